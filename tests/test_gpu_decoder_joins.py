"""GPU: layers that follow one another and share buffers, some of them of their own widths."""
import pytest
import torch

from test_gpu_attn_half import DEV, _gpu, draw, gen  # noqa: F401
from test_gpu_decoder_dense import D, HEADS, KV, SINKS, WINDOW

pytestmark = pytest.mark.gpu
from any_precision_bit_pw_gb300 import synth  # noqa: E402
from any_precision_bit_pw_gb300.decoder import DecoderLayer, DecoderWeights, Fp8Weight, Head, PagedCache  # noqa: E402
from any_precision_bit_pw_gb300.layer import APLMoEStack, load_layer  # noqa: E402

WIDTHS = [None, 640, 200, 200, 640]   # of the layers' dense blocks; None: experts


def parts():
    wl = synth.TINY_LAYER
    sh = wl.shape
    H, g = sh.hidden, gen(21)
    stack = APLMoEStack(H, sh.intermediate, sh.experts, sh.top_k, 1, wl.parent_bits, wl.seed_bits, DEV)
    load_layer(stack, 0, synth.layer_inputs(wl, device=DEV))
    stack.sync()
    norm = lambda: (1 + 0.1 * torch.randn(H, generator=g)).half().to(DEV)  # noqa: E731
    matrix = lambda n, k: Fp8Weight.quantize(draw(g, n, k, scale=k ** -0.5))  # noqa: E731
    ws = []
    for w in WIDTHS:
        a = (norm(), norm(), matrix((HEADS + 2 * KV) * D, H), matrix(H, HEADS * D))
        block = dict(gate=matrix(w, H), up=matrix(w, H), down=matrix(H, w)) if w else dict(
            router=torch.randn(sh.experts, H, generator=g).to(DEV) * H ** -0.5)
        ws.append(DecoderWeights(*a, **block, post_attn_norm=norm(), post_ffn_norm=norm(), residual_scale=0.75))
    return stack, ws, (norm(), matrix(1000, H))


def model(stack, ws, end, shared):
    layers = []
    for w in ws:
        cache = PagedCache(16, 16, KV, D, device=DEV)
        layers.append(DecoderLayer(stack, 0, w, HEADS, cache, 32, window=WINDOW, sinks=SINKS, after=layers[-1] if layers else None,
                                   share=layers[0] if layers and shared else None))
    return layers, Head(*end, tokens=32, top=3, after=layers[-1])


def run(layers, head, x, batch, stream=None):
    r = None
    for L in layers:
        x, r = L(x, r, batch, stream=stream)
    return head(x, r, stream=stream)


@pytest.mark.parametrize("side", [False, True])
def test_shared_buffers_of_several_widths(side):
    """Experts and dense blocks of two widths on one set of buffers, made while the current stream still works and called on
    another one: the results of layers that share nothing."""
    stack, ws, end = parts()
    x = draw(gen(2), 21, stack.H)
    layers, head = model(stack, ws, end, False)
    want = run(layers, head, x, layers[0].cache.batch([0, 1], [14, 7]))
    want = [t.clone() for t in (want.logits, want.lse, want.top_ids)]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream() if side else None
    # work on the current stream on memory that is free again for the constructors
    torch.cuda._sleep(50_000_000)
    for shape in ((32, stack.H), (32, 640), (32, 208), (32, 5)):
        torch.empty(shape, dtype=torch.float16, device=DEV).fill_(float("nan"))
    layers, head = model(stack, ws, end, True)
    assert all(L.x8 is layers[0].x8 for L in layers) and layers[1].ff8.shape == (32, 640) and layers[2].ff8.shape == (32, 200)
    batch = layers[0].cache.batch([0, 1], [14, 7])
    got = run(layers, head, x, batch, stream)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, (got.logits, got.lse, got.top_ids)))
    assert int(layers[0].status.item()) == 0 and int(head.status.item()) == 0
