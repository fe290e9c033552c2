"""GPU: the decoder layer as a server uses it: on a stream of its own, with
changing token counts, several layers in a row."""
import pytest
import torch

from test_gpu_attn_half import _gpu, draw, gen  # noqa: F401
from any_precision_bit_pw_gb300.decoder import DecoderLayer, PagedCache
from test_gpu_decoder import build

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("raw", [False, True], ids=["stream", "handle"])
def test_given_stream(raw):
    """The whole layer runs on the stream that it is given, torch's part too:
    that stream starts late, the current one has nothing to wait for."""
    L, _ = build()
    g, H = gen(31), L.stack.H
    x, res = draw(g, 40, H), draw(g, 40, H)
    out, r2 = L(x, res, L.cache.batch([0, 1], [33, 7]))
    want, want_r = out.clone(), r2.clone()
    other, other_res = draw(g, 40, H), draw(g, 40, H)
    L(other, other_res, L.cache.batch([4, 5], [33, 7]))      # leaves the buffers with other values
    batch = L.cache.batch([2, 3], [33, 7])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    out, r2 = L(x, res, batch, stream=side.cuda_stream if raw else side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(r2, want_r) and torch.equal(out, want)
    assert int(L.status.item()) == 0 and int(L.moe(40).status.item()) == 0


def test_ragged_chunks_take_no_more_memory():
    """Many token counts, one set of buffers; a count's result is that of a
    layer made for it."""
    L, _ = build(tokens=96)
    g, H = gen(32), L.stack.H
    x = draw(g, 96, H)
    batches = [L.cache.batch([i], [n]) for i, n in enumerate((96, 1, 17, 64, 5))]
    L(x[:96], None, batches[0])
    for i, b in enumerate(batches[1:], 1):
        held = torch.cuda.memory_allocated()
        out, r = L(x[: b.tokens], None, b)
        assert out.shape == r.shape == (b.tokens, H) and torch.cuda.memory_allocated() == held
        own, _ = build(tokens=b.tokens)
        want, want_r = own(x[: b.tokens], None, own.cache.batch([i], [b.tokens]))
        assert torch.equal(out, want) and torch.equal(r, want_r)
        del own, want, want_r
    assert int(L.status.item()) == 0 and L.moe(1).status is L.status


def test_layers_share_buffers_and_tables():
    """Three layers in a row, each with its own cache: with the first one's
    buffers and batches, the results are those of layers with their own."""
    g = gen(33)
    stacks = [build(tokens=48)[0] for _ in range(2)]
    x = draw(g, 48, stacks[0].stack.H)
    results = []
    for first, shared in zip(stacks, (False, True)):
        def another():
            c = PagedCache(64, 16, first.kv_heads, first.head_dim, device="cuda")
            return DecoderLayer(first.stack, 0, first.w, first.heads, c, 48, share=first if shared else None)
        layers = [first, another(), another()]
        for n in (48, 5, 1):
            batches = [L.cache.batch([1, 2], [n - n // 3, n // 3]) for L in (layers[:1] if shared else layers)] * (3 if shared else 1)
            h, r = x[:n], None
            for L, b in zip(layers, batches):
                h, r = L(h, r, b)
            results.append((h.clone(), r.clone()))
        assert all(int(L.status.item()) == 0 for L in layers)
    for (h, r), (h2, r2) in zip(results[:3], results[3:]):
        assert torch.equal(h, h2) and torch.equal(r, r2)
    with pytest.raises(ValueError):
        DecoderLayer(first.stack, 0, first.w, first.heads, first.cache, 47, share=first)
