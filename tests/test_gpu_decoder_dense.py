"""GPU: a model of a dense layer and a layer of experts with norms on both sides of
every block, gates, windows with first keys, and its head, run as a program runs it:
every stage is compared with the 64-bit oracle on the buffers before it."""
import math

import numpy as np
import pytest
import torch

from oracle import attn_half as ref
from oracle import more_ops
from test_gpu_attn_half import DEV, TINY, U, _gpu, draw, f64, gen, pw, within  # noqa: F401
from test_gpu_gated import check_codes as check_gated
from test_gpu_norms import EPS, bound_y, check_q

pytestmark = pytest.mark.gpu
from any_precision_bit_pw_gb300 import synth  # noqa: E402
from any_precision_bit_pw_gb300.decoder import DecoderLayer, DecoderWeights, Fp8Weight, Head, PagedCache  # noqa: E402
from any_precision_bit_pw_gb300.layer import APLMoEStack, load_layer  # noqa: E402

F16 = torch.float16
HEADS, KV, D, I, V, WINDOW, SINKS = 4, 2, 64, 640, 3001, 24, 3
u, tiny = U[F16], TINY[F16]


class Model:
    def __init__(self, tokens=64, pages=64, seed=5):
        wl = synth.TINY_LAYER
        sh = wl.shape
        self.H = H = sh.hidden
        stack = APLMoEStack(H, sh.intermediate, sh.experts, sh.top_k, 1, wl.parent_bits, wl.seed_bits, DEV)
        load_layer(stack, 0, synth.layer_inputs(wl, device=DEV))
        stack.sync()
        g = gen(seed)
        norm = lambda: (1 + 0.1 * torch.randn(H, generator=g)).to(F16).to(DEV)  # noqa: E731
        matrix = lambda n, k: Fp8Weight.quantize(draw(g, n, k, scale=k ** -0.5))  # noqa: E731
        both = dict(post_attn_norm=norm(), post_ffn_norm=norm(), attn_gate=norm(), ffn_gate=norm(), residual_scale=0.75)
        attn = lambda: (norm(), norm(), matrix((HEADS + 2 * KV) * D, H), matrix(H, HEADS * D))  # noqa: E731
        caches = [PagedCache(pages, 16, KV, D, device=DEV) for _ in range(2)]
        for c in caches:
            c.k.fill_(float("nan"))
            c.v.fill_(float("nan"))
        kw = dict(window=WINDOW, sinks=SINKS)
        self.dense = DecoderLayer(stack, 0, DecoderWeights(*attn(), gate=matrix(I, H), up=matrix(I, H), down=matrix(H, I), **both),
                                  HEADS, caches[0], tokens, activation=pw.PW_ACT_GELU_TANH, **kw)
        self.moe = DecoderLayer(stack, 0, DecoderWeights(*attn(), torch.randn(sh.experts, H, generator=g).to(DEV) * H ** -0.5,
                                                         **both), HEADS, caches[1], tokens, share=self.dense, after=self.dense, **kw)
        self.head = Head(norm(), matrix(V, H), tokens, top=4, given=2, after=self.moe, temperature=0.7)
        self.cache = caches[0]

    def __call__(self, x, batch, targets=None):
        y, r = self.dense(x, None, batch)
        y, r = self.moe(y, r, batch)
        return self.head(y, r, targets)


def num(t):
    return t.contiguous().view(torch.uint8).cpu().numpy()


def product(a, a_scale, w, got):
    want, mag = ref.fp8_linear(num(a), f64(a_scale), num(w.codes), f64(w.scale))
    within(got, want, u * np.abs(want) * 1.01 + 2.0 ** -13 * mag + tiny)


def join(x, residual, before, weight, r_got=None, y=None, q=None, scale=None, after_attention=False):
    """A block's output and the residual: what was kept, and the norm's result in 16 or 8 bits."""
    w = before
    post, gate = (w.post_attn_norm, w.attn_gate) if after_attention else (w.post_ffn_norm, w.ffn_gate)
    r, want, mag = more_ops.norm_add_norm(f64(x), f64(residual), EPS, f64(post), f64(weight), f64(gate), w.residual_scale)
    if r_got is not None:
        within(r_got, r, u * np.abs(r) * 1.01 + 2.0 ** -17 * mag + tiny)
    if y is not None:
        within(y, want, bound_y(u, tiny, r, want, mag, f64(weight)))
    if q is not None:
        check_q(q, scale, r, want, mag, f64(weight))


def attention(L, batch):
    T = batch.tokens
    want, _, mag, dots = ref.attention(f64(L.q[:T]), f64(L.cache.k), f64(L.cache.v), batch.page_table.cpu().numpy(),
                                       batch.q_offsets.tolist(), batch.kv_lens.tolist(), D ** -0.5, True, WINDOW, SINKS)
    within(L.attn[:T], want, u * np.abs(want) * 1.01 + (u + 2.0 ** -15 * dots + 2.0 ** -16)[..., None] * mag + tiny)
    product(L.attn8[:T], L.attn8_scale[:T], L.w.out, L.o[:T])


def check_step(M, x, batch, targets):
    T, L = batch.tokens, M.dense
    y, r = L(x, None, batch)
    attention(L, batch)
    join(L.o[:T], L.residual[0][:T], L.w, L.w.ffn_norm, r, q=L.x8[:T], scale=L.x8_scale[:T], after_attention=True)
    g, mg = ref.fp8_linear(num(L.x8[:T]), f64(L.x8_scale[:T]), num(L.w.gate.codes), f64(L.w.gate.scale))
    up, mu = ref.fp8_linear(num(L.x8[:T]), f64(L.x8_scale[:T]), num(L.w.up.codes), f64(L.w.up.scale))
    v, t = more_ops.activation(g, "gelu_tanh")
    off = 1.13 * 2.0 ** -13 * mg * (np.abs(up) + 2.0 ** -13 * mu) + np.abs(v) * 2.0 ** -13 * mu + (2.0 ** -20 + 2.0 ** -22 * t) * np.abs(v * up)
    check_gated(L.ff8[:T], L.ff8_scale[:T], v * up, off)
    product(L.ff8[:T], L.ff8_scale[:T], L.w.down, y)
    y1, r1 = y.clone(), r.clone()              # the next layer has these buffers too
    L = M.moe
    y, r = L(y, r, batch)
    join(y1, r1, M.dense.w, L.w.attn_norm, L.residual[0][:T])
    attention(L, batch)
    join(L.o[:T], L.residual[0][:T], L.w, L.w.ffn_norm, r, y=L.h[:T], after_attention=True)
    assert int(L.status.item()) == 0
    s = M.head(y, r, targets)
    join(y, r, L.w, M.head.norm, q=M.head.x8[:T], scale=M.head.x8_scale[:T])
    product(M.head.x8[:T], M.head.x8_scale[:T], M.head.weight, s.logits)
    lp, lse, h, ids, top = more_ops.token_logprobs(f64(s.logits), targets.cpu().numpy(), 4, float(np.float32(1 / 0.7)))
    for got, want in ((s.logprobs, lp), (s.lse, lse), (s.entropy, h), (s.top_logprobs, top)):
        within(got, want, 2.0 ** -16 * (1 + np.abs(want)))
    assert np.array_equal(s.top_ids.cpu().numpy(), ids) and int(M.head.status.item()) == 0


def test_prompts_then_tokens():
    M, g = Model(), gen(3)
    for seqs, new in [([0, 1], [50, 9]), ([0, 2], [11, 40]), ([2, 0, 1], [1, 1, 1]), ([1], [1]), ([0, 1, 2], [1, 5, 1])]:
        for s in seqs:
            M.cache.trim(s, WINDOW, SINKS)     # only what no token sees any more is given back
        batch = M.cache.batch(seqs, new)
        check_step(M, draw(g, batch.tokens, M.H), batch,
                   torch.randint(0, V, (batch.tokens, 2), generator=g, dtype=torch.int32).to(DEV))
    assert any(p < 0 for p in M.cache.pages[0])


def test_scores_of_a_text_in_chunks_and_by_single_tokens():
    """The same text as one chunk and token by token, its pages given back on the way.  The
    products' kernels differ in the order of their sums, so codes next to a border differ
    by a step: a norm of the difference, a few e4m3 roundings (2^-4) of some values, is all that is asked."""
    M, g = Model(), gen(9)
    x = draw(g, 40, M.H)
    text = torch.randint(0, V, (40, 1), generator=g, dtype=torch.int32).to(DEV)
    whole = M(x, M.cache.batch([0], [40]), text).logits.float().clone()
    one = []
    for i in range(40):
        one.append(M(x[i:i + 1], M.cache.batch([1], [1]), text[i:i + 1]).logits.float().clone())
        M.cache.trim(1, WINDOW, SINKS)
    one = torch.cat(one)
    assert float((one - whole).norm() / whole.norm()) < 2.0 ** -4 and int(M.dense.status.item()) == 0


def test_a_step_in_a_graph_and_on_another_stream():
    M, g = Model(), gen(4)
    x = draw(g, 2, M.H)
    M(draw(g, 60, M.H), M.cache.batch([0, 1], [40, 20]))
    batch = M.cache.batch([0, 1], [1, 1], width=4)
    batch.max_kv_len = 64
    text = torch.tensor([[5], [-1]], dtype=torch.int32, device=DEV)
    names = ("logits", "lse", "entropy", "logprobs", "top_ids", "top_logprobs")
    want = [getattr(M(x, batch, text), n).clone() for n in names]
    assert want[3][1, 0] == 0 and want[3][0, 0] < 0
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    y, r = M.dense(x, None, batch, stream=side)
    y, r = M.moe(y, r, batch, stream=side)
    s = M.head(y, r, text, stream=side)
    side.synchronize()
    assert all(torch.equal(a, getattr(s, n)) for a, n in zip(want, names))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = M(x, batch, text)
    for n in names:
        getattr(s, n).zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, getattr(s, n)) for a, n in zip(want, names))


def test_a_dense_model_needs_no_stack():
    g, H = gen(1), 256
    norm = lambda: torch.ones(H, dtype=F16, device=DEV)  # noqa: E731
    matrix = lambda n, k: Fp8Weight.quantize(draw(g, n, k, scale=k ** -0.5))  # noqa: E731
    w = DecoderWeights(norm(), norm(), matrix((HEADS + 2 * KV) * D, H), matrix(H, HEADS * D), gate=matrix(200, H),
                       up=matrix(200, H), down=matrix(H, 200))
    L = DecoderLayer(None, 0, w, HEADS, PagedCache(8, 16, KV, D, device=DEV), 16)
    y, r = L(draw(g, 9, H), None, L.cache.batch([0], [9]))
    assert y.isfinite().all() and r.isfinite().all() and int(L.status.item()) == 0
    product(L.ff8[:9], L.ff8_scale[:9], w.down, y)
