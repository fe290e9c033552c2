"""GPU: a decoder layer run as a program runs it: ragged prompts in chunks,
then single tokens, over a paged cache, with the routed experts behind the
attention.  Every stage's buffer is compared with the 64-bit oracle of that
stage on the buffers before it."""
import numpy as np
import pytest
import torch

from oracle import apl
from oracle import attn_half as ref
from test_gpu_attn_half import DEV, TINY, U, _gpu, check_codes, draw, f64, gen, within  # noqa: F401

pytestmark = pytest.mark.gpu

pw = pytest.importorskip("any_precision_bit_pw_gb300.pw")
from any_precision_bit_pw_gb300 import synth  # noqa: E402
from any_precision_bit_pw_gb300.decoder import DecoderLayer, DecoderWeights, Fp8Weight, PagedCache  # noqa: E402
from any_precision_bit_pw_gb300.layer import APLMoEStack, load_layer  # noqa: E402

F16 = torch.float16


def build(heads=4, kv_heads=2, head_dim=64, pages=64, page_size=16, tokens=96, **kw):
    wl = synth.TINY_LAYER
    sh = wl.shape
    stack = APLMoEStack(sh.hidden, sh.intermediate, sh.experts, sh.top_k, 1, wl.parent_bits, wl.seed_bits, DEV)
    inputs = synth.layer_inputs(wl, device=DEV)
    load_layer(stack, 0, inputs)
    stack.sync()
    g, H = gen(77), sh.hidden
    norm = lambda: (1 + 0.1 * torch.randn(H, generator=g)).to(F16).to(DEV)  # noqa: E731
    w = DecoderWeights(norm(), norm(), Fp8Weight.quantize(draw(g, (heads + 2 * kv_heads) * head_dim, H, scale=H ** -0.5)),
                       Fp8Weight.quantize(draw(g, H, heads * head_dim, scale=(heads * head_dim) ** -0.5)),
                       torch.randn(sh.experts, H, generator=g).to(DEV) * H ** -0.5)
    cache = PagedCache(pages, page_size, kv_heads, head_dim, device=DEV)
    cache.k.fill_(float("nan"))
    cache.v.fill_(float("nan"))
    return DecoderLayer(stack, 0, w, heads, cache, tokens, **kw), (wl, inputs)


def check_stages(L, x, residual, batch, out, r2, moe):
    """Each stage from the buffers that went into it."""
    T, w, D, hq, hk = batch.tokens, L.w, L.head_dim, L.heads, L.kv_heads
    u, tiny = U[F16], TINY[F16]
    near = lambda got, want: within(got, want, u * np.abs(want) * (1 + 2.0 ** -8) + tiny)  # noqa: E731
    r, y = ref.add_rmsnorm(f64(x), f64(w.attn_norm), L.eps, None if residual is None else f64(residual))
    near(L.residual[0][:T], r)
    check_codes(L.x8[:T], L.x8_scale[:T], y, 1)

    def product(a, a_scale, weight, got):
        want, mag = ref.fp8_linear(a.view(torch.uint8).cpu().numpy(), f64(a_scale),
                                   weight.codes.view(torch.uint8).cpu().numpy(), f64(weight.scale))
        within(got, want, u * np.abs(want) * 1.01 + 2.0 ** -13 * mag + tiny)
    product(L.x8[:T], L.x8_scale[:T], w.qkv, L.qkv[:T].reshape(T, -1))
    at = ref.token_positions(batch.q_offsets.tolist(), batch.kv_lens.tolist())
    freq = L.turns.cpu().numpy().astype(np.float64) * 2.0 ** -64 * 2 * np.pi
    qkv = f64(L.qkv[:T])
    rot = ref.rotate(qkv[:, : hq + hk], np.array([p for _, p in at]), freq, L.rope_factor, L.interleaved)
    big = np.abs(qkv[:, : hq + hk]).max() * 1.5 * L.rope_factor
    within(L.q[:T], rot[:, :hq], u * np.abs(rot[:, :hq]) * 1.001 + 2.0 ** -20 * big + tiny)
    table, ps = batch.page_table.cpu().numpy(), L.cache.page_size
    page, row = [int(table[s, p // ps]) for s, p in at], [p % ps for _, p in at]
    within(L.cache.k[page, row], rot[:, hq:], u * np.abs(rot[:, hq:]) * 1.001 + 2.0 ** -20 * big + tiny)
    assert torch.equal(L.cache.v[page, row], L.qkv[:T, hq + hk:])
    want, _, mag, dots = ref.attention(f64(L.q[:T]), f64(L.cache.k), f64(L.cache.v), table, batch.q_offsets.tolist(),
                                       batch.kv_lens.tolist(), D ** -0.5, True, L.window)
    within(L.attn[:T], want, u * np.abs(want) * 1.01 + (u + 2.0 ** -15 * dots + 2.0 ** -16)[..., None] * mag + tiny)
    check_codes(L.attn8[:T], L.attn8_scale[:T], f64(L.attn[:T]).reshape(T, -1), 1)
    product(L.attn8[:T], L.attn8_scale[:T], w.out, L.o[:T])
    r, y = ref.add_rmsnorm(f64(L.o[:T]), f64(w.ffn_norm), L.eps, f64(L.residual[0][:T]))
    near(r2, r)
    near(L.h[:T], y)
    # the experts: routing from the layer's own logits, products as in the layer's parity tests
    wl, inputs = moe
    sh = wl.shape
    route = apl.route_topk(L.logits[:T].cpu().numpy(), sh.top_k)
    assert np.array_equal(L.moe(T).route.ids.cpu().numpy()[:T], route["ids"])
    planes = {key: apl.pack_bitplanes(v.cpu().numpy(), wl.parent_bits) for key, v in inputs.idx.items()}

    def blocks(e, which):
        N, K = (2 * sh.intermediate, sh.hidden) if which == 0 else (sh.hidden, sh.intermediate)
        return apl.Block(planes[(e, which)], {b: t.cpu().numpy() for b, t in inputs.luts[(e, which)].items()},
                         inputs.bits[2 * e + which], N, K)
    want = apl.moe_layer(L.h[:T].cpu().numpy(), route["ids"], route["w"], sh.intermediate, blocks)
    m = apl.compare(want, out.float().cpu().numpy())
    assert m["rel_l2"] <= 2e-3 and m["max_abs_over_rms"] <= 1e-2, m
    assert int(L.status.item()) == 0 and int(L.moe(T).status.item()) == 0


@pytest.mark.parametrize("kw", [dict(), dict(interleaved=True, rotary_dim=32, window=20),
                                dict(heads=6, kv_heads=1, head_dim=128, page_size=8,
                                     rope_scaling=pw.pw_rope_scaling(pw.PW_ROPE_YARN, 0, 4.0, 32.0, 32.0, 1.0))],
                         ids=["plain", "interleaved_window", "yarn_128"])
def test_prompts_then_tokens(kw):
    L, moe = build(**kw)
    g, H = gen(5), L.stack.H
    for seqs, new in [([0, 1], [70, 9]), ([0, 2], [11, 40]), ([2, 0, 1], [1, 1, 1]), ([1], [1]), ([0, 1, 2], [1, 5, 1])]:
        batch = L.cache.batch(seqs, new)
        x, res = draw(g, batch.tokens, H), draw(g, batch.tokens, H, scale=2)
        residual = None if seqs == [1] else res
        out, r2 = L(x, residual, batch)
        check_stages(L, x, residual, batch, out, r2, moe)
    L.cache.release(0)
    with pytest.raises(RuntimeError):
        L.cache.batch([9], [10 ** 6])
    with pytest.raises(ValueError):
        L(draw(g, 3, H), None, L.cache.batch([1], [1]))


def test_chunks_and_single_tokens_agree():
    """The same tokens as one chunk, in three, and one by one: the attention
    of the last token differs by roundings only."""
    g = gen(11)
    L, _ = build(tokens=64)
    x = draw(g, 48, L.stack.H)
    last = []
    for i, cuts in enumerate(([48], [20, 27, 1], [1] * 48)):
        at = 0
        for n in cuts:
            L(x[at:at + n], None, L.cache.batch([i], [n]))
            at += n
        last.append(f64(L.attn[cuts[-1] - 1]))
    # the chunks give the same 16-bit queries, keys and values where the products' tiles agree on every bit; else a
    # 16-bit rounding apart each.  The bound is the attention's own plus one rounding of keys and values.
    want = last[0]
    scale = np.abs(f64(L.cache.v[L.cache.pages[0]][: 3])).max()
    for got in last[1:]:
        assert np.abs(got - want).max() <= 8 * U[F16] * scale


def test_decode_step_in_a_graph():
    """A captured step replays bit for bit; the batch's tensors are refilled in
    place for the next token."""
    L, _ = build()
    g, H = gen(21), L.stack.H
    prompt = L.cache.batch([0, 1, 2], [30, 17, 1])
    L(draw(g, prompt.tokens, H), None, prompt)
    x, res = draw(g, 3, H), draw(g, 3, H)
    first = L.cache.batch([0, 1, 2], [1, 1, 1], width=8)
    first.max_kv_len = 8 * L.cache.page_size
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, r2 = L(x, res, first)
    torch.cuda.current_stream().wait_stream(side)
    want, want_r = out.clone(), r2.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, r2 = L(x, res, first)
    out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(r2, want_r)
    second = L.cache.batch([0, 1, 2], [1, 1, 1], width=8)
    x2 = draw(g, 3, H)
    first.page_table.copy_(second.page_table)
    first.kv_lens.copy_(second.kv_lens)
    x.copy_(x2)
    graph.replay()
    torch.cuda.synchronize()
    got, got_r = out.clone(), r2.clone()
    out, r2 = L(x2, res, second)
    assert int(L.status.item()) == 0
    assert torch.equal(r2, got_r) and torch.equal(out, got)
