"""GPU: the norms on both sides of a block with gate and scaled residual,
against the 64-bit oracle.

Tolerances: u = 2^-11 (fp16) or 2^-8 (bf16) of a result rounded once; below that
32-bit arithmetic: a row's mean square is off by at most 2^-18 (64 terms a thread in a
row, then trees, 2^-24 each), its root by half of that, and the two terms of the sum by
a handful of roundings: 2^-17 of their magnitudes in all."""
import numpy as np
import pytest
import torch

from oracle import more_ops as ref
from test_gpu_attn_half import DEV, DTYPES, IDS, TINY, U, _gpu, draw, f64, gen, pw, within  # noqa: F401

pytestmark = pytest.mark.gpu
EPS = 1e-5


def bound_y(u, tiny, r, y, mag, w):
    rms = np.sqrt(np.mean(r * r, axis=1, keepdims=True) + EPS)
    return u * np.abs(y) * 1.01 + 2.0 ** -17 * (np.abs(y) + mag / rms * np.abs(w)) + tiny


def check_q(q, sc, r, want, mag, w):
    """The scales and codes of the 32-bit y: what it may be off by, in scales and then in codes."""
    cols = want.shape[1]
    off = bound_y(0.0, 0.0, r, want, mag, w)
    top = np.stack([np.abs(want[:, c:c + 128]).max(1) for c in range(0, cols, 128)], 1)
    slack = np.stack([off[:, c:c + 128].max(1) for c in range(0, cols, 128)], 1)
    within(sc, np.maximum(top / 448, 2.0 ** -100), slack / 448 + top * 2.0 ** -30)
    s = np.repeat(f64(sc), 128, 1)[:, :cols]
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(want / s), 2.0 ** -6))) - 3)
    within(q.view(torch.float8_e4m3fn).double(), want / s, 0.5 * step * 1.0001 + 2 * off / s)


def inputs(rows, cols, dtype, seed=0):
    g = gen(rows * 40000 + cols + seed)
    x, res = draw(g, rows, cols, dtype=dtype), draw(g, rows, cols, dtype=dtype, scale=3)
    post, w = (draw(g, cols, dtype=dtype) for _ in range(2))
    return g, x, res, post, w


SIZES = [(1, 1), (3, 7), (1, 128), (5, 129), (2, 1000), (33, 2048), (4, 4095), (2, 5121), (2, 6144), (3, 6152), (1, 8200),
         (3, 16392), (2, 32768), (2, 32761), (700, 256), (650, 1025), (400, 5120), (321, 6145)]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("rows,cols", SIZES)
def test_norm_add_norm(rows, cols, dtype):
    g, x, res, post, w = inputs(rows, cols, dtype)
    gates = [None, draw(g, cols, dtype=dtype), draw(g, rows, cols, dtype=dtype)]
    u, tiny = U[dtype], TINY[dtype]
    for i, gate in enumerate(gates):
        y, ro = torch.empty_like(x), torch.empty_like(x)
        q = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device=DEV)
        sc = torch.empty(rows, -(-cols // 128), device=DEV)
        a, b = (1.0, 1.0) if i == 0 else (0.75, -1.5)
        p = None if i == 1 else post
        pw.pw_norm_add_norm(x, res, EPS, post_weight=p, weight=w, gate=gate, residual_scale=a, block_scale=b,
                            residual_out=ro, y=y, q=q, scale=sc)
        r, want, mag = ref.norm_add_norm(f64(x), f64(res), EPS, None if p is None else f64(p), f64(w),
                                         None if gate is None else f64(gate), a, b)
        within(ro, r, u * np.abs(r) * 1.01 + 2.0 ** -17 * mag + tiny)
        within(y, want, bound_y(u, tiny, r, want, mag, f64(w)))
        check_q(q, sc, r, want, mag, f64(w))
        # one output each, in place
        res2, x2, q2 = res.clone(), x.clone(), torch.empty(rows, cols, dtype=torch.uint8, device=DEV)
        pw.pw_norm_add_norm(x2, res2, EPS, post_weight=p, gate=gate, residual_scale=a, block_scale=b, residual_out=res2)
        assert torch.equal(res2, ro)
        pw.pw_norm_add_norm(x2, res, EPS, post_weight=p, weight=w, gate=gate, residual_scale=a, block_scale=b, y=x2)
        assert torch.equal(x2, y)
        x2.copy_(x)
        pw.pw_norm_add_norm(x2, res, EPS, post_weight=p, weight=w, gate=gate, residual_scale=a, block_scale=b,
                            residual_out=x2, q=q2, scale=sc)
        assert torch.equal(x2, ro) and torch.equal(q2, q.view(torch.uint8))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("rows", [5, 401])
@pytest.mark.parametrize("cols,pads,shifts", [
    (256, (8, 8, 8, 8, 8), (0, 0, 0, 0, 0)), (256, (3, 0, 8, 1, 5), (0, 0, 0, 0, 0)), (256, (8, 16, 0, 8, 8), (1, 2, 3, 4, 5)),
    (1030, (0, 1, 2, 3, 4), (5, 6, 7, 0, 1)), (5121, (0, 0, 0, 0, 0), (0, 0, 0, 0, 0)), (5121, (7, 1, 0, 3, 2), (7, 3, 1, 5, 6)),
    (2, (0, 1, 2, 3, 4), (5, 6, 7, 0, 1)), (9001, (1, 2, 3, 4, 5), (1, 0, 1, 0, 1))])
def test_strides_and_alignment(rows, cols, pads, shifts, dtype):
    """Rows cut out of wider ones, each tensor at a stride and an address of its
    own: the same result, and nothing beside it is written."""
    g, x, res, post, w = inputs(rows, cols, dtype)
    gate = draw(g, rows, cols, dtype=dtype)

    def wide(t, pad, shift):
        buf = torch.full((rows * (cols + pad) + shift + 8,), 7.0, dtype=t.dtype, device=DEV)
        v = buf[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, :cols]
        v.copy_(t)
        return buf, v
    kept = [wide(t, p, s) for t, p, s in zip((x, res, gate, x * 0, x * 0), pads, shifts)]
    (_, xv), (_, rv), (_, gv), (rob, ro), (yb, y) = kept
    pv, wv = torch.empty(cols + 3, dtype=dtype, device=DEV)[3:], torch.empty(cols + 1, dtype=dtype, device=DEV)[1:]
    pv.copy_(post), wv.copy_(w)
    q, sc = torch.empty(rows, cols, dtype=torch.uint8, device=DEV), torch.empty(rows, -(-cols // 128), device=DEV)
    pw.pw_norm_add_norm(xv, rv, EPS, post_weight=pv, weight=wv, gate=gv, residual_scale=0.5, residual_out=ro, y=y, q=q, scale=sc)
    r, want, mag = ref.norm_add_norm(f64(x), f64(res), EPS, f64(post), f64(w), f64(gate), 0.5)
    u, tiny = U[dtype], TINY[dtype]
    within(ro, r, u * np.abs(r) * 1.01 + 2.0 ** -17 * mag + tiny)
    within(y, want, bound_y(u, tiny, r, want, mag, f64(w)))
    for (b, _), pad, shift in zip(kept[3:], pads[3:], shifts[3:]):
        side = b[shift:shift + rows * (cols + pad)].view(rows, cols + pad)[:, cols:]
        assert (side == 7).all() and (b[:shift] == 7).all() and (b[shift + rows * (cols + pad):] == 7).all()
    # codes in wider rows, whole and ragged
    for pitch in (cols + 5, cols + (-cols % 16)):
        room = torch.full((rows, pitch), 9, dtype=torch.uint8, device=DEV)
        sc2 = torch.empty_like(sc)
        pw.pw_norm_add_norm(xv, rv, EPS, post_weight=pv, weight=wv, gate=gv, residual_scale=0.5, q=room[:, :cols], scale=sc2)
        # (rows of codes that start elsewhere may change the accesses, and with them the order of the sums)
        check_q(room[:, :cols], sc2, r, want, mag, f64(w))
        assert (room[:, cols:] == 9).all()


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("cols,pitch", [(130, 131), (5, 16), (300, 304), (1000, 1001), (5121, 5121), (9000, 9016), (16383, 16383)])
@pytest.mark.parametrize("shift", [0, 1, 9, 15])
def test_rows_that_all_start_alike(cols, pitch, shift, dtype):
    """Every matrix at the same place of its 32-byte cells, the codes too: groups of a scale that begin inside a cell."""
    rows = 7
    g, x, res, post, w = inputs(rows, cols, dtype, shift)
    gate = draw(g, rows, cols, dtype=dtype)

    def wide(t, fill=7):
        buf = torch.full((rows * pitch + shift + 40,), fill, dtype=t.dtype, device=DEV)
        v = buf[shift:shift + rows * pitch].view(rows, pitch)[:, :cols]
        v.copy_(t)
        return buf, v
    (_, xv), (_, rv), (_, gv), (rob, ro), (yb, y) = (wide(t) for t in (x, res, gate, x * 0, x * 0))
    qb, q = wide(torch.zeros(rows, cols, dtype=torch.uint8, device=DEV))
    sc = torch.empty(rows, -(-cols // 128), device=DEV)
    r, want, mag = ref.norm_add_norm(f64(x), f64(res), EPS, f64(post), f64(w), f64(gate), 0.5, 2.0)
    for g_, outs in ((gv, dict(residual_out=ro, y=y, q=q, scale=sc)), (gv, dict(y=y)), (gv, dict(q=q, scale=sc))):
        pw.pw_norm_add_norm(xv, rv, EPS, post_weight=post, weight=w, gate=g_, residual_scale=0.5, block_scale=2.0, **outs)
    u, tiny = U[dtype], TINY[dtype]
    within(ro, r, u * np.abs(r) * 1.01 + 2.0 ** -17 * mag + tiny)
    within(y, want, bound_y(u, tiny, r, want, mag, f64(w)))
    check_q(q, sc, r, want, mag, f64(w))
    for b in (rob, yb, qb):
        side = b[shift:shift + rows * pitch].view(rows, pitch)[:, cols:]
        assert (side == 7).all() and (b[:shift] == 7).all() and (b[shift + rows * pitch:] == 7).all()
    # in place, and a gate that is a row at an address of its own
    want_y = torch.empty_like(x)
    pw.pw_norm_add_norm(xv, rv, EPS, post_weight=post, weight=w, gate=gate[0], residual_out=ro, y=y)
    pw.pw_norm_add_norm(x, res, EPS, post_weight=post, weight=w, gate=gate[0].clone(), residual_out=res, y=want_y)
    within(y, f64(want_y), 2 * (u * np.abs(f64(want_y)) + tiny))   # both are rounded, by half a step each
    pw.pw_norm_add_norm(xv, rv, EPS, post_weight=post, weight=w, gate=gate[0], residual_out=rv, y=xv)
    assert torch.equal(rv, ro) and torch.equal(xv, y)


def test_extremes():
    """Rows of zeros, values at the types' ends, and NaN or infinity: they stay in their rows."""
    for dtype in DTYPES:
        x = torch.ones(6, 384, dtype=dtype, device=DEV)
        res = torch.ones_like(x)
        x[0], res[0] = 0, 0
        x[1, 5], x[2, 7], res[3, 9] = float("nan"), float("inf"), float("inf")
        x[4] = torch.finfo(dtype).smallest_normal
        ro, y = torch.empty_like(x), torch.empty_like(x)
        one = torch.ones(384, dtype=dtype, device=DEV)
        pw.pw_norm_add_norm(x, res, EPS, post_weight=one, weight=one, residual_out=ro, y=y)
        assert (ro[0] == 0).all() and (y[0] == 0).all()
        assert ro[1].isnan().all() and y[1].isnan().all()
        # the root of an infinite mean square divides every finite value to 0; the infinite one is NaN
        assert ro[2, 7].isnan() and y[2].isnan().all() and (ro[2, :7] == 1).all()
        assert ro[3, 9].isinf() and y[3, 9].isnan() and (y[3, :9] == 0).all()
        r, want, mag = ref.norm_add_norm(f64(x[4:]), f64(res[4:]), EPS, np.ones(384), np.ones(384))
        within(ro[4:], r, U[dtype] * np.abs(r) * 1.01 + 2.0 ** -17 * mag)
        within(y[4:], want, bound_y(U[dtype], 0.0, r, want, mag, np.ones(384)))


def test_single_norm_is_that_of_add_rmsnorm():
    """Without a norm of the block, gate and scales: pw_add_rmsnorm's function."""
    g, x, res, _, w = inputs(40, 4096, torch.float16)
    y, ro, y2, ro2 = (torch.empty_like(x) for _ in range(4))
    pw.pw_norm_add_norm(x, res, EPS, weight=w, residual_out=ro, y=y)
    pw.pw_add_rmsnorm(x, w, EPS, residual=res, residual_out=ro2, y=y2)
    assert torch.equal(ro, ro2)
    within(y, f64(y2), 2 * U[torch.float16] * np.abs(f64(y2)) + TINY[torch.float16])


def test_stream_graph_and_repeats():
    g, x, res, post, w = inputs(300, 2048, torch.bfloat16)
    want, got = torch.empty_like(x), torch.empty_like(x)
    pw.pw_norm_add_norm(x, res, EPS, post_weight=post, weight=w, y=want)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    pw.pw_norm_add_norm(x, res, EPS, post_weight=post, weight=w, y=got, stream=s)
    s.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pw.pw_norm_add_norm(x, res, EPS, post_weight=post, weight=w, y=got)
    for seed in (1, 2):
        x.copy_(draw(gen(seed), 300, 2048, dtype=torch.bfloat16))
        got.zero_()
        graph.replay()
        pw.pw_norm_add_norm(x, res, EPS, post_weight=post, weight=w, y=want)
        assert torch.equal(got, want)


def test_refusals():
    x = torch.zeros(4, 64, dtype=torch.float16, device=DEV)
    for bad in (dict(residual_out=x[:, :32]), dict(residual_out=x.bfloat16()), dict(residual_out=x, weight=x[0]),
                dict(y=x), dict(residual_out=x.cpu()), dict(residual_out=x, post_weight=x[0, :32]),
                dict(residual_out=x, gate=x[:2]), dict(residual_out=x, gate=x[0].float()), dict(), dict(q=x, weight=x[0]),
                dict(residual_out=x.t().contiguous().t())):
        with pytest.raises((ValueError, pw.PwError)):
            pw.pw_norm_add_norm(x, x, EPS, **bad)
    pw.pw_norm_add_norm(x[:0], x[:0], EPS, residual_out=x[:0])
