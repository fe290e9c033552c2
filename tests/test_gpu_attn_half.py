"""GPU: the attention half (norm, 8-bit quantisation and product, rotary
positions with the paged cache, attention over it) against the 64-bit oracle.

Tolerances are bounds of the roundings that the kernels make: u = 2^-11 (fp16)
or 2^-8 (bf16) for a result rounded once, the same for softmax weights that
are rounded before they meet the values, 32-bit arithmetic below that."""
import os

import numpy as np
import pytest
import torch

from oracle import attn_half as ref

pytestmark = pytest.mark.gpu

pw = pytest.importorskip("any_precision_bit_pw_gb300.pw")

DEV = "cuda"
U = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float16: 2.0 ** -25, torch.bfloat16: 2.0 ** -134}   # half a step among the subnormals
DTYPES = [torch.float16, torch.bfloat16]
IDS = ["fp16", "bf16"]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    if not os.path.exists(pw.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    pw.lib()
    torch.cuda.set_device(0)


def gen(seed):
    return torch.Generator().manual_seed(seed)


def draw(g, *shape, dtype=torch.float16, scale=1.0):
    return (torch.randn(*shape, generator=g) * scale).to(dtype).to(DEV)


def f64(t):
    return t.detach().double().cpu().numpy()


def status():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


def within(got, want, bound):
    got = f64(got) if isinstance(got, torch.Tensor) else got
    assert np.isfinite(got).all()
    err = np.abs(got - want)
    worst = np.argmax(err - bound)
    assert (err <= bound).all(), (err.flat[worst], np.asarray(bound).flat[worst] if np.ndim(bound) else bound, worst)


def check_codes(codes, scale, y, block_rows):
    """Codes and scales of y (64 bits, exact up to `2^-20` relative)."""
    want = ref.group_scales(y, block_rows)
    within(scale, want, want * 2.0 ** -20)
    s = ref.spread(f64(scale), y.shape, block_rows)
    # half a step, and the 32-bit arithmetic before it
    within(ref.e4m3_decode(codes.view(torch.uint8).cpu().numpy()), y / s,
           0.5 * ref.e4m3_step(y / s) + np.abs(y / s) * 2.0 ** -19)


# ---------------------------------------------------------------- norm and quantisation
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 7), (1, 128), (5, 129), (2, 1000), (33, 2048), (4, 4095), (2, 6144),
                                       (1, 8200), (3, 16392), (2, 32768), (700, 256)])
def test_add_rmsnorm(rows, cols, dtype):
    g = gen(rows * 40000 + cols)
    x, res = draw(g, rows, cols, dtype=dtype), draw(g, rows, cols, dtype=dtype, scale=3)
    w = (1 + 0.2 * torch.randn(cols, generator=g)).to(dtype).to(DEV)
    y, ro = torch.empty_like(x), torch.empty_like(x)
    q = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device=DEV)
    sc = torch.empty(rows, -(-cols // 128), device=DEV)
    pw.pw_add_rmsnorm(x, w, 1e-5, residual=res, residual_out=ro, y=y, q=q, scale=sc)
    r, want = ref.add_rmsnorm(f64(x), f64(w), 1e-5, f64(res))
    u = U[dtype]
    within(ro, r, u * np.abs(r) * (1 + 2.0 ** -10) + TINY[dtype])
    within(y, want, u * np.abs(want) * (1 + 2.0 ** -8) + TINY[dtype])
    check_codes(q, sc, want, 1)
    # without a residual, one output each, in place
    x2 = x.clone()
    pw.pw_add_rmsnorm(x2, w, 1e-5, y=x2)
    _, want = ref.add_rmsnorm(f64(x), f64(w), 1e-5)
    within(x2, want, u * np.abs(want) * (1 + 2.0 ** -8) + TINY[dtype])
    res2 = res.clone()
    q2 = torch.empty(rows, cols, dtype=torch.uint8, device=DEV)
    pw.pw_add_rmsnorm(x, w, 1e-5, residual=res2, residual_out=res2, q=q2, scale=sc)
    assert torch.equal(res2, ro) and torch.equal(q2, q.view(torch.uint8))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("cols,pad,shift", [(256, 8, 0), (256, 3, 0), (256, 8, 1), (130, 6, 0), (4096, 4096, 8)])
def test_norm_strides_and_alignment(cols, pad, shift, dtype):
    """Rows cut out of wider ones, at odd strides and addresses: the same
    result bit for bit, and nothing beside it is written."""
    g = gen(cols + pad + shift)
    rows = 5
    x, res = draw(g, rows, cols, dtype=dtype), draw(g, rows, cols, dtype=dtype)
    w = draw(g, cols, dtype=dtype)

    def wide(t):
        buf = torch.full((rows * (cols + pad) + shift,), 7.0, dtype=t.dtype, device=DEV)
        v = buf[shift:].view(rows, cols + pad)[:, :cols]
        v.copy_(t)
        return buf, v
    y, ro = torch.empty_like(x), torch.empty_like(x)
    q, sc = torch.empty(rows, cols, dtype=torch.uint8, device=DEV), torch.empty(rows, -(-cols // 128), device=DEV)
    pw.pw_add_rmsnorm(x, w, 1e-6, residual=res, residual_out=ro, y=y, q=q, scale=sc)
    (_, xv), (_, rv), (yb, yv), (rob, rov), (qb, qv) = wide(x), wide(res), wide(y * 0), wide(ro * 0), wide(q * 0)
    pw.pw_add_rmsnorm(xv, w, 1e-6, residual=rv, residual_out=rov, y=yv, q=qv, scale=sc)
    assert torch.equal(rov, ro)
    u = U[dtype]
    within(yv, f64(y), 2 * u * np.abs(f64(y)) + TINY[dtype])   # another order of the 32-bit sum may round once apart
    for b in (yb, rob, qb):
        side = b[shift:].view(rows, cols + pad)[:, cols:]
        assert (side == 7).all() and (b[:shift] == 7).all()


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 127), (97, 130), (128, 128), (129, 640), (300, 1001), (257, 4096)])
def test_quantize(rows, cols, block_rows, dtype):
    g = gen(rows * 5000 + cols)
    x = draw(g, rows, cols, dtype=dtype, scale=5)
    x[:, ::37] *= 50
    x[rows // 2] = 0
    x[:, : cols // 3] *= 1e-3
    q = torch.empty(rows, cols, dtype=torch.uint8, device=DEV)
    sc = torch.empty(-(-rows // block_rows), -(-cols // 128), device=DEV)
    pw.pw_quantize_fp8(x, q, sc, block_rows=block_rows)
    check_codes(q, sc, f64(x), block_rows)


def test_quantize_extremes():
    """Zeros, the type's extremes, and NaN or infinity: their group is NaN when
    multiplied out, its neighbours are not."""
    for dtype in DTYPES:
        top = torch.finfo(dtype).max
        x = torch.ones(4, 384, dtype=dtype, device=DEV)
        x[0] = 0
        x[1, :128], x[1, 128:256], x[1, 256:] = top, torch.finfo(dtype).smallest_normal, -top
        x[2, 130], x[3, 5] = float("nan"), float("inf")
        q, sc = torch.empty(4, 384, dtype=torch.uint8, device=DEV), torch.empty(4, 3, device=DEV)
        pw.pw_quantize_fp8(x, q, sc)
        y = ref.e4m3_decode(q.cpu().numpy()) * np.repeat(f64(sc), 128, 1)
        assert np.all(y[0] == 0) and f64(sc)[0, 0] == 2.0 ** -100
        big = f64(torch.tensor(top, dtype=dtype))
        assert np.allclose(y[1, :128], big, rtol=2.0 ** -4) and np.allclose(y[1, 256:], -big, rtol=2.0 ** -4)
        if dtype == torch.float16:   # bf16's smallest numbers are below the smallest scale: zeros
            assert np.allclose(y[1, 128:256], 2.0 ** -14, rtol=2.0 ** -4)
        bad = np.isnan(y)
        assert bad[2, 130] and bad[3, 5] and not bad[2, :128].any() and not bad[2, 256:].any() and not bad[3, 128:].any()


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quantize_same_result_at_any_alignment(block_rows):
    rows, cols = 200, 336
    x0 = draw(gen(6), rows, cols, dtype=torch.bfloat16)
    want = None
    for offset, pitch in ((0, 336), (16, 352), (8, 336), (0, 344), (1, 337)):
        x = torch.empty(rows * pitch + 64, dtype=torch.bfloat16, device=DEV)[offset:offset + rows * pitch].view(rows, pitch)[:, :cols]
        x.copy_(x0)
        q = torch.zeros(rows * pitch + 64, dtype=torch.uint8, device=DEV)[offset:offset + rows * pitch].view(rows, pitch)[:, :cols]
        sc = torch.empty(-(-rows // block_rows), -(-cols // 128), device=DEV)
        pw.pw_quantize_fp8(x, q, sc, block_rows=block_rows)
        if want is None:
            want = (q.clone(), sc)
            check_codes(q, sc, f64(x), block_rows)
        assert torch.equal(q, want[0]) and torch.equal(sc, want[1])


# ---------------------------------------------------------------- the 8-bit product
LINEAR = [(1, 1, 16), (1, 128, 128), (3, 17, 130), (7, 200, 100), (8, 1000, 512), (9, 128, 1000), (16, 64, 2048),
          (17, 130, 256), (33, 129, 384), (64, 384, 144), (65, 1, 640), (100, 300, 1024), (128, 256, 128), (129, 513, 257),
          (200, 640, 4096), (257, 128, 16), (300, 1030, 900), (512, 512, 512), (1000, 260, 2000)]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("m,n,k", LINEAR)
def test_fp8_linear(m, n, k, dtype):
    g = gen(m * 7919 + n * 131 + k)
    kb, pad = -(-k // 128), -k % 16
    def codes(rows):
        t = (torch.randn(rows, k + pad, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
        t[:, k:] = float("nan")                    # past the columns: anything
        return t.to(DEV)[:, :k]
    a, b = codes(m), codes(n)
    sa = torch.exp(torch.randn(m, kb, generator=g)).to(DEV)
    sb = torch.exp(torch.randn(-(-n // 128), kb, generator=g) - 6).to(DEV)
    y = torch.full((m, n + 3), 7.0, dtype=dtype, device=DEV)
    st = status()
    pw.pw_fp8_linear(a, sa, b, sb, y[:, :n], st)
    want, mag = ref.fp8_linear(a.view(torch.uint8).cpu().numpy(), f64(sa), b.view(torch.uint8).cpu().numpy(), f64(sb))
    # one rounding to 16 bits; the tensor cores add the exact products of a group with at least 13 bits below the
    # largest of them
    bound = U[dtype] * np.abs(want) * 1.01 + 2.0 ** -13 * mag + TINY[dtype]
    got, top = f64(y[:, :n]), torch.finfo(dtype).max
    # a sum past the type's largest number is an infinity of its sign; one within `bound` of the border may be either
    over = np.isinf(got)
    assert (np.abs(want[over]) + bound[over] > top).all() and (np.sign(want[over]) == np.sign(got[over])).all()
    within(got[~over], want[~over], bound[~over])
    rel = np.linalg.norm(got[~over] - want[~over]) / np.linalg.norm(want[~over])
    assert rel <= U[dtype], rel
    assert (y[:, n:] == 7).all() and int(st.item()) == 0


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("m,n,k", [(9, 33, 100), (15, 1000, 2048), (24, 130, 2000), (32, 4000, 300), (10, 520, 2064),
                                   (31, 100, 4000), (12, 6000, 512), (48, 1000, 1600), (50, 300, 800), (100, 300, 2100),
                                   (128, 200, 5000)])
def test_fp8_linear_between_kernels(m, n, k, dtype):
    """Sizes on both sides of the choices of a kernel and of its split."""
    test_fp8_linear(m, n, k, dtype)


@pytest.mark.parametrize("offset,pitch", [(0, 272), (16, 272), (16, 288), (32, 288)])
@pytest.mark.parametrize("m", [3, 13, 29, 60])
def test_fp8_linear_row_alignment(m, offset, pitch):
    """Rows at 16-byte addresses, whichever of them are at 32-byte ones too."""
    g, n, k = gen(m), 50, 240
    def codes(rows):
        t = (torch.randn(rows * pitch + 64, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn).to(DEV)
        return t[offset:offset + rows * pitch].view(rows, pitch)[:, :k]
    a, b = codes(m), codes(n)
    sa, sb = torch.rand(m, 2, generator=g).to(DEV), torch.rand(1, 2, generator=g).to(DEV) / 64
    y, st = torch.empty(m, n, dtype=torch.bfloat16, device=DEV), status()
    pw.pw_fp8_linear(a, sa, b, sb, y, st)
    want, mag = ref.fp8_linear(a.contiguous().view(torch.uint8).cpu().numpy(), f64(sa),
                               b.contiguous().view(torch.uint8).cpu().numpy(), f64(sb))
    within(f64(y), want, U[torch.bfloat16] * np.abs(want) * 1.01 + 2.0 ** -13 * mag + TINY[torch.bfloat16])
    assert int(st.item()) == 0


def test_fp8_linear_same_result_twice():
    g = gen(5)
    for m in (5, 70, 300):
        a, b = [(torch.randn(r, 1024, generator=g) * 60).to(torch.float8_e4m3fn).to(DEV) for r in (m, 700)]
        sa, sb = torch.rand(m, 8, generator=g).to(DEV), torch.rand(6, 8, generator=g).to(DEV)
        out = [torch.empty(m, 700, dtype=torch.float16, device=DEV) for _ in range(3)]
        st = status()
        for y in out:
            pw.pw_fp8_linear(a, sa, b, sb, y, st)
        assert torch.equal(out[0], out[1]) and torch.equal(out[0], out[2])


# ---------------------------------------------------------------- the paged cache
class Batch:
    """Sequences in a paged cache whose pages are handed out at random and
    whose unused rows are NaN."""

    def __init__(self, q_lens, kv_lens, heads, kv_heads, d, ps, dtype, seed, heads_first=False, spare=3):
        g = gen(seed)
        self.q_lens, self.kv = q_lens, kv_lens
        need = [-(-n // ps) for n in kv_lens]
        pages = sum(need) + spare
        order = torch.randperm(pages, generator=g).tolist()
        width = max(need + [1]) + 1
        table = torch.full((len(kv_lens), width), -1, dtype=torch.int32)
        for b, n in enumerate(need):
            for j in range(n):
                table[b, j] = order.pop()
        self.offsets = torch.tensor([0] + list(np.cumsum(q_lens)), dtype=torch.int32).to(DEV)
        self.lens = torch.tensor(kv_lens, dtype=torch.int32).to(DEV)
        self.T = int(sum(q_lens))
        shape = (pages, kv_heads, ps, d) if heads_first else (pages, ps, kv_heads, d)

        def cache():
            t = torch.full(shape, float("nan"), dtype=dtype, device=DEV)
            return t.permute(0, 2, 1, 3) if heads_first else t
        self.k, self.v = cache(), cache()
        for b, n in enumerate(kv_lens):
            for j in range(need[b]):
                m = min(ps, n - j * ps)
                for t in (self.k, self.v):
                    t[int(table[b, j]), :m] = draw(g, m, kv_heads, d, dtype=dtype)
        self.table = table.to(DEV)
        self.q = draw(g, self.T, heads, d, dtype=dtype, scale=1.5)
        self.qkv = draw(g, self.T, heads + 2 * kv_heads, d, dtype=dtype)
        self.heads, self.kv_heads, self.d, self.ps, self.dtype = heads, kv_heads, d, ps, dtype


ROPE = [  # q_lens, kv_lens, heads, kv_heads, d, rotary, page, heads_first
    ([1], [1], 1, 1, 64, 64, 16, False),
    ([1, 1, 1], [5, 33, 70], 8, 2, 128, 128, 16, True),
    ([3, 0, 17], [3, 9, 40], 6, 2, 64, 24, 7, False),
    ([40, 5], [40, 200], 4, 4, 128, 64, 32, True),
    ([2, 2], [2, 9], 3, 1, 20, 10, 3, False),
    ([1] * 300, [11] * 300, 2, 1, 64, 64, 16, False),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("case", range(len(ROPE)))
def test_rope_append(case, interleaved, dtype):
    ql, kl, h, hk, d, rd, ps, hf = ROPE[case]
    b = Batch(ql, kl, h, hk, d, ps, dtype, case, hf)
    sc = pw.pw_rope_scaling(pw.PW_ROPE_YARN, 0, 4.0, 64.0, 32.0, 1.0) if case % 2 else None
    turns, factor = pw.pw_rope_turns(rd, 1e4, sc)
    q, k, v = b.qkv[:, :h], b.qkv[:, h:h + hk], b.qkv[:, h + hk:]
    q_out = torch.empty(b.T, h, d, dtype=dtype, device=DEV)
    kc, vc, st = b.k.clone(), b.v.clone(), status()
    pw.pw_rope_append(q, k, v, turns.to(DEV), kc, vc, b.table, b.offsets, b.lens, q_out, st, interleaved=interleaved,
                      factor=factor)
    assert int(st.item()) == 0
    freq = turns.numpy().astype(np.float64) * 2.0 ** -64 * 2 * np.pi
    at = ref.token_positions(b.offsets.tolist(), kl)
    pos = np.array([p for _, p in at])
    x = f64(b.qkv)
    want = ref.rotate(x[:, :h + hk], pos, freq, factor, interleaved)
    pair = np.sqrt(ref.rotate(x[:, :h + hk] ** 2, pos * 0, freq, 1.0, interleaved))   # |x|
    half = rd // 2
    i = np.arange(half)
    u_, v_ = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    mag = pair.copy()
    mag[..., u_] = mag[..., v_] = np.hypot(pair[..., u_], pair[..., v_]) * factor
    bound = U[dtype] * np.abs(want) * 1.001 + 2.0 ** -20 * mag + TINY[dtype]
    within(q_out, want[:, :h], bound[:, :h])
    page = [int(b.table[s, p // ps]) for s, p in at]
    row = [p % ps for _, p in at]
    within(kc[page, row], want[:, h:], bound[:, h:])
    assert torch.equal(vc[page, row], v)
    # nothing else in the cache has changed
    kc[page, row], vc[page, row] = b.k[page, row], b.v[page, row]
    same = lambda s, t: torch.equal(s.contiguous().view(torch.int16), t.contiguous().view(torch.int16))  # noqa: E731
    assert same(kc, b.k) and same(vc, b.v)
    # queries alone and in place, positions given
    q2 = q.contiguous()
    pw.pw_rope_append(q2, None, None, turns.to(DEV), None, None, None, b.offsets, b.lens, q2, st, interleaved=interleaved,
                      factor=factor, positions=torch.tensor(pos, dtype=torch.int32, device=DEV))
    assert torch.equal(q2, q_out)


def test_rope_far_positions():
    """The angle stays exact at positions where p * f in 32 bits is off by radians."""
    turns, factor = pw.pw_rope_turns(128, 1e4)
    n = 64
    g = gen(9)
    q = draw(g, n, 2, 128)
    pos = torch.randint(0, 2 ** 31 - 1, (n,), generator=g, dtype=torch.int64)
    pos[0] = 2 ** 31 - 1
    st, out = status(), torch.empty_like(q)
    pw.pw_rope_append(q, None, None, turns.to(DEV), None, None, None, torch.tensor([0, n], dtype=torch.int32, device=DEV),
                      torch.tensor([n], dtype=torch.int32, device=DEV), out, st, factor=factor,
                      positions=pos.to(torch.int32).to(DEV))
    # the reference angle in whole numbers
    frac = np.array([[(int(t) * int(p)) % 2 ** 64 / 2.0 ** 64 for t in turns.tolist()] for p in pos.tolist()])
    c, s = np.cos(2 * np.pi * frac)[:, None], np.sin(2 * np.pi * frac)[:, None]
    x = f64(q)
    a, b = x[..., :64], x[..., 64:]
    want = np.concatenate((a * c - b * s, a * s + b * c), -1)
    mag = np.concatenate((np.hypot(a, b),) * 2, -1)
    within(out, want, U[torch.float16] * np.abs(want) * 1.001 + 2.0 ** -20 * mag + 2.0 ** -25)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("rotary", [128, 64, 16, 8])
def test_rope_same_result_at_any_alignment(rotary, interleaved):
    """Accesses of 16, 8, 4 and 1 values give the same bits."""
    b = Batch([5, 1, 20], [30, 7, 20], 3, 2, 128, 16, torch.float16, 4)
    turns, _ = pw.pw_rope_turns(rotary)
    rows = 3 + 2 * 2
    want = None
    for offset, pitch in ((0, rows * 128), (8, rows * 128 + 8), (4, rows * 128 + 4), (3, rows * 128 + 1)):
        room = torch.empty(b.T * pitch + 64, dtype=torch.float16, device=DEV)
        qkv = room[offset:offset + b.T * pitch].view(b.T, pitch)[:, :rows * 128].unflatten(1, (rows, 128))
        qkv.copy_(b.qkv)
        kc, vc, st = b.k.clone(), b.v.clone(), status()
        qo = torch.empty(b.T, 3, 128, dtype=torch.float16, device=DEV)
        pw.pw_rope_append(qkv[:, :3], qkv[:, 3:5], qkv[:, 5:], turns.to(DEV), kc, vc, b.table, b.offsets, b.lens, qo, st,
                          interleaved=interleaved)
        assert int(st.item()) == 0
        got = [t.view(torch.int16) for t in (qo, kc, vc)]
        if want is None:
            want = got
        assert all(torch.equal(x, y) for x, y in zip(got, want))


def test_rope_reports_missing_pages():
    b = Batch([2], [20], 2, 1, 64, 16, torch.float16, 1)
    turns, _ = pw.pw_rope_turns(64)
    q, k, v = b.qkv[:, :2], b.qkv[:, 2:3], b.qkv[:, 3:]
    for bad in (-1, b.k.shape[0], 10 ** 9):
        t = b.table.clone()
        t[0, 1] = bad
        kc, vc, st, qo = b.k.clone(), b.v.clone(), status(), torch.empty(2, 2, 64, dtype=torch.float16, device=DEV)
        pw.pw_rope_append(q, k, v, turns.to(DEV), kc, vc, t, b.offsets, b.lens, qo, st)
        assert int(st.item()) == pw.PW_ERR_NOT_RESIDENT
        assert torch.equal(kc.view(torch.int16), b.k.view(torch.int16))
    st = status()
    pw.pw_rope_append(q, k, v, turns.to(DEV), b.k, b.v, b.table, torch.tensor([0, 1], dtype=torch.int32, device=DEV), b.lens,
                      qo, st)                       # the second token belongs to no sequence
    assert int(st.item()) == pw.PW_ERR_INVALID_ARG


# ---------------------------------------------------------------- attention
def attend(b, ws=None, **kw):
    out = torch.full((b.T, b.heads, b.d), 7.0, dtype=b.dtype, device=DEV)
    lse, st = torch.empty(b.T, b.heads, device=DEV), status()
    if ws is None:
        n = pw.pw_paged_attention_workspace(b.T, len(b.kv), b.heads, b.kv_heads, b.d)
        ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    kw.setdefault("max_q_len", max(b.q_lens))
    kw.setdefault("max_kv_len", max(b.kv))
    pw.pw_paged_attention(b.q, b.k, b.v, b.table, b.offsets, b.lens, out, ws, st, scale=b.d ** -0.5, lse=lse, **kw)
    return out, lse, int(st.item())


def check_attention(b, out, lse, causal=True, window=0):
    want, wl, mag, dots = ref.attention(f64(b.q), f64(b.k), f64(b.v), b.table.cpu().numpy(), b.offsets.tolist(), b.kv,
                                        b.d ** -0.5, causal, window)
    u = U[b.dtype]
    # scores are off by 2^-16 of the sum of their terms' magnitudes at most (32-bit sums of d exact products)
    ds = 2.0 ** -16 * dots
    within(out, want, u * np.abs(want) * 1.01 + (u + 2 * ds + 2.0 ** -16)[..., None] * mag + TINY[b.dtype])
    got, seen = f64(lse), np.isfinite(wl)
    assert np.array_equal(np.isneginf(got), ~seen)
    err = np.abs(got[seen] - wl[seen])
    assert (err <= ds[seen] + 2.0 ** -18 * (1 + np.abs(wl[seen]))).all(), err.max()


ATTN = [  # q_lens, kv_lens, heads, kv_heads, d, page, heads_first, causal, window
    ([1], [1], 1, 1, 64, 16, False, True, 0),
    ([1], [1], 8, 8, 128, 1, False, True, 0),
    ([1, 1, 1, 1], [3, 64, 65, 700], 8, 2, 128, 16, True, True, 0),
    ([1, 1], [900, 31], 16, 1, 64, 13, False, True, 0),
    ([1] * 40, list(range(1, 41)), 4, 4, 64, 16, False, True, 0),
    ([4, 3, 2], [100, 3, 257], 6, 1, 128, 32, False, True, 0),
    ([5, 0, 7], [5, 40, 300], 12, 4, 64, 64, True, True, 0),
    ([20], [20], 4, 2, 128, 16, False, True, 0),
    ([130, 33], [130, 190], 4, 1, 128, 16, True, True, 0),
    ([70, 140], [300, 140], 6, 2, 64, 32, False, True, 0),
    ([65, 1, 64], [129, 500, 64], 4, 4, 128, 128, False, True, 0),
    ([1, 1], [200, 7], 8, 2, 128, 16, False, True, 33),
    ([50, 10], [200, 10], 4, 2, 64, 16, True, True, 17),
    ([100], [400], 2, 1, 128, 64, False, True, 130),
    ([9, 30], [50, 3], 4, 2, 128, 16, False, False, 0),      # more queries than keys
    ([40, 8], [0, 100], 4, 2, 64, 16, False, False, 0),      # nothing to see
    ([10, 3], [4, 0], 4, 2, 128, 16, False, True, 0),        # the first rows see nothing
    ([200], [64], 4, 4, 128, 32, True, True, 0),
    ([37], [150], 4, 4, 128, 48, False, True, 0),            # pages that end inside a block
]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("case", range(len(ATTN)))
def test_paged_attention(case, dtype):
    ql, kl, h, hk, d, ps, hf, causal, window = ATTN[case]
    b = Batch(ql, kl, h, hk, d, ps, dtype, 100 + case, hf)
    out, lse, st = attend(b, causal=causal, window=window)
    assert st == 0
    check_attention(b, out, lse, causal, window)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_attention_every_kernel_for_the_same_batch(dtype):
    """The length bounds only choose the kernel and the grid."""
    b = Batch([1, 12, 70], [300, 12, 260], 8, 2, 128, 16, dtype, 3)
    for mq in (1, 8, 64, 1000):
        for mk in (1, 300, 100000):
            out, lse, st = attend(b, max_q_len=mq, max_kv_len=mk)
            assert st == 0
            check_attention(b, out, lse)


def test_attention_workspace_is_left_ready():
    """One workspace for many calls of different shapes; the same call gives
    the same bits."""
    n = max(pw.pw_paged_attention_workspace(400, 64, 8, 2, d) for d in (64, 128))
    ws = torch.zeros(n, dtype=torch.uint8, device=DEV)
    first = {}
    for rep in range(2):
        for i, (ql, kl, d) in enumerate([([1], [5000], 128), ([1, 1], [3000, 40], 64), ([100, 1], [300, 999], 128),
                                         ([1] * 64, [50] * 64, 128), ([7], [2000], 64)]):
            b = Batch(ql, kl, 8, 2, d, 16, torch.float16, i)
            out, lse, st = attend(b, ws)
            assert st == 0
            if rep == 0:
                check_attention(b, out, lse)
                first[i] = (out, lse)
            else:
                assert torch.equal(out, first[i][0]) and torch.equal(lse, first[i][1])


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("ql,kl,h,hk,d", [
    ([1], [9000], 4, 1, 64),           # many pieces of few rows
    ([4], [9000], 8, 2, 128),          # and of sixteen
    ([3, 1], [7000, 2500], 15, 3, 64), # heads that do not divide the CTAs
    ([70], [9000], 4, 1, 128),         # full tiles, joined in two steps
    ([100], [9000], 9, 3, 64),
    ([300, 5], [1500, 4000], 10, 5, 128),
    ([260], [700], 2, 2, 64)])
def test_attention_pieces_of_a_unit(ql, kl, h, hk, d, dtype):
    """A unit that many CTAs share, joined in one step and in two; the same bits every time."""
    b = Batch(ql, kl, h, hk, d, 16, dtype, 7)
    ws = torch.zeros(pw.pw_paged_attention_workspace(b.T, len(kl), h, hk, d), dtype=torch.uint8, device=DEV)
    out, lse, st = attend(b, ws)
    assert st == 0
    check_attention(b, out, lse)
    for _ in range(3):
        again, lse2, st = attend(b, ws)
        assert st == 0 and torch.equal(out, again) and torch.equal(lse, lse2)


def test_attention_strided_rows():
    """q and out inside wider rows; nothing beside out is written."""
    for ql in ([1, 1], [40, 3]):
        b = Batch(ql, [77, 200], 4, 2, 128, 16, torch.float16, 8)
        want, _, _ = attend(b)
        wide = torch.randn(b.T, 10, 128, device=DEV).half()
        wide[:, 1:5] = b.q
        out = torch.full((4, b.T, 136), 7.0, dtype=torch.float16, device=DEV)   # heads outermost
        ws = torch.zeros(pw.pw_paged_attention_workspace(b.T, 2, 4, 2, 128), dtype=torch.uint8, device=DEV)
        st = status()
        pw.pw_paged_attention(wide[:, 1:5], b.k, b.v, b.table, b.offsets, b.lens, out.permute(1, 0, 2)[..., :128], ws, st,
                              scale=128 ** -0.5, max_q_len=max(ql), max_kv_len=200)
        assert torch.equal(out.permute(1, 0, 2)[..., :128], want) and (out[..., 128:] == 7).all()


def test_attention_window_ignores_freed_pages():
    """Pages that have left every window may be gone."""
    for ql in (1, 3, 60):
        b = Batch([ql], [500], 4, 2, 128, 16, torch.float16, 6)
        want, wl, _ = attend(b, window=100)
        gone = (500 - ql - 100 + 1) // 16
        for p in b.table[0, :gone].tolist():
            b.k[p], b.v[p] = float("nan"), float("nan")
        b.table[0, :gone] = -1
        out, lse, st = attend(b, window=100)
        assert st == 0 and torch.equal(out, want) and torch.equal(lse, wl)


def test_attention_reports_what_it_cannot_follow():
    for ql in (1, 50):
        b = Batch([ql, ql], [100, 90], 4, 2, 128, 16, torch.float16, 2)
        good, _, _ = attend(b)
        for bad in (-1, b.k.shape[0], 10 ** 9):
            t = b.table.clone()
            b.table[0, 2] = bad
            out, _, st = attend(b)
            assert st == pw.PW_ERR_NOT_RESIDENT and torch.equal(out[ql:], good[ql:])
            b.table = t
        lens = b.lens.clone()
        for bad in (-5, 10 ** 9):
            b.lens[1] = bad
            out, _, st = attend(b)
            assert st in (pw.PW_ERR_INVALID_ARG, pw.PW_ERR_NOT_RESIDENT) and torch.equal(out[:ql], good[:ql])
            b.lens.copy_(lens)
        b.offsets[2] = 10 ** 6
        out, _, st = attend(b)
        assert st == pw.PW_ERR_INVALID_ARG and torch.equal(out[:ql], good[:ql])


def test_attention_scores_of_any_size():
    """Scores far apart, equal, and at the type's ends: no overflow, no NaN."""
    for ql in (1, 60):
        b = Batch([ql], [333], 4, 2, 64, 16, torch.float16, 4)
        b.q *= 30
        out, lse, st = attend(b)
        want, wl, mag, dots = ref.attention(f64(b.q), f64(b.k), f64(b.v), b.table.cpu().numpy(), b.offsets.tolist(), b.kv, 0.125)
        u = U[torch.float16]
        within(out, want, 2 * u * mag + 2.0 ** -14 * dots[..., None] * mag + 2.0 ** -25)
        assert np.abs(f64(lse) - wl).max() <= 2.0 ** -15 * dots.max()
        b.q.zero_()
        out, lse, st = attend(b)
        check_attention(b, out, lse)


def test_long_cache_offsets_pass_32_bits():
    """A cache of more than 2^31 values: pages at its far end."""
    ps, hk, d = 16, 8, 128
    pages = (2 ** 31) // (ps * hk * d) + 64
    k = torch.zeros(pages, ps, hk, d, dtype=torch.float16, device=DEV)
    v = torch.zeros_like(k)
    for ql in (1, 40):
        b = Batch([ql], [100], 16, 8, 128, 16, torch.float16, 12)
        want, wl, _ = attend(b)
        table = b.table.clone()
        for j in range(7):
            far = pages - 1 - 9 * j
            k[far], v[far] = b.k[int(b.table[0, j])], b.v[int(b.table[0, j])]
            table[0, j] = far
        b.k, b.v, b.table = k, v, table
        out, lse, st = attend(b)
        assert st == 0 and torch.equal(out, want) and torch.equal(lse, wl)
        turns, _ = pw.pw_rope_turns(128)
        qo, s = torch.empty_like(b.q), status()
        b.lens = torch.tensor([100], dtype=torch.int32, device=DEV)
        pw.pw_rope_append(b.qkv[:, :16], b.qkv[:, 16:24], b.qkv[:, 24:], turns.to(DEV), k, v, table, b.offsets, b.lens, qo, s)
        assert int(s.item()) == 0
        at = torch.arange(100 - ql, 100)
        assert torch.equal(v[table[0, at // 16].long().cpu(), at % 16], b.qkv[:, 24:])


def test_other_stream():
    b = Batch([1, 30], [300, 60], 8, 2, 128, 16, torch.float16, 15)
    want, wl, _ = attend(b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, lse, st = attend(b)
    torch.cuda.current_stream().wait_stream(side)
    assert st == 0 and torch.equal(out, want) and torch.equal(lse, wl)
