"""GPU: the kernels and loops of the attention half that only larger calls
reach, against the 64-bit oracle: CTAs with several tiles, rows or tokens, pairs
of CTAs, batches of more sequences than threads.  Sizes are the smallest that
get there, ragged, with few column groups.  What a call launches is asked of the
profiler, so that a change of the rules cannot take a path out of the tests."""
import numpy as np
import pytest
import torch

from oracle import attn_half as ref
from test_gpu_attn_half import (Batch, DEV, DTYPES, IDS, TINY, U, _gpu, attend, check_attention, check_codes, draw, f64,  # noqa: F401
                                gen, pw, status, within)

pytestmark = pytest.mark.gpu


def launches(f):
    """Names of the kernels that f launches; f has run before."""
    from torch.profiler import ProfilerActivity, profile
    torch.cuda.synchronize()
    for _ in range(3):      # a process's first recording may come back empty
        with profile(activities=[ProfilerActivity.CUDA]) as p:
            f()
            torch.cuda.synchronize()
        names = [e.name for e in p.events()]
        if names:
            break
    return names


def launched(f, kernel, *numbers):
    """Whether f launches `kernel` with these template numbers."""
    names = launches(f)
    if not names:
        pytest.skip("the profiler records no kernels here")
    plain = ", ".join(str(n) for n in numbers)
    coded = "".join(f"Li{n}E" for n in numbers)
    return any(kernel in n and (plain in n or coded in n) for n in names)


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


# ---------------------------------------------------------------- the 8-bit product
def product(m, n, k, dtype, scale_pad=0, y_pad=0):
    g = gen(m * 31 + n * 7 + k)
    kb, pad = -(-k // 128), -k % 16

    def codes(rows):
        t = (torch.randn(rows, k + pad, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
        t[:, k:] = float("nan")                    # past the columns: anything
        return t.to(DEV)[:, :k]

    def scales(rows, shift):
        t = torch.full((rows, kb + scale_pad), float("nan"))
        t[:, :kb] = torch.exp(torch.randn(rows, kb, generator=g) - shift)
        return t.to(DEV)[:, :kb]
    a, b, sa, sb = codes(m), codes(n), scales(m, 0), scales(-(-n // 128), 6)
    y = torch.full((m, n + y_pad), 7.0, dtype=dtype, device=DEV)
    st = status()
    run = lambda: pw.pw_fp8_linear(a, sa, b, sb, y[:, :n], st)  # noqa: E731
    run()
    want, mag = ref.fp8_linear(a.view(torch.uint8).cpu().numpy(), f64(sa), b.view(torch.uint8).cpu().numpy(), f64(sb))
    # the bound of the smaller sizes: one rounding to 16 bits, and 13 bits below a group's largest product
    bound = U[dtype] * np.abs(want) * 1.01 + 2.0 ** -13 * mag + TINY[dtype]
    got, top = f64(y[:, :n]), torch.finfo(dtype).max
    over = np.isinf(got)
    assert (np.abs(want[over]) + bound[over] > top).all() and (np.sign(want[over]) == np.sign(got[over])).all()
    within(got[~over], want[~over], bound[~over])
    assert (y[:, n:] == 7).all() and int(st.item()) == 0
    first = y.clone()
    run()
    assert torch.equal(y, first)
    return run


# scale_pad makes rows of scales start at 16-byte addresses (or not), y_pad rows of y
PAIR = [(1900, 4700, 256, 2, 4), (1900, 4701, 640, 3, 3), (2300, 2048, 272, 1, 0), (2300, 2040, 128, 0, 0), (4300, 2048, 300, 0, 0),
        (4300, 2044, 1100, 3, 4), (4090, 2048, 1152, 0, 1)]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("m,n,k,scale_pad,y_pad", PAIR)
def test_product_by_pairs_of_ctas(m, n, k, scale_pad, y_pad, dtype):
    """256 x 256 tiles: ragged edges, one and two tiles a pair, several strips of
    tokens; 1 to 9 groups of columns; scales and results by wide and narrow ways."""
    run = product(m, n, k, dtype, scale_pad, y_pad)
    assert launched(run, "linear_tile_kernel", 256, 256)


@pytest.mark.parametrize("m,n,k,scale_pad,y_pad,tile", [
    (270, 12800, 256, 2, 0, 128), (300, 12900, 640, 3, 4, 128), (290, 12801, 300, 0, 0, 128), (260, 12800, 128, 0, 0, 128),
    (50, 20000, 256, 2, 0, 64), (64, 19999, 700, 2, 1, 64), (33, 20100, 100, 0, 4, 64)])
def test_product_several_tiles_a_cta(m, n, k, scale_pad, y_pad, tile):
    """More tiles than SMs by single CTAs: rings, scale slots and the way out go on across tiles."""
    assert -(-m // tile) * -(-n // 128) > sms()
    run = product(m, n, k, DTYPES[n % 2], scale_pad, y_pad)
    assert launched(run, "linear_tile_kernel", tile, 128)


@pytest.mark.parametrize("m,n,k,groups,warps", [
    (1, 500, 1300, 1, 16), (5, 1000, 4096, 1, 16), (8, 4096, 2000, 1, 16), (7, 5000, 1400, 1, 8), (3, 300, 1000, 1, 8),
    (16, 500, 1300, 2, 16), (30, 500, 2000, 4, 16), (16, 5000, 1300, 2, 8), (20, 4000, 2048, 4, 8)])
def test_product_streamed(m, n, k, groups, warps):
    run = product(m, n, k, DTYPES[m % 2], -k % 3)
    assert launched(run, "linear_stream_kernel", groups, warps)


# ---------------------------------------------------------------- norm and quantisation
ROWS = [(12001, 256), (12001, 251), (3001, 6144), (1500, 6143), (1201, 8200), (1000, 8191), (701, 16392), (500, 16391), (301, 32768)]


@pytest.mark.parametrize("rows,cols", ROWS)
def test_norm_of_more_rows_than_ctas(rows, cols):
    """A CTA walks over rows: the next row is under way while this one is finished."""
    dtype = DTYPES[rows % 2]
    g = gen(rows + cols)
    x, res = draw(g, rows, cols, dtype=dtype), draw(g, rows, cols, dtype=dtype, scale=3)
    x *= torch.exp(torch.randn(rows, 1, generator=g)).to(dtype).to(DEV)          # rows that differ
    w = (1 + 0.2 * torch.randn(cols, generator=g)).to(dtype).to(DEV)
    y, ro = torch.empty_like(x), torch.empty_like(x)
    q, sc = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device=DEV), torch.empty(rows, -(-cols // 128), device=DEV)
    pw.pw_add_rmsnorm(x, w, 1e-5, residual=res, residual_out=ro, y=y, q=q, scale=sc)
    r, want = ref.add_rmsnorm(f64(x), f64(w), 1e-5, f64(res))
    u = U[dtype]
    within(ro, r, u * np.abs(r) * (1 + 2.0 ** -10) + TINY[dtype])
    within(y, want, u * np.abs(want) * (1 + 2.0 ** -8) + TINY[dtype])
    check_codes(q, sc, want, 1)
    # in place: the row that is loaded ahead is another one
    y2, res2 = x.clone(), res.clone()
    pw.pw_add_rmsnorm(y2, w, 1e-5, residual=res2, residual_out=res2, y=y2)
    assert torch.equal(y2, y) and torch.equal(res2, ro)


@pytest.mark.parametrize("rows,cols", ROWS)
def test_row_quantisation_of_more_rows_than_ctas(rows, cols):
    x = draw(gen(rows * 3 + cols), rows, cols, dtype=DTYPES[(rows + 1) % 2], scale=5)
    x *= torch.exp(torch.randn(rows, 1, generator=gen(rows))).to(x.dtype).to(DEV)
    q, sc = torch.empty(rows, cols, dtype=torch.uint8, device=DEV), torch.empty(rows, -(-cols // 128), device=DEV)
    pw.pw_quantize_fp8(x, q, sc)
    check_codes(q, sc, f64(x), 1)


# ---------------------------------------------------------------- rotary append
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("h,hk,d,rd,heads_first", [(3, 1, 128, 128, True), (4, 2, 64, 32, False), (2, 1, 24, 8, False),
                                                   (2, 2, 20, 10, True)])
def test_rope_two_tokens_a_cta(h, hk, d, rd, heads_first, interleaved, dtype):
    """More than 8 tokens an SM: CTAs share the search among two tokens, of one
    sequence or of two; their number is odd."""
    ql = [700, 1, 0, 513, 3] + [1, 2] * 40 + [8 * sms() - 1217 + 300]
    ql[-1] += 1 - sum(ql) % 2
    kl = [n + 37 * i % 300 for i, n in enumerate(ql)]
    assert sum(ql) > 8 * sms() and sum(ql) % 2 == 1
    b = Batch(ql, kl, h, hk, d, 16, dtype, 40, heads_first)
    turns, factor = pw.pw_rope_turns(rd, 1e4, pw.pw_rope_scaling(pw.PW_ROPE_LINEAR, 0, 4.0, 0, 0, 0))
    q_out, kc, vc, st = torch.empty(b.T, h, d, dtype=dtype, device=DEV), b.k.clone(), b.v.clone(), status()
    pw.pw_rope_append(b.qkv[:, :h], b.qkv[:, h:h + hk], b.qkv[:, h + hk:], turns.to(DEV), kc, vc, b.table, b.offsets, b.lens,
                      q_out, st, interleaved=interleaved, factor=factor)
    assert int(st.item()) == 0
    freq = turns.numpy().astype(np.float64) * 2.0 ** -64 * 2 * np.pi
    at = ref.token_positions(b.offsets.tolist(), kl)
    x = f64(b.qkv)
    want = ref.rotate(x[:, : h + hk], np.array([p for _, p in at]), freq, factor, interleaved)
    bound = U[dtype] * np.abs(want) * 1.001 + 2.0 ** -20 * 2 * np.abs(x).max() + TINY[dtype]
    within(q_out, want[:, :h], bound[:, :h])
    table = b.table.cpu().numpy()
    page, row = [int(table[s, p // 16]) for s, p in at], [p % 16 for _, p in at]
    within(kc[page, row], want[:, h:], bound[:, h:])
    assert torch.equal(vc[page, row], b.qkv[:, h + hk:])
    kc[page, row], vc[page, row] = b.k[page, row], b.v[page, row]     # nothing else has changed
    for got, before in ((kc, b.k), (vc, b.v)):
        assert torch.equal(got.contiguous().view(torch.int16), before.contiguous().view(torch.int16))


# ---------------------------------------------------------------- attention
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("h,hk,window", [(4, 2, 0), (3, 3, 0), (8, 1, 20)])
def test_attention_of_many_sequences(h, hk, window, dtype):
    """More sequences than the 128 threads of the kernel for few rows, some without new tokens or keys."""
    ql = [(1, 1, 2, 0, 1)[i % 5] for i in range(301)]
    kl = [0 if i % 41 == 7 else 1 + i * 29 % 90 for i in range(301)]
    b = Batch(ql, kl, h, hk, 64, 16, dtype, 50)
    out, lse, st = attend(b, window=window)
    assert st == 0
    check_attention(b, out, lse, True, window)
    assert launched(lambda: attend(b, window=window), "attn_stream_kernel", 64)


@pytest.mark.parametrize("h,hk,causal", [(16, 2, True), (24, 3, False)])
def test_chunk_attention_of_many_sequences(h, hk, causal):
    """More sequences than the 384 threads of the kernel for chunks."""
    ql = [(3, 1, 0, 4)[i % 4] for i in range(901)]
    kl = [0 if i % 97 == 5 else 1 + i * 13 % 40 for i in range(901)]
    b = Batch(ql, kl, h, hk, 64, 16, DTYPES[hk % 2], 51)
    out, lse, st = attend(b, causal=causal)
    assert st == 0
    check_attention(b, out, lse, causal)
    assert launched(lambda: attend(b, causal=causal), "attn_tile_kernel", 64)
