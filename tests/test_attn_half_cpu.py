"""The attention half without a GPU: the oracle against independent values,
the frequency table, and the argument checks that come before any launch."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

from oracle import attn_half as ref

pw = pytest.importorskip("any_precision_bit_pw_gb300.pw")
FAKE = 0x7F0000000000  # never dereferenced


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(pw.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return pw.lib()


def test_e4m3_values_match_torch():
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    got = ref.e4m3_decode(codes.numpy())
    assert np.array_equal(np.isnan(want), np.isnan(got))
    assert np.array_equal(want[~np.isnan(want)], got[~np.isnan(got)])
    at = got[:127]                           # the values from 0 to 448, ascending
    assert np.array_equal(ref.e4m3_step(at[:-1]), np.diff(at))


def test_oracle_attention_against_a_closed_form():
    # equal scores: the mean of the visible values
    rng = np.random.default_rng(0)
    v = rng.standard_normal((3, 4, 1, 8))
    q, k = np.zeros((2, 2, 8)), rng.standard_normal((3, 4, 1, 8))
    table = np.array([[2, 0, 1]])
    out, lse, _, _ = ref.attention(q, k, v, table, [0, 2], [7], 0.5)
    flat = v[[2, 0, 1]].reshape(-1, 8)
    assert np.allclose(out[0, 0], flat[:6].mean(0)) and np.allclose(out[1, 1], flat[:7].mean(0))
    assert np.allclose(lse, np.log([[6, 6], [7, 7]]))
    out, _, _, _ = ref.attention(q, k, v, table, [0, 2], [7], 0.5, window=2)
    assert np.allclose(out[0, 0], flat[4:6].mean(0))
    out, lse, _, _ = ref.attention(q, k, v, table, [0, 2], [1], 0.5)
    assert np.all(out[0] == 0) and np.all(lse[0] == -np.inf) and np.allclose(out[1, 0], flat[0])


def test_oracle_rotation_is_a_rotation():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((4, 2, 16))
    f, _ = ref.frequencies(8, 100.0)
    for inter in (False, True):
        y = ref.rotate(x, np.array([0, 1, 5, 900]), f, 1.0, inter)
        assert np.allclose(y[0], x[0]) and np.array_equal(y[..., 8:], x[..., 8:])
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
        # scores depend on the distance of positions only
        a = ref.rotate(x, np.array([3, 10, 20, 30]), f, 1.0, inter)
        b = ref.rotate(x, np.array([8, 15, 25, 35]), f, 1.0, inter)
        assert np.allclose((a[0] * a[1]).sum(), (b[0] * b[1]).sum())


SCALINGS = [("plain", 0, {}), ("linear", 1, dict(scale=4.0)), ("ntk", 2, dict(scale=8.0)),
            ("yarn", 3, dict(scale=16.0, original=4096.0, fast=32.0, slow=1.0)),
            ("bands", 4, dict(scale=8.0, original=8192.0, fast=4.0, slow=1.0))]


@pytest.mark.parametrize("d", [2, 24, 64, 128])
@pytest.mark.parametrize("name,kind,kw", SCALINGS, ids=[s[0] for s in SCALINGS])
def test_rope_turns(L, d, name, kind, kw):
    if name == "ntk" and d < 4:
        pytest.skip("the base change needs two pairs")
    sc = pw.pw_rope_scaling(kind, 0, kw.get("scale", 0.0), kw.get("original", 0.0), kw.get("fast", 0.0), kw.get("slow", 0.0))
    turns, factor = pw.pw_rope_turns(d, 5e5, sc)
    f, want = ref.frequencies(d, 5e5, name, **kw)
    got = turns.numpy().astype(np.float64) * 2.0 ** -64 * 2 * math.pi
    # a few roundings of 64-bit arithmetic (pow, log), and half a unit of 2^-64 turns
    assert np.all(np.abs(got - f) <= 2.0 ** -46 * f + 2.0 ** -61)
    assert abs(factor - want) <= 2.0 ** -23 * want


@pytest.mark.parametrize("d,base,sc", [
    (0, 1e4, None), (7, 1e4, None), (2048, 1e4, None), (64, 1.0, None), (64, math.nan, None), (64, math.inf, None),
    (64, 1e4, (5, 2.0, 0, 0, 0)), (64, 1e4, (-1, 2.0, 0, 0, 0)), (64, 1e4, (1, 0.5, 0, 0, 0)),
    (64, 1e4, (1, math.nan, 0, 0, 0)), (2, 1e4, (2, 2.0, 0, 0, 0)), (64, 1e4, (3, 2.0, 0, 32, 1)),
    (64, 1e4, (3, 2.0, 4096, 1, 32)), (64, 1e4, (4, 2.0, 4096, 4, 0))])
def test_rope_turns_refusals(L, d, base, sc):
    s = None if sc is None else pw.pw_rope_scaling(sc[0], 0, sc[1], sc[2], sc[3], sc[4])
    with pytest.raises(pw.PwError):
        pw.pw_rope_turns(d, base, s)


def _call(f, struct, defaults, kw):
    a = struct()
    for k, v in {**defaults, **kw}.items():
        setattr(a, k, v)
    return f(ctypes.byref(a), None)


def _norm(L, **kw):
    return _call(L.pw_add_rmsnorm, pw.pw_norm_args, dict(
        x=FAKE, x_stride=64, residual=FAKE, residual_stride=64, weight=FAKE, rows=4, cols=64, eps=1e-5, dtype=0,
        residual_out=FAKE, residual_out_stride=64, y=FAKE, y_stride=64, q=FAKE, q_stride=64, scale=FAKE, scale_stride=1), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), -2), (dict(rows=-1), -1), (dict(cols=0), -1), (dict(cols=32769, x_stride=40000), -2),
    (dict(eps=-1.0), -1), (dict(eps=math.nan), -1), (dict(y=None, q=None, scale=None), -1), (dict(q=None), -1),
    (dict(scale=None), -1), (dict(x_stride=63), -1), (dict(residual_stride=63), -1), (dict(residual_out_stride=1), -1),
    (dict(y_stride=63), -1), (dict(q_stride=63), -1), (dict(scale_stride=0), -1), (dict(x=None), -1), (dict(weight=None), -1),
    (dict(x=FAKE + 1), -1), (dict(scale=FAKE + 2), -1)])
def test_norm_refusals(L, kw, code):
    assert _norm(L, **kw) == code and "add_rmsnorm" in pw.pw_last_error()
    assert L.pw_add_rmsnorm(None, None) == -1


def _quant(L, **kw):
    return _call(L.pw_quantize_fp8, pw.pw_quant_args, dict(
        x=FAKE, x_stride=64, rows=4, cols=64, dtype=0, block_rows=1, q=FAKE, q_stride=64, scale=FAKE, scale_stride=1), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), -2), (dict(block_rows=64), -2), (dict(rows=-4), -1), (dict(cols=0), -1), (dict(x_stride=63), -1),
    (dict(q_stride=63), -1), (dict(cols=129, x_stride=129, q_stride=129), -1), (dict(x=None), -1), (dict(q=None), -1),
    (dict(scale=None), -1), (dict(cols=1 << 16, x_stride=1 << 16, q_stride=1 << 16, scale_stride=1 << 9), -2),
    (dict(rows=1 << 23, block_rows=128), -2), (dict(x=FAKE + 1), -1), (dict(scale=FAKE + 1), -1)])
def test_quantize_refusals(L, kw, code):
    assert _quant(L, **kw) == code and "quantize_fp8" in pw.pw_last_error()
    assert L.pw_quantize_fp8(None, None) == -1


def _linear(L, **kw):
    return _call(L.pw_fp8_linear, pw.pw_linear_args, dict(
        a=FAKE, lda=256, a_scale=FAKE, a_scale_stride=2, b=FAKE, ldb=256, b_scale=FAKE, b_scale_stride=2, m=4, n=128, k=256,
        dtype=0, y=FAKE, ldy=128, status=FAKE), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), -2), (dict(m=-1), -1), (dict(n=0), -1), (dict(k=0), -1), (dict(m=(1 << 20) + 1), -2),
    (dict(lda=240), -1), (dict(ldb=240), -1), (dict(ldy=127), -1), (dict(a_scale_stride=1), -1), (dict(b_scale_stride=1), -1),
    (dict(a=None), -1), (dict(a_scale=None), -1), (dict(b=None), -1), (dict(b_scale=None), -1), (dict(y=None), -1),
    (dict(status=None), -1), (dict(a=FAKE + 8), -1), (dict(b=FAKE + 4), -1), (dict(lda=264), -1), (dict(ldb=257), -1),
    (dict(a_scale=FAKE + 1), -1), (dict(status=FAKE + 2), -1), (dict(ldb=1 << 39), -2)])
def test_linear_refusals(L, kw, code):
    assert _linear(L, **kw) == code and "fp8_linear" in pw.pw_last_error()
    assert L.pw_fp8_linear(None, None) == -1


def test_empty_calls_touch_nothing(L):
    assert _norm(L, rows=0, x=None, weight=None) == 0
    assert _quant(L, rows=0, x=None, q=None, scale=None) == 0
    assert _linear(L, m=0, a=None, b=None, y=None, status=None) == 0


def _rope_args(**kw):
    a = pw.pw_rope_args()
    for n in ("q", "q_out", "k", "v", "k_cache", "v_cache", "turns", "page_table", "q_offsets", "kv_lens", "status"):
        setattr(a, n, FAKE)
    a.tokens, a.batch, a.heads, a.kv_heads, a.head_dim, a.rotary_dim = 4, 2, 4, 2, 64, 64
    a.page_size, a.num_pages, a.pages_per_seq, a.page_table_stride, a.factor = 16, 8, 4, 4, 1.0
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), -2), (dict(tokens=-1), -1), (dict(batch=-1), -1), (dict(head_dim=0), -1), (dict(rotary_dim=65), -1),
    (dict(rotary_dim=66), -1), (dict(rotary_dim=-2), -1), (dict(head_dim=2048), -2), (dict(factor=math.inf), -1),
    (dict(k=None), -1), (dict(v=None), -1), (dict(k_cache=None), -1), (dict(q_out=None), -1), (dict(q=None), -1),
    (dict(q=None, q_out=None, k=None, v=None, k_cache=None, v_cache=None), -1), (dict(q_offsets=None), -1),
    (dict(kv_lens=None), -1), (dict(status=None), -1), (dict(turns=None), -1), (dict(batch=0), -1), (dict(page_table=None), -1),
    (dict(page_size=0), -1), (dict(num_pages=0), -1), (dict(pages_per_seq=0), -1), (dict(page_table_stride=3), -1),
    (dict(k_cache=FAKE + 1), -1)])
def test_rope_refusals(L, kw, code):
    assert L.pw_rope_append(ctypes.byref(_rope_args(**kw)), None) == code and "rope_append" in pw.pw_last_error()
    assert L.pw_rope_append(None, None) == -1


def _attn_args(**kw):
    a = pw.pw_attn_args()
    for n in ("q", "out", "k_cache", "v_cache", "page_table", "q_offsets", "kv_lens", "status"):
        setattr(a, n, FAKE)
    a.tokens, a.batch, a.heads, a.kv_heads, a.head_dim = 4, 2, 4, 2, 128
    a.page_size, a.num_pages, a.pages_per_seq, a.page_table_stride = 16, 8, 4, 4
    a.max_q_len, a.max_kv_len, a.causal, a.scale = 2, 64, 1, 0.1
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=5), -2), (dict(tokens=-1), -1), (dict(heads=5), -1), (dict(kv_heads=0), -1), (dict(head_dim=96), -2),
    (dict(window=-1), -1), (dict(window=4, causal=0), -1), (dict(scale=math.nan), -1), (dict(page_size=0), -1),
    (dict(pages_per_seq=0), -1), (dict(page_table_stride=2), -1), (dict(page_size=1 << 29), -2), (dict(tokens=1 << 29), -2),
    (dict(q=None), -1), (dict(out=None), -1), (dict(k_cache=None), -1), (dict(v_cache=None), -1), (dict(page_table=None), -1),
    (dict(q_offsets=None), -1), (dict(kv_lens=None), -1), (dict(status=None), -1), (dict(q_stride_token=4), -1),
    (dict(k_stride_page=1), -1), (dict(out=FAKE + 2), -1), (dict(v_cache=FAKE + 8), -1), (dict(max_q_len=-1), -1)])
def test_attention_refusals(L, kw, code):
    rc = L.pw_paged_attention(ctypes.byref(_attn_args(**kw)), FAKE, 1 << 30, None)
    assert rc == code and "paged_attention" in pw.pw_last_error()


@pytest.mark.parametrize("name,offset", [("page_table", 2), ("q_offsets", 1), ("kv_lens", 2), ("status", 3)])
def test_misaligned_words_are_refused(L, name, offset):
    kw = {name: FAKE + offset}
    assert L.pw_rope_append(ctypes.byref(_rope_args(**kw)), None) == pw.PW_ERR_INVALID_ARG
    assert L.pw_paged_attention(ctypes.byref(_attn_args(**kw)), FAKE, 1 << 30, None) == pw.PW_ERR_INVALID_ARG
    assert L.pw_paged_attention(ctypes.byref(_attn_args(lse=FAKE + offset)), FAKE, 1 << 30, None) == pw.PW_ERR_INVALID_ARG
    for word in (dict(positions=FAKE + offset), dict(turns=FAKE + 4)):
        assert L.pw_rope_append(ctypes.byref(_rope_args(**word)), None) == pw.PW_ERR_INVALID_ARG


def test_attention_workspace(L):
    need = pw.pw_paged_attention_workspace(4, 2, 4, 2, 128)
    assert need > 0
    assert pw.pw_paged_attention_workspace(4, 2, 5, 2, 128) == 0 and pw.pw_paged_attention_workspace(4, 2, 4, 2, 80) == 0
    a = _attn_args()
    assert L.pw_paged_attention(ctypes.byref(a), FAKE, need - 1, None) == pw.PW_ERR_WORKSPACE
    assert L.pw_paged_attention(ctypes.byref(a), FAKE + 16, need, None) == pw.PW_ERR_WORKSPACE
    assert L.pw_paged_attention(ctypes.byref(a), None, need, None) == pw.PW_ERR_INVALID_ARG
    assert L.pw_paged_attention(None, FAKE, need, None) == pw.PW_ERR_INVALID_ARG
    assert L.pw_paged_attention(ctypes.byref(_attn_args(tokens=0)), FAKE, 0, None) == 0


def test_binding_checks():
    x = torch.zeros(4, 64, dtype=torch.float16)
    with pytest.raises(ValueError):          # not on the GPU
        pw.pw_add_rmsnorm(x, x[0], 1e-5, y=x)
    with pytest.raises(ValueError):          # fp32
        pw.pw_quantize_fp8(x.float(), x, x)
    with pytest.raises(ValueError):
        pw.pw_rope_append(None, None, None, x, None, None, None, x, x, None, x)


def test_paged_cache_hands_out_pages():
    from any_precision_bit_pw_gb300.decoder import PagedCache
    c = PagedCache(6, 4, 1, 8, device="cpu")
    b = c.batch([5, 9], [7, 0])
    assert (b.tokens, b.max_q_len, b.max_kv_len) == (7, 7, 7)
    assert b.q_offsets.tolist() == [0, 7, 7] and b.kv_lens.tolist() == [7, 0]
    assert b.page_table.tolist() == [c.pages[5], [-1, -1]] and len(set(c.pages[5])) == 2
    before = list(c.pages[5])
    b = c.batch([9, 5], [1, 1], width=3)                 # sequence 5 still has room in its second page
    assert c.pages[5] == before and b.kv_lens.tolist() == [1, 8] and b.page_table.shape == (2, 3)
    assert len(c.free_pages) == 3 and b.page_table[0, 1:].tolist() == [-1, -1]
    for bad in (dict(seqs=[5, 5], new_tokens=[1, 1]), dict(seqs=[5], new_tokens=[-1]), dict(seqs=[5], new_tokens=[4], width=2)):
        with pytest.raises((ValueError, RuntimeError)):
            c.batch(**bad)
    with pytest.raises(RuntimeError):
        c.batch([5], [40])
    free = len(c.free_pages)
    held = len(c.pages[5])
    c.release(5)
    assert len(c.free_pages) == free + held and 5 not in c.lens
    c.release(5)                                         # nothing left to return
    assert len(c.free_pages) == free + held
