"""The operators around the attention half without a GPU: the oracle against
independent values, and the argument checks that come before any launch."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

from oracle import more_ops as ref

pw = pytest.importorskip("any_precision_bit_pw_gb300.pw")
FAKE = 0x7F0000000000  # never dereferenced


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(pw.LIB_PATH):
        import __graft_entry__
        __graft_entry__.build()
    return pw.lib()


def test_oracle_norms():
    rng = np.random.default_rng(0)
    x, res, w = rng.standard_normal((3, 8)), rng.standard_normal((3, 8)), rng.standard_normal(8)
    r, y, _ = ref.norm_add_norm(x, res, 0.0, post_weight=np.ones(8), weight=w, residual_scale=0.0, block_scale=3.0)
    assert np.allclose((r ** 2).mean(axis=1), 9.0)           # a normed row has mean square 1
    assert np.allclose(((y / w) ** 2).mean(axis=1), 1.0)
    r, y, _ = ref.norm_add_norm(x, res, 1e-5, gate=w, residual_scale=2.0)
    assert y is None and np.allclose(r, 2 * res + x * w)


def test_oracle_logprobs():
    z = np.log(np.array([[0.5, 0.25, 0.25, 0.0], [1.0, 0.0, 0.0, 0.0]]) + 0.0, where=np.array([[1, 1, 1, 0], [1, 0, 0, 0]], bool),
               out=np.full((2, 4), -np.inf))
    lp, lse, h, ids, top = ref.token_logprobs(z + 3.0, np.array([[1, -1], [0, 9]]), 3, 1.0)
    assert np.allclose(lse, 3.0) and np.allclose(h, [1.5 * math.log(2), 0.0])
    assert np.allclose(lp[0], [math.log(0.25), 0.0]) and lp[1, 0] == 0.0 and np.isnan(lp[1, 1])
    assert ids.tolist() == [[0, 1, 2], [0, 1, 2]] and np.allclose(top[0], np.log([0.5, 0.25, 0.25]))
    assert np.isneginf(top[1, 1:]).all()
    lp, lse, h, _, _ = ref.token_logprobs(np.full((1, 5), -np.inf), np.array([[2]]), 1, 1.0)
    assert np.isneginf(lse).all() and np.isneginf(lp).all() and h[0] == 0.0


def _call(f, struct, defaults, kw):
    a = struct()
    for k, v in {**defaults, **kw}.items():
        setattr(a, k, v)
    return f(ctypes.byref(a), None)


def _norms(L, **kw):
    return _call(L.pw_norm_add_norm, pw.pw_norms_args, dict(
        x=FAKE, x_stride=64, residual=FAKE, residual_stride=64, post_weight=FAKE, gate=FAKE, gate_stride=64, weight=FAKE,
        rows=4, cols=64, eps=1e-5, residual_scale=1.0, block_scale=1.0, dtype=0, residual_out=FAKE, residual_out_stride=64,
        y=FAKE, y_stride=64, q=FAKE, q_stride=64, scale=FAKE, scale_stride=1), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), -2), (dict(rows=-1), -1), (dict(cols=0), -1), (dict(cols=32769, x_stride=40000), -2),
    (dict(eps=-1.0), -1), (dict(eps=math.nan), -1), (dict(residual_scale=math.inf), -1), (dict(block_scale=math.nan), -1),
    (dict(residual_out=None, y=None, q=None, scale=None, weight=None), -1), (dict(q=None), -1), (dict(scale=None), -1),
    (dict(weight=None), -1), (dict(y=None, q=None, scale=None), -1), (dict(x_stride=63), -1), (dict(residual_stride=63), -1),
    (dict(gate_stride=63), -1), (dict(gate_stride=-64), -1), (dict(residual_out_stride=1), -1), (dict(y_stride=63), -1),
    (dict(q_stride=63), -1), (dict(scale_stride=0), -1), (dict(x=None), -1), (dict(residual=None), -1), (dict(x=FAKE + 1), -1),
    (dict(gate=FAKE + 1), -1), (dict(weight=FAKE + 1), -1), (dict(scale=FAKE + 2), -1)])
def test_norms_refusals(L, kw, code):
    assert _norms(L, **kw) == code and "norm_add_norm" in pw.pw_last_error()
    assert L.pw_norm_add_norm(None, None) == -1


def _logprobs(L, **kw):
    return _call(L.pw_token_logprobs, pw.pw_logprob_args, dict(
        logits=FAKE, stride=1000, vocab=1000, rows=4, targets=FAKE, targets_stride=2, logprobs=FAKE, logprobs_stride=2, given=2,
        lse=FAKE, entropy=FAKE, top_ids=FAKE, top_ids_stride=5, top_logprobs=FAKE, top_logprobs_stride=5, top=5, dtype=1,
        scale=1.0), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=3), -2), (dict(dtype=-1), -2), (dict(rows=-1), -1), (dict(vocab=0), -1), (dict(given=-1), -1), (dict(top=-1), -1),
    (dict(top=33, top_ids_stride=33, top_logprobs_stride=33), -2), (dict(top=5, vocab=4), -1), (dict(rows=1 << 25), -2),
    (dict(vocab=1 << 29, stride=1 << 29), -2), (dict(scale=0.0), -1), (dict(scale=-1.0), -1), (dict(scale=math.nan), -1),
    (dict(scale=math.inf), -1), (dict(stride=999), -1), (dict(targets_stride=1), -1), (dict(logprobs_stride=1), -1),
    (dict(top_ids_stride=4), -1), (dict(top_logprobs_stride=4), -1), (dict(logits=None), -1), (dict(targets=None), -1),
    (dict(logprobs=None), -1), (dict(top_ids=None), -1), (dict(top_logprobs=None), -1),
    (dict(given=0, top=0, lse=None, entropy=None), -1), (dict(logits=FAKE + 1), -1), (dict(logits=FAKE + 2, dtype=2), -1),
    (dict(targets=FAKE + 2), -1), (dict(logprobs=FAKE + 1), -1), (dict(lse=FAKE + 2), -1), (dict(entropy=FAKE + 2), -1),
    (dict(top_ids=FAKE + 2), -1), (dict(top_logprobs=FAKE + 2), -1)])
def test_logprobs_refusals(L, kw, code):
    assert _logprobs(L, **kw) == code and "token_logprobs" in pw.pw_last_error()
    assert L.pw_token_logprobs(None, None) == -1


def test_empty_calls_touch_nothing(L):
    assert _norms(L, rows=0, x=None, residual=None, y=None, residual_out=None, q=None, scale=None) == 0
    assert _logprobs(L, rows=0, logits=None, targets=None, logprobs=None, lse=None, entropy=None, top_ids=None) == 0


def test_binding_checks():
    x = torch.zeros(4, 64, dtype=torch.float16)
    with pytest.raises(ValueError):          # not on the GPU
        pw.pw_norm_add_norm(x, x, 1e-5, residual_out=x)
    with pytest.raises(ValueError):          # fp32
        pw.pw_norm_add_norm(x.float(), x, 1e-5, residual_out=x)
    with pytest.raises(ValueError):
        pw.pw_token_logprobs(x, lse=torch.zeros(4))
    with pytest.raises(ValueError):
        pw.pw_token_logprobs(x.double(), lse=torch.zeros(4))
    with pytest.raises(ValueError):          # one without the other
        pw.pw_token_logprobs(x, targets=torch.zeros(4, 1, dtype=torch.int32))


def test_oracle_attention_with_first_keys():
    from oracle import attn_half
    # equal scores: the mean of the visible values
    rng = np.random.default_rng(0)
    v = rng.standard_normal((4, 4, 1, 8))
    q, k = np.zeros((2, 2, 8)), rng.standard_normal((4, 4, 1, 8))
    table = np.array([[2, 0, 1, 3]])
    flat = v[[2, 0, 1, 3]].reshape(-1, 8)
    out, lse, _, _ = attn_half.attention(q, k, v, table, [0, 2], [15], 0.5, window=3, sinks=2)
    assert np.allclose(out[0, 0], flat[[0, 1, 11, 12, 13]].mean(0)) and np.allclose(out[1, 1], flat[[0, 1, 12, 13, 14]].mean(0))
    assert np.allclose(lse, math.log(5))
    # the first keys end where the token is, and where the window begins
    out, _, _, _ = attn_half.attention(q, k, v, table, [0, 2], [2], 0.5, window=1, sinks=5)
    assert np.allclose(out[0, 0], flat[0]) and np.allclose(out[1, 0], flat[:2].mean(0))


def _attention(L, **options):
    a = pw.pw_attn_args()
    for n in ("q", "out", "k_cache", "v_cache", "page_table", "q_offsets", "kv_lens", "status"):
        setattr(a, n, FAKE)
    a.tokens, a.batch, a.heads, a.kv_heads, a.head_dim = 0, 2, 4, 2, 128
    a.page_size, a.num_pages, a.pages_per_seq, a.page_table_stride = 16, 8, 4, 4
    a.max_q_len, a.max_kv_len, a.causal, a.scale, a.window = 2, 64, 1, 0.1, 8
    o = pw.pw_attn_options()
    reserved = options.pop("reserved", None)
    if reserved is not None:
        o.reserved[reserved] = 1
    for k, v in options.items():
        setattr(o, k, v)
    return L.pw_paged_attention_ex(ctypes.byref(a), ctypes.byref(o), FAKE, 1 << 30, None)


@pytest.mark.parametrize("kw", [dict(sinks=-1), dict(sinks=(1 << 30) + 1), dict(reserved=0), dict(reserved=6)])
def test_attention_option_refusals(L, kw):
    assert _attention(L, **kw) == pw.PW_ERR_INVALID_ARG and "paged_attention" in pw.pw_last_error()
    assert _attention(L, sinks=4) == 0                                   # no tokens
    assert L.pw_paged_attention_ex(None, None, FAKE, 1 << 30, None) == pw.PW_ERR_INVALID_ARG


def test_oracle_activations():
    g = np.linspace(-30, 30, 101)
    t = torch.from_numpy(g)
    v, _ = ref.activation(g, "silu")
    assert np.allclose(v, torch.nn.functional.silu(t).numpy(), rtol=1e-12)
    v, _ = ref.activation(g, "gelu_tanh")
    # (1 + tanh x cancels where x is far below 0: 2^-52 of g)
    assert np.allclose(v, torch.nn.functional.gelu(t, approximate="tanh").numpy(), rtol=1e-12, atol=1e-14)


def _gated(L, **kw):
    return _call(L.pw_fp8_gated_linear, pw.pw_gated_args, dict(
        a=FAKE, lda=256, a_scale=FAKE, a_scale_stride=2, gate=FAKE, ld_gate=256, gate_scale=FAKE, gate_scale_stride=2, up=FAKE,
        ld_up=256, up_scale=FAKE, up_scale_stride=2, m=4, n=128, k=256, dtype=0, y=FAKE, ldy=128, q=FAKE, ldq=128, scale=FAKE,
        scale_stride=1, status=FAKE), kw)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), -2), (dict(activation=2), -2), (dict(activation=-1), -2), (dict(m=-1), -1), (dict(n=0), -1), (dict(k=0), -1),
    (dict(m=(1 << 20) + 1), -2), (dict(lda=240), -1), (dict(ld_gate=240), -1), (dict(ld_up=240), -1), (dict(ldy=127), -1),
    (dict(ldq=127), -1), (dict(scale_stride=0), -1), (dict(a_scale_stride=1), -1), (dict(gate_scale_stride=1), -1),
    (dict(up_scale_stride=1), -1), (dict(a=None), -1), (dict(a_scale=None), -1), (dict(gate=None), -1), (dict(gate_scale=None), -1),
    (dict(up=None), -1), (dict(up_scale=None), -1), (dict(status=None), -1), (dict(q=None), -1), (dict(scale=None), -1),
    (dict(y=None, q=None, scale=None), -1), (dict(a=FAKE + 8), -1), (dict(gate=FAKE + 8), -1), (dict(up=FAKE + 4), -1),
    (dict(lda=264), -1), (dict(ld_gate=257), -1), (dict(ld_up=264), -1), (dict(a_scale=FAKE + 1), -1), (dict(scale=FAKE + 2), -1),
    (dict(y=FAKE + 1), -1), (dict(status=FAKE + 2), -1), (dict(ld_up=1 << 39), -2), (dict(ldy=1 << 40), -2)])
def test_gated_refusals(L, kw, code):
    assert _gated(L, **kw) == code and "fp8_gated_linear" in pw.pw_last_error()
    assert L.pw_fp8_gated_linear(None, None) == -1
    assert _gated(L, m=0, a=None, y=None, q=None, scale=None, status=None) == 0


def test_logprobs_scales(L):
    """The sums run in powers of two: scale * log2(e) has to be finite."""
    assert _logprobs(L, scale=3e38) == -1 and "scale" in pw.pw_last_error()
    assert _logprobs(L, scale=2.0 ** 127, rows=0) == 0
