"""GPU: log probabilities of given tokens, entropy and alternatives, against the
64-bit oracle.

Tolerances: differences of logits and their product by scale * log2(e) are rounded
(2^-23 of |z| and of the largest |z| at most), the exponentials carry 2^-22, the sums of positive terms 2^-24 a term in a
thread (at most 1024 / 2 of them, in pairs) and 2^-24 a join: relative errors of S and T
of at most 2^-14.9 in the worst case and, as roundings cancel, below 2^-19; the logarithms and
results round at 2^-23 of their size."""
import math

import numpy as np
import pytest
import torch

from oracle import more_ops as ref
from test_gpu_attn_half import DEV, _gpu, f64, gen, pw, within  # noqa: F401

pytestmark = pytest.mark.gpu
DTYPES = [torch.float16, torch.bfloat16, torch.float32]
IDS = ["fp16", "bf16", "fp32"]


def call(logits, targets=None, top=0, scale=1.0, stats=True, **kw):
    rows = logits.shape[0]
    out = dict(lse=torch.empty(rows, device=DEV), entropy=torch.empty(rows, device=DEV)) if stats else {}
    if targets is not None:
        out.update(logprobs=torch.empty(targets.shape, device=DEV))
    if top:
        out.update(top_ids=torch.empty(rows, top, dtype=torch.int32, device=DEV), top_logprobs=torch.empty(rows, top, device=DEV))
    pw.pw_token_logprobs(logits, targets=targets, scale=scale, **out, **kw)
    return out


def same(got, want, bound):
    got = f64(got)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isneginf(got), np.isneginf(want))
    ok = np.isfinite(want)
    within(got[ok], want[ok], np.broadcast_to(bound, want.shape)[ok])


def check(logits, targets, top, scale, out):
    z, t = f64(logits), targets.cpu().numpy()
    lp, lse, h, ids, best = ref.token_logprobs(z, t, top, scale)
    big = np.abs(np.where(np.isfinite(z), z, 0.0) * scale).max(axis=1) + np.abs(np.where(np.isfinite(lse), lse, 0.0))
    row = 2.0 ** -18 + 2.0 ** -21 * big
    same(out["lse"], lse, row)
    # T / S: its terms are off by as much as z, times at most the entropy's own size
    same(out["entropy"], h, row + 2.0 ** -18 * np.maximum(h, 0))
    if t.shape[1]:
        same(out["logprobs"], lp, row[:, None])
    if top:
        assert np.array_equal(out["top_ids"].cpu().numpy(), ids)
        same(out["top_logprobs"], best, row[:, None])


def make(rows, vocab, dtype, seed, pad=0, offset=0, step=0.0):
    g = gen(seed)
    z = torch.randn(rows, vocab, generator=g) * 3
    if step:
        z = (z / step).round() * step          # many equal values
    buf = torch.full((rows * (vocab + pad) + offset + 64,), float("nan"), dtype=dtype, device=DEV)
    v = buf[offset:offset + rows * (vocab + pad)].view(rows, vocab + pad)[:, :vocab]
    v.copy_(z)
    targets = torch.randint(0, vocab, (rows, 3), generator=g, dtype=torch.int32)
    targets[:, 1] = targets[:, 0]
    return v, targets.to(DEV)


SHAPES = [(1, 1, 1), (1, 2, 2), (3, 5, 5), (2, 31, 7), (4, 33, 32), (1, 257, 20), (2, 1000, 1), (5, 4095, 3), (3, 4096, 8),
          (1, 9001, 20), (2, 32000, 32), (40, 32000, 20), (80, 8191, 5), (160, 5000, 5), (700, 1500, 2), (7, 50257, 10),
          (1, 131072, 32), (3, 262143, 20), (320, 20011, 32)]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("rows,vocab,top", SHAPES)
def test_logprobs(rows, vocab, top, dtype):
    for i, (pad, offset, step, scale) in enumerate([(0, 0, 0.0, 1.0), (3, 1, 0.5, 1.25)]):
        z, targets = make(rows, vocab, dtype, rows + vocab + i, pad, offset, step)
        check(z, targets, top, scale, call(z, targets, top, scale))


@pytest.mark.parametrize("offset", range(16))
def test_addresses(offset):
    """A row that starts and ends anywhere in a vector; its neighbours are NaN."""
    for dtype in DTYPES:
        z, targets = make(2, 300 + offset, dtype, offset, pad=5, offset=offset)
        check(z, targets, 6, 1.0, call(z, targets, 6))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_masked_rows(dtype):
    """-inf for most tokens, for all but one, for all."""
    z, targets = make(6, 20000, dtype, 5)
    z[0, torch.rand(20000, generator=gen(1)).to(DEV) < 0.9] = -math.inf
    z[1] = -math.inf
    z[2] = -math.inf
    z[2, 777] = -4
    z[3, :19990] = -math.inf
    z[4, 10:] = -math.inf
    z[5] = torch.finfo(dtype).min if dtype is torch.float16 else -1e30
    z[5, 123] = 1
    targets[2, 2], targets[5, 2] = 777, 123
    for top in (1, 20):
        out = call(z, targets, top)
        check(z, targets, top, 1.0, out)
        assert out["entropy"][1] == 0 and out["entropy"][2] == 0 and out["logprobs"][2, 2] == 0


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "zeros", "blocks"])
@pytest.mark.parametrize("rows", [1, 400])
def test_orders(rows, kind, dtype):
    """Ties everywhere and sorted rows: the order is that of (value, lowest id)."""
    vocab = 30011
    i = torch.arange(vocab, device=DEV, dtype=torch.float32)
    z = {"equal": i * 0 + 2, "rising": (i / 16).floor() / 256, "falling": -(i / 16).floor() / 256,
         "zeros": torch.where(i % 2 == 0, 0.0, -0.0), "blocks": (i / 1024).floor() % 5}[kind].to(dtype)
    z = z.expand(rows, vocab).contiguous()
    targets = torch.tensor([[0, vocab - 1]], dtype=torch.int32, device=DEV).expand(rows, 2).contiguous()
    out = call(z, targets, 32)
    # (equal rows start at different places of a vector: their sums run in different orders)
    check(z, targets, 32, 1.0, out)
    assert (out["top_ids"] == out["top_ids"][:1]).all()


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("vocab", [5, 3000, 40000])
def test_bad_rows(vocab, dtype):
    """NaN and +inf: their rows are NaN, other rows are not; ids in the logits' order, NaN last."""
    z, targets = make(5, vocab, dtype, 9)
    z[1, vocab // 2] = float("nan")
    z[2, vocab - 1] = float("inf")
    z[3] = float("nan")
    out = call(z, targets, 3)
    for r in (1, 2, 3):
        for k in ("lse", "entropy", "logprobs", "top_logprobs"):
            assert out[k][r].isnan().all(), (k, r)
    clean = torch.where(z.isnan(), -math.inf, z.double()).cpu().numpy()
    want = np.argsort(-clean, axis=1, kind="stable")[:, :3]
    assert np.array_equal(out["top_ids"].cpu().numpy(), want)
    good = [0, 4]
    check(z[good], targets[good], 3, 1.0, {k: v[good] for k, v in out.items()})


def test_targets():
    """Ids outside the vocabulary are not followed; any number of them; rows of wider tensors."""
    z, _ = make(4, 1000, torch.bfloat16, 2)
    room = torch.full((4, 400), -7, dtype=torch.int32, device=DEV)
    t = room[:, 20:320]
    t.copy_(torch.randint(-3, 1003, (4, 300), generator=gen(3), dtype=torch.int32))
    t[0, :4] = torch.tensor([-2 ** 31, 2 ** 31 - 1, 1000, -1])
    lp = torch.full((4, 310), 5.0, device=DEV)
    pw.pw_token_logprobs(z, targets=t, logprobs=lp[:, :300])
    want = ref.token_logprobs(f64(z), t.cpu().numpy(), 1, 1.0)[0]
    same(lp[:, :300], want, 2.0 ** -16)
    assert (lp[:, 300:] == 5).all() and lp[0, 0] == 0 and lp[0, 1].isnan() and lp[0, 2].isnan() and lp[0, 3] == 0


@pytest.mark.parametrize("scale", [1e-4, 0.01, 0.7, 50.0, 1000.0])
def test_scales(scale):
    for dtype in (torch.float16, torch.float32):
        z, targets = make(3, 5000, dtype, 4)
        z[0, 17] = -math.inf
        z[1] *= 1000
        check(z, targets, 4, float(np.float32(scale)), call(z, targets, 4, scale))


def test_confident_rows():
    """Nearly all of the probability on one token: the entropy's terms do not cancel."""
    z = torch.zeros(3, 10000, device=DEV)
    z[0, 5], z[1, 9999], z[2, 0] = 20.0, 40.0, 60.0
    h = call(z)["entropy"]
    _, _, want, _, _ = ref.token_logprobs(f64(z), np.zeros((3, 0), dtype=int), 1, 1.0)
    # T / S has 2^-18 of its size.  S is 1 and a little: the other terms of the maximum's thread (10000 / 256 in two
    # sums: 20 at most) and 5 + 7 joins are added to a number between 1 and 2, each with an error of up to half of
    # its step of 2^-23, so ln S is off by up to 32 * 2^-24 = 2^-19.
    within(h, want, 2.0 ** -18 * want + 2.0 ** -19)


def test_each_output_alone_and_repeats():
    z, targets = make(9, 40001, torch.float16, 6)
    every = call(z, targets, 20)
    for _ in range(3):
        again = call(z, targets, 20)
        assert all(torch.equal(every[k], again[k]) for k in every)
    lse = torch.empty(9, device=DEV)
    pw.pw_token_logprobs(z, lse=lse)
    assert torch.equal(lse, every["lse"])
    assert torch.equal(call(z, targets, stats=False)["logprobs"], every["logprobs"])
    one = call(z, top=1, stats=False)
    assert torch.equal(one["top_ids"][:, 0], every["top_ids"][:, 0])
    # results in wider tensors
    ids, best = torch.full((9, 30), -9, dtype=torch.int32, device=DEV), torch.full((9, 33), 9.0, device=DEV)
    pw.pw_token_logprobs(z, top_ids=ids[:, :20], top_logprobs=best[:, :20])
    assert torch.equal(ids[:, :20], every["top_ids"]) and torch.equal(best[:, :20], every["top_logprobs"])
    assert (ids[:, 20:] == -9).all() and (best[:, 20:] == 9).all()


def test_stream_and_graph():
    z, targets = make(5, 30000, torch.bfloat16, 8)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out = call(z, targets, 5)
    s.synchronize()
    check(z, targets, 5, 1.0, out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(z, targets, 5)
    z.copy_(make(5, 30000, torch.bfloat16, 11)[0])
    graph.replay()
    check(z, targets, 5, 1.0, out)


def test_refusals():
    z = torch.zeros(4, 64, device=DEV)
    t, lp, lse = torch.zeros(4, 2, dtype=torch.int32, device=DEV), torch.zeros(4, 2, device=DEV), torch.zeros(4, device=DEV)
    ids, best = torch.zeros(4, 5, dtype=torch.int32, device=DEV), torch.zeros(4, 5, device=DEV)
    for bad in (dict(), dict(lse=lse[:3]), dict(lse=lse.half()), dict(targets=t.long(), logprobs=lp), dict(targets=t, logprobs=lp[:, :1]),
                dict(targets=t, logprobs=lp.cpu()), dict(top_ids=ids, top_logprobs=best[:, :4]), dict(lse=lse, scale=0.0),
                dict(lse=lse, scale=float("nan")),
                dict(top_ids=torch.zeros(4, 33, dtype=torch.int32, device=DEV), top_logprobs=torch.zeros(4, 33, device=DEV))):
        with pytest.raises((ValueError, pw.PwError)):
            pw.pw_token_logprobs(z, **bad)
    with pytest.raises(ValueError):
        pw.pw_token_logprobs(z.t(), lse=torch.zeros(64, device=DEV))
    pw.pw_token_logprobs(z[:0], lse=lse[:0])


@pytest.mark.parametrize("scale", [1.0, 0.5])
@pytest.mark.parametrize("rows,vocab", [(3, 40), (2, 5000), (1, 40000)])
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_masks_of_the_types_lowest_value(dtype, rows, vocab, scale):
    """Masked tokens have finite log probabilities, of the mask's size; the others
    do not notice them.  (A product and a sum round a masked token's: 2^-23.)"""
    lowest = torch.finfo(dtype).min
    z, _ = make(rows, vocab, dtype, 12)
    z[:, 0::2] = lowest
    z[-1, 33:] = lowest                       # fewer unmasked tokens than alternatives
    targets = torch.tensor([[0, 1, 2, 31]], dtype=torch.int32, device=DEV).repeat(rows, 1)
    out = call(z, targets, 32, scale)
    lp, lse, h, ids, best = ref.token_logprobs(f64(z), targets.cpu().numpy(), 32, scale)
    big = 2.0 ** -18 + 2.0 ** -21 * 2 * (np.abs(f64(z[:, 1::2][:, :16])).max() + 40)
    within(out["lse"], lse, big)
    within(out["entropy"], h, big + 2.0 ** -18 * h)
    for got, want in ((out["logprobs"], lp), (out["top_logprobs"], best)):
        assert np.isfinite(want).all()
        within(got, want, np.where(np.abs(want) > 1e3, 2.0 ** -22 * np.abs(want), big))
    assert np.array_equal(out["top_ids"].cpu().numpy(), ids)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_rows_of_nothing_but_the_lowest_value(dtype):
    z = torch.full((2, 1000), torch.finfo(dtype).min, dtype=dtype, device=DEV)
    out = call(z, torch.tensor([[7], [999]], dtype=torch.int32, device=DEV), 3)
    for name in ("logprobs", "top_logprobs"):
        within(out[name], np.full(out[name].shape, -math.log(1000)), 2.0 ** -18)
    within(out["entropy"], np.full(2, math.log(1000)), 2.0 ** -17)
    assert out["top_ids"].tolist() == [[0, 1, 2]] * 2 and torch.isfinite(out["lse"]).all()
