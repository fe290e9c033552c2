"""GPU: log probabilities of many rows of short or middle vocabularies, which run in CTAs of 128 threads:
what tests/test_gpu_logprobs.py asks of few rows, with its tolerances (a thread has 32 vectors at most)."""
import math

import numpy as np
import pytest
import torch

from test_gpu_attn_half import DEV, _gpu, f64, gen, pw, within  # noqa: F401
from test_gpu_large_paths import launched, sms
from test_gpu_logprobs import DTYPES, IDS, call, check, make, same
from oracle import more_ops as ref

pytestmark = pytest.mark.gpu
ROWS = 700


def some(rows):
    """Rows of each address in a vector, and the last ones."""
    return list(range(min(rows, 33))) + [rows // 2, rows - 2, rows - 1]


def check_some(z, targets, top, scale, out):
    pick = some(z.shape[0])
    check(z[pick], targets[pick], top, scale, {k: v[pick] for k, v in out.items()})


@pytest.fixture(autouse=True)
def _many_rows():
    if ROWS <= 4 * sms():
        pytest.skip("the rule counts SMs")


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_the_kernel(dtype):
    z, targets = make(ROWS, 3000, dtype, 1)
    assert launched(lambda: call(z, targets, 20), "logprobs_kernel", 128)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("rows,vocab,top", [
    (700, 1, 1), (700, 5, 5), (900, 31, 20), (700, 33, 32), (3001, 128, 32), (700, 257, 20), (700, 1000, 1), (700, 2049, 32),
    (1000, 4095, 20), (700, 8191, 5), (620, 20011, 32), (700, 32750, 20), (700, 1500, 0)])
def test_sizes(rows, vocab, top, dtype):
    """From rows of fewer vectors than alternatives to the longest; rows at every address of a vector (odd strides)."""
    for i, (pad, offset, step, scale) in enumerate([(0, 0, 0.0, 1.0), (2 - vocab % 2, 1, 0.5, 1.25)]):
        z, targets = make(rows, vocab, dtype, rows + vocab + i, pad, offset, step)
        out = call(z, targets, top, scale)
        if not top:
            out.update(top_ids=torch.zeros(rows, 0, dtype=torch.int32, device=DEV), top_logprobs=torch.zeros(rows, 0, device=DEV))
        check_some(z, targets, top, scale, out)


@pytest.mark.parametrize("offset", range(16))
def test_addresses(offset):
    """Every row starts at the same place of a vector; its neighbours are NaN."""
    for dtype in DTYPES:
        z, targets = make(ROWS, 320 + offset, dtype, offset, pad=32 - (320 + offset) % 16, offset=offset)
        check_some(z, targets, 20, 1.0, call(z, targets, 20))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "zeros", "blocks"])
@pytest.mark.parametrize("vocab", [40, 1999, 30011])
def test_orders(vocab, kind, dtype):
    """Ties everywhere and sorted rows: the order is that of (value, lowest id)."""
    i = torch.arange(vocab, device=DEV, dtype=torch.float32)
    z = {"equal": i * 0 + 2, "rising": (i / 16).floor() / 256, "falling": -(i / 16).floor() / 256,
         "zeros": torch.where(i % 2 == 0, 0.0, -0.0), "blocks": (i / 1024).floor() % 5}[kind].to(dtype)
    z = z.expand(ROWS, vocab).contiguous()
    targets = torch.tensor([[0, vocab - 1]], dtype=torch.int32, device=DEV).expand(ROWS, 2).contiguous()
    for top in (1, 20, 32):
        out = call(z, targets, top)
        check_some(z, targets, top, 1.0, out)
        assert (out["top_ids"] == out["top_ids"][:1]).all()


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("vocab", [40, 900, 20001])
def test_masked_rows(vocab, dtype):
    """-inf for most tokens, for all but a few (fewer than alternatives), for all; the type's lowest value."""
    z, targets = make(ROWS, vocab, dtype, 5)
    z[0, torch.rand(vocab, generator=gen(1)).to(DEV) < 0.9] = -math.inf
    z[0, 3] = 1
    z[1] = -math.inf
    z[2] = -math.inf
    z[2, 37] = -4
    z[3, :-3] = -math.inf
    z[4, 10:] = -math.inf
    z[-1] = -math.inf
    z[-1, 5] = 2
    targets[2, 2] = 37
    for top in (1, 20, 32):
        out = call(z, targets, top)
        check_some(z, targets, top, 1.0, out)
        assert out["entropy"][1] == 0 and out["entropy"][2] == 0 and out["logprobs"][2, 2] == 0 and out["entropy"][-1] == 0
    z[:, 0::2] = torch.finfo(dtype).min
    z[-1] = torch.finfo(dtype).min
    z[-1, 5] = 1                                        # fewer unmasked tokens than alternatives
    z[1:5, 1::2] = 0
    out = call(z, targets, 32)
    pick = some(ROWS)
    lp, lse, h, ids, best = ref.token_logprobs(f64(z[pick]), targets[pick].cpu().numpy(), 32, 1.0)
    seen = f64(z[pick])
    big = 2.0 ** -18 + 2.0 ** -21 * 2 * (np.abs(np.where(np.abs(seen) < 1e3, seen, 0)).max() + 40)
    within(out["lse"][pick], lse, big)
    within(out["entropy"][pick], h, big + 2.0 ** -18 * h)
    for got, want in ((out["logprobs"][pick], lp), (out["top_logprobs"][pick], best)):
        assert np.isfinite(want).any()                  # (row 0 keeps tokens of -inf beside those of the lowest value)
        same(got, want, np.where(np.abs(want) > 1e3, 2.0 ** -22 * np.abs(want), big))
    assert np.array_equal(out["top_ids"][pick].cpu().numpy(), ids)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("vocab", [40, 3000, 20001])
@pytest.mark.parametrize("top", [3, 32])
def test_bad_rows(top, vocab, dtype):
    """NaN and +inf: their rows are NaN, other rows are not; ids in the logits' order, NaN last."""
    z, targets = make(ROWS, vocab, dtype, 9)
    z[1, vocab // 2] = float("nan")
    z[2, vocab - 1] = float("inf")
    z[3] = float("nan")
    z[-1, 0] = float("inf")
    out = call(z, targets, top)
    for r in (1, 2, 3, ROWS - 1):
        for k in ("lse", "entropy", "logprobs", "top_logprobs"):
            assert out[k][r].isnan().all(), (k, r)
    pick = some(ROWS)
    clean = torch.where(z[pick].isnan(), -math.inf, z[pick].double()).cpu().numpy()
    want = np.argsort(-clean, axis=1, kind="stable")[:, :top]
    assert np.array_equal(out["top_ids"][pick].cpu().numpy(), want)
    good = [r for r in pick if r not in (1, 2, 3, ROWS - 1)]
    check(z[good], targets[good], top, 1.0, {k: v[good] for k, v in out.items()})
    every = torch.ones(ROWS, dtype=torch.bool, device=DEV)
    every[[1, 2, 3, ROWS - 1]] = False
    assert all(out[k][every].isfinite().all() for k in ("lse", "entropy", "logprobs", "top_logprobs"))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_repeats_streams_and_graphs(dtype):
    z, targets = make(ROWS, 5001, dtype, 6)
    want = call(z, targets, 20)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = call(z, targets, 20)
    s.synchronize()
    assert all(torch.equal(want[k], got[k]) for k in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call(z, targets, 20)
    z.copy_(make(ROWS, 5001, dtype, 7)[0])
    graph.replay()
    want = call(z, targets, 20)
    assert all(torch.equal(want[k], got[k]) for k in want)
    check_some(z, targets, 20, 1.0, got)
