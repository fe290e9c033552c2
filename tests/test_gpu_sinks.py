"""GPU: attention with a window and the first keys of each sequence, against the
64-bit oracle.  Tolerances as for the attention without them."""
import numpy as np
import pytest
import torch

from oracle import attn_half as ref
from test_gpu_attn_half import (Batch, DEV, DTYPES, IDS, TINY, U, _gpu, attend, f64, pw, status, within)  # noqa: F401

pytestmark = pytest.mark.gpu


def check(b, out, lse, window, sinks):
    want, wl, mag, dots = ref.attention(f64(b.q), f64(b.k), f64(b.v), b.table.cpu().numpy(), b.offsets.tolist(), b.kv,
                                        b.d ** -0.5, True, window, sinks)
    u = U[b.dtype]
    ds = 2.0 ** -16 * dots
    within(out, want, u * np.abs(want) * 1.01 + (u + 2 * ds + 2.0 ** -16)[..., None] * mag + TINY[b.dtype])
    got, seen = f64(lse), np.isfinite(wl)
    assert np.array_equal(np.isneginf(got), ~seen)
    assert (np.abs(got[seen] - wl[seen]) <= ds[seen] + 2.0 ** -18 * (1 + np.abs(wl[seen]))).all()


def forget(b, window, sinks):
    """What no token of the call sees: pages given back, rows of the others NaN."""
    for i, (m, n) in enumerate(zip(b.q_lens, b.kv)):
        first = n - m - window + 1
        for j in range(-(-n // b.ps)):
            keys = range(j * b.ps, (j + 1) * b.ps)
            hidden = [k for k in keys if k >= n or (k < first and k >= sinks)]
            page = int(b.table[i, j])
            if len(hidden) == b.ps:
                b.table[i, j] = -1
            for t in (b.k, b.v):
                t[page, [k % b.ps for k in hidden]] = float("nan")


CASES = [  # q_lens, kv_lens, heads, kv_heads, d, page, heads_first, window, sinks
    ([1], [1], 1, 1, 64, 16, False, 1, 1),
    ([1], [300], 8, 2, 128, 16, False, 1, 1),
    ([1], [700], 8, 2, 128, 16, True, 33, 4),
    ([1, 1, 1, 1], [3, 64, 165, 700], 8, 2, 128, 16, False, 40, 4),
    ([1, 1], [900, 31], 16, 1, 64, 13, False, 100, 70),
    ([1] * 40, list(range(1, 41)), 4, 4, 64, 16, False, 7, 3),
    ([1, 1], [300, 300], 4, 1, 64, 16, True, 64, 64),          # whole blocks
    ([1, 1], [500, 200], 4, 1, 128, 16, False, 100, 400),      # more first keys than lie before the window
    ([1], [200], 4, 1, 128, 16, False, 50, 1 << 30),           # all of them
    ([4, 3, 2], [100, 3, 257], 6, 1, 128, 32, False, 20, 5),
    ([5, 0, 7], [5, 40, 300], 12, 4, 64, 64, True, 64, 65),
    ([50, 10], [400, 10], 4, 2, 64, 16, True, 17, 4),
    ([100], [900], 2, 1, 128, 64, False, 130, 1),
    ([100], [900], 2, 1, 128, 64, False, 130, 127),
    ([100], [900], 2, 1, 128, 64, False, 130, 128),
    ([100], [900], 2, 1, 64, 64, True, 130, 129),
    ([100, 40], [900, 700], 2, 1, 128, 32, False, 60, 300),
    ([130, 33], [130, 590], 4, 1, 128, 8, True, 20, 40),
    ([200], [64], 4, 4, 128, 32, True, 9, 3),                  # rows that see nothing
    ([10, 3], [4, 0], 4, 2, 128, 16, False, 2, 2),
    ([37], [450], 4, 4, 128, 48, False, 60, 50),               # pages that end inside a block
    ([300], [1000], 1, 1, 128, 16, False, 1, 2),               # several tiles
    ([1, 1], [20000, 9000], 4, 1, 64, 32, False, 5000, 200),   # pieces of a unit
    ([70], [9000], 4, 1, 128, 32, False, 3000, 513),
]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("case", range(len(CASES)))
def test_window_and_first_keys(case, dtype):
    ql, kl, h, hk, d, ps, hf, window, sinks = CASES[case]
    b = Batch(ql, kl, h, hk, d, ps, dtype, 300 + case, hf)
    every = attend(b, window=window, sinks=sinks)
    assert every[2] == 0
    check(b, every[0], every[1], window, sinks)
    # with nothing but what the tokens see: the same bits
    forget(b, window, sinks)
    out, lse, st = attend(b, window=window, sinks=sinks)
    assert st == 0 and torch.equal(out, every[0]) and torch.equal(lse, every[1])


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_every_kernel_for_the_same_batch(dtype):
    """The length bounds only choose the kernel and the grid."""
    b = Batch([1, 12, 70], [300, 12, 460], 8, 2, 128, 16, dtype, 3)
    forget(b, 90, 30)
    for mq in (1, 8, 64, 1000):
        for mk in (1, 300, 100000):
            out, lse, st = attend(b, max_q_len=mq, max_kv_len=mk, window=90, sinks=30)
            assert st == 0
            check(b, out, lse, 90, 30)


def test_without_a_window_they_change_nothing():
    for ql in (1, 40):
        b = Batch([ql], [500], 4, 2, 128, 16, torch.float16, 6)
        want = attend(b)
        got = attend(b, sinks=4)
        assert got[2] == 0 and torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        # a window that reaches the first key is no window
        got = attend(b, sinks=4, window=500)
        check(b, got[0], got[1], 0, 0)


def test_missing_pages_are_reported():
    for ql in (1, 60):
        for page, window in ((0, 100), (1, 100), (31, 20)):
            b = Batch([ql], [500], 4, 2, 128, 16, torch.float16, 6)
            b.table[0, page] = -1
            assert attend(b, window=window, sinks=20)[2] == pw.PW_ERR_NOT_RESIDENT
            b.table[0, page] = 1 << 30
            assert attend(b, window=window, sinks=20)[2] == pw.PW_ERR_NOT_RESIDENT


def test_workspace_stream_and_graph():
    """One workspace with and without first keys in turn; another stream; a replayed graph."""
    ws = torch.zeros(pw.pw_paged_attention_workspace(400, 64, 8, 2, 128), dtype=torch.uint8, device=DEV)
    batches = [Batch([1], [5000], 8, 2, 128, 16, torch.float16, 1), Batch([100, 1], [900, 999], 8, 2, 128, 16, torch.float16, 2)]
    first = {}
    for rep in range(2):
        for i, b in enumerate(batches):
            for sinks in (0, 5):
                out, lse, st = attend(b, ws, window=200, sinks=sinks)
                assert st == 0
                assert rep == 0 or (torch.equal(out, first[i, sinks][0]) and torch.equal(lse, first[i, sinks][1]))
                first.setdefault((i, sinks), (out, lse))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        out, lse, st = attend(batches[0], ws, window=200, sinks=5)
    s.synchronize()
    assert st == 0 and torch.equal(out, first[0, 5][0])
    b = batches[1]
    out, st, graph = torch.empty_like(b.q), status(), torch.cuda.CUDAGraph()
    call = lambda: pw.pw_paged_attention(b.q, b.k, b.v, b.table, b.offsets, b.lens, out, ws, st, scale=b.d ** -0.5,  # noqa: E731
                                         window=200, sinks=5, max_q_len=100, max_kv_len=999)
    with torch.cuda.graph(graph):
        call()
    b.q.mul_(0.5)
    graph.replay()
    got = out.clone()
    call()
    assert torch.equal(out, got) and int(st.item()) == 0


def test_refusals():
    b = Batch([1], [50], 4, 2, 64, 16, torch.float16, 1)
    for kw in (dict(sinks=-1, window=5), dict(sinks=(1 << 30) + 1, window=5), dict(sinks=4, window=5, causal=False)):
        with pytest.raises(pw.PwError):
            attend(b, **kw)
