"""GPU: the gated feed-forward block in e4m3 against the 64-bit oracle.

Tolerances: both projections as the 8-bit product (the tensor cores add the exact
products of a group with at least 13 bits below the largest of them): dg, du =
2^-13 of the terms' magnitudes; an activation's slope is at most 1.13; the
exponential's argument t is off by 2^-22 |t|, it and the quotient by 2^-20; one
rounding to 16 bits, or half a step of e4m3 with the scale's 2^-22."""
import numpy as np
import pytest
import torch

from oracle import attn_half as ref
from oracle import more_ops
from test_gpu_attn_half import DEV, DTYPES, IDS, TINY, U, _gpu, f64, gen, pw, status, within  # noqa: F401

pytestmark = pytest.mark.gpu
ACTS = {"silu": 0, "gelu_tanh": 1}


def problem(m, n, k, seed=0, pad=None):
    g = gen(m * 7919 + n * 131 + k + seed)
    kb, nb, pad = -(-k // 128), -(-n // 128), -k % 16 if pad is None else pad

    def codes(rows):
        t = (torch.randn(rows, k + pad, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn)
        t[:, k:] = float("nan")                    # past the columns: anything
        return t.to(DEV)[:, :k]
    a, gate, up = codes(m), codes(n), codes(n)
    s = 1 / 60 / k ** 0.5                          # projections of about 1
    sa = torch.exp(torch.randn(m, kb, generator=g)).to(DEV) / 60
    sg, su = (s * torch.exp(0.5 * torch.randn(nb, kb, generator=g)).to(DEV) for _ in range(2))
    return a, sa, gate, sg, up, su


def oracle(a, sa, gate, sg, up, su, act):
    """(h, what it may be off by before it is rounded)"""
    num = lambda t: t.contiguous().view(torch.uint8).cpu().numpy()  # noqa: E731
    g, mg = ref.fp8_linear(num(a), f64(sa), num(gate), f64(sg))
    u, mu = ref.fp8_linear(num(a), f64(sa), num(up), f64(su))
    v, t = more_ops.activation(g, act)
    dg, du = 2.0 ** -13 * mg, 2.0 ** -13 * mu
    return v * u, 1.13 * dg * (np.abs(u) + du) + np.abs(v) * du + (2.0 ** -20 + 2.0 ** -22 * t) * np.abs(v * u)


def check_codes(q, sc, h, off):
    rows, cols = h.shape
    top = np.stack([np.abs(h[:, c:c + 128]).max(1) for c in range(0, cols, 128)], 1)
    slack = np.stack([off[:, c:c + 128].max(1) for c in range(0, cols, 128)], 1)
    within(sc, np.maximum(top / 448, 2.0 ** -100), (slack + top * 2.0 ** -22) / 448)
    s = np.repeat(f64(sc), 128, 1)[:, :cols]
    step = 2.0 ** (np.floor(np.log2(np.maximum(np.abs(h / s), 2.0 ** -6))) - 3)
    # near a border of two steps the larger one counts
    within(q.double(), h / s, 0.5 * np.maximum(step, 2.0 ** (np.floor(np.log2(np.maximum((np.abs(h) + off) / s, 2.0 ** -6))) - 3))
           + off / s + np.abs(h / s) * 2.0 ** -22)


def run(m, n, k, dtype, act, y_pad=3, q_pad=None, seed=0, strides=None):
    args = problem(m, n, k, seed)
    if strides:
        args = strides(args)
    h, off = oracle(*args, act)
    u = U[dtype]
    st = status()
    q_pad = -n % 16 if q_pad is None else q_pad
    y = torch.full((m, n + y_pad), 7.0, dtype=dtype, device=DEV)
    q = torch.full((m, n + q_pad), 9, dtype=torch.uint8, device=DEV)
    sc = torch.full((m, -(-n // 128) + 2), 5.0, device=DEV)
    codes = q.view(torch.float8_e4m3fn)[:, :n]
    nb = -(-n // 128)
    pw.pw_fp8_gated_linear(*args, st, y=y[:, :n], q=codes, scale=sc[:, :nb], activation=ACTS[act])
    assert int(st.item()) == 0
    within(y[:, :n], h, u * np.abs(h) * 1.01 + off * 1.01 + TINY[dtype])
    check_codes(codes, sc[:, :nb], h, off)
    assert (y[:, n:] == 7).all() and (q[:, n:] == 9).all() and (sc[:, nb:] == 5).all()
    # one output alone (other tiles may add in another order)
    y2, q2, sc2 = torch.zeros_like(y), torch.zeros_like(q), torch.zeros_like(sc)
    pw.pw_fp8_gated_linear(*args, st, y=y2[:, :n], activation=ACTS[act])
    pw.pw_fp8_gated_linear(*args, st, q=q2[:, :n], scale=sc2[:, :nb], activation=ACTS[act])
    within(y2[:, :n], h, u * np.abs(h) * 1.01 + off * 1.01 + TINY[dtype])
    check_codes(q2.view(torch.float8_e4m3fn)[:, :n], sc2[:, :nb], h, off)
    assert int(st.item()) == 0 and (y2[:, n:] == 0).all() and (q2[:, n:] == 0).all()


SIZES = [(1, 1, 16), (1, 128, 128), (3, 17, 130), (7, 200, 100), (8, 1000, 512), (8, 130, 2064), (9, 128, 1000), (16, 64, 2048),
         (17, 130, 256), (33, 129, 384), (64, 384, 144), (50, 300, 2100), (65, 1, 640), (100, 300, 1024), (128, 256, 128),
         (129, 513, 257), (200, 640, 4096), (257, 128, 16), (300, 1030, 900), (512, 512, 512), (1000, 260, 2000), (5, 4096, 256),
         (60, 2048, 1024), (100, 1408, 2048)]


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("m,n,k", SIZES)
def test_gated(m, n, k, dtype):
    run(m, n, k, dtype, "silu" if (m + n) % 2 else "gelu_tanh")


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k", [(2, 300, 512), (30, 300, 512), (100, 300, 512), (600, 4000, 512), (2400, 2000, 256),
                                   (1300, 3000, 384)])
def test_every_kernel(m, n, k, act):
    """Single tokens, 64- and 128-token tiles, pairs of CTAs with several tiles each."""
    run(m, n, k, torch.bfloat16, act, y_pad=8 - n % 8)


@pytest.mark.parametrize("m", [1, 6, 40, 100, 700])
@pytest.mark.parametrize("n,y_pad,q_pad", [(100, 4, 12), (129, 7, 15), (4, 4, 4), (255, 1, 0), (190, 66, 2), (64, 8, 64), (130, 1, 1),
                                           (2045, 3, 3)])
def test_nothing_beside_the_columns(m, n, y_pad, q_pad):
    run(m, n, 400, torch.bfloat16, "silu", y_pad, q_pad)


@pytest.mark.parametrize("m", [3, 40, 100, 300])
def test_strides_and_halves_of_one_matrix(m):
    """Both weights out of one matrix; scales at odd strides; rows at 16-byte addresses only."""
    n, k = 256, 700

    def halves(args):
        a, sa, gate, sg, up, su = args
        w = torch.cat((gate.view(torch.uint8), up.view(torch.uint8)))
        both = torch.zeros(2 * n, 720, dtype=torch.uint8, device=DEV)[:, :k]
        both.copy_(w)
        both = both.view(torch.float8_e4m3fn)
        s = torch.cat((sg, su))
        return a, sa, both[:n], s[:2], both[n:], s[2:]
    run(m, n, k, torch.float16, "silu", strides=halves)

    def odd(args):
        def wide(s):
            t = torch.full((s.shape[0], s.shape[1] + 3), 1e30, device=DEV)[:, 1:-2]
            t.copy_(s)
            return t

        def shifted(c):
            t = torch.zeros(c.shape[0] * 736 + 16, dtype=torch.uint8, device=DEV)[16:].view(-1, 736)[:, :k]
            t.copy_(c.view(torch.uint8))
            return t.view(torch.float8_e4m3fn)
        a, sa, gate, sg, up, su = args
        return shifted(a), wide(sa), shifted(gate), wide(sg), shifted(up), wide(su)
    run(m, n, k, torch.float16, "gelu_tanh", strides=odd)


def test_extremes():
    """Gates far on both sides, zeros, and NaN: its row's group is NaN, others are not."""
    for m in (4, 40, 100, 300):
        n, k = 256, 128
        a = torch.zeros(m, k, device=DEV)
        a[:, 0] = 1
        gate, up = torch.zeros(n, k, device=DEV), torch.zeros(n, k, device=DEV)
        gate[:, 0] = torch.linspace(-448, 448, n, device=DEV)
        up[:, 0] = 1
        a[1] = 0
        a[2, 1] = float("nan")
        f8 = lambda t: t.to(torch.float8_e4m3fn)  # noqa: E731
        one = lambda r, c: torch.ones(r, c, device=DEV)  # noqa: E731
        for act in ACTS:
            st, y = status(), torch.empty(m, n, dtype=torch.bfloat16, device=DEV)
            q, sc = torch.empty(m, n, dtype=torch.uint8, device=DEV), torch.empty(m, 2, device=DEV)
            pw.pw_fp8_gated_linear(f8(a), one(m, 1), f8(gate), one(2, 1), f8(up), one(2, 1), st, y=y,
                                   q=q.view(torch.float8_e4m3fn), scale=sc, activation=ACTS[act])
            g = f64(f8(gate)[:, 0])
            v, t = more_ops.activation(g, act)
            # (a quotient by a number above 2^126 is 0: |g| 2^-126 is lost at most, |g| <= 448)
            within(y[0], v, U[torch.bfloat16] * np.abs(v) * 1.01 + (2.0 ** -20 + 2.0 ** -22 * t) * np.abs(v) + 448 * 2.0 ** -126)
            assert (y[1] == 0).all() and (q[1] & 127 == 0).all() and (sc[1] == 2.0 ** -100).all()
            assert y[2].isnan().all() and sc[2].isnan().all() and y[3:].isfinite().all() and sc[3:].isfinite().all()
            assert torch.equal(y[3], y[0]) and torch.equal(q[3], q[0]) and int(st.item()) == 0


def test_stream_graph_and_repeats():
    for m in (5, 50, 500):
        args, st = problem(m, 1024, 1024), status()
        new = lambda: (torch.empty(m, 1024, dtype=torch.float16, device=DEV),  # noqa: E731
                       torch.empty(m, 1024, dtype=torch.uint8, device=DEV), torch.empty(m, 8, device=DEV))

        def call(out, stream=None):
            pw.pw_fp8_gated_linear(*args, st, y=out[0], q=out[1].view(torch.float8_e4m3fn), scale=out[2], stream=stream)
        want, got = new(), new()
        call(want)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        for _ in range(3):
            call(got, s)
        s.synchronize()
        assert all(torch.equal(x, z) for x, z in zip(want, got))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call(got)
        args[0].copy_(problem(m, 1024, 1024, 1)[0])
        graph.replay()
        call(want)
        assert all(torch.equal(x, z) for x, z in zip(want, got)) and int(st.item()) == 0


def test_the_block_with_its_down_projection():
    """h in 8 bits is what the 8-bit product reads: the whole feed-forward block."""
    for m in (3, 200):
        H, n = 384, 640
        a, sa, gate, sg, up, su = problem(m, n, H)
        down = (torch.randn(H, n, generator=gen(4)) * 60).clamp(-448, 448).to(torch.float8_e4m3fn).to(DEV)
        sd = torch.full((3, 5), 1 / 60 / n ** 0.5, device=DEV)
        st, y = status(), torch.empty(m, H, dtype=torch.bfloat16, device=DEV)
        q, sc = torch.empty(m, n, dtype=torch.float8_e4m3fn, device=DEV), torch.empty(m, 5, device=DEV)
        pw.pw_fp8_gated_linear(a, sa, gate, sg, up, su, st, q=q, scale=sc)
        pw.pw_fp8_linear(q, sc, down, sd, y, st)
        h, off = oracle(a, sa, gate, sg, up, su, "silu")
        num = lambda t: t.view(torch.uint8).cpu().numpy()  # noqa: E731
        W = ref.e4m3_decode(num(down)) * ref.spread(f64(sd), (H, n), 128)
        # each value of h is off by half a step of its group's largest magnitude / 448 at most: 2^-4 of itself, or
        # of the smallest normal number, 2^-6
        s = np.repeat(f64(sc), 128, 1)[:, :n]
        dh = 2.0 ** -4 * np.maximum(np.abs(h) + off, 2.0 ** -6 * s) * 1.01 + off
        want = h @ W.T
        bound = dh @ np.abs(W).T + 2.0 ** -13 * (np.abs(h) + dh) @ np.abs(W).T
        within(y, want, bound * 1.01 + U[torch.bfloat16] * (np.abs(want) + bound) * 1.01)
        assert int(st.item()) == 0


def test_refusals():
    a, sa, gate, sg, up, su = problem(4, 256, 256)
    st, y = status(), torch.empty(4, 256, dtype=torch.float16, device=DEV)
    q, sc = torch.empty(4, 256, dtype=torch.uint8, device=DEV), torch.empty(4, 2, device=DEV)
    good = dict(a=a, a_scale=sa, gate=gate, gate_scale=sg, up=up, up_scale=su, status=st)
    for bad in (dict(), dict(y=y[:, :128]), dict(y=y.float()), dict(q=q), dict(scale=sc, y=y), dict(q=q, scale=sc[:, :1]),
                dict(y=y, up=up[:128]), dict(y=y, gate_scale=sg[:1]), dict(y=y, activation=2), dict(y=y, a=a[:, :255]),
                dict(y=y, status=st.cpu()), dict(y=y, a_scale=sa.half()), dict(y=y, gate=gate.float())):
        with pytest.raises((ValueError, pw.PwError)):
            pw.pw_fp8_gated_linear(**{**good, **bad})
    pw.pw_fp8_gated_linear(**{**good, "a": a[:0], "a_scale": sa[:0]}, y=y[:0])
