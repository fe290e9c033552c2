"""GPU: what only larger calls of the operators around the attention half reach (CTAs
with several tiles or rows, clusters, several segments of a row), replays of captured clusters,
tensors of another GPU, and the refusal of each missing tensor."""
import numpy as np
import pytest
import torch

from oracle import more_ops as ref
from test_gpu_attn_half import Batch, DEV, TINY, U, _gpu, draw, f64, gen, pw, status, within  # noqa: F401
from test_gpu_gated import oracle, problem, run
from test_gpu_large_paths import launched, sms
from test_gpu_logprobs import call, check, make
from test_gpu_norms import EPS, bound_y, check_q

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- the gated block
def gated(m, n, k, q=True):
    args, st = problem(m, n, k), status()
    out = dict(q=torch.empty(m, n + -n % 16, dtype=torch.float8_e4m3fn, device=DEV)[:, :n],
               scale=torch.empty(m, -(-n // 128), device=DEV)) if q else dict(y=torch.empty(m, n, dtype=torch.float16, device=DEV))
    f = lambda: pw.pw_fp8_gated_linear(*args, st, **out)  # noqa: E731
    f()
    return f


@pytest.mark.parametrize("m,n,k,q,kernel,numbers", [
    (5, 300, 400, True, "gated_stream_kernel", (1, 2, 8)), (5, 6000, 256, True, "gated_stream_kernel", (1, 4, 2)),
    (5, 6000, 256, False, "gated_stream_kernel", (1, 2, 8)), (13, 500, 300, True, "gated_stream_kernel", (2, 2, 8)),
    (27, 500, 300, False, "gated_stream_kernel", (4, 2, 8)), (27, 500, 300, True, "linear_tile_kernel", (64, 256)),
    (40, 20000, 256, True, "linear_tile_kernel", (64, 256)),         # more tiles than SMs
    (128, 300, 2048, True, "linear_tile_kernel", (64, 256)),         # 4 CTAs a tile
    (240, 1408, 4096, True, "linear_tile_kernel", (128, 256)),       # and of 128 tokens
    (1100, 4200, 256, True, "linear_tile_kernel", (128, 256)),
    (509, 1408, 700, False, "linear_tile_kernel", (128, 128)), (60, 700, 2048, False, "linear_tile_kernel", (128, 128)),
    (2000, 1500, 256, False, "linear_tile_kernel", (128, 128)),
    (2500, 1100, 256, True, "linear_tile_kernel", (256, 256))])
def test_every_kernel_of_the_gated_block(m, n, k, q, kernel, numbers):
    if sms() != 152:
        pytest.skip("the rules count SMs")
    assert launched(gated(m, n, k, q), kernel, *numbers)
    run(m, n, k, torch.bfloat16, "silu")


@pytest.mark.parametrize("m,n,k", [(1, 1, 1), (3, 5, 5), (9, 17, 33), (70, 3, 7), (300, 130, 1)])
def test_gated_with_few_columns(m, n, k):
    run(m, n, k, torch.float16, "gelu_tanh")


# ---------------------------------------------------------------- log probabilities
@pytest.mark.parametrize("rows,vocab,dtype", [(1, 131072, torch.float16), (30, 66001, torch.bfloat16), (70, 34000, torch.float32),
                                              (310, 140001, torch.bfloat16), (310, 70000, torch.float32)])
def test_clusters_and_segments(rows, vocab, dtype):
    """8, 4 and 2 CTAs a row, and four segments a thread; a captured call replays on other logits."""
    z, targets = make(rows, vocab, dtype, rows, pad=1)
    out = call(z, targets, 7)
    pick = sorted({0, rows // 2, rows - 1})
    check(z[pick], targets[pick], 7, 1.0, {k: v[pick] for k, v in out.items()})
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call(z, targets, 7)
    z.copy_(make(rows, vocab, dtype, rows + 1)[0])
    graph.replay()
    again = call(z, targets, 7)
    assert all(torch.equal(out[k], again[k]) for k in out)
    check(z[pick], targets[pick], 7, 1.0, {k: v[pick] for k, v in out.items()})


@pytest.mark.parametrize("rows", [1, 310])
def test_the_largest_values_in_one_place(rows):
    """All alternatives in one segment of a thread, in one vector, and at the row's ends."""
    vocab = 140000
    for places in (torch.arange(32) * 4096, torch.arange(32), vocab - 1 - torch.arange(32), 5000 + torch.arange(32) // 2 * 17):
        z = torch.randn(rows, vocab, generator=gen(1)).to(DEV)
        z[:, places.to(DEV)] = 20 + torch.randn(32, generator=gen(2)).to(DEV).round()
        z = z.half()
        targets = torch.zeros(rows, 1, dtype=torch.int32, device=DEV)
        out = call(z, targets, 32)
        pick = sorted({0, rows - 1})
        check(z[pick], targets[pick], 32, 1.0, {k: v[pick] for k, v in out.items()})


def test_rows_past_32_bits():
    """Offsets of more than 2^31 values: the last rows of a batch of logits, of norms and of a product's result."""
    rows, vocab = 17000, 131072
    z = torch.empty(rows, vocab, dtype=torch.bfloat16, device=DEV)
    z[0], z[-1] = draw(gen(1), 2, vocab, dtype=torch.bfloat16, scale=3)
    z[1:-1] = 0
    ids, best = torch.empty(rows, 3, dtype=torch.int32, device=DEV), torch.empty(rows, 3, device=DEV)
    lse = torch.empty(rows, device=DEV)
    pw.pw_token_logprobs(z, lse=lse, top_ids=ids, top_logprobs=best)
    _, wl, _, wi, wb = ref.token_logprobs(f64(z[[0, -1]]), np.zeros((2, 0), dtype=int), 3, 1.0)
    within(lse[[0, -1]], wl, 2.0 ** -16)
    within(best[[0, -1]], wb, 2.0 ** -16)
    assert np.array_equal(ids[[0, -1]].cpu().numpy(), wi) and (ids[1:-1] == torch.arange(3, device=DEV)).all()
    del z
    rows, cols = 70000, 32768
    x = torch.zeros(rows, cols, dtype=torch.float16, device=DEV)
    x[-1] = draw(gen(2), cols)
    one = torch.ones(cols, dtype=torch.float16, device=DEV)
    pw.pw_norm_add_norm(x, x, EPS, post_weight=one, residual_out=x)
    want, _, mag = ref.norm_add_norm(f64(draw(gen(2), cols))[None], f64(draw(gen(2), cols))[None], EPS, np.ones(cols))
    within(x[-1:], want, U[torch.float16] * np.abs(want) * 1.01 + 2.0 ** -17 * mag + TINY[torch.float16])
    assert (x[:-1] == 0).all()


# ---------------------------------------------------------------- norms
@pytest.mark.parametrize("rows,cols", [(400, 9001), (700, 16384), (330, 9008), (170, 16512), (160, 20001), (700, 33)])
def test_norms_of_several_rows_a_cta(rows, cols):
    g = gen(cols)
    x, res, gate = (draw(g, rows, cols, dtype=torch.bfloat16) for _ in range(3))
    post, w = (draw(g, cols, dtype=torch.bfloat16) for _ in range(2))
    y, ro, sc = torch.empty_like(x), torch.empty_like(x), torch.empty(rows, -(-cols // 128), device=DEV)
    q = torch.empty(rows, cols, dtype=torch.float8_e4m3fn, device=DEV)
    for gt in (gate, gate[0]):
        pw.pw_norm_add_norm(x, res, EPS, post_weight=post, weight=w, gate=gt, residual_out=ro, y=y, q=q, scale=sc)
        r, want, mag = ref.norm_add_norm(f64(x), f64(res), EPS, f64(post), f64(w), f64(gt))
        u, tiny = U[torch.bfloat16], TINY[torch.bfloat16]
        within(ro, r, u * np.abs(r) * 1.01 + 2.0 ** -17 * mag + tiny)
        within(y, want, bound_y(u, tiny, r, want, mag, f64(w)))
        check_q(q, sc, r, want, mag, f64(w))


def test_an_expanded_gate_is_one_row():
    g = gen(3)
    x, res, gate = draw(g, 9, 512), draw(g, 9, 512), draw(g, 1, 512)
    a, b = torch.empty_like(x), torch.empty_like(x)
    pw.pw_norm_add_norm(x, res, EPS, gate=gate.expand(9, 512), residual_out=a)
    pw.pw_norm_add_norm(x, res, EPS, gate=gate[0], residual_out=b)
    assert torch.equal(a, b)


# ---------------------------------------------------------------- tensors and devices
def calls():
    """(call, its tensors by name, other arguments); outputs hold 7."""
    half = lambda *s: torch.full(s, 7.0, dtype=torch.float16, device=DEV)  # noqa: E731
    f32 = lambda *s: torch.full(s, 7.0, device=DEV)  # noqa: E731
    code = lambda *s: torch.full(s, 7, dtype=torch.uint8, device=DEV)  # noqa: E731
    i32 = lambda *s: torch.full(s, 7, dtype=torch.int32, device=DEV)  # noqa: E731
    yield pw.pw_norm_add_norm, dict(x=half(3, 64), residual=half(3, 64), post_weight=half(64), weight=half(64), gate=half(3, 64),
                                    residual_out=half(3, 64), y=half(3, 64), q=code(3, 64), scale=f32(3, 1)), dict(eps=1e-5)
    yield pw.pw_fp8_gated_linear, dict(a=code(3, 64), a_scale=f32(3, 1), gate=code(5, 64), gate_scale=f32(1, 1), up=code(5, 64),
                                       up_scale=f32(1, 1), y=half(3, 5), q=code(3, 5), scale=f32(3, 1), status=i32(1)), {}
    yield pw.pw_token_logprobs, dict(logits=half(3, 100), targets=i32(3, 2), logprobs=f32(3, 2), lse=f32(3), entropy=f32(3),
                                     top_ids=i32(3, 5), top_logprobs=f32(3, 5)), {}
    b = Batch([2], [20], 2, 1, 64, 16, torch.float16, 1)
    ws = torch.zeros(pw.pw_paged_attention_workspace(2, 1, 2, 1, 64), dtype=torch.uint8, device=DEV)
    yield pw.pw_paged_attention, dict(q=half(2, 2, 64), k_cache=half(*b.k.shape), v_cache=half(*b.v.shape), page_table=b.table,
                                      q_offsets=b.offsets, kv_lens=b.lens, out=half(2, 2, 64), ws=ws, status=i32(1),
                                      lse=f32(2, 2)), dict(scale=0.1, window=5, sinks=2)


def test_another_gpus_tensors_are_refused(monkeypatch):
    before = torch._C._cuda_getDevice()
    for f, tensors, kw in calls():
        kept = {n: t.clone() for n, t in tensors.items()}
        monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: before + 1)
        with pytest.raises(ValueError, match="current device"):
            f(**tensors, **kw)
        monkeypatch.undo()
        torch.cuda.synchronize()
        assert all(torch.equal(t, kept[n]) for n, t in tensors.items())


def test_each_tensor_has_to_be_there():
    for f, tensors, kw in calls():
        for name in tensors:
            with pytest.raises(ValueError):
                f(**{**tensors, name: tensors[name].cpu()}, **kw)
        f(**tensors, **kw)
    torch.cuda.synchronize()


def test_two_streams_at_once():
    """Calls that overlap share nothing but their inputs."""
    args, st = problem(100, 1408, 1024), status()
    z, targets = make(40, 50001, torch.bfloat16, 3)
    g = gen(8)
    x, res, w = draw(g, 300, 2048), draw(g, 300, 2048), draw(g, 2048)

    def all_three():
        q, sc = torch.empty(100, 1408, dtype=torch.float8_e4m3fn, device=DEV), torch.empty(100, 11, device=DEV)
        y = torch.empty_like(x)
        pw.pw_fp8_gated_linear(*args, st, q=q, scale=sc)
        out = call(z, targets, 9)
        pw.pw_norm_add_norm(x, res, EPS, post_weight=w, weight=w, y=y)
        return [q.view(torch.uint8), sc, y, *out.values()]
    want = all_three()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams * 3:
        with torch.cuda.stream(s):
            got.append(all_three())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for one in got for a, b in zip(want, one)) and int(st.item()) == 0
