"""GPU: arguments of the attention that only bound something."""
import pytest
import torch

from test_gpu_attn_half import Batch, _gpu, pw  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("tokens", [1, 64])
def test_a_bound_of_any_length_costs_nothing(tokens):
    """max_kv_len 2^31 - 1 ("any") is a bound like another: the same bits as the
    table's own length, and no fewer CTAs (a wrapped bound left one: 20 times as
    long here)."""
    b = Batch([tokens], [16384], 4, 1, 128, 128, torch.float16, 2)
    ws = torch.zeros(pw.pw_paged_attention_workspace(b.T, 1, 4, 1, 128), dtype=torch.uint8, device="cuda")
    out, took = {}, {}
    for bound in (b.table.shape[1] * 128, 2 ** 31 - 1):
        times = []
        for _ in range(12):
            start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            torch.cuda._sleep(2_000_000)             # the host is ahead of the GPU
            start.record()
            o, lse, _ = call(b, ws, bound)
            end.record()
            torch.cuda.synchronize()
            times.append(start.elapsed_time(end))
        out[bound], took[bound] = (o, lse), min(times)
    (a, x), (c, y) = out.values()
    assert torch.equal(a, c) and torch.equal(x, y)
    exact, any_length = took.values()
    assert any_length < 3 * exact, (exact, any_length)


def call(b, ws, bound):
    out, lse = torch.empty_like(b.q), torch.empty(b.T, b.heads, device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    pw.pw_paged_attention(b.q, b.k, b.v, b.table, b.offsets, b.lens, out, ws, st, scale=b.d ** -0.5, lse=lse,
                          max_q_len=b.T, max_kv_len=bound)
    return out, lse, st


def test_one_row_of_a_wider_lse():
    """A single token's log-sums may be a row of anything; several tokens' rows
    have to follow each other."""
    b = Batch([1], [30], 4, 2, 64, 16, torch.float16, 3)
    ws = torch.zeros(pw.pw_paged_attention_workspace(1, 1, 4, 2, 64), dtype=torch.uint8, device="cuda")
    _, want, _ = call(b, ws, 30)
    wide = torch.full((5, 9), 7.0, device="cuda")
    out, st = torch.empty_like(b.q), torch.zeros(1, dtype=torch.int32, device="cuda")
    pw.pw_paged_attention(b.q, b.k, b.v, b.table, b.offsets, b.lens, out, ws, st, scale=0.125, lse=wide[2:3, 3:7])
    assert torch.equal(wide[2:3, 3:7], want) and int((wide == 7).sum()) == 41 and int(st.item()) == 0
    two = Batch([2], [30], 4, 2, 64, 16, torch.float16, 3)
    with pytest.raises(ValueError):
        pw.pw_paged_attention(two.q, two.k, two.v, two.table, two.offsets, two.lens, torch.empty_like(two.q), ws, st,
                              scale=0.125, lse=wide[2:4, 3:7])
