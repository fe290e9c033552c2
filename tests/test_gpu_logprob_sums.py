"""GPU: sums over very many tokens, and rows as they are shared by threads, of log probabilities.

Tolerances: a thread adds at most 512 numbers in a row to one of two sums, and those
sums at most 1024 times to the total (2^28 tokens on 256 threads); each addition rounds by
2^-24 of the sum, the exponentials by 2^-22: relative errors of S and T of at most 2^-13.4 (1536 x 2^-24), so
of ln S and of T / S twice that at the very most; below 2^18 tokens a thread has 1024 numbers at most in all."""
import math

import pytest
import torch

from test_gpu_attn_half import DEV, _gpu, f64, pw, within  # noqa: F401
from test_gpu_logprobs import DTYPES, IDS, call

pytestmark = pytest.mark.gpu


def nearly_equal(rows, vocab, dtype, low):
    """Tokens of one logit and, here and there (so that every thread's addends are relative to them), of a larger one:
    lse, entropy and log probability of both, by their closed forms."""
    z = torch.full((rows, vocab), low, dtype=dtype, device=DEV)
    z[:, ::1001] = 1.0
    n1 = -(-vocab // 1001)
    e = (vocab - n1) * math.exp(low - 1.0)
    lse = 1.0 + math.log(n1 + e)
    entropy = lse - 1.0 - e * (low - 1.0) / (n1 + e)
    targets = torch.tensor([[2002, 2003]], dtype=torch.int32, device=DEV).repeat(rows, 1)
    return z, targets, lse, entropy, [1.0 - lse, low - lse]


@pytest.mark.parametrize("rows,vocab,dtype", [
    (1, 1 << 28, torch.float16), (1, 1 << 28, torch.float32), (160, 1 << 24, torch.bfloat16), (160, (1 << 22) + 5, torch.float32),
    (3, (1 << 26) + 1, torch.bfloat16)], ids=str)
@pytest.mark.parametrize("low", [0.9375, -0.5, 0.0625, -2.0])
def test_sums_of_nearly_equal_logits(rows, vocab, dtype, low):
    """Equal addends round the same way every time: the errors of one running sum of 65536 of them reach 2^-10."""
    z, targets, lse, entropy, lp = nearly_equal(rows, vocab, dtype, low)
    out = call(z, targets, 2)
    bound = 1536 * 2.0 ** -24
    within(out["lse"], torch.full((rows,), lse).double().numpy(), bound + 2.0 ** -21 * abs(lse))
    within(out["entropy"], torch.full((rows,), entropy).double().numpy(), 2 * bound + 2.0 ** -21 * abs(entropy))
    within(out["logprobs"], torch.tensor([lp], dtype=torch.float64).repeat(rows, 1).numpy(), bound + 2.0 ** -21 * abs(lse))
    assert (out["top_ids"] == torch.tensor([0, 1001], device=DEV)).all()


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_a_maximum_that_rises_late_over_many_tokens(dtype):
    """What has been added up before is moved with the rest: a row that rises in steps of 1, far apart."""
    vocab = 1 << 24
    step = torch.arange(vocab, device=DEV) // (vocab // 8)
    z = (step.to(torch.float32) - 4).to(dtype)[None].repeat(2, 1)
    out = call(z)
    n = vocab // 8
    s = sum(n * math.exp(k - 7) for k in range(8))
    t = sum(n * math.exp(k - 7) * (k - 7) for k in range(8))
    bound = 1536 * 2.0 ** -24
    want = 3 + math.log(s), math.log(s) - t / s
    within(out["lse"], torch.full((2,), want[0]).double().numpy(), bound + 2.0 ** -21 * want[0])
    within(out["entropy"], torch.full((2,), want[1]).double().numpy(), 2 * bound + 2.0 ** -21 * want[1])
