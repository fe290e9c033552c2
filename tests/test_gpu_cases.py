"""GPU: the measured cases' inputs are a function of the case and the seed alone."""
import pytest
import torch

from test_gpu_attn_half import _gpu  # noqa: F401

pytestmark = pytest.mark.gpu
from perf import more_operators  # noqa: E402


@pytest.mark.parametrize("dtype", ["fp16", "bf16", "fp32"])
@pytest.mark.parametrize("rows,vocab", [(300, 531), (700, 800), (1531, 1024), (4096, 512)])
def test_logits_repeat(rows, vocab, dtype):
    """Short vocabularies: rows that draw one likely position twice."""
    case = {"op": "logprobs", "rows": rows, "vocab": vocab, "pad": 0, "given": 1, "top": 1, "dtype": dtype, "masked": False}
    for seed in range(3):
        want = more_operators.prepare(case, seed)
        plain = [t.clone() for t in more_operators.run(want)]
        for _ in range(10):
            again = more_operators.prepare(case, seed)
            assert torch.equal(again["logits"], want["logits"]) and torch.equal(again["targets"], want["targets"])
        assert all(torch.equal(a, b) for a, b in zip(plain, more_operators.run(again)))
