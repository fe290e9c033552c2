"""GPU: a NaN in a weight of the gated block: its column in 16 bits, its group of 128 columns in 8 bits,
where the scale takes it up; what lies beside them is what it is without the NaN."""
import pytest
import torch

from test_gpu_attn_half import DEV, _gpu, pw, status  # noqa: F401
from test_gpu_gated import ACTS, problem

pytestmark = pytest.mark.gpu


def call(args, m, n, act):
    st, y = status(), torch.empty(m, n, dtype=torch.bfloat16, device=DEV)
    q, sc = torch.empty(m, n, dtype=torch.uint8, device=DEV), torch.empty(m, -(-n // 128), device=DEV)
    pw.pw_fp8_gated_linear(*args, st, y=y, q=q.view(torch.float8_e4m3fn), scale=sc, activation=ACTS[act])
    assert int(st.item()) == 0
    return y, q, sc


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("which", [2, 4], ids=["gate", "up"])
@pytest.mark.parametrize("m,n,k", [(4, 400, 256), (13, 400, 256), (40, 400, 256), (100, 300, 1024), (100, 400, 2048), (2500, 1100, 256)])
def test_a_weight_that_is_nan(m, n, k, which, act):
    args = problem(m, n, k)
    want = call(args, m, n, act)
    args[which].view(torch.uint8)[200, 7] = 0x7F        # NaN
    y, q, sc = call(args, m, n, act)
    beside = torch.arange(n, device=DEV) != 200
    assert y[:, 200].isnan().all() and torch.equal(y[:, beside], want[0][:, beside])
    group = torch.arange(n, device=DEV) // 128 == 1
    assert sc[:, 1].isnan().all() and (q[:, group] & 127 == 127).all()
    others = [g for g in range(sc.shape[1]) if g != 1]
    assert torch.equal(q[:, ~group], want[1][:, ~group]) and torch.equal(sc[:, others], want[2][:, others])
