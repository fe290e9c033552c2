"""GPU: the 8-bit product writes its columns and nothing beside them, whatever
the width of the result and of the rows that hold it."""
import numpy as np
import pytest
import torch

from oracle import attn_half as ref
from test_gpu_attn_half import DEV, TINY, U, _gpu, f64, gen, pw, status, within  # noqa: F401

pytestmark = pytest.mark.gpu


# single tokens, 64-token tiles, 128 x 128 tiles, groups split over a cluster, pairs of CTAs
@pytest.mark.parametrize("m,k", [(5, 256), (50, 256), (100, 256), (50, 2048), (300, 2100), (2300, 128)])
@pytest.mark.parametrize("n,pitch", [(100, 104), (129, 136), (4, 8), (255, 256), (190, 256), (192, 200), (64, 72), (130, 131),
                                     (2045, 2048), (2050, 2056)])
def test_nothing_beside_the_columns(m, k, n, pitch):
    g = gen(m + n + k)
    kb = -(-k // 128)
    a, b = [(torch.randn(r, k + -k % 16, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn).to(DEV)[:, :k] for r in (m, n)]
    sa, sb = torch.rand(m, kb, generator=g).to(DEV), torch.rand(-(-n // 128), kb, generator=g).to(DEV) / 64
    room = torch.full((m + 2, pitch), 7.0, dtype=torch.bfloat16, device=DEV)
    y, st = room[1:-1], status()
    pw.pw_fp8_linear(a, sa, b, sb, y[:, :n], st)
    assert (room[0] == 7).all() and (room[-1] == 7).all() and (y[:, n:] == 7).all() and int(st.item()) == 0
    want, mag = ref.fp8_linear(a.view(torch.uint8).cpu().numpy(), f64(sa), b.view(torch.uint8).cpu().numpy(), f64(sb))
    u = U[torch.bfloat16]
    within(y[:, :n], want, u * np.abs(want) * 1.01 + 2.0 ** -13 * mag + TINY[torch.bfloat16])
