"""GPU: windows with first keys whose scores stand 5 to 10 above the others', which is what first keys are kept
for: they hold the maximum of nearly every row.  Tolerances as for the attention."""
import pytest
import torch

from test_gpu_attn_half import Batch, DTYPES, IDS, _gpu, attend, draw, gen, pw  # noqa: F401
from test_gpu_sinks import check, forget

pytestmark = pytest.mark.gpu


def raise_first_keys(b, sinks, seed, lowest=5.0, highest=10.0, order="any"):
    """The first component of queries is 6; that of the first keys makes up the rest."""
    b.q[..., 0] = 6.0
    for i, n in enumerate(b.kv):
        m = min(sinks, n)
        up = lowest + (highest - lowest) * torch.rand(m, generator=gen(seed + i))
        up = {"any": up, "rising": up.sort().values, "falling": up.sort(descending=True).values}[order]
        for key in range(m):
            b.k[int(b.table[i, key // b.ps]), key % b.ps, :, 0] = float(up[key]) * b.d ** 0.5 / 6.0
        for j in range(-(-n // b.ps)):                  # the others have nothing of it
            rows = [r for r in range(b.ps) if sinks <= j * b.ps + r < n]
            b.k[int(b.table[i, j]), rows, :, 0] = 0.0


@pytest.mark.parametrize("order", ["any", "rising", "falling"])
@pytest.mark.parametrize("sinks", [1, 4, 64, 200])
@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_first_keys_that_hold_the_maximum(dtype, sinks, order):
    for ql, kl, h, hk, d, ps, window in [([1, 1, 1], [900, 40, 333], 8, 2, 128, 16, 100), ([5, 3], [700, 300], 4, 2, 64, 32, 60),
                                         ([100, 40], [900, 700], 4, 2, 128, 32, 260), ([70], [600], 2, 1, 64, 16, 130),
                                         ([1], [9000], 4, 1, 128, 32, 3000)]:
        b = Batch(ql, kl, h, hk, d, ps, dtype, 40 + sinks, False)
        raise_first_keys(b, sinks, 7, order=order)
        forget(b, window, sinks)
        out, lse, st = attend(b, window=window, sinks=sinks)
        assert st == 0
        check(b, out, lse, window, sinks)


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_first_keys_far_above_and_far_below(dtype):
    """Nearly all of the weight on them, or nearly none: 40 above and 40 below."""
    for ql in (1, 90):
        for up in (40.0, -40.0):
            b = Batch([ql], [700], 4, 2, 128, 32, dtype, 3)
            raise_first_keys(b, 6, 5, up, up)
            forget(b, 150, 6)
            out, lse, st = attend(b, window=150, sinks=6)
            assert st == 0
            check(b, out, lse, 150, 6)
