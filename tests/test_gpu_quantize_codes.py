"""GPU: e4m3 codes are those of value / scale in 32 bits, code for code."""
import pytest
import torch

from test_gpu_attn_half import DEV, DTYPES, IDS, _gpu, draw, gen, pw  # noqa: F401

pytestmark = pytest.mark.gpu


def codes_of(y, scale, block_rows):
    """e4m3(y / scale) by torch's own division and conversion, and the scales of y."""
    rows, cols = y.shape
    y = y.float().cpu()
    r, c = -(-rows // block_rows), -(-cols // 128)
    pad = torch.nn.functional.pad(y, (0, c * 128 - cols, 0, r * block_rows - rows))
    top = pad.view(r, block_rows, c, 128).abs().amax(dim=(1, 3))
    want = (top / 448.0).clamp(min=2.0 ** -100)
    assert torch.equal(scale.cpu(), want)
    s = want.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :cols]
    return (y / s).to(torch.float8_e4m3fn).view(torch.uint8)


def quantize(x, block_rows):
    rows, cols = x.shape
    q = torch.empty(rows, cols, dtype=torch.uint8, device=DEV)
    scale = torch.empty(-(-rows // block_rows), -(-cols // 128), device=DEV)
    pw.pw_quantize_fp8(x, q, scale, block_rows=block_rows)
    return q.cpu(), scale


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("block_rows", [1, 128])
@pytest.mark.parametrize("rows,cols", [(1, 5), (200, 136), (1030, 2048), (1000, 1001), (129, 8200)])
def test_codes_are_the_quotients(rows, cols, block_rows, dtype):
    """Large enough that a product with the reciprocal differs somewhere."""
    x = draw(gen(rows + cols), rows, cols, dtype=dtype, scale=5)
    x[:, ::37] *= 50
    q, scale = quantize(x, block_rows)
    assert torch.equal(q, codes_of(x, scale, block_rows))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
@pytest.mark.parametrize("block_rows", [1, 128])
def test_codes_of_every_value(block_rows, dtype):
    """Every finite number of the type, sorted, so that a group's values are of
    one magnitude, and shuffled, so that they are of all; zeros keep their sign."""
    x = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dtype)
    x = x[torch.isfinite(x)]
    x = torch.cat((x, torch.zeros(-x.numel() % 1024, dtype=dtype)))
    for order in (x.float().argsort(), torch.randperm(x.numel(), generator=gen(3))):
        v = x[order].view(-1, 1024).to(DEV)
        q, scale = quantize(v, block_rows)
        assert torch.equal(q, codes_of(v, scale, block_rows))


@pytest.mark.parametrize("dtype", DTYPES, ids=IDS)
def test_norm_codes_follow_its_scales(dtype):
    """The norm's own 8-bit output, on values whose norm is exact in 32 bits: rows
    of +-1 with an eps of 0 have the root mean square 1."""
    rows, cols = 300, 1024
    g = gen(8)
    x = torch.where(torch.rand(rows, cols, generator=g) < 0.5, -1.0, 1.0).to(dtype).to(DEV)
    w = draw(g, cols, dtype=dtype, scale=3)
    q, scale = torch.empty(rows, cols, dtype=torch.uint8, device=DEV), torch.empty(rows, 8, device=DEV)
    pw.pw_add_rmsnorm(x, w, 0.0, q=q, scale=scale)
    assert torch.equal(q.cpu(), codes_of(x.float() * w.float(), scale, 1))
