"""Codes of the join where the rows' scales are at the end of fp32's range."""
import pytest
import torch

import fp8_w8a8_quantized_gb300 as fp8

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("K", [64, 4096])
def test_rows_whose_scale_rounds_to_zero(K):
    # one value a row, 2^-j gamma with eps = 1: the norm's factor is 1, the row's z exact down to
    # fp32's smallest number, and a 448th of it passes the border below which nothing is left
    gamma = torch.full((K,), 2.0 ** -45, dtype=torch.bfloat16, device=DEV)
    size = torch.tensor([2.0 ** -j for j in range(80, 107)], dtype=torch.float64, device=DEV)
    h = torch.zeros(len(size), K, dtype=torch.bfloat16, device=DEV)
    h[:, 5] = size.to(torch.bfloat16)
    y = torch.zeros_like(h)
    _, _, xq, s = fp8.fp8_residual_norm_quant(h, y, gamma, eps=1.0)
    torch.cuda.synchronize()
    z = torch.zeros(len(size), K, dtype=torch.float64, device=DEV)
    z[:, 5] = (size * 2.0 ** -45).float().double()
    want = (z[:, 5] / 448).float()
    assert (want == 0).any() and (want > 0).any()
    assert torch.equal(s, torch.where(want > 0, want, 1.0))
    value = xq.view(torch.float8_e4m3fn).double() * s[:, None].double()
    # half a step of the codes; where the scale has few bits left, the most that its rounding (half of
    # 2^-149) takes from a value of 448 scales
    off = (value - z).abs() - (z * 2.0 ** -4 + 448 * 2.0 ** -150)
    assert not torch.isnan(value).any()
    assert (off <= 0).all(), off.max()
    assert (value[:, :5] == 0).all() and (value[:, 6:] == 0).all()
