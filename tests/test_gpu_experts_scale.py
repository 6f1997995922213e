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


def test_rows_whose_squares_leave_fp32():
    # as the header says: normed to zeros, the stream itself kept; the rows beside them as ever
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    h = torch.randn(5, 256, generator=g, device=DEV).to(torch.bfloat16)
    y, one = torch.zeros_like(h), torch.ones(256, dtype=torch.bfloat16, device=DEV)
    plain = fp8.fp8_residual_norm_quant(h, y, one)
    big = h.clone()
    big[[1, 3], 7] = 2.0 ** 70
    out, z, xq, s = fp8.fp8_residual_norm_quant(big, y, one)
    torch.cuda.synchronize()
    assert torch.equal(out, big)
    for got, want in zip((z, xq, s), plain[1:]):
        assert torch.equal(got[[0, 2, 4]], want[[0, 2, 4]])
    assert (z[[1, 3]] == 0).all() and (s[[1, 3]] == 1).all()
    assert (xq[[1, 3]].view(torch.float8_e4m3fn).float() == 0).all()
    # (the branch's own norm: nothing is left of it, and the stream stays)
    out = fp8.fp8_residual_norm_quant(h, big, one, gamma_post=one)[0]
    assert torch.equal(out[[1, 3]], h[[1, 3]])


def test_rows_of_zeros_without_eps_are_divided_by_zero():
    h = torch.zeros(3, 64, dtype=torch.bfloat16, device=DEV)
    h[1] = 2.0
    one = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    out, z, xq, s = fp8.fp8_residual_norm_quant(h, torch.zeros_like(h), one, eps=0.0)
    torch.cuda.synchronize()
    assert torch.equal(out, h) and torch.isnan(z[[0, 2]].float()).all() and (z[1] == 1).all()
    assert torch.isnan(xq[[0, 2]].view(torch.float8_e4m3fn).float()).all()
