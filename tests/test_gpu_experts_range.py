"""The expert block's operators where offsets pass 32 bits: weights, outputs and
token matrices of more than 2^31 elements, checked in places of all parts."""
import pytest
import torch

import experts_ref as ref
import fp8_w8a8_quantized_gb300 as fp8

pytestmark = pytest.mark.gpu
DEV = "cuda"
F8 = torch.float8_e4m3fn


def within(got, want, tol):
    off = (got.double() - want).abs() - tol
    assert not torch.isnan(off).any() and (off <= 0).all(), off.max()


def codes(g, *shape):
    out = torch.empty(*shape, dtype=torch.uint8, device=DEV)
    for row in out.view(-1, shape[-1]).split(1 << 15):  # (a value in 32 bits for 2^15 rows at a time)
        row.copy_((torch.randn(row.shape, generator=g, device=DEV) * 100).clamp(-448, 448).to(F8).view(torch.uint8))
    return out


def test_weights_of_more_than_2_31_bytes():
    g = torch.Generator(device=DEV)
    g.manual_seed(1)
    E, N, K = 3, 49152, 16384
    wq = codes(g, E, N, K)
    assert wq.numel() > 1 << 31
    s_w = (0.5 + torch.rand(E, N, generator=g, device=DEV)) / (100 * K ** 0.5)
    xq, s_tok = codes(g, 9, K), torch.full((9,), 0.01, device=DEV)
    offsets = torch.tensor([0, 4, 5, 9], dtype=torch.int32, device=DEV)
    y = fp8.fp8_grouped_gemm(xq, s_tok, wq, s_w, offsets)
    at = torch.tensor([0, 1, 8191, 20000, 43690, 43691, N - 2, N - 1], device=DEV)
    want, tol = ref.grouped(xq.view(F8), s_tok, wq[:, at].view(F8), s_w[:, at], offsets, False)
    within(y[:, at], want, tol)
    torch.cuda.synchronize()
    assert fp8.fp8_device_status() == fp8.FP8_OK


@pytest.mark.parametrize("swiglu", [False, True])
def test_outputs_of_more_than_2_31_elements(swiglu):
    g = torch.Generator(device=DEV)
    g.manual_seed(2)
    E, R, K, F = 2, 140001, 32, 16384
    N = 2 * F if swiglu else F
    wq = codes(g, E, N, K)
    s_w = (0.5 + torch.rand(E, N, generator=g, device=DEV)) / (100 * K ** 0.5)
    xq, s_tok = codes(g, R, K), torch.full((R,), 0.01, device=DEV)
    offsets = torch.tensor([0, 70000, R], dtype=torch.int32, device=DEV)
    y = fp8.fp8_grouped_gemm(xq, s_tok, wq, s_w, offsets, swiglu=swiglu)
    assert y.numel() > 1 << 31
    for rows in (slice(0, 300), slice(69900, 70000), slice(70000, 70100), slice(131000, 131200), slice(R - 300, R)):
        e = 0 if rows.stop <= 70000 else 1
        n = rows.stop - rows.start
        want, tol = ref.grouped(xq[rows].view(F8), s_tok[rows], wq[e: e + 1].view(F8), s_w[e: e + 1],
                                torch.tensor([0, n]), swiglu)
        within(y[rows], want, tol)
    torch.cuda.synchronize()
    assert fp8.fp8_device_status() == fp8.FP8_OK


def test_join_of_more_than_2_31_elements():
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    T, K = 70001, 32768
    h = torch.empty(T, K, dtype=torch.bfloat16, device=DEV).normal_(0, 2, generator=g)
    y = torch.empty(T, K, dtype=torch.bfloat16, device=DEV).normal_(0, 1, generator=g)
    assert h.numel() > 1 << 31
    gamma = (1 + 0.1 * torch.randn(K, generator=g, device=DEV)).to(torch.bfloat16)
    rows = torch.randperm(T, generator=g, device=DEV)[:, None].int()
    out, z, xq, s = fp8.fp8_residual_norm_quant(h, y, gamma, token_row=rows, gamma_post=gamma, gate=h)
    at = torch.tensor([0, 1, 32767, 65535, 65536, 66000, T - 1], device=DEV)
    want = ref.residual_norm(h[at], y[rows[at, 0].long()], gamma, 1e-6, gamma, h[at], 1.0, 1.0, None, None)
    within(out[at], want[0], want[3])
    within(z[at], want[1], want[4])
    within(s[at], want[2], want[5])
    value = xq[at].view(F8).double() * s[at][:, None].double()
    within(value, want[1], want[4] + want[1].abs() * (ref.HALF["e4m3"] + 2.0 ** -20) + s[at][:, None].double() * 2.0 ** -10)
    torch.cuda.synchronize()
    assert fp8.fp8_device_status() == fp8.FP8_OK
