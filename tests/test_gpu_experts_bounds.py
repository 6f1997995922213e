"""Grouped products of bounds that go back or lie outside the rows: the rows of each
expert are those of the bounds cut to 0 .. R, each raised to the largest up to it."""
import pytest
import torch

import fp8_w8a8_quantized_gb300 as fp8

pytestmark = pytest.mark.gpu
DEV = "cuda"


def operands(E, R, N, K, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def codes(*shape):
        return (torch.randn(*shape, generator=g, device=DEV) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)

    return codes(R, K), torch.rand(R, generator=g, device=DEV), codes(E, N, K), torch.rand(E, N, generator=g, device=DEV)


# (R up to 32: bounds read behind the wait alone; up to 128 an expert: a tile an SM; beyond: pairs)
@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("R,bounds", [
    (20, [0, 10, 5, 20]), (20, [20, 0, 20, 0]), (20, [7, 3, 3, 1]), (20, [-4, 40, 2, 12]),
    (90, [0, 60, 10, 90]), (90, [90, 80, 85, 90]), (90, [30, 0, 70, 69]),
    (700, [0, 500, 100, 700]), (700, [650, 0, 700, 1]), (700, [0, 1 << 30, -(1 << 31), 300])])
def test_no_row_has_two_experts(R, bounds, swiglu):
    N, K, E = 320, 528, 3
    xq, s_tok, wq, s_w = operands(E, R, N, K, R)
    raised = torch.tensor(bounds).clamp(0, R).cummax(0).values
    y = [torch.full((R, N // 2 if swiglu else N), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for off, out in zip((torch.tensor(bounds), raised), y):
        fp8.fp8_grouped_gemm(xq, s_tok, wq, s_w, off.int().to(DEV), swiglu=swiglu, y=out)
    torch.cuda.synchronize()
    assert fp8.fp8_device_status() == fp8.FP8_OK
    assert torch.equal(*y)
    first, last = raised[0].item(), raised[-1].item()
    assert (y[0][:first] == 7).all() and (y[0][last:] == 7).all()


def test_many_experts_whose_bounds_go_back():
    E, R, N, K = 1024, 600, 48, 64
    xq, s_tok, wq, s_w = operands(E, R, N, K, 1)
    g = torch.Generator().manual_seed(2)
    off = torch.randint(-50, R + 50, (E + 1,), generator=g)
    x = torch.randn(R, K, device=DEV).to(torch.bfloat16)
    raised = off.clamp(0, R).cummax(0).values.int().to(DEV)
    first, last = raised[0].item(), raised[-1].item()
    off = off.int().to(DEV)
    for f in (lambda o: fp8.fp8_grouped_gemm(xq, s_tok, wq, s_w, o),
              lambda o: fp8.fp8_grouped_linear(x, wq, s_w, o)):
        assert torch.equal(f(off)[first:last], f(raised)[first:last])
    torch.cuda.synchronize()
    assert fp8.fp8_device_status() == fp8.FP8_OK
