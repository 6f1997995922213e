"""Refusals of the expert block's calls, on the host: each rejected call answers
before anything is launched, so no GPU is needed."""
import math

import pytest
import torch

INVALID, UNSUP, WS, CUDA = 1, 2, 3, 4
P = 1 << 20  # never dereferenced


@pytest.fixture(scope="module")
def L():
    from fp8_w8a8_quantized_gb300 import build
    build.build()
    import fp8_w8a8_quantized_gb300 as pkg
    return pkg.lib()


def call(f, defaults, **changed):
    assert set(changed) <= set(defaults)
    return f(*{**defaults, **changed}.values())


ROUTE = dict(logits=P, fp32=1, ld=64, T=4096, E=64, k=8, renorm=1, scale=1.0, ids=P, weights=P, offsets=P, rows=P,
             back=P, ws=P, bytes=1 << 30, stream=None)
GEMM = dict(xq=P, s_tok=P, wq=P, s_w=P, offsets=P, E=8, R=64, N=256, K=512, swiglu=0, y=P, ws=P, bytes=1 << 30,
            stream=None)
LINEAR = dict(x=P, T=32, ldx=512, rows=P, wq=P, s_w=P, offsets=P, E=8, R=64, N=256, K=512, swiglu=0, y=P, ws=P,
              bytes=1 << 30, stream=None)
JOIN = dict(h=P, ldh=512, y=P, ldy=512, R=64, rows=P, weights=P, k=2, post=P, gate=P, ldg=0, gamma=P, eps=1e-6, rs=1.0,
            bs=1.0, T=32, K=512, h_out=P, ldho=512, z=P, xq=P, ldq=512, s_tok=P, stream=None)


@pytest.mark.parametrize("changed,want", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(k=0), INVALID), (dict(k=65), INVALID), (dict(E=-4), INVALID),
    (dict(scale=math.nan), INVALID), (dict(scale=math.inf), INVALID), (dict(E=1025, ld=2000), UNSUP),
    (dict(k=33), UNSUP), (dict(T=1 << 28, k=8), UNSUP), (dict(T=1 << 31), INVALID), (dict(logits=None), INVALID),
    (dict(ids=None), INVALID), (dict(weights=None), INVALID), (dict(offsets=None), INVALID), (dict(rows=None), INVALID),
    (dict(back=None), INVALID), (dict(ld=63), INVALID), (dict(ld=1 << 40), INVALID), (dict(logits=P + 2), UNSUP),
    (dict(fp32=0, logits=P + 1), UNSUP), (dict(ids=P + 2), UNSUP), (dict(weights=P + 1), UNSUP),
    (dict(offsets=P + 2), UNSUP), (dict(rows=P + 2), UNSUP), (dict(back=P + 2), UNSUP), (dict(ws=None), WS),
    (dict(bytes=3), WS), (dict(ws=P + 8), WS)])
def test_route_refusals(L, changed, want):
    assert call(L.fp8_moe_route, ROUTE, **changed) == want


SIZES = [(dict(E=0), INVALID), (dict(E=-1), INVALID), (dict(R=-1), INVALID), (dict(N=-1), INVALID), (dict(K=-16), INVALID),
         (dict(E=1025), UNSUP), (dict(K=0), UNSUP), (dict(N=257, swiglu=1), INVALID), (dict(R=1 << 31), INVALID),
         (dict(N=1 << 29), UNSUP), (dict(wq=None), INVALID), (dict(s_w=None), INVALID), (dict(offsets=None), INVALID),
         (dict(y=None), INVALID), (dict(wq=P + 8), UNSUP), (dict(s_w=P + 2), UNSUP), (dict(offsets=P + 2), UNSUP),
         (dict(y=P + 8), UNSUP), (dict(N=0), 0)]


@pytest.mark.parametrize("changed,want", SIZES + [
    (dict(K=520), UNSUP), (dict(R=0), 0), (dict(xq=None), INVALID), (dict(s_tok=None), INVALID), (dict(xq=P + 8), UNSUP),
    (dict(s_tok=P + 2), UNSUP)])
def test_grouped_gemm_refusals(L, changed, want):
    assert call(L.fp8_grouped_gemm, GEMM, **changed) == want


@pytest.mark.parametrize("changed,want", SIZES + [
    (dict(K=520, ldx=520), UNSUP), (dict(R=0), 0), (dict(T=-1), INVALID), (dict(rows=None), INVALID),
    (dict(x=None), INVALID), (dict(ldx=504), INVALID), (dict(ldx=516), UNSUP), (dict(x=P + 8), UNSUP),
    (dict(rows=P + 2), UNSUP), (dict(ws=None), WS), (dict(bytes=64 * 512), WS), (dict(ws=P + 128), WS),
    (dict(rows=None, T=64, ws=None), WS)])
def test_grouped_linear_refusals(L, changed, want):
    assert call(L.fp8_grouped_linear, LINEAR, **changed) == want


@pytest.mark.parametrize("changed,want", [
    (dict(T=-1), INVALID), (dict(R=-1), INVALID), (dict(K=-16), INVALID), (dict(k=-1), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=math.nan), INVALID), (dict(eps=math.inf), INVALID), (dict(rs=math.inf), INVALID), (dict(bs=math.nan), INVALID),
    (dict(k=0), INVALID), (dict(K=0), UNSUP), (dict(K=520, ldh=520), UNSUP), (dict(K=32784), UNSUP), (dict(k=33), UNSUP),
    (dict(rows=None), INVALID), (dict(xq=None), INVALID), (dict(s_tok=None), INVALID), (dict(gamma=None), INVALID),
    (dict(gamma=None, z=None), INVALID), (dict(h=None), INVALID), (dict(y=None), INVALID), (dict(h_out=None), INVALID),
    (dict(ldh=504), INVALID), (dict(ldy=504), INVALID), (dict(ldho=504), INVALID), (dict(ldg=504), INVALID),
    (dict(ldg=516), UNSUP), (dict(ldh=516), UNSUP), (dict(ldq=504), INVALID), (dict(ldq=520), UNSUP), (dict(h=P + 8), UNSUP),
    (dict(y=P + 8), UNSUP), (dict(h_out=P + 8), UNSUP), (dict(gate=P + 8), UNSUP), (dict(post=P + 8), UNSUP),
    (dict(gamma=P + 8), UNSUP), (dict(z=P + 8), UNSUP), (dict(xq=P + 8), UNSUP), (dict(s_tok=P + 2), UNSUP),
    (dict(rows=P + 2), UNSUP), (dict(weights=P + 2), UNSUP), (dict(ldh=1 << 40), INVALID), (dict(T=0), 0)])
def test_join_refusals(L, changed, want):
    assert call(L.fp8_residual_norm_quant, JOIN, **changed) == want


def test_workspaces(L):
    need = L.fp8_grouped_linear_workspace_size(8, 64, 256, 512)
    assert need >= 64 * 512 + 256
    assert call(L.fp8_grouped_linear, LINEAR, bytes=need - 1) == WS
    need = L.fp8_grouped_gemm_workspace_size(8, 64, 256, 512)
    if need:
        assert call(L.fp8_grouped_gemm, GEMM, bytes=need - 1) == WS
        assert call(L.fp8_grouped_gemm, GEMM, ws=None) == WS
        assert call(L.fp8_grouped_gemm, GEMM, ws=P + 128) == WS
    need = L.fp8_moe_route_workspace_size(4096, 64, 8)
    assert need > 0
    assert call(L.fp8_moe_route, ROUTE, bytes=need - 1) == WS
    for bad in ((0, 64, 256, 512), (8, -1, 256, 512), (8, 64, 256, 500), (8, 0, 256, 512), (8, 64, 0, 512),
                (1025, 64, 256, 512), (8, 64, 1 << 29, 512)):
        assert L.fp8_grouped_gemm_workspace_size(*bad) == 0 and L.fp8_grouped_linear_workspace_size(*bad) == 0
    for bad in ((-1, 64, 8), (32, 0, 1), (32, 64, 0), (32, 64, 65), (32, 1025, 8), (32, 64, 33), (1 << 29, 64, 8)):
        assert L.fp8_moe_route_workspace_size(*bad) == 0


def test_calls_that_pass_the_checks_report_a_cuda_error_without_a_device(L):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; this case needs a machine without one")
    assert call(L.fp8_moe_route, ROUTE) == CUDA
    assert call(L.fp8_grouped_gemm, GEMM) == CUDA
    assert call(L.fp8_grouped_linear, LINEAR) == CUDA
    assert call(L.fp8_grouped_linear, LINEAR, rows=None, T=64) == CUDA
    assert call(L.fp8_residual_norm_quant, JOIN) == CUDA
    assert call(L.fp8_residual_norm_quant, JOIN, k=0, R=32, rows=None, weights=None, post=None, gate=None) == CUDA
    assert call(L.fp8_residual_norm_quant, JOIN, gamma=None, z=None, xq=None, s_tok=None, ldq=0) == CUDA


def test_binding_rejects_tensors_the_kernels_cannot_take():
    import fp8_w8a8_quantized_gb300 as pkg
    x, i32 = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    codes, one = torch.zeros(3, 8, 64, dtype=torch.uint8), torch.ones(3, 8)
    with pytest.raises(ValueError, match="logits must be a CUDA"):
        pkg.fp8_moe_route(x, 2)
    with pytest.raises(ValueError, match="logits must be a CUDA"):
        pkg.fp8_moe_route(x.half(), 2)
    with pytest.raises(ValueError, match="x must be a CUDA"):
        pkg.fp8_grouped_linear(x, codes, one, i32)
    with pytest.raises(ValueError, match="xq must be a CUDA"):
        pkg.fp8_grouped_gemm(codes[0], one[0], codes, one, i32)
    with pytest.raises(ValueError, match="h must be a CUDA"):
        pkg.fp8_residual_norm_quant(x, x, x[0])
    with pytest.raises(ValueError, match="logits must be a CUDA tensor; got list"):
        pkg.fp8_moe_route([1.0], 1)
    for name, f in (("renormalize", lambda v: pkg.fp8_moe_route(x, 2, renormalize=v)),
                    ("swiglu", lambda v: pkg.fp8_grouped_linear(x, codes, one, i32, swiglu=v)),
                    ("codes", lambda v: pkg.fp8_residual_norm_quant(x, x, x[0], codes=v))):
        with pytest.raises(ValueError, match=name + " must be true or false"):
            f(torch.zeros(2))
