"""The expert block's launches that only larger calls take: joins of two and four
chunks a thread, the gathering quantizer of several chunks a thread, routing in one
CTA, one cluster and two launches for each number of logits a lane and type."""
import pytest
import torch

import experts_ref as ref
import fp8_w8a8_quantized_gb300 as fp8
from test_gpu_experts import bounds, check_join, check_route, clean, gen, normal, weights, within

pytestmark = pytest.mark.gpu
DEV = "cuda"


# ------------------------------------------------------------------------------------- the join

# (tokens x columns / 8 beyond 155648, or columns beyond 8192: the widths lie on both sides of where
# the number of threads a token changes; tokens that leave the last CTA of several a part)
@pytest.mark.parametrize("post,gate,rows,codes", [(False, "none", True, True), (True, "channel", False, True),
                                                  (True, "token", True, False)])
@pytest.mark.parametrize("k", [0, 3])
@pytest.mark.parametrize("T,K", [(5003, 272), (5003, 512), (2501, 528), (2501, 1024), (2501, 1040), (1021, 2048),
                                 (701, 2064), (701, 2880), (701, 4096), (307, 4112), (301, 8176), (155, 8208),
                                 (77, 16384), (39, 16400)])
def test_join_of_several_chunks_a_thread(T, K, k, post, gate, rows, codes):
    check_join(T, K, k, post, gate, rows=rows, codes=codes, rs=0.5, bs=0.22, holes=k > 0)


@pytest.mark.parametrize("k", [0, 1, 2])
@pytest.mark.parametrize("T,K", [(8192, 1024), (2048, 4096), (9001, 144)])
def test_join_of_prompts(T, K, k):
    check_join(T, K, k, False, "none", rows=False)


# ------------------------------------------------------------------------------------- rows gathered and quantized

# (R K / 16 beyond 155648, so two chunks a thread, four of the widest; or one row's chunks beyond 1024)
@pytest.mark.parametrize("R,K", [(5003, 512), (5003, 528), (2501, 1040), (1301, 2064), (701, 4112), (311, 8208),
                                 (157, 16400), (67, 40000), (5, 20000), (3, 40016)])
@pytest.mark.parametrize("gathered", [True, False])
def test_gathered_rows_of_several_chunks_a_thread(R, K, gathered):
    g = gen(R + K)
    E, N, T = 3, 40, R // 2 + 1 if gathered else R
    wq, s_w = weights(g, E, N, K)
    w8 = wq.view(torch.uint8)
    x = normal(g, T, K + 16, scale=3.0)[:, 8:K + 8]  # rows of a wider matrix
    x[0] = 0
    rows = None
    if gathered:
        rows = torch.randint(0, T, (R,), generator=g, device=DEV).int()
        rows[torch.rand(R, generator=g, device=DEV) < 0.1] = -1
        rows[R // 2], rows[R - 1] = T, T - 1
    offsets = bounds([R // 3, 0, R - R // 3])
    ws = torch.empty(fp8.fp8_grouped_linear_workspace_size(E, R, N, K), dtype=torch.uint8, device=DEV)
    y = fp8.fp8_grouped_linear(x, w8, s_w, offsets, row_token=rows, workspace=ws)
    clean()
    at = torch.arange(R, device=DEV) if rows is None else rows.long()
    absent = (at < 0) | (at >= T)
    codes, s = fp8.fp8_quant_per_token(x[at.clamp(0, T - 1)].contiguous())
    codes[absent], s[absent] = 0, 1
    want_codes, want_s = ref.quant(torch.where(absent[:, None], 0.0, x[at.clamp(0, T - 1)].float()))
    assert torch.equal(s, want_s) and torch.equal(codes, want_codes.view(torch.uint8))
    # (the workspace begins with the rows' codes, and at the next multiple of 256 bytes their scales)
    assert torch.equal(ws[: R * K].view(R, K), codes)
    begin = (R * K + 255) // 256 * 256
    assert torch.equal(ws[begin: begin + 4 * R].view(torch.float32), s)
    assert torch.equal(y, fp8.fp8_grouped_gemm(codes, s, w8, s_w, offsets))
    assert (y[absent] == 0).all()
    clean()


# ------------------------------------------------------------------------------------- routing

# (one CTA, one cluster, two launches; 1, 2, 4, 8, 16 and 32 logits a lane)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("T", [9, 100, 600])
@pytest.mark.parametrize("E,k", [(20, 3), (60, 4), (100, 8), (128, 8), (250, 8), (400, 6), (1000, 32)])
def test_route_launches(T, E, k, dtype):
    x = (torch.randn(T, E, generator=gen(T + E), device=DEV) * 2).to(dtype)
    x[:, E // 2] = -torch.inf
    x[T // 2] = -torch.inf
    x[T // 3, : E - 2] = float("nan")
    x[T - 1] = 0
    check_route(x, k, renorm=T != 100, scale=2.5)


def check_route_large(x, k, renorm):
    """As check_route, in whole-tensor steps on the GPU."""
    T, E = x.shape
    got = fp8.fp8_moe_route(x, k, renormalize=renorm)
    clean()
    value, ids = torch.sort(x.float(), dim=1, descending=True, stable=True)
    value, ids = value[:, :k], ids[:, :k]
    there = value > -torch.inf
    ids = torch.where(there, ids, -1)
    assert torch.equal(got[0], ids.int())
    flat = ids.reshape(-1)
    key = torch.where(flat < 0, E, flat)
    rank = torch.sort(key, stable=True).indices
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=DEV)
    offsets[1:] = torch.bincount(key, minlength=E + 1)[:E].cumsum(0)
    assert torch.equal(got[2], offsets.int())
    at = torch.arange(T * k, device=DEV)
    assert torch.equal(got[3], torch.where(at < offsets[-1], rank // k, -1).int())
    back = torch.empty_like(rank)
    back[rank] = at
    assert torch.equal(got[4], torch.where(flat < 0, -1, back).view(T, k).int())
    best = torch.where(there[:, :1], value[:, :1], 0.0).double()
    p = torch.where(there, torch.exp(value.double() - best), 0.0)
    total = p.sum(1, keepdim=True) if renorm else torch.exp(x.double() - best).sum(1, keepdim=True)
    want = p / torch.where(total > 0, total, 1.0)
    # (the bound of ref.route)
    tol = want * (torch.where(there, best - value.double(), 0.0) + 57) * ref.HALF["fp32"]
    within(got[1], want, tol, "weights")


@pytest.mark.parametrize("T,E,k", [(40000, 60, 8), (20011, 1000, 32), (65536, 8, 2)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_route_of_many_pairs_a_warp(T, E, k, dtype):
    x = (torch.randn(T, E, generator=gen(T), device=DEV) * 2).to(dtype)
    x[::7] = -torch.inf
    x[5::11, ::2] = -torch.inf
    check_route_large(x, k, renorm=dtype == torch.bfloat16)


@pytest.mark.parametrize("one", [True, False])
def test_route_of_the_most_tokens(one):
    # 55189 tokens a part, all of them or most of them of one expert: counts beyond 2^15
    T = 1 << 23
    x = torch.zeros(T, 2, device=DEV)
    x[:, 1] = 1.0
    if not one:
        x[:, 0] = torch.randn(T, generator=gen(1), device=DEV) - 0.5
        x[::1000] = -torch.inf
    check_route_large(x, 1, renorm=False)
