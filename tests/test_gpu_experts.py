"""The expert block's operators against plain forms in 64 bits: routing, products
grouped by expert, the join with the residual stream."""
import math

import pytest
import torch

import experts_ref as ref
import fp8_w8a8_quantized_gb300 as fp8

pytestmark = pytest.mark.gpu
DEV = "cuda"


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, generator=g, device=DEV) * scale).to(torch.bfloat16)


def clean():
    torch.cuda.synchronize()
    assert fp8.fp8_device_status() == fp8.FP8_OK


def within(got, want, tol, what):
    off = (got.double() - want).abs() - tol
    assert not torch.isnan(off).any(), f"{what}: NaN"
    assert (off <= 0).all(), f"{what}: outside its bound by {off.max().item():.3g}"


# ------------------------------------------------------------------------------------- routing

def check_route(logits, k, renorm=True, scale=1.0):
    got = fp8.fp8_moe_route(logits, k, renormalize=renorm, scale=scale)
    clean()
    ids, w, tol, offsets, row_token, token_row = ref.route(logits, k, renorm, scale)
    for name, a, b in zip(("ids", "offsets", "row_token", "token_row"), (got[0], got[2], got[3], got[4]),
                          (ids, offsets, row_token, token_row)):
        assert a.dtype == torch.int32 and torch.equal(a.cpu(), b), name
    within(got[1].cpu(), w, tol, "weights")
    return got


@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 257, 1021, 4999])
@pytest.mark.parametrize("E,k", [(1, 1), (8, 2), (60, 4), (64, 8), (256, 8)])
def test_route(T, E, k):
    g = gen(T * 1000 + E)
    check_route(torch.randn(T, E, generator=g, device=DEV) * 2, k, renorm=T % 2 == 0, scale=1.0 if E < 64 else 2.5)


@pytest.mark.parametrize("E,k", [(33, 32), (128, 32), (500, 17), (1000, 8), (1024, 32)])
def test_route_many_experts(E, k):
    check_route(torch.randn(300, E, generator=gen(E), device=DEV), k, renorm=False)


@pytest.mark.parametrize("E,k", [(16, 4), (200, 8)])
def test_route_ties_of_16_bits(E, k):
    x = torch.randint(-3, 4, (777, E), generator=gen(5), device=DEV).to(torch.bfloat16)
    x[5] = 0.0
    x[6, ::2] = -0.0  # (equal to zero: the lower number first)
    x[6, 1::2] = 0.0
    check_route(x, k)


def test_route_experts_that_are_off():
    x = torch.randn(100, 24, generator=gen(7), device=DEV)
    x[:, 3] = -math.inf
    x[10] = -math.inf              # a token of padding
    x[11, :22] = -math.inf         # fewer than k left
    x[12] = math.nan
    x[13, ::2] = math.nan
    x[14] = -3.0e38                # the lowest values are values
    x[15] = torch.finfo(torch.float32).min
    x[99] = -math.inf
    for renorm in (True, False):
        got = check_route(x, 6, renorm)
        assert (got[0][10] == -1).all() and (got[1][10] == 0).all() and (got[4][10] == -1).all()
    check_route(torch.full((9, 5), -math.inf, device=DEV), 2)


def test_route_rows_of_a_wider_matrix_and_no_tokens():
    wide = torch.randn(70, 100, generator=gen(8), device=DEV)
    check_route(wide[:, 3:67], 5)
    check_route(wide[::2, :64], 5)
    ids, w, offsets, row_token, token_row = fp8.fp8_moe_route(wide[:0, :64], 4)
    clean()
    assert ids.shape == (0, 4) and row_token.numel() == 0 and (offsets == 0).all() and offsets.numel() == 65


def test_route_all_tokens_to_one_expert():
    x = torch.zeros(3001, 40, device=DEV)
    x[:, 17] = 9.0
    check_route(x, 1)


def test_route_writes_into_given_tensors():
    x = torch.randn(50, 16, generator=gen(9), device=DEV)
    out = dict(expert_ids=torch.empty(50, 3, dtype=torch.int32, device=DEV),
               weights=torch.empty(50, 3, device=DEV), offsets=torch.empty(17, dtype=torch.int32, device=DEV),
               row_token=torch.empty(150, dtype=torch.int32, device=DEV),
               token_row=torch.empty(50, 3, dtype=torch.int32, device=DEV))
    got = fp8.fp8_moe_route(x, 3, **out)
    for a, b in zip(got, out.values()):
        assert a.data_ptr() == b.data_ptr()
    for a, b in zip(got, fp8.fp8_moe_route(x, 3)):
        assert torch.equal(a, b)


# ------------------------------------------------------------------------------------- products

def weights(g, E, N, K):
    wq = (torch.randn(E, N, K, generator=g, device=DEV) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    s_w = (0.5 + torch.rand(E, N, generator=g, device=DEV)) / (100 * K ** 0.5)
    return wq, s_w


def bounds(counts, start=0):
    at = [start]
    for c in counts:
        at.append(at[-1] + c)
    return torch.tensor(at, dtype=torch.int32, device=DEV)


def check_grouped(counts, N, K, swiglu, seed=0, start=0, extra=0):
    g = gen(seed + 17 * N + K)
    E, R = len(counts), start + sum(counts) + extra
    wq, s_w = weights(g, E, N, K)
    xq = (torch.randn(R, K, generator=g, device=DEV) * 100).clamp(-448, 448).to(torch.float8_e4m3fn)
    s_tok = (0.5 + torch.rand(R, generator=g, device=DEV)) / 100
    offsets = bounds(counts, start)
    F = N // 2 if swiglu else N
    y = torch.full((R, F), 7.0, dtype=torch.bfloat16, device=DEV)
    fp8.fp8_grouped_gemm(xq.view(torch.uint8), s_tok, wq.view(torch.uint8), s_w, offsets, swiglu=swiglu, y=y)
    clean()
    want, tol = ref.grouped(xq, s_tok, wq, s_w, offsets, swiglu)
    end = start + sum(counts)
    within(y[start:end], want[start:end], tol[start:end], "y")
    assert (y[:start] == 7).all() and (y[end:] == 7).all(), "rows outside the groups were written"
    again = torch.empty_like(y)
    fp8.fp8_grouped_gemm(xq.view(torch.uint8), s_tok, wq.view(torch.uint8), s_w, offsets, swiglu=swiglu, y=again)
    assert torch.equal(again[start:end], y[start:end])
    return y


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("counts", [[1], [0, 1, 0], [2, 0, 0, 3], [32] * 4, [33, 1, 64, 0, 127], [128, 129, 5],
                                    [255, 256, 257], [0, 0, 700, 1], [0, 0, 0]])
def test_grouped_sizes_of_groups(counts, swiglu):
    check_grouped(counts, 320, 272, swiglu)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("N,K", [(2, 16), (8, 32), (16, 128), (34, 144), (256, 256), (258, 1024), (512, 528),
                                 (1026, 400)])
def test_grouped_sizes_of_weights(N, K, swiglu):
    check_grouped([3, 0, 40, 17, 1, 200], N, K, swiglu)


@pytest.mark.parametrize("N,K", [(1, 16), (3, 64), (127, 256), (129, 2048), (257, 128)])
def test_grouped_odd_outputs(N, K):
    check_grouped([5, 130, 0, 61], N, K, False)


@pytest.mark.parametrize("swiglu", [False, True])
def test_grouped_long_sums_of_few_rows(swiglu):
    # few tiles: the sums are split over the SMs
    check_grouped([1, 0, 1], 512, 16384, swiglu)
    check_grouped([0, 60, 5], 256, 8192 + 16, swiglu)
    check_grouped([300], 256, 4096, swiglu)


@pytest.mark.parametrize("swiglu", [False, True])
def test_grouped_rows_outside_stay_as_they_are(swiglu):
    check_grouped([4, 0, 30], 96, 160, swiglu, start=5, extra=9)
    check_grouped([200, 100], 512, 4096, swiglu, start=1, extra=300)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("N", [2, 62, 64, 66, 126, 128, 130, 200, 254, 258, 384, 642])
def test_grouped_many_rows_of_few_outputs(N, swiglu):
    # tiles over two SMs; experts that end in each part of a tile
    check_grouped([400, 130, 20, 256, 0, 385], N, 400, swiglu)


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("K", [16, 32, 112, 128, 144, 272, 1008, 4112])
def test_grouped_many_rows_of_any_depth(K, swiglu):
    check_grouped([290, 129, 128, 511], 288, K, swiglu)


@pytest.mark.parametrize("swiglu", [False, True])
def test_grouped_cut_tiles_of_many_rows(swiglu):
    # one round of few tiles with long sums: cut, each part of up to 256 rows
    check_grouped([256], 256, 32768, swiglu)
    check_grouped([700, 140, 20], 320, 16384 + 48, swiglu)


@pytest.mark.parametrize("rows", [3, 300])
def test_grouped_gates_of_any_size(rows):
    # gates from -inf over +-120 to inf, and values beside them: one product a row and column
    K, F = 16, 64
    xq = torch.zeros(rows, K, device=DEV)
    xq[:, 0] = 1.0
    gates = torch.cat([torch.linspace(-120, 120, F - 8, device=DEV),
                       torch.tensor([0.0, -0.0, 1e-30, -1e-30, -87.5, -88.5, -103.0, 3e38], device=DEV)])
    wq = torch.zeros(1, 2 * F, K, device=DEV)
    wq[0, :, 0] = 1.0
    s_w = torch.cat([gates, torch.full((F,), 1.5, device=DEV)])[None]  # (scales stand for the values)
    s_tok = torch.ones(rows, device=DEV)
    f8 = torch.float8_e4m3fn
    y = fp8.fp8_grouped_gemm(xq.to(f8).view(torch.uint8), s_tok, wq.to(f8).view(torch.uint8), s_w, bounds([rows]),
                             swiglu=True)
    g = gates.double()
    want = torch.where(g >= 0, g / (1 + torch.exp(-g.abs())), g * torch.exp(-g.abs()) / (1 + torch.exp(-g.abs()))) * 1.5
    # exp of an argument of up to 120: rounded to 2^-24 of it, 2^-17; the rest is within 2^-20; below
    # the normal numbers (of fp32 and bf16) half a step
    tol = want.abs() * (ref.HALF["bf16"] + 2.0 ** -16) + 2.0 ** -133
    # (4.5e38 lies beyond the largest bf16, 3.39e38 and half a step: infinity)
    far = want.abs() > 3.4e38
    assert far.sum() == 1 and torch.isinf(y[:, far].float()).all()
    within(y[:, ~far], want[~far].expand(rows, -1), tol[~far].expand(rows, -1), "y")
    clean()


def test_grouped_rows_without_any_group():
    check_grouped([0, 0, 0], 64, 128, False, start=3, extra=5)
    check_grouped([0], 64, 128, True, start=0, extra=700)


def test_grouped_workspace_need_not_be_clean():
    g = gen(21)
    wq, s_w = weights(g, 4, 256, 8192)
    xq = torch.randint(0, 120, (70, 8192), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.ones(70, device=DEV) * 1e-4
    x = normal(g, 70, 8192)
    w8 = wq.view(torch.uint8)
    need = max(fp8.fp8_grouped_gemm_workspace_size(4, 70, 256, 8192), fp8.fp8_grouped_linear_workspace_size(4, 70, 256, 8192))
    ws = torch.empty(need, dtype=torch.uint8, device=DEV)
    for counts in ([70, 0, 0, 0], [1, 2, 3, 64], [30, 30, 5, 5]):
        off = bounds(counts)
        good = fp8.fp8_grouped_gemm(xq, s, w8, s_w, off), fp8.fp8_grouped_linear(x, w8, s_w, off)
        for fill in (0, 255, 1):
            ws.fill_(fill)
            assert torch.equal(fp8.fp8_grouped_gemm(xq, s, w8, s_w, off, workspace=ws), good[0])
            assert torch.equal(fp8.fp8_grouped_gemm(xq, s, w8, s_w, off, workspace=ws), good[0])
            ws.fill_(fill)
            assert torch.equal(fp8.fp8_grouped_linear(x, w8, s_w, off, workspace=ws), good[1])
            assert torch.equal(fp8.fp8_grouped_linear(x, w8, s_w, off, workspace=ws), good[1])
    clean()


def test_grouped_many_experts():
    counts = [(7 * i) % 5 for i in range(1024)]
    check_grouped(counts, 48, 64, False)
    check_grouped(counts, 48, 64, True)


@pytest.mark.parametrize("swiglu", [False, True])
def test_grouped_large(swiglu):
    check_grouped([511, 0, 1025, 258, 64, 1900], 2304, 1040, swiglu)


def test_grouped_rows_do_not_depend_on_their_neighbours():
    # the same rows and weights among others; NaN codes in a neighbouring group stay there
    g = gen(3)
    wq, s_w = weights(g, 3, 160, 512)
    xq = (torch.randn(90, 512, generator=g, device=DEV) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    s = torch.ones(90, device=DEV) * 0.01
    w8 = wq.view(torch.uint8)
    y = fp8.fp8_grouped_gemm(xq, s, w8, s_w, bounds([30, 30, 30]))
    bad = xq.clone()
    bad[:30] = 0x7F
    bad[60:] = 0xFF
    z = fp8.fp8_grouped_gemm(bad, s, w8, s_w, bounds([30, 30, 30]))
    clean()
    assert torch.equal(y[30:60], z[30:60])
    assert torch.isnan(z[:30].float()).all() and torch.isnan(z[60:].float()).all()


def test_grouped_bounds_outside_the_rows_are_cut():
    g = gen(4)
    wq, s_w = weights(g, 3, 64, 128)
    xq = torch.randint(0, 120, (20, 128), generator=g, device=DEV, dtype=torch.uint8)
    s = torch.ones(20, device=DEV) * 0.01
    w8 = wq.view(torch.uint8)
    good = fp8.fp8_grouped_gemm(xq, s, w8, s_w, bounds([6, 4, 10]))
    off = torch.tensor([-5, 6, 10, 1 << 30], dtype=torch.int32, device=DEV)
    assert torch.equal(fp8.fp8_grouped_gemm(xq, s, w8, s_w, off), good)
    clean()


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("T,E,k,K,N", [(1, 8, 2, 256, 128), (33, 8, 3, 1040, 320), (300, 5, 1, 64, 64), (64, 16, 8, 4096, 96)])
def test_grouped_linear_is_its_parts(T, E, k, K, N, swiglu):
    g = gen(T + K)
    wq, s_w = weights(g, E, N, K)
    x = normal(g, T, K + 16)[:, 8:K + 8]  # rows of a wider matrix
    x[0] = 0
    _, _, offsets, row_token, _ = fp8.fp8_moe_route(torch.randn(T, E, generator=g, device=DEV), k)
    y = fp8.fp8_grouped_linear(x, wq.view(torch.uint8), s_w, offsets, row_token=row_token, swiglu=swiglu)
    xq, s = fp8.fp8_quant_per_token(x[row_token.long()].contiguous())
    assert torch.equal(y, fp8.fp8_grouped_gemm(xq, s, wq.view(torch.uint8), s_w, offsets, swiglu=swiglu))
    z = fp8.fp8_grouped_linear(x[row_token.long()], wq.view(torch.uint8), s_w, offsets, swiglu=swiglu)
    assert torch.equal(y, z)
    codes, s_ref = ref.quant(x[row_token.long()])
    assert torch.equal(s, s_ref) and torch.equal(xq, codes.view(torch.uint8))
    want, tol = ref.grouped(codes, s_ref, wq, s_w, offsets, swiglu)
    within(y, want, tol, "y")
    clean()


def test_grouped_linear_rows_without_a_token_are_zeros():
    g = gen(11)
    wq, s_w = weights(g, 2, 64, 128)
    x = normal(g, 10, 128)
    rows = torch.tensor([3, -1, 9, 10, 0, 1 << 30], dtype=torch.int32, device=DEV)
    y = fp8.fp8_grouped_linear(x, wq.view(torch.uint8), s_w, bounds([3, 3]), row_token=rows)
    clean()
    assert (y[[1, 3, 5]] == 0).all()
    full = fp8.fp8_grouped_linear(x[[3, 9, 0]], wq.view(torch.uint8), s_w, bounds([2, 1]))
    assert torch.equal(y[[0, 2, 4]], full)
    assert fp8.fp8_grouped_linear(x[:0], wq.view(torch.uint8), s_w, bounds([0, 0])).shape == (0, 64)
    none = fp8.fp8_grouped_linear(x[:0], wq.view(torch.uint8), s_w, bounds([3, 3]), row_token=rows)
    clean()
    assert (none == 0).all()


def test_grouped_linear_long_rows():
    # rows that the quantizer streams
    g = gen(12)
    K = 65536 + 64
    wq, s_w = weights(g, 2, 32, K)
    x = normal(g, 3, K)
    rows = torch.tensor([2, 0, -1, 1], dtype=torch.int32, device=DEV)
    offsets = bounds([1, 3])
    y = fp8.fp8_grouped_linear(x, wq.view(torch.uint8), s_w, offsets, row_token=rows)
    codes, s = ref.quant(x)
    pick = torch.tensor([2, 0, 0, 1], device=DEV)
    codes, s = codes.view(torch.uint8)[pick].clone(), s[pick].clone()
    codes[2], s[2] = 0, 1
    want, tol = ref.grouped(codes.view(torch.float8_e4m3fn), s, wq, s_w, offsets, False)
    within(y, want, tol, "y")
    clean()


# ------------------------------------------------------------------------------------- the join

def check_join(T, K, k, post, gate, rows=True, codes=True, rs=1.0, bs=1.0, seed=0, eps=1e-6, weighted=True, holes=False,
               ld=0):
    g = gen(seed + T + 7 * K + k)
    h = normal(g, T, K + ld, scale=4.0)[:, :K]
    R = T * k if k else T
    y = normal(g, R, K + 2 * ld)[:, ld:K + ld]
    token_row = w = None
    if k:
        token_row = torch.randperm(R, generator=g, device=DEV).view(T, k).int()
        if holes:
            token_row[torch.rand(T, k, generator=g, device=DEV) < 0.3] = -1
            token_row[0] = -1
            token_row[T // 2, 0] = R
        w = torch.rand(T, k, generator=g, device=DEV) if weighted else None
    gamma = normal(g, K, scale=0.1) + 1
    gp = normal(g, K, scale=0.1) + 1 if post else None
    gt = {"none": None, "channel": normal(g, K), "token": normal(g, T, K + ld)[:, :K]}[gate]
    got = fp8.fp8_residual_norm_quant(h, y, gamma if rows or codes else None, eps=eps, gamma_post=gp, gate=gt,
                                      residual_scale=rs, branch_scale=bs, token_row=token_row, weights=w, rows=rows,
                                      codes=codes)
    clean()
    out, z, s, th, tz, ts = ref.residual_norm(h, y, gamma, eps, gp, gt, rs, bs, token_row, w)
    within(got[0], out, th, "h_out")
    if rows:
        within(got[1], z, tz, "z")
    else:
        assert got[1] is None
    if codes:
        within(got[3], s, ts, "s_tok")
        value = got[2].view(torch.float8_e4m3fn).double() * got[3][:, None].double()
        # half a step of the codes, or half a subnormal step
        room = tz + z.abs() * (ref.HALF["e4m3"] + 2.0 ** -20) + got[3][:, None].double() * 2.0 ** -10
        within(value, z, room, "codes")
        assert (got[2].view(torch.float8_e4m3fn).float().abs().amax(1) == 448).all() or T == 0 or K < 16
    else:
        assert got[2] is None and got[3] is None
    return (h, y, gamma, gp, gt, token_row, w), got


@pytest.mark.parametrize("T", [1, 3, 64, 501])
@pytest.mark.parametrize("K", [16, 256, 272, 528, 1040, 2880, 4096, 8192 - 16, 16384 - 16, 32768])
def test_join_widths(T, K):
    check_join(T, K, 2 if T % 2 else 0, post=K % 32 == 0, gate=["none", "channel", "token"][T % 3])


@pytest.mark.parametrize("k", [0, 1, 2, 4, 7, 32])
@pytest.mark.parametrize("gate", ["none", "channel", "token"])
@pytest.mark.parametrize("post", [False, True])
def test_join_forms(k, gate, post):
    check_join(37, 544, k, post, gate, rs=0.5, bs=0.22, weighted=k != 2)


@pytest.mark.parametrize("rows,codes", [(False, False), (True, False), (False, True)])
def test_join_outputs_that_are_left_out(rows, codes):
    check_join(21, 1024, 2, True, "channel", rows, codes)
    check_join(21, 1024, 0, False, "none", rows, codes)


def test_join_tokens_without_rows():
    check_join(40, 512, 3, False, "none", holes=True)
    check_join(40, 512, 3, True, "token", holes=True)
    h = torch.zeros(3, 64, dtype=torch.bfloat16, device=DEV)
    y = torch.zeros(0, 64, dtype=torch.bfloat16, device=DEV)
    none = torch.full((3, 2), -1, dtype=torch.int32, device=DEV)
    one = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    out, z, xq, s = fp8.fp8_residual_norm_quant(h, y, one, token_row=none, gamma_post=one)
    clean()
    assert (out == 0).all() and (z == 0).all() and (xq == 0).all() and (s == 1).all()


def test_join_rows_of_wider_matrices():
    check_join(19, 320, 2, True, "token", ld=16)
    check_join(19, 320, 0, False, "channel", ld=8)


def test_join_values_in_skipped_rows_do_not_matter():
    g = gen(2)
    h, y, one = normal(g, 4, 64), normal(g, 8, 64), torch.ones(64, dtype=torch.bfloat16, device=DEV)
    rows = torch.tensor([[0, -1], [2, 3], [-1, -1], [7, 5]], dtype=torch.int32, device=DEV)
    a = fp8.fp8_residual_norm_quant(h, y, one, token_row=rows)
    y[[1, 4, 6]] = math.nan
    b = fp8.fp8_residual_norm_quant(h, y, one, token_row=rows)
    for p, q in zip(a, b):
        assert torch.equal(p, q)
    y[2] = math.inf  # a token's own values are its own
    c = fp8.fp8_residual_norm_quant(h, y, one, token_row=rows)
    clean()
    for i, (p, q) in enumerate(zip(a, c)):
        assert torch.equal(p[[0, 2, 3]], q[[0, 2, 3]])
    assert torch.isinf(c[0][1].float()).all()


def test_join_in_place():
    (h, y, gamma, gp, gt, rows, w), got = check_join(33, 768, 2, True, "channel")
    again = h.clone()
    out = fp8.fp8_residual_norm_quant(again, y, gamma, gamma_post=gp, gate=gt, token_row=rows, weights=w, h_out=again)
    clean()
    assert out[0].data_ptr() == again.data_ptr()
    for p, q in zip(out, got):
        assert torch.equal(p, q)


def test_join_sizes_of_zero():
    h = torch.zeros(0, 64, dtype=torch.bfloat16, device=DEV)
    one = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    out = fp8.fp8_residual_norm_quant(h, h, one)
    assert [t.shape[0] for t in out] == [0, 0, 0, 0]


def test_join_small_and_large_values():
    # scales below the normal numbers, and rows whose squares leave bf16 but not fp32
    for scale in (1e-30, 1e15):
        g = gen(6)
        h = normal(g, 5, 256, scale=scale)
        gamma = torch.ones(256, dtype=torch.bfloat16, device=DEV)
        y = normal(g, 5, 256, scale=scale)
        got = fp8.fp8_residual_norm_quant(h, y, gamma, eps=1e-6)
        out, z, s, th, tz, ts = ref.residual_norm(h, y, gamma, 1e-6, None, None, 1.0, 1.0, None, None)
        within(got[0], out, th, "h_out")
        within(got[1], z, tz, "z")
        within(got[3], s, ts, "s_tok")
        clean()
