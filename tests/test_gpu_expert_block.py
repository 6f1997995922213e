"""The expert block's operators together, as a serving step runs them: against
plain forms in 64 bits step by step, captured into a graph, on other streams."""
import os
import sys

import pytest
import torch

import experts_ref as ref
import fp8_w8a8_quantized_gb300 as fp8

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import expert_block  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = "cuda"


def within(got, want, tol):
    off = (got.double() - want).abs() - tol
    assert not torch.isnan(off).any() and (off <= 0).all(), off.max()


def inputs(T, hidden, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return [torch.randn(T, hidden, generator=g, device=DEV).to(torch.bfloat16) for _ in range(2)]


@pytest.mark.parametrize("T,post", [(1, False), (5, True), (64, False), (700, True)])
def test_block_step_by_step(T, post):
    block = expert_block.ExpertBlock(hidden=512, inner=704, experts=12, top=3, post_norm=post)
    h, attended = inputs(T, 512, T)
    h1, z, _, _ = fp8.fp8_residual_norm_quant(h, attended, block.gamma, codes=False)
    out, want_z, _, th, tz, _ = ref.residual_norm(h, attended, block.gamma, 1e-6, None, None, 1.0, 1.0, None, None)
    within(h1, out, th)
    within(z, want_z, tz)
    logits = z @ block.router.t()
    ids, weights, offsets, row_token, token_row = fp8.fp8_moe_route(logits, 3)
    want = ref.route(logits, 3, True, 1.0)
    assert torch.equal(ids.cpu(), want[0]) and torch.equal(offsets.cpu(), want[3])
    assert torch.equal(row_token.cpu(), want[4]) and torch.equal(token_row.cpu(), want[5])
    inner = fp8.fp8_grouped_linear(z, block.w_in, block.s_in, offsets, row_token=row_token, swiglu=True)
    f8 = torch.float8_e4m3fn
    within(inner, *ref.grouped(*ref.quant(z[row_token.long()]), block.w_in.view(f8), block.s_in, offsets, True))
    rows = fp8.fp8_grouped_linear(inner, block.w_out, block.s_out, offsets)
    within(rows, *ref.grouped(*ref.quant(inner), block.w_out.view(f8), block.s_out, offsets, False))
    h2, _, codes, scales = fp8.fp8_residual_norm_quant(h1, rows, block.gamma_next, gamma_post=block.gamma_post,
                                                       token_row=token_row, weights=weights, rows=False)
    out, want_z, s, th, _, ts = ref.residual_norm(h1, rows, block.gamma_next, 1e-6, block.gamma_post, None, 1.0, 1.0,
                                                  token_row, weights)
    within(h2, out, th)
    within(scales, s, ts)
    for a, b in zip(block.forward(h, attended), (h2, codes, scales)):
        assert torch.equal(a, b)
    assert fp8.fp8_device_status() == fp8.FP8_OK


@pytest.mark.parametrize("T", [3, 300])
def test_block_in_a_graph_with_other_inputs_and_routes(T):
    block = expert_block.ExpertBlock(hidden=256, inner=320, experts=9, top=2, post_norm=True)
    h, attended = inputs(T, 256, 1)
    block.forward(h, attended)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block.forward(h, attended)
    for seed in range(4):
        a, b = inputs(T, 256, 10 + seed)
        if seed == 2:  # every token to the same experts
            b[:], a[:] = b[:1].clone(), a[:1].clone()
        h.copy_(a)
        attended.copy_(b)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip(out, block.forward(a, b)):
            assert torch.equal(x, y)
    assert fp8.fp8_device_status() == fp8.FP8_OK


def test_two_blocks_at_once_on_streams_of_their_own():
    blocks = [expert_block.ExpertBlock(hidden=512, inner=640, experts=8, top=2, seed=s) for s in (1, 2)]
    data = [inputs(T, 512, T) for T in (33, 260)]
    want = [b.forward(*d) for b, d in zip(blocks, data)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in blocks]
    for _ in range(10):
        got = []
        for s, b, d in zip(streams, blocks, data):
            with torch.cuda.stream(s):
                got.append(b.forward(*d))
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            for p, q in zip(x, y):
                assert torch.equal(p, q)
    assert fp8.fp8_device_status() == fp8.FP8_OK


def test_calls_take_a_stream():
    s = torch.cuda.Stream()
    block = expert_block.ExpertBlock(hidden=256, inner=256, experts=4, top=2)
    h, y = inputs(40, 256, 3)
    s.wait_stream(torch.cuda.current_stream())
    a = fp8.fp8_moe_route(h[:, :4].float().contiguous(), 2, stream=s)
    b = fp8.fp8_grouped_linear(h, block.w_in, block.s_in, a[2], row_token=a[3], swiglu=True, stream=s)
    c = fp8.fp8_residual_norm_quant(h, y, block.gamma, stream=s.cuda_stream)
    torch.cuda.synchronize()
    d = fp8.fp8_moe_route(h[:, :4].float().contiguous(), 2)
    for p, q in zip(a, d):
        assert torch.equal(p, q)
    assert torch.equal(b, fp8.fp8_grouped_linear(h, block.w_in, block.s_in, d[2], row_token=d[3], swiglu=True))
    for p, q in zip(c, fp8.fp8_residual_norm_quant(h, y, block.gamma)):
        assert torch.equal(p, q)


def test_padded_tokens_make_no_rows():
    block = expert_block.ExpertBlock(hidden=256, inner=256, experts=6, top=2)
    h, _ = inputs(50, 256, 4)
    logits = (h @ block.router.t()).float()
    padded = torch.cat([logits, torch.full((14, 6), -torch.inf, device=DEV)])
    z = torch.cat([h, torch.full((14, 256), float("nan"), dtype=torch.bfloat16, device=DEV)])
    a, b = fp8.fp8_moe_route(logits, 2), fp8.fp8_moe_route(padded, 2)
    assert torch.equal(a[2], b[2]) and torch.equal(a[3], b[3][:100]) and (b[3][100:] == -1).all()
    y = fp8.fp8_grouped_linear(h, block.w_out, block.s_out, a[2], row_token=a[3])
    x = torch.zeros(128, 256, dtype=torch.bfloat16, device=DEV)
    fp8.fp8_grouped_linear(z, block.w_out, block.s_out, b[2], row_token=b[3], y=x)
    assert torch.equal(x[:100], y) and (x[100:] == 0).all()
    big = torch.zeros(64, 256, dtype=torch.bfloat16, device=DEV)
    big[:50] = h
    p = fp8.fp8_residual_norm_quant(h, y, block.gamma, token_row=a[4], weights=a[1])
    q = fp8.fp8_residual_norm_quant(big, x, block.gamma, token_row=b[4], weights=b[1])
    for u, v in zip(p, q):
        assert torch.equal(u, v[:50])
    assert (q[0][50:] == 0).all() and (q[3][50:] == 1).all()
    assert fp8.fp8_device_status() == fp8.FP8_OK


def test_refusals_with_tensors_on_the_gpu():
    h, y = inputs(8, 64, 5)
    one = torch.ones(64, dtype=torch.bfloat16, device=DEV)
    logits = torch.randn(8, 16, device=DEV)
    wq, s_w = torch.zeros(2, 32, 64, dtype=torch.uint8, device=DEV), torch.ones(2, 32, device=DEV)
    offsets = torch.tensor([0, 3, 8], dtype=torch.int32, device=DEV)
    for k in (0, 17, 33):
        with pytest.raises(ValueError, match="top_k"):
            fp8.fp8_moe_route(logits, k)
    with pytest.raises(ValueError, match="weights"):
        fp8.fp8_moe_route(logits, 2, weights=torch.empty(8, 3, device=DEV))
    with pytest.raises(ValueError, match="unit stride"):
        fp8.fp8_moe_route(logits.t(), 2)
    with pytest.raises(ValueError, match="offsets"):
        fp8.fp8_grouped_linear(h, wq, s_w, offsets[:2])
    with pytest.raises(ValueError, match="offsets"):
        fp8.fp8_grouped_linear(h, wq, s_w, offsets.long())
    with pytest.raises(ValueError, match="wq"):
        fp8.fp8_grouped_linear(h[:, :32], wq, s_w, offsets)
    with pytest.raises(ValueError, match="s_w"):
        fp8.fp8_grouped_linear(h, wq, s_w[:, :31], offsets)
    with pytest.raises(ValueError, match="swiglu needs"):
        fp8.fp8_grouped_linear(h, wq[:, :31].contiguous(), s_w[:, :31].contiguous(), offsets, swiglu=True)
    with pytest.raises(ValueError, match="y must"):
        fp8.fp8_grouped_linear(h, wq, s_w, offsets, swiglu=True, y=torch.empty(8, 32, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(fp8.Fp8Error, match="WORKSPACE"):
        fp8.fp8_grouped_linear(h, wq, s_w, offsets, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    with pytest.raises(fp8.Fp8Error, match="UNSUPPORTED"):
        fp8.fp8_grouped_linear(h[:, :40], wq[:, :, :40].contiguous(), s_w, offsets)
    with pytest.raises(ValueError, match="gate"):
        fp8.fp8_residual_norm_quant(h, y, one, gate=one[:32])
    with pytest.raises(ValueError, match="y must"):
        fp8.fp8_residual_norm_quant(h, y[:4], one)
    with pytest.raises(ValueError, match="weights need"):
        fp8.fp8_residual_norm_quant(h, y, one, weights=torch.ones(8, 1, device=DEV))
    with pytest.raises(ValueError, match="gamma must"):
        fp8.fp8_residual_norm_quant(h, y, None)
    with pytest.raises(ValueError, match="rows that do not overlap"):
        fp8.fp8_residual_norm_quant(one[None].expand(8, 64), y, one)
    with pytest.raises(ValueError, match="z needs"):
        fp8.fp8_residual_norm_quant(h, y, one, rows=False, z=torch.empty_like(h))
    with pytest.raises(fp8.Fp8Error, match="INVALID"):
        fp8.fp8_residual_norm_quant(h, y, one, eps=-1.0)
    with pytest.raises(ValueError, match="y must"):
        fp8.fp8_residual_norm_quant(h, y.cpu(), one)
