"""The operators together, as examples/attention_block.py runs them: prompts,
a shared beginning, and steps over the cache.  What the block attends to is
checked against the plain 64-bit forms on the block's own queries and cache
(tolerances as in test_gpu_attention.py), the cache against the cache writer
bit for bit."""
import importlib.util
import os

import pytest
import torch

import attention_ref as ref
import fp8_w8a8_quantized_gb300 as pkg
from conftest import ROOT

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("attention_block",
                                                  os.path.join(ROOT, "examples", "attention_block.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def settled():
    torch.cuda.synchronize()
    assert pkg.fp8_device_status() == pkg.FP8_OK


@pytest.mark.parametrize("q_heads,kv_heads,dim,page,norm", [(8, 2, 64, 16, True), (6, 3, 80, 20, False),
                                                            (4, 4, 128, 32, True)])
def test_prompts_then_steps(example, q_heads, kv_heads, dim, page, norm):
    lens = [37, 1, 130, 64]
    block = example.AttentionBlock(hidden=256, q_heads=q_heads, kv_heads=kv_heads, dim=dim, pages=64,
                                   page_size=page, requests=4, table_width=16, norm=norm)
    g = torch.Generator(device=DEV)
    g.manual_seed(3)
    x = torch.randn(sum(lens), 256, generator=g, device=DEV).to(torch.bfloat16)
    new = torch.tensor(lens, dtype=torch.int32, device=DEV)

    slots, positions, cu, _ = block.place(new, x.shape[0])
    q, k, v = block.project(x, positions, slots, cache_only=False)
    attended = pkg.fp8_attention_prompt(q, k, v, cu)
    settled()
    want, size = ref.prompt(q, k, v, cu, dim ** -0.5)
    ref.check(attended, want, ref.U_BF16 * want.abs() + (ref.U_BF16 + ref.SUMS) * size, "prompt")
    assert positions.tolist() == [i for n in lens for i in range(n)]
    # the cache holds what the cache writer would have written
    kc, vc = torch.zeros_like(block.k_cache), torch.zeros_like(block.v_cache)
    pkg.fp8_kv_cache_quant_kv(k, v.contiguous(), block.k_scale, block.v_scale, kc, vc, slot_mapping=slots)
    settled()
    assert torch.equal(kc, block.k_cache) and torch.equal(vc, block.v_cache)

    for step in range(3):
        x = torch.randn(4, 256, generator=g, device=DEV).to(torch.bfloat16)
        one = torch.ones(4, dtype=torch.int32, device=DEV)
        slots, positions, _, now = block.place(one, 4)
        assert positions.tolist() == [n + step for n in lens] and now.tolist() == [n + step + 1 for n in lens]
        q, none, _ = block.project(x, positions, slots, cache_only=True)
        assert none is None
        got = pkg.fp8_attention_decode(q, block.k_cache, block.v_cache, block.k_scale, block.v_scale, block.table,
                                       now, page)
        settled()
        want, size = ref.decode(q, block.k_cache, block.v_cache, block.k_scale, block.v_scale, block.table, now,
                                page, 0, dim ** -0.5)
        ref.check(got, want, ref.U_BF16 * want.abs() + (ref.U_FP16 + ref.SUMS) * size, "decode")
        assert torch.isfinite(block.output(x, got)).all()


def test_shared_system_prompt(example):
    block = example.AttentionBlock(hidden=256, q_heads=8, kv_heads=8, dim=64, pages=400, requests=120,
                                   table_width=120)
    g = torch.Generator(device=DEV)
    g.manual_seed(4)
    x = torch.randn(1700, 256, generator=g, device=DEV).to(torch.bfloat16)
    y = block.prompt(x, torch.tensor([1700], dtype=torch.int32, device=DEV), slice(0, 1))
    shared = block.share(1700)
    assert shared == 1696 and torch.isfinite(y).all()
    for _ in range(2):
        x = torch.randn(120, 256, generator=g, device=DEV).to(torch.bfloat16)
        slots, positions, _, lens = block.place(torch.ones(120, dtype=torch.int32, device=DEV), 120)
        q, _, _ = block.project(x, positions, slots, cache_only=True)
        got = pkg.fp8_attention_decode(q, block.k_cache, block.v_cache, block.k_scale, block.v_scale, block.table,
                                       lens, 16, prefix_len=shared)
        settled()
        want, size = ref.decode(q, block.k_cache, block.v_cache, block.k_scale, block.v_scale, block.table, lens,
                                16, shared, 64 ** -0.5)
        ref.check(got, want, ref.U_BF16 * want.abs() + (ref.U_FP16 + ref.SUMS) * size, "shared")
    assert torch.isfinite(block.step(x, prefix_len=shared)).all()


def test_the_pool_runs_out(example):
    block = example.AttentionBlock(hidden=256, q_heads=4, kv_heads=2, dim=64, pages=3, requests=2, table_width=8)
    with pytest.raises(RuntimeError, match="4 pages wanted, 3 free"):
        block.place(torch.tensor([30, 20], dtype=torch.int32, device=DEV), 50)
