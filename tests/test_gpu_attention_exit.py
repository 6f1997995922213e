"""Tokens without a slot: their values are fetched but go nowhere.  The caches
stay as they are, queries and keys are turned all the same, and what runs next
in the same shared memory is not disturbed."""
import pytest
import torch

DEV = "cuda"


@pytest.mark.gpu
@pytest.mark.parametrize("T,Hq,Hkv,D", [(3, 4, 8, 128), (2000, 1, 8, 128), (5000, 2, 16, 64)])
def test_no_token_has_a_slot(T, Hq, Hkv, D):
    import fp8_w8a8_quantized_gb300 as pkg
    g = torch.Generator(device=DEV)
    g.manual_seed(T)
    q, k, v = (torch.randn(T, h, D, generator=g, device=DEV).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
    pos = torch.arange(T, dtype=torch.int32, device=DEV)
    turns = pkg.fp8_rope_turns(rot_dim=D)
    one = torch.ones(1, device=DEV)
    kc, vc = (torch.full((64, Hkv, D), 0x41, dtype=torch.uint8, device=DEV) for _ in range(2))
    slot = torch.full((T,), -1, dtype=torch.int64, device=DEV)
    slot[1::2] = 64
    want = pkg.fp8_qk_norm_rope(q, k, pos, turns)
    again = []
    for _ in range(5):
        got = pkg.fp8_qk_norm_rope(q, k, pos, turns, v=v, k_scale=one, v_scale=one, slot_mapping=slot, k_cache=kc,
                                   v_cache=vc)
        again.append((got, pkg.fp8_qk_norm_rope(q, k, pos, turns)))
    torch.cuda.synchronize()
    assert pkg.fp8_device_status() == pkg.FP8_OK
    for got, after in again:
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(after, want))
    assert bool((kc == 0x41).all()) and bool((vc == 0x41).all())
