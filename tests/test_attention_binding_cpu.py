"""Refusals of the attention block's Python binding that come before any tensor
is looked at, so they can be seen without a GPU."""
import pytest
import torch


@pytest.fixture(scope="module")
def pkg():
    from fp8_w8a8_quantized_gb300 import build
    build.build()
    import fp8_w8a8_quantized_gb300 as pkg
    return pkg


@pytest.mark.parametrize("room", [-1, 1 << 31, 1 << 40, 1 << 61, (1 << 63) - 1])
def test_slots_refuse_room_that_the_call_cannot_have(pkg, room):
    # (before anything of that size is allocated, or its bytes are counted in 64 bits)
    n = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="max_tokens must be"):
        pkg.fp8_kv_slots(n, n, n, 16, n[:, None], room)


@pytest.mark.parametrize("name", ["interleaved", "cache_only"])
def test_rotation_refuses_what_is_neither_true_nor_false(pkg, name):
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i32, i64 = torch.zeros(4, dtype=torch.int32), torch.zeros(32, dtype=torch.int64)
    with pytest.raises(ValueError, match=name + " must be true or false"):
        pkg.fp8_qk_norm_rope(x, x, i32, i64, **{name: torch.zeros(2)})
