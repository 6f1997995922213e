"""Refusals of the attention block's calls, on the host: each rejected call
answers before anything is launched, so no GPU is needed."""
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


SLOTS = dict(ctx=P, new=P, B=4, free=P, n_free=9, page=16, table=P, width=8, ld=8, T=32, slot=P, pos=P,
             cu=P, lens=P, used=P, stream=None)
ROPE = dict(q=P, ldq=512, k=P, ldk=128, v=P, ldv=128, T=4, Hq=8, Hkv=2, D=64, gq=P, gk=P, eps=1e-6, pos=P,
            turns=P, rot=64, inter=0, qo=P, ldqo=512, ko=P, ldko=128, ks=P, vs=P, stride=1, slot=P, kc=P, vc=P,
            n_slots=64, stream=None)
PROMPT = dict(q=P, ldq=512, k=P, ldk=128, v=P, ldv=128, T=40, Hq=8, Hkv=2, D=64, cu=P, S=2, scale=0.125,
              out=P, ldo=512, stream=None)
DECODE = dict(q=P, ldq=512, B=3, Hq=8, Hkv=2, D=64, kc=P, vc=P, n_slots=640, ks=P, vs=P, stride=1, table=P,
              width=8, ld=8, page=16, lens=P, prefix=0, scale=0.125, out=P, ldo=512, ws=P, bytes=1 << 30,
              stream=None)


@pytest.mark.parametrize("changed,want", [
    (dict(B=-1), INVALID), (dict(n_free=-1), INVALID), (dict(page=0), INVALID), (dict(T=-1), INVALID),
    (dict(width=-1), INVALID), (dict(T=1 << 31), INVALID), (dict(ctx=None), INVALID), (dict(new=None), INVALID),
    (dict(free=None), INVALID), (dict(table=None), INVALID), (dict(ld=7), INVALID), (dict(slot=None), INVALID),
    (dict(pos=None), INVALID), (dict(cu=None), INVALID), (dict(lens=None), INVALID), (dict(used=None), INVALID),
    (dict(ctx=P + 2), UNSUP), (dict(slot=P + 4), UNSUP), (dict(table=P + 1), UNSUP)])
def test_slots_refusals(L, changed, want):
    assert call(L.fp8_kv_slots, SLOTS, **changed) == want


@pytest.mark.parametrize("changed,want", [
    (dict(T=-1), INVALID), (dict(rot=80), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=math.nan), INVALID),
    (dict(eps=math.inf), INVALID), (dict(D=40, rot=0), UNSUP), (dict(D=272, rot=0), UNSUP), (dict(rot=24), UNSUP),
    (dict(Hq=65536), UNSUP), (dict(pos=None), INVALID), (dict(turns=None), INVALID), (dict(kc=None), INVALID),
    (dict(vc=None), INVALID), (dict(ks=None), INVALID), (dict(vs=None), INVALID), (dict(v=None), INVALID),
    (dict(kc=None, vc=None, ko=None), INVALID), (dict(q=None), INVALID), (dict(qo=None), INVALID),
    (dict(ldq=504), INVALID), (dict(ldq=516), UNSUP), (dict(ldko=120), INVALID), (dict(q=P + 8), UNSUP),
    (dict(ko=P + 8), UNSUP), (dict(v=P + 8), UNSUP), (dict(gq=P + 2), UNSUP), (dict(turns=P + 4), UNSUP),
    (dict(pos=P + 2), UNSUP), (dict(kc=P + 4), UNSUP), (dict(slot=P + 4), UNSUP), (dict(stride=-1), INVALID),
    (dict(n_slots=-1), INVALID), (dict(T=0), 0), (dict(Hq=0, Hkv=0), 0)])
def test_rope_refusals(L, changed, want):
    assert call(L.fp8_qk_norm_rope, ROPE, **changed) == want


HEADS = [(dict(Hq=7), INVALID), (dict(Hkv=0), INVALID), (dict(Hq=0), INVALID), (dict(D=0), INVALID),
         (dict(D=24), UNSUP), (dict(D=144, ldq=2048, ldo=2048), UNSUP), (dict(Hq=130, ldq=1 << 14, ldo=1 << 14), UNSUP),
         (dict(scale=0.0), INVALID), (dict(scale=-1.0), INVALID), (dict(scale=math.nan), INVALID),
         (dict(scale=math.inf), INVALID), (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(ldq=504), INVALID),
         (dict(ldq=516), UNSUP), (dict(ldo=504), INVALID), (dict(q=P + 2), UNSUP), (dict(out=P + 8), UNSUP),
         (dict(ldq=1 << 40), INVALID)]


@pytest.mark.parametrize("changed,want", HEADS + [
    (dict(T=-1), INVALID), (dict(S=-1), INVALID), (dict(cu=None), INVALID), (dict(cu=P + 2), UNSUP),
    (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(ldk=120), INVALID), (dict(ldv=132), UNSUP),
    (dict(k=P + 8), UNSUP), (dict(T=(1 << 31) - 1), UNSUP), (dict(T=0), 0), (dict(S=0), 0)])
def test_prompt_refusals(L, changed, want):
    assert call(L.fp8_attention_prompt, PROMPT, **changed) == want


@pytest.mark.parametrize("changed,want", HEADS + [
    (dict(B=-1), INVALID), (dict(page=0), INVALID), (dict(prefix=-1), INVALID), (dict(prefix=129), INVALID),
    (dict(ks=None), INVALID), (dict(vs=None), INVALID), (dict(lens=None), INVALID), (dict(table=None), INVALID),
    (dict(ld=7), INVALID), (dict(kc=None), INVALID), (dict(vc=None), INVALID), (dict(kc=P + 8), UNSUP),
    (dict(ks=P + 2), UNSUP), (dict(lens=P + 2), UNSUP), (dict(table=P + 2), UNSUP), (dict(stride=-1), INVALID),
    (dict(width=1 << 28, ld=1 << 28), UNSUP), (dict(B=1 << 23), UNSUP), (dict(B=0), 0)])
def test_decode_refusals(L, changed, want):
    assert call(L.fp8_attention_decode, DECODE, **changed) == want


def test_decode_workspace(L):
    size = L.fp8_attention_decode_workspace_size
    need = size(3, 8, 2, 64, 8, 16, 0)
    if need:
        assert call(L.fp8_attention_decode, DECODE, ws=None) == WS
        assert call(L.fp8_attention_decode, DECODE, bytes=need - 1) == WS
        assert call(L.fp8_attention_decode, DECODE, ws=P + 128) == WS
    for bad in ((-1, 8, 2, 64, 8, 16, 0), (3, 7, 2, 64, 8, 16, 0), (3, 8, 2, 60, 8, 16, 0), (3, 8, 2, 64, -1, 16, 0),
                (3, 8, 2, 64, 8, 0, 0), (3, 8, 2, 64, 8, 16, 129), (0, 8, 2, 64, 8, 16, 0)):
        assert size(*bad) == 0


def test_calls_that_pass_the_checks_report_a_cuda_error_without_a_device(L):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present; this case needs a machine without one")
    assert call(L.fp8_kv_slots, SLOTS) == CUDA
    assert call(L.fp8_qk_norm_rope, ROPE) == CUDA
    assert call(L.fp8_qk_norm_rope, ROPE, kc=None, vc=None, v=None, ks=None, vs=None, slot=None) == CUDA
    assert call(L.fp8_qk_norm_rope, ROPE, ko=None, gq=None, gk=None) == CUDA
    assert call(L.fp8_attention_prompt, PROMPT) == CUDA
    assert call(L.fp8_attention_decode, DECODE) == CUDA


def test_binding_rejects_tensors_the_kernels_cannot_take():
    import fp8_w8a8_quantized_gb300 as pkg
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    i32, i64 = torch.zeros(4, dtype=torch.int32), torch.zeros(32, dtype=torch.int64)
    codes, one = torch.zeros(64, 2, 64, dtype=torch.uint8), torch.ones(2)
    with pytest.raises(ValueError, match="q must be a CUDA"):
        pkg.fp8_attention_prompt(x, x, x, i32)
    with pytest.raises(ValueError, match="q must be a CUDA"):
        pkg.fp8_attention_decode(x, codes, codes, one, one, i32[:, None], i32, 16)
    with pytest.raises(ValueError, match="q must be a CUDA"):
        pkg.fp8_qk_norm_rope(x, x, i32, i64)
    with pytest.raises(ValueError, match="ctx_lens must be a CUDA"):
        pkg.fp8_kv_slots(i32, i32, i32, 16, i32[:, None], 8)
