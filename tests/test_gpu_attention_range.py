"""GPU tests of decode attention where one token takes nearly all of the weight
and holds a value of zero, as a first token often does: what the others say is
all that is left, with weights far below the largest one.  Tolerances as in
test_gpu_attention_prefix.py, derived before the first run: each weight is
rounded to f16, 2^-11 of its share of the weighted |v|, wherever it lies above
2^-21 of the largest weight."""
import math

import pytest
import torch

import attention_ref as ref
from test_gpu_attention_prefix import DEV, cached, decode, formula, settled

CASES = [(200, 16, 8, 64, 16, 0, 2000), (160, 32, 8, 128, 16, 0, 1200), (24, 32, 8, 128, 16, 8192, 40),
         (128, 16, 8, 64, 16, 8000, 40)]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("log2", [-12.3, -16.6, -20.6])
def test_one_token_takes_nearly_all(case, log2):
    B, Hq, Hkv, D, page, prefix, own = case
    args = cached(17, B, Hq, Hkv, D, page, prefix, own=own)
    q, kc, vc, ks, vs, table, lens = args
    lens.fill_(prefix + own - 1)
    # keys are zero but token 0's, whose score is -log2 in log2 units for every query
    kc.zero_()
    first = table[:, 0].long() * page
    kc[first, :, 0] = 0x38                     # 1.0
    ks.fill_(1.0)
    q.zero_()
    q[:, :, 0] = 1.0
    vc.fill_(0x38)
    vc[first] = 0
    scale = -log2 * math.log(2.0)
    got = decode(args, page, prefix, scale=scale)
    settled()
    want, size = formula(*args, page, prefix, scale=scale)
    assert torch.isfinite(want).all() and (want > 0).all()
    ref.check(got, want, ref.U_BF16 * want.abs() + (ref.U_FP16 + ref.SUMS) * size, "sink")
