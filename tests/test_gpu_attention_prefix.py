"""GPU tests of decode attention's shared-prefix kernel where a CTA has three
key tiles and more: its ring of keys and values goes round, running maxima move
on past the second tile, and the prefix ends inside a tile or has pages that do
not exist.  Checked against the 64-bit formula, and every case a hundred times
for the same bits.

Tolerances: bf16's rounding of the result (2^-8), f16's of each weight (2^-11 of
its share of the weighted |v|), 2^-12 of the weighted |v| for fp32 products,
sums and exponentials."""
import pytest
import torch

import attention_ref as ref

DEV = "cuda"

# requests, query heads, key heads, dim, page, prefix
CASES = [(24, 32, 8, 128, 16, 8200), (64, 8, 8, 64, 16, 12000), (128, 16, 8, 64, 16, 8016),
         (100, 32, 8, 64, 20, 3001), (64, 64, 8, 128, 16, 4001), (33, 8, 8, 64, 7, 20001),
         (24, 32, 32, 64, 1, 4200), (150, 64, 8, 128, 64, 1100), (300, 64, 32, 64, 16, 705),
         (90, 28, 4, 80, 16, 5000)]


def cached(seed, B, Hq, Hkv, D, page, prefix, own=40):
    """Queries, a cache in shuffled pages, a table whose rows share the prefix's whole pages, lengths past it."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    lens = prefix + torch.randint(0, own, (B,), generator=g, device=DEV, dtype=torch.int32)
    width, shared = -(-(prefix + own) // page), prefix // page
    n_pages = shared + B * (width - shared) + 2
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.cat([order[:shared].expand(B, shared),
                       order[shared: shared + B * (width - shared)].view(B, width - shared)], 1).contiguous()
    codes = [(torch.randn(n_pages * page, Hkv, D, generator=g, device=DEV) * 3).to(torch.float8_e4m3fn)
             .view(torch.uint8) for _ in range(2)]
    scales = [torch.rand(Hkv, generator=g, device=DEV) * 0.2 + 0.2 for _ in range(2)]
    q = torch.randn(B, Hq, D, generator=g, device=DEV).to(torch.bfloat16)
    return [q, codes[0], codes[1], scales[0], scales[1], table, lens]


def formula(q, k_cache, v_cache, k_scale, v_scale, table, lens, page, prefix, scale=None):
    """(out, weighted |v|) in 64 bits."""
    values = ref.e4m3_values().to(DEV)
    B, Hq, D = q.shape
    Hkv = k_cache.shape[1]
    n_pages = k_cache.shape[0] // page
    out, size = (torch.zeros(B, Hq, D, dtype=torch.float64, device=DEV) for _ in range(2))
    for b, n in enumerate(lens.tolist()):
        j = torch.arange(max(0, min(n, table.shape[1] * page)), device=DEV)
        pg = torch.where(j < prefix, table[0].long()[j // page], table[b].long()[j // page])
        slots = (pg * page + j % page)[(pg >= 0) & (pg < n_pages)]
        if not slots.numel():
            continue
        k = values[k_cache[slots].long()] * k_scale.double()[:, None]
        v = values[v_cache[slots].long()] * v_scale.double()[:, None]
        s = torch.einsum("hgd,nhd->hgn", q[b].double().view(Hkv, -1, D), k) * (D ** -0.5 if scale is None else scale)
        w = torch.softmax(s, -1)
        out[b] = torch.einsum("hgn,nhd->hgd", w, v).view(Hq, D)
        size[b] = torch.einsum("hgn,nhd->hgd", w, v.abs()).view(Hq, D)
    return out.cpu(), size.cpu()


def settled():
    import fp8_w8a8_quantized_gb300 as pkg
    torch.cuda.synchronize()
    assert pkg.fp8_device_status() == pkg.FP8_OK


def decode(args, page, prefix, **more):
    import fp8_w8a8_quantized_gb300 as pkg
    return pkg.fp8_attention_decode(*args, page, prefix_len=prefix, **more)


def check(args, page, prefix, what, times=100):
    first = decode(args, page, prefix)
    again = [decode(args, page, prefix) for _ in range(times)]
    settled()
    want, size = formula(*args, page, prefix)
    ref.check(first, want, ref.U_BF16 * want.abs() + (ref.U_FP16 + ref.SUMS) * size, what)
    assert all(torch.equal(first, x) for x in again), what


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: "-".join(map(str, c)))
def test_ring(case):
    B, Hq, Hkv, D, page, prefix = case
    args = cached(prefix + D, *case)
    check(args, page, prefix, "whole")
    # pages that do not exist: in the last key tile, in the one two before it, and further on
    table = args[5]
    for tile in {max(0, -(-prefix // 128) - 1 - i) for i in (0, 2, 5, 9, 13)}:
        table[0, (128 * tile + 3) // page] = -1
    check(args, page, prefix, "missing pages")
    # requests that end inside the prefix
    lens = args[6]
    lens[1], lens[2], lens[B // 2], lens[B - 1] = 0, 1, prefix // 2, prefix - 129
    check(args, page, prefix, "short requests")



@pytest.mark.gpu
@pytest.mark.parametrize("case", [CASES[0], CASES[2], CASES[3], CASES[8], CASES[9]], ids=lambda c: "-".join(map(str, c)))
def test_nan_codes_reach_only_the_requests_that_see_them(case):
    B, Hq, Hkv, D, page, prefix = case
    args = cached(prefix + 7, *case)
    lens, row = args[6], args[5][0].tolist()
    g, head, channel = Hq // Hkv, Hkv - 1, D - 3
    # requests that end at many places of the prefix; the others see all of it
    for b in range(1, B, 3):
        lens[b] = (b * 977 + 1) % prefix
    clean = decode(args, page, prefix)
    settled()
    assert torch.isfinite(clean).all()
    # a value that some requests see, in the first key tile, in the middle and at the end
    for tok in (1, prefix // 2, prefix - 1):
        slot = row[tok // page] * page + tok % page
        bad = list(args)
        bad[2] = args[2].clone()
        bad[2][slot, head, channel] = 0xFF
        got = decode(bad, page, prefix)
        settled()
        sees = (lens > tok).cpu()
        assert sees.any() and (tok == 1 or not sees.all())
        mine = torch.zeros(B, Hq, D, dtype=torch.bool)
        mine[sees, head * g: (head + 1) * g, channel] = True
        assert torch.isnan(got.cpu()[mine]).all(), tok
        assert torch.equal(got.cpu()[~mine], clean.cpu()[~mine]), tok
        # and a key: the heads that read it
        bad = list(args)
        bad[1] = args[1].clone()
        bad[1][slot, 0, 5] = 0x7F
        got = decode(bad, page, prefix)
        settled()
        mine = torch.zeros(B, Hq, D, dtype=torch.bool)
        mine[sees, :g] = True
        assert torch.isnan(got.cpu()[mine]).all(), tok
        assert torch.equal(got.cpu()[~mine], clean.cpu()[~mine]), tok
    # values that nobody sees
    bad = list(args)
    bad[2] = args[2].clone()
    keep = int(lens.max())
    lens.clamp_(max=prefix - 300)
    clean = decode(args, page, prefix)
    for tok in range(prefix - 300, prefix):
        bad[2][row[tok // page] * page + tok % page] = 0x7F
    got = decode(bad, page, prefix)
    settled()
    assert keep > prefix and torch.equal(got, clean) and torch.isfinite(got).all()


@pytest.mark.gpu
@pytest.mark.parametrize("case", [CASES[0], CASES[2], CASES[7]], ids=lambda c: "-".join(map(str, c)))
@pytest.mark.parametrize("exponent", [-133, -126, -120])
def test_queries_at_the_end_of_bf16(case, exponent):
    # the largest element of a query is a power of two as small as bf16 has: all weights alike, and the
    # factor that turns products into logarithms of weights has no digits left in fp32
    B, Hq, Hkv, D, page, prefix = case
    args = cached(prefix + 11, *case)
    args[0] = (args[0].float().sign() * 2.0 ** exponent).to(torch.bfloat16)
    assert args[0].any()
    args[3] = torch.full_like(args[3], 2.0 ** -9)
    args[6][1::4] = prefix - 200
    got, alone = decode(args, page, prefix), decode(args, page, 0)
    settled()
    want, size = formula(*args, page, prefix)
    tol = ref.U_BF16 * want.abs() + (ref.U_FP16 + ref.SUMS) * size
    ref.check(got, want, tol, "shared")
    if prefix % page == 0:
        ref.check(alone, want, tol, "alone")


@pytest.mark.gpu
@pytest.mark.parametrize("case", [CASES[0], CASES[2]], ids=lambda c: "-".join(map(str, c)))
def test_a_nan_query_stays_one(case):
    B, Hq, Hkv, D, page, prefix = case
    args = cached(prefix + 13, *case)
    lens = args[6]
    lens[3], lens[4], lens[5] = prefix, prefix + 5, prefix - 1000
    clean = decode(args, page, prefix)
    bad = list(args)
    bad[0] = args[0].clone()
    mine = torch.zeros(B, Hq, D, dtype=torch.bool)
    for b in (3, 4, 5, B - 1):
        bad[0][b, Hq - 2, 1] = float("nan")
        mine[b, Hq - 2] = True
    got = decode(bad, page, prefix)
    settled()
    assert torch.isnan(got.cpu()[mine]).all()
    assert torch.equal(got.cpu()[~mine], clean.cpu()[~mine])
