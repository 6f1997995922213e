"""GPU tests of the attention block: slot maps, norms and rotation, prompt
attention, decode attention over the paged FP8 cache, each against its plain
64-bit form.

Tolerances.  A result rounded to bf16 is off by at most 2^-8 relative.  The
prompt kernel may round each softmax weight to bf16 (2^-8 of its share of the
weighted |v|), the decode kernel to fp16 (2^-11); 2^-12 of the weighted |v|
covers fp32 products, sums and exponentials.  The rotation's terms are fp32
(a relative 2^-19 of |y_a| + |y_b| covers norm, angle, sine and products).
Codes, slots, tables and lengths are equal bit for bit."""
import math
import random

import pytest
import torch

import attention_ref as ref
import fp8_w8a8_quantized_gb300 as pkg

pytestmark = pytest.mark.gpu
DEV = "cuda"


def gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEV).to(torch.bfloat16)


def int32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def settled():
    torch.cuda.synchronize()
    assert pkg.fp8_device_status() == pkg.FP8_OK


# ------------------------------------------------------------------ slot maps

def slot_case(B, max_ctx, max_new, page, seed, spare=0):
    rng = random.Random(seed)
    ctx = [rng.randint(0, max_ctx) for _ in range(B)]
    new = [rng.randint(0, max_new) for _ in range(B)]
    width = -(-(max_ctx + max_new) // page) + spare
    pages = list(range(3 * B * width + 5))
    rng.shuffle(pages)
    table = torch.full((B, width), -7, dtype=torch.int32)
    for b in range(B):
        for j in range(-(-ctx[b] // page)):
            table[b, j] = pages.pop()
    return ctx, new, table, pages


def check_slots(ctx, new, free, page, table, room, table_gpu=None):
    want = ref.slots(torch.tensor(ctx), torch.tensor(new), free, page, table, room)
    t = table.to(DEV) if table_gpu is None else table_gpu
    got = pkg.fp8_kv_slots(int32(ctx), int32(new), int32(free), page, t, room)
    settled()
    assert torch.equal(t.cpu(), want[0]), "block_table"
    for g, w, name in zip(got, want[1:], ("slots", "positions", "cu", "lens", "used")):
        assert g.cpu().tolist() == (w if isinstance(w, list) else [w]), name


@pytest.mark.parametrize("B,max_ctx,max_new,page", [(1, 0, 1, 1), (1, 1000, 300, 16), (7, 50, 1, 16),
                                                    (33, 100, 90, 20), (256, 64, 3, 1), (300, 40, 200, 64),
                                                    (2048, 9, 2, 4), (2049, 9, 2, 4), (5000, 5, 1, 3)])
def test_slots(B, max_ctx, max_new, page):
    ctx, new, table, free = slot_case(B, max_ctx, max_new, page, B + page)
    check_slots(ctx, new, free[:B * max_new + B], page, table, sum(new) + 11)


def test_slots_room_pages_and_table_run_out():
    ctx, new, table, free = slot_case(40, 60, 70, 16, 5)
    check_slots(ctx, new, free, 16, table, sum(new) // 2)          # tokens dropped
    check_slots(ctx, new, free, 16, table, 0)
    check_slots(ctx, new, free[:9], 16, table, sum(new))           # the free list ends
    check_slots(ctx, new, [], 16, table, sum(new))
    check_slots(ctx, new, free, 16, table[:, :3].contiguous(), sum(new))  # table rows full
    check_slots([-5, 3, -1], [2, -4, 0], free[:4], 16, torch.full((3, 2), 9, dtype=torch.int32), 6)
    free_bad = [-1, 4, -3] + free[:100]
    check_slots(ctx, new, free_bad, 16, table, sum(new))


def test_slots_no_requests_and_a_strided_table():
    check_slots([], [], [3], 16, torch.zeros((0, 4), dtype=torch.int32), 5)
    ctx, new, table, free = slot_case(9, 30, 40, 8, 3)
    wide = torch.full((9, table.shape[1] + 5), -9, dtype=torch.int32, device=DEV)
    view = wide[:, : table.shape[1]]
    view.copy_(table)
    check_slots(ctx, new, free, 8, table, sum(new), view)
    assert bool((wide[:, table.shape[1]:] == -9).all())


# ------------------------------------------------------------ norm and rotation

def inv_freq(rot, theta=500000.0):
    return [theta ** (-2.0 * i / rot) for i in range(rot // 2)]


def check_rope(T, Hq, Hkv, D, rot, norm, interleaved, seed, max_pos=131072):
    g = gen(seed)
    qkv = normal(g, T, (Hq + 2 * Hkv) * D)
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
    gq, gk = normal(g, D), normal(g, D)
    pos = torch.randint(0, max_pos, (T,), generator=g, device=DEV, dtype=torch.int32)
    turns = pkg.fp8_rope_turns(rot_dim=rot)
    n_slots = T + 3
    slot = torch.randperm(n_slots, generator=g, device=DEV)[:T]
    slot[::5] = -1
    slot[1::7] = n_slots
    ks = torch.rand(Hkv, generator=g, device=DEV) * 0.02 + 0.01
    vs = torch.rand(Hkv, generator=g, device=DEV) * 0.02 + 0.01
    kc, vc = (torch.full((n_slots, Hkv, D), 0x55, dtype=torch.uint8, device=DEV) for _ in range(2))
    qo, ko = pkg.fp8_qk_norm_rope(q, k, pos, turns, gamma_q=gq if norm else None,
                                  gamma_k=gk if norm else None, eps=1e-5, interleaved=interleaved,
                                  v=v, k_scale=ks, v_scale=vs, slot_mapping=slot, k_cache=kc, v_cache=vc)
    settled()
    for got, x, gamma, name in ((qo, q, gq, "q"), (ko, k, gk, "k")):
        want, size = ref.norm_rope(x, pos, inv_freq(rot), gamma if norm else None, 1e-5, interleaved)
        ref.check(got, want, ref.U_BF16 * want.abs() + 2.0 ** -19 * size, name)
    kc2, vc2 = (torch.full((n_slots, Hkv, D), 0x55, dtype=torch.uint8, device=DEV) for _ in range(2))
    pkg.fp8_kv_cache_quant_kv(ko, v.contiguous(), ks, vs, kc2, vc2, slot_mapping=slot)
    settled()
    assert torch.equal(kc, kc2) and torch.equal(vc, vc2)
    # the cache alone, and in place: the same bits
    kc3, vc3 = (torch.full((n_slots, Hkv, D), 0x55, dtype=torch.uint8, device=DEV) for _ in range(2))
    more = dict(gamma_q=gq if norm else None, gamma_k=gk if norm else None, eps=1e-5, interleaved=interleaved)
    q2, none = pkg.fp8_qk_norm_rope(q, k, pos, turns, v=v, k_scale=ks, v_scale=vs, slot_mapping=slot,
                                    k_cache=kc3, v_cache=vc3, cache_only=True, **more)
    assert none is None
    pkg.fp8_qk_norm_rope(q, k, pos, turns, q_out=q, k_out=k, **more)
    settled()
    assert torch.equal(kc, kc3) and torch.equal(vc, vc3) and torch.equal(q2, qo)
    assert torch.equal(q, qo) and torch.equal(k, ko)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("T,Hq,Hkv,D,rot,norm", [(1, 1, 1, 16, 16, True), (3, 5, 1, 32, 32, False),
                                                 (37, 14, 2, 64, 32, True), (5, 6, 3, 80, 80, True),
                                                 (9, 4, 4, 96, 32, False), (130, 32, 8, 128, 128, True),
                                                 (8, 9, 3, 256, 64, True), (6, 3, 1, 128, 0, True),
                                                 (700, 8, 2, 112, 96, False)])
def test_norm_rope(T, Hq, Hkv, D, rot, norm, interleaved):
    check_rope(T, Hq, Hkv, D, rot, norm, interleaved, T + D)


def test_norm_rope_far_positions_one_gamma_and_single_scales():
    g = gen(8)
    q, k = normal(g, 50, 4, 64), normal(g, 50, 2, 64)
    pos = torch.randint(0, 2 ** 31 - 1, (50,), generator=g, device=DEV, dtype=torch.int32)
    gamma = normal(g, 64)
    # exactly the angle that the 64-bit turns say, at positions where fp32 has none left
    turns = pkg.fp8_rope_turns(rot_dim=64)
    exact = [2 * math.pi * (t / 2.0 ** 64) for t in turns.tolist()]
    qo, ko = pkg.fp8_qk_norm_rope(q, k, pos, turns, gamma_k=gamma, eps=0.0)
    settled()
    want, size = ref.norm_rope(q, pos, exact, None, 0.0, False)
    ref.check(qo, want, ref.U_BF16 * want.abs() + 2.0 ** -19 * size, "q")
    want, size = ref.norm_rope(k, pos, exact, gamma, 0.0, False)
    ref.check(ko, want, ref.U_BF16 * want.abs() + 2.0 ** -19 * size, "k")


def test_rope_turns_of_given_frequencies():
    f = [1.0, 0.25, 3.5, 7.0, 1e-6]
    got = pkg.fp8_rope_turns(inv_freq=f, device="cpu")
    for x, n in zip(f, got.tolist()):
        off = (n / 2.0 ** 64 - x / (2 * math.pi)) % 1.0
        assert min(off, 1 - off) < 1e-15


# ------------------------------------------------------------- prompt attention

def packed(g, lens, Hq, Hkv, D, extra=0):
    T = sum(lens) + extra
    qkv = normal(g, T, (Hq + 2 * Hkv) * D)
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
    return q, k, v, int32([sum(lens[:i]) for i in range(len(lens) + 1)])


def prompt_tol(want, size):
    return ref.U_BF16 * want.abs() + (ref.U_BF16 + ref.SUMS) * size


PROMPTS = [([1], 1, 1, 16), ([2, 0, 1, 3], 2, 1, 32), ([129], 4, 1, 128), ([128, 127, 1, 255], 8, 2, 64),
           ([300, 5, 0, 0, 77], 6, 2, 80), ([64, 65, 63], 7, 1, 96), ([513], 3, 3, 112),
           ([1] * 70, 8, 8, 128), ([200, 40], 64, 1, 128), ([257, 256, 31], 12, 4, 48),
           ([1000, 1025], 4, 2, 128), ([33] * 40, 5, 5, 64),
           ([1500, 2, 1999], 16, 16, 128), ([3001], 32, 4, 64)]


@pytest.mark.parametrize("lens,Hq,Hkv,D", PROMPTS)
def test_prompt(lens, Hq, Hkv, D):
    q, k, v, cu = packed(gen(sum(lens) + D), lens, Hq, Hkv, D)
    out = pkg.fp8_attention_prompt(q, k, v, cu)
    settled()
    want, size = ref.prompt(q, k, v, cu, D ** -0.5)
    ref.check(out, want, prompt_tol(want, size), "prompt")


@pytest.mark.parametrize("scale", [1e-3, 1.0, 4.0])
def test_prompt_scales_and_strides(scale):
    # a small scale (uniform weights), and large ones (one key takes all)
    g = gen(4)
    q, k, v, cu = packed(g, [190, 70], 4, 2, 64)
    wide = torch.full((260, 4, 96), 5.0, dtype=torch.bfloat16, device=DEV)
    out = torch.as_strided(wide.flatten(), (260, 4, 64), (4 * 96, 64, 1))
    before = wide.clone()
    assert pkg.fp8_attention_prompt(q, k.contiguous(), v, cu, scale=scale, out=out) is out
    settled()
    want, size = ref.prompt(q, k, v, cu, scale)
    # the scores' own fp32 error grows with them: 64 products of up to 16, 2^-24 each, times the scale
    tol = prompt_tol(want, size) + scale * 64 * 16 * 2.0 ** -23 * size
    ref.check(out, want, tol, "prompt")
    assert torch.equal(wide.view(260, -1)[:, 256:], before.view(260, -1)[:, 256:])


def test_prompt_growing_scores():
    # every key beats all earlier ones by far: the running maximum moves at each tile
    g = gen(14)
    n, D = 700, 64
    q, k, v, cu = (t.contiguous() for t in packed(g, [n], 2, 1, D))
    k.copy_((torch.arange(n, device=DEV).float()[:, None, None] / 8).expand(n, 1, D).to(torch.bfloat16))
    q.fill_(0.25)
    out = pkg.fp8_attention_prompt(q, k, v, cu)
    out2 = pkg.fp8_attention_prompt(q, -k, v, cu)
    settled()
    for got, kk in ((out, k), (out2, -k)):
        want, size = ref.prompt(q, kk, v, cu, D ** -0.5)
        ref.check(got, want, prompt_tol(want, size) + 2.0 ** -13 * size, "prompt")


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_prompt_unseen_values_have_no_influence(bad):
    lens, Hq, Hkv, D = [150, 90, 40], 4, 2, 64
    q, k, v, cu = (t.contiguous() for t in packed(gen(21), lens, Hq, Hkv, D, extra=30))
    clean = pkg.fp8_attention_prompt(q, k, v, cu)
    settled()
    # the last key and value of sequence 0, the one after all sequences, and token 70 of sequence 1
    for t in (149, 280, 220):
        k2, v2 = k.clone(), v.clone()
        k2[t, 0, 3] = bad
        v2[t, 1, 5] = bad
        got = pkg.fp8_attention_prompt(q, k2, v2, cu)
        settled()
        seen = torch.zeros(310, dtype=torch.bool)
        seen[t:{149: 150, 280: 280, 220: 240}[t]] = True
        keep = ~seen[:280]
        assert torch.equal(got[:280][keep], clean[:280][keep]), t
        if t == 280:
            continue
        # the value's channel is not finite for those that see it, the other channels of its heads are
        # untouched; the key's heads are judged where its score is NaN for sure
        assert not torch.isfinite(got[t:{149: 150, 220: 240}[t], 2:, 5]).any()
        rest = [d for d in range(D) if d != 5]
        assert torch.equal(got[t:, 2:][..., rest][:280 - t], clean[t:, 2:][..., rest][:280 - t])
        if math.isnan(bad):
            assert torch.isnan(got[t:{149: 150, 220: 240}[t], :2]).all()


@pytest.mark.parametrize("D", [64, 80, 128])
def test_prompt_bits_do_not_depend_on_its_company(D):
    # alone, before many short ones (one query tile a CTA), four times over (two)
    q, k, v, _ = packed(gen(23), [700] + [20] * 300, 32, 8, D)
    parts = [t[:700].contiguous() for t in (q, k, v)]
    alone = pkg.fp8_attention_prompt(*parts, int32([0, 700]))
    among = pkg.fp8_attention_prompt(q, k, v, int32([0] + [700 + 20 * i for i in range(301)]))
    four = pkg.fp8_attention_prompt(*(torch.cat([t] * 4) for t in parts), int32([0, 700, 1400, 2100, 2800]))
    settled()
    assert torch.equal(among[:700], alone)
    assert all(torch.equal(four[700 * i: 700 * i + 700], alone) for i in range(4))


def test_prompt_rows_outside_every_sequence_are_left():
    q, k, v, _ = packed(gen(3), [60], 4, 4, 64)
    out = torch.full((60, 4, 64), 9.0, dtype=torch.bfloat16, device=DEV)
    cu = int32([10, 30, 30, 45])
    pkg.fp8_attention_prompt(q, k, v, cu, out=out)
    settled()
    want, size = ref.prompt(q, k, v, cu, 0.125)
    ref.check(out[10:45], want[10:45], prompt_tol(want, size)[10:45], "prompt")
    assert bool((out[:10] == 9).all()) and bool((out[45:] == 9).all())
    pkg.fp8_attention_prompt(q, k, v, int32([7]), out=out)      # no sequence: a no-op
    assert pkg.fp8_attention_prompt(q[:0], k[:0], v[:0], int32([0, 0])).shape == (0, 4, 64)
    settled()


def test_prompt_is_deterministic_on_another_stream_and_in_a_graph():
    q, k, v, cu = packed(gen(6), [400, 1, 333], 8, 2, 128)
    first = pkg.fp8_attention_prompt(q, k, v, cu)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    second = pkg.fp8_attention_prompt(q, k, v, cu, stream=s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    third = torch.empty_like(first)
    with torch.cuda.graph(graph):
        pkg.fp8_attention_prompt(q, k, v, cu, out=third)
    graph.replay()
    settled()
    assert torch.equal(first, second) and torch.equal(first, third)


# ------------------------------------------------------------- decode attention

def cached(g, lens, Hq, Hkv, D, page, prefix=0, bad_pages=False):
    n = len(lens)
    width = max(1, -(-max(lens) // page))
    shared = prefix // page
    n_pages = shared + n * (width - shared) + 2
    order = torch.randperm(n_pages, generator=g, device=DEV).to(torch.int32)
    table = torch.cat([order[:shared].expand(n, shared),
                       order[shared: shared + n * (width - shared)].view(n, width - shared)], 1).contiguous()
    codes = [(torch.randn(n_pages * page, Hkv, D, generator=g, device=DEV) * 3).to(torch.float8_e4m3fn)
             .view(torch.uint8) for _ in range(2)]
    # slots that no request sees hold NaN codes
    seen = torch.zeros(n_pages * page, dtype=torch.bool, device=DEV)
    for b, x in enumerate(lens):
        j = torch.arange(max(0, min(x, width * page)), device=DEV)
        seen[table[b].long()[j // page] * page + j % page] = True
    for c in codes:
        c[~seen] = 0x7F
    if bad_pages:
        table[0, 0] = -1
        table[-1, -1] = n_pages
        table[n // 2, 0] = 2 ** 31 - 1
    scales = [torch.rand(Hkv, generator=g, device=DEV) * 0.2 + 0.2 for _ in range(2)]
    return normal(g, n, Hq, D), codes[0], codes[1], scales[0], scales[1], table, int32(lens)


def decode_tol(want, size):
    return ref.U_BF16 * want.abs() + (ref.U_FP16 + ref.SUMS) * size


def check_decode(args, page, prefix=0, scale=None, what="decode"):
    q = args[0]
    out = pkg.fp8_attention_decode(*args, page, prefix_len=prefix, scale=scale)
    settled()
    want, size = ref.decode(*args, page, prefix, q.shape[2] ** -0.5 if scale is None else scale)
    ref.check(out, want, decode_tol(want, size), what)
    return out


DECODES = [([1], 1, 1, 16, 1), ([0, 1, 2, 0], 2, 1, 32, 16), ([17, 300, 16, 15], 8, 2, 64, 16),
           ([128, 129, 127, 5], 32, 8, 128, 16), ([1000], 32, 8, 128, 64), ([63, 64, 65], 14, 2, 64, 20),
           ([500, 1, 77], 6, 3, 80, 7), ([2500, 30], 8, 1, 128, 128), ([90] * 40, 4, 4, 96, 32),
           ([40, 41], 64, 1, 112, 16), ([33, 7], 16, 16, 128, 16), ([260, 999], 24, 8, 48, 48),
           ([70, 150], 40, 2, 128, 16), ([31, 64], 26, 13, 64, 16), ([5000, 4999, 3], 7, 1, 128, 16)]


@pytest.mark.parametrize("lens,Hq,Hkv,D,page", DECODES)
def test_decode(lens, Hq, Hkv, D, page):
    check_decode(cached(gen(sum(lens) + D), lens, Hq, Hkv, D, page), page)


PREFIXES = [([300, 310, 257, 256], 8, 2, 64, 16, 256), ([1030] * 5, 32, 8, 128, 16, 1024),
            ([520 + i for i in range(33)], 8, 1, 128, 32, 512), ([140, 20, 0, 130, 64], 6, 3, 80, 20, 120),
            ([200 + i for i in range(70)], 4, 2, 96, 16, 192), ([700], 4, 1, 128, 64, 640),
            ([400 + i % 3 for i in range(150)], 2, 2, 64, 16, 400), ([257, 258], 7, 1, 112, 1, 250),
            ([2300 + 5 * i for i in range(20)], 16, 2, 128, 64, 2240), ([90, 90], 64, 1, 128, 16, 64),
            # (from here on enough requests for the shared-prefix kernel)
            ([900 + i for i in range(170)], 8, 8, 128, 20, 880), ([710 + i % 70 for i in range(260)], 24, 8, 80, 16, 704),
            ([2101 + i % 40 for i in range(200)], 14, 2, 64, 1, 2100), ([2020 + 9 * i for i in range(66)], 32, 8, 128, 32, 2016),
            ([3710 + i % 7 for i in range(120)], 64, 2, 112, 16, 3700), ([4003 + i % 50 for i in range(100)], 32, 2, 128, 64, 4001)]


@pytest.mark.parametrize("lens,Hq,Hkv,D,page,prefix", PREFIXES)
def test_decode_shared_prefix(lens, Hq, Hkv, D, page, prefix):
    args = cached(gen(sum(lens) + D), lens, Hq, Hkv, D, page, prefix)
    check_decode(args, page, prefix, what="prefix")
    # the same tokens without being told that they are shared
    check_decode(args, page, 0, what="no prefix")


def test_decode_prefix_inside_a_page_and_beyond_every_request():
    args = cached(gen(5), [100, 60, 101, 0], 8, 2, 64, 16, 96)
    check_decode(args, 16, 37)
    args = cached(gen(6), [90, 33, 5], 4, 2, 64, 16, 80)
    # (requests shorter than the prefix see their own part of it)
    args[5][:] = args[5][0]
    args[1][args[1] == 0x7F] = 0x20
    args[2][args[2] == 0x7F] = 0x20
    check_decode(args, 16, 96)


def test_decode_long_shared_prefix_with_hidden_pages_and_short_requests():
    lens = [1700 + 3 * i for i in range(80)]
    args = cached(gen(31), lens, 32, 8, 64, 16, 1696)
    args[5][0, 3] = -1               # a page of the shared part that does not exist
    args[5][0, 79] = 2 ** 31 - 1
    args[6][4], args[6][5], args[6][6], args[6][7] = 0, 1, 1000, -3
    check_decode(args, 16, 1696)
    args[0][2, 3] = 0                # a zero query: all weights alike
    check_decode(args, 16, 1677)
    args[5][0, :] = -1               # nothing of the shared part exists
    check_decode(args, 16, 1696)


def test_decode_bad_pages_and_lengths_are_hidden():
    for page, prefix in ((16, 0), (20, 0), (16, 16)):
        args = cached(gen(page), [100, 50, 170, 81, 20], 8, 2, 64, page, bad_pages=True)
        # a length beyond the table, a negative one
        args[6][3] = 2 ** 31 - 1
        args[6][1] = -4
        args[1][args[1] == 0x7F] = 0x31
        args[2][args[2] == 0x7F] = 0x31
        check_decode(args, page, prefix)


def test_decode_more_requests_than_are_cut_by_tokens():
    lens = [(7 * i) % 23 for i in range(4100)]
    check_decode(cached(gen(41), lens, 2, 1, 16, 8), 8)
    lens[17] = 700
    check_decode(cached(gen(42), lens, 18, 1, 32, 16), 16)


@pytest.mark.parametrize("lens,Hq,Hkv,D", [([160 + i % 41 for i in range(200)], 16, 8, 128),
                                           ([161 + i % 7 for i in range(301)], 8, 8, 64),
                                           ([0 if i % 3 else 170 for i in range(400)], 8, 8, 128),
                                           ([1300 + i for i in range(90)], 4, 2, 128),
                                           ([4000, 0, 1, 0], 32, 8, 128), ([150, 9000], 8, 8, 80)])
def test_decode_cuts_everywhere_in_a_request(lens, Hq, Hkv, D):
    # CTAs begin at every place of a request, before its first token too
    check_decode(cached(gen(49 + D), lens, Hq, Hkv, D, 16), 16)


def test_decode_one_long_request_among_many_short_ones():
    lens = [5 + i % 90 for i in range(200)]
    lens[77] = 6001
    check_decode(cached(gen(43), lens, 8, 8, 64, 16), 16)
    check_decode(cached(gen(44), lens, 8, 1, 128, 16), 16)


def test_decode_cache_beyond_32_bits():
    # 5 GB a cache: the pages at its end, at a byte offset past 2^32
    Hkv, D, page, n_pages = 8, 128, 64, 82000
    small = list(cached(gen(45), [300, 1, 129], 16, Hkv, D, page))
    far = list(small)
    have = small[1].shape[0]
    far[1], far[2] = (torch.zeros(n_pages * page, Hkv, D, dtype=torch.uint8, device=DEV) for _ in range(2))
    far[1][-have:], far[2][-have:] = small[1], small[2]
    far[5] = small[5] + (n_pages - have // page)
    assert far[1].numel() > 2 ** 32
    near = pkg.fp8_attention_decode(*small, page)
    got = pkg.fp8_attention_decode(*far, page)
    settled()
    assert torch.equal(near, got)
    # the same through the shared-prefix kernel
    small = list(cached(gen(46), [2001 + i for i in range(70)], 32, Hkv, D, page, 1984))
    have = small[1].shape[0]
    far[1].zero_()
    far[2].zero_()
    far[1][-have:], far[2][-have:] = small[1], small[2]
    far = [small[0], far[1], far[2], small[3], small[4], small[5] + (n_pages - have // page), small[6]]
    near = pkg.fp8_attention_decode(*small, page, prefix_len=1984)
    got = pkg.fp8_attention_decode(*far, page, prefix_len=1984)
    settled()
    assert torch.equal(near, got)
    # and the cache write on the way of the rotation
    q, k, v = (normal(gen(47), 3, h, D) for h in (2, Hkv, Hkv))
    slot = torch.tensor([n_pages * page - 1, 5, n_pages * page - 1 - 4 * 10 ** 6], device=DEV)
    one = torch.ones(1, device=DEV)
    pkg.fp8_qk_norm_rope(q, k, int32([1, 2, 3]), pkg.fp8_rope_turns(rot_dim=D), v=v, k_scale=one, v_scale=one,
                         slot_mapping=slot, k_cache=far[1], v_cache=far[2])
    settled()
    assert torch.equal(far[2][slot].view(torch.float8_e4m3fn).float(), v.to(torch.float8_e4m3fn).float())


def test_prompt_beyond_32_bits():
    # tokens whose queries and outputs lie past 2^32 bytes
    g = gen(48)
    T, Hq, Hkv, D = 270000, 64, 8, 128
    qkv = torch.zeros(T, (Hq + 2 * Hkv) * D, dtype=torch.bfloat16, device=DEV)
    qkv[-400:] = normal(g, 400, qkv.shape[1])
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([Hq * D, Hkv * D, Hkv * D], 1))
    far = pkg.fp8_attention_prompt(q, k, v, int32([T - 400, T - 100, T]))
    near = pkg.fp8_attention_prompt(q[-400:].contiguous(), k[-400:].contiguous(), v[-400:].contiguous(),
                                    int32([0, 300, 400]))
    settled()
    assert far.numel() * 2 > 2 ** 32 and torch.equal(far[-400:], near)


def test_decode_single_scale_strides_large_queries_and_scales():
    args = list(cached(gen(15), [333, 40], 8, 4, 64, 16))
    args[3], args[4] = args[3][:1], args[4][:1]
    wide = normal(gen(2), 2, 8 * 64 + 128)
    # queries at the ends of bf16's range: powers of two are taken out exactly
    for factor in (1.0, 2.0 ** 60, 2.0 ** -60):
        args[0] = (wide * factor)[:, : 8 * 64].unflatten(1, (8, 64))
        check_decode(args, 16, scale=0.3 / factor)
    args[0] = wide[:, : 8 * 64].unflatten(1, (8, 64))
    out = torch.full((2, 8 * 64 + 64), 3.0, dtype=torch.bfloat16, device=DEV)
    view = out[:, : 8 * 64].unflatten(1, (8, 64))
    pkg.fp8_attention_decode(*args, 16, out=view)
    settled()
    assert torch.equal(view, pkg.fp8_attention_decode(*args, 16)) and bool((out[:, 8 * 64:] == 3).all())


def test_decode_is_deterministic_on_another_stream_and_in_a_graph():
    args = cached(gen(9), [1500, 3, 800, 64], 16, 4, 128, 16, 0)
    first = pkg.fp8_attention_decode(*args, 16)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    second = pkg.fp8_attention_decode(*args, 16, stream=s)
    s.synchronize()
    ws = torch.empty(max(1, pkg.fp8_attention_decode_workspace_size(4, 16, 4, 128, args[5].shape[1], 16)),
                     dtype=torch.uint8, device=DEV)
    ws.fill_(0xFF)  # nothing in it needs to start at zero
    third = torch.empty_like(first)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkg.fp8_attention_decode(*args, 16, out=third, workspace=ws)
    graph.replay()
    torch.cuda.synchronize()
    # the lengths are the device's: a replay sees new ones
    assert torch.equal(first, second) and torch.equal(first, third)
    args[6][0] = 700
    graph.replay()
    settled()
    want, size = ref.decode(*args, 16, 0, 128 ** -0.5)
    ref.check(third, want, decode_tol(want, size), "replayed")


def test_decode_no_requests_and_no_pages():
    args = list(cached(gen(9), [5, 6], 4, 2, 64, 16))
    none = [a[:0] if i in (0, 5, 6) else a for i, a in enumerate(args)]
    assert pkg.fp8_attention_decode(*none, 16).shape == (0, 4, 64)
    empty = list(args)
    empty[5] = args[5][:, :0]
    assert not pkg.fp8_attention_decode(*empty, 16).any()
    empty = list(args)
    empty[1], empty[2] = args[1][:0], args[2][:0]
    assert not pkg.fp8_attention_decode(*empty, 16).any()
    settled()
