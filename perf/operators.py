"""The attention block's operators, as cases that can be timed and compared.

Between the QKV projection and the output projection a serving step needs
  slots   block tables, slot maps and positions built on the GPU from request lengths
  rope    per-head norms of queries and keys with the rotation in the same pass, keys and values
          quantized into the FP8 cache on the way
  prompt  causal attention over packed prompts of different lengths, grouped heads
  decode  attention of one new token per request over the paged FP8 cache, a prefix that all requests
          share read once for all

`listed()` names the cases, `draw(rng)` gives more of the same ranges, `prepare(case, seed)` makes the
inputs, `run(state)` makes one pass: the plain form in elementary torch operations, or, where `own` is
true, the framework's calls.  `exact(case, seed)` is the operator's definition in 64 bits.
"""
import math
import random

import torch

own = False

DEVICE = "cuda"
EPS = 1e-6
THETA = 500000.0
E4M3_MAX = 448.0


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # every decode step of a busy engine: one new token for each of 256 requests
        dict(name="slots_step_256", op="slots", requests=256, max_ctx=8192, max_new=1, page=16),
        # admission of many prompts at once, some of them continuing a cached context
        dict(name="slots_prompts_96", op="slots", requests=96, max_ctx=2048, max_new=1365, page=64),
        # decode step of the 8B layer shapes: 32 tokens, rotation only
        dict(name="rope_step_32", op="rope", tokens=32, q_heads=32, kv_heads=8, dim=128, rot=128,
             norm=False, interleaved=False, max_pos=131072),
        # prompt of the 70B layer shapes, with norms of queries and keys
        dict(name="rope_prompt_8192", op="rope", tokens=8192, q_heads=64, kv_heads=8, dim=128, rot=128,
             norm=True, interleaved=False, max_pos=8192),
        # small heads, a rotation of half of each head in interleaved pairs, an odd number of tokens
        dict(name="rope_partial_1021", op="rope", tokens=1021, q_heads=14, kv_heads=2, dim=64, rot=32,
             norm=True, interleaved=True, max_pos=32768),
        # short chat turns packed together: latency and tile waste count
        dict(name="prompt_short_24", op="prompt", requests=24, min_len=1, max_len=257, q_heads=32,
             kv_heads=8, dim=128),
        # a packed prefill batch of very different lengths
        dict(name="prompt_ragged_9", op="prompt", requests=9, min_len=129, max_len=2801, q_heads=64,
             kv_heads=8, dim=128),
        # one long prompt at the 8B shapes
        dict(name="prompt_long_8192", op="prompt", requests=1, min_len=8192, max_len=8192, q_heads=32,
             kv_heads=8, dim=128),
        # one request over a long context: the latency of a single user's token
        dict(name="decode_one_16k", op="decode", requests=1, prefix=0, min_len=16383, max_len=16383,
             q_heads=32, kv_heads=8, dim=128, page=16),
        # a busy engine: 64 requests of very different lengths at the 70B shapes
        dict(name="decode_ragged_64", op="decode", requests=64, prefix=0, min_len=257, max_len=16001,
             q_heads=64, kv_heads=8, dim=128, page=64),
        # 64 requests that share a long system prompt and differ in their own turns
        dict(name="decode_prefix_64", op="decode", requests=64, prefix=8192, min_len=1, max_len=777,
             q_heads=32, kv_heads=8, dim=128, page=16),
        # a few short requests with small heads and pages of an odd size
        dict(name="decode_short_7", op="decode", requests=7, prefix=0, min_len=1, max_len=301,
             q_heads=14, kv_heads=2, dim=64, page=20),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    kv = rng.choice([1, 2, 4, 8])
    return dict(q_heads=kv * rng.choice([1, 2, 4, 7, 8]), kv_heads=kv, dim=rng.choice([64, 80, 96, 128]))


def draw(rng):
    op = rng.choice(["slots", "rope", "prompt", "prompt", "decode", "decode"])
    if op == "slots":
        requests = _spread(rng, 1, 1024)
        return dict(op=op, requests=requests, max_ctx=_spread(rng, 1, 16384),
                    max_new=_spread(rng, 1, max(2, 98304 // requests)), page=rng.choice([1, 16, 20, 64, 128]))
    if op == "rope":
        c = dict(op=op, tokens=_spread(rng, 1, 8192), **_heads(rng))
        c.update(rot=rng.choice([c["dim"], 32]), norm=rng.random() < 0.5, interleaved=rng.random() < 0.5,
                 max_pos=_spread(rng, 64, 131072))
        return c
    if op == "prompt":
        requests = _spread(rng, 1, 48)
        hi = _spread(rng, 2, max(2, min(4096, 12288 // requests)))
        c = dict(op=op, requests=requests, min_len=_spread(rng, 1, hi), max_len=hi, **_heads(rng))
        c["q_heads"] = min(c["q_heads"], 32)
        return c
    requests = _spread(rng, 1, 128)
    prefix = rng.choice([0, 0, _spread(rng, 16, 16384)])
    hi = _spread(rng, 1, max(1, min(16384, 262144 // requests)))
    return dict(op=op, requests=requests, prefix=prefix, min_len=_spread(rng, 1, hi), max_len=hi,
                page=rng.choice([16, 20, 32, 64]), **_heads(rng))


# --------------------------------------------------------------------------- inputs

def _lengths(case, seed):
    """The case's lengths: a geometric spread from min_len to max_len in an order of the seed."""
    n, lo, hi = case["requests"], case["min_len"], case["max_len"]
    got = [int(round(lo * (hi / lo) ** (i / max(1, n - 1)))) for i in range(n)]
    random.Random(seed).shuffle(got)
    return got


def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 17)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE).to(torch.bfloat16)


def _codes(g, *shape):
    """E4M3 codes of normal values."""
    return (torch.randn(*shape, generator=g, device=DEVICE) * 3.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device=DEVICE)


def _inv_freq(rot):
    return THETA ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)


def _capacity(case):
    """Tokens and table width that a program's buffers have room for."""
    if case["op"] == "slots":
        return case["requests"] * case["max_new"], -(-(case["max_ctx"] + case["max_new"]) // case["page"])
    return case["requests"], -(-(case["prefix"] + case["max_len"]) // case["page"])


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    if case["op"] == "slots":
        n, page = case["requests"], case["page"]
        tokens, width = _capacity(case)
        ctx = torch.randint(0, case["max_ctx"] + 1, (n,), generator=g, device=DEVICE, dtype=torch.int32)
        new = torch.randint(min(1, case["max_new"] - 1), case["max_new"] + 1, (n,), generator=g, device=DEVICE,
                            dtype=torch.int32)
        pages = torch.randperm(2 * n * width, generator=g, device=DEVICE).to(torch.int32)
        table = torch.full((n, width), -1, dtype=torch.int32, device=DEVICE)
        have = (ctx + page - 1) // page
        filled = torch.arange(width, device=DEVICE)[None, :] < have[:, None]
        table = torch.where(filled, pages[: n * width].view(n, width), table).contiguous()
        s.update(ctx=ctx, new=new, free=pages[n * width:].contiguous(), table=table, tokens=tokens)
        return s
    if case["op"] == "rope":
        T, hq, hkv, d = case["tokens"], case["q_heads"], case["kv_heads"], case["dim"]
        qkv = _normal(g, T, (hq + 2 * hkv) * d)
        s["q"] = qkv[:, : hq * d].unflatten(1, (hq, d))
        s["k"] = qkv[:, hq * d: (hq + hkv) * d].unflatten(1, (hkv, d))
        s["v"] = qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
        s["gamma_q"] = (1 + 0.1 * torch.randn(d, generator=g, device=DEVICE)).to(torch.bfloat16)
        s["gamma_k"] = (1 + 0.1 * torch.randn(d, generator=g, device=DEVICE)).to(torch.bfloat16)
        s["positions"] = torch.randint(0, case["max_pos"], (T,), generator=g, device=DEVICE, dtype=torch.int32)
        # the plan of the rotation: each pair's frequency as a 2^-64 fraction of a turn per position
        s["turns"] = (_inv_freq(case["rot"]) / (2 * math.pi) * 2.0 ** 64).to(torch.int64).to(DEVICE)
        s["slots"] = torch.randperm(T + 7, generator=g, device=DEVICE)[:T]
        s["k_scale"] = 0.01 + 0.01 * torch.rand(hkv, generator=g, device=DEVICE)
        s["v_scale"] = 0.01 + 0.01 * torch.rand(hkv, generator=g, device=DEVICE)
        s["k_cache"] = torch.zeros(T + 7, hkv, d, dtype=torch.uint8, device=DEVICE)
        s["v_cache"] = torch.zeros(T + 7, hkv, d, dtype=torch.uint8, device=DEVICE)
        return s
    lens = _lengths(case, seed)
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "prompt":
        total = sum(lens)
        qkv = _normal(g, total, (hq + 2 * hkv) * d)
        s["q"] = qkv[:, : hq * d].unflatten(1, (hq, d))
        s["k"] = qkv[:, hq * d: (hq + hkv) * d].unflatten(1, (hkv, d))
        s["v"] = qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
        s["cu"] = _int32([sum(lens[:i]) for i in range(len(lens) + 1)])
        return s
    n, page, shared = case["requests"], case["page"], case["prefix"] // case["page"]
    _, width = _capacity(case)
    n_pages = shared + n * (width - shared) + 3
    order = torch.randperm(n_pages, generator=g, device=DEVICE).to(torch.int32)
    table = order[shared: shared + n * (width - shared)].view(n, width - shared)
    s["table"] = torch.cat([order[:shared].expand(n, shared), table], 1).contiguous()
    s["prefix"] = shared * page  # whole pages are shared, as an engine's prefix cache shares them
    s["lens"] = _int32([case["prefix"] + x for x in lens])
    s["q"] = _normal(g, n, hq, d)
    s["k_cache"] = _codes(g, n_pages * page, hkv, d)
    s["v_cache"] = _codes(g, n_pages * page, hkv, d)
    s["k_scale"] = 0.2 + 0.2 * torch.rand(hkv, generator=g, device=DEVICE)
    s["v_scale"] = 0.2 + 0.2 * torch.rand(hkv, generator=g, device=DEVICE)
    return s


# --------------------------------------------------------------------------- one pass

def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_slots(s):
    import fp8_w8a8_quantized_gb300 as fp8
    slots, positions, cu, lens, used = fp8.fp8_kv_slots(s["ctx"], s["new"], s["free"], s["page"], s["table"],
                                                        s["tokens"])
    return dict(table=s["table"], slots=slots, positions=positions, cu=cu, lens=lens, used=used)


def _own_rope(s):
    import fp8_w8a8_quantized_gb300 as fp8
    q, k = fp8.fp8_qk_norm_rope(s["q"], s["k"], s["positions"], s["turns"],
                                gamma_q=s["gamma_q"] if s["norm"] else None,
                                gamma_k=s["gamma_k"] if s["norm"] else None, eps=EPS,
                                interleaved=s["interleaved"], v=s["v"], k_scale=s["k_scale"],
                                v_scale=s["v_scale"], slot_mapping=s["slots"], k_cache=s["k_cache"],
                                v_cache=s["v_cache"])
    return dict(q=q, k=k, k_cache=s["k_cache"].view(torch.float8_e4m3fn),
                v_cache=s["v_cache"].view(torch.float8_e4m3fn))


def _own_prompt(s):
    import fp8_w8a8_quantized_gb300 as fp8
    return fp8.fp8_attention_prompt(s["q"], s["k"], s["v"], s["cu"])


def _own_decode(s):
    import fp8_w8a8_quantized_gb300 as fp8
    return fp8.fp8_attention_decode(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["table"],
                                    s["lens"], s["page"], prefix_len=s["prefix"])


_own = dict(slots=_own_slots, rope=_own_rope, prompt=_own_prompt, decode=_own_decode)


def _plain_slots(s):
    ctx, new, page, table = s["ctx"].long(), s["new"].long(), s["page"], s["table"]
    n, width = table.shape
    have, need = (ctx + page - 1) // page, (ctx + new + page - 1) // page
    first = torch.cumsum(need - have, 0) - (need - have)
    column = torch.arange(width, device=table.device)[None, :]
    taken = (column >= have[:, None]) & (column < need[:, None])
    entry = (first[:, None] + column - have[:, None]).clamp(0, s["free"].numel() - 1)
    table.copy_(torch.where(taken, s["free"][entry], table))
    cu = torch.zeros(n + 1, dtype=torch.int64, device=table.device)
    cu[1:] = torch.cumsum(new, 0)
    t = torch.arange(s["tokens"], device=table.device)
    b = torch.searchsorted(cu[1:], t, right=True).clamp(max=n - 1)
    live = t < cu[-1]
    position = torch.where(live, ctx[b] + t - cu[b], 0)
    slot = table[b, position // page].long() * page + position % page
    return dict(table=table, slots=torch.where(live, slot, -1), positions=position.int(), cu=cu.int(),
                lens=(ctx + new).int(), used=(need - have).sum().int().reshape(1))


def _rotate(x, angle, interleaved):
    rot = 2 * angle.shape[-1]
    c, n = angle.cos().float()[:, None, :], angle.sin().float()[:, None, :]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * c - b * n, b * c + a * n], -1).flatten(-2)
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        turned = torch.cat([a * c - b * n, b * c + a * n], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_rope(s):
    angle = (s["positions"].long()[:, None] * s["turns"][None, :]).double() * (2 * math.pi * 2.0 ** -64)

    def normed(x, gamma):
        x = x.float()
        if not s["norm"]:
            return x
        return x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * gamma.float()

    q = _rotate(normed(s["q"], s["gamma_q"]), angle, s["interleaved"]).to(torch.bfloat16)
    k = _rotate(normed(s["k"], s["gamma_k"]), angle, s["interleaved"]).to(torch.bfloat16)

    def write(cache, x, scale):
        y = (x.float() / scale[None, :, None]).clamp(-E4M3_MAX, E4M3_MAX)
        cache[s["slots"]] = y.to(torch.float8_e4m3fn).view(torch.uint8)
        return cache.view(torch.float8_e4m3fn)

    return dict(q=q, k=k, k_cache=write(s["k_cache"], k, s["k_scale"]),
                v_cache=write(s["v_cache"], s["v"], s["v_scale"]))


def _attend(q, k, v, mask):
    """softmax(q k^T / sqrt(D)) v over the keys that `mask` leaves, zero where it leaves none."""
    score = (q @ k.transpose(-1, -2)) / math.sqrt(q.shape[-1])
    score = score.masked_fill(~mask, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(-1, keepdim=True)
    return (p @ v) / torch.where(total == 0, 1.0, total)


def _plain_prompt(s):
    cu, n, L = s["cu"].long(), s["requests"], s["max_len"]
    T, hq, d = s["q"].shape
    hkv = s["k"].shape[1]
    at = torch.arange(L, device=cu.device)
    lens = cu[1:] - cu[:-1]
    row = (cu[:-1, None] + at[None, :]).clamp(max=T - 1)
    k = s["k"][row].float().transpose(1, 2)                                          # [n, hkv, L, d]
    v = s["v"][row].float().transpose(1, 2)
    q = s["q"][row].float().view(n, L, hkv, hq // hkv, d).permute(0, 2, 3, 1, 4)      # [n, hkv, g, L, d]
    mask = (at[None, :] <= at[:, None])[None] & (at[None, None, :] < lens[:, None, None])
    out = _attend(q, k.unsqueeze(2), v.unsqueeze(2), mask[:, None, None])
    out = out.permute(0, 3, 1, 2, 4).reshape(n * L, hq, d)
    t = torch.arange(T, device=cu.device)
    b = torch.searchsorted(cu[1:], t, right=True)
    return out[b * L + t - cu[b]].to(torch.bfloat16)


def _plain_decode(s):
    n, hq, d = s["q"].shape
    hkv, page, L = s["k_cache"].shape[1], s["page"], s["table"].shape[1] * s["page"]
    at = torch.arange(L, device=s["q"].device)
    slot = s["table"].long()[:, at // page] * page + at % page                         # [n, L]

    def values(cache, scale):
        x = cache[slot].view(torch.float8_e4m3fn).float() * scale[None, None, :, None]
        return x.transpose(1, 2)                                                     # [n, hkv, L, d]

    q = s["q"].float().view(n, hkv, hq // hkv, d)
    mask = at[None, :] < s["lens"].long()[:, None]
    out = _attend(q, values(s["k_cache"], s["k_scale"]), values(s["v_cache"], s["v_scale"]), mask[:, None, None])
    return out.reshape(n, hq, d).to(torch.bfloat16)


_plain = dict(slots=_plain_slots, rope=_plain_rope, prompt=_plain_prompt, decode=_plain_decode)


# --------------------------------------------------------------------------- work and exact values

def work(case):
    if case["op"] == "slots":
        n, (tokens, width) = case["requests"], _capacity(case)
        new = case["max_new"] / 2 if case["max_new"] > 1 else 1
        taken = n * new / case["page"]
        return dict(bytes=8 * n + 8 * taken + 12 * tokens + 8 * n + 4, flops=0)
    hq, hkv, d = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "rope":
        T = case["tokens"]
        return dict(bytes=T * (2 * (2 * hq + 3 * hkv) * d + 2 * hkv * d + 12), flops=T * (hq + hkv) * (3 * d + 3 * case["rot"]))
    lens = _lengths(case, 0)
    if case["op"] == "prompt":
        return dict(bytes=sum(lens) * 2 * d * (2 * hq + 2 * hkv), flops=4 * d * hq * sum(x * (x + 1) // 2 for x in lens))
    shared = case["prefix"] // case["page"] * case["page"]
    read = shared + sum(case["prefix"] - shared + x for x in lens)
    return dict(bytes=read * 2 * hkv * d + 4 * d * hq * len(lens) + 4 * read / case["page"],
                flops=4 * d * hq * sum(case["prefix"] + x for x in lens))


def _e4m3_values():
    """The value of each of the 256 codes, from the format's fields."""
    got = []
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        got.append(-x if code & 128 else x)
    got[0x7F] = got[0xFF] = math.nan
    return torch.tensor(got, dtype=torch.float64, device=DEVICE)


def _softmax_rows(score):
    w = torch.exp2((score - score.max(-1, keepdim=True).values) * math.log2(math.e))
    return w / w.sum(-1, keepdim=True)


def _exact_rope(case, s):
    T, half = case["tokens"], case["rot"] // 2
    angle = torch.outer(s["positions"].double(), _inv_freq(case["rot"]).to(DEVICE))
    turn = torch.polar(torch.ones_like(angle), angle)[:, None, :]

    def turned(x, gamma):
        x = x.double()
        if case["norm"]:
            x = x * torch.rsqrt((x * x).sum(-1, keepdim=True) / case["dim"] + EPS) * gamma.double()
        y = x.clone()
        if case["interleaved"]:
            z = torch.complex(x[..., 0: 2 * half: 2], x[..., 1: 2 * half: 2]) * turn
            y[..., 0: 2 * half: 2], y[..., 1: 2 * half: 2] = z.real, z.imag
        else:
            z = torch.complex(x[..., :half], x[..., half: 2 * half]) * turn
            y[..., :half], y[..., half: 2 * half] = z.real, z.imag
        return y

    return dict(q=turned(s["q"], s["gamma_q"]), k=turned(s["k"], s["gamma_k"]), k_cache=None, v_cache=None)


def _exact_prompt(case, s):
    T, hq, d = s["q"].shape
    g = hq // case["kv_heads"]
    out = torch.empty(T, hq, d, dtype=torch.float64, device=DEVICE)
    bounds = s["cu"].tolist()
    for a, e in zip(bounds[:-1], bounds[1:]):
        future = torch.ones(e - a, e - a, dtype=torch.bool, device=DEVICE).triu(1)
        for h in range(hq):
            score = s["q"][a:e, h].double() @ s["k"][a:e, h // g].double().T * d ** -0.5
            score[future] = -math.inf
            out[a:e, h] = _softmax_rows(score) @ s["v"][a:e, h // g].double()
    return out


def _exact_decode(case, s):
    n, hq, d = s["q"].shape
    hkv, page = case["kv_heads"], case["page"]
    value = _e4m3_values()
    out = torch.empty(n, hkv, hq // hkv, d, dtype=torch.float64, device=DEVICE)
    for b, length in enumerate(s["lens"].tolist()):
        pages = s["table"][b].long()
        slot = (pages[:, None] * page + torch.arange(page, device=DEVICE)).flatten()[:length]
        k = value[s["k_cache"][slot].long()] * s["k_scale"].double()[:, None]
        v = value[s["v_cache"][slot].long()] * s["v_scale"].double()[:, None]
        q = s["q"][b].double().view(hkv, hq // hkv, d)
        w = _softmax_rows(torch.einsum("hgd,lhd->hgl", q, k) / math.sqrt(d))
        out[b] = torch.einsum("hgl,lhd->hgd", w, v)
    return out.view(n, hq, d)


def exact(case, seed):
    if case["op"] == "slots":
        return None  # whole numbers
    return dict(rope=_exact_rope, prompt=_exact_prompt, decode=_exact_decode)[case["op"]](case, prepare(case, seed))
