"""The expert block's operators, as cases that can be timed and compared.

A serving step whose feed-forward layers are split into experts needs, between the attention block
and the next layer,
  route    each token's best experts with their weights, and the tokens' rows sorted by expert
  grouped  FP8 products of the rows of each expert with that expert's weights (ragged sizes, known on
           the GPU alone), the gated activation in the first of the two
  join     the experts' rows of a token summed by weight, normed, gated, scaled and added to the
           residual stream, and the norm and FP8 quantization that the next layer starts with

`listed()` names the cases, `draw(rng)` gives more of the same ranges, `prepare(case, seed)` makes the
inputs, `run(state)` makes one pass: the plain form in elementary torch operations, or, where `own` is
true, the framework's calls.  `exact(case, seed)` is the operator's definition in 64 bits.
"""
import math

import torch

own = False

DEVICE = "cuda"
EPS = 1e-6
E4M3_MAX = 448.0


# --------------------------------------------------------------------------- cases

def listed():
    return [
        # a decode step of 32 tokens over many small experts: latency counts
        dict(name="route_step_32", op="route", tokens=32, experts=64, top=8, dtype="float32", renorm=True,
             masked=0, scale=1.0),
        # a prefill batch over the most experts
        dict(name="route_prompt_8192", op="route", tokens=8192, experts=256, top=8, dtype="float32", renorm=True,
             masked=0, scale=2.5),
        # 16-bit logits with many ties, an odd number of experts, some of them switched off
        dict(name="route_odd_1021", op="route", tokens=1021, experts=60, top=4, dtype="bfloat16", renorm=False,
             masked=7, scale=1.0),
        # one user's token, two of eight experts of the 8B shapes: weights read once bound it
        dict(name="grouped_one_gate", op="grouped", tokens=1, experts=8, top=2, width=4096, out=28672, gated=True,
             gather=True, skew=1.0),
        # a decode step's second product, rows already in the experts' order
        dict(name="grouped_step_down", op="grouped", tokens=32, experts=8, top=2, width=14336, out=4096,
             gated=False, gather=False, skew=1.0),
        # a busy engine with many small experts, about 32 rows each, some with few and some with many
        dict(name="grouped_small_experts", op="grouped", tokens=253, experts=64, top=8, width=2048, out=2816,
             gated=True, gather=True, skew=1.0),
        # a prefill batch at the 8B shapes: the tensor cores bound it
        dict(name="grouped_prompt_gate", op="grouped", tokens=4096, experts=8, top=2, width=4096, out=28672,
             gated=True, gather=True, skew=0.5),
        # a ragged prefill of small experts, loads that differ much and experts without a row
        dict(name="grouped_ragged_down", op="grouped", tokens=3001, experts=40, top=6, width=1408, out=2048,
             gated=False, gather=False, skew=2.0),
        # the end of a decode step's expert block: two rows a token joined, and the next layer's norm
        dict(name="join_step_32", op="join", tokens=32, width=4096, top=2, post=False, gate="none", branch=1.0,
             residual=1.0, codes=True, rows=False),
        # a prompt's block with a norm behind it and a gate a channel; codes for the next FP8 layer
        dict(name="join_prompt_8192", op="join", tokens=8192, width=4096, top=0, post=True, gate="channel",
             branch=0.22, residual=1.0, codes=True, rows=True),
        # four rows a token, a gate of its own for each token, an odd width and number of tokens
        dict(name="join_gated_1021", op="join", tokens=1021, width=2880, top=4, post=True, gate="token",
             branch=1.0, residual=0.5, codes=False, rows=True),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["route", "grouped", "grouped", "join"])
    if op == "route":
        experts = _spread(rng, 4, 256)
        top = rng.randint(1, min(8, experts))
        return dict(op=op, tokens=_spread(rng, 1, 8192), experts=experts, top=top,
                    dtype=rng.choice(["float32", "bfloat16"]), renorm=rng.random() < 0.5,
                    masked=rng.choice([0, 0, rng.randint(0, experts - 1)]), scale=rng.choice([1.0, 2.5]))
    if op == "grouped":
        experts = _spread(rng, 1, 64)
        top = rng.randint(1, min(8, experts))
        width = 16 * _spread(rng, 16, 448)
        most = 8 * 28672 * 4096 // (experts * width)                    # weights of the largest listed case
        out = 16 * _spread(rng, 8, max(8, min(1792, most // 16)))
        rows = int(min(8192, 8192 * 28672 * 4096 / (width * out)))        # and its products
        return dict(op=op, tokens=_spread(rng, 1, max(1, min(4096, rows // top))), experts=experts, top=top,
                    width=width, out=out, gated=rng.random() < 0.5, gather=rng.random() < 0.5,
                    skew=rng.choice([0.0, 0.5, 1.0, 2.0]))
    width = 16 * _spread(rng, 8, 512)
    codes = rng.random() < 0.7
    return dict(op=op, tokens=_spread(rng, 1, min(8192, 8192 * 4096 // width)), width=width,
                top=rng.choice([0, 1, 2, 4]), post=rng.random() < 0.5,
                gate=rng.choice(["none", "channel", "token"]), branch=rng.choice([1.0, 0.22]),
                residual=rng.choice([1.0, 0.5]), codes=codes, rows=not codes or rng.random() < 0.5)


# --------------------------------------------------------------------------- inputs

def _generator(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(int(seed) * 2654435761 % (1 << 62) + 29)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device=DEVICE).to(torch.bfloat16)


def _order(ids, experts):
    """Rows sorted by expert, in the tokens' order within one: (offsets, row_token, token_row)."""
    flat = ids.reshape(-1).long()
    none = flat < 0
    key = torch.where(none, experts, flat)
    rank = torch.sort(key, stable=True).indices
    counts = (key[:, None] == torch.arange(experts, device=key.device)[None, :]).sum(0)
    offsets = torch.zeros(experts + 1, dtype=torch.int64, device=key.device)
    offsets[1:] = torch.cumsum(counts, 0)
    at = torch.arange(flat.numel(), device=key.device)
    row_token = torch.where(at < offsets[-1], rank // ids.shape[1], -1)
    back = torch.empty_like(rank)
    back[rank] = at
    token_row = torch.where(none, -1, back).reshape(ids.shape)
    return offsets.int(), row_token.int(), token_row.int()


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case)
    T = case["tokens"]
    if case["op"] == "route":
        logits = 2.0 * torch.randn(T, case["experts"], generator=g, device=DEVICE)
        if case["masked"]:  # experts that are switched off for all tokens
            off = torch.randperm(case["experts"], generator=g, device=DEVICE)[: case["masked"]]
            logits[:, off] = -math.inf
        s["logits"] = logits.to(getattr(torch, case["dtype"]))
        return s
    if case["op"] == "grouped":
        E, K, N = case["experts"], case["width"], case["out"]
        # experts differ in how often they are chosen, by exp(skew * normal)
        likes = case["skew"] * torch.randn(E, generator=g, device=DEVICE)
        noise = -torch.log(-torch.log(torch.rand(T, E, generator=g, device=DEVICE).clamp(1e-7, 1 - 1e-6)))
        ids = torch.sort(likes[None, :] + noise, descending=True, stable=True).indices[:, : case["top"]]
        s["offsets"], row_token, _ = _order(ids, E)
        s["row_token"] = row_token if case["gather"] else None
        s["x"] = _normal(g, T if case["gather"] else T * case["top"], K)
        s["wq"] = (105.0 * torch.randn(E, N, K, generator=g, device=DEVICE)).clamp(-E4M3_MAX, E4M3_MAX).to(
            torch.float8_e4m3fn).view(torch.uint8)
        s["s_w"] = (0.5 + torch.rand(E, N, generator=g, device=DEVICE)) / (105.0 * math.sqrt(K))
        s["most"] = int((s["offsets"][1:] - s["offsets"][:-1]).max())  # rows of the busiest expert
        return s
    K, top = case["width"], case["top"]
    s["h"] = (4.0 * torch.randn(T, K, generator=g, device=DEVICE)).to(torch.bfloat16)
    s["y"] = _normal(g, T * max(1, top), K)
    s["token_row"] = s["weights"] = None
    if top:
        s["token_row"] = torch.randperm(T * top, generator=g, device=DEVICE).view(T, top).int()
        w = torch.rand(T, top, generator=g, device=DEVICE)
        s["weights"] = w / w.sum(-1, keepdim=True)
    s["gamma"] = (1 + 0.1 * torch.randn(K, generator=g, device=DEVICE)).to(torch.bfloat16)
    s["gamma_post"] = (1 + 0.1 * torch.randn(K, generator=g, device=DEVICE)).to(torch.bfloat16) if case["post"] else None
    s["g"] = None
    if case["gate"] == "channel":
        s["g"] = _normal(g, K)
    elif case["gate"] == "token":
        s["g"] = _normal(g, T, K)
    return s


# --------------------------------------------------------------------------- one pass

def run(s):
    return (_own if own else _plain)[s["op"]](s)


def _own_route(s):
    import fp8_w8a8_quantized_gb300 as fp8
    ids, weights, offsets, row_token, token_row = fp8.fp8_moe_route(s["logits"], s["top"], renormalize=s["renorm"],
                                                                    scale=s["scale"])
    return dict(ids=ids, weights=weights, offsets=offsets, row_token=row_token, token_row=token_row)


def _own_grouped(s):
    import fp8_w8a8_quantized_gb300 as fp8
    return fp8.fp8_grouped_linear(s["x"], s["wq"], s["s_w"], s["offsets"], row_token=s["row_token"],
                                  swiglu=s["gated"])


def _own_join(s):
    import fp8_w8a8_quantized_gb300 as fp8
    h, z, codes, scale = fp8.fp8_residual_norm_quant(
        s["h"], s["y"], s["gamma"], eps=EPS, gamma_post=s["gamma_post"], gate=s["g"], residual_scale=s["residual"],
        branch_scale=s["branch"], token_row=s["token_row"], weights=s["weights"], rows=s["rows"], codes=s["codes"])
    return dict(h=h, z=z, codes=codes if codes is None else codes.view(torch.float8_e4m3fn), scale=scale)


_own = dict(route=_own_route, grouped=_own_grouped, join=_own_join)


def _plain_route(s):
    x = s["logits"].float()
    x = torch.where(torch.isnan(x), -math.inf, x)
    value, ids = torch.sort(x, dim=-1, descending=True, stable=True)
    value, ids = value[:, : s["top"]], ids[:, : s["top"]]
    there = value != -math.inf
    best = torch.where(value[:, :1] == -math.inf, 0.0, value[:, :1])
    weight = torch.where(there, torch.exp(value - best), 0.0)
    total = weight.sum(-1, keepdim=True) if s["renorm"] else torch.exp(x - best).sum(-1, keepdim=True)
    weight = torch.where(there, weight / torch.where(total == 0, 1.0, total) * s["scale"], 0.0)
    ids = torch.where(there, ids, -1).int()
    offsets, row_token, token_row = _order(ids, x.shape[1])
    return dict(ids=ids, weights=weight, offsets=offsets, row_token=row_token, token_row=token_row)


def _plain_grouped(s):
    x = s["x"].float()
    if s["row_token"] is not None:
        x = x[s["row_token"].long()]
    amax = x.abs().amax(-1, keepdim=True)
    s_x = torch.where(amax > 0, amax / torch.full_like(amax, E4M3_MAX), 1.0)
    codes = (x / s_x).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).float()
    # the rows of each expert side by side, as many places as the busiest one has rows
    offsets = s["offsets"].long()
    place = torch.arange(s["most"], device=x.device)[None, :]
    row = offsets[:-1, None] + place
    there = row < offsets[1:, None]
    acc = codes[row.clamp(max=x.shape[0] - 1)] @ s["wq"].view(torch.float8_e4m3fn).float().transpose(1, 2)
    out = acc[there] * s_x * s["s_w"].repeat_interleave(offsets[1:] - offsets[:-1], dim=0, output_size=x.shape[0])
    if s["gated"]:
        gate, up = out.chunk(2, -1)
        out = gate / (1 + torch.exp(-gate)) * up
    return out.to(torch.bfloat16)


def _norm(x, gamma):
    return x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * gamma.float()


def _plain_join(s):
    y = s["y"].float()
    if s["token_row"] is not None:
        y = (y[s["token_row"].long()] * s["weights"][:, :, None]).sum(1)
    if s["gamma_post"] is not None:
        y = _norm(y, s["gamma_post"])
    if s["g"] is not None:
        y = y * s["g"].float()
    h = s["residual"] * s["h"].float() + s["branch"] * y
    z = _norm(h, s["gamma"])
    codes = scale = None
    if s["codes"]:
        amax = z.abs().amax(-1)
        scale = torch.where(amax > 0, amax / torch.full_like(amax, E4M3_MAX), 1.0)
        codes = (z / scale[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return dict(h=h.to(torch.bfloat16), z=z.to(torch.bfloat16) if s["rows"] else None, codes=codes, scale=scale)


_plain = dict(route=_plain_route, grouped=_plain_grouped, join=_plain_join)


# --------------------------------------------------------------------------- work and exact values

def work(case):
    T = case["tokens"]
    if case["op"] == "route":
        E, k = case["experts"], case["top"]
        return dict(bytes=T * E * (4 if case["dtype"] == "float32" else 2) + 16 * T * k + 4 * (E + 1), flops=3 * T * E)
    K = case["width"]
    if case["op"] == "grouped":
        E, N, rows = case["experts"], case["out"], T * case["top"]
        # experts that are expected to have a row, all chosen alike
        busy = E * (1 - (1 - case["top"] / E) ** T)
        out = N // 2 if case["gated"] else N
        return dict(bytes=busy * N * (K + 4) + 2 * K * (T if case["gather"] else rows) + 2 * rows * out,
                    flops=2 * rows * N * K)
    top = case["top"]
    per = 2 * K * (1 + max(1, top)) + 8 * top + (2 * K if case["gate"] == "token" else 0)
    per += 2 * K + (2 * K if case["rows"] else 0) + (K + 4 if case["codes"] else 0)
    return dict(bytes=T * per + 6 * K, flops=T * K * (10 + 2 * top))


def _codes_of(x):
    """The nearest E4M3 value of each |x| <= 448, ties to the even code, from the format's fields."""
    size = x.abs()
    step = torch.exp2(torch.floor(torch.log2(size.clamp(min=2.0 ** -6))).clamp(min=-6) - 3)
    step = torch.where(size >= 16 * step, 2 * step, step)  # (log2 rounded up to the next binade, or down)
    step = torch.where((size < 8 * step) & (step > 2.0 ** -9), step / 2, step)
    return torch.sign(x) * torch.round(size / step) * step


def _exact_route(case, s):
    x = s["logits"].double()
    order = torch.argsort(-x, dim=1, stable=True)[:, : case["top"]]
    p = torch.softmax(x, 1).gather(1, order)
    if case["renorm"]:
        p = p / p.sum(1, keepdim=True)
    return dict(ids=None, weights=p * case["scale"], offsets=None, row_token=None, token_row=None)


def _exact_grouped(case, s):
    N, K = case["out"], case["width"]
    if 2 * case["tokens"] * case["top"] * N * K > 6e12:
        return None
    x = s["x"] if s["row_token"] is None else s["x"][s["row_token"].long()]
    top = x.float().abs().max(1, keepdim=True).values
    # the scale is an fp32 number by definition: the quotient rounded once
    s_x = torch.where(top == 0, torch.ones_like(top), (top.double() / E4M3_MAX).float())
    codes = _codes_of((x.float() / s_x).double().clamp(-E4M3_MAX, E4M3_MAX))
    out = torch.empty(x.shape[0], N // 2 if case["gated"] else N, dtype=torch.float64, device=DEVICE)
    bounds = s["offsets"].tolist()
    for e, (a, b) in enumerate(zip(bounds[:-1], bounds[1:])):
        if a == b:
            continue
        w = s["wq"][e].view(torch.float8_e4m3fn).double() * s["s_w"][e].double()[:, None]
        y = torch.mm(codes[a:b] * s_x[a:b].double(), w.t())
        out[a:b] = torch.sigmoid(y[:, : N // 2]) * y[:, : N // 2] * y[:, N // 2:] if case["gated"] else y
    return out


def _exact_join(case, s):
    def normed(x, gamma):
        return x * torch.rsqrt((x * x).sum(1, keepdim=True) / case["width"] + EPS) * gamma.double()

    if case["top"]:
        y = torch.zeros(case["tokens"], case["width"], dtype=torch.float64, device=DEVICE)
        for j in range(case["top"]):
            y += s["weights"][:, j: j + 1].double() * s["y"].double().index_select(0, s["token_row"][:, j].long())
    else:
        y = s["y"].double()
    if case["post"]:
        y = normed(y, s["gamma_post"])
    if case["gate"] != "none":
        y = y * s["g"].double()
    h = case["residual"] * s["h"].double() + case["branch"] * y
    z = normed(h, s["gamma"])
    return dict(h=h, z=z if case["rows"] else None, codes=None,
                scale=z.abs().max(1).values / E4M3_MAX if case["codes"] else None)


def exact(case, seed):
    return dict(route=_exact_route, grouped=_exact_grouped, join=_exact_join)[case["op"]](case, prepare(case, seed))
