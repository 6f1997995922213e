"""The expert block's operators in 64 bits, from their definitions, with the
bounds that their outputs have to keep (tests of csrc/moe_route.cu,
gemm_grouped.cu and residual_norm.cu)."""
import torch

E4M3_MAX = 448.0
HALF = dict(bf16=2.0 ** -8, fp32=2.0 ** -24, e4m3=2.0 ** -4)  # half a step, relative


def route(logits, k, renorm, scale):
    """(ids, weights, bound on the weights, offsets, row_token, token_row); on the CPU."""
    x = logits.double().cpu()
    x = torch.where(torch.isnan(x), -torch.inf, x)
    T, E = x.shape
    order = torch.argsort(-x, dim=1, stable=True)[:, :k]
    value = x.gather(1, order)
    there = value > -torch.inf
    best = torch.where(there[:, :1], value[:, :1], 0.0)
    p = torch.exp(value - best)
    total = (p if renorm else torch.exp(x - best)).sum(1, keepdim=True)
    w = torch.where(there, p / torch.where(total > 0, total, 1.0) * scale, 0.0)
    # the difference is rounded to fp32 and exp multiplies its error (its size times 2^-24, on
    # average over the sum at most log E = 7 times), the rest (exp, sum of up to 32 a lane and 5
    # levels, quotient, product) is within 50 roundings
    tol = w.abs() * (torch.where(there, best - value, 0.0) + 57) * HALF["fp32"]
    ids = torch.where(there, order, -1)
    pairs = [(e, t, j) for t, row in enumerate(ids.tolist()) for j, e in enumerate(row) if e >= 0]
    pairs.sort(key=lambda q: (q[0], q[1]))
    row_token = torch.full((T * k,), -1, dtype=torch.int32)
    token_row = torch.full((T, k), -1, dtype=torch.int32)
    if pairs:
        e, t, j = (torch.tensor(v) for v in zip(*pairs))
        row_token[: len(pairs)] = t.int()
        token_row[t, j] = torch.arange(len(pairs), dtype=torch.int32)
        counts = torch.bincount(e, minlength=E)
    else:
        counts = torch.zeros(E, dtype=torch.int64)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).int()
    return ids.int(), w, tol, offsets, row_token, token_row


def quant(x):
    """Codes' values and scales of rows, by the rule of fp8_quant_per_token."""
    x = x.float()
    amax = x.abs().amax(1)
    # (through 64 bits, as a quotient by a number may be taken as a product with its reciprocal)
    s = torch.where(amax > 0, (amax.double() / E4M3_MAX).float(), torch.ones_like(amax))
    codes = (x / s[:, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return codes, s


def grouped(xv, s_tok, wv, s_w, offsets, swiglu):
    """(y, bound) of code values xv [R, K], wv [E, N, K] (float8); NaN outside the groups."""
    R, K = xv.shape
    E, N, _ = wv.shape
    F = N // 2 if swiglu else N
    y = torch.full((R, F), float("nan"), dtype=torch.float64, device=xv.device)
    tol = torch.zeros_like(y)
    at = offsets.tolist()
    for e in range(E):
        a, b = at[e], at[e + 1]
        if a >= b:
            continue
        x, w = xv[a:b].double(), wv[e].double()
        scale = s_tok[a:b, None].double() * s_w[e][None].double()
        v = x @ w.T * scale
        # each MMA step adds 32 products to the sum with an error below 2 units of 2^-23 of what it
        # adds and what it has; two products with the scales
        err = (x.abs() @ w.abs().T) * scale.abs() * (K / 32 + 4) * 2.0 ** -22
        if swiglu:
            g, u, eg, eu = v[:, :F], v[:, F:], err[:, :F], err[:, F:]
            s = torch.sigmoid(g)
            y[a:b] = s * g * u
            # |silu'| < 1.1; silu in fp32 (exp of an argument of up to 100: 2^-17)
            tol[a:b] = 1.1 * eg * u.abs() + (s * g).abs() * eu + eg * eu * 1.1 + (s * g * u).abs() * 2.0 ** -16
        else:
            y[a:b], tol[a:b] = v, err
    return y, tol + y.abs().nan_to_num(0) * HALF["bf16"] + 1e-38


def residual_norm(h, y, gamma, eps, gamma_post, gate, rs, bs, token_row, weights):
    """(h', z, s, bounds of h_out, z_out and s) in 64 bits."""
    h, T, K = h.double(), h.shape[0], h.shape[1]
    if token_row is None:
        b = y.double()
        size = b.abs()
    else:
        b = torch.zeros_like(h)
        size = torch.zeros_like(h)
        for j in range(token_row.shape[1]):
            r = token_row[:, j].long()
            ok = (r >= 0) & (r < y.shape[0])
            w = weights[:, j].double() if weights is not None else torch.ones(T, dtype=torch.float64, device=h.device)
            v = torch.where(ok[:, None], y.double()[r.clamp(0, max(0, y.shape[0] - 1))] * w[:, None], 0.0) \
                if y.shape[0] else torch.zeros_like(h)
            b, size = b + v, size + v.abs()
    if gamma_post is not None:
        inv = 1 / torch.sqrt(b.square().mean(1, keepdim=True) + eps)
        b, size = b * inv * gamma_post.double(), size * inv * gamma_post.double().abs()
    if gate is not None:
        b, size = b * gate.double(), size * gate.double().abs()
    out = rs * h + bs * b
    # sizes of the terms; every sum over the row or over the rows of a token is within 64 roundings
    size = (abs(rs) * h.abs() + abs(bs) * size) * 64 * HALF["fp32"]
    if gamma is None:
        return out, None, None, out.abs() * HALF["bf16"] + size, None, None
    inv = 1 / torch.sqrt(out.square().mean(1, keepdim=True) + eps)
    z = out * inv * gamma.double()
    # (the row's norm takes the terms' errors once more, and 64 roundings of its own)
    err = (size + size.square().mean(1, keepdim=True).sqrt() * inv * out.abs()) * inv * gamma.double().abs()
    err = err + z.abs() * 64 * HALF["fp32"]
    amax = z.abs().amax(1)
    s = torch.where(amax > 0, amax / E4M3_MAX, torch.ones_like(amax))
    return (out, z, s, out.abs() * HALF["bf16"] + size + 1e-38, z.abs() * HALF["bf16"] + err + 1e-38,
            err.amax(1) / E4M3_MAX + s * 4 * HALF["fp32"])
