"""Plain 64-bit forms of the attention block's operators, for the tests: loops
over requests and heads, written from the formulas, sharing nothing with the
CUDA path.  Everything is computed on the host."""
import math

import torch

U_BF16 = 2.0 ** -8   # half a step of bf16, relative
U_FP16 = 2.0 ** -11
SUMS = 2.0 ** -12    # fp32 products, sums and exponentials of values near 1, with room


def e4m3_values() -> torch.Tensor:
    """The value of each of the 256 codes, from the format's fields."""
    got = []
    for code in range(256):
        e, m = (code >> 3) & 15, code & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        got.append(math.nan if code & 127 == 127 else -x if code & 128 else x)
    return torch.tensor(got, dtype=torch.float64)


def attend(q, k, v, scale):
    """(softmax(scale q k^T) v, softmax(scale q k^T) |v|) of one query [D] over
    the given keys and values [n, D]; zeros for n = 0."""
    if k.shape[0] == 0:
        return torch.zeros(v.shape[1], dtype=torch.float64), torch.zeros(v.shape[1], dtype=torch.float64)
    s = (k @ q) * scale
    w = torch.exp(s - s.max())
    w = w / w.sum()
    return w @ v, w @ v.abs()


def prompt(q, k, v, cu, scale):
    """Causal attention over packed sequences, (out, weighted |v|) in 64 bits;
    rows outside every sequence are NaN."""
    q, k, v = (t.detach().cpu().double() for t in (q, k, v))
    T, Hq, D = q.shape
    g = Hq // k.shape[1]
    out = torch.full((T, Hq, D), math.nan, dtype=torch.float64)
    size = torch.zeros(T, Hq, D, dtype=torch.float64)
    bounds = cu.tolist()
    for a, e in zip(bounds[:-1], bounds[1:]):
        n = e - a
        if n == 0:
            continue
        mask = torch.ones(n, n, dtype=torch.bool).triu(1)
        for h in range(Hq):
            s = (q[a:e, h] @ k[a:e, h // g].T * scale).masked_fill(mask, -math.inf)
            w = torch.exp(s - s.max(1, keepdim=True).values)
            w = w / w.sum(1, keepdim=True)
            out[a:e, h] = w @ v[a:e, h // g]
            size[a:e, h] = w @ v[a:e, h // g].abs()
    return out, size


def decode(q, k_cache, v_cache, k_scale, v_scale, table, lens, page, prefix, scale):
    """One query per request over the paged cache, (out, weighted |v|)."""
    values = e4m3_values()
    q = q.detach().cpu().double()
    k_cache, v_cache, table = k_cache.cpu(), v_cache.cpu(), table.cpu()
    n, Hq, D = q.shape
    Hkv = k_cache.shape[1]
    ks, vs = (t.detach().cpu().double().expand(Hkv) for t in (k_scale, v_scale))
    n_pages = k_cache.shape[0] // page
    out = torch.zeros(n, Hq, D, dtype=torch.float64)
    size = torch.zeros(n, Hq, D, dtype=torch.float64)
    for b in range(n):
        slots = []
        for j in range(max(0, min(int(lens[b]), table.shape[1] * page))):
            pg = int(table[0 if j < prefix else b, j // page])
            if 0 <= pg < n_pages:
                slots.append(pg * page + j % page)
        k = values[k_cache[slots].long()]
        v = values[v_cache[slots].long()]
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            out[b, h], size[b, h] = attend(q[b, h], k[:, hk] * ks[hk], v[:, hk] * vs[hk], scale)
    return out, size


def slots(ctx, new, free, page, table, room):
    """(table, slot_mapping, positions, cu_seqlens, seq_lens, pages_used)."""
    table = table.cpu().clone()
    width, taken, t = table.shape[1], 0, 0
    slot, pos, cu = [-1] * room, [0] * room, [0]
    for b, (c, n) in enumerate(zip(ctx.tolist(), new.tolist())):
        c, n = max(c, 0), max(n, 0)
        have, need = min(width, -(-c // page)), min(width, -(-(c + n) // page))
        for j in range(have, need):
            table[b, j] = int(free[taken]) if taken < len(free) else -1
            taken += 1
        for i in range(n):
            if t < room:
                pg = int(table[b, (c + i) // page]) if (c + i) // page < width else -1
                slot[t] = -1 if pg < 0 else pg * page + (c + i) % page
                pos[t] = c + i
            t += 1
        cu.append(min(t, room))
    lens = [max(c, 0) + max(n, 0) for c, n in zip(ctx.tolist(), new.tolist())]
    return table, slot, pos, cu, lens, taken


def norm_rope(x, positions, inv_freq, gamma, eps, interleaved):
    """(rotated, |y_a| + |y_b| of each element's pair) in 64 bits."""
    y = x.detach().cpu().double()
    if gamma is not None:
        y = y / torch.sqrt((y * y).mean(-1, keepdim=True) + eps) * gamma.cpu().double()
    out, size = y.clone(), y.abs()
    for i, f in enumerate(inv_freq):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + len(inv_freq))
        w = positions.cpu().double()[:, None] * f
        c, s = torch.cos(w), torch.sin(w)
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
        size[..., a] = size[..., b] = y[..., a].abs() + y[..., b].abs()
    return out, size


def check(got, ref, tol, what):
    got = got.detach().cpu().double()
    assert got.shape == ref.shape, (what, got.shape, ref.shape)
    bad = ~((got - ref).abs() <= tol) & ~(got.isnan() & ref.isnan()) & ~(got == ref)
    if bad.any():
        at = tuple(torch.nonzero(bad)[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} outside, first at {at}: "
                             f"got {got[at].item()!r}, ref {ref[at].item()!r}, tol {tol[at].item()!r}")
