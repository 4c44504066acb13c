"""Plain implementations, in 64 bits on the CPU, of the operators on the 8-bit
paged cache, for their tests."""
from __future__ import annotations

import math

import torch


def decode(codes):
    """uint8 e4m3 codes as float64."""
    return codes.view(torch.float8_e4m3fn).double()


def encode(x):
    """float64 values to e4m3 codes: to nearest even, saturating; NaN stays NaN.  Every finite value
    is found among the 127 magnitudes of the grid."""
    grid = decode(torch.arange(127, dtype=torch.uint8))
    a = x.abs().clamp(max=448.0)
    hi = torch.searchsorted(grid, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    below, above = a - grid[lo], grid[hi] - a
    pick = torch.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    code = pick.to(torch.uint8) | torch.where(torch.signbit(x), 128, 0).to(torch.uint8)
    return torch.where(torch.isnan(x), torch.tensor(127, dtype=torch.uint8), code)


def same_codes(a, b):
    """Equal values; a NaN equals a NaN and -0 equals 0."""
    x, y = decode(a), decode(b)
    return bool(((x == y) | (x.isnan() & y.isnan())).all())


def block_scale(amax):
    """The smallest power of two, 2^-64 at least, that brings amax to at most 448."""
    s = 2.0 ** -64
    while s * 448 < amax:
        s *= 2
    return s


def store(k, v, kc, vc, ks, vs, slots, num_blocks):
    """In place; caches [slots, heads, dim] uint8, scales [blocks, heads], all on the CPU."""
    bs = kc.shape[0] // num_blocks
    runs, previous = [], None
    for t, s in enumerate(slots.tolist()):
        b = s // bs if 0 <= s < kc.shape[0] else None
        if b is not None:
            if b != previous:
                runs.append((b, []))
            runs[-1][1].append(t)
        previous = b
    for x, cache, scale in ((k, kc, ks), (v, vc, vs)):
        x = x.double()
        for b, tokens in runs:
            offsets = [int(slots[t]) - b * bs for t in tokens]
            first = min(offsets)
            lines = x[tokens]                                             # [run, heads, dim]
            mags = torch.where(lines.isfinite(), lines.abs(), 0.0).amax((0, 2))
            for h in range(cache.shape[1]):
                new = block_scale(float(mags[h]))
                if first > 0:
                    old = float(scale[b, h])
                    if old >= new:
                        new = old
                    else:
                        held = cache[b * bs:b * bs + first, h]
                        cache[b * bs:b * bs + first, h] = encode(decode(held) * (old / new))
                scale[b, h] = new
                for t, o in zip(tokens, offsets):
                    cache[b * bs + o, h] = encode(x[t, h] / new)


def attention(q, kc, vc, ks, vs, tables, starts, lens, scale, window, weights=None):
    """q [T, hq, d]; caches [slots, heads, d] uint8.  Returns out, lse, and what the tolerances are
    made of: sum p |v| per element and the largest sum |q k| of a row's logits."""
    T, hq, d = q.shape
    blocks, heads = ks.shape
    bs, group = kc.shape[0] // blocks, hq // heads
    out = torch.zeros(T, hq, d, dtype=torch.float64)
    size = torch.zeros_like(out)
    reach = torch.zeros(T, hq, dtype=torch.float64)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64)
    for i, length in enumerate(lens):
        a, b = starts[i], starts[i + 1]
        keys = [s for s in range(max(length, 0)) if s // bs < tables.shape[1] and 0 <= tables[i, s // bs] < blocks]
        if a == b or not keys:
            continue
        at = torch.tensor(keys)
        block = tables[i].long()[at // bs]
        slot = block * bs + at % bs
        pos = length - b + torch.arange(a, b)                              # of the queries
        seen = at[None, :] <= pos[:, None]
        if window:
            seen &= at[None, :] > pos[:, None] - window
        some = seen.any(1)
        for h in range(heads):
            k = decode(kc[slot, h]) * ks[block, h].double()[:, None]
            v = decode(vc[slot, h]) * vs[block, h].double()[:, None]
            x = q[a:b, h * group:(h + 1) * group].double()
            logits = (x @ k.T * scale).masked_fill(~seen[:, None], -math.inf)
            top = torch.logsumexp(logits, -1)
            p = torch.exp(logits - top[..., None]).masked_fill(~seen[:, None], 0.0)
            hs = slice(h * group, (h + 1) * group)
            # a value that is NaN reaches the rows that see it and no other
            plain = torch.where(v.isnan(), 0.0, v)
            out[a:b, hs] = p @ plain
            hit = (seen.double() @ v.isnan().double()) > 0
            out[a:b, hs] = out[a:b, hs].masked_fill(hit[:, None, :], math.nan)
            size[a:b, hs] = p @ plain.abs()
            far = (x.abs() @ torch.where(k.isnan(), 0.0, k).abs().T * abs(scale)).masked_fill(~seen[:, None], 0.0)
            reach[a:b, hs] = far.amax(-1)
            lse[a:b, hs] = top
            if weights is not None:
                weights.index_add_(0, slot, p.sum((0, 1)))
            none = torch.arange(a, b)[~some]
            out[none, hs], lse[none, hs] = 0.0, -math.inf
    return out, lse, size, reach


def carried(q, kc, vc, ks, vs, tables, starts, lens, scale, window):
    """Per (query, head) of `attention`'s rows: the largest p * v_scale of a token it sees, and how many it sees."""
    T, hq, _ = q.shape
    blocks, heads = ks.shape
    bs, group = kc.shape[0] // blocks, hq // heads
    most, count = torch.zeros(T, hq, dtype=torch.float64), torch.zeros(T, dtype=torch.float64)
    for i, length in enumerate(lens):
        a, b = starts[i], starts[i + 1]
        keys = [s for s in range(max(length, 0)) if s // bs < tables.shape[1] and 0 <= tables[i, s // bs] < blocks]
        if a == b or not keys:
            continue
        at = torch.tensor(keys)
        block = tables[i].long()[at // bs]
        pos = length - b + torch.arange(a, b)
        seen = at[None, :] <= pos[:, None]
        if window:
            seen &= at[None, :] > pos[:, None] - window
        count[a:b] = seen.sum(1).double()
        for h in range(heads):
            k = decode(kc[block * bs + at % bs, h]) * ks[block, h].double()[:, None]
            logits = (q[a:b, h * group:(h + 1) * group].double() @ k.T * scale).masked_fill(~seen[:, None], -math.inf)
            p = torch.exp(logits - torch.logsumexp(logits, -1)[..., None]).masked_fill(~seen[:, None], 0.0)
            most[a:b, h * group:(h + 1) * group] = (p * vs[block, h].double()).amax(-1)
    return most, count


def evict(kc, vc, ks, vs, weights, tables, lens, fresh, budget, first, last):
    """In place on the CPU tensors; returns new lengths and kept positions."""
    blocks = ks.shape[0]
    bs = kc.shape[0] // blocks
    kept = torch.full((len(lens), budget), -1, dtype=torch.int32)
    new = []
    for i, length in enumerate(lens):
        slot = [int(tables[i, s // bs]) * bs + s % bs for s in range(length)]
        chosen = list(range(length))
        if length > budget:
            def rank(s):
                w = float(weights[slot[s]])
                return (math.isnan(w), -w if not math.isnan(w) else 0.0, s)
            middle = sorted(range(first, length - last), key=rank)[:budget - first - last]
            chosen = sorted(list(range(first)) + middle + list(range(length - last, length)))
        new.append(len(chosen))
        kept[i, :len(chosen)] = torch.tensor(chosen, dtype=torch.int32)
        to = [int(fresh[i, j // bs]) * bs + j % bs for j in range(len(chosen))]
        for j in range(0, len(chosen), bs):
            group = range(j, min(j + bs, len(chosen)))
            for cache, scale in ((kc, ks), (vc, vs)):
                old = torch.stack([scale[slot[chosen[m]] // bs] for m in group]).double()
                now = old.amax(0)
                for m, o in zip(group, old):
                    cache[to[m]] = encode(decode(cache[slot[chosen[m]]]) * (o / now)[:, None])
                scale[to[j] // bs] = now.float()
            for m in group:
                weights[to[m]] = weights[slot[chosen[m]]]
    return new, kept
