"""Plain implementations, in 64 bits on the CPU, of the appending rotation, the
operators on the 4-bit paged cache and the verification of drafts, for their tests."""
from __future__ import annotations

import math

import numpy as np
import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def e4m3(codes):
    """uint8 e4m3 codes as float64."""
    return codes.view(torch.float8_e4m3fn).double()


def scale_code(x):
    """float64 (>= 0) to an e4m3 code: to nearest even, saturating; NaN stays NaN.  Found among the 127
    magnitudes of the grid."""
    grid = e4m3(torch.arange(127, dtype=torch.uint8))
    a = x.clamp(max=448.0)
    hi = torch.searchsorted(grid, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    below, above = a - grid[lo], grid[hi] - a
    pick = torch.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    return torch.where(x.isnan(), 127, pick).to(torch.uint8)


def element_code(x):
    """float64 to an e2m1 code with the sign in bit 3: to nearest even, saturating."""
    a = x.abs().clamp(max=6.0)
    hi = torch.searchsorted(E2M1, a.contiguous()).clamp(max=7)
    lo = (hi - 1).clamp(min=0)
    below, above = a - E2M1[lo], E2M1[hi] - a
    pick = torch.where((below < above) | ((below == above) & (lo % 2 == 0)), lo, hi)
    return (pick + 8 * torch.signbit(x)).to(torch.uint8)


def pack(codes):
    return codes[..., 0::2] | (codes[..., 1::2] << 4)


def unpack(packed):
    codes = torch.stack([packed & 15, packed >> 4], -1).flatten(-2).long()
    return torch.where(codes >= 8, -E2M1[codes % 8], E2M1[codes % 8])


def values(packed, scales, unit):
    """float64 values of codes [.., dim / 2] and scale codes [.., dim / 16]."""
    return unpack(packed) * e4m3(scales).repeat_interleave(16, -1) * unit


def quantise(x, unit):
    """x float64 [.., dim]: element codes [.., dim], scale codes [.., dim / 16], and which groups hold
    a NaN (their codes are 0, their scale NaN)."""
    y = x.unflatten(-1, (-1, 16))
    nan = y.isnan().any(-1)
    scale = scale_code(torch.where(nan, math.nan, y.abs().amax(-1) / (6.0 * unit)))
    by = e4m3(scale) * unit
    safe = torch.where((by > 0) & ~nan, by, 1.0)[..., None]
    codes = element_code(torch.where(((by > 0) & ~nan)[..., None], y / safe, 0.0))
    return codes.flatten(-2), scale, nan


def rotate32(x, positions, table, axes, interleaved):
    """x [T, heads, dim] float32, every operation rounded to float32; positions [axes, T]."""
    x, rot = x.float(), table.shape[1]
    pairs = rot // 2
    at = torch.stack([positions[a] for a in (axes or [0] * pairs)], 1).long()       # [T, pairs]
    cos, sin = (table[:, o:o + pairs].gather(0, at)[:, None] for o in (0, pairs))
    first = torch.arange(pairs) * (2 if interleaved else 1)
    second = first + (1 if interleaved else pairs)
    a, b = x[..., first], x[..., second]
    y = x.clone()
    y[..., first], y[..., second] = a * cos - b * sin, b * cos + a * sin
    return y


def store(k, v, caches, scales, slots, k_unit, v_unit):
    """In place: caches [blocks, heads, bs, dim / 2], scales [blocks, heads, bs, dim / 16]; k, v float64
    [T, heads, dim]."""
    blocks, _, bs, _ = caches[0].shape
    kc, ks, _ = quantise(k, k_unit)
    vc, vs, vnan = quantise(v, v_unit)
    vs = torch.where(vnan, torch.zeros_like(vs), vs)
    ks = ks.clone()
    ks[..., 0] = torch.where(vnan.any(-1), torch.full_like(ks[..., 0], 127), ks[..., 0])
    for t, s in enumerate(slots.tolist()):
        if 0 <= s < blocks * bs:
            for cache, scale, c, f in ((caches[0], scales[0], kc, ks), (caches[1], scales[1], vc, vs)):
                cache[s // bs, :, s % bs], scale[s // bs, :, s % bs] = pack(c[t]), f[t]


def attention(q, caches, scales, units, tables, starts, lens, scale, window):
    """Returns out, lse, and what the tolerances are made of: sum p |v| per element, the largest sum
    |q k| of a row's logits, and how many tokens a row sees."""
    T, hq, d = q.shape
    blocks, heads, bs, _ = caches[0].shape
    group = hq // heads
    out = torch.zeros(T, hq, d, dtype=torch.float64)
    size = torch.zeros_like(out)
    reach = torch.zeros(T, hq, dtype=torch.float64)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64)
    count = torch.zeros(T, dtype=torch.float64)
    for i, length in enumerate(lens):
        a, b = starts[i], starts[i + 1]
        keys = [s for s in range(max(length, 0)) if s // bs < tables.shape[1] and 0 <= tables[i, s // bs] < blocks]
        if a == b or not keys:
            continue
        at = torch.tensor(keys)
        block = tables[i].long()[at // bs]
        pos = length - b + torch.arange(a, b)                              # of the queries
        seen = at[None, :] <= pos[:, None]
        if window:
            seen &= at[None, :] > pos[:, None] - window
        some = seen.any(1)
        count[a:b] = seen.sum(1).double()
        for h in range(heads):
            k = values(caches[0][block, h, at % bs], scales[0][block, h, at % bs], units[0])
            v = values(caches[1][block, h, at % bs], scales[1][block, h, at % bs], units[1])
            v = torch.where(seen.any(0)[:, None], v, 0.0)                  # what no row sees may be anything
            x = q[a:b, h * group:(h + 1) * group].double()
            bad = k.isnan().any(1)
            plain = torch.where(k.isnan(), 0.0, k)
            logits = (x @ plain.T * scale).masked_fill(~seen[:, None], -math.inf)
            top = torch.logsumexp(logits, -1)
            p = torch.exp(logits - top[..., None]).masked_fill(~seen[:, None], 0.0)
            hs = slice(h * group, (h + 1) * group)
            out[a:b, hs], size[a:b, hs] = p @ v, p @ v.abs()
            reach[a:b, hs] = (x.abs() @ plain.abs().T * abs(scale)).masked_fill(~seen[:, None], 0.0).amax(-1)
            lse[a:b, hs] = top
            hit = (seen & bad[None]).any(1)                                # a NaN key: all of the row
            out[a:b, hs] = out[a:b, hs].masked_fill(hit[:, None, None], math.nan)
            lse[a:b, hs] = lse[a:b, hs].masked_fill(hit[:, None], math.nan)
            none = torch.arange(a, b)[~some]
            out[none, hs], lse[none, hs] = 0.0, -math.inf
    return out, lse, size, reach, count


def verify(target, ids, starts, u, most, draft=None):
    """tokens, accepted; target, draft: float32 [rows, vocab] on the CPU."""
    n, vocab = len(starts) - 1, target.shape[1]
    tokens = torch.full((n, most + 1), -1, dtype=torch.int32)
    accepted = torch.zeros(n, dtype=torch.int32)
    u64 = u.double().tolist()
    for i in range(n):
        a, b = starts[i], starts[i + 1]
        if not 0 <= a < b <= target.shape[0] or b - a > most + 1:
            continue
        r = a
        while r < b - 1:
            x = int(ids[r])
            if not 0 <= x < vocab:
                break
            q = float(draft[r, x]) if draft is not None else 1.0
            if not u64[r] * q < float(target[r, x]):
                break
            tokens[i, r - a] = x
            r += 1
        accepted[i] = r - a
        rows = [target[r].numpy()]
        if r < b - 1:
            if draft is not None:
                rows.insert(0, target[r].numpy() - draft[r].numpy())
            else:
                w = target[r].numpy().copy()
                if 0 <= int(ids[r]) < vocab:
                    w[int(ids[r])] = 0
                rows.insert(0, w)
        for w in rows:
            with np.errstate(invalid="ignore"):
                w = np.where(w > 0, np.minimum(w, np.float32(1)), np.float32(0)).astype(np.float64)
            below = np.cumsum(np.rint(w * 2.0 ** 40).astype(np.int64))
            if below[-1] > 0:
                aim = min(max(int(math.floor(u64[b - 1] * float(below[-1]))), 0), int(below[-1]) - 1)
                tokens[i, r - a] = int(np.searchsorted(below, aim, side="right"))
                break
    return tokens, accepted
