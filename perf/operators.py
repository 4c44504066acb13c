"""Measured cases of the operators on a paged KV cache held in 8 bits.

The cache keeps one e4m3 byte per element and one float32 scale for each
(block of tokens, KV head), a power of two when the store made it.  Three
operators work on it:

* the store quantises a step's new K/V lines into their blocks,
* the attention reads the cache for a prepared batch (single tokens, prompt
  chunks or both), and on request adds up the attention weight that each
  cached token received,
* the eviction keeps the tokens of a request that received most weight and
  copies them into new blocks.

``run`` computes them with elementary torch operations, or, with ``own`` set,
through paged_kv_prep_gb300.
"""
import math
import random

import torch

own = False

E4M3_MAX = 448.0
MIN_EXPONENT = -64      # the smallest scale the store gives a block is 2^-64
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _store(name, requests, tokens, block, heads=8, dim=128, dtype="bf16", lens_seed=1):
    return {"name": name, "op": "store", "requests": requests, "tokens": tokens, "block": block,
            "heads": heads, "dim": dim, "dtype": dtype, "lens_seed": lens_seed}


def _attention(name, decodes, ctx, block, group, chunks=0, chunk_lo=0, chunk_hi=0, ctx_lo=1,
               window=0, weights=False, heads=8, dim=128, dtype="bf16", lens_seed=1):
    return {"name": name, "op": "attention", "decodes": decodes, "ctx_lo": ctx_lo, "ctx": ctx,
            "block": block, "group": group, "chunks": chunks, "chunk_lo": chunk_lo,
            "chunk_hi": chunk_hi, "window": window, "weights": weights, "heads": heads,
            "dim": dim, "dtype": dtype, "lens_seed": lens_seed}


def _evict(name, requests, ctx, budget, first, last, block, ctx_lo=1, heads=8, dim=128,
           lens_seed=1):
    return {"name": name, "op": "evict", "requests": requests, "ctx_lo": ctx_lo, "ctx": ctx,
            "budget": budget, "first": first, "last": last, "block": block, "heads": heads,
            "dim": dim, "lens_seed": lens_seed}


def listed():
    return [
        # one decode step of a small batch: eight requests, one line each; latency counts
        _store("store_8_decodes", 8, 8, 16),
        # the large step's token budget: thousands of decodes beside prompt chunks, 32-token blocks
        _store("store_16384_tokens", 4096, 16384, 32),
        # the smallest serving batch: eight single tokens on short contexts
        _attention("attn_8_decodes", 8, 200, 16, 4),
        # an ordinary decode batch, contexts spread up to 8192 (8 KV heads shared by 32 heads)
        _attention("attn_256_decodes", 256, 8192, 16, 4),
        # few requests with very long contexts (64 heads): the work is along the cache
        _attention("attn_4_long_decodes", 4, 131072, 32, 8, ctx_lo=65536),
        # chunked prefill beside decodes, contexts up to 16384
        _attention("attn_mixed_prefill", 64, 16384, 16, 4, chunks=6, chunk_lo=512, chunk_hi=2048),
        # a sliding-window group: decodes and short chunks, blocks before the window are freed
        _attention("attn_window_fp16", 231, 32768, 16, 4, chunks=25, chunk_lo=1, chunk_hi=256,
                   window=4096, dtype="fp16"),
        # a decode step that also adds up the attention each cached token receives
        _attention("attn_weights_decodes", 64, 8192, 16, 4, weights=True),
        # the same for a prompt's chunks, where the weights of a prompt come from
        _attention("attn_weights_prefill", 0, 8192, 16, 4, chunks=3, chunk_lo=512, chunk_hi=2048,
                   weights=True),
        # a few short requests shrink to 64 tokens; latency counts
        _evict("evict_8_short", 8, 200, 64, 4, 16, 16),
        # a decode batch at its memory limit: contexts up to 8192 shrink to 2048
        _evict("evict_256_requests", 256, 8192, 2048, 4, 256, 16),
        # long prompts shrink to an odd budget that ends inside a block
        _evict("evict_4_long", 4, 131072, 8191, 4, 1024, 32, ctx_lo=65536),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["store", "attention", "attention", "attention", "evict"])
    block = rng.choice([16, 32])
    heads, dim = rng.choice([(8, 128), (4, 128), (2, 128), (8, 64), (1, 128)])
    seed = rng.randrange(1 << 30)
    if op == "store":
        requests = _log_int(rng, 1, 4096)
        c = _store("", requests, min(16384, requests * _log_int(rng, 1, 512)), block, heads, dim,
                   rng.choice(["bf16", "fp16"]), seed)
    elif op == "evict":
        ctx = _log_int(rng, 64, 131072)
        requests = _log_int(rng, 1, max(1, min(256, (1 << 19) // ctx)))
        budget = _log_int(rng, 16, min(8192, ctx))
        first = rng.randint(0, min(4, budget // 4))
        c = _evict("", requests, ctx, budget, first, rng.randint(0, budget // 2), block,
                   rng.randint(1, ctx), heads, dim, seed)
    else:
        group = rng.choice([1, 2, 4, 5, 7, 8])
        kind = rng.choice(["decode", "decode", "mixed", "chunks"])
        window = rng.choice([0, 0, 0, _log_int(rng, 64, 8192)])
        dtype = rng.choice(["bf16", "bf16", "fp16"])
        weights = rng.random() < 0.3
        if kind == "decode":
            ctx = _log_int(rng, 32, 131072)
            decodes = _log_int(rng, 1, max(1, min(512, (1 << 20) // ctx)))
            c = _attention("", decodes, ctx, block, group, ctx_lo=rng.randint(1, ctx),
                           window=window, weights=weights, heads=heads, dim=dim, dtype=dtype,
                           lens_seed=seed)
        else:
            ctx = _log_int(rng, 64, 16384)
            hi = _log_int(rng, 2, min(2048, ctx))
            c = _attention("", rng.randint(1, 64) if kind == "mixed" else 0, ctx, block, group,
                           chunks=rng.randint(1, 5), chunk_lo=rng.randint(1, hi), chunk_hi=hi,
                           window=window, weights=weights, heads=heads, dim=dim, dtype=dtype,
                           lens_seed=seed)
    del c["name"]
    return c


# --------------------------------------------------------------------------
# the lengths a case stands for (the same for every seed of its values)
# --------------------------------------------------------------------------
def _lengths(case):
    """(scheduled tokens, sequence length) of each request, fewer tokens first as a prepared
    batch has them."""
    rng = random.Random(case["lens_seed"])
    if case["op"] == "store":
        n, total = case["requests"], case["tokens"]
        counts = [1] * n
        left = total - n
        while left > 0:      # the first requests hold prompt chunks, the rest decode
            c = min(left, rng.randint(1, 4095))
            counts[rng.randrange(n)] += c
            left -= c
        reqs = [(c, c + rng.randint(0, 4 * case["block"])) for c in counts]
    elif case["op"] == "evict":
        reqs = [(0, rng.randint(case["ctx_lo"], case["ctx"])) for _ in range(case["requests"])]
    else:
        reqs = [(1, rng.randint(case["ctx_lo"], case["ctx"])) for _ in range(case["decodes"])]
        for _ in range(case["chunks"]):
            c = rng.randint(case["chunk_lo"], case["chunk_hi"])
            reqs.append((c, rng.randint(c, max(c, case["ctx"]))))
    return sorted(reqs, key=lambda r: r[0])


def _pairs(count, length, window):
    """Visible (query, key) pairs of one request, and the cached tokens that some query sees."""
    if not window or window >= length:
        return count * length - count * (count - 1) // 2, length
    pairs = sum(min(p + 1, window) for p in range(length - count, length))
    return pairs, length - max(0, length - count - window + 1)


def work(case):
    reqs, line = _lengths(case), case["heads"] * case["dim"]
    if case["op"] == "store":
        t = sum(c for c, _ in reqs)
        blocks = sum(-(-length // case["block"]) - (length - c) // case["block"] for c, length in reqs)
        return {"bytes": 2 * t * line * 3 + 8 * t + 2 * blocks * case["heads"] * 4, "flops": 4 * t * line}
    if case["op"] == "evict":
        kept = [min(length, case["budget"]) for _, length in reqs]
        moved = sum(kept)
        seen = sum(length for _, length in reqs)
        scales = 2 * case["heads"] * 4 * (seen + moved) // case["block"]
        return {"bytes": 4 * seen + 2 * moved * (2 * line + 4) + scales, "flops": 2 * 2 * moved * line}
    heads = case["heads"] * case["group"]
    tokens = sum(c for c, _ in reqs)
    pairs = [_pairs(c, length, case["window"]) for c, length in reqs]
    seen = sum(p[1] for p in pairs)
    byte = 2 * seen * line + 2 * seen * case["heads"] * 4 // case["block"]
    byte += 2 * tokens * heads * case["dim"] * 2 + tokens * heads * 4
    if case["weights"]:
        byte += 8 * seen
    return {"bytes": byte, "flops": 4 * case["dim"] * heads * sum(p[0] for p in pairs)}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _scale_of(amax):
    """The smallest power of two that brings amax to at most 448."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(min=MIN_EXPONENT)
    e = torch.where(amax > 0, e, MIN_EXPONENT)
    return ((e.int() + 127) << 23).view(torch.float32)      # 2^e, made from its bits


def _filled_cache(gen, blocks, case):
    """A cache whose lines were stored block by block from normally distributed values; some
    channels are larger than others, as keys have them."""
    bs, h, d = case["block"], case["heads"], case["dim"]
    channel = torch.exp(0.5 * torch.randn(h, d, generator=gen, device="cuda"))
    codes = torch.empty(blocks, bs, h, d, dtype=torch.uint8, device="cuda")
    scale = torch.empty(blocks, h, device="cuda")
    step = max(1, (1 << 28) // (bs * h * d))
    for a in range(0, blocks, step):
        x = torch.randn(min(step, blocks - a), bs, h, d, generator=gen, device="cuda") * channel
        s = _scale_of(x.abs().amax(dim=(1, 3)))
        codes[a:a + step] = (x / s[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scale[a:a + step] = s
    return codes.view(blocks * bs, h * d), scale


def _tables(gen, lens, bs, width, first_blocks=None):
    """Block tables of distinct blocks in random order (-1 past a request's blocks and before its
    window), and how many blocks they name."""
    n = len(lens)
    logical = torch.arange(width, device="cuda")[None, :]
    have = torch.tensor([-(-x // bs) for x in lens], device="cuda")[:, None]
    first = torch.tensor(first_blocks or [0] * n, device="cuda")[:, None]
    used = (logical < have) & (logical >= first)
    total = int(used.sum())
    table = torch.full((n, width), -1, dtype=torch.int32, device="cuda")
    table[used] = torch.randperm(total, generator=gen, device="cuda").to(torch.int32)
    return table, total


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    reqs = _lengths(case)
    counts, lens = [r[0] for r in reqs], [r[1] for r in reqs]
    bs, h, d = case["block"], case["heads"], case["dim"]
    s = {"case": case, "counts": counts, "lens": lens,
         "seq_lens": torch.tensor(lens, dtype=torch.int32, device="cuda")}
    width = -(-max(lens) // bs)
    if case["op"] == "evict":
        table, blocks = _tables(gen, lens, bs, width)
        kept = [min(x, case["budget"]) for x in lens]
        fresh, more = _tables(gen, kept, bs, -(-case["budget"] // bs))
        s["block_tables"] = table
        s["new_block_tables"] = torch.where(fresh >= 0, fresh + blocks, fresh)
        blocks += more
        # accumulated attention is heavy-tailed: a few tokens hold most of it, many hold
        # next to nothing, and tokens that no query has reached yet hold zero
        w = torch.exp(3.0 * torch.randn(blocks * bs, generator=gen, device="cuda"))
        s["weights"] = w * (torch.rand(blocks * bs, generator=gen, device="cuda") < 0.9)
    else:
        first = None
        if case["op"] == "attention" and case["window"]:
            first = [max(0, x - c - case["window"] + 1) // bs for c, x in reqs]
        s["block_tables"], blocks = _tables(gen, lens, bs, width, first)
    s["k_cache"], s["k_scale"] = _filled_cache(gen, blocks, case)
    s["v_cache"], s["v_scale"] = _filled_cache(gen, blocks, case)
    if case["op"] == "evict":
        return s
    starts = [0]
    for c in counts:
        starts.append(starts[-1] + c)
    tokens, dtype = starts[-1], DTYPES[case["dtype"]]
    s["query_start_loc"] = torch.tensor(starts, dtype=torch.int32, device="cuda")
    if case["op"] == "store":
        # the fused projection's rows: K and V are views of it, and outliers come now and then
        rows = torch.randn(tokens, 2 * h * d, generator=gen, device="cuda")
        rows *= torch.exp2(torch.randint(-2, 3, (tokens, 1), generator=gen, device="cuda"))
        rows = rows.to(dtype)
        s["k"], s["v"] = rows[:, :h * d], rows[:, h * d:]
        req = torch.repeat_interleave(torch.arange(len(reqs), device="cuda"),
                                      torch.tensor(counts, device="cuda"))
        pos = torch.arange(tokens, device="cuda") - s["query_start_loc"][req]
        pos = pos + (s["seq_lens"] - torch.tensor(counts, device="cuda"))[req]
        s["slot_mapping"] = s["block_tables"][req, pos // bs].long() * bs + pos % bs
        return s
    hq = h * case["group"]
    rows = torch.randn(tokens, (hq + 2 * h) * d, generator=gen, device="cuda").to(dtype)
    s["q"] = rows[:, :hq * d].view(tokens, hq, d)
    s["softmax_scale"] = d ** -0.5
    if case["weights"]:
        s["weights_before"] = torch.rand(blocks * bs, generator=gen, device="cuda")
        s["weights"] = torch.empty_like(s["weights_before"])
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"store": _own_store, "attention": _own_attention, "evict": _own_evict}[op](state)
    return {"store": _plain_store, "attention": _plain_attention, "evict": _plain_evict}[op](state)


def _cache_outputs(s):
    return {"k_cache": s["k_cache"].view(torch.float8_e4m3fn), "k_scale": s["k_scale"],
            "v_cache": s["v_cache"].view(torch.float8_e4m3fn), "v_scale": s["v_scale"]}


def _own_store(s):
    import paged_kv_prep_gb300 as pkv

    pkv.kv8_store(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                  s["slot_mapping"])
    return _cache_outputs(s)


def _own_attention(s):
    import paged_kv_prep_gb300 as pkv

    case = s["case"]
    if case["weights"]:
        s["weights"].copy_(s["weights_before"])
    out, lse = pkv.kv8_attention(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                 s["block_tables"], s["query_start_loc"], s["seq_lens"],
                                 softmax_scale=s["softmax_scale"], window=case["window"],
                                 weights=s["weights"] if case["weights"] else None)
    return {"out": out, "lse": lse, "weights": s["weights"]} if case["weights"] else {"out": out, "lse": lse}


def _own_evict(s):
    import paged_kv_prep_gb300 as pkv

    case = s["case"]
    new_lens, kept = pkv.kv8_evict(s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"],
                                   s["weights"], s["block_tables"], s["seq_lens"],
                                   s["new_block_tables"], case["budget"],
                                   keep_first=case["first"], keep_last=case["last"])
    return {"seq_lens": new_lens, "kept": kept, "weights": s["weights"], **_cache_outputs(s)}


def _codes(cache, case):
    return cache.view(torch.float8_e4m3fn).view(-1, case["block"], case["heads"], case["dim"])


def _store_one(x, cache, scale, slots, case):
    bs, h, d = case["block"], case["heads"], case["dim"]
    x = x.reshape(-1, h, d).float()
    block, offset = slots // bs, slots % bs
    # the step's tokens of one block stand next to each other
    starts = torch.ones_like(block, dtype=torch.bool)
    starts[1:] = block[1:] != block[:-1]
    run_of = torch.cumsum(starts, 0) - 1
    touched = block[starts]
    runs = touched.numel()
    first = torch.full((runs,), bs, device=x.device).scatter_reduce(0, run_of, offset, "amin")
    amax = torch.zeros(runs, h, device=x.device).index_reduce_(0, run_of, x.abs().amax(2), "amax")
    held = torch.arange(bs, device=x.device)[None, :] < first[:, None]      # lines kept from before
    before = scale[touched]
    after = torch.maximum(_scale_of(amax), torch.where(first[:, None] > 0, before, 0.0))
    codes = _codes(cache, case)
    old = codes[touched]
    again = (old.float() * (before / after)[:, None, :, None]).to(torch.float8_e4m3fn)
    keep = held[:, :, None, None]
    codes.view(torch.uint8)[touched] = torch.where(keep, again.view(torch.uint8), old.view(torch.uint8))
    scale[touched] = after
    new = (x / after[run_of][:, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    codes.view(torch.uint8)[block, offset] = new.view(torch.uint8)


def _plain_store(s):
    _store_one(s["k"], s["k_cache"], s["k_scale"], s["slot_mapping"], s["case"])
    _store_one(s["v"], s["v_cache"], s["v_scale"], s["slot_mapping"], s["case"])
    return _cache_outputs(s)


def _groups(s):
    """Requests a..b that are computed together, so that their padded logits stay within 8 GB."""
    case, at, out = s["case"], 0, []
    hq = case["heads"] * case["group"]
    while at < len(s["lens"]):
        end, most_c, most_l = at, 0, 0
        while end < len(s["lens"]):
            c, x = max(most_c, s["counts"][end]), max(most_l, s["lens"][end])
            size = (end + 1 - at) * x * max(c * hq, case["heads"] * case["dim"])
            if end > at and size > 1 << 31:
                break
            end, most_c, most_l = end + 1, c, x
        out.append((at, end, most_c, most_l))
        at = end
    return out


def _plain_attention(s):
    case = s["case"]
    bs, h, d, group = case["block"], case["heads"], case["dim"], case["group"]
    q = s["q"]
    tokens = q.shape[0]
    out = torch.zeros(tokens, h * group, d, device=q.device)
    lse = torch.full((tokens, h * group), -math.inf, device=q.device)
    kc, vc = _codes(s["k_cache"], case), _codes(s["v_cache"], case)
    if case["weights"]:
        s["weights"].copy_(s["weights_before"])
    for a, b, count, length in _groups(s):
        n = b - a
        blocks = -(-length // bs)
        length = blocks * bs
        table = s["block_tables"][a:b, :blocks].long()
        real = table >= 0
        table = table.clamp(min=0)
        k = kc[table].float() * s["k_scale"][table][:, :, None, :, None]
        v = vc[table].float() * s["v_scale"][table][:, :, None, :, None]
        k = k.view(n, length, h, d).permute(0, 2, 3, 1)
        v = v.view(n, length, h, d).permute(0, 2, 1, 3)
        starts, ends = s["query_start_loc"][a:b, None].long(), s["query_start_loc"][a + 1:b + 1, None].long()
        row = starts + torch.arange(count, device=q.device)
        valid = row < ends
        pos = s["seq_lens"][a:b, None].long() - (ends - row)                 # [n, count]
        x = q[row.clamp(max=tokens - 1)].float().view(n, count, h, group, d)
        x = x.permute(0, 2, 3, 1, 4).reshape(n, h, group * count, d)
        logits = torch.matmul(x, k).mul_(s["softmax_scale"]).view(n, h, group, count, length)
        key = torch.arange(length, device=q.device)
        seen = (key <= pos[:, :, None]) & real.repeat_interleave(bs, 1)[:, None, :] & valid[:, :, None]
        if case["window"]:
            seen &= key > pos[:, :, None] - case["window"]
        logits.masked_fill_(~seen[:, None, None], -math.inf)
        top = logits.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
        p = logits.sub_(top).exp_()
        total = p.sum(-1, keepdim=True)
        mean = torch.matmul(p.view(n, h, group * count, length), v)
        mean = mean.view(n, h, group, count, d) / torch.where(total == 0, 1.0, total)
        found = (top + torch.log(total)).squeeze(-1)
        out[row[valid]] = mean.permute(0, 3, 1, 2, 4)[valid].reshape(-1, h * group, d)
        lse[row[valid]] = found.permute(0, 3, 1, 2)[valid].reshape(-1, h * group)
        if case["weights"]:
            p /= torch.where(total == 0, 1.0, total)
            got = p.sum((1, 2, 3)).view(n, blocks, bs)
            s["weights"].view(-1, bs)[table[real]] += got[real]
    answer = {"out": out.to(q.dtype), "lse": lse}
    if case["weights"]:
        answer["weights"] = s["weights"]
    return answer


def _plain_evict(s):
    case, device = s["case"], s["k_cache"].device
    bs, budget = case["block"], case["budget"]
    table, fresh, lens = s["block_tables"].long(), s["new_block_tables"].long(), s["seq_lens"].long()[:, None]
    n, width = table.shape
    pos = torch.arange(width * bs, device=device)[None, :].expand(n, -1)
    slot = table.repeat_interleave(bs, 1) * bs + pos % bs
    w = s["weights"][slot.clamp(min=0)]
    w = torch.where(torch.isnan(w), -math.inf, w)
    # 2: kept in any case, 1: by weight, 0: past the end
    tier = (pos < lens).int() + ((pos < lens) & ((pos < case["first"]) | (pos >= lens - case["last"]))).int()
    order = torch.sort(w, dim=1, descending=True, stable=True).indices
    order = order.gather(1, torch.sort(tier.gather(1, order), dim=1, descending=True, stable=True).indices)
    new_lens = lens.clamp(max=budget)
    if order.shape[1] < budget:
        order = torch.nn.functional.pad(order, (0, budget - order.shape[1]), value=0)
    place = torch.arange(budget, device=device)[None, :]
    real = place < new_lens
    kept = torch.where(real, order[:, :budget], width * bs).sort(1).values
    src_slot = slot.gather(1, torch.where(real, kept, 0))
    req = torch.arange(n, device=device)[:, None].expand(n, budget)
    dst_block = fresh[req, place // bs].clamp(min=0)
    src, dst = src_slot[real], (dst_block * bs + place % bs)[real]
    for cache, scale in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])):
        codes = _codes(cache, case).view(torch.uint8).view(-1, case["heads"], case["dim"])
        before = scale[src // bs]
        touched = torch.unique(dst // bs)
        scale[touched] = 0.0
        scale.index_reduce_(0, dst // bs, before, "amax")
        ratio = before / scale[dst // bs]
        line = codes[src].view(torch.float8_e4m3fn).float() * ratio[:, :, None]
        codes[dst] = line.to(torch.float8_e4m3fn).view(torch.uint8)
    s["weights"][dst] = s["weights"][src]
    return {"seq_lens": new_lens[:, 0].int(), "kept": torch.where(real, kept, -1).int(),
            "weights": s["weights"], **_cache_outputs(s)}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def _nearest_e4m3(x):
    """float64 values rounded to the e4m3 grid, ties to even, at most 448."""
    exponent = torch.frexp(x)[1].clamp(min=-5) - 4       # the grid's step is 2^exponent, 2^-9 at least
    step = ((exponent.long() + 1023) << 52).view(torch.float64)
    return (torch.round(x / step) * step).clamp(-448.0, 448.0)


def _power_at_least(x):
    """For each positive x the smallest power of two at or above it (and at least 2^-64)."""
    e = torch.ceil(torch.log2(x.clamp(min=2.0 ** MIN_EXPONENT)))
    p = ((e.long() + 1023) << 52).view(torch.float64)
    return torch.where(p / 2 >= x, p / 2, p).clamp(min=2.0 ** MIN_EXPONENT)


def exact(case, seed):
    s = prepare(case, seed)
    return {"store": _exact_store, "attention": _exact_attention, "evict": _exact_evict}[case["op"]](case, s)


def _exact_store(case, s):
    bs, h, d = case["block"], case["heads"], case["dim"]
    slots = s["slot_mapping"].cpu()
    blocks = torch.unique(slots // bs)
    lowest = {}
    for slot in slots.tolist():
        lowest[slot // bs] = min(lowest.get(slot // bs, bs), slot % bs)
    first = torch.tensor([lowest[b] for b in blocks.tolist()])
    result = {}
    for name in ("k", "v"):
        values = s[name + "_cache"].view(torch.float8_e4m3fn).double().cpu().view(-1, h, d)
        scale = s[name + "_scale"].double().cpu()
        x = s[name].double().cpu().view(-1, h, d)
        lines = torch.zeros_like(values)
        lines[slots] = x
        need = lines.view(-1, bs, h, d)[blocks].abs().amax((1, 3)) / 448
        now = _power_at_least(need)
        now = torch.where((first > 0)[:, None], torch.maximum(now, scale[blocks]), now)
        ratio = torch.ones_like(scale)
        ratio[blocks] = scale[blocks] / now
        scale[blocks] = now
        held = torch.zeros(values.shape[0], dtype=torch.bool)
        held.view(-1, bs)[blocks] = torch.arange(bs)[None, :] < first[:, None]
        of = torch.arange(values.shape[0]) // bs
        values[held] = _nearest_e4m3(values[held] * ratio[of[held]][:, :, None])
        values[slots] = _nearest_e4m3(x / scale[slots // bs][:, :, None])
        result[name + "_cache"], result[name + "_scale"] = values.view(-1, h * d), scale
    return result


def _exact_attention(case, s):
    if work(case)["flops"] > 2e12:
        return None
    bs, h, d, group, dev = case["block"], case["heads"], case["dim"], case["group"], "cuda"
    tokens = s["q"].shape[0]
    out = torch.zeros(tokens, h * group, d, dtype=torch.float64, device=dev)
    lse = torch.full((tokens, h * group), -math.inf, dtype=torch.float64, device=dev)
    weights = s["weights_before"].double() if case["weights"] else None
    at = 0
    for i, (count, length) in enumerate(zip(s["counts"], s["lens"])):
        begin = max(0, length - count - case["window"] + 1) if case["window"] else 0
        places = torch.arange(begin, length, device=dev)
        blocks = s["block_tables"][i].long()[places // bs]
        slots = blocks * bs + places % bs
        k = s["k_cache"].view(torch.float8_e4m3fn)[slots].double().view(-1, h, d) * s["k_scale"][blocks].double()[:, :, None]
        v = s["v_cache"].view(torch.float8_e4m3fn)[slots].double().view(-1, h, d) * s["v_scale"][blocks].double()[:, :, None]
        for j in range(0, count, 512):
            rows = torch.arange(j, min(count, j + 512), device=dev)
            where = (length - count + rows)[:, None]
            hidden = places[None, :] > where
            if case["window"]:
                hidden |= places[None, :] <= where - case["window"]
            for head in range(h):
                x = s["q"][at + rows, head * group:(head + 1) * group].double()
                logits = (x.reshape(-1, d) @ k[:, head].T).view(len(rows), group, -1) * s["softmax_scale"]
                logits.masked_fill_(hidden[:, None, :], -math.inf)
                total = torch.logsumexp(logits, -1)
                p = torch.exp(logits - total[:, :, None])
                out[at + rows, head * group:(head + 1) * group] = (p.view(-1, p.shape[-1]) @ v[:, head]).view(len(rows), group, d)
                lse[at + rows, head * group:(head + 1) * group] = total
                if weights is not None:
                    weights[slots] += p.sum((0, 1))
        at += count
    answer = {"out": out, "lse": lse}
    if weights is not None:
        answer["weights"] = weights
    return answer


def _exact_evict(case, s):
    bs, h, d, budget = case["block"], case["heads"], case["dim"], case["budget"]
    all_weights = s["weights"].double().cpu()
    tables, fresh = s["block_tables"].long().cpu(), s["new_block_tables"].long().cpu()
    kept = torch.full((len(s["lens"]), budget), -1, dtype=torch.int32)
    sources, targets = [], []
    for i, length in enumerate(s["lens"]):
        places = torch.arange(length)
        slots = tables[i][places // bs] * bs + places % bs
        if length > budget:
            rank = all_weights[slots].clone()
            rank[:case["first"]] = math.inf
            rank[length - case["last"]:] = math.inf
            chosen = torch.argsort(rank, descending=True, stable=True)[:budget]
            places = torch.sort(chosen).values
        kept[i, :len(places)] = places
        to = torch.arange(len(places))
        sources.append(slots[places])
        targets.append(fresh[i][to // bs] * bs + to % bs)
    src, dst = torch.cat(sources), torch.cat(targets)
    all_weights[dst] = all_weights[src]
    answer = {"seq_lens": torch.tensor([min(x, budget) for x in s["lens"]], dtype=torch.int32),
              "kept": kept, "weights": all_weights}
    src, dst = src.cuda(), dst.cuda()
    for name in ("k", "v"):
        values = s[name + "_cache"].view(torch.float8_e4m3fn).view(-1, h, d)
        scale = s[name + "_scale"].double()
        from_scale = scale[src // bs]
        for head in range(h):
            top = torch.zeros(scale.shape[0], dtype=torch.float64, device="cuda")
            top.scatter_reduce_(0, dst // bs, from_scale[:, head], "amax")
            scale[:, head] = torch.where(top > 0, top, scale[:, head])
        result = values.double()
        for a in range(0, len(src), 1 << 16):
            x, y = src[a:a + (1 << 16)], dst[a:a + (1 << 16)]
            ratio = from_scale[a:a + (1 << 16)] / scale[y // bs]
            result[y] = _nearest_e4m3(values[x].double() * ratio[:, :, None])
        answer[name + "_cache"], answer[name + "_scale"] = result.view(-1, h * d), scale
    return answer
