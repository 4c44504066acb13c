"""Measured cases of the operators around a paged KV cache held in 4 bits.

The cache keeps e2m1 codes (4 bits an element) and an e4m3 scale for every 16
of them along the head dimension; one number for all keys and one for all
values multiply the scales.  Measured are

* the append of a step's keys and values to a 16-bit paged cache with the
  rotation by position applied on the way, to the queries too; a token may have
  positions on several axes (time, height, width),
* the same into the 4-bit cache, and reading stored lines back,
* the attention of a prepared batch (single tokens, drafted tokens, prompt
  chunks) over the 4-bit cache,
* the verification of drafted tokens against the target's probabilities, from
  given random numbers.

``run`` computes them with elementary torch operations, or, with ``own`` set,
through paged_kv_prep_gb300.
"""
import math
import random

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
GRID = 40               # probabilities are added up in whole multiples of 2^-40


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def _append(name, op, requests, tokens, block, group, heads=8, dim=128, rot=128, axes=1, interleaved=False,
            dtype="bf16", ctx=8192, lens_seed=1):
    return {"name": name, "op": op, "requests": requests, "tokens": tokens, "block": block, "group": group,
            "heads": heads, "dim": dim, "rot": rot, "axes": axes, "interleaved": interleaved, "dtype": dtype,
            "ctx": ctx, "lens_seed": lens_seed}


def _attention(name, requests, ctx, block, group, ctx_lo=1, run_lo=1, run_hi=1, chunks=0, chunk_lo=0, chunk_hi=0,
               window=0, heads=8, dim=128, dtype="bf16", lens_seed=1):
    return {"name": name, "op": "attention", "requests": requests, "run_lo": run_lo, "run_hi": run_hi,
            "ctx_lo": ctx_lo, "ctx": ctx, "chunks": chunks, "chunk_lo": chunk_lo, "chunk_hi": chunk_hi,
            "block": block, "group": group, "window": window, "heads": heads, "dim": dim, "dtype": dtype,
            "lens_seed": lens_seed}


def _verify(name, requests, drafts, vocab, dtype="fp32", draft_probs=True, lens_seed=1):
    return {"name": name, "op": "verify", "requests": requests, "drafts": drafts, "vocab": vocab, "dtype": dtype,
            "draft_probs": draft_probs, "lens_seed": lens_seed}


def listed():
    return [
        # one decode step of a small batch: eight tokens; latency counts
        _append("rope_8_decodes", "rope", 8, 8, 16, 4),
        # the large step's token budget: thousands of decodes beside prompt chunks
        _append("rope_16384_tokens", "rope", 4096, 16384, 32, 4),
        # prompts of video frames: three axes, half of each head rotated, neighbouring elements paired
        _append("rope_video_fp16", "rope", 5, 6007, 16, 7, heads=4, rot=64, axes=3, interleaved=True, dtype="fp16"),
        # one decode step into the 4-bit cache, its lines read back; latency counts
        _append("kv4_store_8_decodes", "kv4_store", 8, 8, 16, 4),
        # prompt chunks of frames beside decodes, three axes
        _append("kv4_store_16384_tokens", "kv4_store", 256, 16384, 32, 4, axes=3),
        # the smallest serving batch: eight single tokens on short contexts
        _attention("attn4_8_decodes", 8, 200, 16, 4),
        # an ordinary decode batch, contexts spread up to 8192 (8 KV heads shared by 32 heads)
        _attention("attn4_256_decodes", 256, 8192, 16, 4),
        # few requests with very long contexts (64 heads): the work is along the cache
        _attention("attn4_4_long_decodes", 4, 131072, 32, 8, ctx_lo=65536),
        # drafted tokens to be verified: two to six tokens a request, under a sliding window
        _attention("attn4_drafts_fp16", 96, 16384, 16, 5, run_lo=2, run_hi=6, window=4096, dtype="fp16"),
        # chunked prefill beside decodes, contexts up to 16384
        _attention("attn4_mixed_prefill", 64, 16384, 16, 4, chunks=6, chunk_lo=512, chunk_hi=2048),
        # a small batch proposed by lookup: no draft probabilities, an odd vocabulary
        _verify("verify_8_lookup", 8, 3, 32003, draft_probs=False),
        # a full decode batch with a draft model's probabilities
        _verify("verify_256_drafts", 256, 4, 131072),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "kv4_store", "attention", "attention", "attention", "verify"])
    block = rng.choice([16, 32])
    heads, dim = rng.choice([(8, 128), (4, 128), (2, 128), (8, 64), (1, 128)])
    group = rng.choice([1, 2, 4, 5, 7, 8])
    seed = rng.randrange(1 << 30)
    if op == "verify":
        vocab = _log_int(rng, 1000, 131072)
        c = _verify("", _log_int(rng, 1, 256), rng.randint(1, 8), vocab, rng.choice(["fp32", "fp32", "bf16", "fp16"]),
                    rng.random() < 0.6, seed)
        c["requests"] = min(c["requests"], max(1, (256 * 131072) // vocab // c["drafts"]))
    elif op != "attention":
        requests = _log_int(rng, 1, 4096)
        rot = rng.choice([dim, dim, dim // 2, dim // 4])
        c = _append("", op, requests, min(16384, requests * _log_int(rng, 1, 512)), block, min(group, 32 // heads),
                    heads, dim, rot, rng.choice([1, 1, 3]), rng.random() < 0.3, rng.choice(["bf16", "fp16"]),
                    _log_int(rng, 512, 32768), seed)
    else:
        kind = rng.choice(["decode", "decode", "drafts", "mixed", "chunks"])
        window = rng.choice([0, 0, 0, _log_int(rng, 64, 8192)])
        dtype = rng.choice(["bf16", "bf16", "fp16"])
        if kind in ("decode", "drafts"):
            ctx = _log_int(rng, 32, 131072)
            requests = _log_int(rng, 1, max(1, min(512, (1 << 20) // ctx)))
            hi = rng.randint(2, 8) if kind == "drafts" else 1
            c = _attention("", requests, ctx, block, group, ctx_lo=rng.randint(1, ctx), run_lo=rng.randint(1, hi),
                           run_hi=hi, window=window, heads=heads, dim=dim, dtype=dtype, lens_seed=seed)
        else:
            ctx = _log_int(rng, 64, 16384)
            hi = _log_int(rng, 2, min(2048, ctx))
            c = _attention("", rng.randint(1, 64) if kind == "mixed" else 0, ctx, block, group,
                           chunks=rng.randint(1, 5), chunk_lo=rng.randint(1, hi), chunk_hi=hi, window=window,
                           heads=heads, dim=dim, dtype=dtype, lens_seed=seed)
    del c["name"]
    return c


# --------------------------------------------------------------------------
# the lengths and positions a case stands for (the same for every seed of its values)
# --------------------------------------------------------------------------
def _lengths(case):
    """(scheduled tokens, sequence length) of each request, fewer tokens first as a prepared batch
    has them; (rows, 0) for a verification."""
    rng = random.Random(case["lens_seed"])
    if case["op"] == "verify":
        return [(1 + rng.randint(0, case["drafts"]), 0) for _ in range(case["requests"])]
    if case["op"] == "attention":
        reqs = []
        for _ in range(case["requests"]):
            c = rng.randint(case["run_lo"], case["run_hi"])
            reqs.append((c, rng.randint(max(c, case["ctx_lo"]), max(c, case["ctx"]))))
        for _ in range(case["chunks"]):
            c = rng.randint(case["chunk_lo"], case["chunk_hi"])
            reqs.append((c, rng.randint(c, max(c, case["ctx"]))))
    else:
        n = case["requests"]
        counts = [1] * n
        left = case["tokens"] - n
        while left > 0:      # the first requests hold prompt chunks, the rest decode
            c = min(left, rng.randint(1, 4095))
            counts[rng.randrange(n)] += c
            left -= c
        reqs = [(c, c + rng.randint(0, max(0, case["ctx"] - c))) for c in counts]
    return sorted(reqs, key=lambda r: r[0])


def _positions(case, reqs):
    """Each token's positions, [axes, tokens].  With three axes a prompt is 64 tokens of text and then
    frames of 24 x 24 patches: a patch has its frame, row and column."""
    at = torch.cat([torch.arange(x - c, x) for c, x in reqs])
    if case["axes"] == 1:
        return at[None]
    m = (at - 64).clamp(min=0)
    patch = at >= 64
    return torch.stack([torch.where(patch, 64 + m // 576, at), torch.where(patch, 64 + m % 576 // 24, at),
                        torch.where(patch, 64 + m % 24, at)])


def _axis_of(case):
    """The axis that each rotated pair follows: a quarter of the pairs go by time, three eighths each
    by height and width."""
    pairs = case["rot"] // 2
    if case["axes"] == 1:
        return [0] * pairs
    a, b = pairs // 4, pairs // 4 + pairs * 3 // 8
    return [0 if i < a else 1 if i < b else 2 for i in range(pairs)]


def _pairs(count, length, window):
    """Visible (query, key) pairs of one request, and the cached tokens that some query sees."""
    if not window or window >= length:
        return count * length - count * (count - 1) // 2, length
    pairs = sum(min(p + 1, window) for p in range(length - count, length))
    return pairs, length - max(0, length - count - window + 1)


def work(case):
    reqs = _lengths(case)
    if case["op"] == "verify":
        # a row of the target's probabilities for each request; and one of the draft's for those that
        # reject a draft (about one draft in four is, on these inputs)
        rows = sum(1 + (1 - 0.75 ** (c - 1)) * case["draft_probs"] for c, _ in reqs)
        size = 4 if case["dtype"] == "fp32" else 2
        tokens = sum(c for c, _ in reqs)
        return {"bytes": int(rows * case["vocab"] * size) + tokens * (8 + 8 * size) + 4 * len(reqs) * (case["drafts"] + 2),
                "flops": int(rows * case["vocab"] * 2)}
    h, d = case["heads"], case["dim"]
    hq = h * case["group"]
    if case["op"] != "attention":
        t = sum(c for c, _ in reqs)
        line = 2 * h * d                                            # 16-bit bytes of a token's keys
        pos = _positions(case, reqs)
        table = max(len(torch.unique(p)) for p in pos) * case["rot"] * 4
        small = 8 * t + 4 * t * case["axes"] + table
        byte = 2 * t * hq * d * 2 + small
        if case["op"] == "rope":
            byte += 4 * t * line                                    # keys and values, read and written
        else:
            byte += 4 * t * line + 2 * 2 * t * h * (d // 2 + d // 16) + 8 * t   # stored, and read back
        return {"bytes": byte, "flops": 3 * t * (hq + h) * case["rot"]}
    tokens = sum(c for c, _ in reqs)
    pairs = [_pairs(c, length, case["window"]) for c, length in reqs]
    seen = sum(p[1] for p in pairs)
    byte = 2 * seen * h * (d // 2 + d // 16) + 2 * tokens * hq * d * 2 + tokens * hq * 4
    return {"bytes": byte, "flops": 4 * d * hq * sum(p[0] for p in pairs)}


# --------------------------------------------------------------------------
# the 4-bit format
# --------------------------------------------------------------------------
def _e2m1_codes(x):
    """fp32 values rounded to the e2m1 grid (to nearest, a tie to the even code), as codes with the
    sign in bit 3."""
    a = x.abs()
    code = (a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0)
    return (code + 8 * torch.signbit(x)).to(torch.uint8)


def _quantise(x, unit):
    """x [..., dim] in fp32: (packed codes [..., dim / 2], e4m3 scales [..., dim / 16] as bytes)."""
    y = x.unflatten(-1, (-1, 16))
    # quotients, not products with a reciprocal: a value half way between two codes stays there
    scale = (y.abs().amax(-1) / (6.0 * unit)).clamp(max=448.0).to(torch.float8_e4m3fn)
    by = (scale.float() * unit)[..., None]
    codes = _e2m1_codes(torch.where(by > 0, y / by, 0.0)).flatten(-2)
    return codes[..., 0::2] | (codes[..., 1::2] << 4), scale.view(torch.uint8)


def _value_table(device):
    """The two elements that each byte of codes stands for, [256, 2]."""
    one = torch.tensor(E2M1 + [-v for v in E2M1], device=device)
    byte = torch.arange(256, device=device)
    return torch.stack([one[byte % 16], one[byte // 16]], 1)


def _values(codes, scale, unit, table):
    """fp32 values of packed codes [..., dim / 2] and scale bytes [..., dim / 16]."""
    x = table[codes.int()].flatten(-2).unflatten(-1, (-1, 16))
    return (x * (scale.view(torch.float8_e4m3fn).float()[..., None] * unit)).flatten(-2)


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _filled_cache(gen, blocks, case, unit):
    """A cache of normally distributed lines; some channels are larger than others, as keys have them."""
    bs, h, d = case["block"], case["heads"], case["dim"]
    channel = torch.exp(0.5 * torch.randn(h, 1, d, generator=gen, device="cuda"))
    codes = torch.empty(blocks, h, bs, d // 2, dtype=torch.uint8, device="cuda")
    scale = torch.empty(blocks, h, bs, d // 16, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 28) // (bs * h * d))
    for a in range(0, blocks, step):
        x = torch.randn(min(step, blocks - a), h, bs, d, generator=gen, device="cuda") * channel
        codes[a:a + step], scale[a:a + step] = _quantise(x, unit)
    return codes, scale


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


def _starts(counts):
    starts = [0]
    for c in counts:
        starts.append(starts[-1] + c)
    return starts


def _prepare_verify(case, s, gen):
    """Peaked target rows, a draft that is near them, and drafts drawn from the draft's rows."""
    rows, vocab, dtype = s["starts"][-1], case["vocab"], DTYPES[case["dtype"]]
    s["target_probs"] = torch.empty(rows, vocab, dtype=dtype, device="cuda")
    s["draft_probs"] = torch.empty(rows, vocab, dtype=dtype, device="cuda") if case["draft_probs"] else None
    s["draft_ids"] = torch.empty(rows, dtype=torch.int32, device="cuda")
    step = max(1, (1 << 26) // vocab)
    for a in range(0, rows, step):
        logits = 3.0 * torch.randn(min(step, rows - a), vocab, generator=gen, device="cuda")
        s["target_probs"][a:a + step] = torch.softmax(logits, -1).to(dtype)
        if case["draft_probs"]:
            logits += 0.7 * torch.randn(logits.shape, generator=gen, device="cuda")
        q = torch.softmax(logits, -1).to(dtype)
        if case["draft_probs"]:
            s["draft_probs"][a:a + step] = q
            at = torch.rand(len(q), 1, generator=gen, device="cuda", dtype=torch.float64)
            below = torch.cumsum(q.double(), -1)
            s["draft_ids"][a:a + step] = torch.searchsorted(below, at * below[:, -1:]).clamp(max=vocab - 1)[:, 0].int()
        else:
            s["draft_ids"][a:a + step] = q.argmax(-1).int()
    s["uniforms"] = torch.rand(rows, generator=gen, device="cuda")
    return s


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    reqs = _lengths(case)
    counts, lens = [r[0] for r in reqs], [r[1] for r in reqs]
    starts = _starts(counts)
    s = {"case": case, "counts": counts, "lens": lens, "starts": starts,
         "query_start_loc": torch.tensor(starts, dtype=torch.int32, device="cuda")}
    if case["op"] == "verify":
        return _prepare_verify(case, s, gen)
    bs, h, d, tokens, dtype = case["block"], case["heads"], case["dim"], starts[-1], DTYPES[case["dtype"]]
    hq = h * case["group"]
    rows = torch.randn(tokens, (hq + 2 * h) * d, generator=gen, device="cuda")
    if case["op"] == "attention":
        first = None
        if case["window"]:
            first = [max(0, x - c - case["window"] + 1) // bs for c, x in reqs]
        s["seq_lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["block_tables"], blocks = _tables(gen, lens, bs, -(-max(lens) // bs), first)
        s["units"] = (2.0, 0.5)
        s["k_cache"], s["k_scale"] = _filled_cache(gen, blocks, case, 2.0)
        s["v_cache"], s["v_scale"] = _filled_cache(gen, blocks, case, 0.5)
        s["q"] = rows.to(dtype)[:, :hq * d].view(tokens, hq, d)
        s["softmax_scale"] = d ** -0.5
        s["values"] = _value_table("cuda")
        return s
    # the fused projection's rows: queries, keys and values are views of them, with outliers now and then
    rows *= torch.exp2(torch.randint(-2, 3, (tokens, 1), generator=gen, device="cuda"))
    rows = rows.to(dtype)
    s["q"], s["k"], s["v"] = (x.unflatten(1, (-1, d)) for x in rows.split([hq * d, h * d, h * d], 1))
    positions = _positions(case, reqs)
    s["positions"] = positions.to("cuda", torch.int32).contiguous()
    s["axes"] = _axis_of(case)
    s["axis_rows"] = torch.tensor(s["axes"], device="cuda")
    pair = torch.arange(case["rot"] // 2, dtype=torch.float64, device="cuda")
    angle = torch.arange(max(case["ctx"], int(positions.max()) + 1), dtype=torch.float64, device="cuda")[:, None] * \
        10000.0 ** (-pair / (case["rot"] // 2))
    s["table"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    # blocks that hold the step's tokens, in random order: a token's slot goes by its place in its request
    req = torch.repeat_interleave(torch.arange(len(reqs)), torch.tensor(counts))
    place = torch.cat([torch.arange(x - c, x) for c, x in reqs])
    name, index = torch.unique(torch.stack([req, place // bs], 1), dim=0, return_inverse=True)
    blocks = len(name)
    order = torch.randperm(blocks, generator=gen, device="cuda")
    s["slot_mapping"] = order[index.cuda()] * bs + (place % bs).cuda()
    if case["op"] == "rope":
        s["k_cache"] = torch.zeros(blocks * bs, h, d, dtype=dtype, device="cuda")
        s["v_cache"] = torch.zeros_like(s["k_cache"])
    else:
        s["units"] = (1.0, 1.0)
        s["k_cache"], s["v_cache"] = (torch.zeros(blocks, h, bs, d // 2, dtype=torch.uint8, device="cuda") for _ in range(2))
        s["k_scale"], s["v_scale"] = (torch.zeros(blocks, h, bs, d // 16, dtype=torch.uint8, device="cuda") for _ in range(2))
        s["values"] = _value_table("cuda")
    return s


# --------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------
def run(state):
    op = state["case"]["op"]
    if own:
        return {"rope": _own_rope, "kv4_store": _own_store, "attention": _own_attention, "verify": _own_verify}[op](state)
    return {"rope": _plain_rope, "kv4_store": _plain_store, "attention": _plain_attention,
            "verify": _plain_verify}[op](state)


def _own_rope(s):
    import paged_kv_prep_gb300 as pkv

    q = pkv.rope_store(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slot_mapping"], s["positions"], s["table"],
                       axes=s["axes"], interleaved=s["case"]["interleaved"], q=s["q"])
    return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _own_store(s):
    import paged_kv_prep_gb300 as pkv

    cache = s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"]
    q = pkv.kv4_store(s["k"], s["v"], *cache, s["slot_mapping"], positions=s["positions"], table=s["table"],
                      axes=s["axes"], interleaved=s["case"]["interleaved"], q=s["q"], k_unit=s["units"][0],
                      v_unit=s["units"][1])
    k, v = pkv.kv4_load(*cache, s["slot_mapping"], dtype=s["k"].dtype, k_unit=s["units"][0], v_unit=s["units"][1])
    return {"q": q, "k": k, "v": v}


def _own_attention(s):
    import paged_kv_prep_gb300 as pkv

    out, lse = pkv.kv4_attention(s["q"], s["k_cache"], s["v_cache"], s["k_scale"], s["v_scale"], s["block_tables"],
                                 s["query_start_loc"], s["seq_lens"], softmax_scale=s["softmax_scale"],
                                 window=s["case"]["window"], k_unit=s["units"][0], v_unit=s["units"][1])
    return {"out": out, "lse": lse}


def _own_verify(s):
    import paged_kv_prep_gb300 as pkv

    tokens, accepted = pkv.verify_drafts(s["target_probs"], s["draft_ids"], s["query_start_loc"], s["uniforms"],
                                         s["case"]["drafts"], draft_probs=s["draft_probs"])
    return {"tokens": tokens, "accepted": accepted}


def _rotated(s, x):
    """x [tokens, heads, dim] in fp32, its first `rot` elements rotated by the token's positions."""
    case = s["case"]
    x, rot = x.float(), case["rot"]
    pairs = rot // 2
    at = s["positions"].long()[s["axis_rows"]].T                                   # [tokens, pairs]
    cos = s["table"][:, :pairs].gather(0, at)[:, None]
    sin = s["table"][:, pairs:].gather(0, at)[:, None]
    if case["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :pairs], x[..., pairs:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_rope(s):
    dtype = s["q"].dtype
    s["k_cache"][s["slot_mapping"]] = _rotated(s, s["k"]).to(dtype)
    s["v_cache"][s["slot_mapping"]] = s["v"]
    return {"q": _rotated(s, s["q"]).to(dtype), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_store(s):
    dtype, bs = s["q"].dtype, s["case"]["block"]
    block, offset = s["slot_mapping"] // bs, s["slot_mapping"] % bs
    back = {"q": _rotated(s, s["q"]).to(dtype)}
    for name, x, unit in (("k", _rotated(s, s["k"]), s["units"][0]), ("v", s["v"].float(), s["units"][1])):
        codes, scale = s[name + "_cache"], s[name + "_scale"]
        codes[block, :, offset], scale[block, :, offset] = _quantise(x, unit)
        back[name] = _values(codes[block, :, offset], scale[block, :, offset], unit, s["values"]).to(dtype)
    return back


def _groups(s):
    """Requests a..b that are computed together, so that their padded logits stay within 4 GB."""
    case, at, out = s["case"], 0, []
    hq = case["heads"] * case["group"]
    while at < len(s["lens"]):
        end, most_c, most_l = at, 0, 0
        while end < len(s["lens"]):
            c, x = max(most_c, s["counts"][end]), max(most_l, s["lens"][end])
            size = (end + 1 - at) * x * max(c * hq, case["heads"] * case["dim"])
            if end > at and size > 1 << 30:
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
    for a, b, count, length in _groups(s):
        n = b - a
        blocks = -(-length // bs)
        length = blocks * bs
        table = s["block_tables"][a:b, :blocks].long()
        real = table >= 0
        table = table.clamp(min=0)
        k = _values(s["k_cache"][table], s["k_scale"][table], s["units"][0], s["values"])   # [n, blocks, h, bs, d]
        v = _values(s["v_cache"][table], s["v_scale"][table], s["units"][1], s["values"])
        k = k.permute(0, 2, 4, 1, 3).reshape(n, h, d, length)
        v = v.permute(0, 2, 1, 3, 4).reshape(n, h, length, d)
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
    return {"out": out.to(q.dtype), "lse": lse}


def _plain_verify(s):
    case, device = s["case"], s["uniforms"].device
    n, most, vocab = len(s["counts"]), case["drafts"], case["vocab"]
    start, end = s["query_start_loc"][:-1].long(), s["query_start_loc"][1:].long()
    rows = s["target_probs"].shape[0]
    j = torch.arange(most, device=device)
    row = start[:, None] + j                                                  # [n, most]
    is_draft = row < end[:, None] - 1
    row = row.clamp(max=rows - 1)
    ids = s["draft_ids"][row].long()
    p = s["target_probs"][row, ids].double()
    q = s["draft_probs"][row, ids].double() if case["draft_probs"] else torch.ones_like(p)
    passes = is_draft & (s["uniforms"][row].double() * q < p)
    accepted = torch.cumprod(passes.int(), 1).sum(1)
    last = start + accepted                                                   # the row that gives the next token
    rejected = last < end - 1
    weight = s["target_probs"][last].float()
    if case["draft_probs"]:
        weight = torch.where(rejected[:, None], weight - s["draft_probs"][last].float(), weight)
    else:
        drafted = torch.arange(vocab, device=device)[None] == s["draft_ids"][last].long()[:, None]
        weight = torch.where(rejected[:, None] & drafted, 0.0, weight)
    weight = torch.where(weight > 0, weight, 0.0).clamp(max=1.0)
    count = torch.round(weight.double() * 2.0 ** GRID).long()
    below = torch.cumsum(count, 1)
    total = below[:, -1]
    aim = torch.floor(s["uniforms"][end - 1].double() * total.double()).long()
    aim = torch.minimum(aim, total - 1).clamp(min=0)
    drawn = torch.searchsorted(below, aim[:, None], right=True)[:, 0]
    k = torch.arange(most + 1, device=device)
    drafted = s["draft_ids"][(start[:, None] + k).clamp(max=rows - 1)]
    tokens = torch.where(k < accepted[:, None], drafted, -1)
    tokens = torch.where(k == accepted[:, None], drawn[:, None].int(), tokens)
    return {"tokens": tokens.int(), "accepted": accepted.int()}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    return {"rope": _exact_rope, "kv4_store": _exact_store, "attention": _exact_attention,
            "verify": _exact_verify}[case["op"]](case, s)


def _turn(case, s, x):
    """Every pair as a complex number, multiplied by that of its angle."""
    x, half = x.double(), case["rot"] // 2
    where = torch.stack([s["positions"][a] for a in s["axes"]], 1).long()          # [tokens, pairs]
    pair = torch.arange(half, device=x.device)[None].expand_as(where)
    by = torch.complex(s["table"].double()[where, pair], s["table"].double()[where, half + pair])[:, None]
    first = torch.arange(half, device=x.device) * (2 if case["interleaved"] else 1)
    second = first + (1 if case["interleaved"] else half)
    z = torch.complex(x[..., first], x[..., second]) * by
    y = x.clone()
    y[..., first], y[..., second] = z.real, z.imag
    return y


def _exact_rope(case, s):
    answer = {"q": _turn(case, s, s["q"])}
    for name, x in (("k", _turn(case, s, s["k"])), ("v", s["v"].double())):
        cache = s[name + "_cache"].double()
        cache[s["slot_mapping"]] = x
        answer[name + "_cache"] = cache
    return answer


def _bits_value(codes):
    """e2m1 codes by their fields: sign, two exponent bits, one fraction bit."""
    e, m = (codes >> 1) & 3, codes & 1
    size = torch.where(e == 0, 0.5 * m, torch.exp2(e.double() - 1) * (1 + 0.5 * m))
    return torch.where(codes >= 8, -size, size)


def _exact_store(case, s):
    grid = _bits_value(torch.arange(8, device="cuda").double().int())
    between = (grid[1:] + grid[:-1]) / 2
    answer = {"q": _turn(case, s, s["q"])}
    for name, x, unit in (("k", _turn(case, s, s["k"]), s["units"][0]), ("v", s["v"].double(), s["units"][1])):
        y = x.view(*x.shape[:-1], -1, 16)
        need = y.abs().amax(-1, keepdim=True) / (6.0 * unit)
        step = torch.exp2((torch.frexp(need)[1] - 4).clamp(min=-9).double())
        scale = (torch.round(need / step) * step).clamp(max=448.0) * unit
        t = (y / torch.where(scale > 0, scale, 1.0)).abs()
        low, high = torch.bucketize(t, between, right=False), torch.bucketize(t, between, right=True)
        even = torch.where(low % 2 == 0, low, high)                            # where the two differ: a tie
        answer[name] = (grid[even] * torch.sign(y) * scale).view(x.shape)
    return answer


def _exact_attention(case, s):
    if work(case)["flops"] > 2e12:
        return None
    bs, h, d, group, dev = case["block"], case["heads"], case["dim"], case["group"], "cuda"
    tokens = s["q"].shape[0]
    out = torch.zeros(tokens, h * group, d, dtype=torch.float64, device=dev)
    lse = torch.full((tokens, h * group), -math.inf, dtype=torch.float64, device=dev)
    lines = {}
    at = 0
    for i, (count, length) in enumerate(zip(s["counts"], s["lens"])):
        begin = max(0, length - count - case["window"] + 1) if case["window"] else 0
        places = torch.arange(begin, length, device=dev)
        blocks, offset = s["block_tables"][i].long()[places // bs], places % bs
        for name, unit in (("k", s["units"][0]), ("v", s["units"][1])):
            byte = s[name + "_cache"][blocks, :, offset].int()                  # [seen, h, d / 2]
            line = _bits_value(torch.stack([byte & 15, byte >> 4], -1)).view(-1, h, d // 16, 16)
            scale = s[name + "_scale"].view(torch.float8_e4m3fn)[blocks, :, offset].double()
            lines[name] = (line * scale[..., None] * unit).view(-1, h, d)
        for j in range(0, count, 512):
            rows = torch.arange(j, min(count, j + 512), device=dev)
            where = (length - count + rows)[:, None]
            hidden = places[None, :] > where
            if case["window"]:
                hidden |= places[None, :] <= where - case["window"]
            for head in range(h):
                x = s["q"][at + rows, head * group:(head + 1) * group].double()
                logits = (x.reshape(-1, d) @ lines["k"][:, head].T).view(len(rows), group, -1) * s["softmax_scale"]
                logits.masked_fill_(hidden[:, None, :], -math.inf)
                total = torch.logsumexp(logits, -1)
                p = torch.exp(logits - total[:, :, None])
                mean = p.view(-1, p.shape[-1]) @ lines["v"][:, head]
                out[at + rows, head * group:(head + 1) * group] = mean.view(len(rows), group, d)
                lse[at + rows, head * group:(head + 1) * group] = total
        at += count
    return {"out": out, "lse": lse}


def _exact_verify(case, s):
    tokens = torch.full((len(s["counts"]), case["drafts"] + 1), -1, dtype=torch.int32)
    accepted = torch.zeros(len(s["counts"]), dtype=torch.int32)
    u, ids = s["uniforms"].double().tolist(), s["draft_ids"].tolist()
    for i, count in enumerate(s["counts"]):
        row, end = s["starts"][i], s["starts"][i + 1]
        while row < end - 1:
            p = float(s["target_probs"][row, ids[row]])
            q = float(s["draft_probs"][row, ids[row]]) if case["draft_probs"] else 1.0
            if not u[row] * q < p:
                break
            tokens[i, row - s["starts"][i]] = ids[row]
            row += 1
        weight = s["target_probs"][row].float()
        if row < end - 1:
            if case["draft_probs"]:
                weight = (weight - s["draft_probs"][row].float()).clamp(min=0)
            else:
                weight = weight.clone()
                weight[ids[row]] = 0.0
        below = torch.cumsum((weight.double() * 2.0 ** GRID).round().long(), 0)
        aim = min(int(u[end - 1] * float(below[-1])), int(below[-1]) - 1)
        accepted[i] = row - s["starts"][i]
        tokens[i, row - s["starts"][i]] = int((below <= max(aim, 0)).sum())
    return {"tokens": tokens, "accepted": accepted}
