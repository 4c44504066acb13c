// Attention over the 4-bit paged cache for requests with many query rows
// (prompt chunks, drafted tokens of large groups), on the tensor cores.
//
// Mathematics: as in pkv_kv4_decode.cu.  S = q . k comes from the tensor core with keys that
// carry their scales, so x = S * a - R with one a per row; w = 2^(x - R) goes into the second
// product as f16, the softmax sum adds it in fp32.  R is 9 below the row's maximum over its first
// unit, rounded up to an integer, and then follows lazily: it moves only when the sum of 64 w,
// which is needed anyway, exceeds 2^15, and by a whole power of two, so that
// weights which are f16 already are not rounded again (unless they turn subnormal).
// w is off by 2^-11 of itself, or by 2^-25 where it is below 2^-14, and as much again if the reference
// moves after it: 2^-32 of the largest weight together, so n such tokens put the output off by
// n 2^-32 of the largest |value| at most.
//
// Bound: the tensor pipe (4 D flops per visible pair); beside it per tile of
// 256 rows x 128 tokens 32768 exponentials and 32768 codes turned into f16 and scaled.
//
// Layout.  A CTA holds 256 (query, head) rows of one KV head in two tiles of
// 128.  Warps 0-3 and 4-7 do the softmax of one tile each, a thread per row;
// warps 8-11 (keys) and 12-15 (values) read the codes of 128 tokens a unit ahead into registers, turn
// them into f16 times their scales (exact) and lay them out for the tensor core, so one
// conversion serves both tiles; warp 16 issues the products: S = Q K^T (both in shared memory),
// O += P V with P in TMEM in the place of S; warp 17 goes through the CTA's units and block tables
// and tells the others.  While one tile's softmax runs, the tensor core works on the other; a tile's
// second product begins when half of its weights are there.  The next row tile's queries are loaded
// while the last products of this one run.
// A row tile of at most 128 rows is taken by both softmax warpgroups: one does the units of even
// numbers, the other those of odd ones, each with an accumulator of its own; they are put together
// at the end, out of TMEM.
// The batch's (row tile, KV head, 128 tokens) units are split evenly over the CTAs, by what they cost; a row
// tile that is cut leaves partial results for a merge in a fixed order.
//
// Every wait has a limit; one that runs out sets PKV_DEVERR_TIMEOUT, the other
// waits give up after it, and the CTA drains its products and frees its TMEM.
//
// Measured: two chunks of 2048 tokens, 32 query and 8 KV heads of 128, contexts up to 16384 (522 GFLOP) 460 us
// with the merge, 1.13 PFLOP/s, 60 % of the measured rate of bf16 products.  A unit of 256 rows x 128 tokens takes 3900 cycles of
// which the tensor pipe works 2048 (the rest is the way scores -> weights -> products with its barriers); a row tile 25000
// cycles beside its units.  What was slower, in turn with the form of its time (465 to 500 us, not this one): two issuing warps,
// 1.13 times as long; scores in halves of 64 tokens, two in TMEM, 1.08; fetching codes ahead into L2, 1.04; waits that sleep
// in hardware, 1.08; codes copied to shared memory (by bulk copies or by warps of their own) instead of into registers,
// 1.55 for a step of chunks and decodes.  Without any exponentials and conversions a form that took 495 us, whose second
// products did not begin by halves, took 390.
#include "pkv_kv4_attention.cuh"
#include "pkv_tcgen05.cuh"

namespace pkv {
namespace {

constexpr int kRows = 256;              // rows of a CTA, two tiles of 128
constexpr int kKeys = 128;              // tokens per unit
constexpr int kSoftWarps = 8, kConvWarps = 4;          // converting warps: as many for the keys as for the values
constexpr int kThreads = 32 * (kSoftWarps + 2 * kConvWarps + 4);   // and a warpgroup: issue, walk, two idle warps
constexpr int kUnits = 8;                // units that are known ahead
// Registers a thread: launched with 96; 256 x 144 + 256 x 64 + 128 x 64 = 640 x 96.
constexpr int kSoftRegs = 144, kConvRegs = 64, kIssueRegs = 64;
static_assert(32 * (kSoftWarps * kSoftRegs + 2 * kConvWarps * kConvRegs + 4 * kIssueRegs) <= kThreads * 96, "registers");
constexpr uint32_t kTries = 1u << 22;   // polls before a wait gives up (half a second or more)
constexpr float kHead = 9.f;            // how far below a row's maximum (log2) R is set
constexpr float kMostSum = 32768.f;     // sum of 64 w that makes it move
constexpr float kHuge = 0x1p20f;        // a reference from which on a logit's rounding may count
// Costs, in units of a row tile that one warpgroup's half of the units takes: a unit of two tiles, and what a
// row tile costs beside its units (queries, first scores, output).  A mixed call with 3 for the latter 954 us, with 6
// 858, 10 817, 12 813, 14 810; long chunks with 3 488, 6 479, 10 472, 14 473.
constexpr int kPairCost = 2, kTileCost = 12;

// Kinds of units: of two tiles, a row tile's last of this CTA, the CTA's last; no unit at all.
constexpr int kPair = 1, kTileEnd = 2, kEnd = 4, kNone = 8;
constexpr int kItems = 16;

// One stretch of units: a row tile, a KV head, and which of its 128-token units.
struct Item {
    int start, count, len;              // of the request: first token, scheduled and cached tokens; count 0: the end
    int lo, hi, base, units;            // keys that the tile's rows see, the 16-aligned start of its units
    int i, rt, head, ua, ub;
    int64_t last;                       // the cost at which the row tile's last unit begins
    bool pair;                          // more than 128 rows
};

template <int D>
struct Smem {
    char q[2][128 * D * 2];
    char k[2][kKeys * D * 2];
    char v[2][kKeys * D * 2];
    float top[128], sum[128];           // the odd units' statistics of a row tile that both warpgroups take
    uint64_t q_full[2], k_full[2], v_full[2], k_free[2], v_free[2], s_full[2], p_half[2], p_full[2], h_done[2], o_full[2];
    uint64_t unit_full[kUnits], unit_free[kUnits], side_full, side_free, item_full[kItems], done;
    // Of the units from the walking warp: first token that some row sees, the token behind the last one, which groups of
    // 16 have a block, what kind of unit it is; and the groups' first lines.
    int4 unit[kUnits];
    int64_t line[kUnits][8];
    Item item[kItems];                  // row tiles, from the walking warp; a last one without rows
    uint32_t tmem;
    int32_t failed;
};

// The keys that rows f0 .. of a tile see: [lo, hi), and the 16-aligned start of their units.
struct Span {
    int lo, hi, base, units;
};
__device__ __forceinline__ Span span_of(const AttnParams &p, const Req &r, int rt) {
    const int rows = r.count * p.G, f0 = rt * kRows, f1 = min(rows, f0 + kRows) - 1;
    const int back = r.len - r.count, pos0 = back + f0 / p.G, pos1 = back + f1 / p.G;
    Span s;
    s.lo = lo_of(p, pos0);
    s.hi = min(pos1 + 1, r.keys);
    s.base = s.lo & ~15;
    s.units = s.hi > s.base ? (s.hi - s.base + kKeys - 1) / kKeys : 1;   // a tile without keys writes zeros
    return s;
}
__device__ __forceinline__ bool is_pair(int64_t rows, int rt) { return rows - static_cast<int64_t>(rt) * kRows > 128; }
__device__ __forceinline__ int64_t cost_of(const Span &s, bool pair) { return kTileCost + static_cast<int64_t>(s.units) * (pair ? kPairCost : 1); }
__device__ __forceinline__ int64_t cost_of_tile(const AttnParams &p, const Req &r, int64_t rows, int rt) {
    return cost_of(span_of(p, r, rt), is_pair(rows, rt)) * p.Hkv;
}
// Row tiles of a request.
__device__ __forceinline__ int tiles_of(const AttnParams &p, const Req &r, int64_t rows) {
    return r.count <= 0 || rows <= p.short_rows ? 0 : static_cast<int>((rows + kRows - 1) / kRows);
}
// A request's cost, by a thread, or by a warp (a lane for each row tile).
__device__ __forceinline__ int64_t cost_of_request(const AttnParams &p, const Req &r, int lane = 0, int step = 1) {
    const int64_t rows = static_cast<int64_t>(r.count) * p.G;
    const int tiles = tiles_of(p, r, rows);
    int64_t sum = 0;
    for (int rt = lane; rt < tiles; rt += step) sum += cost_of_tile(p, r, rows, rt);
    return sum;
}

// Costs u .. end - 1 of the batch; a unit belongs to whoever has the cost at which it begins.
struct Walk {
    const AttnParams &p;
    int64_t u, end, at;                 // at: where the row tile `rt` begins
    int i, rt;
    Req r;

    // By a whole warp: a lane looks at every 32nd row tile of the request that u lies in.  `costs`: the requests'.
    template <typename CostOf>
    __device__ __forceinline__ Walk(const AttnParams &p_, const int64_t *prefix, int64_t u0, int64_t u1, CostOf costs) : p(p_), u(u0), end(u1) {
        const int lane = threadIdx.x & 31;
        i = plan_find<kThreads>(prefix, p.n, u, costs, &at);
        r = request_of(p, i);
        const int64_t rows = static_cast<int64_t>(r.count) * p.G;
        const int tiles = tiles_of(p, r, rows);
        for (rt = 0; rt + 32 < tiles; rt += 32) {
            int64_t sum = cost_of_tile(p, r, rows, rt + lane);
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
            if (u < at + sum) break;
            at += sum;
        }
    }
    __device__ __forceinline__ bool next(Item &x) {
        while (u < end) {
            const int64_t rows = static_cast<int64_t>(r.count) * p.G;
            if (r.count <= 0 || rows <= p.short_rows || static_cast<int64_t>(rt) * kRows >= rows) {
                r = request_of(p, ++i);
                rt = 0;
                continue;
            }
            const Span s = span_of(p, r, rt);
            const bool pair = is_pair(rows, rt);
            const int64_t one = cost_of(s, pair), all = one * p.Hkv;
            if (u >= at + all) {
                at += all;
                rt++;
                continue;
            }
            x.head = static_cast<int>((u - at) / one);
            const int64_t tile = at + x.head * one + kTileCost;              // where its first unit begins
            const int step = pair ? kPairCost : 1;
            const int64_t a = (u - tile + step - 1) / step, b = (end - tile + step - 1) / step;
            x.ua = u > tile ? static_cast<int>(a) : 0;
            x.ub = end <= tile ? 0 : b < s.units ? static_cast<int>(b) : s.units;
            u = tile - kTileCost + one;
            if (x.ua >= x.ub) continue;
            x.start = r.start;
            x.count = r.count;
            x.len = r.len;
            x.lo = s.lo;
            x.hi = s.hi;
            x.base = s.base;
            x.units = s.units;
            x.i = i;
            x.rt = rt;
            x.pair = pair;
            x.last = tile + static_cast<int64_t>(s.units - 1) * step;
            return true;
        }
        x.count = 0;
        return false;
    }
};

template <int D>
__device__ __forceinline__ bool wait(Smem<D> *sm, uint64_t *bar, uint32_t parity) {
    if (mbar_try(bar, parity)) return true;
    volatile int32_t *failed = &sm->failed;
    for (uint32_t k = 0; k < kTries; k++) {
        if (mbar_try(bar, parity)) return true;
        if ((k & 63) == 63 && *failed) return false;
    }
    *failed = 1;
    return false;
}
template <int D>
__device__ __forceinline__ bool wait_all(Smem<D> *sm, uint64_t *bar, uint32_t parity) {
    return __all_sync(~0u, wait(sm, bar, parity)) != 0;
}
// What a warp's threads have written counts as there once its first lane has arrived.
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// What a row sees of a unit: columns lo .. hi, and of those the groups of 16 that have a block.
struct Seen {
    bool whole;
    int lo, hi;
    uint32_t named;
    __device__ __forceinline__ void apply(uint32_t (&s)[32], int c) const {
#pragma unroll
        for (int k = 0; k < 32; k++)
            if (k > hi - 32 * c || k < lo - 32 * c || !((named >> (2 * c + (k >> 4))) & 1)) s[k] = 0xff800000u;
    }
};

// 2^d of an integer d <= 0 (0 below 2^-126, and of -inf).
__device__ __forceinline__ float power2_down(float d) {
    return d >= -126.f ? __uint_as_float(static_cast<uint32_t>(static_cast<int>(d) + 127) << 23) : d < 0.f ? 0.f : d;
}

// Largest score of a row in the unit.
__device__ __forceinline__ float row_max(uint32_t ts, const Seen &seen) {
    float most = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < 4; c++) {
        uint32_t s[32];
        tmem_ld32(s, ts + 32 * c);
        tc_wait_ld();
        if (!seen.whole) seen.apply(s, c);
#pragma unroll
        for (int k = 0; k < 32; k += 2) most = max3(most, __uint_as_float(s[k]), __uint_as_float(s[k + 1]));
    }
    return most;
}

// w = 2^(a s + b) of 32 columns as f16; returns their sum.  kTwice: a s is rounded before b is added, so that the
// largest logit minus itself is 0 whatever its size; rounded once, it may be off by 2^-24 of the logit.
// (Not packed: the assembler made one operation of a packed product and sum.)
template <bool kTwice>
__device__ __forceinline__ float weights32(const uint32_t (&s)[32], uint32_t (&w)[16], float a, float b) {
    const uint64_t aa = pair_of(a, a), bb = pair_of(b, b);
    uint64_t part[2] = {0, 0};
#pragma unroll
    for (int k = 0; k < 32; k += 2) {
        const uint64_t y = pair_of(__uint_as_float(s[k]), __uint_as_float(s[k + 1]));
        const uint64_t x = kTwice ? pair_of(__fadd_rn(__fmul_rn(low_of(y), a), b), __fadd_rn(__fmul_rn(high_of(y), a), b)) : fma2(y, aa, bb);
        const float y0 = exp2_fast(low_of(x)), y1 = exp2_fast(high_of(x));
        part[(k >> 1) & 1] = add2(part[(k >> 1) & 1], pair_of(y0, y1));
        w[k / 2] = pack_f16(y0, y1);
    }
    const uint64_t both = add2(part[0], part[1]);
    return low_of(both) + high_of(both);
}

// Columns 64 h .. + 63, where some row's weights outgrow its reference or its logits are huge: the reference
// moves to 9 below the next integer of their largest x, with the row's sum, its weights of these columns
// so far and its accumulator (o_cols columns, 0 while it holds nothing).  Rare.
__device__ __forceinline__ void grow_rows(int h, uint32_t ts, uint32_t to, int o_cols, float a, float &top, float &sum, const Seen &seen) {
#pragma unroll 1
    for (int c = 2 * h; c < 2 * h + 2; c++) {
        uint32_t s[32], w[16];
        tc_wait_st();
        tmem_ld32(s, ts + 32 * c);
        tc_wait_ld();
        seen.apply(s, c);
        float most = -INFINITY;
#pragma unroll
        for (int k = 0; k < 32; k++) most = fmaxf(most, __uint_as_float(s[k]));
        most *= a;
        const bool grow = most > top + kHead;
        // an infinite maximum cannot be followed: its row is NaN
        most = most == INFINITY ? NAN : ceilf(most) - kHead;
        const float f = grow ? power2_down(top - most) : 1.f;
        if (grow) top = most;
        sum *= f;
        if (c & 1) {
            uint32_t y[16];
            tmem_ld16(y, ts + 16 * (c - 1));
            tc_wait_ld();
#pragma unroll
            for (int q = 0; q < 16; q++) {
                const float2 z = __half22float2(*reinterpret_cast<const __half2 *>(&y[q]));
                y[q] = pack_f16(z.x * f, z.y * f);       // f may be below f16's range
            }
            tmem_st16(ts + 16 * (c - 1), y);
        }
#pragma unroll 1
        for (int k = 0; k < o_cols; k += 16) {
            uint32_t y[16];
            tmem_ld16(y, to + k);
            tc_wait_ld();
#pragma unroll
            for (int q = 0; q < 16; q++) y[q] = __float_as_uint(__uint_as_float(y[q]) * f);
            tmem_st16(to + k, y);
        }
        sum += weights32<true>(s, w, a, top == -INFINITY ? 0.f : -top);
        tmem_st16(ts + 16 * c, w);
    }
}

// Columns 64 h .. + 63 of a unit: their exponentials, sums and packing are one block of independent work.
// Weights stand in the place of S (32 columns of scores become 16 of packed f16).  False where the
// rows' references have to be looked at first (nothing is changed then).
__device__ __forceinline__ bool row_weights(int h, uint32_t ts, float a, float top, float &sum, const Seen &seen) {
    const float ref = top == -INFINITY ? 0.f : -top;
    uint32_t s0[32], s1[32], w0[16], w1[16];
    tmem_ld32(s0, ts + 64 * h);
    tmem_ld32(s1, ts + 64 * h + 32);
    tc_wait_ld();
    if (!seen.whole) {
        seen.apply(s0, 2 * h);
        seen.apply(s1, 2 * h + 1);
    }
    const float p0 = weights32<false>(s0, w0, a, ref);
    const float p1 = weights32<false>(s1, w1, a, ref);
    if (__any_sync(~0u, p0 + p1 > kMostSum || fabsf(ref) > kHuge)) return false;
    sum += p0 + p1;
    tmem_st16(ts + 32 * h, w0);
    tmem_st16(ts + 32 * h + 16, w1);
    return true;
}

// Loads a warp's 32 query rows (`mine`: where this lane's row begins, -1: no row) as f16, each scaled by a power of
// two 2^(14 - E) (negated for a negative softmax scale, so that a larger S is a larger x), into rows row0 ..
// of a tile; returns this lane's E.  All loads are on their way at once.
template <int D, bool fp16>
__device__ __forceinline__ int load_rows(const Kv4Params &p, char *qs, int row0, int64_t mine) {
    constexpr int kLine = D / 8, kAtOnce = 32 / kLine;                // lanes of a row, rows of a step
    const int lane = threadIdx.x & 31, c = lane % kLine;
    const float sign = p.scale_log2 < 0.f ? -1.f : 1.f;
    uint4 raw[kLine];
#pragma unroll
    for (int i = 0; i < kLine; i++) {
        const int64_t from = __shfl_sync(~0u, mine, i * kAtOnce + lane / kLine);
        raw[i] = make_uint4(0, 0, 0, 0);
        if (from >= 0) raw[i] = __ldg(reinterpret_cast<const uint4 *>(p.q + from) + c);
    }
    int own = 0;
#pragma unroll
    for (int i = 0; i < kLine; i++) {
        const uint4 y = raw[i];
        uint32_t most = __vmaxu2(__vmaxu2(y.x & 0x7fff7fffu, y.y & 0x7fff7fffu), __vmaxu2(y.z & 0x7fff7fffu, y.w & 0x7fff7fffu));
#pragma unroll
        for (int o = kLine / 2; o; o >>= 1) most = __vmaxu2(most, __shfl_xor_sync(~0u, most, o));
        const float2 two = widen2(most, fp16);
        const int e = row_exponent((most & 0xffffu) > (most >> 16) ? two.x : two.y);
        const int theirs = __shfl_sync(~0u, e, lane % kAtOnce * kLine);
        if (lane / kAtOnce == i) own = theirs;
        const float f = sign * power2(14 - e);
        uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int k = 0; k < 4; k++) {
            const float2 z = widen2(w[k], fp16);
            w[k] = pack_f16(z.x * f, z.y * f);
        }
        const int row = row0 + i * kAtOnce + lane / kLine;
        *reinterpret_cast<uint4 *>(qs + (c >> 3) * (128 * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return own;
}

// ---- softmax warps: a thread per row ----------------------------------------------------------
template <int D, bool fp16>
__device__ void softmax_role(const Kv4Params &p, Smem<D> *sm, int64_t total, int64_t ranges) {
    constexpr int kPart = kRows * (D + 2);
    const int m = threadIdx.x >> 7, row = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>((threadIdx.x >> 5) & 3) << 21;      // TMEM lane of the warp
    const uint32_t ts = sm->tmem + lanes + m * 128, to = sm->tmem + lanes + 256 + m * D;
    uint32_t unit = 0, s_phase = 0, o_phase[2] = {0, 0}, h_phase = 0, side = 0;
    int4 note = make_int4(-1, 0, 0, 0);

    // This thread's row of an item: its number among the request's rows.
    auto row_of = [&](const Item &x) { return x.rt * kRows + (x.pair ? m * 128 : 0) + row; };
    // The next item's place; its queries' loading, and its rows' factor.
    uint32_t items = 0;
    auto find = [&](bool &ok) -> const Item & {
        const uint32_t k = items % kItems;
        ok = wait_all(sm, &sm->item_full[k], items / kItems & 1);
        items++;
        return sm->item[k];
    };
    auto load = [&](const Item &x) {
        const int f = row_of(x), j = f / p.G;
        const int64_t at = static_cast<int64_t>(x.start + j) * p.q_stride + 2 * static_cast<int64_t>(x.head * p.G + f - j * p.G) * D;
        const int e = load_rows<D, fp16>(p, sm->q[m], row & ~31, f < x.count * p.G ? at : -1);
        fence_async_shared();
        warp_arrive(&sm->q_full[m]);
        return fmaxf(fabsf(p.scale_log2) * power2(e - 14), 1e-37f);          // never zero, so that a hidden score stays -inf
    };
    // Whether this tile has units of it (the second of a row tile that both take has none of a single one).
    auto needs = [&](const Item &x) { return x.count && (x.pair || m == 0 || x.ub - x.ua > 1); };
    bool ok = true;
    const Item *now = &find(ok);
    if (!ok) return;
    float next_a = 0.f;
    if (needs(*now)) next_a = load(*now);
    while (now->count) {
        const Item &x = *now;
        const float a = next_a;
        const int nu = x.ub - x.ua, rows = x.count * p.G, f = row_of(x), j = f / p.G;
        const bool pair = x.pair;
        const bool live = f < rows;
        const int back = x.len - x.count, first_key = x.base + x.ua * kKeys, pos = live ? back + j : -1;
        const int f0 = f - row, f1 = min(rows, f0 + 128) - 1;
        const int pos0 = back + f0 / p.G, pos1 = back + f1 / p.G;
        // a row past the tile's last sees nothing and needs no reference to be looked for
        float top = live ? -INFINITY : 0.f, sum = 0.f;
        const int begin = pair ? 0 : m, step = pair ? 1 : 2;
        bool first = true;
        for (int t = begin; t < nu; t += step) {
            if (!wait_all(sm, &sm->s_full[m], s_phase)) return;
            s_phase ^= 1;
            tc_fence_after();
            const int s0 = first_key + t * kKeys;
            Seen seen;
            seen.named = static_cast<uint32_t>(sm->unit[(unit + t) % kUnits].z);
            seen.whole = s0 + kKeys - 1 <= pos0 && (p.window <= 0 || s0 > pos1 - p.window) && seen.named == 0xffu;
            seen.hi = pos - s0;                                              // columns lo .. hi are visible
            seen.lo = p.window > 0 && p.window <= pos ? pos - p.window + 1 - s0 : -0x40000000;
            // the first unit that shows a row anything sets its reference (no weight has been added before)
            if (__any_sync(~0u, top == -INFINITY)) {
                const float most = row_max(ts, seen) * a;
                if (top == -INFINITY) top = most == INFINITY ? NAN : ceilf(most) - kHead;
            }
            // one body for both halves, not unrolled: a whole unit's would not stay in the instruction cache
#pragma unroll 1
            for (int h = 0; h < 2; h++) {
                if (!row_weights(h, ts, a, top, sum, seen)) {
                    // the accumulator is not touched while the first half's product is under way
                    if (h == 1 && !wait_all(sm, &sm->h_done[m], h_phase)) return;
                    tc_fence_after();
                    grow_rows(h, ts, to, first && h == 0 ? 0 : D, a, top, sum, seen);
                }
                tc_wait_st();
                tc_fence_before();
                warp_arrive(h ? &sm->p_full[m] : &sm->p_half[m]);
            }
            h_phase ^= 1;
            first = false;
        }
        unit += nu;
        // All scores of this tile are there: its queries' place takes the next item's.
        const Item &y = find(ok);
        if (!ok) return;
        if (needs(y)) next_a = load(y);

        const bool full = x.ua == 0 && x.ub == x.units;
        const int hq = x.head * p.G + f - j * p.G;
        float scale = 1.f, scale2 = 0.f;          // of this warpgroup's accumulator, and of the other's
        if (!first) {
            if (!wait_all(sm, &sm->o_full[m], o_phase[m])) return;
            o_phase[m] ^= 1;
            tc_fence_after();
        }
        if (!pair) {
            side ^= 1;
            if (m == 1) {
                // leave the statistics, and the accumulator in TMEM, until the other warpgroup has read them
                sm->top[row] = top;
                sm->sum[row] = sum;
                tc_fence_before();
                warp_arrive(&sm->side_full);
                if (!wait_all(sm, &sm->side_free, side ^ 1)) return;
                now = &y;
                continue;
            }
            if (!wait_all(sm, &sm->side_full, side ^ 1)) return;
            tc_fence_after();
            const float top2 = sm->top[row], sum2 = sm->sum[row];
            const bool none2 = top2 == -INFINITY && sum2 == 0.f, none1 = top == -INFINITY && sum == 0.f;
            if (!none2) {
                const float most = none1 ? top2 : fmaxf(top, top2);          // references are integers (or NaN)
                scale = none1 ? 0.f : power2_down(top - most);
                scale2 = power2_down(top2 - most);
                sum = (none1 ? 0.f : sum * scale) + sum2 * scale2;
                top = top != top || top2 != top2 ? NAN : most;
            }
        }
        const bool none = !live || (top == -INFINITY && sum == 0.f);
        const float inv = full ? (none ? 0.f : p.v_unit / sum) : p.v_unit;
        scale *= inv;
        scale2 *= inv;
        float *part = p.part + (2LL * blockIdx.x + (x.ua == 0)) * kPart;
        char *out = p.out + static_cast<int64_t>(x.start + j) * p.out_stride + 2 * static_cast<int64_t>(hq) * D;
        const bool both = !pair && __any_sync(~0u, scale2 != 0.f);        // NaN too; a pair's second tile has no other
#pragma unroll 1
        for (int c = 0; c < D / 32; c++) {
            uint32_t o[32];
            tmem_ld32(o, to + 32 * c);
            tc_wait_ld();
#pragma unroll
            for (int k = 0; k < 32; k++) o[k] = none || scale == 0.f ? 0u : __float_as_uint(__uint_as_float(o[k]) * scale);
            if (both) {
                uint32_t o2[32];
                tmem_ld32(o2, to + D + 32 * c);
                tc_wait_ld();
#pragma unroll
                for (int k = 0; k < 32; k++)
                    if (scale2 != 0.f) o[k] = __float_as_uint(fmaf(__uint_as_float(o2[k]), scale2, __uint_as_float(o[k])));
            }
            if (full && live) {
                uint32_t y16[16];
#pragma unroll
                for (int k = 0; k < 16; k++) y16[k] = pack_out(__uint_as_float(o[2 * k]), __uint_as_float(o[2 * k + 1]), fp16);
#pragma unroll
                for (int k = 0; k < 4; k++)
                    *reinterpret_cast<uint4 *>(out + 64 * c + 16 * k) = make_uint4(y16[4 * k], y16[4 * k + 1], y16[4 * k + 2], y16[4 * k + 3]);
            } else if (live) {
                float *at = part + 2 * kRows + ((pair ? m * 128 : 0) + row) * D + 32 * c;
#pragma unroll
                for (int k = 0; k < 8; k++)
                    *reinterpret_cast<uint4 *>(at + 4 * k) = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
            }
            __syncwarp();
        }
        if (live) {
            if (full) {
                if (p.lse)
                    p.lse[static_cast<int64_t>(x.start + j) * p.Hkv * p.G + hq] = none ? -INFINITY : (top + log2f(sum)) * kLn2;
            } else {
                part[(pair ? m * 128 : 0) + row] = top;
                part[kRows + (pair ? m * 128 : 0) + row] = sum;
            }
        }
        if (!full && x.ua == 0) {
            const int64_t last = ((x.last + 1) * ranges - 1) / total;        // the range with the tile's last unit
            note = make_int4(x.i, x.rt, static_cast<int>(last - blockIdx.x) + 1, x.head);
        }
        tc_fence_before();
        if (!pair) warp_arrive(&sm->side_free);
        now = &y;
    }
    if (m == 0 && row == 0) p.meta[blockIdx.x] = note;
}

// ---- converting warps: codes to f16 operand tiles ---------------------------------------------
// A warpgroup for the keys, one for the values.  A thread's codes and scales of the next unit are on their way
// into registers while it converts this one's.
template <int D>
__device__ void convert_role(const Kv4Params &p, Smem<D> *sm, bool values) {
    constexpr int kC = D / 32;                       // 16-byte pieces of a token's codes
    constexpr int kTok = 32 * kConvWarps / kC;       // tokens per round of the threads, a multiple of 16
    constexpr int kRounds = kKeys / kTok;
    const int i = (threadIdx.x - 32 * kSoftWarps) % (32 * kConvWarps);
    const int c = i % kC, tok = i / kC;              // this thread's piece, and its token within a round
    // The four 16-byte places of a piece's 32 converted codes in a 128-byte row; threads of the upper 64
    // dimensions begin with the third, so that eight neighbours write to eight bank groups.
    const int turn = (c >> 1) << 1;
    const uint32_t row = (c >> 1) * (kKeys * 128) + tok * 128;
    uint32_t to[4];
#pragma unroll
    for (int k = 0; k < 4; k++) to[k] = row + ((((c & 1) * 4 + (k ^ turn)) ^ (tok & 7)) << 4);
    const uint8_t *codes = (values ? p.vc : p.kc) + (tok & 15) * (D / 2) + 16 * c;
    const uint8_t *scales = (values ? p.v_sf : p.k_sf) + (tok & 15) * (D / 16) + 2 * c;
    char *dst = values ? sm->v[0] : sm->k[0];
    uint64_t *freed = values ? sm->v_free : sm->k_free, *filled = values ? sm->v_full : sm->k_full;

    uint4 y[kRounds];
    uint32_t sc[kRounds];
    // A token that no row sees, or without a block: scales of zero (codes are finite whatever they are).
    auto load = [&](uint32_t unit, const int4 &of, int r) {
        const int k = r * kTok + tok;
        const bool on = k >= of.x && k < of.y && ((of.z >> (k >> 4)) & 1);
        const int64_t line = sm->line[unit % kUnits][k >> 4];
        sc[r] = 0;
        if (on) {
            y[r] = __ldg(reinterpret_cast<const uint4 *>(codes + line * (D / 2)));
            sc[r] = __ldg(reinterpret_cast<const uint16_t *>(scales + line * (D / 16)));
        }
    };
    if (!wait_all(sm, &sm->unit_full[0], 0)) return;
    int4 of = sm->unit[0];
    if (of.w & kNone) {
        warp_arrive(&filled[0]);
        return;
    }
#pragma unroll
    for (int r = 0; r < kRounds; r++) {
        y[r] = make_uint4(0, 0, 0, 0);
        load(0, of, r);
    }
    for (uint32_t unit = 0;; unit++) {
        const uint32_t stage = unit & 1, next = unit + 1;
        const bool end = of.w & kEnd;
        if (!end) {
            if (!wait_all(sm, &sm->unit_full[next % kUnits], next / kUnits & 1)) return;
            of = sm->unit[next % kUnits];
        }
        if (!wait_all(sm, &freed[stage], ((unit >> 1) & 1) ^ 1)) return;
        char *at = dst + stage * (kKeys * D * 2);
#pragma unroll
        for (int r = 0; r < kRounds; r++) {
            const uint32_t s = f16x2_of(sc[r]), s0 = turn ? high_twice(s) : low_twice(s), s1 = turn ? low_twice(s) : high_twice(s);
            const uint32_t w[4] = {turn ? y[r].z : y[r].x, turn ? y[r].w : y[r].y, turn ? y[r].x : y[r].z, turn ? y[r].y : y[r].w};
#pragma unroll
            for (int k = 0; k < 4; k++) {
                uint32_t h[4];
                f16_of_e2m1x8(w[k], h);
                const uint32_t f = k < 2 ? s0 : s1;
                *reinterpret_cast<uint4 *>(at + to[k] + r * kTok * 128) =
                    make_uint4(mul_f16x2(h[0], f), mul_f16x2(h[1], f), mul_f16x2(h[2], f), mul_f16x2(h[3], f));
            }
        }
        fence_async_shared();
        warp_arrive(&filled[stage]);
        if (end) return;
#pragma unroll
        for (int r = 0; r < kRounds; r++) load(next, of, r);
    }
}

// ---- walking warp -----------------------------------------------------------------------------
// Finds the CTA's units and where their lines are, and tells the others; lane g looks up group g.
template <int D>
__device__ void walk_role(const Kv4Params &p, Smem<D> *sm, Walk &walk) {
    const int lane = threadIdx.x & 31, g = lane & 7;
    const int jump = kKeys / p.bs, rest = kKeys - jump * p.bs;
    uint32_t items = 0;
    Item x;
    const int32_t *table = nullptr;
    int s = 0, entry = 0, offset = 0;                // the group's first token, its table entry and place in the block
    auto next = [&]() {
        const bool more = walk.next(x);
        if (lane == 0) {
            sm->item[items % kItems] = x;
            mbar_arrive(&sm->item_full[items % kItems]);
        }
        items++;
        table = p.tables + static_cast<int64_t>(x.i) * p.table_row;
        s = x.base + x.ua * kKeys + 16 * g;
        entry = s / p.bs;
        offset = s - entry * p.bs;
        return more;
    };
    // a block id that has been asked for but not yet looked at, of the unit after the one that is told of
    int32_t id = -1;
    auto ask = [&]() { id = s < x.hi && s + 16 > x.lo && entry < p.W ? table[entry] : -1; };
    bool more = next();
    if (more) {
        ask();
    } else if (lane == 0) {
        sm->unit[0] = make_int4(0, 0, 0, kNone);
        mbar_arrive(&sm->unit_full[0]);
    }
    int left = x.ub - x.ua;
    for (uint32_t unit = 0; more; unit++) {
        if (id >= p.num_blocks) {
            if (p.err) atomicOr(p.err, PKV_DEVERR_BLOCK);
            id = -1;
        }
        const int64_t line = (static_cast<int64_t>(id) * p.Hkv + x.head) * p.bs + offset;
        const uint32_t named = __ballot_sync(~0u, id >= 0) & 0xffu;
        const int at = s - 16 * g;
        int4 of = make_int4(x.lo - at, x.hi - at, static_cast<int>(named), x.pair ? kPair : 0);
        s += kKeys;
        entry += jump;
        offset += rest;
        if (offset >= p.bs) {
            offset -= p.bs;
            entry++;
        }
        if (--left == 0) {
            more = next();
            left = x.ub - x.ua;
            of.w |= kTileEnd | (more ? 0 : kEnd);
        }
        if (more) ask();                             // on its way while this unit's place becomes free
        if (!wait_all(sm, &sm->unit_free[unit % kUnits], (unit / kUnits & 1) ^ 1)) return;
        if (lane < 8) sm->line[unit % kUnits][g] = line;
        if (lane == 0) sm->unit[unit % kUnits] = of;
        warp_arrive(&sm->unit_full[unit % kUnits]);
    }
}

// ---- issuing warp ------------------------------------------------------------------------------
// The whole warp goes through the units, so that addresses and descriptors stay in uniform registers; one
// lane issues.  (A warp for each tile took 1.13 times as long: the tiles' products delay each other.)
// Operand descriptors as in smem_desc: the upper word is the same for all, the lower one holds the address.
constexpr uint32_t kDescHigh = (1024 >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t lead) { return ((addr & 0x3ffffu) >> 4) | (lead >> 4 << 16); }
__device__ __forceinline__ uint64_t desc_of(uint32_t low) { return static_cast<uint64_t>(kDescHigh) << 32 | low; }

template <int D>
__device__ void issue_role(Smem<D> *sm) {
    constexpr uint32_t kQk = f16_idesc(128, kKeys, false), kPv = f16_idesc(128, D, true);
    constexpr uint32_t kStage = kKeys * D * 2 >> 4;
    const uint32_t q_low = desc_low(smem_addr(sm->q[0]), 16), k_low = desc_low(smem_addr(sm->k[0]), 16);
    const uint32_t v_low = desc_low(smem_addr(sm->v[0]), kKeys * 128);
    uint32_t unit = 0, q_phase[2] = {0, 0}, p_phase[2] = {0, 0};
    const bool leader = elect_one();
    bool ok = true;
    auto commit = [&](uint64_t *bar) {
        if (leader) tc_commit(bar);
        __syncwarp();
    };
    // Scores of unit u in tile m, whose keys are there.  (All of TMEM is this CTA's: its addresses begin at 0.)
    auto qk = [&](auto tile, uint32_t u) {
        constexpr int m = decltype(tile)::value;
        if (leader && ok) {
            const uint32_t da = q_low + m * (128 * D * 2 >> 4), db = k_low + (u & 1) * kStage;
#pragma unroll
            for (int k = 0; k < D / 16; k++) {
                constexpr uint32_t kPanel = 128 * 128;
                const uint32_t off = ((k >> 2) * kPanel + (k & 3) * 32) >> 4;
                mma_ss(m * 128, desc_of(da + off), desc_of(db + off), kQk, k > 0);
            }
            mbar_arrive(&sm->s_full[m]);             // what this warp knows of the unit, as well as the products
            tc_commit(&sm->s_full[m]);
        }
        __syncwarp();
    };
    // Waits for a unit's keys; what kind of unit it is.
    auto keys = [&](uint32_t u) {
        ok = ok && wait_all(sm, &sm->k_full[u & 1], (u >> 1) & 1);
        tc_fence_after();
        return ok ? __shfl_sync(~0u, sm->unit[u % kUnits].w, 0) : kNone;
    };
    // A tile's second product, in two halves of 64 tokens.
    auto pv = [&](auto tile, uint32_t u, bool add) {
        constexpr int m = decltype(tile)::value;
        const uint32_t db = v_low + (u & 1) * kStage;
        ok = ok && wait(sm, &sm->v_full[u & 1], (u >> 1) & 1) && wait(sm, &sm->p_half[m], p_phase[m]);
        tc_fence_after();
        if (leader && ok) {
#pragma unroll
            for (int k = 0; k < kKeys / 32; k++) mma_ts(256 + m * D, m * 128 + 8 * k, desc_of(db + k * (2048 >> 4)), kPv, add || k > 0);
            tc_commit(&sm->h_done[m]);
        }
        __syncwarp();
        ok = ok && wait(sm, &sm->p_full[m], p_phase[m]);
        p_phase[m] ^= 1;
        tc_fence_after();
        if (leader && ok) {
#pragma unroll
            for (int k = kKeys / 32; k < kKeys / 16; k++) mma_ts(256 + m * D, m * 128 + 8 * k, desc_of(db + k * (2048 >> 4)), kPv, true);
        }
        ok = __all_sync(~0u, ok);
    };
    constexpr std::integral_constant<int, 0> tile0{};
    constexpr std::integral_constant<int, 1> tile1{};
    for (int kind = 0; ok && !(kind & kEnd);) {
        kind = keys(unit);
        if (kind & kNone) break;
        for (int m = 0; m < 2 && ok; m++) {
            if (m == 1 && !(kind & kPair) && (kind & kTileEnd)) continue;    // the second tile has no unit of it
            ok = wait_all(sm, &sm->q_full[m], q_phase[m]);
            q_phase[m] ^= 1;
        }
        if (!ok) break;
        tc_fence_after();
        if (kind & kPair) {
            qk(tile0, unit);
            qk(tile1, unit);
            commit(&sm->k_free[unit & 1]);
            for (bool add = false; ok; add = true, unit++) {
                const bool end = kind & kTileEnd;
                int next = kind;
                pv(tile0, unit, add);
                if (!end) next = keys(unit + 1);
                if (!ok) break;
                if (end) commit(&sm->o_full[0]);
                else qk(tile0, unit + 1);
                pv(tile1, unit, add);
                if (!ok) break;
                if (leader) {
                    mbar_arrive(&sm->unit_free[unit % kUnits]);
                    tc_commit(&sm->v_free[unit & 1]);
                }
                __syncwarp();
                if (end) {
                    commit(&sm->o_full[1]);
                    break;
                }
                qk(tile1, unit + 1);
                commit(&sm->k_free[(unit + 1) & 1]);
                kind = next;
            }
            unit++;
        } else {
            // tile t & 1 takes unit t: the same rows
            qk(tile0, unit);
            commit(&sm->k_free[unit & 1]);
            int next = kind;                         // the kind of the unit after this one, if there is one
            if (!(kind & kTileEnd)) {
                next = keys(unit + 1);
                if (!ok) break;
                qk(tile1, unit + 1);
                commit(&sm->k_free[(unit + 1) & 1]);
            }
            for (int t = 0; ok; t++, unit++) {
                if (t & 1) pv(tile1, unit, t > 1);
                else pv(tile0, unit, t > 1);
                if (!ok) break;
                if (leader) mbar_arrive(&sm->unit_free[unit % kUnits]);
                commit(&sm->v_free[unit & 1]);
                int after = next;
                if (!((kind | next) & kTileEnd)) {
                    after = keys(unit + 2);
                    if (!ok) break;
                    if (t & 1) qk(tile1, unit + 2);
                    else qk(tile0, unit + 2);
                    commit(&sm->k_free[unit & 1]);
                } else {
                    commit(&sm->o_full[t & 1]);
                }
                if (kind & kTileEnd) break;
                kind = next;
                next = after;
            }
            unit++;
        }
    }
    // the products end before the TMEM is freed
    commit(&sm->done);
    for (uint32_t k = 0; k < kTries; k++)
        if (mbar_try(&sm->done, 0)) break;
}

template <int D, bool fp16>
__global__ void __launch_bounds__(kThreads, 1) kv4_prefill_kernel(const Kv4Params p) {
    extern __shared__ char s_raw[];
    // the swizzle goes by address bits: the operand tiles start on 1024 bytes
    Smem<D> *sm = reinterpret_cast<Smem<D> *>(s_raw + (-smem_addr(s_raw) & 1023u));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (warp == 0) tmem_alloc(&sm->tmem, 512);
    if (threadIdx.x == 32) {
        for (int k = 0; k < 2; k++) {
            mbar_init(&sm->q_full[k], 4);
            mbar_init(&sm->k_full[k], kConvWarps);
            mbar_init(&sm->v_full[k], kConvWarps);
            mbar_init(&sm->k_free[k], 1);
            mbar_init(&sm->v_free[k], 1);
            mbar_init(&sm->s_full[k], 2);
            mbar_init(&sm->p_half[k], 4);
            mbar_init(&sm->p_full[k], 4);
            mbar_init(&sm->h_done[k], 1);
            mbar_init(&sm->o_full[k], 1);
        }
        for (int k = 0; k < kUnits; k++) {
            mbar_init(&sm->unit_full[k], 1);
            mbar_init(&sm->unit_free[k], 1);
        }
        for (int k = 0; k < kItems; k++) mbar_init(&sm->item_full[k], 1);
        mbar_init(&sm->side_full, 4);
        mbar_init(&sm->side_free, 4);
        mbar_init(&sm->done, 1);
        sm->failed = 0;
        fence_mbar_init();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();
    pdl_trigger();
    // The plan's sums lie where the first keys go: these wait for the walking warp, which has read them then.  The
    // costs of the requests of a small batch are found by whole warps, and lie where the first values go.
    int64_t *prefix = reinterpret_cast<int64_t *>(sm->k), *each = reinterpret_cast<int64_t *>(sm->v);
    const bool together = p.n <= kThreads;
    if (together) {
        for (int i = warp; i < p.n; i += kThreads / 32) {
            int64_t sum = cost_of_request(p, request_of(p, i, blockIdx.x == 0 && lane == 0), lane, 32);
#pragma unroll
            for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
            if (lane == 0) each[i] = sum;
        }
        __syncthreads();
    }
    const int64_t total = plan_prefix<kThreads>(prefix, prefix + kThreads + 1, p.n, [&](int i) {
        return together ? each[i] : cost_of_request(p, request_of(p, i, blockIdx.x == 0));
    });
    __syncthreads();                                 // everybody has the total
    // at least kPairCost each, so that every range inside a row tile's units has one
    const int64_t ranges = total / kPairCost < gridDim.x ? total / kPairCost : gridDim.x;
    if (blockIdx.x < ranges) {
        if (warp < kSoftWarps) {
            more_registers<kSoftRegs>();
            softmax_role<D, fp16>(p, sm, total, ranges);
        } else if (warp < kSoftWarps + 2 * kConvWarps) {
            fewer_registers<kConvRegs>();
            convert_role<D>(p, sm, warp >= kSoftWarps + kConvWarps);
        } else {
            fewer_registers<kIssueRegs>();
            if (warp == kSoftWarps + 2 * kConvWarps) issue_role<D>(sm);
            if (warp == kSoftWarps + 2 * kConvWarps + 1) {
                Walk walk(p, prefix, blockIdx.x * total / ranges, (blockIdx.x + 1) * total / ranges,
                          [&](int i) { return together ? each[i] : cost_of_request(p, request_of(p, i)); });
                __syncwarp();
                walk_role<D>(p, sm, walk);
            }
        }
    } else if (threadIdx.x == 0) {
        p.meta[blockIdx.x] = make_int4(-1, 0, 0, 0);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (threadIdx.x == 0 && sm->failed) {
        p.meta[blockIdx.x] = make_int4(-1, 0, 0, 0);
        if (p.err) atomicOr(p.err, PKV_DEVERR_TIMEOUT);
    }
    if (warp == 0) {
        __syncwarp();
        tmem_free(sm->tmem, 512);
    }
}

template <int D, bool fp16>
int launch(const Kv4Params &p, int sms, cudaStream_t s) {
    constexpr size_t smem = sizeof(Smem<D>) + 1024;
    static_assert(smem <= 227 * 1024, "shared memory");
    static bool set[64] = {false};
    const int rc = kv8_allow_smem(reinterpret_cast<const void *>(kv4_prefill_kernel<D, fp16>), static_cast<int>(smem), set);
    if (rc != PKV_OK) return rc;
    PKV_CUDA_TRY(launch_pdl(kv4_prefill_kernel<D, fp16>, dim3(sms), dim3(kThreads), smem, s, p));
    return kv4_launch_merge(p, D, kRows, sms, 1, sms, s);
}

}  // namespace

int64_t kv4_prefill_workspace(int32_t head_dim, int sms) {
    return head_dim > 128 ? 0 : static_cast<int64_t>(sms) * (2LL * kRows * (head_dim + 2) * 4 + 16);
}

int kv4_launch_prefill(const Kv4Params &p, int32_t head_dim, int sms, cudaStream_t s) {
    if (p.fp16) return head_dim == 64 ? launch<64, true>(p, sms, s) : launch<128, true>(p, sms, s);
    return head_dim == 64 ? launch<64, false>(p, sms, s) : launch<128, false>(p, sms, s);
}

}  // namespace pkv
