// Attention over the 8-bit paged cache for requests with many query rows
// (prompt chunks), on the tensor cores.
//
// Mathematics: as in pkv_kv8_decode.cu.  x = S * a_b + lv_b with S = q . code_k
// from the tensor core, a_b = k_scale * softmax_scale * log2(e) and lv_b =
// log2(v_scale), both constant over 16 tokens; w = 2^(x - R) goes into the
// second product as f16, the softmax sum adds w / v_scale in fp32.  R is the
// row's maximum over its first unit, rounded up to an integer, and then follows
// lazily: it moves only when the sum of 64 w, which is needed anyway, exceeds
// 2^14, and by a whole power of two, so that weights which are f16 already are
// not rounded again (unless they turn subnormal).  So later units
// take no pass for the maximum, the accumulator is hardly ever rescaled, and w
// stays inside f16's range: it is off by 2^-11 of itself, or by 2^-25 of the
// reference's weight (w = 1) where it is 2^-14 or less and f16 is subnormal.
//
// Bound: the tensor pipe (4 D flops per visible pair); beside it per tile of
// 256 rows x 128 tokens 32768 exponentials and 32768 codes turned into f16.
//
// Layout.  A CTA holds 256 (query, head) rows of one KV head in two tiles of
// 128.  Warps 0-3 and 4-7 do the softmax of one tile each, a thread per row;
// warps 8-11 read the codes of 128 tokens, turn them into f16 (exact) and lay
// them out for the tensor core, so one conversion serves both tiles; warp 12
// issues the products: S = Q K^T (both in shared memory), O += P V with P in
// TMEM in the place of S.  While one tile's softmax runs, the tensor core
// works on the other.  The batch's (row tile, KV head, 128 tokens) units are
// split evenly over the CTAs; a row tile that is cut leaves partial results
// for a merge in a fixed order.
//
// Measured: 913 GFLOP of chunks (2 x 2048 tokens, 4 heads a group, contexts up to
// 16384) 803 us, 1.14 PFLOP/s, 58 % of the measured rate, the tensor pipe active
// 48 % of the time.  A unit takes about 4150 cycles against 2048 of products: the
// way from a tile's scores through its softmax (2100 cycles at two warps a
// scheduler) and back into its next scores is longer than the other tile's
// products.  Not kept: a second issuing warp (1020 us), eight converting warps
// (990 us, registers), bodies unrolled over a unit (instruction cache, 2 x slower).
//
// Every wait has a limit; one that runs out sets PKV_DEVERR_TIMEOUT, the other
// waits give up after it, and the CTA drains its products and frees its TMEM.
#include "pkv_kv8_attention.cuh"
#include "pkv_tcgen05.cuh"

namespace pkv {
namespace {

constexpr int kRows = 256;              // rows of a CTA, two tiles of 128
constexpr int kKeys = 128;              // tokens per unit
constexpr int kSub = kKeys / 16;
constexpr int kSoftWarps = 8, kConvWarps = 4;
constexpr int kThreads = 32 * (kSoftWarps + kConvWarps + 4);   // and a warpgroup whose first warp issues
// Registers a thread: launched with 128; 256 x 176 + 128 x 104 + 128 x 56 = 512 x 128.
constexpr int kSoftRegs = 176, kConvRegs = 104, kIssueRegs = 56;
static_assert(32 * (kSoftWarps * kSoftRegs + kConvWarps * kConvRegs + 4 * kIssueRegs) <= 65536, "registers");
static_assert((kThreads + 1 + kThreads / 32) * 8 <= 2 * kKeys * 64, "the plan's sums lie in the raw codes' place");
constexpr uint32_t kTries = 1u << 22;   // polls before a wait gives up (half a second or more)
constexpr float kMostSum = 16384.f;     // sum of 64 w that makes R follow the row's maximum

template <int D>
struct Smem {
    char q[2][128 * D * 2];
    char k[2][kKeys * D * 2];
    char v[2][kKeys * D * 2];
    char raw[2][kKeys * D];             // codes of the unit that is converted next: keys, values
    alignas(16) float ks[4][kSub], lv[4][kSub], iv[4][kSub];   // per 16 tokens: k_scale, log2(v_scale), 1 / v_scale
    uint64_t q_full[2], k_full[2], v_full[2], k_free[2], v_free[2], s_full[2], p_full[2], o_full[2], done;
    uint32_t tmem;
    int32_t failed;
    int32_t nan_seen;                   // this CTA has met a V code that is NaN,
    uint8_t nan_units[1024];            // in units of these numbers, modulo 1024
};

// The keys that rows f0 .. of a tile see: [lo, hi), and the 16-aligned start of their units.
struct Span {
    int lo, hi, base, units;
};
__device__ __forceinline__ Span span_of(const AttnParams &p, const Req &r, int rt) {
    const int rows = r.count * p.G, f0 = rt * kRows, f1 = min(rows, f0 + kRows) - 1;
    const int back = r.len - r.count, pos0 = back + f0 / p.G, pos1 = back + f1 / p.G;
    Span s;
    s.lo = p.window > 0 ? max(0, pos0 - p.window + 1) : 0;
    s.hi = min(pos1 + 1, r.keys);
    s.base = s.lo & ~15;
    s.units = s.hi > s.base ? (s.hi - s.base + kKeys - 1) / kKeys : 1;   // a tile without keys writes zeros
    return s;
}
__device__ __forceinline__ int64_t units_of_request(const AttnParams &p, const Req &r) {
    const int64_t rows = static_cast<int64_t>(r.count) * p.G;
    if (r.count <= 0 || rows <= p.short_rows) return 0;
    int64_t sum = 0;
    for (int rt = 0; rt * kRows < rows; rt++) sum += span_of(p, r, rt).units;
    return sum * p.Hkv;
}

// One stretch of units: a row tile, a KV head, and which of its 128-token units.
struct Item {
    Req r;
    Span s;
    const int32_t *table;
    int i, rt, head, ua, ub, tiles;     // tiles: 128-row tiles with rows in them
    int64_t tile;                       // the row tile's (and head's) first unit
};

template <int D>
struct Walk {
    const AttnParams &p;
    int64_t u, end, first;
    int i, rt;
    int64_t rt_first;                   // first unit of the row tile `rt`

    __device__ __forceinline__ Walk(const AttnParams &p_, const int64_t *prefix, int64_t u0, int64_t u1) : p(p_), u(u0), end(u1) {
        i = plan_find<kThreads>(prefix, p.n, u, [&](int k) { return units_of_request(p, request_of(p, k)); }, &first);
        rt = 0;
        rt_first = first;
    }
    __device__ __forceinline__ bool next(Item &x) {
        if (u >= end) return false;
        for (;;) {
            const Req r = request_of(p, i);
            const int64_t rows = static_cast<int64_t>(r.count) * p.G;
            if (r.count <= 0 || rows <= p.short_rows || static_cast<int64_t>(rt) * kRows >= rows) {
                i++;
                rt = 0;
                continue;
            }
            const Span s = span_of(p, r, rt);
            const int64_t all = static_cast<int64_t>(s.units) * p.Hkv;
            if (u >= rt_first + all) {
                rt_first += all;
                rt++;
                continue;
            }
            x.r = r;
            x.s = s;
            x.i = i;
            x.rt = rt;
            x.table = p.tables + static_cast<int64_t>(i) * p.W;
            x.head = static_cast<int>((u - rt_first) / s.units);
            x.tile = rt_first + static_cast<int64_t>(x.head) * s.units;
            x.ua = static_cast<int>(u - x.tile);
            x.ub = static_cast<int>(end - x.tile < s.units ? end - x.tile : s.units);
            x.tiles = rows - static_cast<int64_t>(rt) * kRows > 128 ? 2 : 1;
            u = x.tile + x.ub;
            return true;
        }
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

// Scores outside columns lo .. hi become -inf (of 32 columns).
__device__ __forceinline__ void hide(uint32_t (&s)[32], int lo, int hi) {
#pragma unroll
    for (int k = 0; k < 32; k++)
        if (k > hi || k < lo) s[k] = 0xff800000u;
}

// The factors of two 16-token groups; never zero, so that a hidden score stays -inf.
__device__ __forceinline__ float2 factors(float cf, float2 ks) {
    const float a = cf * ks.x, b = cf * ks.y;
    return make_float2(a < 1e-37f ? 1e-37f : a, b < 1e-37f ? 1e-37f : b);
}

// Largest x of a row in the unit.
template <int D>
__device__ __forceinline__ float row_max(const Smem<D> *sm, uint32_t ts, int ring, float cf, int lo, int hi) {
    float most = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < 4; c++) {
        uint32_t s[32];
        tmem_ld32(s, ts + 32 * c);
        const float2 a = factors(cf, *reinterpret_cast<const float2 *>(&sm->ks[ring][2 * c]));
        const float2 lv = *reinterpret_cast<const float2 *>(&sm->lv[ring][2 * c]);
        tc_wait_ld();
        hide(s, lo - 32 * c, hi - 32 * c);
#pragma unroll
        for (int h = 0; h < 2; h++) {
            float mx = __uint_as_float(s[16 * h]);
#pragma unroll
            for (int k = 1; k < 15; k += 2) mx = max3(mx, __uint_as_float(s[16 * h + k]), __uint_as_float(s[16 * h + k + 1]));
            mx = fmaxf(mx, __uint_as_float(s[16 * h + 15]));
            most = fmaxf(most, fmaf(mx, h ? a.y : a.x, h ? lv.y : lv.x));
        }
    }
    return most;
}

// w = 2^(a s + b) of 32 columns as f16; returns the two groups' sums.
__device__ __forceinline__ float2 weights32(const uint32_t (&s)[32], uint32_t (&w)[16], float2 a, float2 b) {
    float2 sums;
#pragma unroll
    for (int h = 0; h < 2; h++) {
        const uint64_t aa = h ? pair_of(a.y, a.y) : pair_of(a.x, a.x), bb = h ? pair_of(b.y, b.y) : pair_of(b.x, b.x);
        uint64_t part = 0;
#pragma unroll
        for (int k = 0; k < 16; k += 2) {
            const uint64_t x = fma2(pair_of(__uint_as_float(s[16 * h + k]), __uint_as_float(s[16 * h + k + 1])), aa, bb);
            const float y0 = exp2_fast(low_of(x)), y1 = exp2_fast(high_of(x));
            part = add2(part, pair_of(y0, y1));
            w[8 * h + k / 2] = pack_f16(y0, y1);
        }
        (h ? sums.y : sums.x) = low_of(part) + high_of(part);
    }
    return sums;
}

// 2^d of an integer d <= 0 (0 below 2^-126, and of -inf).
__device__ __forceinline__ float power2_down(float d) {
    return d >= -126.f ? __uint_as_float(static_cast<uint32_t>(static_cast<int>(d) + 127) << 23) : d < 0.f ? 0.f : d;
}

// Columns 32 c .. of a unit from `c` on, where some row's weights outgrow its reference: the reference
// moves up to the next integer of their largest x, with the row's sum, its weights of this unit so far and its
// accumulator (o_cols columns, 0 while it holds nothing).  Rare.
template <int D>
__device__ __forceinline__ void grow_rows(const Smem<D> *sm, int c, uint32_t ts, uint32_t to, int o_cols, int ring, float cf,
                                          float &top, float &sum, int lo, int hi) {
#pragma unroll 1
    for (; c < 4; c++) {
        uint32_t s[32], w[16];
        tc_wait_st();
        tmem_ld32(s, ts + 32 * c);
        const float2 a = factors(cf, *reinterpret_cast<const float2 *>(&sm->ks[ring][2 * c]));
        const float2 lv = *reinterpret_cast<const float2 *>(&sm->lv[ring][2 * c]);
        const float2 iv = *reinterpret_cast<const float2 *>(&sm->iv[ring][2 * c]);
        tc_wait_ld();
        hide(s, lo - 32 * c, hi - 32 * c);
        float most = -INFINITY;
#pragma unroll
        for (int k = 0; k < 32; k++) most = fmaxf(most, fmaf(__uint_as_float(s[k]), k < 16 ? a.x : a.y, k < 16 ? lv.x : lv.y));
        const bool grow = most > top;
        // an infinite maximum cannot be followed: its row is NaN
        most = most == INFINITY ? NAN : ceilf(most);
        const float f = grow ? power2_down(top - most) : 1.f;
        if (grow) top = most;
        sum *= f;
#pragma unroll 1
        for (int k = 0; k < c; k++) {
            uint32_t y[16];
            tmem_ld16(y, ts + 16 * k);
            tc_wait_ld();
#pragma unroll
            for (int q = 0; q < 16; q++) {
                const float2 z = __half22float2(*reinterpret_cast<const __half2 *>(&y[q]));
                y[q] = pack_f16(z.x * f, z.y * f);       // f may be below f16's range
            }
            tmem_st16(ts + 16 * k, y);
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
        const float ref = top == -INFINITY ? 0.f : top;
        const float2 part = weights32(s, w, a, make_float2(lv.x - ref, lv.y - ref));
        sum = fmaf(part.x, iv.x, fmaf(part.y, iv.y, sum));
        tmem_st16(ts + 16 * c, w);
    }
}

// All of a unit's columns, 64 at a time: their exponentials, sums and packing are one block of
// independent work, which hides its own latencies (a call of chunks and decodes 1704 us, one under a
// window 771; 32 columns at a time, the next on their way, 1711 and 776).  Weights stand in the place
// of S (32 columns of scores become 16 of packed f16).  The loop is not unrolled: the body of a whole
// unit would not stay in the instruction cache beside the other warps' code.
template <int D>
__device__ __forceinline__ void row_weights(const Smem<D> *sm, uint32_t ts, uint32_t to, int o_cols, int ring, float cf,
                                            float &top, float &sum, bool whole, int lo, int hi) {
    const float ref = top == -INFINITY ? 0.f : top;
    int c = 0;
#pragma unroll 1
    for (; c < 4; c += 2) {
        uint32_t s0[32], s1[32], w0[16], w1[16];
        tmem_ld32(s0, ts + 32 * c);
        tmem_ld32(s1, ts + 32 * (c + 1));
        const float4 ks = *reinterpret_cast<const float4 *>(&sm->ks[ring][2 * c]);
        const float4 lv = *reinterpret_cast<const float4 *>(&sm->lv[ring][2 * c]);
        const float4 iv = *reinterpret_cast<const float4 *>(&sm->iv[ring][2 * c]);
        const float2 a0 = factors(cf, make_float2(ks.x, ks.y)), a1 = factors(cf, make_float2(ks.z, ks.w));
        tc_wait_ld();
        if (!whole) {
            hide(s0, lo - 32 * c, hi - 32 * c);
            hide(s1, lo - 32 * c - 32, hi - 32 * c - 32);
        }
        const float2 p0 = weights32(s0, w0, a0, make_float2(lv.x - ref, lv.y - ref));
        const float2 p1 = weights32(s1, w1, a1, make_float2(lv.z - ref, lv.w - ref));
        if (__any_sync(~0u, (p0.x + p0.y) + (p1.x + p1.y) > kMostSum)) break;
        sum += fmaf(p0.x, iv.x, p0.y * iv.y) + fmaf(p1.x, iv.z, p1.y * iv.w);
        tmem_st16(ts + 16 * c, w0);
        tmem_st16(ts + 16 * (c + 1), w1);
    }
    if (c < 4) grow_rows<D>(sm, c, ts, to, o_cols, ring, cf, top, sum, lo, hi);
}

// Which of 16 bytes are NaN codes, a bit each.
__device__ __forceinline__ uint32_t nan_bytes(uint4 v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t bits = 0;
#pragma unroll
    for (int k = 0; k < 4; k++)
        bits |= (((__vcmpeq4(w[k] & 0x7f7f7f7fu, 0x7f7f7f7fu) & 0x08040201u) * 0x01010101u) >> 24) << (4 * k);
    return bits;
}

// Which of a row's dimensions 32 c .. + 31 (at `values` within a line) meet a NaN value: its tokens s0 .. s1 - 1,
// of which those from `a` on are in units numbered from `unit` on, where the converting warps met one.  (Looked
// for in all of a long context, one NaN would hold its rows up for longer than the other warps wait.)
__device__ __forceinline__ uint32_t nan_dims(const AttnParams &p, const uint8_t *units, const int32_t *table, const uint8_t *values,
                                             int64_t line, uint32_t unit, int a, int s0, int s1) {
    uint32_t hit = 0;
#pragma unroll 1
    for (; a < s1 && hit != ~0u; a += kKeys, unit++) {
        if (!*static_cast<const volatile uint8_t *>(&units[unit & 1023])) continue;
#pragma unroll 1
        for (int g = a; g < a + kKeys; g += 16) {
            if (g + 16 <= s0 || g >= s1) continue;
            const int b = block_of(p, table, g);     // 16 tokens from a multiple of 16 on lie in one block
            if (b < 0) continue;
            const uint8_t *v = values + (static_cast<int64_t>(b) * p.bs + g % p.bs) * line;
            const int from = max(s0 - g, 0), to = min(s1 - g, 16);
#pragma unroll 2
            for (int k = from; k < to; k++) {
                const uint4 *at = reinterpret_cast<const uint4 *>(v + k * line);
                hit |= nan_bytes(__ldg(at)) | nan_bytes(__ldg(at + 1)) << 16;
            }
        }
    }
    return hit;
}

// ---- softmax warps: a thread per row ----------------------------------------------------------
template <int D>
__device__ void softmax_role(const AttnParams &p, Smem<D> *sm, Walk<D> &walk, int64_t total, int64_t ranges) {
    constexpr int kPart = kRows * (D + 2);
    const int m = threadIdx.x >> 7, row = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>((threadIdx.x >> 5) & 3) << 21;      // TMEM lane of the warp
    const uint32_t ts = sm->tmem + lanes + m * 128, to = sm->tmem + lanes + 256 + m * D;
    const bool fp16 = p.fp16 != 0;
    char *qs = sm->q[m];
    uint32_t unit = 0, s_phase = 0, o_phase = 0;
    int4 note = make_int4(-1, 0, 0, 0);
    Item x;
    while (walk.next(x)) {
        const int nu = x.ub - x.ua;
        if (m >= x.tiles) {
            unit += nu;
            continue;
        }
        const int rows = x.r.count * p.G, f = x.rt * kRows + m * 128 + row;
        const bool live = f < rows;
        const int j = f / p.G, hq = x.head * p.G + f - j * p.G;
        const int back = x.r.len - x.r.count;
        const int pos = live ? back + j : -1;
        // this row's query as f16, scaled by a power of two
        float cf;
        {
            const char *src = p.q + static_cast<int64_t>(x.r.start + j) * p.q_stride + 2 * static_cast<int64_t>(hq) * D;
            float largest = 0.f;
            if (live) {
#pragma unroll 4
                for (int c = 0; c < D / 8; c++) {
                    const uint4 y = __ldg(reinterpret_cast<const uint4 *>(src) + c);
                    const uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        const float2 z = widen2(w[k], fp16);
                        largest = fmaxf(largest, fmaxf(fabsf(z.x), fabsf(z.y)));
                    }
                }
            }
            const int e = row_exponent(largest);
            // a negative softmax scale moves into the query, so that a larger S is a larger x
            const float fq = p.scale_log2 < 0.f ? -power2(14 - e) : power2(14 - e);
            cf = fabsf(p.scale_log2) * power2(e - 14);
#pragma unroll 4
            for (int c = 0; c < D / 8; c++) {
                uint4 y = make_uint4(0, 0, 0, 0);
                if (live) y = __ldg(reinterpret_cast<const uint4 *>(src) + c);
                uint32_t w[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    const float2 z = widen2(w[k], fp16);
                    w[k] = pack_f16(z.x * fq, z.y * fq);
                }
                *reinterpret_cast<uint4 *>(qs + (c >> 3) * (128 * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4)) =
                    make_uint4(w[0], w[1], w[2], w[3]);
            }
        }
        fence_async_shared();
        mbar_arrive(&sm->q_full[m]);

        const int f0 = x.rt * kRows + m * 128, f1 = min(rows, f0 + 128) - 1;
        const int pos0 = back + f0 / p.G, pos1 = back + f1 / p.G;
        // a row past the tile's last sees nothing and needs no reference to be looked for
        float top = live ? -INFINITY : 0.f, sum = 0.f;
        bool ok = true;
        for (int t = 0; t < nu && ok; t++, unit++) {
            ok = wait(sm, &sm->s_full[m], s_phase);
            s_phase ^= 1;
            ok = __all_sync(~0u, ok);
            if (!ok) break;
            tc_fence_after();
            const int s0 = x.s.base + (x.ua + t) * kKeys, ring = unit & 3;
            const bool whole = s0 + kKeys - 1 <= pos0 && (p.window <= 0 || s0 > pos1 - p.window);
            const int hi = pos - s0;                                         // columns lo .. hi are visible
            const int lo = p.window > 0 && p.window <= pos ? pos - p.window + 1 - s0 : -0x40000000;
            // the first unit that shows a row anything sets its reference (no weight has been added before)
            if (__any_sync(~0u, top == -INFINITY)) {
                const float most = row_max<D>(sm, ts, ring, cf, lo, hi);
                if (top == -INFINITY) top = most == INFINITY ? NAN : ceilf(most);
            }
            row_weights<D>(sm, ts, to, t > 0 ? D : 0, ring, cf, top, sum, whole, lo, hi);
            tc_wait_st();
            tc_fence_before();
            mbar_arrive(&sm->p_full[m]);
        }
        if (!ok) return;
        ok = wait(sm, &sm->o_full[m], o_phase);
        o_phase ^= 1;
        if (!__all_sync(~0u, ok)) return;
        tc_fence_after();
        const bool nan = *static_cast<volatile int32_t *>(&sm->nan_seen) != 0;
        const bool full = x.ua == 0 && x.ub == x.s.units;
        const bool none = top == -INFINITY && sum == 0.f;
        const float inv = none ? 0.f : 1.f / sum;
        float *part = p.part + (2LL * blockIdx.x + (x.ua == 0)) * kPart;
        char *out = p.out + static_cast<int64_t>(x.r.start + j) * p.out_stride + 2 * static_cast<int64_t>(hq) * D;
#pragma unroll 1
        for (int c = 0; c < D / 32; c++) {
            // NaN codes were left out of the product: they go to the rows that see their token
            uint32_t hit = 0;
            if (nan && live)
                hit = nan_dims(p, sm->nan_units, x.table, p.vc + x.head * D + 32 * c, static_cast<int64_t>(p.Hkv) * D, unit - nu,
                               x.s.base + x.ua * kKeys, lo_of(p, pos), min(min(pos + 1, x.s.hi), x.s.base + x.ub * kKeys));
            __syncwarp();
            uint32_t o[32];
            tmem_ld32(o, to + 32 * c);
            tc_wait_ld();
            if (nan) {
#pragma unroll
                for (int k = 0; k < 32; k++)
                    if ((hit >> k) & 1) o[k] = 0x7fffffffu;
            }
            if (full && live) {
                uint32_t y[16];
#pragma unroll
                for (int k = 0; k < 16; k++)
                    y[k] = none ? 0u : pack_out(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv, fp16);
#pragma unroll
                for (int k = 0; k < 4; k++)
                    *reinterpret_cast<uint4 *>(out + 64 * c + 16 * k) = make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
            } else if (live) {
                float *at = part + 2 * kRows + (m * 128 + row) * D + 32 * c;
#pragma unroll
                for (int k = 0; k < 8; k++)
                    *reinterpret_cast<uint4 *>(at + 4 * k) = make_uint4(o[4 * k], o[4 * k + 1], o[4 * k + 2], o[4 * k + 3]);
            }
            __syncwarp();
        }
        if (live) {
            if (full) {
                if (p.lse)
                    p.lse[static_cast<int64_t>(x.r.start + j) * p.Hkv * p.G + hq] = none ? -INFINITY : (top + log2f(sum)) * kLn2;
            } else {
                part[m * 128 + row] = top;
                part[kRows + m * 128 + row] = sum;
            }
        }
        if (!full && x.ua == 0) {
            const int64_t last = ((x.tile + x.s.units) * ranges - 1) / total;
            note = make_int4(x.i, x.rt, static_cast<int>(last - blockIdx.x) + 1, x.head);
        }
        tc_fence_before();
    }
    if (m == 0 && row == 0) p.meta[blockIdx.x] = note;
}

// ---- converting warps: codes to f16 operand tiles ---------------------------------------------
// What a unit's copies need: for the 16-token group (lane & 7), where its codes begin (-1: not
// read) and its scales; klo, khi: the unit's tokens that some row sees.
struct Feed {
    int64_t at;
    int klo, khi;
    float ks, vs;
};

template <int D>
__device__ void convert_role(const AttnParams &p, Smem<D> *sm, Walk<D> &walk) {
    constexpr int kC = D / 16;                       // 16-byte pieces of a token's codes
    constexpr int kTok = 32 * kConvWarps / kC;       // tokens per round of the threads, a multiple of 16
    constexpr int kRounds = kKeys / kTok, kStep = kRounds < 4 ? kRounds : 4, kRaw = 32 * kConvWarps * 16;
    const int i = threadIdx.x - 32 * kSoftWarps, lane = i & 31;
    const int c = i % kC, tok = i / kC;              // this thread's piece, and its token within a round
    const int64_t line = static_cast<int64_t>(p.Hkv) * D;
    const int64_t mine = (tok & 15) * line + 16 * c; // this thread's place within a group of 16 tokens
    // places of the two halves of 16 converted codes; threads of the upper 64 dimensions write
    // their second half first, so that eight neighbours write to eight bank groups
    const int second = (c >> 2) & 1;
    const uint32_t row = (c >> 2) * (kKeys * 128) + tok * 128;
    const uint32_t to0 = row + ((((c & 3) * 2 + second) ^ (tok & 7)) << 4);
    const uint32_t to1 = row + ((((c & 3) * 2 + (second ^ 1)) ^ (tok & 7)) << 4);

    Item x;
    int t = 0;
    bool more = walk.next(x);
    if (!more) return;
    t = x.ua;
    // a block id that has been asked for but not yet looked at
    int32_t id = -1;
    auto ask = [&]() {
        const int s = x.s.base + t * kKeys + 16 * (lane & 7);
        id = -1;
        if (s < x.s.hi && s + 16 > x.s.lo) id = p.table_at(x.table, s);
    };
    auto resolve = [&]() {
        Feed f;
        const int s = x.s.base + t * kKeys + 16 * (lane & 7);
        if (id >= p.num_blocks) {
            if (p.err) atomicOr(p.err, PKV_DEVERR_BLOCK);
            id = -1;
        }
        f.at = -1;
        f.ks = 0.f;
        f.vs = -1.f;                                 // no block
        if (id >= 0) {
            f.at = (static_cast<int64_t>(id) * p.bs + s % p.bs) * line + x.head * D;
            if (i < kSub) {
                f.ks = p.ks[static_cast<int64_t>(id) * p.Hkv + x.head];
                f.vs = p.vs[static_cast<int64_t>(id) * p.Hkv + x.head];
            }
        }
        f.klo = x.s.lo - x.s.base - t * kKeys;
        f.khi = x.s.hi - x.s.base - t * kKeys;
        return f;
    };
    auto advance = [&]() {
        t++;
        if (t == x.ub) {
            more = walk.next(x);
            t = x.ua;
        }
        if (more) ask();
    };
    // Each thread copies its own 16-byte pieces and reads only those back: no barrier.
    auto fetch = [&](const uint8_t *cache, const Feed &f, int r, char *raw) {
        const int k = r * kTok + tok;
        const int64_t from = __shfl_sync(~0u, f.at, k >> 4);
        const bool live = from >= 0 && k >= f.klo && k < f.khi;
        cp_async<16>(smem_addr(raw + r * kRaw + i * 16), cache + (live ? from + mine : 0), live);
    };
    // Turn a half (keys or values) of unit `a` into f16, and refill its pieces with the next unit's.
    auto half = [&](const uint8_t *cache, char *raw, char *dst, const Feed &b, bool next, bool values, uint32_t unit) {
        bool nan = false;
#pragma unroll 1
        for (int r0 = 0; r0 < kRounds; r0 += kStep) {
            uint4 y[kStep];
#pragma unroll
            for (int r = 0; r < kStep; r++) y[r] = *reinterpret_cast<const uint4 *>(raw + (r0 + r) * kRaw + i * 16);
            if (values) {
                // 0x7f + 1 carries into the sign bit of its byte: NaN codes leave the product (the
                // softmax warps bring them back for the rows that see their token)
                uint32_t hit = 0;
#pragma unroll
                for (int r = 0; r < kStep; r++)
                    hit |= ((y[r].x & 0x7f7f7f7fu) + 0x01010101u) | ((y[r].y & 0x7f7f7f7fu) + 0x01010101u) |
                           ((y[r].z & 0x7f7f7f7fu) + 0x01010101u) | ((y[r].w & 0x7f7f7f7fu) + 0x01010101u);
                if (hit & 0x80808080u) {
#pragma unroll
                    for (int r = 0; r < kStep; r++) {
                        y[r].x &= ~__vcmpeq4(y[r].x & 0x7f7f7f7fu, 0x7f7f7f7fu);
                        y[r].y &= ~__vcmpeq4(y[r].y & 0x7f7f7f7fu, 0x7f7f7f7fu);
                        y[r].z &= ~__vcmpeq4(y[r].z & 0x7f7f7f7fu, 0x7f7f7f7fu);
                        y[r].w &= ~__vcmpeq4(y[r].w & 0x7f7f7f7fu, 0x7f7f7f7fu);
                    }
                    nan = true;
                }
            }
#pragma unroll
            for (int r = 0; r < kStep; r++) {
                // the half that goes first (see to0)
                const uint32_t w0 = second ? y[r].z : y[r].x, w1 = second ? y[r].w : y[r].y;
                const uint32_t w2 = second ? y[r].x : y[r].z, w3 = second ? y[r].y : y[r].w;
                *reinterpret_cast<uint4 *>(dst + to0 + (r0 + r) * kTok * 128) =
                    make_uint4(f16x2_of(w0), f16x2_of(w0 >> 16), f16x2_of(w1), f16x2_of(w1 >> 16));
                *reinterpret_cast<uint4 *>(dst + to1 + (r0 + r) * kTok * 128) =
                    make_uint4(f16x2_of(w2), f16x2_of(w2 >> 16), f16x2_of(w3), f16x2_of(w3 >> 16));
            }
            if (next)
#pragma unroll
                for (int r = 0; r < kStep; r++) fetch(cache, b, r0 + r, raw);
        }
        if (nan) {
            *static_cast<volatile uint8_t *>(&sm->nan_units[unit & 1023]) = 1;
            *static_cast<volatile int32_t *>(&sm->nan_seen) = 1;
        }
        cp_commit();
    };

    ask();
    Feed a = resolve();
#pragma unroll 1
    for (int r = 0; r < kRounds; r++) fetch(p.kc, a, r, sm->raw[0]);
    cp_commit();
#pragma unroll 1
    for (int r = 0; r < kRounds; r++) fetch(p.vc, a, r, sm->raw[1]);
    cp_commit();
    advance();
    bool ok = true, now = true;
    for (uint32_t unit = 0; now; unit++) {
        const bool next = more;
        Feed b = {};
        if (next) {
            b = resolve();
            advance();                               // the block ids of the unit after it are on their way
        }
        const int stage = unit & 1;
        const uint32_t parity = ((unit >> 1) & 1) ^ 1;
        cp_wait<1>();
        ok = wait(sm, &sm->k_free[stage], parity);
        if (!__all_sync(~0u, ok)) break;
        if (i < kSub) {
            const int ring = unit & 3;
            const bool named = a.at >= 0;
            const float v = value_scale(a.vs);
            sm->ks[ring][i] = named ? a.ks : 0.f;
            sm->lv[ring][i] = named ? __log2f(v) : -INFINITY;
            sm->iv[ring][i] = named ? __frcp_rn(v) : 0.f;
        }
        half(p.kc, sm->raw[0], sm->k[stage], b, next, false, unit);
        fence_async_shared();
        mbar_arrive(&sm->k_full[stage]);
        cp_wait<1>();
        ok = wait(sm, &sm->v_free[stage], parity);
        if (!__all_sync(~0u, ok)) break;
        half(p.vc, sm->raw[1], sm->v[stage], b, next, true, unit);
        fence_async_shared();
        mbar_arrive(&sm->v_full[stage]);
        a = b;
        now = next;
    }
    cp_wait<0>();
}

// ---- issuing warp ------------------------------------------------------------------------------
// The whole warp walks the units, so that addresses and descriptors stay in uniform registers; one
// lane issues.
template <int D>
__device__ void issue_role(Smem<D> *sm, Walk<D> &walk) {
    constexpr uint32_t kQk = f16_idesc(128, kKeys, false), kPv = f16_idesc(128, D, true);
    const uint32_t tmem = __shfl_sync(~0u, sm->tmem, 0);
    uint32_t unit = 0, q_phase[2] = {0, 0}, p_phase[2] = {0, 0};
    const bool leader = elect_one();
    Item x;
    bool ok = true;
    auto all = [&](uint64_t *bar, uint32_t parity) { return __all_sync(~0u, wait(sm, bar, parity)) != 0; };
    auto qk = [&](int m, int stage) {
        const uint64_t da = smem_desc(smem_addr(sm->q[m]), 16), db = smem_desc(smem_addr(sm->k[stage]), 16);
        if (leader) {
#pragma unroll
            for (int k = 0; k < D / 16; k++) {
                constexpr int kPanel = 128 * 128;
                const uint64_t off = ((k >> 2) * kPanel + (k & 3) * 32) >> 4;
                mma_ss(tmem + m * 128, da + off, db + off, kQk, k > 0);
            }
            mbar_arrive(&sm->s_full[m]);
            tc_commit(&sm->s_full[m]);
        }
        __syncwarp();
    };
    auto pv = [&](int m, int stage, bool add) {
        const uint64_t db = smem_desc(smem_addr(sm->v[stage]), kKeys * 128);
        if (leader) {
#pragma unroll
            for (int k = 0; k < kKeys / 16; k++)
                mma_ts(tmem + 256 + m * D, tmem + m * 128 + 8 * k, db + k * (2048 >> 4), kPv, add || k > 0);
        }
        __syncwarp();
    };
    auto commit = [&](uint64_t *bar) {
        if (leader) tc_commit(bar);
        __syncwarp();
    };
    while (ok && walk.next(x)) {
        const int nu = __shfl_sync(~0u, x.ub - x.ua, 0), tiles = __shfl_sync(~0u, x.tiles, 0);
        for (int m = 0; m < tiles && ok; m++) {
            ok = all(&sm->q_full[m], q_phase[m]);
            q_phase[m] ^= 1;
        }
        ok = ok && all(&sm->k_full[unit & 1], (unit >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        for (int m = 0; m < tiles; m++) qk(m, unit & 1);
        commit(&sm->k_free[unit & 1]);
        for (int t = 0; t < nu && ok; t++, unit++) {
            const int stage = unit & 1, next = stage ^ 1;
            for (int m = 0; m < tiles && ok; m++) {
                if (m == 0) {
                    // the operands are usually there before the weights are: off the weights' path
                    ok = all(&sm->v_full[stage], (unit >> 1) & 1) && (t + 1 == nu || all(&sm->k_full[next], ((unit + 1) >> 1) & 1));
                }
                ok = ok && all(&sm->p_full[m], p_phase[m]);
                p_phase[m] ^= 1;
                if (!ok) break;
                tc_fence_after();
                pv(m, stage, t > 0);
                if (t + 1 < nu) {
                    qk(m, next);
                } else {
                    commit(&sm->o_full[m]);
                }
            }
            if (!ok) break;
            commit(&sm->v_free[stage]);
            if (t + 1 < nu) commit(&sm->k_free[next]);
        }
    }
    // the products end before the TMEM is freed
    commit(&sm->done);
    for (uint32_t k = 0; k < kTries; k++)
        if (mbar_try(&sm->done, 0)) break;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1) kv8_prefill_kernel(const AttnParams p) {
    extern __shared__ char s_raw[];
    // the swizzle goes by address bits: the operand tiles start on 1024 bytes
    Smem<D> *sm = reinterpret_cast<Smem<D> *>(s_raw + (-smem_addr(s_raw) & 1023u));
    const int warp = threadIdx.x >> 5;
    if (warp == 0) tmem_alloc(&sm->tmem, 512);
    if (threadIdx.x == 32) {
        for (int k = 0; k < 2; k++) {
            mbar_init(&sm->q_full[k], 128);
            mbar_init(&sm->k_full[k], 32 * kConvWarps);
            mbar_init(&sm->v_full[k], 32 * kConvWarps);
            mbar_init(&sm->k_free[k], 1);
            mbar_init(&sm->v_free[k], 1);
            mbar_init(&sm->s_full[k], 2);
            mbar_init(&sm->p_full[k], 128);
            mbar_init(&sm->o_full[k], 1);
        }
        mbar_init(&sm->done, 1);
        sm->failed = 0;
        sm->nan_seen = 0;
        fence_mbar_init();
    }
    for (int k = threadIdx.x; k < 1024; k += kThreads) sm->nan_units[k] = 0;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();
    pdl_trigger();
    int64_t *prefix = reinterpret_cast<int64_t *>(sm->raw);
    const int64_t total = plan_prefix<kThreads>(prefix, prefix + kThreads + 1, p.n, [&](int i) {
        return units_of_request(p, request_of(p, i, blockIdx.x == 0));
    });
    const int64_t ranges = total < gridDim.x ? total : gridDim.x;
    if (blockIdx.x < ranges) {
        Walk<D> walk(p, prefix, blockIdx.x * total / ranges, (blockIdx.x + 1) * total / ranges);
        __syncthreads();                             // the sums' place is the converting warps' from here on
        if (warp < kSoftWarps) {
            more_registers<kSoftRegs>();
            softmax_role<D>(p, sm, walk, total, ranges);
        } else if (warp < kSoftWarps + kConvWarps) {
            fewer_registers<kConvRegs>();
            convert_role<D>(p, sm, walk);
        } else {
            fewer_registers<kIssueRegs>();
            if (warp == kSoftWarps + kConvWarps) issue_role<D>(sm, walk);
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

template <int D>
int launch(const AttnParams &p, int sms, cudaStream_t s) {
    constexpr size_t smem = sizeof(Smem<D>) + 1024;
    static_assert(smem <= 227 * 1024, "shared memory");
    static bool set[64] = {false};
    const int rc = kv8_allow_smem(reinterpret_cast<const void *>(kv8_prefill_kernel<D>), static_cast<int>(smem), set);
    if (rc != PKV_OK) return rc;
    PKV_CUDA_TRY(launch_pdl(kv8_prefill_kernel<D>, dim3(sms), dim3(kThreads), smem, s, p));
    return kv8_launch_merge(p, D, kRows, sms, 1, s);
}

}  // namespace

int64_t kv8_prefill_workspace(int32_t head_dim, int sms) {
    return head_dim > 128 ? 0 : static_cast<int64_t>(sms) * (2LL * kRows * (head_dim + 2) * 4 + 16);
}

int kv8_launch_prefill(const AttnParams &p, int32_t head_dim, int sms, cudaStream_t s) {
    return head_dim == 64 ? launch<64>(p, sms, s) : launch<128>(p, sms, s);
}

}  // namespace pkv
