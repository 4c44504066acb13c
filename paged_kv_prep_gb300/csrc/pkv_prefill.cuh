// The walk over the units of requests with many query rows, shared by the prefill
// kernels: a unit is 128 tokens for one KV head and a row tile of 256 (query, head) rows.
#pragma once

#include "pkv_kv8_attention.cuh"
#include "pkv_tcgen05.cuh"

namespace pkv {

constexpr int kRows = 256;              // rows of a CTA, two tiles of 128
constexpr int kKeys = 128;              // tokens per unit
constexpr int kSub = kKeys / 16;
constexpr int kSoftWarps = 8, kConvWarps = 4;
constexpr int kThreads = 32 * (kSoftWarps + kConvWarps + 4);   // and a warpgroup whose first warp issues
constexpr uint32_t kTries = 1u << 22;   // polls before a wait gives up (half a second or more)

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

// A wait with a limit; `sm` is the CTA's shared memory, whose `failed` ends every other wait too.
template <typename Smem>
__device__ __forceinline__ bool wait(Smem *sm, uint64_t *bar, uint32_t parity) {
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

// 2^d of an integer d <= 0 (0 below 2^-126, and of -inf).
__device__ __forceinline__ float power2_down(float d) {
    return d >= -126.f ? __uint_as_float(static_cast<uint32_t>(static_cast<int>(d) + 127) << 23) : d < 0.f ? 0.f : d;
}

}  // namespace pkv
