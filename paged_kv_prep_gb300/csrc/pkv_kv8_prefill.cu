// Attention over the 8-bit paged cache for requests with many query rows
// (prompt chunks), on the tensor cores.
//
// Mathematics: as in pkv_kv8_decode.cu.  x = S * a_b + lv_b with S = q . code_k
// from the tensor core, a_b = k_scale * softmax_scale * log2(e) and lv_b =
// log2(v_scale), both constant over 16 tokens; w = 2^(x - R) goes into the
// second product as f16, the softmax sum adds w / v_scale in fp32.  R follows
// the running maximum lazily: it moves only when a row's maximum has grown by
// more than 2^8, so that the accumulator is rarely rescaled and w stays below
// 2^8, far inside f16's range.
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
constexpr int kThreads = 32 * (kSoftWarps + kConvWarps + 1);
constexpr uint32_t kTries = 1u << 19;   // polls of about a microsecond before a wait gives up
constexpr float kSlack = 8.f;           // growth of a row's maximum (log2) that R does not follow

template <int D>
struct Smem {
    char q[2][128 * D * 2];
    char k[2][kKeys * D * 2];
    char v[2][kKeys * D * 2];
    float ks[4][kSub], lv[4][kSub], iv[4][kSub];   // per 16 tokens: k_scale, log2(v_scale), 1 / v_scale
    uint64_t q_full[2], k_full[2], v_full[2], k_free[2], v_free[2], s_full[2], p_full[2], o_full[2], done;
    int64_t prefix[kThreads + 1];
    int64_t warp_sum[kThreads / 32];
    uint32_t tmem;
    int32_t failed;
    int32_t nan_seen;                   // this CTA has met a V code that is NaN
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

    __device__ __forceinline__ Walk(const AttnParams &p_, const Smem<D> &sm, int64_t u0, int64_t u1) : p(p_), u(u0), end(u1) {
        i = plan_find<kThreads>(sm.prefix, p.n, u, [&](int k) { return units_of_request(p, request_of(p, k)); }, &first);
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
    volatile int32_t *failed = &sm->failed;
    for (uint32_t k = 0; k < kTries; k++) {
        if (mbar_wait(bar, parity, 1)) return true;
        if (*failed) return false;
    }
    *failed = 1;
    return false;
}

// ---- softmax warps: a thread per row ----------------------------------------------------------
template <int D>
__device__ void softmax_role(const AttnParams &p, Smem<D> *sm, int64_t u0, int64_t u1, int64_t total, int64_t ranges) {
    constexpr int kPart = kRows * (D + 2);
    const int m = threadIdx.x >> 7, row = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>((threadIdx.x >> 5) & 3) << 21;      // TMEM lane of the warp
    const uint32_t ts = sm->tmem + lanes + m * 128, to = sm->tmem + lanes + 256 + m * D;
    const bool fp16 = p.fp16 != 0;
    char *qs = sm->q[m];
    uint32_t unit = 0, s_phase = 0, o_phase = 0;
    int4 note = make_int4(-1, 0, 0, 0);
    Walk<D> walk(p, *sm, u0, u1);
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
        float top = -INFINITY, sum = 0.f;
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
            const int lo = p.window > 0 ? pos - p.window + 1 - s0 : -0x7fffffff;
            float most = -INFINITY;
#pragma unroll
            for (int c = 0; c < 4; c++) {
                uint32_t s[32];
                tmem_ld32(s, ts + 32 * c);
                tc_wait_ld();
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    float mx = -INFINITY;
                    if (whole) {
#pragma unroll
                        for (int k = 0; k < 16; k++) mx = fmaxf(mx, __uint_as_float(s[16 * h + k]));
                    } else {
#pragma unroll
                        for (int k = 0; k < 16; k++) {
                            const int col = 32 * c + 16 * h + k;
                            mx = fmaxf(mx, col <= hi && col >= lo ? __uint_as_float(s[16 * h + k]) : -INFINITY);
                        }
                    }
                    const float a = cf * sm->ks[ring][2 * c + h], lv = sm->lv[ring][2 * c + h];
                    most = fmaxf(most, mx == -INFINITY ? -INFINITY : fmaf(mx, a, lv));
                }
            }
            const bool grow = most > top + kSlack || (top == -INFINITY && most > -INFINITY);
            if (__any_sync(~0u, grow)) {
                const float f2 = grow ? exp2_fast(top - most) : 1.f;
                if (grow) top = most;
                sum *= f2;
                if (t > 0) {
#pragma unroll
                    for (int c = 0; c < D / 32; c++) {
                        uint32_t o[32];
                        tmem_ld32(o, to + 32 * c);
                        tc_wait_ld();
#pragma unroll
                        for (int k = 0; k < 32; k++) o[k] = __float_as_uint(__uint_as_float(o[k]) * f2);
                        tmem_st32(to + 32 * c, o);
                    }
                }
            }
            const float ref = top == -INFINITY ? 0.f : top;
#pragma unroll
            for (int c = 0; c < 4; c++) {
                uint32_t s[32], w[16];
                tmem_ld32(s, ts + 32 * c);
                tc_wait_ld();
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const float a = cf * sm->ks[ring][2 * c + h], b = sm->lv[ring][2 * c + h] - ref;
                    float part = 0.f;
#pragma unroll
                    for (int k = 0; k < 16; k += 2) {
                        float y0 = exp2_fast(fmaf(__uint_as_float(s[16 * h + k]), a, b));
                        float y1 = exp2_fast(fmaf(__uint_as_float(s[16 * h + k + 1]), a, b));
                        if (!whole) {
                            const int col = 32 * c + 16 * h + k;
                            y0 = col <= hi && col >= lo ? y0 : 0.f;
                            y1 = col + 1 <= hi && col + 1 >= lo ? y1 : 0.f;
                        }
                        part += y0 + y1;
                        w[8 * h + k / 2] = pack_f16(y0, y1);
                    }
                    sum = fmaf(part, sm->iv[ring][2 * c + h], sum);
                }
                tmem_st16(ts + 16 * c, w);
            }
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
            uint32_t o[32];
            tmem_ld32(o, to + 32 * c);
            tc_wait_ld();
            if (nan && live) {
                // NaN codes were left out of the product: they go to the rows that see their token
                uint32_t hit = 0;
                const int s1 = min(min(pos + 1, x.s.hi), x.s.base + x.ub * kKeys);
                for (int s = max(max(lo_of(p, pos), x.s.lo), x.s.base + x.ua * kKeys); s < s1; s++) {
                    const int b = block_of(p, x.table, s);
                    if (b < 0) continue;
                    const uint8_t *v = p.vc + ((static_cast<int64_t>(b) * p.bs + s % p.bs) * p.Hkv + x.head) * D + 32 * c;
                    for (int k = 0; k < 32; k++) hit |= ((v[k] & 127) == 127 ? 1u : 0u) << k;
                }
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
template <int D>
__device__ void convert_role(const AttnParams &p, Smem<D> *sm, int64_t u0, int64_t u1) {
    constexpr int kC = D / 16;                       // 16-byte pieces of a token's codes
    constexpr int kTok = 128 / kC;                   // tokens per round of the 128 threads
    constexpr int kRounds = kKeys / kTok;
    const int i = threadIdx.x - 32 * kSoftWarps, lane = i & 31;
    const int c = i % kC, tok = i / kC;              // this thread's piece, and its token within a round
    const int64_t line = static_cast<int64_t>(p.Hkv) * D;

    Walk<D> walk(p, *sm, u0, u1);
    Item x;
    bool more = walk.next(x);
    int t = x.ua;
    // block id of 16-token group (lane & 7) of unit t, -1 where no row of the item sees it
    auto groups = [&]() {
        const int s = x.s.base + t * kKeys + 16 * (lane & 7);
        return s < x.s.hi && s + 16 > x.s.lo ? block_of(p, x.table, s) : -1;
    };
    auto load = [&](uint4 (&y)[kRounds], const uint8_t *cache, int blocks, const Item &it, int tu) {
#pragma unroll
        for (int r = 0; r < kRounds; r++) {
            const int k = r * kTok + tok;            // token of the unit
            const int b = __shfl_sync(~0u, blocks, k >> 4);
            const int s = it.s.base + tu * kKeys + k;
            y[r] = make_uint4(0, 0, 0, 0);
            if (b >= 0 && s >= it.s.lo && s < it.s.hi)
                y[r] = __ldg(reinterpret_cast<const uint4 *>(cache + (static_cast<int64_t>(b) * p.bs + s % p.bs) * line +
                                                             it.head * D + 16 * c));
        }
    };
    auto lay = [&](const uint4 (&y)[kRounds], char *dst) {
#pragma unroll
        for (int r = 0; r < kRounds; r++) {
            const int k = r * kTok + tok;
            const uint32_t w[4] = {y[r].x, y[r].y, y[r].z, y[r].w};
            uint4 h[2];
            h[0] = make_uint4(f16x2_of(w[0]), f16x2_of(w[0] >> 16), f16x2_of(w[1]), f16x2_of(w[1] >> 16));
            h[1] = make_uint4(f16x2_of(w[2]), f16x2_of(w[2] >> 16), f16x2_of(w[3]), f16x2_of(w[3] >> 16));
            char *panel = dst + (c >> 2) * (kKeys * 128) + k * 128;
            // the upper panel's threads write their second half first: eight neighbours, eight bank groups
            const int first = (c >> 2) & 1;
#pragma unroll
            for (int g = 0; g < 2; g++) {
                const int half = g ^ first;
                *reinterpret_cast<uint4 *>(panel + ((((c & 3) * 2 + half) ^ (k & 7)) << 4)) = half ? h[1] : h[0];
            }
        }
    };
    if (!more) return;
    uint4 kreg[kRounds], vreg[kRounds];
    int blocks = groups();
    load(kreg, p.kc, blocks, x, t);
    uint32_t unit = 0;
    bool ok = true;
    while (more && ok) {
        load(vreg, p.vc, blocks, x, t);
        const int stage = unit & 1;
        const uint32_t parity = ((unit >> 1) & 1) ^ 1;
        ok = wait(sm, &sm->k_free[stage], parity);
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        if (i < kSub) {
            // i == lane & 7 here: this thread knows the group's block
            const int64_t at = static_cast<int64_t>(blocks) * p.Hkv + x.head;
            const int ring = unit & 3;
            float k = 0.f, lv = -INFINITY, iv = 0.f;
            if (blocks >= 0) {
                k = p.ks[at];
                const float v = value_scale(p.vs[at]);
                lv = __log2f(v);
                iv = __frcp_rn(v);
            }
            sm->ks[ring][i] = k;
            sm->lv[ring][i] = lv;
            sm->iv[ring][i] = iv;
        }
        lay(kreg, sm->k[stage]);
        fence_async_shared();
        mbar_arrive(&sm->k_full[stage]);
        // the next unit's keys are on their way while this unit's values are laid out
        t++;
        const bool last = t == x.ub;
        if (last) {
            more = walk.next(x);
            t = x.ua;
        }
        if (more) {
            blocks = groups();
            load(kreg, p.kc, blocks, x, t);
        }
        ok = wait(sm, &sm->v_free[stage], parity);
        ok = __all_sync(~0u, ok);
        if (!ok) break;
        {
            bool nan = false;
#pragma unroll
            for (int r = 0; r < kRounds; r++) {
                uint32_t *w = reinterpret_cast<uint32_t *>(&vreg[r]);
#pragma unroll
                for (int k = 0; k < 4; k++) {
                    // 0x7f + 1 carries into the sign bit of its byte
                    if ((((w[k] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0) {
                        w[k] &= ~__vcmpeq4(w[k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                        nan = true;
                    }
                }
            }
            if (nan) *static_cast<volatile int32_t *>(&sm->nan_seen) = 1;
        }
        lay(vreg, sm->v[stage]);
        fence_async_shared();
        mbar_arrive(&sm->v_full[stage]);
        unit++;
    }
}

// ---- issuing thread ----------------------------------------------------------------------------
template <int D>
__device__ void issue_role(const AttnParams &p, Smem<D> *sm, int64_t u0, int64_t u1) {
    constexpr uint32_t kQk = f16_idesc(128, kKeys, false), kPv = f16_idesc(128, D, true);
    const uint32_t tmem = sm->tmem;
    uint32_t unit = 0, q_phase[2] = {0, 0}, p_phase[2] = {0, 0};
    Walk<D> walk(p, *sm, u0, u1);
    Item x;
    bool ok = true;
    auto qk = [&](int m, int stage) {
        const uint32_t a = smem_addr(sm->q[m]), b = smem_addr(sm->k[stage]);
#pragma unroll
        for (int k = 0; k < D / 16; k++) {
            const uint32_t off = (k >> 2) * (128 * 128) + (k & 3) * 32;
            mma_ss(tmem + m * 128, smem_desc(a + off, 16), smem_desc(b + off, 16), kQk, k > 0);
        }
        mbar_arrive(&sm->s_full[m]);
        tc_commit(&sm->s_full[m]);
    };
    auto pv = [&](int m, int stage, bool add) {
        const uint32_t b = smem_addr(sm->v[stage]);
#pragma unroll
        for (int k = 0; k < kKeys / 16; k++)
            mma_ts(tmem + 256 + m * D, tmem + m * 128 + 8 * k, smem_desc(b + k * 2048, kKeys * 128), kPv, add || k > 0);
    };
    while (ok && walk.next(x)) {
        const int nu = x.ub - x.ua;
        for (int m = 0; m < x.tiles && ok; m++) {
            ok = wait(sm, &sm->q_full[m], q_phase[m]);
            q_phase[m] ^= 1;
        }
        ok = ok && wait(sm, &sm->k_full[unit & 1], (unit >> 1) & 1);
        if (!ok) break;
        tc_fence_after();
        for (int m = 0; m < x.tiles; m++) qk(m, unit & 1);
        tc_commit(&sm->k_free[unit & 1]);
        for (int t = 0; t < nu && ok; t++, unit++) {
            const int stage = unit & 1, next = (unit + 1) & 1;
            for (int m = 0; m < x.tiles && ok; m++) {
                if (m == 0) ok = wait(sm, &sm->v_full[stage], (unit >> 1) & 1);
                ok = ok && wait(sm, &sm->p_full[m], p_phase[m]);
                p_phase[m] ^= 1;
                if (!ok) break;
                tc_fence_after();
                pv(m, stage, t > 0);
                if (t + 1 < nu) {
                    if (m == 0) {
                        ok = wait(sm, &sm->k_full[next], ((unit + 1) >> 1) & 1);
                        if (!ok) break;
                        tc_fence_after();
                    }
                    qk(m, next);
                } else {
                    tc_commit(&sm->o_full[m]);
                }
            }
            if (!ok) break;
            tc_commit(&sm->v_free[stage]);
            if (t + 1 < nu) tc_commit(&sm->k_free[next]);
        }
    }
    // the products end before the TMEM is freed
    tc_commit(&sm->done);
    for (uint32_t k = 0; k < kTries; k++)
        if (mbar_wait(&sm->done, 0, 1)) break;
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
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_wait();
    pdl_trigger();
    const int64_t total = plan_prefix<kThreads>(sm->prefix, sm->warp_sum, p.n, [&](int i) {
        return units_of_request(p, request_of(p, i, blockIdx.x == 0));
    });
    const int64_t ranges = total < gridDim.x ? total : gridDim.x;
    const int64_t u0 = ranges ? blockIdx.x * total / ranges : 0, u1 = ranges ? (blockIdx.x + 1) * total / ranges : 0;
    if (blockIdx.x < ranges) {
        if (warp < kSoftWarps)
            softmax_role<D>(p, sm, u0, u1, total, ranges);
        else if (warp < kSoftWarps + kConvWarps)
            convert_role<D>(p, sm, u0, u1);
        else if ((threadIdx.x & 31) == 0)
            issue_role<D>(p, sm, u0, u1);
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
    PKV_CUDA_TRY(cudaFuncSetAttribute(kv8_prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      static_cast<int>(smem)));
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
