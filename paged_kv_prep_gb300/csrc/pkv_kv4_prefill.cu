// Attention over the 4-bit paged cache for requests with many query rows
// (prompt chunks), on the tensor cores.
//
// Mathematics: as in pkv_kv4_decode.cu.  S = q . k comes from the tensor core with keys that
// carry their scales, so x = S * a - R with one a per row; w = 2^(x - R) goes into the second
// product as f16, the softmax sum adds it in fp32.  R is 9 below the row's maximum over its first
// unit, rounded up to an integer, and then follows lazily: it moves only when the sum of 64 w,
// which is needed anyway, exceeds 2^15, and by a whole power of two, so that
// weights which are f16 already are not rounded again (unless they turn subnormal).
// w is off by 2^-11 of itself, or by 2^-25 where it is below 2^-14: 2^-33 of the largest weight, at
// most 2^-11 of the output (nonzero values are less than 2^22 apart).
//
// Bound: the tensor pipe (4 D flops per visible pair); beside it per tile of
// 256 rows x 128 tokens 32768 exponentials and 32768 codes turned into f16 and scaled.
//
// Layout.  A CTA holds 256 (query, head) rows of one KV head in two tiles of
// 128.  Warps 0-3 and 4-7 do the softmax of one tile each, a thread per row;
// warps 8-11 read the codes of 128 tokens, turn them into f16 times their scales (exact) and
// lay them out for the tensor core, so one conversion serves both tiles; warp 12
// issues the products: S = Q K^T (both in shared memory), O += P V with P in
// TMEM in the place of S.  While one tile's softmax runs, the tensor core
// works on the other.  The batch's (row tile, KV head, 128 tokens) units are
// split evenly over the CTAs; a row tile that is cut leaves partial results
// for a merge in a fixed order.
//
// Every wait has a limit; one that runs out sets PKV_DEVERR_TIMEOUT, the other
// waits give up after it, and the CTA drains its products and frees its TMEM.
#include "pkv_kv4_attention.cuh"
#include "pkv_prefill.cuh"

namespace pkv {
namespace {

// Registers a thread: launched with 128; 256 x 176 + 128 x 104 + 128 x 56 = 512 x 128.
constexpr int kSoftRegs = 176, kConvRegs = 104, kIssueRegs = 56;
static_assert(32 * (kSoftWarps * kSoftRegs + kConvWarps * kConvRegs + 4 * kIssueRegs) <= 65536, "registers");
static_assert((kThreads + 1 + kThreads / 32) * 8 <= 2 * kKeys * 32, "the plan's sums lie in the raw codes' place");
constexpr float kHead = 9.f;            // how far below a row's maximum (log2) R is set
constexpr float kMostSum = 32768.f;     // sum of 64 w that makes it move
constexpr float kHuge = 0x1p20f;        // a reference from which on a logit's rounding may count

template <int D>
struct Smem {
    char q[2][128 * D * 2];
    char k[2][kKeys * D * 2];
    char v[2][kKeys * D * 2];
    char raw[2][kKeys * D / 2];         // codes of the unit that is converted next: keys, values
    uint64_t q_full[2], k_full[2], v_full[2], k_free[2], v_free[2], s_full[2], p_full[2], o_full[2], done;
    uint32_t named[4];                  // which groups of 16 of a unit's tokens lie in a block, a bit each
    uint32_t tmem;
    int32_t failed;
};

// Scores of 32 columns, of which groups 2 c, 2 c + 1 may have no block.
__device__ __forceinline__ void hide_unnamed(uint32_t (&s)[32], uint32_t two) {
#pragma unroll
    for (int h = 0; h < 2; h++)
        if (!((two >> h) & 1)) {
#pragma unroll
            for (int k = 0; k < 16; k++) s[16 * h + k] = 0xff800000u;
        }
}

// What a row sees of a unit: columns lo .. hi, and of those the named groups'.
struct Seen {
    bool whole;
    int lo, hi;
    uint32_t named;
    __device__ __forceinline__ void apply(uint32_t (&s)[32], int c) const {
        hide(s, lo - 32 * c, hi - 32 * c);
        hide_unnamed(s, named >> (2 * c));
    }
};

// Largest score of a row in the unit.
__device__ __forceinline__ float row_max(uint32_t ts, const Seen &seen) {
    float most = -INFINITY;
#pragma unroll 1
    for (int c = 0; c < 4; c++) {
        uint32_t s[32];
        tmem_ld32(s, ts + 32 * c);
        tc_wait_ld();
        seen.apply(s, c);
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

// Columns 32 c .. of a unit from `c` on, where some row's weights outgrow its reference or its logits are huge: the reference
// moves to 9 below the next integer of their largest x, with the row's sum, its weights of this unit so far and its
// accumulator (o_cols columns, 0 while it holds nothing).  Rare.
__device__ __forceinline__ void grow_rows(int c, uint32_t ts, uint32_t to, int o_cols, float a, float &top, float &sum, const Seen &seen) {
#pragma unroll 1
    for (; c < 4; c++) {
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
        sum += weights32<true>(s, w, a, top == -INFINITY ? 0.f : -top);
        tmem_st16(ts + 16 * c, w);
    }
}

// All of a unit's columns, 64 at a time: their exponentials, sums and packing are one block of
// independent work.  Weights stand in the place of S (32 columns of scores become 16 of packed
// f16).  The loop is not unrolled: the body of a whole unit would not stay in the instruction cache
// beside the other warps' code.
__device__ __forceinline__ void row_weights(uint32_t ts, uint32_t to, int o_cols, float a, float &top, float &sum, const Seen &seen) {
    const float ref = top == -INFINITY ? 0.f : -top;
    int c = 0;
    const bool huge = __any_sync(~0u, fabsf(ref) > kHuge);
#pragma unroll 1
    for (; c < 4 && !huge; c += 2) {
        uint32_t s0[32], s1[32], w0[16], w1[16];
        tmem_ld32(s0, ts + 32 * c);
        tmem_ld32(s1, ts + 32 * (c + 1));
        tc_wait_ld();
        if (!seen.whole) {
            seen.apply(s0, c);
            seen.apply(s1, c + 1);
        }
        const float p0 = weights32<false>(s0, w0, a, ref);
        const float p1 = weights32<false>(s1, w1, a, ref);
        if (__any_sync(~0u, p0 + p1 > kMostSum)) break;
        sum += p0 + p1;
        tmem_st16(ts + 16 * c, w0);
        tmem_st16(ts + 16 * (c + 1), w1);
    }
    if (c < 4) grow_rows(c, ts, to, o_cols, a, top, sum, seen);
}

// ---- softmax warps: a thread per row ----------------------------------------------------------
template <int D>
__device__ void softmax_role(const Kv4Params &p, Smem<D> *sm, Walk &walk, int64_t total, int64_t ranges) {
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
            if (cf < 1e-37f) cf = 1e-37f;                // never zero, so that a hidden score stays -inf
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
            const int s0 = x.s.base + (x.ua + t) * kKeys;
            Seen seen;
            seen.named = sm->named[unit & 3];
            seen.whole = s0 + kKeys - 1 <= pos0 && (p.window <= 0 || s0 > pos1 - p.window) && seen.named == 0xffu;
            seen.hi = pos - s0;                                              // columns lo .. hi are visible
            seen.lo = p.window > 0 && p.window <= pos ? pos - p.window + 1 - s0 : -0x40000000;
            // the first unit that shows a row anything sets its reference (no weight has been added before)
            if (__any_sync(~0u, top == -INFINITY)) {
                const float most = row_max(ts, seen) * cf;
                if (top == -INFINITY) top = most == INFINITY ? NAN : ceilf(most) - kHead;
            }
            row_weights(ts, to, t > 0 ? D : 0, cf, top, sum, seen);
            tc_wait_st();
            tc_fence_before();
            mbar_arrive(&sm->p_full[m]);
        }
        if (!ok) return;
        ok = wait(sm, &sm->o_full[m], o_phase);
        o_phase ^= 1;
        if (!__all_sync(~0u, ok)) return;
        tc_fence_after();
        const bool full = x.ua == 0 && x.ub == x.s.units;
        const bool none = top == -INFINITY && sum == 0.f;
        const float inv = full ? (none ? 0.f : p.v_unit / sum) : p.v_unit;
        float *part = p.part + (2LL * blockIdx.x + (x.ua == 0)) * kPart;
        char *out = p.out + static_cast<int64_t>(x.r.start + j) * p.out_stride + 2 * static_cast<int64_t>(hq) * D;
#pragma unroll 1
        for (int c = 0; c < D / 32; c++) {
            uint32_t o[32];
            tmem_ld32(o, to + 32 * c);
            tc_wait_ld();
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
                    *reinterpret_cast<float4 *>(at + 4 * k) =
                        make_float4(__uint_as_float(o[4 * k]) * inv, __uint_as_float(o[4 * k + 1]) * inv,
                                    __uint_as_float(o[4 * k + 2]) * inv, __uint_as_float(o[4 * k + 3]) * inv);
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
// What a unit's copies need: the first line of the 16-token group (lane & 7) (-1: not read); klo,
// khi: the unit's tokens that some row sees.
struct Feed {
    int64_t line;
    int klo, khi;
};

template <int D>
__device__ void convert_role(const Kv4Params &p, Smem<D> *sm, Walk &walk) {
    constexpr int kC = D / 32;                       // 16-byte pieces of a token's codes
    constexpr int kTok = 32 * kConvWarps / kC;       // tokens per round of the threads, a multiple of 16
    constexpr int kRounds = kKeys / kTok, kRaw = 32 * kConvWarps * 16;
    const int i = threadIdx.x - 32 * kSoftWarps, lane = i & 31;
    const int c = i % kC, tok = i / kC;              // this thread's piece, and its token within a round
    // The four 16-byte places of a piece's 32 converted codes in a 128-byte row; threads of the upper 64
    // dimensions begin with the third, so that eight neighbours write to eight bank groups.
    const int turn = (c >> 1) << 1;
    const uint32_t row = (c >> 1) * (kKeys * 128) + tok * 128;
    uint32_t to[4];
#pragma unroll
    for (int k = 0; k < 4; k++) to[k] = row + ((((c & 1) * 4 + (k ^ turn)) ^ (tok & 7)) << 4);

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
        f.line = id >= 0 ? (static_cast<int64_t>(id) * p.Hkv + x.head) * p.bs + s % p.bs : -1;
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
    // Each thread copies its own 16-byte pieces and reads only those back: no barrier.  A piece's two
    // scales wait in a register.
    auto fetch = [&](const uint8_t *cache, const uint8_t *scales, const Feed &f, int r, char *raw) {
        const int k = r * kTok + tok;
        const int64_t from = __shfl_sync(~0u, f.line, k >> 4);
        const bool live = from >= 0 && k >= f.klo && k < f.khi;
        const int64_t line = live ? from + (k & 15) : 0;
        cp_async<16>(smem_addr(raw + r * kRaw + i * 16), cache + line * (D / 2) + 16 * c, live);
        return live ? static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t *>(scales + line * (D / 16)) + c)) : 0u;
    };
    // Turn a half (keys or values) of unit `a` into f16, and refill its pieces with the next unit's.
    auto half = [&](const uint8_t *cache, const uint8_t *scales, char *raw, char *dst, const Feed &b, bool next, uint32_t (&sc)[kRounds]) {
#pragma unroll
        for (int r = 0; r < kRounds; r++) {
            const uint4 y = *reinterpret_cast<const uint4 *>(raw + r * kRaw + i * 16);
            const uint32_t s = f16x2_of(sc[r]), s0 = turn ? high_twice(s) : low_twice(s), s1 = turn ? low_twice(s) : high_twice(s);
            const uint32_t w[4] = {turn ? y.z : y.x, turn ? y.w : y.y, turn ? y.x : y.z, turn ? y.y : y.w};
#pragma unroll
            for (int k = 0; k < 4; k++) {
                uint32_t h[4];
                f16_of_e2m1x8(w[k], h);
                const uint32_t m = k < 2 ? s0 : s1;
                *reinterpret_cast<uint4 *>(dst + to[k] + r * kTok * 128) =
                    make_uint4(mul_f16x2(h[0], m), mul_f16x2(h[1], m), mul_f16x2(h[2], m), mul_f16x2(h[3], m));
            }
            if (next) sc[r] = fetch(cache, scales, b, r, raw);
        }
        cp_commit();
    };

    uint32_t ksc[kRounds], vsc[kRounds];
    ask();
    Feed a = resolve();
#pragma unroll
    for (int r = 0; r < kRounds; r++) ksc[r] = fetch(p.kc, p.k_sf, a, r, sm->raw[0]);
    cp_commit();
#pragma unroll
    for (int r = 0; r < kRounds; r++) vsc[r] = fetch(p.vc, p.v_sf, a, r, sm->raw[1]);
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
        const uint32_t named = __ballot_sync(~0u, a.line >= 0) & 0xffu;
        if (i == 0) sm->named[unit & 3] = named;
        half(p.kc, p.k_sf, sm->raw[0], sm->k[stage], b, next, ksc);
        fence_async_shared();
        mbar_arrive(&sm->k_full[stage]);
        cp_wait<1>();
        ok = wait(sm, &sm->v_free[stage], parity);
        if (!__all_sync(~0u, ok)) break;
        half(p.vc, p.v_sf, sm->raw[1], sm->v[stage], b, next, vsc);
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
__device__ void issue_role(Smem<D> *sm, Walk &walk) {
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
__global__ void __launch_bounds__(kThreads, 1) kv4_prefill_kernel(const Kv4Params p) {
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
        fence_mbar_init();
    }
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
        Walk walk(p, prefix, blockIdx.x * total / ranges, (blockIdx.x + 1) * total / ranges);
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
int launch(const Kv4Params &p, int sms, cudaStream_t s) {
    constexpr size_t smem = sizeof(Smem<D>) + 1024;
    static_assert(smem <= 227 * 1024, "shared memory");
    static bool set[64] = {false};
    const int rc = kv8_allow_smem(reinterpret_cast<const void *>(kv4_prefill_kernel<D>), static_cast<int>(smem), set);
    if (rc != PKV_OK) return rc;
    PKV_CUDA_TRY(launch_pdl(kv4_prefill_kernel<D>, dim3(sms), dim3(kThreads), smem, s, p));
    return kv8_launch_merge(p, D, kRows, sms, 1, s);
}

}  // namespace

int64_t kv4_prefill_workspace(int32_t head_dim, int sms) {
    return head_dim > 128 ? 0 : static_cast<int64_t>(sms) * (2LL * kRows * (head_dim + 2) * 4 + 16);
}

int kv4_launch_prefill(const Kv4Params &p, int32_t head_dim, int sms, cudaStream_t s) {
    return head_dim == 64 ? launch<64>(p, sms, s) : launch<128>(p, sms, s);
}

}  // namespace pkv
