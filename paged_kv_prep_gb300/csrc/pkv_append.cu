// Appending a step's keys and values to a paged cache with the rotation by
// position on the way (the queries rotated beside them), to a 16-bit cache or
// to the 4-bit one, and reading lines of the 4-bit cache back.
//
// Mathematics.  Pair (x0, x1) with cosine c and sine s of its axis's position:
// (x0 c - x1 s, x1 c + x0 s) in fp32, each operation rounded by itself, so that
// an elementwise restatement gives the same bits; one rounding to the element
// type.  4 bits: of 16 neighbours the scale is e4m3(max |x| / (6 unit)), a code
// e2m1(x / (scale unit)); both are true quotients, because 16-bit inputs often
// lie exactly half way between two codes and a product with a reciprocal would
// move them.  A quotient is such a product with its error x - y (scale unit), exact in a fused
// multiply-add, brought back once (Markstein's correction): exact where the quotient is a
// floating-point number, as those middles are; 3 operations where a division takes a dozen.  A scale's reciprocal is
// the hardware's approximation after one step of Newton's.
//
// Bound: HBM (every line read and written once), or launch latency for a decode
// step.
//
// Layout.  A warp takes one token and a few of its query lines or KV heads; a lane moves 16 bytes
// of a line and keeps the cosines and sines of its eight elements in registers for all of the
// warp's lines.  All lines are asked for before the token's position is known, so the chain position -> table row
// runs beside them.  A pair's other element comes by a shuffle.
//
// Measured, 16384 tokens, 32 query and 8 KV heads of 128: into the 16-bit cache (407 MB) 61 us, 98 % of the
// copy rate; into the 4-bit one and the lines read back (321 and 120 MB, three axes) 82 us, 79 %: the append takes 69, bound
// by instructions (half of them conversions and maxima on the integer pipe), the reading 13.5, most of it from and to L2.
// The two with divisions 115 us where 101 remained; with the scale's quotient a division 85.7 where 84.3 remained, with maxima
// of bit patterns 84.3 and 83.7.
#include "pkv_kv4.cuh"
#include "pkv_kv8_attention.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
// Line steps of a warp: queries; keys and values together.  Threads of a CTA, and CTAs that an SM holds, by the cache.
// (16384 tokens, 32 query and 8 KV heads x 128, and 6007 of fewer heads on three axes, both into the 16-bit cache: 61.1 and 19.4
// us; 8 and 4 steps 60.9 and 20.0, 7 and 2 66.8 and 19.3; with CTAs of 128 threads 61.6 and 20.2, of 32 60.7 and 20.8;
// without streaming loads and stores 63.6 and 20.5.  Into the 4-bit cache, with the reading back: 82 us; 8 and 2 steps 88,
// 4 and 1 92, CTAs of 64 threads 91, of 256 87; eight CTAs an SM 82.6, six 87, nine 89.)
constexpr int kQSteps = 4, kKvSteps = 2;
constexpr int threads_of(bool kv4) { return kv4 ? 128 : 64; }
constexpr int resident_of(bool kv4) { return kv4 ? 7 : 12; }
constexpr int kLoadSteps = 4;            // (append and reading back together: 82.6 us; two 83.7, one 88.0)
constexpr int kMaxAxes = 8;

struct Rope {
    const float *table;
    const int32_t *pos;
    int64_t axis_stride;
    int32_t rot, max_position, axes, interleaved;     // rot 0: no rotation
    uint64_t axis8[16];                               // axes of pairs 8 i .. 8 i + 7, a byte each
};

struct AppendParams {
    Rope rope;
    const char *q, *k, *v;
    char *q_out;
    int64_t q_stride, q_out_stride, k_stride, v_stride;
    uint8_t *kc, *vc, *ks, *vs;
    const int64_t *slots;
    int64_t num_slots, jobs;
    float k_unit, v_unit, k_six, v_six, k_sixth, v_sixth;      // six times the unit, and its reciprocal
    int32_t T, Hq, H, bs, q_parts, parts;
    int32_t *err;
};

// Cosines and sines for a lane's eight elements: element i becomes x c[i] + (its pair's other) s[i].
struct Turn {
    float c[8], s[8];
    int from;                                         // lane that has the other elements
    bool on;
};

// False where the token has a position outside the table.
template <int D>
__device__ __forceinline__ bool make_turn(const Rope &r, int64_t t, Turn &w, int32_t *err) {
    constexpr int kLine = D / 8;
    const int lane = threadIdx.x & 31, l = lane % kLine, e0 = 8 * l, half = r.rot >> 1;
    w.on = e0 < r.rot;
    w.from = lane;
    if (r.rot == 0) return true;
    int32_t pos = 0;
    if (lane < r.axes) pos = r.pos[lane * r.axis_stride + t];
    if (__any_sync(~0u, pos < 0 || pos >= r.max_position)) {
        if (lane == 0 && err) atomicOr(err, PKV_DEVERR_POSITION);
        return false;
    }
    const bool second = !r.interleaved && e0 >= half;
    const int pair = !w.on ? 0 : r.interleaved ? e0 >> 1 : second ? e0 - half : e0;     // of the first element
    if (!r.interleaved && w.on) w.from = lane + (second ? -half : half) / 8;
    // positions of the pairs (four where neighbours are paired)
    int32_t at[8];
    const int32_t first = __shfl_sync(~0u, pos, 0);
#pragma unroll
    for (int i = 0; i < 8; i++) at[i] = first;
    bool same = true;
    if (r.axes > 1) {
        const uint64_t names = r.axis8[pair >> 3] >> (8 * (pair & 7));
#pragma unroll
        for (int i = 0; i < 8; i++) {
            at[i] = __shfl_sync(~0u, pos, static_cast<int>(names >> (8 * i)) & 7);
            if (i < (r.interleaved ? 4 : 8)) same &= at[i] == at[0];
        }
    }
    float c[8], s[8];
    const float *row = r.table + static_cast<int64_t>(at[0]) * r.rot + pair;
    if (same) {
#pragma unroll
        for (int i = 0; i < 8; i += 4) {
            if (i && r.interleaved) break;
            const float4 a = __ldg(reinterpret_cast<const float4 *>(row + i));
            const float4 b = __ldg(reinterpret_cast<const float4 *>(row + half + i));
            c[i] = a.x, c[i + 1] = a.y, c[i + 2] = a.z, c[i + 3] = a.w;
            s[i] = b.x, s[i + 1] = b.y, s[i + 2] = b.z, s[i + 3] = b.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            if (i >= 4 && r.interleaved) break;
            const float *one = r.table + static_cast<int64_t>(at[i]) * r.rot + pair + i;
            c[i] = __ldg(one);
            s[i] = __ldg(one + half);
        }
    }
#pragma unroll
    for (int i = 0; i < 8; i++) {
        w.c[i] = r.interleaved ? c[i >> 1] : c[i];
        const float y = r.interleaved ? s[i >> 1] : s[i];
        w.s[i] = (r.interleaved ? !(i & 1) : !second) ? -y : y;
    }
    return true;
}

template <bool kFp16>
__device__ __forceinline__ void widen8(uint4 v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const float2 y = widen2(w[i], kFp16);
        x[2 * i] = y.x;
        x[2 * i + 1] = y.y;
    }
}

// The lane's eight elements, rotated, in fp32.  All lanes of the warp call it together.
template <bool kFp16>
__device__ __forceinline__ void turned(const Rope &r, const Turn &w, uint4 v, float (&x)[8]) {
    widen8<kFp16>(v, x);
    if (r.rot == 0) return;
    float y[8];
    if (r.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; i++) y[i] = x[i ^ 1];
    } else {
        uint4 u;
        u.x = __shfl_sync(~0u, v.x, w.from);
        u.y = __shfl_sync(~0u, v.y, w.from);
        u.z = __shfl_sync(~0u, v.z, w.from);
        u.w = __shfl_sync(~0u, v.w, w.from);
        widen8<kFp16>(u, y);
    }
    if (w.on) {
#pragma unroll
        for (int i = 0; i < 8; i++) x[i] = __fadd_rn(__fmul_rn(x[i], w.c[i]), __fmul_rn(y[i], w.s[i]));
    }
}

template <bool kFp16>
__device__ __forceinline__ uint4 rounded(const float (&x)[8]) {
    return make_uint4(pack_out(x[0], x[1], kFp16), pack_out(x[2], x[3], kFp16), pack_out(x[4], x[5], kFp16),
                      pack_out(x[6], x[7], kFp16));
}

// The largest of three, NaN if one is.
__device__ __forceinline__ float nan_max3(float a, float b, float c) {
    float y;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Eight of a group's 16 elements (the neighbouring lane has the others): codes, and the group's scale.
struct Quantised {
    uint32_t codes, scale;
    bool nan;
};
__device__ __forceinline__ Quantised quantise(const float (&x)[8], float unit, float six, float sixth) {
    float most = nan_max3(nan_max3(nan_max3(fabsf(x[0]), fabsf(x[1]), fabsf(x[2])), fabsf(x[3]), fabsf(x[4])), fabsf(x[5]), fabsf(x[6]));
    most = nan_max3(most, fabsf(x[7]), 0.f);
    most = nan_max3(most, __shfl_xor_sync(~0u, most, 1), 0.f);
    Quantised z;
    z.nan = most != most;
    const float first = most * sixth;                 // corrected where it is not far past the largest scale
    z.scale = e4m3x2(first < 1024.f ? fmaf(fmaf(-first, six, most), sixth, first) : first, 0.f) & 0xffu;
    const float by = floats_of(z.scale).x * unit, guess = rcp_fast(by), inverse = fmaf(fmaf(-by, guess, 1.f), guess, guess);
    float y[8];
    if (most * inverse < 0x1p64f) {
#pragma unroll
        for (int i = 0; i < 8; i++) {
            const float near = x[i] * inverse;
            y[i] = fmaf(fmaf(-near, by, x[i]), inverse, near);
        }
        z.codes = e2m1x8(y);
    } else {                                          // infinities among them, or far too large; a scale of 0 or NaN
#pragma unroll
        for (int i = 0; i < 8; i++) y[i] = __fdiv_rn(x[i], by);
        z.codes = by > 0.f ? e2m1x8(y) : 0;
    }
    return z;
}

// A line's scales, a byte of every second lane, as words in the lanes 8 i.
__device__ __forceinline__ uint32_t scale_word(uint32_t scale, int l) {
    uint32_t w = scale << (8 * ((l >> 1) & 3));
    w |= __shfl_xor_sync(~0u, w, 2);
    w |= __shfl_xor_sync(~0u, w, 4);
    return w;
}

template <int D, bool kFp16, bool kKv4>
__global__ void __launch_bounds__(threads_of(kKv4), resident_of(kKv4)) append_kernel(const AppendParams p) {
    constexpr int kLine = D / 8, kAtOnce = 32 / kLine;             // lanes of a line, lines of a step
    constexpr int kWarps = threads_of(kKv4) / 32;
    pdl_wait();
    pdl_trigger();
    const int64_t job = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (job >= p.jobs) return;
    const int64_t t = job / p.parts;
    const int part = static_cast<int>(job - t * p.parts);
    const int lane = threadIdx.x & 31, l = lane % kLine, mine = lane / kLine;
    Turn w;
    if (part < p.q_parts) {
        const int h0 = part * kQSteps * kAtOnce + mine;
        const char *src = p.q + t * p.q_stride + 16 * l;
        char *dst = p.q_out + t * p.q_out_stride + 16 * l;
        uint4 raw[kQSteps];
#pragma unroll
        for (int i = 0; i < kQSteps; i++) {
            raw[i] = make_uint4(0, 0, 0, 0);
            if (h0 + i * kAtOnce < p.Hq) raw[i] = __ldcs(reinterpret_cast<const uint4 *>(src + 2LL * D * (h0 + i * kAtOnce)));
        }
        if (!make_turn<D>(p.rope, t, w, p.err)) return;
#pragma unroll
        for (int i = 0; i < kQSteps; i++) {
            float x[8];
            turned<kFp16>(p.rope, w, raw[i], x);
            if (w.on) raw[i] = rounded<kFp16>(x);
            if (h0 + i * kAtOnce < p.Hq) __stcs(reinterpret_cast<uint4 *>(dst + 2LL * D * (h0 + i * kAtOnce)), raw[i]);
        }
        return;
    }
    const int h0 = (part - p.q_parts) * kKvSteps * kAtOnce + mine;
    const char *ksrc = p.k + t * p.k_stride + 16 * l, *vsrc = p.v + t * p.v_stride + 16 * l;
    uint4 rk[kKvSteps], rv[kKvSteps];
    const int64_t slot = p.slots[t];
#pragma unroll
    for (int i = 0; i < kKvSteps; i++) {
        const int h = h0 + i * kAtOnce;
        rk[i] = rv[i] = make_uint4(0, 0, 0, 0);
        if (h < p.H) {
            rk[i] = __ldcs(reinterpret_cast<const uint4 *>(ksrc + 2LL * D * h));
            rv[i] = __ldcs(reinterpret_cast<const uint4 *>(vsrc + 2LL * D * h));
        }
    }
    if (!make_turn<D>(p.rope, t, w, p.err)) return;
    if (slot < 0 || slot >= p.num_slots) {
        if (slot >= p.num_slots && lane == 0 && p.err) atomicOr(p.err, PKV_DEVERR_SLOT);
        return;
    }
    const uint32_t block = static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.bs);
    const uint32_t offset = static_cast<uint32_t>(slot) - block * static_cast<uint32_t>(p.bs);
#pragma unroll
    for (int i = 0; i < kKvSteps; i++) {
        const int h = h0 + i * kAtOnce;
        float x[8];
        turned<kFp16>(p.rope, w, rk[i], x);
        if constexpr (kKv4) {
            Quantised a = quantise(x, p.k_unit, p.k_six, p.k_sixth);
            widen8<kFp16>(rv[i], x);
            Quantised b = quantise(x, p.v_unit, p.v_six, p.v_sixth);
            // a NaN value is noted in the line's first key scale
            const uint32_t nan = __ballot_sync(~0u, b.nan) >> (mine * kLine);
            if (b.nan) b.scale = b.codes = 0;
            if (l < 2 && (nan & (0xffffffffu >> (32 - kLine)))) a.scale = 0x7f;
            const uint32_t sa = scale_word(a.scale, l), sb = scale_word(b.scale, l);
            if (h < p.H) {
                const int64_t line = (static_cast<int64_t>(block) * p.H + h) * p.bs + offset;
                *reinterpret_cast<uint32_t *>(p.kc + line * (D / 2) + 4 * l) = a.codes;
                *reinterpret_cast<uint32_t *>(p.vc + line * (D / 2) + 4 * l) = b.codes;
                if ((l & 7) == 0) {
                    *reinterpret_cast<uint32_t *>(p.ks + line * (D / 16) + (l >> 1)) = sa;
                    *reinterpret_cast<uint32_t *>(p.vs + line * (D / 16) + (l >> 1)) = sb;
                }
            }
        } else {
            if (w.on) rk[i] = rounded<kFp16>(x);
            if (h < p.H) {
                const int64_t at = (slot * p.H + h) * (2 * D) + 16 * l;
                __stcs(reinterpret_cast<uint4 *>(p.kc + at), rk[i]);
                __stcs(reinterpret_cast<uint4 *>(p.vc + at), rv[i]);
            }
        }
    }
}

struct LoadParams {
    const uint8_t *kc, *vc, *ks, *vs;
    const int64_t *slots;
    int64_t num_slots, jobs;
    char *k, *v;
    float k_unit, v_unit;
    int32_t H, bs, parts;
    int32_t *err;
};

// The lane's eight values: code * scale is exact in f16, the unit multiplies it in fp32.
template <bool kFp16>
__device__ __forceinline__ uint4 values_of(uint32_t codes, uint32_t scale, float unit) {
    uint32_t h[4];
    f16_of_e2m1x8(codes, h);
    const uint32_t s = low_twice(f16x2_of(scale));
    float x[8];
#pragma unroll
    for (int i = 0; i < 4; i++) {
        const uint32_t y = mul_f16x2(h[i], s);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&y));
        x[2 * i] = f.x * unit;
        x[2 * i + 1] = f.y * unit;
    }
    return rounded<kFp16>(x);
}

template <int D, bool kFp16>
__global__ void __launch_bounds__(kThreads) kv4_load_kernel(const LoadParams p) {
    constexpr int kLine = D / 8, kAtOnce = 32 / kLine;
    pdl_wait();
    pdl_trigger();
    const int64_t job = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (job >= p.jobs) return;
    const int64_t i = job / p.parts;
    const int lane = threadIdx.x & 31, l = lane % kLine;
    const int h0 = static_cast<int>(job - i * p.parts) * kLoadSteps * kAtOnce + lane / kLine;
    const int64_t slot = p.slots[i];
    const bool live = slot >= 0 && slot < p.num_slots;
    if (slot >= p.num_slots && lane == 0 && p.err) atomicOr(p.err, PKV_DEVERR_SLOT);
    const uint32_t block = live ? static_cast<uint32_t>(slot) / static_cast<uint32_t>(p.bs) : 0;
    const uint32_t offset = static_cast<uint32_t>(slot) - block * static_cast<uint32_t>(p.bs);
    uint32_t kcode[kLoadSteps], vcode[kLoadSteps], kscale[kLoadSteps], vscale[kLoadSteps];
#pragma unroll
    for (int n = 0; n < kLoadSteps; n++) {
        const int h = h0 + n * kAtOnce;
        kcode[n] = vcode[n] = kscale[n] = vscale[n] = 0;
        if (live && h < p.H) {
            const int64_t line = (static_cast<int64_t>(block) * p.H + h) * p.bs + offset;
            if (p.k) {
                kcode[n] = __ldg(reinterpret_cast<const uint32_t *>(p.kc + line * (D / 2)) + l);
                kscale[n] = __ldg(p.ks + line * (D / 16) + (l >> 1));
            }
            if (p.v) {
                vcode[n] = __ldg(reinterpret_cast<const uint32_t *>(p.vc + line * (D / 2)) + l);
                vscale[n] = __ldg(p.vs + line * (D / 16) + (l >> 1));
            }
        }
    }
#pragma unroll
    for (int n = 0; n < kLoadSteps; n++) {
        const int h = h0 + n * kAtOnce;
        if (h >= p.H) continue;
        const int64_t at = (i * p.H + h) * (2 * D) + 16 * l;
        if (p.k) *reinterpret_cast<uint4 *>(p.k + at) = values_of<kFp16>(kcode[n], kscale[n], p.k_unit);
        if (p.v) *reinterpret_cast<uint4 *>(p.v + at) = values_of<kFp16>(vcode[n], vscale[n], p.v_unit);
    }
}

int check_rope(const pkv_rope *r, int32_t head_dim, int32_t num_tokens, Rope *out) {
    if (r->rot_dim < 16 || r->rot_dim % 16 || r->rot_dim > head_dim || r->num_axes < 1 || r->num_axes > kMaxAxes ||
        r->max_position < 1 || (r->num_axes > 1 && r->axis_stride < num_tokens) || !r->table || !r->positions)
        return PKV_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(r->table) & 15) || (reinterpret_cast<uintptr_t>(r->positions) & 3)) return PKV_ERR_ALIGN;
    out->table = r->table;
    out->pos = r->positions;
    out->axis_stride = r->axis_stride;
    out->rot = r->rot_dim;
    out->max_position = r->max_position;
    out->axes = r->num_axes;
    out->interleaved = r->interleaved != 0;
    for (int i = 0; i < r->rot_dim / 2; i++) {
        const uint64_t a = r->pair_axes ? r->pair_axes[i] : 0;
        if (a >= static_cast<uint64_t>(r->num_axes)) return PKV_ERR_INVALID_ARG;
        out->axis8[i >> 3] |= a << (8 * (i & 7));
    }
    return PKV_OK;
}

// The sources and the queries; p's cache is filled in already.
int check_rows(AppendParams &p, bool kv4, const void *k, const void *v, int32_t head_dim, int32_t dtype, const void *q, void *q_out) {
    if (!kv8_head_dim(head_dim) || (dtype != PKV_BF16 && dtype != PKV_FP16) || p.T < 0 || p.T >= PKV_MAX_TOKENS || p.H < 1 ||
        p.H > kMaxHeads || p.Hq < 0 || p.Hq > (1 << 20) || p.k_stride < 0 || p.v_stride < 0 || p.q_stride < 0 ||
        p.q_out_stride < 0)
        return PKV_ERR_INVALID_ARG;
    if (p.T == 0) return PKV_OK;
    if (!k || !v || !p.slots || (p.Hq > 0 && (!q || !q_out))) return PKV_ERR_INVALID_ARG;
    const uintptr_t all = reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v) | reinterpret_cast<uintptr_t>(q) |
                          reinterpret_cast<uintptr_t>(q_out) | static_cast<uintptr_t>(p.k_stride | p.v_stride);
    if ((all & 15) || (p.Hq > 0 && ((p.q_stride | p.q_out_stride) & 15)) || (reinterpret_cast<uintptr_t>(p.slots) & 7))
        return PKV_ERR_ALIGN;
    const int64_t line = 2LL * p.H * head_dim, row = 2LL * p.Hq * head_dim;
    if (p.T > 1 && (p.k_stride < line || p.v_stride < line || (p.Hq > 0 && (p.q_stride < row || p.q_out_stride < row))))
        return PKV_ERR_INVALID_ARG;
    const int lines = 32 / (head_dim / 8);
    const int q_lines = kQSteps * lines, kv_lines = kKvSteps * lines;
    p.q_parts = (p.Hq + q_lines - 1) / q_lines;
    p.parts = p.q_parts + (p.H + kv_lines - 1) / kv_lines;
    p.jobs = static_cast<int64_t>(p.T) * p.parts;
    p.k = static_cast<const char *>(k);
    p.v = static_cast<const char *>(v);
    p.q = static_cast<const char *>(q);
    p.q_out = static_cast<char *>(q_out);
    const int warps = threads_of(kv4) / 32;
    return (p.jobs + warps - 1) / warps > 0x7fffffff ? PKV_ERR_INVALID_ARG : PKV_OK;
}

template <bool kKv4>
int launch_append(const AppendParams &p, int32_t head_dim, int32_t dtype, cudaStream_t s) {
    const bool h = dtype == PKV_FP16;
    auto kernel = head_dim == 64    ? (h ? append_kernel<64, true, kKv4> : append_kernel<64, false, kKv4>)
                  : head_dim == 128 ? (h ? append_kernel<128, true, kKv4> : append_kernel<128, false, kKv4>)
                                    : (h ? append_kernel<256, true, kKv4> : append_kernel<256, false, kKv4>);
    constexpr int warps = threads_of(kKv4) / 32;
    PKV_CUDA_TRY(launch_pdl(kernel, dim3(static_cast<unsigned>((p.jobs + warps - 1) / warps)), dim3(32 * warps), 0, s, p));
    return PKV_OK;
}

}  // namespace
}  // namespace pkv

extern "C" {

int pkv_rope_store(const pkv_rope *rope, const void *k, const void *v, int64_t k_stride_bytes, int64_t v_stride_bytes,
                   int32_t num_heads, int32_t head_dim, int32_t dtype, const void *q, int64_t q_stride_bytes,
                   int32_t num_q_heads, void *q_out, int64_t q_out_stride_bytes, void *k_cache, void *v_cache,
                   int64_t num_slots, const int64_t *slot_mapping, int32_t num_tokens, int32_t *d_error,
                   pkv_stream_t stream) {
    if (!rope || num_slots < 0 || num_slots > 0xffffffffLL) return PKV_ERR_INVALID_ARG;
    pkv::AppendParams p = {};
    p.T = num_tokens;
    p.H = num_heads;
    p.Hq = num_q_heads;
    p.k_stride = k_stride_bytes;
    p.v_stride = v_stride_bytes;
    p.q_stride = q_stride_bytes;
    p.q_out_stride = q_out_stride_bytes;
    p.kc = static_cast<uint8_t *>(k_cache);
    p.vc = static_cast<uint8_t *>(v_cache);
    p.slots = slot_mapping;
    p.num_slots = num_slots;
    p.bs = 1;
    p.err = d_error;
    int rc = pkv::check_rows(p, false, k, v, head_dim, dtype, q, q_out);
    if (rc == PKV_OK && num_tokens > 0) rc = pkv::check_rope(rope, head_dim, num_tokens, &p.rope);
    if (rc != PKV_OK || num_tokens == 0) return rc;
    if (num_slots > 0 && (!k_cache || !v_cache)) return PKV_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache)) & 15) return PKV_ERR_ALIGN;
    return pkv::launch_append<false>(p, head_dim, dtype, pkv::as_stream(stream));
}

int pkv_kv4_store(const pkv_kv4_cache *cache, const pkv_rope *rope, const void *k, const void *v, int64_t k_stride_bytes,
                  int64_t v_stride_bytes, int32_t dtype, const void *q, int64_t q_stride_bytes, int32_t num_q_heads,
                  void *q_out, int64_t q_out_stride_bytes, const int64_t *slot_mapping, int32_t num_tokens,
                  int32_t *d_error, pkv_stream_t stream) {
    int rc = pkv::kv4_check_cache(cache);
    if (rc != PKV_OK) return rc;
    if (!rope && num_q_heads != 0) return PKV_ERR_INVALID_ARG;
    pkv::AppendParams p = {};
    p.T = num_tokens;
    p.H = cache->num_heads;
    p.Hq = num_q_heads;
    p.k_stride = k_stride_bytes;
    p.v_stride = v_stride_bytes;
    p.q_stride = q_stride_bytes;
    p.q_out_stride = q_out_stride_bytes;
    p.kc = static_cast<uint8_t *>(cache->k_cache);
    p.vc = static_cast<uint8_t *>(cache->v_cache);
    p.ks = static_cast<uint8_t *>(cache->k_scale);
    p.vs = static_cast<uint8_t *>(cache->v_scale);
    p.slots = slot_mapping;
    p.num_slots = cache->num_blocks * cache->block_size;
    p.bs = cache->block_size;
    p.k_unit = cache->k_unit;
    p.v_unit = cache->v_unit;
    p.k_six = 6.f * cache->k_unit;
    p.v_six = 6.f * cache->v_unit;
    p.k_sixth = 1.f / p.k_six;
    p.v_sixth = 1.f / p.v_six;
    p.err = d_error;
    rc = pkv::check_rows(p, true, k, v, cache->head_dim, dtype, q, q_out);
    if (rc == PKV_OK && num_tokens > 0 && rope) rc = pkv::check_rope(rope, cache->head_dim, num_tokens, &p.rope);
    if (rc != PKV_OK || num_tokens == 0) return rc;
    return pkv::launch_append<true>(p, cache->head_dim, dtype, pkv::as_stream(stream));
}

int pkv_kv4_load(const pkv_kv4_cache *cache, const int64_t *slots, int32_t count, int32_t dtype, void *k, void *v,
                 int32_t *d_error, pkv_stream_t stream) {
    const int rc = pkv::kv4_check_cache(cache);
    if (rc != PKV_OK) return rc;
    if (count < 0 || (dtype != PKV_BF16 && dtype != PKV_FP16)) return PKV_ERR_INVALID_ARG;
    if (count == 0 || (!k && !v)) return PKV_OK;
    if (!slots) return PKV_ERR_INVALID_ARG;
    if (((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 15) || (reinterpret_cast<uintptr_t>(slots) & 7))
        return PKV_ERR_ALIGN;
    pkv::LoadParams p = {};
    p.kc = static_cast<const uint8_t *>(cache->k_cache);
    p.vc = static_cast<const uint8_t *>(cache->v_cache);
    p.ks = static_cast<const uint8_t *>(cache->k_scale);
    p.vs = static_cast<const uint8_t *>(cache->v_scale);
    p.slots = slots;
    p.num_slots = cache->num_blocks * cache->block_size;
    p.k = static_cast<char *>(k);
    p.v = static_cast<char *>(v);
    p.k_unit = cache->k_unit;
    p.v_unit = cache->v_unit;
    p.H = cache->num_heads;
    p.bs = cache->block_size;
    p.err = d_error;
    const int D = cache->head_dim, lines = 32 / (D / 8) * pkv::kLoadSteps;
    p.parts = (p.H + lines - 1) / lines;
    p.jobs = static_cast<int64_t>(count) * p.parts;
    const int64_t grid = (p.jobs + pkv::kWarps - 1) / pkv::kWarps;
    if (grid > 0x7fffffff) return PKV_ERR_INVALID_ARG;
    const bool h = dtype == PKV_FP16;
    auto kernel = D == 64    ? (h ? pkv::kv4_load_kernel<64, true> : pkv::kv4_load_kernel<64, false>)
                  : D == 128 ? (h ? pkv::kv4_load_kernel<128, true> : pkv::kv4_load_kernel<128, false>)
                             : (h ? pkv::kv4_load_kernel<256, true> : pkv::kv4_load_kernel<256, false>);
    PKV_CUDA_TRY(pkv::launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(pkv::kThreads), 0, pkv::as_stream(stream), p));
    return PKV_OK;
}

}  // extern "C"
