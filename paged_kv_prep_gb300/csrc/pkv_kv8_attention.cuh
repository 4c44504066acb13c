// Pieces shared by the attention kernels on the 8-bit paged cache: launch
// parameters, the plan over ragged requests, warp-level matrix products.
#pragma once

#include <type_traits>

#include "pkv_async.cuh"
#include "pkv_kv8.cuh"

namespace pkv {

// Positions that are seen lie below this, so that the end of a unit, or of the one after it, fits 32 bits.
constexpr int32_t kMostKeys = 0x7fffffff - 4095;

struct AttnParams {
    const char *q;                 // [T][Hq][D], bytes below
    int64_t q_stride;
    char *out;
    int64_t out_stride;
    float *lse;                    // [T][Hq]
    const uint8_t *kc, *vc;
    const float *ks, *vs;
    float *weights;                // [num_slots] or NULL
    const int32_t *tables;
    const int32_t *qsl;
    const int32_t *lens;
    int64_t num_blocks;
    int32_t n, T, W;               // W: a table's entries that are looked at, those of blocks below kMostKeys
    int32_t table_row;             // entries of a table
    int32_t bs, Hkv, G;
    int32_t window;
    int32_t fp16;
    float scale_log2;              // softmax_scale * log2(e)
    int32_t whole;                 // decode kernel: row tiles are not cut (no merge follows)
    int32_t short_rows;            // requests with more (query, head) rows than this take the prefill kernel
    float *part;                   // partial results, see pkv_kv8_decode.cu
    int4 *meta;
    int32_t *err;

    // A table's width and what of it is looked at (a limit here costs the kernels nothing; one in request_of cost a step of
    // chunks and decodes 16 us of 802).
    void set_table(int32_t width, int32_t block_size) {
        table_row = width;
        W = width < kMostKeys / block_size ? width : kMostKeys / block_size;
    }

    // The table's entry for a position, unchecked but for the table's end (-1 past it).
    __device__ __forceinline__ int32_t table_at(const int32_t *table, int32_t pos) const {
        const int32_t j = pos / bs;
        return j < W ? table[j] : -1;
    }
};

// Warps that one launch of the decode kernel may have: sixteen an SM, or one for each KV head (rounded up
// to whole CTAs) where the heads are more than that.
constexpr int kMaxWarps = 16;
inline int64_t kv8_most_workers(int sms) {
    const int64_t a = static_cast<int64_t>(sms) * kMaxWarps, b = kMaxHeads + kMaxWarps;
    return a > b ? a : b;
}

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;

// One request's share of the batch.
struct Req {
    int32_t start;                 // its first token in the batch
    int32_t count;                 // scheduled tokens (0: nothing to do)
    int32_t len;                   // cached tokens, those of this step included
    int32_t lo;                    // first key that any of its queries sees
    int32_t keys;                  // keys that its block table can name
};

__device__ __forceinline__ Req request_of(const AttnParams &p, int i, bool report = false) {
    Req r;
    const int32_t a = p.qsl[i], b = p.qsl[i + 1];
    r.start = a;
    r.count = b - a;
    r.len = p.lens[i];
    if (a < 0 || b < a || b > p.T) {
        if (report && p.err) atomicOr(p.err, PKV_DEVERR_COUNT);
        r.count = 0;
    }
    const int64_t cap = static_cast<int64_t>(p.W) * p.bs;
    if (r.len > cap && report && p.err && r.count > 0) atomicOr(p.err, PKV_DEVERR_BLOCK);
    r.keys = r.len < cap ? r.len : static_cast<int32_t>(cap);
    r.lo = 0;
    if (p.window > 0) {
        const int64_t lo = static_cast<int64_t>(r.len) - r.count - p.window + 1;
        r.lo = lo > 0 ? static_cast<int32_t>(lo) : 0;
    }
    return r;
}

// First position that a query at `pos` sees.  (Before position 0, pos - window may pass the smallest integer.)
__device__ __forceinline__ int32_t lo_of(const AttnParams &p, int32_t pos) {
    return p.window > 0 ? max(0, max(pos, 0) - p.window + 1) : 0;
}

// Value scales below 2^-100 (an unwritten block's zero among them) count as 2^-100, so that their
// logarithm and reciprocal stay finite.
__device__ __forceinline__ float value_scale(float s) { return s < 0x1p-100f ? 0x1p-100f : s; }

// Block id of a position, -1 where there is none to read.
__device__ __forceinline__ int32_t block_of(const AttnParams &p, const int32_t *table, int32_t pos) {
    const int32_t b = p.table_at(table, pos);
    if (b >= p.num_blocks) {
        if (p.err) atomicOr(p.err, PKV_DEVERR_BLOCK);
        return -1;
    }
    return b < 0 ? -1 : b;
}

// Units of `tokens` that the tables' longest request can have, and two; no more than 2^20, which is more than any launch
// has warps, so that a product with row tiles and heads fits 64 bits.
inline int64_t most_units(const AttnParams &p, int tokens) {
    const int64_t units = static_cast<int64_t>(p.W) * p.bs / tokens + 2;
    return units < (1 << 20) ? units : 1 << 20;
}

// Prefix sums of the requests' units: thread c of the CTA holds requests c * per .. (c + 1) * per - 1.
// s_prefix[kThreads + 1] gets the exclusive sums; the total is s_prefix[kThreads].
template <int kThreads, typename UnitsOf>
__device__ __forceinline__ int64_t plan_prefix(int64_t *s_prefix, int64_t *s_warp, int n, UnitsOf units_of) {
    const int per = (n + kThreads - 1) / kThreads;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    int64_t sum = 0;
    for (int k = 0; k < per; k++) {
        const int i = tid * per + k;
        if (i < n) sum += units_of(i);
    }
    int64_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(~0u, incl, o);
        if (lane >= o) incl += u;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int64_t base = 0;
    for (int w = 0; w < warp; w++) base += s_warp[w];
    s_prefix[tid] = base + incl - sum;
    if (tid == kThreads - 1) s_prefix[kThreads] = base + incl;
    __syncthreads();
    return s_prefix[kThreads];
}

// The request that unit u (0 <= u < total) belongs to; its first unit goes to *first.
template <int kThreads, typename UnitsOf>
__device__ __forceinline__ int plan_find(const int64_t *s_prefix, int n, int64_t u, UnitsOf units_of,
                                         int64_t *first) {
    int a = 0, b = kThreads;                       // s_prefix[a] <= u < s_prefix[b]
    while (b - a > 1) {
        const int m = (a + b) >> 1;
        if (s_prefix[m] <= u) a = m;
        else b = m;
    }
    const int per = (n + kThreads - 1) / kThreads;
    int64_t at = s_prefix[a];
    int i = a * per;
    for (;; i++) {
        const int64_t k = units_of(i);
        if (u < at + k || i + 1 >= n) break;
        at += k;
    }
    *first = at;
    return i;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Transpose an 8 x 8 matrix of 16-bit values held as lane -> (row lane / 4, columns 2 * (lane % 4) ..+1).
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t pack_out(float lo, float hi, bool fp16) {
    uint32_t r;
    if (fp16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float2 widen2(uint32_t x, bool fp16) {
    if (fp16) return __half22float2(*reinterpret_cast<const __half2 *>(&x));
    return make_float2(__uint_as_float(x << 16), __uint_as_float(x & 0xffff0000u));
}

// Queries go into the products as f16 after a power of two has brought their row's largest
// magnitude into [2^14, 2^15): a value keeps all its bits from 2^-28 (fp16; bf16: 2^-31) of the
// row's largest on; a smaller one is off by 2^-39 of the largest at most, below fp32's own rounding of
// a sum that the largest is part of.
// Returns the exponent E with 2^E <= largest (clamped), so that the factor is 2^(14 - E).
__device__ __forceinline__ int row_exponent(float largest) {
    const int e = static_cast<int>(__float_as_uint(largest) >> 23) - 127;
    return e < -100 ? -100 : e;
}
__device__ __forceinline__ float power2(int e) { return __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

// Merge partial results (kv8_merge_kernel in pkv_kv8_decode.cu): worker w's note names a tile of
// `rows` rows that begins with it and how many workers, `stride` apart, hold a piece of it.
int kv8_launch_merge(const AttnParams &p, int32_t head_dim, int rows, int workers, int stride, cudaStream_t s);

template <int kBytes>
__device__ __forceinline__ void cp_async(uint32_t dst, const void *src, bool live) {
    const int n = live ? kBytes : 0;
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kBytes), "r"(n)
                     : "memory");
}
template <int kBytes>
__device__ __forceinline__ void cp_async_full(uint32_t dst, const void *src) {
    if constexpr (kBytes == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
    else
        asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(kBytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Rows of codes in shared memory: a row's 16-byte pieces are permuted by f(token) = (token & 6) ^
// ((token & 1) << 2) (pairs of 64-byte rows: by token >> 1), which makes the fragment reads free of
// bank conflicts: K rows g and g + 1 fall into different halves of the banks, V tokens 2t into
// different quarters.
template <int D>
__device__ __forceinline__ int swizzle(int piece, int token) {
    return D == 64 ? piece ^ ((token >> 1) & 3) : piece ^ (token & 6) ^ ((token & 1) << 2);
}

// Loads one (query, head) row's f16 fragments of a query tile: element pairs of this lane's
// dimensions 64 u + 16 t + 4 i .. + 3 in qb[4 u + i], scaled by 2^(14 - E); returns E.
template <int D>
__device__ __forceinline__ int load_query(uint32_t (&qb)[D / 16][2], const char *row, bool live, int t, bool fp16) {
    uint2 raw[D / 16];
    float largest = 0.f;
#pragma unroll
    for (int j = 0; j < D / 16; j++) {
        raw[j] = make_uint2(0, 0);
        if (live) raw[j] = __ldg(reinterpret_cast<const uint2 *>(row + 2 * (64 * (j / 4) + 16 * t + 4 * (j % 4))));
        const float2 a = widen2(raw[j].x, fp16), b = widen2(raw[j].y, fp16);
        largest = fmaxf(fmaxf(largest, fmaxf(fabsf(a.x), fabsf(a.y))), fmaxf(fabsf(b.x), fabsf(b.y)));
    }
    largest = fmaxf(largest, __shfl_xor_sync(~0u, largest, 1));
    largest = fmaxf(largest, __shfl_xor_sync(~0u, largest, 2));
    const int e = row_exponent(largest);
    const float f = power2(14 - e);
#pragma unroll
    for (int j = 0; j < D / 16; j++) {
        const float2 a = widen2(raw[j].x, fp16), b = widen2(raw[j].y, fp16);
        qb[j][0] = pack_f16(a.x * f, a.y * f);
        qb[j][1] = pack_f16(b.x * f, b.y * f);
    }
    return e;
}

}  // namespace pkv
