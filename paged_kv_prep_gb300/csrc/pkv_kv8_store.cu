// Quantising store into the 8-bit paged cache.
//
// Mathematics.  The tokens of one block stand next to each other in the step's
// slot_mapping; such a run covers the block's offsets from `first` on.  Per
// (block, head): amax = the largest finite |x| of the run,
//   s = max(2^ceil(log2(amax / 448)), the block's scale if first > 0),
//   new lines: code = rne_e4m3(x / s), held lines (offset < first): code =
//   rne_e4m3(code * s_old / s).
// With scales that are powers of two a rescaled code keeps its mantissa, so a
// block that is filled token by token loses nothing but what falls below the
// grid's smallest step (2^-9 of its scale).  The only rounding is that to e4m3.
//
// Bound: HBM (2 bytes read and 1 written per element), or launch latency for a
// decode step.
//
// Layout.  A CTA takes the runs that start among kChunk consecutive tokens, for
// 256 consecutive elements of the K or the V line (one to four heads); a run
// that reaches past the chunk is followed to its end.  A warp moves one
// token's 256 elements with 16 bytes a lane; the chunk's tokens are asked for
// before anything is known about them and stay in registers between the maximum
// and the rounding, while every warp finds the runs by itself (a lane per
// token) and the blocks' scales are on their way.  The maxima of a run meet in
// shared memory as integers (order-free); one barrier stands between them and
// the rounding.
// Measured (16384 tokens, 4096 of them first in their run, 8 heads x 128, bf16;
// 101 MB, floor 15.1 us): 41 us; reading the runs' slots and scales, the two
// barriers and the integer work around eight elements a lane hold it there
// (0.55 instructions issued a cycle).  One search of the runs per segment: 46 us;
// without holding the lines past the chunk in registers: 58 us.
#include <type_traits>

#include "pkv_async.cuh"
#include "pkv_kv8.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 32;
constexpr int kHold = kChunk / kWarps;
constexpr int kSegment = 256;      // elements of a line per CTA

struct StoreParams {
    const char *x[2];              // K, V sources
    int64_t stride[2];             // bytes from token to token
    uint8_t *cache[2];
    float *scale[2];
    const int64_t *slots;
    int64_t num_slots;
    int32_t T, bs, shift, heads, segments;   // shift: log2(bs), -1 if it is not a power of two
    int32_t *err;
};

// Eight bf16 or fp16 values as floats.
template <typename T>
__device__ __forceinline__ float2 widen1(uint32_t w) {
    if constexpr (std::is_same<T, __half>::value) return __half22float2(*reinterpret_cast<const __half2 *>(&w));
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ void widen(uint4 v, float (&f)[8]) {
    const float2 a = widen1<T>(v.x), b = widen1<T>(v.y), c = widen1<T>(v.z), d = widen1<T>(v.w);
    f[0] = a.x;
    f[1] = a.y;
    f[2] = b.x;
    f[3] = b.y;
    f[4] = c.x;
    f[5] = c.y;
    f[6] = d.x;
    f[7] = d.y;
}

// Largest finite magnitude of the pairs' elements, as bits of T in each half (magnitudes order as
// their bits).  Infinities saturate and NaNs pass; neither sets the scale.
template <typename T>
__device__ __forceinline__ uint32_t largest8(uint4 v) {
    constexpr uint32_t kInf = std::is_same<T, __half>::value ? 0x7c00u : 0x7f80u;
    uint32_t a = v.x & 0x7fff7fffu, b = v.y & 0x7fff7fffu, c = v.z & 0x7fff7fffu, d = v.w & 0x7fff7fffu;
    uint32_t m = __vmaxu2(__vmaxu2(a, b), __vmaxu2(c, d));
    if ((m & 0xffffu) >= kInf || (m >> 16) >= kInf) {
        const uint32_t inf = kInf | kInf << 16;
        a &= ~__vcmpgeu2(a, inf);
        b &= ~__vcmpgeu2(b, inf);
        c &= ~__vcmpgeu2(c, inf);
        d &= ~__vcmpgeu2(d, inf);
        m = __vmaxu2(__vmaxu2(a, b), __vmaxu2(c, d));
    }
    return m;
}

template <typename T>
__device__ __forceinline__ uint2 quantise8(uint4 v, float s) {
    float f[8];
    widen<T>(v, f);
    const float r = __frcp_rn(s);       // exact for a power of two: the product is the quotient
#pragma unroll
    for (int i = 0; i < 8; i++) f[i] *= r;
    return make_uint2(pkv::e4m3x2(f[0], f[1]) | (pkv::e4m3x2(f[2], f[3]) << 16),
                      pkv::e4m3x2(f[4], f[5]) | (pkv::e4m3x2(f[6], f[7]) << 16));
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads, 3) kv8_store_kernel(const StoreParams p) {
    constexpr int kLanes = D / 8;              // lanes per head
    constexpr int kHeads = kSegment / D;       // heads per segment
    __shared__ uint32_t s_amax[kChunk][kHeads];
    __shared__ float s_old[kChunk][kHeads];    // the run's block's scales before
    __shared__ int32_t s_first[kChunk];        // the run's smallest offset

    pkv::pdl_wait();
    pkv::pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kChunk;
    // A token's slot (fewer than 2^32) and block; kNone where it is not stored.
    constexpr uint32_t kNone = 0xffffffffu;
    auto slot_of = [&](int64_t t, bool report) {
        if (t < 0 || t >= p.T) return kNone;
        const int64_t s = p.slots[t];
        if (s >= p.num_slots && report && p.err) atomicOr(p.err, PKV_DEVERR_SLOT);
        return s < 0 || s >= p.num_slots ? kNone : static_cast<uint32_t>(s);
    };
    auto block_of = [&](uint32_t s) {
        return s == kNone ? kNone : p.shift >= 0 ? s >> p.shift : s / static_cast<uint32_t>(p.bs);
    };
    uint32_t slot = slot_of(t0 + lane, blockIdx.y == 0 && warp == 0);
    const uint32_t edge = lane == 0 ? slot_of(t0 - 1, false) : kNone;
    const uint32_t beyond = slot_of(t0 + kChunk + lane, false);
    const uint32_t block = block_of(slot);
    uint32_t before = __shfl_up_sync(~0u, block, 1);
    if (lane == 0) before = block_of(edge);
    const bool leader = block != kNone && block != before;
    const uint32_t leaders = __ballot_sync(~0u, leader);
    if (!leaders) return;                                  // the whole CTA: every warp sees the same tokens
    // tokens of a run that starts before the chunk belong to another CTA
    const uint32_t upto = leaders & (0xffffffffu >> (31 - lane));
    if (!upto) slot = kNone;
    const int run = __popc(upto) - 1, runs = __popc(leaders);
    const uint32_t offset = slot - block * static_cast<uint32_t>(p.bs);
    const uint32_t last = __shfl_sync(~0u, slot == kNone ? kNone : block, 31);

    // the chunk's last run goes on past it
    int extra = 0;
    uint32_t extra_first = kNone;                          // smallest offset among them
    if (last != kNone) {
        for (int64_t a = t0 + kChunk; a < p.T; a += 32) {
            const uint32_t s = a == t0 + kChunk ? beyond : slot_of(a + lane, false);
            const uint32_t same = __ballot_sync(~0u, s != kNone && block_of(s) == last);
            const int c = same == ~0u ? 32 : __ffs(~same) - 1;
            if (lane < c) extra_first = min(extra_first, s - last * static_cast<uint32_t>(p.bs));
            extra += c;
            if (c < 32) break;
        }
    }
    for (int y = blockIdx.y; y < 2 * p.segments; y += gridDim.y) {
        const int which = y & 1, seg = y >> 1;
        if (y != static_cast<int>(blockIdx.y)) __syncthreads();   // the round before has left shared memory
        const int e0 = seg * kSegment + lane * 8;              // this lane's first element
        const bool live = e0 < p.heads * D;
        const int hs = lane / kLanes;                          // head within the segment
        const char *src = (which ? p.x[1] : p.x[0]) + 2 * e0;
        const int64_t stride = which ? p.stride[1] : p.stride[0];
        float *const scales = which ? p.scale[1] : p.scale[0];
        uint8_t *const cache = which ? p.cache[1] : p.cache[0];
        auto load = [&](int64_t t, bool there) {
            return live && there ? __ldg(reinterpret_cast<const uint4 *>(src + t * stride)) : make_uint4(0, 0, 0, 0);
        };
        uint4 held[kHold];
#pragma unroll
        for (int i = 0; i < kHold; i++) held[i] = load(t0 + warp + i * kWarps, t0 + warp + i * kWarps < p.T);
        uint4 more[kHold];                                     // of the tokens past the chunk: the first 32
#pragma unroll
        for (int i = 0; i < kHold; i++) more[i] = load(t0 + kChunk + warp + i * kWarps, warp + i * kWarps < extra);

        if (warp == 0) {
            s_first[lane] = p.bs;
#pragma unroll
            for (int h = 0; h < kHeads; h++) s_amax[lane][h] = 0;
            __syncwarp();
            if (slot != kNone) atomicMin(&s_first[run], static_cast<int32_t>(offset));
            if (extra_first != kNone) atomicMin(&s_first[runs - 1], static_cast<int32_t>(extra_first));
            if (leader) {
#pragma unroll
                for (int h = 0; h < kHeads; h++)
                    if (seg * kHeads + h < p.heads)
                        s_old[run][h] = scales[static_cast<int64_t>(block) * p.heads + seg * kHeads + h];
            }
        }
        __syncthreads();

        auto measure = [&](uint4 v, int r) {
            uint32_t m = largest8<T>(v);
#pragma unroll
            for (int o = kLanes / 2; o; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(~0u, m, o));
            const uint32_t top = max(m & 0xffffu, m >> 16);
            if ((lane & (kLanes - 1)) == 0) atomicMax(&s_amax[r][hs], __float_as_uint(widen1<T>(top).x));
        };
#pragma unroll
        for (int i = 0; i < kHold; i++) {
            const int j = warp + i * kWarps;
            if (__shfl_sync(~0u, slot, j) != kNone) measure(held[i], __shfl_sync(~0u, run, j));
        }
#pragma unroll
        for (int i = 0; i < kHold; i++)
            if (warp + i * kWarps < extra) measure(more[i], runs - 1);
        for (int j = warp + kChunk; j < extra; j += kWarps) measure(load(t0 + kChunk + j, true), runs - 1);
        __syncthreads();

        // a run's scale, and how held codes change with it
        auto scale_of = [&](int r, float &ratio) {
            float s = pkv::scale_for(__uint_as_float(s_amax[r][hs]));
            ratio = 1.f;
            if (s_first[r] > 0 && live) {
                const float old = s_old[r][hs];
                if (old >= s) s = old;
                else ratio = old * __frcp_rn(s);   // s is a power of two here
            }
            return s;
        };
        const int64_t line = static_cast<int64_t>(p.heads) * D;
        auto write = [&](uint4 v, float s, uint32_t at) {
            if (live) *reinterpret_cast<uint2 *>(cache + at * line + e0) = quantise8<T>(v, s);
        };
#pragma unroll
        for (int i = 0; i < kHold; i++) {
            const int j = warp + i * kWarps;
            const uint32_t at = __shfl_sync(~0u, slot, j);
            if (at == kNone) continue;
            const int r = __shfl_sync(~0u, run, j);
            float ratio;
            const float s = scale_of(r, ratio);
            write(held[i], s, at);
            if ((leaders >> j) & 1) {
                // the run's first token brings the scale, and the lines that the block already held
                const uint32_t b = __shfl_sync(~0u, block, j);
                if (live && (lane & (kLanes - 1)) == 0) scales[static_cast<int64_t>(b) * p.heads + seg * kHeads + hs] = s;
                if (__any_sync(~0u, ratio != 1.f)) {
                    const int first = s_first[r];
                    for (int o = 0; o < first; o++) {
                        if (ratio == 1.f) continue;
                        uint2 *held_line = reinterpret_cast<uint2 *>(cache + (b * static_cast<int64_t>(p.bs) + o) * line + e0);
                        uint2 c = *held_line;
                        c.x = pkv::requantise4(c.x, ratio);
                        c.y = pkv::requantise4(c.y, ratio);
                        *held_line = c;
                    }
                }
            }
        }
        if (extra) {
            float ratio;
            const float s = scale_of(runs - 1, ratio);
#pragma unroll
            for (int i = 0; i < kHold; i++) {
                const int j = warp + i * kWarps;
                const uint32_t at = __shfl_sync(~0u, beyond, j);
                if (j < extra) write(more[i], s, at);
            }
            for (int j = warp + kChunk; j < extra; j += kWarps)
                write(load(t0 + kChunk + j, true), s, static_cast<uint32_t>(p.slots[t0 + kChunk + j]));
        }
    }
}

template <typename T>
int launch_store(const StoreParams &p, int32_t head_dim, int sms, cudaStream_t s) {
    const int chunks = (p.T + kChunk - 1) / kChunk;
    // about 12 CTAs an SM (four waves); fewer segments per CTA than that would repeat the runs' search
    const int want = (12 * sms + chunks - 1) / chunks;
    const dim3 grid(chunks, want < 2 * p.segments ? want : 2 * p.segments);
    cudaError_t e;
    if (head_dim == 64)
        e = pkv::launch_pdl(kv8_store_kernel<T, 64>, grid, dim3(kThreads), 0, s, p);
    else if (head_dim == 128)
        e = pkv::launch_pdl(kv8_store_kernel<T, 128>, grid, dim3(kThreads), 0, s, p);
    else
        e = pkv::launch_pdl(kv8_store_kernel<T, 256>, grid, dim3(kThreads), 0, s, p);
    PKV_CUDA_TRY(e);
    return PKV_OK;
}

}  // namespace

extern "C" int pkv_kv8_store(const pkv_kv8_cache *cache, const void *k, const void *v,
                             int64_t k_stride_bytes, int64_t v_stride_bytes, int32_t dtype,
                             const int64_t *slot_mapping, int32_t num_tokens, int32_t *d_error,
                             pkv_stream_t stream) {
    int rc = pkv::kv8_check_cache(cache);
    if (rc != PKV_OK) return rc;
    if (num_tokens < 0 || num_tokens >= PKV_MAX_TOKENS || (dtype != PKV_BF16 && dtype != PKV_FP16) ||
        k_stride_bytes < 0 || v_stride_bytes < 0)
        return PKV_ERR_INVALID_ARG;
    if (num_tokens == 0) return PKV_OK;
    if (!k || !v || !slot_mapping) return PKV_ERR_INVALID_ARG;
    const int64_t row = 2LL * cache->num_heads * cache->head_dim;
    if ((k_stride_bytes & 15) || (v_stride_bytes & 15) || (reinterpret_cast<uintptr_t>(k) & 15) ||
        (reinterpret_cast<uintptr_t>(v) & 15))
        return PKV_ERR_ALIGN;
    if (num_tokens > 1 && (k_stride_bytes < row || v_stride_bytes < row)) return PKV_ERR_INVALID_ARG;
    StoreParams p;
    p.x[0] = static_cast<const char *>(k);
    p.x[1] = static_cast<const char *>(v);
    p.stride[0] = k_stride_bytes;
    p.stride[1] = v_stride_bytes;
    p.cache[0] = static_cast<uint8_t *>(cache->k_cache);
    p.cache[1] = static_cast<uint8_t *>(cache->v_cache);
    p.scale[0] = cache->k_scale;
    p.scale[1] = cache->v_scale;
    p.slots = slot_mapping;
    p.num_slots = cache->num_blocks * cache->block_size;
    p.T = num_tokens;
    p.bs = cache->block_size;
    p.shift = (p.bs & (p.bs - 1)) ? -1 : 31 - __builtin_clz(static_cast<unsigned>(p.bs));
    p.heads = cache->num_heads;
    p.segments = static_cast<int32_t>((row / 2 + kSegment - 1) / kSegment);
    p.err = d_error;
    int sms = 0;
    rc = pkv::kv8_sm_count(&sms);
    if (rc != PKV_OK) return rc;
    return dtype == PKV_FP16 ? launch_store<__half>(p, cache->head_dim, sms, pkv::as_stream(stream))
                             : launch_store<__nv_bfloat16>(p, cache->head_dim, sms, pkv::as_stream(stream));
}
