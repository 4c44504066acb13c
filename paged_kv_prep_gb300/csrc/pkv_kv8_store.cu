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
// that reaches past the chunk is followed to its end, so every token belongs
// to one CTA and is read once.  A warp moves one token's 256 elements with 16
// bytes a lane and keeps up to kHold tokens in registers between the maximum
// and the rounding; the maxima of a run meet in shared memory as integers
// (order-free).
#include <type_traits>

#include "pkv_async.cuh"
#include "pkv_kv8.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk = 32;
constexpr int kHold = 8;
constexpr int kSegment = 256;      // elements of a line per CTA

struct StoreParams {
    const char *x[2];              // K, V sources
    int64_t stride[2];             // bytes from token to token
    uint8_t *cache[2];
    float *scale[2];
    const int64_t *slots;
    int64_t num_slots;
    int32_t T, bs, heads, segments;
    int32_t *err;
};

// Eight bf16 or fp16 values as floats.
template <typename T>
__device__ __forceinline__ void widen(const uint4 &v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        float2 p;
        if constexpr (std::is_same<T, __half>::value)
            p = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
        else
            p = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]));
        f[2 * i] = p.x;
        f[2 * i + 1] = p.y;
    }
}

// Largest finite magnitude (infinities saturate and NaNs pass; neither sets the scale).
__device__ __forceinline__ float amax8(const float (&f)[8]) {
    float m = 0.f;
#pragma unroll
    for (int i = 0; i < 8; i++) {
        const float a = fabsf(f[i]);
        m = fmaxf(m, a < INFINITY ? a : 0.f);
    }
    return m;
}

template <typename T>
__device__ __forceinline__ uint2 quantise8(const uint4 &v, float s) {
    float f[8];
    widen<T>(v, f);
    if ((__float_as_uint(s) & 0x7fffffu) == 0) {   // a power of two: the product is the quotient
        const float r = 1.f / s;
#pragma unroll
        for (int i = 0; i < 8; i++) f[i] *= r;
    } else {
#pragma unroll
        for (int i = 0; i < 8; i++) f[i] = __fdiv_rn(f[i], s);
    }
    return make_uint2(pkv::e4m3x2(f[0], f[1]) | (pkv::e4m3x2(f[2], f[3]) << 16),
                      pkv::e4m3x2(f[4], f[5]) | (pkv::e4m3x2(f[6], f[7]) << 16));
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) kv8_store_kernel(const StoreParams p) {
    constexpr int kLanes = D / 8;              // lanes per head
    constexpr int kHeads = kSegment / D;       // heads per segment
    __shared__ int64_t s_slot[kChunk];         // -1: not stored
    __shared__ int64_t s_block[kChunk];        // of run r
    __shared__ int32_t s_first[kChunk];        // of run r: smallest offset
    __shared__ uint32_t s_amax[kChunk][kHeads];
    __shared__ float s_new[kChunk][kHeads];
    __shared__ float s_ratio[kChunk][kHeads];
    __shared__ uint32_t s_leaders;
    __shared__ int32_t s_extra;

    pkv::pdl_wait();
    pkv::pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int which = blockIdx.y & 1, seg = blockIdx.y >> 1;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * kChunk;
    const int64_t bs = p.bs;

    // the chunk's runs
    if (warp == 0) {
        const int64_t t = t0 + lane;
        int64_t slot = -1, block = -1;
        if (t < p.T) {
            slot = p.slots[t];
            if (slot >= p.num_slots) {
                if (p.err && blockIdx.y == 0) atomicOr(p.err, PKV_DEVERR_SLOT);
                slot = -1;
            }
            if (slot < 0) slot = -1;
            else block = slot / bs;
        }
        int64_t before = __shfl_up_sync(~0u, block, 1);
        if (lane == 0) {
            before = -1;
            if (t > 0) {
                const int64_t s = p.slots[t - 1];
                if (s >= 0 && s < p.num_slots) before = s / bs;
            }
        }
        const uint32_t leaders = __ballot_sync(~0u, block >= 0 && block != before);
        // tokens of a run that starts before the chunk belong to another CTA
        const uint32_t upto = leaders & (0xffffffffu >> (31 - lane));
        if (!upto) slot = -1;
        s_slot[lane] = slot;
        if ((leaders >> lane) & 1) s_block[__popc(upto) - 1] = block;
        s_first[lane] = p.bs;
        // the chunk's last run goes on past it
        const int64_t last = __shfl_sync(~0u, slot >= 0 ? block : -1, 31);
        int32_t extra = 0;
        if (last >= 0) {
            for (int64_t a = t0 + kChunk; a < p.T; a += 32) {
                const int64_t u = a + lane;
                bool same = false;
                if (u < p.T) {
                    const int64_t s = p.slots[u];
                    same = s >= 0 && s < p.num_slots && s / bs == last;
                }
                const uint32_t b = __ballot_sync(~0u, same);
                const int c = b == ~0u ? 32 : __ffs(~b) - 1;
                extra += c;
                if (c < 32) break;
            }
        }
        if (lane == 0) {
            s_leaders = leaders;
            s_extra = extra;
        }
    }
    for (int i = threadIdx.x; i < kChunk * kHeads; i += kThreads) (&s_amax[0][0])[i] = 0;
    __syncthreads();
    const uint32_t leaders = s_leaders;
    if (!leaders) return;
    const int runs = __popc(leaders);
    const int count = kChunk + s_extra;

    const int e0 = seg * kSegment + lane * 8;              // this lane's first element
    const bool live = e0 < p.heads * D;
    const int hs = lane / kLanes;                          // head within the segment
    const char *src = p.x[which] + 2 * e0;
    uint8_t *cache = p.cache[which];
    const int64_t line = static_cast<int64_t>(p.heads) * D;

    // run and slot of the j-th token
    auto place = [&](int j, int &run, int64_t &slot) {
        if (j < kChunk) {
            slot = s_slot[j];
            run = __popc(leaders & (0xffffffffu >> (31 - j))) - 1;
        } else {
            slot = p.slots[t0 + j];
            run = runs - 1;
        }
        return slot >= 0;
    };
    auto load = [&](int j) {
        return live ? __ldg(reinterpret_cast<const uint4 *>(src + (t0 + j) * p.stride[which]))
                    : make_uint4(0, 0, 0, 0);
    };
    auto measure = [&](const uint4 &v, int run, int64_t slot) {
        float f[8];
        widen<T>(v, f);
        float m = amax8(f);
#pragma unroll
        for (int o = kLanes / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
        if ((lane & (kLanes - 1)) == 0) atomicMax(&s_amax[run][hs], __float_as_uint(m));
        if (lane == 0) atomicMin(&s_first[run], static_cast<int32_t>(slot - s_block[run] * bs));
    };

    uint4 held[kHold];
    int64_t slot[kHold];
    int run[kHold];
#pragma unroll
    for (int i = 0; i < kHold; i++) {
        const int j = warp + i * kWarps;
        slot[i] = -1;
        run[i] = 0;
        if (j < count && place(j, run[i], slot[i])) held[i] = load(j);
    }
#pragma unroll
    for (int i = 0; i < kHold; i++)
        if (slot[i] >= 0) measure(held[i], run[i], slot[i]);
    for (int j = warp + kHold * kWarps; j < count; j += kWarps) {   // blocks of more than 32 tokens
        int r;
        int64_t s;
        if (place(j, r, s)) measure(load(j), r, s);
    }
    __syncthreads();

    // the runs' scales
    for (int i = threadIdx.x; i < runs * kHeads; i += kThreads) {
        const int r = i / kHeads, h = i % kHeads;
        if (seg * kHeads + h < p.heads) {
            float *at = p.scale[which] + s_block[r] * p.heads + seg * kHeads + h;
            float s = pkv::scale_for(__uint_as_float(s_amax[r][h])), ratio = 1.f;
            if (s_first[r] > 0) {
                const float old = *at;
                if (old >= s) s = old;
                else ratio = old / s;
            }
            *at = s;
            s_new[r][h] = s;
            s_ratio[r][h] = ratio;
        }
    }
    __syncthreads();

    auto write = [&](const uint4 &v, int r, int64_t s) {
        if (live)
            *reinterpret_cast<uint2 *>(cache + s * line + e0) = quantise8<T>(v, s_new[r][hs]);
    };
#pragma unroll
    for (int i = 0; i < kHold; i++)
        if (slot[i] >= 0) write(held[i], run[i], slot[i]);
    for (int j = warp + kHold * kWarps; j < count; j += kWarps) {
        int r;
        int64_t s;
        if (place(j, r, s)) write(load(j), r, s);
    }
    // lines that the blocks already held, where the scale grew
    for (int r = 0; r < runs; r++) {
        const int first = s_first[r];
        if (first == 0) continue;
        const float ratio = live ? s_ratio[r][hs] : 1.f;
        if (!__any_sync(~0u, ratio != 1.f)) continue;
        for (int o = warp; o < first; o += kWarps) {
            if (ratio == 1.f) continue;
            uint2 *at = reinterpret_cast<uint2 *>(cache + (s_block[r] * bs + o) * line + e0);
            uint2 c = *at;
            c.x = pkv::requantise4(c.x, ratio);
            c.y = pkv::requantise4(c.y, ratio);
            *at = c;
        }
    }
}

template <typename T>
int launch_store(const StoreParams &p, int32_t head_dim, cudaStream_t s) {
    const dim3 grid((p.T + kChunk - 1) / kChunk, 2 * p.segments);
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
    p.heads = cache->num_heads;
    p.segments = static_cast<int32_t>((row / 2 + kSegment - 1) / kSegment);
    p.err = d_error;
    return dtype == PKV_FP16 ? launch_store<__half>(p, cache->head_dim, pkv::as_stream(stream))
                             : launch_store<__nv_bfloat16>(p, cache->head_dim, pkv::as_stream(stream));
}
