// Shared by the kernels on the 8-bit paged cache: e4m3 conversions, scale
// arithmetic, argument checks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <string.h>

#include "pkv_common.cuh"

namespace pkv {

constexpr float kE4m3Max = 448.f;
constexpr int kMaxHeads = 1024;     // KV heads of a cache
constexpr int kMinScaleExp = -64;   // the store's smallest block scale is 2^-64

// Two floats rounded to e4m3 (to nearest even, saturating at 448; NaN stays NaN): `lo` in the
// low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two e4m3 codes (low byte first) as f16x2: exact, every e4m3 value is an f16 value.
__device__ __forceinline__ uint32_t f16x2_of(uint32_t codes) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(codes)));
    return r;
}

__device__ __forceinline__ float2 floats_of(uint32_t codes) {
    const uint32_t h = f16x2_of(codes);
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// The smallest power of two 2^e >= amax / 448 with e >= -64 (448 = 1.75 * 2^8, so e follows from
// amax's exponent and whether its fraction is above 0.75).  amax is finite and >= 0.
__device__ __forceinline__ float scale_for(float amax) {
    const uint32_t b = __float_as_uint(amax);
    int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u);
    e = e < kMinScaleExp ? kMinScaleExp : e;
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// Requantise four codes from a block scale to a larger one; ratio = old / new <= 1.
__device__ __forceinline__ uint32_t requantise4(uint32_t c, float ratio) {
    const float2 a = floats_of(c & 0xffffu), b = floats_of(c >> 16);
    return e4m3x2(a.x * ratio, a.y * ratio) | (e4m3x2(b.x * ratio, b.y * ratio) << 16);
}

// Thread-block clusters: CTAs in this one, a barrier over them, a value of CTA `rank`.
__device__ __forceinline__ int cluster_size() {
    uint32_t n;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(n));
    return static_cast<int>(n);
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive;" ::: "memory");
    asm volatile("barrier.cluster.wait;" ::: "memory");
}
template <typename T>
__device__ __forceinline__ T cluster_read(const T *at, uint32_t rank) {
    static_assert(sizeof(T) == 4, "32-bit values");
    uint32_t a, v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(a)
                 : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(at))), "r"(rank));
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    T r;
    memcpy(&r, &v, 4);
    return r;
}

inline bool kv8_head_dim(int32_t d) { return d == 64 || d == 128 || d == 256; }

// The cache's own arguments: sizes, pointers, alignment.
inline int kv8_check_cache(const pkv_kv8_cache *c) {
    if (!c) return PKV_ERR_INVALID_ARG;
    if (c->num_blocks < 0 || c->block_size < 1 || c->num_heads < 1 || c->num_heads > kMaxHeads ||
        !kv8_head_dim(c->head_dim) || c->num_blocks > 0x7fffffff ||
        c->num_blocks * c->block_size > 0xffffffffLL)    // slots fit 32 bits
        return PKV_ERR_INVALID_ARG;
    if (c->num_blocks == 0) return PKV_OK;
    if (!c->k_cache || !c->v_cache || !c->k_scale || !c->v_scale) return PKV_ERR_INVALID_ARG;
    const uintptr_t lines = reinterpret_cast<uintptr_t>(c->k_cache) | reinterpret_cast<uintptr_t>(c->v_cache);
    const uintptr_t scales = reinterpret_cast<uintptr_t>(c->k_scale) | reinterpret_cast<uintptr_t>(c->v_scale);
    if ((lines & 15) || (scales & 3)) return PKV_ERR_ALIGN;
    return PKV_OK;
}

// Lets a kernel take `bytes` of dynamic shared memory; asked for once per device (`set` is the
// kernel's own record).
inline int kv8_allow_smem(const void *kernel, int bytes, bool (&set)[64]) {
    int dev = 0;
    PKV_CUDA_TRY(cudaGetDevice(&dev));
    if (dev < 64 && set[dev]) return PKV_OK;
    PKV_CUDA_TRY(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes));
    if (dev < 64) set[dev] = true;
    return PKV_OK;
}

// SMs of the current device (asked once per device).
inline int kv8_sm_count(int *out) {
    int dev = 0;
    PKV_CUDA_TRY(cudaGetDevice(&dev));
    static int cached[64] = {0};
    if (dev >= 0 && dev < 64 && cached[dev]) {
        *out = cached[dev];
        return PKV_OK;
    }
    int n = 0;
    PKV_CUDA_TRY(cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev));
    if (dev >= 0 && dev < 64) cached[dev] = n;
    *out = n;
    return PKV_OK;
}

}  // namespace pkv
