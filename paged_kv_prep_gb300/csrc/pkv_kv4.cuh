// Shared by the kernels on the 4-bit paged cache: e2m1 conversions, where a
// block's codes and scales lie, argument checks.
#pragma once

#include "pkv_kv8.cuh"

namespace pkv {

// Eight e2m1 codes (low four bits first) as four f16x2: exact.
__device__ __forceinline__ void f16_of_e2m1x8(uint32_t codes, uint32_t (&h)[4]) {
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "mov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
        "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
        "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(codes));
}

// Eight floats rounded to e2m1 (to nearest even, saturating at 6), the first in the low four bits.
__device__ __forceinline__ uint32_t e2m1x8(const float (&x)[8]) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(r)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return r;
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Both halves of an f16x2 in both places.
__device__ __forceinline__ uint32_t low_twice(uint32_t h) { return __byte_perm(h, h, 0x1010); }
__device__ __forceinline__ uint32_t high_twice(uint32_t h) { return __byte_perm(h, h, 0x3232); }

// The cache's own arguments: sizes, pointers, alignment.
inline int kv4_check_cache(const pkv_kv4_cache *c) {
    if (!c) return PKV_ERR_INVALID_ARG;
    if (c->num_blocks < 0 || c->block_size < 1 || c->block_size % 16 || c->num_heads < 1 || c->num_heads > kMaxHeads ||
        !kv8_head_dim(c->head_dim) || c->num_blocks > 0x7fffffff ||
        c->num_blocks * c->block_size > 0xffffffffLL)        // slots fit 32 bits
        return PKV_ERR_INVALID_ARG;
    if (!(c->k_unit >= 0x1p-64f && c->k_unit <= 0x1p64f && c->v_unit >= 0x1p-64f && c->v_unit <= 0x1p64f))
        return PKV_ERR_INVALID_ARG;
    if (c->num_blocks == 0) return PKV_OK;
    if (!c->k_cache || !c->v_cache || !c->k_scale || !c->v_scale) return PKV_ERR_INVALID_ARG;
    const uintptr_t all = reinterpret_cast<uintptr_t>(c->k_cache) | reinterpret_cast<uintptr_t>(c->v_cache) |
                          reinterpret_cast<uintptr_t>(c->k_scale) | reinterpret_cast<uintptr_t>(c->v_scale);
    return all & 15 ? PKV_ERR_ALIGN : PKV_OK;
}

}  // namespace pkv
