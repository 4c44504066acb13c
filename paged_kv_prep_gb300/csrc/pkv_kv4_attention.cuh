// Pieces shared by the attention kernels on the 4-bit paged cache.
#pragma once

#include "pkv_kv4.cuh"
#include "pkv_kv8_attention.cuh"

namespace pkv {

// The 8-bit cache's parameters (its scales unused; scale_log2 holds the keys' unit too) and the scales.
struct Kv4Params : AttnParams {
    const uint8_t *k_sf, *v_sf;        // e4m3, a byte for each 16 elements
    float v_unit;
};

// Requests with more (query, head) rows than this take the prefill kernel.
constexpr int kKv4PrefillRows = 32;

// Merge partial results: worker w's note names a tile of `rows` rows (8, 16 or 256) that begins with it and how many
// workers, `stride` apart, hold a piece of it.
int kv4_launch_merge(const AttnParams &p, int32_t head_dim, int rows, int workers, int stride, int sms, cudaStream_t s);
int64_t kv4_decode_workspace(int32_t head_dim, int sms);
int64_t kv4_prefill_workspace(int32_t head_dim, int sms);
int kv4_launch_decode(const Kv4Params &p, int32_t head_dim, bool one_tile, int sms, cudaStream_t s);
int kv4_launch_prefill(const Kv4Params &p, int32_t head_dim, int sms, cudaStream_t s);

}  // namespace pkv
