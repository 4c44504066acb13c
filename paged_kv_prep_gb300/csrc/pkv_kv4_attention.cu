// Host side of the attention over the 4-bit paged cache: argument checks, which
// kernels take which requests.
#include <cmath>

#include "pkv_kv4_attention.cuh"

namespace pkv {
namespace {

int64_t workspace_of(int32_t head_dim, int sms) {
    const int64_t a = kv4_decode_workspace(head_dim, sms), b = kv4_prefill_workspace(head_dim, sms);
    return ((a > b ? a : b) + 255) & ~255LL;
}

}  // namespace
}  // namespace pkv

extern "C" {

int pkv_kv4_attention_workspace(int32_t head_dim, int64_t *bytes) {
    if (!bytes || !pkv::kv8_head_dim(head_dim)) return PKV_ERR_INVALID_ARG;
    int sms = 0;
    const int rc = pkv::kv8_sm_count(&sms);
    if (rc != PKV_OK) return rc;
    *bytes = pkv::workspace_of(head_dim, sms);
    return PKV_OK;
}

int pkv_kv4_attention(const pkv_kv4_cache *cache, const void *q, int64_t q_stride_bytes, int32_t dtype,
                      int32_t num_q_heads, const int32_t *block_tables, int32_t table_width,
                      const int32_t *query_start_loc, const int32_t *seq_lens, int32_t n, int32_t num_tokens,
                      float softmax_scale, int32_t window, void *out, int64_t out_stride_bytes, float *lse,
                      void *workspace, int64_t workspace_bytes, int32_t *d_error, pkv_stream_t stream) {
    int rc = pkv::kv4_check_cache(cache);
    if (rc != PKV_OK) return rc;
    if (n < 0 || n > PKV_MAX_BATCH || num_tokens < 0 || num_tokens >= PKV_MAX_TOKENS ||
        (dtype != PKV_BF16 && dtype != PKV_FP16) || num_q_heads < 1 || num_q_heads % cache->num_heads ||
        table_width < 0 || window < 0 || q_stride_bytes < 0 || out_stride_bytes < 0)
        return PKV_ERR_INVALID_ARG;
    // the kernels take the larger of a row's factor and a tiny number, which would hide a NaN
    const float scale_log2 = softmax_scale * pkv::kLog2e * cache->k_unit;
    if (!std::isfinite(scale_log2)) return PKV_ERR_INVALID_ARG;
    const int64_t row = 2LL * num_q_heads * cache->head_dim;
    // (query, head) rows are counted in 32 bits, with room for a last tile
    if (static_cast<int64_t>(num_tokens) * (num_q_heads / cache->num_heads) >= (1LL << 31) - 1024 || row >= (1LL << 31))
        return PKV_ERR_INVALID_ARG;
    if (n == 0 || num_tokens == 0) return PKV_OK;
    if (!q || !out || !query_start_loc || !seq_lens || (table_width > 0 && !block_tables) || !workspace)
        return PKV_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(q) & 15) || (reinterpret_cast<uintptr_t>(out) & 15) || (q_stride_bytes & 15) ||
        (out_stride_bytes & 15) || (reinterpret_cast<uintptr_t>(workspace) & 15))
        return PKV_ERR_ALIGN;
    if (num_tokens > 1 && (q_stride_bytes < row || out_stride_bytes < row)) return PKV_ERR_INVALID_ARG;
    int sms = 0;
    rc = pkv::kv8_sm_count(&sms);
    if (rc != PKV_OK) return rc;
    if (workspace_bytes < pkv::workspace_of(cache->head_dim, sms)) return PKV_ERR_INVALID_ARG;
    pkv::Kv4Params p = {};
    p.q = static_cast<const char *>(q);
    p.q_stride = q_stride_bytes;
    p.out = static_cast<char *>(out);
    p.out_stride = out_stride_bytes;
    p.lse = lse;
    p.kc = static_cast<const uint8_t *>(cache->k_cache);
    p.vc = static_cast<const uint8_t *>(cache->v_cache);
    p.k_sf = static_cast<const uint8_t *>(cache->k_scale);
    p.v_sf = static_cast<const uint8_t *>(cache->v_scale);
    p.v_unit = cache->v_unit;
    p.tables = block_tables;
    p.qsl = query_start_loc;
    p.lens = seq_lens;
    p.num_blocks = cache->num_blocks;
    p.n = n;
    p.T = num_tokens;
    p.set_table(table_width, cache->block_size);
    p.bs = cache->block_size;
    p.Hkv = cache->num_heads;
    p.G = num_q_heads / cache->num_heads;
    p.window = window;
    p.fp16 = dtype == PKV_FP16;
    p.scale_log2 = scale_log2;
    p.meta = static_cast<int4 *>(workspace);
    p.part = reinterpret_cast<float *>(p.meta + pkv::kv8_most_workers(sms));
    p.err = d_error;
    cudaStream_t s = pkv::as_stream(stream);
    // The prefill kernel takes the requests of many rows.  It needs head_dim <= 128 (two accumulators beside two
    // score tiles in TMEM); otherwise the decode kernel's row tiles take everything.  Up to 32 rows, two of the
    // decode kernel's tiles, it would be mostly empty: 96 requests of two to six tokens with five heads a KV head
    // under a window of 4096: 218 us; with the requests of more than 16 rows on the prefill kernel 294 us, of more than 8
    // 374 us.  Where the requests have many rows on average the step has prompt chunks, and the others are single
    // tokens as a rule: the decode kernel then takes what fits its eight-row tiles, which go through the cache
    // faster than sixteen (a step of chunks and decodes 938 us; with up to 32 rows and tiles of sixteen 979 us).
    const bool chunks = static_cast<int64_t>(num_tokens) * p.G > 32LL * n && p.G <= 8;
    const int rows = chunks ? 8 : pkv::kKv4PrefillRows;
    const bool prefill = cache->head_dim <= 128 && num_tokens > n && static_cast<int64_t>(num_tokens - n + 1) * p.G > rows;
    // A warp takes a whole row tile, and no merge follows, where the tables hold at most 64 tokens, or at most 256 and
    // the batch two tiles an SM.  Single tokens, 8 KV heads, whole and cut: tables of 64
    // tokens, 8 requests 9.6 and 11.2 us, 2048 requests 68 and 78; of 256 tokens, 32 requests 18.1 and 13.2, 64 17.8 and
    // 17.9, 128 18.3 and 22.9, 2048 128 and 127; of 512 tokens, 128 requests 29.1 and 27.5, 32 27.6 and 18.7.
    const int64_t most = static_cast<int64_t>(p.W) * p.bs;
    p.whole = most <= 64 || (most <= 256 && static_cast<int64_t>(n) * p.Hkv >= 2 * sms);
    // The prefill kernel takes everything, without a second pair of launches, where the requests have more than 8 rows on
    // average and there is one of them, or no more row tiles of single tokens than SMs, and of 128-token units, by the
    // tables' width, no more than 32 an SM.  8 KV heads, two chunks of 300 tokens and single tokens, alone and with
    // the decode kernel: 16 on 1000 tokens 52 and 61 us, on 4000 82 and 83, on 16000 198 and 160; 32 on 1000 68 and 63, on
    // 4000 120 and 100; a chunk of 256 tokens by itself 29 and 36; eight requests of two to six tokens, five heads a KV head, on
    // up to 2000 tokens 29 and 37, of two to five on up to 8000 with one KV head 31 and 55.
    const int64_t tiles = static_cast<int64_t>(n) * p.Hkv;
    const bool alone = prefill && static_cast<int64_t>(num_tokens) * p.G > 8LL * n &&
                       (n == 1 || (tiles <= sms && tiles * (most / 128 + 1) <= 32LL * sms));
    p.short_rows = alone ? 0 : prefill ? rows : 0x7fffffff;
    // These rules go by the tables' width and by counts that may be padded, since the host knows no lengths.  Tables of
    // 131072 tokens instead of the longest request's: two chunks of 300 tokens beside eight single ones 53 us instead of
    // 45, eight requests of two to six tokens 37 instead of 28, 2048 single tokens on up to 64 tokens 86 instead of 74.
    // Idle requests hide a chunk from `prefill`: one of 60 tokens on a context of 37000 takes 60 us by itself, 220 among
    // 63 of them.  Rows behind the last request do the opposite: 256 single tokens in 512 rows 334 us instead of 220.
    // one 8-row tile holds every request that the decode kernel takes
    const bool one_tile = (num_tokens <= n && p.G <= 8) || (prefill && chunks);
    if (prefill) {
        rc = pkv::kv4_launch_prefill(p, cache->head_dim, sms, s);
        if (rc != PKV_OK || alone) return rc;
    }
    return pkv::kv4_launch_decode(p, cache->head_dim, one_tile, sms, s);
}

}  // extern "C"
