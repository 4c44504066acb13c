// Host side of the attention over the 8-bit paged cache, and the kernel that
// adds up the attention weight each cached token received.
//
// weights[slot] += sum over the step's queries and heads of exp(x - lse): the
// row's lse is known once the attention has run, so a token's weight is a sum
// over rows that one CTA can own.  A CTA takes 64 tokens of a request; its
// warps share out the KV heads, each recomputes K Q^T of its head for all rows
// of the request, and the warps' sums meet in a fixed order.  No atomics unless
// requests share a block: the addition to global memory itself is atomic, so
// that shared blocks lose nothing.
//
// Bound: for single tokens HBM (D bytes of K per token and KV head, the second
// read of K), for chunks the tensor pipe (mma.sync).
#include "pkv_kv8_attention.cuh"

namespace pkv {

int64_t kv8_decode_workspace(int32_t head_dim, int sms);
int kv8_launch_decode(const AttnParams &p, int32_t head_dim, bool one_tile, int sms, cudaStream_t s);
int64_t kv8_prefill_workspace(int32_t head_dim, int sms);
int kv8_launch_prefill(const AttnParams &p, int32_t head_dim, int sms, cudaStream_t s);

namespace {

constexpr int kPrefillRows = 32;

constexpr int kWTokens = 64;
constexpr int kWWarps = 8;

__device__ __forceinline__ int64_t weight_units(const AttnParams &p, const Req &r) {
    if (r.count <= 0) return 0;
    const int lo = r.lo & ~(kWTokens - 1);
    return r.keys > lo ? (r.keys - lo + kWTokens - 1) / kWTokens : 0;
}

template <int D>
__global__ void __launch_bounds__(32 * kWWarps) kv8_weights_kernel(const AttnParams p) {
    constexpr int kThreads = 32 * kWWarps, S = D / 16, kSub = kWTokens / 16, kPieces = D / 64;
    __shared__ int64_t s_prefix[kThreads + 1];
    __shared__ int64_t s_warp[kWWarps];
    __shared__ float s_sum[kWWarps][kWTokens];
    __shared__ int32_t s_block[kWTokens];
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    auto units = [&](int i) { return weight_units(p, request_of(p, i)); };
    const int64_t total = plan_prefix<kThreads>(s_prefix, s_warp, p.n, units);
    const int64_t line = static_cast<int64_t>(p.Hkv) * D;
    const bool fp16 = p.fp16 != 0;
    for (int64_t u = blockIdx.x; u < total; u += gridDim.x) {
        int64_t first;
        const int i = plan_find<kThreads>(s_prefix, p.n, u, units, &first);
        const Req r = request_of(p, i);
        const int32_t *table = p.tables + static_cast<int64_t>(i) * p.W;
        const int s0 = (r.lo & ~(kWTokens - 1)) + static_cast<int>(u - first) * kWTokens;
        if (tid < kWTokens) {
            const int s = s0 + tid;
            s_block[tid] = s >= r.lo && s < r.len ? block_of(p, table, s) : -1;
        }
        __syncthreads();
        // rows that see some token of the tile: query j sees s in (pos_j - window, pos_j], pos_j = len - count + j
        const int back = r.len - r.count;
        const int j0 = max(0, s0 - back);
        const int64_t j1w = p.window > 0 ? static_cast<int64_t>(s0) + kWTokens - 1 + p.window - 1 - back : r.count - 1;
        const int j1 = static_cast<int>(j1w < r.count - 1 ? j1w : r.count - 1);
        const int f0 = j0 * p.G, f1 = (j1 + 1) * p.G;
        float acc[kSub][2];
#pragma unroll
        for (int k = 0; k < kSub; k++) acc[k][0] = acc[k][1] = 0.f;
        int64_t slot[kSub][2];
        uint32_t live = 0;
#pragma unroll
        for (int k = 0; k < kSub; k++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                const int x = 16 * k + g + 8 * h, b = s_block[x];
                slot[k][h] = b >= 0 ? static_cast<int64_t>(b) * p.bs + (s0 + x) % p.bs : 0;
                live |= (b >= 0 ? 1u : 0u) << (2 * k + h);
            }
        for (int head = warp; head < p.Hkv; head += kWWarps) {
            float ks[kSub][2];
#pragma unroll
            for (int k = 0; k < kSub; k++)
#pragma unroll
                for (int h = 0; h < 2; h++)
                    ks[k][h] = (live >> (2 * k + h)) & 1
                                   ? p.ks[static_cast<int64_t>(s_block[16 * k + g + 8 * h]) * p.Hkv + head] : 0.f;
            const uint8_t *kh = p.kc + head * D + 16 * t;
            for (int f8 = f0; f8 < f1; f8 += 8) {
                uint32_t qb[S][2];
                const int f = f8 + g, j = f / p.G;
                const char *row = p.q + static_cast<int64_t>(r.start + j) * p.q_stride +
                                  2 * static_cast<int64_t>(head * p.G + f - j * p.G) * D;
                const int e = load_query<D>(qb, row, f < f1, t, fp16);
                float cf[2], lse[2];
                int pos[2];
#pragma unroll
                for (int c = 0; c < 2; c++) {
                    const int fc = f8 + 2 * t + c, jc = fc / p.G;
                    cf[c] = p.scale_log2 * power2(__shfl_sync(~0u, e, (2 * t + c) * 4) - 14);
                    pos[c] = fc < f1 ? back + jc : -1;
                    lse[c] = fc < f1 ? p.lse[static_cast<int64_t>(r.start + jc) * p.Hkv * p.G + head * p.G + fc - jc * p.G] * kLog2e
                                     : 0.f;
                    if (lse[c] == -INFINITY) pos[c] = -1;      // an empty row gives no weight
                }
#pragma unroll
                for (int k = 0; k < kSub; k++) {
                    float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int c = 0; c < kPieces; c++) {
                        uint4 ka = make_uint4(0, 0, 0, 0), kb = ka;
                        if ((live >> (2 * k)) & 1) ka = __ldg(reinterpret_cast<const uint4 *>(kh + slot[k][0] * line + 64 * c));
                        if ((live >> (2 * k + 1)) & 1) kb = __ldg(reinterpret_cast<const uint4 *>(kh + slot[k][1] * line + 64 * c));
                        const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
                        for (int q = 0; q < 4; q++) {
                            const uint32_t a[4] = {f16x2_of(wa[q]), f16x2_of(wb[q]), f16x2_of(wa[q] >> 16), f16x2_of(wb[q] >> 16)};
                            mma_f16(x, a, qb[4 * c + q][0], qb[4 * c + q][1]);
                        }
                    }
#pragma unroll
                    for (int c = 0; c < 4; c++) {
                        const int h = c >> 1, col = c & 1, s = s0 + 16 * k + g + 8 * h;
                        const bool ok = ((live >> (2 * k + h)) & 1) && s <= pos[col] &&
                                        (p.window <= 0 || s > pos[col] - p.window);
                        if (ok) acc[k][h] += exp2_fast(fmaf(x[c], cf[col] * ks[k][h], -lse[col]));
                    }
                }
            }
        }
#pragma unroll
        for (int k = 0; k < kSub; k++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                float a = acc[k][h];
                a += __shfl_xor_sync(~0u, a, 1);
                a += __shfl_xor_sync(~0u, a, 2);
                if (t == 0) s_sum[warp][16 * k + g + 8 * h] = a;
            }
        __syncthreads();
        if (tid < kWTokens && s_block[tid] >= 0) {
            float a = 0.f;
#pragma unroll
            for (int w = 0; w < kWWarps; w++) a += s_sum[w][tid];
            atomicAdd(p.weights + static_cast<int64_t>(s_block[tid]) * p.bs + (s0 + tid) % p.bs, a);
        }
        __syncthreads();
    }
}

int64_t workspace_of(int32_t head_dim, int sms) {
    const int64_t a = kv8_decode_workspace(head_dim, sms), b = kv8_prefill_workspace(head_dim, sms);
    return a > b ? a : b;
}

int launch_weights(const AttnParams &p, int32_t head_dim, int sms, cudaStream_t s) {
    const dim3 grid(2 * sms), block(32 * kWWarps);
    if (head_dim == 64)
        PKV_CUDA_TRY(launch_pdl(kv8_weights_kernel<64>, grid, block, 0, s, p));
    else if (head_dim == 128)
        PKV_CUDA_TRY(launch_pdl(kv8_weights_kernel<128>, grid, block, 0, s, p));
    else
        PKV_CUDA_TRY(launch_pdl(kv8_weights_kernel<256>, grid, block, 0, s, p));
    return PKV_OK;
}

}  // namespace
}  // namespace pkv

extern "C" {

int pkv_kv8_attention_workspace(int32_t num_heads, int32_t head_dim, int64_t *bytes) {
    if (!bytes || num_heads < 1 || num_heads > 1024 || !pkv::kv8_head_dim(head_dim)) return PKV_ERR_INVALID_ARG;
    int sms = 0;
    const int rc = pkv::kv8_sm_count(&sms);
    if (rc != PKV_OK) return rc;
    *bytes = pkv::workspace_of(head_dim, sms);
    return PKV_OK;
}

int pkv_kv8_attention(const pkv_kv8_cache *cache, const void *q, int64_t q_stride_bytes, int32_t dtype,
                      int32_t num_q_heads, const int32_t *block_tables, int32_t table_width,
                      const int32_t *query_start_loc, const int32_t *seq_lens, int32_t n,
                      int32_t num_tokens, float softmax_scale, int32_t window, void *out,
                      int64_t out_stride_bytes, float *lse, float *weights, void *workspace,
                      int64_t workspace_bytes, int32_t *d_error, pkv_stream_t stream) {
    int rc = pkv::kv8_check_cache(cache);
    if (rc != PKV_OK) return rc;
    if (n < 0 || n > PKV_MAX_BATCH || num_tokens < 0 || num_tokens >= PKV_MAX_TOKENS ||
        (dtype != PKV_BF16 && dtype != PKV_FP16) || num_q_heads < 1 || num_q_heads % cache->num_heads ||
        table_width < 0 || window < 0 || q_stride_bytes < 0 || out_stride_bytes < 0)
        return PKV_ERR_INVALID_ARG;
    const int64_t row = 2LL * num_q_heads * cache->head_dim;
    // (query, head) rows are counted in 32 bits, with room for a last tile
    if (static_cast<int64_t>(num_tokens) * (num_q_heads / cache->num_heads) >= (1LL << 31) - 1024 ||
        row >= (1LL << 31))
        return PKV_ERR_INVALID_ARG;
    if (n == 0 || num_tokens == 0) return PKV_OK;
    if (!q || !out || !query_start_loc || !seq_lens || (table_width > 0 && !block_tables) || !workspace ||
        (weights && !lse))
        return PKV_ERR_INVALID_ARG;
    if ((reinterpret_cast<uintptr_t>(q) & 15) || (reinterpret_cast<uintptr_t>(out) & 15) ||
        (q_stride_bytes & 15) || (out_stride_bytes & 15) || (reinterpret_cast<uintptr_t>(workspace) & 15))
        return PKV_ERR_ALIGN;
    if (num_tokens > 1 && (q_stride_bytes < row || out_stride_bytes < row)) return PKV_ERR_INVALID_ARG;
    int sms = 0;
    rc = pkv::kv8_sm_count(&sms);
    if (rc != PKV_OK) return rc;
    if (workspace_bytes < pkv::workspace_of(cache->head_dim, sms)) return PKV_ERR_INVALID_ARG;
    pkv::AttnParams p = {};
    p.q = static_cast<const char *>(q);
    p.q_stride = q_stride_bytes;
    p.out = static_cast<char *>(out);
    p.out_stride = out_stride_bytes;
    p.lse = lse;
    p.kc = static_cast<const uint8_t *>(cache->k_cache);
    p.vc = static_cast<const uint8_t *>(cache->v_cache);
    p.ks = cache->k_scale;
    p.vs = cache->v_scale;
    p.weights = weights;
    p.tables = block_tables;
    p.qsl = query_start_loc;
    p.lens = seq_lens;
    p.num_blocks = cache->num_blocks;
    p.n = n;
    p.T = num_tokens;
    p.W = table_width;
    p.bs = cache->block_size;
    p.Hkv = cache->num_heads;
    p.G = num_q_heads / cache->num_heads;
    p.window = window;
    p.fp16 = dtype == PKV_FP16;
    p.scale_log2 = softmax_scale * pkv::kLog2e;
    p.short_rows = 0x7fffffff;
    p.meta = static_cast<int4 *>(workspace);
    p.part = reinterpret_cast<float *>(p.meta + static_cast<int64_t>(sms) * 16);
    p.err = d_error;
    cudaStream_t s = pkv::as_stream(stream);
    // The prefill kernel takes the requests with more than kPrefillRows rows.  It needs head_dim <= 128
    // (two accumulators beside two score tiles in TMEM) and 16-token groups that lie in one block;
    // otherwise the decode kernel's row tiles take everything.
    const bool prefill = cache->head_dim <= 128 && p.bs % 16 == 0 &&
                         static_cast<int64_t>(num_tokens - n + 1) * p.G > pkv::kPrefillRows && num_tokens > n;
    p.short_rows = prefill ? pkv::kPrefillRows : 0x7fffffff;
    // one 8-row tile holds every request of a pure decode step
    const bool one_tile = num_tokens <= n && p.G <= 8;
    if (prefill) {
        rc = pkv::kv8_launch_prefill(p, cache->head_dim, sms, s);
        if (rc != PKV_OK) return rc;
    }
    rc = pkv::kv8_launch_decode(p, cache->head_dim, one_tile, sms, s);
    if (rc != PKV_OK || !weights) return rc;
    return pkv::launch_weights(p, cache->head_dim, sms, s);
}

}  // extern "C"
