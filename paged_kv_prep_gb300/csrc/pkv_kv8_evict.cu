// Eviction from the 8-bit paged cache by accumulated attention weight.
//
// Mathematics.  A request of length L with L > budget keeps its first
// `keep_first` tokens, its last `keep_last`, and of those between the
// r = budget - keep_first - keep_last with the largest weights; equal weights
// go to the lower position, NaN counts below every number.  Kept tokens move,
// in order, to positions 0.. of new blocks.  A new block's scale is the
// largest of its tokens' old scales per head and its codes are
// rne_e4m3(code * s_old / s_new); weights move along.  Nothing of the old
// blocks changes, so they may be shared.
//
// Selection: the r-th largest weight by a radix select over order-preserving
// integer keys, eight bits a pass, then one ordered pass in which a token's
// place follows from two running counts (larger ones, equal ones).  A CTA per
// request; bound by the passes' latency.
//
// Copy: a CTA per new block; bound by HBM (4 * line bytes per kept token).
#include "pkv_async.cuh"
#include "pkv_kv8.cuh"

namespace {

constexpr int kSelThreads = 1024;
constexpr int kCopyThreads = 256;
constexpr int kCopyLines = 64;     // lines whose sources a CTA holds at a time

struct EvictParams {
    const uint8_t *kc, *vc;
    uint8_t *kd, *vd;
    float *ks, *vs;
    float *weights;
    const int32_t *tables, *new_tables;
    const int32_t *lens;
    int64_t num_blocks;
    int32_t bs, heads, line;
    int32_t W, W2;
    int32_t budget, first, last;
    int32_t *new_lens, *kept;
    int32_t *err;
};

// Larger weights have larger keys; NaN has key 0, and -0 the key of +0.
__device__ __forceinline__ uint32_t key_of(float w) {
    const uint32_t b = __float_as_uint(w + 0.f);
    if ((b & 0x7fffffffu) > 0x7f800000u) return 0;
    return (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) kv8_select_kernel(const EvictParams p) {
    __shared__ uint32_t s_hist[256];
    __shared__ uint32_t s_bad;
    __shared__ uint32_t s_prefix, s_need;
    __shared__ uint64_t s_warp[kSelThreads / 32];
    pkv::pdl_wait();
    pkv::pdl_trigger();
    const int req = blockIdx.x, tid = threadIdx.x;
    const int lane = tid & 31, warp = tid >> 5;
    const int32_t *table = p.tables + static_cast<int64_t>(req) * p.W;
    const int32_t *fresh = p.new_tables + static_cast<int64_t>(req) * p.W2;
    int32_t *kept = p.kept + static_cast<int64_t>(req) * p.budget;
    const int64_t L64 = p.lens[req];
    const int bs = p.bs;
    if (tid == 0) s_bad = 0;
    __syncthreads();
    const int64_t n64 = L64 < p.budget ? L64 : p.budget;
    uint32_t bad = 0;
    if (L64 < 0 || L64 > static_cast<int64_t>(p.W) * bs || n64 > static_cast<int64_t>(p.W2) * bs)
        bad = PKV_DEVERR_POSITION;
    if (!bad) {
        for (int64_t j = tid; j * bs < L64; j += kSelThreads)
            if (table[j] < 0 || table[j] >= p.num_blocks) bad = PKV_DEVERR_BLOCK;
        for (int64_t j = tid; j * bs < n64; j += kSelThreads)
            if (fresh[j] < 0 || fresh[j] >= p.num_blocks) bad = PKV_DEVERR_BLOCK;
    }
    if (bad) atomicOr(&s_bad, bad);
    __syncthreads();
    if (s_bad) {
        if (tid == 0) {
            p.new_lens[req] = -1;
            if (p.err) atomicOr(p.err, static_cast<int32_t>(s_bad));
        }
        for (int j = tid; j < p.budget; j += kSelThreads) kept[j] = -1;
        return;
    }
    const int L = static_cast<int>(L64), n = static_cast<int>(n64);
    if (tid == 0) p.new_lens[req] = n;
    for (int j = n + tid; j < p.budget; j += kSelThreads) kept[j] = -1;
    if (L <= p.budget) {
        for (int j = tid; j < n; j += kSelThreads) kept[j] = j;
        return;
    }
    auto weight_key = [&](int pos) {
        const int b = pos / bs;
        return key_of(p.weights[static_cast<int64_t>(table[b]) * bs + (pos - b * bs)]);
    };
    const int lo = p.first, hi = L - p.last;           // candidates lo..hi-1
    const int r = p.budget - p.first - p.last;
    for (int j = tid; j < p.first; j += kSelThreads) kept[j] = j;
    for (int j = tid; j < p.last; j += kSelThreads) kept[p.budget - p.last + j] = hi + j;
    if (r == 0) return;
    if (tid == 0) {
        s_prefix = 0;
        s_need = static_cast<uint32_t>(r);
    }
    // the r-th largest key, eight bits at a time from the top
    for (int shift = 24; shift >= 0; shift -= 8) {
        for (int i = tid; i < 256; i += kSelThreads) s_hist[i] = 0;
        __syncthreads();
        const uint32_t prefix = s_prefix;
        const uint32_t above = shift == 24 ? 0 : 0xffffffffu << (shift + 8);
        for (int pos = lo + tid; pos < hi; pos += kSelThreads) {
            const uint32_t k = weight_key(pos);
            if ((k & above) == prefix) atomicAdd(&s_hist[(k >> shift) & 255], 1u);
        }
        __syncthreads();
        if (warp == 0) {
            // lane l holds digits 255 - 8l .. 248 - 8l, largest first
            uint32_t c[8], sum = 0;
#pragma unroll
            for (int i = 0; i < 8; i++) {
                c[i] = s_hist[255 - 8 * lane - i];
                sum += c[i];
            }
            uint32_t incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t u = __shfl_up_sync(~0u, incl, o);
                if (lane >= o) incl += u;
            }
            const uint32_t need = s_need;
            uint32_t seen = incl - sum;
            if (seen < need && need <= incl) {
#pragma unroll
                for (int i = 0; i < 8; i++) {
                    if (seen < need && need <= seen + c[i]) {
                        s_prefix = prefix | (static_cast<uint32_t>(255 - 8 * lane - i) << shift);
                        s_need = need - seen;
                        seen = need;               // found: no later digit matches
                    } else {
                        seen += c[i];
                    }
                }
            }
        }
        __syncthreads();
    }
    const uint32_t pivot = s_prefix, ties = s_need;    // keep every key > pivot and the first `ties` equal ones
    // places in order: larger ones in the low word of the count, equal ones in the high word
    uint64_t base = 0;
    for (int at = lo; at < hi; at += kSelThreads) {
        const int pos = at + tid;
        uint32_t k = 0;
        bool in = pos < hi;
        if (in) k = weight_key(pos);
        const bool gt = in && k > pivot, eq = in && k == pivot;
        const uint32_t bg = __ballot_sync(~0u, gt), be = __ballot_sync(~0u, eq);
        if (lane == 0) s_warp[warp] = static_cast<uint64_t>(__popc(bg)) | (static_cast<uint64_t>(__popc(be)) << 32);
        __syncthreads();
        uint64_t mine = lane < warp ? s_warp[lane] : 0, all = s_warp[lane];
#pragma unroll
        for (int o = 16; o; o >>= 1) {
            mine += __shfl_xor_sync(~0u, mine, o);
            all += __shfl_xor_sync(~0u, all, o);
        }
        const uint32_t below = (1u << lane) - 1;
        const uint64_t before = base + mine;
        const uint32_t g = static_cast<uint32_t>(before) + __popc(bg & below);
        const uint32_t e = static_cast<uint32_t>(before >> 32) + __popc(be & below);
        if (gt || (eq && e < ties)) kept[lo + g + (e < ties ? e : ties)] = pos;
        base += all;
        __syncthreads();
    }
}

// grid (new blocks per request, requests, K and V)
__global__ void __launch_bounds__(kCopyThreads) kv8_copy_kernel(const EvictParams p) {
    __shared__ int64_t s_src[kCopyLines];
    extern __shared__ float s_scale[];                 // [heads]
    pkv::pdl_wait();
    pkv::pdl_trigger();
    const int req = blockIdx.y, tid = threadIdx.x, bs = p.bs;
    const bool is_v = blockIdx.z != 0;
    const int n = p.new_lens[req];
    const int64_t d0 = static_cast<int64_t>(blockIdx.x) * bs;
    if (d0 >= n) return;                               // also a refused request (-1)
    const int lines = n - d0 < bs ? static_cast<int>(n - d0) : bs;
    const int32_t *table = p.tables + static_cast<int64_t>(req) * p.W;
    const int32_t *kept = p.kept + static_cast<int64_t>(req) * p.budget + d0;
    const int64_t block = p.new_tables[static_cast<int64_t>(req) * p.W2 + blockIdx.x];
    const uint8_t *from = is_v ? p.vc : p.kc;
    uint8_t *to = is_v ? p.vd : p.kd;
    float *scale = is_v ? p.vs : p.ks;
    const int heads = p.heads;

    for (int h = tid; h < heads; h += kCopyThreads) s_scale[h] = 0.f;
    __syncthreads();
    for (int i = tid; i < lines * heads; i += kCopyThreads) {
        const int l = i / heads, h = i - l * heads;
        const int64_t b = table[kept[l] / bs];
        // positive floats order as integers
        atomicMax(reinterpret_cast<int *>(&s_scale[h]), __float_as_int(scale[b * heads + h]));
    }
    __syncthreads();
    for (int h = tid; h < heads; h += kCopyThreads) scale[block * heads + h] = s_scale[h];
    const int chunks = p.line / 16, per_head = chunks / heads;
    for (int l0 = 0; l0 < lines; l0 += kCopyLines) {
        const int m = lines - l0 < kCopyLines ? lines - l0 : kCopyLines;
        __syncthreads();
        if (tid < m) {
            const int pos = kept[l0 + tid], b = pos / bs;
            const int64_t src = static_cast<int64_t>(table[b]) * bs + (pos - b * bs);
            s_src[tid] = src;
            if (!is_v) p.weights[block * bs + l0 + tid] = p.weights[src];
        }
        __syncthreads();
        for (int i = tid; i < m * chunks; i += kCopyThreads) {
            const int l = i / chunks, c = i - l * chunks, h = c / per_head;
            const int64_t src = s_src[l];
            uint4 v = *reinterpret_cast<const uint4 *>(from + src * p.line + c * 16);
            const float old = scale[src / bs * heads + h];
            if (old != s_scale[h]) {
                const float ratio = __fdiv_rn(old, s_scale[h]);
                v.x = pkv::requantise4(v.x, ratio);
                v.y = pkv::requantise4(v.y, ratio);
                v.z = pkv::requantise4(v.z, ratio);
                v.w = pkv::requantise4(v.w, ratio);
            }
            *reinterpret_cast<uint4 *>(to + (block * bs + l0 + l) * p.line + c * 16) = v;
        }
    }
}

}  // namespace

extern "C" int pkv_kv8_evict(const pkv_kv8_cache *cache, float *weights,
                             const int32_t *block_tables, int32_t table_width,
                             const int32_t *seq_lens, int32_t n, const int32_t *new_block_tables,
                             int32_t new_table_width, int32_t budget, int32_t keep_first,
                             int32_t keep_last, int32_t *new_seq_lens, int32_t *kept,
                             int32_t *d_error, pkv_stream_t stream) {
    int rc = pkv::kv8_check_cache(cache);
    if (rc != PKV_OK) return rc;
    if (n < 0 || n > PKV_MAX_BATCH || table_width < 1 || new_table_width < 1 || budget < 1 ||
        keep_first < 0 || keep_last < 0 || static_cast<int64_t>(keep_first) + keep_last > budget)
        return PKV_ERR_INVALID_ARG;
    if (n == 0) return PKV_OK;
    if (cache->num_blocks == 0 || !weights || !block_tables || !seq_lens || !new_block_tables ||
        !new_seq_lens || !kept)
        return PKV_ERR_INVALID_ARG;
    EvictParams p;
    p.kc = p.kd = static_cast<uint8_t *>(cache->k_cache);
    p.vc = p.vd = static_cast<uint8_t *>(cache->v_cache);
    p.ks = cache->k_scale;
    p.vs = cache->v_scale;
    p.weights = weights;
    p.tables = block_tables;
    p.new_tables = new_block_tables;
    p.lens = seq_lens;
    p.num_blocks = cache->num_blocks;
    p.bs = cache->block_size;
    p.heads = cache->num_heads;
    p.line = cache->num_heads * cache->head_dim;
    p.W = table_width;
    p.W2 = new_table_width;
    p.budget = budget;
    p.first = keep_first;
    p.last = keep_last;
    p.new_lens = new_seq_lens;
    p.kept = kept;
    p.err = d_error;
    cudaStream_t s = pkv::as_stream(stream);
    PKV_CUDA_TRY(pkv::launch_pdl(kv8_select_kernel, dim3(n), dim3(kSelThreads), 0, s, p));
    const unsigned blocks = static_cast<unsigned>((static_cast<int64_t>(budget) + p.bs - 1) / p.bs);
    PKV_CUDA_TRY(pkv::launch_pdl(kv8_copy_kernel, dim3(blocks, n, 2), dim3(kCopyThreads),
                                 p.heads * sizeof(float), s, p));
    return PKV_OK;
}
