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
// integer keys in three passes of 11, 11 and 10 bits, then one ordered pass in
// which a token's place follows from two running counts (larger ones, equal
// ones).  A request is one CTA's, or a cluster's of eight where tables are
// long; the keys stay in shared memory after the first pass, and the clusters'
// histograms and counts meet through distributed shared memory.  Bound by the
// passes' latency.
//
// Copy: a CTA per new block moves its K and V lines; the lines are on their way
// before the new scales are known.  Bound by HBM (4 * line bytes per kept
// token): 465 MB for 64 requests in 82 us, 5.7 TB/s, 85 % of the measured copy
// rate.
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

template <int kCluster>
__device__ __forceinline__ void sync_all() {
    if constexpr (kCluster == 1) {
        __syncthreads();
    } else {
        pkv::cluster_sync();
    }
}

// One cluster of kCluster CTAs per request; `cap` keys fit the dynamic shared memory.
template <int kCluster>
__global__ void __launch_bounds__(kSelThreads) kv8_select_kernel(const EvictParams p, int cap) {
    constexpr int kBins = 2048, kWarps = kSelThreads / 32;
    extern __shared__ uint32_t s_key[];
    __shared__ uint32_t s_hist[2][kBins];              // two, so that a pass clears while others still read
    __shared__ uint32_t s_bad;
    __shared__ uint32_t s_digit, s_before;
    __shared__ uint32_t s_gt[kWarps + 1], s_eq[kWarps + 1];   // by warp; the last: the CTA's totals
    __shared__ uint32_t s_sum[kWarps];
    pkv::pdl_wait();
    pkv::pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int req = blockIdx.x / kCluster, rank = blockIdx.x % kCluster, all = rank * kSelThreads + tid;
    constexpr int kAll = kCluster * kSelThreads;
    const int32_t *table = p.tables + static_cast<int64_t>(req) * p.W;
    const int32_t *fresh = p.new_tables + static_cast<int64_t>(req) * p.W2;
    int32_t *kept = p.kept + static_cast<int64_t>(req) * p.budget;
    const int64_t L64 = p.lens[req];
    const int bs = p.bs;
    if (tid == 0) s_bad = 0;
    for (int i = tid; i < 2 * kBins; i += kSelThreads) (&s_hist[0][0])[i] = 0;
    __syncthreads();
    const int64_t n64 = L64 < p.budget ? L64 : p.budget;
    uint32_t bad = 0;
    if (L64 < 0 || L64 > static_cast<int64_t>(p.W) * bs || n64 > static_cast<int64_t>(p.W2) * bs)
        bad = PKV_DEVERR_POSITION;
    if (!bad) {
        for (int64_t j = all; j * bs < L64; j += kAll)
            if (table[j] < 0 || table[j] >= p.num_blocks) bad = PKV_DEVERR_BLOCK;
        for (int64_t j = all; j * bs < n64; j += kAll)
            if (fresh[j] < 0 || fresh[j] >= p.num_blocks) bad = PKV_DEVERR_BLOCK;
    }
    if (bad) atomicOr(&s_bad, bad);
    sync_all<kCluster>();
    bad = 0;
#pragma unroll
    for (int c = 0; c < kCluster; c++) bad |= pkv::cluster_read(&s_bad, c);
    if (bad) {
        if (all == 0) {
            p.new_lens[req] = -1;
            if (p.err) atomicOr(p.err, static_cast<int32_t>(bad));
        }
        for (int j = all; j < p.budget; j += kAll) kept[j] = -1;
        sync_all<kCluster>();                          // nobody leaves while its memory is read
        return;
    }
    const int L = static_cast<int>(L64), n = static_cast<int>(n64);
    if (all == 0) p.new_lens[req] = n;
    for (int j = n + all; j < p.budget; j += kAll) kept[j] = -1;
    const int lo = p.first, hi = L - p.last;           // candidates lo..hi-1
    const int r = p.budget - p.first - p.last;
    if (L <= p.budget) {
        for (int j = all; j < n; j += kAll) kept[j] = j;
    } else {
        for (int j = all; j < p.first; j += kAll) kept[j] = j;
        for (int j = all; j < p.last; j += kAll) kept[p.budget - p.last + j] = hi + j;
    }
    if (L <= p.budget || r == 0) {
        sync_all<kCluster>();
        return;
    }
    // this CTA's candidates, a stretch per warp
    const int stretch = 32 * ((hi - lo + kAll - 1) / kAll);
    const int begin = lo + (rank * kWarps + warp) * stretch;
    const int mine = min(max(hi - begin, 0), stretch);
    const bool hold = stretch * kWarps <= cap;
    uint32_t *keys = s_key + warp * stretch;
    auto weight_key = [&](int i) {
        const int pos = begin + i, b = pos / bs;
        return key_of(p.weights[static_cast<int64_t>(table[b]) * bs + (pos - b * bs)]);
    };
    uint32_t prefix = 0, need = static_cast<uint32_t>(r);
    // the r-th largest key, from the top digit down
#pragma unroll 1
    for (int pass = 0; pass < 3; pass++) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
        uint32_t *hist = s_hist[pass & 1];
        const uint32_t above = pass == 0 ? 0u : 0xffffffffu << (pass == 1 ? 21 : 10);
        for (int i = lane; i < mine; i += 32) {
            uint32_t k;
            if (pass > 0 && hold) {
                k = keys[i];
            } else {
                k = weight_key(i);
                if (hold) keys[i] = k;
            }
            if ((k & above) == prefix) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1u);
        }
        sync_all<kCluster>();
        // thread t holds digits bins-1 - 2t and the one below it, largest first
        uint32_t c0 = 0, c1 = 0;
        const int d0 = bins - 1 - 2 * tid;
        if (d0 > 0) {
#pragma unroll
            for (int c = 0; c < kCluster; c++) {
                c0 += pkv::cluster_read(&hist[d0], c);
                c1 += pkv::cluster_read(&hist[d0 - 1], c);
            }
        }
        uint32_t incl = c0 + c1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t u = __shfl_up_sync(~0u, incl, o);
            if (lane >= o) incl += u;
        }
        if (lane == 31) s_sum[warp] = incl;
        __syncthreads();
        uint32_t base = lane < warp ? s_sum[lane] : 0;
#pragma unroll
        for (int o = 16; o; o >>= 1) base += __shfl_xor_sync(~0u, base, o);
        incl += base;
        const uint32_t before = incl - c0 - c1;
        if (before < need && need <= incl) {           // one thread
            const bool second = before + c0 < need;
            s_digit = static_cast<uint32_t>(d0 - second);
            s_before = before + (second ? c0 : 0);
        }
        // the other histogram is free: everyone is past its last reading
        for (int i = tid; i < kBins; i += kSelThreads) s_hist[(pass & 1) ^ 1][i] = 0;
        __syncthreads();
        prefix |= s_digit << shift;
        need -= s_before;
    }
    const uint32_t pivot = prefix, ties = need;        // keep every key > pivot and the first `ties` equal ones
    // places in order: counts of larger and equal keys before each stretch
    uint32_t gt = 0, eq = 0;
    for (int i = lane; i < mine; i += 32) {
        const uint32_t k = hold ? keys[i] : weight_key(i);
        gt += k > pivot;
        eq += k == pivot;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        gt += __shfl_xor_sync(~0u, gt, o);
        eq += __shfl_xor_sync(~0u, eq, o);
    }
    if (lane == 0) {
        s_gt[warp] = gt;
        s_eq[warp] = eq;
    }
    __syncthreads();
    uint32_t g = lane < warp ? s_gt[lane] : 0, e = lane < warp ? s_eq[lane] : 0, ag = s_gt[lane], ae = s_eq[lane];
#pragma unroll
    for (int o = 16; o; o >>= 1) {
        g += __shfl_xor_sync(~0u, g, o);
        e += __shfl_xor_sync(~0u, e, o);
        ag += __shfl_xor_sync(~0u, ag, o);
        ae += __shfl_xor_sync(~0u, ae, o);
    }
    if (tid == 0) {
        s_gt[kWarps] = ag;
        s_eq[kWarps] = ae;
    }
    sync_all<kCluster>();
#pragma unroll
    for (int c = 0; c + 1 < kCluster; c++)
        if (c < rank) {
            g += pkv::cluster_read(&s_gt[kWarps], c);
            e += pkv::cluster_read(&s_eq[kWarps], c);
        }
    const uint32_t below = (1u << lane) - 1;
    for (int i0 = 0; i0 < mine; i0 += 32) {
        const int i = i0 + lane;
        uint32_t k = 0;
        if (i < mine) k = hold ? keys[i] : weight_key(i);
        const uint32_t bg = __ballot_sync(~0u, i < mine && k > pivot), be = __ballot_sync(~0u, i < mine && k == pivot);
        const uint32_t here = e + __popc(be & below);
        const bool is_gt = (bg >> lane) & 1, is_eq = (be >> lane) & 1;
        if (is_gt || (is_eq && here < ties)) kept[lo + g + __popc(bg & below) + (here < ties ? here : ties)] = begin + i;
        g += __popc(bg);
        e += __popc(be);
    }
    sync_all<kCluster>();                              // nobody leaves while its memory is read
}

// grid (new blocks per request, at most the new tables' width; requests)
constexpr int kCopyHold = 4;                           // 16-byte pieces of K (and of V) that a thread holds

__global__ void __launch_bounds__(kCopyThreads, 4) kv8_copy_kernel(const EvictParams p, int chunk_shift, int head_shift) {
    __shared__ uint32_t s_src[kCopyLines];             // slot and block that a line comes from
    __shared__ int32_t s_block[kCopyLines];
    extern __shared__ float s_scale[];                 // [2][heads]
    pkv::pdl_wait();
    pkv::pdl_trigger();
    const int req = blockIdx.y, tid = threadIdx.x, bs = p.bs, heads = p.heads;
    const int64_t d0 = static_cast<int64_t>(blockIdx.x) * bs;
    // what the block is made from is asked for together: its lines' old positions, its new id
    const int first = d0 + tid < p.budget && tid < kCopyLines ? p.kept[static_cast<int64_t>(req) * p.budget + d0 + tid] : -1;
    const int64_t block = p.new_tables[static_cast<int64_t>(req) * p.W2 + blockIdx.x];
    const int n = p.new_lens[req];
    if (d0 >= n) return;                               // also a refused request (-1)
    const int lines = n - d0 < bs ? static_cast<int>(n - d0) : bs;
    const int32_t *table = p.tables + static_cast<int64_t>(req) * p.W;
    const int32_t *kept = p.kept + static_cast<int64_t>(req) * p.budget + d0;
    const int chunks = p.line / 16;                    // a head has 2^head_shift of them

    for (int h = tid; h < 2 * heads; h += kCopyThreads) s_scale[h] = 0.f;
    for (int l0 = 0; l0 < lines; l0 += kCopyLines) {
        const int m = lines - l0 < kCopyLines ? lines - l0 : kCopyLines;
        __syncthreads();
        if (tid < m) {
            const int pos = l0 == 0 ? first : kept[l0 + tid], b = pos / bs;
            const int32_t id = table[b];
            const uint32_t src = static_cast<uint32_t>(id) * static_cast<uint32_t>(bs) + static_cast<uint32_t>(pos - b * bs);
            s_src[tid] = src;
            s_block[tid] = id;
            p.weights[block * bs + l0 + tid] = p.weights[src];
        }
        __syncthreads();
        // the first round's pieces and their scales are on their way before the new scales are known
        const int count = m * chunks;
        for (int i0 = 0; i0 < count; i0 += kCopyThreads * kCopyHold) {
            uint4 kv[kCopyHold][2];
            float old[kCopyHold][2];
#pragma unroll
            for (int u = 0; u < kCopyHold; u++) {
                const int i = i0 + u * kCopyThreads + tid;
                if (i < count) {
                    const int l = chunk_shift >= 0 ? i >> chunk_shift : i / chunks, c = i - l * chunks;
                    const int64_t from = static_cast<int64_t>(s_src[l]) * p.line + c * 16;
                    const int64_t at = static_cast<int64_t>(s_block[l]) * heads + (c >> head_shift);
                    kv[u][0] = __ldg(reinterpret_cast<const uint4 *>(p.kc + from));
                    kv[u][1] = __ldg(reinterpret_cast<const uint4 *>(p.vc + from));
                    old[u][0] = p.ks[at];
                    old[u][1] = p.vs[at];
                }
            }
            if (l0 == 0 && i0 == 0) {
                // positive floats order as integers
                for (int i = tid; i < lines * heads; i += kCopyThreads) {
                    const int l = i / heads, h = i - l * heads;
                    const int64_t b = l < kCopyLines ? s_block[l] : table[kept[l] / bs], at = b * heads + h;
                    atomicMax(reinterpret_cast<int *>(&s_scale[h]), __float_as_int(p.ks[at]));
                    atomicMax(reinterpret_cast<int *>(&s_scale[heads + h]), __float_as_int(p.vs[at]));
                }
                __syncthreads();
                for (int h = tid; h < heads; h += kCopyThreads) {
                    p.ks[block * heads + h] = s_scale[h];
                    p.vs[block * heads + h] = s_scale[heads + h];
                }
            }
#pragma unroll
            for (int u = 0; u < kCopyHold; u++) {
                const int i = i0 + u * kCopyThreads + tid;
                if (i < count) {
                    const int l = chunk_shift >= 0 ? i >> chunk_shift : i / chunks, c = i - l * chunks, h = c >> head_shift;
                    const int64_t to = (block * bs + l0 + l) * p.line + c * 16;
#pragma unroll
                    for (int w = 0; w < 2; w++) {
                        const float now = s_scale[w * heads + h];
                        uint4 v = kv[u][w];
                        if (old[u][w] != now) {
                            const float ratio = old[u][w] * __frcp_rn(now);    // exact between powers of two
                            v.x = pkv::requantise4(v.x, ratio);
                            v.y = pkv::requantise4(v.y, ratio);
                            v.z = pkv::requantise4(v.z, ratio);
                            v.w = pkv::requantise4(v.w, ratio);
                        }
                        *reinterpret_cast<uint4 *>((w ? p.vd : p.kd) + to) = v;
                    }
                }
            }
        }
    }
}

constexpr int kSelCap = 16384;                         // keys held per CTA: 64 KB

template <int kCluster>
int launch_select(const EvictParams &p, int n, cudaStream_t s) {
    static bool set[64] = {false};
    const int rc = pkv::kv8_allow_smem(reinterpret_cast<const void *>(kv8_select_kernel<kCluster>), kSelCap * 4, set);
    if (rc != PKV_OK) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(n) * kCluster);
    cfg.blockDim = dim3(kSelThreads);
    // a CTA holds what its share of the longest table row needs, kSelCap at most
    const int64_t share = (static_cast<int64_t>(p.W) * p.bs + kCluster * kSelThreads - 1) / (kCluster * kSelThreads) * kSelThreads;
    const int cap = share < kSelCap ? static_cast<int>(share) : kSelCap;
    cfg.dynamicSmemBytes = static_cast<size_t>(cap) * 4;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = kCluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kCluster == 1 ? 1 : 2;
    PKV_CUDA_TRY(cudaLaunchKernelEx(&cfg, kv8_select_kernel<kCluster>, p, cap));
    return PKV_OK;
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
    // Eight CTAs share a request where tables reach past 16384 tokens (one CTA holds that many keys):
    // four requests of up to 131072 tokens take 33 us so, 195 us with a CTA each; 64 requests of up to
    // 8192 tokens take 16 us with a CTA each.  The host knows no lengths, so many short requests in wide tables
    // get a cluster each as well: 256 requests of up to 8192 tokens take 603 us in tables of 131072 tokens,
    // 344 in tables of 8192 (the copy included).
    rc = static_cast<int64_t>(p.W) * p.bs > kSelCap ? launch_select<8>(p, n, s) : launch_select<1>(p, n, s);
    if (rc != PKV_OK) return rc;
    // No request fills more blocks than the budget needs, than its new table names or than its old one
    // named; with that the copy's reads of new_block_tables stay in their row.
    int64_t blocks = (static_cast<int64_t>(budget) + p.bs - 1) / p.bs;
    blocks = blocks < p.W2 ? blocks : p.W2;
    blocks = blocks < p.W ? blocks : p.W;
    const int chunks = p.line / 16;
    const int chunk_shift = (chunks & (chunks - 1)) ? -1 : 31 - __builtin_clz(static_cast<unsigned>(chunks));
    const int head_shift = cache->head_dim == 64 ? 2 : cache->head_dim == 128 ? 3 : 4;
    PKV_CUDA_TRY(pkv::launch_pdl(kv8_copy_kernel, dim3(static_cast<unsigned>(blocks), n), dim3(kCopyThreads), 2 * p.heads * sizeof(float), s, p,
                                 chunk_shift, head_shift));
    return PKV_OK;
}
