// Verification of drafted tokens against the target's probabilities, from given
// random numbers.
//
// Mathematics.  Draft j stands while u_j q_j(x_j) < p_j(x_j) (the product of two fp32
// numbers is exact in fp64).  The next token is drawn by inverting the running sum
// of w = max(0, p - q) at the first rejected draft, or of w = p: the first token whose
// running sum exceeds floor(u total).  Sums are whole numbers: round(w 2^40), put
// together from the two roundings h = round(w 2^20) and round((w 2^20 - h) 2^20), each made by
// adding 2^23 (1.5 2^23) in fp32, whose low bits are then the integer.  Integer sums are the same in
// any order, so one pass over the row split over a cluster gives the sequential answer.
//
// Bound: HBM, one row of p (and of q where a draft was rejected) per request.
//
// Layout.  A cluster of one to eight CTAs takes a request; every warp of it owns one stretch of
// the row and walks it with 16-byte loads, eight of p and q each on their way at a time.  Every
// warp works out for itself which drafts stand, a lane per draft.  The warps' totals meet through
// distributed shared memory; the warp whose stretch holds the aim walks it again (from L2) to
// name the token, while the other CTAs make room for the next requests'.
// Measured: 256 requests of up to four drafts over 131072 fp32 probabilities (188 MB of rows) 41 us,
// 4.6 TB/s, 68 % of the measured copy rate (199 MB are read in all).  Six instructions an element: with every element's place checked
// (thirty) 58 us.  CTAs of 256 threads 44 us; clusters of four 42 us, of two 54 us; four loads at a
// time 44 us.  The rest is latency: offsets, drafts, their probabilities, the row come one after the
// other, and the last wave's walk for the token.
#include "pkv_kv4.cuh"
#include "pkv_kv8_attention.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kResident = 8;               // CTAs of an SM

struct VerifyParams {
    const char *p, *q;
    int64_t p_stride, q_stride;            // bytes
    const int32_t *ids, *qsl;
    const float *u;
    int32_t *tokens, *accepted;
    int32_t *err;
    int32_t rows, vocab, n, most;          // most: drafts that a request may have
};

template <typename T>
__device__ __forceinline__ float one_of(const char *row, int64_t i) {
    if constexpr (sizeof(T) == 4) return __ldg(reinterpret_cast<const float *>(row) + i);
    else {
        const uint32_t b = __ldg(reinterpret_cast<const unsigned short *>(row) + i);
        return widen2(b, std::is_same<T, __half>::value).x;
    }
}

template <typename T, int N>
__device__ __forceinline__ void floats_of_vector(uint4 v, float (&x)[N]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; i++) {
        if constexpr (sizeof(T) == 4) x[i] = __uint_as_float(w[i]);
        else {
            const float2 y = widen2(w[i], std::is_same<T, __half>::value);
            x[2 * i] = y.x;
            x[2 * i + 1] = y.y;
        }
    }
}

constexpr uint32_t kMagicHigh = 0x4b000000u, kMagicLow = 0x4b400000u;     // 2^23, 1.5 * 2^23

// A weight's two integer parts, each still with its magic constant's bits.
__device__ __forceinline__ void parts_of(float w, uint32_t &high, uint32_t &low) {
    const float t = fmaf(w, 0x1p20f, 0x1p23f);
    high = __float_as_uint(t);
    const float r = fmaf(w, 0x1p20f, 0x1p23f - t);                       // exact
    low = __float_as_uint(fmaf(r, 0x1p20f, 0x1.8p23f));
}
__device__ __forceinline__ int64_t count_of(float w) {
    uint32_t h, l;
    parts_of(w, h, l);
    return (static_cast<int64_t>(h - kMagicHigh) << 20) + static_cast<int32_t>(l - kMagicLow);
}

__device__ __forceinline__ int64_t warp_sum(int64_t x) {
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(~0u, x, o);
    return x;
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait;" ::: "memory"); }
__device__ __forceinline__ int64_t cluster_read64(const int64_t *at, uint32_t rank) {
    uint32_t a;
    int64_t v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                 : "=r"(a)
                 : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(at))), "r"(rank));
    asm volatile("ld.shared::cluster.s64 %0, [%1];" : "=l"(v) : "r"(a) : "memory");
    return v;
}

// One row's weights: where they are, and what is taken from the target's probabilities.
struct Row {
    const char *p, *q;                     // q NULL: nothing is subtracted
    int32_t without;                       // a token whose weight is 0, -1: none
};

// A row is walked in steps of 32 vectors (16 bytes a lane), counted from the aligned address at or before its
// first element; a step is whole where all its elements are the row's and p and q are aligned alike.
template <typename T>
struct Walk {
    static constexpr int N = 16 / sizeof(T);           // elements of a lane's load
    static constexpr int kStep = 32 * N;                // of a warp's
    static constexpr int kBatch = 8;                   // whole steps whose loads are on their way together
    static constexpr int kFlush = 512 / N;              // steps whose 32-bit sums cannot overflow (4096 elements a lane would)

    Row row;
    int64_t lead;                                       // elements from the aligned address to the row
    int32_t vocab;
    bool alike;

    __device__ __forceinline__ Walk(const Row &r, int32_t v) : row(r), vocab(v) {
        lead = static_cast<int64_t>(reinterpret_cast<uintptr_t>(r.p) & 15) / static_cast<int64_t>(sizeof(T));
        alike = r.q == nullptr || ((reinterpret_cast<uintptr_t>(r.q) ^ reinterpret_cast<uintptr_t>(r.p)) & 15) == 0;
    }
    __device__ __forceinline__ int64_t first_of(int64_t step) const { return step * kStep + (threadIdx.x & 31) * N - lead; }
    // Steps a .. b - 1 without those that are not whole.
    __device__ __forceinline__ void whole_of(int64_t a, int64_t b, int64_t &from, int64_t &to) const {
        from = lead > 0 && a == 0 ? 1 : a;
        const int64_t full = (vocab + lead) / kStep;    // steps that end inside the row
        to = alike ? (b < full ? b : full) : from;
        if (to < from) to = from;
    }
    // Weights of the lane's elements first .. + N - 1; what is not the row's weighs nothing.
    __device__ __forceinline__ void any_weights(int64_t first, float (&w)[N]) const {
#pragma unroll
        for (int i = 0; i < N; i++) {
            const int64_t e = first + i;
            w[i] = 0.f;
            if (e >= 0 && e < vocab && e != row.without) {
                const float x = one_of<T>(row.p, e);
                w[i] = __saturatef(row.q ? x - one_of<T>(row.q, e) : x);
            }
        }
    }
    static __device__ __forceinline__ void whole_weights(uint4 a, uint4 b, float (&w)[N]) {
        float y[N];
        floats_of_vector<T, N>(a, w);
        floats_of_vector<T, N>(b, y);
#pragma unroll
        for (int i = 0; i < N; i++) w[i] = __saturatef(w[i] - y[i]);      // NaN becomes 0
    }
    // The lane's sum over whole steps a .. b - 1; a token that is left out counts all the same.
    template <bool kQ>
    __device__ __forceinline__ int64_t whole_sum(int64_t a, int64_t b) const {
        const char *p = row.p + first_of(a) * static_cast<int64_t>(sizeof(T)), *q = kQ ? row.q + first_of(a) * static_cast<int64_t>(sizeof(T)) : nullptr;
        int64_t total = 0;
        while (a < b) {
            const int n = static_cast<int>(b - a < kFlush ? b - a : kFlush);
            uint32_t high = 0, low = 0;
#pragma unroll 1
            for (int k0 = 0; k0 < n; k0 += kBatch) {
                uint4 x[kBatch], y[kBatch];
#pragma unroll
                for (int k = 0; k < kBatch; k++) {
                    x[k] = y[k] = make_uint4(0, 0, 0, 0);
                    if (k0 + k < n) {
                        x[k] = __ldg(reinterpret_cast<const uint4 *>(p + 512 * k));
                        if constexpr (kQ) y[k] = __ldg(reinterpret_cast<const uint4 *>(q + 512 * k));
                    }
                }
                p += 512 * kBatch;
                if constexpr (kQ) q += 512 * kBatch;
#pragma unroll
                for (int k = 0; k < kBatch; k++) {
                    float w[N];
                    whole_weights(x[k], y[k], w);
#pragma unroll
                    for (int i = 0; i < N; i++) {
                        uint32_t h, l;
                        parts_of(w[i], h, l);
                        high += h;
                        low += l;
                    }
                }
            }
            const uint32_t count = static_cast<uint32_t>((n + kBatch - 1) / kBatch * kBatch * N);
            total += (static_cast<int64_t>(high - count * kMagicHigh) << 20) + static_cast<int32_t>(low - count * kMagicLow);
            a += n;
        }
        return total;
    }
    // The lane's sum over steps a .. b - 1, none of them taken to be whole.
    __device__ __forceinline__ int64_t any_sum(int64_t a, int64_t b) const {
        int64_t total = 0;
#pragma unroll 1
        for (; a < b; a++) {
            float w[N];
            any_weights(first_of(a), w);
#pragma unroll
            for (int i = 0; i < N; i++) total += count_of(w[i]);
        }
        return total;
    }
    // The sum over steps a .. b - 1 of the row, by the whole warp.
    __device__ __forceinline__ int64_t sum(int64_t a, int64_t b) const {
        int64_t from, to;
        whole_of(a, b, from, to);
        int64_t total = row.q ? whole_sum<true>(from, to) : whole_sum<false>(from, to);
        if (row.without >= 0) {
            const int64_t at = row.without + lead;      // the left-out token's place
            if (at >= from * kStep && at < to * kStep && (threadIdx.x & 31) == 0)
                total -= count_of(__saturatef(one_of<T>(row.p, row.without)));
        }
        total += any_sum(a, from < b ? from : b);
        total += any_sum(to > a ? to : a, b);
        return warp_sum(total);
    }
    // The first token of steps a .. b - 1 at which the running sum exceeds `aim` (it does before their end).
    __device__ __forceinline__ int32_t find(int64_t a, int64_t b, int64_t aim) const {
        const int lane = threadIdx.x & 31;
#pragma unroll 1
        for (; b - a > kBatch; a += kBatch) {           // the batch that holds it
            const int64_t part = sum(a, a + kBatch);
            if (part > aim) {
                b = a + kBatch;
                break;
            }
            aim -= part;
        }
#pragma unroll 1
        for (; a < b; a++) {
            const int64_t first = first_of(a);
            float w[N];
            any_weights(first, w);
            int64_t mine = 0;
#pragma unroll
            for (int i = 0; i < N; i++) mine += count_of(w[i]);
            int64_t upto = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t z = __shfl_up_sync(~0u, upto, o);
                if (lane >= o) upto += z;
            }
            const uint32_t past = __ballot_sync(~0u, upto > aim);
            if (past) {
                int64_t at = upto - mine;
                int32_t token = -1;
#pragma unroll
                for (int i = 0; i < N; i++) {
                    at += count_of(w[i]);
                    if (token < 0 && at > aim) token = static_cast<int32_t>(first + i);
                }
                return __shfl_sync(~0u, token, __ffs(past) - 1);
            }
            aim -= __shfl_sync(~0u, upto, 31);
        }
        return -1;
    }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, kResident) verify_kernel(const VerifyParams v) {
    __shared__ int64_t s_sum[2][kWarps];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int mates = cluster_size(), rank = blockIdx.x % mates, i = blockIdx.x / mates;
    const int32_t a = v.qsl[i], b = v.qsl[i + 1];
    int32_t *tokens = v.tokens + static_cast<int64_t>(i) * (v.most + 1);
    if (a < 0 || b < a || b > v.rows || static_cast<int64_t>(b) - a > static_cast<int64_t>(v.most) + 1 || a == b) {
        if (a != b && rank == 0 && threadIdx.x == 0 && v.err) atomicOr(v.err, PKV_DEVERR_COUNT);
        if (rank == 0) {
            for (int k = threadIdx.x; k <= v.most; k += kThreads) tokens[k] = -1;
            if (threadIdx.x == 0) v.accepted[i] = 0;
        }
        return;                                        // the whole cluster
    }
    // the drafts that stand, by every warp for itself
    const int drafts = b - a - 1;
    int stand = drafts;
    for (int j0 = 0; j0 < drafts; j0 += 32) {
        const int j = j0 + lane;
        bool passes = true;
        if (j < drafts) {
            const int64_t r = a + j;
            const int32_t x = v.ids[r];
            passes = false;
            if (x >= 0 && x < v.vocab) {
                const double p = one_of<T>(v.p + r * v.p_stride, x);
                const double q = v.q ? one_of<T>(v.q + r * v.q_stride, x) : 1.f;
                passes = static_cast<double>(v.u[r]) * q < p;
            }
        }
        const uint32_t falls = __ballot_sync(~0u, !passes);
        if (falls) {
            stand = j0 + __ffs(falls) - 1;
            break;
        }
    }
    const int64_t r = static_cast<int64_t>(a) + stand;
    if (rank == 0) {
        for (int k = threadIdx.x; k <= v.most; k += kThreads)
            if (k != stand) tokens[k] = k < stand ? v.ids[a + k] : -1;
        if (threadIdx.x == 0) v.accepted[i] = stand;
    }
    const float u = v.u[b - 1];
    Row row = {v.p + r * v.p_stride, nullptr, -1};
    if (stand < drafts) {
        if (v.q) row.q = v.q + r * v.q_stride;
        else row.without = v.ids[r];
    }
    // this warp's stretch of the row's steps
    const int64_t lead = static_cast<int64_t>(reinterpret_cast<uintptr_t>(row.p) & 15) / static_cast<int64_t>(sizeof(T));
    const int64_t steps = (v.vocab + lead + Walk<T>::kStep - 1) / Walk<T>::kStep, owners = static_cast<int64_t>(mates) * kWarps;
    const int64_t me = rank * kWarps + warp, from = steps * me / owners, to = steps * (me + 1) / owners;
    bool found = false;
    for (int pass = 0; pass < 2 && !found; pass++) {
        const Walk<T> walk(row, v.vocab);
        const int64_t mine = walk.sum(from, to);
        if (lane == 0) s_sum[pass][warp] = mine;
        if (mates > 1) cluster_sync();
        else __syncthreads();
        // every lane takes the totals of up to two warps
        int64_t before = 0, total = 0;
        for (int o = lane; o < owners; o += 32) {
            const int64_t x = mates > 1 ? cluster_read64(&s_sum[pass][o % kWarps], o / kWarps) : s_sum[pass][o];
            total += x;
            if (o < me) before += x;
        }
        total = warp_sum(total);
        before = warp_sum(before);
        if (mates > 1) cluster_arrive();               // this CTA has read the others' sums
        if (total > 0) {
            found = true;
            const double near = __ll2double_rn(total);
            double product = __dmul_rn(static_cast<double>(u), near);
            // rounded once: what a total past 2^53 loses in fp64 (2^8 at most) times u's 24 bits is exact
            if (total >> 53) product = __fma_rn(u, near, __dmul_rn(u, __ll2double_rn(total - __double2ll_rn(near))));
            int64_t aim = __double2ll_rd(product);
            aim = aim >= total ? total - 1 : aim < 0 ? 0 : aim;
            if (before <= aim && aim < before + mine) {
                const int32_t token = walk.find(from, to, aim - before);
                if (lane == 0) tokens[stand] = token;
            }
        } else if (!row.q && row.without < 0) {
            if (rank == 0 && threadIdx.x == 0) tokens[stand] = -1;
            found = true;
        } else {
            row.q = nullptr;                           // nothing is left of p - q: p itself
            row.without = -1;
        }
        if (mates > 1) cluster_wait();                 // nobody leaves while its sums are read
    }
}

template <typename T>
int launch(const VerifyParams &v, cudaStream_t s) {
    // A CTA for every 16384 bytes of a row, one batch of its four warps, up to eight.
    const int64_t bytes = static_cast<int64_t>(v.vocab) * sizeof(T);
    int mates = 1;
    while (mates < kMaxCluster && bytes > mates * 16384LL) mates *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(v.n) * mates);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(mates);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    PKV_CUDA_TRY(cudaLaunchKernelEx(&cfg, verify_kernel<T>, v));
    return PKV_OK;
}

}  // namespace
}  // namespace pkv

extern "C" int pkv_verify_drafts(const void *target_probs, int64_t target_stride, const void *draft_probs,
                                 int64_t draft_stride, int32_t dtype, int32_t vocab, int32_t num_rows,
                                 const int32_t *draft_ids, const int32_t *query_start_loc, int32_t n,
                                 const float *uniforms, int32_t max_drafts, int32_t *tokens, int32_t *accepted,
                                 int32_t *d_error, pkv_stream_t stream) {
    if (n < 0 || n > PKV_MAX_BATCH || num_rows < 0 || num_rows >= PKV_MAX_TOKENS || vocab < 1 || vocab > (1 << 22) ||
        max_drafts < 0 || max_drafts >= PKV_MAX_TOKENS || target_stride < 0 || draft_stride < 0 ||
        target_stride > (1LL << 40) || draft_stride > (1LL << 40) || (dtype != PKV_BF16 && dtype != PKV_FP16 && dtype != PKV_FP32))
        return PKV_ERR_INVALID_ARG;
    if (n == 0) return PKV_OK;
    if (!query_start_loc || !tokens || !accepted) return PKV_ERR_INVALID_ARG;
    if (num_rows > 0 && (!target_probs || !uniforms || (num_rows > 1 && !draft_ids))) return PKV_ERR_INVALID_ARG;
    if (num_rows > 1 && (target_stride < vocab || (draft_probs && draft_stride < vocab))) return PKV_ERR_INVALID_ARG;
    const int size = dtype == PKV_FP32 ? 4 : 2;
    if (((reinterpret_cast<uintptr_t>(target_probs) | reinterpret_cast<uintptr_t>(draft_probs)) & (size - 1)) ||
        ((reinterpret_cast<uintptr_t>(draft_ids) | reinterpret_cast<uintptr_t>(query_start_loc) | reinterpret_cast<uintptr_t>(uniforms) |
          reinterpret_cast<uintptr_t>(tokens) | reinterpret_cast<uintptr_t>(accepted)) & 3))
        return PKV_ERR_ALIGN;
    pkv::VerifyParams v = {};
    v.p = static_cast<const char *>(target_probs);
    v.q = static_cast<const char *>(draft_probs);
    v.p_stride = target_stride * size;
    v.q_stride = draft_stride * size;
    v.ids = draft_ids;
    v.qsl = query_start_loc;
    v.u = uniforms;
    v.tokens = tokens;
    v.accepted = accepted;
    v.err = d_error;
    v.rows = num_rows;
    v.vocab = vocab;
    v.n = n;
    v.most = max_drafts;
    cudaStream_t s = pkv::as_stream(stream);
    return dtype == PKV_FP32 ? pkv::launch<float>(v, s) : dtype == PKV_FP16 ? pkv::launch<__half>(v, s) : pkv::launch<__nv_bfloat16>(v, s);
}
