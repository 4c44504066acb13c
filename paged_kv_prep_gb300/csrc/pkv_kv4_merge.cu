// Merging the partial results of the attention kernels on the 4-bit paged cache.
//
// Mathematics.  A (query, head) row that was cut has pieces (R_k, sum_k, O_k); with R = max R_k it is sum =
// sum_k 2^(R_k - R) sum_k and O likewise, in the order of the pieces.
//
// Bound: latency (the note, the request, the references, the rows come one after the other); the pieces lie in L2.
//
// Layout.  A CTA belongs to one note.  Row tiles of chunks have 256 rows in two or three pieces: a warp takes four rows, all
// of their loads on their way at once.  Few tokens have eight rows or sixteen: a warp each, or, where few requests
// are cut into long chains, four warps a row, which share out its pieces and meet in shared memory; few notes are
// real then, so a CTA looks at several.
// Measured: 256 decodes 9.9 us, four long ones 13.8 us, a mixed call's chunks 20.8 us (one warp a row
// that reads its note itself: 13.8, 18.5 and 26 us).
#include "pkv_kv4_attention.cuh"

namespace pkv {
namespace {

constexpr int kThreads = 256, kChainThreads = 1024;
constexpr int kWarps = kThreads / 32, kTeamWarps = 4;

// Rows row0 .. + kRows - 1 of a note's tile by one warp (kTeam 1), or one row by kTeam warps, of which this is `rank`;
// s_acc is theirs, and all of the CTA's warps are here together.  kBatch: pieces whose rows are on their way together.
template <int D, int kRows, int kTeam, int kBatch>
__device__ __forceinline__ void merge_rows(const AttnParams &p, int rows, int stride, int worker, int4 note, int row0, int rank,
                                           float (*s_acc)[D + 1]) {
    constexpr int kPer = D / 32;                       // elements of a lane
    const int lane = threadIdx.x & 31;
    const Req r = request_of(p, note.x);
    const int pieces = note.z, head = note.w;
    const int64_t f0 = static_cast<int64_t>(note.y) * rows + row0, all = static_cast<int64_t>(r.count) * p.G;
    if (kTeam == 1 && f0 >= all) return;
    const int64_t size = static_cast<int64_t>(rows) * (D + 2);
    auto part = [&](int k) { return p.part + (2LL * (worker + static_cast<int64_t>(k) * stride) + (k == 0)) * size; };
    float top[kRows], sum[kRows], acc[kRows][kPer];
#pragma unroll
    for (int i = 0; i < kRows; i++) {
        top[i] = -INFINITY;
        sum[i] = 0.f;
#pragma unroll
        for (int c = 0; c < kPer; c++) acc[i][c] = 0.f;
    }
    for (int k = lane; k < pieces; k += 32) {
#pragma unroll
        for (int i = 0; i < kRows; i++) top[i] = fmaxf(top[i], part(k)[row0 + i]);
    }
#pragma unroll
    for (int i = 0; i < kRows; i++)
#pragma unroll
        for (int o = 16; o; o >>= 1) top[i] = fmaxf(top[i], __shfl_xor_sync(~0u, top[i], o));
    for (int k0 = rank; k0 < pieces; k0 += kTeam * kBatch) {
        float m[kBatch][kRows], l[kBatch][kRows], y[kBatch][kRows][kPer];
#pragma unroll
        for (int b = 0; b < kBatch; b++) {
            const float *a = part(min(k0 + b * kTeam, pieces - 1));
#pragma unroll
            for (int i = 0; i < kRows; i++) {
                m[b][i] = a[row0 + i];
                l[b][i] = a[rows + row0 + i];
                const float *o = a + 2 * rows + (row0 + i) * D + lane * kPer;
                if constexpr (kPer == 2) {
                    const float2 z = *reinterpret_cast<const float2 *>(o);
                    y[b][i][0] = z.x, y[b][i][1] = z.y;
                } else {
#pragma unroll
                    for (int c = 0; c < kPer; c += 4) {
                        const float4 z = *reinterpret_cast<const float4 *>(o + c);
                        y[b][i][c] = z.x, y[b][i][c + 1] = z.y, y[b][i][c + 2] = z.z, y[b][i][c + 3] = z.w;
                    }
                }
            }
        }
#pragma unroll
        for (int b = 0; b < kBatch; b++) {
            if (k0 + b * kTeam >= pieces) break;
#pragma unroll
            for (int i = 0; i < kRows; i++) {
                // a piece without a reference adds nothing, unless its logits were NaN
                const float f = m[b][i] == -INFINITY ? (l[b][i] == 0.f ? 0.f : NAN) : exp2_fast(m[b][i] - top[i]);
                if (f != 0.f || l[b][i] != l[b][i]) {  // a NaN counts however small its piece is
                    sum[i] = fmaf(f, l[b][i], sum[i]);
#pragma unroll
                    for (int c = 0; c < kPer; c++) acc[i][c] = fmaf(f, y[b][i][c], acc[i][c]);
                }
            }
        }
    }
    if constexpr (kTeam > 1) {
#pragma unroll
        for (int c = 0; c < kPer; c++) s_acc[rank][lane * kPer + c] = acc[0][c];
        if (lane == 0) s_acc[rank][D] = sum[0];
        __syncthreads();
        if (rank || f0 >= all) return;
#pragma unroll
        for (int w = 1; w < kTeam; w++) {
            sum[0] += s_acc[w][D];
#pragma unroll
            for (int c = 0; c < kPer; c++) acc[0][c] += s_acc[w][lane * kPer + c];
        }
    }
#pragma unroll
    for (int i = 0; i < kRows; i++) {
        if (f0 + i >= all) break;
        const bool none = top[i] == -INFINITY && sum[i] == 0.f;
        const float inv = none ? 0.f : 1.f / sum[i];
        const int f = static_cast<int>(f0) + i, j = f / p.G, hq = head * p.G + f - j * p.G;
        uint32_t z[kPer / 2];
#pragma unroll
        for (int c = 0; c < kPer; c += 2) z[c / 2] = pack_out(acc[i][c] * inv, acc[i][c + 1] * inv, p.fp16);
        char *out = p.out + static_cast<int64_t>(r.start + j) * p.out_stride + 2 * (static_cast<int64_t>(hq) * D + lane * kPer);
        if constexpr (kPer == 2) *reinterpret_cast<uint32_t *>(out) = z[0];
        else if constexpr (kPer == 4) *reinterpret_cast<uint2 *>(out) = make_uint2(z[0], z[1]);
        else *reinterpret_cast<uint4 *>(out) = make_uint4(z[0], z[1], z[2], z[3]);
        if (lane == 0 && p.lse)
            p.lse[static_cast<int64_t>(r.start + j) * p.Hkv * p.G + hq] = none ? -INFINITY : (top[i] + log2f(sum[i])) * kLn2;
    }
}

template <int D, int kRows, int kBatch>
__global__ void __launch_bounds__(kThreads) kv4_merge_kernel(const AttnParams p, int rows, int stride) {
    pdl_wait();
    pdl_trigger();
    const int parts = rows / (kWarps * kRows), worker = blockIdx.x / parts;
    const int4 note = p.meta[worker];                  // request, row tile, pieces, KV head
    if (note.x < 0) return;
    merge_rows<D, kRows, 1, kBatch>(p, rows, stride, worker, note, ((blockIdx.x - worker * parts) * kWarps + (threadIdx.x >> 5)) * kRows,
                                    0, nullptr);
}

// Eight rows of tiles of `rows`; a CTA looks at up to 32 workers' notes.
template <int D>
__global__ void __launch_bounds__(kChainThreads) kv4_merge_chains_kernel(const AttnParams p, int rows, int workers, int stride) {
    __shared__ float s_acc[8][kTeamWarps][D + 1];
    static_assert(kChainThreads / 32 == 8 * kTeamWarps, "eight rows");
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, row = (threadIdx.x >> 5) / kTeamWarps, eights = rows / 8;
    const int step = gridDim.x / eights, first = blockIdx.x / eights, row0 = 8 * (blockIdx.x - first * eights);
    // neighbouring workers, which begin the same request's heads, go to different CTAs
    const int mine = first + lane * step;
    uint32_t real = __ballot_sync(~0u, mine < workers && p.meta[mine < workers ? mine : 0].x >= 0);
    for (; real; real &= real - 1) {
        const int worker = first + (__ffs(real) - 1) * step;
        merge_rows<D, 1, kTeamWarps, 4>(p, rows, stride, worker, p.meta[worker], row0 + row, (threadIdx.x >> 5) % kTeamWarps, s_acc[row]);
        __syncthreads();                               // the sums have been read
    }
}

template <int D>
int launch(const AttnParams &p, int rows, int workers, int stride, int sms, cudaStream_t s) {
    // chains: the row tiles (of all heads) that the batch can have are an eighth of the workers or fewer (calls of two
    // requests' four drafts on 60000 tokens 54 us so, 71 with a warp a row; of eight single tokens of 16 heads 19.6 and 24)
    const int64_t tiles = (static_cast<int64_t>(p.T) * p.G / rows + p.n) * p.Hkv;
    if (rows <= 16 && tiles * 8 <= workers) {
        const int grid = workers < 32 * sms ? sms : (workers + 31) / 32;
        PKV_CUDA_TRY(launch_pdl(kv4_merge_chains_kernel<D>, dim3((workers < grid ? workers : grid) * (rows / 8)), dim3(kChainThreads), 0, s, p,
                                rows, workers, stride));
        return PKV_OK;
    }
    constexpr int kTileRows = D == 256 ? 2 : 4;
    auto kernel = rows > 16 ? kv4_merge_kernel<D, kTileRows, 2> : kv4_merge_kernel<D, 1, 4>;
    const int own = kWarps * (rows > 16 ? kTileRows : 1);
    PKV_CUDA_TRY(launch_pdl(kernel, dim3(static_cast<unsigned>(workers) * (rows / own)), dim3(kThreads), 0, s, p, rows, stride));
    return PKV_OK;
}

}  // namespace

int kv4_launch_merge(const AttnParams &p, int32_t head_dim, int rows, int workers, int stride, int sms, cudaStream_t s) {
    if (head_dim == 64) return launch<64>(p, rows, workers, stride, sms, s);
    if (head_dim == 128) return launch<128>(p, rows, workers, stride, sms, s);
    return launch<256>(p, rows, workers, stride, sms, s);
}

}  // namespace pkv
