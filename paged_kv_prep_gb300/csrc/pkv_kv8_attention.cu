// Host side of the attention over the 8-bit paged cache, and the kernel that
// adds up the attention weight each cached token received.
//
// weights[slot] += sum over the step's queries and heads of exp(x - lse): the
// row's lse is known once the attention has run, so a token's weight is a sum
// over rows that one CTA can own.  No atomics unless requests share a block:
// the addition to global memory itself is atomic, so that shared blocks lose
// nothing.
//
// Layout.  A first kernel packs the rows (f16, scaled by a power of two, in the
// order of the fragments) with their factors, so that rows of one KV head lie
// behind one another.  A CTA owns kT token groups of 32 of a request and walks
// the KV heads: a head's codes come by cp.async while the head before is worked
// on, become f16 fragments in registers once, and meet the request's rows in
// chunks that bulk copies bring two chunks ahead.  With kT = 8 (single tokens: few
// rows) a warp per group; with kT = 4 (chunks: many rows) two warps share a group's
// rows and a cluster shares the KV heads, so that the tokens that thousands of rows
// see do not hold the launch up; the sums meet in a fixed order.
//
// Bound: for single tokens HBM (D bytes of K per token and KV head, the second
// read of K), for chunks the tensor pipe (mma.sync) and the exponentials.
// Measured: 32 single tokens on 8192 cached (271 MB) 75 us, 3.6 TB/s, held by the
// barriers and row copies of each (256 tokens, head) step; three chunks (145 GFLOP
// of attention) 267 us with the tensor pipe active 46 % of the time.  Chunks with
// kT = 1 and 128 rows a chunk 291 us, kT = 2 and 96 rows 286 (a row is fetched by
// four or two times as many CTAs); rows shared out over the cluster as well 278.
#include "pkv_kv8_attention.cuh"
#include "pkv_tcgen05.cuh"

namespace pkv {

int64_t kv8_decode_workspace(int32_t head_dim, int sms);
int kv8_launch_decode(const AttnParams &p, int32_t head_dim, bool one_tile, int sms, cudaStream_t s);
int64_t kv8_prefill_workspace(int32_t head_dim, int sms);
int kv8_launch_prefill(const AttnParams &p, int32_t head_dim, int sms, cudaStream_t s);

namespace {

constexpr int kPrefillRows = 32;

constexpr int kWWarps = 8, kWThreads = 32 * kWWarps, kWStages = 3;
constexpr uint32_t kNone = 0xffffffffu;                       // no slot: slots fit 32 bits with room
template <int D, int kT>
constexpr int kWRows = kT < 8 ? (D > 128 ? 32 : 64) : (D > 128 ? 16 : 32);   // rows of a chunk

template <int D, int kT>
struct WeightsShape {
    static constexpr int kSubs = D <= 128 ? 2 : 1;            // 16-token fragments per warp
    static constexpr int kGroup = 16 * kSubs, kTokens = kGroup * kT;
    static constexpr int kTeams = kWWarps / kT;               // warps that share a group's rows
};

template <int D, int kT>
struct WeightsSmem {
    static constexpr int kTokens = WeightsShape<D, kT>::kTokens;
    alignas(16) char k[2][kTokens * D];                       // this head's codes, the next one's
    alignas(16) char q[kWStages][kWRows<D, kT> * D * 2];                         // packed rows
    alignas(16) float2 fac[kWStages][kWRows<D, kT> + 2];                            // factor of S, -lse (both for base 2)
    uint64_t full[kWStages], free[kWStages];
    int32_t block[2][kTokens];                                // by unit parity; -1: not read
    uint32_t slot[2][kTokens];
    float ks[2][kTokens];
    float sum[kWWarps][WeightsShape<D, kT>::kGroup];
    float total[2][kTokens];                                  // by unit parity: this CTA's heads
    int64_t prefix[kWThreads + 1];
    int64_t warp_sum[kWWarps];
};

// Wait for a bulk copy; gives up after half a second or more.
__device__ __forceinline__ bool wait_rows(uint64_t *bar, uint32_t parity) {
    for (uint32_t k = 0; k < (1u << 22); k++)
        if (mbar_try(bar, parity)) return true;
    return false;
}

// Packed rows of a call: [KV head][token * G + head of the group], a row of D f16 values whose
// 16-byte pieces stand as (step pair, lane t), the odd rows' with the halves of 128 bytes swapped (so
// that two neighbouring rows fall into different banks); and their factors.
struct Packed {
    char *rows;
    float2 *fac;
};

// A warp per 32 * 8 / D rows of a token, D / 8 lanes per row.
template <int D>
__global__ void __launch_bounds__(256) kv8_pack_kernel(const AttnParams p, const Packed out) {
    constexpr int kPieces = D / 8, kAtOnce = 32 / kPieces;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, piece = lane % kPieces;
    const bool fp16 = p.fp16 != 0;
    const int hq = p.Hkv * p.G, per = (hq + kAtOnce - 1) / kAtOnce;
    const int64_t jobs = static_cast<int64_t>(p.T) * per;
    for (int64_t job = (blockIdx.x * 256LL + threadIdx.x) >> 5; job < jobs; job += gridDim.x * 8LL) {
        const int64_t tok = job / per;
        const int h = static_cast<int>(job - tok * per) * kAtOnce + lane / kPieces;
        uint4 y = make_uint4(0, 0, 0, 0);
        float lse = -INFINITY;
        if (h < hq) {
            y = __ldg(reinterpret_cast<const uint4 *>(p.q + tok * p.q_stride + 2 * (static_cast<int64_t>(h) * D + 8 * piece)));
            lse = p.lse[tok * hq + h];
        }
        const float2 a = widen2(y.x, fp16), b = widen2(y.y, fp16), c = widen2(y.z, fp16), d = widen2(y.w, fp16);
        float m = fmaxf(fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(b.x), fabsf(b.y))),
                        fmaxf(fmaxf(fabsf(c.x), fabsf(c.y)), fmaxf(fabsf(d.x), fabsf(d.y))));
#pragma unroll
        for (int o = kPieces / 2; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(~0u, m, o));
        const int e = row_exponent(m);
        const float s = power2(14 - e);
        if (h < hq) {
            const int head = h / p.G;
            const int64_t row = (static_cast<int64_t>(head) * p.T + tok) * p.G + h - head * p.G;
            // dimensions 8 piece ..: fragment steps 4 u + i and the one after it, lane t
            const int dim = 8 * piece, pair = (4 * (dim / 64) + (dim % 16) / 4) >> 1, t = (dim % 64) / 16;
            const int at = (4 * pair + t) ^ (static_cast<int>(row & 1) << 2);
            *reinterpret_cast<uint4 *>(out.rows + row * (2 * D) + 16 * at) =
                make_uint4(pack_f16(a.x * s, a.y * s), pack_f16(b.x * s, b.y * s), pack_f16(c.x * s, c.y * s),
                           pack_f16(d.x * s, d.y * s));
            if (piece == 0) out.fac[row] = make_float2(p.scale_log2 * power2(e - 14), -lse * kLog2e);
        }
    }
}

template <int D, int kT>
__global__ void __launch_bounds__(kWThreads, 2) kv8_weights_kernel(const AttnParams p, const Packed packed) {
    using Shape = WeightsShape<D, kT>;
    constexpr int S = D / 16, kSubs = Shape::kSubs, kGroup = Shape::kGroup, kTokens = Shape::kTokens, kTeams = Shape::kTeams;
    extern __shared__ __align__(16) char s_raw[];
    auto &sm = *reinterpret_cast<WeightsSmem<D, kT> *>(s_raw);
    pdl_wait();
    pdl_trigger();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
    const int group = warp % kT, team = warp / kT;
    const int64_t line = static_cast<int64_t>(p.Hkv) * D;
    if (tid == 0) {
        for (int k = 0; k < kWStages; k++) {
            mbar_init(&sm.full[k], 1);
            mbar_init(&sm.free[k], kWWarps);
        }
        fence_mbar_init();
    }
    auto units = [&](int i) -> int64_t {
        const Req r = request_of(p, i);
        const int lo = r.lo & ~(kTokens - 1);
        return r.count > 0 && r.keys > lo ? (r.keys - lo + kTokens - 1) / kTokens : 0;
    };
    const int64_t total = plan_prefix<kWThreads>(sm.prefix, sm.warp_sum, p.n, units);
    const int64_t all = gridDim.x / cluster_size(), ranges = total < all ? total : all;
    const int mates = cluster_size(), rank = blockIdx.x % mates, range = blockIdx.x / mates;
    if (range >= ranges) return;
    // Single tokens: a stretch of units each, all alike.  Chunks: every ranges-th unit, since the tokens
    // at a chunk's front are seen by more rows than those at its end.
    constexpr bool kStretch = kT == 8;
    const int64_t step = kStretch ? 1 : ranges, end = kStretch ? (range + 1) * total / ranges : total;
    int64_t u = kStretch ? range * total / ranges : range;

    // One unit: a request, the tokens s0 .. s0 + kTokens - 1, and the rows f0 .. f1 - 1 that see one of them.
    struct Unit {
        Req r;
        int i, s0, f0, f1;
    };
    struct Walk {
        int64_t first;                                        // first unit of request `at`
        int at;
    };
    Walk walk;
    walk.at = plan_find<kWThreads>(sm.prefix, p.n, u, units, &walk.first);
    auto unit_of = [&](Walk &w, int64_t v) {
        Unit x;
        for (;;) {
            const int64_t k = units(w.at);
            if (v < w.first + k) break;
            w.first += k;
            w.at++;
        }
        x.i = w.at;
        x.r = request_of(p, w.at);
        x.s0 = (x.r.lo & ~(kTokens - 1)) + static_cast<int>(v - w.first) * kTokens;
        const int back = x.r.len - x.r.count;
        // query j (at position back + j) sees token s if s <= back + j < s + window
        const int j0 = max(0, x.s0 - back);
        const int64_t j1 = p.window > 0 ? static_cast<int64_t>(x.s0) + kTokens - 1 + p.window - 1 - back : x.r.count - 1;
        x.f0 = j0 * p.G;
        x.f1 = (static_cast<int>(j1 < x.r.count - 1 ? j1 : x.r.count - 1) + 1) * p.G;
        return x;
    };
    auto find_blocks = [&](const Unit &x, int parity) {
        if (tid < kTokens) {
            const int s = x.s0 + tid;
            const int b = s >= x.r.lo && s < x.r.keys ? block_of(p, p.tables + static_cast<int64_t>(x.i) * p.W, s) : -1;
            sm.block[parity][tid] = b;
            sm.slot[parity][tid] = b < 0 ? kNone : static_cast<uint32_t>(b) * static_cast<uint32_t>(p.bs) + static_cast<uint32_t>(s % p.bs);
        }
    };
    // the codes and scales of one head
    auto fetch = [&](const Unit &x, int parity, int head, int place) {
        constexpr int kRowLanes = D / 16, kStep = kWThreads / kRowLanes;
        const int piece = tid % kRowLanes;
#pragma unroll
        for (int i = 0; i < (kTokens + kStep - 1) / kStep; i++) {
            const int tok = i * kStep + tid / kRowLanes;
            if (tok < kTokens) {
                const uint32_t slot = sm.slot[parity][tok];
                cp_async<16>(smem_addr(sm.k[place] + tok * D + 16 * swizzle<D>(piece, tok)),
                             p.kc + (slot != kNone ? slot * line + head * D + 16 * piece : 0), slot != kNone);
            }
        }
        if (tid < kTokens) {
            const int b = sm.block[parity][tid];
            cp_async<4>(smem_addr(&sm.ks[place][tid]), p.ks + (b >= 0 ? static_cast<int64_t>(b) * p.Hkv + head : 0), b >= 0);
        }
        cp_commit();
    };
    // The rows' chunks in the order in which they are used; thread 0 asks for them two ahead, into the
    // place of the chunk before.
    struct Feed {
        Walk walk;
        int64_t u;
        Unit x;
        int head, f;
        uint32_t count;
    };
    Feed feed = {};
    auto ask_rows = [&]() {
        if (feed.u >= end) return;
        const int stage = feed.count % kWStages;
        // every warp has left the chunk that had this place before
        if (feed.count >= kWStages && !wait_rows(&sm.free[stage], (feed.count / kWStages - 1) & 1) && p.err)
            atomicOr(p.err, PKV_DEVERR_TIMEOUT);
        const int rows = min(kWRows<D, kT>, feed.x.f1 - feed.f);
        const int64_t row = (static_cast<int64_t>(feed.head) * p.T + feed.x.r.start) * p.G + feed.f;
        // the factors' copy starts on an even row and the two sides' offsets agree
        const int odd = static_cast<int>(row & 1);
        const uint32_t facs = static_cast<uint32_t>((rows + odd + 1) & ~1) * 8;
        mbar_arrive_expect_tx(&sm.full[stage], rows * 2 * D + facs);
        bulk_g2s(sm.q[stage], packed.rows + row * (2 * D), rows * 2 * D, &sm.full[stage]);
        bulk_g2s(sm.fac[stage], packed.fac + row - odd, facs, &sm.full[stage]);
        feed.count++;
        feed.f += kWRows<D, kT>;
        if (feed.f >= feed.x.f1) {
            feed.head += mates;
            if (feed.head >= p.Hkv) {
                feed.head = rank;
                feed.u += step;
                if (feed.u < end) feed.x = unit_of(feed.walk, feed.u);
            }
            feed.f = feed.x.f0;
        }
    };

    feed.walk = walk;
    feed.u = u;
    Unit x = unit_of(walk, u);
    feed.x = x;
    feed.head = rank;
    feed.f = x.f0;
    feed.count = 0;
    if (rank >= p.Hkv) feed.u = end;
    int parity = 0;
    uint32_t chunk = 0, step_no = 0;
    find_blocks(x, parity);
    __syncthreads();
    if (rank < p.Hkv) fetch(x, parity, rank, 0);
    if (tid == 0) {
        ask_rows();
        ask_rows();
    }
    while (true) {
        const bool more = u + step < end;
        Unit y = x;
        if (more) {
            y = unit_of(walk, u + step);
            find_blocks(y, parity ^ 1);
        }
        float acc[kSubs][2];
#pragma unroll
        for (int k = 0; k < kSubs; k++) acc[k][0] = acc[k][1] = 0.f;
        for (int head = rank; head < p.Hkv; head += mates) {
            // this head's codes are here, and everyone has left the place of the head before: the next
            // head's are on their way for a whole step
            cp_wait<0>();
            __syncthreads();
            const int place = step_no++ & 1;
            const bool last = head + mates >= p.Hkv;
            if (!last) fetch(x, parity, head + mates, place ^ 1);
            else if (more) fetch(y, parity ^ 1, rank, place ^ 1);
            uint32_t kf[kSubs][S][4];
            float ks[kSubs][2];
#pragma unroll
            for (int k = 0; k < kSubs; k++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const int tok = group * kGroup + 16 * k + g + 8 * h;
                    ks[k][h] = sm.ks[place][tok];
#pragma unroll
                    for (int c = 0; c < D / 64; c++) {
                        const uint4 v = *reinterpret_cast<const uint4 *>(sm.k[place] + tok * D + 16 * swizzle<D>(4 * c + t, tok));
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int i = 0; i < 4; i++) {
                            kf[k][4 * c + i][h] = f16x2_of(w[i]);
                            kf[k][4 * c + i][2 + h] = f16x2_of(w[i] >> 16);
                        }
                    }
                }
            const int back = x.r.len - x.r.count;
            // rows whose position is at least the tile's last token and whose window reaches its first
            const auto rows_to = [&](int64_t j) { return static_cast<int>(min(max(j, int64_t{0}) * p.G, int64_t{0x7fffffff})); };
            const int whole0 = rows_to(static_cast<int64_t>(x.s0) + kTokens - 1 - back);
            const int whole1 = p.window > 0 ? rows_to(static_cast<int64_t>(x.s0) + p.window - back) : 0x7fffffff;
            const int64_t row0 = (static_cast<int64_t>(head) * p.T + x.r.start) * p.G;
            for (int f = x.f0; f < x.f1; f += kWRows<D, kT>, chunk++) {
                if (tid == 0) ask_rows();
                const int stage = chunk % kWStages;
                if (!wait_rows(&sm.full[stage], (chunk / kWStages) & 1) && p.err) atomicOr(p.err, PKV_DEVERR_TIMEOUT);
                const int odd = static_cast<int>((row0 + f) & 1);
                // every row of the chunk sees every token of the tile (tokens that are not read do not count:
                // their sums are dropped)
                const bool chunk_whole = f >= whole0 && min(f + kWRows<D, kT>, x.f1) <= whole1;
                int nt = team;
                if constexpr (kT < 8) {
                    // two tiles of rows at a time where nothing is masked: twice the independent products (three
                    // chunks 518 us with the attention, a tile at a time 537)
#pragma unroll 1
                    for (; chunk_whole && nt + kTeams < kWRows<D, kT> / 8 && f + 8 * (nt + kTeams) + 8 <= x.f1; nt += 2 * kTeams) {
                        float c[2][kSubs][4];
#pragma unroll
                        for (int w = 0; w < 2; w++)
#pragma unroll
                            for (int k = 0; k < kSubs; k++) c[w][k][0] = c[w][k][1] = c[w][k][2] = c[w][k][3] = 0.f;
                        const char *row = sm.q[stage] + (8 * nt + g) * (2 * D);
                        const int flip = ((g + odd) & 1) << 2;
#pragma unroll
                        for (int j = 0; j < S; j += 2) {
#pragma unroll
                            for (int w = 0; w < 2; w++) {
                                const uint4 b = *reinterpret_cast<const uint4 *>(row + w * (8 * kTeams * 2 * D) + 16 * ((2 * j + t) ^ flip));
#pragma unroll
                                for (int k = 0; k < kSubs; k++) mma_f16(c[w][k], kf[k][j], b.x, b.y);
#pragma unroll
                                for (int k = 0; k < kSubs; k++) mma_f16(c[w][k], kf[k][j + 1], b.z, b.w);
                            }
                        }
#pragma unroll
                        for (int w = 0; w < 2; w++) {
                            const float2 fa = sm.fac[stage][odd + 8 * (nt + w * kTeams) + 2 * t];
                            const float2 fb = sm.fac[stage][odd + 8 * (nt + w * kTeams) + 2 * t + 1];
#pragma unroll
                            for (int k = 0; k < kSubs; k++)
#pragma unroll
                                for (int h = 0; h < 2; h++)
                                    acc[k][h] += exp2_fast(fmaf(c[w][k][2 * h], fa.x * ks[k][h], fa.y)) +
                                                 exp2_fast(fmaf(c[w][k][2 * h + 1], fb.x * ks[k][h], fb.y));
                        }
                    }
                }
#pragma unroll 1
                for (; nt < kWRows<D, kT> / 8; nt += kTeams) {
                    if (f + 8 * nt >= x.f1) break;
                    float c[kSubs][4];
#pragma unroll
                    for (int k = 0; k < kSubs; k++) c[k][0] = c[k][1] = c[k][2] = c[k][3] = 0.f;
                    const char *row = sm.q[stage] + (8 * nt + g) * (2 * D);
                    const int flip = ((g + odd) & 1) << 2;
#pragma unroll
                    for (int j = 0; j < S; j += 2) {
                        const uint4 b = *reinterpret_cast<const uint4 *>(row + 16 * ((2 * j + t) ^ flip));
#pragma unroll
                        for (int k = 0; k < kSubs; k++) {
                            mma_f16(c[k], kf[k][j], b.x, b.y);
                            mma_f16(c[k], kf[k][j + 1], b.z, b.w);
                        }
                    }
                    const float2 fa = sm.fac[stage][odd + 8 * nt + 2 * t], fb = sm.fac[stage][odd + 8 * nt + 2 * t + 1];
                    const int first = f + 8 * nt;
                    float v[kSubs][4];
#pragma unroll
                    for (int k = 0; k < kSubs; k++)
#pragma unroll
                        for (int q = 0; q < 4; q++)
                            v[k][q] = exp2_fast(fmaf(c[k][q], (q & 1 ? fb.x : fa.x) * ks[k][q >> 1], q & 1 ? fb.y : fa.y));
                    if (!chunk_whole) {
                        const int r0 = first + 2 * t;
                        const int pa = r0 < x.f1 ? back + r0 / p.G : -1, pb = r0 + 1 < x.f1 ? back + (r0 + 1) / p.G : -1;
#pragma unroll
                        for (int k = 0; k < kSubs; k++)
#pragma unroll
                            for (int q = 0; q < 4; q++) {
                                const int pos = q & 1 ? pb : pa, s = x.s0 + group * kGroup + 16 * k + g + 8 * (q >> 1);
                                // an empty row (-lse = inf) gives no weight
                                const bool ok = s <= pos && s >= lo_of(p, pos) && (q & 1 ? fb.y : fa.y) != INFINITY;
                                if (!ok) v[k][q] = 0.f;
                            }
                    } else if (first + 8 > x.f1) {
#pragma unroll
                        for (int k = 0; k < kSubs; k++)
#pragma unroll
                            for (int q = 0; q < 4; q++)
                                if (first + 2 * t + (q & 1) >= x.f1) v[k][q] = 0.f;
                    }
#pragma unroll
                    for (int k = 0; k < kSubs; k++)
#pragma unroll
                        for (int h = 0; h < 2; h++) acc[k][h] += v[k][2 * h] + v[k][2 * h + 1];
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.free[stage]);
            }
        }
#pragma unroll
        for (int k = 0; k < kSubs; k++)
#pragma unroll
            for (int h = 0; h < 2; h++) {
                float a = acc[k][h];
                a += __shfl_xor_sync(~0u, a, 1);
                a += __shfl_xor_sync(~0u, a, 2);
                if (t == 0) sm.sum[warp][16 * k + g + 8 * h] = a;
            }
        __syncthreads();
        if (tid < kTokens) {
            float a = 0.f;
#pragma unroll
            for (int w = 0; w < kTeams; w++) a += sm.sum[w * kT + tid / kGroup][tid % kGroup];
            sm.total[parity][tid] = a;
        }
        cluster_sync();
        if (rank == 0 && tid < kTokens && sm.block[parity][tid] >= 0) {
            float a = sm.total[parity][tid];
            for (int c = 1; c < mates; c++) a += cluster_read(&sm.total[parity][tid], c);
            atomicAdd(p.weights + sm.slot[parity][tid], a);
        }
        if (!more) break;
        __syncthreads();
        x = y;
        u += step;
        parity ^= 1;
    }
    cp_wait<0>();
    cluster_sync();                                           // nobody leaves while its totals are read
}

int64_t workspace_of(int32_t head_dim, int sms) {
    const int64_t a = kv8_decode_workspace(head_dim, sms), b = kv8_prefill_workspace(head_dim, sms);
    return ((a > b ? a : b) + 255) & ~255LL;
}

template <int D, int kT>
int launch_weights_as(const AttnParams &p, const Packed &packed, int mates, int sms, cudaStream_t s) {
    constexpr int smem = static_cast<int>(sizeof(WeightsSmem<D, kT>));
    static_assert(smem <= 113 * 1024, "two CTAs an SM");
    static bool set[64] = {false};
    const int rc = kv8_allow_smem(reinterpret_cast<const void *>(kv8_weights_kernel<D, kT>), smem, set);
    if (rc != PKV_OK) return rc;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(2 * sms / mates * mates));
    cfg.blockDim = dim3(kWThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(mates);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    // Clusters that become resident while the packing still runs end up unevenly placed: three chunks
    // took 608 us with the early start and 518 us without it, the attention included.
    cfg.attrs = mates == 1 ? attr : attr + 1;
    cfg.numAttrs = mates == 1 ? 2 : 1;
    // Every cluster takes one stretch of the units, so no more of them are started than run at once
    // (the SMs of a GPC are not a multiple of eight); asked for once per device and cluster size.
    static int known[64][4] = {{0}};
    int dev = 0;
    PKV_CUDA_TRY(cudaGetDevice(&dev));
    const int log = mates == 1 ? 0 : mates == 2 ? 1 : mates == 4 ? 2 : 3;
    int clusters = dev < 64 ? known[dev][log] : 0;
    if (!clusters) {
        cudaLaunchConfig_t alone = cfg;
        alone.attrs = attr + 1;
        alone.numAttrs = 1;
        PKV_CUDA_TRY(cudaOccupancyMaxActiveClusters(&clusters, kv8_weights_kernel<D, kT>, &alone));
        if (clusters < 1) clusters = 1;
        if (dev < 64) known[dev][log] = clusters;
    }
    if (clusters * mates < 2 * sms) cfg.gridDim = dim3(static_cast<unsigned>(clusters * mates));
    const int64_t pack = (static_cast<int64_t>(p.T) * p.Hkv * p.G * D + 2047) / 2048;   // CTAs that hold all rows
    PKV_CUDA_TRY(launch_pdl(kv8_pack_kernel<D>, dim3(static_cast<unsigned>(pack < 8 * sms ? pack : 8 * sms)), dim3(256), 0, s, p, packed));
    PKV_CUDA_TRY(cudaLaunchKernelEx(&cfg, kv8_weights_kernel<D, kT>, p, packed));
    return PKV_OK;
}

int launch_weights(const AttnParams &p, char *workspace, int32_t head_dim, int sms, cudaStream_t s) {
    Packed packed;
    packed.rows = workspace;
    packed.fac = reinterpret_cast<float2 *>(workspace + 2LL * p.T * p.Hkv * p.G * head_dim);
    // a step of single tokens has few rows a request: the warps share out its tokens
    const bool single = p.T <= p.n;
    const int mates = single || p.Hkv < 2 ? 1 : p.Hkv < 4 ? 2 : p.Hkv < 8 ? 4 : 8;
    if (head_dim == 64)
        return single ? launch_weights_as<64, 8>(p, packed, mates, sms, s) : launch_weights_as<64, 4>(p, packed, mates, sms, s);
    if (head_dim == 128)
        return single ? launch_weights_as<128, 8>(p, packed, mates, sms, s) : launch_weights_as<128, 4>(p, packed, mates, sms, s);
    return single ? launch_weights_as<256, 8>(p, packed, mates, sms, s) : launch_weights_as<256, 4>(p, packed, mates, sms, s);
}

// Bytes of the packed rows and their factors (a pair of factors may be read past the last row).
int64_t packed_bytes(int64_t rows, int32_t head_dim) { return rows * (2LL * head_dim + 8) + 16; }

}  // namespace
}  // namespace pkv

extern "C" {

int pkv_kv8_attention_workspace(int32_t num_tokens, int32_t num_q_heads, int32_t head_dim, int32_t with_weights,
                                int64_t *bytes) {
    if (!bytes || num_tokens < 0 || num_tokens >= PKV_MAX_TOKENS || num_q_heads < 1 || num_q_heads > (1 << 20) ||
        !pkv::kv8_head_dim(head_dim))
        return PKV_ERR_INVALID_ARG;
    int sms = 0;
    const int rc = pkv::kv8_sm_count(&sms);
    if (rc != PKV_OK) return rc;
    *bytes = pkv::workspace_of(head_dim, sms);
    if (with_weights) *bytes += pkv::packed_bytes(static_cast<int64_t>(num_tokens) * num_q_heads, head_dim);
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
    const int64_t own = pkv::workspace_of(cache->head_dim, sms);
    if (workspace_bytes < own + (weights ? pkv::packed_bytes(static_cast<int64_t>(num_tokens) * num_q_heads, cache->head_dim) : 0))
        return PKV_ERR_INVALID_ARG;
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
    p.part = reinterpret_cast<float *>(p.meta + pkv::kv8_most_workers(sms));
    p.err = d_error;
    cudaStream_t s = pkv::as_stream(stream);
    // The prefill kernel takes the requests with more than kPrefillRows rows.  It needs head_dim <= 128
    // (two accumulators beside two score tiles in TMEM) and 16-token groups that lie in one block;
    // otherwise the decode kernel's row tiles take everything.
    const bool prefill = cache->head_dim <= 128 && p.bs % 16 == 0 &&
                         static_cast<int64_t>(num_tokens - n + 1) * p.G > pkv::kPrefillRows && num_tokens > n;
    // Tables of at most 256 tokens (eight units) and tiles enough for two warps an SM: a warp takes a
    // whole row tile, and no merge follows.  Contexts of 100 to 200 tokens, 8 KV heads of 4 query heads,
    // cut / whole: 8 requests 13.7 / 18.7 us, 64 requests 20.3 / 18.8, 512 requests 55.2 / 48.6; contexts of
    // 250 to 500, 64 requests 24.2 / 32.0.  The host knows no lengths: short requests in wide tables are cut.
    p.whole = static_cast<int64_t>(p.W) * p.bs <= 256 && static_cast<int64_t>(n) * p.Hkv >= 2 * sms;
    p.short_rows = prefill ? pkv::kPrefillRows : 0x7fffffff;
    // one 8-row tile holds every request of a pure decode step
    const bool one_tile = num_tokens <= n && p.G <= 8;
    if (prefill) {
        rc = pkv::kv8_launch_prefill(p, cache->head_dim, sms, s);
        if (rc != PKV_OK) return rc;
    }
    rc = pkv::kv8_launch_decode(p, cache->head_dim, one_tile, sms, s);
    if (rc != PKV_OK || !weights) return rc;
    return pkv::launch_weights(p, static_cast<char *>(workspace) + own, cache->head_dim, sms, s);
}

}  // extern "C"
