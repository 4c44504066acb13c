// Attention over the 8-bit paged cache for requests with few query rows
// (single-token decodes, short chunks).
//
// Mathematics.  Row r = (query j, head of the KV head's group), key s in block
// b: x = (q . code_k) * k_scale[b] * softmax_scale * log2(e) + log2(v_scale[b]).
// With R = the running maximum of x, w = 2^(x - R) <= 1 already carries the
// value scale, so it can be rounded to f16 for the second product without
// leaving f16's range whatever the scales are; the softmax sum adds
// w / v_scale[b] in fp32.  out = sum w * code_v / sum, lse = R ln 2 + ln sum.
//
// Bound: HBM, 2 * D bytes per (cached token, KV head), each read once.
//
// Layout.  Every warp works alone: it owns one KV head and a contiguous range
// of 16-token units of the batch; the warps of the KV heads of one range are
// neighbours, so a token's line is read by one CTA at one time.  Keys are the
// M side of the products (S^T = K Q^T, O^T = V^T P^T), so eight rows fill the
// N side.  Each lane copies with cp.async exactly the codes that its own
// fragments need into its own slots of a ring, so the ring needs no barrier
// and no transpose: K by token rows, V as pairs of tokens merged with a byte
// permute; e4m3 turns into f16 exactly on the way into the fragments, and P
// moves from accumulator to operand layout with movmatrix.
// A range that ends inside a request leaves a partial result (R, sum, O) that
// a second kernel merges in a fixed order.
#include "pkv_kv8_attention.cuh"

namespace pkv {
namespace {

constexpr int kUnit = 16;          // tokens per unit
constexpr int kStages = 3;

template <int D>
struct Stage {
    static constexpr int kKPieces = D / 64;                   // 16-byte pieces per lane and token row
    static constexpr int kVBytes = D / 8 < 16 ? D / 8 : 16;   // bytes per piece
    static constexpr int kVPieces = D / 8 / kVBytes;
    uint4 k[2][kKPieces][32];
    char v[4][kVPieces][32 * kVBytes];
    float ks[kUnit], vs[kUnit];
};

template <int D, int NT>
constexpr int warps_of() { return NT == 1 && D <= 128 ? 16 : 8; }

// Units of a request: 16-token units of its visible range, once per tile of 8 * NT rows.
template <int NT>
__device__ __forceinline__ int64_t units_of_request(const AttnParams &p, const Req &r, int *per_tile) {
    *per_tile = 1;
    const int64_t rows = static_cast<int64_t>(r.count) * p.G;
    if (r.count <= 0 || rows > p.short_rows) return 0;
    const int lo = r.lo & ~(kUnit - 1);
    const int u = r.keys > lo ? (r.keys - lo + kUnit - 1) / kUnit : 1;   // a request without keys writes zeros
    *per_tile = u;
    return static_cast<int64_t>(u) * ((rows + 8 * NT - 1) / (8 * NT));
}

// One warp's pass over units ua..ub-1 of row tile `rt` of a request and one KV head.
template <int D, int NT>
struct Tile {
    float o[NT][D / 16][4];
    float top[NT][2], sum[NT][2];          // of columns 2t, 2t + 1

    __device__ __forceinline__ void run(const AttnParams &p, const Req &r, const int32_t *table, int head,
                                        int rt, int ua, int ub, Stage<D> *ring, uint32_t *valid) {
        constexpr int S = D / 16;
        using St = Stage<D>;
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const int rows = r.count * p.G;
        const bool fp16 = p.fp16 != 0;

        // row positions of this lane's columns, and the tile's key range
        int pos[NT][2];
        float cf[NT][2];
        uint32_t qb[NT][S][2];
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
            const int f = rt * 8 * NT + nt * 8 + g;
            const int j = f / p.G;
            const char *row = p.q + static_cast<int64_t>(r.start + j) * p.q_stride +
                              2 * static_cast<int64_t>(head * p.G + f - j * p.G) * D;
            const int e = load_query<D>(qb[nt], row, f < rows, t, fp16);
#pragma unroll
            for (int c = 0; c < 2; c++) {
                const int fc = rt * 8 * NT + nt * 8 + 2 * t + c;
                pos[nt][c] = fc < rows ? r.len - r.count + fc / p.G : -1;
                cf[nt][c] = p.scale_log2 * power2(__shfl_sync(~0u, e, (2 * t + c) * 4) - 14);
                top[nt][c] = -INFINITY;
                sum[nt][c] = 0.f;
            }
#pragma unroll
            for (int j2 = 0; j2 < S; j2++)
#pragma unroll
                for (int c = 0; c < 4; c++) o[nt][j2][c] = 0.f;
        }
        const int first_row = rt * 8 * NT, last_row = min(rows, first_row + 8 * NT) - 1;
        const int pos_first = r.len - r.count + first_row / p.G, pos_last = r.len - r.count + last_row / p.G;
        const int base = r.lo & ~(kUnit - 1);
        // keys that some row of the tile sees, and those that every row sees
        const int some_lo = p.window > 0 ? max(0, pos_first - p.window + 1) : 0, some_hi = min(pos_last + 1, r.keys);
        const int all_lo = p.window > 0 ? max(0, pos_last - p.window + 1) : 0, all_hi = pos_first + 1;
        ua = max(ua, (some_lo - base) / kUnit);
        ub = min(ub, some_hi > base ? (some_hi - base + kUnit - 1) / kUnit : 0);
        if (ua >= ub) return;

        const int64_t line = static_cast<int64_t>(p.Hkv) * D;
        const uint8_t *kh = p.kc + head * D + 16 * t;
        const uint8_t *vh = p.vc + head * D + St::kVBytes * g;

        auto block_at = [&](int u) {           // block id of token (lane & 15) of unit u, -1 if not read
            const int s = base + u * kUnit + (lane & 15);
            return u < ub && s >= some_lo && s < some_hi ? block_of(p, table, s) : -1;
        };
        auto issue = [&](int u, int block) {
            if (u < ub) {
                St &st = ring[(u - ua) % kStages];
                const int s = base + u * kUnit + (lane & 15);
                const int64_t slot = block >= 0 ? static_cast<int64_t>(block) * p.bs + s % p.bs : -1;
                const uint32_t mask = __ballot_sync(~0u, block >= 0) & 0xffffu;
                if (lane == 0) valid[(u - ua) % kStages] = mask;
                const float *sc = (lane < 16 ? p.ks : p.vs) + (block >= 0 ? static_cast<int64_t>(block) * p.Hkv + head : 0);
                cp_async<4>(smem_addr(lane < 16 ? &st.ks[lane] : &st.vs[lane - 16]), sc, block >= 0);
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const int64_t x = __shfl_sync(~0u, slot, g + 8 * h);
                    const uint8_t *src = kh + (x >= 0 ? x * line : 0);
#pragma unroll
                    for (int c = 0; c < St::kKPieces; c++) cp_async<16>(smem_addr(&st.k[h][c][lane]), src + 64 * c, x >= 0);
                }
#pragma unroll
                for (int h = 0; h < 4; h++) {
                    const int64_t x = __shfl_sync(~0u, slot, 2 * t + (h & 1) + 8 * (h >> 1));
                    const uint8_t *src = vh + (x >= 0 ? x * line : 0);
#pragma unroll
                    for (int c = 0; c < St::kVPieces; c++)
                        cp_async<St::kVBytes>(smem_addr(&st.v[h][c][lane * St::kVBytes]), src + 128 * c, x >= 0);
                }
            }
            cp_commit();
        };

        __syncwarp();
        int ahead = block_at(ua);
#pragma unroll
        for (int k = 0; k < kStages - 1; k++) {
            const int b = ahead;
            ahead = block_at(ua + k + 1);
            issue(ua + k, b);
        }
        for (int u = ua; u < ub; u++) {
            cp_wait<kStages - 2>();
            __syncwarp();
            {
                const int b = ahead;
                ahead = block_at(u + kStages);
                issue(u + kStages - 1, b);
            }
            const St &st = ring[(u - ua) % kStages];
            const uint32_t mask = valid[(u - ua) % kStages];
            const int s0 = base + u * kUnit;

            float x[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int c = 0; c < 4; c++) x[nt][c] = 0.f;
#pragma unroll
            for (int c = 0; c < St::kKPieces; c++) {
                const uint4 ka = st.k[0][c][lane], kb = st.k[1][c][lane];
                const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    const uint32_t a[4] = {f16x2_of(wa[i]), f16x2_of(wb[i]), f16x2_of(wa[i] >> 16), f16x2_of(wb[i] >> 16)};
#pragma unroll
                    for (int nt = 0; nt < NT; nt++) mma_f16(x[nt], a, qb[nt][4 * c + i][0], qb[nt][4 * c + i][1]);
                }
            }
            const float ks[2] = {st.ks[g], st.ks[g + 8]}, vs[2] = {value_scale(st.vs[g]), value_scale(st.vs[g + 8])};
            const float lv[2] = {__log2f(vs[0]), __log2f(vs[1])}, iv[2] = {__frcp_rn(vs[0]), __frcp_rn(vs[1])};
            const bool whole = mask == 0xffffu && s0 >= all_lo && s0 + kUnit <= all_hi;
            uint32_t pb[NT][2], seen[NT];
            bool moved = false;
            float next[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
                seen[nt] = 15;
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    const int h = c >> 1, col = c & 1;
                    x[nt][c] = fmaf(x[nt][c], cf[nt][col] * ks[h], lv[h]);
                    if (!whole) {
                        const int s = s0 + g + 8 * h;
                        const bool ok = ((mask >> (g + 8 * h)) & 1) && s <= pos[nt][col] &&
                                        (p.window <= 0 || s > pos[nt][col] - p.window);
                        if (!ok) {
                            x[nt][c] = -INFINITY;
                            seen[nt] &= ~(1u << c);
                        }
                    }
                }
#pragma unroll
                for (int col = 0; col < 2; col++) {
                    float m = fmaxf(x[nt][col], x[nt][2 + col]);
                    m = fmaxf(m, __shfl_xor_sync(~0u, m, 4));
                    m = fmaxf(m, __shfl_xor_sync(~0u, m, 8));
                    m = fmaxf(m, __shfl_xor_sync(~0u, m, 16));
                    next[nt][col] = fmaxf(top[nt][col], m);
                    moved |= next[nt][col] > top[nt][col];
                }
            }
            if (__any_sync(~0u, moved)) {
#pragma unroll
                for (int nt = 0; nt < NT; nt++) {
                    float a[2];
#pragma unroll
                    for (int col = 0; col < 2; col++) {
                        a[col] = next[nt][col] > top[nt][col] ? exp2_fast(top[nt][col] - next[nt][col]) : 1.f;
                        sum[nt][col] *= a[col];
                        top[nt][col] = next[nt][col];
                    }
#pragma unroll
                    for (int j = 0; j < S; j++)
#pragma unroll
                        for (int c = 0; c < 4; c++) o[nt][j][c] *= a[c & 1];
                }
            }
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
                float w[4];
#pragma unroll
                for (int c = 0; c < 4; c++) {
                    w[c] = (seen[nt] >> c) & 1 ? exp2_fast(x[nt][c] - top[nt][c & 1]) : 0.f;
                    sum[nt][c & 1] += (seen[nt] >> c) & 1 ? w[c] * iv[c >> 1] : 0.f;
                }
                pb[nt][0] = transpose8x8(pack_f16(w[0], w[1]));
                pb[nt][1] = transpose8x8(pack_f16(w[2], w[3]));
            }
#pragma unroll
            for (int c = 0; c < St::kVPieces; c++) {
                uint32_t w[4][St::kVBytes / 4];
#pragma unroll
                for (int h = 0; h < 4; h++) {
                    if constexpr (St::kVBytes == 16) {
                        const uint4 y = *reinterpret_cast<const uint4 *>(&st.v[h][c][lane * 16]);
                        w[h][0] = y.x;
                        w[h][1] = y.y;
                        w[h][2] = y.z;
                        w[h][3] = y.w;
                    } else {
                        const uint2 y = *reinterpret_cast<const uint2 *>(&st.v[h][c][lane * 8]);
                        w[h][0] = y.x;
                        w[h][1] = y.y;
                    }
                }
                bool nan = false;
                if (!whole && r.count > 1) {
                    // A row must not see a NaN code in a token that only other rows see: such codes leave
                    // the product and come back below for the rows that do see them.
#pragma unroll
                    for (int h = 0; h < 4; h++)
#pragma unroll
                        for (int i = 0; i < St::kVBytes / 4; i++)
                            nan |= __vcmpeq4(w[h][i] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
                    nan = __any_sync(~0u, nan);
                }
#pragma unroll
                for (int i = 0; i < St::kVBytes / 4; i++) {
#pragma unroll
                    for (int half = 0; half < 2; half++) {
                        // dimensions 4 i + 2 half (row g) and + 1 (row g + 8), tokens (2t, 2t+1) and (2t+8, 2t+9)
                        const uint32_t sel = half ? 0x7362 : 0x5140;
                        uint32_t lo = __byte_perm(w[0][i], w[1][i], sel), hi = __byte_perm(w[2][i], w[3][i], sel);
                        const int j = c * (St::kVBytes / 2) + 2 * i + half;
                        if (nan) {
                            const uint32_t nl = __vcmpeq4(lo & 0x7f7f7f7fu, 0x7f7f7f7fu), nh = __vcmpeq4(hi & 0x7f7f7f7fu, 0x7f7f7f7fu);
                            lo &= ~nl;
                            hi &= ~nh;
                            const uint32_t a[4] = {f16x2_of(nl & 0x38383838u), f16x2_of((nl & 0x38383838u) >> 16),
                                                   f16x2_of(nh & 0x38383838u), f16x2_of((nh & 0x38383838u) >> 16)};
#pragma unroll
                            for (int nt = 0; nt < NT; nt++) {
                                const uint32_t one = 0x3c00u;
                                const uint32_t s01 = ((seen[nt] & 1) ? one : 0) | ((seen[nt] & 2) ? one << 16 : 0);
                                const uint32_t s23 = ((seen[nt] & 4) ? one : 0) | ((seen[nt] & 8) ? one << 16 : 0);
                                float hit[4] = {0.f, 0.f, 0.f, 0.f};
                                mma_f16(hit, a, transpose8x8(s01), transpose8x8(s23));
#pragma unroll
                                for (int k = 0; k < 4; k++)
                                    if (hit[k] > 0.f) o[nt][j][k] = NAN;
                            }
                        }
                        const uint32_t a[4] = {f16x2_of(lo), f16x2_of(lo >> 16), f16x2_of(hi), f16x2_of(hi >> 16)};
#pragma unroll
                        for (int nt = 0; nt < NT; nt++) mma_f16(o[nt][j], a, pb[nt][0], pb[nt][1]);
                    }
                }
            }
        }
        cp_wait<0>();
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int col = 0; col < 2; col++) {
                float l = sum[nt][col];
                l += __shfl_xor_sync(~0u, l, 4);
                l += __shfl_xor_sync(~0u, l, 8);
                l += __shfl_xor_sync(~0u, l, 16);
                sum[nt][col] = l;
            }
    }

    // Dimensions of this lane's accumulators: piece c covers 128 c + kVBytes g .., pairs in order.
    __device__ __forceinline__ void write(const AttnParams &p, const Req &r, int head, int rt) const {
        using St = Stage<D>;
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const int rows = r.count * p.G;
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int col = 0; col < 2; col++) {
                const int f = rt * 8 * NT + nt * 8 + 2 * t + col;
                if (f >= rows) continue;
                const int j = f / p.G, hq = head * p.G + f - j * p.G;
                // nothing visible (a row of NaN logits leaves top at -inf too, but its sum is NaN)
                const bool none = top[nt][col] == -INFINITY && sum[nt][col] == 0.f;
                const float inv = none ? 0.f : 1.f / sum[nt][col];
                char *row = p.out + static_cast<int64_t>(r.start + j) * p.out_stride + 2 * static_cast<int64_t>(hq) * D;
#pragma unroll
                for (int c = 0; c < St::kVPieces; c++)
#pragma unroll
                    for (int i = 0; i < St::kVBytes / 8; i++) {
                        uint32_t y[4];
#pragma unroll
                        for (int k = 0; k < 4; k++) {
                            const float *a = o[nt][c * (St::kVBytes / 2) + 4 * i + k];
                            y[k] = pack_out(none ? 0.f : a[col] * inv, none ? 0.f : a[2 + col] * inv, p.fp16);
                        }
                        *reinterpret_cast<uint4 *>(row + 2 * (128 * c + St::kVBytes * g + 8 * i)) =
                            make_uint4(y[0], y[1], y[2], y[3]);
                    }
                if (g == 0 && p.lse)
                    p.lse[static_cast<int64_t>(r.start + j) * p.Hkv * p.G + hq] =
                        none ? -INFINITY : (top[nt][col] + log2f(sum[nt][col])) * kLn2;
            }
    }

    // A partial result: 8 NT tops, 8 NT sums, then rows of D floats.
    __device__ __forceinline__ void spill(float *part) const {
        using St = Stage<D>;
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
        for (int nt = 0; nt < NT; nt++)
#pragma unroll
            for (int col = 0; col < 2; col++) {
                const int row = nt * 8 + 2 * t + col;
                if (g == 0) {
                    part[row] = top[nt][col];
                    part[8 * NT + row] = sum[nt][col];
                }
                float *at = part + 16 * NT + row * D;
#pragma unroll
                for (int c = 0; c < St::kVPieces; c++)
#pragma unroll
                    for (int i = 0; i < St::kVBytes / 4; i++) {
                        const float *a = o[nt][c * (St::kVBytes / 2) + 2 * i], *b = o[nt][c * (St::kVBytes / 2) + 2 * i + 1];
                        *reinterpret_cast<float4 *>(at + 128 * c + St::kVBytes * g + 4 * i) =
                            make_float4(a[col], a[2 + col], b[col], b[2 + col]);
                    }
            }
    }
};

template <int D, int NT>
__global__ void __launch_bounds__(32 * warps_of<D, NT>(), 1) kv8_decode_kernel(const AttnParams p) {
    constexpr int kWarps = warps_of<D, NT>(), kThreads = 32 * kWarps;
    constexpr int kPart = 8 * NT * (D + 2);
    extern __shared__ __align__(16) char s_ring[];
    __shared__ int64_t s_prefix[kThreads + 1];
    __shared__ int64_t s_warp[kWarps];
    __shared__ uint32_t s_valid[kWarps][kStages];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    auto units = [&](int i) {
        int per;
        return units_of_request<NT>(p, request_of(p, i), &per);
    };
    const int64_t total = plan_prefix<kThreads>(s_prefix, s_warp, p.n, [&](int i) {
        int per;
        return units_of_request<NT>(p, request_of(p, i, blockIdx.x == 0), &per);
    });
    const int worker = blockIdx.x * kWarps + warp;
    const int64_t all = static_cast<int64_t>(gridDim.x) * kWarps / p.Hkv;     // ranges the batch is cut into
    const int64_t ranges = total < all ? total : all;
    const int range = worker / p.Hkv, head = worker - range * p.Hkv;
    int4 note = make_int4(-1, 0, 0, 0);
    if (range < ranges) {
        int64_t u = range * total / ranges;
        const int64_t end = (range + 1) * total / ranges;
        Stage<D> *ring = reinterpret_cast<Stage<D> *>(s_ring) + warp * kStages;
        int64_t first;
        int i = plan_find<kThreads>(s_prefix, p.n, u, units, &first);
        while (u < end) {
            const Req r = request_of(p, i);
            int per;
            const int64_t k = units_of_request<NT>(p, r, &per);
            if (u >= first + k) {
                first += k;
                i++;
                continue;
            }
            const int rt = static_cast<int>((u - first) / per);
            const int64_t tile = first + static_cast<int64_t>(rt) * per;      // the tile's first unit
            const int ua = static_cast<int>(u - tile);
            const int ub = static_cast<int>(end - tile < per ? end - tile : per);
            Tile<D, NT> x;
            x.run(p, r, p.tables + static_cast<int64_t>(i) * p.W, head, rt, ua, ub, ring, s_valid[warp]);
            if (ua == 0 && ub == per) {
                x.write(p, r, head, rt);
            } else {
                // slot 1: the range where a tile begins, slot 0: one that goes on with it
                x.spill(p.part + (2LL * worker + (ua == 0)) * kPart);
                if (ua == 0) {
                    const int64_t last = ((tile + per) * ranges - 1) / total; // the range with the tile's last unit
                    note = make_int4(i, rt, static_cast<int>(last - range) + 1, head);
                }
            }
            u = tile + ub;
        }
    }
    if (lane == 0) p.meta[worker] = note;
}

// Merge the partial results of the tiles that were cut, a warp per (worker, row).
constexpr int kMergeThreads = 256;

template <int D>
__global__ void __launch_bounds__(kMergeThreads) kv8_merge_kernel(const AttnParams p, int rows, int workers, int stride) {
    constexpr int kPer = D / 32;
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int job = blockIdx.x * (kMergeThreads / 32) + (threadIdx.x >> 5);
    const int worker = job / rows, row = job - worker * rows;
    if (worker >= workers) return;
    const int4 note = p.meta[worker];                // request, row tile, pieces, KV head
    if (note.x < 0) return;
    const Req r = request_of(p, note.x);
    const int64_t f64 = static_cast<int64_t>(note.y) * rows + row;
    if (f64 >= static_cast<int64_t>(r.count) * p.G) return;
    const int f = static_cast<int>(f64), pieces = note.z, head = note.w;
    const int64_t size = static_cast<int64_t>(rows) * (D + 2);
    auto part = [&](int k) { return p.part + (2LL * (worker + static_cast<int64_t>(k) * stride) + (k == 0)) * size; };
    float top = -INFINITY;
    for (int k = lane; k < pieces; k += 32) top = fmaxf(top, part(k)[row]);
#pragma unroll
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
    float sum = 0.f, acc[kPer];
#pragma unroll
    for (int c = 0; c < kPer; c++) acc[c] = 0.f;
#pragma unroll 8
    for (int k = 0; k < pieces; k++) {
        const float *a = part(k);
        const float m = a[row], l = a[rows + row];
        // a piece without a top adds nothing, unless its logits were NaN
        const float f2 = m == -INFINITY ? (l == 0.f ? 0.f : NAN) : exp2_fast(m - top);
        sum += f2 * l;
        const float *o = a + 2 * rows + row * D + lane * kPer;
#pragma unroll
        for (int c = 0; c < kPer; c += 2) {
            const float2 y = *reinterpret_cast<const float2 *>(o + c);
            acc[c] += f2 == 0.f ? 0.f : f2 * y.x;
            acc[c + 1] += f2 == 0.f ? 0.f : f2 * y.y;
        }
    }
    const bool none = top == -INFINITY && sum == 0.f;
    const int j = f / p.G, hq = head * p.G + f - j * p.G;
    const float inv = none ? 0.f : 1.f / sum;
    char *out = p.out + static_cast<int64_t>(r.start + j) * p.out_stride + 2 * (static_cast<int64_t>(hq) * D + lane * kPer);
#pragma unroll
    for (int c = 0; c < kPer; c += 2)
        *reinterpret_cast<uint32_t *>(out + 2 * c) = pack_out(acc[c] * inv, acc[c + 1] * inv, p.fp16);
    if (lane == 0 && p.lse)
        p.lse[static_cast<int64_t>(r.start + j) * p.Hkv * p.G + hq] = none ? -INFINITY : (top + log2f(sum)) * kLn2;
}

template <int D, int NT>
int launch(const AttnParams &p, int sms, cudaStream_t s) {
    constexpr int kWarps = warps_of<D, NT>();
    constexpr size_t smem = sizeof(Stage<D>) * kStages * kWarps;
    static bool set[64] = {false};
    int dev = 0;
    PKV_CUDA_TRY(cudaGetDevice(&dev));
    if (dev < 0 || dev >= 64 || !set[dev]) {
        PKV_CUDA_TRY(cudaFuncSetAttribute(kv8_decode_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                          static_cast<int>(smem)));
        if (dev >= 0 && dev < 64) set[dev] = true;
    }
    PKV_CUDA_TRY(launch_pdl(kv8_decode_kernel<D, NT>, dim3(sms), dim3(32 * kWarps), smem, s, p));
    return kv8_launch_merge(p, D, 8 * NT, sms * kWarps, p.Hkv, s);
}

template <int D>
int launch_rows(const AttnParams &p, bool one_tile, int sms, cudaStream_t s) {
    return one_tile ? launch<D, 1>(p, sms, s) : launch<D, 2>(p, sms, s);
}

}  // namespace

int kv8_launch_merge(const AttnParams &p, int32_t head_dim, int rows, int workers, int stride, cudaStream_t s) {
    const dim3 grid((static_cast<unsigned>(workers) * rows + kMergeThreads / 32 - 1) / (kMergeThreads / 32)), block(kMergeThreads);
    if (head_dim == 64)
        PKV_CUDA_TRY(launch_pdl(kv8_merge_kernel<64>, grid, block, 0, s, p, rows, workers, stride));
    else if (head_dim == 128)
        PKV_CUDA_TRY(launch_pdl(kv8_merge_kernel<128>, grid, block, 0, s, p, rows, workers, stride));
    else
        PKV_CUDA_TRY(launch_pdl(kv8_merge_kernel<256>, grid, block, 0, s, p, rows, workers, stride));
    return PKV_OK;
}

int64_t kv8_decode_workspace(int32_t head_dim, int sms) {
    // the widest variant: 16 workers an SM, two partial results each of 16 rows
    return static_cast<int64_t>(sms) * 16 * (2LL * 16 * (head_dim + 2) * 4 + 16);
}

int kv8_launch_decode(const AttnParams &p, int32_t head_dim, bool one_tile, int sms, cudaStream_t s) {
    if (head_dim == 64) return launch_rows<64>(p, one_tile, sms, s);
    if (head_dim == 128) return launch_rows<128>(p, one_tile, sms, s);
    return launch_rows<256>(p, one_tile, sms, s);
}

}  // namespace pkv
