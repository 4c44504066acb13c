// Attention over the 8-bit paged cache for requests with few query rows
// (single-token decodes, short chunks).
//
// Mathematics.  Row r = (query j, head of the KV head's group), key s in block
// b: x = (q . code_k) * k_scale[b] * softmax_scale * log2(e) + log2(v_scale[b]).
// With R = a row's reference, at most 14 below the running maximum of x, w =
// 2^(x - R) <= 2^14 already carries the value scale, so it can be rounded to f16
// for the second product without leaving f16's range whatever the scales are; the softmax sum adds
// w / v_scale[b] in fp32.  out = sum w * code_v / sum, lse = R ln 2 + ln sum.
//
// Bound: HBM, 2 * D bytes per (cached token, KV head), each read once.
//
// Layout.  Every warp works alone: it owns one KV head and a contiguous range
// of 32-token units of the batch; the warps of the KV heads of one range are
// neighbours, so a token's line is read by one CTA at one time.  Keys are the
// M side of the products (S^T = K Q^T, O^T = V^T P^T), so eight rows fill the
// N side.  A warp copies its unit's rows with cp.async into a stage of its own, whose
// halves (keys, values) it refills as soon as it has taken them out; V comes
// out as pairs of tokens merged with a byte permute, no transpose; e4m3 turns into f16 exactly on the way into the fragments, and P
// moves from accumulator to operand layout with movmatrix.
// The copies go by whole 128-byte pieces of a line: fetched as the fragments
// want them (16 bytes of four to eight lines an instruction) the kernel stood at
// 4.3 TB/s with or without its arithmetic.
// A range that ends inside a request leaves a partial result (R, sum, O) that
// a second kernel merges in a fixed order.
// Measured: 256 single tokens on contexts up to 8192 (2.1 GB, floor 316 us) 377 to
// 389 us with the merge, 5.4 to 5.6 TB/s, 81 to 84 % of the measured copy rate.  Without its arithmetic it reaches 5.7 TB/s.
#include "pkv_kv8_attention.cuh"

namespace pkv {
namespace {

constexpr int kUnit = 32;          // tokens per unit, two groups of 16
constexpr int kDepth = 1;           // units whose codes are held or on their way; two measured no faster
constexpr float kSlack = 14.f;     // growth of a row's maximum (log2) that R does not follow

// A unit's codes, a row of D bytes per token (pieces permuted by swizzle()), and its scales.
template <int D>
struct Stage {
    static constexpr int kKPieces = D / 64;                   // 16-byte pieces per lane and token row
    static constexpr int kVBytes = D / 8 < 16 ? D / 8 : 16;   // bytes per piece
    static constexpr int kVPieces = D / 8 / kVBytes;
    static constexpr int kRowLanes = D / 16;                  // lanes that copy a token's row
    static constexpr int kRows = 32 / kRowLanes;              // rows of one copy instruction
    char k[kUnit * D], v[kUnit * D];
    float ks[kUnit], vs[kUnit];                               // by token, or by group
};

template <int D, int NT>
constexpr int warps_of() { return D == 256 ? 6 : NT == 2 ? 8 : D == 128 ? 12 : 16; }

// Units of a request: 32-token units of its visible range, once per tile of 8 * NT rows.
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

// One warp's pass over units ua..ub-1 of row tile `rt` of a request and one KV head.  kGrouped: 16
// tokens from a multiple of 16 on lie in one block, so a group has one address and one pair of scales.
template <int D, int NT, bool kGrouped>
struct Tile {
    float o[NT][D / 16][4];
    float top[NT][2], sum[NT][2];          // of columns 2t, 2t + 1

    __device__ __forceinline__ void run(const AttnParams &p, const Req &r, const int32_t *table, int head,
                                        int rt, int ua, int ub, Stage<D> *ring) {
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
        const int some_lo = lo_of(p, pos_first), some_hi = min(pos_last + 1, r.keys);
        const int all_lo = lo_of(p, pos_last), all_hi = min(pos_first + 1, r.keys);
        ua = max(ua, (some_lo - base) / kUnit);
        ub = min(ub, some_hi > base ? (some_hi - base + kUnit - 1) / kUnit : 0);
        if (ua >= ub) return;

        const int64_t line = static_cast<int64_t>(p.Hkv) * D;
        // copying: this lane moves 16 bytes of every kRows-th row, so that eight lanes ask for 128 (or
        // 64) consecutive bytes
        const int crow = lane / St::kRowLanes, cpiece = lane % St::kRowLanes;
        const uint8_t *kh = p.kc + head * D + 16 * cpiece + (kGrouped ? crow * line : 0);
        const uint8_t *vh = p.vc + head * D + 16 * cpiece + (kGrouped ? crow * line : 0);

        // Block id of token `lane`'s (group of) unit u: asked for one unit ahead, looked at by place().
        auto ask = [&](int u) {
            const int s = base + u * kUnit + (kGrouped ? lane & 16 : lane);
            return u < ub && s < some_hi ? p.table_at(table, s) : -1;
        };
        // Where a unit's lines are: a bit for each token that is read; the offset of each group's first
        // line (kGrouped) or this lane's token's slot.
        struct Place {
            uint32_t mask, slot;
            int64_t at[2];
            int32_t block;
        };
        auto place = [&](int u, int block) {
            Place y;
            const int s = base + u * kUnit + lane;
            if (block >= p.num_blocks) {
                if (p.err && s >= some_lo && s < some_hi) atomicOr(p.err, PKV_DEVERR_BLOCK);
                block = -1;
            }
            y.block = block;
            y.mask = __ballot_sync(~0u, u < ub && block >= 0 && s >= some_lo && s < some_hi);
            y.slot = static_cast<uint32_t>(block) * static_cast<uint32_t>(p.bs) + static_cast<uint32_t>(s) % static_cast<uint32_t>(p.bs);
            if constexpr (kGrouped) {
                y.at[0] = static_cast<int64_t>(__shfl_sync(~0u, y.slot, 0)) * line;
                y.at[1] = static_cast<int64_t>(__shfl_sync(~0u, y.slot, 16)) * line;
            }
            return y;
        };
        auto fetch = [&](const Place &y, const uint8_t *from, char *to) {
            if (kGrouped && y.mask == ~0u) {
#pragma unroll
                for (int i = 0; i < kUnit; i += St::kRows) {
                    const int r = i + crow;
                    cp_async_full<16>(smem_addr(to + r * D + 16 * swizzle<D>(cpiece, r)), from + y.at[i >> 4] + (i & 15) * line);
                }
            } else {
#pragma unroll
                for (int i = 0; i < kUnit; i += St::kRows) {
                    const int r = i + crow;
                    const bool on = (y.mask >> r) & 1;
                    const int64_t x = kGrouped ? y.at[i >> 4] + (i & 15) * line
                                               : static_cast<int64_t>(__shfl_sync(~0u, y.slot, r)) * line;
                    cp_async<16>(smem_addr(to + r * D + 16 * swizzle<D>(cpiece, r)), from + (on ? x : 0), on);
                }
            }
        };
        // A stage's keys are refilled when every lane has taken them out, then its values.
        auto fetch_k = [&](const Place &y, Stage<D> &st) {
            // a group's scales count where some row sees one of its tokens: whatever those of an unseen block
            // hold (one given away before the window) stays out
            const bool on = (y.mask >> (kGrouped ? lane & 16 : lane)) & (kGrouped ? 0xffffu : 1u);
            const int64_t sc = on ? static_cast<int64_t>(y.block) * p.Hkv + head : 0;
            if constexpr (kGrouped) {
                // lanes 0, 16: K scales; lanes 1, 17: V scales
                if ((lane & 15) < 2) cp_async<4>(smem_addr(&(lane & 1 ? st.vs : st.ks)[lane >> 4]), (lane & 1 ? p.vs : p.ks) + sc, on);
            } else {
                cp_async<4>(smem_addr(&st.ks[lane]), p.ks + sc, on);
                cp_async<4>(smem_addr(&st.vs[lane]), p.vs + sc, on);
            }
            fetch(y, kh, st.k);
            cp_commit();
        };
        auto fetch_v = [&](const Place &y, Stage<D> &st) {
            fetch(y, vh, st.v);
            cp_commit();
        };

        __syncwarp();
        uint32_t masks[kDepth];                // of units u, u + 1, ..
#pragma unroll
        for (int k = 0; k < kDepth; k++) {
            const Place y = place(ua + k, ask(ua + k));
            masks[k] = y.mask;
            fetch_k(y, ring[(ua + k) % kDepth]);
            fetch_v(y, ring[(ua + k) % kDepth]);
        }
        int ahead = ask(ua + kDepth);
        for (int u = ua; u < ub; u++) {
            Stage<D> &st = ring[u % kDepth];
            const Place next = place(u + kDepth, ahead);
            ahead = ask(u + kDepth + 1);
            const uint32_t mask = masks[0];
            const int s0 = base + u * kUnit;
            cp_wait<2 * kDepth - 1>();         // the keys are here, all later copies may be on their way
            __syncwarp();
            float ks[2][2], vs[2][2];
#pragma unroll
            for (int q = 0; q < 2; q++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const int at = kGrouped ? q : 16 * q + g + 8 * h;
                    ks[q][h] = st.ks[at];
                    vs[q][h] = value_scale(st.vs[at]);
                }
            float x[2][NT][4];
#pragma unroll
            for (int q = 0; q < 2; q++) {
#pragma unroll
                for (int nt = 0; nt < NT; nt++)
#pragma unroll
                    for (int c = 0; c < 4; c++) x[q][nt][c] = 0.f;
            }
#pragma unroll
            for (int c = 0; c < St::kKPieces; c++) {
                uint4 ka[2], kb[2];
#pragma unroll
                for (int q = 0; q < 2; q++) {
                    const char *row = st.k + (16 * q + g) * D + 16 * swizzle<D>(4 * c + t, g);
                    ka[q] = *reinterpret_cast<const uint4 *>(row);
                    kb[q] = *reinterpret_cast<const uint4 *>(row + 8 * D);
                }
#pragma unroll
                for (int i = 0; i < 4; i++)
#pragma unroll
                    for (int q = 0; q < 2; q++) {
                        const uint32_t wa = i == 0 ? ka[q].x : i == 1 ? ka[q].y : i == 2 ? ka[q].z : ka[q].w;
                        const uint32_t wb = i == 0 ? kb[q].x : i == 1 ? kb[q].y : i == 2 ? kb[q].z : kb[q].w;
                        const uint32_t a[4] = {f16x2_of(wa), f16x2_of(wb), f16x2_of(wa >> 16), f16x2_of(wb >> 16)};
#pragma unroll
                        for (int nt = 0; nt < NT; nt++) mma_f16(x[q][nt], a, qb[nt][4 * c + i][0], qb[nt][4 * c + i][1]);
                    }
            }
            __syncwarp();
            fetch_k(next, st);
            const bool whole = mask == ~0u && s0 >= all_lo && s0 + kUnit <= all_hi;
            float iv[2][2];                    // of the lane's tokens g, g + 8 of both groups
            uint32_t seen[NT];                 // bit 4 q + c: the lane's value is visible
#pragma unroll
            for (int nt = 0; nt < NT; nt++) seen[nt] = 255;
#pragma unroll
            for (int q = 0; q < 2; q++)
#pragma unroll
                for (int h = 0; h < 2; h++) {
                    const float lv = __log2f(vs[q][h]);
                    iv[q][h] = __frcp_rn(vs[q][h]);
#pragma unroll
                    for (int nt = 0; nt < NT; nt++)
#pragma unroll
                        for (int col = 0; col < 2; col++) {
                            float &y = x[q][nt][2 * h + col];
                            y = fmaf(y, cf[nt][col] * ks[q][h], lv);
                        }
                }
            if (!whole) {
#pragma unroll
                for (int q = 0; q < 2; q++)
#pragma unroll
                    for (int nt = 0; nt < NT; nt++)
#pragma unroll
                        for (int c = 0; c < 4; c++) {
                            const int tok = 16 * q + g + 8 * (c >> 1), s = s0 + tok;
                            const bool ok = ((mask >> tok) & 1) && s <= pos[nt][c & 1] && s >= lo_of(p, pos[nt][c & 1]);
                            if (!ok) {
                                x[q][nt][c] = -INFINITY;
                                seen[nt] &= ~(1u << (4 * q + c));
                            }
                        }
            }
            // R follows the maximum only where a row's values outgrow it (or it has seen nothing yet)
            bool grow = false;
            float most[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int col = 0; col < 2; col++) {
                    most[nt][col] = fmaxf(fmaxf(x[0][nt][col], x[0][nt][2 + col]), fmaxf(x[1][nt][col], x[1][nt][2 + col]));
                    grow |= most[nt][col] > top[nt][col] + kSlack;
                }
            if (__any_sync(~0u, grow)) {
#pragma unroll
                for (int nt = 0; nt < NT; nt++) {
                    float a[2];
#pragma unroll
                    for (int col = 0; col < 2; col++) {
                        float m = most[nt][col];
                        m = fmaxf(m, __shfl_xor_sync(~0u, m, 4));
                        m = fmaxf(m, __shfl_xor_sync(~0u, m, 8));
                        m = fmaxf(m, __shfl_xor_sync(~0u, m, 16));
                        m = fmaxf(m, top[nt][col]);
                        a[col] = m > top[nt][col] ? exp2_fast(top[nt][col] - m) : 1.f;
                        top[nt][col] = m;
                        sum[nt][col] *= a[col];
                    }
#pragma unroll
                    for (int j = 0; j < S; j++)
#pragma unroll
                        for (int c = 0; c < 4; c++) o[nt][j][c] *= a[c & 1];
                }
            }
            uint32_t pb[2][NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
                const float ref[2] = {top[nt][0] == -INFINITY ? 0.f : top[nt][0], top[nt][1] == -INFINITY ? 0.f : top[nt][1]};
#pragma unroll
                for (int q = 0; q < 2; q++) {
                    float w[4];
#pragma unroll
                    for (int c = 0; c < 4; c++) {
                        w[c] = exp2_fast(x[q][nt][c] - ref[c & 1]);
                        sum[nt][c & 1] = fmaf(w[c], iv[q][c >> 1], sum[nt][c & 1]);
                    }
                    pb[q][nt][0] = transpose8x8(pack_f16(w[0], w[1]));
                    pb[q][nt][1] = transpose8x8(pack_f16(w[2], w[3]));
                }
            }
            cp_wait<2 * kDepth - 1>();         // the values are here
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 2; q++)
#pragma unroll
                for (int c = 0; c < St::kVPieces; c++) {
                    uint32_t w[4][St::kVBytes / 4];
#pragma unroll
                    for (int h = 0; h < 4; h++) {
                        const int r = 16 * q + 2 * t + (h & 1) + 8 * (h >> 1);
                        if constexpr (St::kVBytes == 16) {
                            const uint4 y = *reinterpret_cast<const uint4 *>(st.v + r * D + 16 * swizzle<D>(8 * c + g, r));
                            w[h][0] = y.x;
                            w[h][1] = y.y;
                            w[h][2] = y.z;
                            w[h][3] = y.w;
                        } else {
                            const uint2 y = *reinterpret_cast<const uint2 *>(st.v + r * D + 16 * swizzle<D>(g >> 1, r) + 8 * (g & 1));
                            w[h][0] = y.x;
                            w[h][1] = y.y;
                        }
                    }
                    if (!whole && r.count > 1) keep_nan_apart(w, q, c, seen);
#pragma unroll
                    for (int i = 0; i < St::kVBytes / 4; i++)
#pragma unroll
                        for (int half = 0; half < 2; half++) {
                            // dimensions 4 i + 2 half (row g) and + 1 (row g + 8), tokens (2t, 2t+1) and (2t+8, 2t+9)
                            const uint32_t sel = half ? 0x7362 : 0x5140;
                            const uint32_t lo = __byte_perm(w[0][i], w[1][i], sel), hi = __byte_perm(w[2][i], w[3][i], sel);
                            const int j = c * (St::kVBytes / 2) + 2 * i + half;
                            const uint32_t a[4] = {f16x2_of(lo), f16x2_of(lo >> 16), f16x2_of(hi), f16x2_of(hi >> 16)};
#pragma unroll
                            for (int nt = 0; nt < NT; nt++) mma_f16(o[nt][j], a, pb[q][nt][0], pb[q][nt][1]);
                        }
                }
            __syncwarp();
            fetch_v(next, st);
#pragma unroll
            for (int k = 0; k + 1 < kDepth; k++) masks[k] = masks[k + 1];
            masks[kDepth - 1] = next.mask;
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

    // Where rows differ in the tokens they see, a row must not meet a NaN code of a token that only
    // other rows see (0 * NaN): such codes leave the product, and the accumulators of the rows that do
    // see them become NaN.
    __device__ __forceinline__ void keep_nan_apart(uint32_t (&w)[4][Stage<D>::kVBytes / 4], int q, int c, const uint32_t (&seen)[NT]) {
        constexpr int kWords = Stage<D>::kVBytes / 4;
        bool nan = false;
#pragma unroll
        for (int h = 0; h < 4; h++)
#pragma unroll
            for (int i = 0; i < kWords; i++) nan |= (((w[h][i] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
        if (!__any_sync(~0u, nan)) return;
#pragma unroll
        for (int i = 0; i < kWords; i++)
#pragma unroll
            for (int half = 0; half < 2; half++) {
                const uint32_t sel = half ? 0x7362 : 0x5140;
                const uint32_t nl = __vcmpeq4(__byte_perm(w[0][i], w[1][i], sel) & 0x7f7f7f7fu, 0x7f7f7f7fu) & 0x38383838u;
                const uint32_t nh = __vcmpeq4(__byte_perm(w[2][i], w[3][i], sel) & 0x7f7f7f7fu, 0x7f7f7f7fu) & 0x38383838u;
                const uint32_t a[4] = {f16x2_of(nl), f16x2_of(nl >> 16), f16x2_of(nh), f16x2_of(nh >> 16)};   // ones
#pragma unroll
                for (int nt = 0; nt < NT; nt++) {
                    const uint32_t one = 0x3c00u, m = seen[nt] >> (4 * q);
                    const uint32_t s01 = ((m & 1) ? one : 0) | ((m & 2) ? one << 16 : 0);
                    const uint32_t s23 = ((m & 4) ? one : 0) | ((m & 8) ? one << 16 : 0);
                    float hit[4] = {0.f, 0.f, 0.f, 0.f};
                    mma_f16(hit, a, transpose8x8(s01), transpose8x8(s23));
#pragma unroll
                    for (int k = 0; k < 4; k++)
                        if (hit[k] > 0.f) o[nt][c * (2 * kWords) + 2 * i + half][k] = NAN;
                }
            }
#pragma unroll
        for (int h = 0; h < 4; h++)
#pragma unroll
            for (int i = 0; i < kWords; i++) w[h][i] &= ~__vcmpeq4(w[h][i] & 0x7f7f7f7fu, 0x7f7f7f7fu);
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

template <int D, int NT, bool kGrouped>
__global__ void __launch_bounds__(32 * warps_of<D, NT>(), 1) kv8_decode_kernel(const AttnParams p) {
    constexpr int kWarps = warps_of<D, NT>(), kThreads = 32 * kWarps;
    constexpr int kPart = 8 * NT * (D + 2);
    extern __shared__ __align__(16) char s_ring[];
    __shared__ int64_t s_prefix[kThreads + 1];
    __shared__ int64_t s_warp[kWarps];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // what the ranges are cut from: a request's units, or its row tiles
    auto share = [&](const Req &r) {
        int per;
        const int64_t k = units_of_request<NT>(p, r, &per);
        return p.whole ? k / per : k;
    };
    auto units = [&](int i) { return share(request_of(p, i)); };
    const int64_t total = plan_prefix<kThreads>(s_prefix, s_warp, p.n, [&](int i) { return share(request_of(p, i, blockIdx.x == 0)); });
    const int worker = blockIdx.x * kWarps + warp;
    const int64_t all = static_cast<int64_t>(gridDim.x) * kWarps / p.Hkv;     // ranges the batch is cut into
    const int64_t ranges = total < all ? total : all;
    const int range = worker / p.Hkv, head = worker - range * p.Hkv;
    int4 note = make_int4(-1, 0, 0, 0);
    if (range < ranges) {
        int64_t u = range * total / ranges;
        const int64_t end = (range + 1) * total / ranges;
        Stage<D> *ring = reinterpret_cast<Stage<D> *>(s_ring) + warp * kDepth;
        int64_t first;
        int i = plan_find<kThreads>(s_prefix, p.n, u, units, &first);
        while (u < end) {
            const Req r = request_of(p, i);
            int per;
            const int64_t all_units = units_of_request<NT>(p, r, &per);
            const int64_t k = p.whole ? all_units / per : all_units;
            if (u >= first + k) {
                first += k;
                i++;
                continue;
            }
            const int cut = p.whole ? 1 : per;                                // shares of a row tile
            const int rt = static_cast<int>((u - first) / cut);
            const int64_t tile = first + static_cast<int64_t>(rt) * cut;      // the tile's first share
            const int ua = p.whole ? 0 : static_cast<int>(u - tile);
            const int ub = p.whole ? per : static_cast<int>(end - tile < per ? end - tile : per);
            Tile<D, NT, kGrouped> x;
            x.run(p, r, p.tables + static_cast<int64_t>(i) * p.W, head, rt, ua, ub, ring);
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
            u = p.whole ? u + 1 : tile + ub;
        }
    }
    if (lane == 0) p.meta[worker] = note;
}

// Merge the partial results of the tiles that were cut, a warp per (worker, row).
constexpr int kMergeThreads = 256;

// kBatch: partial rows on their way at a time.  Sixteen for the long chains of a few decodes (four long
// ones 139 us, with eight 144), eight for a full batch (256 decodes 389 us, with sixteen 398: fewer
// warps resident), two for the thousands of rows of row tiles, mostly of two pieces.
template <int D, int kBatch>
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
    for (int k0 = 0; k0 < pieces; k0 += 32) {
        // a piece's factor, in the lane of its number; a piece without a top adds nothing, unless its
        // logits were NaN
        float fac = 0.f;
        if (k0 + lane < pieces) {
            const float *a = part(k0 + lane);
            const float m = a[row], l = a[rows + row];
            fac = m == -INFINITY ? (l == 0.f ? 0.f : NAN) : exp2_fast(m - top);
            sum += fac * l;
        }
        const int n = min(32, pieces - k0);
        for (int k1 = 0; k1 < n; k1 += kBatch) {
            float y[kBatch][kPer];
#pragma unroll
            for (int k = 0; k < kBatch; k++) {
                const float *o = part(k0 + min(k1 + k, n - 1)) + 2 * rows + row * D + lane * kPer;
#pragma unroll
                for (int c = 0; c < kPer; c += 2) {
                    const float2 z = *reinterpret_cast<const float2 *>(o + c);
                    y[k][c] = z.x;
                    y[k][c + 1] = z.y;
                }
            }
#pragma unroll
            for (int k = 0; k < kBatch; k++) {
                const float f2 = __shfl_sync(~0u, fac, k1 + k);
                if (k1 + k < n && f2 != 0.f) {
#pragma unroll
                    for (int c = 0; c < kPer; c++) acc[c] = fmaf(f2, y[k][c], acc[c]);
                }
            }
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
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

template <int D, int NT, bool kGrouped>
int launch(const AttnParams &p, int sms, cudaStream_t s) {
    constexpr int kWarps = warps_of<D, NT>();
    constexpr size_t smem = sizeof(Stage<D>) * kDepth * kWarps;
    static_assert(smem <= 220 * 1024, "shared memory");
    static bool set[64] = {false};
    const int rc = kv8_allow_smem(reinterpret_cast<const void *>(kv8_decode_kernel<D, NT, kGrouped>), static_cast<int>(smem), set);
    if (rc != PKV_OK) return rc;
    static_assert(kWarps <= kMaxWarps, "the workspace holds this many");
    // One CTA an SM, or as many as the longest requests the tables can name would give a unit a warp; but a
    // warp for each KV head at least (with head_dim 256 there are more heads than warps from 913 on), or
    // the batch would have no range.
    const int64_t tiles = static_cast<int64_t>(p.T) * p.G / (8 * NT) + p.n;
    const int64_t most = tiles * (static_cast<int64_t>(p.W) * p.bs / kUnit + 2) * p.Hkv;
    const int least = (p.Hkv + kWarps - 1) / kWarps, full = sms > least ? sms : least;
    const int grid = most < static_cast<int64_t>(full) * kWarps ? static_cast<int>((most + kWarps - 1) / kWarps) : full;
    PKV_CUDA_TRY(launch_pdl(kv8_decode_kernel<D, NT, kGrouped>, dim3(grid), dim3(32 * kWarps), smem, s, p));
    return p.whole ? PKV_OK : kv8_launch_merge(p, D, 8 * NT, grid * kWarps, p.Hkv, s);
}

template <int D>
int launch_rows(const AttnParams &p, bool one_tile, int sms, cudaStream_t s) {
    if (p.bs % 16 == 0) return one_tile ? launch<D, 1, true>(p, sms, s) : launch<D, 2, true>(p, sms, s);
    return one_tile ? launch<D, 1, false>(p, sms, s) : launch<D, 2, false>(p, sms, s);
}

}  // namespace

int kv8_launch_merge(const AttnParams &p, int32_t head_dim, int rows, int workers, int stride, cudaStream_t s) {
    const dim3 grid((static_cast<unsigned>(workers) * rows + kMergeThreads / 32 - 1) / (kMergeThreads / 32)), block(kMergeThreads);
    const int64_t tiles = (static_cast<int64_t>(p.T) * p.G / rows + p.n) * p.Hkv;
    const bool tile = rows > 16, chains = tiles * 8 <= workers;
    auto kernel = head_dim == 64    ? (tile ? kv8_merge_kernel<64, 2> : chains ? kv8_merge_kernel<64, 16> : kv8_merge_kernel<64, 8>)
                  : head_dim == 128 ? (tile ? kv8_merge_kernel<128, 2> : chains ? kv8_merge_kernel<128, 16> : kv8_merge_kernel<128, 8>)
                                    : kv8_merge_kernel<256, 8>;
    PKV_CUDA_TRY(launch_pdl(kernel, grid, block, 0, s, p, rows, workers, stride));
    return PKV_OK;
}

int64_t kv8_decode_workspace(int32_t head_dim, int sms) {
    // a note and two partial results of 16 rows (the widest variant's) for each warp
    return kv8_most_workers(sms) * (2LL * 16 * (head_dim + 2) * 4 + 16);
}

int kv8_launch_decode(const AttnParams &p, int32_t head_dim, bool one_tile, int sms, cudaStream_t s) {
    if (head_dim == 64) return launch_rows<64>(p, one_tile, sms, s);
    if (head_dim == 128) return launch_rows<128>(p, one_tile, sms, s);
    return launch_rows<256>(p, one_tile, sms, s);
}

}  // namespace pkv
