// Attention over the 4-bit paged cache for requests with few query rows
// (single tokens, drafted tokens).
//
// Mathematics.  Row r = (query j, head of the KV head's group), key s: x = (q . k) *
// softmax_scale * log2(e) * k_unit, with k = code * scale exact in f16 (an e2m1 value has two
// significant bits, an e4m3 scale four).  R, a row's reference, is 11 to 15 below the running
// maximum of x.  w = 2^(x - R) <= 2^15 is rounded to f16 for the second product: off by 2^-11 of
// itself, or by 2^-25 where it is below 2^-14, which is 2^-36 of the largest weight: n such tokens put
// the output off by n 2^-36 of the largest |value| at most.  out = v_unit * sum w v / sum w, lse = R ln 2 +
// ln sum w, both sums in fp32.
//
// Bound: HBM, 2 * (D / 2 + D / 16) bytes per (cached token, KV head), each read once; next to it
// the conversions, one cvt and one multiplication by the scale for every two elements.
//
// Layout.  Every warp works alone: it owns one KV head and a contiguous range of
// 32-token units of the batch.  The lines of a (block, head) stand next to each other, so a
// copy instruction asks for 512 consecutive bytes.  Keys are the M side of the products (S^T = K
// Q^T, O^T = V^T P^T), so eight rows fill the N side.  A warp copies its units with
// cp.async into a stage of its own, whose halves (keys, values) it refills as soon as it
// has taken them out.  Codes of two tokens are merged nibble by nibble (two shifts and two
// selections for 16 codes) before the conversion, so V needs no transpose; P moves from
// accumulator to operand layout with movmatrix.
// A range that ends inside a request leaves a partial result (R, sum, O) that a second
// kernel merges in a fixed order.
//
// Measured, with the merge: 256 single tokens, 32 query and 8 KV heads of 128, contexts up to 8192 (1.16 GB) 221 us,
// 78 % of the copy rate; four of 64 query heads on 65536 to 131072 tokens (455 MB) 96 us, 70 %; 96 requests
// of two to six tokens, 40 query heads, a window of 4096 (411 MB; a request of more than 16 rows takes two tiles,
// which both go through its lines) 220 us.  Of head_dim 256, 4 KV heads: 256 single tokens as many bytes 218 us; 96 requests
// of two to six tokens 198 us (324 bytes of registers spilled a thread); prompt chunks, which the prefill kernel does not
// take, 2330 us for the 522 GFLOP that it does in 460 of head_dim 128.
// Instructions bound it next to HBM: 129 for 1 KB of codes with eight rows, 0.6 a cycle issued, the
// integer pipe 50 % busy with the conversions.  Tiles of eight rows: twelve warps an SM, 221 us for the 256; eight 262, ten
// 264, thirteen 261, fourteen 246, sixteen (spilling) 236; queries in registers 224; a second unit on its way 224.  Tiles of
// sixteen rows: eight warps 218 us for the 96 requests; twelve 222, queries in registers
// 227 and (twelve, spilling) 232; 24 rows 262; as many groups of eight rows as a request needs, up to 32, 269.
// Of head_dim 64 sixteen warps 151 us for the 256 where twelve take 159, with sixteen rows twelve 274 where eight take 326; of
// 256 queries in registers 223 us (128 requests of up to five tokens) where shared memory takes 227.
#include "pkv_kv4_attention.cuh"
#include "pkv_tcgen05.cuh"

namespace pkv {
namespace {

constexpr int kUnit = 32;          // tokens per unit, two groups of 16, each inside one block
constexpr int kDepth = 1;          // units whose codes are held or on their way
constexpr float kHead = 11.f;      // how far below a row's maximum (log2) R is set,
constexpr float kSlack = 15.f;     // and how far it may come to be

// A unit's codes (places: at<D>()) and scales, D / 16 bytes a token.
template <int D>
struct Stage {
    char k[kUnit * D / 2], v[kUnit * D / 2];
    char ks[kUnit * D / 16], vs[kUnit * D / 16];
};

// Where a token's 16-byte piece of codes lies in a stage.  Rows and pieces are permuted so that the
// fragment reads (keys: eight tokens, 8 or 16 bytes a lane; values: the tokens 2 t + h, 4, 8 or 16
// bytes a lane) meet every bank once.
template <int D>
__device__ __forceinline__ int at(int token, int piece) {
    if constexpr (D == 64) return (token ^ ((token >> 2) & 1)) * 32 + 16 * piece;
    if constexpr (D == 128) return (token ^ ((token >> 1) & 1)) * 64 + 16 * (piece ^ ((token & 4) >> 1));
    return token * 128 + 16 * (piece ^ (token & 6) ^ ((token & 1) << 2));
}

// Warps of an SM.  Four schedulers share them, so that numbers between these are slower than both neighbours.
template <int D, int NT>
constexpr int warps_of() { return D == 64 ? (NT > 1 ? 12 : 16) : D == 128 && NT == 1 ? 12 : 8; }

// Queries lie in shared memory (with the accumulator they are more than the registers that leave enough warps): fragments
// of two steps, 16 bytes a lane, for each eight rows.  For D = 256 registers spill either way.
template <int D, int NT>
constexpr int query_bytes() { return D < 256 ? 8 * NT * D * 2 : 0; }

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

// One (query, head) row's fragments, scaled by 2^(14 - E) (and negated for a negative softmax scale, so
// that a larger product is a larger x): element pairs of this lane's dimensions (step
// j has four: of D = 64 16 t + 4 j, otherwise 128 (j / 8) + 32 t + 4 (j % 8)); returns E.
template <int D>
__device__ __forceinline__ int load_row(uint32_t (&qb)[D / 16][2], const char *row, bool live, int t, bool fp16, bool negative) {
    uint2 raw[D / 16];
    float largest = 0.f;
#pragma unroll
    for (int j = 0; j < D / 16; j++) {
        raw[j] = make_uint2(0, 0);
        const int dim = D == 64 ? 16 * t + 4 * j : 128 * (j / 8) + 32 * t + 4 * (j % 8);
        if (live) raw[j] = __ldg(reinterpret_cast<const uint2 *>(row + 2 * dim));
        const float2 a = widen2(raw[j].x, fp16), b = widen2(raw[j].y, fp16);
        largest = fmaxf(fmaxf(largest, fmaxf(fabsf(a.x), fabsf(a.y))), fmaxf(fabsf(b.x), fabsf(b.y)));
    }
    largest = fmaxf(largest, __shfl_xor_sync(~0u, largest, 1));
    largest = fmaxf(largest, __shfl_xor_sync(~0u, largest, 2));
    const int e = row_exponent(largest);
    const float f = negative ? -power2(14 - e) : power2(14 - e);
#pragma unroll
    for (int j = 0; j < D / 16; j++) {
        const float2 a = widen2(raw[j].x, fp16), b = widen2(raw[j].y, fp16);
        qb[j][0] = pack_f16(a.x * f, a.y * f);
        qb[j][1] = pack_f16(b.x * f, b.y * f);
    }
    return e;
}

// One warp's pass over units ua..ub-1 of row tile `rt` of a request and one KV head.
template <int D, int NT>
struct Tile {
    static constexpr int kOwn = D / 8;     // dimensions of O that a lane holds, in order from kOwn * g on
    float o[NT][D / 16][4];
    float top[NT][2], sum[NT][2];          // R and the sum of w, of columns 2t, 2t + 1

    __device__ __forceinline__ void run(const Kv4Params &p, const Req &r, const int32_t *table, int head, int rt, int ua, int ub,
                                        Stage<D> *ring, uint4 *queries) {
        constexpr int S = D / 16;
        constexpr bool kShared = query_bytes<D, NT>() > 0;
        constexpr int kPieces = D / 32;                    // 16-byte pieces of a token's codes
        const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
        const int rows = r.count * p.G;
        const bool fp16 = p.fp16 != 0;

        float cf[NT][2];
        uint32_t qb[kShared ? 1 : NT][S][2];
        __syncwarp();                          // the last tile's queries have been read
#pragma unroll
        for (int nt = 0; nt < NT; nt++) {
            const int f = rt * 8 * NT + nt * 8 + g;
            const int j = f / p.G;
            const char *row = p.q + static_cast<int64_t>(r.start + j) * p.q_stride +
                              2 * static_cast<int64_t>(head * p.G + f - j * p.G) * D;
            uint32_t(&fr)[S][2] = qb[kShared ? 0 : nt];
            const int e = load_row<D>(fr, row, f < rows, t, fp16, p.scale_log2 < 0.f);
            if constexpr (kShared) {
#pragma unroll
                for (int j2 = 0; j2 < S; j2 += 2)
                    queries[(j2 / 2 * NT + nt) * 32 + lane] = make_uint4(fr[j2][0], fr[j2][1], fr[j2 + 1][0], fr[j2 + 1][1]);
            }
#pragma unroll
            for (int c = 0; c < 2; c++) {
                // never zero, so that a hidden score stays -inf
                cf[nt][c] = fmaxf(fabsf(p.scale_log2) * power2(__shfl_sync(~0u, e, (2 * t + c) * 4) - 14), 1e-37f);
                top[nt][c] = -INFINITY;
                sum[nt][c] = 0.f;
            }
#pragma unroll
            for (int j2 = 0; j2 < S; j2++)
#pragma unroll
                for (int c = 0; c < 4; c++) o[nt][j2][c] = 0.f;
        }
        // position of the row in column 2 t + c of eight rows, -1 where there is none
        auto pos_of = [&](int nt, int c) {
            const int f = rt * 8 * NT + nt * 8 + 2 * t + c;
            return f < rows ? r.len - r.count + f / p.G : -1;
        };
        const int first_row = rt * 8 * NT, last_row = min(rows, first_row + 8 * NT) - 1;
        const int pos_first = r.len - r.count + first_row / p.G, pos_last = r.len - r.count + last_row / p.G;
        const int base = r.lo & ~(kUnit - 1);
        // keys that some row of the tile sees, and those that every row sees
        const int some_lo = lo_of(p, pos_first), some_hi = min(pos_last + 1, r.keys);
        const int all_lo = lo_of(p, pos_last), all_hi = min(pos_first + 1, r.keys);
        ua = max(ua, (some_lo - base) / kUnit);
        ub = min(ub, some_hi > base ? (some_hi - base + kUnit - 1) / kUnit : 0);
        if (ua >= ub) return;

        // Each half of the warp copies one of a unit's two groups: its block's table entry and the group's
        // place in the block, for the unit that is asked for next; 32 tokens further without a division.
        const int half = lane >> 4, own = lane & 15;
        const int jump = kUnit / p.bs, rest = kUnit - jump * p.bs;
        int entry = (base + ua * kUnit + 16 * half) / p.bs, offset = base + ua * kUnit + 16 * half - entry * p.bs;
        struct Asked {
            int block, offset;
        };
        auto ask = [&](int u) {
            Asked y;
            const int s = base + u * kUnit + 16 * half;
            y.block = u < ub && s < some_hi && entry < p.W ? table[entry] : -1;
            y.offset = offset;
            entry += jump;
            offset += rest;
            if (offset >= p.bs) {
                offset -= p.bs;
                entry++;
            }
            return y;
        };
        // Where a unit's lines are: a bit for each token that is read, the half's first line.
        struct Place {
            uint32_t mask;
            int64_t line;
        };
        auto place = [&](int u, Asked x) {
            Place y;
            const int s = base + u * kUnit + lane;
            if (x.block >= p.num_blocks) {
                if (p.err && s >= some_lo && s < some_hi) atomicOr(p.err, PKV_DEVERR_BLOCK);
                x.block = -1;
            }
            y.mask = __ballot_sync(~0u, u < ub && x.block >= 0 && s >= some_lo && s < some_hi);
            y.line = (static_cast<int64_t>(x.block) * p.Hkv + head) * p.bs + x.offset;
            return y;
        };
        // Lane `own` copies the pieces own, own + 16, .. of its half's codes (they lie one behind the other), and
        // one piece of its scales, which are those of 256 / D tokens.  What is not read becomes zeros.
        const uint32_t place0 = static_cast<uint32_t>(at<D>(16 * half + own / kPieces, own % kPieces));
        auto fetch = [&](const Place &y, const uint8_t *codes, const uint8_t *scales, char *to, char *to_scales) {
            const uint8_t *from = codes + y.line * (D / 2) + 16 * own, *sf = scales + y.line * (D / 16) + 16 * own;
            const uint32_t dst = smem_addr(to) + place0, sdst = smem_addr(to_scales) + half * D + 16 * own;
            // the place of piece own + 16 i, by the permutations of at()
            auto piece = [&](int i) {
                return D == 64 ? dst + 256 * i : D == 128 ? (dst ^ (32 * (i & 1))) + 256 * i : (dst ^ (32 * (i & 3))) + 256 * i;
            };
            if (y.mask == ~0u) {
#pragma unroll
                for (int i = 0; i < kPieces; i++) cp_async_full<16>(piece(i), from + 256 * i);
                if (own < D / 16) cp_async_full<16>(sdst, sf);
            } else {
                const uint32_t on = y.mask >> (16 * half);
#pragma unroll
                for (int i = 0; i < kPieces; i++) {
                    const bool yes = (on >> ((own + 16 * i) / kPieces)) & 1;
                    cp_async<16>(piece(i), yes ? from + 256 * i : codes, yes);
                }
                constexpr int kTok = 256 / D, kBytes = D / 16;
                if (own < D / 16) {
#pragma unroll
                    for (int w = 0; w < kTok; w++) {
                        const bool yes = (on >> (own * kTok + w)) & 1;
                        cp_async<kBytes>(sdst + kBytes * w, yes ? sf + kBytes * w : scales, yes);
                    }
                }
            }
        };
        // A stage's keys are refilled when every lane has taken them out, then its values.
        auto fetch_k = [&](const Place &y, Stage<D> &st) {
            fetch(y, p.kc, p.k_sf, st.k, st.ks);
            cp_commit();
        };
        auto fetch_v = [&](const Place &y, Stage<D> &st) {
            fetch(y, p.vc, p.v_sf, st.v, st.vs);
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
        Asked ahead = ask(ua + kDepth);
        for (int u = ua; u < ub; u++) {
            Stage<D> &st = ring[u % kDepth];
            const Place next = place(u + kDepth, ahead);
            ahead = ask(u + kDepth + 1);
            const uint32_t mask = masks[0];
            const int s0 = base + u * kUnit;
            cp_wait<2 * kDepth - 1>();         // the keys are here, all later copies may be on their way
            __syncwarp();
            float x[2][NT][4];
#pragma unroll
            for (int q = 0; q < 2; q++) {
#pragma unroll
                for (int nt = 0; nt < NT; nt++)
#pragma unroll
                    for (int c = 0; c < 4; c++) x[q][nt][c] = 0.f;
            }
            // step 2 i + half of word i: dimensions 8 i + 4 half .. + 3 of a lane's piece; rows g, g + 8
            auto words = [&](uint32_t wa, uint32_t wb, uint32_t sa, uint32_t sb, int q, int step) {
                uint32_t a[4], b[4];
                f16_of_e2m1x8(wa, a);
                f16_of_e2m1x8(wb, b);
#pragma unroll
                for (int i = 0; i < 4; i++) {
                    a[i] = mul_f16x2(a[i], sa);
                    b[i] = mul_f16x2(b[i], sb);
                }
                const uint32_t f0[4] = {a[0], b[0], a[1], b[1]}, f1[4] = {a[2], b[2], a[3], b[3]};
#pragma unroll
                for (int nt = 0; nt < NT; nt++) {
                    uint4 y;
                    if constexpr (kShared) y = queries[(step / 2 * NT + nt) * 32 + lane];
                    else y = make_uint4(qb[nt][step][0], qb[nt][step][1], qb[nt][step + 1][0], qb[nt][step + 1][1]);
                    mma_f16(x[q][nt], f0, y.x, y.y);
                    mma_f16(x[q][nt], f1, y.z, y.w);
                }
            };
#pragma unroll
            for (int q = 0; q < 2; q++) {
                const int ta = 16 * q + g, tb = ta + 8;
                if constexpr (D == 64) {
                    const uint2 ka = *reinterpret_cast<const uint2 *>(st.k + at<D>(ta, t >> 1) + 8 * (t & 1));
                    const uint2 kb = *reinterpret_cast<const uint2 *>(st.k + at<D>(tb, t >> 1) + 8 * (t & 1));
                    const uint32_t sa = low_twice(f16x2_of(static_cast<uint8_t>(st.ks[ta * 4 + t])));
                    const uint32_t sb = low_twice(f16x2_of(static_cast<uint8_t>(st.ks[tb * 4 + t])));
                    words(ka.x, kb.x, sa, sb, q, 0);
                    words(ka.y, kb.y, sa, sb, q, 2);
                } else {
#pragma unroll
                    for (int c = 0; c < D / 128; c++) {
                        const uint4 ka = *reinterpret_cast<const uint4 *>(st.k + at<D>(ta, 4 * c + t));
                        const uint4 kb = *reinterpret_cast<const uint4 *>(st.k + at<D>(tb, 4 * c + t));
                        const uint32_t sa = f16x2_of(*reinterpret_cast<const uint16_t *>(st.ks + ta * (D / 16) + 8 * c + 2 * t));
                        const uint32_t sb = f16x2_of(*reinterpret_cast<const uint16_t *>(st.ks + tb * (D / 16) + 8 * c + 2 * t));
                        words(ka.x, kb.x, low_twice(sa), low_twice(sb), q, 8 * c);
                        words(ka.y, kb.y, low_twice(sa), low_twice(sb), q, 8 * c + 2);
                        words(ka.z, kb.z, high_twice(sa), high_twice(sb), q, 8 * c + 4);
                        words(ka.w, kb.w, high_twice(sa), high_twice(sb), q, 8 * c + 6);
                    }
                }
            }
            __syncwarp();
            fetch_k(next, st);
            const bool whole = mask == ~0u && s0 >= all_lo && s0 + kUnit <= all_hi;
            if (!whole) {
#pragma unroll
                for (int nt = 0; nt < NT; nt++)
#pragma unroll
                    for (int col = 0; col < 2; col++) {
                        const int pos = pos_of(nt, col), lo = lo_of(p, pos);
#pragma unroll
                        for (int q = 0; q < 2; q++)
#pragma unroll
                            for (int h = 0; h < 2; h++) {
                                const int tok = 16 * q + g + 8 * h, s = s0 + tok;
                                if (!((mask >> tok) & 1) || s > pos || s < lo) x[q][nt][2 * h + col] = -INFINITY;
                            }
                    }
            }
            // R moves only where a row's values outgrow it (or it has seen nothing yet)
            bool grow = false;
            float most[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
#pragma unroll
                for (int col = 0; col < 2; col++) {
                    most[nt][col] = max3(fmaxf(x[0][nt][col], x[0][nt][2 + col]), x[1][nt][col], x[1][nt][2 + col]) * cf[nt][col];
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
                        m = fmaxf(m - kHead, top[nt][col]);
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
                const float ref[2] = {top[nt][0] == -INFINITY ? 0.f : -top[nt][0], top[nt][1] == -INFINITY ? 0.f : -top[nt][1]};
#pragma unroll
                for (int q = 0; q < 2; q++) {
                    float w[4];
#pragma unroll
                    for (int c = 0; c < 4; c++) {
                        // two roundings: the largest logit minus itself is 0, whatever its size
                        w[c] = exp2_fast(__fadd_rn(__fmul_rn(x[q][nt][c], cf[nt][c & 1]), ref[c & 1]));
                        sum[nt][c & 1] += w[c];
                    }
                    pb[q][nt][0] = transpose8x8(pack_f16(w[0], w[1]));
                    pb[q][nt][1] = transpose8x8(pack_f16(w[2], w[3]));
                }
            }
            cp_wait<2 * kDepth - 1>();         // the values are here
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 2; q++) {
                constexpr int kWords = kOwn / 8;
                // words of the lane's dimensions and their scales, of tokens 2t, 2t + 1, 2t + 8, 2t + 9
                uint32_t w[4][kWords], sc[4];
#pragma unroll
                for (int h = 0; h < 4; h++) {
                    const int tok = 16 * q + 2 * t + (h & 1) + 8 * (h >> 1);
                    if constexpr (D == 64) {
                        w[h][0] = *reinterpret_cast<const uint32_t *>(st.v + at<D>(tok, g >> 2) + 4 * (g & 3));
                        sc[h] = static_cast<uint8_t>(st.vs[tok * 4 + (g >> 1)]);
                    } else if constexpr (D == 128) {
                        const uint2 y = *reinterpret_cast<const uint2 *>(st.v + at<D>(tok, g >> 1) + 8 * (g & 1));
                        w[h][0] = y.x;
                        w[h][1] = y.y;
                        sc[h] = static_cast<uint8_t>(st.vs[tok * 8 + g]);
                    } else {
                        const uint4 y = *reinterpret_cast<const uint4 *>(st.v + at<D>(tok, g));
                        w[h][0] = y.x;
                        w[h][1] = y.y;
                        w[h][2] = y.z;
                        w[h][3] = y.w;
                        sc[h] = *reinterpret_cast<const uint16_t *>(st.vs + tok * 16 + 2 * g);
                    }
                }
#pragma unroll
                for (int i = 0; i < kWords; i++) {
                    // scales of the token pairs in this word's group
                    const uint32_t sel = D == 256 && i >= 2 ? 0x0051u : 0x0040u;
                    const uint32_t s01 = f16x2_of(__byte_perm(sc[0], sc[1], sel)), s23 = f16x2_of(__byte_perm(sc[2], sc[3], sel));
                    // even dimensions of both tokens in a byte, then odd ones
                    auto merge = [](uint32_t lo, uint32_t hi, bool odd) {
                        return odd ? ((lo >> 4) & 0x0f0f0f0fu) | (hi & 0xf0f0f0f0u) : (lo & 0x0f0f0f0fu) | ((hi << 4) & 0xf0f0f0f0u);
                    };
                    uint32_t a0[4], a1[4], a2[4], a3[4];
                    f16_of_e2m1x8(merge(w[0][i], w[1][i], false), a0);
                    f16_of_e2m1x8(merge(w[0][i], w[1][i], true), a1);
                    f16_of_e2m1x8(merge(w[2][i], w[3][i], false), a2);
                    f16_of_e2m1x8(merge(w[2][i], w[3][i], true), a3);
#pragma unroll
                    for (int b = 0; b < 4; b++) {
                        const uint32_t f[4] = {mul_f16x2(a0[b], s01), mul_f16x2(a1[b], s01), mul_f16x2(a2[b], s23), mul_f16x2(a3[b], s23)};
#pragma unroll
                        for (int nt = 0; nt < NT; nt++) mma_f16(o[nt][4 * i + b], f, pb[q][nt][0], pb[q][nt][1]);
                    }
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

    __device__ __forceinline__ void write(const Kv4Params &p, const Req &r, int head, int rt) const {
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
                const float inv = none ? 0.f : p.v_unit / sum[nt][col];
                char *row = p.out + static_cast<int64_t>(r.start + j) * p.out_stride + 2 * static_cast<int64_t>(hq) * D;
#pragma unroll
                for (int i = 0; i < D / 16; i += 4) {
                    uint32_t y[4];
#pragma unroll
                    for (int k = 0; k < 4; k++) {
                        const float *a = o[nt][i + k];
                        y[k] = pack_out(none ? 0.f : a[col] * inv, none ? 0.f : a[2 + col] * inv, p.fp16);
                    }
                    *reinterpret_cast<uint4 *>(row + 2 * (kOwn * g + 2 * i)) = make_uint4(y[0], y[1], y[2], y[3]);
                }
                if (g == 0 && p.lse)
                    p.lse[static_cast<int64_t>(r.start + j) * p.Hkv * p.G + hq] =
                        none ? -INFINITY : (top[nt][col] + log2f(sum[nt][col])) * kLn2;
            }
    }

    // A partial result: 8 NT tops, 8 NT sums, then rows of D floats.
    __device__ __forceinline__ void spill(float *part, float v_unit) const {
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
                float *to = part + 16 * NT + row * D + kOwn * g;
#pragma unroll
                for (int i = 0; i < D / 16; i += 2) {
                    const float *a = o[nt][i], *b = o[nt][i + 1];
                    *reinterpret_cast<float4 *>(to + 2 * i) =
                        make_float4(a[col] * v_unit, a[2 + col] * v_unit, b[col] * v_unit, b[2 + col] * v_unit);
                }
            }
    }
};

template <int D, int NT>
__global__ void __launch_bounds__(32 * warps_of<D, NT>(), 1) kv4_decode_kernel(const Kv4Params p) {
    constexpr int kWarps = warps_of<D, NT>(), kThreads = 32 * kWarps;
    constexpr int kPart = 8 * NT * (D + 2);
    extern __shared__ __align__(128) char s_ring[];     // at() permutes address bits up to 64
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
        uint4 *queries = reinterpret_cast<uint4 *>(s_ring + sizeof(Stage<D>) * kDepth * kWarps + warp * query_bytes<D, NT>());
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
            Tile<D, NT> x;
            x.run(p, r, p.tables + static_cast<int64_t>(i) * p.table_row, head, rt, ua, ub, ring, queries);
            if (ua == 0 && ub == per) {
                x.write(p, r, head, rt);
            } else {
                // slot 1: the range where a tile begins, slot 0: one that goes on with it
                x.spill(p.part + (2LL * worker + (ua == 0)) * kPart, p.v_unit);
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

template <int D, int NT>
int launch(const Kv4Params &p, int sms, cudaStream_t s) {
    constexpr int kWarps = warps_of<D, NT>();
    constexpr size_t smem = (sizeof(Stage<D>) * kDepth + query_bytes<D, NT>()) * kWarps;
    static_assert(smem <= 220 * 1024, "shared memory");
    static bool set[64] = {false};
    const int rc = kv8_allow_smem(reinterpret_cast<const void *>(kv4_decode_kernel<D, NT>), static_cast<int>(smem), set);
    if (rc != PKV_OK) return rc;
    static_assert(kWarps <= kMaxWarps, "the workspace holds this many");
    // One CTA an SM, or as many as the longest requests the tables can name would give a unit a warp; but a
    // warp for each KV head at least, or the batch would have no range.
    const int64_t tiles = static_cast<int64_t>(p.T) * p.G / (8 * NT) + p.n;
    const int64_t most = tiles * most_units(p, kUnit) * p.Hkv;
    const int least = (p.Hkv + kWarps - 1) / kWarps, full = sms > least ? sms : least;
    const int grid = most < static_cast<int64_t>(full) * kWarps ? static_cast<int>((most + kWarps - 1) / kWarps) : full;
    PKV_CUDA_TRY(launch_pdl(kv4_decode_kernel<D, NT>, dim3(grid), dim3(32 * kWarps), smem, s, p));
    return p.whole ? PKV_OK : kv4_launch_merge(p, D, 8 * NT, grid * kWarps, p.Hkv, sms, s);
}

}  // namespace

int64_t kv4_decode_workspace(int32_t head_dim, int sms) {
    // a note and two partial results of 16 rows (the widest variant's) for each warp
    return kv8_most_workers(sms) * (2LL * 16 * (head_dim + 2) * 4 + 16);
}

int kv4_launch_decode(const Kv4Params &p, int32_t head_dim, bool one_tile, int sms, cudaStream_t s) {
    if (head_dim == 64) return one_tile ? launch<64, 1>(p, sms, s) : launch<64, 2>(p, sms, s);
    if (head_dim == 128) return one_tile ? launch<128, 1>(p, sms, s) : launch<128, 2>(p, sms, s);
    return one_tile ? launch<256, 1>(p, sms, s) : launch<256, 2>(p, sms, s);
}

}  // namespace pkv
