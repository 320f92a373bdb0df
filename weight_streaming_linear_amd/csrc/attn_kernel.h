// The attention kernel of attn_decode, for one cache format per translation unit.
#pragma once

#include "attn.h"

namespace wsl {
namespace {

typedef short s16x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ bf16x8 as_bf16x8(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

__device__ __forceinline__ f32x4 mfma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
}

__device__ __forceinline__ float scale_of(uint32_t byte) { return __builtin_bit_cast(float, byte << 23); }

__device__ __forceinline__ uint32_t fp8_pair(uint32_t w, float s, bool hi) {
    return hi ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, true))
              : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, s, false));
}

// 32 keys or values of one head as loaded: bf16 elements, or e4m3 codes with a scale per token.
template <int FMT, int DP>
struct Keys {
    static constexpr int kLoads = FMT == WSL_KV_BF16 ? DP / 32 : DP / 64;   // 16 bytes each
    u32x4 x[2][kLoads];
    uint32_t e[2];
};
template <int FMT, int DP>
struct Values {
    static constexpr int kVec = DP >= 128 ? 8 : DP / 16;                    // elements of a load
    static constexpr int kLoads = DP / (16 * kVec);
    static constexpr int kWords = FMT == WSL_KV_BF16 ? kVec / 2 : kVec / 4;
    uint32_t x[8][kLoads][kWords];
    uint32_t e[8];
};

// Where a wave's 32 tokens lie.  UNI: a page holds whole groups of 16 tokens, so the two
// groups' addresses are the same for all lanes; otherwise each lane keeps its own tokens'.
template <bool UNI>
struct Place;
template <>
struct Place<true> {
    int64_t off[2];      // byte offset of the group's first token
    int64_t cell[2];     // its index among the scale bytes
    bool ok[2];
};
template <>
struct Place<false> {
    int64_t koff[2], voff[8];
    int64_t kcell[2], vcell[8];
    uint32_t kok, vok;   // bit i: token i of the lane is there
};

// Token t of the sequence: its byte offset and scale index; false (and a safe offset) where the
// sequence ends before it or its page is none of the cache's.
__device__ __forceinline__ bool find_token(const AttnArgs &a, const int32_t *table, int32_t h, int32_t len, int32_t t,
                                           int64_t &off, int64_t &cell, bool &bad) {
    int32_t page = 0, at = 0;
    bool ok = t < len;
    if (ok) {
        const int32_t i = static_cast<uint32_t>(t) / static_cast<uint32_t>(a.page_size);
        at = t - i * a.page_size;
        page = table[i];
        if (static_cast<uint32_t>(page) >= static_cast<uint32_t>(a.n_pages)) {
            ok = false;
            bad = true;
            page = at = 0;
        }
    }
    off = page * a.page_stride + h * a.head_stride + at * a.token_stride;
    cell = (static_cast<int64_t>(page) * a.n_kv + h) * a.page_size + at;
    return ok;
}

template <bool UNI>
__device__ __forceinline__ Place<UNI> find_tokens(const AttnArgs &a, const int32_t *table, int32_t h, int32_t len,
                                                  int32_t base, bool &bad) {
    Place<UNI> p;
    const int lane = static_cast<int>(threadIdx.x & 63);
    if constexpr (UNI) {
#pragma unroll
        for (int i = 0; i < 2; ++i) p.ok[i] = find_token(a, table, h, len, base + 16 * i, p.off[i], p.cell[i], bad);
    } else {
        p.kok = p.vok = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            p.kok |= find_token(a, table, h, len, base + 16 * i + (lane & 15), p.koff[i], p.kcell[i], bad) ? 1u << i : 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int32_t t = base + 16 * (i >> 2) + 4 * (lane >> 4) + (i & 3);
            p.vok |= find_token(a, table, h, len, t, p.voff[i], p.vcell[i], bad) ? 1u << i : 0;
        }
    }
    return p;
}

// Keys as the A operand of S^T = K Q^T: lane l holds key l % 16 and, of its head_dim, the
// 8 consecutive elements per matrix instruction that lane group l / 16 owns.
template <int FMT, int DP, bool UNI>
__device__ __forceinline__ void load_keys(const AttnArgs &a, const Place<UNI> &p, Keys<FMT, DP> &k) {
    const int lane = static_cast<int>(threadIdx.x & 63);
    constexpr int kElem = FMT == WSL_KV_BF16 ? 2 : 1, kPer = 16 / kElem;    // elements of a 16-byte load
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const char *row;
        if constexpr (UNI) row = a.k + p.off[i] + static_cast<uint32_t>((lane & 15) * static_cast<int32_t>(a.token_stride));
        else row = a.k + p.koff[i];
#pragma unroll
        for (int c = 0; c < Keys<FMT, DP>::kLoads; ++c) {
            const int d = c * 4 * kPer + (lane >> 4) * kPer;
            const bool in = d < a.head_dim;
            k.x[i][c] = *reinterpret_cast<const u32x4 *>(row + (in ? d : 0) * kElem);
            if (a.head_dim != DP && !in) k.x[i][c] = u32x4{0, 0, 0, 0};
        }
        if constexpr (FMT == WSL_KV_E4M3) {
            if constexpr (UNI) k.e[i] = a.ke[p.cell[i] + (lane & 15)];
            else k.e[i] = a.ke[p.kcell[i]];
        }
    }
}

// Values for the A operand of O^T = V^T P: lane l takes its group's 8 tokens (those whose scores
// S^T leaves in this lane) and, of each, the kVec elements that start at (l % 16) * kVec: whole
// rows are read in order, and the 8 x kVec block is transposed inside the lane.
template <int FMT, int DP, bool UNI>
__device__ __forceinline__ void load_values(const AttnArgs &a, const Place<UNI> &p, Values<FMT, DP> &v) {
    typedef Values<FMT, DP> V;
    const int lane = static_cast<int>(threadIdx.x & 63);
    constexpr int kElem = FMT == WSL_KV_BF16 ? 2 : 1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const char *row;
        if constexpr (UNI)
            row = a.v + p.off[i >> 2] +
                  static_cast<uint32_t>((4 * (lane >> 4) + (i & 3)) * static_cast<int32_t>(a.token_stride));
        else row = a.v + p.voff[i];
#pragma unroll
        for (int n = 0; n < V::kLoads; ++n) {
            int d = n * 16 * V::kVec + (lane & 15) * V::kVec;
            d = d < a.head_dim ? d : 0;              // columns past head_dim: computed, never written
            const uint32_t *src = reinterpret_cast<const uint32_t *>(row + d * kElem);
            if constexpr (V::kWords == 4) {
                const u32x4 w = *reinterpret_cast<const u32x4 *>(src);
                v.x[i][n][0] = w.x, v.x[i][n][1] = w.y, v.x[i][n][2] = w.z, v.x[i][n][3] = w.w;
            } else if constexpr (V::kWords == 2) {
                const u32x2 w = *reinterpret_cast<const u32x2 *>(src);
                v.x[i][n][0] = w.x, v.x[i][n][1] = w.y;
            } else {
                v.x[i][n][0] = src[0];
            }
        }
        if constexpr (FMT == WSL_KV_E4M3) {
            if constexpr (UNI) v.e[i] = a.ve[p.cell[i >> 2] + 4 * (lane >> 4) + (i & 3)];
            else v.e[i] = a.ve[p.vcell[i]];
        }
    }
}

// Token pair (2t, 2t + 1) of element word w (two bf16 elements) of load n.
template <int FMT, int DP>
__device__ __forceinline__ uint32_t value_word(const Values<FMT, DP> &v, int t, int n, int w) {
    if constexpr (FMT == WSL_KV_BF16) return v.x[t][n][w];
    else return fp8_pair(v.x[t][n][w >> 1], scale_of(v.e[t]), (w & 1) != 0);
}

// A pair of bf16 numbers with its NaNs and infinities replaced by zero.
__device__ __forceinline__ uint32_t finite_pair(uint32_t x) {
    x = (x & 0x7f80u) == 0x7f80u ? x & 0xffff0000u : x;
    return (x & 0x7f800000u) == 0x7f800000u ? x & 0xffffu : x;
}

// O^T += V^T (hi + lo) for MT blocks of 16 rows.
// CAREFUL: only over the values whose bit of `keep` is set and only into the rows that `rows` picks
// (bit m: the lane's row of block m), with lo (which may be zero or negative) times the finite
// values alone, so that an infinity gives the infinity that the weight itself would.
template <int FMT, int DP, int MT, bool CAREFUL>
__device__ __forceinline__ void add_values(const Values<FMT, DP> &v, const u32x4 (&hi)[MT], const u32x4 (&lo)[MT],
                                           f32x4 (&acc)[MT][DP / 16], uint32_t keep, uint32_t rows) {
    typedef Values<FMT, DP> V;
#pragma unroll
    for (int n = 0; n < V::kLoads; ++n)
#pragma unroll
        for (int w = 0; w < V::kVec / 2; ++w) {
            uint32_t x[8];
#pragma unroll
            for (int t = 0; t < 8; ++t) {
                x[t] = value_word<FMT, DP>(v, t, n, w);
                if constexpr (CAREFUL) x[t] = (keep >> t) & 1 ? x[t] : 0;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int j = n * V::kVec + 2 * w + e;
                u32x4 both, fine;
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    both[t] = __builtin_amdgcn_perm(x[2 * t + 1], x[2 * t], e ? 0x07060302u : 0x05040100u);
                    fine[t] = CAREFUL ? finite_pair(both[t]) : both[t];
                }
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const f32x4 sum = mfma(fine, lo[m], mfma(both, hi[m], acc[m][j]));
                    if constexpr (CAREFUL) {
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[m][j][r] = (rows >> m) & 1 ? sum[r] : acc[m][j][r];
                    } else {
                        acc[m][j] = sum;
                    }
                }
            }
        }
}

template <int FMT, int DP>
__device__ __forceinline__ void keep_values(Values<FMT, DP> &v, uint32_t keep) {
    typedef Values<FMT, DP> V;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
        const bool on = (keep >> t) & 1;
#pragma unroll
        for (int n = 0; n < V::kLoads; ++n)
#pragma unroll
            for (int w = 0; w < V::kWords; ++w) v.x[t][n][w] = on ? v.x[t][n][w] : 0;
        if constexpr (FMT == WSL_KV_E4M3) v.e[t] = on ? v.e[t] : 127;    // 0 * an unused scale may be NaN
    }
}

// Query rows as the B operand: lane l holds row l % 16 and the elements that match load_keys.
// QT == 1: bf16 queries; QT == 3: fp32 queries as a sum of three bf16 numbers (24 bits).
template <int FMT, int DP, int MT, int QT>
__device__ __forceinline__ void load_queries(const AttnArgs &a, int32_t seq, int32_t h, int32_t row0,
                                             u32x4 (&q)[MT][QT][DP / 32]) {
    const int lane = static_cast<int>(threadIdx.x & 63), g = lane >> 4;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
        const int32_t row = row0 + 16 * m + (lane & 15);
        const bool in_row = row < a.rows;
        const int32_t i = in_row ? row / a.group : 0, head = h * a.group + (in_row ? row - i * a.group : 0);
        const int64_t at = (static_cast<int64_t>(seq) * a.q_len + i) * a.ld_q + static_cast<int64_t>(head) * a.head_dim;
#pragma unroll
        for (int c = 0; c < DP / 32; ++c) {
            const int d = FMT == WSL_KV_BF16 ? c * 32 + g * 8 : (c >> 1) * 64 + g * 16 + (c & 1) * 8;
            const bool in = in_row && d < a.head_dim;
            if constexpr (QT == 1) {
                u32x4 x = {0, 0, 0, 0};
                if (in) x = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.q) + at + d);
                q[m][0][c] = x;
            } else {
                f32x4 x[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
                if (in) {
                    const f32x4 *src = reinterpret_cast<const f32x4 *>(static_cast<const float *>(a.q) + at + d);
                    x[0] = src[0], x[1] = src[1];
                }
#pragma unroll
                for (int t = 0; t < QT; ++t)
#pragma unroll
                    for (int w = 0; w < 4; ++w) {
                        const int half = w >> 1, e = 2 * (w & 1);
                        const uint32_t b = pack_bf16x2(x[half][e], x[half][e + 1]);
                        q[m][t][c][w] = b;
                        x[half][e] -= bf16_lo(b);
                        x[half][e + 1] -= bf16_hi(b);
                    }
            }
        }
    }
}

// One pass over a range of token tiles with the running maximum and sum of a softmax:
//     S = scale * Q K^T;  m' = max(m, max S);  P = exp(S - m');
//     l = l * exp(m - m') + sum P;  O = O * exp(m - m') + P V.
// Everything stays in registers.  S^T = K Q^T leaves the scores of query row l % 16 for the keys
// 4 (l / 16) .. + 3 of each group of 16 in lane l, which is the B operand of O^T = V^T P^T when
// the matrix instruction's 8 reduction slots of a lane group are taken to be those 8 keys: the
// order of the reduction is free as long as V's lanes use the same.  The rows' maxima and sums
// then sit in the lanes that hold the rows' outputs.
// P enters the matrix instruction as the sum of two bf16 numbers (16 bits): one alone would add an
// error as large as a bf16 result's own rounding.
template <int FMT, int DP, int MT, int QT, bool UNI>
__global__ __launch_bounds__(kAttnThreads, MT *DP *(QT == 1 ? 1 : 2) <= 128 ? 2 : 1) void attn_kernel(AttnArgs a) {
    constexpr int kPad = DP + 4;
    __shared__ float lds_o[kAttnWaves][16][kPad];
    __shared__ float lds_m[kAttnWaves][16], lds_l[kAttnWaves][16];
    __shared__ int64_t lds_plan[4];
    __shared__ int64_t lds_at[2];

    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int items = a.n_kv * a.row_tiles;

    // this workgroup's range of the tiles of all (sequence, head, row tile)
    const AttnPlan plan = attn_plan(a, lds_plan);
    const int64_t total = plan.total * items;
    const int64_t workers = attn_workers(a, total);
    if (blockIdx.x >= workers) return;
    const int64_t begin = attn_start(total, blockIdx.x, workers), end = attn_start(total, blockIdx.x + 1, workers);
    {
        const int64_t y = begin / items;
        if (plan.before <= y && y < plan.before + plan.mine) {
            int64_t before = plan.before;
            int32_t b = tid * plan.each;
            for (;; ++b) {
                const int32_t n = attn_span(a, b).tiles;
                if (y < before + n) break;
                before += n;
            }
            lds_at[0] = b, lds_at[1] = before;
        }
        __syncthreads();
    }
    int32_t seq = __builtin_amdgcn_readfirstlane(static_cast<int32_t>(lds_at[0]));
    AttnSpan span = attn_span(a, seq);
    const int64_t rest = begin - lds_at[1] * items;
    int32_t item = __builtin_amdgcn_readfirstlane(static_cast<int32_t>(rest / span.tiles));
    int32_t tile = __builtin_amdgcn_readfirstlane(static_cast<int32_t>(rest - static_cast<int64_t>(item) * span.tiles));
    bool bad = false;

    for (int64_t x = begin; x < end;) {
        const int32_t left = span.tiles - tile;
        const int32_t n = end - x < left ? static_cast<int32_t>(end - x) : left;
        const int32_t h = item / a.row_tiles, row0 = (item - h * a.row_tiles) * a.tile_rows;
        const int32_t len = __builtin_amdgcn_readfirstlane(span.len);
        const int32_t *table = a.table + seq * a.ld_table;
        bad |= span.bad;

        u32x4 q[MT][QT][DP / 32];
        load_queries<FMT, DP, MT, QT>(a, seq, h, row0, q);
        f32x4 acc[MT][DP / 16];
        float m[MT], l[MT];
        int32_t hi_t[MT];         // last position that the lane's row sees
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int32_t row = row0 + 16 * i + (lane & 15);
            hi_t[i] = row < a.rows ? len - a.q_len + row / a.group : -1;
        }
        // positions that every row sees: [all_lo, all_hi]; that some row sees: from any_lo on
        const int32_t all_hi = len - a.q_len;
        const int64_t all_lo = a.window > 0 ? static_cast<int64_t>(len) - a.window : 0;
        const int64_t any_lo = a.window > 0 ? static_cast<int64_t>(len) - a.q_len - a.window + 1 : 0;

        const int32_t t0 = (span.first + tile) * kAttnTile + wave * kAttnSub;
        const int32_t t1 = (span.first + tile + n) * kAttnTile < len ? (span.first + tile + n) * kAttnTile : len;
        // A NaN or an infinity among the values can reach rows that do not see it (0 * inf) and turn
        // hi * inf + lo * inf into NaN.  Both end in a NaN sum; a wave that finds one goes over its
        // tokens once more, carefully.
        for (bool careful = false;;) {
#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int j = 0; j < DP / 16; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
            m[i] = -__builtin_huge_valf();
            l[i] = 0.f;
        }
        Keys<FMT, DP> k;
        Values<FMT, DP> v;
        Place<UNI> place;
        if (t0 < t1) {
            place = find_tokens<UNI>(a, table, h, len, t0, bad);
            load_keys<FMT, DP, UNI>(a, place, k);
        }
        for (int32_t t = t0; t < t1; t += kAttnTile) {
            load_values<FMT, DP, UNI>(a, place, v);
            // scores
            f32x4 s[2][MT];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int j = 0; j < MT; ++j) s[i][j] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < DP / 32; ++c) {
                    u32x4 kc;
                    if constexpr (FMT == WSL_KV_BF16) {
                        kc = k.x[i][c];
                    } else {
                        const float sc = scale_of(k.e[i]);
                        const uint32_t w0 = k.x[i][c >> 1][(c & 1) * 2], w1 = k.x[i][c >> 1][(c & 1) * 2 + 1];
                        kc = u32x4{fp8_pair(w0, sc, false), fp8_pair(w0, sc, true), fp8_pair(w1, sc, false),
                                   fp8_pair(w1, sc, true)};
                    }
#pragma unroll
                    for (int j = 0; j < MT; ++j)
#pragma unroll
                        for (int e = 0; e < QT; ++e) s[i][j] = mfma(kc, q[j][e][c], s[i][j]);
                }
            }
            // which of the lane's 8 tokens (values) are there at all
            uint32_t there;
            if constexpr (UNI) there = (place.ok[0] ? 0x0fu : 0u) | (place.ok[1] ? 0xf0u : 0u);
            else there = place.vok;
            // the next keys, in flight under the softmax and the product with V
            if (t + kAttnTile < t1) {
                place = find_tokens<UNI>(a, table, h, len, t + kAttnTile, bad);
                load_keys<FMT, DP, UNI>(a, place, k);
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < MT; ++j) s[i][j] *= a.scale_log2;
            const bool whole = t + kAttnSub - 1 <= all_hi && t >= all_lo && __all(there == 0xffu);
            bool mixed = false;
            if (!whole) {
                uint32_t keep = 0;
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int32_t at = t + 16 * i + 4 * g + r;
                        const bool ok = ((there >> (4 * i + r)) & 1) && at < len && at >= any_lo;
                        keep |= ok ? 1u << (4 * i + r) : 0u;
                        mixed |= ok && (at > all_hi || at < all_lo);
#pragma unroll
                        for (int j = 0; j < MT; ++j) {
                            const bool see = ok && at <= hi_t[j] && (a.window == 0 || at > hi_t[j] - a.window);
                            s[i][j][r] = see ? s[i][j][r] : -__builtin_huge_valf();
                        }
                    }
                keep_values<FMT, DP>(v, keep);     // what no row sees may hold anything
                mixed = __any(mixed);
            }
            u32x4 p_hi[MT], p_lo[MT];
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                float top = fmaxf(fmaxf(fmaxf(s[0][j][0], s[0][j][1]), fmaxf(s[0][j][2], s[0][j][3])),
                                  fmaxf(fmaxf(s[1][j][0], s[1][j][1]), fmaxf(s[1][j][2], s[1][j][3])));
                top = fmaxf(top, __shfl_xor(top, 16, 64));
                top = fmaxf(top, __shfl_xor(top, 32, 64));
                const float next = fmaxf(m[j], top);
                const float ref = next == -__builtin_huge_valf() ? 0.f : next;
                if (__any(next != m[j])) {
                    const float f = __builtin_amdgcn_exp2f(m[j] - ref);
                    l[j] *= f;
#pragma unroll
                    for (int d = 0; d < DP / 16; ++d) acc[j][d] *= f;
                    m[j] = next;
                }
                float p[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) p[i] = __builtin_amdgcn_exp2f(s[i >> 2][j][i & 3] - ref);
                l[j] += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t b = pack_bf16x2(p[2 * i], p[2 * i + 1]);
                    p_hi[j][i] = b;
                    p_lo[j][i] = pack_bf16x2(p[2 * i] - bf16_lo(b), p[2 * i + 1] - bf16_hi(b));
                }
            }
            if (careful) {
                // values that some rows see and others do not: one query position at a time
                for (int32_t i = 0; i < (mixed ? a.q_len : 1); ++i) {
                    const int32_t last = all_hi + i;
                    uint32_t keep = 0, rows = 0;
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int32_t at = t + 16 * (e >> 2) + 4 * g + (e & 3);
                        keep |= !mixed || (at <= last && (a.window == 0 || at > last - a.window)) ? 1u << e : 0u;
                    }
#pragma unroll
                    for (int j = 0; j < MT; ++j) rows |= !mixed || hi_t[j] == last ? 1u << j : 0u;
                    add_values<FMT, DP, MT, true>(v, p_hi, p_lo, acc, keep, rows);
                }
            } else {
                add_values<FMT, DP, MT, false>(v, p_hi, p_lo, acc, 0, 0);
            }
        }
        if (careful) break;
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int d = 0; d < DP / 16; ++d)
#pragma unroll
                for (int r = 0; r < 4; ++r) careful |= acc[j][d][r] != acc[j][d][r];
        careful = __any(careful);
        if (!careful) break;
        }

        // join the waves; then the rows are done, or partial where the item goes on elsewhere
        const bool full = tile == 0 && n == span.tiles;
        const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (tile == 0 ? 1 : 0);
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            l[j] += __shfl_xor(l[j], 16, 64);
            l[j] += __shfl_xor(l[j], 32, 64);
            if (g == 0) lds_m[wave][lane] = m[j];
            __syncthreads();
            float top = lds_m[0][lane & 15];
#pragma unroll
            for (int w = 1; w < kAttnWaves; ++w) top = fmaxf(top, lds_m[w][lane & 15]);
            const float ref = top == -__builtin_huge_valf() ? 0.f : top;
            const float f = __builtin_amdgcn_exp2f(m[j] - ref);
            if (g == 0) lds_l[wave][lane] = l[j] * f;
            // acc[j][n * kVec + e][r] is element n * 16 * kVec + (4 g + r) * kVec + e of row l % 16
            constexpr int kVec = Values<FMT, DP>::kVec;
#pragma unroll
            for (int c = 0; c < Values<FMT, DP>::kLoads; ++c)
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int e = 0; e < kVec; e += 4) {
                        const int i = c * kVec + e;
                        *reinterpret_cast<f32x4 *>(&lds_o[wave][lane & 15][c * 16 * kVec + (4 * g + r) * kVec + e]) =
                            f32x4{acc[j][i][r] * f, acc[j][i + 1][r] * f, acc[j][i + 2][r] * f, acc[j][i + 3][r] * f};
                    }
            __syncthreads();
            for (int i = tid; i < 16 * (DP / 4); i += kAttnThreads) {
                const int r = i / (DP / 4), d = (i - r * (DP / 4)) * 4;
                const int32_t in_tile = 16 * j + r, row = row0 + in_tile;
                if (d < a.head_dim && in_tile < a.tile_rows && row < a.rows) {
                    f32x4 o = {0, 0, 0, 0};
                    float sum = 0.f, mx = lds_m[0][r];
#pragma unroll
                    for (int w = 0; w < kAttnWaves; ++w) {
                        o += *reinterpret_cast<const f32x4 *>(&lds_o[w][r][d]);
                        sum += lds_l[w][r];
                        mx = fmaxf(mx, lds_m[w][r]);
                    }
                    if (full) {
                        attn_finish(a, seq, len, h, row, d, make_float4(o.x, o.y, o.z, o.w), mx, sum);
                    } else {
                        *reinterpret_cast<f32x4 *>(a.part_o + (slot * a.tile_rows + in_tile) * a.head_dim + d) = o;
                        if (d == 0) a.part_ml[slot * a.tile_rows + in_tile] = make_float2(mx, sum);
                    }
                }
            }
            __syncthreads();
        }

        x += n;
        tile = 0;
        if (n == left && ++item == items) {
            item = 0;
            ++seq;
            if (x < end) span = attn_span(a, seq);
        }
    }
    if (__any(bad) && lane == 0 && a.status != nullptr) atomicOr(a.status, WSL_STATUS_INDEX);
}

template <int FMT, int DP, int MT, int QT>
void go(const AttnArgs &a, bool uni, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(a.workers)), block(kAttnThreads);
    if (uni) hipLaunchKernelGGL((attn_kernel<FMT, DP, MT, QT, true>), grid, block, 0, s, a);
    else hipLaunchKernelGGL((attn_kernel<FMT, DP, MT, QT, false>), grid, block, 0, s, a);
}

template <int FMT, int DP>
void go_rows(const AttnArgs &a, bool uni, int mt, hipStream_t s) {
    if (a.qfmt == WSL_OUT_BF16) {
        if (mt == 1) go<FMT, DP, 1, 1>(a, uni, s);
        else if (mt == 2 || DP == 256) go<FMT, DP, 2, 1>(a, uni, s);
        else if constexpr (DP < 256) go<FMT, DP, 4, 1>(a, uni, s);
    } else {
        if (mt == 1 || DP == 256) go<FMT, DP, 1, 3>(a, uni, s);
        else if constexpr (DP < 256) go<FMT, DP, 2, 3>(a, uni, s);
    }
}

}  // namespace

template <int FMT>
int launch_attn_fmt(const AttnArgs &a, int mt, hipStream_t s) {
    // groups of 16 tokens that never leave a page, and reach less than 2 GiB
    const bool uni = a.page_size % 16 == 0 && a.token_stride < (int64_t(1) << 26);
    if (a.head_dim <= 64) go_rows<FMT, 64>(a, uni, mt, s);
    else if (a.head_dim <= 128) go_rows<FMT, 128>(a, uni, mt, s);
    else go_rows<FMT, 256>(a, uni, mt, s);
    return WSL_OK;
}

}  // namespace wsl
