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

// The lane's number and the kernel's arguments, made out anew: what is derived from them for an item's
// end or a rare case is not computed before the loop over the tokens and held in registers throughout
// (that took 80 vector registers and spilled as many scalar ones).
__device__ __forceinline__ int fresh(int v) {
    asm volatile("" : "+v"(v));
    return v;
}
__device__ __forceinline__ const AttnArgs &fresh_args() {
    auto p = __builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *(const AttnArgs *)p;
}

// Two bf16 numbers of two e4m3 codes (exact).
__device__ __forceinline__ uint32_t fp8_pair(uint32_t w, bool hi) {
    return hi ? __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, true))
              : __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, false));
}

// 32 keys or values of one head as loaded: bf16 elements or e4m3 codes.
template <int FMT, int DP>
struct Keys {
    static constexpr int kLoads = FMT == WSL_KV_BF16 ? DP / 32 : DP / 64;   // 16 bytes each
    u32x4 x[2][kLoads];
};
template <int FMT, int DP>
struct Values {
    static constexpr int kVec = DP % 128 == 0 ? 8 : 4;                      // elements of a load
    static constexpr int kLoads = DP / (16 * kVec);
    static constexpr int kWords = FMT == WSL_KV_BF16 ? kVec / 2 : kVec / 4;
    uint32_t x[8][kLoads][kWords];
};

// One wave's part of LDS: where its 32 tokens lie, and their scales.
struct WaveLds {
    int64_t off[kAttnSub];
    float ks[kAttnSub], vs[kAttnSub];
};

// Orders one wave's LDS accesses across its lanes (they are carried out in order: no instruction).
__device__ __forceinline__ void wave_lds_fence() {
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
}

// Lane l's token (l % 32) of 32 successive ones: its place in its page, and its page as the table
// names it.  The table is read two rounds before the tokens are, so that nobody waits for it.  Tokens
// from `end` on stand for the last one before it (and for the first, if there is none): the load is
// made in any case, as all are (see attn_kernel).
struct Look {
    int32_t at, page;
};

__device__ __forceinline__ Look look_up(const AttnArgs &a, const int32_t *table, int32_t end, int32_t t) {
    t += static_cast<int32_t>(threadIdx.x & 31);
    t = t < end ? t : end - 1;
    t = t < 0 ? 0 : t;
    const uint32_t i = attn_over(static_cast<uint32_t>(t), a.over_page);
    Look p;
    p.at = t - static_cast<int32_t>(i * static_cast<uint32_t>(a.page_size));
    p.page = table[i];
    return p;
}

// The byte offsets of the 32 tokens from t on go into LDS (their scale bytes are fetched); returns
// which of the tokens are there at all: from `low` on and before `end`, on a page that the cache has
// (bad: one between the two is not).  A token that is not there gets a safe offset and the scale 1.
// `low`, the lowest position that some row sees, may lie inside the first tile: what is before it is
// nobody's, and its page may be gone.
template <int FMT>
__device__ __forceinline__ uint32_t find_tokens(const AttnArgs &a, WaveLds &w, const Look &p, int32_t h, int32_t low,
                                                int32_t end, int32_t t, uint32_t &kb, uint32_t &vb, bool &bad) {
    const int32_t lane = static_cast<int32_t>(threadIdx.x & 31);
    const bool in = t + lane >= low && t + lane < end, ok = in && static_cast<uint32_t>(p.page) < static_cast<uint32_t>(a.n_pages);
    bad |= in && !ok;
    const int64_t page = ok ? p.page : 0, at = ok ? p.at : 0;
    wave_lds_fence();
    w.off[lane] = page * a.page_stride + h * a.head_stride + at * a.token_stride;
    if constexpr (FMT == WSL_KV_E4M3) {
        const int64_t cell = (page * a.n_kv + h) * a.page_size + at;
        kb = a.ke[cell], vb = a.ve[cell];
    }
    wave_lds_fence();
    return static_cast<uint32_t>(__ballot(ok));
}

// Keys as the A operand of S^T = K Q^T: lane l holds key l % 16 and, of its head_dim, the
// 8 consecutive elements per matrix instruction that lane group l / 16 owns.
// FULL: head_dim is DP; else the places past it are read from the row's beginning and dropped.
template <int FMT, int DP, bool FULL>
__device__ __forceinline__ void load_keys(const AttnArgs &a, const WaveLds &w, Keys<FMT, DP> &k) {
    const int lane = static_cast<int>(threadIdx.x & 63);
    constexpr int kElem = FMT == WSL_KV_BF16 ? 2 : 1, kPer = 16 / kElem;    // elements of a 16-byte load
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const char *row = a.k + w.off[16 * i + (lane & 15)];
#pragma unroll
        for (int c = 0; c < Keys<FMT, DP>::kLoads; ++c) {
            const int d = c * 4 * kPer + (lane >> 4) * kPer;
            k.x[i][c] = *reinterpret_cast<const u32x4 *>(row + (FULL || d < a.head_dim ? d : 0) * kElem);
        }
    }
}

// Values for the A operand of O^T = V^T P: lane l takes its group's 8 tokens (those whose scores
// S^T leaves in this lane) and, of each, the kVec elements that start at (l % 16) * kVec: whole
// rows are read in order, and the 8 x kVec block is transposed inside the lane.  They are streamed: a
// line of values is read by one instruction once, where one of keys is read by two.  (Keys and values
// streamed alike, or neither: 30.4, 29.2 against 27.6 us for 16 sequences of up to 4224 tokens with five
// queries, 43.6, 48.9 against 42.2 for 32 of up to 8192 in e4m3, 160, 185 against 164 for 8 of 32768.)
template <int FMT, int DP, bool FULL>
__device__ __forceinline__ void load_values(const AttnArgs &a, const WaveLds &w, Values<FMT, DP> &v) {
    typedef Values<FMT, DP> V;
    const int lane = static_cast<int>(threadIdx.x & 63);
    constexpr int kElem = FMT == WSL_KV_BF16 ? 2 : 1;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const char *row = a.v + w.off[16 * (i >> 2) + 4 * (lane >> 4) + (i & 3)];
#pragma unroll
        for (int n = 0; n < V::kLoads; ++n) {
            int d = n * 16 * V::kVec + (lane & 15) * V::kVec;
            d = FULL || d < a.head_dim ? d : 0;      // columns past head_dim: computed, never written
            const uint32_t *src = reinterpret_cast<const uint32_t *>(row + d * kElem);
            if constexpr (V::kWords == 4) {
                const u32x4 x = __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(src));
                v.x[i][n][0] = x.x, v.x[i][n][1] = x.y, v.x[i][n][2] = x.z, v.x[i][n][3] = x.w;
            } else if constexpr (V::kWords == 2) {
                const u32x2 x = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(src));
                v.x[i][n][0] = x.x, v.x[i][n][1] = x.y;
            } else {
                v.x[i][n][0] = __builtin_nontemporal_load(src);
            }
        }
    }
}

// Element word w (two bf16 elements) of load n of token t.  Codes are converted as they are: their
// powers of two go into the scores and the weights, which is exact.
template <int FMT, int DP>
__device__ __forceinline__ uint32_t value_word(const Values<FMT, DP> &v, int t, int n, int w) {
    if constexpr (FMT == WSL_KV_BF16) return v.x[t][n][w];
    else return fp8_pair(v.x[t][n][w >> 1], (w & 1) != 0);
}

// O^T += V^T P for MT blocks of 16 rows, P as a sum of PT bf16 numbers.
template <int FMT, int DP, int MT, int PT>
__device__ __forceinline__ void add_values(const Values<FMT, DP> &v, const u32x4 (&p)[MT][PT],
                                           f32x4 (&acc)[MT][DP / 16]) {
    typedef Values<FMT, DP> V;
#pragma unroll
    for (int n = 0; n < V::kLoads; ++n)
#pragma unroll
        for (int w = 0; w < V::kVec / 2; ++w) {
            uint32_t x[8];
#pragma unroll
            for (int t = 0; t < 8; ++t) x[t] = value_word<FMT, DP>(v, t, n, w);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int j = n * V::kVec + 2 * w + e;
                u32x4 col;
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    col[t] = __builtin_amdgcn_perm(x[2 * t + 1], x[2 * t], e ? 0x07060302u : 0x05040100u);
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int i = 0; i < PT; ++i) acc[m][j] = mfma(col, p[m][i], acc[m][j]);
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
    }
}

// Query rows as the B operand: lane l holds row l % 16 and the elements that match load_keys.
// QT == 1: bf16 queries; QT == 3: fp32 queries as a sum of three bf16 numbers (24 bits).  All loads are
// made, a row past the last one being the first again: a load in a branch could not be counted.
template <int DP, int QT>
struct Queries {
    u32x4 x[DP / 32][QT == 1 ? 1 : 2];      // as loaded
};
template <int FMT, int DP, int QT, bool FULL>
__device__ __forceinline__ void load_queries(const AttnArgs &a, int32_t seq, int32_t h, int32_t row, Queries<DP, QT> &q) {
    const int g = static_cast<int>(threadIdx.x & 63) >> 4;
    row = row < a.rows ? row : 0;
    const int32_t i = static_cast<int32_t>(attn_over(static_cast<uint32_t>(row), a.over_group)), head = h * a.group + row - i * a.group;
    const int64_t at = (static_cast<int64_t>(seq) * a.q_len + i) * a.ld_q + static_cast<int64_t>(head) * a.head_dim;
#pragma unroll
    for (int c = 0; c < DP / 32; ++c) {
        const int d = FMT == WSL_KV_BF16 ? c * 32 + g * 8 : (c >> 1) * 64 + g * 16 + (c & 1) * 8;
        const int64_t from = at + (FULL || d < a.head_dim ? d : 0);
        if constexpr (QT == 1) {
            q.x[c][0] = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(a.q) + from);
        } else {
            const u32x4 *src = reinterpret_cast<const u32x4 *>(static_cast<const float *>(a.q) + from);
            q.x[c][0] = src[0], q.x[c][1] = src[1];
        }
    }
}
template <int FMT, int DP, int QT, bool FULL>
__device__ __forceinline__ void split_queries(const AttnArgs &a, const Queries<DP, QT> &q, u32x4 (&out)[QT][DP / 32]) {
    const int g = static_cast<int>(threadIdx.x & 63) >> 4;
#pragma unroll
    for (int c = 0; c < DP / 32; ++c) {
        const int d = FMT == WSL_KV_BF16 ? c * 32 + g * 8 : (c >> 1) * 64 + g * 16 + (c & 1) * 8;
        const bool in = FULL || d < a.head_dim;
        if constexpr (QT == 1) {
#pragma unroll
            for (int w = 0; w < 4; ++w) out[0][c][w] = in ? q.x[c][0][w] : 0;
        } else {
            f32x4 x[2] = {__builtin_bit_cast(f32x4, q.x[c][0]), __builtin_bit_cast(f32x4, q.x[c][1])};
#pragma unroll
            for (int w = 0; w < 4; ++w) x[0][w] = in ? x[0][w] : 0.f, x[1][w] = in ? x[1][w] : 0.f;
#pragma unroll
            for (int t = 0; t < QT; ++t)
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const int half = w >> 1, e = 2 * (w & 1);
                    const uint32_t b = pack_bf16x2(x[half][e], x[half][e + 1]);
                    out[t][c][w] = b;
                    x[half][e] -= bf16_lo(b);
                    x[half][e + 1] -= bf16_hi(b);
                }
        }
    }
}

// Element d of a row of keys or values, exactly.
template <int FMT>
__device__ __forceinline__ float element(const char *row, int32_t d, float scale) {
    if constexpr (FMT == WSL_KV_BF16) return bf16_lo(reinterpret_cast<const uint16_t *>(row)[d]);
    else return bf16_lo(fp8_pair(reinterpret_cast<const uint8_t *>(row)[d], false)) * scale;
}

// A wave's part of one row block (the lane's row), token by token in fp32: a row's sums take nothing
// from a token that it does not see.  Only for tokens among which a NaN or an infinity was found.
template <int FMT, int DP>
__device__ __forceinline__ void again(const int32_t *table, int32_t seq, int32_t h, int32_t row,
                                      int32_t len, int32_t t0, int32_t t1, int32_t hi, f32x4 (&acc)[DP / 16], float &m,
                                      float &l) {
    constexpr int kVec = Values<FMT, DP>::kVec;
    const AttnArgs &a = fresh_args();
    const int g = fresh(static_cast<int>(threadIdx.x & 63)) >> 4;
    const int32_t pos = row < a.rows ? static_cast<int32_t>(attn_over(static_cast<uint32_t>(row), a.over_group)) : 0, head = h * a.group + (row < a.rows ? row - pos * a.group : 0);
    const int64_t at_q = (static_cast<int64_t>(seq) * a.q_len + pos) * a.ld_q + static_cast<int64_t>(head) * a.head_dim;
    m = -__builtin_huge_valf();
    l = 0.f;
#pragma unroll
    for (int j = 0; j < DP / 16; ++j) acc[j] = f32x4{0, 0, 0, 0};
    for (int32_t sub = t0; sub < t1; sub += kAttnTile)
        for (int32_t t = sub; t < sub + kAttnSub && t < len; ++t) {
            const uint32_t i = attn_over(static_cast<uint32_t>(t), a.over_page);
            const int64_t page = table[i], at = t - static_cast<int32_t>(i * static_cast<uint32_t>(a.page_size));
            const bool see = t <= hi && (a.window == 0 || t > hi - a.window);
            if (page < 0 || page >= a.n_pages || !__any(see)) continue;
            const int64_t off = page * a.page_stride + h * a.head_stride + at * a.token_stride;
            float ks = 1.f, vs = 1.f;
            if constexpr (FMT == WSL_KV_E4M3) {
                const int64_t cell = (page * a.n_kv + h) * a.page_size + at;
                ks = __builtin_bit_cast(float, static_cast<uint32_t>(a.ke[cell]) << 23);
                vs = __builtin_bit_cast(float, static_cast<uint32_t>(a.ve[cell]) << 23);
            }
            float s = 0.f;
            for (int32_t d = g; d < a.head_dim; d += 4) {
                const float q = a.qfmt == WSL_OUT_F32 ? static_cast<const float *>(a.q)[at_q + d]
                                                      : bf16_lo(static_cast<const uint16_t *>(a.q)[at_q + d]);
                s = __builtin_fmaf(q, element<FMT>(a.k + off, d, ks), s);
            }
            s += __shfl_xor(s, 16, 64);
            s += __shfl_xor(s, 32, 64);
            s = see ? s * a.scale_log2 : -__builtin_huge_valf();
            const float best = fmaxf(m, s), ref = best == -__builtin_huge_valf() ? 0.f : best;
            const float f = __builtin_amdgcn_exp2f(m - ref), p = __builtin_amdgcn_exp2f(s - ref);
            m = best;
            l = l * f + p;
#pragma unroll
            for (int c = 0; c < DP / (16 * kVec); ++c)
#pragma unroll
                for (int e = 0; e < kVec; ++e)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int32_t d = c * 16 * kVec + (4 * g + r) * kVec + e;
                        const float x = d < a.head_dim ? element<FMT>(a.v + off, d, vs) : 0.f;
                        const float o = acc[c * kVec + e][r] * f;
                        acc[c * kVec + e][r] = see ? __builtin_fmaf(p, x, o) : o;
                    }
        }
    l = g == 0 ? l : 0.f;       // the lanes of a row add theirs up
}

// Waves of a SIMD that the registers are shared among (a workgroup is one wave on each): as many as do
// without scratch memory.  What is in flight has to cover the memory's latency, and a wave has a round's
// keys and values under way; more waves with spilled registers lost (8 sequences of 8192 tokens in e4m3,
// heads of 256, fp32 queries: 92 us with two, 52 with one; 16 of up to 4224 with 25 rows of 64 20.4 with
// three, 20.2 with two), and more without did not help (three instead of two in e4m3 at 128: 32 ragged
// sequences 44.9 against 42.2).
template <int FMT, int DP, int MT, int QT>
constexpr int attn_waves() {
    if (DP > 128) return FMT == WSL_KV_BF16 || (DP > 192 && QT == 3) ? 1 : 2;
    return QT == 3 && MT == 2 ? 1 : DP == 64 && MT == 1 ? 3 : 2;
}

// One pass over a range of token tiles with the running maximum and sum of a softmax:
//     S = scale * Q K^T;  m' = max(m, max S);  P = exp(S - m');
//     l = l * exp(m - m') + sum P;  O = O * exp(m - m') + P V.
// Everything stays in registers.  S^T = K Q^T leaves the scores of query row l % 16 for the keys
// 4 (l / 16) .. + 3 of each group of 16 in lane l, which is the B operand of O^T = V^T P^T when
// the matrix instruction's 8 reduction slots of a lane group are taken to be those 8 keys: the
// order of the reduction is free as long as V's lanes use the same.  The rows' maxima and sums
// then sit in the lanes that hold the rows' outputs.
// P enters the matrix instruction as the sum of PT bf16 numbers: of three (24 bits), or of two (16 bits)
// where queries and result are both bf16, whose own rounding is 2^8 times as large (one number alone would
// add an error of its size).  (Three there too: 16 sequences of up to 4224 tokens with five queries 28.1 us
// against 27.6, 32 of up to 8192 in e4m3 42.1 against 41.9, and as many results, one or two in 1000, fall
// to the other side of a rounding as with two: sums in another order do that.)
// Each wave works on 32 tokens of its own in a round, and the four join at an item's end.  In a
// round it asks for this round's values, then works on the keys that it asked for a round before,
// asks for the next round's keys and the table's entries for the round after that.
// No load stands in a branch: the waits count the loads since, and where there may be more or fewer of
// them the compiler waits for all.  So a wave without tokens, and the keys after a range's last round, are
// a row of the cache that nobody uses.
// Bound: the cached keys and values, read once.  8 sequences of 32768 tokens, 8 kv heads of 128, bf16
// (1.07 GB): 159 us, 6.7 TB/s, against 7.3 of a plain read.  Short calls are a chain of five trips to
// memory (lengths, table, keys, values, result): 6.3 us for one sequence of 37 tokens.
template <int FMT, int DP, int MT, int QT, int PT, bool FULL>
__global__ __launch_bounds__(kAttnThreads, (attn_waves<FMT, DP, MT, QT>())) void attn_kernel(AttnArgs a) {
    constexpr int kPad = DP + 4;
    __shared__ float lds_o[kAttnWaves][16 * MT][kPad];
    __shared__ float lds_m[kAttnWaves][16 * MT], lds_l[kAttnWaves][16 * MT];
    __shared__ WaveLds lds_w[kAttnWaves];

    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    WaveLds &mem = lds_w[wave];

    const AttnPlan plan = attn_plan(a, blockIdx.x);
    int32_t begin = 0, end = 1;
    if (!a.whole) {
        begin = static_cast<int32_t>(blockIdx.x) * plan.each;
        end = plan.total - begin < plan.each ? plan.total : begin + plan.each;
    }
    AttnOpen open = {0, 0, 0, 1};
    bool bad = false;
    int32_t seq = plan.seq, head = 0, unit = 0;
    AttnSpan span = {};
    if (begin < end) {
        span = attn_span(a, attn_len(a, plan, seq));
        const int32_t units = span.tiles + plan.cost;
        const int32_t rest = a.whole ? static_cast<int32_t>(blockIdx.x - static_cast<uint32_t>(seq * a.n_kv)) * units
                                     : begin - plan.before * a.n_kv;
        head = static_cast<int32_t>(static_cast<uint32_t>(rest) / static_cast<uint32_t>(units));
        head = head < a.n_kv ? head : a.n_kv - 1;      // (as in attn_plan)
        unit = rest - head * units;
        unit = unit < units ? unit : units - 1;
        if (a.whole) end = units;
    }

    for (int32_t x = begin; x < end;) {
        const int32_t left = span.tiles + plan.cost - unit;
        const int32_t used = end - x < left ? end - x : left;
        const int32_t tile = unit > plan.cost ? unit - plan.cost : 0;
        const int32_t n = unit + used - plan.cost - tile;      // tiles; none where the units all stand for its beginning
        if (n > 0) {
        const int32_t row0 = static_cast<int32_t>(blockIdx.y) * a.tile_rows;
        const int32_t len = span.len;
        const int32_t *table = a.table + seq * a.ld_table;
        bad |= span.bad;

        const int32_t t0 = (span.first + tile) * kAttnTile + wave * kAttnSub;
        const int32_t t1 = (span.first + tile + n) * kAttnTile < len ? (span.first + tile + n) * kAttnTile : len;
        const Look here = look_up(a, table, t1, t0);
        Queries<DP, QT> raw[MT];
#pragma unroll
        for (int i = 0; i < MT; ++i)
            load_queries<FMT, DP, QT, FULL>(a, seq, head, row0 + 16 * i + (lane & 15), raw[i]);
        f32x4 acc[MT][DP / 16];
        float m[MT], l[MT];
        int32_t hi_t[MT];         // last position that the lane's row sees
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            const int32_t row = row0 + 16 * i + (lane & 15);
            hi_t[i] = row < a.rows ? len - a.q_len + static_cast<int32_t>(attn_over(static_cast<uint32_t>(row), a.over_group)) : -1;
        }
        // positions that every row sees: [all_lo, all_hi]; that some row sees: from low on
        const int32_t all_hi = len - a.q_len;
        const int32_t all_lo = a.window > 0 ? len - a.window : 0;
        const int32_t low = attn_lowest(a, len);

#pragma unroll
        for (int i = 0; i < MT; ++i) {
#pragma unroll
            for (int j = 0; j < DP / 16; ++j) acc[i][j] = f32x4{0, 0, 0, 0};
#pragma unroll
            for (int j = 0; j < DP / 16; ++j) asm volatile("" : "+v"(acc[i][j]));   // now, not after the first loads
            m[i] = -__builtin_huge_valf();
            l[i] = 0.f;
        }
        __builtin_amdgcn_sched_barrier(0);
        Keys<FMT, DP> k;
        Values<FMT, DP> v;
        uint32_t kb = 127, vb = 127;
        u32x4 q[MT][QT][DP / 32];
        uint32_t there_next = find_tokens<FMT>(a, mem, here, head, low, t1, t0, kb, vb, bad);
        load_keys<FMT, DP, FULL>(a, mem, k);
        Look next = look_up(a, table, t1, t0 + kAttnTile);
#pragma unroll
        for (int i = 0; i < MT; ++i) {
            split_queries<FMT, DP, QT, FULL>(a, raw[i], q[i]);
            // they are here before the loop: in it, their wait would be one for a round's own loads
#pragma unroll
            for (int e = 0; e < QT; ++e)
#pragma unroll
                for (int c = 0; c < DP / 32; ++c) asm volatile("" : "+v"(q[i][e][c]));
        }
        for (int32_t t = t0; t < t1; t += kAttnTile) {
            const uint32_t there = there_next;
            load_values<FMT, DP, FULL>(a, mem, v);
            __builtin_amdgcn_sched_barrier(0);       // asked for before anything waits for the keys
            f32x4 ks[2], vs[2];
            if constexpr (FMT == WSL_KV_E4M3) {
                // (a byte of 255 is none that a write leaves; 254 keeps what it gives finite)
                const bool ok = (there >> (lane & 31)) & 1;
                mem.ks[lane & 31] = __builtin_bit_cast(float, (ok ? (kb < 254u ? kb : 254u) : 127u) << 23);
                mem.vs[lane & 31] = __builtin_bit_cast(float, (ok ? (vb < 254u ? vb : 254u) : 127u) << 23);
                wave_lds_fence();
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    ks[i] = *reinterpret_cast<const f32x4 *>(&mem.ks[16 * i + 4 * g]);
                    vs[i] = *reinterpret_cast<const f32x4 *>(&mem.vs[16 * i + 4 * g]);
                }
            }
            // scores
            f32x4 s[2][MT];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int j = 0; j < MT; ++j) s[i][j] = f32x4{0, 0, 0, 0};
#pragma unroll
                for (int c = 0; c < DP / 32; ++c) {
                    u32x4 kc;
                    int d;
                    if constexpr (FMT == WSL_KV_BF16) {
                        kc = k.x[i][c];
                        d = c * 32 + g * 8;
                    } else {
                        const uint32_t w0 = k.x[i][c >> 1][(c & 1) * 2], w1 = k.x[i][c >> 1][(c & 1) * 2 + 1];
                        kc = u32x4{fp8_pair(w0, false), fp8_pair(w0, true), fp8_pair(w1, false), fp8_pair(w1, true)};
                        d = (c >> 1) * 64 + g * 16;
                    }
                    if constexpr (!FULL) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) kc[e] = d < a.head_dim ? kc[e] : 0;
                    }
#pragma unroll
                    for (int j = 0; j < MT; ++j)
#pragma unroll
                        for (int e = 0; e < QT; ++e) s[i][j] = mfma(kc, q[j][e][c], s[i][j]);
                }
            }
            // the next keys, in flight under the softmax and the product with V
            there_next = find_tokens<FMT>(a, mem, next, head, low, t1, t + kAttnTile, kb, vb, bad);
            load_keys<FMT, DP, FULL>(a, mem, k);
            next = look_up(a, table, t1, t + 2 * kAttnTile);
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < MT; ++j) {
                    if constexpr (FMT == WSL_KV_E4M3) s[i][j] *= ks[i];
                    s[i][j] *= a.scale_log2;
                }
            const bool whole = t + kAttnSub - 1 <= all_hi && t >= all_lo && there == 0xffffffffu;
            if (!whole) {
                uint32_t keep = 0;
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int r = 0; r < 4; ++r) {
                        const int32_t at = t + 16 * i + 4 * g + r;
                        const bool ok = (there >> (16 * i + 4 * g + r)) & 1;
                        keep |= ok ? 1u << (4 * i + r) : 0u;
#pragma unroll
                        for (int j = 0; j < MT; ++j) {
                            const bool see = ok && at <= hi_t[j] && (a.window == 0 || at > hi_t[j] - a.window);
                            s[i][j][r] = see ? s[i][j][r] : -__builtin_huge_valf();
                        }
                    }
                keep_values<FMT, DP>(v, keep);     // what no row sees may hold anything
            }
            u32x4 p_t[MT][PT];
#pragma unroll
            for (int j = 0; j < MT; ++j) {
                float top = fmaxf(fmaxf(fmaxf(s[0][j][0], s[0][j][1]), fmaxf(s[0][j][2], s[0][j][3])),
                                  fmaxf(fmaxf(s[1][j][0], s[1][j][1]), fmaxf(s[1][j][2], s[1][j][3])));
                top = fmaxf(top, __shfl_xor(top, 16, 64));
                top = fmaxf(top, __shfl_xor(top, 32, 64));
                const float best = fmaxf(m[j], top);
                const float ref = best == -__builtin_huge_valf() ? 0.f : best;
                if (__any(best != m[j])) {
                    const float f = __builtin_amdgcn_exp2f(m[j] - ref);
                    l[j] *= f;
#pragma unroll
                    for (int d = 0; d < DP / 16; ++d) acc[j][d] *= f;
                    m[j] = best;
                }
                float p[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) p[i] = __builtin_amdgcn_exp2f(s[i >> 2][j][i & 3] - ref);
                l[j] += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
                if constexpr (FMT == WSL_KV_E4M3) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) p[i] *= vs[i >> 2][i & 3];
                }
#pragma unroll
                for (int e = 0; e < PT; ++e)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t b = pack_bf16x2(p[2 * i], p[2 * i + 1]);
                        p_t[j][e][i] = b;
                        p[2 * i] -= bf16_lo(b);
                        p[2 * i + 1] -= bf16_hi(b);
                    }
            }
            add_values<FMT, DP, MT, PT>(v, p_t, acc);
        }
        // A NaN or an infinity among the values can reach rows that do not see it (0 * inf) and turn
        // the sum of a weight's terms times it into NaN.  Both end in a NaN sum; a wave that finds
        // one goes over its tokens once more, one by one.
        bool odd = false;
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int d = 0; d < DP / 16; ++d)
#pragma unroll
                for (int r = 0; r < 4; ++r) odd |= acc[j][d][r] != acc[j][d][r];
        if (__any(odd)) {
#pragma unroll
            for (int i = 0; i < MT; ++i)
                again<FMT, DP>(table, seq, head, row0 + 16 * i + fresh(lane & 15), len, t0, t1, hi_t[i], acc[i], m[i], l[i]);
        }

        // join the waves; then the rows are done, or partial where the item goes on elsewhere
        const bool full = tile == 0 && n == span.tiles;
        {
        const AttnArgs a = fresh_args();
        const int tid = fresh(static_cast<int>(threadIdx.x)), lane = tid & 63, g = lane >> 4;
        const int64_t slot = (static_cast<int64_t>(blockIdx.y) * a.workers + blockIdx.x) * 2 + (tile == 0 ? 1 : 0);
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            l[j] += __shfl_xor(l[j], 16, 64);
            l[j] += __shfl_xor(l[j], 32, 64);
            if (g == 0) lds_m[wave][16 * j + lane] = m[j];
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < MT; ++j) {
            float top = lds_m[0][16 * j + (lane & 15)];
#pragma unroll
            for (int w = 1; w < kAttnWaves; ++w) top = fmaxf(top, lds_m[w][16 * j + (lane & 15)]);
            const float ref = top == -__builtin_huge_valf() ? 0.f : top;
            const float f = __builtin_amdgcn_exp2f(m[j] - ref);
            if (g == 0) lds_l[wave][16 * j + lane] = l[j] * f;
            // acc[j][n * kVec + e][r] is element n * 16 * kVec + (4 g + r) * kVec + e of row l % 16
            constexpr int kVec = Values<FMT, DP>::kVec;
#pragma unroll
            for (int c = 0; c < Values<FMT, DP>::kLoads; ++c)
#pragma unroll
                for (int r = 0; r < 4; ++r)
#pragma unroll
                    for (int e = 0; e < kVec; e += 4) {
                        const int i = c * kVec + e;
                        *reinterpret_cast<f32x4 *>(&lds_o[wave][16 * j + (lane & 15)][c * 16 * kVec + (4 * g + r) * kVec + e]) =
                            f32x4{acc[j][i][r] * f, acc[j][i + 1][r] * f, acc[j][i + 2][r] * f, acc[j][i + 3][r] * f};
                    }
        }
        __syncthreads();
        for (int i = tid; i < 16 * MT * (DP / 4); i += kAttnThreads) {
            const int r = i / (DP / 4), d = (i - r * (DP / 4)) * 4;
            const int32_t row = row0 + r;
            if (d < a.head_dim && r < a.tile_rows && row < a.rows) {
                f32x4 o = {0, 0, 0, 0};
                float sum = 0.f, mx = lds_m[0][r];
#pragma unroll
                for (int w = 0; w < kAttnWaves; ++w) {
                    o += *reinterpret_cast<const f32x4 *>(&lds_o[w][r][d]);
                    sum += lds_l[w][r];
                    mx = fmaxf(mx, lds_m[w][r]);
                }
                if (full) {
                    attn_finish(a, seq, head, row, d, o, mx, sum);
                } else {
                    *reinterpret_cast<f32x4 *>(a.part_o + (slot * a.tile_rows + r) * a.head_dim + d) = o;
                    if (d == 0) a.part_ml[slot * a.tile_rows + r] = make_float2(mx, sum);
                }
            }
        }
        if (tile == 0 && a.open != nullptr) {
            const uint32_t last = static_cast<uint32_t>(x + left - 1) / static_cast<uint32_t>(plan.each);
            open = {seq, head, static_cast<int32_t>(blockIdx.x), static_cast<int32_t>(last - blockIdx.x) + 1};
            if (a.by_item && blockIdx.y == 0 && tid == 0) a.open[seq * a.n_kv + head] = open;
        }
        }
        if (x + used < end) __syncthreads();      // LDS is free again
        }

        x += used;
        unit = 0;
        if (used == left && ++head == a.n_kv) {
            head = 0;
            if (++seq >= a.n_seq) break;
            if (x < end) span = attn_span(a, attn_len(a, plan, seq));
        }
    }
    if (a.open != nullptr && !a.by_item && blockIdx.y == 0 && tid == 0) a.open[blockIdx.x] = open;
    if (__any(bad) && lane == 0 && a.status != nullptr) atomicOr(a.status, WSL_STATUS_INDEX);
}

// There is a workgroup for each whole item and row tile; or else, over bf16, one for each compute unit:
// its four waves' rounds of 16 KB keep the memory busy, and fewer shares have fewer beginnings, ends and
// parts (two on each: 16 sequences of up to 4224 tokens with five queries 30.1 us against 27.6, 64 of up to
// 2048 48.1 against 44.5, 8 of 32768 164.7 against 163.9); over e4m3, whose rounds are half as long, as
// many as the registers allow.  There many short sequences and fp32 queries gain (two against one: 64 of up
// to 2048 28.7 against 30.1, the 16 with five queries 25.3 against 25.7, 32 of up to 8192 with fp32 queries
// 44.6 against 45.3) and few long ones lose (4 of 8192 20.4 against 18.7, 8 of up to 16384 26.5 against 24.9,
// 32 of up to 8192 42.2 against 41.8).
// Those of one token range lie `workers` apart, a multiple of 8 where it can be, so that they run at the
// same time on the same XCD and what one reads the others find in its L2.
template <int FMT, int DP, int MT, int QT, int PT>
void go(AttnArgs &a, hipStream_t s) {
    const int fit = kAttnCus * (FMT == WSL_KV_BF16 ? 1 : attn_waves<FMT, DP, MT, QT>());
    static_assert(attn_waves<FMT, DP, MT, QT>() <= kAttnMaxWaves, "workspaces are for so many");
    const int most = a.row_tiles * 8 >= fit ? 8 : fit / a.row_tiles / 8 * 8;
    if (a.whole) a.workers = a.n_seq * a.n_kv;
    else a.workers = a.workers < most ? a.workers : most;
    const dim3 grid(static_cast<unsigned>(a.workers), static_cast<unsigned>(a.row_tiles));
    if (a.head_dim == DP) hipLaunchKernelGGL((attn_kernel<FMT, DP, MT, QT, PT, true>), grid, dim3(kAttnThreads), 0, s, a);
    else hipLaunchKernelGGL((attn_kernel<FMT, DP, MT, QT, PT, false>), grid, dim3(kAttnThreads), 0, s, a);
}

template <int FMT, int DP>
void go_rows(AttnArgs &a, int mt, hipStream_t s) {
    if (a.qfmt != WSL_OUT_BF16) {
        if (mt == 1) go<FMT, DP, 1, 3, 3>(a, s);
        else if constexpr (attn_two_blocks(FMT, WSL_OUT_F32, DP)) go<FMT, DP, 2, 3, 3>(a, s);
        return;
    }
    const bool exact = a.ofmt != WSL_OUT_BF16;
    if (mt == 1) exact ? go<FMT, DP, 1, 1, 3>(a, s) : go<FMT, DP, 1, 1, 2>(a, s);
    else if constexpr (attn_two_blocks(FMT, WSL_OUT_BF16, DP))
        exact ? go<FMT, DP, 2, 1, 3>(a, s) : go<FMT, DP, 2, 1, 2>(a, s);
}

}  // namespace

template <int FMT>
int launch_attn_fmt(AttnArgs &a, int mt, hipStream_t s) {
    if (a.head_dim <= 64) go_rows<FMT, 64>(a, mt, s);
    else if (a.head_dim <= 128) go_rows<FMT, 128>(a, mt, s);
    else if (a.head_dim <= 192) go_rows<FMT, 192>(a, mt, s);
    else go_rows<FMT, 256>(a, mt, s);
    return WSL_OK;
}

}  // namespace wsl
