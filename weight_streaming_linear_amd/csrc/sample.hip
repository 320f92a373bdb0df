// Sampling from logits (sample_logits) for gfx950.
//
// A row's entries are ordered by value, equal ones by index: by the 64-bit number
//     order(j) = ordered bits of z_j, then ~j,
// no two of which are equal.  Whatever top-k, top-p and min-p keep is a beginning of that order, so a
// row needs one border and not a sort:
//     y = 8 log2(e) (z - max z) / T,  w = 2^(y / 8)  (the greatest weigh 1 exactly),
//     cell of an entry = min(-rint(y), 255): an eighth of a power of two each, in order;
// counts and weight sums of the cells say which cell the border of top-k (or top-p) lies in, and only that
// cell's entries are looked at further: up to kList of them are put in order, more are first
// narrowed by 256 ranges of order(j).  Weights come from 64-bit arithmetic; in a cell they are
// added up as whole numbers of 2^-40 of the cell's unit, which no order of adding changes.
// The token is then found as in verify_drafts: sums of segments in the order of the entries, and the
// segment that passes u * total looked through.
#include "row_scan.h"

namespace wsl {
namespace {

constexpr int kWaves = 16, kSegs = 2, kChunk = kWaves * kSegs * kSeg;      // entries in registers together
constexpr int kCells = 256, kList = 256;
constexpr int kMostSegs = (1 << 22) / kSeg;
constexpr double kUnit = 1099511627776.0;      // 2^40: whole numbers to the unit; 2^22 entries of it fit 64 bits

struct SampleArgs {
    const void *logits;
    const float *u;
    int32_t *tokens;
    float *probs;
    uint32_t *status;
    int64_t vocab, ld, ld_probs;
    wsl_sampling how;
};

// 2^(n / 8) for n of any size.
__device__ __forceinline__ double eighths(double n) {
    constexpr double kRoots[8] = {1.0, 1.0905077326652577, 1.189207115002721, 1.2968395546510096,
                                  1.4142135623730951, 1.5422108254079407, 1.681792830507429, 1.8340080864093424};
    n = n < -16000 ? -16000 : (n > 8000 ? 8000 : n);
    const int i = static_cast<int>(n);
    double r = kRoots[0];
#pragma unroll
    for (int e = 1; e < 8; ++e) r = (i & 7) == e ? kRoots[e] : r;
    return __builtin_ldexp(r, i >> 3);
}
// 2^(f / 8), |f| <= 1/2: the Taylor series of exp(f ln 2 / 8) to the 7th power, right to 2^-50 (and 1 for
// an f that is nearly 0: logits that a high temperature makes equal weigh the same).
__device__ __forceinline__ double part(double f) {
    const double x = f * 0.08664339756999316;
    double r = 1.0 / 5040;
    r = __builtin_fma(r, x, 1.0 / 720);
    r = __builtin_fma(r, x, 1.0 / 120);
    r = __builtin_fma(r, x, 1.0 / 24);
    r = __builtin_fma(r, x, 1.0 / 6);
    r = __builtin_fma(r, x, 0.5);
    r = __builtin_fma(r, x, 1.0);
    return __builtin_fma(r, x, 1.0);
}

__device__ __forceinline__ bool in_row(float z) { return z > -__builtin_huge_valf(); }

__device__ __forceinline__ uint64_t order_of(float z, uint32_t index) {
    const uint32_t b = __builtin_bit_cast(uint32_t, z + 0.f);      // -0 is 0
    const uint32_t key = b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
    return static_cast<uint64_t>(key) << 32 | ~index;
}
__device__ __forceinline__ float logit_of(uint64_t order) {
    const uint32_t key = static_cast<uint32_t>(order >> 32);
    return __builtin_bit_cast(float, key ^ (key >> 31 ? 0x80000000u : 0xffffffffu));
}

// A row's settings and its greatest entry.
struct Scale {
    double c8, m;          // y = c8 * (z - m)
    __device__ __forceinline__ double y(float z) const { return c8 * (static_cast<double>(z) - m); }
    __device__ __forceinline__ int cell(double y) const {
        const double d = -__builtin_rint(y);
        return static_cast<int>(d < kCells - 1 ? d : kCells - 1);
    }
    // weight, and as a whole number of a cell's units
    __device__ __forceinline__ double weight(float z) const {
        const double v = y(z), n = __builtin_rint(v);
        return part(v - n) * eighths(n);
    }
    __device__ __forceinline__ uint64_t whole(double y, int cell) const {
        const double n = __builtin_rint(y);
        double w = part(y - n);
        if (cell == kCells - 1) w *= eighths(n + (kCells - 1));
        return static_cast<uint64_t>(__builtin_fma(w, kUnit, 0.5));
    }
};

// Counts and sums of 256 cells (or ranges), and where a count or a sum is reached.
struct Bins {
    uint64_t sum[kCells];
    uint32_t count[kCells];
};
struct Border {
    int bin;
    uint32_t before, in;           // entries before the bin, and in it
    double w_before, w_all;        // weights before it, and of all bins
};
// The first bin up to which there are `count` entries (by_count), or a sum of `sum`; where rounding lets
// none, the last that holds any.  unit(i): what a sum of bin i counts.  Every wave comes to the same.
template <typename Unit>
__device__ __forceinline__ Border border_of(const Bins &b, bool by_count, uint32_t count, double sum, Unit unit) {
    const int lane = static_cast<int>(threadIdx.x & 63);
    constexpr int kMine = kCells / 64;
    uint32_t c[kMine], cs = 0;
    double w[kMine], ws = 0;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        c[i] = b.count[lane * kMine + i];
        w[i] = static_cast<double>(b.sum[lane * kMine + i]) * unit(lane * kMine + i);
        cs += c[i], ws += w[i];
    }
    const double up_w = lanes_before(ws), up_c = lanes_before(static_cast<double>(cs));
    double at_w = up_w - ws;
    uint32_t at_c = static_cast<uint32_t>(up_c) - cs;
    int hit = -1, last = -1;
    uint32_t hit_c = 0, hit_in = 0, last_c = 0, last_in = 0;
    double hit_w = 0, last_w = 0;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        if (c[i]) {
            last = i, last_c = at_c, last_in = c[i], last_w = at_w;
            if (hit < 0 && (by_count ? at_c + c[i] >= count : at_w + w[i] >= sum)) hit = i, hit_c = at_c, hit_in = c[i], hit_w = at_w;
        }
        at_c += c[i], at_w += w[i];
    }
    const uint64_t hits = __ballot(hit >= 0), some = __ballot(last >= 0);
    Border o = {0, 0, 0, 0, lane_value(up_w, 63)};
    if (!some) return o;
    const int l = hits ? __builtin_ctzll(hits) : 63 - __builtin_clzll(some);
    o.bin = l * kMine + __builtin_amdgcn_readlane(hits ? hit : last, l);
    o.before = __builtin_amdgcn_readlane(static_cast<int>(hits ? hit_c : last_c), l);
    o.in = __builtin_amdgcn_readlane(static_cast<int>(hits ? hit_in : last_in), l);
    o.w_before = lane_value(hits ? hit_w : last_w, l);
    return o;
}

struct Shared {
    Bins bins;
    uint64_t list[kList], sorted[kList];
    uint64_t least[kWaves], most[kWaves];
    float top[kWaves];
    uint32_t n, bad;
};

// Every entry of a row, by all waves of a workgroup: fn(z, index).  LOOP: rows longer than kChunk, read
// again each time.
template <int FMT, bool LOOP>
struct Row {
    const char *p;
    int64_t vocab;
    float z[kSegs][kEach];
    __device__ __forceinline__ void load(int64_t j0) {
#pragma unroll
        for (int i = 0; i < kSegs; ++i) load_seg<FMT>(p, j0 + i * kSeg, vocab, z[i], -__builtin_huge_valf());
    }
    template <typename Fn>
    __device__ __forceinline__ void each(Fn fn) {
        const int lane = static_cast<int>(threadIdx.x & 63);
        const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
        for (int64_t j0 = wave * kSegs * kSeg; j0 < vocab; j0 += kChunk) {
            if constexpr (LOOP) load(j0);
#pragma unroll
            for (int i = 0; i < kSegs; ++i)
#pragma unroll
                for (int e = 0; e < kEach; ++e) fn(z[i][e], static_cast<uint32_t>(j0) + i * kSeg + entry_of<FMT>(lane, e));
            if constexpr (!LOOP) break;
        }
    }
};

// The least order that is kept, of the first `count` entries or of the first whose sum reaches `sum`;
// w_kept: the weight of what is kept.  s.bins holds the cells.
template <typename R>
__device__ uint64_t keep_from(R &row, Shared &s, const Scale &sc, bool by_count, uint32_t count, double sum, double &w_kept) {
    const uint32_t tid = threadIdx.x;
    const int lane = static_cast<int>(tid & 63), wave = static_cast<int>(tid >> 6);
    Border b = border_of(s.bins, by_count, count, sum, [](int i) { return eighths(-i) / kUnit; });
    const int cell = b.bin;
    const double unit = eighths(-cell) / kUnit;
    uint64_t lo = 0, hi = ~0ull;
    const auto inside = [&](float z, uint32_t j, double &y, uint64_t &o) {
        if (!in_row(z)) return false;
        y = sc.y(z);
        o = order_of(z, j);
        return sc.cell(y) == cell && o >= lo && o <= hi;
    };
    count -= b.before, sum -= b.w_before;
    w_kept = b.w_before;
    Bins &bins = s.bins;
    while (b.in > kList) {
        uint64_t least = ~0ull, most = 0;
        row.each([&](float z, uint32_t j) {
            double y;
            uint64_t o;
            if (inside(z, j, y, o)) least = o < least ? o : least, most = o > most ? o : most;
        });
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) {
            const uint64_t l = __shfl_xor(static_cast<unsigned long long>(least), off, 64);
            const uint64_t m = __shfl_xor(static_cast<unsigned long long>(most), off, 64);
            least = l < least ? l : least, most = m > most ? m : most;
        }
        __syncthreads();                           // the bins have been read
        if (lane == 0) s.least[wave] = least, s.most[wave] = most;
        if (tid < kCells) bins.sum[tid] = 0, bins.count[tid] = 0;
        __syncthreads();
        for (int w = 0; w < static_cast<int>(blockDim.x >> 6); ++w) {
            least = s.least[w] < least ? s.least[w] : least;
            most = s.most[w] > most ? s.most[w] : most;
        }
        lo = least, hi = most;
        const int bits = 64 - __builtin_clzll(hi - lo | 1), shift = bits > 8 ? bits - 8 : 0;
        row.each([&](float z, uint32_t j) {
            double y;
            uint64_t o;
            if (inside(z, j, y, o)) {
                const int at = static_cast<int>((hi - o) >> shift);
                atomicAdd(&bins.count[at], 1u);
                atomicAdd(reinterpret_cast<unsigned long long *>(&bins.sum[at]), static_cast<unsigned long long>(sc.whole(y, cell)));
            }
        });
        __syncthreads();
        b = border_of(bins, by_count, count, sum, [&](int) { return unit; });
        count -= b.before, sum -= b.w_before;
        w_kept += b.w_before;
        hi -= static_cast<uint64_t>(b.bin) << shift;
        const uint64_t width = (1ull << shift) - 1;
        lo = hi - lo > width ? hi - width : lo;
    }
    __syncthreads();
    if (tid == 0) s.n = 0;
    __syncthreads();
    row.each([&](float z, uint32_t j) {
        double y;
        uint64_t o;
        if (inside(z, j, y, o)) s.list[atomicAdd(&s.n, 1u)] = o;
    });
    __syncthreads();
    const uint32_t n = s.n;                        // b.in
    if (tid < n) {
        const uint64_t mine = s.list[tid];
        uint32_t rank = 0;
        for (uint32_t i = 0; i < n; ++i) rank += s.list[i] > mine ? 1u : 0u;
        s.sorted[rank] = mine;
    }
    __syncthreads();
    // every wave: four successive entries a lane
    constexpr int kMine = kList / 64;
    double w[kMine], ws = 0;
    uint64_t o[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const uint32_t at = lane * kMine + i;
        o[i] = at < n ? s.sorted[at] : 0;
        w[i] = at < n ? sc.weight(logit_of(o[i])) : 0;
        ws += w[i];
    }
    const double up = lanes_before(ws);
    double at = up - ws;
    int hit = -1, last = -1;
    double hit_w = 0, last_w = 0;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        at += w[i];
        const uint32_t place = lane * kMine + i;
        if (place < n) {
            last = i, last_w = at;
            if (hit < 0 && (by_count ? place + 1 >= count : at >= sum)) hit = i, hit_w = at;
        }
    }
    const uint64_t hits = __ballot(hit >= 0), some = __ballot(last >= 0);
    const int l = hits ? __builtin_ctzll(hits) : 63 - __builtin_clzll(some);
    w_kept += lane_value(hits ? hit_w : last_w, l);
    const int which = __builtin_amdgcn_readlane(hits ? hit : last, l);
    __syncthreads();
    return s.sorted[l * kMine + which];
}

template <int FMT, bool LOOP>
__global__ __launch_bounds__(kWaves * 64) void sample_kernel(SampleArgs a) {
    __shared__ Shared s;
    __shared__ double seg_sum[LOOP ? kMostSegs : kWaves * kSegs];
    constexpr int kSize = FMT == WSL_OUT_F32 ? 4 : 2;
    const int64_t r = blockIdx.x;
    const uint32_t tid = threadIdx.x;
    const int lane = static_cast<int>(tid & 63), wave = __builtin_amdgcn_readfirstlane(static_cast<int>(tid >> 6));
    const int waves = static_cast<int>(blockDim.x >> 6);
    Row<FMT, LOOP> row;
    row.p = static_cast<const char *>(a.logits) + r * a.ld * kSize;
    row.vocab = a.vocab;
    if constexpr (!LOOP) row.load(wave * kSegs * kSeg);
    const float t = a.how.d_temperature ? a.how.d_temperature[r] : a.how.temperature;
    const float top_p = a.how.d_top_p ? a.how.d_top_p[r] : a.how.top_p;
    const float min_p = a.how.d_min_p ? a.how.d_min_p[r] : a.how.min_p;
    int64_t k = a.how.d_top_k ? a.how.d_top_k[r] : a.how.top_k;
    const bool greedy = !(t > 0) || k == 1 || top_p <= 0;
    if (k <= 0 || k > a.vocab) k = a.vocab;

    // the greatest entry
    float m = -__builtin_huge_valf();
    bool bad = false;
    row.each([&](float z, uint32_t) {
        bad |= !(z < __builtin_huge_valf());
        m = z > m ? z : m;
    });
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
        const float o = __shfl_xor(m, off, 64);
        m = o > m ? o : m;
    }
    const bool any_bad = __ballot(bad) != 0;
    if (tid == 0) s.bad = 0, s.n = ~0u;
    if (tid < kCells) s.bins.sum[tid] = 0, s.bins.count[tid] = 0;
    __syncthreads();
    if (lane == 0) {
        s.top[wave] = m;
        if (any_bad) atomicOr(&s.bad, 1u);
    }
    __syncthreads();
    for (int w = 0; w < waves; ++w) m = s.top[w] > m ? s.top[w] : m;
    if (s.bad || !in_row(m)) {
        if (a.probs)
            for (int64_t j = tid; j < a.vocab; j += blockDim.x) a.probs[r * a.ld_probs + j] = 0.f;
        if (tid == 0) {
            if (a.tokens) a.tokens[r] = -1;
            if (a.status) atomicOr(a.status, WSL_STATUS_NONFINITE);
        }
        return;
    }
    if (greedy) {
        uint32_t at = ~0u;
        row.each([&](float z, uint32_t j) { at = z == m && j < at ? j : at; });
        if (at != ~0u) atomicMin(&s.n, at);
        __syncthreads();
        at = s.n;
        if (a.probs)
            for (int64_t j = tid; j < a.vocab; j += blockDim.x) a.probs[r * a.ld_probs + j] = j == at ? 1.f : 0.f;
        if (a.tokens && tid == 0) a.tokens[r] = static_cast<int32_t>(at);
        return;
    }
    Scale sc;
    sc.c8 = 11.541560327111707 / static_cast<double>(t);           // 8 log2(e)
    sc.m = m;
    uint64_t from = 0;
    if (k < a.vocab || top_p < 1) {
        row.each([&](float z, uint32_t) {
            if (in_row(z)) {
                const double y = sc.y(z);
                const int c = sc.cell(y);
                atomicAdd(&s.bins.count[c], 1u);
                atomicAdd(reinterpret_cast<unsigned long long *>(&s.bins.sum[c]), static_cast<unsigned long long>(sc.whole(y, c)));
            }
        });
        __syncthreads();
        double w_kept = 0, w_top = 0;
        const Border all = border_of(s.bins, true, static_cast<uint32_t>(a.vocab) + 1, 0, [](int i) { return eighths(-i) / kUnit; });
        w_kept = all.w_all;
        if (k < all.before + all.in) {
            from = keep_from(row, s, sc, true, static_cast<uint32_t>(k), 0, w_kept);
            if (top_p < 1) {                       // the cells again: narrowing may have taken their place
                __syncthreads();
                if (tid < kCells) s.bins.sum[tid] = 0, s.bins.count[tid] = 0;
                __syncthreads();
                row.each([&](float z, uint32_t) {
                    if (in_row(z)) {
                        const double y = sc.y(z);
                        const int c = sc.cell(y);
                        atomicAdd(&s.bins.count[c], 1u);
                        atomicAdd(reinterpret_cast<unsigned long long *>(&s.bins.sum[c]), static_cast<unsigned long long>(sc.whole(y, c)));
                    }
                });
                __syncthreads();
            }
        }
        if (top_p < 1) {
            const uint64_t p_from = keep_from(row, s, sc, false, 0, static_cast<double>(top_p) * w_kept, w_top);
            from = p_from > from ? p_from : from;
        }
    }
    const double least_y = min_p > 0 ? 8 * log2(static_cast<double>(min_p < 1 ? min_p : 1.f)) : -__builtin_huge_val();
    const auto weight = [&](float z, uint32_t j) {
        return in_row(z) && order_of(z, j) >= from && sc.y(z) >= least_y ? sc.weight(z) : 0.0;
    };
    // sums of the segments, in the order of the entries
    for (int64_t j0 = wave * kSegs * kSeg; j0 < a.vocab; j0 += kChunk) {
        if constexpr (LOOP) row.load(j0);
#pragma unroll
        for (int i = 0; i < kSegs; ++i) {
            double w = 0;
#pragma unroll
            for (int e = 0; e < kEach; ++e) w += weight(row.z[i][e], static_cast<uint32_t>(j0) + i * kSeg + entry_of<FMT>(lane, e));
            w = lanes_total(w);
            if (lane == 0) seg_sum[j0 / kSeg + i] = w;
        }
        if constexpr (!LOOP) break;
    }
    __syncthreads();
    const int segs = static_cast<int>((a.vocab + kSeg - 1) / kSeg), each = (segs + 63) / 64;
    const int c0 = each * lane < segs ? each * lane : segs, c1 = c0 + each < segs ? c0 + each : segs;
    double mine = 0;
    for (int c = c0; c < c1; ++c) mine += seg_sum[c];
    const double up = lanes_before(mine), total = lane_value(up, 63);
    if (a.tokens) {
        double target = static_cast<double>(a.u[r]) * total;       // NaN is passed by none: the last one
        if (target < 0) target = 0;
        int hit = -1, last = -1;
        double at = up - mine, hit_at = 0, last_at = 0;
        for (int c = c0; c < c1; ++c) {
            const double w = seg_sum[c];
            if (w > 0) last = c, last_at = at;
            if (hit < 0 && w > 0 && at + w > target) hit = c, hit_at = at;
            at += w;
        }
        const uint64_t hits = __ballot(hit >= 0), some = __ballot(last >= 0);
        const int l = hits ? __builtin_ctzll(hits) : 63 - __builtin_clzll(some);
        const int seg = __builtin_amdgcn_readlane(hits ? hit : last, l);
        const double run = lane_value(hits ? hit_at : last_at, l);
        const int j0 = seg * kSeg;
        if constexpr (LOOP) {
            if (wave == 0) {
                float z[kEach];
                load_seg<FMT>(row.p, j0, a.vocab, z, -__builtin_huge_valf());
                const int32_t token = look_through<FMT>([&](int i) { return weight(z[i], j0 + entry_of<FMT>(lane, i)); }, j0, target, run);
                if (lane == 0) a.tokens[r] = token;
            }
        } else {
#pragma unroll
            for (int q = 0; q < kSegs; ++q)
                if (seg == wave * kSegs + q) {
                    const int32_t token = look_through<FMT>([&](int i) { return weight(row.z[q][i], j0 + entry_of<FMT>(lane, i)); }, j0, target, run);
                    if (lane == 0) a.tokens[r] = token;
                }
        }
    }
    if (a.probs) {
        float *out = a.probs + r * a.ld_probs;
        row.each([&](float z, uint32_t j) {
            if (j < a.vocab) out[j] = static_cast<float>(weight(z, j) / total);
        });
    }
}

template <int FMT>
void go(const SampleArgs &a, int64_t n_rows, hipStream_t s) {
    const unsigned rows = static_cast<unsigned>(n_rows);
    if (a.vocab <= kChunk) {
        const int64_t waves = (a.vocab + kSegs * kSeg - 1) / (kSegs * kSeg);
        hipLaunchKernelGGL((sample_kernel<FMT, false>), dim3(rows), dim3(static_cast<unsigned>(waves < 4 ? 4 : waves) * 64), 0, s, a);
    } else {
        hipLaunchKernelGGL((sample_kernel<FMT, true>), dim3(rows), dim3(kWaves * 64), 0, s, a);
    }
}

}  // namespace

size_t sample_ws_bytes(int64_t, int64_t) { return 0; }

int launch_sample(const void *logits, int zfmt, int64_t n_rows, int64_t vocab, int64_t ld, const wsl_sampling *how,
                  const float *u, int32_t *tokens, float *probs, int64_t ld_probs, void *, uint32_t *status, hipStream_t s) {
    SampleArgs a;
    a.logits = logits, a.u = u, a.tokens = tokens, a.probs = probs, a.status = status;
    a.vocab = vocab, a.ld = ld, a.ld_probs = ld_probs;
    if (how) a.how = *how;
    else a.how = {nullptr, nullptr, nullptr, nullptr, 1.f, 0, 1.f, 0.f};
    if (zfmt == WSL_OUT_F32) go<WSL_OUT_F32>(a, n_rows, s);
    else go<WSL_OUT_BF16>(a, n_rows, s);
    return WSL_OK;
}

}  // namespace wsl
