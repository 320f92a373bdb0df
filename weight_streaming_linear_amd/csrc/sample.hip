// Sampling from logits (sample_logits) for gfx950.
//
// A row's entries are ordered by value, equal ones by index: by the 64-bit number
//     order(j) = ordered bits of z_j, then ~j,
// no two of which are equal.  Whatever top-k, top-p and min-p keep is a beginning of that order, so a
// row needs one border and not a sort:
//     w = exp((z - max z) / T) = 2^((y - max y) / 8),  y = c z,  c = 8 log2(e) / T,
//     cell of an entry = min(rint(max y) - rint(y), 255): an eighth of a power of two each, in order;
// counts and weight sums of the cells say which cell the border of top-k, top-p or min-p lies in, and only
// that cell's entries are looked at further: up to kList of them are put in order, more are first
// narrowed by 256 ranges of order(j).  Weights come from 64-bit arithmetic; in a cell they are
// added up as whole numbers (of 2^-32 or 2^-40 of the cell's unit), which no order of adding changes.  The
// greatest entries weigh 1 exactly, so that rows of equal logits have exact sums.
// The token is then found as in verify_drafts: sums of segments in the order of the entries, and the
// segment that passes u * total looked through.
//
// A row up to kChunk entries is one workgroup's, in registers.  Longer ones are cut into segments, a
// workgroup each, so that few rows fill the chip too, in up to four launches: cells of each segment
// (relative to its own greatest entry, shifted by whole cells when they are put together); the entries
// of the border's cells as a list; the border and the token, one workgroup a row; the probabilities.
// The first two read the row, the second mostly from the caches.
#include "row_scan.h"

namespace wsl {
namespace {

constexpr int kSegs = 2;                       // segments of kSeg entries that a wave of a short row holds
constexpr int kSmallWaves = 4, kChunk = kSmallWaves * kSegs * kSeg;
constexpr int kCells = 256, kList = 256;
constexpr int kMostWaves = 16, kMostParts = 256;
constexpr int kGathered = 8192;                // entries that a row's list holds
constexpr double kUnit = 1099511627776.0;      // 2^40: whole numbers to a cell's unit; 2^22 entries of it fit 64 bits
constexpr double kPartUnit = 4294967296.0;     // 2^32, and 2^14 entries of a part fit 48 bits
constexpr float kInf = __builtin_huge_valf();

// What a part of a long row finds.
struct PartHead {
    float m;                                   // its greatest entry
    uint32_t first;                            // the first that is as great (greedy rows)
    uint32_t bad;
    uint32_t at;                               // where its entries begin in the row's list
};
// Which cells' entries are needed one by one, and what is on.
struct Plan {
    int32_t k_on, p_on;
    int32_t one, lo, hi, min;                  // cells: of top-k, from .. to of top-p, of min-p; -1: none
    uint32_t n;                                // their entries
    __device__ __forceinline__ bool wants(int c) const { return c == one || (c >= lo && c <= hi) || c == min; }
};
// Counts and weights of 256 cells (or ranges).
struct Bins {
    double w[kCells];
    uint32_t count[kCells];
};
struct RowPlan {
    Bins cells;
    Plan plan;
    uint32_t pad;
};
// What is decided of a long row, for the probabilities.
struct RowOut {
    double total;                              // 0: every probability is 0
    double least;                              // of y, by min-p
    uint64_t from;                             // of order
    float m;
    int32_t only;                              // the one entry kept, or -1
};

struct SampleArgs {
    const void *logits;
    const float *u;
    int32_t *tokens;
    float *probs;
    uint32_t *status;
    int64_t vocab, ld, ld_probs;
    wsl_sampling how;
    // long rows
    PartHead *heads;                           // [rows][parts]
    uint64_t *cells;                           // [rows][parts][kCells]: count in the upper 16 bits, sum
    uint64_t *list;                            // [rows][kGathered]
    RowPlan *plans;                            // [rows]
    RowOut *outs;                              // [rows]
    int32_t parts, part;                       // of a row, and entries of one
};

// A row's settings.
struct How {
    double c8;                                 // y = c8 * z
    double log_min_p;                          // 8 log2(min_p), or -infinity
    float top_p;                               // 1: off
    uint32_t k;                                // vocab: off
    bool greedy;
};
__device__ __forceinline__ How how_of(const SampleArgs &a, int64_t r) {
    const float t = a.how.d_temperature ? a.how.d_temperature[r] : a.how.temperature;
    const float top_p = a.how.d_top_p ? a.how.d_top_p[r] : a.how.top_p;
    const float min_p = a.how.d_min_p ? a.how.d_min_p[r] : a.how.min_p;
    const int32_t k = a.how.d_top_k ? a.how.d_top_k[r] : a.how.top_k;
    How h;
    h.greedy = !(t > 0) || k == 1 || top_p <= 0;
    h.c8 = 11.541560327111707 / static_cast<double>(t > 0 ? t : 1.f);          // 8 log2(e) / T
    h.top_p = top_p < 1 ? top_p : 1.f;
    h.k = k <= 0 || k > a.vocab ? static_cast<uint32_t>(a.vocab) : static_cast<uint32_t>(k);
    h.log_min_p = min_p > 0 ? 8 * log2(static_cast<double>(min_p < 1 ? min_p : 1.f)) : -__builtin_huge_val();
    return h;
}

// 2^(n / 8) for whole n of any size.
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
// 2^(f / 8), |f| <= 1/2: the Taylor series of exp(f ln 2 / 8) to the 7th power, right to 2^-50 (and 1 for an
// f that is nearly 0: logits that a high temperature makes equal weigh the same).
constexpr double kEighth = 0.08664339756999316;        // ln 2 / 8
__device__ __forceinline__ double power(double f) {
    const double x = f * kEighth;
    double r = __builtin_fma(1.0 / 5040, x, 1.0 / 720);
    r = __builtin_fma(r, x, 1.0 / 120);
    r = __builtin_fma(r, x, 1.0 / 24);
    r = __builtin_fma(r, x, 1.0 / 6);
    r = __builtin_fma(r, x, 0.5);
    r = __builtin_fma(r, x, 1.0);
    return __builtin_fma(r, x, 1.0);
}
// The same to the 5th power (2^-36), as a whole number of 2^-32: the last sum is above 2^52, whose fraction
// ends at 1, so its low bits are the number, rounded once.
__device__ __forceinline__ uint64_t whole_power(double f) {
    constexpr double k1 = kEighth * kPartUnit, k2 = kEighth * k1 / 2, k3 = kEighth * k2 / 3, k4 = kEighth * k3 / 4,
                     k5 = kEighth * k4 / 5;
    double r = __builtin_fma(k5, f, k4);
    r = __builtin_fma(r, f, k3);
    r = __builtin_fma(r, f, k2);
    r = __builtin_fma(r, f, k1);
    return __builtin_bit_cast(uint64_t, __builtin_fma(r, f, kPartUnit + 4503599627370496.0)) & 0x3ffffffffull;
}

__device__ __forceinline__ bool in_row(float z) { return z > -kInf; }

__device__ __forceinline__ uint64_t order_of(float z, uint32_t index) {
    const uint32_t b = __builtin_bit_cast(uint32_t, z + 0.f);      // -0 is 0
    const uint32_t key = b ^ (b >> 31 ? 0xffffffffu : 0x80000000u);
    return static_cast<uint64_t>(key) << 32 | ~index;
}
__device__ __forceinline__ float logit_of(uint64_t order) {
    const uint32_t key = static_cast<uint32_t>(order >> 32);
    return __builtin_bit_cast(float, key ^ (key >> 31 ? 0x80000000u : 0xffffffffu));
}

// A row's cells and weights, once its greatest entry m is known.
struct Scale {
    double c8, m, n_m;                         // n_m = rint(c8 * m)
    __device__ __forceinline__ Scale(double c8_, float m_) : c8(c8_), m(m_), n_m(__builtin_rint(c8_ * static_cast<double>(m_))) {}
    __device__ __forceinline__ double y(float z) const { return c8 * static_cast<double>(z); }
    __device__ __forceinline__ int cell(double y) const {
        const double d = n_m - __builtin_rint(y);
        return static_cast<int>(d < kCells - 1 ? d : kCells - 1);
    }
    __device__ __forceinline__ double weight(float z) const {
        const double v = c8 * (static_cast<double>(z) - m), n = __builtin_rint(v);
        return power(v - n) * eighths(n);
    }
    // a power of two near the weights of a cell, and a weight as a whole number of 2^-40 of it
    static __device__ __forceinline__ double unit(int cell) { return __builtin_ldexp(1.0, -(cell >> 3)); }
    __device__ __forceinline__ uint64_t whole(float z, int cell) const {
        return static_cast<uint64_t>(__builtin_fma(__builtin_ldexp(weight(z), cell >> 3), kUnit, 0.5));
    }
};

// Where a count or a sum is reached.
struct Border {
    int bin;
    uint32_t before, in;           // entries before the bin, and in it
    double w_before, w_all;        // weights before it, and of all bins
};
// The first bin up to which there are `count` entries (by_count), or a sum of `sum`; where rounding lets
// none, the last that holds any.  Every wave comes to the same.
__device__ __forceinline__ Border border_of(const Bins &b, bool by_count, uint32_t count, double sum) {
    const int lane = static_cast<int>(threadIdx.x & 63);
    constexpr int kMine = kCells / 64;
    uint32_t c[kMine], cs = 0;
    double w[kMine], ws = 0;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        c[i] = b.count[lane * kMine + i];
        w[i] = b.w[lane * kMine + i];
        cs += c[i], ws += w[i];
    }
    const double up_w = lanes_before(ws);
    double at_w = up_w - ws;
    uint32_t at_c = lanes_before(cs) - cs;
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
    Bins cells, bins;
    uint64_t sum[kCells];
    uint64_t list[kList], sorted[kList];
    uint32_t rank[kList];
    uint64_t least[kMostWaves], most[kMostWaves];
    float top[kMostWaves];
    uint32_t n, bad;
};

// What keep_from goes over, by all waves of a workgroup: fn(z, order).  A short row, in registers:
template <int FMT>
struct ShortRow {
    float z[kSegs][kEach];
    template <typename Fn>
    __device__ __forceinline__ void each(Fn fn) const {
        const int lane = static_cast<int>(threadIdx.x & 63);
        const uint32_t j0 = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6)) * kSegs * kSeg;
#pragma unroll
        for (int i = 0; i < kSegs; ++i)
#pragma unroll
            for (int e = 0; e < kEach; ++e) fn(z[i][e], order_of(z[i][e], j0 + i * kSeg + entry_of<FMT>(lane, e)));
    }
};
// A long row that its list has no room for, read again each time:
template <int FMT>
struct LongRow {
    const char *p;
    int64_t vocab;
    template <typename Fn>
    __device__ __forceinline__ void each(Fn fn) const {
        const int lane = static_cast<int>(threadIdx.x & 63);
        const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
        for (int64_t j0 = wave * kSeg; j0 < vocab; j0 += static_cast<int64_t>(blockDim.x) / 64 * kSeg) {
            float z[kEach];
            load_seg<FMT>(p, j0, vocab, z, -kInf);
#pragma unroll
            for (int e = 0; e < kEach; ++e) fn(z[e], order_of(z[e], static_cast<uint32_t>(j0) + entry_of<FMT>(lane, e)));
        }
    }
};
// The list of a long row's border cells, in registers; entries that are none have order 0.
constexpr int kHeld = kGathered / (kMostWaves * 64);
struct Gathered {
    uint64_t o[kHeld];
    template <typename Fn>
    __device__ __forceinline__ void each(Fn fn) const {
#pragma unroll
        for (int i = 0; i < kHeld; ++i) fn(o[i] ? logit_of(o[i]) : -kInf, o[i]);
    }
};

// The least order that is kept, of the first `count` entries or of the first whose sum reaches `sum`;
// w_kept: the weight of what is kept; cell: the cell it lies in.  s.cells holds the cells of all.
template <typename From>
__device__ uint64_t keep_from(const From &row, Shared &s, const Scale &sc, bool by_count, uint32_t count, double sum,
                              double &w_kept, int &cell) {
    const uint32_t tid = threadIdx.x;
    const int lane = static_cast<int>(tid & 63), wave = static_cast<int>(tid >> 6);
    Border b = border_of(s.cells, by_count, count, sum);
    cell = b.bin;
    const int in_cell = cell;
    const double unit = Scale::unit(cell) / kUnit;
    uint64_t lo = 0, hi = ~0ull;
    const auto inside = [&](float z, uint64_t o) {
        return in_row(z) && o >= lo && o <= hi && sc.cell(sc.y(z)) == in_cell;
    };
    count -= b.before, sum -= b.w_before;
    w_kept = b.w_before;
    while (b.in > kList) {
        uint64_t least = ~0ull, most = 0;
        row.each([&](float z, uint64_t o) {
            if (inside(z, o)) least = o < least ? o : least, most = o > most ? o : most;
        });
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) {
            const uint64_t l = __shfl_xor(static_cast<unsigned long long>(least), off, 64);
            const uint64_t m = __shfl_xor(static_cast<unsigned long long>(most), off, 64);
            least = l < least ? l : least, most = m > most ? m : most;
        }
        __syncthreads();                           // the bins have been read
        if (lane == 0) s.least[wave] = least, s.most[wave] = most;
        if (tid < kCells) s.sum[tid] = 0, s.bins.count[tid] = 0;
        __syncthreads();
        for (int w = 0; w < static_cast<int>(blockDim.x >> 6); ++w) {
            least = s.least[w] < least ? s.least[w] : least;
            most = s.most[w] > most ? s.most[w] : most;
        }
        lo = least, hi = most;
        const int bits = 64 - __builtin_clzll(hi - lo | 1), shift = bits > 8 ? bits - 8 : 0;
        row.each([&](float z, uint64_t o) {
            if (inside(z, o)) {
                const int at = static_cast<int>((hi - o) >> shift);
                atomicAdd(&s.bins.count[at], 1u);
                atomicAdd(reinterpret_cast<unsigned long long *>(&s.sum[at]), static_cast<unsigned long long>(sc.whole(z, in_cell)));
            }
        });
        __syncthreads();
        if (tid < kCells) s.bins.w[tid] = static_cast<double>(s.sum[tid]) * unit;
        __syncthreads();
        b = border_of(s.bins, by_count, count, sum);
        count -= b.before, sum -= b.w_before;
        w_kept += b.w_before;
        hi -= static_cast<uint64_t>(b.bin) << shift;
        const uint64_t width = (1ull << shift) - 1;
        lo = hi - lo > width ? hi - width : lo;
    }
    if (tid == 0) s.n = 0;
    __syncthreads();
    row.each([&](float z, uint64_t o) {
        if (inside(z, o)) {
            const uint32_t at = atomicAdd(&s.n, 1u);
            if (at < kList) s.list[at] = o;
        }
    });
    __syncthreads();
    const uint32_t n = s.n < kList ? s.n : kList;  // b.in
    // an entry's place: as many threads as there are for each, a part of the list each
    const uint32_t shares = blockDim.x / kList, entry = tid % kList, share = tid / kList;
    if (tid < kList) s.rank[tid] = 0;
    __syncthreads();
    if (entry < n) {
        const uint64_t mine = s.list[entry];
        const uint32_t i0 = n * share / shares, i1 = n * (share + 1) / shares;
        uint32_t rank = 0;
#pragma unroll 8
        for (uint32_t i = i0; i < i1; ++i) rank += s.list[i] > mine ? 1u : 0u;
        atomicAdd(&s.rank[entry], rank);
    }
    __syncthreads();
    if (tid < n) s.sorted[s.rank[tid]] = s.list[tid];
    __syncthreads();
    // every wave: four successive entries a lane
    constexpr int kMine = kList / 64;
    double w[kMine], ws = 0;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
        const uint32_t at = lane * kMine + i;
        w[i] = at < n ? sc.weight(logit_of(s.sorted[at])) : 0;
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
    if (!some) return ~0ull;                       // (a border lies in a cell that holds something)
    const int l = hits ? __builtin_ctzll(hits) : 63 - __builtin_clzll(some);
    w_kept += lane_value(hits ? hit_w : last_w, l);
    const int which = __builtin_amdgcn_readlane(hits ? hit : last, l);
    const uint64_t from = s.sorted[l * kMine + which];
    __syncthreads();                               // the list and the bins may be used again
    return from;
}

// In the order of n sums (LDS): the first that passes the target, or the last that is not zero, and what lies
// before it.  Every wave comes to the same; n is at most 64 * what a lane takes.
struct Place {
    int at;
    double before;
};
__device__ __forceinline__ Place place_of(const double *sums, int n, double target) {
    const int lane = static_cast<int>(threadIdx.x & 63), each = (n + 63) / 64;
    const int c0 = each * lane < n ? each * lane : n, c1 = c0 + each < n ? c0 + each : n;
    double mine = 0;
    for (int c = c0; c < c1; ++c) mine += sums[c];
    double at = lanes_before(mine) - mine;
    int hit = -1, last = -1;
    double hit_at = 0, last_at = 0;
    for (int c = c0; c < c1; ++c) {
        const double w = sums[c];
        if (w > 0) last = c, last_at = at;
        if (hit < 0 && w > 0 && at + w > target) hit = c, hit_at = at;
        at += w;
    }
    const uint64_t hits = __ballot(hit >= 0), some = __ballot(last >= 0);
    if (!some) return Place{0, 0.0};
    const int l = hits ? __builtin_ctzll(hits) : 63 - __builtin_clzll(some);
    return Place{__builtin_amdgcn_readlane(hits ? hit : last, l), lane_value(hits ? hit_at : last_at, l)};
}
__device__ __forceinline__ double total_of(const double *sums, int n) {
    const int lane = static_cast<int>(threadIdx.x & 63), each = (n + 63) / 64;
    double mine = 0;
    for (int c = each * lane; c < each * (lane + 1) && c < n; ++c) mine += sums[c];
    return lanes_total(mine);
}
// What running sums have to pass; NaN is passed by none: the last entry, as for u >= 1.
__device__ __forceinline__ double target_of(const SampleArgs &a, int64_t r, double total) {
    const double t = static_cast<double>(a.u[r]) * total;
    return t < 0 ? 0 : t;
}

// ------------------------------------------------------------------ short rows
template <int FMT>
__global__ __launch_bounds__(kSmallWaves * 64) void sample_short_kernel(SampleArgs a) {
    __shared__ Shared s;
    __shared__ double seg_sum[kSmallWaves * kSegs];
    constexpr int kSize = FMT == WSL_OUT_F32 ? 4 : 2;
    const int64_t r = blockIdx.x;
    const uint32_t tid = threadIdx.x;
    const int lane = static_cast<int>(tid & 63), wave = __builtin_amdgcn_readfirstlane(static_cast<int>(tid >> 6));
    const char *p = static_cast<const char *>(a.logits) + r * a.ld * kSize;
    ShortRow<FMT> row;
#pragma unroll
    for (int i = 0; i < kSegs; ++i) load_seg<FMT>(p, (wave * kSegs + i) * kSeg, a.vocab, row.z[i], -kInf);
    const How h = how_of(a, r);

    // the greatest entry
    float m = -kInf;
    bool bad = false;
#pragma unroll
    for (int i = 0; i < kSegs; ++i)
#pragma unroll
        for (int e = 0; e < kEach; ++e) bad |= !(row.z[i][e] < kInf), m = row.z[i][e] > m ? row.z[i][e] : m;
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
        const float o = __shfl_xor(m, off, 64);
        m = o > m ? o : m;
    }
    const bool any_bad = __ballot(bad) != 0;
    if (tid == 0) s.bad = 0, s.n = ~0u;
    if (tid < kCells) s.sum[tid] = 0, s.cells.count[tid] = 0;
    __syncthreads();
    if (lane == 0) {
        s.top[wave] = m;
        if (any_bad) atomicOr(&s.bad, 1u);
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSmallWaves; ++w) m = s.top[w] > m ? s.top[w] : m;
    if (s.bad || !in_row(m)) {
        if (a.probs)
            for (int64_t j = tid; j < a.vocab; j += blockDim.x) a.probs[r * a.ld_probs + j] = 0.f;
        if (tid == 0) {
            if (a.tokens) a.tokens[r] = -1;
            if (a.status) atomicOr(a.status, WSL_STATUS_NONFINITE);
        }
        return;
    }
    if (h.greedy) {
        uint64_t first = 0;                        // the greatest order
        row.each([&](float z, uint64_t o) { first = z == m && o > first ? o : first; });
        if (first) atomicMin(&s.n, ~static_cast<uint32_t>(first));
        __syncthreads();
        const uint32_t at = s.n;
        if (a.probs)
            for (int64_t j = tid; j < a.vocab; j += blockDim.x) a.probs[r * a.ld_probs + j] = j == at ? 1.f : 0.f;
        if (a.tokens && tid == 0) a.tokens[r] = static_cast<int32_t>(at);
        return;
    }
    const Scale sc(h.c8, m);
    uint64_t from = 0;
    if (h.k < a.vocab || h.top_p < 1) {
        row.each([&](float z, uint64_t) {
            if (in_row(z)) {
                const int c = sc.cell(sc.y(z));
                atomicAdd(&s.cells.count[c], 1u);
                atomicAdd(reinterpret_cast<unsigned long long *>(&s.sum[c]), static_cast<unsigned long long>(sc.whole(z, c)));
            }
        });
        __syncthreads();
        if (tid < kCells) s.cells.w[tid] = static_cast<double>(s.sum[tid]) * (Scale::unit(tid) / kUnit);
        __syncthreads();
        const Border all = border_of(s.cells, true, ~0u, 0);
        double w_kept = all.w_all, w_top;
        int cell;
        if (h.k < all.before + all.in) from = keep_from(row, s, sc, true, h.k, 0, w_kept, cell);
        if (h.top_p < 1) {
            const uint64_t p_from = keep_from(row, s, sc, false, 0, static_cast<double>(h.top_p) * w_kept, w_top, cell);
            from = p_from > from ? p_from : from;
        }
    }
    const double least = sc.y(m) + h.log_min_p;
    const auto weight = [&](float z, uint32_t j) {
        return in_row(z) && order_of(z, j) >= from && sc.y(z) >= least ? sc.weight(z) : 0.0;
    };
    const uint32_t j0 = wave * kSegs * kSeg;
#pragma unroll
    for (int i = 0; i < kSegs; ++i) {
        double w = 0;
#pragma unroll
        for (int e = 0; e < kEach; ++e) w += weight(row.z[i][e], j0 + i * kSeg + entry_of<FMT>(lane, e));
        w = lanes_total(w);
        if (lane == 0) seg_sum[wave * kSegs + i] = w;
    }
    __syncthreads();
    const double total = total_of(seg_sum, kSmallWaves * kSegs);
    if (a.tokens) {
        const double target = target_of(a, r, total);
        const Place at = place_of(seg_sum, kSmallWaves * kSegs, target);
#pragma unroll
        for (int i = 0; i < kSegs; ++i)
            if (at.at == wave * kSegs + i) {
                const int32_t token = look_through<FMT>(
                    [&](int e) { return weight(row.z[i][e], at.at * kSeg + entry_of<FMT>(lane, e)); }, at.at * kSeg, target, at.before);
                if (lane == 0) a.tokens[r] = token;
            }
    }
    if (a.probs) {
        float *out = a.probs + r * a.ld_probs;
#pragma unroll
        for (int i = 0; i < kSegs; ++i)
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const uint32_t j = j0 + i * kSeg + entry_of<FMT>(lane, e);
                if (j < a.vocab) out[j] = static_cast<float>(weight(row.z[i][e], j) / total);
            }
    }
}

// ------------------------------------------------------------------ long rows
// Cells of one part: blockIdx (part, row), a wave a segment.  Bound by the 64-bit arithmetic, about 16
// instructions an entry (an exponential in 32 bits would take as many and leave 2^-22 of a weight).
template <int FMT>
__global__ __launch_bounds__(kMostWaves * 64) void sample_cells_kernel(SampleArgs a) {
    __shared__ uint64_t cells[kCells];
    __shared__ float top[kMostWaves];
    __shared__ uint32_t first, bad;
    constexpr int kSize = FMT == WSL_OUT_F32 ? 4 : 2;
    const int64_t r = blockIdx.y;
    const uint32_t tid = threadIdx.x;
    const int lane = static_cast<int>(tid & 63), wave = __builtin_amdgcn_readfirstlane(static_cast<int>(tid >> 6));
    const int waves = static_cast<int>(blockDim.x >> 6);
    const int64_t j0 = static_cast<int64_t>(blockIdx.x) * a.part + wave * kSeg;
    float z[kEach];
    load_seg<FMT>(static_cast<const char *>(a.logits) + r * a.ld * kSize, j0, a.vocab, z, -kInf);
    const How h = how_of(a, r);
    if (tid == 0) first = ~0u, bad = 0;
    if (tid < kCells) cells[tid] = 0;
    float m = -kInf;
    bool mine_bad = false;
#pragma unroll
    for (int e = 0; e < kEach; ++e) mine_bad |= !(z[e] < kInf), m = z[e] > m ? z[e] : m;
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
        const float o = __shfl_xor(m, off, 64);
        m = o > m ? o : m;
    }
    const bool any_bad = __ballot(mine_bad) != 0;
    if (lane == 0) top[wave] = m;
    __syncthreads();
    if (lane == 0 && any_bad) atomicOr(&bad, 1u);
    for (int w = 0; w < waves; ++w) m = top[w] > m ? top[w] : m;
    if (h.greedy) {
        uint32_t at = ~0u;
#pragma unroll
        for (int e = kEach - 1; e >= 0; --e) at = z[e] == m ? static_cast<uint32_t>(j0) + entry_of<FMT>(lane, e) : at;
        if (at != ~0u) atomicMin(&first, at);
    } else if (in_row(m)) {
        const double n_m = __builtin_rint(h.c8 * static_cast<double>(m));
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const double y = h.c8 * static_cast<double>(z[e]), n = __builtin_rint(y), d = n_m - n;
            uint64_t v = whole_power(y - n) + (1ull << 48);
            int c = static_cast<int>(d);
            bool put = d < kCells - 1;
            if (__ballot(!put)) {              // the last cell's entries count by how far they are behind it
                if (!put) {
                    c = kCells - 1, put = in_row(z[e]);
                    const float w = exp2f(static_cast<float>(y - (n_m - (kCells - 1))) * 0.125f) * 4294967296.f;
                    v = static_cast<uint64_t>(w) + (1ull << 48);
                }
            }
            if (put) atomicAdd(reinterpret_cast<unsigned long long *>(&cells[c]), static_cast<unsigned long long>(v));
        }
    }
    __syncthreads();
    const int64_t at = r * a.parts + blockIdx.x;
    if (tid < kCells && !h.greedy) a.cells[at * kCells + tid] = cells[tid];
    if (tid == 0) a.heads[at] = PartHead{m, first, bad, 0};
}

// A long row put together from its parts.
struct LongShared {
    float m[kMostParts];
    double below[kMostParts];                      // cells that a part's lie below the row's
    int32_t shift[kMostParts];                     // the same, 255 at most
    double part_sum[kMostParts];
    uint32_t part_count[kMostParts];
    double w[kMostWaves / 4][kCells];
    uint32_t count[kMostWaves / 4][kCells];
    double rest[kMostWaves];
    uint32_t rest_count[kMostWaves];
    uint32_t bad, first;
};
struct Whole {
    float m;
    uint32_t bad, first;
};

__device__ __forceinline__ Whole heads_of(const SampleArgs &a, int64_t r, double c8, LongShared &s) {
    const uint32_t tid = threadIdx.x;
    if (tid == 0) s.bad = 0, s.first = ~0u;
    PartHead p = {-kInf, ~0u, 0, 0};
    if (tid < static_cast<uint32_t>(a.parts)) {
        p = a.heads[r * a.parts + tid];
        s.m[tid] = p.m;
    }
    __syncthreads();
    Whole o;
    o.m = -kInf;
    for (int i = 0; i < a.parts; ++i) o.m = s.m[i] > o.m ? s.m[i] : o.m;
    if (p.bad) atomicOr(&s.bad, 1u);
    if (p.m == o.m && p.first != ~0u) atomicMin(&s.first, p.first);
    if (tid < static_cast<uint32_t>(a.parts)) {
        const double d = __builtin_rint(c8 * static_cast<double>(o.m)) - __builtin_rint(c8 * static_cast<double>(p.m));
        s.below[tid] = d < 100000 ? d : 100000;    // (a part of -infinities, and infinite temperature: NaN)
        s.shift[tid] = static_cast<int>(d < kCells - 1 ? d : kCells - 1);
    }
    __syncthreads();
    o.bad = s.bad, o.first = s.first;
    return o;
}

// The sum of a cell's whole numbers as a weight: by the number of the greatest entry, which weighs 1.
__device__ __forceinline__ double top_whole(const Scale &sc) {
    const double y = sc.y(static_cast<float>(sc.m));
    return static_cast<double>(whole_power(y - sc.n_m));
}

// The row's cells from its parts': groups of 256 threads take every so many parts, a thread a cell of the
// row, and of the part where that lies in or behind the last.
__device__ __forceinline__ void put_together(const SampleArgs &a, int64_t r, const Scale &sc, LongShared &s, Bins &cells) {
    const uint32_t tid = threadIdx.x, cell = tid & (kCells - 1), group = tid / kCells, groups = blockDim.x / kCells;
    const int lane = static_cast<int>(tid & 63), wave = static_cast<int>(tid >> 6);
    uint64_t sum = 0;
    double rest = 0;
    uint32_t count = 0, rest_count = 0;
    const uint64_t *mine = a.cells + r * a.parts * kCells;
    const double whole = top_whole(sc);
#pragma unroll 4
    for (int i = group; i < a.parts; i += groups) {
        const int shift = s.shift[i], from = static_cast<int>(cell) - shift;
        const bool here = from >= 0 && cell < kCells - 1, behind = static_cast<int>(cell) + shift >= kCells - 1;
        const uint64_t v = here ? mine[i * kCells + from] : 0, u = behind ? mine[i * kCells + cell] : 0;
        sum += v & 0xffffffffffffull;
        count += static_cast<uint32_t>(v >> 48);
        if (u) {
            rest += static_cast<double>(u & 0xffffffffffffull) / whole * eighths(-(s.below[i] + cell));
            rest_count += static_cast<uint32_t>(u >> 48);
        }
    }
    const double unit = eighths(-static_cast<double>(cell));
    rest = lanes_total(rest);
    rest_count = lane_value(lanes_before(rest_count), 63);
    s.w[group][cell] = static_cast<double>(sum), s.count[group][cell] = count;
    if (lane == 0) s.rest[wave] = rest, s.rest_count[wave] = rest_count;
    __syncthreads();
    if (tid < kCells) {
        double w = 0;
        count = 0;
        for (uint32_t g = 0; g < groups; ++g) w += s.w[g][cell], count += s.count[g][cell];
        w = w / whole * unit;
        if (cell == kCells - 1)
            for (uint32_t i = 0; i < groups * 4; ++i) w += s.rest[i], count += s.rest_count[i];
        cells.w[cell] = w, cells.count[cell] = count;
    }
    __syncthreads();
}

__device__ __forceinline__ Plan plan_of(const Bins &cells, const Scale &sc, const How &h, double least) {
    const Border all = border_of(cells, true, ~0u, 0);
    Plan p;
    p.k_on = h.k < all.before + all.in, p.p_on = h.top_p < 1;
    p.one = p.min = p.lo = -1, p.hi = -2, p.n = 0;
    double least_w = all.w_all, most_w = all.w_all;
    if (p.k_on) {
        const Border b = border_of(cells, true, h.k, 0);
        p.one = b.bin;
        // between the lightest and the heaviest that (k - before) entries of the cell can be: 2^(1/16) either way
        // of its middle, which is as far from the greatest's, and a little
        const double some = static_cast<double>(h.k - b.before), unit = eighths(-b.bin);
        least_w = b.w_before + (b.bin < kCells - 1 ? 0.916 * unit * some : 0.0);
        most_w = b.w_before + 1.091 * unit * some;
    }
    if (p.p_on) {
        p.lo = border_of(cells, false, 0, static_cast<double>(h.top_p) * least_w * (1 - 1e-6)).bin;
        p.hi = border_of(cells, false, 0, static_cast<double>(h.top_p) * most_w * (1 + 1e-6)).bin;
    }
    if (least > -__builtin_huge_val()) {
        const double d = sc.n_m - __builtin_rint(least);
        const int c = static_cast<int>(d < kCells - 1 ? d : kCells - 1);
        const int first = p.k_on ? (p.p_on && p.lo < p.one ? p.lo : p.one) : (p.p_on ? p.lo : kCells);
        if (c < first) p.k_on = p.p_on = false, p.one = p.lo = -1, p.hi = -2, p.min = c;       // it alone decides
        else if (c <= (p.p_on ? p.hi : first)) p.min = c;
    }
    for (int i = static_cast<int>(threadIdx.x & 63); i < kCells; i += 64) p.n += p.wants(i) ? cells.count[i] : 0u;
    p.n = lane_value(lanes_before(p.n), 63);
    return p;
}

// Entries of each part that the plan wants; a wave a part.
__device__ __forceinline__ void count_parts(const SampleArgs &a, int64_t r, const Plan &p, LongShared &s) {
    const int lane = static_cast<int>(threadIdx.x & 63), wave = static_cast<int>(threadIdx.x >> 6);
    const int waves = static_cast<int>(blockDim.x >> 6);
    for (int i = wave; i < a.parts; i += waves) {
        uint32_t n = 0;
#pragma unroll
        for (int e = 0; e < kCells; e += 64) {
            const int c = e + lane + s.shift[i];
            if (p.wants(c < kCells - 1 ? c : kCells - 1)) n += static_cast<uint32_t>(a.cells[(r * a.parts + i) * kCells + e + lane] >> 48);
        }
        n = lane_value(lanes_before(n), 63);
        if (lane == 0) s.part_count[i] = n;
    }
    __syncthreads();
}

// Whether a row's settings leave entries out (else its cells are all that is needed of it).
__device__ __forceinline__ bool filters(const SampleArgs &a, const How &h) {
    return h.k < a.vocab || h.top_p < 1 || h.log_min_p > -__builtin_huge_val();
}

// The entries of the border's cells, in an order that is the same on every run: blockIdx (part, row).
template <int FMT>
__global__ __launch_bounds__(kMostWaves * 64) void sample_border_kernel(SampleArgs a) {
    __shared__ LongShared s;
    __shared__ Bins cells;
    __shared__ uint32_t found[kMostWaves];
    constexpr int kSize = FMT == WSL_OUT_F32 ? 4 : 2;
    const int64_t r = blockIdx.y;
    const int lane = static_cast<int>(threadIdx.x & 63), wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    const How h = how_of(a, r);
    if (h.greedy || !filters(a, h)) return;
    const Whole all = heads_of(a, r, h.c8, s);
    if (all.bad || !in_row(all.m)) return;
    const Scale sc(h.c8, all.m);
    put_together(a, r, sc, s, cells);
    const Plan p = plan_of(cells, sc, h, sc.y(all.m) + h.log_min_p);
    const bool fits = p.n > 0 && p.n <= kGathered;
    if (fits) count_parts(a, r, p, s);
    if (blockIdx.x == 0) {                         // for the next launch
        RowPlan &out = a.plans[r];
        for (uint32_t i = threadIdx.x; i < kCells; i += blockDim.x) out.cells.w[i] = cells.w[i], out.cells.count[i] = cells.count[i];
        if (threadIdx.x == 0) out.plan = p;
        if (fits && threadIdx.x < static_cast<uint32_t>(a.parts)) {
            uint32_t at = 0;
            for (uint32_t i = 0; i < threadIdx.x; ++i) at += s.part_count[i];
            a.heads[r * a.parts + threadIdx.x].at = at;
        }
    }
    if (!fits || s.part_count[blockIdx.x] == 0) return;
    const int64_t j0 = static_cast<int64_t>(blockIdx.x) * a.part + wave * kSeg;
    float z[kEach];
    load_seg<FMT>(static_cast<const char *>(a.logits) + r * a.ld * kSize, j0, a.vocab, z, -kInf);
    // nearly all entries are outside of what the wanted cells span: looked at in 32 bits, with a margin
    float low = -kInf, high = kInf;
    if (h.c8 > 0) {
        int c0 = p.min >= 0 ? p.min : kCells, c1 = p.min;
        if (p.one >= 0) c0 = p.one < c0 ? p.one : c0, c1 = p.one > c1 ? p.one : c1;
        if (p.hi >= 0) c0 = p.lo < c0 ? p.lo : c0, c1 = p.hi > c1 ? p.hi : c1;
        const double to = (sc.n_m - c0 + 0.51) / h.c8, from = (sc.n_m - c1 - 0.51) / h.c8;
        high = static_cast<float>(to + __builtin_fabs(to) * 1e-6);
        if (c1 < kCells - 1) low = static_cast<float>(from - __builtin_fabs(from) * 1e-6);
    }
    uint32_t mine = 0, n = 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        bool w = z[e] >= low && z[e] <= high;
        if (__ballot(w)) {
            w = w && in_row(z[e]) && p.wants(sc.cell(sc.y(z[e])));
            mine |= w ? 1u << e : 0u;
            n += static_cast<uint32_t>(__popcll(__ballot(w)));
        }
    }
    if (lane == 0) found[wave] = n;
    __syncthreads();
    uint32_t at = 0;
    for (uint32_t i = 0; i < blockIdx.x; ++i) at += s.part_count[i];
    for (int w = 0; w < wave; ++w) at += found[w];
    if (n == 0) return;
    uint64_t *list = a.list + r * kGathered;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const bool w = mine >> e & 1u;
        const uint64_t who = __ballot(w);
        if (who) {
            const uint32_t to = at + static_cast<uint32_t>(__popcll(who & ((1ull << lane) - 1)));
            if (w && to < kGathered) list[to] = order_of(z[e], static_cast<uint32_t>(j0) + entry_of<FMT>(lane, e));
            at += static_cast<uint32_t>(__popcll(who));
        }
    }
}

// The border and the token of a row.
template <int FMT>
__global__ __launch_bounds__(kMostWaves * 64) void sample_pick_kernel(SampleArgs a) {
    __shared__ LongShared s;
    __shared__ Shared t;
    __shared__ double seg_sum[kMostWaves];
    constexpr int kSize = FMT == WSL_OUT_F32 ? 4 : 2;
    const int64_t r = blockIdx.x;
    const uint32_t tid = threadIdx.x;
    const int lane = static_cast<int>(tid & 63), wave = __builtin_amdgcn_readfirstlane(static_cast<int>(tid >> 6));
    const How h = how_of(a, r);
    const char *p_row = static_cast<const char *>(a.logits) + r * a.ld * kSize;
    const bool some = !h.greedy && filters(a, h);
    Plan p = {0, 0, -1, -1, -2, -1, 0};
    if (some) {                                    // (read before it is known that there is anything to sample)
        p = a.plans[r].plan;
        if (tid < kCells) t.cells.w[tid] = a.plans[r].cells.w[tid], t.cells.count[tid] = a.plans[r].cells.count[tid];
    }
    const Whole all = heads_of(a, r, h.c8, s);
    if (all.bad || !in_row(all.m) || h.greedy) {
        const bool fine = !all.bad && in_row(all.m);
        if (tid == 0) {
            if (a.tokens) a.tokens[r] = fine ? static_cast<int32_t>(all.first) : -1;
            if (!fine && a.status) atomicOr(a.status, WSL_STATUS_NONFINITE);
            a.outs[r] = RowOut{0, 0, 0, 0, fine ? static_cast<int32_t>(all.first) : -1};
        }
        return;
    }
    const Scale sc(h.c8, all.m);
    const double least = sc.y(all.m) + h.log_min_p;
    const bool listed = p.n <= kGathered;
    uint64_t from = 0;
    int border = kCells;                           // the cell that is kept in part; those before it are whole
    if (p.n && (p.k_on || p.p_on)) {
        Gathered g;
        const LongRow<FMT> row = {p_row, a.vocab};
#pragma unroll
        for (int i = 0; i < kHeld; ++i) {
            const uint32_t at = i * (kMostWaves * 64) + tid;
            g.o[i] = listed && at < p.n ? a.list[r * kGathered + at] : 0;
        }
        const auto keep = [&](bool by_count, double sum, double &w_kept) {
            int cell;
            const uint64_t o = listed ? keep_from(g, t, sc, by_count, h.k, sum, w_kept, cell)
                                      : keep_from(row, t, sc, by_count, h.k, sum, w_kept, cell);
            from = o > from ? o : from;
            border = cell < border ? cell : border;
        };
        double w_kept = 0, w_top;
        if (p.k_on) keep(true, 0, w_kept);
        else w_kept = border_of(t.cells, true, ~0u, 0).w_all;
        if (p.p_on) keep(false, static_cast<double>(h.top_p) * w_kept, w_top);
    }
    if (p.min >= 0 && p.min < border) border = p.min;      // (which may hold nothing)
    const auto weight = [&](float z, uint64_t o) { return in_row(z) && o >= from && sc.y(z) >= least ? sc.weight(z) : 0.0; };
    // the kept weight of each part; a wave a part: whole cells, and entries of the border's
    const double whole = top_whole(sc);
    for (int i = wave; i < a.parts; i += kMostWaves) {
        double w = 0;
#pragma unroll
        for (int e = 0; e < kCells; e += 64) {
            const int c = e + lane, to = c + s.shift[i];
            if ((to < kCells - 1 ? to : kCells - 1) < border)
                w += static_cast<double>(a.cells[(r * a.parts + i) * kCells + c] & 0xffffffffffffull) / whole * eighths(-(s.below[i] + c));
        }
        if (border < kCells && p.n) {
            if (listed) {
                const uint32_t end = i + 1 < a.parts ? a.heads[r * a.parts + i + 1].at : p.n;
                for (uint32_t at = a.heads[r * a.parts + i].at + lane; at < end; at += 64) {
                    const uint64_t o = a.list[r * kGathered + at];
                    const float z = logit_of(o);
                    if (sc.cell(sc.y(z)) == border) w += weight(z, o);
                }
            } else {
                for (int64_t j0 = static_cast<int64_t>(i) * a.part; j0 < static_cast<int64_t>(i + 1) * a.part && j0 < a.vocab; j0 += kSeg) {
                    float z[kEach];
                    load_seg<FMT>(p_row, j0, a.vocab, z, -kInf);
#pragma unroll
                    for (int e = 0; e < kEach; ++e)
                        if (in_row(z[e]) && sc.cell(sc.y(z[e])) == border)
                            w += weight(z[e], order_of(z[e], static_cast<uint32_t>(j0) + entry_of<FMT>(lane, e)));
                }
            }
        }
        w = lanes_total(w);
        if (lane == 0) s.part_sum[i] = w;
    }
    __syncthreads();
    const double total = total_of(s.part_sum, a.parts);
    if (tid == 0) a.outs[r] = RowOut{total, least, from, all.m, -1};
    if (!a.tokens) return;
    const double target = target_of(a, r, total);
    const Place in = place_of(s.part_sum, a.parts, target);
    // the part's segments, a wave each
    const int64_t j0 = static_cast<int64_t>(in.at) * a.part + wave * kSeg;
    float z[kEach];
    double w = 0;
    if (wave * kSeg < a.part) {
        load_seg<FMT>(p_row, j0, a.vocab, z, -kInf);
#pragma unroll
        for (int e = 0; e < kEach; ++e) w += weight(z[e], order_of(z[e], static_cast<uint32_t>(j0) + entry_of<FMT>(lane, e)));
        w = lanes_total(w);
    }
    if (lane == 0) seg_sum[wave] = w;
    __syncthreads();
    const Place at = place_of(seg_sum, a.part / kSeg, target - in.before);
    if (wave == at.at) {
        const int32_t token = look_through<FMT>(
            [&](int e) { return weight(z[e], order_of(z[e], static_cast<uint32_t>(j0) + entry_of<FMT>(lane, e))); }, j0,
            target - in.before, at.before);
        if (lane == 0) a.tokens[r] = token;
    }
}

// The probabilities of a long row: a wave a segment.
template <int FMT>
__global__ __launch_bounds__(256) void sample_probs_kernel(SampleArgs a) {
    constexpr int kSize = FMT == WSL_OUT_F32 ? 4 : 2;
    const int64_t r = blockIdx.y;
    const int lane = static_cast<int>(threadIdx.x & 63);
    const int64_t j0 = (static_cast<int64_t>(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6))) * kSeg;
    if (j0 >= a.vocab) return;
    const RowOut o = a.outs[r];
    float *out = a.probs + r * a.ld_probs;
    float z[kEach];
    if (o.total > 0) load_seg<FMT>(static_cast<const char *>(a.logits) + r * a.ld * kSize, j0, a.vocab, z, -kInf);
    const Scale sc(how_of(a, r).c8, o.m);
    const double each = o.total > 0 ? 1 / o.total : 0;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        const uint32_t j = static_cast<uint32_t>(j0) + entry_of<FMT>(lane, e);
        float v = static_cast<int32_t>(j) == o.only ? 1.f : 0.f;
        if (o.total > 0 && in_row(z[e]) && order_of(z[e], j) >= o.from && sc.y(z[e]) >= o.least)
            v = static_cast<float>(sc.weight(z[e]) * each);
        if (j < a.vocab) out[j] = v;
    }
}

// Waves of a part: about eight parts a row and more, of up to 16384 entries.
int waves_of(int64_t vocab) { return vocab <= 65536 ? 4 : (vocab <= 131072 ? 8 : kMostWaves); }

template <int FMT>
void go(const SampleArgs &a, int64_t n_rows, hipStream_t s) {
    const unsigned rows = static_cast<unsigned>(n_rows);
    if (a.vocab <= kChunk) {
        hipLaunchKernelGGL(sample_short_kernel<FMT>, dim3(rows), dim3(kSmallWaves * 64), 0, s, a);
        return;
    }
    const dim3 grid(static_cast<unsigned>(a.parts), rows), block(static_cast<unsigned>(a.part / kSeg * 64));
    hipLaunchKernelGGL(sample_cells_kernel<FMT>, grid, block, 0, s, a);
    const bool some = a.how.d_top_k || a.how.d_top_p || a.how.d_min_p || a.how.top_k > 0 || a.how.top_p < 1 || a.how.min_p > 0;
    if (some) hipLaunchKernelGGL(sample_border_kernel<FMT>, grid, block, 0, s, a);
    hipLaunchKernelGGL(sample_pick_kernel<FMT>, dim3(rows), dim3(kMostWaves * 64), 0, s, a);
    if (a.probs)
        hipLaunchKernelGGL(sample_probs_kernel<FMT>, dim3(static_cast<unsigned>((a.vocab + 4 * kSeg - 1) / (4 * kSeg)), rows), dim3(256), 0, s, a);
}

struct Sizes {
    int64_t parts, part;
    size_t row;                                    // bytes of workspace
};
Sizes sizes_of(int64_t vocab) {
    Sizes z;
    z.part = static_cast<int64_t>(waves_of(vocab)) * kSeg;
    z.parts = (vocab + z.part - 1) / z.part;
    z.row = sizeof(RowOut) + sizeof(RowPlan) + static_cast<size_t>(z.parts) * (sizeof(PartHead) + kCells * sizeof(uint64_t)) + kGathered * sizeof(uint64_t);
    return z;
}

}  // namespace

size_t sample_ws_bytes(int64_t n_rows, int64_t vocab) {
    return vocab <= kChunk ? 0 : static_cast<size_t>(n_rows) * sizes_of(vocab).row;
}

int launch_sample(const void *logits, int zfmt, int64_t n_rows, int64_t vocab, int64_t ld, const wsl_sampling *how,
                  const float *u, int32_t *tokens, float *probs, int64_t ld_probs, void *ws, uint32_t *status, hipStream_t s) {
    SampleArgs a = {};
    a.logits = logits, a.u = u, a.tokens = tokens, a.probs = probs, a.status = status;
    a.vocab = vocab, a.ld = ld, a.ld_probs = ld_probs;
    if (how) a.how = *how;
    else a.how = {nullptr, nullptr, nullptr, nullptr, 1.f, 0, 1.f, 0.f};
    const Sizes z = sizes_of(vocab);
    a.parts = static_cast<int32_t>(z.parts), a.part = static_cast<int32_t>(z.part);
    a.cells = static_cast<uint64_t *>(ws);
    a.list = a.cells + n_rows * z.parts * kCells;
    a.plans = reinterpret_cast<RowPlan *>(a.list + n_rows * kGathered);
    a.heads = reinterpret_cast<PartHead *>(a.plans + n_rows);
    a.outs = reinterpret_cast<RowOut *>(a.heads + n_rows * z.parts);
    if (zfmt == WSL_OUT_F32) go<WSL_OUT_F32>(a, n_rows, s);
    else go<WSL_OUT_BF16>(a, n_rows, s);
    return WSL_OK;
}

}  // namespace wsl
