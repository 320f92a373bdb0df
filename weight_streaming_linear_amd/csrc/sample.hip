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
// narrowed by ranges of order(j), 256 at a time.  Weights come from 64-bit arithmetic; in a cell they are
// added up as whole numbers of 2^-32 of the cell's unit, which no order of adding changes.  The
// greatest entries weigh 1 exactly, so that rows of equal logits have exact sums.
// The token is then found as in verify_drafts: sums of segments in the order of the entries, and the
// segment that passes u * total looked through.
//
// A row up to kChunk entries is one workgroup's, in LDS.  Longer ones are cut into parts, a workgroup
// each, so that few rows fill the chip too, in up to four launches: cells of each part
// (relative to its own greatest entry, shifted by whole cells when they are put together); the entries
// of the border's cells as a list; the border and the token, one workgroup a row; the probabilities.
// The first two read the row, the second mostly from the caches.  A workgroup passes through most of this
// code once, so what bounds it besides the loads is how fast instructions come in: loops over LDS are
// kept rolled.
//
// Measured, top-k and top-p of each row's own: 64 rows of 151937 fp32 entries (38.9 MB, 7.6 us as a copy) 51 us: cells 16.1, border
// 15.1, pick 19.8; one row of 32000, 25: 6.4, 8.4 and 10.8; 40 bf16 rows of 32000 with their probabilities 41: 7.2, 9.5, 16.4 and 8.
// Rows so flat that a border's cells hold more than kHeld entries have no list: one workgroup goes through the row in memory for each
// step, and time grows with the row.  Top-p 0.9 of 64 rows of 151937 normal logits of spread 0.5: 530 us, of 2.5: 64; of equal ones 980;
// one row of 2^22 of spread 2.5: 14 ms.
#include "row_scan.h"

namespace wsl {
namespace {

constexpr int kCells = 256, kList = 256;
constexpr int kWaves = 8, kPartSegs = 16;      // waves of a workgroup, and segments of a part, at most
constexpr int kMostParts = 256, kFewParts = 16;
constexpr int kHeld = 8192;                    // orders that a workgroup holds: a short row, or a long one's list
// Entries of a short row, at most.  Against long rows' launches, in us (top-k 50 and top-p 0.9 in a graph, as all figures here): 8192
// entries, 1, 64 and 512 rows: 18, 18.4 and 35, the others 24, 26 and 43.5.
constexpr int kChunk = kHeld;
// Short rows of up to 4096 entries beyond which four waves take one, with a segment each, instead of eight.  (LDS has room for two rows
// a CU either way.)  Eight and four, 4000 entries: 14.5 and 17.3 for 1 row, 15.5 and 18.5 for 256, 28 and 20 for 512, 55 and 39 for 1024.
constexpr int64_t kManyRows = 256;
// Parts of all rows up to which a part is 8 segments and not 16.  8 and 16: 32000 entries, 1, 64, 128 and 256 rows (1024 parts):
// 24.7 and 29.6, 27 and 32, 31.3 and 33.7, 46.3 and 43.7; 65536, 64 rows (512) and 128: 31.5 and 33.8, 46 and 41; 131072, 1, 32
// (512) and 64: 27 and 30.3, 34.7 and 35.5, 49 and 43.8.
constexpr int64_t kFill = 512;
constexpr double kPartUnit = 4294967296.0;     // 2^32: whole numbers to a cell's unit; 2^14 entries of it fit 48 bits
constexpr float kInf = __builtin_huge_valf();

// What a part of a long row finds.
struct PartHead {
    float m;                                   // its greatest entry
    uint32_t first;                            // the first that is as great (greedy rows)
    uint32_t bad;
    uint32_t at;                               // where its entries begin in the row's list
};
// Counts and weights of 256 cells (or ranges).
struct Bins {
    double w[kCells];
    uint32_t count[kCells];
};
// Where a count or a sum is reached.
struct Border {
    int32_t bin;
    uint32_t before, in, all;                  // entries before the bin, in it, and of all bins
    double w_before, w_all;                    // weights before it, and of all
};
// Which cells' entries are needed one by one, and what is on.
struct Plan {
    int32_t k_on, p_on;
    int32_t one, lo, hi, min;                  // cells: of top-k, from .. to of top-p, of min-p; -1: none
    uint32_t n;                                // their entries
    uint32_t pad;
    Border k, p;                               // of top-k; of top-p where lo is hi
    __device__ __forceinline__ bool wants(int c) const { return c == one || (c >= lo && c <= hi) || c == min; }
};
struct RowPlan {
    Bins cells;
    Plan plan;
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
    uint64_t *list;                            // [rows][kHeld]
    RowPlan *plans;                            // [rows]
    RowOut *outs;                              // [rows]
    int32_t parts, part;                       // of a row, and entries of one
};

// A row's settings.
struct How {
    double c8;                                 // y = c8 * z
    double log_min_p;                          // 8 log2(min_p), or -infinity: off
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
    h.greedy = !(t > 0) || k == 1 || top_p <= 0 || min_p > 1;                  // (the greatest weight is 1)
    h.c8 = 11.541560327111707 / static_cast<double>(t > 0 ? t : 1.f);          // 8 log2(e) / T
    h.top_p = top_p < 1 ? top_p : 1.f;
    h.k = k <= 0 || k > a.vocab ? static_cast<uint32_t>(a.vocab) : static_cast<uint32_t>(k);
    h.log_min_p = min_p > 0 ? 8 * log2(static_cast<double>(min_p)) : -__builtin_huge_val();
    return h;
}

// 2^(v / 8): the Taylor series of exp(x) to the 12th power, |x| <= ln 2 / 2, right to 2^-50 (and 1 for a v that
// is nearly 0: logits that a high temperature makes equal weigh the same).
constexpr double kEighth = 0.08664339756999316;        // ln 2 / 8
__device__ __forceinline__ double power(double v) {
    v = v < -16000 ? -16000 : v;
    const double n = __builtin_rint(v * 0.125), x = (v - 8 * n) * kEighth;
    double r = __builtin_fma(1.0 / 479001600, x, 1.0 / 39916800);
    r = __builtin_fma(r, x, 1.0 / 3628800);
    r = __builtin_fma(r, x, 1.0 / 362880);
    r = __builtin_fma(r, x, 1.0 / 40320);
    r = __builtin_fma(r, x, 1.0 / 5040);
    r = __builtin_fma(r, x, 1.0 / 720);
    r = __builtin_fma(r, x, 1.0 / 120);
    r = __builtin_fma(r, x, 1.0 / 24);
    r = __builtin_fma(r, x, 1.0 / 6);
    r = __builtin_fma(r, x, 0.5);
    r = __builtin_fma(r, x, 1.0);
    return __builtin_ldexp(__builtin_fma(r, x, 1.0), static_cast<int>(n));
}
// The same of |f| <= 1/2 to the 5th power (2^-36), as a whole number of 2^-32: the last sum is above 2^52, whose
// fraction ends at 1, so its low bits are the number, rounded once.
__device__ __forceinline__ uint64_t whole_power(double f) {
    double k0 = kPartUnit + 4503599627370496.0, k1 = kEighth * kPartUnit, k2 = kEighth * k1 / 2, k3 = kEighth * k2 / 3, k4 = kEighth * k3 / 4,
           k5 = kEighth * k4 / 5;
    // (in scalar registers: a sum into its own constant would need that made anew each time)
    asm("" : "+s"(k0), "+s"(k1), "+s"(k2), "+s"(k3), "+s"(k4), "+s"(k5));
    double r = __builtin_fma(k5, f, k4);
    r = __builtin_fma(r, f, k3);
    r = __builtin_fma(r, f, k2);
    r = __builtin_fma(r, f, k1);
    return __builtin_bit_cast(uint64_t, __builtin_fma(r, f, k0)) & 0x3ffffffffull;
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
        return power(c8 * (static_cast<double>(z) - m));
    }
    // A weight in cell c as a whole number of 2^-32 of the cell's unit, and what the sum of such numbers weighs:
    // the greatest entry's own number weighs 1.
    __device__ __forceinline__ uint64_t whole(float z, int cell) const {
        const double v = y(z);
        if (cell < kCells - 1) return whole_power(v - __builtin_rint(v));
        return static_cast<uint64_t>(weight(z) * 2147483648.0 * kPartUnit);    // the last is open: 2^-31 and less
    }
    __device__ __forceinline__ double top() const { return static_cast<double>(whole_power(y(static_cast<float>(m)) - n_m)); }
    __device__ __forceinline__ double weight_of(double sum, int cell) const {
        return cell < kCells - 1 ? sum / top() * power(-cell) : sum / kPartUnit / 2147483648.0;
    }
};

// The first bin up to which there are `count` entries (by_count), or a sum of `sum`; where rounding lets
// none, the last that holds any.  By one wave: the others wait, for what all of them did would take as many times as long.
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
    Border o = {0, 0, 0, lane_value(at_c, 63), 0, lane_value(up_w, 63)};
    if (!some) return o;
    const int l = hits ? __builtin_ctzll(hits) : 63 - __builtin_clzll(some);
    o.bin = l * kMine + __builtin_amdgcn_readlane(hits ? hit : last, l);
    o.before = __builtin_amdgcn_readlane(static_cast<int>(hits ? hit_c : last_c), l);
    o.in = __builtin_amdgcn_readlane(static_cast<int>(hits ? hit_in : last_in), l);
    o.w_before = lane_value(hits ? hit_w : last_w, l);
    return o;
}

// What one wave found, for all: the same in every lane.
__device__ __forceinline__ uint32_t same(uint32_t v) { return static_cast<uint32_t>(__builtin_amdgcn_readfirstlane(static_cast<int>(v))); }
__device__ __forceinline__ double same(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    return __builtin_bit_cast(double, static_cast<uint64_t>(same(static_cast<uint32_t>(b >> 32))) << 32 | same(static_cast<uint32_t>(b)));
}
__device__ __forceinline__ Border same(const Border &b) {
    return Border{static_cast<int32_t>(same(static_cast<uint32_t>(b.bin))), same(b.before), same(b.in), same(b.all), same(b.w_before), same(b.w_all)};
}

struct Shared {
    uint64_t held[kHeld];                          // orders; 0: none
    Bins cells, bins;
    uint64_t sum[kCells];
    uint64_t list[kList], sorted[kList];
    uint32_t rank[kList];
    Border border;
    uint64_t from;
    double w_kept;
    uint64_t least[kWaves], most[kWaves];
    float top[kWaves];
    uint32_t n, bad;
};

// What keep_from goes over, by all waves of a workgroup: orders in LDS, or, where they have no room there, a row
// itself, read again each time.
template <int FMT>
struct Entries {
    const uint64_t *held;
    uint32_t n;
    const char *row;
    uint32_t vocab;                                // 0: held
    template <typename Fn>
    __device__ __forceinline__ void each(Fn fn) const {
        const uint32_t all = vocab ? vocab : n;
#pragma unroll 1
        for (uint32_t i0 = 0; i0 < all; i0 += blockDim.x) {
            const uint32_t i = i0 + threadIdx.x;
            uint64_t o = 0;
            if (vocab) {
                const float z = i < vocab ? load_one<FMT>(row, i) : -kInf;
                o = in_row(z) ? order_of(z, i) : 0;
            } else if (i < n) {
                o = held[i];
            }
            fn(o);
        }
    }
};

// The least order that is kept, of the first `count` entries or of the first whose sum reaches `sum`; b: the
// border among the cells; w_kept: the weight of what is kept.
template <int FMT>
__device__ __forceinline__ uint64_t keep_from(const Entries<FMT> &row, Shared &s, const Scale &sc, Border b, bool by_count,
                                              uint32_t count, double sum, double &w_kept) {
    const uint32_t tid = threadIdx.x;
    const int lane = static_cast<int>(tid & 63), wave = static_cast<int>(tid >> 6);
    const int cell = b.bin;
    uint64_t lo = 1, hi = ~0ull;
    const auto inside = [&](uint64_t o) {
        return o >= lo && o <= hi && sc.cell(sc.y(logit_of(o))) == cell;
    };
    count -= b.before, sum -= b.w_before;
    w_kept = b.w_before;
    while (b.in > kList) {
        uint64_t least = ~0ull, most = 0;
        row.each([&](uint64_t o) {
            if (inside(o)) least = o < least ? o : least, most = o > most ? o : most;
        });
#pragma unroll
        for (int off = 32; off >= 1; off >>= 1) {
            const uint64_t l = __shfl_xor(static_cast<unsigned long long>(least), off, 64);
            const uint64_t m = __shfl_xor(static_cast<unsigned long long>(most), off, 64);
            least = l < least ? l : least, most = m > most ? m : most;
        }
        __syncthreads();                           // the round before has been read
        if (lane == 0) s.least[wave] = least, s.most[wave] = most;
        if (tid < kCells) s.sum[tid] = 0, s.bins.count[tid] = 0;
        __syncthreads();
        for (int w = 0; w < static_cast<int>(blockDim.x >> 6); ++w) {
            least = s.least[w] < least ? s.least[w] : least;
            most = s.most[w] > most ? s.most[w] : most;
        }
        lo = least, hi = most;
        const int bits = 64 - __builtin_clzll(hi - lo | 1), shift = bits > 8 ? bits - 8 : 0;
        row.each([&](uint64_t o) {
            const float z = logit_of(o);
            bool in = inside(o);
            const int at = in ? static_cast<int>((hi - o) >> shift) : -1;
            const uint64_t v = in ? sc.whole(z, cell) : 0;
            // equal logits would queue for one bin: the first lane adds those of its like at once
            for (uint64_t left = __ballot(in); left;) {
                const int first = __builtin_ctzll(left);
                const uint64_t like = __ballot(in && at == __builtin_amdgcn_readlane(at, first) &&
                                               z == __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, z), first)));
                const uint32_t n = static_cast<uint32_t>(__popcll(like));
                if (n < 8) break;
                if (lane == first) {
                    atomicAdd(&s.bins.count[at], n);
                    atomicAdd(reinterpret_cast<unsigned long long *>(&s.sum[at]), static_cast<unsigned long long>(n * v));
                }
                in = in && !(like >> lane & 1u);
                left &= ~like;
            }
            if (in) {
                atomicAdd(&s.bins.count[at], 1u);
                atomicAdd(reinterpret_cast<unsigned long long *>(&s.sum[at]), static_cast<unsigned long long>(v));
            }
        });
        __syncthreads();
        if (tid < kCells) s.bins.w[tid] = sc.weight_of(static_cast<double>(s.sum[tid]), cell);
        __syncthreads();
        if (wave == 0) {
            b = border_of(s.bins, by_count, count, sum);
            if (lane == 0) s.border = b;
        }
        __syncthreads();
        b = same(s.border);
        count -= b.before, sum -= b.w_before;
        w_kept += b.w_before;
        hi -= static_cast<uint64_t>(b.bin) << shift;
        const uint64_t width = (1ull << shift) - 1;
        lo = hi - lo > width ? hi - width : lo;
    }
    if (tid == 0) s.n = 0;
    if (tid < kList) s.rank[tid] = 0;
    __syncthreads();
    row.each([&](uint64_t o) {
        if (inside(o)) {
            const uint32_t at = atomicAdd(&s.n, 1u);
            if (at < kList) s.list[at] = o;
        }
    });
    __syncthreads();
    const uint32_t n = s.n < kList ? s.n : kList;                      // b.in
    if (n > 64) {
        // an entry's place: as many threads as there are for each, a part of the list each
        const uint32_t shares = blockDim.x / kList, entry = tid % kList, share = tid / kList;
        if (entry < n) {
            const uint64_t mine = s.list[entry];
            uint32_t rank = 0;
#pragma unroll 4
            for (uint32_t i = n * share / shares; i < n * (share + 1) / shares; ++i) rank += s.list[i] > mine ? 1u : 0u;
            atomicAdd(&s.rank[entry], rank);
        }
        __syncthreads();
        if (tid < n) s.sorted[s.rank[tid]] = s.list[tid];
        __syncthreads();
    }
    if (wave == 0) {
        uint64_t from = ~0ull;                     // (a border lies in a cell that holds something)
        double w = 0;
        if (n <= 64) {                             // a lane an entry, brought into their order
            const bool in = static_cast<uint32_t>(lane) < n;
            const uint64_t mine = in ? s.list[lane] : 0;
            uint32_t place = 0;
#pragma unroll 4
            for (uint32_t i = 0; i < n; ++i) place += s.list[i] > mine ? 1u : 0u;
            const int to = static_cast<int>(in ? place : lane) * 4;
            const auto push = [&](uint64_t v) {
                const uint32_t l = static_cast<uint32_t>(__builtin_amdgcn_ds_permute(to, static_cast<int>(v)));
                const uint32_t h = static_cast<uint32_t>(__builtin_amdgcn_ds_permute(to, static_cast<int>(v >> 32)));
                return static_cast<uint64_t>(h) << 32 | l;
            };
            const uint64_t sorted = push(mine);
            const double at = lanes_before(in ? sc.weight(logit_of(sorted)) : 0.0);
            const uint64_t hits = __ballot(in && (by_count ? static_cast<uint32_t>(lane) + 1 >= count : at >= sum));
            if (n) {
                const int l = hits ? __builtin_ctzll(hits) : static_cast<int>(n) - 1;
                w = lane_value(at, l);
                from = static_cast<uint64_t>(lane_value(static_cast<uint32_t>(sorted >> 32), l)) << 32 |
                       lane_value(static_cast<uint32_t>(sorted), l);
            }
        } else {                                   // successive entries of a lane
            constexpr uint32_t kMine = kList / 64;
            double ws = 0;
#pragma unroll 1
            for (uint32_t i = 0; i < kMine; ++i) {
                const uint32_t at = lane * kMine + i;
                ws += at < n ? sc.weight(logit_of(s.sorted[at])) : 0;
            }
            // the lane, then which of its entries
            const double up = lanes_before(ws);
            const uint32_t end = (lane + 1) * kMine < n ? (lane + 1) * kMine : n;
            const uint64_t hits = __ballot(lane * kMine < n && (by_count ? end >= count : up >= sum));
            const uint32_t l = hits ? static_cast<uint32_t>(__builtin_ctzll(hits)) : (n - 1) / kMine;
            w = lane_value(up, l) - lane_value(ws, l);
            uint32_t at = l * kMine;
#pragma unroll 1
            for (;; ++at) {
                w += sc.weight(logit_of(s.sorted[at]));
                if (at + 1 >= n || at + 1 >= (l + 1) * kMine || (by_count ? at + 1 >= count : w >= sum)) break;
            }
            from = s.sorted[at];
        }
        if (lane == 0) s.from = from, s.w_kept = w;
    }
    __syncthreads();                               // the list and the bins may be used again
    w_kept += same(s.w_kept);
    const uint64_t from = s.from;
    return static_cast<uint64_t>(same(static_cast<uint32_t>(from >> 32))) << 32 | same(static_cast<uint32_t>(from));
}

// In the order of n sums (LDS): the first that passes u times their total (share; else u itself), or the last
// that is not zero, and what lies before it.  Every wave comes to the same.
struct Place {
    int at;
    double before, target, total;
};
__device__ __forceinline__ Place place_of(const double *sums, int n, bool share, double u) {
    const int lane = static_cast<int>(threadIdx.x & 63), each = (n + 63) / 64;
    const int c0 = each * lane < n ? each * lane : n, c1 = c0 + each < n ? c0 + each : n;
    double mine = 0;
    for (int c = c0; c < c1; ++c) mine += sums[c];
    const double up = lanes_before(mine);
    Place o = {0, 0.0, u, lane_value(up, 63)};
    if (share) {                                   // NaN is passed by none: the last one, as for u >= 1
        o.target = u * o.total;
        if (o.target < 0) o.target = 0;
    }
    double at = up - mine;
    int hit = -1, last = -1;
    double hit_at = 0, last_at = 0;
    for (int c = c0; c < c1; ++c) {
        const double w = sums[c];
        if (w > 0) last = c, last_at = at;
        if (hit < 0 && w > 0 && at + w > o.target) hit = c, hit_at = at;
        at += w;
    }
    const uint64_t hits = __ballot(hit >= 0), some = __ballot(last >= 0);
    if (!some) return o;
    const int l = hits ? __builtin_ctzll(hits) : 63 - __builtin_clzll(some);
    o.at = __builtin_amdgcn_readlane(hits ? hit : last, l);
    o.before = lane_value(hits ? hit_at : last_at, l);
    return o;
}

// A segment by one wave, lane l taking its entries kEach * l and on: the weights up to each lane's last, and the
// lane's own.  weight(i) is that of entry i.
struct Lanes {
    double up, mine;
};
template <typename Weight>
__device__ __forceinline__ Lanes lanes_of(Weight weight) {
    const int lane = static_cast<int>(threadIdx.x & 63);
    double w = 0;
#pragma unroll 2
    for (int i = 0; i < kEach; ++i) w += weight(lane * kEach + i);
    return Lanes{lanes_before(w), w};
}
// The first of its entries whose running sum passes the target, or the last with a weight.
template <typename Weight>
__device__ __forceinline__ int entry_in(Weight weight, const Lanes &s, double target, double run) {
    const int lane = static_cast<int>(threadIdx.x & 63);
    uint64_t hits = __ballot(s.mine > 0 && run + s.up > target), some = __ballot(s.mine > 0);
    if (!some) return -1;
    const int l = hits ? __builtin_ctzll(hits) : 63 - __builtin_clzll(some);
    run += lane_value(s.up, l) - lane_value(s.mine, l);
    const double w = lane < kEach ? weight(l * kEach + lane) : 0.0, up = lanes_before(w);
    hits = __ballot(w > 0 && run + up > target), some = __ballot(w > 0);
    return l * kEach + (hits ? __builtin_ctzll(hits) : 63 - __builtin_clzll(some));
}

// ------------------------------------------------------------------ short rows
template <int FMT>
__global__ __launch_bounds__(kWaves * 64) void sample_short_kernel(SampleArgs a) {
    __shared__ Shared s;
    __shared__ double seg_sum[kWaves];
    constexpr int kSize = FMT == WSL_OUT_F32 ? 4 : 2;
    const int64_t r = blockIdx.x;
    const uint32_t tid = threadIdx.x, vocab = static_cast<uint32_t>(a.vocab);
    const int lane = static_cast<int>(tid & 63), wave = __builtin_amdgcn_readfirstlane(static_cast<int>(tid >> 6));
    const int waves = static_cast<int>(blockDim.x >> 6);       // a segment each
    float z[kEach];
    load_seg<FMT>(static_cast<const char *>(a.logits) + r * a.ld * kSize, wave * kSeg, a.vocab, z, -kInf);
    const float u = a.tokens ? a.u[r] : 0.f;
    const How h = how_of(a, r);

    // the greatest entry
    float m = -kInf;
    bool bad = false;
#pragma unroll
    for (int e = 0; e < kEach; ++e) {
        bad |= !(z[e] < kInf), m = z[e] > m ? z[e] : m;
        const uint32_t j = wave * kSeg + entry_of<FMT>(lane, e);
        s.held[j] = in_row(z[e]) ? order_of(z[e], j) : 0;
    }
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
        const float o = __shfl_xor(m, off, 64);
        m = o > m ? o : m;
    }
    const bool any_bad = __ballot(bad) != 0;
    if (tid == 0) s.bad = 0, s.n = ~0u;
    for (uint32_t i = tid; i < kCells; i += blockDim.x) s.sum[i] = 0, s.cells.count[i] = 0;
    __syncthreads();
    if (lane == 0) {
        s.top[wave] = m;
        if (any_bad) atomicOr(&s.bad, 1u);
    }
    __syncthreads();
    for (int w = 0; w < waves; ++w) m = s.top[w] > m ? s.top[w] : m;
    if (s.bad || !in_row(m)) {
        if (a.probs)
            for (uint32_t j = tid; j < vocab; j += blockDim.x) a.probs[r * a.ld_probs + j] = 0.f;
        if (tid == 0) {
            if (a.tokens) a.tokens[r] = -1;
            if (a.status) atomicOr(a.status, WSL_STATUS_NONFINITE);
        }
        return;
    }
    if (h.greedy) {
        uint32_t at = ~0u;
#pragma unroll
        for (int e = kEach - 1; e >= 0; --e) at = z[e] == m ? static_cast<uint32_t>(wave * kSeg + entry_of<FMT>(lane, e)) : at;
        if (at != ~0u) atomicMin(&s.n, at);
        __syncthreads();
        at = s.n;
        if (a.probs)
            for (uint32_t j = tid; j < vocab; j += blockDim.x) a.probs[r * a.ld_probs + j] = j == at ? 1.f : 0.f;
        if (a.tokens && tid == 0) a.tokens[r] = static_cast<int32_t>(at);
        return;
    }
    const Scale sc(h.c8, m);
    const Entries<FMT> row = {s.held, vocab, nullptr, 0};
    uint64_t from = 0;
    if (h.k < vocab || h.top_p < 1) {
        row.each([&](uint64_t o) {
            if (o) {
                const float x = logit_of(o);
                const int c = sc.cell(sc.y(x));
                atomicAdd(&s.cells.count[c], 1u);
                atomicAdd(reinterpret_cast<unsigned long long *>(&s.sum[c]), static_cast<unsigned long long>(sc.whole(x, c)));
            }
        });
        __syncthreads();
        for (uint32_t i = tid; i < kCells; i += blockDim.x) s.cells.w[i] = sc.weight_of(static_cast<double>(s.sum[i]), i);
        __syncthreads();
        // top-k, then top-p of what it leaves
        double w_kept = 0;
#pragma unroll 1
        for (int by_count = 1; by_count >= (h.top_p < 1 ? 0 : 1); --by_count) {
            const double sum = by_count ? 0 : static_cast<double>(h.top_p) * w_kept;
            if (wave == 0) {
                const Border found = border_of(s.cells, by_count != 0, h.k, sum);
                if (lane == 0) s.border = found;
            }
            __syncthreads();
            const Border b = same(s.border);
            if (by_count) w_kept = b.w_all;
            if (by_count && h.k >= b.all) {
                __syncthreads();                   // all have read it
                continue;
            }
            const uint64_t o = keep_from(row, s, sc, b, by_count != 0, h.k, sum, w_kept);
            from = o > from ? o : from;
        }
    }
    const double least = sc.y(m) + h.log_min_p;
    const auto weight = [&](uint64_t o) {
        const float x = logit_of(o);
        return o && o >= from && sc.y(x) >= least ? sc.weight(x) : 0.0;
    };
    const auto mine = [&](int i) { return weight(s.held[wave * kSeg + i]); };
    const Lanes lanes = lanes_of(mine);
    if (lane == 63) seg_sum[wave] = lanes.up;
    __syncthreads();
    const Place at = place_of(seg_sum, waves, true, u);
    if (a.tokens && at.at == wave) {
        const int token = entry_in(mine, lanes, at.target, at.before);
        if (lane == 0) a.tokens[r] = wave * kSeg + token;
    }
    if (a.probs) {
        float *out = a.probs + r * a.ld_probs;
#pragma unroll 1
        for (uint32_t j = tid; j < vocab; j += blockDim.x) out[j] = static_cast<float>(weight(s.held[j]) / at.total);
    }
}

// ------------------------------------------------------------------ long rows
// Cells of one part: blockIdx (part, row), a wave SEGS segments of it.  Bound by the loads (10.5 us of 64 rows' 17) and
// the 64-bit arithmetic and atomics in LDS behind them, about 16 instructions an entry (an exponential in 32 bits would
// take as many and leave 2^-22 of a weight).
template <int FMT, int SEGS>
__global__ __launch_bounds__(kWaves * 64) void sample_cells_kernel(SampleArgs a) {
    __shared__ uint64_t cells[kCells];
    __shared__ float top[kWaves];
    __shared__ uint32_t first, bad;
    constexpr int kSize = FMT == WSL_OUT_F32 ? 4 : 2;
    const int64_t r = blockIdx.y;
    const uint32_t tid = threadIdx.x;
    const int lane = static_cast<int>(tid & 63), wave = __builtin_amdgcn_readfirstlane(static_cast<int>(tid >> 6));
    const int waves = static_cast<int>(blockDim.x >> 6);
    const int64_t j0 = static_cast<int64_t>(blockIdx.x) * a.part + wave * SEGS * kSeg;
    float z[SEGS][kEach];
#pragma unroll
    for (int i = 0; i < SEGS; ++i) load_seg<FMT>(static_cast<const char *>(a.logits) + r * a.ld * kSize, j0 + i * kSeg, a.vocab, z[i], -kInf);
    const How h = how_of(a, r);
    if (tid == 0) first = ~0u, bad = 0;
    if (tid < kCells) cells[tid] = 0;
    float m = -kInf;
    bool mine_bad = false;
#pragma unroll
    for (int i = 0; i < SEGS; ++i)
#pragma unroll
        for (int e = 0; e < kEach; ++e) mine_bad |= !(z[i][e] < kInf), m = z[i][e] > m ? z[i][e] : m;
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
        for (int i = SEGS - 1; i >= 0; --i)
#pragma unroll
            for (int e = kEach - 1; e >= 0; --e)
                at = z[i][e] == m ? static_cast<uint32_t>(j0) + i * kSeg + entry_of<FMT>(lane, e) : at;
        if (at != ~0u) atomicMin(&first, at);
    } else if (in_row(m)) {
        const double n_m = __builtin_rint(h.c8 * static_cast<double>(m));
        // the last cell's entries count by how far they are behind it: weights of less than 2^-31, for which an
        // exponential of 32 bits does (2^-23 of them; of 2^22 entries together 2^-33), added up in 64 by their lane
        double behind = 0;
        uint32_t n_behind = 0;
#pragma unroll
        for (int i = 0; i < SEGS; ++i)
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const double y = h.c8 * static_cast<double>(z[i][e]), n = __builtin_rint(y), d = n_m - n;
                if (d < kCells - 1) {
                    const uint64_t v = whole_power(y - n) + (1ull << 48);
                    atomicAdd(reinterpret_cast<unsigned long long *>(&cells[static_cast<int>(d)]), static_cast<unsigned long long>(v));
                } else if (in_row(z[i][e])) {
                    behind += static_cast<double>(__builtin_amdgcn_exp2f(static_cast<float>(y - (n_m - (kCells - 1))) * 0.125f));
                    ++n_behind;
                }
            }
        const double sum = lanes_total(behind);
        n_behind = lane_value(lanes_before(n_behind), 63);
        if (lane == 0 && n_behind)
            atomicAdd(reinterpret_cast<unsigned long long *>(&cells[kCells - 1]),
                      static_cast<unsigned long long>(static_cast<uint64_t>(sum * kPartUnit) + (static_cast<uint64_t>(n_behind) << 48)));
    }
    __syncthreads();
    const int64_t at = r * a.parts + blockIdx.x;
    if (tid < kCells && !h.greedy) a.cells[at * kCells + tid] = cells[tid];
    if (tid == 0) a.heads[at] = PartHead{m, first, bad, 0};
}

// A long row put together from its parts.
template <int PARTS, int WAVES>
struct LongShared {
    float m[PARTS];
    double below[PARTS];                           // cells that a part's lie below the row's
    int32_t shift[PARTS];                          // the same, 255 at most
    double part_sum[PARTS];
    uint32_t part_count[PARTS];
    double w[WAVES / 4][kCells];
    uint32_t count[WAVES / 4][kCells];
    double rest[WAVES];
    uint32_t rest_count[WAVES];
    uint32_t bad, first;
};
template <bool FEW>
constexpr int kPartsOf = FEW ? kFewParts : kMostParts;
struct Whole {
    float m;
    uint32_t bad, first;
};

// p: a thread's part's head.
template <typename S>
__device__ __forceinline__ Whole heads_of(const SampleArgs &a, const PartHead &p, double c8, S &s) {
    const uint32_t tid = threadIdx.x;
    const bool mine = tid < static_cast<uint32_t>(a.parts);
    if (tid == 0) s.bad = 0, s.first = ~0u;
    if (mine) s.m[tid] = p.m;
    __syncthreads();
    Whole o;
    o.m = -kInf;
    for (int i = 0; i < a.parts; ++i) o.m = s.m[i] > o.m ? s.m[i] : o.m;
    if (mine) {
        if (p.bad) atomicOr(&s.bad, 1u);
        if (p.m == o.m && p.first != ~0u) atomicMin(&s.first, p.first);
        const double d = __builtin_rint(c8 * static_cast<double>(o.m)) - __builtin_rint(c8 * static_cast<double>(p.m));
        s.below[tid] = d < 100000 ? d : 100000;    // (a part of -infinities, and infinite temperature: NaN)
        s.shift[tid] = static_cast<int>(d < kCells - 1 ? d : kCells - 1);
    }
    __syncthreads();
    o.bad = s.bad, o.first = s.first;
    return o;
}

// The cells of a row's parts: of up to kFewParts in LDS, asked for before anything is known (take, put), or where
// they lie.
template <bool FEW>
struct PartCells;
template <>
struct PartCells<true> {
    static constexpr int kThreads = kWaves * 64, kMine = kFewParts * kCells / kThreads;
    uint64_t raw[kMine];
    __device__ __forceinline__ void take(const uint64_t *from, int parts) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const uint32_t at = i * kThreads + threadIdx.x;
            raw[i] = at < static_cast<uint32_t>(parts) * kCells ? from[at] : 0;
        }
    }
    __device__ __forceinline__ void put(uint64_t *lds, int parts) const {
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
            const uint32_t at = i * kThreads + threadIdx.x;
            if (at < static_cast<uint32_t>(parts) * kCells) lds[at] = raw[i];
        }
    }
    static __device__ __forceinline__ const uint64_t *of(const uint64_t *, const uint64_t *lds) { return lds; }
};
template <>
struct PartCells<false> {
    __device__ __forceinline__ void take(const uint64_t *, int) {}
    __device__ __forceinline__ void put(uint64_t *, int) const {}
    static __device__ __forceinline__ const uint64_t *of(const uint64_t *from, const uint64_t *) { return from; }
};

// The row's cells from its parts': groups of 256 threads take every so many parts, a thread a cell of the
// row, and of the part where that lies in or behind the last.
template <typename S>
__device__ __forceinline__ void put_together(int parts, const uint64_t *mine, const Scale &sc, S &s, Bins &cells) {
    const uint32_t tid = threadIdx.x, cell = tid & (kCells - 1), group = tid / kCells, groups = blockDim.x / kCells;
    const int lane = static_cast<int>(tid & 63), wave = static_cast<int>(tid >> 6);
    uint64_t sum = 0;
    double rest = 0;
    uint32_t count = 0, rest_count = 0;
    const double top = sc.top(), one = 1 / top;
    for (int i = group; i < parts; i += groups) {
        const int shift = s.shift[i], from = static_cast<int>(cell) - shift;
        const bool here = from >= 0 && cell < kCells - 1, behind = static_cast<int>(cell) + shift >= kCells - 1;
        const uint64_t v = here ? mine[i * kCells + from] : 0, u = behind ? mine[i * kCells + cell] : 0;
        sum += v & 0xffffffffffffull;
        count += static_cast<uint32_t>(v >> 48);
        if (__ballot(u != 0)) {
            rest += static_cast<double>(u & 0xffffffffffffull) * one * power(-(s.below[i] + cell));
            rest_count += static_cast<uint32_t>(u >> 48);
        }
    }
    rest = lanes_total(rest);
    rest_count = lane_value(lanes_before(rest_count), 63);
    s.w[group][cell] = static_cast<double>(sum), s.count[group][cell] = count;
    if (lane == 0) s.rest[wave] = rest, s.rest_count[wave] = rest_count;
    __syncthreads();
    if (tid < kCells) {
        double w = 0;
        count = 0;
        for (uint32_t g = 0; g < groups; ++g) w += s.w[g][cell], count += s.count[g][cell];
        w = w / top * power(-static_cast<double>(cell));
        if (cell == kCells - 1)
            for (uint32_t i = 0; i < groups * 4; ++i) w += s.rest[i], count += s.rest_count[i];
        cells.w[cell] = w, cells.count[cell] = count;
    }
    __syncthreads();
}

__device__ __forceinline__ Plan plan_of(const Bins &cells, const Scale &sc, const How &h, double least) {
    Plan p;
    p.p_on = h.top_p < 1;
    p.one = p.min = p.lo = -1, p.hi = -2, p.n = 0, p.pad = 0;
    // the border of top-k, and of the least and the most that top-p may keep
    double sum = 0, most = 0;
#pragma unroll 1
    for (int step = 0; step < 3; ++step) {
        const Border b = border_of(cells, step == 0, h.k, sum);
        if (step == 0) {
            p.k = p.p = b;
            p.k_on = h.k < b.all;
            double least_w = b.w_all, most_w = b.w_all;
            if (p.k_on) {
                p.one = b.bin;
                // between the lightest and the heaviest that (k - before) entries of the cell can be: 2^(1/16) either
                // way of its middle, which is as far from the greatest's, and a little
                const double some = static_cast<double>(h.k - b.before), unit = power(-p.one);
                least_w = b.w_before + (p.one < kCells - 1 ? 0.916 * unit * some : 0.0);
                most_w = b.w_before + 1.091 * unit * some;
            }
            if (!p.p_on) break;
            sum = static_cast<double>(h.top_p) * least_w * (1 - 1e-6);
            most = static_cast<double>(h.top_p) * most_w * (1 + 1e-6);
        } else if (step == 1) {
            p.p = b;
            p.lo = p.hi = b.bin;
            if (most < b.w_before + cells.w[b.bin]) break;
            sum = most;
        } else {
            p.hi = b.bin;
        }
    }
    if (least > -__builtin_huge_val()) {
        const double d = sc.n_m - __builtin_rint(least);
        const int c = static_cast<int>(d < kCells - 1 ? d : kCells - 1);
        const int first = p.k_on ? (p.p_on && p.lo < p.one ? p.lo : p.one) : (p.p_on ? p.lo : kCells);
        if (c < first) p.k_on = p.p_on = 0, p.one = p.lo = -1, p.hi = -2, p.min = c;           // it alone decides
        else if (c <= (p.p_on ? p.hi : first)) p.min = c;
    }
    for (int i = static_cast<int>(threadIdx.x & 63); i < kCells; i += 64) p.n += p.wants(i) ? cells.count[i] : 0u;
    p.n = lane_value(lanes_before(p.n), 63);
    return p;
}

// Entries of each part that the plan wants; a wave a part.
template <typename S>
__device__ __forceinline__ void count_parts(int parts, const uint64_t *cells, const Plan &p, S &s) {
    const int lane = static_cast<int>(threadIdx.x & 63), wave = static_cast<int>(threadIdx.x >> 6);
    const int waves = static_cast<int>(blockDim.x >> 6);
    for (int i = wave; i < parts; i += waves) {
        uint32_t n = 0;
#pragma unroll
        for (int e = 0; e < kCells; e += 64) {
            const int c = e + lane + s.shift[i];
            if (p.wants(c < kCells - 1 ? c : kCells - 1)) n += static_cast<uint32_t>(cells[i * kCells + e + lane] >> 48);
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
template <int FMT, int SEGS, bool FEW>
__global__ __launch_bounds__(kWaves * 64) void sample_border_kernel(SampleArgs a) {
    __shared__ LongShared<kPartsOf<FEW>, kWaves> s;
    __shared__ uint64_t held[FEW ? kFewParts * kCells : 1];
    __shared__ Bins cells;
    __shared__ uint32_t found[kWaves];
    constexpr int kSize = FMT == WSL_OUT_F32 ? 4 : 2;
    const int64_t r = blockIdx.y;
    const int lane = static_cast<int>(threadIdx.x & 63), wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    PartCells<FEW> raw;
    PartHead head = {-kInf, ~0u, 0, 0};
    if (threadIdx.x < static_cast<uint32_t>(a.parts)) head = a.heads[r * a.parts + threadIdx.x];
    raw.take(a.cells + r * a.parts * kCells, a.parts);
    const How h = how_of(a, r);
    if (h.greedy || !filters(a, h)) return;
    const int64_t j0 = static_cast<int64_t>(blockIdx.x) * a.part + wave * SEGS * kSeg;
    float z[SEGS][kEach];
#pragma unroll
    for (int i = 0; i < SEGS; ++i) load_seg<FMT>(static_cast<const char *>(a.logits) + r * a.ld * kSize, j0 + i * kSeg, a.vocab, z[i], -kInf);
    raw.put(held, a.parts);
    const Whole all = heads_of(a, head, h.c8, s);
    if (all.bad || !in_row(all.m)) return;
    const Scale sc(h.c8, all.m);
    const uint64_t *mine_cells = PartCells<FEW>::of(a.cells + r * a.parts * kCells, held);
    put_together(a.parts, mine_cells, sc, s, cells);
    __shared__ Plan plan;
    if (wave == 0) {
        const Plan o = plan_of(cells, sc, h, sc.y(all.m) + h.log_min_p);
        if (lane == 0) plan = o;
    }
    __syncthreads();
    Plan p = plan;
    p.one = static_cast<int32_t>(same(static_cast<uint32_t>(p.one))), p.lo = static_cast<int32_t>(same(static_cast<uint32_t>(p.lo)));
    p.hi = static_cast<int32_t>(same(static_cast<uint32_t>(p.hi))), p.min = static_cast<int32_t>(same(static_cast<uint32_t>(p.min)));
    p.n = same(p.n);
    const bool fits = p.n > 0 && p.n <= kHeld;
    if (fits) count_parts(a.parts, mine_cells, p, s);
    if (blockIdx.x == 0) {                         // for the next launch
        RowPlan &out = a.plans[r];
        for (uint32_t i = threadIdx.x; i < kCells; i += blockDim.x) out.cells.w[i] = cells.w[i], out.cells.count[i] = cells.count[i];
        if (threadIdx.x == 0) out.plan = plan;
        if (fits && threadIdx.x < static_cast<uint32_t>(a.parts)) {
            uint32_t at = 0;
            for (uint32_t i = 0; i < threadIdx.x; ++i) at += s.part_count[i];
            a.heads[r * a.parts + threadIdx.x].at = at;
        }
    }
    if (!fits || s.part_count[blockIdx.x] == 0) return;
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
    for (int i = 0; i < SEGS; ++i)
#pragma unroll
        for (int e = 0; e < kEach; ++e) mine |= z[i][e] >= low && z[i][e] <= high ? 1u << (i * kEach + e) : 0u;
    // the few that are left, from the caches again: which are wanted, and then where they go
    const char *row = static_cast<const char *>(a.logits) + r * a.ld * kSize;
    const auto index = [&](uint32_t bit) {
        return static_cast<uint32_t>(j0) + bit / kEach * kSeg + entry_of<FMT>(lane, static_cast<int>(bit % kEach));
    };
#pragma unroll 1
    for (uint32_t left = mine; left; left &= left - 1) {
        const uint32_t bit = static_cast<uint32_t>(__builtin_ctz(left)), j = index(bit);
        const float x = j < a.vocab ? load_one<FMT>(row, j) : -kInf;
        if (!(in_row(x) && p.wants(sc.cell(sc.y(x))))) mine &= ~(1u << bit);
    }
    n = static_cast<uint32_t>(__builtin_popcount(mine));
    const uint32_t up = lanes_before(n);
    if (lane == 63) found[wave] = up;
    __syncthreads();
    uint32_t at = up - n;
    for (uint32_t i = 0; i < blockIdx.x; ++i) at += s.part_count[i];
    for (int w = 0; w < wave; ++w) at += found[w];
    uint64_t *list = a.list + r * kHeld;
#pragma unroll 1
    for (uint32_t left = mine; left; left &= left - 1) {
        const uint32_t j = index(static_cast<uint32_t>(__builtin_ctz(left)));
        if (at < kHeld) list[at] = order_of(load_one<FMT>(row, j), j);
        ++at;
    }
}

// The border and the token of a row.
template <int FMT, bool FEW>
__global__ __launch_bounds__(kWaves * 64) void sample_pick_kernel(SampleArgs a) {
    __shared__ LongShared<kPartsOf<FEW>, kWaves> s;
    __shared__ uint64_t held[FEW ? kFewParts * kCells : 1];
    __shared__ Shared t;
    __shared__ double seg_sum[kPartSegs];
    constexpr int kSize = FMT == WSL_OUT_F32 ? 4 : 2;
    const int64_t r = blockIdx.x;
    const uint32_t tid = threadIdx.x;
    const int lane = static_cast<int>(tid & 63), wave = __builtin_amdgcn_readfirstlane(static_cast<int>(tid >> 6));
    const char *p_row = static_cast<const char *>(a.logits) + r * a.ld * kSize;
    // asked for before it is known what of it there is
    PartCells<FEW> raw;
    PartHead head = {-kInf, ~0u, 0, 0};
    if (tid < static_cast<uint32_t>(a.parts)) head = a.heads[r * a.parts + tid];
    raw.take(a.cells + r * a.parts * kCells, a.parts);
    constexpr int kMine = kHeld / (kWaves * 64);
    uint64_t orders[kMine];
#pragma unroll
    for (int i = 0; i < kMine; ++i) orders[i] = a.list[r * kHeld + i * (kWaves * 64) + tid];
    const float u = a.tokens ? a.u[r] : 0.f;
    Plan p = a.plans[r].plan;
    const How h = how_of(a, r);
    raw.put(held, a.parts);
    if (h.greedy || !filters(a, h)) p.n = 0, p.k_on = p.p_on = 0, p.one = p.lo = p.min = -1, p.hi = -2;
    else if (p.lo != p.hi && tid < kCells) t.cells.w[tid] = a.plans[r].cells.w[tid], t.cells.count[tid] = a.plans[r].cells.count[tid];
    const Whole all = heads_of(a, head, h.c8, s);
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
    const bool listed = p.n <= kHeld;
    uint64_t from = 0;
    int border = kCells;                           // the cell that is kept in part; those before it are whole
    if (p.n && (p.k_on || p.p_on)) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) t.held[i * (kWaves * 64) + tid] = orders[i];
        __syncthreads();
        const Entries<FMT> g = {t.held, listed ? p.n : 0, p_row, listed ? 0 : static_cast<uint32_t>(a.vocab)};
        // top-k, then top-p of what it leaves
        double w_kept = p.k.w_all;
#pragma unroll 1
        for (int by_count = p.k_on; by_count >= (p.p_on ? 0 : 1); --by_count) {
            const double sum = by_count ? 0 : static_cast<double>(h.top_p) * w_kept;
            Border b = by_count ? p.k : p.p;
            if (!by_count && p.lo != p.hi) {
                if (wave == 0) {
                    b = border_of(t.cells, false, 0, sum);
                    if (lane == 0) t.border = b;
                }
                __syncthreads();
                b = same(t.border);
            }
            const uint64_t o = keep_from(g, t, sc, b, by_count != 0, h.k, sum, w_kept);
            from = o > from ? o : from;
            border = b.bin < border ? b.bin : border;
        }
    }
    if (p.min >= 0 && p.min < border) border = p.min;      // (which may hold nothing)
    const auto weight = [&](float z, uint32_t j) {
        return in_row(z) && order_of(z, j) >= from && sc.y(z) >= least ? sc.weight(z) : 0.0;
    };
    // the kept weight of each part; a wave a part: whole cells, and entries of the border's
    const double top = sc.top();
    const uint64_t *mine_cells = PartCells<FEW>::of(a.cells + r * a.parts * kCells, held);
    for (int i = wave; i < a.parts; i += kWaves) {
        double w = 0;
#pragma unroll
        for (int e = 0; e < kCells; e += 64) {
            const int c = e + lane, to = c + s.shift[i];
            if ((to < kCells - 1 ? to : kCells - 1) < border)
                w += static_cast<double>(mine_cells[i * kCells + c] & 0xffffffffffffull) / top * power(-(s.below[i] + c));
        }
        if (border < kCells && p.n) {
            if (listed) {
                const uint32_t end = i + 1 < a.parts ? a.heads[r * a.parts + i + 1].at : p.n;
                for (uint32_t at = a.heads[r * a.parts + i].at + lane; at < end; at += 64) {
                    const uint64_t o = a.list[r * kHeld + at];
                    const float z = logit_of(o);
                    if (sc.cell(sc.y(z)) == border) w += weight(z, ~static_cast<uint32_t>(o));
                }
            } else {
                const uint32_t j1 = static_cast<uint32_t>((i + 1) * a.part < a.vocab ? (i + 1) * a.part : a.vocab);
                for (uint32_t j = i * a.part + lane; j < j1; j += 64) {
                    const float z = load_one<FMT>(p_row, j);
                    if (in_row(z) && sc.cell(sc.y(z)) == border) w += weight(z, j);
                }
            }
        }
        w = lanes_total(w);
        if (lane == 0) s.part_sum[i] = w;
    }
    __syncthreads();
    const Place in = place_of(s.part_sum, a.parts, true, u);
    if (tid == 0) a.outs[r] = RowOut{in.total, least, from, all.m, -1};
    if (!a.tokens) return;
    // the part's segments
    const int64_t j0 = static_cast<int64_t>(in.at) * a.part;
    const int segs = a.part / kSeg;
    float *logits = reinterpret_cast<float *>(t.held);         // the orders are done with
    static_assert(sizeof(t.held) >= kPartSegs * kSeg * sizeof(float), "a part's logits in place of the orders");
    __syncthreads();
    constexpr int kEachWave = kPartSegs / kWaves;
    float z[kEachWave][kEach];
#pragma unroll
    for (int q = 0; q < kEachWave; ++q)
        if (wave + q * kWaves < segs) load_seg<FMT>(p_row, j0 + (wave + q * kWaves) * kSeg, a.vocab, z[q], -kInf);
#pragma unroll
    for (int q = 0; q < kEachWave; ++q)
        if (wave + q * kWaves < segs) {
#pragma unroll
            for (int e = 0; e < kEach; ++e) logits[(wave + q * kWaves) * kSeg + entry_of<FMT>(lane, e)] = z[q][e];
        }
    const auto weight_in = [&](int seg, int i) {
        return weight(logits[seg * kSeg + i], static_cast<uint32_t>(j0) + seg * kSeg + i);
    };
    Lanes lanes[kEachWave];
#pragma unroll
    for (int q = 0; q < kEachWave; ++q) {
        const int seg = wave + q * kWaves;
        lanes[q] = Lanes{0, 0};
        if (seg < segs) {
            lanes[q] = lanes_of([&](int i) { return weight_in(seg, i); });
            if (lane == 63) seg_sum[seg] = lanes[q].up;
        }
    }
    __syncthreads();
    const Place at = place_of(seg_sum, segs, false, in.target - in.before);
    if (wave == at.at % kWaves) {
        const Lanes mine = at.at < kWaves ? lanes[0] : lanes[kEachWave - 1];
        static_assert(kEachWave <= 2, "one of two");
        const int token = entry_in([&](int i) { return weight_in(at.at, i); }, mine, in.target - in.before, at.before);
        if (lane == 0) a.tokens[r] = static_cast<int32_t>(j0) + at.at * kSeg + token;
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

// Entries of a part, a segment or two of them to each of eight waves.
int64_t parts_of(int64_t vocab, int64_t segs) { return (vocab + segs * kSeg - 1) / (segs * kSeg); }
int64_t segs_of(int64_t n_rows, int64_t vocab) {
    const int64_t parts = parts_of(vocab, kWaves);
    return parts <= kFewParts && n_rows * parts <= kFill ? kWaves : kPartSegs;
}

template <int FMT, int SEGS, bool FEW>
void go_long(const SampleArgs &a, unsigned rows, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(a.parts), rows), block(kWaves * 64);
    hipLaunchKernelGGL((sample_cells_kernel<FMT, SEGS>), grid, block, 0, s, a);
    const bool some = a.how.d_top_k || a.how.d_top_p || a.how.d_min_p || a.how.top_k > 0 || a.how.top_p < 1 || a.how.min_p > 0;
    if (some) hipLaunchKernelGGL((sample_border_kernel<FMT, SEGS, FEW>), grid, block, 0, s, a);
    hipLaunchKernelGGL((sample_pick_kernel<FMT, FEW>), dim3(rows), dim3(kWaves * 64), 0, s, a);
    if (a.probs)
        hipLaunchKernelGGL(sample_probs_kernel<FMT>, dim3(static_cast<unsigned>((a.vocab + 4 * kSeg - 1) / (4 * kSeg)), rows), dim3(256), 0, s, a);
}

template <int FMT>
void go(const SampleArgs &a, int64_t n_rows, hipStream_t s) {
    const unsigned rows = static_cast<unsigned>(n_rows);
    const unsigned waves = a.vocab <= 4 * kSeg && n_rows > kManyRows ? 4 : kWaves;
    if (a.vocab <= kChunk) hipLaunchKernelGGL(sample_short_kernel<FMT>, dim3(rows), dim3(waves * 64), 0, s, a);
    else if (a.part == kWaves * kSeg) go_long<FMT, 1, true>(a, rows, s);
    else if (a.parts <= kFewParts) go_long<FMT, 2, true>(a, rows, s);
    else go_long<FMT, 2, false>(a, rows, s);
}

}  // namespace

size_t sample_ws_bytes(int64_t n_rows, int64_t vocab) {
    if (vocab <= kChunk) return 0;
    // (what the shorter parts take: more rows never take less)
    const size_t parts = static_cast<size_t>(parts_of(vocab, parts_of(vocab, kWaves) <= kFewParts ? kWaves : kPartSegs));
    return static_cast<size_t>(n_rows) * (sizeof(RowOut) + sizeof(RowPlan) + parts * (sizeof(PartHead) + kCells * sizeof(uint64_t)) +
                                          kHeld * sizeof(uint64_t));
}

int launch_sample(const void *logits, int zfmt, int64_t n_rows, int64_t vocab, int64_t ld, const wsl_sampling *how,
                  const float *u, int32_t *tokens, float *probs, int64_t ld_probs, void *ws, uint32_t *status, hipStream_t s) {
    SampleArgs a = {};
    a.logits = logits, a.u = u, a.tokens = tokens, a.probs = probs, a.status = status;
    a.vocab = vocab, a.ld = ld, a.ld_probs = ld_probs;
    if (how) a.how = *how;
    else a.how = {nullptr, nullptr, nullptr, nullptr, 1.f, 0, 1.f, 0.f};
    const int64_t segs = segs_of(n_rows, vocab), parts = parts_of(vocab, segs);
    a.parts = static_cast<int32_t>(parts), a.part = static_cast<int32_t>(segs * kSeg);
    a.cells = static_cast<uint64_t *>(ws);
    a.list = a.cells + n_rows * parts * kCells;
    a.plans = reinterpret_cast<RowPlan *>(a.list + n_rows * kHeld);
    a.heads = reinterpret_cast<PartHead *>(a.plans + n_rows);
    a.outs = reinterpret_cast<RowOut *>(a.heads + n_rows * parts);
    if (zfmt == WSL_OUT_F32) go<WSL_OUT_F32>(a, n_rows, s);
    else go<WSL_OUT_BF16>(a, n_rows, s);
    return WSL_OK;
}

}  // namespace wsl
