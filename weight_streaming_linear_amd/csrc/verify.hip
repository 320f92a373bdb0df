// Verification of drafted tokens (verify_drafts) for gfx950.
//
// TCPP README, "Quickstart": one sweep scores every position of a context; Tarfa 2,
// "Speculative decoding": drafts are kept only where the target agrees.  For a sequence with
// drafts x_0 .. x_{n-1}, target rows p_0 .. p_n, draft rows q_i (or none: a deterministic
// drafter, q_i = 1 at x_i) and numbers u_0 .. in [0, 1):
//     draft i stands iff every earlier one does and u_i * q_i(x_i) < p_i(x_i);
//     r = the number that stand;
//     w_j = max(p_r(j) - q_r(j), 0) if r < n (a draft fell), max(p_n(j), 0) if all stand;
//     if the w_j sum to zero, w_j = max(p_r(j), 0);
//     the next token is the least j with w_0 + .. + w_j > u_last * (w_0 + .. + w_{V-1}).
// The accepted token then has the target's distribution.  Everything is decided in 64 bits:
// u * q of two fp32 numbers is exact there, and a sum of V differences is off by about
// 2^-53 * V, so the token does not depend on how the sum is split.
//
// Bound: the two rows that are read, V * (4 + 4) bytes per sequence, and at small sizes the chain
// drafts -> their probabilities -> the row -> its sum -> the token.  A wave takes segments of 1024
// entries, each lane 16 bytes at a time.  Up to kSmallVocab one workgroup a sequence asks for the whole
// rows at once and one launch does all of it.  Beyond, one launch sums the segments, so that
// one sequence alone spreads over the chip, and a second, one wave a sequence, finds the segment that
// holds the target sum and looks through that one.  (fp32, 64 sequences of 8 drafts over 151937 entries:
// 14.5 us, 5.4 TB/s, and 4.6; one of 4 over 32000 in one launch: 5.8 us.)
#include "device_common.h"

namespace wsl {
namespace {

constexpr int kSeg = 1024;                             // entries a wave takes together
constexpr int kEach = kSeg / 64;                       // of a lane
constexpr int kSmallWaves = 16, kSmallSegs = 2;
constexpr int64_t kSmallVocab = kSmallWaves * kSmallSegs * kSeg;

// What one sequence samples from: r drafts stand; of n.
struct Verdict {
    int32_t n, r, one_hot;           // one_hot: the index whose weight is zero, or -1
    uint32_t bad;                    // a draft outside the vocabulary
};

struct VerifyArgs {
    const void *p, *q;
    const int32_t *drafts, *n_drafts;
    const float *u;
    int32_t *accepted, *tokens;
    double2 *sums;                   // [n_seq][segs]: sums of w and of max(p, 0)
    Verdict *verdicts;               // [n_seq]
    uint32_t *status;
    int64_t ld_p, ld_q, vocab, segs;
    int32_t width;                   // drafts per sequence, at most 64
};

template <int FMT>
__device__ __forceinline__ float load_one(const void *p, uint32_t i) {
    if constexpr (FMT == WSL_OUT_F32) return static_cast<const float *>(p)[i];
    return bf16_lo(static_cast<const uint16_t *>(p)[i]);
}

// Every lane of a wave comes to the same Verdict: lane i judges draft i, a ballot finds the first
// that falls.
template <int FMT>
__device__ __forceinline__ Verdict judge(const VerifyArgs &a, int64_t seq) {
    constexpr int kSize = FMT == WSL_OUT_F32 ? 4 : 2;
    const int lane = static_cast<int>(threadIdx.x & 63);
    Verdict o;
    o.n = a.width;
    if (a.n_drafts != nullptr) {
        o.n = __builtin_amdgcn_readfirstlane(a.n_drafts[seq]);
        o.n = o.n < 0 ? 0 : (o.n > a.width ? a.width : o.n);
    }
    bool stands = true, bad = false;
    int32_t x = -1;
    if (lane < o.n) {
        x = a.drafts[seq * a.width + lane];
        const float u = a.u[seq * (a.width + 1) + lane];
        bad = x < 0 || x >= a.vocab;
        stands = false;
        if (!bad) {
            const char *p = static_cast<const char *>(a.p) + (seq * (a.width + 1) + lane) * a.ld_p * kSize;
            const char *q = static_cast<const char *>(a.q) + (seq * a.width + lane) * a.ld_q * kSize;
            const double px = load_one<FMT>(p, x);
            const double qx = a.q ? static_cast<double>(load_one<FMT>(q, x)) : 1.0;
            stands = static_cast<double>(u) * qx < px;
        }
    }
    const uint64_t fell = __ballot(!stands);
    o.bad = __ballot(bad) != 0;
    o.r = fell ? __builtin_ctzll(fell) : o.n;
    o.one_hot = o.r < o.n && !a.q ? __builtin_amdgcn_readlane(x, o.r) : -1;
    return o;
}

// The row that is sampled and the one that is taken off it (null where there is none).
template <int FMT>
__device__ __forceinline__ void rows_of(const VerifyArgs &a, int64_t seq, const Verdict &o, const char *&p,
                                        const char *&q) {
    constexpr int kSize = FMT == WSL_OUT_F32 ? 4 : 2;
    p = static_cast<const char *>(a.p) + (seq * (a.width + 1) + o.r) * a.ld_p * kSize;
    q = o.r < o.n && a.q ? static_cast<const char *>(a.q) + (seq * a.width + o.r) * a.ld_q * kSize : nullptr;
}

// Entries j0 .. j0 + kSeg - 1 of a row, zeros past its end.  Element i of lane l is entry
// entry_of(l, i): 16 bytes of a lane are read at once (rows need not be aligned for that).
template <int FMT>
constexpr int kVec = FMT == WSL_OUT_F32 ? 4 : 8;
template <int FMT>
__device__ __forceinline__ int entry_of(int lane, int i) {
    return (i / kVec<FMT>) * 64 * kVec<FMT> + lane * kVec<FMT> + i % kVec<FMT>;
}
typedef u32x4 u32x4_any __attribute__((aligned(2)));
typedef f32x4 f32x4_word __attribute__((aligned(4)));
template <int FMT>
__device__ __forceinline__ void load_seg(const char *row, int64_t j0, int64_t vocab, float (&x)[kEach]) {
    constexpr uint32_t kSize = FMT == WSL_OUT_F32 ? 4 : 2;
    const int lane = static_cast<int>(threadIdx.x & 63);
    const char *base = row + j0 * kSize;               // the same for the whole wave
    if (j0 + kSeg <= vocab) {
#pragma unroll
        for (int i = 0; i < kEach; i += kVec<FMT>) {
            const uint32_t at = static_cast<uint32_t>(entry_of<FMT>(lane, i)) * kSize;
            if constexpr (FMT == WSL_OUT_F32) {
                const f32x4 w = *reinterpret_cast<const f32x4_word *>(base + at);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[i + e] = w[e];
            } else {
                const u32x4 w = *reinterpret_cast<const u32x4_any *>(base + at);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[i + 2 * e] = bf16_lo(w[e]), x[i + 2 * e + 1] = bf16_hi(w[e]);
            }
        }
    } else {
        const int left = static_cast<int>(vocab - j0);  // may be none
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int j = entry_of<FMT>(lane, i);
            x[i] = 0.f;
            if (j < left) x[i] = load_one<FMT>(base, static_cast<uint32_t>(j));
        }
    }
}

// A segment of p and of what is taken off it: nothing, q, or infinity at the one draft that fell.
struct Seg {
    float p[kEach], q[kEach];
};
template <int FMT>
__device__ __forceinline__ void load(const char *p, const char *q, int64_t j0, int64_t vocab, int32_t one_hot, Seg &s) {
    load_seg<FMT>(p, j0, vocab, s.p);
    if (q) {
        load_seg<FMT>(q, j0, vocab, s.q);
    } else {
        const int64_t at = one_hot - j0;
        const int lane = static_cast<int>(threadIdx.x & 63);
#pragma unroll
        for (int i = 0; i < kEach; ++i) s.q[i] = entry_of<FMT>(lane, i) == at ? __builtin_huge_valf() : 0.f;
    }
}
// Weights: NaN and negative ones count as zero (the maximum with zero is zero for both).
__device__ __forceinline__ double top_of(const Seg &s, int i) { return __builtin_fmax(static_cast<double>(s.p[i]), 0.0); }
__device__ __forceinline__ double weight_of(const Seg &s, int i) {
    return __builtin_fmax(static_cast<double>(s.p[i]) - static_cast<double>(s.q[i]), 0.0);
}

// Sums over lanes 0 .. l, by moves inside the rows of 16 lanes and from row to row.
template <int CTRL, int ROWS>
__device__ __forceinline__ double lanes_add(double v) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_update_dpp(0, static_cast<int>(b), CTRL, ROWS, 0xf, false);
    const uint32_t hi = __builtin_amdgcn_update_dpp(0, static_cast<int>(b >> 32), CTRL, ROWS, 0xf, false);
    return v + __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
__device__ __forceinline__ double lanes_before(double v) {
    v = lanes_add<0x111, 0xf>(v);      // from 1, 2, 4 and 8 lanes before in the row
    v = lanes_add<0x112, 0xf>(v);
    v = lanes_add<0x114, 0xf>(v);
    v = lanes_add<0x118, 0xf>(v);
    v = lanes_add<0x142, 0xa>(v);      // rows 1 and 3: the row before's last lane
    return lanes_add<0x143, 0xc>(v);   // rows 2 and 3: lane 31
}
__device__ __forceinline__ double lane_value(double v, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(b), lane);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(b >> 32), lane);
    return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
__device__ __forceinline__ double lanes_total(double v) { return lane_value(lanes_before(v), 63); }

// A segment's sums over the wave: of the weights, and of the tops if that is zero.  They are asked for
// only where all weights of a row are zero, and then each segment's are.
__device__ __forceinline__ double2 sums_of(const Seg &s) {
    double sw = 0, sp = 0;
#pragma unroll
    for (int i = 0; i < kEach; ++i) sw += weight_of(s, i);
    sw = lanes_total(sw);
    if (sw == 0) {
#pragma unroll
        for (int i = 0; i < kEach; ++i) sp += top_of(s, i);
        sp = lanes_total(sp);
    }
    return make_double2(sw, sp);
}

// In the order of the entries: the first of a segment whose running sum (from `run` on) passes the
// target; where none does, the last with a weight.
template <int FMT>
__device__ __forceinline__ int32_t look_through(const Seg &s, int64_t j0, bool tops, double target, double run) {
    constexpr int V = kVec<FMT>;
    int64_t last = -1;
#pragma unroll
    for (int b = 0; b < kEach; b += V) {
        double w[V], sum = 0;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            w[e] = tops ? top_of(s, b + e) : weight_of(s, b + e);
            sum += w[e];
        }
        const double up = lanes_before(sum);
        double at = run + (up - sum);
        int hit = -1, end = -1;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            at += w[e];
            if (w[e] > 0) end = e;
            if (hit < 0 && w[e] > 0 && at > target) hit = e;
        }
        const uint64_t hits = __ballot(hit >= 0), ends = __ballot(end >= 0);
        const int64_t here = j0 + b / V * 64 * V;
        if (ends) {
            const int l = 63 - __builtin_clzll(ends);
            last = here + l * V + __builtin_amdgcn_readlane(end, l);
        }
        if (hits) {
            const int l = __builtin_ctzll(hits);
            return static_cast<int32_t>(here + l * V + __builtin_amdgcn_readlane(hit, l));
        }
        run += lane_value(up, 63);
    }
    return static_cast<int32_t>(last);
}

// What running sums have to pass; NaN passes none: the last entry, as for u >= 1.
__device__ __forceinline__ double target_of(const VerifyArgs &a, int64_t seq, double total) {
    const double t = static_cast<double>(a.u[seq * (a.width + 1) + a.width]) * total;
    return t < 0 ? 0 : t;
}

// One wave writes a sequence's results.
__device__ __forceinline__ void write_out(const VerifyArgs &a, int64_t seq, const Verdict &o, int32_t token) {
    const int lane = static_cast<int>(threadIdx.x & 63);
    for (int i = lane; i <= a.width; i += 64)
        a.tokens[seq * (a.width + 1) + i] = i < o.r ? a.drafts[seq * a.width + i] : (i == o.r ? token : -1);
    if (lane == 0) {
        a.accepted[seq] = o.r;
        const uint32_t st = (o.bad ? WSL_STATUS_INDEX : 0u) | (token < 0 ? WSL_STATUS_NONFINITE : 0u);
        if (st && a.status != nullptr) atomicOr(a.status, st);
    }
}

template <int FMT>
__global__ __launch_bounds__(kSmallWaves * 64) void verify_small_kernel(VerifyArgs a) {
    __shared__ double lds_w[kSmallWaves * kSmallSegs], lds_p[kSmallWaves * kSmallSegs];
    const int64_t seq = blockIdx.x;
    const int lane = static_cast<int>(threadIdx.x & 63), waves = static_cast<int>(blockDim.x >> 6);
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    const Verdict o = judge<FMT>(a, seq);
    const char *p, *q;
    rows_of<FMT>(a, seq, o, p, q);
    Seg s[kSmallSegs];
#pragma unroll
    for (int i = 0; i < kSmallSegs; ++i) load<FMT>(p, q, (wave * kSmallSegs + i) * kSeg, a.vocab, o.one_hot, s[i]);
#pragma unroll
    for (int i = 0; i < kSmallSegs; ++i) {
        const double2 sums = sums_of(s[i]);
        if (lane == 0) lds_w[wave * kSmallSegs + i] = sums.x, lds_p[wave * kSmallSegs + i] = sums.y;
    }
    __syncthreads();
    // (the entries stay in registers as they were read: not the weights, which take twice as many)
#pragma unroll
    for (int i = 0; i < kSmallSegs; ++i)
#pragma unroll
        for (int e = 0; e < kEach; ++e) asm volatile("" : "+v"(s[i].p[e]), "+v"(s[i].q[e]));
    double mine = lane < waves * kSmallSegs ? lds_w[lane] : 0.0, up = lanes_before(mine), total = lane_value(up, 63);
    const bool tops = !(total > 0);        // nothing left of p once q is off: sample p itself
    if (tops) {
        mine = lane < waves * kSmallSegs ? lds_p[lane] : 0.0;
        up = lanes_before(mine);
        total = lane_value(up, 63);
    }
    if (!(total > 0 && total < __builtin_huge_val())) {
        if (wave == 0) write_out(a, seq, o, -1);
        return;
    }
    const double target = target_of(a, seq, total);
    // the first segment whose running sum passes the target; where rounding (or u >= 1) lets none
    // pass, the last one that holds anything
    const uint64_t hits = __ballot(mine > 0 && up > target), some = __ballot(mine > 0);
    const int which = hits ? __builtin_ctzll(hits) : 63 - __builtin_clzll(some);
#pragma unroll
    for (int i = 0; i < kSmallSegs; ++i)
        if (which == wave * kSmallSegs + i)
            write_out(a, seq, o, look_through<FMT>(s[i], which * kSeg, tops, target, which == 0 ? 0.0 : lane_value(up, which - 1)));
}

template <int FMT>
__global__ __launch_bounds__(256) void verify_sum_kernel(VerifyArgs a) {
    const int64_t seq = blockIdx.y;
    const int64_t seg = static_cast<int64_t>(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x >> 6));
    const int lane = static_cast<int>(threadIdx.x & 63);
    if (seg >= a.segs) return;
    const Verdict o = judge<FMT>(a, seq);
    const char *p, *q;
    rows_of<FMT>(a, seq, o, p, q);
    Seg s;
    load<FMT>(p, q, seg * kSeg, a.vocab, o.one_hot, s);
    const double2 sums = sums_of(s);
    if (lane == 0) {
        a.sums[seq * a.segs + seg] = sums;
        if (seg == 0) a.verdicts[seq] = o;
    }
}

// One wave a sequence; each lane holds `each` successive segments.
template <int FMT>
__global__ __launch_bounds__(64) void verify_pick_kernel(VerifyArgs a) {
    const int64_t seq = blockIdx.x;
    const int lane = static_cast<int>(threadIdx.x & 63);
    const Verdict o = a.verdicts[seq];
    const double2 *sums = a.sums + seq * a.segs;
    const int64_t each = (a.segs + 63) / 64;
    const int64_t c0 = each * lane < a.segs ? each * lane : a.segs, c1 = c0 + each < a.segs ? c0 + each : a.segs;
    double sw = 0, sp = 0;
#pragma unroll 4
    for (int64_t c = c0; c < c1; ++c) {
        const double2 s = sums[c];
        sw += s.x, sp += s.y;
    }
    double mine = sw, up = lanes_before(mine), total = lane_value(up, 63);
    const bool tops = !(total > 0);
    if (tops) {
        mine = sp;
        up = lanes_before(mine);
        total = lane_value(up, 63);
    }
    int32_t token = -1;
    if (total > 0 && total < __builtin_huge_val()) {
        const double target = target_of(a, seq, total);
        int64_t hit = -1, last = -1;
        double at = up - mine, hit_at = 0, last_at = 0;
        for (int64_t c = c0; c < c1; ++c) {
            const double s = tops ? sums[c].y : sums[c].x;
            if (s > 0) last = c, last_at = at;
            if (hit < 0 && s > 0 && at + s > target) hit = c, hit_at = at;
            at += s;
        }
        const uint64_t hits = __ballot(hit >= 0), some = __ballot(last >= 0);
        const int l = hits ? __builtin_ctzll(hits) : 63 - __builtin_clzll(some);
        const int64_t seg = __builtin_amdgcn_readlane(static_cast<int>(hits ? hit : last), l);
        const double run = lane_value(hits ? hit_at : last_at, l);
        const char *p, *q;
        rows_of<FMT>(a, seq, o, p, q);
        Seg s;
        load<FMT>(p, q, seg * kSeg, a.vocab, o.one_hot, s);
        token = look_through<FMT>(s, seg * kSeg, tops, target, run);
    }
    write_out(a, seq, o, token);
}

template <int FMT>
void go(const VerifyArgs &a, int64_t n_seq, hipStream_t s) {
    const unsigned seqs = static_cast<unsigned>(n_seq);
    if (a.vocab <= kSmallVocab) {
        const unsigned waves = static_cast<unsigned>((a.segs + kSmallSegs - 1) / kSmallSegs);
        hipLaunchKernelGGL(verify_small_kernel<FMT>, dim3(seqs), dim3(waves * 64), 0, s, a);
        return;
    }
    hipLaunchKernelGGL(verify_sum_kernel<FMT>, dim3(static_cast<unsigned>((a.segs + 3) / 4), seqs), dim3(256), 0, s, a);
    hipLaunchKernelGGL(verify_pick_kernel<FMT>, dim3(seqs), dim3(64), 0, s, a);
}

int64_t segs_of(int64_t vocab) { return (vocab + kSeg - 1) / kSeg; }

}  // namespace

size_t verify_ws_bytes(int64_t n_seq, int64_t vocab) {
    if (vocab <= kSmallVocab) return 0;
    return static_cast<size_t>(n_seq) * (static_cast<size_t>(segs_of(vocab)) * sizeof(double2) + sizeof(Verdict));
}

int launch_verify(const void *p, const void *q, int pfmt, int64_t n_seq, int64_t width, int64_t vocab, int64_t ld_p,
                  int64_t ld_q, const int32_t *drafts, const int32_t *n_drafts, const float *u, int32_t *accepted,
                  int32_t *tokens, void *ws, uint32_t *status, hipStream_t s) {
    VerifyArgs a;
    a.p = p, a.q = q, a.drafts = drafts, a.n_drafts = n_drafts, a.u = u, a.accepted = accepted, a.tokens = tokens;
    a.status = status;
    a.ld_p = ld_p, a.ld_q = ld_q, a.vocab = vocab, a.segs = segs_of(vocab);
    a.width = static_cast<int32_t>(width);
    a.sums = static_cast<double2 *>(ws);
    a.verdicts = reinterpret_cast<Verdict *>(a.sums + n_seq * a.segs);
    if (pfmt == WSL_OUT_F32) go<WSL_OUT_F32>(a, n_seq, s);
    else go<WSL_OUT_BF16>(a, n_seq, s);
    return WSL_OK;
}

}  // namespace wsl
