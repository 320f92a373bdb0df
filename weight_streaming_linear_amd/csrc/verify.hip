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
// Bound: the two rows that are read, V * (4 + 4) bytes per sequence.  A first kernel sums
// chunks of kChunk entries (one workgroup each, so that one sequence alone spreads over the
// chip); a second, one workgroup per sequence, finds the chunk that holds the target sum and
// looks only through that one.
#include "device_common.h"

namespace wsl {
namespace {

constexpr int kChunk = 4096;         // entries per workgroup: 16 per lane
constexpr int kPerLane = kChunk / 256;

struct VerifyArgs {
    const void *p, *q;
    const int32_t *drafts, *n_drafts;
    const float *u;
    int32_t *accepted, *tokens;
    double *sums;                    // [n_seq][chunks][2]: sums of w and of max(p, 0)
    uint32_t *status;
    int64_t ld_p, ld_q, vocab, chunks;
    int32_t width;                   // drafts per sequence, at most 64
};

template <int FMT>
__device__ __forceinline__ float load_one(const void *p, int64_t i) {
    if constexpr (FMT == WSL_OUT_F32) return static_cast<const float *>(p)[i];
    return bf16_lo(static_cast<const uint16_t *>(p)[i]);
}

// What a sequence samples from: the row's pointers, q null where there is nothing to take off.
struct Row {
    int32_t n, r, one_hot;           // one_hot: the index whose weight is zero, or -1
    bool bad;                        // a draft outside the vocabulary
    const char *p, *q;
};

// Every lane of every wave comes to the same Row: lane i judges draft i, a ballot finds the first
// that falls.
template <int FMT>
__device__ __forceinline__ Row judge(const VerifyArgs &a, int64_t seq) {
    constexpr int kSize = FMT == WSL_OUT_F32 ? 4 : 2;
    const int lane = static_cast<int>(threadIdx.x & 63);
    Row o;
    o.n = a.width;
    if (a.n_drafts != nullptr) {
        o.n = a.n_drafts[seq];
        o.n = o.n < 0 ? 0 : (o.n > a.width ? a.width : o.n);
    }
    const char *p0 = static_cast<const char *>(a.p) + seq * (a.width + 1) * a.ld_p * kSize;
    const char *q0 = a.q ? static_cast<const char *>(a.q) + seq * a.width * a.ld_q * kSize : nullptr;
    bool stands = true, bad = false;
    int32_t x = -1;
    if (lane < o.n) {
        x = a.drafts[seq * a.width + lane];
        bad = x < 0 || x >= a.vocab;
        stands = false;
        if (!bad) {
            const double px = load_one<FMT>(p0 + lane * a.ld_p * kSize, x);
            const double qx = q0 ? static_cast<double>(load_one<FMT>(q0 + lane * a.ld_q * kSize, x)) : 1.0;
            stands = static_cast<double>(a.u[seq * (a.width + 1) + lane]) * qx < px;
        }
    }
    const uint64_t fell = __ballot(!stands);
    o.bad = __ballot(bad) != 0;
    o.r = fell ? __builtin_ctzll(fell) : o.n;
    o.one_hot = -1;
    o.p = p0 + o.r * a.ld_p * kSize;
    o.q = nullptr;
    if (o.r < o.n) {
        if (q0) o.q = q0 + o.r * a.ld_q * kSize;
        else o.one_hot = __shfl(x, o.r, 64);
    }
    return o;
}

// Weights of entry j: NaN and negative ones count as zero.
template <int FMT>
__device__ __forceinline__ void weights(const Row &o, int64_t j, double &w, double &top) {
    const double p = load_one<FMT>(o.p, j);
    top = p > 0 ? p : 0;
    w = top;
    if (o.q) {
        const double d = p - static_cast<double>(load_one<FMT>(o.q, j));
        w = d > 0 ? d : 0;
    } else if (j == o.one_hot) {
        w = 0;
    }
}

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
    return v;
}

template <int FMT>
__global__ __launch_bounds__(256) void verify_sum_kernel(VerifyArgs a) {
    __shared__ double part[4][2];
    const int64_t seq = blockIdx.y;
    const Row o = judge<FMT>(a, seq);
    double sw = 0, sp = 0;
#pragma unroll
    for (int i = 0; i < kPerLane; ++i) {
        const int64_t j = static_cast<int64_t>(blockIdx.x) * kChunk + i * 256 + threadIdx.x;
        if (j < a.vocab) {
            double w, top;
            weights<FMT>(o, j, w, top);
            sw += w;
            sp += top;
        }
    }
    sw = wave_sum64(sw);
    sp = wave_sum64(sp);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6][0] = sw, part[threadIdx.x >> 6][1] = sp;
    __syncthreads();
    if (threadIdx.x < 2)
        a.sums[(seq * a.chunks + blockIdx.x) * 2 + threadIdx.x] =
            (part[0][threadIdx.x] + part[1][threadIdx.x]) + (part[2][threadIdx.x] + part[3][threadIdx.x]);
}

// Sums before each thread's own value (exclusive, in thread order) and over all 256.
__device__ __forceinline__ double block_before(double v, double *lds, double &total) {
    const int lane = static_cast<int>(threadIdx.x & 63), wave = static_cast<int>(threadIdx.x >> 6);
    double run = v;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const double o = __shfl_up(run, off, 64);
        if (lane >= off) run += o;
    }
    if (lane == 63) lds[wave] = run;
    __syncthreads();
    double before = 0;
    total = 0;
    for (int i = 0; i < 4; ++i) {
        if (i < wave) before += lds[i];
        total += lds[i];
    }
    __syncthreads();
    return before + (run - v);
}

// The least index over the workgroup, or 0x7fffffff... of the ones given.
__device__ __forceinline__ int64_t block_least(int64_t v, int64_t *lds) {
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) {
        const int64_t o = __shfl_xor(v, off, 64);
        v = o < v ? o : v;
    }
    if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
    __syncthreads();
    int64_t m = lds[0];
    for (int i = 1; i < 4; ++i) m = lds[i] < m ? lds[i] : m;
    __syncthreads();
    return m;
}

template <int FMT>
__global__ __launch_bounds__(256) void verify_pick_kernel(VerifyArgs a) {
    __shared__ double lds[4];
    __shared__ int64_t ldi[4];
    __shared__ double before_chunk;
    constexpr int64_t kNone = INT64_MAX;
    const int64_t seq = blockIdx.x;
    const Row o = judge<FMT>(a, seq);
    const double *sums = a.sums + seq * a.chunks * 2;
    // each thread takes `each` successive chunks
    const int64_t each = (a.chunks + 255) / 256;
    const int64_t c0 = each * threadIdx.x, c1 = c0 + each < a.chunks ? c0 + each : a.chunks;
    double mine = 0, top = 0, total;
    for (int64_t c = c0; c < c1; ++c) mine += sums[2 * c], top += sums[2 * c + 1];
    double before = block_before(mine, lds, total);
    int which = 0;
    if (!(total > 0)) {               // nothing left of p once q is off: sample p itself
        which = 1;
        mine = top;
        before = block_before(mine, lds, total);
    }
    int32_t token = -1;
    if (total > 0 && total < __builtin_huge_val()) {
        double target = static_cast<double>(a.u[seq * (a.width + 1) + a.width]) * total;
        target = target < 0 ? 0 : target;    // NaN passes no sum: the last entry, as u >= 1
        // the first chunk whose running sum passes the target; where rounding (or u >= 1) lets
        // none pass, the last one that holds anything
        int64_t hit = kNone, last = -1;
        double at = before, hit_before = 0, last_before = 0;
        for (int64_t c = c0; c < c1; ++c) {
            const double s = sums[2 * c + which];
            if (s > 0) last = c, last_before = at;
            if (hit == kNone && s > 0 && at + s > target) hit = c, hit_before = at;
            at += s;
        }
        int64_t chunk = block_least(hit, ldi);
        if (chunk == kNone) {
            chunk = -block_least(-last, ldi);
            hit = last, hit_before = last_before;
        }
        if (hit == chunk) before_chunk = hit_before;
        __syncthreads();
        // its entries, 16 successive ones a thread
        const int64_t j0 = chunk * kChunk + static_cast<int64_t>(threadIdx.x) * kPerLane;
        double w[kPerLane], sum = 0, all;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
            w[i] = 0;
            if (j0 + i < a.vocab) {
                double t;
                weights<FMT>(o, j0 + i, w[i], t);
                if (which) w[i] = t;
            }
            sum += w[i];
        }
        double run = before_chunk + block_before(sum, lds, all);
        int64_t first = kNone, end = -1;
#pragma unroll
        for (int i = 0; i < kPerLane; ++i) {
            run += w[i];
            if (w[i] > 0) end = j0 + i;
            if (first == kNone && w[i] > 0 && run > target) first = j0 + i;
        }
        first = block_least(first, ldi);
        if (first == kNone) first = -block_least(-end, ldi);
        token = static_cast<int32_t>(first);
    }
    if (threadIdx.x <= static_cast<unsigned>(a.width)) {
        const int i = static_cast<int>(threadIdx.x);
        a.tokens[seq * (a.width + 1) + i] = i < o.r ? a.drafts[seq * a.width + i] : (i == o.r ? token : -1);
    }
    if (threadIdx.x == 0) {
        a.accepted[seq] = o.r;
        const uint32_t st = (o.bad ? WSL_STATUS_INDEX : 0u) | (token < 0 ? WSL_STATUS_NONFINITE : 0u);
        if (st && a.status != nullptr) atomicOr(a.status, st);
    }
}

}  // namespace

size_t verify_ws_bytes(int64_t n_seq, int64_t vocab) {
    return static_cast<size_t>(n_seq) * static_cast<size_t>((vocab + kChunk - 1) / kChunk) * 2 * sizeof(double);
}

int launch_verify(const void *p, const void *q, int pfmt, int64_t n_seq, int64_t width, int64_t vocab, int64_t ld_p,
                  int64_t ld_q, const int32_t *drafts, const int32_t *n_drafts, const float *u, int32_t *accepted,
                  int32_t *tokens, void *ws, uint32_t *status, hipStream_t s) {
    VerifyArgs a;
    a.p = p, a.q = q, a.drafts = drafts, a.n_drafts = n_drafts, a.u = u, a.accepted = accepted, a.tokens = tokens;
    a.sums = static_cast<double *>(ws), a.status = status;
    a.ld_p = ld_p, a.ld_q = ld_q, a.vocab = vocab, a.chunks = (vocab + kChunk - 1) / kChunk;
    a.width = static_cast<int32_t>(width);
    const dim3 grid(static_cast<unsigned>(a.chunks), static_cast<unsigned>(n_seq));
    if (pfmt == WSL_OUT_F32) {
        hipLaunchKernelGGL(verify_sum_kernel<WSL_OUT_F32>, grid, dim3(256), 0, s, a);
        hipLaunchKernelGGL(verify_pick_kernel<WSL_OUT_F32>, dim3(grid.y), dim3(256), 0, s, a);
    } else {
        hipLaunchKernelGGL(verify_sum_kernel<WSL_OUT_BF16>, grid, dim3(256), 0, s, a);
        hipLaunchKernelGGL(verify_pick_kernel<WSL_OUT_BF16>, dim3(grid.y), dim3(256), 0, s, a);
    }
    return WSL_OK;
}

}  // namespace wsl
