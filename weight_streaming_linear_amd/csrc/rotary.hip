// Rotary positions (rotary_embed) for gfx950.
//
// For the token at position p and pair i, the angle is p * f_i radians.  Far positions lose it in
// binary32 (p = 10^6 leaves 2^-4 of a radian) and, rounded, in 64 bits too (2^-24 at 2^29), so the product is kept as
// the sum of two doubles, and brought to turns with 1 / 2 pi as two more:
//     t + t' = p f,  r = frac((t + t') / 2 pi) = (h - rint(h)) + l,   h + l = t * (C1 + C2) + t' * C1,
// (off by 2^-50 while |p f| < 2^52), then to the nearest quarter turn: |angle| <= pi / 4, sin and cos by their Taylor series
// (to x^11 and x^12: below 2^-33), rounded once to binary32.
//
// Bound: the heads' bytes in and out once.  One workgroup a token: its first waves make the rot_dim / 2
// pairs of cos and sin once for all heads, in LDS.  Measured: 2.8 us for one token of 40 and 8 heads of 128 (the launch); 8192 tokens
// of 48 and 8 (235 MB) 46.5 from memory, a copy's 5.1 TB/s, and 35.7 where the last-level cache holds some of it.
// Halves that are no multiple of 8 go an element at a time: 8192 tokens of 40 heads of 80 bf16 elements, turned by 40, 50 us, by 80
// 18.7.
#include "device_common.h"

namespace wsl {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMostGroups = int64_t(1) << 20;      // of a launch (which takes 2^32 threads at most): beyond, each goes on

struct RotaryArgs {
    const void *q, *k;
    void *q_out, *k_out;
    int64_t ld_q, ld_k, ld_q_out, ld_k_out;
    const int64_t *positions;
    const double *freqs;
    double amplitude;
    int64_t count;
    uint32_t heads, kv_heads, head_dim, half;      // half: rot_dim / 2
};

__device__ __forceinline__ float2 cos_sin(int64_t position, double freq, double amplitude) {
    constexpr double kTurns = 0.15915494309189535, kTurnsLow = -9.839338337591243e-18;   // 1 / 2 pi
    constexpr double kTau = 6.283185307179586;
    // the position's halves are doubles; what their sum loses (from 2^53 on) is the rest
    const double upper = static_cast<double>(static_cast<int32_t>(position >> 32)) * 4294967296.0;
    const double lower = static_cast<double>(static_cast<uint32_t>(position));
    const double p = upper + lower, rest = lower - (p - upper);
    const double angle = p * freq, more = __builtin_fma(p, freq, -angle) + rest * freq;
    const double h = angle * kTurns;
    const double l = __builtin_fma(angle, kTurns, -h) + (angle * kTurnsLow + more * kTurns);
    const double r = (h - __builtin_rint(h)) + l;      // about -0.5 .. 0.5 turns
    const double quarter = __builtin_rint(4 * r);
    const double x = (r - 0.25 * quarter) * kTau, y = x * x;
    double s = -1.0 / 39916800, c = 1.0 / 479001600;
    s = __builtin_fma(s, y, 1.0 / 362880), c = __builtin_fma(c, y, -1.0 / 3628800);
    s = __builtin_fma(s, y, -1.0 / 5040), c = __builtin_fma(c, y, 1.0 / 40320);
    s = __builtin_fma(s, y, 1.0 / 120), c = __builtin_fma(c, y, -1.0 / 720);
    s = __builtin_fma(s, y, -1.0 / 6), c = __builtin_fma(c, y, 1.0 / 24);
    s = __builtin_fma(s, y, 1.0), c = __builtin_fma(c, y, -0.5);
    s *= x, c = __builtin_fma(c, y, 1.0);
    const int q = static_cast<int>(quarter) & 3;
    const double co = q & 1 ? s : c, si = q & 1 ? c : s;
    return make_float2(static_cast<float>(amplitude * (q == 1 || q == 2 ? -co : co)),
                       static_cast<float>(amplitude * (q >= 2 ? -si : si)));
}

template <int FMT>
__device__ __forceinline__ void load8(const void *p, int64_t at, float (&x)[8]) {
    if constexpr (FMT == WSL_OUT_F32) {
        const f32x4 *f = reinterpret_cast<const f32x4 *>(static_cast<const float *>(p) + at);
        const f32x4 lo = f[0], hi = f[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = lo[i], x[4 + i] = hi[i];
    } else {
        const u32x4 w = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(p) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[2 * i] = bf16_lo(w[i]), x[2 * i + 1] = bf16_hi(w[i]);
    }
}
template <int FMT>
__device__ __forceinline__ void store8(void *p, int64_t at, const float (&x)[8]) {
    if constexpr (FMT == WSL_OUT_F32) {
        f32x4 *f = reinterpret_cast<f32x4 *>(static_cast<float *>(p) + at);
        f[0] = f32x4{x[0], x[1], x[2], x[3]};
        f[1] = f32x4{x[4], x[5], x[6], x[7]};
    } else {
        *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(p) + at) =
            u32x4{pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7])};
    }
}
template <int FMT>
__device__ __forceinline__ float load1(const void *p, int64_t at) {
    if constexpr (FMT == WSL_OUT_F32) return static_cast<const float *>(p)[at];
    return bf16_lo(static_cast<const uint16_t *>(p)[at]);
}
template <int FMT>
__device__ __forceinline__ void store1(void *p, int64_t at, float x) {
    if constexpr (FMT == WSL_OUT_F32) static_cast<float *>(p)[at] = x;
    else static_cast<uint16_t *>(p)[at] = static_cast<uint16_t>(pack_bf16x2(x, x));
}

__device__ __forceinline__ void turn(float &a, float &b, float2 cs) {
    const float y = a * cs.x - b * cs.y, z = a * cs.y + b * cs.x;
    a = y, b = z;
}

enum { kHalves = 0, kPairs = 1, kSingles = 2 };

// LAYOUT kHalves: 16 elements a task, eight and their partners half a rotation's width on, or eight
// to be copied twice (rot_dim a multiple of 16).  kPairs: eight, which hold whole pairs.  kSingles: one
// element and its partner, for halves of other widths.
template <int XF, int OF, int LAYOUT>
__global__ __launch_bounds__(kThreads) void rotary_kernel(RotaryArgs a) {
    __shared__ float2 cs[128];
    const uint32_t tid = threadIdx.x;
    // tasks of a head: pairs first, then what is copied
    const uint32_t turned = LAYOUT == kHalves ? a.half / 8 : (LAYOUT == kPairs ? a.head_dim / 8 : a.half);
    const uint32_t rest = LAYOUT == kHalves ? (a.head_dim - 2 * a.half) / 8 : (LAYOUT == kPairs ? 0 : a.head_dim - 2 * a.half);
    const uint32_t tasks = turned + rest, n = (a.heads + a.kv_heads) * tasks;
    for (int64_t t = blockIdx.x; t < a.count; t += gridDim.x) {
        if (tid < a.half) cs[tid] = cos_sin(a.positions[t], a.freqs[tid], a.amplitude);
        __syncthreads();
        for (uint32_t i = tid; i < n; i += kThreads) {
            const uint32_t h = i / tasks, e = i - h * tasks;
            const bool is_k = h >= a.heads;
            const void *x = is_k ? a.k : a.q;
            void *y = is_k ? a.k_out : a.q_out;
            const int64_t head = static_cast<int64_t>(is_k ? h - a.heads : h) * a.head_dim;
            const int64_t from = t * (is_k ? a.ld_k : a.ld_q) + head, to = t * (is_k ? a.ld_k_out : a.ld_q_out) + head;
            if constexpr (LAYOUT == kHalves) {
                float u[8], v[8];
                if (e < turned) {
                    load8<XF>(x, from + 8 * e, u);
                    load8<XF>(x, from + a.half + 8 * e, v);
    #pragma unroll
                    for (int j = 0; j < 8; ++j) turn(u[j], v[j], cs[8 * e + j]);
                    store8<OF>(y, to + 8 * e, u);
                    store8<OF>(y, to + a.half + 8 * e, v);
                } else {
                    const uint32_t at = 2 * a.half + 8 * (e - turned);
                    load8<XF>(x, from + at, u);
                    store8<OF>(y, to + at, u);
                }
            } else if constexpr (LAYOUT == kPairs) {
                float u[8];
                load8<XF>(x, from + 8 * e, u);
    #pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (4 * e + j < a.half) turn(u[2 * j], u[2 * j + 1], cs[4 * e + j]);
                store8<OF>(y, to + 8 * e, u);
            } else {
                if (e < turned) {
                    float u = load1<XF>(x, from + e), v = load1<XF>(x, from + a.half + e);
                    turn(u, v, cs[e]);
                    store1<OF>(y, to + e, u);
                    store1<OF>(y, to + a.half + e, v);
                } else {
                    const uint32_t at = a.half + e;        // 2 * half + (e - half)
                    store1<OF>(y, to + at, load1<XF>(x, from + at));
                }
            }
        }
        __syncthreads();
    }
}

template <int XF, int OF>
void go(const RotaryArgs &a, bool interleaved, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(a.count < kMostGroups ? a.count : kMostGroups));
    if (interleaved) hipLaunchKernelGGL((rotary_kernel<XF, OF, kPairs>), grid, dim3(kThreads), 0, s, a);
    else if (a.half % 8 == 0) hipLaunchKernelGGL((rotary_kernel<XF, OF, kHalves>), grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((rotary_kernel<XF, OF, kSingles>), grid, dim3(kThreads), 0, s, a);
}

}  // namespace

int launch_rotary(const void *q, int64_t n_heads, int64_t ld_q, const void *k, int64_t n_kv, int64_t ld_k, int xfmt,
                  int64_t count, int64_t head_dim, int64_t rot_dim, const int64_t *positions, const double *freqs,
                  double amplitude, int flags, void *q_out, int64_t ld_q_out, void *k_out, int64_t ld_k_out, int ofmt,
                  hipStream_t s) {
    RotaryArgs a;
    a.q = q, a.k = k, a.q_out = q_out, a.k_out = k_out;
    a.ld_q = ld_q, a.ld_k = ld_k, a.ld_q_out = ld_q_out, a.ld_k_out = ld_k_out;
    a.positions = positions, a.freqs = freqs, a.amplitude = amplitude, a.count = count;
    a.heads = static_cast<uint32_t>(n_heads), a.kv_heads = k ? static_cast<uint32_t>(n_kv) : 0;
    a.head_dim = static_cast<uint32_t>(head_dim), a.half = static_cast<uint32_t>(rot_dim / 2);
    const bool pairs = (flags & WSL_ROTARY_INTERLEAVED) != 0;
    if (xfmt == WSL_OUT_F32) {
        ofmt == WSL_OUT_F32 ? go<WSL_OUT_F32, WSL_OUT_F32>(a, pairs, s) : go<WSL_OUT_F32, WSL_OUT_BF16>(a, pairs, s);
    } else {
        ofmt == WSL_OUT_F32 ? go<WSL_OUT_BF16, WSL_OUT_F32>(a, pairs, s) : go<WSL_OUT_BF16, WSL_OUT_BF16>(a, pairs, s);
    }
    return WSL_OK;
}

}  // namespace wsl
