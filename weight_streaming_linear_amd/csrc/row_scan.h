// Rows of a vocabulary taken by waves: segments of 1024 entries, and sums over the lanes in 64 bits.
#pragma once

#include "device_common.h"

namespace wsl {
namespace {

constexpr int kSeg = 1024;                             // entries a wave takes together
constexpr int kEach = kSeg / 64;                       // of a lane

template <int FMT>
__device__ __forceinline__ float load_one(const void *p, uint32_t i) {
    if constexpr (FMT == WSL_OUT_F32) return static_cast<const float *>(p)[i];
    return bf16_lo(static_cast<const uint16_t *>(p)[i]);
}

// Entries j0 .. j0 + kSeg - 1 of a row, `pad` past its end.  Element i of lane l is entry
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
__device__ __forceinline__ void load_seg(const char *row, int64_t j0, int64_t vocab, float (&x)[kEach],
                                         float pad = 0.f) {
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
            x[i] = pad;
            if (j < left) x[i] = load_one<FMT>(base, static_cast<uint32_t>(j));
        }
    }
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
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t lanes_add(uint32_t v) {
    return v + static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), CTRL, ROWS, 0xf, false));
}
__device__ __forceinline__ uint32_t lanes_before(uint32_t v) {
    v = lanes_add<0x111, 0xf>(v);
    v = lanes_add<0x112, 0xf>(v);
    v = lanes_add<0x114, 0xf>(v);
    v = lanes_add<0x118, 0xf>(v);
    v = lanes_add<0x142, 0xa>(v);
    return lanes_add<0x143, 0xc>(v);
}
__device__ __forceinline__ uint32_t lane_value(uint32_t v, int lane) {
    return static_cast<uint32_t>(__builtin_amdgcn_readlane(static_cast<int>(v), lane));
}
__device__ __forceinline__ double lane_value(double v, int lane) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = __builtin_amdgcn_readlane(static_cast<int>(b), lane);
    const uint32_t hi = __builtin_amdgcn_readlane(static_cast<int>(b >> 32), lane);
    return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
__device__ __forceinline__ double lanes_total(double v) { return lane_value(lanes_before(v), 63); }

// A segment in the order of its entries: the first whose running sum of weights (from `run` on) passes the
// target; where none does, the last with a weight.  weight(i) is that of a lane's element i.
template <int FMT, typename Weight>
__device__ __forceinline__ int32_t look_through(Weight weight, int64_t j0, double target, double run) {
    constexpr int V = kVec<FMT>;
    int64_t last = -1;
#pragma unroll
    for (int b = 0; b < kEach; b += V) {
        double w[V], sum = 0;
#pragma unroll
        for (int e = 0; e < V; ++e) {
            w[e] = weight(b + e);
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

}  // namespace
}  // namespace wsl
