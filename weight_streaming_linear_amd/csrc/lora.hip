// Low-rank adapters of many requests beside a shared projection (lora_add) for gfx950.
//
//     h = A[a] x          (rank x k, summed in fp32, k in parts so that few tokens fill the chip)
//     out = base + scale[a] * B[a] h
// Two launches, the second adding up the parts of h.  Few tokens, each with an adapter of its own: one
// workgroup a token and part, dot products on the vector units, every byte of A and B read as it lies.
// More tokens: waves of 16 tokens on the matrix cores, once for each adapter among the 16 (a prompt's
// tokens share theirs).  There h goes in as three bf16 numbers (hi + mid + lo, 24 bits): its
// rounding to one would be the largest error of the result.
//
// Bound: base and out once each, x, and A and B of the adapters in use.
#include "device_common.h"

namespace wsl {
namespace {

constexpr int64_t kFewTokens = 64;
constexpr int kPart = 512;                 // least elements of k in a part
constexpr int64_t kMostParts = 16;

struct LoraArgs {
    const uint16_t *a, *b, *x;
    const int32_t *ids;
    const float *scales;
    const void *base;
    void *out;
    float *h;                              // [parts][m][rank]
    uint32_t *status;
    int64_t n_adapters, n_out, k, m, ldx, ld_base, ld_out;
    int64_t part;                          // elements of k in a part
    int32_t rank, parts, wide;             // wide: rows of base and out are 16-byte aligned
};

// A token's adapter, or -1; the first launch reports a bad one.
__device__ __forceinline__ int32_t adapter_of(const LoraArgs &a, int64_t t, bool report) {
    const int32_t id = a.ids[t];
    if (id >= 0 && id < a.n_adapters) return id;
    if (report && id != -1 && a.status != nullptr) atomicOr(a.status, WSL_STATUS_INDEX);
    return -1;
}

// ------------------------------------------------------------------ few tokens
// blockIdx: (token, part of k).  A wave takes 128 elements of k at a time, 16 lanes of 8 each, four rows
// of A side by side; ROWS of them one after the other.
template <int ROWS>
__global__ __launch_bounds__(256) void shrink_few_kernel(LoraArgs a) {
    __shared__ float lds[4][ROWS * 4];
    const int64_t t = blockIdx.x;
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wave = tid >> 6, g = lane >> 4;
    const int32_t id = adapter_of(a, t, blockIdx.y == 0 && tid == 0);
    if (id < 0) return;
    const uint16_t *w = a.a + static_cast<int64_t>(id) * a.rank * a.k, *x = a.x + t * a.ldx;
    const int64_t k0 = blockIdx.y * a.part, k1 = k0 + a.part < a.k ? k0 + a.part : a.k;
    float acc[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) acc[i] = 0.f;
    for (int64_t kk = k0 + wave * 128 + (lane & 15) * 8; kk < k1; kk += 512) {
        const u32x4 xv = *reinterpret_cast<const u32x4 *>(x + kk);
        u32x4 wv[ROWS];
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            wv[i] = u32x4{0, 0, 0, 0};
            if (4 * i + g < a.rank) wv[i] = *reinterpret_cast<const u32x4 *>(w + (4 * i + g) * a.k + kk);
        }
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                acc[i] = __builtin_fmaf(bf16_lo(wv[i][e]), bf16_lo(xv[e]), acc[i]);
                acc[i] = __builtin_fmaf(bf16_hi(wv[i][e]), bf16_hi(xv[e]), acc[i]);
            }
    }
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
#pragma unroll
        for (int off = 8; off >= 1; off >>= 1) acc[i] += __shfl_xor(acc[i], off, 64);
        if ((lane & 15) == 0) lds[wave][4 * i + g] = acc[i];
    }
    __syncthreads();
    if (tid < a.rank)
        a.h[(blockIdx.y * a.m + t) * a.rank + tid] = (lds[0][tid] + lds[1][tid]) + (lds[2][tid] + lds[3][tid]);
}

template <int FMT>
__device__ __forceinline__ float get(const void *p, int64_t i) {
    if constexpr (FMT == WSL_OUT_F32) return static_cast<const float *>(p)[i];
    return bf16_lo(static_cast<const uint16_t *>(p)[i]);
}
template <int FMT>
__device__ __forceinline__ void put(void *p, int64_t i, float v) {
    if constexpr (FMT == WSL_OUT_F32) static_cast<float *>(p)[i] = v;
    else static_cast<uint16_t *>(p)[i] = static_cast<uint16_t>(pack_bf16x2(v, v));
}

template <int FMT>
__device__ __forceinline__ void copy1(void *to, int64_t i, const void *from, int64_t j) {
    if constexpr (FMT == WSL_OUT_F32) static_cast<uint32_t *>(to)[i] = static_cast<const uint32_t *>(from)[j];
    else static_cast<uint16_t *>(to)[i] = static_cast<const uint16_t *>(from)[j];
}

// blockIdx: (token, 256 outputs); a lane's row of B is rank * 2 bytes in one piece.
template <int FMT>
__global__ __launch_bounds__(256) void expand_few_kernel(LoraArgs a) {
    __shared__ float h[128];
    const int64_t t = blockIdx.x, n = static_cast<int64_t>(blockIdx.y) * 256 + threadIdx.x;
    const int tid = static_cast<int>(threadIdx.x);
    const int32_t id = adapter_of(a, t, false);
    if (id < 0 && a.base == a.out) return;
    if (id >= 0 && tid < a.rank) {
        float v = 0;
        for (int p = 0; p < a.parts; ++p) v += a.h[(p * a.m + t) * a.rank + tid];
        h[tid] = a.scales ? a.scales[id] * v : v;
    }
    __syncthreads();
    if (n >= a.n_out) return;
    if (id < 0) {
        copy1<FMT>(a.out, t * a.ld_out + n, a.base, t * a.ld_base + n);
        return;
    }
    const u32x4 *w = reinterpret_cast<const u32x4 *>(a.b + (id * a.n_out + n) * a.rank);
    float y = 0;
    for (int r = 0; r < a.rank; r += 8) {
        const u32x4 v = w[r / 8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            y = __builtin_fmaf(bf16_lo(v[e]), h[r + 2 * e], y);
            y = __builtin_fmaf(bf16_hi(v[e]), h[r + 2 * e + 1], y);
        }
    }
    put<FMT>(a.out, t * a.ld_out + n, get<FMT>(a.base, t * a.ld_base + n) + y);
}

// ------------------------------------------------------------------ more tokens
__device__ __forceinline__ bf16x8 frag(u32x4 v) { return __builtin_bit_cast(bf16x8, v); }

// blockIdx: (64 tokens, part of k); a wave's 16 tokens are the rows, 16 rows of A the columns.
template <int BLOCKS>
__global__ __launch_bounds__(256) void shrink_many_kernel(LoraArgs a) {
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wave = tid >> 6, col = lane & 15, g = lane >> 4;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * 64 + wave * 16;
    if (t0 >= a.m) return;
    const int64_t mine = t0 + col < a.m ? t0 + col : a.m - 1;
    const int32_t id = t0 + col < a.m ? adapter_of(a, mine, blockIdx.y == 0 && g == 0) : -1;
    const int64_t k0 = blockIdx.y * a.part, k1 = k0 + a.part < a.k ? k0 + a.part : a.k;
    const uint16_t *x = a.x + mine * a.ldx;
    uint32_t todo = static_cast<uint32_t>(__ballot(id >= 0)) & 0xffffu;
    while (todo) {
        const int32_t which = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
        const uint32_t same = static_cast<uint32_t>(__ballot(id == which)) & 0xffffu;
        todo &= ~same;
        const uint16_t *w = a.a + static_cast<int64_t>(which) * a.rank * a.k;
        f32x4 acc[BLOCKS];
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) acc[b] = f32x4{0, 0, 0, 0};
#pragma unroll 4
        for (int64_t kk = k0; kk < k1; kk += 32) {
            const int64_t at = kk + g * 8;
            u32x4 xv = {0, 0, 0, 0};
            if (at < k1) xv = *reinterpret_cast<const u32x4 *>(x + at);
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b) {
                u32x4 wv = {0, 0, 0, 0};
                if (at < k1 && 16 * b + col < a.rank) wv = *reinterpret_cast<const u32x4 *>(w + (16 * b + col) * a.k + at);
                acc[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(xv), frag(wv), acc[b], 0, 0, 0);
            }
        }
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if ((same >> (4 * g + i) & 1u) && 16 * b + col < a.rank)
                    a.h[(blockIdx.y * a.m + t0 + 4 * g + i) * a.rank + 16 * b + col] = acc[b][i];
    }
}

// x = hi + mid + lo, each a bf16 number: part p of it.
__device__ __forceinline__ float third(float x, int p) {
    const float hi = bf16_lo(pack_bf16x2(x, x));
    if (p == 0) return hi;
    if (!(__builtin_fabsf(hi) < __builtin_huge_valf())) return 0.f;        // infinite: hi alone
    const float rest = x - hi, mid = bf16_lo(pack_bf16x2(rest, rest));
    return p == 1 ? mid : rest - mid;
}

// blockIdx: (64 tokens, outputs).  The products run over (part of h, rank), 32 at a time.  Rows: 16
// outputs, columns: a wave's 16 tokens; the outputs of four products are shuffled so that a lane ends
// up with 16 successive ones of its token.
template <int FMT, int STEPS>
__global__ __launch_bounds__(256) void expand_many_kernel(LoraArgs a, int64_t each) {
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wave = tid >> 6, col = lane & 15, g = lane >> 4;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * 64 + wave * 16;
    if (t0 >= a.m) return;
    const bool there = t0 + col < a.m;
    const int64_t t = there ? t0 + col : a.m - 1;
    const int32_t id = there ? adapter_of(a, t, false) : -1;
    const uint32_t some = static_cast<uint32_t>(__ballot(id >= 0)) & 0xffffu;
    if (!some && a.base == a.out) return;
    u32x4 h[STEPS];
    int at[STEPS];
    const float scale = id >= 0 && a.scales ? a.scales[id] : 1.f;
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int slot = 32 * s + 8 * g, p = slot / a.rank, r = slot - p * a.rank;
        at[s] = p < 3 ? r : 0;
        float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (id >= 0 && p < 3)
            for (int c = 0; c < a.parts; ++c) {
                const float *from = a.h + (c * a.m + t) * a.rank + r;
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] += from[e];
            }
#pragma unroll
        for (int e = 0; e < 4; ++e) h[s][e] = pack_bf16x2(third(scale * v[2 * e], p), third(scale * v[2 * e + 1], p));
    }
    const int64_t n0 = blockIdx.y * each, n1 = n0 + each < a.n_out ? n0 + each : a.n_out;
    for (int64_t n = n0; n < n1; n += 64) {
        f32x4 acc[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[q] = f32x4{0, 0, 0, 0};
        uint32_t todo = some;
        while (todo) {
            const int32_t which = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
            todo &= ~static_cast<uint32_t>(__ballot(id == which));
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int64_t row = n + (col >> 2) * 16 + q * 4 + (col & 3);
                const uint16_t *w = a.b + (which * a.n_out + (row < a.n_out ? row : a.n_out - 1)) * a.rank;
                f32x4 d = {0, 0, 0, 0};
#pragma unroll
                for (int s = 0; s < STEPS; ++s)
                    d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(*reinterpret_cast<const u32x4 *>(w + at[s])),
                                                                frag(h[s]), d, 0, 0, 0);
                if (id == which) acc[q] = d;           // whatever this adapter makes of other tokens is left
            }
        }
        if (!there) continue;
        const int64_t mine = n + g * 16;
        const int64_t from = t * a.ld_base + mine, to = t * a.ld_out + mine;
        if (a.wide && mine + 16 <= a.n_out) {
            constexpr int kWide = FMT == WSL_OUT_F32 ? 4 : 2, kSize = FMT == WSL_OUT_F32 ? 4 : 2;
            const u32x4 *in = reinterpret_cast<const u32x4 *>(static_cast<const char *>(a.base) + from * kSize);
            u32x4 *out = reinterpret_cast<u32x4 *>(static_cast<char *>(a.out) + to * kSize), v[kWide];
#pragma unroll
            for (int q = 0; q < kWide; ++q) v[q] = in[q];
            if (id >= 0) {
#pragma unroll
                for (int q = 0; q < kWide; ++q)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t w = v[q][e];
                        if constexpr (FMT == WSL_OUT_F32)
                            v[q][e] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, w) + acc[q][e]);
                        else
                            v[q][e] = pack_bf16x2(bf16_lo(w) + acc[2 * q + e / 2][2 * (e % 2)],
                                                  bf16_hi(w) + acc[2 * q + e / 2][2 * (e % 2) + 1]);
                    }
            }
#pragma unroll
            for (int q = 0; q < kWide; ++q) out[q] = v[q];
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if (mine + 4 * q + i < a.n_out) {
                        if (id >= 0) put<FMT>(a.out, to + 4 * q + i, get<FMT>(a.base, from + 4 * q + i) + acc[q][i]);
                        else copy1<FMT>(a.out, to + 4 * q + i, a.base, from + 4 * q + i);
                    }
        }
    }
}

// Parts of k: few tokens, as many as there are kPart elements; more, until there are enough workgroups.
int64_t parts_of(int64_t m, int64_t k) {
    int64_t most = kMostParts;
    if (m > kFewTokens) {
        const int64_t tiles = (m + 63) / 64;
        most = (512 + tiles - 1) / tiles;
        if (most > kMostParts) most = kMostParts;
    }
    const int64_t parts = (k + kPart - 1) / kPart;
    return parts < most ? parts : most;
}

template <int FMT>
void go_expand(const LoraArgs &a, hipStream_t s) {
    if (a.m <= kFewTokens) {
        hipLaunchKernelGGL(expand_few_kernel<FMT>, dim3(static_cast<unsigned>(a.m), static_cast<unsigned>((a.n_out + 255) / 256)),
                           dim3(256), 0, s, a);
        return;
    }
    const int64_t each = 512;
    const dim3 grid(static_cast<unsigned>((a.m + 63) / 64), static_cast<unsigned>((a.n_out + each - 1) / each));
    const int steps = (3 * a.rank + 31) / 32;
    if (steps <= 2) hipLaunchKernelGGL((expand_many_kernel<FMT, 2>), grid, dim3(256), 0, s, a, each);
    else if (steps <= 3) hipLaunchKernelGGL((expand_many_kernel<FMT, 3>), grid, dim3(256), 0, s, a, each);
    else if (steps <= 6) hipLaunchKernelGGL((expand_many_kernel<FMT, 6>), grid, dim3(256), 0, s, a, each);
    else hipLaunchKernelGGL((expand_many_kernel<FMT, 12>), grid, dim3(256), 0, s, a, each);
}

}  // namespace

size_t lora_ws_bytes(int64_t m, int64_t rank, int64_t k) {
    return static_cast<size_t>(parts_of(m, k)) * static_cast<size_t>(m) * static_cast<size_t>(rank) * sizeof(float);
}

int launch_lora(const void *d_a, const void *d_b, int64_t n_adapters, int64_t rank, int64_t n_out, int64_t k,
                const int32_t *ids, const float *scales, const void *x, int64_t m, int64_t ldx, const void *base,
                int64_t ld_base, void *out, int64_t ld_out, int fmt, void *ws, uint32_t *status, hipStream_t s) {
    LoraArgs a;
    a.a = static_cast<const uint16_t *>(d_a), a.b = static_cast<const uint16_t *>(d_b);
    a.x = static_cast<const uint16_t *>(x);
    a.ids = ids, a.scales = scales, a.base = base, a.out = out, a.h = static_cast<float *>(ws), a.status = status;
    a.n_adapters = n_adapters, a.n_out = n_out, a.k = k, a.m = m, a.ldx = ldx, a.ld_base = ld_base, a.ld_out = ld_out;
    a.rank = static_cast<int32_t>(rank);
    const int64_t parts = parts_of(m, k);
    a.part = ((k + parts - 1) / parts + kPart - 1) / kPart * kPart;
    a.parts = static_cast<int32_t>((k + a.part - 1) / a.part);
    const int64_t step = fmt == WSL_OUT_F32 ? 4 : 8;
    a.wide = ld_base % step == 0 && ld_out % step == 0 && reinterpret_cast<uintptr_t>(base) % 16 == 0 &&
             reinterpret_cast<uintptr_t>(out) % 16 == 0;
    if (m <= kFewTokens) {
        const dim3 grid(static_cast<unsigned>(m), static_cast<unsigned>(a.parts));
        if (rank <= 8) hipLaunchKernelGGL(shrink_few_kernel<2>, grid, dim3(256), 0, s, a);
        else if (rank <= 16) hipLaunchKernelGGL(shrink_few_kernel<4>, grid, dim3(256), 0, s, a);
        else if (rank <= 32) hipLaunchKernelGGL(shrink_few_kernel<8>, grid, dim3(256), 0, s, a);
        else if (rank <= 64) hipLaunchKernelGGL(shrink_few_kernel<16>, grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL(shrink_few_kernel<32>, grid, dim3(256), 0, s, a);
    } else {
        const dim3 grid(static_cast<unsigned>((m + 63) / 64), static_cast<unsigned>(a.parts));
        if (rank <= 16) hipLaunchKernelGGL(shrink_many_kernel<1>, grid, dim3(256), 0, s, a);
        else if (rank <= 32) hipLaunchKernelGGL(shrink_many_kernel<2>, grid, dim3(256), 0, s, a);
        else if (rank <= 64) hipLaunchKernelGGL(shrink_many_kernel<4>, grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL(shrink_many_kernel<8>, grid, dim3(256), 0, s, a);
    }
    if (fmt == WSL_OUT_F32) go_expand<WSL_OUT_F32>(a, s);
    else go_expand<WSL_OUT_BF16>(a, s);
    return WSL_OK;
}

}  // namespace wsl
