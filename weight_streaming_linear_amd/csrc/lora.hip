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
// Bound: base and out once each, x, and A and B of the adapters in use.  Measured, launches behind one another in a graph (as all
// figures here, fp32 and on inputs that the caches may hold): one token, 5120 to 5120, rank 16, 6.1 us (3 and 3; half of it is the
// launches); 48 tokens of 7168 to 5120, 24 adapters, 7.5; 4224 tokens of 6144 to 5120, 21 adapters, 50.2 (225 MB of x, base and
// out: 4.5 TB/s); rank 64, 78.5.  Rows of base and out that are not 16-byte aligned go an element at a time: 4224 tokens
// of 6144, 12 adapters, to 6144 outputs 52.5, to 6145 148; in bf16 37.5 and 157.
#include "device_common.h"

namespace wsl {
namespace {

// Tokens one by one up to here.  That costs by the tokens, and adapters that caches do not hold; tiles of 16 cost by the adapters among
// them, which the host does not know.  5120 to 5120, one against the other, in us: tokens with an adapter each, rank 16: 14 and
// 44 for 128, 34 and 51 for 512, 85 and 107 for 1024; requests of 200 tokens: 8.8 and 10.2, 20.3 and 14.1, 36 and 20.  Rank 64: 41.5
// and 94.5 for 128, 82 and 148 for 256; requests: 23.4 and 14.3, 38.5 and 17.7.  So next to the border either side loses up to twice for
// some ids.
constexpr int64_t kFewRows = 8192;         // m * rank
bool few(int64_t m, int64_t rank) { return m * rank <= kFewRows; }
// Least elements of k in a part; more only add partial sums to write and read.  512 against 1024, in us: one token of 5120, rank 16:
// 6.4 and 6.1; 48 tokens of 7168: 8.9 and 7.5; 128 of 5120: 15.3 and 14.0; 1024 in requests: 20.1 and 20.1; but 256 with 128 adapters,
// rank 64: 91 and 97.
constexpr int kPart = 1024;
// Parts at most.  8, 16 and 32, 14336 to 5120, rank 64: one token 13.0, 12.7 and 12.7; 8 tokens 11.9, 10.5 and 10.5.
constexpr int64_t kMostParts = 16;
// Workgroups of 16 tokens that keep the chip busy: one a CU.  128, 256 and 512: 600 tokens, 5120 to 5120, rank 16: 15.3, 14.8 and
// 14.9; 2048: 30.0, 29.1 and 30.3; 1024 of 14336, rank 64: 42.9, 37.4 and 40.5.
constexpr int64_t kGroups = 256;
constexpr int kXcds = 8;                   // (another number costs locality alone)
constexpr int64_t kMostTiles = 32768;      // of 16 tokens along a grid's y, which ends at 65535

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

// 16 rows of C * 8 elements, by one wave: from C lanes a row, as they are loaded, to the operands of C / 4 products (a row
// to 16 lanes; as loads those would be 64 pieces of 16 bytes, which take four times as long to ask for).
template <int C>
struct Turn {
    static constexpr int kLoads = C / 4, kRows = 64 / C;       // rows of a load
    u32x4 at[16 * (C + 1)];                        // a row and 16 bytes: no two rows in the same banks
    static __device__ __forceinline__ int row(int load) { return load * kRows + static_cast<int>(threadIdx.x & 63) / C; }
    static __device__ __forceinline__ int element() { return static_cast<int>(threadIdx.x) % C * 8; }
    __device__ __forceinline__ void operator()(u32x4 (&v)[kLoads]) {
        const int lane = static_cast<int>(threadIdx.x & 63), col = lane & 15, g = lane >> 4;
        // (the wave's own, in order: what was read before is out before this comes in)
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int i = 0; i < kLoads; ++i) at[row(i) * (C + 1) + lane % C] = v[i];
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
        __builtin_amdgcn_wave_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
#pragma unroll
        for (int s = 0; s < kLoads; ++s) v[s] = at[col * (C + 1) + 4 * s + g];
    }
};

// A workgroup: 16 tokens and a part of k, those of an XCD in turn so that its L2 holds what they have of A (4224 tokens of 6144, 21
// adapters, rank 16, 55.3 -> 50.2 us, the whole; rank 64, 96 -> 78.5).  The tokens
// are the rows, 16 rows of A the columns; the waves take 128 elements of k in turn, all of their loads made
// before the first product, and are added up in LDS, so that one part is enough where tokens are many.
template <int BLOCKS, int WAVES>
__global__ __launch_bounds__(WAVES * 64) void shrink_many_kernel(LoraArgs a) {
    __shared__ union {
        Turn<16> turn[WAVES];
        f32x4 sums[WAVES][BLOCKS][64];
    } lds;
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, col = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t at = (blockIdx.x % kXcds) * (gridDim.x / kXcds) + blockIdx.x / kXcds;
    const uint32_t tiles = static_cast<uint32_t>((a.m + 15) / 16), part = at / tiles;
    if (part >= static_cast<uint32_t>(a.parts)) return;
    const int64_t t0 = static_cast<int64_t>(at - part * tiles) * 16;
    const bool there = t0 + col < a.m;
    const int32_t id = there ? adapter_of(a, t0 + col, part == 0 && tid < 16) : -1;
    const int64_t k0 = part * a.part, k1 = k0 + a.part < a.k ? k0 + a.part : a.k;
    const auto token = [&](int row) { return t0 + row < a.m ? t0 + row : a.m - 1; };
    const uint16_t *x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = a.x + token(4 * i + g) * a.ldx + col * 8;
    const uint32_t lane_at = static_cast<uint32_t>(g * a.k + col * 8) * 2;     // k < 2^22
    uint32_t todo = static_cast<uint32_t>(__ballot(id >= 0)) & 0xffffu;
    while (todo) {
        // two adapters at a time: most tiles where requests meet have two
        int32_t which[2];
        uint32_t same[2] = {0, 0};
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            which[p] = p ? which[0] : -1;
            if (todo) {
                which[p] = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
                same[p] = static_cast<uint32_t>(__ballot(id == which[p])) & 0xffffu;
                todo &= ~same[p];
            }
        }
        f32x4 acc[2][BLOCKS];
#pragma unroll
        for (int b = 0; b < BLOCKS; ++b) acc[0][b] = acc[1][b] = f32x4{0, 0, 0, 0};
        int64_t kk = k0 + wave * 128;
        for (; kk + 128 <= k1; kk += 128 * WAVES) {
            constexpr int kOnce = BLOCKS < 2 ? BLOCKS : 2;     // (more have no room in the registers)
            u32x4 xv[4], wv[kOnce][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) xv[i] = *reinterpret_cast<const u32x4 *>(x[i] + kk);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                if (!same[p]) continue;
                // rows behind the rank (8 of 16, or blocks of them) are read again and not kept
                const char *w = reinterpret_cast<const char *>(a.a + static_cast<int64_t>(which[p]) * a.rank * a.k + kk);
#pragma unroll
                for (int b0 = 0; b0 < BLOCKS; b0 += kOnce) {
#pragma unroll
                    for (int b = 0; b < kOnce; ++b)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int row = 16 * (b0 + b) + 4 * i;
                            wv[b][i] = *reinterpret_cast<const u32x4 *>(w + (row < a.rank ? row : 0) * a.k * 2 + lane_at);
                        }
                    if (p == 0 && b0 == 0) lds.turn[wave](xv);
#pragma unroll
                    for (int b = 0; b < kOnce; ++b) {
                        lds.turn[wave](wv[b]);
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            acc[p][b0 + b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(xv[s]), frag(wv[b][s]), acc[p][b0 + b], 0, 0, 0);
                    }
                }
            }
        }
        for (; kk < k1; kk += 32) {                // fewer than 128 left: this wave's alone, and read as it is needed
            const bool in = kk + g * 8 < k1;
            u32x4 xv = {0, 0, 0, 0};
            if (in) xv = *reinterpret_cast<const u32x4 *>(a.x + token(col) * a.ldx + kk + g * 8);
#pragma unroll
            for (int p = 0; p < 2; ++p) {
                const uint16_t *w = a.a + static_cast<int64_t>(which[p]) * a.rank * a.k + kk + g * 8;
#pragma unroll
                for (int b = 0; b < BLOCKS; ++b) {
                    u32x4 wv = {0, 0, 0, 0};
                    if (in) wv = *reinterpret_cast<const u32x4 *>(w + (16 * b + col < a.rank ? 16 * b + col : 0) * a.k);
                    acc[p][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(xv), frag(wv), acc[p][b], 0, 0, 0);
                }
            }
        }
        __syncthreads();                           // the sums lie where the waves turn their rows
#pragma unroll
        for (int p = 0; p < 2; ++p) {
            if (!same[p]) continue;
#pragma unroll
            for (int b = 0; b < BLOCKS; ++b) lds.sums[wave][b][lane] = acc[p][b];
            __syncthreads();
            for (int b = wave; b < BLOCKS; b += WAVES) {
                f32x4 v = lds.sums[0][b][lane];
#pragma unroll
                for (int q = 1; q < WAVES; ++q) {
                    const f32x4 u = lds.sums[q][b][lane];
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] += u[i];
                }
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    if ((same[p] >> (4 * g + i) & 1u) && 16 * b + col < a.rank)
                        a.h[(part * a.m + t0 + 4 * g + i) * a.rank + 16 * b + col] = v[i];
            }
            __syncthreads();
        }
    }
}

// x = hi + mid + lo, each a bf16 number: part p of it.  hi is cut off: rounded, the finite numbers next to the largest
// would become infinite.  (A NaN is a quiet one here, its mark in the upper half.)
__device__ __forceinline__ float third(float x, int p) {
    const float hi = __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, x) & 0xffff0000u);
    if (p == 0) return hi;
    if (!(__builtin_fabsf(hi) < __builtin_huge_valf())) return 0.f;        // infinite: hi alone
    const float rest = x - hi, mid = bf16_lo(pack_bf16x2(rest, rest));
    return p == 1 ? mid : rest - mid;
}

// blockIdx: (outputs, 16 tokens): what runs together covers whole rows of base and out, and the parts of h are made
// once for the four waves (before, a wave had 16 tokens of its own: 1024 tokens, 5120 outputs, rank 64, 31.4 -> 21.7 us).  The products run over
// (part of h, rank), 32 at a time.  Rows: 16 outputs, columns: a wave's 16 tokens; the outputs of four products are
// shuffled so that a lane ends up with 16 successive bytes of its token's row for each access, the four lanes of a token
// with 64.  A wave has kTiles * 64 outputs, whose base it asks for before it knows its adapters: waiting for those, and
// for h, would otherwise take as long as the rest.  (B asked for as early takes registers for it, and half the
// waves.)  kTiles 1, 2 and 4, the whole call, to 5120, rank 16: 1024 tokens of 5120: 18.8, 20.0 and 23.3 us, 2048: 29.1, 29.2 and
// 28.6, 8192: 98.4, 95.5 and 99.6; 4224 of 6144: 51.4, 50.2 and 52.9; rank 64: 31.6, 29.8 and 34.4 for 1024, 78.2, 78.5 and 86.9 for
// 4224.  The rows
// of B that go with the three parts of h are the same: PERIOD of them are different (STEPS where the rank neither divides
// 32 nor is a multiple of it).
constexpr int kTiles = 2;
// The output of row i of product q: four successive rows make 16 bytes of fp32, those of two products 16 bytes of bf16.
template <int FMT>
__device__ __forceinline__ int output_of(int q, int i) {
    if constexpr (FMT == WSL_OUT_F32) return 16 * q + i;
    return (q >> 1) * 32 + (i >> 2) * 8 + (q & 1) * 4 + (i & 3);
}
template <int FMT, int STEPS, int PERIOD>
__global__ __launch_bounds__(256) void expand_many_kernel(LoraArgs a) {
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wave = tid >> 6, col = lane & 15, g = lane >> 4;
    const int64_t t0 = (static_cast<int64_t>(blockIdx.z) * kMostTiles + blockIdx.y) * 16;
    if (t0 >= a.m) return;
    constexpr bool kTurned = PERIOD > 1 && PERIOD < STEPS;     // rows of B are PERIOD * 32 elements
    __shared__ u32x4 shared[STEPS][64];
    __shared__ Turn<PERIOD * 4> turn[kTurned ? 4 : 1];
    constexpr int kWide = FMT == WSL_OUT_F32 ? 4 : 2, kSize = FMT == WSL_OUT_F32 ? 4 : 2;
    const bool there = t0 + col < a.m;
    const int64_t t = there ? t0 + col : a.m - 1, n0 = (static_cast<int64_t>(blockIdx.x) * 4 + wave) * (kTiles * 64);
    u32x4 v[kTiles][kWide];
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
        const int64_t n = n0 + 64 * i;
        if (a.wide && n + 64 <= a.n_out) {
            const u32x4 *in = reinterpret_cast<const u32x4 *>(static_cast<const char *>(a.base) + (t * a.ld_base + n) * kSize) + g;
#pragma unroll
            for (int q = 0; q < kWide; ++q) v[i][q] = in[4 * q];
        }
    }
    const int32_t id = there ? adapter_of(a, t, false) : -1;
    const uint32_t some = static_cast<uint32_t>(__ballot(id >= 0)) & 0xffffu;
    if (!some && a.base == a.out) return;
    const float scale = id >= 0 && a.scales ? a.scales[id] : 1.f;
    for (int s = wave; s < STEPS; s += 4) {
        const int slot = 32 * s + 8 * g, p = slot / a.rank;
        float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (id >= 0 && p < 3)
            for (int c = 0; c < a.parts; ++c) {
                const f32x4 *from = reinterpret_cast<const f32x4 *>(a.h + (c * a.m + t) * a.rank + slot - p * a.rank);
                const f32x4 lo = from[0], hi = from[1];
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] += lo[e], x[4 + e] += hi[e];
            }
        u32x4 w;
#pragma unroll
        for (int e = 0; e < 4; ++e) w[e] = pack_bf16x2(third(scale * x[2 * e], p), third(scale * x[2 * e + 1], p));
        shared[s][lane] = w;
    }
    __syncthreads();
    u32x4 h[STEPS];
    int at[STEPS];
#pragma unroll
    for (int s = 0; s < STEPS; ++s) {
        const int slot = 32 * s + 8 * g, p = slot / a.rank;
        at[s] = p < 3 || PERIOD < STEPS ? slot - p * a.rank : 0;
        h[s] = shared[s][lane];
    }
#pragma unroll
    for (int i = 0; i < kTiles; ++i) {
        const int64_t n = n0 + 64 * i;
        if (n >= a.n_out) break;
        f32x4 acc[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[q] = f32x4{0, 0, 0, 0};
        uint32_t todo = some;
        while (todo) {
            const int32_t which = __builtin_amdgcn_readlane(id, __builtin_ctz(todo));
            todo &= ~static_cast<uint32_t>(__ballot(id == which));
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const auto row_of = [&](int i) {
                    const int64_t row = n + output_of<FMT>(q, i);
                    return a.b + (which * a.n_out + (row < a.n_out ? row : a.n_out - 1)) * a.rank;
                };
                u32x4 b[PERIOD];
                if constexpr (kTurned) {
                    using T = Turn<PERIOD * 4>;
#pragma unroll
                    for (int s = 0; s < PERIOD; ++s) b[s] = *reinterpret_cast<const u32x4 *>(row_of(T::row(s)) + T::element());
                    turn[wave](b);
                } else {
                    const uint16_t *w = row_of(col);
#pragma unroll
                    for (int s = 0; s < PERIOD; ++s) b[s] = *reinterpret_cast<const u32x4 *>(w + at[s]);
                }
                f32x4 d = {0, 0, 0, 0};
#pragma unroll
                for (int s = 0; s < STEPS; ++s)
                    d = __builtin_amdgcn_mfma_f32_16x16x32_bf16(frag(b[s % PERIOD]), frag(h[s]), d, 0, 0, 0);
                if (id == which) acc[q] = d;           // whatever this adapter makes of other tokens is left
            }
        }
        if (there && a.wide && n + 64 <= a.n_out) {
            u32x4 *out = reinterpret_cast<u32x4 *>(static_cast<char *>(a.out) + (t * a.ld_out + n) * kSize) + g;
            if (id >= 0) {
#pragma unroll
                for (int q = 0; q < kWide; ++q)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t w = v[i][q][e];
                        if constexpr (FMT == WSL_OUT_F32)
                            v[i][q][e] = __builtin_bit_cast(uint32_t, __builtin_bit_cast(float, w) + acc[q][e]);
                        else
                            v[i][q][e] = pack_bf16x2(bf16_lo(w) + acc[2 * q + e / 2][2 * (e % 2)],
                                                     bf16_hi(w) + acc[2 * q + e / 2][2 * (e % 2) + 1]);
                    }
            }
#pragma unroll
            for (int q = 0; q < kWide; ++q) out[4 * q] = v[i][q];
        } else if (there) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (const int64_t row = n + output_of<FMT>(q, 4 * g + e); row < a.n_out) {
                        if (id >= 0) put<FMT>(a.out, t * a.ld_out + row, get<FMT>(a.base, t * a.ld_base + row) + acc[q][e]);
                        else copy1<FMT>(a.out, t * a.ld_out + row, a.base, t * a.ld_base + row);
                    }
        }
    }
}

// Parts of k: as many as there are kPart elements, of more tokens only until there are enough workgroups.
int64_t parts_of(int64_t m, int64_t rank, int64_t k) {
    int64_t most = kMostParts;
    if (!few(m, rank)) {
        const int64_t tiles = (m + 15) / 16;
        most = (kGroups + tiles - 1) / tiles;
        if (most > kMostParts) most = kMostParts;
    }
    const int64_t parts = (k + kPart - 1) / kPart;
    return parts < most ? parts : most;
}

template <int FMT>
void go_expand(const LoraArgs &a, hipStream_t s) {
    if (few(a.m, a.rank)) {
        hipLaunchKernelGGL(expand_few_kernel<FMT>, dim3(static_cast<unsigned>(a.m), static_cast<unsigned>((a.n_out + 255) / 256)),
                           dim3(256), 0, s, a);
        return;
    }
    const int64_t tiles = (a.m + 15) / 16;
    const dim3 grid(static_cast<unsigned>((a.n_out + kTiles * 256 - 1) / (kTiles * 256)), static_cast<unsigned>(tiles < kMostTiles ? tiles : kMostTiles),
                    static_cast<unsigned>((tiles + kMostTiles - 1) / kMostTiles));
    const auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, a); };
    const int rank = a.rank, steps = (3 * rank + 31) / 32;
    if (rank <= 8) go(expand_many_kernel<FMT, 1, 1>);
    else if (rank == 16) go(expand_many_kernel<FMT, 2, 1>);
    else if (rank == 32) go(expand_many_kernel<FMT, 3, 1>);
    else if (rank == 64) go(expand_many_kernel<FMT, 6, 2>);
    else if (rank == 128) go(expand_many_kernel<FMT, 12, 4>);
    else if (steps <= 6) go(expand_many_kernel<FMT, 6, 6>);
    else go(expand_many_kernel<FMT, 12, 12>);
}

}  // namespace

size_t lora_ws_bytes(int64_t m, int64_t rank, int64_t k) {
    // At least parts_of * m, and never less for more tokens: m times all parts of k while they go one by one; from there on parts_of is
    // below kGroups * 16 / m + 1.
    const int64_t parts = parts_of(1, rank, k), last = kFewRows / rank;
    int64_t sums = m * parts;
    if (!few(m, rank)) {
        if (sums > m + kGroups * 16) sums = m + kGroups * 16;
        if (sums < last * parts) sums = last * parts;
    }
    return static_cast<size_t>(sums) * static_cast<size_t>(rank) * sizeof(float);
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
    const int64_t parts = parts_of(m, rank, k);
    a.part = ((k + parts - 1) / parts + kPart - 1) / kPart * kPart;
    a.parts = static_cast<int32_t>((k + a.part - 1) / a.part);
    const int64_t vec = fmt == WSL_OUT_F32 ? 4 : 8;
    a.wide = ld_base % vec == 0 && ld_out % vec == 0 && reinterpret_cast<uintptr_t>(base) % 16 == 0 &&
             reinterpret_cast<uintptr_t>(out) % 16 == 0;
    if (few(m, rank)) {
        const dim3 grid(static_cast<unsigned>(m), static_cast<unsigned>(a.parts));
        if (rank <= 8) hipLaunchKernelGGL(shrink_few_kernel<2>, grid, dim3(256), 0, s, a);
        else if (rank <= 16) hipLaunchKernelGGL(shrink_few_kernel<4>, grid, dim3(256), 0, s, a);
        else if (rank <= 32) hipLaunchKernelGGL(shrink_few_kernel<8>, grid, dim3(256), 0, s, a);
        else if (rank <= 64) hipLaunchKernelGGL(shrink_few_kernel<16>, grid, dim3(256), 0, s, a);
        else hipLaunchKernelGGL(shrink_few_kernel<32>, grid, dim3(256), 0, s, a);
    } else {
        const dim3 grid(static_cast<unsigned>(((m + 15) / 16 * a.parts + kXcds - 1) / kXcds * kXcds));
        if (rank <= 16) hipLaunchKernelGGL((shrink_many_kernel<1, 8>), grid, dim3(512), 0, s, a);
        else if (rank <= 32) hipLaunchKernelGGL((shrink_many_kernel<2, 8>), grid, dim3(512), 0, s, a);
        else if (rank <= 64) hipLaunchKernelGGL((shrink_many_kernel<4, 8>), grid, dim3(512), 0, s, a);
        else hipLaunchKernelGGL((shrink_many_kernel<8, 8>), grid, dim3(512), 0, s, a);
    }
    if (fmt == WSL_OUT_F32) go_expand<WSL_OUT_F32>(a, s);
    else go_expand<WSL_OUT_BF16>(a, s);
    return WSL_OK;
}

}  // namespace wsl
