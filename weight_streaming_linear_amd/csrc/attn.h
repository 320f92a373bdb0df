// What the host side of attn_decode tells its kernels, and the split of the work that the
// attention kernel and the joining kernel both derive from it.
#pragma once

#include "device_common.h"

namespace wsl {

constexpr int kAttnWaves = 4;                      // waves of a workgroup
constexpr int kAttnSub = 32;                       // tokens a wave takes at a time
constexpr int kAttnTile = kAttnWaves * kAttnSub;   // tokens a workgroup takes at a time
constexpr int kAttnThreads = kAttnWaves * 64;

struct AttnArgs {
    const char *k, *v;
    const uint8_t *ke, *ve;
    const void *q;
    void *out;
    float *lse;
    float *part_o;        // [2 * workers][tile_rows][head_dim]: unnormalised sums
    float2 *part_ml;      // [2 * workers][tile_rows]: running maximum (log2 domain) and sum
    const int32_t *table, *lens;
    uint32_t *status;
    int64_t page_stride, head_stride, token_stride;   // bytes
    int64_t ld_q, ld_out, ld_table;                   // elements
    int64_t window, capacity;                         // capacity: tokens a table row can name
    float scale_log2;
    int32_t n_seq, q_len, n_kv, group, rows, head_dim, page_size, n_pages;
    int32_t row_tiles, tile_rows, workers, qfmt, ofmt;
};

// A sequence's length and the token tiles that some row of it sees.  A sequence with nothing to see
// has one tile, whose worker writes its empty rows.
struct AttnSpan {
    int32_t len, first, tiles;
    bool bad;
};

__device__ __forceinline__ AttnSpan attn_span(const AttnArgs &a, int32_t seq) {
    AttnSpan s;
    const int32_t raw = a.lens[seq];
    s.bad = raw < 0 || raw > a.capacity;
    s.len = raw < 0 ? 0 : (raw > a.capacity ? static_cast<int32_t>(a.capacity) : raw);
    s.first = 0;
    if (a.window > 0) {
        const int64_t lo = static_cast<int64_t>(s.len) - a.q_len - a.window + 1;
        if (lo > 0) s.first = static_cast<int32_t>(lo / kAttnTile);
    }
    const int32_t n = (s.len + kAttnTile - 1) / kAttnTile - s.first;
    s.tiles = n > 0 ? n : 1;
    return s;
}

// Token tiles of all sequences in order.  Every workgroup adds them up for itself (the lengths
// are on the device): thread i takes `each` successive sequences.  lds: 4 int64.
struct AttnPlan {
    int64_t before, mine, total;   // tiles before this thread's sequences, in them, in all
    int32_t each;
};

__device__ __forceinline__ AttnPlan attn_plan(const AttnArgs &a, int64_t *lds) {
    AttnPlan p;
    const int tid = static_cast<int>(threadIdx.x), lane = tid & 63, wave = tid >> 6;
    p.each = (a.n_seq + kAttnThreads - 1) / kAttnThreads;
    p.mine = 0;
    for (int32_t i = 0; i < p.each; ++i) {
        const int64_t b = static_cast<int64_t>(tid) * p.each + i;
        if (b < a.n_seq) p.mine += attn_span(a, static_cast<int32_t>(b)).tiles;
    }
    int64_t run = p.mine;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
        const int64_t o = __shfl_up(run, off, 64);
        if (lane >= off) run += o;
    }
    if (lane == 63) lds[wave] = run;
    __syncthreads();
    p.before = run - p.mine;
    p.total = 0;
    for (int i = 0; i < kAttnWaves; ++i) {
        if (i < wave) p.before += lds[i];
        p.total += lds[i];
    }
    __syncthreads();
    return p;
}

// Worker w takes the global tiles [total * w / workers, total * (w + 1) / workers), with no more
// workers than tiles, so that none is empty.
__device__ __forceinline__ int64_t attn_workers(const AttnArgs &a, int64_t total) {
    return total < a.workers ? total : a.workers;
}
__device__ __forceinline__ int64_t attn_start(int64_t total, int64_t w, int64_t workers) { return total * w / workers; }
__device__ __forceinline__ int64_t attn_worker(int64_t total, int64_t x, int64_t workers) {
    return ((x + 1) * workers - 1) / total;
}

__device__ __forceinline__ void attn_store(const AttnArgs &a, int64_t at, float4 o) {
    if (a.ofmt == WSL_OUT_F32)
        *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = o;
    else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at) =
            make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
}

// Row `row` (query position row / group, head h * group + row % group) of a sequence is done:
// o and l are its sums, m the maximum they are relative to.
__device__ __forceinline__ void attn_finish(const AttnArgs &a, int32_t seq, int32_t len, int32_t h, int32_t row,
                                            int32_t d, float4 o, float m, float l) {
    const int32_t i = row / a.group, head = h * a.group + row - i * a.group;
    const int64_t tok = static_cast<int64_t>(seq) * a.q_len + i;
    const bool seen = len - a.q_len + i >= 0;       // else no token is visible: zeros, not 0 / 0
    const float r = 1.f / l;
    o.x = seen ? o.x * r : 0.f, o.y = seen ? o.y * r : 0.f, o.z = seen ? o.z * r : 0.f, o.w = seen ? o.w * r : 0.f;
    attn_store(a, tok * a.ld_out + static_cast<int64_t>(head) * a.head_dim + d, o);
    if (a.lse != nullptr && d == 0)
        a.lse[tok * (a.n_kv * a.group) + head] =
            seen ? (m + __builtin_amdgcn_logf(l)) * 0.69314718055994530942f : -__builtin_huge_valf();
}

template <int FMT>
int launch_attn_fmt(const AttnArgs &a, int tiles_m, hipStream_t s);

}  // namespace wsl
