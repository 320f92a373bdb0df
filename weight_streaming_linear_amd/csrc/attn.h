// What the host side of attn_decode tells its kernels, and the split of the work among workgroups.
#pragma once

#include "device_common.h"

namespace wsl {

constexpr int kAttnWaves = 4;                      // waves of a workgroup
constexpr int kAttnSub = 32;                       // tokens a wave takes at a time
constexpr int kAttnTile = kAttnWaves * kAttnSub;   // tokens a workgroup takes at a time
constexpr int kAttnThreads = kAttnWaves * 64;
constexpr int kAttnCus = 256;
constexpr int kAttnMaxWaves = 3;                   // of a SIMD, over all variants
constexpr int64_t kAttnMaxTokens = 0x7fffffff - 4 * kAttnTile;   // positions stay in 32 bits some rounds past the end
constexpr int kAttnJoinRows = 4;                   // rows a workgroup of the joining kernel takes

// What became of an item: the worker that began it and how many workers hold parts of it.
struct AttnOpen {
    int32_t seq, head, worker, parts;
};

// Division of a number n < 2^31 by one that the host knows, 1 <= by <= 2^30: with 2^shift the least
// power of two >= by and mul = floor(2^32 (2^shift - by) / by) + 1, n / by = (n mul / 2^32 + n) >> shift.
// (32 ragged sequences over e4m3 43.4 -> 42.4 us against the hardware's steps for a division.)
struct AttnDiv {
    uint32_t mul, shift;
};
inline AttnDiv attn_div(uint32_t by) {
    AttnDiv d = {1, 0};
    while ((uint32_t(1) << d.shift) < by) ++d.shift;
    d.mul = static_cast<uint32_t>((((uint64_t(1) << d.shift) - by) << 32) / by + 1);
    return d;
}
__device__ __forceinline__ uint32_t attn_over(uint32_t n, const AttnDiv &d) { return (__umulhi(n, d.mul) + n) >> d.shift; }

// Two blocks of 16 rows in a workgroup at one time: where the registers allow (figures: blocks_of).
constexpr bool attn_two_blocks(int fmt, int qfmt, int64_t head_dim) {
    if (qfmt == WSL_OUT_BF16) return head_dim <= (fmt == WSL_KV_BF16 ? 192 : 128);
    return fmt == WSL_KV_BF16 && head_dim > 64 && head_dim <= 128;
}

struct AttnArgs {
    AttnDiv over_page, over_group, over_heads;
    const char *k, *v;
    const uint8_t *ke, *ve;
    const void *q;
    void *out;
    float *lse;
    float *part_o;        // [row_tiles][2 * workers][tile_rows][head_dim]: unnormalised sums
    float2 *part_ml;      // [row_tiles][2 * workers][tile_rows]: running maximum (log2 domain) and sum
    AttnOpen *open;       // of each item, or of the last one that each worker began; null if nothing can be split
    const int32_t *table, *lens;
    uint32_t *status;
    int64_t page_stride, head_stride, token_stride;   // bytes
    int64_t ld_q, ld_out, ld_table;                   // elements
    float scale_log2;
    int32_t window;       // below capacity: attn_window
    int32_t capacity;     // tokens a table row can name
    int32_t n_seq, q_len, n_kv, group, rows, head_dim, page_size, n_pages;
    int32_t row_tiles, tile_rows, workers, qfmt, ofmt;
    int32_t whole;        // a workgroup takes one whole item
    int32_t by_item;      // how `open` is indexed: by whichever there are fewer of
};

// A sequence's length and the token tiles that some row of it sees.  A sequence with nothing to see
// has one tile, whose worker writes its empty rows.
struct AttnSpan {
    int32_t len, first, tiles;
    bool bad;
};

// A window as the kernels take it: one that reaches back over all that a table row can name is none (0),
// so that positions less any other stay in 32 bits.
inline int32_t attn_window(int64_t window, int64_t capacity) {
    static_assert(kAttnMaxTokens + 256 <= 0x7fffffff, "a query may stand at up to 256 before the first token");
    capacity = capacity < kAttnMaxTokens ? capacity : kAttnMaxTokens;
    return window < capacity ? static_cast<int32_t>(window) : 0;
}

// The lowest position that some row of a sequence of `len` tokens sees.
__device__ __forceinline__ int32_t attn_lowest(const AttnArgs &a, int32_t len) {
    const int32_t lo = len - a.q_len - a.window + 1;
    return a.window > 0 && lo > 0 ? lo : 0;
}

__device__ __forceinline__ AttnSpan attn_span(const AttnArgs &a, int32_t raw) {
    AttnSpan s;
    s.bad = raw < 0 || raw > a.capacity;
    s.len = raw < 0 ? 0 : (raw > a.capacity ? a.capacity : raw);
    s.first = attn_lowest(a, s.len) / kAttnTile;
    const int32_t n = (s.len + kAttnTile - 1) / kAttnTile - s.first;
    s.tiles = n > 0 ? n : 1;
    return s;
}

// The work of all items in order, an item being a (sequence, kv head): a sequence's first head, its
// next, then the next sequence's.  An item is kAttnCost + tiles units long: the first kAttnCost stand
// for its beginning and end, which a worker spends about as long on as on so many tiles.  Worker w
// takes `each` successive units from w * each on, with the least `each` for which the workers suffice.
// Where equal shares of tiles alone end with the items, or are a tile or two, there is nothing to weigh
// up (cost 0).  (16 sequences of up to 4224 tokens with five queries 29.6 us at cost 0, 29.1, 27.6, 27.5,
// 28.1 and 28.8 at 1, 2, 3, 4 and 6, in e4m3 27.9, 27.0, 25.5, 25.4, 25.2 and 26.1; 32 of up to 8192 76.2,
// 73.4, 73.8, 75.3, 76.3 and 77.3, in e4m3 43.0, 42.7, 42.3, 42.9, 43.2 and 44.7.)
// A few long items are not cut finer than two tiles where that leaves a worker for most compute units:
// half as many parts are to be joined.  That is so over e4m3 alone: over bf16 there are as many workers as
// compute units, and such items have two tiles each anyway.  (One sequence of 8192 tokens, 8 kv heads, in
// e4m3 14.0 -> 12.4 us, two of 4096 13.1 -> 12.5, one of 12000 with heads of 64 13.9 -> 13.1, of 6000 13.5 ->
// 13.9.)
// The lengths are on the device, so every wave works this out for itself: without LDS or barriers,
// each lane adds up the units of `per` successive sequences, a scan over the lanes finds the lane whose
// sequences hold the wanted unit, and its sequences are divided among the lanes again until one is left.
constexpr int kAttnCost = 2;
struct AttnPlan {
    int32_t total, each;      // units in all; of a worker
    int32_t cost;             // units of an item that are not tiles
    int32_t seq, before;      // the worker's first sequence and the units (of one head) before it
    int32_t lens;             // of up to 64 sequences: lane l holds the length of sequence l
};

// Length of a sequence, the same for the whole wave.
__device__ __forceinline__ int32_t attn_len(const AttnArgs &a, const AttnPlan &p, int32_t seq) {
    return a.n_seq <= 64 && !a.whole ? __builtin_amdgcn_readlane(p.lens, seq) : __builtin_amdgcn_readfirstlane(a.lens[seq]);
}

// Sums over lanes 0 .. l, by moves inside the rows of 16 lanes and from row to row.
template <int CTRL, int ROWS>
__device__ __forceinline__ int32_t attn_lanes_add(int32_t v) {
    return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xf, false);
}
__device__ __forceinline__ int32_t attn_lanes_before(int32_t v) {
    v = attn_lanes_add<0x111, 0xf>(v);      // from 1, 2, 4 and 8 lanes before in the row
    v = attn_lanes_add<0x112, 0xf>(v);
    v = attn_lanes_add<0x114, 0xf>(v);
    v = attn_lanes_add<0x118, 0xf>(v);
    v = attn_lanes_add<0x142, 0xa>(v);      // rows 1 and 3: the row before's last lane
    return attn_lanes_add<0x143, 0xc>(v);   // rows 2 and 3: lane 31
}

__device__ __forceinline__ int32_t attn_lane_units(const AttnArgs &a, int32_t first, int32_t count, int32_t per,
                                                   int32_t cost, int32_t &raw) {
    const int lane = static_cast<int>(threadIdx.x & 63);
    int32_t mine = 0;
    raw = 0;
    for (int32_t i = 0; i < per; ++i) {
        const int32_t b = lane * per + i;
        if (b < count) {
            raw = a.lens[first + b];
            mine += attn_span(a, raw).tiles + cost;
        }
    }
    return mine;
}

__device__ __forceinline__ AttnPlan attn_plan(const AttnArgs &a, uint32_t w) {
    AttnPlan p;
    p.seq = p.before = 0;
    const uint32_t heads = static_cast<uint32_t>(a.n_kv), workers = static_cast<uint32_t>(a.workers);
    if (a.whole) {
        p.seq = static_cast<int32_t>(attn_over(w, a.over_heads));
        p.total = a.workers;      // here a unit is a whole item
        p.each = 1;
        p.cost = p.lens = 0;
        return p;
    }
    const int lane = static_cast<int>(threadIdx.x & 63);
    int32_t count = a.n_seq, per = (count + 63) / 64;
    int32_t mine = attn_lane_units(a, 0, count, per, kAttnCost, p.lens), run = attn_lanes_before(mine);
    uint32_t total = static_cast<uint32_t>(__builtin_amdgcn_readlane(run, 63)) * heads;
    p.cost = kAttnCost;
    bool few = false;
    if (per == 1) {
        const uint32_t tiles = total - heads * static_cast<uint32_t>(count) * kAttnCost;
        const uint32_t each = (tiles + workers - 1) / workers;
        few = each == 1 && tiles > kAttnCus && tiles >= 16 * heads * static_cast<uint32_t>(count);
        if (each <= 2 || !__any(lane < count && static_cast<uint32_t>(mine - kAttnCost) % each != 0)) {
            p.cost = 0;
            run -= (lane < count ? lane + 1 : count) * kAttnCost;
            mine -= lane < count ? kAttnCost : 0;
            total = tiles;
        }
    }
    p.total = static_cast<int32_t>(total);
    p.each = few ? 2 : static_cast<int32_t>((total + workers - 1) / workers);
    const uint32_t x = w * static_cast<uint32_t>(p.each);
    if (x >= total || a.n_seq == 1) return p;
    const int32_t y = static_cast<int32_t>(attn_over(x, a.over_heads));
    for (;;) {
        // (the bound holds by itself unless the lengths change while they are read: then the rows are
        // wrong, but nothing outside the tables is touched)
        const int past = __builtin_popcountll(__ballot(p.before + run <= y)), lastj = (count - 1) / per;
        const int j = past < lastj ? past : lastj;
        p.before += __builtin_amdgcn_readlane(run - mine, j);
        p.seq += j * per;
        if (per == 1) return p;
        count = count - j * per < per ? count - j * per : per;
        per = (count + 63) / 64;
        int32_t raw;
        mine = attn_lane_units(a, p.seq, count, per, p.cost, raw);
        run = attn_lanes_before(mine);
    }
}

__device__ __forceinline__ void attn_store(const AttnArgs &a, int64_t at, f32x4 o) {
    if (a.ofmt == WSL_OUT_F32)
        *reinterpret_cast<f32x4 *>(static_cast<float *>(a.out) + at) = o;
    else
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at) =
            make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
}

// Elements d .. d + 3 of row `row` (query position row / group, head h * group + row % group) of a
// sequence are done: o and l are its sums, m the maximum they are relative to.  l is zero where
// nothing was seen but scores of -infinity (and o may be NaN: zero times a value that is not finite), and
// at least one otherwise (the maximum's own term).
__device__ __forceinline__ void attn_finish(const AttnArgs &a, int32_t seq, int32_t h, int32_t row, int32_t d, f32x4 o,
                                            float m, float l) {
    const int32_t i = static_cast<int32_t>(attn_over(static_cast<uint32_t>(row), a.over_group)), head = h * a.group + row - i * a.group;
    const int64_t tok = static_cast<int64_t>(seq) * a.q_len + i;
    const f32x4 none = {0, 0, 0, 0};
    attn_store(a, tok * a.ld_out + static_cast<int64_t>(head) * a.head_dim + d, l == 0.f ? none : o * (1.f / l));
    if (a.lse != nullptr && d == 0)
        a.lse[tok * (a.n_kv * a.group) + head] =
            l == 0.f ? -__builtin_huge_valf() : (m + __builtin_amdgcn_logf(l)) * 0.69314718055994530942f;
}

template <int FMT>
int launch_attn_fmt(AttnArgs &a, int tiles_m, hipStream_t s);

}  // namespace wsl
