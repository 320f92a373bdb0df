// attn_decode on the host: how many rows a workgroup holds, how many workgroups, and the kernel
// that joins the parts of a (sequence, kv head) that several workgroups computed.
#include "attn.h"

namespace wsl {
namespace {

// Workgroup (i, y) joins rows y * kAttnJoinRows .. of the item of entry i, if it has several parts: with the parts' maxima m_i, sums l_i and O_i, M = max m_i, the result is
// sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.  Bound by trips to memory, so the parts are split over
// groups of threads, each of which asks for several at a time and keeps a running maximum; the
// groups are then joined in order.
constexpr int kJoinMany = 1024, kJoinFew = 256, kJoinAhead = 4;
constexpr int kJoinLds = sizeof(f32x4) + 2 * sizeof(float);  // of a thread
__global__ __launch_bounds__(kJoinMany) void attn_join_kernel(AttnArgs a) {
    extern __shared__ f32x4 lds_o[];
    const int threads = static_cast<int>(blockDim.x);
    float *lds_m = reinterpret_cast<float *>(lds_o + threads), *lds_l = lds_m + threads;
    AttnOpen it = a.open[blockIdx.x];
    // (never so unless the lengths changed while the workers read them, and an item was nobody's)
    if (it.worker < 0 || it.worker >= a.workers || it.parts > a.workers - it.worker) return;
    if (it.parts <= 1) return;
    const int32_t w = it.worker;
    if (a.by_item) {
        it.seq = static_cast<int32_t>(blockIdx.x) / a.n_kv;
        it.head = static_cast<int32_t>(blockIdx.x) - it.seq * a.n_kv;
    }
    const int tid = static_cast<int>(threadIdx.x);
    const int per_row = a.head_dim / 4, cells = kAttnJoinRows * per_row;
    const int groups = threads / cells;                      // 1 .. 64
    const int grp = tid / cells, cell = tid - grp * cells, r = cell / per_row, d = (cell - r * per_row) * 4;
    const int32_t row = static_cast<int32_t>(blockIdx.y) * kAttnJoinRows + r;
    const bool in = grp < groups && row < a.rows;
    const int32_t rt = row / a.tile_rows, in_tile = row - rt * a.tile_rows;
    // worker w holds the item's beginning (its second slot), the others go on (their first)
    const int64_t base = static_cast<int64_t>(rt) * a.workers * 2;
    float top = -__builtin_huge_valf(), l = 0.f;
    f32x4 o = {0, 0, 0, 0};
    auto add = [&](float m1, float l1, f32x4 o1) {
        const float best = fmaxf(top, m1), ref = best == -__builtin_huge_valf() ? 0.f : best;
        const float f0 = __builtin_amdgcn_exp2f(top - ref), f1 = __builtin_amdgcn_exp2f(m1 - ref);
        o = o * f0 + o1 * f1;
        l = l * f0 + l1 * f1;
        top = best;
    };
    if (in)
        for (int32_t i0 = grp; i0 < it.parts; i0 += groups * kJoinAhead) {
            float2 ml[kJoinAhead];
            f32x4 po[kJoinAhead];
#pragma unroll
            for (int e = 0; e < kJoinAhead; ++e) {
                const int32_t i = i0 + e * groups;
                const int64_t at = (base + 2 * (w + i) + (i == 0)) * a.tile_rows + in_tile;
                ml[e] = make_float2(-__builtin_huge_valf(), 0.f);
                po[e] = f32x4{0, 0, 0, 0};
                if (i < it.parts) {
                    ml[e] = a.part_ml[at];
                    po[e] = *reinterpret_cast<const f32x4 *>(a.part_o + at * a.head_dim + d);
                }
            }
#pragma unroll
            for (int e = 0; e < kJoinAhead; ++e) add(ml[e].x, ml[e].y, po[e]);
        }
    lds_o[tid] = o;
    lds_m[tid] = top;
    lds_l[tid] = l;
    __syncthreads();
    if (!in || grp != 0) return;
    const int n = groups < it.parts ? groups : it.parts;
    for (int i = 1; i < n; ++i) add(lds_m[i * cells + cell], lds_l[i * cells + cell], lds_o[i * cells + cell]);
    attn_finish(a, it.seq, it.head, row, d, o, top, l);
}

// Short sequences are not split, which saves the joining launch: a workgroup takes an item from end to
// end.  (One sequence of 512 tokens, 40 heads on 8 of 128: 8.9 us against 12.5, 16 of up to 512 9.6
// against 13.0, 64 of them 16.0 against 22.0; of 1024 tokens 13.1 against 12.7, 15.1 against 14.5 and, with
// enough items to fill the chip, 25.8 against 27.5.  What a table has room for decides, not the lengths: one
// of 512 in a table for 8192 takes 12.7.)
bool attn_whole(int64_t tiles, int64_t items) {
    return tiles <= (items >= 2 * kAttnCus ? 8 : 4) && items <= (1 << 23);      // (a grid's limit)
}

struct AttnShape {
    int mt, tile_rows, row_tiles;
    int64_t workers, entries; // at most
    bool whole;
};

// Two blocks of 16 rows for a workgroup, or one; more rows are as many workgroups over the same tokens.
// Two where the registers allow beside the head's width (24 rows of 192, 89 sequences of up to 1839
// tokens, bf16: 104 us against 138 with one; 25 rows of 128, 16 of up to 4224: 27.6 against 32.6, over e4m3
// 25.3 against 26.4, with fp32 queries 30.8 against 34.1, over e4m3 31.1 against 28.2).  Left at one where
// two won in some shapes and lost in others: 192 over e4m3 88 against 96 and 26.0 against 25.8; 256 over
// bf16, with spilled registers, 63.6 against 66.5 and 41.7 against 36.3; fp32 queries of 64 22.0 against
// 24.0 and 24.9 against 25.4.  And where there is enough to do for all compute units (25 rows of 128, one
// sequence of 300 tokens 10.8 against 8.2, of 4000 14.7 against 13.6, of 8192 16.9 against 16.7; 16 of up to
// 500 12.4 against 10.1, 32 of them 13.0 against 17.1, 64 19.2 against 25.7).
int blocks_of(int fmt, int qfmt, int64_t rows, int64_t head_dim, bool whole, int64_t shares) {
    if (rows <= 16 || shares <= (whole ? 1 : 2) * kAttnCus / ((rows + 15) / 16)) return 1;
    return attn_two_blocks(fmt, qfmt, head_dim) ? 2 : 1;
}

AttnShape shape_of(int fmt, int qfmt, int64_t n_seq, int64_t rows, int64_t n_kv, int64_t head_dim, int64_t capacity) {
    AttnShape s;
    const int64_t tiles = (capacity + kAttnTile - 1) / kAttnTile, items = n_seq * n_kv;
    s.whole = attn_whole(tiles, items);
    s.mt = blocks_of(fmt, qfmt, rows, head_dim, s.whole, s.whole || tiles > (1 << 20) ? items : items * tiles);
    s.tile_rows = static_cast<int>(rows < 16 * s.mt ? rows : 16 * s.mt);
    s.row_tiles = static_cast<int>((rows + s.tile_rows - 1) / s.tile_rows);
    const int64_t fit = kAttnCus * kAttnMaxWaves, most = s.row_tiles * 8 >= fit ? 8 : fit / s.row_tiles / 8 * 8;
    s.workers = tiles >= most || items >= most || items * tiles >= most ? most : items * tiles;
    s.entries = items < s.workers ? items : s.workers;
    return s;
}

size_t parts_of(const AttnShape &s) {
    return 2 * static_cast<size_t>(s.workers) * static_cast<size_t>(s.row_tiles) * static_cast<size_t>(s.tile_rows);
}

}  // namespace

// Enough for a cache of either format.
size_t attn_ws_bytes(int qfmt, int64_t n_seq, int64_t rows, int64_t n_kv, int64_t head_dim, int64_t capacity) {
    size_t need = 0;
    for (const int fmt : {WSL_KV_BF16, WSL_KV_E4M3}) {
        const AttnShape s = shape_of(fmt, qfmt, n_seq, rows, n_kv, head_dim, capacity);
        if (s.whole) return 0;
        const size_t bytes = parts_of(s) * (static_cast<size_t>(head_dim) * sizeof(float) + sizeof(float2)) +
                             static_cast<size_t>(s.entries) * sizeof(AttnOpen);
        need = bytes > need ? bytes : need;
    }
    return need;
}

int launch_attn(const wsl_kv_cache *c, const void *q, int qfmt, int64_t n_seq, int64_t q_len, int64_t n_heads,
                int64_t ld_q, const int32_t *table, int64_t ld_table, int64_t pages_per_seq, const int32_t *lens,
                float scale, int64_t window, void *out, int ofmt, int64_t ld_out, float *lse, void *ws,
                uint32_t *status, hipStream_t s) {
    const int64_t elem = c->fmt == WSL_KV_BF16 ? 2 : 1;
    const int64_t group = n_heads / c->n_kv, rows = group * q_len, capacity = pages_per_seq * c->page_size;
    const AttnShape sh = shape_of(static_cast<int>(c->fmt), qfmt, n_seq, rows, c->n_kv, c->head_dim, capacity);
    AttnArgs a;
    a.k = static_cast<const char *>(c->k), a.v = static_cast<const char *>(c->v), a.ke = c->k_exp, a.ve = c->v_exp;
    a.q = q, a.out = out, a.lse = lse, a.table = table, a.lens = lens, a.status = status;
    a.page_stride = c->page_stride * elem, a.head_stride = c->head_stride * elem, a.token_stride = c->token_stride * elem;
    a.ld_q = ld_q, a.ld_out = ld_out, a.ld_table = ld_table;
    a.window = attn_window(window, capacity);
    a.capacity = static_cast<int32_t>(capacity < kAttnMaxTokens ? capacity : kAttnMaxTokens);
    a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.44269504088896340736);
    a.n_seq = static_cast<int32_t>(n_seq), a.q_len = static_cast<int32_t>(q_len), a.n_kv = static_cast<int32_t>(c->n_kv);
    a.group = static_cast<int32_t>(group), a.rows = static_cast<int32_t>(rows);
    a.head_dim = static_cast<int32_t>(c->head_dim), a.page_size = static_cast<int32_t>(c->page_size);
    a.n_pages = static_cast<int32_t>(c->n_pages);
    a.over_page = attn_div(static_cast<uint32_t>(c->page_size)), a.over_group = attn_div(static_cast<uint32_t>(group));
    a.over_heads = attn_div(static_cast<uint32_t>(c->n_kv));
    a.row_tiles = sh.row_tiles, a.tile_rows = sh.tile_rows, a.workers = static_cast<int32_t>(sh.workers);
    a.qfmt = qfmt, a.ofmt = ofmt;
    // the parts' sums first (16-byte aligned), then the open items, then the parts' maxima and sums
    a.part_o = static_cast<float *>(ws);
    a.open = sh.whole ? nullptr : reinterpret_cast<AttnOpen *>(a.part_o + parts_of(sh) * c->head_dim);
    a.part_ml = sh.whole ? nullptr : reinterpret_cast<float2 *>(a.open + sh.entries);
    a.whole = sh.whole ? 1 : 0;
    a.by_item = n_seq * c->n_kv <= sh.workers ? 1 : 0;
    if (c->fmt == WSL_KV_BF16) launch_attn_fmt<WSL_KV_BF16>(a, sh.mt, s);
    else launch_attn_fmt<WSL_KV_E4M3>(a, sh.mt, s);
    if (!sh.whole) {
        // A few long sequences leave items in many parts, many sequences leave many items in two or
        // three.  (One sequence of 8192 tokens, 8 heads of 32 parts: 15.3 us a call with few threads,
        // 14.6 with many, in e4m3 12.9 and 12.4; 16 of up to 4224 with five queries 27.6 with few, 30.0
        // with many, in e4m3 25.5 and 28.8; 32 of up to 8192 in e4m3 42.2 and 44.0.)
        const int threads = a.workers >= 16 * n_seq * c->n_kv ? kJoinMany : kJoinFew;
        hipLaunchKernelGGL(attn_join_kernel,
                           dim3(static_cast<unsigned>(a.by_item ? n_seq * c->n_kv : a.workers),
                                static_cast<unsigned>((rows + kAttnJoinRows - 1) / kAttnJoinRows)),
                           dim3(threads), threads * kJoinLds, s, a);
    }
    return WSL_OK;
}

}  // namespace wsl
