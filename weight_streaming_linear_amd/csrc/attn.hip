// attn_decode on the host: how many rows a workgroup holds, how many workgroups, and the kernel
// that joins the parts of a (sequence, head) that several workgroups computed.
#include "attn.h"

namespace wsl {
namespace {

// For each (sequence, kv head, row tile) whose tiles lie in more than one workgroup's range:
// with the parts' maxima m_i, sums l_i and O_i, M = max m_i, the result is
// sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i, added in the order of the workgroups.
__global__ __launch_bounds__(kAttnThreads) void attn_join_kernel(AttnArgs a) {
    __shared__ int64_t lds_plan[4];
    __shared__ int64_t lds_before;
    const int items = a.n_kv * a.row_tiles;
    const int32_t seq = static_cast<int32_t>(blockIdx.y), item = static_cast<int32_t>(blockIdx.x);
    const AttnPlan plan = attn_plan(a, lds_plan);
    if (static_cast<int32_t>(threadIdx.x) == seq / plan.each) {
        int64_t before = plan.before;
        for (int32_t b = static_cast<int32_t>(threadIdx.x) * plan.each; b < seq; ++b) before += attn_span(a, b).tiles;
        lds_before = before;
    }
    __syncthreads();
    const AttnSpan span = attn_span(a, seq);
    const int64_t total = plan.total * items;
    const int64_t x0 = lds_before * items + static_cast<int64_t>(item) * span.tiles;
    const int64_t workers = attn_workers(a, total);
    const int64_t w0 = attn_worker(total, x0, workers), w1 = attn_worker(total, x0 + span.tiles - 1, workers);
    if (w0 == w1) return;
    const int32_t h = item / a.row_tiles, row0 = (item - h * a.row_tiles) * a.tile_rows;
    const int per_row = a.head_dim / 4;
    for (int32_t i = static_cast<int32_t>(threadIdx.x); i < a.tile_rows * per_row; i += kAttnThreads) {
        const int32_t r = i / per_row, d = (i - r * per_row) * 4;
        if (row0 + r >= a.rows) break;
        // worker w0 holds the item's beginning (its second slot), the others go on (their first)
        float top = -__builtin_huge_valf();
        for (int64_t w = w0; w <= w1; ++w) top = fmaxf(top, a.part_ml[(2 * w + (w == w0)) * a.tile_rows + r].x);
        const float ref = top == -__builtin_huge_valf() ? 0.f : top;
        f32x4 o = {0, 0, 0, 0};
        float l = 0.f;
        for (int64_t w = w0; w <= w1; ++w) {
            const int64_t at = (2 * w + (w == w0)) * a.tile_rows + r;
            const float2 ml = a.part_ml[at];
            const float f = __builtin_amdgcn_exp2f(ml.x - ref);
            o += *reinterpret_cast<const f32x4 *>(a.part_o + at * a.head_dim + d) * f;
            l += ml.y * f;
        }
        attn_finish(a, seq, span.len, h, row0 + r, d, make_float4(o.x, o.y, o.z, o.w), top, l);
    }
}

struct AttnShape {
    int mt, tile_rows, row_tiles;
    int64_t workers;
    bool may_split;
};

// Blocks of 16 rows a workgroup holds: as many as the rows need, up to what the registers hold
// beside the head's width; more rows read the cache once per row tile.
AttnShape shape_of(int qfmt, int64_t n_seq, int64_t rows, int64_t n_kv, int64_t head_dim, int64_t capacity) {
    AttnShape s;
    const int most = qfmt == WSL_OUT_BF16 ? (head_dim > 128 ? 2 : 4) : (head_dim > 128 ? 1 : 2);
    s.mt = rows <= 16 ? 1 : (rows <= 32 ? 2 : 4);
    s.mt = s.mt > most ? most : s.mt;
    s.tile_rows = static_cast<int>(rows < 16 * s.mt ? rows : 16 * s.mt);
    s.row_tiles = static_cast<int>((rows + s.tile_rows - 1) / s.tile_rows);
    const int64_t tiles = (capacity + kAttnTile - 1) / kAttnTile;
    const int64_t items = n_seq * n_kv * s.row_tiles;
    s.may_split = tiles > 1;
    // two workgroups fit on a compute unit
    const int64_t want = 512;
    s.workers = tiles >= want || items >= want ? want : (items * tiles < want ? items * tiles : want);
    return s;
}

}  // namespace

size_t attn_ws_bytes(int qfmt, int64_t n_seq, int64_t rows, int64_t n_kv, int64_t head_dim, int64_t capacity) {
    const AttnShape s = shape_of(qfmt, n_seq, rows, n_kv, head_dim, capacity);
    if (!s.may_split) return 0;
    const size_t parts = 2 * static_cast<size_t>(s.workers) * static_cast<size_t>(s.tile_rows);
    return parts * (static_cast<size_t>(head_dim) * sizeof(float) + sizeof(float2));
}

int launch_attn(const wsl_kv_cache *c, const void *q, int qfmt, int64_t n_seq, int64_t q_len, int64_t n_heads,
                int64_t ld_q, const int32_t *table, int64_t ld_table, int64_t pages_per_seq, const int32_t *lens,
                float scale, int64_t window, void *out, int ofmt, int64_t ld_out, float *lse, void *ws,
                uint32_t *status, hipStream_t s) {
    const int64_t elem = c->fmt == WSL_KV_BF16 ? 2 : 1;
    const int64_t group = n_heads / c->n_kv, rows = group * q_len, capacity = pages_per_seq * c->page_size;
    const AttnShape sh = shape_of(qfmt, n_seq, rows, c->n_kv, c->head_dim, capacity);
    AttnArgs a;
    a.k = static_cast<const char *>(c->k), a.v = static_cast<const char *>(c->v), a.ke = c->k_exp, a.ve = c->v_exp;
    a.q = q, a.out = out, a.lse = lse, a.table = table, a.lens = lens, a.status = status;
    a.page_stride = c->page_stride * elem, a.head_stride = c->head_stride * elem, a.token_stride = c->token_stride * elem;
    a.ld_q = ld_q, a.ld_out = ld_out, a.ld_table = ld_table;
    a.window = window, a.capacity = capacity < 0x7fffffff - kAttnTile ? capacity : 0x7fffffff - kAttnTile;
    a.scale_log2 = static_cast<float>(static_cast<double>(scale) * 1.44269504088896340736);
    a.n_seq = static_cast<int32_t>(n_seq), a.q_len = static_cast<int32_t>(q_len), a.n_kv = static_cast<int32_t>(c->n_kv);
    a.group = static_cast<int32_t>(group), a.rows = static_cast<int32_t>(rows);
    a.head_dim = static_cast<int32_t>(c->head_dim), a.page_size = static_cast<int32_t>(c->page_size);
    a.n_pages = static_cast<int32_t>(c->n_pages);
    a.row_tiles = sh.row_tiles, a.tile_rows = sh.tile_rows, a.workers = static_cast<int32_t>(sh.workers);
    a.qfmt = qfmt, a.ofmt = ofmt;
    // the parts' sums first (16-byte aligned), then their maxima and sums
    a.part_o = static_cast<float *>(ws);
    a.part_ml = reinterpret_cast<float2 *>(a.part_o + 2 * sh.workers * sh.tile_rows * c->head_dim);
    if (c->fmt == WSL_KV_BF16) launch_attn_fmt<WSL_KV_BF16>(a, sh.mt, s);
    else launch_attn_fmt<WSL_KV_E4M3>(a, sh.mt, s);
    if (sh.may_split)
        hipLaunchKernelGGL(attn_join_kernel, dim3(static_cast<unsigned>(a.n_kv * a.row_tiles), static_cast<unsigned>(n_seq)),
                           dim3(kAttnThreads), 0, s, a);
    return WSL_OK;
}

}  // namespace wsl
