// Host-side argument validation of the C ABI (no HIP dependency).
#include "validate.h"

#include "../../include/wsl.h"

namespace wsl {
namespace {

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

bool mul_ok(int64_t a, int64_t b, int64_t *out) {
    if (a < 0 || b < 0) return false;
    if (a != 0 && b > INT64_MAX / a) return false;
    *out = a * b;
    return true;
}

}  // namespace

size_t nf4_bytes(int64_t n_out, int64_t k) {
    if (n_out <= 0 || k <= 0 || (k % kGroup) != 0) return 0;
    if (n_out > kMaxDim || k > kMaxDim) return 0;
    int64_t codes = 0, scales = 0;
    if (!mul_ok(n_out, k / 2, &codes)) return 0;
    if (!mul_ok(n_out, (k / kGroup) * 2, &scales)) return 0;
    if (codes > INT64_MAX - scales) return 0;
    return static_cast<size_t>(codes + scales);
}

int check_pack(const void *w, int64_t n_out, int64_t k, const void *packed) {
    if (!w || !packed) return WSL_E_NULL;
    if (nf4_bytes(n_out, k) == 0) return WSL_E_SHAPE;
    int64_t elems = 0;
    if (!mul_ok(n_out, k, &elems)) return WSL_E_SHAPE;
    if (!aligned(w, 16) || !aligned(packed, 16)) return WSL_E_ALIGN;
    return WSL_OK;
}

int check_dequant_tile(const void *packed, int64_t n_out, int64_t k, int64_t row0, int64_t k0,
                       int64_t rows, int64_t cols, const void *tile, int64_t ld_tile) {
    if (!packed || !tile) return WSL_E_NULL;
    if (nf4_bytes(n_out, k) == 0) return WSL_E_SHAPE;
    if (rows <= 0 || cols <= 0 || ld_tile <= 0) return WSL_E_SHAPE;
    if (rows > kMaxDim || cols > kMaxDim || ld_tile > kMaxDim) return WSL_E_SHAPE;
    if (ld_tile < cols) return WSL_E_SHAPE;
    if (row0 < 0 || k0 < 0 || row0 > n_out - rows || k0 > k - cols) return WSL_E_RANGE;
    int64_t t = 0;
    if (!mul_ok(rows, ld_tile, &t)) return WSL_E_SHAPE;
    if (!aligned(packed, 16) || !aligned(tile, 2)) return WSL_E_ALIGN;
    return WSL_OK;
}

int check_gemv(int wfmt, const void *w, int64_t n_out, int64_t k, const void *x, const void *y) {
    if (wfmt != WSL_W_BF16 && wfmt != WSL_W_NF4) return WSL_E_FORMAT;
    if (!w || !x || !y) return WSL_E_NULL;
    if (n_out <= 0 || k <= 0 || n_out > kMaxDim || k > kMaxDim) return WSL_E_SHAPE;
    if (wfmt == WSL_W_NF4) {
        if (nf4_bytes(n_out, k) == 0) return WSL_E_SHAPE;
    } else {
        int64_t e = 0;
        if ((k % 8) != 0 || !mul_ok(n_out, k, &e) || e > INT64_MAX / 2) return WSL_E_SHAPE;
    }
    if (!aligned(w, 16) || !aligned(x, 16) || !aligned(y, 4)) return WSL_E_ALIGN;
    return WSL_OK;
}

int check_gemm(int wfmt, const void *w, int64_t n_out, int64_t k, const void *x, int64_t m,
               int64_t ldx, const void *y, int ofmt, int64_t ldy, const void *ws, size_t ws_bytes) {
    if (wfmt != WSL_W_BF16 && wfmt != WSL_W_NF4) return WSL_E_FORMAT;
    if (ofmt != WSL_OUT_F32 && ofmt != WSL_OUT_BF16) return WSL_E_FORMAT;
    if (!w || !x || !y) return WSL_E_NULL;
    if (n_out <= 0 || k <= 0 || m <= 0) return WSL_E_SHAPE;
    if (n_out > kMaxDim || k > kMaxDim || m > kMaxDim || ldx > kMaxDim || ldy > kMaxDim) return WSL_E_SHAPE;
    if ((k % kGroup) != 0) return WSL_E_SHAPE;
    if (ldx < k || ldy < n_out) return WSL_E_SHAPE;
    int64_t e = 0;
    if (!mul_ok(m, ldx, &e) || !mul_ok(m, ldy, &e) || !mul_ok(n_out, k, &e)) return WSL_E_SHAPE;
    if ((ldx % 8) != 0) return WSL_E_ALIGN;
    if (!aligned(w, 16) || !aligned(x, 16)) return WSL_E_ALIGN;
    if (!aligned(y, ofmt == WSL_OUT_F32 ? 4 : 2)) return WSL_E_ALIGN;
    if (ws && ws_bytes && !aligned(ws, 16)) return WSL_E_ALIGN;
    return WSL_OK;
}

int check_ring(int wfmt, int64_t count, const void *const *h_w, const int64_t *n_out, const int64_t *k,
               const void *const *x, int64_t m, int64_t ldx, const void *const *y, int ofmt, int64_t ldy,
               const void *ws, size_t ws_bytes, const void *const *slot, size_t slot_bytes, const void *const *events,
               int flags) {
    if (wfmt != WSL_W_BF16 && wfmt != WSL_W_NF4) return WSL_E_FORMAT;
    if (flags & ~WSL_RING_PACE) return WSL_E_FLAGS;
    if (count < 0 || count > kMaxDim) return WSL_E_SHAPE;
    if (count == 0) return WSL_OK;
    if (!h_w || !n_out || !k || !x || !y || !slot || !events) return WSL_E_NULL;
    if (!slot[0] || !slot[1]) return WSL_E_NULL;
    if (!events[0] || !events[1] || !events[2] || !events[3]) return WSL_E_NULL;
    if (!aligned(slot[0], 16) || !aligned(slot[1], 16)) return WSL_E_ALIGN;
    for (int64_t i = 0; i < count; ++i) {
        if (!h_w[i]) return WSL_E_NULL;
        int rc = (m < 0) ? check_gemv(wfmt, slot[0], n_out[i], k[i], x[i], y[i])
                         : check_gemm(wfmt, slot[0], n_out[i], k[i], x[i], m, ldx, y[i], ofmt, ldy, ws, ws_bytes);
        if (rc != WSL_OK) return rc;
        size_t bytes = 0;
        if (wfmt == WSL_W_NF4) {
            bytes = nf4_bytes(n_out[i], k[i]);
        } else {
            int64_t e = 0;
            if (!mul_ok(n_out[i], k[i], &e) || e > INT64_MAX / 2) return WSL_E_SHAPE;
            bytes = static_cast<size_t>(e) * 2;
        }
        if (bytes == 0) return WSL_E_SHAPE;
        if (bytes > slot_bytes) return WSL_E_RANGE;
    }
    return WSL_OK;
}

int check_embed(const void *packed, int64_t n_rows, int64_t k, const void *ids, int64_t count, const void *out,
                int ofmt, int64_t ld_out) {
    if (ofmt != WSL_OUT_F32 && ofmt != WSL_OUT_BF16) return WSL_E_FORMAT;
    if (!packed || (count != 0 && (!ids || !out))) return WSL_E_NULL;   // ids and out may be NULL when count == 0
    if (nf4_bytes(n_rows, k) == 0) return WSL_E_SHAPE;
    if (count < 0 || count > kMaxDim || ld_out < k || ld_out > kMaxDim) return WSL_E_SHAPE;
    int64_t e = 0;
    if (!mul_ok(count, ld_out, &e)) return WSL_E_SHAPE;
    if ((ld_out % (ofmt == WSL_OUT_F32 ? 4 : 8)) != 0) return WSL_E_ALIGN;
    if (!aligned(packed, 16) || !aligned(ids, 8) || !aligned(out, 16)) return WSL_E_ALIGN;
    return WSL_OK;
}

int check_multi(int wfmt, int64_t count, const void *h_stages) {
    if (wfmt != WSL_W_BF16) return WSL_E_FORMAT;
    if (count < 0 || count > WSL_GEMV_MULTI_MAX) return WSL_E_SHAPE;
    if (count == 0) return WSL_OK;
    if (!h_stages) return WSL_E_NULL;
    const wsl_gemv_stage *st = static_cast<const wsl_gemv_stage *>(h_stages);
    for (int64_t i = 0; i < count; ++i) {
        const int rc = check_gemv(WSL_W_BF16, st[i].w, st[i].n_out, st[i].k, st[i].x, st[i].y);
        if (rc != WSL_OK) return rc;
        if (st[i].k != st[0].k) return WSL_E_SHAPE;
    }
    return WSL_OK;
}

int check_sweep(int wfmt, int64_t count, const void *h_stages, const void *d_stages, const void *ws,
                size_t ws_bytes, size_t ws_need) {
    if (wfmt != WSL_W_NF4) return WSL_E_FORMAT;
    if (count < 0 || count > (int64_t(1) << 24)) return WSL_E_SHAPE;
    if (count == 0) return WSL_OK;
    if (!h_stages || !d_stages || !ws) return WSL_E_NULL;
    if (!aligned(d_stages, 8) || !aligned(ws, 128)) return WSL_E_ALIGN;
    if (ws_bytes < ws_need) return WSL_E_RANGE;
    const wsl_gemv_stage *st = static_cast<const wsl_gemv_stage *>(h_stages);
    for (int64_t i = 0; i < count; ++i) {
        const int rc = check_gemv(WSL_W_NF4, st[i].w, st[i].n_out, st[i].k, st[i].x, st[i].y);
        if (rc != WSL_OK) return rc;
        if (st[i].k > 32768) return WSL_E_SHAPE;
    }
    return WSL_OK;
}

int check_kv_cache(const void *h_cache) {
    if (!h_cache) return WSL_E_NULL;
    const wsl_kv_cache &c = *static_cast<const wsl_kv_cache *>(h_cache);
    if (c.fmt != WSL_KV_BF16 && c.fmt != WSL_KV_E4M3) return WSL_E_FORMAT;
    if (!c.k || !c.v) return WSL_E_NULL;
    if (c.fmt == WSL_KV_E4M3 && (!c.k_exp || !c.v_exp)) return WSL_E_NULL;
    if (c.n_pages <= 0 || c.n_pages > 0x7fffffff || c.page_size <= 0 || c.page_size > kMaxDim) return WSL_E_SHAPE;
    if (c.n_kv <= 0 || c.n_kv > (int64_t(1) << 20)) return WSL_E_SHAPE;
    if (c.head_dim < 16 || c.head_dim > 256 || c.head_dim % 16 != 0) return WSL_E_SHAPE;
    const int64_t elem = c.fmt == WSL_KV_BF16 ? 2 : 1, step = 16 / elem;
    const int64_t stride[3] = {c.page_stride, c.head_stride, c.token_stride};
    const int64_t count[3] = {c.n_pages, c.n_kv, c.page_size};
    int64_t reach = c.head_dim, cells = 1;
    for (int i = 0; i < 3; ++i) {
        if (stride[i] < c.head_dim) return WSL_E_SHAPE;
        if (stride[i] % step != 0) return WSL_E_ALIGN;
        int64_t far = 0;
        if (!mul_ok(stride[i], count[i], &far) || far > INT64_MAX / 8 - reach) return WSL_E_SHAPE;
        reach += far;
        if (!mul_ok(cells, count[i], &cells)) return WSL_E_SHAPE;
    }
    if (!aligned(c.k, 16) || !aligned(c.v, 16)) return WSL_E_ALIGN;
    return WSL_OK;
}

namespace {

// Token rows [count][ld] of `width` elements outside the cache.
int check_token_rows(int fmt, int64_t count, int64_t width, int64_t ld) {
    const int64_t step = fmt == WSL_OUT_F32 ? 4 : 8;
    if (ld < width) return WSL_E_SHAPE;
    int64_t all = 0;
    if (!mul_ok(count, ld, &all) || all > INT64_MAX / 8) return WSL_E_SHAPE;
    return ld % step == 0 ? WSL_OK : WSL_E_ALIGN;
}

}  // namespace

int check_kv_rows(const void *h_cache, const void *k, const void *v, int fmt, int64_t count, int64_t ld_k, int64_t ld_v,
                  const void *slots) {
    int rc = check_kv_cache(h_cache);
    if (rc != WSL_OK) return rc;
    if (fmt != WSL_OUT_F32 && fmt != WSL_OUT_BF16) return WSL_E_FORMAT;
    if (count < 0) return WSL_E_SHAPE;
    if (count == 0) return WSL_OK;
    if (!k || !v || !slots) return WSL_E_NULL;
    const wsl_kv_cache &c = *static_cast<const wsl_kv_cache *>(h_cache);
    if (count > (int64_t(1) << 26) / c.n_kv) return WSL_E_SHAPE;
    if ((rc = check_token_rows(fmt, count, c.n_kv * c.head_dim, ld_k)) != WSL_OK) return rc;
    if ((rc = check_token_rows(fmt, count, c.n_kv * c.head_dim, ld_v)) != WSL_OK) return rc;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8)) return WSL_E_ALIGN;
    return WSL_OK;
}

int check_attn_shape(int qfmt, int64_t n_seq, int64_t q_len, int64_t n_heads, int64_t n_kv, int64_t head_dim,
                     int64_t pages_per_seq, int64_t page_size) {
    if (qfmt != WSL_OUT_F32 && qfmt != WSL_OUT_BF16) return WSL_E_FORMAT;
    if (n_seq < 0 || n_seq > 65535 || q_len < 1 || q_len > 256) return WSL_E_SHAPE;
    if (n_kv <= 0 || n_kv > (int64_t(1) << 20) || n_heads <= 0 || n_heads > kMaxDim || n_heads % n_kv != 0)
        return WSL_E_SHAPE;
    if (n_heads / n_kv * q_len > 65536 || n_heads * q_len > (int64_t(1) << 24)) return WSL_E_SHAPE;
    if (head_dim < 16 || head_dim > 256 || head_dim % 16 != 0) return WSL_E_SHAPE;
    if (pages_per_seq < 1 || pages_per_seq > 0x7fffffff || page_size < 1 || page_size > kMaxDim) return WSL_E_SHAPE;
    // the kernels count tiles of 128 tokens, and some more of each, over all sequences and kv heads in 32 bits
    const int64_t capacity = pages_per_seq * page_size, tokens = capacity < 0x7fffffff ? capacity : 0x7fffffff;
    if (n_seq * n_kv > (int64_t(1) << 30) / ((tokens + 127) / 128 + 4)) return WSL_E_SHAPE;
    return WSL_OK;
}

int check_attn(const void *h_cache, const void *q, int qfmt, int64_t n_seq, int64_t q_len, int64_t n_heads,
               int64_t ld_q, const void *table, int64_t ld_table, int64_t pages_per_seq, const void *lens, float scale,
               int64_t window, const void *out, int ofmt, int64_t ld_out, const void *lse) {
    int rc = check_kv_cache(h_cache);
    if (rc != WSL_OK) return rc;
    const wsl_kv_cache &c = *static_cast<const wsl_kv_cache *>(h_cache);
    if (ofmt != WSL_OUT_F32 && ofmt != WSL_OUT_BF16) return WSL_E_FORMAT;
    rc = check_attn_shape(qfmt, n_seq, q_len, n_heads, c.n_kv, c.head_dim, pages_per_seq, c.page_size);
    if (rc != WSL_OK) return rc;
    if (n_seq == 0) return WSL_OK;
    if (!q || !table || !lens || !out) return WSL_E_NULL;
    if (ld_table < pages_per_seq || window < 0 || !(scale - scale == 0.f)) return WSL_E_SHAPE;
    int64_t entries = 0;
    if (!mul_ok(n_seq, ld_table, &entries) || entries > INT64_MAX / 8) return WSL_E_SHAPE;
    if ((rc = check_token_rows(qfmt, n_seq * q_len, n_heads * c.head_dim, ld_q)) != WSL_OK) return rc;
    if ((rc = check_token_rows(ofmt, n_seq * q_len, n_heads * c.head_dim, ld_out)) != WSL_OK) return rc;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(lse, 4))
        return WSL_E_ALIGN;
    return WSL_OK;
}

int check_verify(const void *p, const void *q, int pfmt, int64_t n_seq, int64_t width, int64_t vocab, int64_t ld_p,
                 int64_t ld_q, const void *drafts, const void *n_drafts, const void *u, const void *accepted,
                 const void *tokens) {
    if (pfmt != WSL_OUT_F32 && pfmt != WSL_OUT_BF16) return WSL_E_FORMAT;
    if (n_seq < 0 || n_seq > 65535 || width < 0 || width > WSL_VERIFY_MAX_DRAFTS) return WSL_E_SHAPE;
    if (vocab <= 0 || vocab > kMaxDim) return WSL_E_SHAPE;
    if (n_seq == 0) return WSL_OK;
    if (!p || !u || !accepted || !tokens || (width > 0 && !drafts)) return WSL_E_NULL;
    int64_t all = 0;
    if (ld_p < vocab || (q && ld_q < vocab)) return WSL_E_SHAPE;
    if (!mul_ok(n_seq * (width + 1), ld_p, &all) || all > INT64_MAX / 8) return WSL_E_SHAPE;
    if (q && (!mul_ok(n_seq * (width + 1), ld_q, &all) || all > INT64_MAX / 8)) return WSL_E_SHAPE;
    const uintptr_t elem = pfmt == WSL_OUT_F32 ? 4 : 2;
    if (!aligned(p, elem) || !aligned(q, elem) || !aligned(drafts, 4) || !aligned(n_drafts, 4) || !aligned(u, 4) ||
        !aligned(accepted, 4) || !aligned(tokens, 4))
        return WSL_E_ALIGN;
    return WSL_OK;
}

int check_workspace(const void *ws, size_t ws_bytes, size_t need, size_t alignment) {
    if (need == 0) return WSL_OK;
    if (!ws) return WSL_E_NULL;
    if (ws_bytes < need) return WSL_E_RANGE;
    return aligned(ws, alignment) ? WSL_OK : WSL_E_ALIGN;
}

}  // namespace wsl
