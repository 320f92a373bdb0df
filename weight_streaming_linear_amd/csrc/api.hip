// C ABI entry points (include/wsl.h): validate on the host, check the device,
// enqueue on the caller's stream, report launch errors without synchronizing.
#include <atomic>
#include <cstring>

#include "device_common.h"
#include "validate.h"

namespace wsl {
int launch_pack(const void *w, int64_t n_out, int64_t k, void *packed, uint32_t *status, hipStream_t s);
int launch_dequant_tile(const void *packed, int64_t n_out, int64_t k, int64_t row0, int64_t k0, int64_t rows,
                        int64_t cols, void *tile, int64_t ld, hipStream_t s);
int launch_gemv_bf16(const void *w, int64_t n_out, int64_t k, const void *x, float *y, hipStream_t s);
int launch_gemv_bf16_multi(const wsl_gemv_stage *st, int64_t count, hipStream_t s);
int launch_gemv_nf4(const void *w, int64_t n_out, int64_t k, const void *x, float *y, hipStream_t s);
size_t sweep_ws_bytes();
int launch_gemv_nf4_sweep(const wsl_gemv_stage *d_stages, int64_t count, int64_t max_k, void *ws, hipStream_t s);
int launch_gemm_bf16(const void *w, int64_t n_out, int64_t k, const void *x, int64_t m, int64_t ldx, void *y,
                     int ofmt, int64_t ldy, void *ws, size_t ws_bytes, hipStream_t s);
int launch_gemm_nf4(const void *w, int64_t n_out, int64_t k, const void *x, int64_t m, int64_t ldx, void *y,
                    int ofmt, int64_t ldy, void *ws, size_t ws_bytes, hipStream_t s);
size_t gemm_ws_bytes(int wfmt, int64_t n_out, int64_t k, int64_t m);
int launch_gemm_noalloc(int wfmt, const void *w, int64_t n_out, int64_t k, const void *x, int64_t m, int64_t ldx,
                        void *y, int ofmt, int64_t ldy, hipStream_t s);
int launch_kv_write(const wsl_kv_cache *c, const void *k, const void *v, int xfmt, int64_t count, int64_t ld_k,
                    int64_t ld_v, const int64_t *slots, uint32_t *status, hipStream_t s);
int launch_kv_read(const wsl_kv_cache *c, const int64_t *slots, int64_t count, void *k, void *v, int ofmt,
                   int64_t ld_k, int64_t ld_v, uint32_t *status, hipStream_t s);
size_t attn_ws_bytes(int qfmt, int64_t n_seq, int64_t rows, int64_t n_kv, int64_t head_dim, int64_t capacity);
int launch_attn(const wsl_kv_cache *c, const void *q, int qfmt, int64_t n_seq, int64_t q_len, int64_t n_heads,
                int64_t ld_q, const int32_t *table, int64_t ld_table, int64_t pages_per_seq, const int32_t *lens,
                float scale, int64_t window, void *out, int ofmt, int64_t ld_out, float *lse, void *ws,
                uint32_t *status, hipStream_t s);
size_t verify_ws_bytes(int64_t n_seq, int64_t vocab);
int launch_verify(const void *p, const void *q, int pfmt, int64_t n_seq, int64_t width, int64_t vocab, int64_t ld_p,
                  int64_t ld_q, const int32_t *drafts, const int32_t *n_drafts, const float *u, int32_t *accepted,
                  int32_t *tokens, void *ws, uint32_t *status, hipStream_t s);
size_t grow_ws_bytes(int64_t n_seq, int64_t n_tokens);
int launch_grow(const wsl_kv_pages *p, const int32_t *d_new, int64_t each, int64_t n_tokens, int64_t *slots,
                int64_t *positions, int32_t *starts, void *ws, uint32_t *status, hipStream_t s);
int launch_trim(const wsl_kv_pages *p, const int32_t *lens, uint32_t *status, hipStream_t s);
int launch_rotary(const void *q, int64_t n_heads, int64_t ld_q, const void *k, int64_t n_kv, int64_t ld_k, int xfmt,
                  int64_t count, int64_t head_dim, int64_t rot_dim, const int64_t *positions, const double *freqs,
                  double amplitude, int flags, void *q_out, int64_t ld_q_out, void *k_out, int64_t ld_k_out, int ofmt,
                  hipStream_t s);
size_t sample_ws_bytes(int64_t n_rows, int64_t vocab);
int launch_sample(const void *logits, int zfmt, int64_t n_rows, int64_t vocab, int64_t ld, const wsl_sampling *how,
                  const float *u, int32_t *tokens, float *probs, int64_t ld_probs, void *ws, uint32_t *status,
                  hipStream_t s);
size_t lora_ws_bytes(int64_t m, int64_t rank, int64_t k);
int launch_lora(const void *d_a, const void *d_b, int64_t n_adapters, int64_t rank, int64_t n_out, int64_t k,
                const int32_t *ids, const float *scales, const void *x, int64_t m, int64_t ldx, const void *base,
                int64_t ld_base, void *out, int64_t ld_out, int fmt, void *ws, uint32_t *status, hipStream_t s);
int check_pinned(int64_t count, const void *const *h_w);
int ring_gemv(int wfmt, int64_t count, const void *const *h_w, const int64_t *n_out, const int64_t *k,
              const void *const *x, float *const *y, void *const *slot, hipStream_t copy, hipStream_t compute,
              void *const *events, int flags);
int ring_gemm(int wfmt, int64_t count, const void *const *h_w, const int64_t *n_out, const int64_t *k,
              const void *const *x, int64_t m, int64_t ldx, void *const *y, int ofmt, int64_t ldy, void *ws,
              size_t ws_bytes, void *const *slot, hipStream_t copy, hipStream_t compute, void *const *events,
              int flags);
int launch_stream_read(const void *buf, size_t bytes, uint32_t *sink, hipStream_t s);
int launch_embed_rows(const void *packed, int64_t n_rows, int64_t k, const int64_t *ids, int64_t count, void *out,
                      int ofmt, int64_t ld_out, uint32_t *status, hipStream_t s);

namespace {

constexpr int kMaxDevices = 64;
// 0 = not yet checked, 1 = gfx950, 2 = something else.
std::atomic<int> g_arch[kMaxDevices];

int device_ok() {
    int dev = -1;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0) return WSL_E_DEVICE;
    if (dev >= kMaxDevices) return WSL_E_DEVICE;
    int st = g_arch[dev].load(std::memory_order_acquire);
    if (st == 0) {
        hipDeviceProp_t prop;
        if (hipGetDeviceProperties(&prop, dev) != hipSuccess) return WSL_E_DEVICE;
        st = (std::strncmp(prop.gcnArchName, "gfx950", 6) == 0) ? 1 : 2;
        g_arch[dev].store(st, std::memory_order_release);
    }
    return st == 1 ? WSL_OK : WSL_E_DEVICE;
}

int after_launch(int rc) {
    if (rc != WSL_OK) return rc;
    return hipGetLastError() == hipSuccess ? WSL_OK : WSL_E_LAUNCH;
}

hipStream_t as_stream(void *s) { return static_cast<hipStream_t>(s); }

}  // namespace
}  // namespace wsl

extern "C" {

size_t nf4_packed_bytes(int64_t n_out, int64_t k) { return wsl::nf4_bytes(n_out, k); }

int nf4_codebook(float *out_host) {
    if (!out_host) return WSL_E_NULL;
    for (int i = 0; i < 16; ++i) std::memcpy(&out_host[i], &wsl::kLevelBits[i], sizeof(float));
    return WSL_OK;
}

int nf4_pack(const void *d_w, int64_t n_out, int64_t k, void *d_packed, uint32_t *d_status, void *stream) {
    int rc = wsl::check_pack(d_w, n_out, k, d_packed);
    if (rc != WSL_OK) return rc;
    if ((rc = wsl::device_ok()) != WSL_OK) return rc;
    return wsl::after_launch(wsl::launch_pack(d_w, n_out, k, d_packed, d_status, wsl::as_stream(stream)));
}

int nf4_dequant_tile(const void *d_packed, int64_t n_out, int64_t k, int64_t row0, int64_t k0, int64_t rows,
                     int64_t cols, void *d_tile, int64_t ld_tile, void *stream) {
    int rc = wsl::check_dequant_tile(d_packed, n_out, k, row0, k0, rows, cols, d_tile, ld_tile);
    if (rc != WSL_OK) return rc;
    if ((rc = wsl::device_ok()) != WSL_OK) return rc;
    return wsl::after_launch(
        wsl::launch_dequant_tile(d_packed, n_out, k, row0, k0, rows, cols, d_tile, ld_tile, wsl::as_stream(stream)));
}

int linear_gemv(int wfmt, const void *d_w, int64_t n_out, int64_t k, const void *d_x, float *d_y, void *stream) {
    int rc = wsl::check_gemv(wfmt, d_w, n_out, k, d_x, d_y);
    if (rc != WSL_OK) return rc;
    if ((rc = wsl::device_ok()) != WSL_OK) return rc;
    if (wfmt == WSL_W_NF4) return wsl::after_launch(wsl::launch_gemv_nf4(d_w, n_out, k, d_x, d_y, wsl::as_stream(stream)));
    return wsl::after_launch(wsl::launch_gemv_bf16(d_w, n_out, k, d_x, d_y, wsl::as_stream(stream)));
}

size_t linear_gemv_sweep_workspace_bytes(void) { return wsl::sweep_ws_bytes(); }

int linear_gemv_sweep(int wfmt, int64_t count, const wsl_gemv_stage *h_stages, const wsl_gemv_stage *d_stages,
                      void *d_ws, size_t ws_bytes, void *stream) {
    int rc = wsl::check_sweep(wfmt, count, h_stages, d_stages, d_ws, ws_bytes, wsl::sweep_ws_bytes());
    if (rc != WSL_OK || count == 0) return rc;
    if ((rc = wsl::device_ok()) != WSL_OK) return rc;
    int64_t max_k = 0;
    for (int64_t i = 0; i < count; ++i) max_k = h_stages[i].k > max_k ? h_stages[i].k : max_k;
    return wsl::after_launch(wsl::launch_gemv_nf4_sweep(d_stages, count, max_k, d_ws, wsl::as_stream(stream)));
}

int linear_gemv_multi(int wfmt, int64_t count, const wsl_gemv_stage *h_stages, void *stream) {
    int rc = wsl::check_multi(wfmt, count, h_stages);
    if (rc != WSL_OK || count == 0) return rc;
    if ((rc = wsl::device_ok()) != WSL_OK) return rc;
    return wsl::after_launch(wsl::launch_gemv_bf16_multi(h_stages, count, wsl::as_stream(stream)));
}

size_t linear_gemm_workspace_bytes(int wfmt, int64_t n_out, int64_t k, int64_t m) {
    if (wfmt != WSL_W_BF16 && wfmt != WSL_W_NF4) return 0;
    if (n_out <= 0 || k <= 0 || m <= 0 || (k % 64) != 0) return 0;
    if (n_out > wsl::kMaxDim || k > wsl::kMaxDim || m > wsl::kMaxDim) return 0;
    return wsl::gemm_ws_bytes(wfmt, n_out, k, m);
}

int linear_gemm(int wfmt, const void *d_w, int64_t n_out, int64_t k, const void *d_x, int64_t m, int64_t ldx,
                void *d_y, int ofmt, int64_t ldy, void *d_ws, size_t ws_bytes, void *stream) {
    int rc = wsl::check_gemm(wfmt, d_w, n_out, k, d_x, m, ldx, d_y, ofmt, ldy, d_ws, ws_bytes);
    if (rc != WSL_OK) return rc;
    if ((rc = wsl::device_ok()) != WSL_OK) return rc;
    if (wfmt == WSL_W_NF4)
        return wsl::after_launch(
            wsl::launch_gemm_nf4(d_w, n_out, k, d_x, m, ldx, d_y, ofmt, ldy, d_ws, ws_bytes, wsl::as_stream(stream)));
    return wsl::after_launch(
        wsl::launch_gemm_bf16(d_w, n_out, k, d_x, m, ldx, d_y, ofmt, ldy, d_ws, ws_bytes, wsl::as_stream(stream)));
}

int linear_gemm_noalloc(int wfmt, const void *d_w, int64_t n_out, int64_t k, const void *d_x, int64_t m,
                        int64_t ldx, void *d_y, int ofmt, int64_t ldy, void *stream) {
    int rc = wsl::check_gemm(wfmt, d_w, n_out, k, d_x, m, ldx, d_y, ofmt, ldy, nullptr, 0);
    if (rc != WSL_OK) return rc;
    if ((rc = wsl::device_ok()) != WSL_OK) return rc;
    return wsl::after_launch(
        wsl::launch_gemm_noalloc(wfmt, d_w, n_out, k, d_x, m, ldx, d_y, ofmt, ldy, wsl::as_stream(stream)));
}

int nf4_embed_rows(const void *d_packed, int64_t n_rows, int64_t k, const int64_t *d_ids, int64_t count,
                   void *d_out, int ofmt, int64_t ld_out, uint32_t *d_status, void *stream) {
    int rc = wsl::check_embed(d_packed, n_rows, k, d_ids, count, d_out, ofmt, ld_out);
    if (rc != WSL_OK) return rc;
    if ((rc = wsl::device_ok()) != WSL_OK) return rc;
    return wsl::after_launch(wsl::launch_embed_rows(d_packed, n_rows, k, d_ids, count, d_out, ofmt, ld_out, d_status,
                                                    wsl::as_stream(stream)));
}

int linear_gemv_streamed(int wfmt, int64_t count, const void *const *h_w, const int64_t *n_out, const int64_t *k,
                         const void *const *d_x, float *const *d_y, void *const *d_slot, size_t slot_bytes,
                         void *copy_stream, void *compute_stream, void *const *events, int flags) {
    int rc = wsl::check_ring(wfmt, count, h_w, n_out, k, d_x, -1, 0, reinterpret_cast<const void *const *>(d_y), 0,
                             0, nullptr, 0, d_slot, slot_bytes, events, flags);
    if (rc != WSL_OK || count == 0) return rc;
    if ((rc = wsl::device_ok()) != WSL_OK) return rc;
    if ((rc = wsl::check_pinned(count, h_w)) != WSL_OK) return rc;
    return wsl::ring_gemv(wfmt, count, h_w, n_out, k, d_x, d_y, d_slot, wsl::as_stream(copy_stream),
                          wsl::as_stream(compute_stream), events, flags);
}

int linear_gemm_streamed(int wfmt, int64_t count, const void *const *h_w, const int64_t *n_out, const int64_t *k,
                         const void *const *d_x, int64_t m, int64_t ldx, void *const *d_y, int ofmt, int64_t ldy,
                         void *d_ws, size_t ws_bytes, void *const *d_slot, size_t slot_bytes,
                         void *copy_stream, void *compute_stream, void *const *events, int flags) {
    int rc = wsl::check_ring(wfmt, count, h_w, n_out, k, d_x, m < 0 ? 0 : m, ldx,
                             reinterpret_cast<const void *const *>(d_y), ofmt, ldy, d_ws, ws_bytes, d_slot,
                             slot_bytes, events, flags);
    if (rc != WSL_OK || count == 0) return rc;
    if ((rc = wsl::device_ok()) != WSL_OK) return rc;
    if ((rc = wsl::check_pinned(count, h_w)) != WSL_OK) return rc;
    return wsl::ring_gemm(wfmt, count, h_w, n_out, k, d_x, m, ldx, d_y, ofmt, ldy, d_ws, ws_bytes, d_slot,
                          wsl::as_stream(copy_stream), wsl::as_stream(compute_stream), events, flags);
}

int kv_cache_write(const wsl_kv_cache *h_cache, const void *d_k, const void *d_v, int xfmt, int64_t count,
                   int64_t ld_k, int64_t ld_v, const int64_t *d_slots, uint32_t *d_status, void *stream) {
    int rc = wsl::check_kv_rows(h_cache, d_k, d_v, xfmt, count, ld_k, ld_v, d_slots);
    if (rc != WSL_OK || count == 0) return rc;
    if ((rc = wsl::device_ok()) != WSL_OK) return rc;
    return wsl::after_launch(wsl::launch_kv_write(h_cache, d_k, d_v, xfmt, count, ld_k, ld_v, d_slots, d_status,
                                                  wsl::as_stream(stream)));
}

int kv_cache_read(const wsl_kv_cache *h_cache, const int64_t *d_slots, int64_t count, void *d_k, void *d_v, int ofmt,
                  int64_t ld_k, int64_t ld_v, uint32_t *d_status, void *stream) {
    int rc = wsl::check_kv_rows(h_cache, d_k, d_v, ofmt, count, ld_k, ld_v, d_slots);
    if (rc != WSL_OK || count == 0) return rc;
    if ((rc = wsl::device_ok()) != WSL_OK) return rc;
    return wsl::after_launch(wsl::launch_kv_read(h_cache, d_slots, count, d_k, d_v, ofmt, ld_k, ld_v, d_status,
                                                 wsl::as_stream(stream)));
}

size_t attn_decode_workspace_bytes(int qfmt, int64_t n_seq, int64_t q_len, int64_t n_heads, int64_t n_kv,
                                   int64_t head_dim, int64_t pages_per_seq, int64_t page_size) {
    if (wsl::check_attn_shape(qfmt, n_seq, q_len, n_heads, n_kv, head_dim, pages_per_seq, page_size) != WSL_OK ||
        n_seq == 0)
        return 0;
    return wsl::attn_ws_bytes(qfmt, n_seq, n_heads / n_kv * q_len, n_kv, head_dim, pages_per_seq * page_size);
}

int attn_decode(const wsl_kv_cache *h_cache, const void *d_q, int qfmt, int64_t n_seq, int64_t q_len, int64_t n_heads,
                int64_t ld_q, const int32_t *d_block_table, int64_t ld_table, int64_t pages_per_seq,
                const int32_t *d_kv_lens, float scale, int64_t window, void *d_out, int ofmt, int64_t ld_out,
                float *d_lse, void *d_ws, size_t ws_bytes, uint32_t *d_status, void *stream) {
    int rc = wsl::check_attn(h_cache, d_q, qfmt, n_seq, q_len, n_heads, ld_q, d_block_table, ld_table, pages_per_seq,
                             d_kv_lens, scale, window, d_out, ofmt, ld_out, d_lse);
    if (rc != WSL_OK || n_seq == 0) return rc;
    const size_t need = wsl::attn_ws_bytes(qfmt, n_seq, n_heads / h_cache->n_kv * q_len, h_cache->n_kv,
                                           h_cache->head_dim, pages_per_seq * h_cache->page_size);
    if ((rc = wsl::check_workspace(d_ws, ws_bytes, need, 16)) != WSL_OK) return rc;
    if ((rc = wsl::device_ok()) != WSL_OK) return rc;
    return wsl::after_launch(wsl::launch_attn(h_cache, d_q, qfmt, n_seq, q_len, n_heads, ld_q, d_block_table, ld_table,
                                              pages_per_seq, d_kv_lens, scale, window, d_out, ofmt, ld_out, d_lse, d_ws,
                                              d_status, wsl::as_stream(stream)));
}

size_t verify_drafts_workspace_bytes(int64_t n_seq, int64_t vocab) {
    if (n_seq <= 0 || n_seq > 65535 || vocab <= 0 || vocab > wsl::kMaxDim) return 0;
    return wsl::verify_ws_bytes(n_seq, vocab);
}

int verify_drafts(const void *d_p, const void *d_q, int pfmt, int64_t n_seq, int64_t width, int64_t vocab,
                  int64_t ld_p, int64_t ld_q, const int32_t *d_drafts, const int32_t *d_n_drafts, const float *d_u,
                  int32_t *d_accepted, int32_t *d_tokens, void *d_ws, size_t ws_bytes, uint32_t *d_status,
                  void *stream) {
    int rc = wsl::check_verify(d_p, d_q, pfmt, n_seq, width, vocab, ld_p, ld_q, d_drafts, d_n_drafts, d_u, d_accepted,
                               d_tokens);
    if (rc != WSL_OK || n_seq == 0) return rc;
    if ((rc = wsl::check_workspace(d_ws, ws_bytes, wsl::verify_ws_bytes(n_seq, vocab), 16)) != WSL_OK) return rc;
    if ((rc = wsl::device_ok()) != WSL_OK) return rc;
    return wsl::after_launch(wsl::launch_verify(d_p, d_q, pfmt, n_seq, width, vocab, ld_p, ld_q, d_drafts, d_n_drafts,
                                                d_u, d_accepted, d_tokens, d_ws, d_status, wsl::as_stream(stream)));
}

size_t kv_pages_grow_workspace_bytes(int64_t n_seq, int64_t n_tokens) {
    if (n_seq < 0 || n_seq > 65535 || n_tokens < 0 || n_tokens > wsl::kMaxDim) return 0;
    return wsl::grow_ws_bytes(n_seq, n_tokens);
}

int kv_pages_grow(const wsl_kv_pages *h_pages, const int32_t *d_new, int64_t each, int64_t n_tokens, int64_t *d_slots,
                  int64_t *d_positions, int32_t *d_starts, void *d_ws, size_t ws_bytes, uint32_t *d_status,
                  void *stream) {
    int rc = wsl::check_grow(h_pages, d_new, each, n_tokens, d_slots, d_positions, d_starts);
    if (rc != WSL_OK || (h_pages->n_seq == 0 && n_tokens == 0 && !d_starts)) return rc;
    if ((rc = wsl::check_workspace(d_ws, ws_bytes, wsl::grow_ws_bytes(h_pages->n_seq, n_tokens), 16)) != WSL_OK) return rc;
    if ((rc = wsl::device_ok()) != WSL_OK) return rc;
    return wsl::after_launch(wsl::launch_grow(h_pages, d_new, each, n_tokens, d_slots, d_positions, d_starts, d_ws,
                                              d_status, wsl::as_stream(stream)));
}

int kv_pages_trim(const wsl_kv_pages *h_pages, const int32_t *d_lens, uint32_t *d_status, void *stream) {
    int rc = wsl::check_trim(h_pages, d_lens);
    if (rc != WSL_OK || h_pages->n_seq == 0) return rc;
    if ((rc = wsl::device_ok()) != WSL_OK) return rc;
    return wsl::after_launch(wsl::launch_trim(h_pages, d_lens, d_status, wsl::as_stream(stream)));
}

int rotary_embed(const void *d_q, int64_t n_heads, int64_t ld_q, const void *d_k, int64_t n_kv, int64_t ld_k, int xfmt,
                 int64_t count, int64_t head_dim, int64_t rot_dim, const int64_t *d_positions, const double *d_freqs,
                 double amplitude, int flags, void *d_q_out, int64_t ld_q_out, void *d_k_out, int64_t ld_k_out, int ofmt,
                 void *stream) {
    int rc = wsl::check_rotary(d_q, n_heads, ld_q, d_k, n_kv, ld_k, xfmt, count, head_dim, rot_dim, d_positions, d_freqs,
                               amplitude, flags, d_q_out, ld_q_out, d_k_out, ld_k_out, ofmt);
    if (rc != WSL_OK || count == 0) return rc;
    if ((rc = wsl::device_ok()) != WSL_OK) return rc;
    return wsl::after_launch(wsl::launch_rotary(d_q, n_heads, ld_q, d_k, n_kv, ld_k, xfmt, count, head_dim, rot_dim,
                                                d_positions, d_freqs, amplitude, flags, d_q_out, ld_q_out, d_k_out,
                                                ld_k_out, ofmt, wsl::as_stream(stream)));
}

size_t sample_logits_workspace_bytes(int64_t n_rows, int64_t vocab) {
    if (n_rows <= 0 || n_rows > 65535 || vocab <= 0 || vocab > wsl::kMaxSampleVocab) return 0;
    return wsl::sample_ws_bytes(n_rows, vocab);
}

int sample_logits(const void *d_logits, int zfmt, int64_t n_rows, int64_t vocab, int64_t ld,
                  const wsl_sampling *h_settings, const float *d_u, int32_t *d_tokens, float *d_probs, int64_t ld_probs,
                  void *d_ws, size_t ws_bytes, uint32_t *d_status, void *stream) {
    int rc = wsl::check_sample(d_logits, zfmt, n_rows, vocab, ld, h_settings, d_u, d_tokens, d_probs, ld_probs);
    if (rc != WSL_OK || n_rows == 0) return rc;
    if ((rc = wsl::check_workspace(d_ws, ws_bytes, wsl::sample_ws_bytes(n_rows, vocab), 16)) != WSL_OK) return rc;
    if ((rc = wsl::device_ok()) != WSL_OK) return rc;
    return wsl::after_launch(wsl::launch_sample(d_logits, zfmt, n_rows, vocab, ld, h_settings, d_u, d_tokens, d_probs,
                                                ld_probs, d_ws, d_status, wsl::as_stream(stream)));
}

size_t lora_add_workspace_bytes(int64_t m, int64_t rank, int64_t k) {
    return m > 0 && wsl::lora_shape_ok(m, rank, k) ? wsl::lora_ws_bytes(m, rank, k) : 0;
}

int lora_add(const void *d_a, const void *d_b, int64_t n_adapters, int64_t rank, int64_t n_out, int64_t k,
             const int32_t *d_ids, const float *d_scales, const void *d_x, int64_t m, int64_t ldx, const void *d_base,
             int64_t ld_base, void *d_out, int64_t ld_out, int fmt, void *d_ws, size_t ws_bytes, uint32_t *d_status,
             void *stream) {
    int rc = wsl::check_lora(d_a, d_b, n_adapters, rank, n_out, k, d_ids, d_scales, d_x, m, ldx, d_base, ld_base, d_out,
                             ld_out, fmt);
    if (rc != WSL_OK || m == 0) return rc;
    if ((rc = wsl::check_workspace(d_ws, ws_bytes, wsl::lora_ws_bytes(m, rank, k), 16)) != WSL_OK) return rc;
    if ((rc = wsl::device_ok()) != WSL_OK) return rc;
    return wsl::after_launch(wsl::launch_lora(d_a, d_b, n_adapters, rank, n_out, k, d_ids, d_scales, d_x, m, ldx, d_base,
                                              ld_base, d_out, ld_out, fmt, d_ws, d_status, wsl::as_stream(stream)));
}

int wsl_stream_read(const void *d_buf, size_t bytes, uint32_t *d_sink, void *stream) {
    if (bytes == 0) return WSL_OK;
    if (!d_buf || !d_sink) return WSL_E_NULL;
    if ((bytes % 16) != 0) return WSL_E_SHAPE;
    if ((reinterpret_cast<uintptr_t>(d_buf) % 16) != 0 || (reinterpret_cast<uintptr_t>(d_sink) % 4) != 0)
        return WSL_E_ALIGN;
    int rc;
    if ((rc = wsl::device_ok()) != WSL_OK) return rc;
    return wsl::after_launch(wsl::launch_stream_read(d_buf, bytes, d_sink, wsl::as_stream(stream)));
}

const char *wsl_strerror(int code) {
    switch (code) {
        case WSL_OK: return "ok";
        case WSL_E_NULL: return "a required pointer is NULL";
        case WSL_E_SHAPE: return "invalid shape (non-positive size, k not a multiple of 64, or size overflow)";
        case WSL_E_ALIGN: return "misaligned pointer or leading dimension";
        case WSL_E_FORMAT: return "unknown weight or output format";
        case WSL_E_DEVICE: return "current device is not gfx950 (MI355X) or could not be queried";
        case WSL_E_LAUNCH: return "kernel launch failed";
        case WSL_E_RANGE: return "tile or workspace outside its matrix or buffer";
        case WSL_E_MEMORY: return "host buffer is not pinned (page-locked) host memory";
        case WSL_E_SCRATCH:
            return "linear_gemm_noalloc: the shape's split workspace exceeds WSL_NOALLOC_SCRATCH_BYTES "
                   "(use linear_gemm with a caller workspace)";
        case WSL_E_FLAGS: return "a flags argument holds a bit the call does not define";
        default: return "unknown status code";
    }
}

}  // extern "C"
