// Host-side argument validation of the C ABI (no HIP dependency).
//
// Every entry point validates its arguments here before it enqueues anything,
// so a caller error returns a status code and launches nothing.  This unit is
// plain C++ so it can be built with g++ and exercised under AddressSanitizer
// and UndefinedBehaviorSanitizer on a machine without a GPU.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace wsl {

constexpr int64_t kGroup = 64;          // NF4 group size along k
constexpr int64_t kScaleRowBlock = 16;  // rows per scale block in the device layout

// Size of a packed NF4 matrix, or 0 if the shape is invalid or the size overflows.
size_t nf4_bytes(int64_t n_out, int64_t k);

int check_pack(const void *w, int64_t n_out, int64_t k, const void *packed);
int check_dequant_tile(const void *packed, int64_t n_out, int64_t k, int64_t row0, int64_t k0,
                       int64_t rows, int64_t cols, const void *tile, int64_t ld_tile);
int check_gemv(int wfmt, const void *w, int64_t n_out, int64_t k, const void *x, const void *y);
int check_gemm(int wfmt, const void *w, int64_t n_out, int64_t k, const void *x, int64_t m,
               int64_t ldx, const void *y, int ofmt, int64_t ldy, const void *ws, size_t ws_bytes);
// Copy-ring arguments: the flags, the arrays, the slots, the events, and for each matrix
// check_gemv / check_gemm with the slot as the weight pointer plus the slot size.
// m < 0 selects the GEMV checks.
int check_ring(int wfmt, int64_t count, const void *const *h_w, const int64_t *n_out, const int64_t *k,
               const void *const *x, int64_t m, int64_t ldx, const void *const *y, int ofmt, int64_t ldy,
               const void *ws, size_t ws_bytes, const void *const *slot, size_t slot_bytes, const void *const *events,
               int flags);
// Decode sweep: count in [0, 2^24], the host descriptors (each as check_gemv for NF4,
// plus k <= 32768), the device descriptor array and the workspace.
int check_sweep(int wfmt, int64_t count, const void *h_stages, const void *d_stages, const void *ws,
                size_t ws_bytes, size_t ws_need);
// Several GEMVs in one launch: bf16 only, count in [0, WSL_GEMV_MULTI_MAX], each descriptor
// as check_gemv, every k equal.
int check_multi(int wfmt, int64_t count, const void *h_stages);
int check_embed(const void *packed, int64_t n_rows, int64_t k, const void *ids, int64_t count, const void *out,
                int ofmt, int64_t ld_out);

// A wsl_kv_cache, then kv_cache_write / kv_cache_read: rows outside the cache of type fmt.
int check_kv_cache(const void *h_cache);
int check_kv_rows(const void *h_cache, const void *k, const void *v, int fmt, int64_t count, int64_t ld_k, int64_t ld_v,
                  const void *slots);
int check_attn_shape(int qfmt, int64_t n_seq, int64_t q_len, int64_t n_heads, int64_t n_kv, int64_t head_dim,
                     int64_t pages_per_seq, int64_t page_size);
int check_attn(const void *h_cache, const void *q, int qfmt, int64_t n_seq, int64_t q_len, int64_t n_heads,
               int64_t ld_q, const void *table, int64_t ld_table, int64_t pages_per_seq, const void *lens, float scale,
               int64_t window, const void *out, int ofmt, int64_t ld_out, const void *lse);
int check_verify(const void *p, const void *q, int pfmt, int64_t n_seq, int64_t width, int64_t vocab, int64_t ld_p,
                 int64_t ld_q, const void *drafts, const void *n_drafts, const void *u, const void *accepted,
                 const void *tokens);
// A wsl_kv_pages, then what a call is asked for.
int check_kv_pages(const void *h_pages);
int check_grow(const void *h_pages, const void *d_new, int64_t each, int64_t n_tokens, const void *slots,
               const void *positions, const void *starts);
int check_trim(const void *h_pages, const void *lens);
int check_rotary(const void *q, int64_t n_heads, int64_t ld_q, const void *k, int64_t n_kv, int64_t ld_k, int xfmt,
                 int64_t count, int64_t head_dim, int64_t rot_dim, const void *positions, const void *freqs,
                 double amplitude, int flags, const void *q_out, int64_t ld_q_out, const void *k_out, int64_t ld_k_out,
                 int ofmt);
int check_sample(const void *logits, int zfmt, int64_t n_rows, int64_t vocab, int64_t ld, const void *h_settings,
                 const void *u, const void *tokens, const void *probs, int64_t ld_probs);
int check_lora(const void *a, const void *b, int64_t n_adapters, int64_t rank, int64_t n_out, int64_t k, const void *ids,
               const void *scales, const void *x, int64_t m, int64_t ldx, const void *base, int64_t ld_base,
               const void *out, int64_t ld_out, int fmt);
bool lora_shape_ok(int64_t m, int64_t rank, int64_t k);
// A workspace of ws_bytes at ws where need bytes are needed.
int check_workspace(const void *ws, size_t ws_bytes, size_t need, size_t alignment);

// Upper bound on any single dimension accepted by the library (keeps every
// derived index within int64 and every per-row byte offset within int32).
constexpr int64_t kMaxDim = int64_t(1) << 30;
constexpr int64_t kMaxSampleVocab = int64_t(1) << 22;
constexpr int64_t kMaxLoraDim = int64_t(1) << 22;

}  // namespace wsl
