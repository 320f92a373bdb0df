/*
 * wsl.h -- C ABI of the weight-streaming linear library for AMD Instinct MI355X (gfx950).
 *
 * The library computes the linear layers y = W x of a decoder whose weights W
 * are held either as plain bf16 or as packed NF4 (4-bit codes in groups of 64
 * along K plus one fp16 scale per group).  NF4 weights stay packed in device
 * memory and are dequantized in registers inside the linear kernels; no dense
 * copy of W is ever written back.  Sources:
 *   - deep-fold README, "Метод" section: codes and scales live in video
 *     memory; linear kernels restore only the fragment of the current tile
 *     and never write a dense weight matrix back; a group of 64 weights holds
 *     4-bit NF4 codes and one FP16 scale; prefill is a GEMM that restores
 *     into BF16 register fragments for batches of up to 32 positions, decode
 *     an N=1 GEMV; both paths share one compressed representation (Figure 1).
 *   - TCPP README, "What exact means here": bf16 weights used as stored, no
 *     dequantization; "Quickstart"/"Performance": batch verification scores
 *     every position of a K-token context in one sweep (a wide GEMM).
 *   - IPE page, "What is built": a decode step indexes preallocated buffers
 *     with host integers and never reads device values back; "How it is
 *     checked": zero host-device synchronizations and zero allocator growth.
 *
 * Conventions for every entry point:
 *   - Shapes are int64_t.  W is [n_out][k] row-major (k contiguous), like a
 *     torch Linear weight; y = W x has n_out entries; the GEMM computes
 *     Y[m][n_out] = X[m][k] * W^T for m token positions.
 *   - Pointers named d_* or documented "device" are caller-owned device
 *     memory; "host" pointers are ordinary host memory.  The library never
 *     allocates, frees, copies or synchronizes: every call only validates its
 *     arguments on the host and enqueues kernels on `stream` (a hipStream_t;
 *     NULL means the default stream), so calls are legal inside HIP stream or
 *     graph capture.
 *   - Argument errors are returned synchronously, before anything is
 *     enqueued (nothing is launched).  Launch failures are reported as
 *     WSL_E_LAUNCH (from hipGetLastError, which does not synchronize).
 *     Errors in the *data* (non-finite weights) are reported through an
 *     optional device status word (nf4_pack only).
 *   - The library refuses any device other than gfx950 (WSL_E_DEVICE).
 *   - Results are deterministic: no floating-point atomics; the same inputs
 *     give the same bits on every run.
 *   - Calls that share output buffers and overlap on one device race; calls
 *     on the same stream are ordered.
 */
#ifndef WSL_H
#define WSL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes returned by every entry point. */
enum {
    WSL_OK = 0,
    WSL_E_NULL = 1,    /* a required pointer is NULL */
    WSL_E_SHAPE = 2,   /* a size <= 0 (or < 0 where 0 is allowed), k % 64 != 0, or a size overflow */
    WSL_E_ALIGN = 3,   /* a pointer or leading dimension breaks the documented alignment */
    WSL_E_FORMAT = 4,  /* unknown weight or output format */
    WSL_E_DEVICE = 5,  /* current device is not gfx950, or the device query failed */
    WSL_E_LAUNCH = 6,  /* a kernel launch failed */
    WSL_E_RANGE = 7,   /* a tile or workspace lies outside its matrix or buffer */
    WSL_E_MEMORY = 8,  /* a host buffer of a streamed call is not pinned (page-locked) host memory */
    WSL_E_SCRATCH = 9, /* linear_gemm_noalloc: the shape needs more split workspace than its scratch holds */
    WSL_E_FLAGS = 10   /* a flags argument holds a bit the call does not define */
};

/* Weight formats. */
enum { WSL_W_BF16 = 0, WSL_W_NF4 = 1 };
/* Output formats. */
enum { WSL_OUT_F32 = 0, WSL_OUT_BF16 = 1 };

/* Bits OR-ed into a call's optional device status word. */
#define WSL_STATUS_NONFINITE 1u   /* a group (or cache row) held a NaN or an infinity; verify_drafts, sample_logits: nothing to sample */
#define WSL_STATUS_OVERFLOW  2u   /* a group's absmax rounds to +inf in fp16 (>= 65520) */
#define WSL_STATUS_INDEX     4u   /* a row index, cache slot, page, length or draft was out of range */
#define WSL_STATUS_SWEEP_TIMEOUT 8u   /* linear_gemv_sweep: a stage barrier waited past its bound */
#define WSL_STATUS_DESCRIPTOR    16u  /* linear_gemv_sweep: a device stage descriptor was invalid (skipped) */
#define WSL_STATUS_PAGES         32u  /* kv_pages_grow: a sequence needed more pages than were free */

/* Flags of linear_gemv_streamed / linear_gemm_streamed. */
#define WSL_RING_PACE 1   /* the host keeps the copies at most two matrices ahead of the kernels */

/*
 * nf4_packed_bytes -- size in bytes of one packed NF4 matrix.
 *   = n_out*k/2 (codes, 4 bits each) + n_out*(k/64)*2 (fp16 scales),
 *   i.e. 17/32 byte per weight (deep-fold README, "Метод": the payload is
 *   about 3.76x smaller than BF16 for aligned matrices).
 *   Returns 0 if n_out <= 0, k <= 0, k % 64 != 0 or the size overflows.
 */
size_t nf4_packed_bytes(int64_t n_out, int64_t k);

/*
 * nf4_codebook -- copies the 16 binary32 NF4 levels (ascending; c[0] = -1,
 * c[7] = +0, c[15] = +1) into host memory out_host[0..15].  The levels are
 * normal quantiles with an exact zero, scaled to [-1, 1] (NF4 as introduced
 * in QLoRA, credited in deep-fold README, "Метод").  Returns WSL_E_NULL if
 * out_host is NULL.
 */
int nf4_codebook(float *out_host);

/*
 * nf4_pack -- encode a bf16 weight matrix into the packed NF4 device layout.
 *   (deep-fold README, "Метод": per group of 64 weights, 4-bit NF4 codes and
 *   one FP16 scale; the compressor there runs offline on the CPU.)
 * d_w       device, bf16 [n_out][k], 16-byte aligned (read only).
 * n_out, k  n_out >= 1, k >= 64, k % 64 == 0.
 * d_packed  device, nf4_packed_bytes(n_out, k) bytes, 16-byte aligned (written).
 * d_status  device uint32 or NULL.  If non-NULL, the kernel ORs
 *           WSL_STATUS_* bits into it for groups it cannot encode (the
 *           caller zeroes it first).  Such a group is written as s = +0 with
 *           every code 7, i.e. as zeros.
 * Encoding per row and group of 64 consecutive k: s = fp16_RNE(max|w|);
 * code = nearest level to w/s with ties to the lower index, decided
 * exactly as #{i : w > m_i * s} in fp64, m_i = (c_i + c_{i+1}) / 2; an
 * all-zero or fp16-underflowing group stores s = +0 and codes 7.
 * Layout written:
 *   codes  bytes [0, n_out*k/2): row-major, two codes per byte (even k in the
 *          low nibble), and every aligned little-endian 32-bit word (codes
 *          k = 8j..8j+7 of a row) rotated left by 2 bits;
 *   scales fp16 following the codes; rows in blocks of 16 (the last block
 *          may have rb < 16 rows), ordered [group][row] inside a block:
 *          scale(n, g) at index (n/16)*16*(k/64) + g*rb + n%16.
 * Bit-exact and deterministic.
 */
int nf4_pack(const void *d_w, int64_t n_out, int64_t k, void *d_packed,
             uint32_t *d_status, void *stream);

/*
 * nf4_dequant_tile -- restore a rectangular tile of a packed NF4 matrix to bf16.
 *   (deep-fold README, "Метод": kernels restore only the current tile's
 *   fragment into BF16.)  A test and diagnostic export: the linear kernels
 *   restore tiles in registers and never call it.
 * Value written for (r, c): bf16_RNE(fp32_RN(level[code] * s)) of weight
 * (row0 + r, k0 + c).  Tile: rows x cols at d_tile[r*ld_tile + c] (bf16).
 * Requires 0 <= row0, rows >= 1, row0 + rows <= n_out, 0 <= k0, cols >= 1,
 * k0 + cols <= k (else WSL_E_RANGE), ld_tile >= cols, d_tile 2-byte aligned.
 */
int nf4_dequant_tile(const void *d_packed, int64_t n_out, int64_t k,
                     int64_t row0, int64_t k0, int64_t rows, int64_t cols,
                     void *d_tile, int64_t ld_tile, void *stream);

/*
 * linear_gemv -- decode (one position): y[n] = sum_k W[n][k] * x[k], fp32 result.
 *   (deep-fold README, "Метод" table: decode is an N=1 NF4 GEMV; TCPP
 *   README: bf16 weights used as stored.)
 * wfmt      WSL_W_BF16: d_w is bf16 [n_out][k], 16-byte aligned;
 *           WSL_W_NF4 : d_w is a packed NF4 matrix (nf4_pack layout).
 * d_x       device bf16 [k], 16-byte aligned.   d_y device fp32 [n_out], 4-byte aligned.
 * n_out >= 1; k >= 64 and k % 64 == 0 for NF4; k >= 8 and k % 8 == 0 for bf16.
 * Accumulation is fp32.  NF4 multiplies the binary32 level by x and applies
 * the fp32 scale once per group partial sum; each row satisfies
 * |y - y_exact| <= 1e-4 * sum_k |w_hat x| with w_hat = level * s exactly.
 */
int linear_gemv(int wfmt, const void *d_w, int64_t n_out, int64_t k,
                const void *d_x, float *d_y, void *stream);

/* One stage of linear_gemv_sweep: y = W x with W a packed NF4 [n_out][k] matrix. */
typedef struct wsl_gemv_stage {
    const void *w;   /* device, packed NF4 (nf4_pack layout), 16-byte aligned */
    const void *x;   /* device, bf16 [k], 16-byte aligned */
    float *y;        /* device, fp32 [n_out], 4-byte aligned */
    int64_t n_out;   /* >= 1 */
    int64_t k;       /* 64 <= k <= 32768, k % 64 == 0 */
} wsl_gemv_stage;

/*
 * linear_gemv_sweep_workspace_bytes -- size of the synchronization workspace that
 * linear_gemv_sweep needs (a few KB of counters).
 */
size_t linear_gemv_sweep_workspace_bytes(void);

/*
 * linear_gemv_sweep -- a decode sweep: `count` NF4 GEMVs (the linear stages of every
 * layer of a decoder, in decoder order) in one launch.
 *   (deep-fold README, "Метод" table: decode runs N=1 NF4 GEMVs inside one graph of
 *   the whole greedy step; a token's step sweeps every layer's weights once.)
 * Computes, for i = 0 .. count-1, what linear_gemv(WSL_W_NF4, ...) of stage i computes
 * (same per-row tolerance: |y - y_exact| <= 1e-4 * sum_k |w_hat x|).  The stages run in
 * order: no part of stage i + 1 starts (nor reads its x) before every part of stage i
 * has finished (a device-wide barrier between stages); the loads of its weights may
 * begin earlier.  No stage may read another stage's output: every y must be disjoint
 * from every w and x of the call.  Every y is written when the call completes.
 * wfmt       WSL_W_NF4 (bf16 weights return WSL_E_FORMAT).
 * count      number of stages, 0 <= count <= 2^24 (0 enqueues nothing).
 * h_stages   host array of count descriptors: every argument is validated from it
 *            before anything is enqueued (as linear_gemv validates; k <= 32768).
 * d_stages   device array holding the same count descriptors (8-byte aligned), which
 *            the kernel reads.  If the two differ the results are undefined; a device
 *            descriptor that is invalid is skipped and WSL_STATUS_DESCRIPTOR is ORed
 *            into the status word.
 * d_ws       device workspace of at least linear_gemv_sweep_workspace_bytes() bytes,
 *            128-byte aligned, all zero before the first call; every call leaves it
 *            zero again except the status word, its uint32 at byte offset 1280, into
 *            which WSL_STATUS_SWEEP_TIMEOUT / WSL_STATUS_DESCRIPTOR bits are ORed (a
 *            caller that sees a nonzero status zeroes the workspace before reuse).
 *            Calls that share a workspace must not overlap.
 * The call launches one workgroup per compute unit and needs all of them resident at
 * once (nothing else occupying the GPU's compute units); a barrier that is not reached
 * within about a second is abandoned with WSL_STATUS_SWEEP_TIMEOUT so the kernel always
 * ends.  Deterministic: the same inputs give the same bits.
 */
int linear_gemv_sweep(int wfmt, int64_t count, const wsl_gemv_stage *h_stages,
                      const wsl_gemv_stage *d_stages, void *d_ws, size_t ws_bytes, void *stream);

/*
 * linear_gemv_multi -- several independent bf16 GEMVs in one launch: y_i = W_i x_i for
 * i < count, bit for bit what count linear_gemv calls give.  For matrices that read the
 * same k and none of whose outputs another reads -- a layer's q, k and v projections, or
 * its gate and up projections, kept as separate tensors (TCPP README, "What 'exact' means
 * here": weights used as stored) -- so that they share one launch instead of paying one
 * launch each (IPE page, "How it is benchmarked": a decode step's linear layers).
 * wfmt      WSL_W_BF16 (WSL_W_NF4: WSL_E_FORMAT; linear_gemv_sweep serves NF4 layers).
 * count     0 <= count <= WSL_GEMV_MULTI_MAX; 0 enqueues nothing.
 * h_stages  host array of count descriptors (read before the call returns), each with
 *           linear_gemv's bf16 arguments: w bf16 [n_out][k] 16-byte aligned, x bf16 [k]
 *           16-byte aligned, y fp32 [n_out] 4-byte aligned, n_out >= 1, k >= 8,
 *           k % 8 == 0; every descriptor has the same k (else WSL_E_SHAPE).
 * Returns linear_gemv's errors for a bad descriptor; asynchronous on stream.
 */
#define WSL_GEMV_MULTI_MAX 8
int linear_gemv_multi(int wfmt, int64_t count, const wsl_gemv_stage *h_stages, void *stream);

/*
 * linear_gemm_workspace_bytes -- workspace linear_gemm can use for a shape
 * (0 if it would not split the reduction): splits * m * n_out * 4 bytes of fp32
 * partials, for a k split of the shared-X kernels or of the 256 x 256 tiles
 * (a launch whose tiles would leave most compute units idle).  Passing a smaller
 * (or NULL) workspace is legal and only selects a path with less parallelism.
 */
size_t linear_gemm_workspace_bytes(int wfmt, int64_t n_out, int64_t k, int64_t m);

/*
 * linear_gemm -- prefill / batch verification: Y[i][n] = sum_k X[i][k] * T[n][k].
 *   (deep-fold README, "Метод" table: prefill is an NF4 GEMM that restores
 *   weights into BF16 register fragments; TCPP README, "Quickstart" and
 *   "Performance": batch verification over thousands of positions.)
 * T is the bf16 weight (WSL_W_BF16) or the restored bf16 tile value
 * bf16_RNE(fp32_RN(level * s)) (WSL_W_NF4).  Products are accumulated in fp32
 * on the matrix cores (MFMA); Y is written as fp32 (WSL_OUT_F32) or rounded
 * once to bf16 (WSL_OUT_BF16, round to nearest even).
 * d_x       device bf16 [m][ldx], ldx >= k, ldx % 8 == 0, 16-byte aligned.
 * d_y       device [m][ldy] of the output type, ldy >= n_out, aligned to its element size.
 * m >= 1.   n_out, k as for linear_gemv (k % 64 == 0 for both formats).
 * d_ws      optional device workspace (16-byte aligned) of ws_bytes bytes.
 *           It holds split-reduction partials; its contents on entry do not
 *           matter.  Calls that share a workspace and overlap race.
 */
int linear_gemm(int wfmt, const void *d_w, int64_t n_out, int64_t k,
                const void *d_x, int64_t m, int64_t ldx,
                void *d_y, int ofmt, int64_t ldy,
                void *d_ws, size_t ws_bytes, void *stream);

/*
 * linear_gemm_noalloc -- linear_gemm for callers that cannot allocate device memory:
 * code under HIP graph capture, tight serving loops, harnesses that forbid hipMalloc.
 * Same arguments and kernels as linear_gemm; instead of a caller workspace, the
 * split-reduction partials go to a scratch array of WSL_NOALLOC_SCRATCH_BYTES that the
 * library holds in device memory of every GPU it runs on, from the first call on that GPU
 * until the process ends.  The call itself allocates nothing: on its first call on a device
 * it looks up that device's copy of the array (hipGetSymbolAddress), afterwards it only
 * enqueues kernels.  When the shape's split workspace (linear_gemm_workspace_bytes) fits in
 * the scratch, the results are bit for bit those of linear_gemm given that workspace.
 * Beyond it, a shape that runs on the 256 x 256 tiles runs them without a k split (bit for
 * bit linear_gemm without a workspace), and any other shape returns WSL_E_SCRATCH,
 * launching nothing (4 MiB is enough for every shape at up to 32 positions with
 * k % 256 == 0, the prefill width); linear_gemm with a caller workspace serves those.
 * Every call on one GPU shares that GPU's scratch: calls
 * that overlap on one device (different streams, or different host threads without
 * ordering) race and may return wrong results; calls ordered on one stream do not.
 */
#define WSL_NOALLOC_SCRATCH_BYTES ((size_t)4 << 20)
int linear_gemm_noalloc(int wfmt, const void *d_w, int64_t n_out, int64_t k,
                        const void *d_x, int64_t m, int64_t ldx,
                        void *d_y, int ofmt, int64_t ldy, void *stream);

/*
 * nf4_embed_rows -- restore only the requested rows of a packed NF4 matrix (a
 * packed embedding table [n_rows][k]).
 *   (deep-fold README, introduction and Figure 1: embeddings stay packed and
 *   only the rows that are asked for are restored, separately from the linear
 *   kernels.)
 * d_packed  device, nf4_pack layout of an [n_rows][k] matrix, 16-byte aligned.
 * d_ids     device int64 [count], the rows to restore (any order, repeats allowed),
 *           8-byte aligned.  Read by the kernel only: indices are never copied
 *           to the host.
 * count     >= 0 (0 launches nothing; d_ids and d_out may then be NULL).
 * d_out     device [count][ld_out], 16-byte aligned; row i receives row d_ids[i]:
 *           WSL_OUT_BF16: bf16_RNE(fp32_RN(level * s)) (the restored tile value,
 *                         bit-identical to nf4_dequant_tile), ld_out % 8 == 0;
 *           WSL_OUT_F32 : fp32_RN(level * s), ld_out % 4 == 0.
 *           ld_out >= k; entries past k are not written.
 * d_status  device uint32 or NULL.  An index outside [0, n_rows) gives an
 *           all-zero output row and ORs WSL_STATUS_INDEX into *d_status.
 * Bit-exact and deterministic.
 */
int nf4_embed_rows(const void *d_packed, int64_t n_rows, int64_t k, const int64_t *d_ids, int64_t count,
                   void *d_out, int ofmt, int64_t ld_out, uint32_t *d_status, void *stream);

/*
 * linear_gemv_streamed / linear_gemm_streamed -- the linear kernels over matrices
 * that live in pinned host memory, brought to the device through two reusable
 * caller-owned device slots (a copy ring).
 *   (deep-fold README, "Метод" table and Figure 1: a model larger than the GPU
 *   budget keeps selected packed matrices in pinned host memory and passes them
 *   through two reusable device slots to the same kernels; the 32B model of the
 *   results keeps 9.5 GiB resident and 6.7 GiB in pinned host memory.)
 * For matrix i (slot s = i % 2) the call enqueues:
 *   copy_stream:    wait events[2 + s]; copy h_w[i] -> d_slot[s]; record events[s];
 *   compute_stream: wait events[s]; linear_gemv / linear_gemm on d_slot[s];
 *                   record events[2 + s].
 * So the copy of matrix i + 1 runs while matrix i is multiplied, and a slot is
 * overwritten only after the kernel that read it finished (also across calls,
 * since the events carry over).  Without WSL_RING_PACE the call enqueues everything
 * without waiting (it may be captured in a graph).  With it, before enqueueing the copy
 * of matrix i >= 2 the host waits for events[2 + s] -- the kernel of matrix i - 2, which
 * that copy waits for on the device anyway -- so the call returns once the kernel of
 * matrix count - 3 has finished.  The pacing is for long streams: when hundreds of copies
 * that each wait on a kernel of another stream are enqueued ahead, the HIP runtime can
 * hold the host inside a copy's enqueue for milliseconds, long enough for the copy engine
 * to run out of queued copies; kept two matrices ahead, the ring stays within a few
 * percent of the rate of plain back-to-back copies.
 * wfmt          WSL_W_NF4 or WSL_W_BF16, the format of every h_w[i].
 * count         number of matrices (>= 0; 0 enqueues nothing).
 * h_w           host array of count pointers to page-locked host buffers (allocated
 *               with hipHostMalloc; any other host memory gives WSL_E_MEMORY), each
 *               holding a matrix in its device format (nf4_pack layout, or bf16
 *               [n_out][k]).  They must stay allocated until the copies complete.
 * n_out, k      host arrays of count shapes (as for linear_gemv / linear_gemm).
 * d_x, d_y      host arrays of count device pointers: GEMV x bf16 [k] and y fp32
 *               [n_out]; GEMM X bf16 [m][ldx] and Y [m][ldy] of type ofmt.
 * m, ldx, ldy, ofmt, d_ws, ws_bytes   GEMM only, shared by every matrix (the
 *               workspace is used by one kernel at a time: all run on compute_stream).
 * d_slot        host array of 2 device pointers, 16-byte aligned, slot_bytes each;
 *               every matrix must fit (else WSL_E_RANGE).
 * copy_stream, compute_stream   hipStream_t (NULL = default stream); inputs and
 *               outputs are ordered on compute_stream.
 * events        host array of 4 hipEvent_t created by the caller.
 * flags         0 or WSL_RING_PACE (other bits: WSL_E_FLAGS).
 * Every argument is validated before anything is enqueued; a HIP error while
 * enqueuing (or waiting, with WSL_RING_PACE) returns WSL_E_LAUNCH (earlier matrices
 * may already be enqueued).
 */
int linear_gemv_streamed(int wfmt, int64_t count, const void *const *h_w, const int64_t *n_out, const int64_t *k,
                         const void *const *d_x, float *const *d_y, void *const *d_slot, size_t slot_bytes,
                         void *copy_stream, void *compute_stream, void *const *events, int flags);
int linear_gemm_streamed(int wfmt, int64_t count, const void *const *h_w, const int64_t *n_out, const int64_t *k,
                         const void *const *d_x, int64_t m, int64_t ldx, void *const *d_y, int ofmt, int64_t ldy,
                         void *d_ws, size_t ws_bytes, void *const *d_slot, size_t slot_bytes,
                         void *copy_stream, void *compute_stream, void *const *events, int flags);

/* Formats of a key-value cache. */
enum { WSL_KV_BF16 = 0, WSL_KV_E4M3 = 1 };

/*
 * A paged key-value cache of one layer, described by the caller (host struct, read before a
 * call returns).  Keys and values are [n_pages][n_kv][page_size][head_dim] each, with the
 * strides given here (the same for both): a token's slot is page * page_size + its place in
 * the page.  A sequence's tokens lie in the pages its row of a block table names, in order.
 *   (deep-fold README, "Метод" table: a decode step reads only the valid prefix of the cache;
 *   IPE page, "What is built": a decode step indexes preallocated buffers.)
 * fmt        WSL_KV_BF16, or WSL_KV_E4M3: 8-bit codes (1 sign, 4 exponent, 3 fraction bits, no
 *            infinities) with one power of two per token and kv head: with a = max|x| over the
 *            head_dim elements, e is the least integer >= -110 with a <= 448 * 2^e, a code is
 *            the e4m3 number nearest to x * 2^-e (ties to even), its value code * 2^e, and the
 *            scale byte e + 127.  A row that holds a NaN or an infinity is kept as NaN codes
 *            with scale byte 127.
 * k, v       device, 16-byte aligned.
 * k_exp, v_exp   device uint8 [n_pages][n_kv][page_size], contiguous (E4M3; else ignored).
 * n_pages    1 .. 2^31 - 1.   page_size 1 .. 2^30, any number.   n_kv 1 .. 2^20.
 * head_dim   16 .. 256, a multiple of 16.
 * page_stride, head_stride, token_stride   in elements, >= head_dim, multiples of 16 bytes.
 */
typedef struct wsl_kv_cache {
    void *k, *v;
    uint8_t *k_exp, *v_exp;
    int64_t fmt;
    int64_t n_pages, n_kv, page_size, head_dim;
    int64_t page_stride, head_stride, token_stride;
} wsl_kv_cache;

/*
 * kv_cache_write -- put the keys and values of count tokens into their slots, rounded to bf16
 * (to nearest even) or quantised as above.
 * d_k, d_v   device [count][ld_k] / [count][ld_v] of xfmt (WSL_OUT_F32 as linear_gemv gives
 *            them, or WSL_OUT_BF16): n_kv * head_dim elements a token, heads in order; 16-byte
 *            aligned, ld_k, ld_v >= n_kv * head_dim and multiples of 16 bytes (so views of a
 *            fused projection's output serve).
 * count      >= 0 (0 launches nothing); count * n_kv <= 2^26.
 * d_slots    device int64 [count]; -1: the token is not kept.  Two tokens of one call must not
 *            name the same slot.
 * d_status   device uint32 or NULL: WSL_STATUS_INDEX is ORed in if a slot is outside the cache
 *            (nothing is written for it), WSL_STATUS_NONFINITE if an E4M3 row held a NaN or an
 *            infinity.
 */
int kv_cache_write(const wsl_kv_cache *h_cache, const void *d_k, const void *d_v, int xfmt, int64_t count,
                   int64_t ld_k, int64_t ld_v, const int64_t *d_slots, uint32_t *d_status, void *stream);

/*
 * kv_cache_read -- the keys and values held in count slots (repeats allowed), as bf16 or fp32:
 * exact in both (a row whose largest element rounded up to 2^128 holds an infinity there, as its
 * bf16 rounding would).  Arguments as for kv_cache_write, d_k and d_v written in ofmt.  Slot -1 gives
 * zeros; a slot outside the cache gives zeros and WSL_STATUS_INDEX.
 */
int kv_cache_read(const wsl_kv_cache *h_cache, const int64_t *d_slots, int64_t count, void *d_k, void *d_v, int ofmt,
                  int64_t ld_k, int64_t ld_v, uint32_t *d_status, void *stream);

/*
 * attn_decode -- attention of the q_len newest tokens of each of n_seq sequences over the
 * sequence's cached keys and values (its own included: write them first).
 *   (TCPP README, "Quickstart": a line of drafted tokens is scored in one sweep; deep-fold
 *   README, "Метод" table: decode reads the valid prefix of the cache.)
 * For sequence b with L = d_kv_lens[b] tokens, query i stands at position p = L - q_len + i and
 * sees the tokens t <= p (with window > 0 only t > p - window):
 *   out = sum_t exp(s_t - max s) V_t / sum_t exp(s_t - max s),   s_t = scale * <q, K_t>,
 * head h reading kv head h / (n_heads / n_kv).  A query that sees nothing (p < 0), or only scores of
 * -infinity, gives zeros.
 * Tokens a query does not see have no part in it, whatever their slots hold.
 * d_q        device [n_seq * q_len][ld_q] of qfmt (WSL_OUT_F32 or WSL_OUT_BF16), n_heads *
 *            head_dim elements a token; 16-byte aligned, ld_q a multiple of 16 bytes.
 * n_seq      0 .. 65535 (0 launches nothing).  q_len 1 .. 256.  n_heads a multiple of n_kv.
 *            q_len * n_heads / n_kv <= 2^16, q_len * n_heads <= 2^24, and n_seq * n_kv *
 *            (ceil(pages_per_seq * page_size / 128) + 4) <= 2^30.
 * d_block_table   device int32 [n_seq][ld_table]: page of token t of a sequence at [t / page_size];
 *            pages_per_seq (1 .. ld_table) entries of a row may be read.
 * d_kv_lens  device int32 [n_seq]: read by the kernels only, so a captured call goes on with
 *            lengths that grow.  One outside [0, pages_per_seq * page_size] is clamped to it
 *            and reported; so is, as if it were not seen, a token that a query sees and whose page is
 *            outside [0, n_pages) (entries of pages that lie wholly behind the window may be anything).
 * scale      the factor of the scores.  window >= 0 (0: none).
 * d_out      device [n_seq * q_len][ld_out] of ofmt, 16-byte aligned, ld_out a multiple of 16 bytes.
 * d_lse      device fp32 [n_seq][q_len][n_heads] or NULL: log sum_t exp(s_t), -infinity where
 *            the sum is zero (for joining with attention over tokens kept elsewhere).
 * d_ws       device workspace, 16-byte aligned, of attn_decode_workspace_bytes (else WSL_E_RANGE):
 *            the length is split over the chip by the actual lengths, and parts of one head are
 *            joined by a second launch.  Its contents on entry do not matter.  Calls that share
 *            a workspace must not overlap.
 * d_status   device uint32 or NULL: WSL_STATUS_INDEX as above.
 * Scores, maxima, sums and products with V are held in fp32.  The matrix instructions take bf16:
 * fp32 queries enter them as three bf16 numbers (24 bits), and so do the weights, but as two (16
 * bits) where queries and result are both bf16.  The sums over V are divided last: they overflow
 * where sum_t exp(s_t - max s) |V_t| reaches 2^128.  Deterministic.
 */
size_t attn_decode_workspace_bytes(int qfmt, int64_t n_seq, int64_t q_len, int64_t n_heads, int64_t n_kv,
                                   int64_t head_dim, int64_t pages_per_seq, int64_t page_size);
int attn_decode(const wsl_kv_cache *h_cache, const void *d_q, int qfmt, int64_t n_seq, int64_t q_len, int64_t n_heads,
                int64_t ld_q, const int32_t *d_block_table, int64_t ld_table, int64_t pages_per_seq,
                const int32_t *d_kv_lens, float scale, int64_t window, void *d_out, int ofmt, int64_t ld_out,
                float *d_lse, void *d_ws, size_t ws_bytes, uint32_t *d_status, void *stream);

/*
 * verify_drafts -- which drafted tokens the target's probabilities let stand, and the token that
 * follows them, from given random numbers.
 *   (TCPP README, "Quickstart": batch verification scores every position in one sweep; Tarfa 2,
 *   "Speculative decoding".)
 * For each of n_seq sequences with n drafts x_0 .. x_{n-1}, rows p_0 .. p_n of the target, rows
 * q_0 .. q_{n-1} of the drafter and numbers u_0 .. u_width:
 *   draft i stands iff all before it do and u_i * q_i(x_i) < p_i(x_i); r = how many stand;
 *   w_j = max(p_r(j) - q_r(j), 0) if r < n, else max(p_n(j), 0); if they sum to 0, max(p_r(j), 0);
 *   the next token is the least j with w_0 + .. + w_j > u_width * sum w.
 * With u uniform in [0, 1) and x_i drawn from q_i, every token has the target's distribution.
 * All of it in 64 bits.  NaN and negative weights count as zero; where no sum passes (u >= 1 or
 * NaN) the last entry with a weight is taken.
 * d_p        device [n_seq][width + 1][ld_p] of pfmt (WSL_OUT_F32 or WSL_OUT_BF16), the first
 *            vocab of each row used; aligned to its element.
 * d_q        device [n_seq][width][ld_q] of pfmt, or NULL: the drafter was certain (q_i = 1 at x_i).
 * n_seq      0 .. 65535 (0 launches nothing).  width 0 .. 64 (0: p_0 is sampled).
 * vocab      1 .. 2^30.
 * d_drafts   device int32 [n_seq][width].  A draft outside [0, vocab) falls (WSL_STATUS_INDEX).
 * d_n_drafts device int32 [n_seq] or NULL (width for all): n, clamped to [0, width].
 * d_u        device fp32 [n_seq][width + 1].
 * d_accepted device int32 [n_seq]: r.   d_tokens device int32 [n_seq][width + 1]: the r drafts
 *            that stand, the next token, then -1.  If the weights do not sum to a positive finite
 *            number the next token is -1 (WSL_STATUS_NONFINITE).
 * d_ws       device workspace, 16-byte aligned, of verify_drafts_workspace_bytes (else WSL_E_RANGE;
 *            none where that is 0: small vocabularies).
 *            Its contents on entry do not matter.  Calls that share a workspace must not overlap.
 */
#define WSL_VERIFY_MAX_DRAFTS 64
size_t verify_drafts_workspace_bytes(int64_t n_seq, int64_t vocab);
int verify_drafts(const void *d_p, const void *d_q, int pfmt, int64_t n_seq, int64_t width, int64_t vocab,
                  int64_t ld_p, int64_t ld_q, const int32_t *d_drafts, const int32_t *d_n_drafts, const float *d_u,
                  int32_t *d_accepted, int32_t *d_tokens, void *d_ws, size_t ws_bytes, uint32_t *d_status,
                  void *stream);

/*
 * The pages of a key-value cache kept on the device, described by the caller (host struct, read
 * before a call returns): which pages each sequence holds, how long it is, and which are free.
 *   (IPE page, "What is built": a decode step indexes preallocated buffers and never reads device
 *   values back; deep-fold README, "Метод": a whole greedy step is one graph.)
 * table      device int32 [n_seq][ld_table]: the block table that attn_decode reads; a sequence of L
 *            tokens holds the first ceil(L / page_size) entries of its row.
 * lens       device int32 [n_seq]: the tokens of each sequence (attn_decode's d_kv_lens).
 * free_pages device int32 [n_pages], a stack: its first *n_free entries are the free pages.
 * n_free     device int32 [1].
 * n_seq 0 .. 65535.  pages_per_seq 1 .. ld_table.  n_pages 1 .. 2^31 - 1.  page_size 1 .. 2^30.
 * A sequence holds at most pages_per_seq * page_size tokens, and 2^31 - 1.  A page is held by one sequence, or free:
 * one that two rows name is given back twice.
 */
typedef struct wsl_kv_pages {
    int32_t *table, *lens, *free_pages, *n_free;
    int64_t n_seq, pages_per_seq, ld_table, n_pages, page_size;
} wsl_kv_pages;

/*
 * kv_pages_grow -- take in new tokens: the pages they need, their cache slots and positions.
 * Sequence b grows by d_new[b] tokens (by `each` where d_new is NULL).  The pages it lacks are taken
 * off the top of the stack, in the order of sequences and of their places; its lens and the stack
 * are moved on.  A call is made once for a step, before the layers' kv_cache_write.
 * d_new       device int32 [n_seq] or NULL.      each   >= 0 (d_new NULL; else ignored).
 * n_tokens    0 .. 2^30: room in d_slots and d_positions.
 * d_slots     device int64 [n_tokens]: the slots for kv_cache_write; the tokens of sequence b lie at
 *             starts[b] .. starts[b] + new[b] - 1, starts the running sum of new.  -1 where there
 *             is no token, or one that is not taken in.
 * d_positions device int64 [n_tokens] or NULL: the tokens' positions in their sequences, or -1.
 * d_starts    device int32 [n_seq + 1] or NULL: starts and their end (at most n_tokens each).
 * A sequence is left as it is, and its tokens get -1, where
 *   - more pages are needed, by it and those before it, than are free (WSL_STATUS_PAGES): from
 *     the first one on only sequences that need no page grow;
 *   - its lens or new is negative, it would grow past its row, or its tokens past n_tokens
 *     (WSL_STATUS_INDEX).  It then asks for no page.
 * A token whose page number is outside [0, n_pages) gets -1 (WSL_STATUS_INDEX).  An *n_free outside
 * [0, n_pages] is clamped to it and reported.
 * d_ws        device workspace, 16-byte aligned, of kv_pages_grow_workspace_bytes (none where that is
 *             0).  Its contents on entry do not matter.  Calls that share a workspace, or the same
 *             pages, must not overlap.
 * d_status    device uint32 or NULL.
 */
size_t kv_pages_grow_workspace_bytes(int64_t n_seq, int64_t n_tokens);
int kv_pages_grow(const wsl_kv_pages *h_pages, const int32_t *d_new, int64_t each, int64_t n_tokens, int64_t *d_slots,
                  int64_t *d_positions, int32_t *d_starts, void *d_ws, size_t ws_bytes, uint32_t *d_status,
                  void *stream);

/*
 * kv_pages_trim -- shorten sequences to d_lens[b] tokens (fallen drafts; 0 for one that is done) and
 * give the pages behind them back.  Of R pages given back, the r-th in the order of sequences
 * and places comes to lie at free_pages[*n_free + R - 1 - r]: growing again by as much takes the same
 * pages.  Table entries are left as they are.  A length at or above a sequence's own leaves it as
 * it is.
 * d_lens     device int32 [n_seq].  A negative one (or a lens outside the row) leaves the sequence as it
 *            is and ORs WSL_STATUS_INDEX into the status word; pages that the stack has no room for are
 *            dropped and reported so too.
 */
int kv_pages_trim(const wsl_kv_pages *h_pages, const int32_t *d_lens, uint32_t *d_status, void *stream);

/*
 * rotary_embed -- rotary positions: pairs of a head's elements turned by position * frequency.
 *   (Between the fused projection of linear_gemm and kv_cache_write / attn_decode.)
 * For the token at position p and pair i < rot_dim / 2, with the angle p * freqs[i]:
 *   (a, b) -> amplitude * (a cos - b sin, a sin + b cos),
 * a and b the elements i and i + rot_dim / 2 of the head (or, with WSL_ROTARY_INTERLEAVED, 2i and
 * 2i + 1); elements from rot_dim on are copied.  Angles are formed and reduced in two 64-bit numbers
 * each: cos and sin are right to 2^-24 where |p * freqs[i]| < 2^48, the products and sums are in fp32.
 * d_q, d_k     device [count][ld] of xfmt (WSL_OUT_F32 or WSL_OUT_BF16): n_heads (n_kv) * head_dim elements a
 *              token; 16-byte aligned, ld a multiple of 16 bytes (views of a fused projection serve).
 *              d_k may be NULL (then d_k_out is ignored).
 * d_q_out, d_k_out   the same of ofmt; each may be its input itself where ofmt is xfmt (and the lds
 *              are equal).  Other overlaps are not allowed.
 * count >= 0 (0 launches nothing).  n_heads, n_kv 1 .. 2^16.  head_dim 16 .. 256, a multiple of 16.
 * rot_dim      2 .. head_dim, even.
 * count * (n_heads + n_kv) * head_dim <= 2^40.
 * d_positions  device int64 [count], any (kv_pages_grow's -1 too).
 * d_freqs      device float64 [rot_dim / 2], radians a position: scaling for long contexts is in them.
 * amplitude    finite.      flags   0 or WSL_ROTARY_INTERLEAVED.
 */
#define WSL_ROTARY_INTERLEAVED 1
int rotary_embed(const void *d_q, int64_t n_heads, int64_t ld_q, const void *d_k, int64_t n_kv, int64_t ld_k, int xfmt,
                 int64_t count, int64_t head_dim, int64_t rot_dim, const int64_t *d_positions, const double *d_freqs,
                 double amplitude, int flags, void *d_q_out, int64_t ld_q_out, void *d_k_out, int64_t ld_k_out, int ofmt,
                 void *stream);

/* Settings of sample_logits (host struct): one value for all rows, or (device, [n_rows]) one for each. */
typedef struct wsl_sampling {
    const float *d_temperature;      /* device or NULL: temperature for all */
    const int32_t *d_top_k;
    const float *d_top_p, *d_min_p;
    float temperature;
    int32_t top_k;
    float top_p, min_p;
} wsl_sampling;

/*
 * sample_logits -- tokens from logits and given random numbers, and the distribution they come from.
 *   (What follows the packed head's GEMM, and, with d_probs, what verify_drafts takes as p and q.)
 * A row's entries z are ordered by value, equal ones by index.
 *   K: the first top_k entries (all where top_k <= 0);
 *   w_j = exp((z_j - max z) / temperature);
 *   P: the entries of K before which less than top_p * (sum of w over K) lies (all where top_p >= 1);
 *   Q: those with w_j >= min_p (all where min_p <= 0; none where it is above 1).
 * The entries in K, P and Q, always the first one, are kept; the token is the least j with
 *   sum of the kept w_0 .. w_j > u * (sum of all kept), or the last kept where none is (u >= 1 or NaN),
 * and probs_j = w_j / (sum of all kept), 0 for the rest.  Where temperature is not above 0 the first
 * entry alone is kept.  A NaN in top_p or min_p counts as off.  Weights and their sums are right to 2^-32,
 * exact where all weights are equal; decisions are made in 64 bits.  The same call gives the same bits; with other
 * rows beside it a long row may be cut elsewhere, and a decision as near to its border as 2^-32 fall the other way.
 * Entries of -infinity are out.  A row that holds a NaN or +infinity, or nothing but -infinity, gives
 * token -1, probabilities 0, and WSL_STATUS_NONFINITE.
 * d_logits   device [n_rows][ld] of zfmt (WSL_OUT_F32 or WSL_OUT_BF16), the first vocab of each row used;
 *            aligned to its element.
 * n_rows     0 .. 65535 (0 launches nothing).      vocab 1 .. 2^22.
 * h_settings NULL: temperature 1, nothing off.
 * d_u        device fp32 [n_rows]; may be NULL where d_tokens is.
 * d_tokens   device int32 [n_rows] or NULL.     d_probs  device fp32 [n_rows][ld_probs] or NULL; one of
 *            them is needed.  Entries of a row past vocab are not written.
 * d_ws       device workspace, 16-byte aligned, of sample_logits_workspace_bytes (none where that is 0; more
 *            rows never take less).  Its contents on entry do not matter.  Calls that share a workspace must not overlap.
 */
size_t sample_logits_workspace_bytes(int64_t n_rows, int64_t vocab);
int sample_logits(const void *d_logits, int zfmt, int64_t n_rows, int64_t vocab, int64_t ld,
                  const wsl_sampling *h_settings, const float *d_u, int32_t *d_tokens, float *d_probs, int64_t ld_probs,
                  void *d_ws, size_t ws_bytes, uint32_t *d_status, void *stream);

/*
 * lora_add -- low-rank adapters of many requests at once, beside a projection they share:
 *   out[t] = base[t] + scale[a] * B[a] (A[a] x[t]),  a = ids[t]; out[t] = base[t] where ids[t] is -1.
 *   (base is what linear_gemm gives for the packed matrix, which no adapter changes.)
 * d_a       device bf16 [n_adapters][rank][k], d_b device bf16 [n_adapters][n_out][rank]: contiguous,
 *           16-byte aligned.  An adapter of a smaller rank has zeros in its last rows of A (or columns of B).
 * n_adapters 1 .. 2^20.   rank 8 .. 128, a multiple of 8.   n_out 1 .. 2^22.   k 8 .. 2^22, a multiple of 8.
 * d_ids     device int32 [m].  One outside [-1, n_adapters) counts as -1 (WSL_STATUS_INDEX).
 * d_scales  device fp32 [n_adapters], or NULL: 1.
 * d_x       device bf16 [m][ldx], 16-byte aligned, ldx a multiple of 8.   m 0 .. 2^20 (0 launches nothing).
 * d_base    device [m][ld_base] of fmt (WSL_OUT_F32 or WSL_OUT_BF16), aligned to its element.
 * d_out     device [m][ld_out] of fmt; may be d_base itself (with the same ld), no other overlap.
 * A x is summed in fp32 and scaled there; its product with B too.  (On the matrix cores A x enters as
 * three bf16 numbers, 24 bits; there an infinity in B gives a NaN.)  The sum with base is rounded once to
 * fmt.  Rows without an adapter are copied.  An adapter has no part in other tokens' rows, whatever
 * it holds.  Deterministic.
 * d_ws      device workspace, 16-byte aligned, of lora_add_workspace_bytes (A x in parts of k; more tokens
 *           never take less).  Its contents on entry do not matter.  Calls that share a workspace must not overlap.
 */
size_t lora_add_workspace_bytes(int64_t m, int64_t rank, int64_t k);
int lora_add(const void *d_a, const void *d_b, int64_t n_adapters, int64_t rank, int64_t n_out, int64_t k,
             const int32_t *d_ids, const float *d_scales, const void *d_x, int64_t m, int64_t ldx, const void *d_base,
             int64_t ld_base, void *d_out, int64_t ld_out, int fmt, void *d_ws, size_t ws_bytes, uint32_t *d_status,
             void *stream);

/*
 * wsl_stream_read -- measurement aid, not part of the linear path: a read-only
 * kernel that reads bytes bytes at d_buf once, with the access form of the GEMV
 * weight stream (16-byte loads that bypass the caches, 1 KB of consecutive bytes
 * per wave instruction; one 8-wave workgroup per compute unit, three such
 * loads in flight per wave), so that its rate over a buffer much larger than
 * the caches is the streaming-read ceiling the GB/s
 * figures are compared with (a figure the pages do not give: measured on the GPU at hand).
 * d_buf    device, 16-byte aligned; bytes a multiple of 16.  bytes == 0 enqueues
 *          nothing and returns 0.
 * d_sink   device uint32 [1], 4-byte aligned: each lane XOR-combines the words it
 *          reads and writes the result to d_sink[0] only if it equals 0x9e3779b9,
 *          so the kernel writes nothing in practice (a test plants that value to
 *          check that every word is read).
 * Returns WSL_E_NULL, WSL_E_SHAPE (bytes % 16 != 0), WSL_E_ALIGN, WSL_E_DEVICE or
 * WSL_E_LAUNCH as the other entry points do; asynchronous on stream.
 */
int wsl_stream_read(const void *d_buf, size_t bytes, uint32_t *d_sink, void *stream);

/* wsl_strerror -- static description of a status code (never NULL). */
const char *wsl_strerror(int code);

#ifdef __cplusplus
}
#endif

#endif /* WSL_H */
