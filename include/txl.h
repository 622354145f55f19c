/*
 * txl.h - C ABI of the GB300 (sm_103a) Transformer-XL relative-position
 * attention library.
 *
 * The operations follow "Transformer-XL: Attentive Language Models Beyond a
 * Fixed-Length Context" (Dai et al.):
 *   - §3.2, segment-level recurrence: the hidden states of earlier segments are
 *     cached (a memory of length M per layer) and prepended, without gradient,
 *     to the current segment as extended context for keys and values;
 *   - §3.3, the relative score
 *       A_ij = q_i.k_j + q_i.W_kR R_{i-j} + u.k_j + v.W_kR R_{i-j}
 *     with the sinusoid table R, then a masked softmax over the extended
 *     context and a product with the values (the N-layer summary);
 *   - Appendix B, the reversed table Q_k = W_kR R_{M+L-1-k} and the left shift
 *     that turns q Q^T into the position term, which the kernel realises by
 *     index arithmetic inside its tiles.
 *
 * Conventions for every entry point:
 *   - All pointers are device pointers unless stated otherwise.  The caller owns
 *     every buffer; the library keeps no reference after the call returns.
 *   - Work is enqueued on `stream` (a cudaStream_t; NULL is the legacy default
 *     stream) and the call returns once it is launched.  Inputs must stay valid
 *     and unmodified until the stream reaches the work.
 *   - Arguments are validated on the host before anything is launched; a bad
 *     argument returns an error code and enqueues nothing.
 *   - Kernels that wait on on-chip barriers give up after a time limit and
 *     record TXL_ERR_TIMEOUT in a device status word; txl_device_status()
 *     reads and clears it.
 *   - Return values are txl_status codes (0 = success).
 */
#ifndef TXL_H
#define TXL_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    TXL_OK = 0,
    TXL_ERR_INVALID_ARG = -1, /* null pointer, negative size, bad dtype code */
    TXL_ERR_UNSUPPORTED = -2, /* a shape or dtype the library has no kernel for */
    TXL_ERR_MISALIGNED = -3,  /* a pointer breaks the stated alignment */
    TXL_ERR_SHAPE = -4,       /* sizes inconsistent with each other */
    TXL_ERR_CUDA = -5,        /* a CUDA runtime or driver call failed */
    TXL_ERR_TIMEOUT = -6,     /* a kernel gave up waiting on an on-chip barrier */
    TXL_ERR_WORKSPACE = -7,   /* workspace missing or too small for the request */
    TXL_ERR_INDEX = -8        /* an index held on the device was out of range (page ids, parents,
                                 source rows, token ids); debug builds: any device-side index check */
} txl_status;

typedef enum {
    TXL_F32 = 0, /* IEEE binary32 */
    TXL_BF16 = 1 /* bfloat16 */
} txl_dtype;

/* Human-readable name of a status code (static string, never NULL). */
const char *txl_status_string(int status);

/* Library version: major*10000 + minor*100 + patch. */
int txl_version(void);

/*
 * txl_rel_pos_emb - the sinusoid relative encoding table R of §3.3 ("R is a
 * sinusoid encoding matrix without learnable parameters"; row p stands for a
 * relative distance of p), written in Appendix B's reversed row order.
 *
 *   R     [K][d_model], dtype `dtype` (TXL_F32 or TXL_BF16), row-major.
 *         Row rho holds distance p = K-1-rho:
 *           R[rho][2k]   = sin(p * w_k),  R[rho][2k+1] = cos(p * w_k),
 *           w_k = 10000^(-2k/d_model).
 *         Multiplying by W_kR^T gives the per-head operand `r` of
 *         txl_relattn_fwd.
 *   K >= 1, d_model even and >= 2.  R must be 4-byte aligned.
 * Errors: TXL_ERR_INVALID_ARG (null R, K < 1, odd or non-positive d_model,
 * bad dtype), TXL_ERR_MISALIGNED, TXL_ERR_CUDA.
 */
int txl_rel_pos_emb(void *R, int K, int d_model, int dtype, void *stream);

/*
 * txl_relattn_workspace_size - bytes of device workspace txl_relattn_fwd needs
 * when it splits the key range of a head over `n_splits` thread blocks
 * (n_splits <= 1 needs none).  Pure host arithmetic.
 */
size_t txl_relattn_workspace_size(int B, int H, int L, int dh, int n_splits);

/* Kernels txl_relattn_fwd may run (reported by txl_relattn_plan). */
typedef enum {
    TXL_KERNEL_TC = 1,     /* bf16: tensor cores (tcgen05, TMEM, TMA), 128-row query tiles */
    TXL_KERNEL_DECODE = 2, /* bf16, L = 1: split-K decode kernel on the CUDA cores, fp32 */
    TXL_KERNEL_F32 = 3,    /* fp32: CUDA cores */
    TXL_KERNEL_DECODE_MMA = 4 /* bf16, 2 <= L <= 8: split-K decode kernel, warp-level tensor-core MMAs */
} txl_kernel;

/*
 * txl_relattn_plan - the kernel and the split txl_relattn_fwd would use for a
 * call with these arguments and a workspace of `workspace_bytes` bytes (0 = no
 * workspace; a non-zero size stands for a 256-byte aligned workspace).  Host
 * arithmetic plus cached device attributes of the current device; launches
 * nothing.
 *   *kernel  a txl_kernel value
 *   *splits  key ranges per query tile (TXL_KERNEL_TC) or per (b, h)
 *            (TXL_KERNEL_DECODE, TXL_KERNEL_DECODE_MMA); 1 for TXL_KERNEL_F32
 * Returns the status the call would return for its sizes (TXL_ERR_WORKSPACE
 * when the split needs more workspace than given), or TXL_ERR_INVALID_ARG for
 * NULL outputs.
 */
int txl_relattn_plan(int B, int H, int M, int L, int r_rows, int dh, int dtype, int n_splits,
                     size_t workspace_bytes, int *kernel, int *splits);

/*
 * txl_relattn_fwd - forward relative-position attention of one layer over the
 * extended context (§3.2 recurrence, §3.3 score and N-layer summary,
 * Appendix B shift).
 *
 * With K = M + L keys (memory rows first, then the segment), for every batch
 * b, head h, query i in [0,L) and key j in [0,K):
 *   delta  = M + i - j                        (relative distance)
 *   A_ij   = scale * ((q_i + u).k_j + (q_i + v_bias).r[row(delta)])  if delta >= 0
 *   A_ij   = -inf                                                     otherwise
 *   out_i  = sum_j softmax_j(A_i.) v_j,   lse_i = log sum_j exp(A_ij)
 * where r[row] = W_kR R_{distance} in Appendix B's reversed order: with
 * r_rows rows per head, row(delta) = r_rows - 1 - delta.  A table built for
 * exactly K keys has r_rows = K; a longer table (r_rows > K, e.g. cached for the
 * largest memory) is used as is.
 *
 * Layouts (dense, row-major, innermost dimension dh contiguous):
 *   q   [B][H][L][dh]        k, v [B][H][K][dh]
 *   r   [H][r_rows][dh]      u, v_bias [H][dh]
 *   out [B][H][L][dh]        lse [B][H][L] fp32, natural log (may be NULL)
 * dtype TXL_BF16: q, k, v, r, u, v_bias and out are bf16; scores, softmax and
 *   accumulation are fp32 on the tensor cores (tcgen05).  dh must be 64; q, k,
 *   v and r must be 16-byte aligned.  Segments of L <= 8 queries (decoding a
 *   few new tokens against a long memory) always take a split-K decode kernel
 *   instead: from L = 2 on the tensor cores' warp-level MMAs with q + u, q + v
 *   and P each carried as a bf16 pair (value and residual), for L = 1 the CUDA
 *   cores in fp32; either way the error before the output's bf16 rounding is
 *   far below that rounding (txl_relattn_plan tells which kernel).  For it n_splits
 *   counts key ranges per (b, h), each a whole number of 32-key chunks,
 *   at most one per 128 keys (larger requests are capped, ranges that would
 *   hold no key are dropped); up to 8 ranges of a head run as one thread-block
 *   cluster and merge in distributed shared memory, needing no workspace.
 * dtype TXL_F32: every tensor is fp32 and the arithmetic is fp32 on the CUDA
 *   cores (no TF32).  dh must be 64.
 * M >= 0, L >= 1, r_rows >= K, B >= 1, H >= 1.
 *
 * n_splits: 0 lets the library choose; 1 processes each head's keys in one
 * thread block; n > 1 splits the key range over n blocks and merges their
 * partial results (needs txl_relattn_workspace_size(B,H,L,dh,n) bytes of
 * workspace, 256-byte aligned, owned by the caller, contents undefined on
 * return).  A workspace that is NULL or too small limits the automatic choice
 * to 1 and makes an explicit n > 1 fail with TXL_ERR_WORKSPACE.
 *
 * Errors: TXL_ERR_INVALID_ARG, TXL_ERR_UNSUPPORTED (dh != 64, bad dtype),
 * TXL_ERR_MISALIGNED, TXL_ERR_SHAPE (r_rows < K), TXL_ERR_WORKSPACE,
 * TXL_ERR_CUDA.
 */
int txl_relattn_fwd(const void *q, const void *k, const void *v, const void *r, int r_rows,
                    const void *u, const void *v_bias, void *out, float *lse, int B, int H,
                    int M, int L, int dh, float scale, int dtype, int n_splits,
                    void *workspace, size_t workspace_bytes, void *stream);

/*
 * txl_relattn_fwd_strided - txl_relattn_fwd with the (b, h) planes of k and v
 * kv_stride elements apart instead of K * dh, so that the K = M + L keys of each
 * plane can be a window of a larger buffer (the memory of §3.2 kept in place,
 * the segment's rows written behind it; see txl_kv_window below) and nothing
 * has to be concatenated before the call.
 *
 *   k, v  plane p = b*H + h starts at k + p * kv_stride (elements); within a
 *         plane the K rows of dh elements are contiguous, memory rows first.
 *         Only those K rows of each plane are read.
 *   kv_stride >= K * dh and a multiple of 8 (16 bytes of bf16: every plane
 *         starts 16-byte aligned when k and v do).
 * Everything else (q, r, u, v_bias, out, lse, n_splits, workspace, the
 * kernels, results and errors) is as for txl_relattn_fwd, which is this call
 * with kv_stride = K * dh.
 * Errors: those of txl_relattn_fwd; TXL_ERR_INVALID_ARG for kv_stride < 1,
 * TXL_ERR_SHAPE for kv_stride < K * dh, TXL_ERR_MISALIGNED for a kv_stride not
 * a multiple of 8.
 */
int txl_relattn_fwd_strided(const void *q, const void *k, const void *v, long long kv_stride,
                            const void *r, int r_rows, const void *u, const void *v_bias,
                            void *out, float *lse, int B, int H, int M, int L, int dh,
                            float scale, int dtype, int n_splits, void *workspace,
                            size_t workspace_bytes, void *stream);

/*
 * TXL_NOALLOC_SCRATCH_BYTES - size of the scratch array built into the library
 * for txl_relattn_fwd_noalloc (32 MiB).
 */
#define TXL_NOALLOC_SCRATCH_BYTES (32u * 1024u * 1024u)

/*
 * txl_relattn_fwd_noalloc - txl_relattn_fwd for callers that cannot allocate
 * device memory when they run it (for example plugins of inference engines
 * whose execute step must not allocate, or runtimes whose device memory budget
 * is fixed at start-up).  The paper has no counterpart: this is a property of
 * the library, not of the method.
 *
 * Same arguments, layouts, results and errors as txl_relattn_fwd, without the
 * workspace.  When a head's key range is split over several blocks, the
 * partial results go to a scratch array that is part of the library: one
 * device array of TXL_NOALLOC_SCRATCH_BYTES that every GPU which loads the
 * library holds until the process exits.  The call itself allocates nothing
 * (no cudaMalloc, cudaFree or allocating library routine).
 *   - A split whose partial results need more than the scratch returns
 *     TXL_ERR_WORKSPACE and launches nothing.  What counts is the split the
 *     call runs, as txl_relattn_plan reports it for workspace_bytes =
 *     TXL_NOALLOC_SCRATCH_BYTES: requests above the key-tile count are capped
 *     first, and decode key ranges merged inside a thread-block cluster need
 *     no scratch; otherwise it needs txl_relattn_workspace_size(B, H, L, dh,
 *     splits) bytes.  n_splits = 0 chooses a split that fits (or none).
 *   - Every call shares the array and leaves its partial results in it; calls
 *     that may run at the same time on the GPU (other streams, or other host
 *     threads without ordering) race on it and must be serialised by the
 *     caller.
 *   - The first call on a device looks up the array's device address (a
 *     runtime query, done once per device with that device current); make that
 *     first call before any stream capture.
 */
int txl_relattn_fwd_noalloc(const void *q, const void *k, const void *v, const void *r,
                            int r_rows, const void *u, const void *v_bias, void *out, float *lse,
                            int B, int H, int M, int L, int dh, float scale, int dtype,
                            int n_splits, void *stream);

/*
 * Segment memory of one layer (§3.2: "cache a predefined length-M old hidden
 * states spanning (possibly) multiple segments"), kept as a ring buffer.
 *
 *   mem  [B][capacity][d] on the device, owned by the caller.
 *   txl_mem_state lives in HOST memory and is owned by the caller:
 *     head     slot that receives the next row
 *     fill     rows currently held (0..capacity)
 *     capacity M, the memory length
 * Logical row t (0 = oldest) of the fill rows sits in slot
 * (head - fill + t) mod capacity.  Initialise with {0, 0, M}.
 */
typedef struct {
    int head;
    int fill;
    int capacity;
} txl_mem_state;

/*
 * txl_mem_concat - the extended context h~ = [SG(m) o h] of §3.2 / §3.3 for
 * the current segment: ext[b] = the fill memory rows oldest-first, then the L
 * rows of h_new.  SG (stop-gradient) is the identity in a forward pass.
 *   ext   [B][fill + L][d]   h_new [B][L][d]   same dtype (TXL_F32 / TXL_BF16)
 * Rows are copied in 16-byte units: d * element size must be a multiple of 16
 * and every pointer 16-byte aligned.
 * Errors: TXL_ERR_INVALID_ARG, TXL_ERR_MISALIGNED, TXL_ERR_SHAPE, TXL_ERR_CUDA.
 */
int txl_mem_concat(void *ext, const void *mem, const txl_mem_state *st, const void *h_new,
                   int B, int L, int d, int dtype, void *stream);

/*
 * txl_mem_update - advance the memory with the current segment's states:
 * the memory becomes the newest `capacity` rows of [m o h_new] (§3.2, the
 * summary's m^n_tau).  Writes at most min(L, capacity) rows into the ring and
 * updates *st on the host (head advances by L mod capacity, fill saturates at
 * capacity).  Same layout and alignment rules as txl_mem_concat.
 * Errors: TXL_ERR_INVALID_ARG, TXL_ERR_MISALIGNED, TXL_ERR_SHAPE, TXL_ERR_CUDA;
 * *st is unchanged on error.
 */
int txl_mem_update(void *mem, txl_mem_state *st, const void *h_new, int B, int L, int d,
                   int dtype, void *stream);

/*
 * A memory of §3.2 ("a predefined length-M old hidden states spanning
 * (possibly) multiple segments") kept as a contiguous window of a larger
 * buffer, one window per plane (e.g. the projected keys or values of each
 * (batch, head)), so that [memory ; segment] is read in place by
 * txl_relattn_fwd_strided.
 *
 *   buf   [planes][capacity][d] on the device, owned by the caller.
 *   txl_kv_window lives in HOST memory and is owned by the caller:
 *     start     row of the oldest memory row in every plane
 *     fill      memory rows held (0..M)
 *     capacity  rows per plane of buf; at least 2 * M + L for segments of L rows
 *     M         memory length
 * Initialise with {0, 0, capacity, M}.  Per segment:
 *   txl_kv_window_append  puts the segment's L rows behind the memory rows;
 *                         afterwards rows [start, start + fill + L) of every
 *                         plane are [memory ; segment] (K = fill + L keys, at a
 *                         plane stride of capacity * d elements);
 *   (attention over that window)
 *   txl_kv_window_advance keeps the newest M rows as the memory (host only).
 */
typedef struct {
    int start;
    int fill;
    int capacity;
    int M;
} txl_kv_window;

/*
 * txl_kv_window_append - copy seg [planes][L][d] into rows start + fill ..
 * start + fill + L - 1 of every plane.  When those rows would run past the
 * buffer's end, the fill memory rows are first copied to rows 0 .. fill - 1 and
 * start becomes 0 (with capacity >= 2M + L the two ranges never overlap).
 * Same dtype and 16-byte rules as txl_mem_update.  Updates w->start on the host.
 * Errors: TXL_ERR_INVALID_ARG (bad state, sizes, pointers or dtype),
 * TXL_ERR_SHAPE (capacity < 2M + L), TXL_ERR_MISALIGNED, TXL_ERR_CUDA; *w is
 * unchanged on error.
 */
int txl_kv_window_append(void *buf, txl_kv_window *w, const void *seg, int planes, int L, int d,
                         int dtype, void *stream);

/*
 * txl_kv_window_advance - after attending to a segment of L rows appended by
 * txl_kv_window_append: the memory becomes the newest min(fill + L, M) rows of
 * [memory ; segment] (§3.2, the summary's m^n_tau).  Host arithmetic only.
 * Errors: TXL_ERR_INVALID_ARG (bad state, L < 0), TXL_ERR_SHAPE (the window
 * would run past the buffer: the segment was not appended).
 */
int txl_kv_window_advance(txl_kv_window *w, int L);

/*
 * txl_qkv_project - one layer's projections for a segment, written where the
 * attention reads them, with the memory update in the same launch ("Transformer-XL:
 * Attentive Language Models Beyond a Fixed-Length Context", §3.3 N-layer
 * summary: q = h W_q^T and k, v = h~ W_kE^T, h~ W_v^T, of which only the
 * segment's rows are new when the memory's k and v are kept in a window; §3.2:
 * the memory takes the newest states).  One GEMM, Y = h W^T over the stacked
 * weights, on the tensor cores (bf16 in, fp32 accumulate, bf16 out), whose
 * epilogue writes
 *   q      [B][H][L][dh]                               (when q != NULL)
 *   k, v   rows start + fill .. start + fill + L - 1 of the window planes of
 *          kv_buf: keys in planes 0 .. B*H-1, values in planes B*H .. 2*B*H-1
 *          ([2*B*H][capacity][dh], plane = b*H + h), exactly as
 *          txl_kv_window_append would place them (moving the memory rows to
 *          the buffer's front first when needed; updates kv_win->start)
 *   mem    the memory ring [B][capacity][d_model] advanced as txl_mem_update
 *          would (when mem != NULL; updates *mem_st)
 * h [B][L][d_model]; w [n_out * H * dh][d_model] with n_out = 3 (rows W_q,
 * W_kE, W_v, head-major inside each) when q != NULL, else 2 (W_kE, W_v).
 * All bf16, dense, 16-byte aligned; dh must be 64 and d_model a multiple of 8.
 * The caller owns every buffer and both states (host memory).  Asynchronous on
 * `stream`.  Errors: TXL_ERR_INVALID_ARG (NULL h, w, kv_buf or kv_win, bad
 * sizes or states, mem without mem_st), TXL_ERR_UNSUPPORTED (dh != 64),
 * TXL_ERR_SHAPE (window capacity < 2M + L, ring row width), TXL_ERR_MISALIGNED,
 * TXL_ERR_CUDA; the states are unchanged on error.
 */
int txl_qkv_project(const void *h, const void *w, int B, int L, int d_model, int H, int dh,
                    void *q, void *kv_buf, txl_kv_window *kv_win, void *mem,
                    txl_mem_state *mem_st, void *stream);

/*
 * txl_relattn_bwd - backward of txl_relattn_fwd for one segment (training
 * backpropagates within a segment, "Transformer-XL: Attentive Language Models
 * Beyond a Fixed-Length Context" §3.2; the memory is SG(m): no gradient leaves
 * through it, but its projected keys and values receive one like the
 * segment's).  With A_ij the §3.3 score times `scale`, P = softmax_j(A) over
 * the kept keys (j <= i + M), O = P v and dout = dL/dO:
 *   D_i   = sum_j P_ij (dout_i . v_j)
 *   g_ij  = scale P_ij (dout_i . v_j - D_i)
 *   dq_i  = sum_j g_ij (k_j + r(M+i-j))       dk_j = sum_i g_ij (q_i + u)
 *   dv_j  = sum_i P_ij dout_i                 du   = sum_{b,i,j} g_ij k_j
 *   dr(d) = sum_{b, i-j = d-M} g_ij (q_i + v) dv_bias = sum_{b,i,j} g_ij r(M+i-j)
 * where r(d) is the table row of distance d (row r_rows - 1 - d of r).  P is
 * recomputed; so are its log-sum-exp and D (exactly, in fp32): nothing from the
 * forward call is needed.
 * Inputs, bf16, dense and 16-byte aligned, layouts as txl_relattn_fwd:
 *   q, dout [B][H][L][dh]   k, v [B][H][M+L][dh]   r [H][r_rows][dh]
 *   u, v_bias [H][dh]
 * Outputs, fp32, dense, written (not accumulated), 16-byte aligned:
 *   dq [B][H][L][dh]   dk, dv [B][H][M+L][dh]   dr [H][r_rows][dh] (rows of
 *   distances >= M+L are zero)   du, dv_bias [H][dh]
 * workspace: txl_relattn_bwd_workspace_size(B, H, L, M) bytes of device
 * memory, 256-byte aligned (per-row statistics, per-block bias and dq
 * partials, and g of every query-key pair: B*H*L rows of M+L rounded up to 64
 * fp32, from which the table gradient is summed); 0 for sizes out of range.  The sums
 * over the batch and the key splits are ordered, so results repeat bit for
 * bit.  dh must be 64 and dtype
 * TXL_DTYPE_BF16.  Asynchronous on `stream`.  Errors: TXL_ERR_INVALID_ARG
 * (NULL pointer, bad sizes), TXL_ERR_UNSUPPORTED (dh, dtype, sizes past the
 * grid limits), TXL_ERR_SHAPE (r_rows < M+L), TXL_ERR_MISALIGNED,
 * TXL_ERR_WORKSPACE, TXL_ERR_CUDA.
 */
size_t txl_relattn_bwd_workspace_size(int B, int H, int L, int M);
int txl_relattn_bwd(const void *q, const void *k, const void *v, const void *r, int r_rows,
                    const void *u, const void *v_bias, const void *dout, float *dq, float *dk,
                    float *dv, float *dr, float *du, float *dv_bias, int B, int H, int M, int L,
                    int dh, float scale, int dtype, void *workspace, size_t workspace_bytes,
                    void *stream);

/*
 * Paged memory.  The memory of §3.2 for sequences whose lengths differ and
 * change on the device: the projected keys and values of a sequence lie in pages
 * of page_rows rows, listed by a page table.  The paper keeps one memory length
 * for a batch; this form serves streams that begin, fork and advance apart (for
 * instance by the accepted part of a drafted tree).
 *
 *   pool    device [2 * layers][n_pages][H][page_rows][dh]: plane 2 l holds layer
 *           l's keys, plane 2 l + 1 its values; a page id names the same page
 *           of every plane.  16-byte aligned.
 *   table   device [B][slots] int32: page ids of a sequence.  Its table rows 0 ..
 *           R-1 (R = slots * page_rows) are a ring: table row x is row x mod
 *           page_rows of page table[b][x / page_rows].
 *   begin   device [B] int32 in [0, R): table row of the oldest memory row
 *   fill    device [B] int32 in [0, R]: memory rows held
 *   ticket  device, one int32, zero before the first use (left at zero)
 * Memory row t (0 = oldest) lies in table row (begin + t) mod R.  A memory that
 * slides (keep rows of it, below) comes around to its own oldest pages, so the
 * table of a sequence need not change as it advances; pages shared with another
 * sequence (a fork) have to be copied before rows are put into them.
 * dh must be 64, page_rows a multiple of 32 (a tile of keys never crosses a
 * page), dtype TXL_BF16 or TXL_F32.
 *
 * What lies on the device is checked on the device.  A page id outside
 * [0, n_pages) is never dereferenced: rows in it are not written and not
 * attended to.  begin and fill are brought into their ranges.  Either records
 * TXL_ERR_INDEX for txl_device_status.
 * The struct lives in HOST memory; its contents are read during the call.
 */
typedef struct {
    void *pool;
    const int *table;
    int *begin;
    int *fill;
    int *ticket;
    int layers;
    int n_pages;
    int H;
    int page_rows;
    int dh;
    int B;
    int slots;
    int dtype;
} txl_paged_kv;

/*
 * A [B][H][rows][dh] operand with strides, in elements, of its first three
 * dimensions (dh contiguous): for instance the heads of a projection's output
 * [B][rows][H * dh].  The pointer must be 16-byte aligned and the strides of
 * dimensions larger than one positive multiples of 16 bytes.
 */
typedef struct {
    void *ptr;
    long long stride_b, stride_h, stride_row;
} txl_rows;

/*
 * txl_paged_append - put new rows behind the memory (§3.2: the memory takes the
 * newest states) and, if asked, advance it.  For layers layer0 .. layer0 +
 * n_layers - 1, every sequence b, head and t < n_new[b]:
 *   memory row fill[b] + t  <-  row (rows ? rows[b][t] : t) of k and v
 *   k, v    layer layer0 + l of them starts l * layer_stride elements on
 *           (layer_stride is a multiple of 16 bytes); N rows each, outside the pool.
 *   n_new   device [B], values taken into [0, max_rows]; NULL: max_rows
 *   rows    device [B][rows_stride >= max_rows] of source rows in [0, N) (the
 *           accepted nodes of a drafted tree, say; the same row may come more
 *           than once), or NULL (then max_rows <= N)
 * A source row outside [0, N) and rows the table has no room for (fill + n >
 * R) are not written and record TXL_ERR_INDEX.
 * begin_out, fill_out (device [B], both or neither): the state advanced to the
 * newest `keep` rows (n' of n_new fit the table), keep in [0, R]:
 *   fill_out = min(fill + n', keep), begin_out = (begin + fill + n' - fill_out) mod R
 * They may be mem->begin and mem->fill themselves.  Then the call uses
 * mem->ticket, and calls on the same memory must not overlap in time; without
 * that, calls for different layers may.  They overlap neither the table, n_new nor rows
 * (TXL_ERR_INVALID_ARG), except that n_new may be one of them where they are the state.
 * Errors: TXL_ERR_INVALID_ARG, TXL_ERR_UNSUPPORTED (dh, page_rows, dtype, sizes
 * past the grid limits), TXL_ERR_MISALIGNED, TXL_ERR_SHAPE, TXL_ERR_CUDA.
 */
int txl_paged_append(const txl_paged_kv *mem, int layer0, int n_layers, const txl_rows *k,
                     const txl_rows *v, long long layer_stride, int N, const int *rows,
                     int rows_stride, const int *n_new, int max_rows, int keep, int *begin_out,
                     int *fill_out, void *stream);

/*
 * txl_paged_advance - the state part of txl_paged_append alone, for a caller
 * that appended layer by layer: begin_out, fill_out (which may be mem->begin
 * and mem->fill, and n_new one of them) from n_new (NULL: max_rows for every sequence), as
 * above.
 * Errors: as txl_paged_append.
 */
int txl_paged_advance(const txl_paged_kv *mem, const int *n_new, int max_rows, int keep,
                      int *begin_out, int *fill_out, void *stream);

/*
 * txl_paged_copy - copy pages src[i] to pages dst[i], i < n (device int32), in
 * every plane of the pool: a forked sequence's own copy of a page it will write,
 * or pages moved together.  No page may be a destination twice, nor a source
 * and a destination (unless src[i] = dst[i], which copies nothing).  A pair with
 * an id outside [0, n_pages) is skipped and records TXL_ERR_INDEX.
 * Errors: as txl_paged_append.
 */
int txl_paged_copy(const txl_paged_kv *mem, const int *src, const int *dst, int n, void *stream);

/*
 * txl_page_pool - host-side accounting of a pool's pages: which are free and by
 * how many sequences each is used.  The caller owns the struct and both arrays
 * of n_pages ints.  Host arithmetic only; not thread-safe.
 *   txl_page_pool_init     every page free
 *   txl_page_pool_alloc    n pages, each with one user; all or none: TXL_ERR_SHAPE when
 *                          fewer are free
 *   txl_page_pool_retain   one user more for each page (a fork shares it)
 *   txl_page_pool_release  one user less; a page without users is free again.
 *                          *n_freed (may be NULL): how many became free
 * Errors: TXL_ERR_INVALID_ARG (NULL pointers, negative counts, ids out of range,
 * pages that have no user; nothing is changed then).
 */
typedef struct {
    int n_pages;
    int n_free;
    int *free_list; /* ids of the free pages, the next one to hand out last */
    int *users;     /* per page */
} txl_page_pool;

int txl_page_pool_init(txl_page_pool *p, int n_pages, int *free_list, int *users);
int txl_page_pool_alloc(txl_page_pool *p, int *pages, int n);
int txl_page_pool_retain(txl_page_pool *p, const int *pages, int n);
int txl_page_pool_release(txl_page_pool *p, const int *pages, int n, int *n_freed);

/*
 * txl_relattn_tree_fwd - relative-position attention (§3.3) of a tree of
 * drafted tokens over a paged memory: the verification step of speculative
 * decoding, and with a chain of nodes (each the parent of the next) or a single
 * node an ordinary decoding step.  Node i of sequence b has parent parents[b][i]
 * in [0, i), or none (-1: it follows the memory directly; any other value is
 * taken as -1 and records TXL_ERR_INDEX).  Its depth d_i is 0 without a parent,
 * else its parent's plus one.  With F = fill[b] memory rows, for node i < n_b:
 *   memory row t   distance F + d_i - t
 *   node a         distance d_i - d_a, visible when a is i or an ancestor of i
 *   A_ij = scale * ((q_i + u).k_j + (q_i + v_bias).r[r_rows - 1 - distance])
 *   out_i = sum_j softmax_j(A_i.) v_j,  lse_i = log sum_j exp(A_ij)
 * over the visible nodes and memory rows whose distance is below r_rows (a
 * memory longer than the table is attended to as far as the table goes).  A node sees
 * itself at least.  Infinite values of what it sees show as in the formula, and so does a row
 * whose every score is -infinity (out NaN, lse -infinity); q.k and u.k, and q.r and
 * v_bias.r, are summed apart: infinities of unlike sign in them make the row NaN.
 *
 *   q, out        [B][H][N][dh]    (strided; out must not overlap the inputs, nor one
 *                 row of it another)
 *   k_new, v_new  [B][H][N][dh]    the nodes' keys and values
 *   mem, layer    the memory and the layer of it to read; nothing is written
 *   r             [H][r_rows][dh] dense, u, v_bias [H][dh]; as txl_relattn_fwd
 *   parents       device [B], parents_stride ints apart (0: one tree for all)
 *   n_nodes       device [B], values taken into [0, N]; NULL: N
 *   lse           [B][H][N] fp32 or NULL
 * Rows i >= n_b of out and lse are left as they were; those rows of q, k_new and
 * v_new, and what the pages hold outside the memory rows, have no influence.
 * All of mem->dtype.  TXL_BF16: products on the tensor cores, fp32 sums; the
 * probabilities enter as bf16 pairs (value and residual), or, for N > 16 (the width of the
 * call, whatever n_nodes says), rounded to one bf16 value.  TXL_F32: fp32 arithmetic.
 * 1 <= N <= 64, dh = 64.  mem's arrays, parents and n_nodes must not change while the call runs.
 * n_splits: key ranges per (b, h), merged inside a thread-block cluster: 0 lets
 * the library choose, at most 8 (larger requests are refused).  No workspace.
 * Errors: TXL_ERR_INVALID_ARG, TXL_ERR_UNSUPPORTED (N > 64, dh, page_rows, dtype,
 * n_splits > 8, sizes past the grid limits), TXL_ERR_MISALIGNED, TXL_ERR_SHAPE
 * (layer not in the pool, r_rows < 1), TXL_ERR_CUDA.
 */
int txl_relattn_tree_fwd(const txl_rows *q, const txl_rows *k_new, const txl_rows *v_new,
                         const txl_paged_kv *mem, int layer, const void *r, int r_rows,
                         const void *u, const void *v_bias, const int *parents,
                         long long parents_stride, const int *n_nodes, const txl_rows *out,
                         float *lse, int N, float scale, int n_splits, void *stream);

/*
 * The two ends of the model: the embedding of tokens (§3.3: h^0 is the word
 * embedding sequence) and the log probabilities of tokens under
 * softmax(h E^T) (§3: the language model's output), each with its gradient.  The
 * table may be tied (one [V][d] array for both).
 *
 * Token ids and targets lie on the device as int32 or int64 (txl_index_type).  -1
 * stands for none (padding); any other value outside [0, V) is taken as -1 and
 * records TXL_ERR_INDEX for txl_device_status.
 * Rows of d elements, d at most 65536 and (but for txl_embed_fwd) 16 bytes' worth or a
 * multiple: of 8 elements, of 4 where all rows are fp32 in txl_embed_bwd.  Row strides in
 * elements, multiples of 16 bytes, at least d (so h may be, say, the last position of every
 * segment); pointers of rows 16-byte, of other arrays as their element, workspaces 256-byte
 * aligned.  txl_embed_fwd takes any d, stride and element-aligned pointers.  Outputs and
 * workspaces that overlap inputs or one another are refused (TXL_ERR_INVALID_ARG), as are
 * scales that are not finite.  Workspaces are the caller's, their contents undefined before
 * and after; calls that may run at the same time need one each.  n, N and V up to 2^28; n or
 * N = 0 is allowed.
 */
typedef enum {
    TXL_I32 = 4,
    TXL_I64 = 8
} txl_index_type;

/*
 * txl_embed_fwd - out_t = scale * emb[token_t] (t < n), a row of zeros without a token.
 *   tokens [n]; emb [V] rows of d, emb_stride apart; out [n][d] dense.  emb and out of dtype
 *   (TXL_F32 or TXL_BF16); the product is rounded once, and with scale = 1 rows are
 *   copied bit for bit.
 * Errors: TXL_ERR_INVALID_ARG, TXL_ERR_UNSUPPORTED, TXL_ERR_MISALIGNED,
 * TXL_ERR_SHAPE (a stride below d), TXL_ERR_CUDA.
 */
int txl_embed_fwd(const void *tokens, int index_type, const void *emb, long long emb_stride,
                  void *out, int n, int V, int d, float scale, int dtype, void *stream);

/*
 * txl_embed_bwd - gradient of the table: demb_v = scale * sum_{t: token_t = v} dout_t.
 *   tokens [n]; dout [n] rows of d, dout_stride apart, of dtype; demb [V][d] dense of
 *   grad_dtype.  Every row of demb is written (zeros for tokens that do not occur); with
 *   accumulate, which needs grad_dtype TXL_F32, the sums are added to demb instead and other
 *   rows are left alone (the gradient of a tied table, say, after txl_logprob_bwd).
 *   dout of positions without a token is not read.
 * Sums are fp32, in an order that the tokens alone determine: results repeat bit for bit.
 *   workspace: txl_embed_bwd_workspace_size(n, V, d) bytes (0 for sizes out of range).
 * Errors: as txl_embed_fwd, and TXL_ERR_WORKSPACE.
 */
size_t txl_embed_bwd_workspace_size(int n, int V, int d);
int txl_embed_bwd(const void *tokens, int index_type, const void *dout, long long dout_stride,
                  void *demb, int n, int V, int d, float scale, int dtype, int grad_dtype,
                  int accumulate, void *workspace, size_t workspace_bytes, void *stream);

/*
 * txl_logprob_fwd - log probabilities of given tokens, the distributions' entropy and their
 * largest alternatives.  With z_ij = scale * h_i.w_j over the vocabulary, for i < N:
 *   lse_i     = log sum_j exp z_ij
 *   logp_i    = z_i,targets[i] - lse_i            (0 without a target)
 *   entropy_i = lse_i - sum_j p_ij z_ij,  p_ij = exp(z_ij - lse_i)
 *   top_ids[i][0 .. top-1]  the `top` largest z_ij in descending order, equal ones by
 *             ascending j;  top_logp the z - lse of them.  The top + 4 largest by their
 *             fp32 sums (up to 256 states without kept logits: those beside them in their fours too) are
 *             ordered by sums carried beyond fp32; of more logits within fp32's rounding of one another
 *             at the end of the list, which ones it holds goes by their fp32 sums.  NaN logits are not
 *             listed; places without a number hold id -1 and NaN.
 * The logits are not kept (with alternatives, those of up to 64 and d / 16 states pass through the workspace).
 *   h [N] rows, w [V] rows of d, strides apart, both of dtype; targets [N] or NULL
 *   logp, lse, entropy [N] fp32, top_logp [N][top] fp32, top_ids [N][top] int32: each may
 *   be NULL (the last two only when top = 0)
 *   top in [0, 16]
 * TXL_BF16: products on the tensor cores, fp32 sums.  TXL_F32: operands as three bf16 terms
 * each (their leading 24 bits; values beneath bf16's subnormals are lost), six products on
 * the tensor cores, fp32 sums; there an infinite element of h or w makes a logit it enters NaN.
 * The tensor cores cut each of a logit's d / 16 additions; it is scaled by the mean of that, which where nothing was
 * cut (a state with one element) is d 2^-30 of its value.  The target's logit and, with alternatives, the
 * largest are formed again without.  Sums of exponentials leave the largest's own 1 out, so log probabilities near 0
 * are as exact as others, relative to their size, down to about 2^-45 times
 * the largest logit.
 * A logit of -infinity has probability zero; a row with a logit of +infinity or NaN gives NaN.  Logits of more
 * than 2^128 ln 2 (2.35e38) in size count as infinite.
 *   workspace: txl_logprob_fwd_workspace_size(N, V, d, top, dtype) bytes (0 for arguments
 *   out of range).
 * Errors: as txl_embed_bwd; TXL_ERR_UNSUPPORTED for top > 16.
 */
size_t txl_logprob_fwd_workspace_size(int N, int V, int d, int top, int dtype);
int txl_logprob_fwd(const void *h, long long h_stride, const void *w, long long w_stride,
                    const void *targets, int index_type, float *logp, float *lse, float *entropy,
                    float *top_logp, int *top_ids, int N, int V, int d, int top, float scale,
                    int dtype, void *workspace, size_t workspace_bytes, void *stream);

/*
 * txl_logprob_bwd - gradients of h and w for dlogp = dL/dlogp and dentropy = dL/dentropy:
 *   G_ij = dlogp_i (1[j = targets[i]] - p_ij) - dentropy_i p_ij (log p_ij + entropy_i)
 *   dh_i = scale sum_j G_ij w_j          dw_j = scale sum_i G_ij h_i
 *   h, w, targets, scale as in the forward call; lse and entropy its outputs (entropy may be
 *   NULL without dentropy).  dlogp, dentropy [N] fp32: targets and dlogp are given together
 *   or both NULL; one of dlogp and dentropy at least is given.
 *   dh [N][d] dense of dtype, dw [V][d] dense of grad_dtype (TXL_F32 h and w: TXL_F32); one of
 *   them may be NULL.  Written, not accumulated.
 * A row without a target and with dentropy 0 (or NULL) has no part, whatever its h and
 * statistics hold: its dh is zero.
 * G enters its products rounded to bf16; as a bf16 pair (value and residual) with h for an fp32
 * dw of bf16 operands, and in both products for N <= 128; and for fp32 operands as three terms.
 * Sums are fp32 in a fixed order: results repeat bit for bit.  The tensor cores cut each of their additions;
 * fp32 results are sums of parts of at most 512 of them, each scaled by the mean of what they cut, which where
 * nothing was cut (one term among zeros) is 8.2e-6 of the value.
 *   workspace: txl_logprob_bwd_workspace_size(N, V, d, dtype, grad_dtype) bytes: G in chunks
 *   of the vocabulary, up to about 1 GiB or 128 columns, h once more (TXL_F32: and w, as three terms each), and
 *   partial sums (past one chunk two fp32 dh or, where a chunk's is split, more).
 * Errors: as txl_logprob_fwd.
 */
size_t txl_logprob_bwd_workspace_size(int N, int V, int d, int dtype, int grad_dtype);
int txl_logprob_bwd(const void *h, long long h_stride, const void *w, long long w_stride,
                    const void *targets, int index_type, const float *lse, const float *entropy,
                    const float *dlogp, const float *dentropy, void *dh, void *dw, int N, int V,
                    int d, float scale, int dtype, int grad_dtype, void *workspace,
                    size_t workspace_bytes, void *stream);

/*
 * txl_device_status - synchronise `stream`, then read and clear the device
 * status word in which kernels record barrier time-outs (and, in a debug
 * build, failed index checks).  Returns TXL_OK, TXL_ERR_TIMEOUT (a time-out was
 * recorded), TXL_ERR_INDEX (only failed index checks were) or TXL_ERR_CUDA.
 */
int txl_device_status(void *stream);

/*
 * txl_set_wait_limit_ns - time limit, in nanoseconds, after which a kernel's
 * on-chip barrier wait gives up (default 1e9).  Applies to later launches from
 * this process.  Returns the previous value.
 */
uint64_t txl_set_wait_limit_ns(uint64_t ns);

/*
 * txl_debug_wait_timeout - launch one small kernel that waits on a barrier no
 * one will complete, with the time limit `ns`; it must give up, record the
 * time-out and return.  Lets a test check the time-out path without hanging
 * anything.  Returns the status txl_device_status() reports afterwards
 * (TXL_ERR_TIMEOUT when the path works).
 */
int txl_debug_wait_timeout(uint64_t ns, void *stream);

/*
 * Debug build.  A library compiled with -DTXL_DEBUG checks, inside its kernels,
 * the index arithmetic of the hot path (work split of each block, every row of
 * the shared-memory ring that applies the Appendix B shift, TMEM columns of the
 * table chunks, output rows, decode key and table ranges, memory ring slots and
 * window rows).  A failed check records TXL_ERR_INDEX in the device status word
 * and the kernel goes on: nothing traps.  Release builds compile the checks
 * away.
 *
 * txl_debug_checks - 1 in a debug build, 0 otherwise.
 * txl_debug_index_probe - launch one small kernel that fails one check on
 *   purpose, then return txl_device_status(stream): TXL_ERR_INDEX in a debug
 *   build (the reporting path works), TXL_OK in a release build.
 */
int txl_debug_checks(void);
int txl_debug_index_probe(void *stream);

#ifdef __cplusplus
}
#endif

#endif /* TXL_H */
