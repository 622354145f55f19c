// Internal launch interface of the model's two ends: the token embedding
// (embed.cu) and the log probabilities of tokens (logprob.cu).  Not part of the
// public ABI.
#pragma once

#include "kernels.h"

namespace txl {

// From txl_api.cu: device status word of the current device (null on a CUDA error), the
// barrier time limit, SMs of the current device.
unsigned int *device_status_word();
unsigned long long wait_limit_ns();
int device_sm_count();
// bf16 view [planes][rows][inner], rows ld elements apart, planes plane elements apart, with a
// 64 x box_rows box and 128-byte swizzle.
bool make_map_planes(CUtensorMap *map, const void *base, long long inner, long long rows,
                     long long ld, long long planes, long long plane, unsigned box_rows);
// The same of fp32 in 32 x box_rows boxes.
bool make_map_planes_f32(CUtensorMap *map, const void *base, long long inner, long long rows,
                         long long ld, long long planes, long long plane, unsigned box_rows);

// A launch in clusters of `cluster` blocks that may begin while its predecessor in the stream
// still runs: every kernel here waits for that one's end and writes (chain_wait) before it reads or
// writes anything, so only launches and set-up overlap.  After a kernel that gives no leave
// (chain_go) it is an ordinary launch.  What such a kernel reads may still be written when its blocks
// become resident, so no load here takes the non-coherent path (__ldg), which is for memory that
// nothing writes in a kernel's lifetime.
template <typename... P, typename... A>
cudaError_t launch_grid(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, cudaStream_t s,
                        unsigned cluster, const A &...args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2] = {};
    cfg.attrs = attr;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 1;
    if (cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = cluster;
        attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}

// ---------------------------------------------------------------------------
// token ids
// ---------------------------------------------------------------------------

__device__ __forceinline__ long long raw_token(const void *tokens, int index_bytes, long long i)
{
    return index_bytes == 8 ? static_cast<const long long *>(tokens)[i] : static_cast<const int *>(tokens)[i];
}

// A token's id in [0, V), or -1 for none.  Any other value is taken as none and recorded.
__device__ __forceinline__ int checked_token(long long t, int V, unsigned int *status)
{
    if (t < -1 || t >= V) {
        atomicOr(status, TXL_STATUS_INDEX);
        return -1;
    }
    return (int)t;
}

// Token i of an int32 or int64 array.
__device__ __forceinline__ int token_at(const void *tokens, int index_bytes, long long i, int V,
                                        unsigned int *status)
{
    return checked_token(raw_token(tokens, index_bytes, i), V, status);
}

// ---------------------------------------------------------------------------
// embedding
// ---------------------------------------------------------------------------

struct EmbedParams {
    const void *tokens;
    const void *emb;       // [V][emb_ld]
    void *out;             // [n][d]
    long long emb_ld;      // elements
    int index_bytes, n, V, d;
    float scale;
    unsigned int *status;
};
cudaError_t launch_embed_fwd(const EmbedParams &p, bool bf16, cudaStream_t s);

struct EmbedBwdParams {
    const void *tokens;
    const void *dout;      // [n][dout_ld]
    void *demb;            // [V][d]
    long long dout_ld;
    int index_bytes, n, V, d;
    float scale;
    int accumulate;
    unsigned int *status;
};
size_t embed_bwd_workspace_bytes(int n, int d);
cudaError_t launch_embed_bwd(const EmbedBwdParams &p, bool bf16, bool grad_bf16, void *workspace,
                             cudaStream_t s);

// ---------------------------------------------------------------------------
// log probabilities
// ---------------------------------------------------------------------------

constexpr int kMaxTop = 16;      // alternatives of a row
constexpr int kSpareTop = 4;     // candidates kept beyond them, for the exact order
constexpr int kMaxStatSplits = 160;  // vocabulary ranges of a row
constexpr int kMaxRowSplits = 32;    // ... of more than kFewRows rows, two halves of tiles each
constexpr int kFewRows = 256;    // states up to which the vocabulary takes the tiles' rows
constexpr int kMaxPieces = 3;    // bf16 terms of an fp32 operand

// Candidates kept per row and vocabulary range for `top` alternatives.
constexpr int list_length(int top) { return top == 0 ? 0 : top <= 8 ? 12 : 20; }

// The tensor core's fp32 accumulators cut each addition instead of rounding it, so a sum of
// `steps` additions (16 products each) comes out too small, on average by 0.2 (terms of random
// sign) to 0.3 (terms of one sign) times steps * 2^-24 of its value (measured for 4 to 256 steps);
// results that are fp32 are scaled by the mean of that.  1024 wide: root mean square error 15 to 19
// times 2^-24 without it, 3 to 9 with it.
__device__ __forceinline__ float uncut_scale(int steps) { return fmaf((float)steps, 0.27f * 5.9604645e-8f, 1.f); }

// Order of floats as unsigned integers; 0 is below every number (NaN has none).
__device__ __forceinline__ uint32_t order_key(float v)
{
    const uint32_t u = __float_as_uint(v);
    return u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k)
{
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

// A sum of exponentials is kept beside its maximum's own term, the 1 that is left out of it: of a nearly
// certain token the others are all that its log probability is, and next to a 1 they would be rounded to 2^-24.

// hi + lo + x, the sum of hi and x exactly (Knuth's two-sum).
__device__ __forceinline__ void two_sum(float &hi, float &lo, float x)
{
    const float s = __fadd_rn(hi, x), bb = __fadd_rn(s, -hi);
    lo += (hi - (s - bb)) + (x - bb);
    hi = s;
}

// One GEMM over 256 x bn tiles (bn 128 with three terms), bf16 operands, fp32 sums.
// Which operands, and what becomes of a tile, is the kernel's mode.
struct GemmParams {
    int M, N;              // rows and columns of the product
    int mb, nb, bn;        // tiles, and columns of one (128 or 256)
    int kb;                // 64-wide steps along the contraction
    int splits;            // statistics: ranges of the columns; products: of the contraction
    int n_items;
    int terms;             // of the operands: 1; 2 (products: two of A by one of B); 3 (three of each)
    int twice;             // dW of few rows: both terms of G in steps of their own (terms 1), or 0
    int a_rows;            // of A's boxes: less than 128 where M is, in the logits and in stacked products
    int stacked;           // dh, M <= 128: a pair's blocks take a term of A each, the same rows and columns; their
                           // sums are two parts
    int b_row0;            // offset of B's rows (the vocabulary chunk's first)
    unsigned int *status;
    unsigned long long wait_ns;
    // statistics and gradient of the logits
    const void *targets;   // or null
    int index_bytes;
    int V;                 // the whole vocabulary
    float scale;
    float4 *stats;         // [2 splits][M] (halves of tiles): maximum, sum beside its own 1, weighted sum (log2
                           // units), target's logit; few states: [splits][M], 0 in the last's place
    float *list_val;       // [2 splits][list][M]
    int *list_id;
    unsigned *group_key;   // few states: [M][nb][32] order of the largest of four logits, or null
    float *logits;         // ... and [M][nb][128] the logits (log2 units; NaN behind V), or null
    float *target_z;       // few states: [M], log2 units (where there is a target)
    const float *lse, *entropy, *dlogp, *dentropy;  // (the last two may be null)
    const float *target_logp;
    int g_pieces;          // terms of G
    // products
    int part;              // fp32 parts [splits][M][N] (stacked: twice as many), or the result directly
    int out_bf16;
};

// A launch: the statistics, the gradient of the logits, or both products (p[0] dh, p[1] dW; one
// of them may have no items).  Operands in boxes of 64 elements; out: boxes of 128 bytes of columns
// and 32 rows for the tiles' stores (G's terms; a product or its parts one behind the other).
struct GemmLaunch {
    struct {
        CUtensorMap a, b, out;
    } maps[2];
    GemmParams p[2];
    int early;             // products: items of the second that pairs with fewer of the first begin with
};

cudaError_t launch_logprob_stats(const GemmLaunch &g, int list, cudaStream_t s);
// h against w for M <= kFewRows states: tiles of 128 vocabulary rows (nb of them, bn states wide),
// `splits` blocks.
cudaError_t launch_logprob_few(const CUtensorMap &tm_w, const CUtensorMap &tm_h, const GemmParams &p,
                               cudaStream_t s);
cudaError_t launch_logprob_grad(const GemmLaunch &g, cudaStream_t s);
// dh = G W (contraction over the vocabulary) and dW = G^T h (over the rows).
cudaError_t launch_products(const GemmLaunch &g, cudaStream_t s);
// out = sum over the parts, in their order; of up to two results (elems 0: none).  out may be the first part.
struct PartsSum {
    const float *part;
    void *out;
    long long elems;
    int parts, bf16;
};
cudaError_t launch_sum_parts(const PartsSum (&r)[2], cudaStream_t s);
// fp32 rows [rows] of d, ld apart, as three bf16 terms: planes [3][rows][plane_ld].
struct SplitRows {
    const float *x;
    long long ld;
    int rows, d, plane_ld;
    __nv_bfloat16 *planes;
};
cudaError_t launch_split_f32(const SplitRows &h, const SplitRows &w, cudaStream_t s);

// h without the rows that have no part (fp32: as terms), and the targets' log probabilities;
// fp32: the table's terms too.
struct GradRowsParams {
    const void *h, *w;
    __nv_bfloat16 *out;    // [N][out_ld], or [3][N][out_ld]
    int out_ld;
    SplitRows table;
    float *target_logp;    // [N]
    long long h_ld, w_ld;
    int N, V, d, index_bytes;
    const void *targets;
    const float *lse, *dentropy;
    float scale;
    unsigned int *status;
};
cudaError_t launch_grad_rows(const GradRowsParams &p, bool bf16, cudaStream_t s);

struct MergeParams {
    const float4 *stats;
    const float *list_val;
    const int *list_id;
    const unsigned *group_key;
    const float *logits;   // or null
    const float *target_z;
    int nb;                // vocabulary tiles of 128
    int splits, N, V, d, top, list;
    const void *h, *w;
    long long h_ld, w_ld;
    const void *targets;
    int index_bytes;
    float scale, c_hi, c_lo;  // c: scale / ln 2 as a pair
    float *logp, *lse, *entropy, *top_logp;
    int *top_ids;
    unsigned int *status;
};
cudaError_t launch_logprob_few_merge(const MergeParams &p, bool bf16, cudaStream_t s);
cudaError_t launch_logprob_merge(const MergeParams &p, bool bf16, cudaStream_t s);

} // namespace txl
