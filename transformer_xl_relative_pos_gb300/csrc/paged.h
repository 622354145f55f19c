// Internal launch interface of the paged memory's kernels (paged.cu) and of the
// attention that reads it (relattn_tree.cu, relattn_tree_f32.cu).  Not part of
// the public ABI.
#pragma once

#include "kernels.h"

namespace txl {

constexpr int kTreeMaxNodes = 64;   // nodes of a drafted tree (one 64-bit ancestor mask)
constexpr int kTreeMaxCluster = 8;  // key ranges of a head: one portable thread-block cluster
constexpr int kTreeMaxSorted = 64;  // sequences whose blocks can be ordered by length
// Key groups of a block in a tree of N nodes: its four warps that compute hold 16 nodes each.
constexpr int tree_key_groups(int N) { return N <= 16 ? 4 : N <= 32 ? 2 : 1; }
constexpr int kPageRowUnit = 32;    // page_rows is a multiple of this: keys of one tile

// Device view of a paged memory (txl_paged_kv).
struct PagedView {
    const int *table;  // [B][slots]
    const int *begin;  // [B]
    const int *fill;   // [B]
    int n_pages, H, P, slots, B;
    int R;             // slots * P: table rows of a sequence
};

// begin and fill of sequence b, brought into their ranges whatever they hold (a
// value outside is recorded).
__device__ __forceinline__ void paged_state(const PagedView &m, int b, unsigned int *status,
                                            int &begin, int &fill)
{
    begin = m.begin[b];
    fill = m.fill[b];
    if (begin < 0 || begin >= m.R || fill < 0 || fill > m.R) {
        atomicOr(status, TXL_STATUS_INDEX);
        begin %= m.R;
        begin += begin < 0 ? m.R : 0;
        fill = min(max(fill, 0), m.R);
    }
}

// Operand [B][H][rows][64] with strides in elements.
struct RowsView {
    const void *ptr;
    long long sb, sh, sr;
};

struct AppendParams {
    PagedView mem;
    void *pool;
    RowsView k, v;
    long long layer_stride;  // elements
    int layer0, n_layers, N, esize;
    const int *rows;
    int rows_stride;
    const int *n_new;
    int max_rows, keep;
    int *begin_out, *fill_out;  // null: the state is not advanced
    int *ticket;                // non-null: the outputs are the state itself
    unsigned int *status;
};

cudaError_t launch_paged_append(const AppendParams &p, cudaStream_t s);
// Only begin_out / fill_out of the parameters' state fields, n_new, max_rows, keep.
cudaError_t launch_paged_advance(const AppendParams &p, cudaStream_t s);
cudaError_t launch_paged_copy(void *pool, int planes, int n_pages, long long page_vec,
                              const int *src, const int *dst, int n, unsigned int *status,
                              cudaStream_t s);

struct TreeParams {
    PagedView mem;
    RowsView q, k, v, out;
    const void *r, *u, *vb;
    const void *kpage, *vpage;  // the layer's key and value planes of the pool
    float *lse;
    const int *parents;
    long long parents_stride;
    const int *n_nodes;
    int N, r_rows, n_splits;
    int by_length;              // blocks of the longest memories first (B <= kTreeMaxSorted)
    float scale_log2;           // scale * log2(e)
    unsigned int *status;
    unsigned long long wait_ns;
};

// bf16: tm_kv over the layer's key planes and then its value planes [2 * n_pages * H][P][64],
// tm_r over the table [H][r_rows][64], in boxes of 32 rows, 128-byte swizzle.
cudaError_t launch_relattn_tree(const CUtensorMap &tm_kv, const CUtensorMap &tm_r, const TreeParams &p,
                                cudaStream_t s);
cudaError_t launch_relattn_tree_f32(const TreeParams &p, cudaStream_t s);
// Thread-block clusters of n_splits blocks that the current device holds at once, for
// trees of N nodes (0 when that cannot be found).
int tree_max_clusters(int N, int n_splits);
int tree_max_clusters_f32(int N, int n_splits);

} // namespace txl
