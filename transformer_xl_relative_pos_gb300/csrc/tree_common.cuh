// Device code shared by the two kernels of txl_relattn_tree_fwd (relattn_tree.cu,
// bf16 on the tensor cores; relattn_tree_f32.cu): the drafted tree's depths and
// ancestors, the split of a memory's keys, and the merge of the warps' and the
// blocks' partial results.
//
// A block's NW warps that compute hold ROWS of the tree's nodes each (node tile mt)
// and take a range of the keys (key group kg): with MT node tiles there are
// NW / MT key groups.  The blocks of one (batch, head) are a thread-block cluster;
// its key groups share the memory in contiguous runs of 32-key chunks.
#pragma once

#include <atomic>
#include <type_traits>

#include "decode_common.cuh"
#include "paged.h"

namespace txl {
namespace tree {

using namespace ptx;
using decode::cluster_addr;
using decode::cluster_rank;
using decode::cluster_sync;
using decode::ex2f;
using decode::ld_cluster_f32;
using decode::ld_cluster_f32x2;

constexpr int DH = kTcDH;  // 64
constexpr int GK = 32;     // keys per chunk
constexpr int kNodesCost = 2;  // the nodes among themselves, in chunks of memory

// max that keeps a NaN: a row with a NaN score gives NaN, as the formula does.
__device__ __forceinline__ float max_nan(float a, float b)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

__device__ __forceinline__ float max3_nan(float a, float b, float c)
{
    float d;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}

// Byte offset of 16-byte piece c of row `row` in a 128-byte-swizzled box of 128-byte rows.
__device__ __forceinline__ uint32_t swz(int row, int c)
{
    return (uint32_t)(row * DH * 2 + ((c ^ (row & 7)) << 4));
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// 16 bytes into shared memory without passing through registers, or zeros.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool there)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(there ? 16 : 0)
                 : "memory");
}

// A bf16 whose exponent bits are all ones (infinity or NaN) in either half.
__device__ __forceinline__ bool nonfinite2(uint32_t w)
{
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// Per node of the block's sequence: depth, and the mask of itself and its ancestors.
struct Topology {
    unsigned long long anc[kTreeMaxNodes];
    int depth[kTreeMaxNodes];
    int hop[kTreeMaxNodes];
    int picked;  // pick_sequence's
};

// Sequence of this block: the ranks of the grid (rank = block / (H * n_splits)) in
// order, or, by_length, longest memory first: with more blocks than are resident at
// once and unlike lengths, the blocks that start last are then the short ones.
// Every block finds the one of its rank: a warp has all lengths in its lanes, and counts for
// its share of the sequences how many come before.  All threads of the block.
__device__ __forceinline__ int pick_sequence(const TreeParams &p, int rank, Topology &topo)
{
    static_assert(kTreeMaxSorted == 64, "two lengths a lane");
    if (!p.by_length) return rank;
    const int B = p.mem.B, lane = threadIdx.x & 31;
    constexpr int NONE = (int)0x80000000;
    const int f0 = lane < B ? p.mem.fill[lane] : NONE, f1 = lane + 32 < B ? p.mem.fill[lane + 32] : NONE;
    for (int i = threadIdx.x >> 5; i < B; i += blockDim.x >> 5) {
        const int mine = __shfl_sync(0xffffffffu, i < 32 ? f0 : f1, i & 31);
        const unsigned before0 = __ballot_sync(0xffffffffu, f0 > mine || (f0 == mine && lane < i));
        const unsigned before1 = __ballot_sync(0xffffffffu, f1 > mine || (f1 == mine && lane + 32 < i));
        if (lane == 0 && __popc(before0) + __popc(before1) == rank) topo.picked = i;
    }
    __syncthreads();
    return topo.picked;
}

// By pointer doubling: after round r a node knows its 2^r nearest ancestors.  A
// parent that is not an earlier node counts as none, so there is no cycle.  All
// threads of the block, thread i with node i's parent; ends with a barrier.
__device__ __forceinline__ void build_topology(Topology &t, int parent, int n,
                                               unsigned int *status)
{
    const int i = threadIdx.x;
    unsigned long long anc = 0;
    int hop = -1, depth = 0;
    if (i < n) {
        hop = parent;
        if (hop < -1 || hop >= i) {
            atomicOr(status, TXL_STATUS_INDEX);
            hop = -1;
        }
        anc = 1ull << i;
        depth = hop >= 0 ? 1 : 0;
    }
    for (int span = 1; span < n; span *= 2) {
        if (i < n) {
            t.anc[i] = anc;
            t.depth[i] = depth;
            t.hop[i] = hop;
        }
        __syncthreads();
        if (hop >= 0) {
            anc |= t.anc[hop];
            depth += t.depth[hop];
            hop = t.hop[hop];
        }
        __syncthreads();
    }
    if (i < n) {
        t.anc[i] = anc;
        t.depth[i] = depth;
    }
    __syncthreads();
}

// The chunks of one key group: 32-row chunks of the table ring, aligned to it
// (so that none crosses a page).  Chunk c holds memory rows 32 c - off .. + 31.
struct Chunks {
    int off;        // begin mod 32
    int c0, count;  // this group's first chunk, and how many
    int slot, row;  // table slot of the first chunk, and its first row there
};

// A head's chunks in contiguous runs over its key groups.  The last group also takes
// the nodes among themselves, which count as `nodes_cost` chunks behind the
// memory's.
__device__ __forceinline__ Chunks group_chunks(const TreeParams &p, int begin, int fill, int nodes_cost,
                                               int group, int groups)
{
    Chunks k;
    k.off = begin & (GK - 1);
    // Rows the table reaches from a node of depth 0; deeper ones reach fewer.
    const int t_lo = max(0, fill - p.r_rows + 1);
    const int first = (k.off + t_lo) / GK;
    const int all = fill > t_lo ? (k.off + fill + GK - 1) / GK - first : 0;
    const int from = min(all, (int)((long long)(all + nodes_cost) * group / groups));
    const int to = min(all, (int)((long long)(all + nodes_cost) * (group + 1) / groups));
    k.c0 = first + from;
    k.count = to - from;
    int x = begin - k.off + k.c0 * GK;  // below 2 R, and R itself when there is no chunk
    x -= x >= p.mem.R ? p.mem.R : 0;
    k.slot = x / p.mem.P;
    k.row = x - k.slot * p.mem.P;
    return k;
}

// Page id in table slot `slot` of sequence b (out of range: -1, and recorded).
__device__ __forceinline__ int page_at(const PagedView &m, int b, int slot, unsigned int *status)
{
    TXL_CHECK(slot >= 0 && slot < m.slots, status);
    const int page = m.table[(long long)b * m.slots + slot];
    if (page >= 0 && page < m.n_pages) return page;
    atomicOr(status, TXL_STATUS_INDEX);
    return -1;
}

// The table position one chunk on.  True when another page begins.
__device__ __forceinline__ bool next_chunk(const PagedView &m, int &slot, int &row)
{
    row += GK;
    if (row < m.P) return false;
    row = 0;
    if (++slot == m.slots) slot = 0;
    return true;
}

// One warp's result for its nodes: running maximum (log2 units), sum of
// probabilities, unnormalised output.
template <int ROWS, int LD = DH>
struct Rec {
    static constexpr int N = ROWS;
    float m[ROWS];
    float l[ROWS];
    float a[ROWS][LD];
};

__device__ __forceinline__ void put_row(__nv_bfloat16 *dst, int lane, float x, float y)
{
    reinterpret_cast<__nv_bfloat162 *>(dst)[lane] = __floats2bfloat162_rn(x, y);
}

__device__ __forceinline__ void put_row(float *dst, int lane, float x, float y)
{
    reinterpret_cast<float2 *>(dst)[lane] = make_float2(x, y);
}

// The last barrier of a cluster: the other blocks have read this one's shared memory
// (their loads are complete: nothing to order).
__device__ __forceinline__ void cluster_done()
{
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// NW warps, after each wrote its record (those of node tile mt: rec(mt), rec(mt + MT), ...,
// KG of them) and all threads of the block entered: merge the key groups of each node, then
// the blocks of the cluster, whose warps share the nodes; write out and lse of the n nodes.
// A partial result stays unnormalised until the last merge:
//   m = max m_g, l = sum 2^(m_g - m) l_g, a = sum 2^(m_g - m) a_g, out = a / l.
// Every node sees itself at least, so l = 0 only where all its scores are -infinity: 0 / 0, NaN
// as in the formula.
template <int NW, int KG, int MT, typename T, typename RecOf>
__device__ __forceinline__ void finish(RecOf rec, const TreeParams &p, int b, int h, int n, int warp,
                                       int lane)
{
    constexpr int ROWS = std::remove_pointer_t<decltype(rec(0))>::N;
    constexpr float LN2 = 0.69314718055994531f;
    T *out = static_cast<T *>(const_cast<void *>(p.out.ptr)) + b * p.out.sb + h * p.out.sh;
    float *lse = p.lse ? p.lse + ((long long)b * p.mem.H + h) * p.N : nullptr;
    auto write = [&](int i, float m, float l, float o0, float o1) {
        const float inv = 1.f / l;
        put_row(out + i * p.out.sr, lane, o0 * inv, o1 * inv);
        if (lse && lane == 0) lse[i] = (m + log2f(l)) * LN2;
    };
    __syncthreads();
    if (KG > 1 || p.n_splits == 1) {
#pragma unroll 2
        for (int i = warp; i < n; i += NW) {
            const int mt = i / ROWS, ii = i % ROWS;
            float m[KG], l[KG];
            float2 a[KG];
            float mx = -INFINITY;
#pragma unroll
            for (int g = 0; g < KG; ++g) {
                const auto *r = rec(g * MT + mt);
                m[g] = r->m[ii];
                l[g] = r->l[ii];
                a[g] = reinterpret_cast<const float2 *>(r->a[ii])[lane];
                mx = max_nan(mx, m[g]);
            }
            const float ref = mx == -INFINITY ? 0.f : mx;
            float ls = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
            for (int g = 0; g < KG; ++g) {
                const float w = ex2f(m[g] - ref);  // (0 from -inf)
                ls = fmaf(w, l[g], ls);
                o0 = fmaf(w, a[g].x, o0);
                o1 = fmaf(w, a[g].y, o1);
            }
            if (p.n_splits == 1) {
                write(i, mx, ls, o0, o1);
            } else {
                // in place of key group 0's (each lane overwrites what it alone has read,
                // or what all have)
                auto *r = rec(mt);
                __syncwarp();
                reinterpret_cast<float2 *>(r->a[ii])[lane] = make_float2(o0, o1);
                if (lane == 0) {
                    r->m[ii] = mx;
                    r->l[ii] = ls;
                }
            }
        }
    }
    if (p.n_splits == 1) return;
    cluster_sync();
    for (int i = (int)cluster_rank() * NW + warp; i < n; i += NW * p.n_splits) {
        const auto *r = rec(i / ROWS);
        const uint32_t at_m = smem_u32(&r->m[i % ROWS]), at_l = smem_u32(&r->l[i % ROWS]);
        const uint32_t at_a = smem_u32(&r->a[i % ROWS][2 * lane]);
        // (every load on its way before the first is used; ranks past the last: rank 0
        // again, its values replaced by an empty result's, as zero weight times an infinity is NaN)
        float m[kTreeMaxCluster], l[kTreeMaxCluster];
        float2 a[kTreeMaxCluster];
#pragma unroll
        for (int s = 0; s < kTreeMaxCluster; ++s) {
            const uint32_t from = s < p.n_splits ? s : 0;
            m[s] = ld_cluster_f32(cluster_addr(at_m, from));
            l[s] = ld_cluster_f32(cluster_addr(at_l, from));
            a[s] = ld_cluster_f32x2(cluster_addr(at_a, from));
        }
        float mx = -INFINITY;
#pragma unroll
        for (int s = 0; s < kTreeMaxCluster; ++s) {
            if (s >= p.n_splits) {
                m[s] = -INFINITY;
                l[s] = a[s].x = a[s].y = 0.f;
            }
            mx = max_nan(mx, m[s]);
        }
        const float ref = mx == -INFINITY ? 0.f : mx;
        float ls = 0.f, o0 = 0.f, o1 = 0.f;
#pragma unroll
        for (int s = 0; s < kTreeMaxCluster; ++s) {
            const float w = ex2f(m[s] - ref);  // (0 from -inf)
            ls = fmaf(w, l[s], ls);
            o0 = fmaf(w, a[s].x, o0);
            o1 = fmaf(w, a[s].y, o1);
        }
        write(i, mx, ls, o0, o1);
    }
    cluster_done();
}

// The barriers of finish, for warps that have no results.
__device__ __forceinline__ void finish_barriers(const TreeParams &p)
{
    __syncthreads();
    if (p.n_splits == 1) return;
    cluster_sync();
    cluster_done();
}

// Configuration of a launch with one cluster of n_splits blocks per (batch, head).
struct ClusterConfig {
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    ClusterConfig(long long blocks, int n_splits, int threads, int smem, cudaStream_t s)
    {
        cfg.gridDim = dim3((unsigned)blocks, 1, 1);
        cfg.blockDim = dim3((unsigned)threads, 1, 1);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)n_splits;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = n_splits > 1 ? 1 : 0;
    }
};

template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kern)(KArgs...), const TreeParams &p, int threads, int smem,
                            cudaStream_t s, const Args &...args)
{
    const long long blocks = (long long)p.mem.B * p.mem.H * p.n_splits;
    if (blocks <= 0 || blocks > 0x7fffffffLL || p.n_splits > kTreeMaxCluster)
        return cudaErrorInvalidValue;
    ClusterConfig c(blocks, p.n_splits, threads, smem, s);
    return cudaLaunchKernelEx(&c.cfg, kern, args...);
}

// Clusters of n_splits blocks the current device holds at once (0: unknown).
template <typename... KArgs>
int max_clusters(void (*kern)(KArgs...), int n_splits, int threads, int smem)
{
    ClusterConfig c(n_splits, n_splits, threads, smem, nullptr);
    c.cfg.numAttrs = 1;  // (a cluster of one block too)
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &c.cfg) != cudaSuccess) {
        cudaGetLastError();  // (no sticky error is left to a later launch check)
        return 0;
    }
    return n;
}

// max_clusters of one kernel, found once per device and size.
struct ClusterCache {
    std::atomic<int> n[64][kTreeMaxCluster + 1] = {};  // plus one; 0: not found yet
    template <typename F>
    int get(int n_splits, F find)
    {
        int dev = 0;
        if (n_splits < 1 || n_splits > kTreeMaxCluster || cudaGetDevice(&dev) != cudaSuccess || dev < 0 ||
            dev >= 64)
            return 0;
        int v = n[dev][n_splits].load(std::memory_order_relaxed);
        if (v == 0) {
            v = find() + 1;
            n[dev][n_splits].store(v, std::memory_order_relaxed);
        }
        return v - 1;
    }
};

} // namespace tree
} // namespace txl
