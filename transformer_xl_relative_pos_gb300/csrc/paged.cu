// Pages of the memory ("Transformer-XL: Attentive Language Models Beyond a
// Fixed-Length Context", §3.2: the cached states of earlier segments) for
// sequences that advance apart: rows put behind a memory, the memory's state
// advanced, pages copied.
//
// All three move bytes and nothing else; what they cannot do without is each
// row read once and written once.
#include "paged.h"

namespace txl {
namespace {

constexpr int kThreads = 256;
constexpr int kRowTile = 16;      // memory rows per block: more make too few blocks for a prompt (below)
constexpr int kVecPerThread = 4;  // 16-byte vectors in flight per thread

// n_new of sequence b taken into [0, max_rows] and to the room its table has.
__device__ __forceinline__ int new_rows(const AppendParams &p, int b, int fill, bool report)
{
    int n = p.n_new ? min(max(p.n_new[b], 0), p.max_rows) : p.max_rows;
    const int room = p.mem.R - fill;
    if (n > room) {
        if (report) atomicOr(p.status, TXL_STATUS_INDEX);
        n = room;
    }
    return n;
}

// begin_out, fill_out of sequence b: the newest `keep` rows of [memory ; new].
// Both inputs are read before either output is written: they may be the same.
__device__ __forceinline__ void advance(const AppendParams &p, int b)
{
    int begin, fill;
    paged_state(p.mem, b, p.status, begin, fill);
    const int total = fill + new_rows(p, b, fill, true);  // <= R
    const int left = min(total, p.keep);
    int nb = begin + (total - left);                      // < 2 R
    nb -= nb >= p.mem.R ? p.mem.R : 0;
    p.begin_out[b] = nb;
    p.fill_out[b] = left;
}

// Rows [16 x, 16 x + 16) of sequence y's new rows into plane z (layer, key or
// value) of its pages.  The addresses of a row (its page, its source) are found once per
// row and block, in shared memory; then the rows' vectors go over the threads, a
// row's heads and vectors innermost (a projection's output [rows][H][64] is read
// in order; each head's row lands as 128 or 256 contiguous bytes of a page).
// Bound by DRAM for prompts: one layer, 16 sequences of 16 heads, 1600 rows each into empty
// memories, 34.7 us for 210 MB read and written (6.05 TB/s, 0.9 of a plain copy's rate; 32 rows a
// block 37.6, 64 rows 41.7: the last wave of blocks is then a larger part).  Bound by the
// chain of dependent loads state -> table -> source -> store for a few rows: the accepted
// paths (1 to 8 rows) of 64 sequences of 16 heads in 12 layers 8 us for 28 MB in L2, 9.5 from HBM, of
// one sequence 2.5 us.  Keys and values by one block, which would walk that chain once: 9.3 and 38 us;
// heads outermost: 8.4 and 36 us; eight vectors in flight: 11.4 and 42 us.
__global__ void __launch_bounds__(kThreads) paged_append_kernel(const AppendParams p)
{
    __shared__ long long s_dst[kRowTile];  // vector index of head 0's row in the plane; -1: none
    __shared__ int s_src[kRowTile];
    __shared__ bool s_last;
    const int b = blockIdx.y;
    const int layer = p.layer0 + (blockIdx.z >> 1), kv = blockIdx.z & 1;
    const PagedView &m = p.mem;
    const int V = 64 * p.esize / 16;       // vectors of a row: 8 or 16
    int begin, fill;
    paged_state(m, b, p.status, begin, fill);
    const int n = new_rows(p, b, fill, true);
    const int t0 = blockIdx.x * kRowTile;
    const int rows = min(kRowTile, n - t0);
    if (rows > 0) {
        if (threadIdx.x < (unsigned)rows) {
            const int t = t0 + threadIdx.x;
            int x = begin + fill + t;          // fill + t < R, begin < R: below 2 R
            x -= x >= m.R ? m.R : 0;
            const int slot = x / m.P;
            const int page = m.table[(long long)b * m.slots + slot];
            const int src = p.rows ? p.rows[(long long)b * p.rows_stride + t] : t;
            const bool ok = page >= 0 && page < m.n_pages && src >= 0 && src < p.N;
            if (!ok) atomicOr(p.status, TXL_STATUS_INDEX);
            s_dst[threadIdx.x] = ok ? (((long long)page * m.H) * m.P + (x - slot * m.P)) * V : -1;
            s_src[threadIdx.x] = src;
        }
        __syncthreads();
        const RowsView &in = kv ? p.v : p.k;
        const long long l_off = (long long)(blockIdx.z >> 1) * p.layer_stride;
        const char *src = static_cast<const char *>(in.ptr) + (l_off + b * in.sb) * p.esize;
        uint4 *dst = static_cast<uint4 *>(p.pool) +
                     (long long)(2 * layer + kv) * m.n_pages * m.H * m.P * V;
        const long long head_vec = (long long)m.P * V;
        const int total = rows * m.H * V;      // <= 16 * H * 16
        for (int i0 = threadIdx.x; i0 < total; i0 += kThreads * kVecPerThread) {
            uint4 val[kVecPerThread];
            long long at[kVecPerThread];
#pragma unroll
            for (int c = 0; c < kVecPerThread; ++c) {
                const int i = i0 + c * kThreads;
                at[c] = -1;
                if (i >= total) continue;
                const int j = i / V, vec = i - j * V;
                const int tt = j / m.H, h = j - tt * m.H;
                const long long d = s_dst[tt];
                if (d < 0) continue;
                at[c] = d + h * head_vec + vec;
                val[c] = reinterpret_cast<const uint4 *>(
                    src + (h * in.sh + s_src[tt] * in.sr) * p.esize)[vec];
            }
#pragma unroll
            for (int c = 0; c < kVecPerThread; ++c)
                if (at[c] >= 0) dst[at[c]] = val[c];
        }
    }
    if (!p.begin_out) return;
    if (!p.ticket) {
        // separate outputs: one block of each sequence writes them
        if (blockIdx.x == 0 && blockIdx.z == 0 && threadIdx.x == 0) advance(p, b);
        return;
    }
    // The outputs are the state that every block reads: the block that takes the
    // last ticket writes them, when all have read it, and leaves the ticket at zero.
    __syncthreads();
    if (threadIdx.x == 0) {
        __threadfence();
        const int blocks = gridDim.x * gridDim.y * gridDim.z;
        s_last = atomicAdd(p.ticket, 1) == blocks - 1;
    }
    __syncthreads();
    if (!s_last) return;
    for (int i = threadIdx.x; i < m.B; i += kThreads) advance(p, i);
    if (threadIdx.x == 0) *p.ticket = 0;
}

__global__ void __launch_bounds__(kThreads) paged_advance_kernel(const AppendParams p)
{
    const int b = blockIdx.x * kThreads + threadIdx.x;
    if (b < p.mem.B) advance(p, b);
}

// Part x mod parts of page src[x / parts] to page dst[x / parts] of plane y; page_vec 16-byte
// vectors a page.  Bound by DRAM: 48 pages of 64 rows and 16 heads in 12 layers 45.1 us for
// 302 MB (6.70 TB/s, a plain copy's rate); a single page of 8 heads 1.8 us in
// L2, 2.3 from HBM, which is the launch and two dependent loads.  With eight vectors a thread 45.5 and 2.0 us.
constexpr int kCopyVec = 2;  // vectors per thread, all in flight at once

__global__ void __launch_bounds__(kThreads) paged_copy_kernel(uint4 *__restrict__ pool, int n_pages,
                                                              long long page_vec,
                                                              const int *__restrict__ src,
                                                              const int *__restrict__ dst,
                                                              int parts, unsigned int *status)
{
    const int i = blockIdx.x / parts, part = blockIdx.x - i * parts;
    const int s = src[i], d = dst[i];
    if (s < 0 || s >= n_pages || d < 0 || d >= n_pages) {
        if (part == 0 && blockIdx.y == 0 && threadIdx.x == 0) atomicOr(status, TXL_STATUS_INDEX);
        return;
    }
    if (s == d) return;
    const long long plane = (long long)blockIdx.y * n_pages;
    const uint4 *from = pool + (plane + s) * page_vec;
    uint4 *to = pool + (plane + d) * page_vec;
    const long long base = (long long)part * kThreads * kCopyVec + threadIdx.x;
    uint4 v[kCopyVec];
#pragma unroll
    for (int c = 0; c < kCopyVec; ++c)
        if (base + c * kThreads < page_vec) v[c] = from[base + c * kThreads];
#pragma unroll
    for (int c = 0; c < kCopyVec; ++c)
        if (base + c * kThreads < page_vec) to[base + c * kThreads] = v[c];
}

} // namespace

cudaError_t launch_paged_append(const AppendParams &p, cudaStream_t s)
{
    const unsigned tiles = (unsigned)((p.max_rows + kRowTile - 1) / kRowTile);
    const dim3 grid(tiles, (unsigned)p.mem.B, (unsigned)(2 * p.n_layers));
    paged_append_kernel<<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_paged_advance(const AppendParams &p, cudaStream_t s)
{
    paged_advance_kernel<<<(unsigned)((p.mem.B + kThreads - 1) / kThreads), kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_paged_copy(void *pool, int planes, int n_pages, long long page_vec,
                              const int *src, const int *dst, int n, unsigned int *status,
                              cudaStream_t s)
{
    const long long per = (long long)kThreads * kCopyVec;
    const long long parts = (page_vec + per - 1) / per;
    if (parts * n > 0x7fffffffLL || planes > 65535) return cudaErrorInvalidValue;
    paged_copy_kernel<<<dim3((unsigned)(parts * n), (unsigned)planes), kThreads, 0, s>>>(
        static_cast<uint4 *>(pool), n_pages, page_vec, src, dst, (int)parts, status);
    return cudaGetLastError();
}

} // namespace txl
