// The token embedding and its gradient ("Transformer-XL: Attentive Language
// Models Beyond a Fixed-Length Context", §3.3: h^0 is the word embedding
// sequence).
//
//   forward   out_t = scale * E[token_t]
//   gradient  dE_v  = scale * sum_{t : token_t = v} dout_t
//
// Both move rows and are bound by HBM.  The gradient first sorts the positions
// by their tokens (a stable radix sort), then sums runs of equal tokens in
// chunks of positions, a warp each; a run that crosses chunks leaves one partial per
// chunk, which a last launch sums in their order.  No sum depends on the order
// in which blocks run, so results repeat bit for bit.
#include <algorithm>

#include "vocab.h"
#include "ptx.cuh"

namespace txl {
namespace {

using namespace ptx;

// ---------------------------------------------------------------------------
// rows as 16-byte vectors
// ---------------------------------------------------------------------------

__device__ __forceinline__ float2 bf2_to_f2(uint32_t v)
{
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}

__device__ __forceinline__ uint32_t f2_to_bf2(float lo, float hi)
{
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
}

template <bool BF16>
__device__ __forceinline__ uint4 scaled(uint4 v, float s)
{
    uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = bf2_to_f2(w[i]);
        w[i] = BF16 ? f2_to_bf2(f.x * s, f.y * s) : __float_as_uint(__uint_as_float(w[i]) * s);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

template <bool BF16>
__device__ __forceinline__ float scaled(float v, float s)
{
    return v * s;
}

template <bool BF16>
__device__ __forceinline__ __nv_bfloat16 scaled(__nv_bfloat16 v, float s)
{
    return __float2bfloat16_rn(__bfloat162float(v) * s);
}

constexpr int kFwdThreads = 256;
constexpr int kFwdVecs = 4;  // vectors a thread keeps in flight

// Flat over (position, vector): 16 bytes, or an element where widths, strides or addresses ask
// for it.
template <bool BF16, typename VEC>
__global__ void __launch_bounds__(kFwdThreads) embed_fwd_kernel(const EmbedParams p, int row_vec,
                                                                long long emb_vec)
{
    const long long total = (long long)p.n * row_vec;
    const long long base = (long long)blockIdx.x * (kFwdThreads * kFwdVecs) + threadIdx.x;
    const VEC *emb = static_cast<const VEC *>(p.emb);
    VEC *out = static_cast<VEC *>(p.out);
    VEC v[kFwdVecs];
    chain_wait();
    chain_go();
#pragma unroll
    for (int k = 0; k < kFwdVecs; ++k) {
        const long long i = base + k * kFwdThreads;
        v[k] = VEC{};
        if (i >= total) continue;
        const int t = (int)(i / row_vec), c = (int)(i - (long long)t * row_vec);
        const int id = token_at(p.tokens, p.index_bytes, t, p.V, p.status);
        if (id >= 0) v[k] = emb[id * emb_vec + c];
    }
#pragma unroll
    for (int k = 0; k < kFwdVecs; ++k) {
        const long long i = base + k * kFwdThreads;
        if (i < total) out[i] = p.scale == 1.f ? v[k] : scaled<BF16>(v[k], p.scale);
    }
}

// ---------------------------------------------------------------------------
// positions sorted by token
// ---------------------------------------------------------------------------
// LSD radix sort of (key, position): key = token, or V for a position without one.  One launch:
// a thread-block cluster, a warp for each stretch of consecutive positions.  A pass counts each warp's digits, exchanges the blocks' counts through distributed
// shared memory, and lets every warp put its stretch in place in order: 32 positions at a time,
// equal digits ranked by match.  Stable, so equal tokens stay in the order of their positions.
// Bound by the scattered stores of a few SMs, hence one of 8 bytes for each position.

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortCluster = 8, kSortWide = 16;  // blocks; more than 8 need the device's consent
constexpr int kHeld = 8;                // rows of 32 positions a warp holds in registers
constexpr int kDigit = 9;                // bits of a pass, at most
constexpr int kBins = 1 << kDigit;      // one bin a thread
static_assert(kBins == kSortThreads, "a thread keeps one bin");

struct SortParams {
    const void *tokens;
    int2 *pair[2];           // (key, position): pass i reads buffer i & 1 and writes the other
    int *crossing;           // counter of the runs that cross chunks, zeroed here
    int index_bytes, n, V, passes, digit, per_warp, blocks;  // digit: bits of a pass
    unsigned int *status;
};

// A word of another block's shared memory (the same place in it).
__device__ __forceinline__ int cluster_word(const int *p, int block)
{
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(cluster_addr(p, (uint32_t)block)) : "memory");
    return v;
}

__global__ void __launch_bounds__(kSortThreads) sort_kernel(const SortParams p)
{
    __shared__ int place[kSortWarps][kBins];    // a warp's counts, then its next places
    __shared__ int total[kBins];                // the block's counts
    __shared__ int warp_sum[kSortWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int block = blockIdx.x;
    const long long lo_ = ((long long)block * kSortWarps + warp) * p.per_warp;
    const int lo = (int)min((long long)p.n, lo_), hi = (int)min((long long)p.n, lo_ + p.per_warp);
    chain_wait();
    chain_go();
    if (block == 0 && tid == 0) *p.crossing = 0;
    for (int pass = 0; pass < p.passes; ++pass) {
        const int shift = pass * p.digit, mask = (1 << p.digit) - 1;
        const bool last = pass + 1 == p.passes;
        const int2 *in = p.pair[pass & 1];
        int2 *out = p.pair[(pass & 1) ^ 1];
        // kHeld rows of 32 positions at a time in registers (all loads before the first is looked at)
        int key[kHeld], pos[kHeld];
        auto load = [&](int i0) {
            if (pass == 0) {
                long long id[kHeld];
#pragma unroll
                for (int k = 0; k < kHeld; ++k) {
                    const int i = i0 + k * 32 + lane;
                    pos[k] = i;
                    id[k] = i < hi ? raw_token(p.tokens, p.index_bytes, i) : -1;
                }
#pragma unroll
                for (int k = 0; k < kHeld; ++k) {
                    const int t = checked_token(id[k], p.V, p.status);
                    key[k] = pos[k] >= hi ? -1 : t < 0 ? p.V : t;
                }
            } else {
#pragma unroll
                for (int k = 0; k < kHeld; ++k) {
                    const int i = i0 + k * 32 + lane;
                    const int2 v = i < hi ? __ldcg(in + i) : make_int2(-1, 0);
                    key[k] = v.x;
                    pos[k] = v.y;
                }
            }
        };
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) place[w][tid] = 0;
        __syncthreads();
        load(lo);
        for (int i0 = lo; i0 < hi; i0 += kHeld * 32) {
            if (i0 > lo) load(i0);
#pragma unroll
            for (int k = 0; k < kHeld; ++k)
                if (key[k] >= 0) atomicAdd(&place[warp][(key[k] >> shift) & mask], 1);
        }
        __syncthreads();
        // thread = bin: the warps' counts to starts within the block
        int sum = 0;
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = place[w][tid];
            place[w][tid] = sum;
            sum += c;
        }
        total[tid] = sum;
        cluster_sync_all();
        int all = 0, before = 0;
#pragma unroll
        for (int b = 0; b < kSortWide; ++b) {
            const int c = b < p.blocks && tid <= mask ? cluster_word(total + tid, b) : 0;
            all += c;
            before += b < block ? c : 0;
        }
        int incl = all;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, incl, o);
            incl += lane >= o ? v : 0;
        }
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        int start = incl - all + before;
        for (int w = 0; w < warp; ++w) start += warp_sum[w];
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) place[w][tid] += start;
        __syncthreads();
        if (hi - lo > kHeld * 32) load(lo);
        for (int i0 = lo; i0 < hi; i0 += kHeld * 32) {
            if (i0 > lo) load(i0);
#pragma unroll
            for (int k = 0; k < kHeld; ++k) {
                if (i0 + k * 32 >= hi) break;
                const bool on = key[k] >= 0;
                const int digit = on ? (key[k] >> shift) & mask : kBins + lane;
                const unsigned same = __match_any_sync(0xffffffffu, digit);
                const int rank = __popc(same & ((1u << lane) - 1));
                int to = 0;
                if (on) to = place[warp][digit] + rank;
                __syncwarp();
                if (on && rank == 0) place[warp][digit] = to + __popc(same);
                __syncwarp();
                if (!on) continue;
                TXL_CHECK(to >= 0 && to < p.n, p.status);
                __stcg(out + to, make_int2(key[k], pos[k]));
            }
        }
        // what this pass has put in place is read by other warps and blocks
        if (last) break;
        __threadfence();
        cluster_sync_all();
    }
    // (no block leaves while another may still read its counts)
    cluster_sync_all();
}

// Up to kRankMost positions: each one's place is the number of keys before it, counted by
// comparing with all of them.  A block places 32 positions, each of its warps against an
// eighth of the keys.  2047 positions 4 us, where a block with two radix passes took 11.
constexpr int kRankMost = 4096;
constexpr int kRankThreads = 256;

__global__ void __launch_bounds__(kRankThreads) rank_sort_kernel(const SortParams p)
{
    __shared__ int4 s_key[kRankMost / 4];
    __shared__ int s_rank[32];
    chain_wait();
    chain_go();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (blockIdx.x == 0 && tid == 0) *p.crossing = 0;
    if (tid < 32) s_rank[tid] = 0;
    int *keys = reinterpret_cast<int *>(s_key);
    const int padded = (p.n + 31) / 32 * 32;
    for (int i = tid; i < padded; i += kRankThreads) {
        int key = 0x7ffffffe;  // (behind the last: after everything)
        if (i < p.n) {
            const int id = token_at(p.tokens, p.index_bytes, i, p.V, p.status);
            key = id < 0 ? p.V : id;
        }
        keys[i] = key;
    }
    __syncthreads();
    const int i0 = blockIdx.x * 32, mine = keys[i0 + lane];
    // rows of 32 keys in turn over the warps: rows before this one count equal keys too
    int rank = 0;
    for (int r = warp; r < padded / 32; r += kRankThreads / 32) {
        const int limit = mine + (r * 32 < i0 ? 1 : 0);
        if (r * 32 == i0) {
#pragma unroll
            for (int j = 0; j < 32; ++j) rank += keys[i0 + j] < mine || (keys[i0 + j] == mine && j < lane);
            continue;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int4 k = s_key[r * 8 + j];
            rank += (k.x < limit) + (k.y < limit) + (k.z < limit) + (k.w < limit);
        }
    }
    atomicAdd(s_rank + lane, rank);
    __syncthreads();
    if (warp == 0 && i0 + lane < p.n) {
        const int to = s_rank[lane];
        TXL_CHECK(to >= 0 && to < p.n, p.status);
        p.pair[0][to] = make_int2(mine, i0 + lane);
    }
}

// ---------------------------------------------------------------------------
// sums over runs
// ---------------------------------------------------------------------------

constexpr int kRow = 32;          // positions at a time
constexpr int kMaxChunk = 64;     // positions of a warp, at most
constexpr int kSumWarps = 4;
constexpr int kBatch = 8;         // rows in flight, and as many being summed
constexpr int kJoinWarps = 16;
constexpr int kClearRows = 8;     // rows of the gradient that a warp looks up and clears

struct SumParams {
    const int2 *pair;             // (key, position), sorted
    const void *dout;
    long long dout_ld;
    void *demb;
    float *part;                  // [chunks][2][part_ld]: of a run from before, of one into the next
    long long part_ld;
    int *crossing;                // runs that begin in a chunk and go on in the next:
    int2 *cross;                  // ... the chunk and the key of each
    int n, V, d, chunk, chunks, slices, accumulate;
    int sum_blocks;               // the blocks behind them clear the rows that no token points to
    float scale;
    unsigned int *status;
};

// Columns of a lane: 16 bytes of dout.
template <bool BF16>
struct Cols {
    static constexpr int N = BF16 ? 8 : 4;
};

template <bool BF16>
__device__ __forceinline__ void add_row(float (&a)[Cols<BF16>::N], const uint4 &r)
{
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (BF16) {
            const float2 f = bf2_to_f2(w[i]);
            a[2 * i] += f.x;
            a[2 * i + 1] += f.y;
        } else {
            a[i] += __uint_as_float(w[i]);
        }
    }
}

// N sums (4 or 8) of a row of demb, from column col on.
template <bool GRAD_BF16, int N>
__device__ __forceinline__ void store_row(const SumParams &p, int v, int col, const float (&a)[N])
{
    const long long at = (long long)v * p.d + col;
#pragma unroll
    for (int q = 0; q < N; q += 4) {
        float4 x = make_float4(a[q] * p.scale, a[q + 1] * p.scale, a[q + 2] * p.scale, a[q + 3] * p.scale);
        if (GRAD_BF16) {
            *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.demb) + at + q) =
                make_uint2(f2_to_bf2(x.x, x.y), f2_to_bf2(x.z, x.w));
        } else {
            float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p.demb) + at + q);
            if (p.accumulate) {
                const float4 y = *o;
                x = make_float4(y.x + x.x, y.y + x.y, y.z + x.z, y.w + x.w);
            }
            *o = x;
        }
    }
}

// kClearRows rows of the table's gradient to a warp: zeros where no token points.  A lane finds whether
// its row's key is among the sorted ones.  (Clearing the whole gradient beside the sort writes
// most rows twice: 65536 tokens, 32000 x 1024 in fp32, 72 us in all instead of 69.5, with the sort 32
// instead of 20; 2047 tokens, 10007 x 520: 16.2 and 14.7.  The sums' own warps clearing the gaps
// between their keys: 82.)
template <bool GRAD_BF16>
__device__ __forceinline__ void clear_rows(const SumParams &p, long long first, int lane)
{
    if (first >= p.V) return;
    const int v = (int)first + lane;
    int lo = 0, hi = p.n;
    while (lo < hi) {
        const int mid = lo + (hi - lo) / 2;
        if (p.pair[mid].x < v) lo = mid + 1;
        else hi = mid;
    }
    const bool absent = lane < kClearRows && v < p.V && !(lo < p.n && p.pair[lo].x == v);
    const int row_vec = p.d * (GRAD_BF16 ? 2 : 4) / 16;
    for (unsigned rows = __ballot_sync(0xffffffffu, absent); rows; rows &= rows - 1) {
        uint4 *row = static_cast<uint4 *>(p.demb) + (first + __ffs(rows) - 1) * row_vec;
        for (int c = lane; c < row_vec; c += 32) row[c] = make_uint4(0, 0, 0, 0);
    }
}

// One warp per (chunk, slice).
template <bool BF16, bool GRAD_BF16>
__global__ void __launch_bounds__(kSumWarps * 32) sum_runs_kernel(const SumParams p)
{
    constexpr int COLS = Cols<BF16>::N, SLICE = 32 * COLS;
    constexpr unsigned FULL = 0xffffffffu;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    chain_wait();
    chain_go();
    if ((int)blockIdx.x >= p.sum_blocks) {
        clear_rows<GRAD_BF16>(p, ((long long)((int)blockIdx.x - p.sum_blocks) * kSumWarps + warp) * kClearRows, lane);
        return;
    }
    const int item = (int)blockIdx.x * kSumWarps + warp;
    const int chunk = item / p.slices, slice = item - chunk * p.slices;
    if (chunk >= p.chunks) return;
    const int col = slice * SLICE + lane * COLS;
    const bool col_on = col < p.d;
    const int lo = (int)min((long long)p.n, (long long)chunk * p.chunk), hi = min(p.n, lo + p.chunk);
    const int prev = lo > 0 ? p.pair[lo - 1].x : -1;
    // 32 positions and the key behind them; positions without a token (key V) come last
    struct Row {
        int key, pos, next, live;
        unsigned ends;   // of runs
    };
    auto load = [&](int i0) {
        Row r;
        const int i = i0 + lane;
        const int2 v = i < hi ? p.pair[i] : make_int2(p.V, 0);
        r.key = v.x;
        r.pos = v.y;
        const int behind = min(i0 + kRow, hi);
        r.next = behind < p.n ? p.pair[behind].x : -1;
        return r;
    };
    auto settle = [&](Row &r, int i0) {
        r.live = __popc(__ballot_sync(FULL, r.key < p.V));
        int after = __shfl_down_sync(FULL, r.key, 1);
        if (lane == 31 || i0 + lane + 1 == hi) after = r.next;
        r.ends = __ballot_sync(FULL, r.key != after || i0 + lane + 1 == hi);
    };
    const char *dout = static_cast<const char *>(p.dout) + (long long)col * (BF16 ? 2 : 4);
    const long long ld = p.dout_ld * (BF16 ? 2 : 4);
    uint4 in[2][kBatch];
    auto fetch = [&](uint4 (&v)[kBatch], const Row &r, int k0) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int t = __shfl_sync(FULL, r.pos, (k0 + k) & 31);
            const int id = __shfl_sync(FULL, r.key, (k0 + k) & 31);
            v[k] = id < p.V && col_on ? __ldcs(reinterpret_cast<const uint4 *>(dout + t * ld))
                                      : make_uint4(0, 0, 0, 0);
        }
    };
    float *part = p.part + (long long)chunk * 2 * p.part_ld + col;
    float a[COLS] = {};
    bool first = true;   // the chunk's first run
    Row cur = load(lo);
    fetch(in[0], cur, 0);
    for (int i0 = lo; i0 < hi; i0 += kRow) {
        settle(cur, i0);
        Row ahead{p.V, 0, -1, 0, 0u};
        if (i0 + kRow < hi) ahead = load(i0 + kRow);
#pragma unroll
        for (int b = 0; b < kRow / kBatch; ++b) {
            const int k0 = b * kBatch;
            if (k0 >= cur.live) break;
            if (b + 1 < kRow / kBatch) fetch(in[(b + 1) & 1], cur, k0 + kBatch);
            else fetch(in[(b + 1) & 1], ahead, 0);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (k0 + k >= cur.live) break;
                add_row<BF16>(a, in[b & 1][k]);
                if (!(cur.ends >> (k0 + k) & 1)) continue;
                const int id = __shfl_sync(FULL, cur.key, k0 + k);
                const bool from_before = first && id == prev;
                const bool into_next = i0 + k0 + k + 1 == hi && id == cur.next;
                if (col_on) {
                    if (from_before || into_next) {
                        float4 *o = reinterpret_cast<float4 *>(part + (from_before ? 0 : p.part_ld));
#pragma unroll
                        for (int q = 0; q < COLS / 4; ++q)
                            o[q] = make_float4(a[4 * q], a[4 * q + 1], a[4 * q + 2], a[4 * q + 3]);
                    } else {
                        store_row<GRAD_BF16>(p, id, col, a);
                    }
                }
                if (into_next && !from_before && slice == 0 && lane == 0)
                    p.cross[atomicAdd(p.crossing, 1)] = make_int2(chunk, id);
#pragma unroll
                for (int c = 0; c < COLS; ++c) a[c] = 0.f;
                first = false;
            }
        }
        if (cur.live < kRow) break;
        cur = ahead;
    }
}

// Runs that begin in a chunk and go on in the next: the chunk's tail, then the heads of the
// chunks the run reaches.  A block takes one run at a time (of the list that the sums left, in
// any order); its warps are 128-column slices by shares of the chunks.
template <bool GRAD_BF16>
__global__ void __launch_bounds__(kJoinWarps * 32) join_runs_kernel(const SumParams p, int wide)
{
    constexpr unsigned FULL = 0xffffffffu;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int shares = kJoinWarps / wide, slice = warp % wide, share = warp / wide;
    __shared__ float4 sums[kJoinWarps][32];
    chain_wait();
    chain_go();
    const int runs = *p.crossing;
    for (int run = blockIdx.x; run < runs; run += gridDim.x) {
        const int2 begin = p.cross[run];
        const int chunk = begin.x, key = begin.y;
        // the last chunk whose first position has the key, 32 chunks at a time
        int in = chunk;
        while (true) {
            const int at = in + 1 + lane;
            const bool has = at < p.chunks && p.pair[(long long)at * p.chunk].x == key;
            const unsigned all = __ballot_sync(FULL, has);
            in += __popc(all);
            if (all != FULL) break;
        }
        for (int c0 = slice * 128; c0 < p.d + wide * 128; c0 += wide * 128) {
            const int col = c0 + lane * 4;
            const bool any = c0 - slice * 128 < p.d;   // (the same for the whole block)
            if (!any) break;
            float a[4] = {};
            // four loads in flight; then the shares' sums in their order
            for (int c = chunk + share; c <= in; c += 4 * shares) {
                float4 x[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int ck = c + k * shares;
                    x[k] = ck <= in && col < p.d
                               ? *reinterpret_cast<const float4 *>(p.part + (2LL * ck + (ck == chunk)) * p.part_ld + col)
                               : make_float4(0.f, 0.f, 0.f, 0.f);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    a[0] += x[k].x;
                    a[1] += x[k].y;
                    a[2] += x[k].z;
                    a[3] += x[k].w;
                }
            }
            sums[warp][lane] = make_float4(a[0], a[1], a[2], a[3]);
            __syncthreads();
            if (share == 0 && col < p.d) {
                for (int w = 1; w < shares; ++w) {
                    const float4 x = sums[w * wide + slice][lane];
                    a[0] += x.x;
                    a[1] += x.y;
                    a[2] += x.z;
                    a[3] += x.w;
                }
                store_row<GRAD_BF16>(p, key, col, a);
            }
            __syncthreads();
        }
    }
}

size_t up(size_t x) { return (x + 255) & ~(size_t)255; }

struct Layout {
    size_t pair[2], cross, part, total;
    long long part_ld;
    int chunk, chunks;
};

// Positions of a warp: as many as leave some 512 warps for each slice of columns, in rows of 32.
// Longer stretches leave fewer partial sums to join and fewer rows in flight (65536 tokens of 1024:
// sums and joins 37 + 25 us with 32 positions, 47 + 8 with 128).
int chunk_of(int n) { return std::min(kMaxChunk, std::max(kRow, n / 512 / kRow * kRow)); }

Layout layout(int n, int d)
{
    Layout l{};
    l.chunk = chunk_of(n);
    l.chunks = (int)(((long long)n + l.chunk - 1) / l.chunk);
    l.part_ld = (d + 31) / 32 * 32;
    size_t o = 0;
    for (int i = 0; i < 2; ++i) {
        l.pair[i] = o;
        o = up(o + (size_t)n * 8);
    }
    l.cross = o;
    o = up(o + ((size_t)l.chunks + 1) * 8);
    l.part = o;
    l.total = up(o + (size_t)l.chunks * 2 * l.part_ld * 4);
    return l;
}

template <bool BF16, bool GRAD_BF16>
cudaError_t sum_and_join(const SumParams &r, cudaStream_t s)
{
    const int rows = kSumWarps * kClearRows;
    const unsigned blocks = (unsigned)(r.sum_blocks + (r.accumulate ? 0 : (r.V + rows - 1) / rows));
    cudaError_t e = launch_grid(sum_runs_kernel<BF16, GRAD_BF16>, dim3(blocks), kSumWarps * 32, 0, s, 1, r);
    if (e == cudaSuccess && r.chunks > 1) {
        int wide = 1;   // slices of 128 columns side by side
        while (wide < 8 && wide * 128 < r.d) wide *= 2;
        const unsigned blocks = (unsigned)std::min(r.chunks - 1, 4 * device_sm_count());
        e = launch_grid(join_runs_kernel<GRAD_BF16>, dim3(blocks), kJoinWarps * 32, 0, s, 1, r, wide);
    }
    return e;
}

// Whether the device takes clusters of kSortWide blocks of the sort (asked once).
bool wide_clusters()
{
    static int known[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return false;
    if (!known[dev]) {
        int n = 0;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(kSortWide);
        cfg.blockDim = dim3(kSortThreads);
        cudaLaunchAttribute attr{};
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = kSortWide;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        const bool ok =
            cudaFuncSetAttribute(sort_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
            cudaOccupancyMaxActiveClusters(&n, sort_kernel, &cfg) == cudaSuccess && n > 0;
        if (!ok) cudaGetLastError();
        known[dev] = ok ? 1 : -1;
    }
    return known[dev] > 0;
}

} // namespace

cudaError_t launch_embed_fwd(const EmbedParams &p, bool bf16, cudaStream_t s)
{
    const int per = bf16 ? 8 : 4;
    const bool wide = p.d % per == 0 && p.emb_ld % per == 0 &&
                      (reinterpret_cast<uintptr_t>(p.emb) | reinterpret_cast<uintptr_t>(p.out)) % 16 == 0;
    const int row_vec = wide ? p.d / per : p.d;
    const long long ld = wide ? p.emb_ld / per : p.emb_ld;
    const long long total = (long long)p.n * row_vec;
    const unsigned grid = (unsigned)((total + kFwdThreads * kFwdVecs - 1) / (kFwdThreads * kFwdVecs));
    auto *kernel = wide ? (bf16 ? embed_fwd_kernel<true, uint4> : embed_fwd_kernel<false, uint4>)
                        : (bf16 ? embed_fwd_kernel<true, __nv_bfloat16> : embed_fwd_kernel<false, float>);
    return launch_grid(kernel, dim3(grid), kFwdThreads, 0, s, 1, p, row_vec, ld);
}

size_t embed_bwd_workspace_bytes(int n, int d) { return layout(n, d).total; }

cudaError_t launch_embed_bwd(const EmbedBwdParams &p, bool bf16, bool grad_bf16, void *workspace,
                             cudaStream_t s)
{
    const Layout l = layout(p.n, p.d);
    char *ws = static_cast<char *>(workspace);
    SortParams q{};
    q.tokens = p.tokens;
    for (int i = 0; i < 2; ++i) q.pair[i] = reinterpret_cast<int2 *>(ws + l.pair[i]);
    q.crossing = reinterpret_cast<int *>(ws + l.cross);
    q.index_bytes = p.index_bytes;
    q.n = p.n;
    q.V = p.V;
    q.status = p.status;
    int bits = 1;
    while (((long long)p.V >> bits) != 0) ++bits;  // (the key V stands for no token)
    q.passes = (bits + kDigit - 1) / kDigit;
    q.digit = (bits + q.passes - 1) / q.passes;
    const bool few = p.n <= kRankMost;
    q.blocks = few ? (p.n + 31) / 32 : p.n <= 16384 || !wide_clusters() ? kSortCluster : kSortWide;
    const int warps = q.blocks * kSortWarps;
    q.per_warp = (int)((((long long)p.n + warps - 1) / warps + 31) / 32 * 32);
    const dim3 grid((unsigned)q.blocks);
    const cudaError_t e = few ? launch_grid(rank_sort_kernel, grid, kRankThreads, 0, s, 1, q)
                              : launch_grid(sort_kernel, grid, kSortThreads, 0, s, (unsigned)q.blocks, q);
    if (e != cudaSuccess) return e;
    const int sorted = few ? 0 : q.passes & 1;

    SumParams r{};
    r.pair = q.pair[sorted];
    r.dout = p.dout;
    r.dout_ld = p.dout_ld;
    r.demb = p.demb;
    r.part = reinterpret_cast<float *>(ws + l.part);
    r.part_ld = l.part_ld;
    r.crossing = q.crossing;
    r.cross = reinterpret_cast<int2 *>(ws + l.cross) + 1;
    r.chunk = l.chunk;
    r.n = p.n;
    r.V = p.V;
    r.d = p.d;
    r.chunks = l.chunks;
    const int slice = bf16 ? 256 : 128;
    r.slices = (p.d + slice - 1) / slice;
    r.accumulate = p.accumulate;
    r.scale = p.scale;
    r.status = p.status;
    r.sum_blocks = (int)(((long long)l.chunks * r.slices + kSumWarps - 1) / kSumWarps);
    if (bf16 && grad_bf16) return sum_and_join<true, true>(r, s);
    if (bf16) return sum_and_join<true, false>(r, s);
    return grad_bf16 ? sum_and_join<false, true>(r, s) : sum_and_join<false, false>(r, s);
}

} // namespace txl
