// The token embedding and its gradient ("Transformer-XL: Attentive Language
// Models Beyond a Fixed-Length Context", §3.3: h^0 is the word embedding
// sequence).
//
//   forward   out_t = scale * E[token_t]
//   gradient  dE_v  = scale * sum_{t : token_t = v} dout_t
//
// Both move rows and are bound by HBM.  The gradient first sorts the positions
// by their tokens (a stable radix sort), then sums runs of equal tokens in
// chunks of kChunk positions; a run that crosses chunks leaves one partial per
// chunk, which a last launch sums in their order.  No sum depends on the order
// in which blocks run, so results repeat bit for bit.
#include "vocab.h"

namespace txl {
namespace {

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

__device__ __forceinline__ uint4 scaled(uint4 v, float s, bool bf16)
{
    if (!bf16)
        return make_uint4(__float_as_uint(__uint_as_float(v.x) * s), __float_as_uint(__uint_as_float(v.y) * s),
                          __float_as_uint(__uint_as_float(v.z) * s), __float_as_uint(__uint_as_float(v.w) * s));
    uint32_t *w = &v.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = bf2_to_f2(w[i]);
        w[i] = f2_to_bf2(f.x * s, f.y * s);
    }
    return v;
}

constexpr int kFwdThreads = 256;
constexpr int kFwdVecs = 4;  // vectors a thread keeps in flight

// Flat over (position, vector).
template <bool BF16>
__global__ void __launch_bounds__(kFwdThreads) embed_fwd_kernel(const EmbedParams p, int row_vec,
                                                                long long emb_vec)
{
    const long long total = (long long)p.n * row_vec;
    const long long base = (long long)blockIdx.x * (kFwdThreads * kFwdVecs) + threadIdx.x;
    const uint4 *emb = static_cast<const uint4 *>(p.emb);
    uint4 *out = static_cast<uint4 *>(p.out);
    uint4 v[kFwdVecs];
#pragma unroll
    for (int k = 0; k < kFwdVecs; ++k) {
        const long long i = base + k * kFwdThreads;
        v[k] = make_uint4(0, 0, 0, 0);
        if (i >= total) continue;
        const int t = (int)(i / row_vec), c = (int)(i - (long long)t * row_vec);
        const int id = token_at(p.tokens, p.index_bytes, t, p.V, p.status);
        if (id >= 0) v[k] = __ldg(emb + id * emb_vec + c);
    }
#pragma unroll
    for (int k = 0; k < kFwdVecs; ++k) {
        const long long i = base + k * kFwdThreads;
        if (i < total) out[i] = p.scale == 1.f ? v[k] : scaled(v[k], p.scale, BF16);
    }
}

// ---------------------------------------------------------------------------
// positions sorted by token
// ---------------------------------------------------------------------------
// LSD radix sort of (key, position): key = token, or V for a position without
// one.  Up to kTiles tiles of consecutive positions, one block each; a pass is
// a histogram per tile and a scatter whose blocks read all histograms.  One tile
// needs no histogram launch.  Within a block, rows of kSortThreads positions are
// ranked in order: by warp (match of equal digits), then over the warps' counts.

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kTiles = 64;
constexpr int kDigit = 9;
constexpr int kBins = 1 << kDigit;  // one bin a thread
static_assert(kBins == kSortThreads, "a thread keeps one bin");

struct SortParams {
    const void *tokens;      // first pass: keys come from here
    const int *key_in, *pos_in;
    int *key_out, *pos_out;
    int *hist;               // [tiles][kBins]
    unsigned int *present;   // bit per token, or null
    int index_bytes, n, V, shift, tile, tiles, present_words;
    unsigned int *status;
};

__device__ __forceinline__ int sort_key(const SortParams &p, int i)
{
    if (p.key_in) return p.key_in[i];
    const int id = token_at(p.tokens, p.index_bytes, i, p.V, p.status);
    return id < 0 ? p.V : id;
}

__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(const SortParams p)
{
    __shared__ int bins[kBins];
    bins[threadIdx.x] = 0;
    if (p.present)
        for (int i = blockIdx.x * kSortThreads + threadIdx.x; i < p.present_words;
             i += gridDim.x * kSortThreads)
            p.present[i] = 0;
    __syncthreads();
    const int lo = blockIdx.x * p.tile, hi = min(p.n, lo + p.tile);
    for (int i = lo + threadIdx.x; i < hi; i += kSortThreads)
        atomicAdd(bins + ((sort_key(p, i) >> p.shift) & (kBins - 1)), 1);
    __syncthreads();
    p.hist[blockIdx.x * kBins + threadIdx.x] = bins[threadIdx.x];
}

__global__ void __launch_bounds__(kSortThreads) sort_scatter_kernel(const SortParams p)
{
    __shared__ int base[kBins];                 // next place of each digit
    __shared__ int count[kSortWarps][kBins];    // of the current row, per warp
    __shared__ int warp_sum[kSortWarps];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // this tile's first place of digit `tid`: all smaller digits, and its own in earlier tiles
    int total = 0, before = 0;
    for (int t = 0; t < p.tiles; ++t) {
        const int c = p.hist[t * kBins + tid];
        total += c;
        before += t < (int)blockIdx.x ? c : 0;
    }
    int incl = total;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        incl += lane >= o ? v : 0;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int prefix = incl - total;
    for (int w = 0; w < warp; ++w) prefix += warp_sum[w];
    base[tid] = prefix + before;
    const int lo = blockIdx.x * p.tile, hi = min(p.n, lo + p.tile);
    for (int row = lo; row < hi; row += kSortThreads) {
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) count[w][tid] = 0;
        __syncthreads();
        const int i = row + tid;
        const bool on = i < hi;
        const int key = on ? sort_key(p, i) : 0;
        const int digit = (key >> p.shift) & (kBins - 1);
        const unsigned live = __ballot_sync(0xffffffffu, on);
        const unsigned same = __match_any_sync(0xffffffffu, digit) & live;
        const int rank = __popc(same & ((1u << lane) - 1));
        if (on && rank == 0) count[warp][digit] = __popc(same);
        __syncthreads();
        // places of each warp's digits in this row, and the next row's base
        int at = base[tid];
#pragma unroll
        for (int w = 0; w < kSortWarps; ++w) {
            const int c = count[w][tid];
            count[w][tid] = at;
            at += c;
        }
        base[tid] = at;
        __syncthreads();
        if (on) {
            const int to = count[warp][digit] + rank;
            TXL_CHECK(to >= 0 && to < p.n, p.status);
            p.key_out[to] = key;
            p.pos_out[to] = p.pos_in ? p.pos_in[i] : i;
            if (p.present && key < p.V) {
                const unsigned bit = 1u << (key & 31);
                if (!(p.present[key >> 5] & bit)) atomicOr(p.present + (key >> 5), bit);
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------------------
// sums over runs
// ---------------------------------------------------------------------------

constexpr int kChunk = 32;        // positions of a warp
constexpr int kSlice = 256;       // columns of a warp (eight a lane)
constexpr int kSumWarps = 4;

struct SumParams {
    const int *key, *pos;
    const unsigned int *present;
    const void *dout;
    long long dout_ld;
    void *demb;
    float *part;                  // [chunks][2][slices * kSlice]: of a run from before, of one into the next
    int n, V, d, chunks, slices, sum_blocks, accumulate;
    float scale;
    unsigned int *status;
};

struct Acc {
    float v[8];
};

template <bool BF16>
__device__ __forceinline__ Acc load_row(const SumParams &p, int t, int col)
{
    Acc a;
    if (BF16) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(
            static_cast<const __nv_bfloat16 *>(p.dout) + t * p.dout_ld + col));
        const float2 f0 = bf2_to_f2(v.x), f1 = bf2_to_f2(v.y), f2 = bf2_to_f2(v.z), f3 = bf2_to_f2(v.w);
        a = {f0.x, f0.y, f1.x, f1.y, f2.x, f2.y, f3.x, f3.y};
    } else {
        const float4 *s = reinterpret_cast<const float4 *>(static_cast<const float *>(p.dout) +
                                                           t * p.dout_ld + col);
        const float4 x = __ldcs(s), y = __ldcs(s + 1);
        a = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
    }
    return a;
}

template <bool GRAD_BF16>
__device__ __forceinline__ void store_row(const SumParams &p, int v, int col, const Acc &a)
{
    const long long at = (long long)v * p.d + col;
    if (GRAD_BF16) {
        uint4 o;
        o.x = f2_to_bf2(a.v[0] * p.scale, a.v[1] * p.scale);
        o.y = f2_to_bf2(a.v[2] * p.scale, a.v[3] * p.scale);
        o.z = f2_to_bf2(a.v[4] * p.scale, a.v[5] * p.scale);
        o.w = f2_to_bf2(a.v[6] * p.scale, a.v[7] * p.scale);
        *reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.demb) + at) = o;
    } else {
        float4 *o = reinterpret_cast<float4 *>(static_cast<float *>(p.demb) + at);
        float4 x = make_float4(a.v[0] * p.scale, a.v[1] * p.scale, a.v[2] * p.scale, a.v[3] * p.scale);
        float4 y = make_float4(a.v[4] * p.scale, a.v[5] * p.scale, a.v[6] * p.scale, a.v[7] * p.scale);
        if (p.accumulate) {
            const float4 ox = o[0], oy = o[1];
            x = make_float4(ox.x + x.x, ox.y + x.y, ox.z + x.z, ox.w + x.w);
            y = make_float4(oy.x + y.x, oy.y + y.y, oy.z + y.z, oy.w + y.w);
        }
        o[0] = x;
        o[1] = y;
    }
}

__device__ __forceinline__ void store_part(float *part, const Acc &a)
{
    float4 *o = reinterpret_cast<float4 *>(part);
    o[0] = make_float4(a.v[0], a.v[1], a.v[2], a.v[3]);
    o[1] = make_float4(a.v[4], a.v[5], a.v[6], a.v[7]);
}

// Blocks below sum_blocks: one warp per (chunk, slice).  The rest write the rows of
// tokens that do not occur, 32 tokens a warp.
template <bool BF16, bool GRAD_BF16>
__global__ void __launch_bounds__(kSumWarps * 32) sum_runs_kernel(const SumParams p)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if ((int)blockIdx.x >= p.sum_blocks) {
        const int word = ((int)blockIdx.x - p.sum_blocks) * kSumWarps + warp;
        const int v0 = word * 32;
        if (v0 >= p.V) return;
        unsigned absent = ~p.present[word];
        if (p.V - v0 < 32) absent &= (1u << (p.V - v0)) - 1;
        Acc zero{};
        for (; absent; absent &= absent - 1) {
            const int v = v0 + __ffs(absent) - 1;
            for (int col = lane * 8; col < p.d; col += kSlice) store_row<GRAD_BF16>(p, v, col, zero);
        }
        return;
    }
    const int item = (int)blockIdx.x * kSumWarps + warp;
    const int chunk = item / p.slices, slice = item - chunk * p.slices;
    if (chunk >= p.chunks) return;
    const int col = slice * kSlice + lane * 8;
    const bool col_on = col < p.d;
    const int lo = chunk * kChunk, cnt = min(kChunk, p.n - lo);
    const int my_key = lane < cnt ? p.key[lo + lane] : p.V;
    const int my_pos = lane < cnt ? p.pos[lo + lane] : 0;
    const int prev = lo > 0 ? p.key[lo - 1] : -1;
    const int next = lo + cnt < p.n ? p.key[lo + cnt] : -1;
    float *part = p.part + ((long long)chunk * 2 * p.slices + slice) * kSlice + lane * 8;
    const long long tail = (long long)p.slices * kSlice;
    int i = 0;
    while (i < cnt) {
        const int key = __shfl_sync(0xffffffffu, my_key, i);
        if (key >= p.V) break;  // (positions without a token come last)
        const unsigned same = __ballot_sync(0xffffffffu, lane < cnt && my_key == key);
        const int end = i + __popc(same);
        Acc a{};
        for (; i < end; i += 4) {
            Acc r[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = __shfl_sync(0xffffffffu, my_pos, (i + k) & 31);
                if (i + k < end && col_on) r[k] = load_row<BF16>(p, t, col);
                else r[k] = Acc{};
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int c = 0; c < 8; ++c) a.v[c] += r[k].v[c];
        }
        i = end;
        const bool from_before = key == prev && end - __popc(same) == 0;
        const bool into_next = end == cnt && key == next;
        if (from_before) store_part(part, a);
        else if (into_next) store_part(part + tail, a);
        else if (col_on) store_row<GRAD_BF16>(p, key, col, a);
    }
}

// Runs that begin in a chunk and go on in the next: the chunk's tail, then the heads of the
// chunks the run reaches.  One block per (chunk, slice), mostly without such a run.
template <bool GRAD_BF16>
__global__ void __launch_bounds__(kSumWarps * 32) join_runs_kernel(const SumParams p)
{
    const int chunk = blockIdx.x, slice = blockIdx.y;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int last = chunk * kChunk + kChunk - 1;
    if (last + 1 >= p.n) return;
    const int key = p.key[last];
    if (key >= p.V || p.key[last + 1] != key) return;
    // (the run began in an earlier chunk)
    if (chunk > 0 && p.key[chunk * kChunk - 1] == key) return;
    // the last chunk whose first position has the key: a search over the sorted keys
    int in = chunk + 1, out = p.chunks;
    while (out - in > 1) {
        const int mid = (in + out) / 2;
        if (p.key[mid * kChunk] == key) in = mid;
        else out = mid;
    }
    __shared__ float sums[kSumWarps][kSlice];
    const long long row = 2LL * p.slices * kSlice;
    const float *part = p.part + (long long)slice * kSlice + lane * 8;
    Acc a{};
    // partials over the warps in turn, then the warps' sums in their order
    for (int c = chunk + warp; c <= in; c += kSumWarps) {
        const float *src = part + c * row + (c == chunk ? (long long)p.slices * kSlice : 0);
        const float4 x = reinterpret_cast<const float4 *>(src)[0], y = reinterpret_cast<const float4 *>(src)[1];
        a.v[0] += x.x; a.v[1] += x.y; a.v[2] += x.z; a.v[3] += x.w;
        a.v[4] += y.x; a.v[5] += y.y; a.v[6] += y.z; a.v[7] += y.w;
    }
    store_part(&sums[warp][lane * 8], a);
    __syncthreads();
    const int col = slice * kSlice + lane * 8;
    if (warp > 0 || col >= p.d) return;
    for (int w = 1; w < kSumWarps; ++w)
#pragma unroll
        for (int c = 0; c < 8; ++c) a.v[c] += sums[w][lane * 8 + c];
    store_row<GRAD_BF16>(p, key, col, a);
}

size_t up(size_t x) { return (x + 255) & ~(size_t)255; }

struct Layout {
    size_t key[2], pos[2], hist, present, part, total;
    int chunks, slices, words;
};

Layout layout(int n, int V, int d)
{
    Layout l{};
    l.chunks = (int)(((long long)n + kChunk - 1) / kChunk);
    l.slices = (d + kSlice - 1) / kSlice;
    l.words = (int)(((long long)V + 31) / 32);
    size_t o = 0;
    for (int i = 0; i < 2; ++i) {
        l.key[i] = o;
        o = up(o + (size_t)n * 4);
        l.pos[i] = o;
        o = up(o + (size_t)n * 4);
    }
    l.hist = o;
    o = up(o + (size_t)kTiles * kBins * 4);
    l.present = o;
    o = up(o + (size_t)l.words * 4);
    l.part = o;
    l.total = up(o + (size_t)l.chunks * 2 * l.slices * kSlice * 4);
    return l;
}

} // namespace

cudaError_t launch_embed_fwd(const EmbedParams &p, bool bf16, cudaStream_t s)
{
    const int per = bf16 ? 8 : 4;
    const int row_vec = p.d / per;
    const long long total = (long long)p.n * row_vec;
    const unsigned grid = (unsigned)((total + kFwdThreads * kFwdVecs - 1) / (kFwdThreads * kFwdVecs));
    if (bf16) embed_fwd_kernel<true><<<grid, kFwdThreads, 0, s>>>(p, row_vec, p.emb_ld / per);
    else embed_fwd_kernel<false><<<grid, kFwdThreads, 0, s>>>(p, row_vec, p.emb_ld / per);
    return cudaGetLastError();
}

size_t embed_bwd_workspace_bytes(int n, int V, int d) { return layout(n, V, d).total; }

cudaError_t launch_embed_bwd(const EmbedBwdParams &p, bool bf16, bool grad_bf16, void *workspace,
                             cudaStream_t s)
{
    const Layout l = layout(p.n, p.V, p.d);
    char *ws = static_cast<char *>(workspace);
    SortParams q{};
    q.tokens = p.tokens;
    q.index_bytes = p.index_bytes;
    q.n = p.n;
    q.V = p.V;
    q.hist = reinterpret_cast<int *>(ws + l.hist);
    q.present_words = l.words;
    q.status = p.status;
    // tiles of whole rows of the block's threads
    q.tile = (int)((((long long)p.n + kTiles - 1) / kTiles + kSortThreads - 1) / kSortThreads * kSortThreads);
    q.tiles = (int)(((long long)p.n + q.tile - 1) / q.tile);
    int bits = 1;
    while (((long long)p.V >> bits) != 0) ++bits;  // (the key V stands for no token)
    int from = 0;
    for (int shift = 0; shift < bits; shift += kDigit) {
        q.shift = shift;
        q.present = shift == 0 ? reinterpret_cast<unsigned int *>(ws + l.present) : nullptr;
        q.key_in = shift == 0 ? nullptr : reinterpret_cast<const int *>(ws + l.key[from]);
        q.pos_in = shift == 0 ? nullptr : reinterpret_cast<const int *>(ws + l.pos[from]);
        q.key_out = reinterpret_cast<int *>(ws + l.key[from ^ 1]);
        q.pos_out = reinterpret_cast<int *>(ws + l.pos[from ^ 1]);
        sort_count_kernel<<<q.tiles, kSortThreads, 0, s>>>(q);
        sort_scatter_kernel<<<q.tiles, kSortThreads, 0, s>>>(q);
        from ^= 1;
    }
    SumParams r{};
    r.key = reinterpret_cast<const int *>(ws + l.key[from]);
    r.pos = reinterpret_cast<const int *>(ws + l.pos[from]);
    r.present = reinterpret_cast<const unsigned int *>(ws + l.present);
    r.dout = p.dout;
    r.dout_ld = p.dout_ld;
    r.demb = p.demb;
    r.part = reinterpret_cast<float *>(ws + l.part);
    r.n = p.n;
    r.V = p.V;
    r.d = p.d;
    r.chunks = l.chunks;
    r.slices = l.slices;
    r.accumulate = p.accumulate;
    r.scale = p.scale;
    r.status = p.status;
    r.sum_blocks = (int)(((long long)l.chunks * l.slices + kSumWarps - 1) / kSumWarps);
    const int fill_blocks = p.accumulate ? 0 : (l.words + kSumWarps - 1) / kSumWarps;
    const unsigned grid = (unsigned)(r.sum_blocks + fill_blocks);
    const int threads = kSumWarps * 32;
    if (bf16 && grad_bf16) sum_runs_kernel<true, true><<<grid, threads, 0, s>>>(r);
    else if (bf16) sum_runs_kernel<true, false><<<grid, threads, 0, s>>>(r);
    else if (grad_bf16) sum_runs_kernel<false, true><<<grid, threads, 0, s>>>(r);
    else sum_runs_kernel<false, false><<<grid, threads, 0, s>>>(r);
    if (l.chunks > 1) {
        const dim3 join((unsigned)(l.chunks - 1), (unsigned)l.slices);
        if (grad_bf16) join_runs_kernel<true><<<join, threads, 0, s>>>(r);
        else join_runs_kernel<false><<<join, threads, 0, s>>>(r);
    }
    return cudaGetLastError();
}

} // namespace txl
