// Log probabilities of tokens: joining the vocabulary ranges of a row, and the small passes
// around the products of logprob.cu.
#include "vocab.h"
#include "ptx.cuh"

namespace txl {
namespace {

using namespace ptx;

// ---------------------------------------------------------------------------
// joining the vocabulary ranges of a row
// ---------------------------------------------------------------------------

// A number as hi + lo, |lo| at most half a unit of hi's last place.
struct Wide {
    float hi, lo;
};

// h_i . w_j to about 2^-45 of its terms' size, over a warp: products split exactly (a bf16
// product is an fp32 value; an fp32 one is a product and its rounding error by fma), sums
// carried with their errors, four chains a lane.  Where that is no number, the plain sum.  (All in
// fp32: the fp64 units give one result where the fp32 ones give 64.)
struct ExactSum {
    float hi[4] = {}, lo[4] = {}, plain = 0.f;

    // Sixteen bytes of each operand.
    template <bool BF16>
    __device__ __forceinline__ void add(const uint4 &x, const uint4 &y)
    {
        const uint32_t xp[4] = {x.x, x.y, x.z, x.w}, yp[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (BF16) {
                const float q0 = __fmul_rn(__uint_as_float(xp[i] << 16), __uint_as_float(yp[i] << 16));
                const float q1 = __fmul_rn(__uint_as_float(xp[i] & 0xffff0000u),
                                           __uint_as_float(yp[i] & 0xffff0000u));
                two_sum(hi[i], lo[i], q0);
                two_sum(hi[i], lo[i], q1);
                plain += q0 + q1;
            } else {
                const float a = __uint_as_float(xp[i]), b = __uint_as_float(yp[i]), q = __fmul_rn(a, b);
                two_sum(hi[i], lo[i], q);
                lo[i] += fmaf(a, b, -q);
                plain += q;
            }
        }
    }

    __device__ __forceinline__ Wide over_warp()
    {
#pragma unroll
        for (int i = 1; i < 4; ++i) {
            two_sum(hi[0], lo[0], hi[i]);
            lo[0] += lo[i];
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float ohi = __shfl_xor_sync(0xffffffffu, hi[0], o), olo = __shfl_xor_sync(0xffffffffu, lo[0], o);
            two_sum(hi[0], lo[0], ohi);
            lo[0] += olo;
        }
        Wide z{__fadd_rn(hi[0], lo[0]), 0.f};
        z.lo = lo[0] - __fadd_rn(z.hi, -hi[0]);
        if (!isfinite(z.hi)) {
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) plain += __shfl_xor_sync(0xffffffffu, plain, o);
            z = {plain, 0.f};
        }
        return z;
    }
};

template <bool BF16>
__device__ __forceinline__ Wide dot_exact(const void *h, const void *w, int d, int lane)
{
    const uint4 *a = static_cast<const uint4 *>(h), *b = static_cast<const uint4 *>(w);
    const int vecs = d / (BF16 ? 8 : 4);
    ExactSum sum;
#pragma unroll 4
    for (int c = lane; c < vecs; c += 32) sum.add<BF16>(a[c], b[c]);
    return sum.over_warp();
}

// Order of scale * z as integers, 0 for no number: by the product's sign (the scale only
// stretches it).
__device__ __forceinline__ unsigned long long wide_key(Wide z, float scale)
{
    if (!(z.hi * scale == z.hi * scale)) return 0ull;
    if (scale == 0.f) return 1ull;
    const float s = scale < 0.f ? -1.f : 1.f;
    return (unsigned long long)order_key(z.hi * s + 0.f) << 32 | order_key(isfinite(z.hi) ? z.lo * s + 0.f : 0.f);
}

constexpr int kMergeWarps = 4;
constexpr int kLaneLists = kMaxStatSplits / 32;
constexpr float kLn2 = 0.6931471805599453f;

// Softmax statistics of a row from its ranges', over a warp: lane s holds ranges s, s + 32, ...
struct RowSums {
    float m, mu, sum, lo, es, zt;
};

// The sum is hi + lo: beside one term near 1 the others count, its logarithm is theirs.
template <int PER>
__device__ __forceinline__ RowSums join_stats(const MergeParams &p, int row, int lane)
{
    constexpr unsigned FULL = 0xffffffffu;
    float4 st[PER];
    RowSums r{-INFINITY, 0.f, 0.f, 0.f, 0.f, 0.f};
    bool nan = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int s = lane + 32 * i;
        st[i] = s < p.splits ? p.stats[(long long)s * p.N + row] : make_float4(-INFINITY, 0.f, 0.f, 0.f);
        r.m = fmaxf(r.m, st[i].x);
        nan = nan || st[i].y != st[i].y;
        r.zt += st[i].w;  // (zero but in the target's range)
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        r.m = fmaxf(r.m, __shfl_xor_sync(FULL, r.m, o));
        r.zt += __shfl_xor_sync(FULL, r.zt, o);
    }
    r.mu = r.m == -INFINITY ? 0.f : r.m;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        if (st[i].x == -INFINITY && st[i].y == 0.f) continue;
        const float d = fmaxf(st[i].x - r.mu, -1e30f), f = exp2f(d);  // (bounded: times a sum it stays finite)
        two_sum(r.sum, r.lo, f);
        two_sum(r.sum, r.lo, st[i].y * f);
        r.es += (st[i].z + (st[i].y + 1.f) * d) * f;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float hi = __shfl_xor_sync(FULL, r.sum, o), lo = __shfl_xor_sync(FULL, r.lo, o);
        two_sum(r.sum, r.lo, hi);
        r.lo += lo;
        r.es += __shfl_xor_sync(FULL, r.es, o);
    }
    if (__any_sync(FULL, nan)) r.sum = __int_as_float(0x7fffffff);
    return r;
}

// scale * z in log2 units less mu.
__device__ __forceinline__ float above(const MergeParams &p, Wide z, float mu)
{
    return fmaf(z.hi, p.c_hi, -mu) + fmaf(z.hi, p.c_lo, z.lo * p.c_hi);
}

// A logit known more exactly (d1 above mu) takes its place in the sums: peaked rows, whose sums
// are a few such terms, are as exact as these.
__device__ __forceinline__ void replace_term(float mu, float was, float d1, float &ds, float &de)
{
    // (as a multiple of the term that was there: of two numbers near 1 the difference would be a rounding)
    const float d0 = was - mu, e0 = ex2(d0);
    if (e0 == 0.f) return;  // (nothing is in the sums; the difference may be anything)
    ds = e0 * expm1f((d1 - d0) * kLn2);
    de = fmaf(ds, d1, e0 * (d1 - d0));
}

// Row outputs from the sums; d_target: the target's logit above mu (log2 units).  Returns
// log(sum): a log probability is its logit above mu, times ln 2, less that.
__device__ __forceinline__ float row_outputs(const MergeParams &p, int row, const RowSums &r, int target,
                                             float d_target, bool write)
{
    float l = logf(r.sum);
    if (isfinite(l)) l += r.lo / r.sum;
    if (write) {
        if (p.logp) p.logp[row] = target >= 0 ? fmaf(d_target, kLn2, -l) : 0.f;
        // (ln 2 to fp64; a maximum of -infinity stands for itself)
        if (p.lse) p.lse[row] = fmaf(r.m, kLn2, r.m > -INFINITY ? fmaf(r.m, -1.9046542e-9f, l) : l);
        if (p.entropy) p.entropy[row] = l - r.es / r.sum * kLn2;
    }
    return l;
}

// Rows of the statistics kernel: one warp each.  Its ranges' lists are two a lane.
template <bool BF16, int LIST>
__global__ void __launch_bounds__(kMergeWarps * 32) logprob_merge_kernel(const MergeParams p)
{
    constexpr unsigned FULL = 0xffffffffu;
    chain_wait();
    chain_go();
    constexpr int PER = 2 * kMaxRowSplits / 32, WANT = LIST > 0 ? LIST : 1;
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
    if (row >= p.N) return;
    const int target = p.targets ? token_at(p.targets, p.index_bytes, row, p.V, p.status) : -1;
    const int esize = BF16 ? 2 : 4;
    const char *h = static_cast<const char *>(p.h) + row * p.h_ld * esize;
    auto exact = [&](int id) {
        return dot_exact<BF16>(h, static_cast<const char *>(p.w) + id * p.w_ld * esize, p.d, lane);
    };
    // the largest of all ranges, from the heads of their lists
    const int want = LIST > 0 ? min(p.top + kSpareTop, LIST) : 0;
    float my_val = 0.f;   // candidate of lane c
    int my_id = -1;
    if (LIST > 0) {
        float val[PER][WANT];
        int id[PER][WANT];
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int s = lane + 32 * i;
#pragma unroll
            for (int j = 0; j < LIST; ++j) {
                const bool on = s < p.splits;
                const long long at = ((long long)s * LIST + j) * p.N + row;
                id[i][j] = on ? p.list_id[at] : -1;
                val[i][j] = on ? p.list_val[at] + 0.f : 0.f;  // (+ 0: zeros of one sign)
            }
        }
        for (int c = 0; c < want; ++c) {
            uint32_t key = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (id[i][0] >= 0) key = max(key, order_key(val[i][0]));
            const uint32_t most = __reduce_max_sync(FULL, key);
            if (!most) break;
            unsigned mine = 0xffffffffu;
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (id[i][0] >= 0 && order_key(val[i][0]) == most) mine = min(mine, (unsigned)id[i][0]);
            const int won = (int)__reduce_min_sync(FULL, mine);
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (id[i][0] == won) {
#pragma unroll
                    for (int j = 0; j + 1 < LIST; ++j) {
                        id[i][j] = id[i][j + 1];
                        val[i][j] = val[i][j + 1];
                    }
                    id[i][WANT - 1] = -1;
                }
            if (lane == c) {
                my_val = key_value(most);
                my_id = won;
            }
        }
    }
    const int found = __popc(__ballot_sync(FULL, my_id >= 0));
    // exact logits of the candidates, and of the target where it is none of them
    RowSums r = join_stats<PER>(p, row, lane);
    float d_mine = my_val - r.mu, d_target = r.zt - r.mu;
    unsigned long long order = my_id >= 0 ? (unsigned long long)order_key(my_val) << 32 : 0ull;
    float ds = 0.f, de = 0.f;
    bool listed = false;
    for (int c = 0; c < found; ++c) {
        const int id = __shfl_sync(FULL, my_id, c);
        const Wide e = exact(id);
        if (lane == c) {
            // (beside infinite ones the rounded logit orders as well)
            const unsigned long long k = wide_key(e, p.scale);
            if (k) order = k;
            if (isfinite(e.hi) && isfinite(my_val)) {
                d_mine = above(p, e, r.mu);
                replace_term(r.mu, my_val, d_mine, ds, de);
            }
        }
        if (id == target) {
            listed = true;
            d_target = __shfl_sync(FULL, d_mine, c);
        }
    }
    if (target >= 0 && !listed) {
        const Wide e = exact(target);
        if (isfinite(e.hi) && isfinite(r.zt)) {
            d_target = above(p, e, r.mu);
            // (found is below 32: this lane has no candidate)
            if (lane == 31) replace_term(r.mu, r.zt, d_target, ds, de);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        ds += __shfl_xor_sync(FULL, ds, o);
        de += __shfl_xor_sync(FULL, de, o);
    }
    two_sum(r.sum, r.lo, ds);
    r.es += de;
    const float l = row_outputs(p, row, r, target, d_target, lane == 0);
    if (LIST == 0) return;
    int rank = 0;
    for (int c = 0; c < found; ++c) {
        const unsigned long long other = __shfl_sync(FULL, order, c);
        const int oid = __shfl_sync(FULL, my_id, c);
        if (other > order || (other == order && oid < my_id)) ++rank;
    }
    if (my_id >= 0 && rank < p.top) {
        p.top_ids[(long long)row * p.top + rank] = my_id;
        p.top_logp[(long long)row * p.top + rank] = fmaf(d_mine, kLn2, -l);
    }
    if (lane >= found && lane < p.top) {  // fewer numbers than places
        p.top_ids[(long long)row * p.top + lane] = -1;
        p.top_logp[(long long)row * p.top + lane] = __int_as_float(0x7fffffff);
    }
}

// Rows of the kernel for few states: a block each.  The `want` largest logits lie in the `want`
// groups of four with the largest maxima.  Those are found by a threshold that at least `want`
// warps' own maxima reach, then ranked among all that reach it.  Where the logits themselves were
// written (FULL: few states beside the width), the `want` largest of the groups' members are the
// candidates, else all members; the candidates' exact products give the order.
constexpr int kFewWarps = 32;
constexpr int kFewThreads = kFewWarps * 32;
constexpr int kFewCap = 256;                          // groups above the threshold
constexpr int kFewWant = kMaxTop + kSpareTop;
constexpr int kFewLoads = 4;                          // 16-byte loads of a thread in flight
static_assert(kFewWant < kFewWarps, "a threshold from the warps' maxima");

template <bool BF16, bool FULL>
__global__ void __launch_bounds__(kFewThreads) logprob_few_merge_kernel(const MergeParams p)
{
    constexpr unsigned ALL = 0xffffffffu;
    __shared__ unsigned s_key[kFewCap];
    __shared__ int s_at[kFewCap];
    __shared__ int s_count;
    __shared__ unsigned s_thr, s_best_key[kFewWarps];
    __shared__ int s_best_at[kFewWarps];
    __shared__ unsigned g_key[kFewWant];              // the groups, in order
    __shared__ int g_at[kFewWant];
    __shared__ unsigned m_key[4 * kFewWant];          // FULL: their members
    __shared__ int c_id[4 * kFewWant];                // the candidates
    __shared__ float c_was[4 * kFewWant];             // ... their logits in the sums (NaN: not known)
    __shared__ Wide s_z[4 * kFewWant + 1];            // ... their exact products, then the target's
    __shared__ unsigned long long s_order[4 * kFewWant];
    __shared__ RowSums s_sums;
    __shared__ float s_l;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.x;
    chain_wait();
    chain_go();
    const int target = p.targets ? token_at(p.targets, p.index_bytes, row, p.V, p.status) : -1;
    const int esize = BF16 ? 2 : 4;
    const char *h = static_cast<const char *>(p.h) + row * p.h_ld * esize;
    const float nan = __int_as_float(0x7fffffff);
    int jobs = 0;                                     // candidates
    if (p.top > 0) {
        // vectors of four groups' maxima; the first kFewLoads of a thread stay in its registers
        const int n = p.nb * 8, want = min(p.top + kSpareTop, kFewWant);
        const uint4 *src = reinterpret_cast<const uint4 *>(p.group_key) + (long long)row * n;
        uint4 held[kFewLoads];
        auto load = [&](uint4 (&k)[kFewLoads], int i0) {
#pragma unroll
            for (int u = 0; u < kFewLoads; ++u) {
                const int i = i0 + u * kFewThreads;
                k[u] = i < n ? src[i] : make_uint4(0, 0, 0, 0);
            }
        };
        // (the code below is run once by a block: it is kept short, a cold instruction costs more
        // than its work)
        const unsigned *one = reinterpret_cast<const unsigned *>(src);
        auto scan = [&](auto take) {   // take(mask of a thread's 16 maxima, place of the first)
            for (int i0 = tid; i0 < n; i0 += kFewThreads * kFewLoads) {
                if (i0 > tid) load(held, i0);
                take(i0);
            }
            if (n > kFewThreads * kFewLoads) load(held, tid);
        };
        load(held, tid);
        unsigned mine = 0;
        scan([&](int) {
#pragma unroll
            for (int u = 0; u < kFewLoads; ++u)
                mine = max(mine, max(max(held[u].x, held[u].y), max(held[u].z, held[u].w)));
        });
        const unsigned most = __reduce_max_sync(ALL, mine);
        if (lane == 0) s_best_key[warp] = most;
        if (tid == 0) s_count = 0;
        __syncthreads();
        // the want-th largest of the warps' maxima (a warp's own: distinct groups)
        if (warp == 0) {
            const unsigned w_key = s_best_key[lane];
            int ahead = 0;
#pragma unroll
            for (int o = 0; o < kFewWarps; ++o) {
                const unsigned other = __shfl_sync(ALL, w_key, o);
                ahead += (other > w_key) | ((other == w_key) & (o < lane));
            }
            const unsigned t = __reduce_max_sync(ALL, ahead == want - 1 ? w_key : 0u);
            if (lane == 0) s_thr = max(1u, t);
        }
        __syncthreads();
        const unsigned thr = s_thr;
        if (mine >= thr)
            scan([&](int i0) {
                unsigned hits = 0;
#pragma unroll
                for (int u = 0; u < kFewLoads; ++u)
                    hits |= ((held[u].x >= thr) | (held[u].y >= thr) << 1 | (held[u].z >= thr) << 2 |
                             (held[u].w >= thr) << 3) << (4 * u);
                for (; hits; hits &= hits - 1) {
                    const int bit = __ffs(hits) - 1, place = (i0 + (bit >> 2) * kFewThreads) * 4 + (bit & 3);
                    const int at = atomicAdd(&s_count, 1);
                    if (at < kFewCap) {
                        s_key[at] = one[place];
                        s_at[at] = place;
                    }
                }
            });
        __syncthreads();
        const int count = s_count;
        int groups = 0;
        if (count <= kFewCap) {
            if (tid < count) {
                int rank = 0;
                const unsigned k = s_key[tid];
                const int at = s_at[tid];
#pragma unroll 4
                for (int c = 0; c < count; ++c) rank += (s_key[c] > k) | ((s_key[c] == k) & (s_at[c] < at));
                if (rank < want) {
                    g_key[rank] = k;
                    g_at[rank] = at;
                }
            }
            groups = min(count, want);
        } else {
            // very many equal maxima: one after the other, the lowest group of equal ones first
            unsigned last_key = 0xffffffffu;
            int last_at = -1;
            for (int c = 0; c < want; ++c) {
                unsigned bk = 0;
                int ba = 0x7fffffff;
                for (int i = tid; i < n * 4; i += kFewThreads) {
                    const unsigned k = one[i];
                    const bool left = k && (k < last_key || (k == last_key && i > last_at));
                    if (left && k > bk) {
                        bk = k;
                        ba = i;
                    }
                }
                unsigned top = __reduce_max_sync(ALL, bk);
                int at = (int)__reduce_min_sync(ALL, bk == top ? (unsigned)ba : 0x7fffffffu);
                __syncthreads();
                if (lane == 0) {
                    s_best_key[warp] = top;
                    s_best_at[warp] = at;
                }
                __syncthreads();
                bk = s_best_key[lane];
                ba = s_best_at[lane];
                top = __reduce_max_sync(ALL, bk);
                at = (int)__reduce_min_sync(ALL, bk == top ? (unsigned)ba : 0x7fffffffu);
                if (!top) break;
                if (tid == 0) {
                    g_key[c] = top;
                    g_at[c] = at;
                }
                last_key = top;
                last_at = at;
                groups = c + 1;
            }
        }
        __syncthreads();
        // the candidates
        const int members = 4 * groups;
        const int id = tid < members ? g_at[tid >> 2] * 4 + (tid & 3) : 0;
        if (FULL) {
            const float *logit = p.logits + (long long)row * p.nb * 128;
            const float v = tid < members ? logit[id] : nan;
            const unsigned k = tid < members && id < p.V && v == v ? order_key(v) : 0u;
            if (tid < members) m_key[tid] = k;
            const int some = __syncthreads_count(k != 0);
            if (k) {
                int rank = 0;
#pragma unroll 4
                for (int o = 0; o < members; ++o) {
                    const int oid = g_at[o >> 2] * 4 + (o & 3);
                    rank += (m_key[o] > k) | ((m_key[o] == k) & (oid < id));
                }
                if (rank < want) {
                    c_id[rank] = id;
                    c_was[rank] = v;
                }
            }
            jobs = min(some, want);
        } else {
            if (tid < members) {
                c_id[tid] = id < p.V ? id : -1;
                c_was[tid] = nan;
            }
            jobs = members;
        }
        __syncthreads();
    }
    // the ranges' sums (last warp); exact logits, the target's first
    if (warp == kFewWarps - 1) {
        const RowSums r = join_stats<kLaneLists>(p, row, lane);
        if (lane == 0) s_sums = r;
    }
    for (int c = warp; c <= jobs; c += kFewWarps) {
        const int id = c == 0 ? target : c_id[c - 1];
        Wide e{nan, 0.f};  // no such token
        if (id >= 0) e = dot_exact<BF16>(h, static_cast<const char *>(p.w) + id * p.w_ld * esize, p.d, lane);
        if (lane == 0) {
            s_z[c == 0 ? 4 * kFewWant : c - 1] = e;
            if (c > 0) s_order[c - 1] = wide_key(e, p.scale);
        }
    }
    __syncthreads();
    if (FULL && warp > 0) return;
    // places in the order, while the first warp finishes the sums; FULL: it does both
    int rank = 0;
    const int c = FULL ? tid : tid - 32;
    const bool on = c >= 0 && c < jobs && s_order[c] != 0;
    if (on) {
        const unsigned long long k = s_order[c];
        const int id = c_id[c];
#pragma unroll 4
        for (int o = 0; o < jobs; ++o) {
            const unsigned long long other = s_order[o];
            rank += (other > k) | ((other == k) & (c_id[o] < id));
        }
    }
    const int found = FULL ? __popc(__ballot_sync(ALL, on)) : __syncthreads_count(on);
    RowSums r = s_sums;
    float l = 0.f;
    if (warp == 0) {
        if (target >= 0) r.zt = p.target_z[row];
        float d_target = r.zt - r.mu, ds = 0.f, de = 0.f;
        bool replaced = false;
        if (lane < (FULL ? jobs : jobs / 4)) {
            // (without the logits themselves: a group's maximum was its largest member's)
            int at = FULL ? lane : 4 * lane;
            if (!FULL)
                for (int i = 1; i < 4; ++i)
                    if (s_order[4 * lane + i] > s_order[at]) at = 4 * lane + i;
            const Wide best = s_z[at];
            const float was = FULL ? c_was[lane] : key_value(g_key[lane]);
            if (isfinite(best.hi) && isfinite(was)) replace_term(r.mu, was, above(p, best, r.mu), ds, de);
            replaced = c_id[at] == target;
        }
        const bool in_sums = __any_sync(ALL, replaced);
        if (target >= 0) {
            const Wide e = s_z[4 * kFewWant];
            if (isfinite(e.hi) && isfinite(r.zt)) {
                d_target = above(p, e, r.mu);
                if (!in_sums && lane == 31) replace_term(r.mu, r.zt, d_target, ds, de);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            ds += __shfl_xor_sync(ALL, ds, o);
            de += __shfl_xor_sync(ALL, de, o);
        }
        two_sum(r.sum, r.lo, ds);
        r.es += de;
        l = row_outputs(p, row, r, target, d_target, lane == 0);
        if (!FULL && lane == 0) s_l = l;
    }
    if (!FULL) {
        __syncthreads();
        l = s_l;
    }
    if (on && rank < p.top) {
        p.top_ids[(long long)row * p.top + rank] = c_id[c];
        const Wide z = s_z[c];
        const float d = isfinite(z.hi) ? above(p, z, r.mu) : z.hi * p.scale - r.mu;
        p.top_logp[(long long)row * p.top + rank] = fmaf(d, kLn2, -l);
    }
    if (tid >= found && tid < p.top) {  // fewer numbers than places
        p.top_ids[(long long)row * p.top + tid] = -1;
        p.top_logp[(long long)row * p.top + tid] = __int_as_float(0x7fffffff);
    }
}

// ---------------------------------------------------------------------------
// small passes
// ---------------------------------------------------------------------------

// Blocks below blocks0 sum the first result, the others the second.  Twelve parts in flight (four: 9 us
// for the 32 parts of 29 x 224).
__global__ void __launch_bounds__(256) sum_parts_kernel(const PartsSum r0, const PartsSum r1, int blocks0)
{
    const bool second = (int)blockIdx.x >= blocks0;
    const PartsSum r = second ? r1 : r0;
    const long long vecs = r.elems / 4;
    const long long i = (long long)((int)blockIdx.x - (second ? blocks0 : 0)) * 256 + threadIdx.x;
    chain_wait();
    chain_go();
    if (i >= vecs) return;
    const float4 *part = reinterpret_cast<const float4 *>(r.part) + i;
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int FLY = 12;
    for (int s = 0; s < r.parts; s += FLY) {
        float4 b[FLY];
#pragma unroll
        for (int k = 0; k < FLY; ++k)
            b[k] = s + k < r.parts ? __ldcs(part + (s + k) * vecs) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < FLY; ++k) {
            a.x += b[k].x;
            a.y += b[k].y;
            a.z += b[k].z;
            a.w += b[k].w;
        }
    }
    if (r.bf16)
        static_cast<uint2 *>(r.out)[i] = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
    else
        static_cast<float4 *>(r.out)[i] = a;
}

// x = t0 + t1 + t2, each the bf16 nearest to what is left (exact but for what falls below
// bf16's range).  An infinite or NaN value is its first term; a finite one that rounds to
// infinity is cut instead.
__device__ __forceinline__ float next_term(float &x)
{
    __nv_bfloat16 n = __float2bfloat16_rn(x);
    if (__hisinf(n) && !isinf(x)) n = __float2bfloat16_rz(x);
    const float t = __bfloat162float(n);
    x = isfinite(x) ? x - t : 0.f;
    return t;
}

// Four values: their terms to the three planes (dst of the first, planes `plane` elements apart).
__device__ __forceinline__ void split4(const uint4 &x, __nv_bfloat16 *dst, long long plane)
{
    float v[4] = {__uint_as_float(x.x), __uint_as_float(x.y), __uint_as_float(x.z), __uint_as_float(x.w)};
#pragma unroll
    for (int t = 0; t < kMaxPieces; ++t) {
        float y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) y[k] = next_term(v[k]);
        *reinterpret_cast<uint2 *>(dst + t * plane) = make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
    }
}

// A thread takes two vectors of eight, `threads` apart.
__device__ __forceinline__ void split_block(const SplitRows &r, long long block, int threads)
{
    const int vecs = r.d / 8;
    const long long total = (long long)r.rows * vecs, base = block * threads * 2 + threadIdx.x;
    const long long plane = (long long)r.rows * r.plane_ld;
    uint4 v[2][2] = {};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const long long i = base + k * threads;
        if (i >= total) continue;
        const int row = (int)(i / vecs), c = (int)(i - (long long)row * vecs);
        const uint4 *src = reinterpret_cast<const uint4 *>(r.x + row * r.ld + c * 8);
        v[k][0] = __ldcs(src);
        v[k][1] = __ldcs(src + 1);
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const long long i = base + k * threads;
        if (i >= total) continue;
        const int row = (int)(i / vecs), c = (int)(i - (long long)row * vecs);
        __nv_bfloat16 *dst = r.planes + (long long)row * r.plane_ld + c * 8;
        float x[8];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            x[4 * j] = __uint_as_float(v[k][j].x);
            x[4 * j + 1] = __uint_as_float(v[k][j].y);
            x[4 * j + 2] = __uint_as_float(v[k][j].z);
            x[4 * j + 3] = __uint_as_float(v[k][j].w);
        }
#pragma unroll
        for (int t = 0; t < kMaxPieces; ++t) {
            float y[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) y[j] = next_term(x[j]);
            *reinterpret_cast<uint4 *>(dst + t * plane) =
                make_uint4(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]), pack_bf16x2(y[4], y[5]),
                           pack_bf16x2(y[6], y[7]));
        }
    }
}

long long split_blocks(const SplitRows &r, int threads)
{
    return ((long long)r.rows * (r.d / 8) + threads * 2 - 1) / (threads * 2);
}

// Two operands in one launch.
__global__ void __launch_bounds__(256) split_f32_kernel(const SplitRows r0, const SplitRows r1, long long blocks0)
{
    chain_wait();
    chain_go();
    if (blockIdx.x < blocks0) split_block(r0, blockIdx.x, 256);
    else split_block(r1, blockIdx.x - blocks0, 256);
}

// One warp per row: a copy of h with zeros in rows that have no part in the gradient (whatever
// those hold), and the log probability of the row's target from its logit summed with rounding (of fp32
// operands: carried beyond fp32), not by the accumulators that cut: G's one large element is the
// difference of 1 and that probability.
template <bool BF16>
__global__ void __launch_bounds__(kMergeWarps * 32) grad_rows_kernel(const GradRowsParams p, int row_blocks)
{
    chain_wait();
    chain_go();
    if (!BF16 && (int)blockIdx.x >= row_blocks) {  // the table's terms, in the same launch
        split_block(p.table, (int)blockIdx.x - row_blocks, kMergeWarps * 32);
        return;
    }
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
    if (row >= p.N) return;
    constexpr int ESIZE = BF16 ? 2 : 4;
    const int vecs = p.d * ESIZE / 16;
    const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const char *>(p.h) + row * p.h_ld * ESIZE);
    // (fp32: as terms)
    __nv_bfloat16 *out = p.out + (long long)row * p.out_ld;
    const long long id = p.targets ? raw_token(p.targets, p.index_bytes, row) : -1;
    // (the row does not wait for the token, the table's row does)
    uint4 h[4];
    auto load = [&](int c0) {
#pragma unroll
        for (int k = 0; k < 4; ++k) h[k] = c0 + 32 * k < vecs ? src[c0 + 32 * k] : make_uint4(0, 0, 0, 0);
    };
    load(lane);
    const int target = checked_token(id, p.V, p.status);
    const bool live = target >= 0 || (p.dentropy && p.dentropy[row] != 0.f);
    const uint4 *w = reinterpret_cast<const uint4 *>(static_cast<const char *>(p.w) + max(target, 0) * p.w_ld * ESIZE);
    ExactSum sum;
    float chain[4] = {};  // (bf16: rounded sums will do beside G's own rounding)
    for (int c0 = lane; c0 < vecs; c0 += 128) {
        if (c0 > lane) load(c0);
        uint4 y[4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            y[k] = target >= 0 && c0 + 32 * k < vecs ? w[c0 + 32 * k] : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int c = c0 + 32 * k;
            if (c < vecs) {
                const uint4 x = live ? h[k] : make_uint4(0, 0, 0, 0);
                if (BF16) reinterpret_cast<uint4 *>(out)[c] = x;
                else split4(x, out + c * 4, (long long)p.N * p.out_ld);
            }
            if (BF16) {
                const uint32_t xp[4] = {h[k].x, h[k].y, h[k].z, h[k].w}, yp[4] = {y[k].x, y[k].y, y[k].z, y[k].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    chain[i] = fmaf(__uint_as_float(xp[i] << 16), __uint_as_float(yp[i] << 16), chain[i]);
                    chain[i] = fmaf(__uint_as_float(xp[i] & 0xffff0000u), __uint_as_float(yp[i] & 0xffff0000u),
                                    chain[i]);
                }
            } else {
                sum.add<BF16>(h[k], y[k]);
            }
        }
    }
    Wide z{(chain[0] + chain[1]) + (chain[2] + chain[3]), 0.f};
    if (BF16) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) z.hi += __shfl_xor_sync(0xffffffffu, z.hi, o);
    } else {
        z = sum.over_warp();
    }
    if (lane == 0) p.target_logp[row] = target < 0 ? 0.f : fmaf(z.hi, p.scale, -p.lse[row]) + z.lo * p.scale;
}

} // namespace

cudaError_t launch_sum_parts(const PartsSum (&r)[2], cudaStream_t s)
{
    const auto blocks = [](const PartsSum &x) { return (int)((x.elems / 4 + 255) / 256); };
    const int b0 = blocks(r[0]), b1 = blocks(r[1]);
    if (b0 + b1 == 0) return cudaSuccess;
    return launch_grid(sum_parts_kernel, dim3((unsigned)(b0 + b1)), 256, 0, s, 1, r[0], r[1], b0);
}

cudaError_t launch_split_f32(const SplitRows &h, const SplitRows &w, cudaStream_t s)
{
    const long long b0 = split_blocks(h, 256), b1 = split_blocks(w, 256);
    return launch_grid(split_f32_kernel, dim3((unsigned)(b0 + b1)), 256, 0, s, 1, h, w, b0);
}

cudaError_t launch_grad_rows(const GradRowsParams &p, bool bf16, cudaStream_t s)
{
    const int threads = kMergeWarps * 32, rows = (p.N + kMergeWarps - 1) / kMergeWarps;
    if (bf16) return launch_grid(grad_rows_kernel<true>, dim3((unsigned)rows), threads, 0, s, 1, p, rows);
    return launch_grid(grad_rows_kernel<false>, dim3((unsigned)(rows + split_blocks(p.table, threads))), threads, 0, s,
                       1, p, rows);
}

cudaError_t launch_logprob_few_merge(const MergeParams &p, bool bf16, cudaStream_t s)
{
    const unsigned grid = (unsigned)p.N;
    auto *kernel = bf16 ? (p.logits ? logprob_few_merge_kernel<true, true> : logprob_few_merge_kernel<true, false>)
                        : (p.logits ? logprob_few_merge_kernel<false, true> : logprob_few_merge_kernel<false, false>);
    return launch_grid(kernel, dim3(grid), kFewThreads, 0, s, 1, p);
}

template <bool BF16, int LIST>
cudaError_t merge(const MergeParams &p, cudaStream_t s)
{
    const unsigned grid = (unsigned)((p.N + kMergeWarps - 1) / kMergeWarps);
    return launch_grid(logprob_merge_kernel<BF16, LIST>, dim3(grid), kMergeWarps * 32, 0, s, 1, p);
}

cudaError_t launch_logprob_merge(const MergeParams &p, bool bf16, cudaStream_t s)
{
    if (bf16) return p.list == 0 ? merge<true, 0>(p, s) : p.list == 12 ? merge<true, 12>(p, s) : merge<true, 20>(p, s);
    return p.list == 0 ? merge<false, 0>(p, s) : p.list == 12 ? merge<false, 12>(p, s) : merge<false, 20>(p, s);
}

} // namespace txl
