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

// a + b exactly as hi + lo (Knuth's two-sum).
__device__ __forceinline__ void two_sum(float &hi, float &lo, float x)
{
    const float s = __fadd_rn(hi, x), bb = __fadd_rn(s, -hi);
    lo += (hi - (s - bb)) + (x - bb);
    hi = s;
}

// h_i . w_j to about 2^-45 of its terms' size, over a warp: products split exactly (a bf16
// product is an fp32 value; an fp32 one is a product and its rounding error by fma), sums
// carried with their errors, four chains a lane.  Where that is no number, the plain sum.
template <bool BF16>
__device__ double dot_exact(const void *h, const void *w, int d, int lane)
{
    float hi[4] = {}, lo[4] = {}, plain = 0.f;
    if (BF16) {
        const uint4 *a = static_cast<const uint4 *>(h), *b = static_cast<const uint4 *>(w);
#pragma unroll 4
        for (int c = lane; c < d / 8; c += 32) {
            const uint4 x = __ldg(a + c), y = __ldg(b + c);
            const uint32_t xp[4] = {x.x, x.y, x.z, x.w}, yp[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float q0 = __fmul_rn(__uint_as_float(xp[i] << 16), __uint_as_float(yp[i] << 16));
                const float q1 = __fmul_rn(__uint_as_float(xp[i] & 0xffff0000u),
                                           __uint_as_float(yp[i] & 0xffff0000u));
                two_sum(hi[i], lo[i], q0);
                two_sum(hi[i], lo[i], q1);
                plain += q0 + q1;
            }
        }
    } else {
        const float4 *a = static_cast<const float4 *>(h), *b = static_cast<const float4 *>(w);
#pragma unroll 4
        for (int c = lane; c < d / 4; c += 32) {
            const float4 x = __ldg(a + c), y = __ldg(b + c);
            const float xp[4] = {x.x, x.y, x.z, x.w}, yp[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float q = __fmul_rn(xp[i], yp[i]);
                two_sum(hi[i], lo[i], q);
                lo[i] += fmaf(xp[i], yp[i], -q);
                plain += q;
            }
        }
    }
#pragma unroll
    for (int i = 1; i < 4; ++i) {
        two_sum(hi[0], lo[0], hi[i]);
        lo[0] += lo[i];
    }
    double z = (double)hi[0] + (double)lo[0];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    if (!isfinite(z)) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) plain += __shfl_xor_sync(0xffffffffu, plain, o);
        z = plain;
    }
    return z;
}

constexpr int kMergeWarps = 4;
constexpr int kLaneLists = kMaxStatSplits / 32;
constexpr float kLn2 = 0.6931471805599453f;

// Softmax statistics of a row from its ranges', over a warp: lane s holds ranges s, s + 32, ...
struct RowSums {
    float m, mu, sum, es, zt;
};

template <int PER>
__device__ __forceinline__ RowSums join_stats(const MergeParams &p, int row, int lane)
{
    constexpr unsigned FULL = 0xffffffffu;
    float4 st[PER];
    RowSums r{-INFINITY, 0.f, 0.f, 0.f, 0.f};
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
        if (st[i].y == 0.f) continue;
        const float d = st[i].x - r.mu, f = exp2f(d);
        r.sum += st[i].y * f;
        r.es += (st[i].z + st[i].y * d) * f;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        r.sum += __shfl_xor_sync(FULL, r.sum, o);
        r.es += __shfl_xor_sync(FULL, r.es, o);
    }
    if (__any_sync(FULL, nan)) r.sum = __int_as_float(0x7fffffff);
    return r;
}

// A logit known more exactly (log2 units) takes its place in the sums: peaked rows, whose sums
// are a few such terms, are as exact as these.
__device__ __forceinline__ void replace_term(float mu, float was, double is, float &ds, float &de)
{
    const float d0 = was - mu, d1 = (float)(is - (double)mu);
    const float e0 = ex2(d0), e1 = exp2f(d1);
    ds = e1 - e0;
    de = e1 * d1 - e0 * d0;
}

// Row outputs from the sums (one thread); returns lse.
__device__ __forceinline__ double row_outputs(const MergeParams &p, int row, const RowSums &r, int target,
                                              double z_target, bool write)
{
    const float l = logf(r.sum);
    const double lse = (double)r.m * 0.6931471805599453 + (double)l;
    if (write) {
        if (p.logp) p.logp[row] = target >= 0 ? (float)(z_target - lse) : 0.f;
        if (p.lse) p.lse[row] = (float)lse;
        if (p.entropy) p.entropy[row] = l - r.es / r.sum * kLn2;
    }
    return lse;
}

// Rows of the statistics kernel: one warp each.  Its ranges' lists are two a lane.
template <bool BF16, int LIST>
__global__ void __launch_bounds__(kMergeWarps * 32) logprob_merge_kernel(const MergeParams p)
{
    constexpr unsigned FULL = 0xffffffffu;
    constexpr int PER = kMaxRowSplits / 32, WANT = LIST > 0 ? LIST : 1;
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
    if (row >= p.N) return;
    const int target = p.targets ? token_at(p.targets, p.index_bytes, row, p.V, p.status) : -1;
    const int esize = BF16 ? 2 : 4;
    const char *h = static_cast<const char *>(p.h) + row * p.h_ld * esize;
    auto logit = [&](int id) {
        return dot_exact<BF16>(h, static_cast<const char *>(p.w) + id * p.w_ld * esize, p.d, lane) *
               (double)p.scale;
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
    double z = (double)my_val * kLn2, z_target = (double)r.zt * kLn2;
    float ds = 0.f, de = 0.f;
    bool listed = false;
    for (int c = 0; c < found; ++c) {
        const int id = __shfl_sync(FULL, my_id, c);
        const double e = logit(id);
        if (lane == c && isfinite(e) && isfinite(my_val)) {
            z = e;
            replace_term(r.mu, my_val, e * 1.4426950408889634, ds, de);
        }
        if (id == target) {
            listed = true;
            z_target = __shfl_sync(FULL, z, c);
        }
    }
    if (target >= 0 && !listed) {
        const double e = logit(target);
        if (isfinite(e) && isfinite(r.zt)) {
            z_target = e;
            if (lane == 31) {   // (found is below 32: this lane has no candidate)
                replace_term(r.mu, r.zt, e * 1.4426950408889634, ds, de);
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        ds += __shfl_xor_sync(FULL, ds, o);
        de += __shfl_xor_sync(FULL, de, o);
    }
    r.sum += ds;
    r.es += de;
    const double lse = row_outputs(p, row, r, target, z_target, lane == 0);
    if (LIST == 0) return;
    int rank = 0;
    for (int c = 0; c < found; ++c) {
        const double oz = __shfl_sync(FULL, z, c);
        const int oid = __shfl_sync(FULL, my_id, c);
        if (oz > z || (oz == z && oid < my_id)) ++rank;
    }
    if (my_id >= 0 && rank < p.top) {
        p.top_ids[(long long)row * p.top + rank] = my_id;
        p.top_logp[(long long)row * p.top + rank] = (float)(z - lse);
    }
    if (lane >= found && lane < p.top) {  // fewer numbers than places
        p.top_ids[(long long)row * p.top + lane] = -1;
        p.top_logp[(long long)row * p.top + lane] = __int_as_float(0x7fffffff);
    }
}

// Rows of the kernel for few states: a block each.  The `want` largest logits lie in the `want`
// groups of four with the largest maxima.  Those are found by a threshold that at least `want`
// threads' own maxima reach (a search over the order's upper bits), then ranked among all that
// reach it; their members' exact logits give the order.
constexpr int kFewThreads = 512;
constexpr int kFewWarps = kFewThreads / 32;
constexpr int kFewCap = 256;                          // groups above the threshold
constexpr int kFewWant = kMaxTop + kSpareTop;
constexpr int kFewLoads = 4;                          // 16-byte loads of a thread in flight

// Order of doubles as integers (their comparisons are slow); 0 stands for no number.
__device__ __forceinline__ unsigned long long wide_key(double z)
{
    z += 0.0;  // (zeros of one sign)
    const long long u = __double_as_longlong(z);
    return z == z ? (unsigned long long)u ^ ((unsigned long long)(u >> 63) | 0x8000000000000000ull) : 0ull;
}

template <bool BF16>
__global__ void __launch_bounds__(kFewThreads) logprob_few_merge_kernel(const MergeParams p)
{
    constexpr unsigned FULL = 0xffffffffu;
    __shared__ unsigned s_key[kFewCap];
    __shared__ int s_at[kFewCap];
    __shared__ int s_count;
    __shared__ unsigned s_best_key[kFewWarps];
    __shared__ int s_best_at[kFewWarps];
    __shared__ unsigned g_key[kFewWant];              // the groups, in order
    __shared__ int g_at[kFewWant];
    __shared__ double s_z[4 * kFewWant + 1];          // members' exact logits, then the target's
    __shared__ unsigned long long s_wide[4 * kFewWant];
    __shared__ RowSums s_sums;
    __shared__ double s_lse;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.x;
    const int target = p.targets ? token_at(p.targets, p.index_bytes, row, p.V, p.status) : -1;
    const int esize = BF16 ? 2 : 4;
    const char *h = static_cast<const char *>(p.h) + row * p.h_ld * esize;
    int groups = 0;                                   // found
    if (p.top > 0) {
        const int n = p.nb * 8, want = min(p.top + kSpareTop, kFewWant);  // (n: of four groups)
        const uint4 *key = reinterpret_cast<const uint4 *>(p.group_key) + (long long)row * n;
        auto scan = [&](auto take) {
            for (int i0 = tid; i0 < n; i0 += kFewThreads * kFewLoads) {
                uint4 k[kFewLoads];
#pragma unroll
                for (int u = 0; u < kFewLoads; ++u) {
                    const int i = i0 + u * kFewThreads;
                    k[u] = i < n ? key[i] : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int u = 0; u < kFewLoads; ++u) take(k[u], (i0 + u * kFewThreads) * 4);
            }
        };
        unsigned mine = 0;
        scan([&](const uint4 &k, int) { mine = max(mine, max(max(k.x, k.y), max(k.z, k.w))); });
        if (tid == 0) s_count = 0;
        unsigned thr = 0;
        for (int bit = 31; bit >= 14; --bit) {
            const unsigned t = thr | 1u << bit;
            if (__syncthreads_count(mine >= t) >= want) thr = t;
        }
        thr = max(thr, 1u);
        if (mine >= thr)
            scan([&](const uint4 &k, int at0) {
                const unsigned ks[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    if (ks[q] >= thr) {
                        const int at = atomicAdd(&s_count, 1);
                        if (at < kFewCap) {
                            s_key[at] = ks[q];
                            s_at[at] = at0 + q;
                        }
                    }
            });
        __syncthreads();
        const int count = s_count;
        if (count <= kFewCap) {
            if (tid < count) {
                int rank = 0;
                const unsigned k = s_key[tid];
                const int at = s_at[tid];
                for (int c = 0; c < count; ++c) rank += s_key[c] > k || (s_key[c] == k && s_at[c] < at);
                if (rank < want) {
                    g_key[rank] = k;
                    g_at[rank] = at;
                }
            }
            __syncthreads();
            groups = min(count, want);
        } else {
            // very many equal maxima: one after the other, the lowest group of equal ones first
            const unsigned *one = reinterpret_cast<const unsigned *>(key);
            unsigned last_key = 0xffffffffu;
            int last_at = -1;
            for (int c = 0; c < want; ++c) {
                unsigned bk = 0;
                int ba = 0x7fffffff;
                for (int i = tid; i < n * 4; i += kFewThreads) {
                    const unsigned k = one[i];
                    const bool left = k < last_key || (k == last_key && i > last_at);
                    if (k && left && k > bk) {
                        bk = k;
                        ba = i;
                    }
                }
                unsigned top = __reduce_max_sync(FULL, bk);
                int at = (int)__reduce_min_sync(FULL, bk == top ? (unsigned)ba : 0x7fffffffu);
                if (lane == 0) {
                    s_best_key[warp] = top;
                    s_best_at[warp] = at;
                }
                __syncthreads();
                bk = lane < kFewWarps ? s_best_key[lane] : 0;
                ba = lane < kFewWarps ? s_best_at[lane] : 0x7fffffff;
                top = __reduce_max_sync(FULL, bk);
                at = (int)__reduce_min_sync(FULL, bk == top ? (unsigned)ba : 0x7fffffffu);
                __syncthreads();
                if (!top) break;
                if (tid == 0) {
                    g_key[c] = top;
                    g_at[c] = at;
                }
                last_key = top;
                last_at = at;
                groups = c + 1;
            }
            __syncthreads();
        }
    }
    // the ranges' sums (last warp); exact logits, the target's first
    if (warp == kFewWarps - 1) {
        const RowSums r = join_stats<kLaneLists>(p, row, lane);
        if (lane == 0) s_sums = r;
    }
    const int jobs = 4 * groups;
    for (int c = warp; c <= jobs; c += kFewWarps) {
        const int id = c == 0 ? target : g_at[(c - 1) >> 2] * 4 + ((c - 1) & 3);
        double e = __longlong_as_double(0x7ff8000000000000LL);  // no such token
        if (id >= 0 && id < p.V)
            e = dot_exact<BF16>(h, static_cast<const char *>(p.w) + id * p.w_ld * esize, p.d, lane) *
                (double)p.scale;
        if (lane == 0) {
            s_z[c == 0 ? 4 * kFewWant : c - 1] = e;
            if (c > 0) s_wide[c - 1] = wide_key(e);
        }
    }
    __syncthreads();
    // places in the order, while the first warp finishes the sums
    int rank = 0;
    const int c = tid - 32;
    const bool on = c >= 0 && c < jobs && s_wide[c] != 0;
    if (on) {
        const unsigned long long k = s_wide[c];
        const int id = g_at[c >> 2] * 4 + (c & 3);
        for (int o = 0; o < jobs; ++o) {
            const unsigned long long ok = s_wide[o];
            rank += ok > k || (ok == k && g_at[o >> 2] * 4 + (o & 3) < id);
        }
    }
    const int found = __syncthreads_count(on);
    if (warp == 0) {
        RowSums r = s_sums;
        if (target >= 0) r.zt = p.target_z[row];
        double z_target = (double)r.zt * kLn2;
        float ds = 0.f, de = 0.f;
        bool replaced = false;
        if (lane < groups) {
            // the group's maximum was its largest member's logit
            int at = 0;
            for (int i = 1; i < 4; ++i)
                if (s_wide[4 * lane + i] > s_wide[4 * lane + at]) at = i;
            const double best = s_z[4 * lane + at];
            const float was = key_value(g_key[lane]);
            if (isfinite(best) && isfinite(was)) replace_term(r.mu, was, best * 1.4426950408889634, ds, de);
            replaced = g_at[lane] * 4 + at == target;
        }
        const bool in_sums = __any_sync(FULL, replaced);
        if (target >= 0) {
            const double e = s_z[4 * kFewWant];
            if (isfinite(e) && isfinite(r.zt)) {
                z_target = e;
                if (!in_sums && lane == 31) replace_term(r.mu, r.zt, e * 1.4426950408889634, ds, de);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            ds += __shfl_xor_sync(FULL, ds, o);
            de += __shfl_xor_sync(FULL, de, o);
        }
        r.sum += ds;
        r.es += de;
        const double lse = row_outputs(p, row, r, target, z_target, lane == 0);
        if (lane == 0) s_lse = lse;
    }
    __syncthreads();
    if (on && rank < p.top) {
        p.top_ids[(long long)row * p.top + rank] = g_at[c >> 2] * 4 + (c & 3);
        p.top_logp[(long long)row * p.top + rank] = (float)(s_z[c] - s_lse);
    }
    if (tid >= found && tid < p.top) {  // fewer numbers than places
        p.top_ids[(long long)row * p.top + tid] = -1;
        p.top_logp[(long long)row * p.top + tid] = __int_as_float(0x7fffffff);
    }
}

// ---------------------------------------------------------------------------
// small passes
// ---------------------------------------------------------------------------

template <bool BF16>
__global__ void __launch_bounds__(256) sum_parts_kernel(const float4 *part, int parts, long long vecs,
                                                        void *out)
{
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= vecs) return;
    float4 a = __ldcs(part + i);
    for (int s = 1; s < parts; ++s) {
        const float4 b = __ldcs(part + s * vecs + i);
        a.x += b.x;
        a.y += b.y;
        a.z += b.z;
        a.w += b.w;
    }
    if (BF16)
        reinterpret_cast<uint2 *>(out)[i] = make_uint2(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w));
    else
        reinterpret_cast<float4 *>(out)[i] = a;
}

// x = t0 + t1 + t2, each the bf16 nearest to what is left (exact but for what falls below
// bf16's range).  An infinite or NaN value is its first term; a finite one that rounds to
// infinity is cut instead.  Eight values a thread.
__global__ void __launch_bounds__(256) split_f32_kernel(const float *x, long long ld, int rows, int vecs,
                                                        __nv_bfloat16 *planes)
{
    const long long total = (long long)rows * vecs;
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= total) return;
    const int r = (int)(i / vecs), c = (int)(i - (long long)r * vecs);
    const float4 *src = reinterpret_cast<const float4 *>(x + r * ld + c * 8);
    const float4 lo = __ldcs(src), hi = __ldcs(src + 1);
    float v[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
#pragma unroll
    for (int t = 0; t < kMaxPieces; ++t) {
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            __nv_bfloat16 n = __float2bfloat16_rn(v[k]);
            if (__hisinf(n) && !isinf(v[k])) n = __float2bfloat16_rz(v[k]);
            v[k] = isfinite(v[k]) ? v[k] - __bfloat162float(n) : 0.f;
            const uint32_t bits = __bfloat16_as_ushort(n);
            o[k / 2] = k & 1 ? o[k / 2] | bits << 16 : bits;
        }
        reinterpret_cast<uint4 *>(planes)[t * total + i] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// One warp per row: a copy of h with zeros in rows that have no part in the gradient (whatever
// those hold), and the log probability of the row's target from its logit's products carried
// beyond fp32: G's one large element is the difference of 1 and that probability.
template <bool BF16>
__global__ void __launch_bounds__(kMergeWarps * 32) grad_rows_kernel(const GradRowsParams p)
{
    const int lane = threadIdx.x & 31;
    const int row = blockIdx.x * kMergeWarps + (threadIdx.x >> 5);
    if (row >= p.N) return;
    constexpr int ESIZE = BF16 ? 2 : 4;
    const int target = p.targets ? token_at(p.targets, p.index_bytes, row, p.V, p.status) : -1;
    const bool live = target >= 0 || (p.dentropy && p.dentropy[row] != 0.f);
    const int vecs = p.d * ESIZE / 16;
    const uint4 *src = reinterpret_cast<const uint4 *>(static_cast<const char *>(p.h) + row * p.h_ld * ESIZE);
    uint4 *dst = static_cast<uint4 *>(p.out) + (long long)row * vecs;
    for (int c = lane; c < vecs; c += 32) dst[c] = live ? __ldg(src + c) : make_uint4(0, 0, 0, 0);
    if (target < 0) {
        if (lane == 0) p.target_logp[row] = 0.f;
        return;
    }
    const double z = dot_exact<BF16>(src, static_cast<const char *>(p.w) + target * p.w_ld * ESIZE, p.d, lane) *
                     (double)p.scale;
    if (lane == 0) p.target_logp[row] = (float)(z - (double)p.lse[row]);
}

} // namespace

cudaError_t launch_sum_parts(const float *part, int parts, long long elems, void *out, bool bf16,
                             cudaStream_t s)
{
    const long long vecs = elems / 4;
    const unsigned grid = (unsigned)((vecs + 255) / 256);
    if (bf16) sum_parts_kernel<true><<<grid, 256, 0, s>>>(reinterpret_cast<const float4 *>(part), parts, vecs, out);
    else sum_parts_kernel<false><<<grid, 256, 0, s>>>(reinterpret_cast<const float4 *>(part), parts, vecs, out);
    return cudaGetLastError();
}

cudaError_t launch_split_f32(const float *x, long long ld, int rows, int d, __nv_bfloat16 *planes,
                             cudaStream_t s)
{
    const long long vecs = (long long)rows * (d / 8);
    split_f32_kernel<<<(unsigned)((vecs + 255) / 256), 256, 0, s>>>(x, ld, rows, d / 8, planes);
    return cudaGetLastError();
}

cudaError_t launch_grad_rows(const GradRowsParams &p, bool bf16, cudaStream_t s)
{
    const unsigned grid = (unsigned)((p.N + kMergeWarps - 1) / kMergeWarps);
    if (bf16) grad_rows_kernel<true><<<grid, kMergeWarps * 32, 0, s>>>(p);
    else grad_rows_kernel<false><<<grid, kMergeWarps * 32, 0, s>>>(p);
    return cudaGetLastError();
}

cudaError_t launch_logprob_few_merge(const MergeParams &p, bool bf16, cudaStream_t s)
{
    if (bf16) logprob_few_merge_kernel<true><<<(unsigned)p.N, kFewThreads, 0, s>>>(p);
    else logprob_few_merge_kernel<false><<<(unsigned)p.N, kFewThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <bool BF16, int LIST>
void merge(const MergeParams &p, cudaStream_t s)
{
    const unsigned grid = (unsigned)((p.N + kMergeWarps - 1) / kMergeWarps);
    logprob_merge_kernel<BF16, LIST><<<grid, kMergeWarps * 32, 0, s>>>(p);
}

cudaError_t launch_logprob_merge(const MergeParams &p, bool bf16, cudaStream_t s)
{
    if (bf16) {
        if (p.list == 0) merge<true, 0>(p, s);
        else if (p.list == 12) merge<true, 12>(p, s);
        else merge<true, 20>(p, s);
    } else {
        if (p.list == 0) merge<false, 0>(p, s);
        else if (p.list == 12) merge<false, 12>(p, s);
        else merge<false, 20>(p, s);
    }
    return cudaGetLastError();
}

} // namespace txl
