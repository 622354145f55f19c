// Log probabilities of tokens and their gradient.
//
//   z_ij   = scale * h_i . w_j                        (w: the tied table, V rows)
//   lse_i  = log sum_j exp z_ij,  logp_i = z_i,t(i) - lse_i
//   H_i    = lse_i - sum_j p_ij z_ij,  the largest few z_ij
//   G_ij   = g_i (1[j = t(i)] - p_ij) - e_i p_ij (log p_ij + H_i)
//   dh_i   = scale sum_j G_ij w_j,  dW_j = scale sum_i G_ij h_i
//
// One GEMM kernel on tcgen05 (bf16 operands, fp32 accumulators in TMEM), in
// three modes that differ in their operands' layout and in what becomes of a tile:
//   kStats   h W^T; a block keeps 128 rows and walks over a range of the
//            vocabulary, each row's running maximum, sum, weighted sum, target
//            logit and largest logits in the registers of the thread that owns it:
//            the N x V logits are never written.  launch_logprob_merge joins the
//            ranges.
//   kGrad    h W^T again; a tile becomes G, as bf16 terms in the workspace
//   kProducts  dh = G W and dW = G^T h, the tiles of both in one launch
// Where G is a bf16 pair, a stage holds both terms beside one tile of the other operand, or (few rows) the
// pair's blocks take one term each in dh, and dW the terms in steps of their own: less room a stage, and half
// the MMAs of dh (the gradient of 64 x 32000 x 1024 60 us, 70 with both terms in each stage).
// fp32 operands are three bf16 terms each (their leading 24 bits); a product of two
// such operands is the six products of terms whose weight is above 2^-24.  A step of them loads
// each term once, three stages for six products (where every product had its own two tiles, the
// gradient of 333 x 5003 x 520 took 73 us, so 61).
#include <type_traits>

#include "vocab.h"
#include "ptx.cuh"

namespace txl {
namespace {

using namespace ptx;

constexpr int BM = 128, BK = 64, MAX_BN = 256;
constexpr int A_BYTES = BM * BK * 2;
constexpr int SLAB = BK * 128;                    // 64 MN elements x BK rows
constexpr uint32_t TM_COLS = 512;                 // two accumulators of 256 columns,
constexpr int REST = 128;                         // ... or of 128 and, behind them, the small products
constexpr int OUT_BYTES = 32 * 128;               // a warp's rows of a stored tile
constexpr int kEpiWarps = 8;                      // two halves of a tile's columns, four warps each
constexpr int kThreads = (4 + kEpiWarps) * 32;

// A pair of blocks multiplies 256 x bn tiles, each block holding half of A's rows and of B's
// columns (a block alone with 128 x bn tiles reads half as much again from L2 for the same work: the
// statistics of 2048 x 131072 306 us, with pairs 287).
constexpr int B_BYTES = MAX_BN / 2 * BK * 2;
constexpr int RING = 192 * 1024, MAX_NS = RING / (A_BYTES + B_BYTES / 2);
constexpr int OFF_OUT = RING;
constexpr int OFF_BAR = OFF_OUT + kEpiWarps * OUT_BYTES;
constexpr int OFF_MISC = OFF_BAR + (2 * MAX_NS + 4) * 8;
constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;  // (slack for the manual alignment)

static_assert(A_BYTES % 1024 == 0 && B_BYTES % 2048 == 0, "swizzled tiles need 1024-byte alignment");
static_assert(SMEM_BYTES <= 232448, "shared memory budget exceeded");

enum Mode { kStats, kGrad, kProducts };

// Tile `t` of the `n_tiles` that item `item` consists of.
struct Tile {
    int m, n, kb_lo, kb_hi;
};

// Item `item` of a launch: of the first of its products, or (kProducts) the second, whose items
// follow.
template <Mode MODE>
struct Item {
    int side, at;

    __device__ __forceinline__ Item(const GemmLaunch &g, int item)
    {
        side = MODE == kProducts && item >= g.p[0].n_items ? 1 : 0;
        at = side ? item - g.p[0].n_items : item;
    }
    // Tiles of it.
    __device__ __forceinline__ int tiles(const GemmParams &p) const
    {
        if (MODE != kStats) return 1;
        const int s = at / p.mb;
        return (int)((long long)(s + 1) * p.nb / p.splits) - (int)((long long)s * p.nb / p.splits);
    }
    __device__ __forceinline__ Tile tile(const GemmParams &p, int t) const
    {
        if (MODE == kStats) {
            const int s = at / p.mb;
            return {at - s * p.mb, (int)((long long)s * p.nb / p.splits) + t, 0, p.kb};
        }
        if (MODE == kGrad) {  // (neighbouring blocks share a tile of w)
            const int n = at / p.mb;
            return {at - n * p.mb, n, 0, p.kb};
        }
        const int per = p.mb * p.nb, s = at / per, mn = at - s * per;
        return {mn / p.nb, mn % p.nb, (int)((long long)s * p.kb / p.splits),
                (int)((long long)(s + 1) * p.kb / p.splits)};
    }
};

// The items of one pair in turn: every pairs-th of the first product, then of the second; pairs that
// have one less of the first take `early` of the second before all share the rest.
template <Mode MODE>
struct Turn {
    int pair, pairs, n0, n1, own0, fewer, early;

    __device__ __forceinline__ Turn(const GemmLaunch &g, int pair_, int pairs_) : pair(pair_), pairs(pairs_)
    {
        n0 = g.p[0].n_items;
        n1 = MODE == kProducts ? g.p[1].n_items : 0;
        own0 = (n0 - pair + pairs - 1) / pairs;  // (n0 >= 0 and pair < pairs: not negative)
        fewer = pairs - n0 % pairs;
        early = MODE == kProducts && pair >= n0 % pairs ? g.early : 0;
    }
    // Item k of the pair, or -1 behind its last.
    __device__ __forceinline__ int item(const GemmLaunch &g, int k) const
    {
        if (k < own0) return pair + k * pairs;
        if (MODE != kProducts) return -1;
        k -= own0;
        const int at = k < early ? pair - (pairs - fewer) + k * fewer : g.early * fewer + pair + (k - early) * pairs;
        return at < n1 ? n0 + at : -1;
    }
};

// What a thread keeps of its row while it walks over the vocabulary (log2 units).
template <int LIST>
struct RowStats {
    float m, s, lo, es, zt;   // the sum is s + lo, and the maximum's own 1
    float val[LIST > 0 ? LIST : 1];
    int id[LIST > 0 ? LIST : 1];

    __device__ __forceinline__ void clear()
    {
        m = -INFINITY;
        s = lo = es = zt = 0.f;
#pragma unroll
        for (int j = 0; j < LIST; ++j) {
            val[j] = __int_as_float(0x7fffffff);  // NaN: an empty place, which any number takes
            id[j] = -1;
        }
    }
    // Places in descending order; an equal value that comes later goes behind.
    __device__ __forceinline__ void insert(float v, int j0)
    {
#pragma unroll
        for (int j = LIST - 1; j > 0; --j) {
            const bool above = !(v <= val[j - 1]), here = !(v <= val[j]);
            val[j] = above ? val[j - 1] : here ? v : val[j];
            id[j] = above ? id[j - 1] : here ? j0 : id[j];
        }
        if (LIST > 0 && !(v <= val[0])) {
            val[0] = v;
            id[0] = j0;
        }
    }
};

__device__ __forceinline__ float pick(const float (&t)[32], int i)
{
    float a[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) a[k] = (i & 16) ? t[k + 16] : t[k];
#pragma unroll
    for (int k = 0; k < 8; ++k) a[k] = (i & 8) ? a[k + 8] : a[k];
#pragma unroll
    for (int k = 0; k < 4; ++k) a[k] = (i & 4) ? a[k + 4] : a[k];
#pragma unroll
    for (int k = 0; k < 2; ++k) a[k] = (i & 2) ? a[k + 2] : a[k];
    return (i & 1) ? a[1] : a[0];
}

// 32 logits of a row, columns col0 .. col0 + cnt - 1 of the vocabulary (t: log2 units, -inf
// behind cnt).
template <int LIST>
__device__ __forceinline__ void take(RowStats<LIST> &r, const float (&t)[32], int col0, int cnt,
                                     int target)
{
    float mx = t[0];
#pragma unroll
    for (int i = 1; i < 32; ++i) mx = fmaxf(mx, t[i]);
    const float m_new = fmaxf(r.m, mx);
    const float mu = m_new == -INFINITY ? 0.f : m_new;
    const bool up = m_new > r.m;
    bool far = false;   // a new maximum beside which the others are small
    if (up) {
        // (bounded: a finite maximum of 1e38 below, times a sum, would be infinite, and times 0 NaN)
        const float diff = fmaxf(r.m - mu, -1e30f);
        const float f = ex2(diff);
        if (r.m > -INFINITY) {  // (the old maximum's 1 is one of the others now)
            two_sum(r.s, r.lo, 1.f);
            r.es = (r.es + r.s * diff) * f;
        }
        r.s *= f;
        r.lo *= f;
        r.m = m_new;
        far = !(f > 0.125f);
    }
    // sums of the 32, as a tree; OWN: without the new maximum's 1 (equal ones beside it are added again).  Else
    // it is taken from the whole: the others are an eighth at least, and lose 5 roundings of 2^-24 of 1.
    // (2048 x 131072 x 1024: 351 us with the first for every new maximum, 346 so.)
    float ce[2] = {0.f, 0.f}, more = 0.f;
    auto sum = [&](auto own) {
        float cs[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            float e[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = t[8 * q + i] - mu;
                e[i] = ex2(d);
                // (a logit of -inf has weight zero)
                ce[i & 1] = fmaf(e[i], fmaxf(d, -1e30f), ce[i & 1]);
                if constexpr (decltype(own)::value) {
                    const float its = far && t[8 * q + i] == mx ? 1.f : 0.f;
                    e[i] -= its;
                    more += its;
                }
            }
            cs[q] = ((e[0] + e[1]) + (e[2] + e[3])) + ((e[4] + e[5]) + (e[6] + e[7]));
        }
        two_sum(r.s, r.lo, (cs[0] + cs[1]) + (cs[2] + cs[3]));
    };
    if (__any_sync(0xffffffffu, far)) sum(std::true_type{});
    else sum(std::false_type{});
    if (up && more != 1.f) two_sum(r.s, r.lo, more - 1.f);
    r.es += ce[0] + ce[1];
    const int at = target - col0;
    if (__any_sync(0xffffffffu, (unsigned)at < (unsigned)cnt)) {
        const float v = pick(t, at & 31);
        if ((unsigned)at < (unsigned)cnt) r.zt = v;
    }
    if (LIST > 0) {
        const float thr = r.val[LIST - 1];
        if (__any_sync(0xffffffffu, !(mx <= thr))) {
            unsigned cand = 0;
#pragma unroll
            for (int i = 0; i < 32; ++i)
                cand |= (!(t[i] <= thr) && t[i] == t[i]) ? 1u << i : 0u;
            if (cnt < 32) cand &= (1u << cnt) - 1;
            while (__any_sync(0xffffffffu, cand != 0)) {
                const int i = cand ? __ffs(cand) - 1 : 0;
                const float v = pick(t, i);
                if (cand && !(v <= r.val[LIST - 1])) r.insert(v, col0 + i);
                cand &= cand - 1;
            }
        }
    }
}

// THREE: three terms of both operands.
template <Mode MODE, int LIST, bool THREE>
__global__ void __launch_bounds__(kThreads, 1)
    vocab_gemm_kernel(const __grid_constant__ GemmLaunch g)
{
    // (products have no list: LIST 1 is their form for few rows, with GemmParams' stacked and twice)
    constexpr bool FEW = MODE == kProducts && LIST > 0;
    // (dW's A operand, G^T, is MN-major; both products' B operand is)
    constexpr bool B_MN = MODE == kProducts;
    // stages of the ring: A's rows (two terms of them, if a product has them), then B's columns
    const bool dual = MODE == kProducts && !THREE && (g.p[0].terms == 2 || g.p[1].terms == 2);
    const int off_b = dual ? 2 * A_BYTES : A_BYTES;
    const int stage = off_b + (THREE ? B_BYTES / 2 : B_BYTES), ns = RING / stage;
    unsigned int *status = g.p[0].status;
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)cluster_rank();
    const Turn<MODE> turn(g, blockIdx.x / 2, gridDim.x / 2);

    // full (counted on block 0), empty, accumulators full and empty (block 0)
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + OFF_BAR);
    uint64_t *empty = full + MAX_NS;
    uint64_t *acc_full = empty + MAX_NS;
    uint64_t *acc_empty = acc_full + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + OFF_MISC);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + OFF_MISC + 4);
    if (threadIdx.x == 0) {
        for (int s = 0; s < ns; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, 1);
        }
        for (int s = 0; s < 2; ++s) {
            mbar_init(acc_full + s, 1);
            mbar_init(acc_empty + s, kEpiWarps * 2);  // (the epilogue's warps)
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 2) {
        tmem_alloc_pair(tmem_slot, TM_COLS);
        tmem_relinquish_pair();
        tc_fence_before_sync();
    }
    __syncthreads();
    cluster_sync_all();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const uint64_t wait_ns = g.p[0].wait_ns;
    chain_wait();
    chain_go();

    if (warp == 0) {
        // ===================== TMA producer =====================================
        if (lane == 0) {
            const uint32_t full0 = cluster_addr(full, 0);
            for (int i = 0; i < (MODE == kProducts ? 2 : 1); ++i) {
                if (g.p[i].n_items == 0) continue;  // (a gradient that is not wanted has no maps)
                prefetch_tensormap(&g.maps[i].a);
                prefetch_tensormap(&g.maps[i].b);
            }
            bool ok = true;
            int it = 0, s = 0;  // stages filled; the next one
            uint32_t phase = 1;
            for (int k = 0, item; ok && (item = turn.item(g, k)) >= 0; ++k) {
                const Item<MODE> i(g, item);
                const GemmParams &p = g.p[i.side];
                // (in registers: the loop below issues a step's copies in a few hundred cycles, and reads
                // of parameters would be repeated after every one)
                const CUtensorMap *tm_a = &g.maps[i.side].a, *tm_b = &g.maps[i.side].b;
                const int bn = p.bn, own_bn = bn / 2;  // columns of B in this block
                const int b_row0 = p.b_row0;
                const bool two = !THREE && p.terms == 2;
                const bool a_mn = MODE == kProducts && i.side, stacked = FEW && p.stacked;
                const int twice = FEW ? p.twice : 0;
                // (whole boxes in the products of many rows: the copies' rate is their bound, and what this would
                // ask of it takes 5 us of 166 there)
                constexpr bool WHOLE = MODE == kProducts && !FEW;
                const uint32_t a_tx = (two ? 2 : 1) * (WHOLE || a_mn ? A_BYTES : p.a_rows * BK * 2), b_tx = own_bn * BK * 2;
                const int M = p.M;
                const int nt = i.tiles(p);
                for (int t = 0; t < nt && ok; ++t) {
                    const Tile w = i.tile(p, t);
                    const int m0 = stacked ? 0 : (w.m * 2 + rank) * BM, n0 = w.n * bn + rank * own_bn;
                    // (rows behind the last are not loaded: what they multiply is not stored)
                    const bool load_a = WHOLE || m0 < M;
                    const uint32_t stage_tx = (WHOLE || stacked || (w.m * 2 + 1) * BM < M ? 2 : 1) * a_tx + 2 * b_tx;
                    const int plane0 = stacked ? rank : 0;
                    for (int k = w.kb_lo << twice; k < w.kb_hi << twice && ok; ++k) {
                        const int kb = k >> twice, plane = plane0 + (k & twice);
                        for (int term = 0; term < (THREE ? 3 : 1); ++term) {
                            if (!(ok = mbar_wait(empty + s, phase, abort_flag, wait_ns))) break;
                            uint8_t *st = smem + s * stage;
                            if (rank == 0) mbar_arrive_expect_tx(full + s, stage_tx);
                            const uint32_t bar = full0 + s * 8;
                            for (int t = 0; t < (MODE == kProducts && two ? 2 : 1) && load_a; ++t) {
                                if (a_mn) {
#pragma unroll
                                    for (int x = 0; x < BM / 64; ++x)
                                        tma_load_3d_pair(st + t * A_BYTES + x * SLAB, tm_a, bar, m0 + x * 64, kb * BK,
                                                         plane + term + t);
                                } else {
                                    tma_load_3d_pair(st + t * A_BYTES, tm_a, bar, kb * BK, m0, plane + term + t);
                                }
                            }
                            if (B_MN) {
#pragma unroll
                                for (int x = 0; x < MAX_BN / 2 / 64; ++x)
                                    if (x * 64 < own_bn)
                                        tma_load_3d_pair(st + off_b + x * SLAB, tm_b, bar, n0 + x * 64, b_row0 + kb * BK, term);
                            } else {
                                tma_load_3d_pair(st + off_b, tm_b, bar, kb * BK, b_row0 + n0, term);
                            }
                            ++it;
                            if (++s == ns) {
                                s = 0;
                                phase ^= 1;
                            }
                        }
                    }
                }
            }
            if (!ok) {
                atomicOr(status, TXL_STATUS_TIMEOUT);
                *abort_flag = 1;
                // copies in flight land before the block ends: counted on block 0's barriers, which
                // the other block gives a millisecond
                const int zero = 0;
                if (rank == 0) {
                    for (int i = max(0, it - ns); i < it; ++i)
                        mbar_wait(full + i % ns, (i / ns) & 1, &zero, wait_ns);
                } else {
                    const uint64_t t0 = globaltimer_ns();
                    while (globaltimer_ns() - t0 < 1000000ull) {
                    }
                }
            }
        }
    } else if (warp == 1) {
        // ===================== MMA issuer (block 0) ==============================
        const uint32_t a0 = smem_u32(smem), b0 = smem_u32(smem + off_b);
        const uint64_t dB = B_MN ? sdesc_sw128_mn(b0, SLAB) : sdesc_sw128(b0);
        constexpr int STEP_B = B_MN ? 16 * 128 / 16 : 2;
        auto elect = []() -> bool {
            uint32_t el;
            asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}"
                         : "=r"(el));
            return el != 0;
        };
        bool ok = true;
        int s = 0, tile = 0;
        uint32_t phase = 0;
        for (int turns = 0, item; ok && rank == 0 && (item = turn.item(g, turns)) >= 0; ++turns) {
            const Item<MODE> i(g, item);
            const GemmParams &p = g.p[i.side];
            const bool a_mn = MODE == kProducts && i.side;
            const uint32_t ID = idesc_bf16_f32(2 * BM, p.bn, B_MN) | (a_mn ? 1u << 15 : 0u);
            const uint64_t dA = a_mn ? sdesc_sw128_mn(a0, SLAB) : sdesc_sw128(a0);
            const int step_a = a_mn ? 16 * 128 / 16 : 2;
            const bool two = MODE == kProducts && !THREE && p.terms == 2;
            const int nt = i.tiles(p);
            for (int t = 0; t < nt && ok; ++t) {
                const Tile w = i.tile(p, t);
                const int steps = (w.kb_hi - w.kb_lo) << (FEW ? p.twice : 0);
                const int buf = tile & 1;
                ok = __all_sync(0xffffffffu, mbar_wait(acc_empty + buf, ((tile >> 1) & 1) ^ 1, abort_flag, wait_ns));
                if (!ok) break;
                tc_fence_after_sync();
                const uint32_t acc = tmem + buf * MAX_BN;
                for (int k = 0; k < steps; ++k) {
                    ok = __all_sync(0xffffffffu, mbar_wait(full + s, phase, abort_flag, wait_ns));
                    if (!ok) break;
                    tc_fence_after_sync();
                    const uint64_t off = (uint64_t)((s * stage) >> 4);
                    if (THREE) {
                        // terms 0, 1, 2 of both in three stages: their products of weight 1 in one
                        // accumulator, those of weight 2^-8 and 2^-16 in another, whose cut
                        // additions do not matter
                        const int first = s;
                        auto product = [&](uint32_t to, uint64_t x, uint64_t y, bool add) {
#pragma unroll
                            for (int kk = 0; kk < BK / 16; ++kk)
                                mma_bf16_ss_pair(to, dA + x + kk * step_a, dB + y + kk * STEP_B, ID,
                                                 add || kk > 0 ? 1u : 0u);
                        };
                        if (elect()) product(acc, off, off, k > 0);
                        __syncwarp();
                        for (int term = 1; term < 3; ++term) {
                            if (++s == ns) {
                                s = 0;
                                phase ^= 1;
                            }
                            ok = __all_sync(0xffffffffu, mbar_wait(full + s, phase, abort_flag, wait_ns));
                            if (!ok) break;
                            tc_fence_after_sync();
                            const uint64_t at = (uint64_t)((s * stage) >> 4);
                            if (elect()) {
                                product(acc + REST, at, off, k > 0 || term > 1);
                                product(acc + REST, off, at, true);
                                if (term == 1) product(acc + REST, at, at, true);
                                mma_commit_pair(empty + s);
                                if (term == 2) mma_commit_pair(empty + first);
                            }
                            __syncwarp();
                        }
                        if (!ok) break;
                    } else if (elect()) {
#pragma unroll
                        for (int kk = 0; kk < BK / 16; ++kk)
                            mma_bf16_ss_pair(acc, dA + off + kk * step_a, dB + off + kk * STEP_B, ID,
                                             k > 0 || kk > 0 ? 1u : 0u);
                        if (two)
#pragma unroll
                            for (int kk = 0; kk < BK / 16; ++kk)
                                mma_bf16_ss_pair(acc, dA + off + (A_BYTES >> 4) + kk * step_a, dB + off + kk * STEP_B,
                                                 ID, 1u);
                        mma_commit_pair(empty + s);
                    }
                    __syncwarp();
                    if (++s == ns) {
                        s = 0;
                        phase ^= 1;
                    }
                }
                if (!ok) break;
                if (elect()) mma_commit_pair(acc_full + buf);
                __syncwarp();
                ++tile;
            }
        }
        if (!ok) {
            // let what was issued drain before the memory is freed
            if (lane == 0) {
                atomicOr(status, TXL_STATUS_TIMEOUT);
                *abort_flag = 1;
            }
            if (elect()) mma_commit_pair(acc_full + (tile & 1));
            __syncwarp();
            const int zero = 0;
            mbar_wait(acc_full + (tile & 1), (tile >> 1) & 1, &zero, wait_ns);
        }
    } else if (warp >= 4) {
        // ===================== epilogue: thread = row, half of the columns =======
        const int wq = warp & 3, half = (warp - 4) >> 2;
        const int row = wq * 32 + lane;
        const uint32_t tq = tmem + ((uint32_t)(wq * 32) << 16);
        uint8_t *out = smem + OFF_OUT + (warp - 4) * OUT_BYTES;
        constexpr float kLog2e = 1.4426950408889634f;
        constexpr float kNoWeight = -1e3f;  // log probabilities below have p = 0, which a gradient times them must not undo
        const float zscale = g.p[0].scale * uncut_scale(g.p[0].kb * (BK / 16)), c2 = zscale * kLog2e;
        // 128 bytes of each of the warp's rows, turned by the swizzle, then one store.  Each warp for
        // itself: with four that met at barriers around one store of 128 rows the products of
        // 64 x 32000 x 1024 took 45.1 us, so 39.9; from 2048 rows on both take the same.
        const CUtensorMap *tm_out = &g.maps[0].out;
        auto store = [&](const uint4 (&v)[8], int c0, int m0, int plane) {
            if (lane == 0) bulk_wait_read();
            __syncwarp();
#pragma unroll
            for (int q = 0; q < 8; ++q) *reinterpret_cast<uint4 *>(out + lane * 128 + ((q ^ (lane & 7)) << 4)) = v[q];
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                tma_store_3d(tm_out, out, c0, m0 + wq * 32, plane);
                bulk_commit();
            }
        };
        auto pack = [](const float (&v)[32], uint4 *o) {
#pragma unroll
            for (int q = 0; q < 4; ++q)
                o[q] = make_uint4(pack_bf16x2(v[8 * q], v[8 * q + 1]), pack_bf16x2(v[8 * q + 2], v[8 * q + 3]),
                                  pack_bf16x2(v[8 * q + 4], v[8 * q + 5]), pack_bf16x2(v[8 * q + 6], v[8 * q + 7]));
        };
        bool ok = true;
        int tile = 0;
        for (int k = 0, item; ok && (item = turn.item(g, k)) >= 0; ++k) {
            const Item<MODE> it(g, item);
            const GemmParams &p = g.p[it.side];
            tm_out = &g.maps[it.side].out;
            const int nt = it.tiles(p);
            RowStats<LIST> r;
            int target = -1;
            float g1 = 0.f, ge = 0.f, lse = 0.f, ent = 0.f, lpt = 0.f;
            if (MODE == kStats || MODE == kGrad) {
                const int m = (it.tile(p, 0).m * 2 + rank) * BM + row;
                if (m < p.M && p.targets) target = token_at(p.targets, p.index_bytes, m, p.V, p.status);
                // (rows without a part: zeros all through, their states have been cleared)
                if (MODE == kGrad && m < p.M && (target >= 0 || (p.dentropy && p.dentropy[m] != 0.f))) {
                    if (target >= 0) {
                        g1 = p.dlogp[m] * p.scale;
                        lpt = p.target_logp[m];
                    }
                    if (p.dentropy) {
                        ge = p.dentropy[m] * p.scale;
                        ent = p.entropy[m];
                    }
                    lse = p.lse[m];
                }
                if (MODE == kStats) r.clear();
            }
            for (int t = 0; t < nt && ok; ++t, ++tile) {
                const Tile w = it.tile(p, t);
                const int buf = tile & 1;
                ok = __all_sync(0xffffffffu, mbar_wait(acc_full + buf, (tile >> 1) & 1, abort_flag, wait_ns)) &&
                     !*abort_flag;
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after_sync();
                const int m0 = FEW && p.stacked ? 0 : (w.m * 2 + rank) * BM, n0 = w.n * p.bn;
                // (a warp whose rows lie behind the last has nothing to do)
                const int c_lo = half * (p.bn / 2),
                          c_hi = m0 + wq * 32 < p.M ? min((half + 1) * (p.bn / 2), p.N - n0) : 0;
                const bool empty_part = w.kb_lo == w.kb_hi;  // (nothing was accumulated)
                auto sums = [&](uint32_t (&raw)[32], int c) {
                    tmem_ld32(tq + buf * MAX_BN + c, raw);
                    if (THREE) {
                        uint32_t rest[32];
                        tmem_ld32(tq + buf * MAX_BN + REST + c, rest);
                        tmem_ld_wait(raw);
                        tmem_ld_wait(rest);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            raw[i] = __float_as_uint(__uint_as_float(raw[i]) + __uint_as_float(rest[i]));
                    } else {
                        tmem_ld_wait(raw);
                    }
                };
                if (MODE == kStats) {
#pragma unroll 1
                    for (int c = c_lo; c < c_hi; c += 32) {
                        uint32_t raw[32];
                        sums(raw, c);
                        const int cnt = min(32, c_hi - c);
                        float v[32];
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = i < cnt ? __uint_as_float(raw[i]) * c2 : -INFINITY;
                        take<LIST>(r, v, n0 + c, cnt, target);
                    }
                } else if (MODE == kGrad) {
                    const int at0 = target < 0 ? -1 : target - p.b_row0 - n0;  // column of the tile
#pragma unroll 1
                    for (int c = c_lo; c < c_hi; c += 64) {
                        float v[2][32];
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            uint32_t raw[32];
                            sums(raw, c + 32 * x);
                            if (p.dentropy) {
#pragma unroll
                                for (int i = 0; i < 32; ++i) {
                                    const float lp = fmaf(__uint_as_float(raw[i]), zscale, -lse);
                                    v[x][i] = -ex2(lp * kLog2e) * fmaf(ge, fmaxf(lp, kNoWeight) + ent, g1);
                                }
                            } else {
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    v[x][i] = ex2(fmaf(__uint_as_float(raw[i]), zscale, -lse) * kLog2e) * -g1;
                            }
                            const int at = at0 - c - 32 * x;
                            if (__any_sync(0xffffffffu, (unsigned)at < 32u && target >= 0)) {
                                // the target's element, from its exact logit
                                const float pt = ex2(lpt * kLog2e);
                                const float f = p.dentropy ? fmaf(ge, fmaxf(lpt, kNoWeight) + ent, g1) : g1;
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    if (i == at && target >= 0) v[x][i] = fmaf(-pt, f, g1);
                            }
                        }
                        for (int piece = 0; piece < p.g_pieces; ++piece) {
                            uint4 o[8];
                            pack(v[0], o);
                            pack(v[1], o + 4);
                            store(o, n0 + c, m0, piece);
                            if (piece + 1 < p.g_pieces)
#pragma unroll
                                for (int i = 0; i < 64; ++i) {
                                    float &y = v[i >> 5][i & 31];
                                    y = isfinite(y) ? y - __bfloat162float(__float2bfloat16_rn(y)) : 0.f;
                                }
                        }
                    }
                } else if (p.part || !p.out_bf16) {
                    const float f = empty_part ? 0.f : uncut_scale((w.kb_hi - w.kb_lo) * (BK / 16) * ((!THREE && p.terms == 2) || (FEW && p.twice) ? 2 : 1));
#pragma unroll 1
                    for (int c = c_lo; c < c_hi; c += 32) {
                        uint32_t raw[32];
                        sums(raw, c);
                        uint4 o[8];
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            (&o[i >> 2].x)[i & 3] = empty_part ? 0u : __float_as_uint(__uint_as_float(raw[i]) * f);
                        const int part = p.part ? it.at / (p.mb * p.nb) : 0;
                        store(o, n0 + c, m0, FEW && p.stacked ? 2 * part + rank : part);
                    }
                } else {
#pragma unroll 1
                    for (int c = c_lo; c < c_hi; c += 64) {
                        uint4 o[8];
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            uint32_t raw[32];
                            sums(raw, c + 32 * x);
                            float v[32];
#pragma unroll
                            for (int i = 0; i < 32; ++i) v[i] = empty_part ? 0.f : __uint_as_float(raw[i]);
                            pack(v, o + 4 * x);
                        }
                        store(o, n0 + c, m0, 0);
                    }
                }
                tc_fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(cluster_addr(acc_empty + buf, 0));
            }
            if (MODE == kStats && ok) {
                const int s = it.at / p.mb, m = ((it.at - s * p.mb) * 2 + rank) * BM + row;
                if (m < p.M) {
                    const long long part = 2 * s + half;
                    p.stats[part * p.M + m] = make_float4(r.m, r.s + r.lo, r.es, r.zt);
#pragma unroll
                    for (int j = 0; j < LIST; ++j) {
                        const long long at = (part * LIST + j) * p.M + m;
                        p.list_val[at] = r.val[j];
                        p.list_id[at] = r.id[j];
                    }
                }
            }
        }
        if (MODE != kStats && lane == 0) bulk_wait_all();
        if (!ok && lane == 0) {
            atomicOr(status, TXL_STATUS_TIMEOUT);
            *abort_flag = 1;
        }
        tc_fence_before_sync();
    }

    __syncthreads();
    cluster_sync_all();
    if (warp == 2) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem, TM_COLS);
    }
}

template <Mode MODE, int LIST, bool THREE>
cudaError_t launch_gemm_of(const GemmLaunch &g, cudaStream_t s)
{
    static bool attr_set[64] = {};  // the attribute is set once per device
    auto *kernel = vocab_gemm_kernel<MODE, LIST, THREE>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    const int items = g.p[0].n_items + (MODE == kProducts ? g.p[1].n_items : 0);
    const unsigned grid = (unsigned)(min(items, device_sm_count() / 2) * 2);
    return launch_grid(kernel, dim3(grid), kThreads, SMEM_BYTES, s, 2, g);
}

template <Mode MODE, int LIST>
cudaError_t launch_gemm(const GemmLaunch &g, cudaStream_t s)
{
    // (products: both have three terms, or neither; one may be absent)
    const bool three = g.p[0].terms == 3 || (MODE == kProducts && g.p[1].terms == 3);
    return three ? launch_gemm_of<MODE, LIST, true>(g, s) : launch_gemm_of<MODE, LIST, false>(g, s);
}

} // namespace

cudaError_t launch_logprob_stats(const GemmLaunch &g, int list, cudaStream_t s)
{
    if (list == 0) return launch_gemm<kStats, 0>(g, s);
    return list == 12 ? launch_gemm<kStats, 12>(g, s) : launch_gemm<kStats, 20>(g, s);
}

cudaError_t launch_logprob_grad(const GemmLaunch &g, cudaStream_t s) { return launch_gemm<kGrad, 0>(g, s); }

cudaError_t launch_products(const GemmLaunch &g, cudaStream_t s)
{
    if (g.p[0].stacked || g.p[1].twice) return launch_gemm_of<kProducts, 1, false>(g, s);
    return launch_gemm<kProducts, 0>(g, s);
}

} // namespace txl
