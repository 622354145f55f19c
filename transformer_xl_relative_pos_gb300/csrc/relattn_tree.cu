// Relative-position attention of a tree of drafted tokens over a paged memory,
// bf16 on the tensor cores ("Transformer-XL: Attentive Language Models Beyond a
// Fixed-Length Context", §3.2 evaluation with a long memory, §3.3 score,
// Appendix B reversed table).
//
// For node i of depth d_i and memory row j of F rows the distance is F + d_i - j:
// the table row it needs is (r_rows - 1 - F) + j - d_i, Appendix B's shift by the
// node's depth instead of its index.  A node a among the keys stands at
// distance d_i - d_a, as a memory row j = F + d_a would.
//
// What it cannot do without is reading each sequence's keys and values once
// (256 bytes a key and head; the table stays in L2 across the batch).  A block's
// warps hold 16 nodes each and share the keys as tree_common.cuh says.  Per
// 32-key chunk a warp computes, with warp-level MMAs (mma.sync m16n8k16, bf16 in,
// fp32 out; a tcgen05 tile would be 64 or 128 rows, mostly padding for the 1 to
// 32 nodes that drafts have, and keeps its scores out of the registers in which
// the online softmax and the next product's operand want them):
//   content  (q_i + u).k_j        4 key tiles x 4 steps of 16 dimensions
//   position (q_i + v).r_t        the chunk's 32 table rows, likewise.  The products go
//            to a ring of 32 + D columns in shared memory (D = 16 MT >= any depth) and
//            are read back shifted by the nodes' depths; the next chunk's
//            window needs D of them again, so no table row is multiplied twice.
//   P.V      2 steps of 16 keys x 8 tiles of 8 dimensions
// q and u (or v) enter as they are, one MMA each into the same accumulator (at most 8
// nodes: q and the bias as the two halves of one tile's rows): the scores are exact products
// summed in fp32.  P enters as two bf16 values (value and residual), to about 2^-17
// relative, so that the output's own rounding is the one that shows; in trees of more than 16
// nodes, where the MMAs count, as one, 2^-8 (half a step of bf16, as large as the output's own
// rounding; 16 sequences of 64 nodes 180 us with residuals, 161 without, at that time).
//
// Measured (16 heads, 3800 rows, graph replays over inputs larger than L2): 19 sequences fill the two
// blocks of every SM, and take 46 us for 8 nodes (0.99 of a plain copy's rate, bound by DRAM), 53 us for 16
// (0.86), 82 us for 32 and 140 us for 64.  The last two are bound by latency: two warps that compute per
// SM quarter, whose matrix instructions, shared-memory accesses and issue slots are each about half
// busy.  One sequence of one node over 1600 rows takes 7.5 us (6.5 when its memory is in L2
// already), of which 2 are an empty kernel's and the rest a chain of
// dependent steps: state, page ids, copies, products, the merges of warps and blocks.
// What was tried for the wide trees and was slower: tcgen05 tiles of 128 rows [q; u; v] (bound by
// shared memory), 32 nodes a warp (registers), three blocks per SM (A operands re-read).
//
// Copies: each key group has a ring of stages [32 k rows | 32 v rows | 32 table
// rows], three TMA boxes on one mbarrier, swizzled so that the matrix loads are
// conflict-free.  Pages are aligned to chunks: a box never crosses one.  Chunk
// rows outside the memory (where it begins and ends inside a tile) hold
// whatever the page holds: their scores are masked and their values, which
// may be NaN, are zeroed in the fragments.
//
// The nodes' own keys and values come through the ring of the last group, ahead of its
// chunks; the table rows before a group's first chunk go from global memory straight into
// fragments while the first copies are on their way.
#include "tree_common.cuh"

namespace txl {
namespace {

using namespace tree;

constexpr int WARPS = 4, ROWS = 16;        // warps that compute, nodes of a warp
constexpr int THREADS = 2 * WARPS * 32;    // and as many for the copies, one per key group
constexpr int ROWB = DH * 2;               // bytes of a row
constexpr int BOX = GK * ROWB;             // 4096: one 32-row box
constexpr int ST_K = 0, ST_V = BOX, ST_R = 2 * BOX;
constexpr int STAGE = 3 * BOX;             // 12288

template <int MT>
struct Cfg {
    static constexpr int KG = WARPS / MT;      // key groups of a block
    static_assert(KG == tree_key_groups(16 * MT), "as the choice of key ranges has it");
    static constexpr int NSTG = MT == 1 ? 2 : MT == 2 ? 3 : 6;  // ring stages of a group
    // With four node tiles the products with u and v, alike for all nodes, are made once per
    // chunk by the three warps that have no copies, in turn (shared_biases): 48 MMAs of a
    // warp's 80 remain.  16 sequences of 16 heads, 64 nodes, 3800 rows: 141 us, 156 without.  With
    // two node tiles (and one such warp per key group) 32 nodes took 87 us against 83.
    static constexpr bool SHARED = MT == 4;
    static constexpr int HELPERS = WARPS - 1;
    static_assert(!SHARED || (KG == 1 && NSTG % HELPERS == 0), "a stage has one helper, which sees its every phase");
    // Registers a thread of the two kinds (warpgroups) after the split of the 128 that two
    // blocks of 256 threads per SM leave.
    static constexpr int REGS_COPY = SHARED ? 64 : 48, REGS_COMPUTE = 256 - REGS_COPY;
    static constexpr int DCAP = 16 * MT;       // depths are below this
    static constexpr int RW = GK + DCAP;       // columns of the product ring
    static constexpr int LD = RW + 8;          // its row stride (floats): 8 mod 16, so that the
                                               // quads' paired stores do not conflict
    static constexpr int SCR = 16 * LD * 4;    // bytes per warp
    static constexpr int OFF_SCR = KG * NSTG * STAGE;
    static constexpr int OFF_BIAS = OFF_SCR + WARPS * SCR;  // SHARED: u.k and v.r of a stage's rows
    static constexpr int OFF_BAR = OFF_BIAS + (SHARED ? NSTG * 2 * GK * 4 : 0);  // full[KG][NSTG], empty, biased
    static constexpr int OFF_TOPO = OFF_BAR + 3 * KG * NSTG * 8;
    static constexpr int OFF_OK = OFF_TOPO + (int)sizeof(Topology);  // page of a stage valid
    static constexpr int OFF_FLAG = OFF_OK + KG * NSTG * 4;
    static constexpr int SMEM = OFF_FLAG + 16 + 1024;  // slack for the manual alignment
    // where a warp leaves its record: its private ring, or (shared ring) its scratch
    static_assert(MT == 1 || sizeof(Rec<ROWS>) <= SCR, "a warp's record fits in its scratch");
    static_assert(sizeof(Rec<ROWS>) <= NSTG * STAGE, "a warp's record fits in its ring");
    static_assert(OFF_BAR % 8 == 0 && OFF_TOPO % 8 == 0, "8-byte alignment");
    static_assert(2 * (SMEM + 1024) <= 228 * 1024, "two blocks per SM");
};

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
                 "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same from a zero accumulator.
__device__ __forceinline__ void mma16816_first(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ void ldsm_x4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

__device__ __forceinline__ void ldsm_x4_t(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

// Scratch accesses by 32-bit shared-memory address.
__device__ __forceinline__ float ld_scr(uint32_t addr)
{
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void ld_scr2(uint32_t addr, float &x, float &y)
{
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(x), "=f"(y) : "r"(addr) : "memory");
}

__device__ __forceinline__ void st_scr2(uint32_t addr, float x, float y)
{
    asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(x), "f"(y) : "memory");
}

// bf16 pair of (x0, x1), and in `res` the pair of what the rounding left over.
__device__ __forceinline__ uint32_t split_bf16x2(float x0, float x1, uint32_t &res)
{
    const uint32_t hi = pack_bf16x2(x0, x1);
    res = pack_bf16x2(x0 - bf_lo(hi), x1 - bf_hi(hi));
    return hi;
}

// The mbarrier's phase also waits for this thread's copies so far (its pending count
// is raised by one until they are there).
__device__ __forceinline__ void cp_async_hold(uint64_t *bar)
{
    asm volatile("cp.async.mbarrier.arrive.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// The running softmax and output of a warp's nodes: NR rows per lane (g, and g + 8
// when NR = 2); its output columns are 8 nd + 2 t, + 1.  LO: the products with the
// probabilities' residuals, kept apart until the end, as a residual (of either sign, or zero)
// times an infinity must not meet the infinity of the product itself.  With NR = 1 (at most 8
// nodes) they are the accumulators' rows g + 8, with NR = 2 accumulators of their own (19 x 16 nodes of
// 3800 rows 53.4 us, 52.2 with one set of accumulators; no registers spill).
template <int NR, bool LO>
struct State {
    static constexpr bool APART = LO && NR == 2;
    float m[NR], l[NR];
    float acc[8][4];
    float res[APART ? 8 : 1][4];
    // Column e (0, 1) of this lane's row r in tile nd: an infinite product stands by itself.
    __device__ __forceinline__ float out(int nd, int r, int e) const
    {
        const float x = acc[nd][2 * r + e];
        if constexpr (!LO) return x;
        const float y = NR == 1 ? acc[nd][2 + e] : res[APART ? nd : 0][2 * r + e];
        return fabsf(x) == INFINITY ? x : x + y;
    }
};

// One chunk's masked scores s (before the scale; s[nt][2 r + e]: row r of this lane, key
// 8 nt + 2 t + e) into probabilities, rescaling the state to the new maximum.
// scale > 0, to log2 units.
template <int NR, bool LO>
__device__ __forceinline__ void softmax_step(State<NR, LO> &st, float (&s)[4][2 * NR], float scale)
{
    float mx[NR], ms[NR];
    bool moved = false;
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        mx[r] = st.m[r];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) mx[r] = max3_nan(mx[r], s[nt][2 * r], s[nt][2 * r + 1]);
        mx[r] = max_nan(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
        mx[r] = max_nan(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
        // a row without a visible key so far: any finite value makes its probabilities zero
        ms[r] = mx[r] == -INFINITY ? 0.f : __fmul_rn(mx[r], scale);
        moved |= !(mx[r] == st.m[r]);
    }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int r = 0; r < NR; ++r) {
            // The old maximum as it was rounded when it was the new one, not fused with the
            // difference: a row whose maximum has not moved is rescaled by exactly one.
            const float f = ex2f(__fmul_rn(st.m[r], scale) - ms[r]);  // (0 from -inf: the sums are zero then)
            st.m[r] = mx[r];
            st.l[r] *= f;
#pragma unroll
            for (int nd = 0; nd < 8; ++nd)
#pragma unroll
                for (int e = 0; e < 4 / NR; ++e) {
                    st.acc[nd][2 * r + e] *= f;
                    if constexpr (State<NR, LO>::APART) st.res[nd][2 * r + e] *= f;
                }
        }
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        float sum[4];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
            s[nt][2 * r] = ex2f(fmaf(s[nt][2 * r], scale, -ms[r]));
            s[nt][2 * r + 1] = ex2f(fmaf(s[nt][2 * r + 1], scale, -ms[r]));
            sum[nt] = s[nt][2 * r] + s[nt][2 * r + 1];
        }
        st.l[r] += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    }
}

// acc += P.V over 16 keys 16 kk .. + 15, v[nd]: their fragments of dimensions 8 nd .. + 7.
// The probabilities enter as bf16 and, with LO (NR = 1: always), their residuals.
template <int NR, bool LO>
__device__ __forceinline__ void pv_step(State<NR, LO> &st, const float (&s)[4][2 * NR], int kk,
                                        const uint32_t (&v)[8][2])
{
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int c = 0; c < 2; ++c)
        if constexpr (!LO && NR == 2) {
            hi[2 * c] = pack_bf16x2(s[2 * kk + c][0], s[2 * kk + c][1]);
            hi[2 * c + 1] = pack_bf16x2(s[2 * kk + c][2], s[2 * kk + c][3]);
        } else if constexpr (NR == 2) {
            hi[2 * c] = split_bf16x2(s[2 * kk + c][0], s[2 * kk + c][1], lo[2 * c]);
            hi[2 * c + 1] = split_bf16x2(s[2 * kk + c][2], s[2 * kk + c][3], lo[2 * c + 1]);
        } else {
            hi[2 * c] = split_bf16x2(s[2 * kk + c][0], s[2 * kk + c][1], hi[2 * c + 1]);
        }
#pragma unroll
    for (int nd = 0; nd < 8; ++nd) mma16816(st.acc[nd], hi, v[nd][0], v[nd][1]);
    if constexpr (LO && NR == 2) {
#pragma unroll
        for (int nd = 0; nd < 8; ++nd) mma16816(st.res[nd], lo, v[nd][0], v[nd][1]);
    }
}

// Step ks of 16 dimensions of (q + bias).b for four tiles of eight rows b, whose
// fragments are words w, w + 1 of f: first the products with q (HALF: with q and the bias at
// once), then those with the bias.
template <bool HALF, int W>
__device__ __forceinline__ void q_products(float (&c)[4][4], const uint32_t (&aq)[4][4],
                                           const uint32_t (&bias)[4][4], int ks, const uint32_t (&f)[4][W],
                                           int w)
{
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
        if constexpr (HALF) {
            if (ks == 0) mma16816_first(c[nt], bias[0], f[nt][w], f[nt][w + 1]);
            else mma16816(c[nt], bias[ks], f[nt][w], f[nt][w + 1]);
        } else {
            if (ks == 0) mma16816_first(c[nt], aq[0], f[nt][w], f[nt][w + 1]);
            else mma16816(c[nt], aq[ks], f[nt][w], f[nt][w + 1]);
        }
    }
}

template <bool HALF, int W>
__device__ __forceinline__ void bias_products(float (&c)[4][4], const uint32_t (&bias)[4][4], int ks,
                                              const uint32_t (&f)[4][W], int w)
{
    if constexpr (!HALF) {
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) mma16816(c[nt], bias[ks], f[nt][w], f[nt][w + 1]);
    }
}

// Element e (0, 1) of this lane's row r in a product's fragment.
template <bool HALF>
__device__ __forceinline__ float element(const float (&c)[4], int r, int e)
{
    return HALF ? c[e] + c[2 + e] : c[2 * r + e];
}

// u.k_j and v.r_t of the block's chunks, every HELPERS-th item from item `first` on (one warp):
// summed by the tensor cores in fp32, as the products with q are.  Per item it waits for
// the copies and arrives on the stage's `biased`, for which every warp that computes waits
// before it lets the stage go: none of the barriers runs ahead of another by two phases.
template <int MT>
__device__ __forceinline__ void shared_biases(const TreeParams &p, int begin, int fill, int n, int h, int split,
                                              int first, uint8_t *smem, int lane)
{
    using C = Cfg<MT>;
    constexpr int NSTG = C::NSTG;
    const int t = lane & 3, lr = lane & 7, lm = lane >> 3;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR), *biased = full + 2 * NSTG;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_FLAG);
    const Chunks ck = group_chunks(p, begin, fill, kNodesCost, split, p.n_splits);
    const int nodes = split == p.n_splits - 1 ? (n + GK - 1) / GK : 0;  // (items without biases)
    const uint32_t sign = p.scale_log2 < 0.f ? 0x80008000u : 0u, some = p.scale_log2 == 0.f ? 0u : ~0u;
    // A operands whose rows are all u, or all v: registers 0 = 1 and 2 = 3 of each step
    uint32_t a[2][4][2];
#pragma unroll
    for (int x = 0; x < 8; ++x) {
        const int w = h * (DH / 2) + 4 * x + t;
        a[0][x >> 1][x & 1] = (__ldg(static_cast<const uint32_t *>(p.u) + w) ^ sign) & some;
        a[1][x >> 1][x & 1] = (__ldg(static_cast<const uint32_t *>(p.vb) + w) ^ sign) & some;
    }
    for (int item = first; item < nodes + ck.count; item += C::HELPERS) {
        const int st = item % NSTG;
        if (!__all_sync(0xffffffffu, mbar_wait(full + st, (item / NSTG) & 1, abort_flag, p.wait_ns))) {
            if (lane == 0) {
                *abort_flag = 1;
                atomicOr(p.status, TXL_STATUS_TIMEOUT);
            }
            return;
        }
        if (item >= nodes) {
            float *out = reinterpret_cast<float *>(smem + C::OFF_BIAS) + st * 2 * GK;
#pragma unroll
            for (int uv = 0; uv < 2; ++uv) {
                const uint32_t rows = smem_u32(smem) + st * STAGE + (uv ? ST_R : ST_K);
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    uint32_t b[2][4];
                    float c[4];
                    ldsm_x4(b[0], rows + swz(8 * nt + lr, lm));
                    ldsm_x4(b[1], rows + swz(8 * nt + lr, 4 + lm));
#pragma unroll
                    for (int ks = 0; ks < 4; ++ks) {
                        const uint32_t a4[4] = {a[uv][ks][0], a[uv][ks][0], a[uv][ks][1], a[uv][ks][1]};
                        if (ks == 0) mma16816_first(c, a4, b[0][0], b[0][1]);
                        else mma16816(c, a4, b[ks >> 1][2 * (ks & 1)], b[ks >> 1][2 * (ks & 1) + 1]);
                    }
                    if (lane < 4) *reinterpret_cast<float2 *>(out + uv * GK + 8 * nt + 2 * t) = make_float2(c[0], c[1]);
                }
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(biased + st);
    }
}

// MT node tiles of 16; HALF: at most 8 nodes (one tile, whose rows 8 to 15 then take u, v
// and the probabilities' residuals: half the MMAs).
template <int MT, bool HALF>
__global__ void __launch_bounds__(THREADS, 2)
    relattn_tree_kernel(const __grid_constant__ CUtensorMap tm_kv,
                        const __grid_constant__ CUtensorMap tm_r, const TreeParams p)
{
    using C = Cfg<MT>;
    static_assert(!HALF || MT == 1, "half a tile");
    constexpr int KG = C::KG, NSTG = C::NSTG, DCAP = C::DCAP, RW = C::RW, LD = C::LD;
    constexpr int NR = HALF ? 1 : 2;           // nodes per lane
    constexpr int TB = DCAP / 8 < 4 ? DCAP / 8 : 4;  // table tiles loaded at once
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int mt = warp % MT, kg = warp / MT;
    const int g = lane >> 2, t = lane & 3;
    const int split = blockIdx.x % p.n_splits;
    const int bh = blockIdx.x / p.n_splits;
    const int rank = bh / p.mem.H, h = bh - rank * p.mem.H;
    const int b = pick_sequence(p, rank, *reinterpret_cast<Topology *>(smem + C::OFF_TOPO));
    int begin, fill;
    paged_state(p.mem, b, p.status, begin, fill);
    const int n = p.n_nodes ? min(max(p.n_nodes[b], 0), p.N) : p.N;
    if (n == 0) return finish_barriers(p);  // nothing of this sequence is written
    const int parent = threadIdx.x < n ? p.parents[b * p.parents_stride + threadIdx.x] : -1;

    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR);  // full, empty, biased, [KG][NSTG] each
    volatile int *stage_ok = reinterpret_cast<volatile int *>(smem + C::OFF_OK);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_FLAG);
    Topology &topo = *reinterpret_cast<Topology *>(smem + C::OFF_TOPO);
    const auto rec = [smem](int w) {
        return reinterpret_cast<Rec<ROWS> *>(MT == 1 ? smem + w * NSTG * STAGE
                                                     : smem + C::OFF_SCR + w * C::SCR);
    };

    if (warp >= WARPS) {
        // ===================== the copies: a warp per key group, its lane 0 ============
        // Boxes are always complete (rows past a tensor's ends arrive as zeros): a page
        // id out of range becomes a plane past the pool's end, and its rows are masked.
        // The id of a page is loaded an item ahead.
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_COPY));
        const int group = warp - WARPS;
        const bool mine = group < KG;
        if (warp == WARPS && lane == 0) *abort_flag = 0;
        if (mine && lane == 0) {
            for (int s = 0; s < NSTG; ++s) {
                mbar_init(bars + group * NSTG + s, 1);
                mbar_init(bars + (KG + group) * NSTG + s, MT);
                mbar_init(bars + (2 * KG + group) * NSTG + s, 1);
            }
            fence_barrier_init();
        }
        __syncwarp();
        Chunks ck{};
        if (mine) ck = group_chunks(p, begin, fill, kNodesCost, split * KG + group, p.n_splits * KG);
        const int nodes = split == p.n_splits - 1 && group == KG - 1 ? (n + GK - 1) / GK : 0;
        const int items = mine ? nodes + ck.count : 0;
        int slot = ck.slot, row = ck.row, page = -1;
        if (mine && ck.count > 0 && lane == 0) page = page_at(p.mem, b, slot, p.status);
        const uint64_t pol_stream = policy_evict_first();  // k, v: read once
        const uint64_t pol_keep = policy_evict_last();     // table: shared by the batch
        const int trow0 = p.r_rows - 1 - fill + ck.c0 * GK - ck.off;  // table row of the first chunk's key 0
        // One item into its stage (the whole warp): for the group that takes the nodes
        // among themselves boxes of them, then its chunks.
        auto issue = [&](int item) {
            const int st = group * NSTG + item % NSTG;
            uint64_t *bar = bars + st;
            uint8_t *dst = smem + st * STAGE;
            if (item < nodes) {
                // 32 rows of the nodes' k and v (past the last: zeros), swizzled as TMA does
                const __nv_bfloat16 *kn = static_cast<const __nv_bfloat16 *>(p.k.ptr) + b * p.k.sb + h * p.k.sh;
                const __nv_bfloat16 *vn = static_cast<const __nv_bfloat16 *>(p.v.ptr) + b * p.v.sb + h * p.v.sh;
                const uint32_t at = smem_u32(dst);
#pragma unroll 2
                for (int x = lane; x < GK * 8; x += 32) {
                    const int a = item * GK + (x >> 3), c = x & 7;
                    const bool there = a < n;
                    cp_async16(at + ST_K + swz(x >> 3, c), kn + (there ? a * p.k.sr + 8 * c : 0), there);
                    cp_async16(at + ST_V + swz(x >> 3, c), vn + (there ? a * p.v.sr + 8 * c : 0), there);
                }
                cp_async_hold(bar);
                __syncwarp();
                if (lane == 0) mbar_arrive(bar);
            } else if (lane == 0) {
                fence_proxy_async_smem();  // (the stage may have held nodes, written without TMA)
                const int planes = p.mem.n_pages * p.mem.H;  // of keys; then as many of values
                const int plane = page >= 0 ? page * p.mem.H + h : 2 * planes;
                stage_ok[st] = page >= 0;
                mbar_arrive_expect_tx(bar, (uint32_t)STAGE);
                tma_load_3d_hint(dst + ST_K, &tm_kv, bar, 0, row, plane, pol_stream);
                tma_load_3d_hint(dst + ST_V, &tm_kv, bar, 0, row, page >= 0 ? plane + planes : plane, pol_stream);
                tma_load_3d_hint(dst + ST_R, &tm_r, bar, 0, trow0 + (item - nodes) * GK, h, pol_keep);
                if (next_chunk(p.mem, slot, row) && item + 1 < items) page = page_at(p.mem, b, slot, p.status);
            }
        };
        int issued = 0;
        for (; issued < min(NSTG, items); ++issued) issue(issued);
        __syncwarp();
        build_topology(topo, parent, n, p.status);
        // refill each stage when the group's warps have left it
        bool ok = true;
        for (; issued < items; ++issued) {
            if (lane == 0)
                ok = mbar_wait(bars + (KG + group) * NSTG + issued % NSTG, (issued / NSTG + 1) & 1, abort_flag,
                               p.wait_ns);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
            issue(issued);
        }
        if (lane == 0) {
            if (!ok) {
                *abort_flag = 1;
                atomicOr(p.status, TXL_STATUS_TIMEOUT);
            }
            // the copies in flight land before shared memory is used for anything else
            const int zero = 0;
            for (int x = max(0, issued - NSTG); x < issued; ++x)
                mbar_wait(bars + group * NSTG + x % NSTG, (x / NSTG) & 1, &zero, p.wait_ns);
        }
        __syncwarp();
        if constexpr (C::SHARED) {
            if (!mine) shared_biases<MT>(p, begin, fill, n, h, split, group - 1, smem, lane);
        }
        finish_barriers(p);
        return;
    }
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_COMPUTE));

    const uint8_t *ring = smem + kg * NSTG * STAGE;
    uint64_t *full = bars + kg * NSTG, *empty = full + KG * NSTG;
    uint64_t *filled = C::SHARED ? empty + KG * NSTG : full;  // an item's data are there
    float *scr = reinterpret_cast<float *>(smem + C::OFF_SCR + warp * C::SCR);
    const uint32_t scr_at = smem_u32(scr);
    const Chunks ck = group_chunks(p, begin, fill, kNodesCost, split * KG + kg, p.n_splits * KG);
    const int trow0 = p.r_rows - 1 - fill + ck.c0 * GK - ck.off;  // table row of the first chunk's key 0

    // A operands, dimensions 16 ks + 2 t, + 1 (registers 0, 1) and + 8, + 9 (2, 3): rows
    // g, g + 8 of the tile's q; u and v, alike in every row.  HALF: au holds q in rows g
    // and u in rows g + 8, av q and v; a product's two rows are then added.
    const int i0 = mt * 16 + g;  // this lane's first node (the second: + 8)
    // With the scale's sign in the A operands (zeros for scale 0) the scores want a
    // positive factor only.
    const float scale = p.scale_log2 == 0.f ? 1.f : fabsf(p.scale_log2);
    const uint32_t sign = p.scale_log2 < 0.f ? 0x80008000u : 0u, some = p.scale_log2 == 0.f ? 0u : ~0u;
    uint32_t aq[4][4], au[4][4], av[4][4];
    {
        const __nv_bfloat16 *qb = static_cast<const __nv_bfloat16 *>(p.q.ptr) + b * p.q.sb + h * p.q.sh;
        const uint32_t *urow = reinterpret_cast<const uint32_t *>(static_cast<const __nv_bfloat16 *>(p.u) + h * DH);
        const uint32_t *vrow = reinterpret_cast<const uint32_t *>(static_cast<const __nv_bfloat16 *>(p.vb) + h * DH);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int w = 8 * ks + 4 * half + t;
#pragma unroll
                for (int r = 0; r < NR; ++r)
                    aq[ks][2 * half + r] =
                        i0 + 8 * r < n
                            ? (reinterpret_cast<const uint32_t *>(qb + (i0 + 8 * r) * p.q.sr)[w] ^ sign) & some
                            : 0;
                au[ks][2 * half + 1] = (__ldg(urow + w) ^ sign) & some;
                av[ks][2 * half + 1] = (__ldg(vrow + w) ^ sign) & some;
                au[ks][2 * half] = HALF ? aq[ks][2 * half] : au[ks][2 * half + 1];
                av[ks][2 * half] = HALF ? aq[ks][2 * half] : av[ks][2 * half + 1];
            }
    }
    auto put_products = [&](const float (&c)[4], int col) {
        TXL_CHECK(col >= 0 && col + 8 <= RW, p.status);
#pragma unroll
        for (int r = 0; r < NR; ++r)
            st_scr2(scr_at + ((g + 8 * r) * LD + col + 2 * t) * 4, element<HALF>(c, r, 0), element<HALF>(c, r, 1));
    };
    // 32 contiguous bytes' worth of a row in fragment order: word x holds dimensions
    // 8 x + 2 t, + 1 (words 2 ks, 2 ks + 1: step ks).
    auto load_row = [&](uint32_t (&w)[8], const __nv_bfloat16 *src, bool there) {
#pragma unroll
        for (int x = 0; x < 8; ++x)
            w[x] = there ? __ldg(reinterpret_cast<const uint32_t *>(src) + 4 * x + t) : 0;
    };
    // TB tiles of eight table rows from global memory (rows outside the table: zero),
    // and their products into ring columns col ...
    const __nv_bfloat16 *table = static_cast<const __nv_bfloat16 *>(p.r) + (long long)h * p.r_rows * DH;
    auto load_table = [&](auto &w, int row0) {
#pragma unroll
        for (int x = 0; x < TB; ++x) {
            const int tr = row0 + 8 * x + g;
            load_row(w[x], table + (long long)tr * DH, tr >= 0 && tr < p.r_rows);
        }
    };
    auto table_products = [&](const auto &w, int col) {
#pragma unroll
        for (int x = 0; x < TB; ++x) {
            float c[4];
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) {
                if (ks == 0) mma16816_first(c, av[0], w[x][0], w[x][1]);
                else mma16816(c, av[ks], w[x][2 * ks], w[x][2 * ks + 1]);
                if (!HALF) mma16816(c, aq[ks], w[x][2 * ks], w[x][2 * ks + 1]);
            }
            put_products(c, col + 8 * x);
        }
    };
    // P.V of one chunk, element by element: for a chunk whose keys are not all
    // visible to the same nodes and whose values hold an infinity or NaN, which must
    // not reach the nodes that do not see the key.  hidden: bit 4 nt + 2 r + e of this
    // lane's elements.  col0: 32 free ring columns.
    State<NR, MT == 1> st;
    auto pv_by_element = [&](const auto &s, uint32_t hidden, int col0, const uint8_t *values) {
        auto at = [&](int key) { const int c = col0 + key; return c >= RW ? c - RW : c; };
        __syncwarp();
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int e = 0; e < 2 * NR; ++e)
                scr[(g + 8 * (e >> 1)) * LD + at(8 * nt + 2 * t + (e & 1))] =
                    (hidden >> (4 * nt + e)) & 1 ? -1.f : s[nt][e];
        __syncwarp();
#pragma unroll 1
        for (int key = 0; key < GK; ++key) {
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const float pr = scr[(g + 8 * r) * LD + at(key)];
                if (pr < 0.f) continue;
#pragma unroll
                for (int nd = 0; nd < 8; ++nd) {
                    const uint32_t v2 = *reinterpret_cast<const uint32_t *>(values + swz(key, nd) + 4 * t);
                    st.acc[nd][2 * r] = fmaf(pr, bf_lo(v2), st.acc[nd][2 * r]);
                    st.acc[nd][2 * r + 1] = fmaf(pr, bf_hi(v2), st.acc[nd][2 * r + 1]);
                }
            }
        }
        __syncwarp();
    };
    // Whether a value row lo .. hi - 1 of a box holds an infinity or NaN (lane = key).
    auto nonfinite_values = [&](const uint8_t *values, int lo, int hi) {
        bool bad = false;
        if (lane >= lo && lane < hi) {
#pragma unroll 1
            for (int x = 0; x < 8; ++x) {
                const uint4 w = *reinterpret_cast<const uint4 *>(values + swz(lane, x));
                bad |= nonfinite2(w.x) | nonfinite2(w.y) | nonfinite2(w.z) | nonfinite2(w.w);
            }
        }
        return __any_sync(0xffffffffu, bad) != 0;
    };
    const int lr = lane & 7, lm = lane >> 3;  // matrix-load roles: row, matrix
    // V fragments of keys 16 kk .. 16 kk + 15 of a box
    auto load_v = [&](uint32_t (&bv)[8][2], uint32_t sv, int kk) {
#pragma unroll
        for (int np = 0; np < 4; ++np) {
            uint32_t w[4];
            ldsm_x4_t(w, sv + swz(16 * kk + (lm & 1) * 8 + lr, 2 * np + (lm >> 1)));
            bv[2 * np][0] = w[0];
            bv[2 * np][1] = w[1];
            bv[2 * np + 1][0] = w[2];
            bv[2 * np + 1][1] = w[3];
        }
    };

    const bool active = mt * 16 < n;  // this warp has nodes
    // The last group takes the nodes among themselves.  The table rows for them, or before
    // the first chunk's, are loaded ahead of the tree's construction.
    const bool nodes_here = split == p.n_splits - 1 && kg == KG - 1, owner = active && nodes_here;
    const int nodes = nodes_here ? (n + GK - 1) / GK : 0;  // boxes of nodes ahead of the chunks
    uint32_t tw[TB][8];
    if (active && (owner || ck.count > 0)) load_table(tw, (owner ? p.r_rows : trow0) - DCAP);
    build_topology(topo, parent, n, p.status);
    int depth[NR], depth_max = 0;
    unsigned long long anc[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        const bool there = i0 + 8 * r < n;
        depth[r] = there ? topo.depth[i0 + 8 * r] : 0;
        anc[r] = there ? topo.anc[i0 + 8 * r] : 0;
        depth_max = max(depth_max, depth[r]);
        st.m[r] = -INFINITY;
        st.l[r] = 0.f;
    }
    depth_max = __reduce_max_sync(0xffffffffu, depth_max);
#pragma unroll
    for (int nd = 0; nd < 8; ++nd)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            st.acc[nd][e] = 0.f;
            if constexpr (decltype(st)::APART) st.res[nd][e] = 0.f;
        }

    bool ok = true;
    if (!active)  // (a warp without nodes only lets the stages go)
        for (int box = 0; box < nodes && ok; ++box) {
            ok = __all_sync(0xffffffffu, mbar_wait(filled + box % NSTG, (box / NSTG) & 1, abort_flag, p.wait_ns));
            if (lane == 0 && ok) mbar_arrive(empty + box % NSTG);
        }
    if (owner) {
        // ---- the nodes among themselves: distances 0 .. DCAP - 1 ------------------
        table_products(tw, 0);
#pragma unroll
        for (int c = TB * 8; c < DCAP; c += TB * 8) {
            load_table(tw, p.r_rows - DCAP + c);
            table_products(tw, c);
        }
        __syncwarp();
        for (int box = 0; box < nodes && ok; ++box) {
            ok = __all_sync(0xffffffffu, mbar_wait(filled + box % NSTG, (box / NSTG) & 1, abort_flag, p.wait_ns));
            // (no node is an ancestor of an earlier one: boxes past this tile are hidden)
            if (ok && box * GK < mt * 16 + 16) {
                const uint8_t *base = ring + (box % NSTG) * STAGE;
                const int a0 = box * GK;
                float c[4][4], s[4][2 * NR];
                const uint32_t sk = smem_u32(base + ST_K);
#pragma unroll
                for (int h2 = 0; h2 < 2; ++h2) {
                    uint32_t bk[4][4];
#pragma unroll
                    for (int nt = 0; nt < 4; ++nt) ldsm_x4(bk[nt], sk + swz(8 * nt + lr, 4 * h2 + lm));
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        q_products<HALF>(c, aq, au, 2 * h2 + x, bk, 2 * x);
                        bias_products<HALF>(c, au, 2 * h2 + x, bk, 2 * x);
                    }
                }
                uint32_t hidden = 0;
#pragma unroll
                for (int r = 0; r < NR; ++r) {
                    const unsigned long long mine = anc[r] >> a0;
#pragma unroll
                    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int a = 8 * nt + 2 * t + e;
                            const bool related = (mine >> a) & 1;
                            const int dist = related ? depth[r] - topo.depth[a0 + a] : 0;
                            const bool seen = related && dist < p.r_rows;
                            TXL_CHECK(dist >= 0 && dist < DCAP, p.status);
                            hidden |= seen ? 0u : 1u << (4 * nt + 2 * r + e);
                            s[nt][2 * r + e] = seen ? element<HALF>(c[nt], r, e) +
                                                          ld_scr(scr_at + ((g + 8 * r) * LD + DCAP - 1 - dist) * 4)
                                                    : -INFINITY;
                        }
                }
                softmax_step(st, s, scale);
                if (nonfinite_values(base + ST_V, 0, GK)) {
                    pv_by_element(s, hidden, DCAP, base + ST_V);
                } else {
#pragma unroll
                    for (int kk = 0; kk < 2; ++kk) {
                        uint32_t bv[8][2];
                        load_v(bv, smem_u32(base + ST_V), kk);
                        pv_step(st, s, kk, bv);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty + box % NSTG);
        }
        __syncwarp();  // the ring's columns are free again
        if (ck.count > 0) load_table(tw, trow0 - DCAP);
    }
    if (active && ck.count > 0) {  // the DCAP table rows before the first chunk's
        table_products(tw, 0);
#pragma unroll
        for (int c = TB * 8; c < DCAP; c += TB * 8) {
            load_table(tw, trow0 - DCAP + c);
            table_products(tw, c);
        }
    }

    // ---- the memory, chunk by chunk ---------------------------------------------
    int wpos = DCAP;  // ring column of the chunk's first table row
    const int items = nodes + ck.count;
    int stg = nodes % NSTG, phase = (nodes / NSTG) & 1;
    bool ready = false;  // the item's stage was seen full ahead of its turn
    for (int item = nodes; ok && item < items; ++item) {
        if (!__all_sync(0xffffffffu, ready)) {
            ok = __all_sync(0xffffffffu, mbar_wait(full + stg, phase, abort_flag, p.wait_ns));
            if (!ok) break;
        }
        const int this_stg = stg, this_phase = phase;
        // (SHARED: the products with u and v of this item are there)
        auto biased = [&] {
            return !C::SHARED ||
                   __all_sync(0xffffffffu, mbar_wait(filled + this_stg, this_phase, abort_flag, p.wait_ns));
        };
        if (++stg == NSTG) {
            stg = 0;
            phase ^= 1;
        }
        const bool page_ok = stage_ok[kg * NSTG + this_stg] != 0;
        ready = false;
        if (active) {
            const uint8_t *base = ring + this_stg * STAGE;
            const uint32_t sk = smem_u32(base + ST_K), sv = smem_u32(base + ST_V), sr = smem_u32(base + ST_R);
            const int j0 = (ck.c0 + item - nodes) * GK - ck.off;  // memory row of the chunk's first key

            // content and position products (SHARED: those with q; the others' sums are added
            // behind them), eight independent accumulators in turn (one
            // after the other, each MMA would wait for the one before)
            float c[4][4], cr[4][4];
#pragma unroll
            for (int h2 = 0; h2 < 2; ++h2) {
                uint32_t bk[4][4], br[4][4];
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    ldsm_x4(bk[nt], sk + swz(8 * nt + lr, 4 * h2 + lm));
                    ldsm_x4(br[nt], sr + swz(8 * nt + lr, 4 * h2 + lm));
                }
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    q_products<HALF>(c, aq, au, 2 * h2 + x, bk, 2 * x);
                    q_products<HALF>(cr, aq, av, 2 * h2 + x, br, 2 * x);
                    bias_products<HALF || C::SHARED>(c, au, 2 * h2 + x, bk, 2 * x);
                    bias_products<HALF || C::SHARED>(cr, av, 2 * h2 + x, br, 2 * x);
                }
            }
            ok = biased();
            if (!ok) break;
            if constexpr (C::SHARED) {
                const uint32_t bias = smem_u32(smem + C::OFF_BIAS) + this_stg * 2 * GK * 4 + 8 * t;
#pragma unroll
                for (int nt = 0; nt < 4; ++nt) {
                    float b0, b1;
                    ld_scr2(bias + 32 * nt, b0, b1);
                    c[nt][0] += b0, c[nt][1] += b1, c[nt][2] += b0, c[nt][3] += b1;
                    ld_scr2(bias + GK * 4 + 32 * nt, b0, b1);
                    cr[nt][0] += b0, cr[nt][1] += b1, cr[nt][2] += b0, cr[nt][3] += b1;
                }
            }
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                const int col = wpos + 8 * nt;
                put_products(cr[nt], col >= RW ? col - RW : col);
            }
            __syncwarp();
            // scores: the position product of key jj and a node of depth d stands
            // d columns before the chunk's own column jj, in the window of RW columns that
            // begins at the ring column after the chunk's last
            int next = wpos + GK;
            next -= next >= RW ? RW : 0;
            float s[4][2 * NR];
#pragma unroll
            for (int r = 0; r < NR; ++r) {
                const int first = next + DCAP + 2 * t - depth[r];
                const uint32_t at = scr_at + ((g + 8 * r) * LD + first) * 4;
#pragma unroll
                for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const int jj = 8 * nt + e;
                        const bool wraps = jj >= RW - first;
                        TXL_CHECK(first + jj - (wraps ? RW : 0) >= 0 && first + jj - (wraps ? RW : 0) < RW, p.status);
                        s[nt][2 * r + e] = element<HALF>(c[nt], r, e) + ld_scr((wraps ? at - RW * 4 : at) + 4 * jj);
                    }
            }
            // Keys that are not memory rows (the chunk sticks out at either end, or its
            // page is unknown) or that the table does not reach from the node.
            const bool out_of_memory = j0 < 0 || j0 + GK > fill || !page_ok;
            const bool partly_hidden = j0 < fill + depth_max - p.r_rows + 1;
            const int key_lo = -j0, key_hi = page_ok ? fill - j0 : 0;  // memory rows of the chunk
            uint32_t hidden = 0;
            if (out_of_memory || partly_hidden) {
#pragma unroll
                for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                    for (int e = 0; e < 2 * NR; ++e) {
                        const int jj = 8 * nt + 2 * t + (e & 1);
                        if (jj < max(0, fill + depth[e >> 1] - p.r_rows + 1) - j0 || jj >= key_hi) {
                            s[nt][e] = -INFINITY;
                            hidden |= 1u << (4 * nt + e);
                        }
                    }
            }
            // what the softmax's latencies leave time for: the values, and whether the next
            // stage is there
            uint32_t bv[2][8][2];
            load_v(bv[0], sv, 0);
            load_v(bv[1], sv, 1);
            ready = item + 1 < items && mbar_test(full + stg, phase);
            softmax_step(st, s, scale);
            if (partly_hidden && nonfinite_values(base + ST_V, key_lo, key_hi)) {
                pv_by_element(s, hidden, next, base + ST_V);
            } else {
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    if (out_of_memory) {
                        // this lane's fragment rows: keys 16 kk + 2 t, + 1 and + 8, + 9
                        const int key = 16 * kk + 2 * t;
                        auto in = [&](int x) { return x >= key_lo && x < key_hi; };
                        const uint32_t keep0 = (in(key) ? 0xffffu : 0u) | (in(key + 1) ? 0xffff0000u : 0u);
                        const uint32_t keep1 = (in(key + 8) ? 0xffffu : 0u) | (in(key + 9) ? 0xffff0000u : 0u);
#pragma unroll
                        for (int nd = 0; nd < 8; ++nd) {
                            bv[kk][nd][0] &= keep0;
                            bv[kk][nd][1] &= keep1;
                        }
                    }
                    pv_step(st, s, kk, bv[kk]);
                }
            }
            wpos = next;
        } else {
            ok = biased();
            if (!ok) break;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(empty + this_stg);  // this warp has read the stage
    }
    if (!ok && lane == 0) {
        *abort_flag = 1;
        atomicOr(p.status, TXL_STATUS_TIMEOUT);
    }

    // ---- this warp's record ------------------------------------------------------
    // over the copies' stages (all of this group's items have landed and been read, and
    // with one node tile nobody else reads them), or over the scratch
    __syncwarp();
    Rec<ROWS> *mine = rec(warp);
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        st.l[r] += __shfl_xor_sync(0xffffffffu, st.l[r], 1);
        st.l[r] += __shfl_xor_sync(0xffffffffu, st.l[r], 2);
        if (t == 0) {
            mine->m[g + 8 * r] = __fmul_rn(st.m[r], scale);  // log2 units
            mine->l[g + 8 * r] = st.l[r];
        }
#pragma unroll
        for (int nd = 0; nd < 8; ++nd)
            *reinterpret_cast<float2 *>(&mine->a[g + 8 * r][8 * nd + 2 * t]) =
                make_float2(st.out(nd, r, 0), st.out(nd, r, 1));
    }
    finish<WARPS, KG, MT, __nv_bfloat16>(rec, p, b, h, n, warp, lane);
}

// The dynamic shared-memory attribute of the kernels, once per device.
cudaError_t ensure_attr()
{
    static bool done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
    const auto set = [](auto *k, int bytes) {
        return cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    };
    if ((e = set(relattn_tree_kernel<1, true>, Cfg<1>::SMEM)) != cudaSuccess) return e;
    if ((e = set(relattn_tree_kernel<1, false>, Cfg<1>::SMEM)) != cudaSuccess) return e;
    if ((e = set(relattn_tree_kernel<2, false>, Cfg<2>::SMEM)) != cudaSuccess) return e;
    if ((e = set(relattn_tree_kernel<4, false>, Cfg<4>::SMEM)) != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) done[dev] = true;
    return cudaSuccess;
}

} // namespace

// f(kernel, its shared memory, its index) for trees of N nodes.
template <typename F>
static auto with_kernel(int N, F f)
{
    if (N <= 8) return f(relattn_tree_kernel<1, true>, Cfg<1>::SMEM, 0);
    if (N <= 16) return f(relattn_tree_kernel<1, false>, Cfg<1>::SMEM, 1);
    if (N <= 32) return f(relattn_tree_kernel<2, false>, Cfg<2>::SMEM, 2);
    return f(relattn_tree_kernel<4, false>, Cfg<4>::SMEM, 3);
}

cudaError_t launch_relattn_tree(const CUtensorMap &tm_kv, const CUtensorMap &tm_r, const TreeParams &p,
                                cudaStream_t s)
{
    const cudaError_t e = ensure_attr();
    if (e != cudaSuccess) return e;
    return with_kernel(p.N, [&](auto *kern, int smem, int) {
        return launch_clusters(kern, p, THREADS, smem, s, tm_kv, tm_r, p);
    });
}

int tree_max_clusters(int N, int n_splits)
{
    static ClusterCache cache[4];
    if (ensure_attr() != cudaSuccess) return 0;
    return with_kernel(N, [&](auto *kern, int smem, int i) {
        return cache[i].get(n_splits, [&] { return max_clusters(kern, n_splits, THREADS, smem); });
    });
}

} // namespace txl
