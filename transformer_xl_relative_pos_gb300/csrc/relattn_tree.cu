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
// q and u (or v) enter as they are, one MMA each into the same accumulator: the
// scores are exact products summed in fp32.  P enters as two bf16 values (value and
// residual), to about 2^-17 relative, so that the output's own rounding is the one
// that shows.
//
// Copies: each key group has a ring of stages [32 k rows | 32 v rows | 32 table
// rows], three TMA boxes on one mbarrier, swizzled so that the matrix loads are
// conflict-free.  Pages are aligned to chunks: a box never crosses one.  Chunk
// rows outside the memory (where it begins and ends inside a tile) hold
// whatever the page holds: their scores are masked and their values, which
// may be NaN, are zeroed in the fragments.
//
// The nodes' own keys and values, and the table rows before a group's first
// chunk, are few: they go from global memory straight into fragments while
// the first copies are on their way.
#include "tree_common.cuh"

namespace txl {
namespace {

using namespace tree;

constexpr int ROWB = DH * 2;               // bytes of a row
constexpr int BOX = GK * ROWB;             // 4096: one 32-row box
constexpr int ST_K = 0, ST_V = BOX, ST_R = 2 * BOX;
constexpr int STAGE = 3 * BOX;             // 12288

template <int MT>
struct Cfg {
    static constexpr int KG = WARPS / MT;      // key groups of a block
    static constexpr int NSTG = MT == 1 ? 2 : MT == 2 ? 3 : 7;  // ring stages of a group
    static constexpr int DCAP = 16 * MT;       // depths are below this
    static constexpr int RW = GK + DCAP;       // columns of the product ring
    static constexpr int LD = RW + 8;          // its row stride (floats): 8 mod 16, so that the
                                               // quads' paired stores do not conflict
    static constexpr int SCR = 16 * LD * 4;    // bytes per warp
    static constexpr int OFF_SCR = KG * NSTG * STAGE;
    static constexpr int OFF_BAR = OFF_SCR + WARPS * SCR;  // full[KG][NSTG], empty[KG][NSTG]
    static constexpr int OFF_TOPO = OFF_BAR + 2 * KG * NSTG * 8;
    static constexpr int OFF_OK = OFF_TOPO + (int)sizeof(Topology);  // page of a stage valid
    static constexpr int OFF_FLAG = OFF_OK + KG * NSTG * 4;
    static constexpr int SMEM = OFF_FLAG + 16 + 1024;  // slack for the manual alignment
    // where a warp leaves its record: its private ring, or (shared ring) its scratch
    static_assert(MT == 1 || sizeof(Rec) <= SCR, "a warp's record fits in its scratch");
    static_assert(sizeof(Rec) <= NSTG * STAGE, "a warp's record fits in its ring");
    static_assert(OFF_BAR % 8 == 0 && OFF_TOPO % 8 == 0, "8-byte alignment");
    static_assert(2 * (SMEM + 1024) <= 228 * 1024, "two blocks per SM");
};

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
                 "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The same for an A operand whose 16 rows are alike.
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[2], uint32_t b0,
                                         uint32_t b1)
{
    const uint32_t rows[4] = {a[0], a[0], a[1], a[1]};
    mma16816(c, rows, b0, b1);
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

// Byte offset of 16-byte piece c of row `row` in a 128-byte-swizzled box.
__device__ __forceinline__ uint32_t swz(int row, int c)
{
    return (uint32_t)(row * ROWB + ((c ^ (row & 7)) << 4));
}

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// bf16 pair of (x0, x1), and in `res` the pair of what the rounding left over.
__device__ __forceinline__ uint32_t split_bf16x2(float x0, float x1, uint32_t &res)
{
    const uint32_t hi = pack_bf16x2(x0, x1);
    res = pack_bf16x2(x0 - bf_lo(hi), x1 - bf_hi(hi));
    return hi;
}

// A bf16 whose exponent bits are all ones (infinity or NaN) in either half.
__device__ __forceinline__ bool nonfinite2(uint32_t w)
{
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
}

// The running softmax and output of a warp's 16 nodes: this lane's rows are g and
// g + 8 (index 0, 1), its output columns 8 nd + 2 t, + 1.
struct State {
    float m[2], l[2];
    float acc[8][4];
};

// One chunk's masked scores s (log2 units; s[nt][e] of row g, s[nt][2 + e] of row
// g + 8, key 8 nt + 2 t + e) into probabilities, rescaling the state to the new maximum.
__device__ __forceinline__ void softmax_step(State &st, float (&s)[4][4])
{
    float mx[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        mx[r] = s[0][2 * r];
#pragma unroll
        for (int nt = 0; nt < 4; ++nt) {
            if (nt) mx[r] = max_nan(mx[r], s[nt][2 * r]);
            mx[r] = max_nan(mx[r], s[nt][2 * r + 1]);
        }
        mx[r] = max_nan(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 1));
        mx[r] = max_nan(mx[r], __shfl_xor_sync(0xffffffffu, mx[r], 2));
        mx[r] = max_nan(mx[r], st.m[r]);
    }
    // (a row without a visible key so far keeps maximum -inf: its sums are zero, and
    // the selects below leave them so)
    const bool moved = !(mx[0] == st.m[0]) || !(mx[1] == st.m[1]);
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const float f = st.m[r] == -INFINITY ? 0.f : ex2f(st.m[r] - mx[r]);
            st.m[r] = mx[r];
            st.l[r] *= f;
#pragma unroll
            for (int nd = 0; nd < 8; ++nd) {
                st.acc[nd][2 * r] *= f;
                st.acc[nd][2 * r + 1] *= f;
            }
        }
    }
#pragma unroll
    for (int nt = 0; nt < 4; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float x = s[nt][e];
            s[nt][e] = x == -INFINITY ? 0.f : ex2f(x - st.m[e >> 1]);
            st.l[e >> 1] += s[nt][e];
        }
}

// A operands of P.V for keys 16 kk .. 16 kk + 15 of a chunk, value and residual.
__device__ __forceinline__ void p_operand(const float (&s)[4][4], int kk, uint32_t (&hi)[4],
                                          uint32_t (&lo)[4])
{
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        hi[2 * c] = split_bf16x2(s[2 * kk + c][0], s[2 * kk + c][1], lo[2 * c]);
        hi[2 * c + 1] = split_bf16x2(s[2 * kk + c][2], s[2 * kk + c][3], lo[2 * c + 1]);
    }
}

template <int MT>
__global__ void __launch_bounds__(WARPS * 32, 2)
    relattn_tree_kernel(const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ CUtensorMap tm_r, const TreeParams p)
{
    using C = Cfg<MT>;
    constexpr int KG = C::KG, NSTG = C::NSTG, DCAP = C::DCAP, RW = C::RW, LD = C::LD;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int mt = warp % MT, kg = warp / MT;
    const int g = lane >> 2, t = lane & 3;
    const int split = blockIdx.x % p.n_splits;
    const int bh = blockIdx.x / p.n_splits;
    const int b = bh / p.mem.H, h = bh - b * p.mem.H;
    const int n = p.n_nodes ? min(max(p.n_nodes[b], 0), p.N) : p.N;
    if (n == 0) return;  // (every block of the cluster)

    uint8_t *ring = smem + kg * NSTG * STAGE;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + C::OFF_BAR) + kg * NSTG;
    uint64_t *empty = full + KG * NSTG;
    volatile int *stage_ok = reinterpret_cast<volatile int *>(smem + C::OFF_OK) + kg * NSTG;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + C::OFF_FLAG);
    Topology &topo = *reinterpret_cast<Topology *>(smem + C::OFF_TOPO);
    float *scr = reinterpret_cast<float *>(smem + C::OFF_SCR + warp * C::SCR);
    const bool leader = mt == 0 && lane == 0;  // issues its key group's copies
    if (threadIdx.x == 0) *abort_flag = 0;
    if (leader) {
        for (int s = 0; s < NSTG; ++s) {
            mbar_init(full + s, 1);
            mbar_init(empty + s, MT);
        }
        fence_barrier_init();
    }
    __syncthreads();

    int begin, fill;
    paged_state(p.mem, b, p.status, begin, fill);
    const Chunks ck = group_chunks(p, begin, fill, split * KG + kg, p.n_splits * KG);
    const uint64_t pol_stream = policy_evict_first();  // k, v: read once
    const uint64_t pol_keep = policy_evict_last();     // table: shared by the batch
    // Copies of this group's item into its stage.  Boxes are always complete (rows
    // past a tensor's ends arrive as zeros): a page id out of range becomes a plane
    // past the pool's end, and its rows are masked.
    auto issue = [&](int item) {
        const int c = ck.c0 + item, st = item % NSTG;
        int page, row;
        chunk_place(p.mem, ck, b, c, p.status, page, row);
        const int plane = page >= 0 ? page * p.mem.H + h : p.mem.n_pages * p.mem.H;
        stage_ok[st] = page >= 0;
        uint8_t *dst = ring + st * STAGE;
        mbar_arrive_expect_tx(full + st, (uint32_t)STAGE);
        tma_load_3d_hint(dst + ST_K, &tm_k, full + st, 0, row, plane, pol_stream);
        tma_load_3d_hint(dst + ST_V, &tm_v, full + st, 0, row, plane, pol_stream);
        tma_load_3d_hint(dst + ST_R, &tm_r, full + st, 0, p.r_rows - 1 - fill + c * GK - ck.off, h,
                         pol_keep);
    };
    int issued = 0;
    if (leader)
        for (; issued < min(NSTG, ck.count); ++issued) issue(issued);

    // A operands, dimensions 16 ks + 2 t, + 1 (registers 0, 1) and + 8, + 9 (2, 3): rows
    // g, g + 8 of the tile's q; u and v, alike in every row.
    uint32_t aq[4][4], au[4][2], av[4][2];
    {
        const __nv_bfloat16 *qb = static_cast<const __nv_bfloat16 *>(p.q.ptr) + b * p.q.sb + h * p.q.sh;
        const uint32_t *urow = reinterpret_cast<const uint32_t *>(static_cast<const __nv_bfloat16 *>(p.u) + h * DH);
        const uint32_t *vrow = reinterpret_cast<const uint32_t *>(static_cast<const __nv_bfloat16 *>(p.vb) + h * DH);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int w = 8 * ks + 4 * half + t;
                au[ks][half] = urow[w];
                av[ks][half] = vrow[w];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const int i = mt * 16 + g + 8 * r;
                    aq[ks][2 * half + r] =
                        i < n ? reinterpret_cast<const uint32_t *>(qb + i * p.q.sr)[w] : 0;
                }
            }
    }
    build_topology(topo, p.parents + b * p.parents_stride, n, p.status);
    const int i0 = mt * 16 + g, i1 = i0 + 8;  // this lane's nodes
    const int d0 = i0 < n ? topo.depth[i0] : 0, d1 = i1 < n ? topo.depth[i1] : 0;

    State st;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        st.m[r] = -INFINITY;
        st.l[r] = 0.f;
    }
#pragma unroll
    for (int nd = 0; nd < 8; ++nd)
#pragma unroll
        for (int e = 0; e < 4; ++e) st.acc[nd][e] = 0.f;

    // Products (q + v).r of 8 table rows from global memory (rows outside the table:
    // zero) into ring columns col .. col + 7.
    const __nv_bfloat16 *table = static_cast<const __nv_bfloat16 *>(p.r) + (long long)h * p.r_rows * DH;
    auto table_tile = [&](int row0, int col) {
        const int row = row0 + g;
        uint32_t w[8];
#pragma unroll
        for (int x = 0; x < 8; ++x) w[x] = 0;
        if (row >= 0 && row < p.r_rows) {
            const uint32_t *src = reinterpret_cast<const uint32_t *>(table + (long long)row * DH);
#pragma unroll
            for (int x = 0; x < 8; ++x) w[x] = __ldg(src + 4 * x + t);
        }
        float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
            mma16816(c, aq[ks], w[2 * ks], w[2 * ks + 1]);
            mma16816(c, av[ks], w[2 * ks], w[2 * ks + 1]);
        }
        TXL_CHECK(col >= 0 && col + 8 <= RW, p.status);
        *reinterpret_cast<float2 *>(scr + g * LD + col + 2 * t) = make_float2(c[0], c[1]);
        *reinterpret_cast<float2 *>(scr + (g + 8) * LD + col + 2 * t) = make_float2(c[2], c[3]);
    };
    // P.V of one chunk, element by element: for a chunk whose keys are not all
    // visible to the same nodes and whose values hold an infinity or NaN, which must
    // not reach the nodes that do not see the key.  hidden: bit 4 nt + e of this lane's
    // elements.  col0: 32 free ring columns.
    auto pv_by_element = [&](const float (&s)[4][4], uint32_t hidden, int col0, auto &&value) {
        auto at = [&](int key) { const int c = col0 + key; return c >= RW ? c - RW : c; };
        __syncwarp();
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                scr[(g + 8 * (e >> 1)) * LD + at(8 * nt + 2 * t + (e & 1))] =
                    (hidden >> (4 * nt + e)) & 1 ? -1.f : s[nt][e];
        __syncwarp();
        for (int key = 0; key < GK; ++key) {
            const float p0 = scr[g * LD + at(key)], p1 = scr[(g + 8) * LD + at(key)];
#pragma unroll
            for (int nd = 0; nd < 8; ++nd)
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float x = value(key, 8 * nd + 2 * t + e);
                    if (!(p0 < 0.f)) st.acc[nd][e] = fmaf(p0, x, st.acc[nd][e]);
                    if (!(p1 < 0.f)) st.acc[nd][2 + e] = fmaf(p1, x, st.acc[nd][2 + e]);
                }
        }
        __syncwarp();
    };

    const bool active = mt * 16 < n;  // this warp has nodes
    if (active && split == p.n_splits - 1 && kg == 0) {
        // ---- the nodes among themselves: distances 0 .. DCAP - 1 ------------------
        for (int c = 0; c < DCAP; c += 8) table_tile(p.r_rows - DCAP + c, c);
        __syncwarp();
        const unsigned long long anc0 = i0 < n ? topo.anc[i0] : 0, anc1 = i1 < n ? topo.anc[i1] : 0;
        const __nv_bfloat16 *kn = static_cast<const __nv_bfloat16 *>(p.k.ptr) + b * p.k.sb + h * p.k.sh;
        const __nv_bfloat16 *vn = static_cast<const __nv_bfloat16 *>(p.v.ptr) + b * p.v.sb + h * p.v.sh;
        // (no node is an ancestor of an earlier one: this tile's nodes see nodes up to their own)
        const int a_end = min(n, mt * 16 + 16);
        for (int a0 = 0; a0 < a_end; a0 += GK) {
            float s[4][4];
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                const int row = a0 + 8 * nt + g;
                uint32_t w[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) w[x] = 0;
                if (row < a_end) {
                    const uint32_t *src = reinterpret_cast<const uint32_t *>(kn + row * p.k.sr);
#pragma unroll
                    for (int x = 0; x < 8; ++x) w[x] = src[4 * x + t];
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
                    mma16816(s[nt], aq[ks], w[2 * ks], w[2 * ks + 1]);
                    mma16816(s[nt], au[ks], w[2 * ks], w[2 * ks + 1]);
                }
            }
            uint32_t hidden = 0;
#pragma unroll
            for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int a = a0 + 8 * nt + 2 * t + (e & 1);
                    const int dist = (e < 2 ? d0 : d1) - (a < n ? topo.depth[a] : 0);
                    const bool seen = a < n && (((e < 2 ? anc0 : anc1) >> a) & 1) && dist < p.r_rows;
                    TXL_CHECK(!seen || (dist >= 0 && dist < DCAP), p.status);
                    hidden |= seen ? 0u : 1u << (4 * nt + e);
                    s[nt][e] = seen ? (s[nt][e] + scr[(g + 8 * (e >> 1)) * LD + DCAP - 1 - dist]) * p.scale_log2
                                    : -INFINITY;
                }
            softmax_step(st, s);
            // V fragments: key rows 16 kk + 2 t, + 1 (and + 8, + 9), column 8 nd + g
            uint32_t vw[2][8][2];
            bool bad = false;
#pragma unroll
            for (int kk = 0; kk < 2; ++kk)
#pragma unroll
                for (int nd = 0; nd < 8; ++nd)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int key = a0 + 16 * kk + 8 * x + 2 * t;
                        const __nv_bfloat16 *src = vn + key * p.v.sr + 8 * nd + g;
                        uint32_t w = 0;
                        if (key < a_end) w = __bfloat16_as_ushort(src[0]);
                        if (key + 1 < a_end) w |= (uint32_t)__bfloat16_as_ushort(src[p.v.sr]) << 16;
                        vw[kk][nd][x] = w;
                        bad |= nonfinite2(w);
                    }
            if (__any_sync(0xffffffffu, bad)) {
                pv_by_element(s, hidden, DCAP, [&](int key, int dim) {
                    return a0 + key < a_end ? __bfloat162float(vn[(a0 + key) * p.v.sr + dim]) : 0.f;
                });
                continue;
            }
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                uint32_t hi[4], lo[4];
                p_operand(s, kk, hi, lo);
#pragma unroll
                for (int nd = 0; nd < 8; ++nd) {
                    mma16816(st.acc[nd], hi, vw[kk][nd][0], vw[kk][nd][1]);
                    mma16816(st.acc[nd], lo, vw[kk][nd][0], vw[kk][nd][1]);
                }
            }
        }
        __syncwarp();  // the ring's columns are free again
    }
    if (active && ck.count > 0)  // the DCAP table rows before the first chunk's
        for (int c = 0; c < DCAP; c += 8)
            table_tile(p.r_rows - 1 - fill + ck.c0 * GK - ck.off - DCAP + c, c);

    // ---- the memory, chunk by chunk ---------------------------------------------
    const int lr = lane & 7, lm = lane >> 3;  // matrix-load roles: row, matrix
    const int depth_max = __reduce_max_sync(0xffffffffu, max(d0, d1));
    int wpos = DCAP;                          // ring column of the chunk's first table row
    bool ok = true;
    for (int item = 0; item < ck.count; ++item) {
        const int stg = item % NSTG;
        ok = __all_sync(0xffffffffu, mbar_wait(full + stg, (item / NSTG) & 1, abort_flag, p.wait_ns));
        if (!ok) break;
        if (active) {
            const uint8_t *base = ring + stg * STAGE;
            const uint32_t sk = smem_u32(base + ST_K), sv = smem_u32(base + ST_V), sr = smem_u32(base + ST_R);
            const int j0 = (ck.c0 + item) * GK - ck.off;  // memory row of the chunk's first key

            // content and position products
            float s[4][4];
#pragma unroll
            for (int nt = 0; nt < 4; ++nt) {
                const int row = 8 * nt + lr;
                float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int e = 0; e < 4; ++e) s[nt][e] = 0.f;
#pragma unroll
                for (int h2 = 0; h2 < 2; ++h2) {
                    uint32_t bk[4], br[4];
                    ldsm_x4(bk, sk + swz(row, 4 * h2 + lm));
                    ldsm_x4(br, sr + swz(row, 4 * h2 + lm));
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int ks = 2 * h2 + x;
                        mma16816(s[nt], aq[ks], bk[2 * x], bk[2 * x + 1]);
                        mma16816(c, aq[ks], br[2 * x], br[2 * x + 1]);
                        mma16816(s[nt], au[ks], bk[2 * x], bk[2 * x + 1]);
                        mma16816(c, av[ks], br[2 * x], br[2 * x + 1]);
                    }
                }
                int col = wpos + 8 * nt;
                col -= col >= RW ? RW : 0;
                TXL_CHECK(col >= 0 && col + 8 <= RW, p.status);
                *reinterpret_cast<float2 *>(scr + g * LD + col + 2 * t) = make_float2(c[0], c[1]);
                *reinterpret_cast<float2 *>(scr + (g + 8) * LD + col + 2 * t) = make_float2(c[2], c[3]);
            }
            __syncwarp();
            // scores: the position product of key jj and a node of depth d stands
            // d columns before the chunk's own column jj
#pragma unroll
            for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    int col = wpos + 8 * nt + 2 * t + (e & 1) - (e < 2 ? d0 : d1);
                    col += col < 0 ? RW : 0;
                    col -= col >= RW ? RW : 0;
                    TXL_CHECK(col >= 0 && col < RW, p.status);
                    s[nt][e] = (s[nt][e] + scr[(g + 8 * (e >> 1)) * LD + col]) * p.scale_log2;
                }
            // Keys that are not memory rows (the chunk sticks out at either end, or its
            // page is unknown) or that the table does not reach from the node.
            const bool page_ok = stage_ok[stg] != 0;
            const bool out_of_memory = j0 < 0 || j0 + GK > fill || !page_ok;
            const bool partly_hidden = j0 < fill + depth_max - p.r_rows + 1;
            uint32_t hidden = 0;
            if (out_of_memory || partly_hidden) {
                const int lo0 = max(0, fill + d0 - p.r_rows + 1) - j0;
                const int lo1 = max(0, fill + d1 - p.r_rows + 1) - j0;
                const int hi = page_ok ? fill - j0 : 0;
#pragma unroll
                for (int nt = 0; nt < 4; ++nt)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int jj = 8 * nt + 2 * t + (e & 1);
                        if (jj < (e < 2 ? lo0 : lo1) || jj >= hi) {
                            s[nt][e] = -INFINITY;
                            hidden |= 1u << (4 * nt + e);
                        }
                    }
            }
            softmax_step(st, s);
            // P.V
            const int key_lo = -j0, key_hi = page_ok ? fill - j0 : 0;  // memory rows of the chunk
            bool bad = false;
            if (partly_hidden) {
                // lane = key: does a memory row hold an infinity or NaN
                if (lane >= key_lo && lane < key_hi) {
#pragma unroll 1
                    for (int x = 0; x < 8; ++x) {
                        const uint4 w = *reinterpret_cast<const uint4 *>(base + ST_V + swz(lane, x));
                        bad |= nonfinite2(w.x) | nonfinite2(w.y) | nonfinite2(w.z) | nonfinite2(w.w);
                    }
                }
                bad = __any_sync(0xffffffffu, bad);
            }
            int next = wpos + GK;
            next -= next >= RW ? RW : 0;
            if (bad) {
                pv_by_element(s, hidden, next, [&](int key, int dim) {
                    const uint8_t *at = base + ST_V + swz(key, dim >> 3) + 2 * (dim & 7);
                    return __bfloat162float(*reinterpret_cast<const __nv_bfloat16 *>(at));
                });
            } else {
#pragma unroll
                for (int kk = 0; kk < 2; ++kk) {
                    uint32_t hi[4], lo[4];
                    p_operand(s, kk, hi, lo);
                    uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
                    if (out_of_memory) {
                        // this lane's fragment rows: keys 16 kk + 2 t, + 1 and + 8, + 9
                        const int key = 16 * kk + 2 * t;
                        auto in = [&](int x) { return x >= key_lo && x < key_hi; };
                        keep0 = (in(key) ? 0xffffu : 0u) | (in(key + 1) ? 0xffff0000u : 0u);
                        keep1 = (in(key + 8) ? 0xffffu : 0u) | (in(key + 9) ? 0xffff0000u : 0u);
                    }
                    const int row = 16 * kk + (lm & 1) * 8 + lr;
#pragma unroll
                    for (int np = 0; np < 4; ++np) {
                        uint32_t bv[4];
                        ldsm_x4_t(bv, sv + swz(row, 2 * np + (lm >> 1)));
                        if (out_of_memory) {
                            bv[0] &= keep0;
                            bv[1] &= keep1;
                            bv[2] &= keep0;
                            bv[3] &= keep1;
                        }
                        mma16816(st.acc[2 * np], hi, bv[0], bv[1]);
                        mma16816(st.acc[2 * np + 1], hi, bv[2], bv[3]);
                        mma16816(st.acc[2 * np], lo, bv[0], bv[1]);
                        mma16816(st.acc[2 * np + 1], lo, bv[2], bv[3]);
                    }
                }
            }
            wpos = next;
        }
        // The stage is read: order this lane's reads before the copy that refills it.
        fence_proxy_async_smem();
        __syncwarp();
        if constexpr (MT == 1) {
            if (item + NSTG < ck.count) {
                if (lane == 0) issue(item + NSTG);
                ++issued;
            }
        } else {
            // The group's other warps may lag: refill the previous item's stage, once
            // all have left it.
            if (lane == 0) mbar_arrive(empty + stg);
            if (item > 0 && item - 1 + NSTG < ck.count) {
                if (leader) {
                    const int prev = item - 1;
                    if (mbar_wait(empty + prev % NSTG, (prev / NSTG) & 1, abort_flag, p.wait_ns)) {
                        issue(prev + NSTG);
                        ++issued;
                    } else {
                        ok = false;
                    }
                }
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) break;
            }
        }
    }
    if (!ok) {
        // Time-out: record it, and let this group's copies in flight land before the
        // block's shared memory is used for anything else or released.
        if (lane == 0) {
            *abort_flag = 1;
            atomicOr(p.status, TXL_STATUS_TIMEOUT);
            const int zero = 0;
            if (leader)
                for (int x = max(0, issued - NSTG); x < issued; ++x)
                    mbar_wait(full + x % NSTG, (x / NSTG) & 1, &zero, p.wait_ns);
        }
        __syncwarp();
    }

    // ---- this warp's record ------------------------------------------------------
    const auto rec = [smem](int w) {
        return reinterpret_cast<Rec *>(MT == 1 ? smem + w * NSTG * STAGE : smem + C::OFF_SCR + w * C::SCR);
    };
    __syncwarp();
    Rec *mine = rec(warp);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
        st.l[r] += __shfl_xor_sync(0xffffffffu, st.l[r], 1);
        st.l[r] += __shfl_xor_sync(0xffffffffu, st.l[r], 2);
        if (t == 0) {
            mine->m[g + 8 * r] = st.m[r];
            mine->l[g + 8 * r] = st.l[r];
        }
#pragma unroll
        for (int nd = 0; nd < 8; ++nd)
            *reinterpret_cast<float2 *>(&mine->a[g + 8 * r][8 * nd + 2 * t]) =
                make_float2(st.acc[nd][2 * r], st.acc[nd][2 * r + 1]);
    }
    finish<MT, __nv_bfloat16>(rec, p, b, h, n, warp, lane);
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
    if ((e = set(relattn_tree_kernel<1>, Cfg<1>::SMEM)) != cudaSuccess) return e;
    if ((e = set(relattn_tree_kernel<2>, Cfg<2>::SMEM)) != cudaSuccess) return e;
    if ((e = set(relattn_tree_kernel<4>, Cfg<4>::SMEM)) != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) done[dev] = true;
    return cudaSuccess;
}

} // namespace

cudaError_t launch_relattn_tree(const CUtensorMap &tm_k, const CUtensorMap &tm_v,
                                const CUtensorMap &tm_r, const TreeParams &p, cudaStream_t s)
{
    const cudaError_t e = ensure_attr();
    if (e != cudaSuccess) return e;
    if (p.N <= 16) return launch_clusters(relattn_tree_kernel<1>, p, Cfg<1>::SMEM, s, tm_k, tm_v, tm_r, p);
    if (p.N <= 32) return launch_clusters(relattn_tree_kernel<2>, p, Cfg<2>::SMEM, s, tm_k, tm_v, tm_r, p);
    return launch_clusters(relattn_tree_kernel<4>, p, Cfg<4>::SMEM, s, tm_k, tm_v, tm_r, p);
}

} // namespace txl
