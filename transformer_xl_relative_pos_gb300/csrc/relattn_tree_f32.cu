// Relative-position attention of a tree of drafted tokens over a paged memory in
// fp32 on the CUDA cores (FFMA, no TF32): the exact path, as relattn_f32.cu is for
// dense segments.  "Transformer-XL: Attentive Language Models Beyond a Fixed-Length
// Context", §3.3 score, Appendix B reversed table; the shift by the nodes' depths
// and the split of the keys are those of relattn_tree.cu.
//
// Per key, head and node it computes 3 x 64 multiply-adds; reading 512 bytes of k
// and v for them, it is bound by those products from a few nodes on.  Each row that
// many products share sits in registers, the other operand comes from shared
// memory four floats at a time:
//   scores   lane = key: the lane's k row (then its table row) against the warp's
//            nodes, whose q + u (q + v) every lane reads alike
//   P.V      lane = two dimensions of 32 value rows, against the probabilities,
//            which every lane reads alike
#include "tree_common.cuh"

namespace txl {
namespace {

using namespace tree;

constexpr int WARPS = 8, ROWS = 8;   // warps of a block, nodes of a warp
constexpr int MAX_MT = kTreeMaxNodes / ROWS;
constexpr int SLD = DH + 4;          // row stride of staged rows (floats): a lane's own row is then
                                     // read without bank conflicts, four floats at a time

template <int MT>
struct CfgF32 {
    static constexpr int DCAP = ROWS * MT;     // depths are below this
    static constexpr int RW = GK + DCAP;       // columns of the product ring
    static constexpr int Q = MT * 2 * ROWS * DH;  // floats: q + u, q + v of the nodes
    // floats per warp: ring, probabilities, 32 rows on their way to the lanes
    static constexpr int WARP = ROWS * RW + ROWS * GK + GK * SLD;
    static constexpr int REC = (int)sizeof(Rec<ROWS>);  // a warp's record goes over them
    static constexpr int OFF_WARP = Q * 4;
    static constexpr int STEP = WARP * 4 > REC ? WARP * 4 : REC;  // bytes per warp
    static constexpr int OFF_TOPO = OFF_WARP + WARPS * STEP;
    static constexpr int SMEM = OFF_TOPO + (int)sizeof(Topology);
    static_assert(SMEM <= 232448, "shared memory budget exceeded");
    static_assert(OFF_TOPO % 16 == 0 && OFF_WARP % 16 == 0 && STEP % 16 == 0, "alignment");
};

template <int MT>
__global__ void __launch_bounds__(WARPS * 32) relattn_tree_f32_kernel(const TreeParams p)
{
    using C = CfgF32<MT>;
    constexpr int KG = WARPS / MT, DCAP = C::DCAP, RW = C::RW;
    extern __shared__ __align__(16) uint8_t smem_f32[];
    uint8_t *smem = smem_f32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int mt = warp % MT, kg = warp / MT;
    const int split = blockIdx.x % p.n_splits;
    const int bh = blockIdx.x / p.n_splits;
    const int rank = bh / p.mem.H, h = bh - rank * p.mem.H;
    const int b = pick_sequence(p, rank, reinterpret_cast<int *>(smem + C::OFF_TOPO));
    const int n = p.n_nodes ? min(max(p.n_nodes[b], 0), p.N) : p.N;
    if (n == 0) return;  // (every block of the cluster)
    const int parent = threadIdx.x < n ? p.parents[b * p.parents_stride + threadIdx.x] : -1;

    float *qs = reinterpret_cast<float *>(smem);
    float *ring = reinterpret_cast<float *>(smem + C::OFF_WARP + warp * C::STEP);
    float *prob = ring + ROWS * RW, *rows32 = prob + ROWS * GK;
    Topology &topo = *reinterpret_cast<Topology *>(smem + C::OFF_TOPO);

    // q + u and q + v of the nodes (those past n: zero)
    for (int e = threadIdx.x; e < MT * ROWS * DH; e += WARPS * 32) {
        const int i = e / DH, c = e % DH;
        const float *q = static_cast<const float *>(p.q.ptr) + b * p.q.sb + h * p.q.sh + i * p.q.sr;
        const float x = i < n ? q[c] : 0.f;
        float *dst = qs + (i / ROWS) * (2 * ROWS * DH) + (i % ROWS) * DH + c;
        dst[0] = x + static_cast<const float *>(p.u)[h * DH + c];
        dst[ROWS * DH] = x + static_cast<const float *>(p.vb)[h * DH + c];
    }
    build_topology(topo, parent, n, p.status);

    int begin, fill;
    paged_state(p.mem, b, p.status, begin, fill);
    const Chunks ck = group_chunks(p, begin, fill, kNodesCost, split * KG + kg, p.n_splits * KG);
    const int rows = min(ROWS, n - mt * ROWS);  // this warp's nodes (none: <= 0)
    const float4 *qu = reinterpret_cast<const float4 *>(qs + mt * (2 * ROWS * DH));
    const float4 *qv = qu + ROWS * DH / 4;
    const float *table = static_cast<const float *>(p.r) + (long long)h * p.r_rows * DH;

    float m[ROWS], l[ROWS], acc[ROWS][2];  // l: this lane's keys only
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        m[i] = -INFINITY;
        l[i] = acc[i][0] = acc[i][1] = 0.f;
    }
    int depth_max = 0;
    for (int i = 0; i < rows; ++i) depth_max = max(depth_max, topo.depth[mt * ROWS + i]);

    // Dot products of the warp's nodes with one row per lane, row(x) of 32 (null: zero).
    // The rows are read in order, half a warp a row, and handed out through shared
    // memory: a lane reading its own row would touch 32 lines at a time.
    auto dots = [&](auto &&row, const float4 *q, float (&out)[ROWS]) {
        float4 x[DH / 4];
#pragma unroll
        for (int c = 0; c < DH / 4; ++c) {
            const float *src = row(2 * c + (lane >> 4));
            x[c] = src ? __ldg(reinterpret_cast<const float4 *>(src) + (lane & 15))
                       : make_float4(0.f, 0.f, 0.f, 0.f);
        }
#pragma unroll
        for (int c = 0; c < DH / 4; ++c)
            *reinterpret_cast<float4 *>(rows32 + (2 * c + (lane >> 4)) * SLD + 4 * (lane & 15)) = x[c];
        __syncwarp();
#pragma unroll
        for (int c = 0; c < DH / 4; ++c) x[c] = *reinterpret_cast<const float4 *>(rows32 + lane * SLD + 4 * c);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            if (i >= rows) break;
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int c = 0; c < DH / 4; ++c) {
                const float4 a = q[i * (DH / 4) + c];
                s0 = fmaf(a.x, x[c].x, s0);
                s1 = fmaf(a.y, x[c].y, s1);
                s0 = fmaf(a.z, x[c].z, s0);
                s1 = fmaf(a.w, x[c].w, s1);
            }
            out[i] = s0 + s1;
        }
    };
    // (q + v).r of table rows row0 .. row0 + 31 (outside the table: zero); this lane's into
    // ring column col, when keep
    auto table_dots = [&](int row0, int col, bool keep) {
        float c[ROWS];
        dots([&](int x) { return row0 + x >= 0 && row0 + x < p.r_rows ? table + (long long)(row0 + x) * DH : nullptr; },
             qv, c);
        TXL_CHECK(!keep || (col >= 0 && col < RW), p.status);
#pragma unroll
        for (int i = 0; i < ROWS; ++i)
            if (i < rows && keep) ring[i * RW + col] = c[i];
    };
    // Masked scores (log2 units) of this lane's key into the running softmax, then
    // P.V over the chunk's value rows.  value(key): the row, or null (zero).  mixed: keys
    // may be hidden from some nodes only (bit i of this lane's `hidden`); the value,
    // which may be an infinity or NaN, then must not reach them.
    auto step = [&](float (&s)[ROWS], bool mixed, unsigned hidden, auto &&value) {
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            if (i >= rows) break;
            float mx = s[i];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            mx = max_nan(mx, m[i]);
            if (!(mx == m[i])) {
                const float f = m[i] == -INFINITY ? 0.f : ex2f(m[i] - mx);
                m[i] = mx;
                l[i] *= f;
                acc[i][0] *= f;
                acc[i][1] *= f;
            }
            const float e = s[i] == -INFINITY ? 0.f : ex2f(s[i] - mx);
            l[i] += e;
            prob[i * GK + lane] = (hidden >> i) & 1 ? -1.f : e;
        }
        float2 v[GK];
#pragma unroll
        for (int key = 0; key < GK; ++key) {
            const float *row = value(key);
            v[key] = row ? __ldg(reinterpret_cast<const float2 *>(row) + lane) : make_float2(0.f, 0.f);
        }
        __syncwarp();
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            if (i >= rows) break;
#pragma unroll
            for (int c = 0; c < GK / 4; ++c) {
                const float4 e = *reinterpret_cast<const float4 *>(prob + i * GK + 4 * c);
                const float w[4] = {e.x, e.y, e.z, e.w};
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    if (mixed && w[x] < 0.f) continue;
                    acc[i][0] = fmaf(w[x], v[4 * c + x].x, acc[i][0]);
                    acc[i][1] = fmaf(w[x], v[4 * c + x].y, acc[i][1]);
                }
            }
        }
        __syncwarp();
    };

    if (rows > 0 && split == p.n_splits - 1 && kg == KG - 1) {
        // ---- the nodes among themselves: distances 0 .. DCAP - 1 ------------------
        for (int c = 0; c < DCAP; c += 32) table_dots(p.r_rows - DCAP + c, c + lane, c + lane < DCAP);
        __syncwarp();
        const float *kn = static_cast<const float *>(p.k.ptr) + b * p.k.sb + h * p.k.sh;
        const float *vn = static_cast<const float *>(p.v.ptr) + b * p.v.sb + h * p.v.sh;
        const int a_end = mt * ROWS + rows;  // (no node is an ancestor of an earlier one)
        for (int a0 = 0; a0 < a_end; a0 += GK) {
            const int a = a0 + lane;
            float s[ROWS];
            dots([&](int x) { return a0 + x < a_end ? kn + (a0 + x) * p.k.sr : nullptr; }, qu, s);
            const int da = a < a_end ? topo.depth[a] : 0;
            unsigned hidden = 0;
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
                if (i >= rows) break;
                const int dist = topo.depth[mt * ROWS + i] - da;
                const bool seen = a < a_end && ((topo.anc[mt * ROWS + i] >> a) & 1) && dist < p.r_rows;
                TXL_CHECK(!seen || (dist >= 0 && dist < DCAP), p.status);
                hidden |= seen ? 0u : 1u << i;
                s[i] = seen ? (s[i] + ring[i * RW + DCAP - 1 - dist]) * p.scale_log2 : -INFINITY;
            }
            step(s, true, hidden, [&](int key) { return a0 + key < a_end ? vn + (a0 + key) * p.v.sr : nullptr; });
        }
    }
    if (rows > 0 && ck.count > 0)  // the DCAP table rows before the first chunk's
        for (int c = 0; c < DCAP; c += 32)
            table_dots(p.r_rows - 1 - fill + ck.c0 * GK - ck.off - DCAP + c, c + lane,
                       c + lane < DCAP);

    // ---- the memory, chunk by chunk ---------------------------------------------
    int wpos = DCAP;  // ring column of the chunk's first table row
    int slot = ck.slot, row = ck.row, page = ck.count > 0 ? page_at(p.mem, b, slot, p.status) : -1;
    for (int item = 0; item < (rows > 0 ? ck.count : 0); ++item) {
        const int c = ck.c0 + item, j0 = c * GK - ck.off;
        const long long at = page >= 0 ? (((long long)page * p.mem.H + h) * p.mem.P + row) * DH : 0;
        const float *kp = static_cast<const float *>(p.kpage) + at;
        const float *vp = static_cast<const float *>(p.vpage) + at;
        const int key_lo = -j0, key_hi = page >= 0 ? fill - j0 : 0;  // memory rows of the chunk
        const bool mine = lane >= key_lo && lane < key_hi;
        float s[ROWS];
        dots([&](int x) { return x >= key_lo && x < key_hi ? kp + x * DH : nullptr; }, qu, s);
        int col = wpos + lane;
        col -= col >= RW ? RW : 0;
        table_dots(p.r_rows - 1 - fill + j0, col, true);
        __syncwarp();
        const int reach = fill - p.r_rows - j0;  // depth d sees keys above reach + d
        const bool mixed = reach + depth_max >= 0;
        unsigned hidden = 0;
#pragma unroll
        for (int i = 0; i < ROWS; ++i) {
            if (i >= rows) break;
            const int d = topo.depth[mt * ROWS + i];
            int x = wpos + lane - d;
            x += x < 0 ? RW : 0;
            x -= x >= RW ? RW : 0;
            const bool seen = mine && lane > reach + d;
            hidden |= mixed && !seen ? 1u << i : 0u;  // (else a missing key's zero value is harmless)
            s[i] = seen ? (s[i] + ring[i * RW + x]) * p.scale_log2 : -INFINITY;
        }
        step(s, mixed, hidden,
             [&](int key) { return key >= key_lo && key < key_hi ? vp + key * DH : nullptr; });
        wpos += GK;
        wpos -= wpos >= RW ? RW : 0;
        if (next_chunk(p.mem, slot, row) && item + 1 < ck.count) page = page_at(p.mem, b, slot, p.status);
    }

    // ---- this warp's record, over its ring ----------------------------------------
    const auto rec = [smem](int w) {
        return reinterpret_cast<Rec<ROWS> *>(smem + C::OFF_WARP + w * C::STEP);
    };
    __syncwarp();
    Rec<ROWS> *r = rec(warp);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        if (i >= rows) break;
        float sum = l[i];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0) {
            r->m[i] = m[i];
            r->l[i] = sum;
        }
        reinterpret_cast<float2 *>(r->a[i])[lane] = make_float2(acc[i][0], acc[i][1]);
    }
    finish<WARPS, KG, MT, float>(rec, p, b, h, n, warp, lane);
}

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
    if ((e = set(relattn_tree_f32_kernel<1>, CfgF32<1>::SMEM)) != cudaSuccess) return e;
    if ((e = set(relattn_tree_f32_kernel<2>, CfgF32<2>::SMEM)) != cudaSuccess) return e;
    if ((e = set(relattn_tree_f32_kernel<4>, CfgF32<4>::SMEM)) != cudaSuccess) return e;
    if ((e = set(relattn_tree_f32_kernel<MAX_MT>, CfgF32<MAX_MT>::SMEM)) != cudaSuccess) return e;
    if (dev >= 0 && dev < 64) done[dev] = true;
    return cudaSuccess;
}

} // namespace

// f(kernel, its shared memory, its index) for trees of N nodes.
template <typename F>
static auto with_kernel(int N, F f)
{
    const int mt = (N + ROWS - 1) / ROWS;
    if (mt <= 1) return f(relattn_tree_f32_kernel<1>, CfgF32<1>::SMEM, 0);
    if (mt <= 2) return f(relattn_tree_f32_kernel<2>, CfgF32<2>::SMEM, 1);
    if (mt <= 4) return f(relattn_tree_f32_kernel<4>, CfgF32<4>::SMEM, 2);
    return f(relattn_tree_f32_kernel<MAX_MT>, CfgF32<MAX_MT>::SMEM, 3);
}

cudaError_t launch_relattn_tree_f32(const TreeParams &p, cudaStream_t s)
{
    const cudaError_t e = ensure_attr();
    if (e != cudaSuccess) return e;
    return with_kernel(p.N, [&](auto *kern, int smem, int) {
        return launch_clusters(kern, p, WARPS * 32, smem, s, p);
    });
}

int tree_max_clusters_f32(int N, int n_splits)
{
    static ClusterCache cache[4];
    if (ensure_attr() != cudaSuccess) return 0;
    return with_kernel(N, [&](auto *kern, int smem, int i) {
        return cache[i].get(n_splits, [&] { return max_clusters(kern, n_splits, WARPS * 32, smem); });
    });
}

} // namespace txl
