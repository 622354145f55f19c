// Relative-position attention of a tree of drafted tokens over a paged memory in
// fp32 on the CUDA cores (FFMA, no TF32): the exact path, as relattn_f32.cu is for
// dense segments.  "Transformer-XL: Attentive Language Models Beyond a Fixed-Length
// Context", §3.3 score, Appendix B reversed table; the shift by the nodes' depths
// and the split of the keys are those of relattn_tree.cu.
//
// Per key, head and node it computes 3 x 64 multiply-adds; reading 512 bytes of k
// and v for them, it is bound by those products from a few nodes on.  A warp has
// ROWS = 4, 8 or 16 nodes and takes 32 keys at a time, whose rows it stages in its own
// shared memory; a lane then keeps a register tile, four floats per load:
//   scores   ROWS / 4 nodes x 4 keys, 16 steps of 4 dimensions
//   P.V      ROWS / 4 nodes x 8 dimensions, 8 steps of 4 keys
// With 16 nodes that is eight loads for 64 multiply-adds.  Row strides of 4 mod 32 floats keep
// the loads free of bank conflicts.  Measured: 13 nodes, two sequences of 8 heads and up to 777
// rows 17.2 us, 14.7 when the memory is in L2 (a lane per key, without register tiles, 29); 64
// nodes, six sequences of 16 heads and 1500 rows 158 us, 153 in L2 (455 without), 23 TFLOP/s: a third of the CUDA cores' rate, the
// operands' loads and the staging between the products taking the rest.
#include "tree_common.cuh"

namespace txl {
namespace {

using namespace tree;

constexpr int WARPS = 4;
constexpr int SLD = DH + 4;                    // stride of staged rows and of q (floats)
constexpr int PLD = GK + 4;                    // stride of the probabilities

template <int MT_, int ROWS_>
struct CfgF32 {
    static constexpr int MT = MT_, ROWS = ROWS_, KG = WARPS / MT;
    static constexpr int NODES = MT * ROWS;
    static_assert(KG == tree_key_groups(NODES), "as the choice of key ranges has it");
    static constexpr int DCAP = NODES;         // depths are below this
    static constexpr int RW = GK + DCAP;       // columns of the product ring
    static constexpr int Q = 2 * NODES * SLD;  // floats: q + u, q + v of the nodes
    // floats per warp: the staged rows, the ring, the probabilities
    static constexpr int RING = GK * SLD, PROB = RING + ROWS * RW, WARP = PROB + ROWS * PLD;
    using WarpRec = Rec<ROWS>;                 // a warp's record, over them
    static constexpr int OFF_WARP = Q * 4;
    static constexpr int OFF_TOPO = OFF_WARP + WARPS * WARP * 4;
    static constexpr int SMEM = OFF_TOPO + (int)sizeof(Topology);
    static_assert(sizeof(WarpRec) <= WARP * 4, "a warp's record fits");
    static_assert(SMEM <= 232448, "shared memory budget exceeded");
    static_assert(OFF_TOPO % 16 == 0 && RING % 4 == 0 && PROB % 4 == 0 && WARP % 4 == 0, "alignment");
};

__device__ __forceinline__ float4 f4(const float *p) { return *reinterpret_cast<const float4 *>(p); }

template <int MT, int ROWS>
__global__ void __launch_bounds__(WARPS * 32, 2) relattn_tree_f32_kernel(const TreeParams p)
{
    using C = CfgF32<MT, ROWS>;
    constexpr int KG = C::KG, DCAP = C::DCAP, RW = C::RW;
    constexpr int XN = ROWS / 4;               // nodes of a lane: quad + 4 x
    extern __shared__ __align__(16) uint8_t smem_f32[];
    uint8_t *smem = smem_f32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int mt = warp % MT, kg = warp / MT;
    const int oct = lane & 7, quad = lane >> 3;  // keys oct + 8 y, or dimensions 4 oct + 32 z; nodes quad + 4 x
    const int split = blockIdx.x % p.n_splits;
    const int bh = blockIdx.x / p.n_splits;
    const int rank = bh / p.mem.H, h = bh - rank * p.mem.H;
    const int b = pick_sequence(p, rank, *reinterpret_cast<Topology *>(smem + C::OFF_TOPO));
    const int n = p.n_nodes ? min(max(p.n_nodes[b], 0), p.N) : p.N;
    if (n == 0) return finish_barriers(p);  // nothing of this sequence is written
    const int parent = threadIdx.x < n ? p.parents[b * p.parents_stride + threadIdx.x] : -1;

    float *qs = reinterpret_cast<float *>(smem);
    float *rows32 = reinterpret_cast<float *>(smem + C::OFF_WARP) + warp * C::WARP;
    float *ring = rows32 + C::RING, *prob = rows32 + C::PROB;
    Topology &topo = *reinterpret_cast<Topology *>(smem + C::OFF_TOPO);

    // q + u and q + v of the nodes (those past n: zero)
    for (int e = threadIdx.x; e < C::NODES * DH; e += WARPS * 32) {
        const int i = e / DH, c = e % DH;
        const float *q = static_cast<const float *>(p.q.ptr) + b * p.q.sb + h * p.q.sh + i * p.q.sr;
        const float x = i < n ? q[c] : 0.f;
        float *dst = qs + (i / ROWS) * (2 * ROWS * SLD) + (i % ROWS) * SLD + c;
        dst[0] = x + static_cast<const float *>(p.u)[h * DH + c];
        dst[ROWS * SLD] = x + static_cast<const float *>(p.vb)[h * DH + c];
    }
    build_topology(topo, parent, n, p.status);

    int begin, fill;
    paged_state(p.mem, b, p.status, begin, fill);
    const Chunks ck = group_chunks(p, begin, fill, kNodesCost, split * KG + kg, p.n_splits * KG);
    const int i0 = mt * ROWS;               // this warp's first node
    const bool active = i0 < n;
    const float *qu = qs + mt * (2 * ROWS * SLD), *qv = qu + ROWS * SLD;
    const float *table = static_cast<const float *>(p.r) + (long long)h * p.r_rows * DH;

    float m[XN], l[XN], acc[XN][8];  // l: this lane's keys only; acc: dimensions 4 oct + e, 32 + 4 oct + e
    int depth[XN], depth_max = 0;
#pragma unroll
    for (int x = 0; x < XN; ++x) {
        m[x] = -INFINITY;
        l[x] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[x][e] = 0.f;
        const int i = i0 + quad + 4 * x;
        depth[x] = i < n ? topo.depth[i] : 0;
        depth_max = max(depth_max, depth[x]);
    }
    depth_max = __reduce_max_sync(0xffffffffu, depth_max);

    // 32 rows, row(x) of each (null: zeros), into the stage: in order, half a warp a row.
    auto load = [&](auto &&row, float4 (&w)[16]) {
#pragma unroll
        for (int c = 0; c < 16; ++c) {
            const float *src = row(2 * c + (lane >> 4));
            w[c] = src ? __ldg(reinterpret_cast<const float4 *>(src) + (lane & 15)) : make_float4(0.f, 0.f, 0.f, 0.f);
        }
    };
    auto stage = [&](const float4 (&w)[16]) {
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 16; ++c)
            *reinterpret_cast<float4 *>(rows32 + (2 * c + (lane >> 4)) * SLD + 4 * (lane & 15)) = w[c];
        __syncwarp();
    };
    // Dot products of nodes quad + 4 x (rows of q) and staged rows oct + 8 y.
    auto dots = [&](const float *q, float (&out)[XN][4]) {
#pragma unroll
        for (int x = 0; x < XN; ++x)
#pragma unroll
            for (int y = 0; y < 4; ++y) out[x][y] = 0.f;
#pragma unroll 4
        for (int d = 0; d < DH; d += 4) {
            float4 a[XN], k[4];
#pragma unroll
            for (int x = 0; x < XN; ++x) a[x] = f4(q + (quad + 4 * x) * SLD + d);
#pragma unroll
            for (int y = 0; y < 4; ++y) k[y] = f4(rows32 + (oct + 8 * y) * SLD + d);
#pragma unroll
            for (int x = 0; x < XN; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    out[x][y] = fmaf(a[x].x, k[y].x, out[x][y]);
                    out[x][y] = fmaf(a[x].y, k[y].y, out[x][y]);
                    out[x][y] = fmaf(a[x].z, k[y].z, out[x][y]);
                    out[x][y] = fmaf(a[x].w, k[y].w, out[x][y]);
                }
        }
    };
    // (q + v).r of the staged table rows into ring columns col ... (those below `past`)
    auto put_products = [&](int col, int past) {
        float c[XN][4];
        dots(qv, c);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
            int at = col + oct + 8 * y;
            const bool keep = at < past;
            at -= at >= RW ? RW : 0;
            TXL_CHECK(at >= 0 && at < RW, p.status);
#pragma unroll
            for (int x = 0; x < XN; ++x)
                if (keep) ring[(quad + 4 * x) * RW + at] = c[x][y];
        }
        __syncwarp();
    };
    auto table_row = [&](int row) {
        return row >= 0 && row < p.r_rows ? table + (long long)row * DH : nullptr;
    };
    // The DCAP table rows before row `end` into ring columns 0 .. DCAP - 1.
    auto table_before = [&](int end) {
        for (int c = 0; c < DCAP; c += GK) {
            float4 w[16];
            load([&](int x) { return table_row(end - DCAP + c + x); }, w);
            stage(w);
            put_products(c, DCAP);
        }
    };
    // Masked scores (log2 units; bit 4 x + y of `hidden`: not seen) into the running
    // softmax, then P.V over the value rows w.  mixed: keys may be hidden from some nodes
    // only; the value, which may be an infinity or NaN, then must not reach them.
    auto step = [&](float (&s)[XN][4], bool mixed, unsigned hidden, const float4 (&w)[16]) {
#pragma unroll
        for (int x = 0; x < XN; ++x) {
            float mx = max3_nan(max_nan(s[x][0], s[x][1]), s[x][2], s[x][3]);
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
            mx = max_nan(mx, m[x]);
            const float ref = mx == -INFINITY ? 0.f : mx;
            if (!(mx == m[x])) {
                const float f = ex2f(m[x] - ref);  // (0 from -inf: the sums are zero then)
                m[x] = mx;
                l[x] *= f;
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[x][e] *= f;
            }
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const float e = ex2f(s[x][y] - ref);
                l[x] += e;
                prob[(quad + 4 * x) * PLD + oct + 8 * y] = mixed && (hidden >> (4 * x + y)) & 1 ? -1.f : e;
            }
        }
        stage(w);
        if (mixed) {
#pragma unroll 1
            for (int key = 0; key < GK; ++key) {
                const float4 v0 = f4(rows32 + key * SLD + 4 * oct), v1 = f4(rows32 + key * SLD + 32 + 4 * oct);
                const float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
                for (int x = 0; x < XN; ++x) {
                    const float e = prob[(quad + 4 * x) * PLD + key];
                    if (e < 0.f) continue;
#pragma unroll
                    for (int d = 0; d < 8; ++d) acc[x][d] = fmaf(e, v[d], acc[x][d]);
                }
            }
            return;
        }
#pragma unroll 2
        for (int key = 0; key < GK; key += 4) {
            float4 e[XN];
#pragma unroll
            for (int x = 0; x < XN; ++x) e[x] = f4(prob + (quad + 4 * x) * PLD + key);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float4 v0 = f4(rows32 + (key + k) * SLD + 4 * oct);
                const float4 v1 = f4(rows32 + (key + k) * SLD + 32 + 4 * oct);
                const float v[8] = {v0.x, v0.y, v0.z, v0.w, v1.x, v1.y, v1.z, v1.w};
#pragma unroll
                for (int x = 0; x < XN; ++x) {
                    const float pe = k == 0 ? e[x].x : k == 1 ? e[x].y : k == 2 ? e[x].z : e[x].w;
#pragma unroll
                    for (int d = 0; d < 8; ++d) acc[x][d] = fmaf(pe, v[d], acc[x][d]);
                }
            }
        }
    };

    if (active && split == p.n_splits - 1 && kg == KG - 1) {
        // ---- the nodes among themselves: distances 0 .. DCAP - 1 ------------------
        table_before(p.r_rows);
        const float *kn = static_cast<const float *>(p.k.ptr) + b * p.k.sb + h * p.k.sh;
        const float *vn = static_cast<const float *>(p.v.ptr) + b * p.v.sb + h * p.v.sh;
        const int a_end = min(n, i0 + ROWS);  // (no node is an ancestor of an earlier one)
        for (int a0 = 0; a0 < a_end; a0 += GK) {
            float4 w[16];
            load([&](int x) { return a0 + x < a_end ? kn + (a0 + x) * p.k.sr : nullptr; }, w);
            stage(w);
            load([&](int x) { return a0 + x < a_end ? vn + (a0 + x) * p.v.sr : nullptr; }, w);
            float s[XN][4];
            dots(qu, s);
            unsigned hidden = 0;
#pragma unroll
            for (int x = 0; x < XN; ++x) {
                const int i = i0 + quad + 4 * x;
                const unsigned long long anc = i < n ? topo.anc[i] : 0;
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int a = a0 + oct + 8 * y;
                    const bool related = a < a_end && (anc >> a) & 1;
                    const int dist = related ? depth[x] - topo.depth[a] : 0;
                    const bool seen = related && dist < p.r_rows;
                    TXL_CHECK(dist >= 0 && dist < DCAP, p.status);
                    hidden |= seen ? 0u : 1u << (4 * x + y);
                    s[x][y] = seen ? (s[x][y] + ring[(quad + 4 * x) * RW + DCAP - 1 - dist]) * p.scale_log2
                                   : -INFINITY;
                }
            }
            step(s, true, hidden, w);
        }
        __syncwarp();
    }
    if (active && ck.count > 0) {
        const int trow0 = p.r_rows - 1 - fill + ck.c0 * GK - ck.off;  // table row of the first chunk's key 0
        table_before(trow0);
        // ---- the memory, chunk by chunk -------------------------------------------
        int wpos = DCAP;  // ring column of the chunk's first table row
        int slot = ck.slot, row = ck.row, page = page_at(p.mem, b, slot, p.status);
        for (int item = 0; item < ck.count; ++item) {
            const int j0 = (ck.c0 + item) * GK - ck.off;
            const long long at = page >= 0 ? (((long long)page * p.mem.H + h) * p.mem.P + row) * DH : 0;
            const float *kp = static_cast<const float *>(p.kpage) + at;
            const float *vp = static_cast<const float *>(p.vpage) + at;
            const int key_lo = -j0, key_hi = page >= 0 ? fill - j0 : 0;  // memory rows of the chunk
            float4 w[16];
            load([&](int x) { return table_row(trow0 + item * GK + x); }, w);
            stage(w);
            load([&](int x) { return x >= key_lo && x < key_hi ? kp + x * DH : nullptr; }, w);
            put_products(wpos, RW + GK);
            stage(w);
            load([&](int x) { return x >= key_lo && x < key_hi ? vp + x * DH : nullptr; }, w);
            float s[XN][4];
            dots(qu, s);
            const int reach = fill - p.r_rows - j0;  // depth d sees keys above reach + d
            unsigned hidden = 0;
#pragma unroll
            for (int x = 0; x < XN; ++x)
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                    const int jj = oct + 8 * y;
                    int c = wpos + jj - depth[x];
                    c += c < 0 ? RW : 0;
                    c -= c >= RW ? RW : 0;
                    const bool seen = jj >= key_lo && jj < key_hi && jj > reach + depth[x];
                    hidden |= seen ? 0u : 1u << (4 * x + y);
                    s[x][y] = seen ? (s[x][y] + ring[(quad + 4 * x) * RW + c]) * p.scale_log2 : -INFINITY;
                }
            step(s, reach + depth_max >= 0, hidden, w);
            wpos += GK;
            wpos -= wpos >= RW ? RW : 0;
            if (next_chunk(p.mem, slot, row) && item + 1 < ck.count) page = page_at(p.mem, b, slot, p.status);
        }
    }

    // ---- this warp's record, over its staged rows ------------------------------------
    const auto rec = [smem](int w) {
        return reinterpret_cast<typename C::WarpRec *>(smem + C::OFF_WARP + w * C::WARP * 4);
    };
    __syncwarp();
    typename C::WarpRec *r = rec(warp);
#pragma unroll
    for (int x = 0; x < XN; ++x) {
        float sum = l[x];
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const int i = quad + 4 * x;
        if (oct == 0) {
            r->m[i] = m[x];
            r->l[i] = sum;
        }
        *reinterpret_cast<float4 *>(&r->a[i][4 * oct]) = make_float4(acc[x][0], acc[x][1], acc[x][2], acc[x][3]);
        *reinterpret_cast<float4 *>(&r->a[i][32 + 4 * oct]) = make_float4(acc[x][4], acc[x][5], acc[x][6], acc[x][7]);
    }
    finish<WARPS, KG, MT, float>(rec, p, b, h, n, warp, lane);
}

// f(kernel, its shared memory, its index) for trees of N nodes: a warp's 4, 8 or 16
// nodes, then node tiles of 16.
template <typename F>
auto with_kernel(int N, F f)
{
    if (N <= 4) return f(relattn_tree_f32_kernel<1, 4>, CfgF32<1, 4>::SMEM, 0);
    if (N <= 8) return f(relattn_tree_f32_kernel<1, 8>, CfgF32<1, 8>::SMEM, 1);
    if (N <= 16) return f(relattn_tree_f32_kernel<1, 16>, CfgF32<1, 16>::SMEM, 2);
    if (N <= 32) return f(relattn_tree_f32_kernel<2, 16>, CfgF32<2, 16>::SMEM, 3);
    return f(relattn_tree_f32_kernel<4, 16>, CfgF32<4, 16>::SMEM, 4);
}

// The dynamic shared-memory attribute of the kernels, once per device.
cudaError_t ensure_attr()
{
    static bool done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 0 && dev < 64 && done[dev]) return cudaSuccess;
    for (int N : {4, 8, 16, 32, 64}) {
        e = with_kernel(N, [](auto *kern, int smem, int) {
            return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
        });
        if (e != cudaSuccess) return e;
    }
    if (dev >= 0 && dev < 64) done[dev] = true;
    return cudaSuccess;
}

} // namespace

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
    static ClusterCache cache[5];
    if (ensure_attr() != cudaSuccess) return 0;
    return with_kernel(N, [&](auto *kern, int smem, int i) {
        return cache[i].get(n_splits, [&] { return max_clusters(kern, n_splits, WARPS * 32, smem); });
    });
}

} // namespace txl
