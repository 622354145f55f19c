// Statistics of the logits of a few states (up to kFewRows): decoding steps, drafted trees.
//
// The table is what such a call reads; it streams through a ring of TMA copies as the A
// operand of tcgen05 (128 vocabulary rows a tile), the states are the B operand (bn of them,
// from L2 again for every tile), so that a tile of logits has its vocabulary in TMEM's lanes
// and the states in its columns.  The epilogue's warps turn 64 columns at a time through
// shared memory; each warp then owns eight states, four logits a lane, and every lane keeps the
// statistics of the logits it has seen.  For the largest logits only the maximum of each four is
// written; logprob_few_merge finds them among those.  Bound by the table's bytes.
//   warp 0      TMA producer
//   warp 1      MMA issuer
//   warp 2      TMEM allocator
//   warps 4-11  epilogue
#include "vocab.h"
#include "ptx.cuh"

namespace txl {
namespace {

using namespace ptx;

constexpr int BM = 128, BK = 64, MAX_NS = 10;
constexpr int A_BYTES = BM * BK * 2;
constexpr int RING = 184 * 1024;
constexpr int TURN_LD = BM + 4;                      // floats of a state's logits
constexpr int OFF_TURN = RING;                       // [64][TURN_LD]
constexpr int OFF_TARGET = OFF_TURN + 64 * TURN_LD * 4;
constexpr int OFF_BAR = OFF_TARGET + kFewRows * 4;
constexpr int N_BAR = 2 * MAX_NS + 4;
constexpr int OFF_MISC = OFF_BAR + N_BAR * 8;
constexpr int SMEM_BYTES = OFF_MISC + 16 + 1024;     // (slack for the manual alignment)
constexpr uint32_t TM_COLS = 512;
constexpr int ACC = 256;                             // columns of an accumulator
constexpr int kEpiWarps = 8;

static_assert(SMEM_BYTES <= 232448, "shared memory budget exceeded");
static_assert(kFewRows <= ACC, "states lie in an accumulator's columns");

__device__ __forceinline__ float min_nan(float a, float b)
{
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

__device__ __forceinline__ void epi_sync()
{
    asm volatile("bar.sync 1, %0;" ::"n"(kEpiWarps * 32) : "memory");
}

// Whether any thread of the epilogue says so; a barrier of its warps.
__device__ __forceinline__ bool epi_any(bool x)
{
    uint32_t r;
    asm volatile("{\n\t.reg .pred a, b;\n\tsetp.ne.u32 a, %1, 0;\n\t"
                 "barrier.cta.red.or.pred b, 1, %2, a;\n\tselp.u32 %0, 1, 0, b;\n\t}"
                 : "=r"(r)
                 : "r"((uint32_t)x), "n"(kEpiWarps * 32)
                 : "memory");
    return r != 0;
}

// Statistics (maximum, sum beside its 1, weighted sum) of eight states from 32 lanes' each ([maximum, sum,
// weighted sum][8][33] floats): lanes 4 j .. 4 j + 3 join state j's.
constexpr int kOwn = 3 * 8 * 33;
static_assert(kEpiWarps * kOwn <= 64 * TURN_LD, "the warps' parts of the turning buffer");

__device__ __noinline__ float4 join_lanes(const float *own, int lane)
{
    constexpr unsigned FULL = 0xffffffffu;
    const float *m = own + (lane >> 2) * 33 + (lane & 3) * 8, *s = m + 8 * 33, *es = s + 8 * 33;
    float top = m[0];
#pragma unroll
    for (int i = 1; i < 8; ++i) top = fmaxf(top, m[i]);
    top = fmaxf(top, __shfl_xor_sync(FULL, top, 1));
    top = fmaxf(top, __shfl_xor_sync(FULL, top, 2));
    const float mu = top == -INFINITY ? 0.f : top;
    float sum = 0.f, lo = 0.f, weighted = 0.f;
#pragma unroll 4
    for (int i = 0; i < 8; ++i) {
        // (before its first number a lane's maximum is -infinity and its sums are zero)
        const float d = fmaxf(m[i] - mu, -1e30f), f = ex2(d);
        two_sum(sum, lo, f);
        two_sum(sum, lo, s[i] * f);
        weighted = fmaf(fmaf(s[i] + 1.f, d, es[i]), f, weighted);
    }
#pragma unroll
    for (int o = 1; o < 4; o *= 2) {
        const float hi = __shfl_xor_sync(FULL, sum, o), olo = __shfl_xor_sync(FULL, lo, o);
        two_sum(sum, lo, hi);
        lo += olo;
        weighted += __shfl_xor_sync(FULL, weighted, o);
    }
    // (the largest one's own 1 is among the terms, so their sum is 1 at least)
    return make_float4(top, top == -INFINITY ? sum : (sum - 1.f) + lo, weighted, 0.f);
}

// THREE: three terms of both operands.
template <int GROUPS, bool THREE>
__global__ void __launch_bounds__((4 + kEpiWarps) * 32, 1)
    logprob_few_kernel(const __grid_constant__ CUtensorMap tm_w, const __grid_constant__ CUtensorMap tm_h,
                       const GemmParams p, int ns)
{
    extern __shared__ uint8_t smem_raw[];
    const uint32_t raw_addr = smem_u32(smem_raw);
    uint8_t *smem = smem_raw + ((1024u - (raw_addr & 1023u)) & 1023u);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    // two accumulators in turn; with three terms, up to 128 states: two of 128 columns with the small
    // products behind each; beyond: one, its small products in the other's place
    constexpr int BUFS = THREE && GROUPS > 2 ? 1 : 2, REST = GROUPS > 2 ? ACC : ACC / 2;
    const int stage_bytes = A_BYTES + p.bn * BK * 2;
    // this block's tiles of the vocabulary
    const int t_lo = (int)((long long)blockIdx.x * p.nb / p.splits);
    const int t_hi = (int)((long long)(blockIdx.x + 1) * p.nb / p.splits);

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
            mbar_init(acc_empty + s, kEpiWarps * 32);
        }
        *abort_flag = 0;
        fence_barrier_init();
    }
    if (warp == 2) {
        tmem_alloc(tmem_slot, TM_COLS);
        tmem_relinquish();
        tc_fence_before_sync();
    }
    __syncthreads();
    tc_fence_after_sync();
    const uint32_t tmem = *tmem_slot;
    const uint64_t wait_ns = p.wait_ns;
    chain_wait();
    chain_go();

    if (warp == 0) {
        if (lane == 0) {
            prefetch_tensormap(&tm_w);
            prefetch_tensormap(&tm_h);
            const uint64_t often = policy_evict_last();
            bool ok = true;
            int it = 0;
            for (int t = t_lo; t < t_hi && ok; ++t)
                for (int kb = 0; kb < p.kb && ok; ++kb) {
                    for (int term = 0; term < (THREE ? 3 : 1); ++term) {
                        const int s = it % ns;
                        if (!(ok = mbar_wait(empty + s, ((it / ns) & 1) ^ 1, abort_flag, wait_ns))) break;
                        uint8_t *st = smem + s * stage_bytes;
                        mbar_arrive_expect_tx(full + s, stage_bytes);
                        tma_load_3d(st, &tm_w, full + s, kb * BK, t * BM, term);
                        tma_load_3d_hint(st + A_BYTES, &tm_h, full + s, kb * BK, 0, term, often);
                        ++it;
                    }
                }
            if (!ok) {
                atomicOr(p.status, TXL_STATUS_TIMEOUT);
                *abort_flag = 1;
                const int zero = 0;
                for (int i = max(0, it - ns); i < it; ++i)
                    mbar_wait(full + i % ns, (i / ns) & 1, &zero, wait_ns);
            }
        }
    } else if (warp == 1) {
        const uint32_t ID = idesc_bf16_f32(BM, p.bn, false);
        auto elect = []() -> bool {
            uint32_t el;
            asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}"
                         : "=r"(el));
            return el != 0;
        };
        const uint64_t dA = sdesc_sw128(smem_u32(smem)), dB = sdesc_sw128(smem_u32(smem + A_BYTES));
        bool ok = true;
        int it = 0, tile = 0;
        for (int t = t_lo; t < t_hi; ++t) {
            const int buf = tile % BUFS;
            ok = __all_sync(0xffffffffu, mbar_wait(acc_empty + buf, ((tile / BUFS) & 1) ^ 1, abort_flag, wait_ns));
            if (!ok) break;
            tc_fence_after_sync();
            const uint32_t acc = tmem + buf * ACC;
            auto product = [&](uint32_t to, uint64_t x, uint64_t y, bool add) {
#pragma unroll
                for (int kk = 0; kk < BK / 16; ++kk)
                    mma_bf16_ss(to, dA + x + kk * 2, dB + y + kk * 2, ID, add || kk > 0 ? 1u : 0u);
            };
            for (int k = 0; k < p.kb && ok; ++k) {
                // the product of the first terms in one accumulator; those of three terms whose weights are
                // 2^-8 and 2^-16 in another, whose cut additions do not matter
                uint64_t first = 0;
                for (int term = 0; term < (THREE ? 3 : 1); ++term, ++it) {
                    const int s = it % ns;
                    ok = __all_sync(0xffffffffu, mbar_wait(full + s, (it / ns) & 1, abort_flag, wait_ns));
                    if (!ok) break;
                    tc_fence_after_sync();
                    const uint64_t at = (uint64_t)((s * stage_bytes) >> 4);
                    if (term == 0) first = at;
                    if (elect()) {
                        if (term == 0) {
                            product(acc, at, at, k > 0);
                        } else {
                            product(acc + REST, at, first, k > 0 || term > 1);
                            product(acc + REST, first, at, true);
                            if (term == 1) product(acc + REST, at, at, true);
                        }
                        // (of three terms, the first stage is free with the last)
                        if (term > 0 || !THREE) mma_commit(empty + s);
                        if (term == 2) mma_commit(empty + (it - 2) % ns);
                    }
                    __syncwarp();
                }
            }
            if (!ok) break;
            if (elect()) mma_commit(acc_full + buf);
            __syncwarp();
            ++tile;
        }
        if (!ok) {
            if (lane == 0) {
                atomicOr(p.status, TXL_STATUS_TIMEOUT);
                *abort_flag = 1;
            }
            if (elect()) mma_commit(acc_full + tile % BUFS);
            __syncwarp();
            const int zero = 0;
            mbar_wait(acc_full + tile % BUFS, (tile / BUFS) & 1, &zero, wait_ns);
        }
    } else if (warp >= 4) {
        constexpr unsigned FULL = 0xffffffffu;
        const int we = warp - 4, quarter = we & 3, half = we >> 2;
        float *turn = reinterpret_cast<float *>(smem + OFF_TURN);
        int *targets = reinterpret_cast<int *>(smem + OFF_TARGET);
        const float c2 = p.scale * uncut_scale(p.kb * (BK / 16)) * 1.4426950408889634f;
        for (int i = threadIdx.x - 128; i < p.M; i += kEpiWarps * 32)
            targets[i] = p.targets ? token_at(p.targets, p.index_bytes, i, p.V, p.status) : -1;
        // running statistics of this lane's logits of state 64 g + 8 we + j; the sums leave the maximum's own 1 out
        float m[GROUPS * 8], sum[GROUPS * 8], es[GROUPS * 8];
#pragma unroll
        for (int i = 0; i < GROUPS * 8; ++i) {
            m[i] = -INFINITY;
            sum[i] = es[i] = 0.f;
        }
        bool ok = true;
        int tile = 0;
        for (int t = t_lo; t < t_hi; ++t, ++tile) {
            const int buf = tile % BUFS;
            ok = __all_sync(FULL, mbar_wait(acc_full + buf, (tile / BUFS) & 1, abort_flag, wait_ns) && !*abort_flag);
            // (all warps of the epilogue meet at its barriers: they leave together)
            if (epi_any(!ok)) {
                ok = false;
                break;
            }
            tc_fence_after_sync();
            const int id0 = t * BM + lane * 4, left = p.N - id0;  // (p.N: the vocabulary)
            const bool whole = (t + 1) * BM <= p.N;
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
                const int c = g * 64 + half * 32;
                if (c < p.M) {
                    uint32_t raw[32];
                    tmem_ld32(tmem + ((uint32_t)(quarter * 32) << 16) + buf * ACC + c, raw);
                    tmem_ld_wait(raw);
                    if (THREE) {
                        uint32_t rest[32];
                        tmem_ld32(tmem + ((uint32_t)(quarter * 32) << 16) + buf * ACC + REST + c, rest);
                        tmem_ld_wait(rest);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            raw[i] = __float_as_uint(__uint_as_float(raw[i]) + __uint_as_float(rest[i]));
                    }
#pragma unroll
                    for (int i = 0; i < 32; ++i)
                        turn[(half * 32 + i) * TURN_LD + quarter * 32 + lane] = __uint_as_float(raw[i]);
                }
                if (g + 1 == GROUPS) {
                    tc_fence_before_sync();
                    mbar_arrive(acc_empty + buf);
                }
                epi_sync();
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int st = g * 64 + we * 8 + j, k = g * 8 + j;
                    if (st >= p.M) break;
                    const float4 z = *reinterpret_cast<const float4 *>(turn + (we * 8 + j) * TURN_LD + lane * 4);
                    float v[4] = {z.x, z.y, z.z, z.w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[i] = fmaf(v[i], c2, 0.f);  // (+ 0: zeros of one sign)
                    if (!whole)
#pragma unroll
                        for (int i = 0; i < 4; ++i) v[i] = i < left ? v[i] : -INFINITY;
                    // the four with their largest first (a maximum passes NaN over, a minimum takes it)
                    const float a = fmaxf(v[0], v[1]), b = fmaxf(v[2], v[3]), top = fmaxf(a, b);
                    const float u[4] = {top, min_nan(a, b), min_nan(v[0], v[1]), min_nan(v[2], v[3])};
                    const float m_new = fmaxf(m[k], top);
                    const float mu = m_new == -INFINITY ? 0.f : m_new;
                    // (before the first number the maximum is -infinity and the sums are zero)
                    const float diff = fmaxf(m[k] - mu, -1e30f), f = ex2(diff);
                    // (a maximum that another takes the place of is one of the others)
                    const float one = top > m[k] ? 1.f : 0.f, others = sum[k] + one;
                    float e_new = fmaf(others, diff, es[k]) * f, e4[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float d = u[i] - mu;
                        e4[i] = ex2(d);
                        e_new = fmaf(e4[i], fmaxf(d, -1e30f), e_new);
                    }
                    m[k] = m_new;
                    sum[k] = fmaf(others, f, ((e4[0] - one) + e4[1]) + (e4[2] + e4[3]));
                    es[k] = e_new;
                    if (p.logits) {
                        const float none = __int_as_float(0x7fffffff);
                        *reinterpret_cast<float4 *>(p.logits + ((long long)st * p.nb + t) * BM + lane * 4) =
                            make_float4(left > 0 ? v[0] : none, left > 1 ? v[1] : none, left > 2 ? v[2] : none,
                                        left > 3 ? v[3] : none);
                    }
                    // the largest of the lane's four: NaN has no place in the order, nor has a lane behind V
                    if (p.group_key)
                        p.group_key[((long long)st * p.nb + t) * 32 + lane] = top == top && left > 0 ? order_key(top) : 0u;
                    const int at = targets[st] - id0;
                    if ((unsigned)at < 4u)
                        p.target_z[st] = at & 2 ? (at & 1 ? v[3] : v[2]) : (at & 1 ? v[1] : v[0]);
                }
                epi_sync();  // (the buffer is free again)
            }
        }
        if (!ok && lane == 0) {
            atomicOr(p.status, TXL_STATUS_TIMEOUT);
            *abort_flag = 1;
        }
        if (ok) {
            // over the lanes, through the warp's part of the turning buffer, four lanes a state (in one
            // copy of the code: a kernel's cold instructions cost more here than the arithmetic)
            float *own = turn + we * kOwn;
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
                if (g * 64 >= p.M) break;
                __syncwarp();
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    own[j * 33 + lane] = m[g * 8 + j];
                    own[(8 + j) * 33 + lane] = sum[g * 8 + j];
                    own[(16 + j) * 33 + lane] = es[g * 8 + j];
                }
                __syncwarp();
                const int st = g * 64 + we * 8 + (lane >> 2);
                const float4 r = join_lanes(own, lane);
                if ((lane & 3) == 0 && st < p.M) p.stats[(long long)blockIdx.x * p.M + st] = r;
            }
        }
        tc_fence_before_sync();
    }

    __syncthreads();
    if (warp == 2) {
        tc_fence_after_sync();
        tmem_dealloc(tmem, TM_COLS);
    }
}

template <int GROUPS, bool THREE>
cudaError_t launch(const CUtensorMap &tm_w, const CUtensorMap &tm_h, const GemmParams &p, cudaStream_t s)
{
    static bool attr_set[64] = {};  // the attribute is set once per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !attr_set[dev]) {
        e = cudaFuncSetAttribute(logprob_few_kernel<GROUPS, THREE>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 SMEM_BYTES);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) attr_set[dev] = true;
    }
    const int ns = min(MAX_NS, RING / (A_BYTES + p.bn * BK * 2));
    return launch_grid(logprob_few_kernel<GROUPS, THREE>, dim3((unsigned)p.splits), (4 + kEpiWarps) * 32, SMEM_BYTES, s, 1,
                       tm_w, tm_h, p, ns);
}

} // namespace

cudaError_t launch_logprob_few(const CUtensorMap &tm_w, const CUtensorMap &tm_h, const GemmParams &p,
                               cudaStream_t s)
{
    const int groups = (p.M + 63) / 64;
    const bool three = p.terms == 3;
    if (groups == 1) return three ? launch<1, true>(tm_w, tm_h, p, s) : launch<1, false>(tm_w, tm_h, p, s);
    if (groups == 2) return three ? launch<2, true>(tm_w, tm_h, p, s) : launch<2, false>(tm_w, tm_h, p, s);
    return three ? launch<4, true>(tm_w, tm_h, p, s) : launch<4, false>(tm_w, tm_h, p, s);
}

} // namespace txl
