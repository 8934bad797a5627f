// The BF16 layers of a deployment (osm_linear_hp): Y = [R +] [gate] act(X W +
// bias) on the tensor cores, W packed transposed [N][kp] by a k = K plan.
//
// Two kernels, by the number of tokens:
//   pair_kernel   CTA pairs on 256 x 256 output tiles (tcgen05 cta_group::2),
//                 persistent, two accumulators in tensor memory: the epilogue
//                 of a tile runs under the MMAs of the next.
//   skinny_kernel few tokens: the weights are what has to be read. The
//                 operands change places -- 128 output channels are the rows
//                 of the MMA, nt tokens its columns -- and the CTAs of a
//                 cluster split K, so that every SM streams weights; the
//                 partial sums are joined through distributed shared memory
//                 in the order of the ranks.
// What bounds them, measured on one B200 (back to back, power not capped): pair_kernel
// the tensor pipe -- BF16 4096 x 5120 x 5120 in 149 us (1440 TFLOP/s), 32760
// gated rows onto BF16 in 1141-1180 (1455-1505; the pipe 86 % active);
// skinny_kernel the weights -- one token, 5120 x 5120, in 14.2 us where the
// weights come from HBM (3.7 TB/s with 4 us of start and end) and 11.3 where they
// stayed in L2, 512 tokens in 33-35, where 1024 take pair_kernel 49. FP32 results
// cost more: 4096 tokens 219 us where BF16 ones take 169 (both power capped), for
// the sums of chunks and an end that runs under no other tile.
// 256 x 256 tiles are the largest of which tensor memory holds two accumulators.
// Every wait is bounded by %globaltimer; one that runs out sets the plan's
// status word and the CTA returns after its copies and MMAs have finished.
// No TMA multicast is used.

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <type_traits>

#include "osm_internal.h"
#include "osm_mx.cuh"
#include "osm_onto.cuh"
#include "osm_ptx.cuh"

namespace osm {
namespace {

constexpr int KSTEP = 64;               // BF16 values of one 128-byte swizzled row
constexpr int ROWS = 128;               // MMA rows per CTA (tensor-memory lanes)
constexpr int TILE = ROWS * 128;        // bytes of one 128-row operand tile of a K-step
constexpr uint16_t PAIR_MASK = 0x3;

struct LinearParams {
    CUtensorMap tm_x;    // X    [M][K] bf16
    CUtensorMap tm_w;    // w_hp [N][kp] bf16, box 64 x 128
    onto::Params end;    // sizes and the end of the product
    uint32_t* status;
    uint64_t wait_limit_ns;
    uint32_t starve;     // bytes that a CTA's first K-step waits for in vain (0 outside of failure tests)
    int ksteps;
    int num_m, num_n, group_m;  // pair_kernel: tiles and raster
};

__host__ __device__ constexpr uint32_t idesc_bf16(int m, int n) {
    // kind::f16: FP32 accumulator, A and B BF16, both K-major
    return (1u << 4) | (1u << 7) | (1u << 10) | (static_cast<uint32_t>(n >> 3) << 17) |
           (static_cast<uint32_t>(m >> 4) << 24);
}

__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr) {
    return ptx::smem_desc(saddr, 16, 1024, ptx::LAYOUT_SW128);
}

// The tensor cores round the accumulator toward zero at every 16 values of K;
// the errors have one sign, so they grow with K (1.6e-5 of the result at K =
// 13824, where FP32 sums rounded to nearest are within 1.5e-6). A BF16 result
// does not see them. For an FP32 result the products of FP32_CHUNK K-steps are
// one sum in tensor memory, and the chunks' sums are added up in registers,
// rounded to nearest, while the MMAs of the next chunk run.
constexpr int FP32_CHUNK = 8;  // K-steps: 512 values, 32 roundings

// ------------------------------------------------------------ pair_kernel

constexpr int PK_STAGES = 6;
constexpr int PK_EPI_WARPS = 8;
// Warpgroup 2 holds the producer and the MMA issuer and gives registers back
// to the epilogue (an FP32 tile's 128 sums, 64 residual words and the slab
// being read); 384 x 168 registers are launched (see osm_gemm.cu).
constexpr int PK_THREADS = 32 * PK_EPI_WARPS + 128;
constexpr int PK_LAUNCH_REGS = 168, PK_CTRL_REGS = 56, PK_EPI_REGS = 224;
static_assert((PK_LAUNCH_REGS - PK_CTRL_REGS) * 128 >= (PK_EPI_REGS - PK_LAUNCH_REGS) * 256, "register split exceeds the launch");
constexpr int PK_PRODUCER = PK_EPI_WARPS, PK_MMA = PK_EPI_WARPS + 1;
constexpr int PK_N = 256;
constexpr uint32_t PK_IDESC = idesc_bf16(256, PK_N);

struct __align__(1024) PairSmem {
    uint8_t a[PK_STAGES][TILE];
    uint8_t b[PK_STAGES][TILE];  // this CTA's half of the 256 output channels
    uint64_t full[PK_STAGES];    // leader: all copies of both CTAs for the slot have landed
    uint64_t empty[PK_STAGES];   // both: the MMAs reading the slot have completed
    uint64_t acc_full[2];        // both: an accumulator is complete (a tile's, or an FP32 chunk's)
    uint64_t acc_empty[2];       // leader: both CTAs have drained it
    onto::Vectors vectors[PK_EPI_WARPS];
    uint64_t drain;
    uint32_t tmem_base;
    int abort_flag;
};

template <class SM>
__device__ __forceinline__ void raise_abort(SM& S, uint32_t* status) {
    S.abort_flag = 1;
    atomicOr(status, OSM_STATUS_TIMEOUT);
}

__device__ __forceinline__ void pair_coords(const LinearParams& p, int tile, int& m, int& n) {
    const int group = p.group_m * p.num_n, g = tile / group, first = g * p.group_m;
    const int gm = min(p.num_m - first, p.group_m), local = tile % group;
    m = first + local % gm;
    n = local / gm;
}

template <bool F32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(PK_THREADS, 1)
    pair_kernel(const __grid_constant__ LinearParams p) {
    extern __shared__ uint8_t smem_raw[];
    PairSmem& S = *reinterpret_cast<PairSmem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = ptx::cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = static_cast<int>(ptx::cluster_id_x()), npairs = static_cast<int>(ptx::num_clusters_x());
    const int tiles = p.num_m * p.num_n;
    const volatile int* abort = &S.abort_flag;
    __shared__ int never;
    const uint64_t drain_ns = p.wait_limit_ns > 200000000ull ? p.wait_limit_ns : 200000000ull;

    if (threadIdx.x == 0) {
        for (int s = 0; s < PK_STAGES; ++s) {
            ptx::mbar_init(ptx::smem_u32(&S.full[s]), 1);
            ptx::mbar_init(ptx::smem_u32(&S.empty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(ptx::smem_u32(&S.acc_full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&S.acc_empty[i]), 2 * PK_EPI_WARPS);
        }
        ptx::mbar_init(ptx::smem_u32(&S.drain), 1);
        S.abort_flag = 0;
        never = 0;
        ptx::fence_mbar_init();
    }
    if (warp == PK_PRODUCER && lane == 0) {
        ptx::prefetch_tmap(&p.tm_x);
        ptx::prefetch_tmap(&p.tm_w);
    }
    if (warp == 1) {
        ptx::tmem_alloc_pair(ptx::smem_u32(&S.tmem_base), 512);
        ptx::tmem_relinquish_pair();
    }
    __syncwarp();
    ptx::tc_fence_before();
    ptx::cluster_sync();
    ptx::tc_fence_after();
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const uint32_t tmem = S.tmem_base;
    const int chunk = F32 ? FP32_CHUNK : p.ksteps;  // K-steps per accumulator
    auto teardown = [&] {
        __syncwarp();
        ptx::tc_fence_before();
        ptx::cluster_sync();
        if (warp == 1) {
            __syncwarp();
            ptx::tc_fence_after();
            ptx::tmem_dealloc_pair(tmem, 512);
        }
    };
    // Each side of the register split ends with its own copy of the teardown.
    if (warp >= PK_EPI_WARPS) {
        ptx::setmaxnreg_dec<PK_CTRL_REGS>();
        if (warp == PK_PRODUCER && ptx::elect_one()) {
            int stage = 0, last_stage = -1;
            uint32_t phase = 0, last_phase = 0, starve = p.starve;
            bool ok = true;
            for (int tile = pair; tile < tiles && ok; tile += npairs) {
                int m, n;
                pair_coords(p, tile, m, n);
                const int arow = m * 256 + static_cast<int>(rank) * ROWS;
                const int brow = n * PK_N + static_cast<int>(rank) * ROWS;
                for (int ks = 0; ks < p.ksteps; ++ks) {
                    if (!ptx::mbar_wait_bounded(ptx::smem_u32(&S.empty[stage]), phase ^ 1u, p.wait_limit_ns, abort)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = ptx::mapa(ptx::smem_u32(&S.full[stage]), 0);
                    if (leader) ptx::mbar_arrive_expect_tx(ptx::smem_u32(&S.full[stage]), 4u * TILE + starve);
                    starve = 0;
                    ptx::tma_load_2d_pair(ptx::smem_u32(S.a[stage]), &p.tm_x, ks * KSTEP, arow, fb);
                    ptx::tma_load_2d_pair(ptx::smem_u32(S.b[stage]), &p.tm_w, ks * KSTEP, brow, fb);
                    last_stage = stage;
                    last_phase = phase;
                    if (++stage == PK_STAGES) { stage = 0; phase ^= 1u; }
                }
            }
            if (!ok) raise_abort(S, p.status);
            // the slot filled last is released after the MMAs that read it: by then every copy has landed
            if (last_stage >= 0 &&
                !ptx::mbar_wait_bounded_cluster(ptx::smem_u32(&S.empty[last_stage]), last_phase, drain_ns, &never))
                ptx::spin_ns(1000000);
        } else if (warp == PK_MMA && leader && ptx::elect_one()) {
            int stage = 0, it = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int tile = pair; tile < tiles && ok; tile += npairs) {
                for (int k0 = 0; k0 < p.ksteps && ok; k0 += chunk, ++it) {
                    const int buf = it & 1, k1 = min(k0 + chunk, p.ksteps);
                    if (!ptx::mbar_wait_bounded_cluster(ptx::smem_u32(&S.acc_empty[buf]), ((it >> 1) & 1) ^ 1u,
                                                        p.wait_limit_ns, abort)) {
                        ok = false;
                        break;
                    }
                    ptx::tc_fence_after();
                    const uint32_t acc = tmem + buf * PK_N;
                    for (int ks = k0; ks < k1; ++ks) {
                        if (!ptx::mbar_wait_bounded(ptx::smem_u32(&S.full[stage]), phase, p.wait_limit_ns, abort)) {
                            ok = false;
                            break;
                        }
                        ptx::tc_fence_after();
                        const uint32_t a = ptx::smem_u32(S.a[stage]), b = ptx::smem_u32(S.b[stage]);
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            ptx::mma_bf16_pair(acc, desc_sw128(a + kk * 32), desc_sw128(b + kk * 32), PK_IDESC,
                                               (ks != k0 || kk != 0) ? 1u : 0u);
                        ptx::tc_commit_pair_mc(ptx::smem_u32(&S.empty[stage]), PAIR_MASK);
                        if (++stage == PK_STAGES) { stage = 0; phase ^= 1u; }
                    }
                    if (!ok) break;
                    ptx::tc_commit_pair_mc(ptx::smem_u32(&S.acc_full[buf]), PAIR_MASK);
                }
            }
            if (!ok) raise_abort(S, p.status);
            ptx::tc_commit_pair_mc(ptx::smem_u32(&S.drain), 0x1);
            ptx::mbar_wait_bounded(ptx::smem_u32(&S.drain), 0, drain_ns, &never);
        }
        teardown();
    } else {
        ptx::setmaxnreg_inc<PK_EPI_REGS>();
        const int q = warp & 3, half = warp >> 2;
        const uint32_t empty_leader = ptx::mapa(ptx::smem_u32(&S.acc_empty[0]), 0);
        onto::Tile<F32> end;
        int it = 0;
        // the accumulator's chunk `it` is complete
        auto wait_full = [&]() -> bool {
            int ok = 1;
            if (lane == 0)
                ok = ptx::mbar_wait_bounded_long(ptx::smem_u32(&S.acc_full[it & 1]), (it >> 1) & 1, p.wait_limit_ns, abort,
                                                 20000u);
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok && lane == 0) raise_abort(S, p.status);
            ptx::tc_fence_after();
            return ok;
        };
        // this warp has read it: the MMAs of the chunk after next may overwrite it
        auto release = [&] {
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive_remote_relaxed(empty_leader + (it & 1) * 8);
            ++it;
        };
        bool ok = true;
        for (int tile = pair; tile < tiles && ok; tile += npairs) {
            int m, n;
            pair_coords(p, tile, m, n);
            end.prepare(p.end, (int64_t)m * 256 + (int64_t)rank * ROWS + q * 32, (int64_t)n * PK_N + half * 128, lane,
                        S.vectors[warp]);
            if constexpr (F32) {
                uint32_t sum[128];
#pragma unroll 1
                for (int k0 = 0; k0 < p.ksteps; k0 += chunk) {
                    if (!(ok = wait_full())) break;
                    const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + (it & 1) * PK_N + half * 128;
                    if (k0 == 0) {
                        ptx::tmem_ld_16x256b_x16(taddr, sum);
                        ptx::tmem_ld_16x256b_x16(taddr + (16u << 16), sum + 64);
                        ptx::tmem_ld_wait();
                    } else {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {  // slab i / 2, columns 64 (i % 2) ..
                            uint32_t r[32];
                            ptx::tmem_ld_16x256b_x8(taddr + (static_cast<uint32_t>(16 * (i >> 1)) << 16) + 64 * (i & 1), r);
                            ptx::tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                sum[32 * i + e] = __float_as_uint(__fadd_rn(__uint_as_float(sum[32 * i + e]), __uint_as_float(r[e])));
                        }
                    }
                    release();
                }
                if (!ok) break;
                end.load_first(p.end, lane);
                if (end.nj > 0) {
#pragma unroll 1
                    for (int sl = 0; sl < 2; ++sl) {
                        end.template store<false, true>(p.end, sl, lane, S.vectors[warp], sum);
#pragma unroll
                        for (int e = 0; e < 64; ++e) sum[e] = sum[e + 64];
                    }
                }
            } else {
                end.load_first(p.end, lane);
                if (!(ok = wait_full())) break;
                const uint32_t taddr = tmem + (static_cast<uint32_t>(q * 32) << 16) + (it & 1) * PK_N + half * 128;
#pragma unroll 1
                for (int sl = 0; sl < 2; ++sl) {
                    uint32_t r[64];
                    ptx::tmem_ld_16x256b_x16(taddr + (static_cast<uint32_t>(16 * sl) << 16), r);
                    ptx::tmem_ld_wait();
                    if (sl == 1) release();
                    if (end.nj > 0) end.template store<false, true>(p.end, sl, lane, S.vectors[warp], r);
                }
            }
        }
        teardown();
    }
}

// ------------------------------------------------------------ skinny_kernel

constexpr int SK_THREADS = 192;  // warps 0-3 drain tensor memory, 4 issues the copies, 5 the MMAs

constexpr int SK_MAX_STAGES = 8;

// Bytes of a ring slot: 128 weight rows and nt token rows of one K-step.
__host__ __device__ constexpr int sk_slot(int nt) { return TILE + nt * 128; }

struct SkinnyControl {
    uint64_t full[SK_MAX_STAGES];
    uint64_t empty[SK_MAX_STAGES];
    uint64_t acc_full[2];   // FP32: a chunk's sum is complete
    uint64_t acc_empty[2];  // FP32: the four draining warps have read it
    uint64_t done;
    uint32_t tmem_base;
    int abort_flag;
};

__device__ __forceinline__ float4 ld_cluster_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Grid: x = clusters of S CTAs over the 128-channel tiles, y = tiles of nt
// tokens (a multiple of 16, at most 256). Rank s of a cluster takes the K-steps
// [s ks / S, (s + 1) ks / S). Once its ring is idle it holds the CTA's partial
// sums [nt][128]. SUMS: 0 for a BF16 result; for an FP32 one the tokens whose
// sums a lane holds (nt <= SUMS).
template <int SUMS>
__global__ void __launch_bounds__(SK_THREADS) skinny_kernel(const __grid_constant__ LinearParams p, int splits, int nt,
                                                           int stages, uint32_t acc_cols) {
    constexpr bool F32 = SUMS > 0;
    using Quad = typename std::conditional<F32, float4, uint2>::type;  // four values of Y's type
    const uint32_t cols = F32 ? 2 * acc_cols : acc_cols;  // tensor-memory columns: a power of two, 32 or more
    extern __shared__ uint8_t smem_raw[];
    __shared__ SkinnyControl S;
    uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float* part = reinterpret_cast<float*>(ring);
    const uint32_t ring_u32 = ptx::smem_u32(ring), slot_bytes = sk_slot(nt);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = splits > 1 ? static_cast<int>(ptx::cluster_ctarank()) : 0;
    const int n0 = (static_cast<int>(blockIdx.x) / splits) * ROWS;
    const int m0 = static_cast<int>(blockIdx.y) * nt;
    const int k0 = static_cast<int>(static_cast<int64_t>(p.ksteps) * rank / splits);
    const int k1 = static_cast<int>(static_cast<int64_t>(p.ksteps) * (rank + 1) / splits);
    const volatile int* abort = &S.abort_flag;
    __shared__ int never;
    const uint64_t drain_ns = p.wait_limit_ns > 200000000ull ? p.wait_limit_ns : 200000000ull;

    if (threadIdx.x == 0) {
        for (int s = 0; s < stages; ++s) {
            ptx::mbar_init(ptx::smem_u32(&S.full[s]), 1);
            ptx::mbar_init(ptx::smem_u32(&S.empty[s]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(ptx::smem_u32(&S.acc_full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&S.acc_empty[i]), 4);
        }
        ptx::mbar_init(ptx::smem_u32(&S.done), 1);
        S.abort_flag = 0;
        never = 0;
        ptx::fence_mbar_init();
    }
    if (warp == 4 && lane == 0) {
        ptx::prefetch_tmap(&p.tm_x);
        ptx::prefetch_tmap(&p.tm_w);
    }
    if (warp == 1) {
        ptx::tmem_alloc(ptx::smem_u32(&S.tmem_base), cols);
        ptx::tmem_relinquish();
    }
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const uint32_t tmem = S.tmem_base;

    if (warp == 4) {
        if (ptx::elect_one()) {
            int stage = 0, issued = 0;
            uint32_t phase = 0, starve = p.starve;
            bool ok = true;
            for (int ks = k0; ks < k1; ++ks, ++issued) {
                if (!ptx::mbar_wait_bounded(ptx::smem_u32(&S.empty[stage]), phase ^ 1u, p.wait_limit_ns, abort)) {
                    ok = false;
                    break;
                }
                const uint32_t fb = ptx::smem_u32(&S.full[stage]);
                ptx::mbar_arrive_expect_tx(fb, slot_bytes + starve);
                starve = 0;
                ptx::tma_load_2d(ring_u32 + stage * slot_bytes, &p.tm_w, ks * KSTEP, n0, fb);
                ptx::tma_load_2d(ring_u32 + stage * slot_bytes + TILE, &p.tm_x, ks * KSTEP, m0, fb);
                if (++stage == stages) { stage = 0; phase ^= 1u; }
            }
            if (!ok) raise_abort(S, p.status);
            // every copy has landed before the ring is used again (the MMAs wait for each of them;
            // an aborted pipeline may not have)
            for (int i = issued > stages ? issued - stages : 0; i < issued; ++i)
                if (!ptx::mbar_wait_bounded(ptx::smem_u32(&S.full[i % stages]), (i / stages) & 1, drain_ns, &never))
                    ptx::spin_ns(1000000);
        }
    } else if (warp == 5) {
        if (ptx::elect_one()) {
            const uint32_t idesc = idesc_bf16(ROWS, nt);
            int stage = 0;
            uint32_t phase = 0;
            bool ok = true;
            for (int ks = k0; ks < k1; ++ks) {
                const int i = (ks - k0) / FP32_CHUNK, buf = F32 ? i & 1 : 0;
                const bool first = F32 ? (ks - k0) % FP32_CHUNK == 0 : ks == k0;
                if (F32 && first &&
                    !ptx::mbar_wait_bounded(ptx::smem_u32(&S.acc_empty[buf]), ((i >> 1) & 1) ^ 1u, p.wait_limit_ns, abort)) {
                    ok = false;
                    break;
                }
                if (!ptx::mbar_wait_bounded(ptx::smem_u32(&S.full[stage]), phase, p.wait_limit_ns, abort)) {
                    ok = false;
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t a = ring_u32 + stage * slot_bytes, b = a + TILE;
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                    ptx::mma_bf16(tmem + buf * acc_cols, desc_sw128(a + kk * 32), desc_sw128(b + kk * 32),
                                  idesc, (!first || kk != 0) ? 1u : 0u);
                ptx::tc_commit(ptx::smem_u32(&S.empty[stage]));
                if (F32 && (ks + 1 == k1 || (ks + 1 - k0) % FP32_CHUNK == 0)) ptx::tc_commit(ptx::smem_u32(&S.acc_full[buf]));
                if (++stage == stages) { stage = 0; phase ^= 1u; }
            }
            if (!ok) raise_abort(S, p.status);
            ptx::tc_commit(ptx::smem_u32(&S.done));
            if (!ptx::mbar_wait_bounded(ptx::smem_u32(&S.done), 0, drain_ns, &never)) raise_abort(S, p.status);
        }
    }
    float4 bias = make_float4(0.0f, 0.0f, 0.0f, 0.0f);  // of the channels that this lane finishes
    if (p.end.bias && n0 + 4 * lane < p.end.N) bias = ptx::ld_f4(p.end.bias + n0 + 4 * lane);
    // FP32: a lane adds up its channel's chunk sums for all tokens
    float sum[F32 ? SUMS : 1];
    if constexpr (F32) {
#pragma unroll
        for (int i = 0; i < SUMS; ++i) sum[i] = 0.0f;
        if (warp < 4) {
            const int chunks = (k1 - k0 + FP32_CHUNK - 1) / FP32_CHUNK;
#pragma unroll 1
            for (int i = 0; i < chunks; ++i) {
                int ok = 1;
                if (lane == 0)
                    ok = ptx::mbar_wait_bounded(ptx::smem_u32(&S.acc_full[i & 1]), (i >> 1) & 1, p.wait_limit_ns, abort);
                ok = __shfl_sync(0xffffffffu, ok, 0);
                if (!ok) {
                    if (lane == 0) raise_abort(S, p.status);
                    break;
                }
                ptx::tc_fence_after();
                const uint32_t taddr = tmem + (static_cast<uint32_t>(warp * 32) << 16) + (i & 1) * acc_cols;
#pragma unroll
                for (int c = 0; c < SUMS; c += 32) {
                    if (c >= static_cast<int>(acc_cols)) break;
                    uint32_t r[32];
                    ptx::tmem_ld_32x32b_x32(taddr + c, r);
                    ptx::tmem_ld_wait();
#pragma unroll
                    for (int e = 0; e < 32; ++e) sum[c + e] = __fadd_rn(sum[c + e], __uint_as_float(r[e]));
                }
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(ptx::smem_u32(&S.acc_empty[i & 1]));
            }
        }
    }
    // All copies have landed and all MMAs completed: the ring becomes the
    // partial sums' buffer.
    __syncwarp();
    ptx::tc_fence_before();
    __syncthreads();
    ptx::tc_fence_after();
    if (F32) {
        if (warp < 4) {
#pragma unroll
            for (int i = 0; i < SUMS; ++i)
                if (i < nt && m0 + i < p.end.M) part[i * ROWS + warp * 32 + lane] = sum[F32 ? i : 0];
        }
    } else if (warp < 4) {
        const uint32_t taddr = tmem + (static_cast<uint32_t>(warp * 32) << 16);
#pragma unroll 1
        for (int c = 0; c < nt; c += 32) {
            uint32_t r[32];
            ptx::tmem_ld_32x32b_x32(taddr + c, r);
            ptx::tmem_ld_wait();
            const bool some = k1 > k0;  // a rank without K-steps adds zeros
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (c + i < nt && m0 + c + i < p.end.M) part[(c + i) * ROWS + warp * 32 + lane] = some ? __uint_as_float(r[i]) : 0.0f;
        }
        ptx::tc_fence_before();
    }
    if (splits > 1) ptx::cluster_sync();
    else __syncthreads();
    if (warp == 1) {
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, cols);
    }
    // Each rank finishes its share of the tile's tokens, a warp a token at a
    // time, a lane four channels of it. Everything that UNROLL tokens read is
    // on its way before the first of them is used.
    constexpr int UNROLL = 4, WARPS = SK_THREADS / 32;
    const int mt = static_cast<int>(min(static_cast<int64_t>(nt), p.end.M - m0)), share = (mt + splits - 1) / splits;
    const int last = min(mt, (rank + 1) * share);
    const int64_t n = n0 + 4 * lane;
    if (n < p.end.N) {
        for (int t0 = rank * share + warp; t0 < last; t0 += UNROLL * WARPS) {
            float4 v[UNROLL], g[UNROLL];
            Quad w[UNROLL];
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int t = t0 + u * WARPS;
                if (t >= last) break;
                const uint32_t off = ring_u32 + (t * ROWS + 4 * lane) * 4;
                v[u] = splits == 1 ? *reinterpret_cast<const float4*>(part + t * ROWS + 4 * lane) : ld_cluster_f4(ptx::mapa(off, 0));
                if (p.end.onto.gate)
                    g[u] = ptx::ld_f4(
                        p.end.onto.gate +
                        (static_cast<uint32_t>(m0 + t) / static_cast<uint32_t>(p.end.onto.gate_rows)) * p.end.onto.gate_stride + n);
                if (p.end.onto.r) w[u] = static_cast<const Quad*>(p.end.onto.r)[((m0 + t) * p.end.N + n) >> 2];
            }
            for (int s = 1; s < splits; ++s) {
#pragma unroll
                for (int u = 0; u < UNROLL; ++u) {
                    const int t = t0 + u * WARPS;
                    if (t >= last) break;
                    const float4 o = ld_cluster_f4(ptx::mapa(ring_u32 + (t * ROWS + 4 * lane) * 4, s));
                    v[u] = make_float4(v[u].x + o.x, v[u].y + o.y, v[u].z + o.z, v[u].w + o.w);
                }
            }
#pragma unroll
            for (int u = 0; u < UNROLL; ++u) {
                const int t = t0 + u * WARPS;
                if (t >= last) break;
                float2 a = make_float2(v[u].x, v[u].y), b = make_float2(v[u].z, v[u].w);
                if (p.end.bias) {
                    a = __fadd2_rn(a, make_float2(bias.x, bias.y));
                    b = __fadd2_rn(b, make_float2(bias.z, bias.w));
                }
                a = onto::activate2(a, p.end.act);
                b = onto::activate2(b, p.end.act);
                if (p.end.onto.gate) {
                    a = __fmul2_rn(a, make_float2(g[u].x, g[u].y));
                    b = __fmul2_rn(b, make_float2(g[u].z, g[u].w));
                }
                Quad out;
                if constexpr (F32) {
                    if (p.end.onto.r) {
                        a = __fadd2_rn(make_float2(w[u].x, w[u].y), a);
                        b = __fadd2_rn(make_float2(w[u].z, w[u].w), b);
                    }
                    out = make_float4(a.x, a.y, b.x, b.y);
                } else {
                    if (p.end.onto.r) {
                        a = __fadd2_rn(onto::from_word<false>(w[u].x), a);
                        b = __fadd2_rn(onto::from_word<false>(w[u].y), b);
                    }
                    out = make_uint2(mx::bf16x2_bits(a.x, a.y), mx::bf16x2_bits(b.x, b.y));
                }
                static_cast<Quad*>(p.end.Y)[((m0 + t) * p.end.N + n) >> 2] = out;
            }
        }
    }
    // a CTA's partial sums stay until every rank has read them
    if (splits > 1) ptx::cluster_sync();
}

// ------------------------------------------------------------ host

struct KernelInfo {
    int clusters = 0;  // co-resident CTA pairs (pair_kernel)
    bool ready = false;
};

int current_device(int* dev) {
    OSM_TRY(check_cuda(cudaGetDevice(dev), "cudaGetDevice"));
    if (*dev < 0 || *dev >= 64) return fail(OSM_ERR_UNSUPPORTED, "device index %d", *dev);
    return OSM_OK;
}

// Larger weights than this are swept by groups of M-tiles (see osm_gemm.cu).
constexpr int64_t W_RESIDENT_BYTES = 48ll << 20;

int launch_pair(LinearParams& p, bool f32, int64_t w_bytes, cudaStream_t st) {
    void (*kern)(LinearParams) = f32 ? pair_kernel<true> : pair_kernel<false>;
    constexpr size_t smem = sizeof(PairSmem) + 1024;
    static_assert(smem <= 232448, "shared memory budget");
    static KernelInfo info[64][2];
    static std::mutex mu;
    int dev = 0;
    OSM_TRY(current_device(&dev));
    KernelInfo& ki = info[dev][f32 ? 1 : 0];
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!ki.ready) {
            // the register split assumes that the launch gives every thread exactly PK_LAUNCH_REGS
            cudaFuncAttributes fa;
            OSM_TRY(check_cuda(cudaFuncGetAttributes(&fa, kern), "linear_hp attributes"));
            if (fa.numRegs != PK_LAUNCH_REGS)
                return fail(OSM_ERR_UNSUPPORTED, "linear_hp: built with %d registers per thread, the split needs %d",
                            fa.numRegs, PK_LAUNCH_REGS);
            OSM_TRY(check_cuda(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                    static_cast<int>(smem)), "linear_hp smem attribute"));
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(2, 1, 1);
            cfg.blockDim = dim3(PK_THREADS, 1, 1);
            cfg.dynamicSmemBytes = smem;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 2;
            attr[0].val.clusterDim.y = 1;
            attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            OSM_TRY(check_cuda(cudaOccupancyMaxActiveClusters(&ki.clusters, kern, &cfg), "linear_hp cluster occupancy"));
            if (ki.clusters < 1) return fail(OSM_ERR_UNSUPPORTED, "linear_hp: no CTA pair fits on this device");
            ki.ready = true;
        }
    }
    p.num_m = static_cast<int>(ceil_div(p.end.M, 256));
    p.num_n = static_cast<int>(ceil_div(p.end.N, PK_N));
    p.group_m = w_bytes <= W_RESIDENT_BYTES ? 1 : 8;
    const int64_t tiles = static_cast<int64_t>(p.num_m) * p.num_n;
    if (tiles > 0x7FFFFFFF) return fail(OSM_ERR_UNSUPPORTED, "linear_hp: too many tiles");
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * static_cast<unsigned>(std::min<int64_t>(tiles, ki.clusters)), 1, 1);
    cfg.blockDim = dim3(PK_THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return check_cuda(cudaLaunchKernelEx(&cfg, kern, p), "linear_hp launch");
}

// A launch of skinny_kernel: tokens per tile, ring slots and K splits.
struct SkinnyShape {
    int nt, stages, splits;
    float us;  // estimated time
};

// Time estimates in microseconds, fitted to sweeps on one B200 (K, N = 5120 x
// 5120, 1504 x 4128, 5120 x 1024, 512 x 13824, 1 to 1536 tokens; within about a
// tenth of the measured times of plain products). Activation, gate and residual
// are not in them: 1001 x 1504 x 4128 FP32 is estimated at 19.8, the plain product
// takes 18.8, with GELU 20.5 (22.7 with inputs that change), with gate and residual 22. A launch of skinny_kernel costs 3.6, a CTA alone on
// its SM takes a K-step of nt tokens in max(0.165, 0.115 + 0.00103 nt) (FP32, with
// its chunks: max(0.22, 0.13 + 0.00103 nt)) and its tile's end in 0.03 a token; two on an SM take 0.86 of twice the steps and 0.042 a
// token. Joining split sums costs 1.6, and the weights come at 6.2 TB/s.
// pair_kernel costs 8.5 and, per round of tiles, 0.29 a K-step, at least 5.2 for the
// epilogue; FP32 0.4 a K-step and 4.5 for the epilogue, which the sums in registers
// keep from running under the next tile.
SkinnyShape skinny_shape(int64_t M, int64_t N, int ksteps, bool f32, int sms) {
    SkinnyShape best{0, 0, 0, 1e30f};
    const int64_t ntiles = ceil_div(N, ROWS);
    const int most = f32 ? 128 : 256;  // an FP32 lane holds its tokens' sums in registers
    const int64_t fewest = ceil_div(M, most);
    for (int64_t tiles = fewest; tiles <= fewest + 8 && (tiles == fewest || ceil_div(M, tiles) > 32); ++tiles) {
        const int nt = static_cast<int>(round_up(ceil_div(M, tiles), 16));
        const float step = f32 ? std::max(0.22f, 0.13f + 0.00103f * nt) : std::max(0.165f, 0.115f + 0.00103f * nt);
        for (int splits = 1; splits <= 8 && (splits == 1 || ksteps >= 4 * splits); splits *= 2) {
            const int64_t ctas = ntiles * ceil_div(M, nt) * splits, per = ceil_div(ksteps, splits);
            if (splits > 1 && ctas > 2 * sms) break;
            const bool two = ctas > sms && nt <= 160;  // three ring slots of 160 tokens still fit twice
            const float rounds = static_cast<float>(ceil_div(ctas, two ? 2 * sms : sms));
            const float work = rounds * (two ? 1.72f * per * step + 0.042f * nt : per * step + 0.03f * nt);
            const float us = 3.6f + (splits > 1 ? 1.6f : 0.0f) + std::max(work, static_cast<float>(N) * ksteps * (KSTEP * 2) / 6.2e6f);
            if (us < best.us) best = SkinnyShape{nt, 0, splits, us};
        }
    }
    // as many slots as two CTAs per SM leave room for (one, where that is all there are); the partial sums
    // take the ring's place
    const int64_t ctas = ntiles * ceil_div(M, best.nt) * best.splits;
    const int slot = sk_slot(best.nt), room = ctas <= sms ? 208 * 1024 : 108 * 1024;
    best.stages = std::min(SK_MAX_STAGES, std::max(room / slot, static_cast<int>(ceil_div(best.nt * ROWS * 4, slot))));
    return best;
}

float pair_us(int64_t M, int64_t N, int ksteps, bool f32, int sms) {
    const int64_t tiles = ceil_div(M, 256) * ceil_div(N, PK_N);
    return 8.5f + static_cast<float>(ceil_div(tiles, sms / 2)) * (f32 ? 0.4f * ksteps + 4.5f : std::max(5.2f, 0.29f * ksteps));
}

template <int SUMS>
int launch_skinny(LinearParams& p, const SkinnyShape& s, cudaStream_t st) {
    void (*kern)(LinearParams, int, int, int, uint32_t) = skinny_kernel<SUMS>;
    const size_t smem = static_cast<size_t>(s.stages) * sk_slot(s.nt) + 1024;
    static KernelInfo info[64];
    static std::mutex mu;
    int dev = 0;
    OSM_TRY(current_device(&dev));
    {
        std::lock_guard<std::mutex> lk(mu);
        if (!info[dev].ready) {
            OSM_TRY(check_cuda(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 220 * 1024),
                               "linear_hp smem attribute"));
            info[dev].ready = true;
        }
    }
    const int64_t mtiles = ceil_div(p.end.M, s.nt);
    if (mtiles > 65535) return fail(OSM_ERR_UNSUPPORTED, "linear_hp: too many token tiles");
    uint32_t acc_cols = 32;
    while (acc_cols < static_cast<uint32_t>(s.nt)) acc_cols *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ceil_div(p.end.N, ROWS) * s.splits), static_cast<unsigned>(mtiles), 1);
    cfg.blockDim = dim3(SK_THREADS, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(s.splits);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = s.splits > 1 ? 2 : 1;
    return check_cuda(cudaLaunchKernelEx(&cfg, kern, p, s.splits, s.nt, s.stages, acc_cols), "linear_hp launch");
}

}  // namespace

int launch_linear_hp(const osm_plan* pl, const uint16_t* X, int64_t M, const uint16_t* w_hp, const float* bias, int act,
                     const Onto& onto, void* Y, int y_dtype, cudaStream_t st) {
    LinearParams p;
    std::memset(&p, 0, sizeof(p));
    p.end = onto::Params{M, pl->N, bias, Y, onto, 1.0f, act};
    p.status = pl->d_status;
    p.wait_limit_ns = pl->wait_limit_ns;
    p.starve = (pl->debug_flags & OSM_DEBUG_STARVE_LINEAR) ? 16u : 0u;
    p.ksteps = static_cast<int>(pl->kp / KSTEP);
    const bool f32 = y_dtype == OSM_DT_F32;
    int dev = 0;
    OSM_TRY(current_device(&dev));
    static std::atomic<int> sm_count[64];
    int sms = sm_count[dev].load(std::memory_order_relaxed);
    if (!sms) {
        OSM_TRY(check_cuda(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev), "SM count"));
        sm_count[dev].store(sms, std::memory_order_relaxed);
    }
    // CTA pairs once there are tokens for more than one of their tiles and
    // they are expected to be done first.
    bool pair = M > 4096;
    SkinnyShape shape{};
    if (!pair) {
        shape = skinny_shape(M, pl->N, p.ksteps, f32, sms);
        pair = M > 128 && pair_us(M, pl->N, p.ksteps, f32, sms) < shape.us;
    }
    const CUtensorMapDataType bf = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    const CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B;
    OSM_TRY(make_map(&p.tm_x, bf, X, pl->K, M, pl->K * 2, KSTEP, pair ? ROWS : shape.nt, sw, "X"));
    OSM_TRY(make_map(&p.tm_w, bf, w_hp, pl->kp, pl->N, pl->kp * 2, KSTEP, ROWS, sw, "w_hp"));
    if (pair) return launch_pair(p, f32, pl->N * pl->kp * 2, st);
    if (!f32) return launch_skinny<0>(p, shape, st);
    if (shape.nt <= 32) return launch_skinny<32>(p, shape, st);
    return shape.nt <= 64 ? launch_skinny<64>(p, shape, st) : launch_skinny<128>(p, shape, st);
}

}  // namespace osm
