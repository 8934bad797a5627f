// The norms before and after a transformer block's sublayers with their
// modulation, gate and residual:
//   norm_modulate   h = bf16((N(x) w + b) (1 + scale) + shift)
//   residual_norm   r' = r + alpha gate P(y), h = N(r') modulated likewise
// One pass over the rows: each row is read once, its statistics are joined
// across its warps (osm_norm.cuh), and the outputs are written from the same
// registers.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <mutex>

#include "osm_internal.h"
#include "osm_norm.cuh"
#include "osm_ptx.cuh"

namespace osm {
namespace {

using norm::Spec;

struct RowParams {
    const void* x;          // [M][D] BF16 or FP32: the rows (norm_modulate) or the residual stream
    const uint16_t* y;      // [M][D] BF16: the sublayer's output (residual_norm)
    void* r_out;            // [M][D] in x's type (residual_norm)
    uint16_t* h;            // [M][D] BF16, or NULL without a pre-norm
    const float* gate;      // gate rows, gate_stride floats apart, or NULL
    int64_t gate_stride;
    float alpha;
    Spec post, pre;         // kind -1: none
    uint32_t M, share;      // tokens of a run: they share their modulation and gate rows
    uint32_t pre_rows, gate_rows;  // tokens per modulation row and per gate row (at most M)
    uint32_t tile_rows, tiles_per_run, tiles;  // row tiles of a run (rows_kernel)
    int D;
};

// h = n a + b of the pre-norm, and (y or its norm) a + b of the gated sum:
// alpha, gate and the post-norm's affine part in one pair; columns j .. j + 3.
__device__ __forceinline__ void post_coefficients4(const RowParams& p, uint32_t row, int j, float2 (&a)[2],
                                                   float2 (&b)[2]) {
    const float2 alpha = make_float2(p.alpha, p.alpha);
    float2 g[2] = {alpha, alpha};
    if (p.gate) {
        const float4 v = ptx::ld_f4(p.gate + (row / p.gate_rows) * p.gate_stride + j);
        g[0] = __fmul2_rn(alpha, make_float2(v.x, v.y));
        g[1] = __fmul2_rn(alpha, make_float2(v.z, v.w));
    }
    a[0] = g[0];
    a[1] = g[1];
    b[0] = b[1] = make_float2(0.0f, 0.0f);
    if (p.post.weight) {
        const float4 v = ptx::ld_f4(p.post.weight + j);
        a[0] = __fmul2_rn(g[0], make_float2(v.x, v.y));
        a[1] = __fmul2_rn(g[1], make_float2(v.z, v.w));
    }
    if (p.post.bias) {
        const float4 v = ptx::ld_f4(p.post.bias + j);
        b[0] = __fmul2_rn(g[0], make_float2(v.x, v.y));
        b[1] = __fmul2_rn(g[1], make_float2(v.z, v.w));
    }
}

// One row by a team of `nw` warps: warp j of it holds the segments j, j + nw,
// ... (NS of them at most) in registers, as they are in memory. total() adds
// up one value per segment over the row (a barrier of the team and a buffer of
// its own, in turn, per call); coef(which, c, a, b) gives chunk c's
// coefficients (0: gated sum, 1: pre-norm).
template <bool F32, bool HAS_Y, int NS, class Total, class Coef>
__device__ __forceinline__ void one_row(const RowParams& p, uint32_t row, int j, int nw, int lane, float inv_d,
                                        Total total, Coef coef) {
    constexpr int XQ = F32 ? 2 : 1;  // 16-byte words of x per chunk
    const int nchunk = p.D / norm::CHUNK;
    const size_t base = static_cast<size_t>(row) * nchunk;
    uint4 xq[NS][XQ], yq[HAS_Y ? NS : 1];
    const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int t = 0; t < NS; ++t) {
        const int c = (j + t * nw) * 32 + lane;
#pragma unroll
        for (int q = 0; q < XQ; ++q)
            xq[t][q] = c < nchunk ? norm::ld_row(reinterpret_cast<const uint4*>(p.x) + (base + c) * XQ + q) : zero;
        if constexpr (HAS_Y)
            yq[t] = c < nchunk ? norm::ld_row(reinterpret_cast<const uint4*>(p.y) + base + c) : zero;
    }
    auto x_of = [&](int t, float2 (&v)[4]) {
        if constexpr (F32) norm::unpack(xq[t][0], xq[t][1], v);
        else norm::unpack(xq[t][0], v);
    };
    // (mean, 1 / deviation) of the row whose chunks get(t, v) gives
    auto statistics = [&](auto get, const Spec& s) -> float2 {
        float part[NS];
        float mean = 0.0f;
        if (s.kind == OSM_NORM_LAYER) {
#pragma unroll
            for (int t = 0; t < NS; ++t) {
                float2 v[4];
                get(t, v);
                part[t] = norm::chunk_sum(v);
            }
            mean = norm::mean_of(total(part), static_cast<float>(p.D), inv_d);
        }
#pragma unroll
        for (int t = 0; t < NS; ++t) {
            float2 v[4];
            get(t, v);
            part[t] = (j + t * nw) * 32 + lane < nchunk ? norm::chunk_m2(v, mean) : 0.0f;
        }
        return make_float2(mean, norm::inverse_deviation(total(part), inv_d, s.eps));
    };
    if constexpr (HAS_Y) {
        float2 st = make_float2(0.0f, 1.0f);
        if (p.post.kind >= 0) st = statistics([&](int t, float2 (&v)[4]) { norm::unpack(yq[t], v); }, p.post);
#pragma unroll
        for (int t = 0; t < NS; ++t) {
            const int c = (j + t * nw) * 32 + lane;
            if (c >= nchunk) continue;
            float2 xv[4], yv[4], a[4], b[4];
            x_of(t, xv);
            norm::unpack(yq[t], yv);
            coef(0, c, a, b);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (p.post.kind >= 0) yv[i] = norm::normalise(yv[i], st);
                xv[i] = __fadd2_rn(xv[i], __ffma2_rn(yv[i], a[i], b[i]));
            }
            // rounded to the residual stream's type: the norm reads what is stored
            if constexpr (F32) {
                xq[t][0] = make_uint4(__float_as_uint(xv[0].x), __float_as_uint(xv[0].y), __float_as_uint(xv[1].x),
                                      __float_as_uint(xv[1].y));
                xq[t][1] = make_uint4(__float_as_uint(xv[2].x), __float_as_uint(xv[2].y), __float_as_uint(xv[3].x),
                                      __float_as_uint(xv[3].y));
            } else {
                xq[t][0] = make_uint4(mx::bf16x2_bits(xv[0].x, xv[0].y), mx::bf16x2_bits(xv[1].x, xv[1].y),
                                      mx::bf16x2_bits(xv[2].x, xv[2].y), mx::bf16x2_bits(xv[3].x, xv[3].y));
            }
#pragma unroll
            for (int q = 0; q < XQ; ++q) reinterpret_cast<uint4*>(p.r_out)[(base + c) * XQ + q] = xq[t][q];
        }
        if (p.pre.kind < 0) return;
    }
    const float2 st = statistics(x_of, p.pre);
#pragma unroll
    for (int t = 0; t < NS; ++t) {
        const int c = (j + t * nw) * 32 + lane;
        if (c >= nchunk) continue;
        float2 xv[4], a[4], b[4];
        x_of(t, xv);
        coef(1, c, a, b);
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 hv = __ffma2_rn(norm::normalise(xv[i], st), a[i], b[i]);
            o[i] = mx::bf16x2_bits(hv.x, hv.y);
        }
        reinterpret_cast<uint4*>(p.h)[base + c] = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// Many rows: a CTA takes a tile of rows of one run, teams of W
// warps a row each. The run's coefficients are laid out once per tile in
// shared memory (FP32, four 16-byte words of a chunk in arrays of their own:
// conflict-free 128-bit reads), where all teams read them.
template <bool F32, bool HAS_Y, int W, int NS, int WARPS, int MINB>
__global__ void __launch_bounds__(32 * WARPS, MINB) rows_kernel(const __grid_constant__ RowParams p) {
    constexpr int TEAMS = WARPS / W;
    ptx::grid_dep_wait();    // launched while the kernel before it finishes
    ptx::grid_dep_launch();
    extern __shared__ __align__(16) uint8_t smem[];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int team = warp / W, j = warp % W;
    const int nchunk = p.D / norm::CHUNK, nseg = (p.D + norm::SEG - 1) / norm::SEG;
    const float inv_d = __frcp_rn(static_cast<float>(p.D));
    float* part = reinterpret_cast<float*>(smem) + team * 2 * W * NS;  // [2][W * NS]
    float4* table = reinterpret_cast<float4*>(smem + TEAMS * 2 * W * NS * 4);
    const int ntab = (HAS_Y ? 4 : 0) + (p.pre.kind >= 0 ? 4 : 0);  // arrays of nchunk words
    int flip = 0;
    auto total = [&](const float (&v)[NS]) -> float {
        float* at = part + flip * W * NS;
        flip ^= 1;
        norm::warp_totals<NS>(v, lane, at + j, W);
        if constexpr (W == 1) __syncwarp();
        else asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(32 * W) : "memory");
        return norm::join_total<W * NS>(at, nseg, lane);
    };
    auto coef = [&](int which, int c, float2 (&a)[4], float2 (&b)[4]) {
        const float4* at = table + (HAS_Y && which ? 4 : 0) * nchunk + c;
        const float4 a0 = at[0], a1 = at[nchunk], b0 = at[2 * nchunk], b1 = at[3 * nchunk];
        a[0] = make_float2(a0.x, a0.y);
        a[1] = make_float2(a0.z, a0.w);
        a[2] = make_float2(a1.x, a1.y);
        a[3] = make_float2(a1.z, a1.w);
        b[0] = make_float2(b0.x, b0.y);
        b[1] = make_float2(b0.z, b0.w);
        b[2] = make_float2(b1.x, b1.y);
        b[3] = make_float2(b1.z, b1.w);
    };
    uint32_t held = 0xffffffffu;
    for (uint32_t tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
        const uint32_t run = tile / p.tiles_per_run;
        const uint32_t first = run * p.share;
        const uint32_t row0 = first + (tile - run * p.tiles_per_run) * p.tile_rows;
        const uint32_t end = min(min(row0 + p.tile_rows, first + p.share), p.M);
        if (held != run) {
            if (held != 0xffffffffu) __syncthreads();  // the rows of the last run are done
            held = run;
            // word w of chunk c: columns 8c + 4 (w & 1) .. + 3 of a (w < 2) or b
            for (int i = threadIdx.x; i < ntab / 2 * nchunk; i += 32 * WARPS) {
                const int k = i / nchunk, c = i - k * nchunk;  // k: table * 2 + half
                const int col = c * norm::CHUNK + 4 * (k & 1);
                float2 a[2], b[2];
                if (HAS_Y && k < 2) post_coefficients4(p, first, col, a, b);
                else norm::coefficients4(p.pre, first / p.pre_rows, col, a, b);
                float4* at = table + ((k >> 1) * 4 + (k & 1)) * nchunk + c;
                at[0] = make_float4(a[0].x, a[0].y, a[1].x, a[1].y);
                at[2 * nchunk] = make_float4(b[0].x, b[0].y, b[1].x, b[1].y);
            }
            __syncthreads();
        }
        for (uint32_t row = row0 + team; row < end; row += TEAMS)
            one_row<F32, HAS_Y, NS>(p, row, j, W, lane, inv_d, total, coef);
    }
}

// Few rows, very wide ones, or a modulation row for each token: a CTA takes one
// row at a time and reads its coefficients from global memory.
template <bool F32, bool HAS_Y, int NS, int MINB>
__global__ void __launch_bounds__(512, MINB) row_kernel(const __grid_constant__ RowParams p) {
    __shared__ float part[2][16 * NS];
    ptx::grid_dep_wait();
    ptx::grid_dep_launch();
    const int lane = threadIdx.x & 31, j = threadIdx.x >> 5, nw = blockDim.x >> 5;
    const int nseg = (p.D + norm::SEG - 1) / norm::SEG;
    const float inv_d = __frcp_rn(static_cast<float>(p.D));
    int flip = 0;
    auto total = [&](const float (&v)[NS]) -> float {
        float* at = part[flip];
        flip ^= 1;
        norm::warp_totals<NS>(v, lane, at + j, nw);
        __syncthreads();
        return norm::join_total<16 * NS>(at, nseg, lane);
    };
    for (uint64_t row = blockIdx.x; row < p.M; row += gridDim.x) {
        const uint32_t r = static_cast<uint32_t>(row);
        auto coef = [&](int which, int c, float2 (&a)[4], float2 (&b)[4]) {
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
                float2 a2[2], b2[2];
                if (HAS_Y && which == 0) post_coefficients4(p, r, c * norm::CHUNK + 2 * i, a2, b2);
                else norm::coefficients4(p.pre, r / p.pre_rows, c * norm::CHUNK + 2 * i, a2, b2);
                a[i] = a2[0], a[i + 1] = a2[1], b[i] = b2[0], b[i + 1] = b2[1];
            }
        };
        one_row<F32, HAS_Y, NS>(p, r, j, nw, lane, inv_d, total, coef);
    }
}

// Resident CTAs of a kernel on the current device, looked up once per device,
// CTA size and shared-memory size (the last few shapes are kept).
struct Setup {
    struct Shape {
        size_t smem = ~size_t(0);
        int threads = 0, ctas = 0;
    };
    std::mutex mu;
    size_t smem_set[64] = {};
    Shape shapes[64][8];
    int next[64] = {};
};
int prepare(Setup& su, const void* kern, int threads, size_t smem, int* ctas) {
    int dev = 0, rc;
    if ((rc = check_cuda(cudaGetDevice(&dev), "cudaGetDevice"))) return rc;
    if (dev < 0 || dev >= 64) return fail(OSM_ERR_UNSUPPORTED, "device index %d", dev);
    std::lock_guard<std::mutex> lk(su.mu);
    for (const Setup::Shape& s : su.shapes[dev])
        if (s.smem == smem && s.threads == threads) {
            *ctas = s.ctas;
            return OSM_OK;
        }
    if (smem > 48 * 1024 && su.smem_set[dev] < smem) {
        if ((rc = check_cuda(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                  static_cast<int>(smem)), "norm smem attribute")))
            return rc;
        su.smem_set[dev] = smem;
    }
    int n = 0, sms = 0;
    if ((rc = check_cuda(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, threads, smem), "norm occupancy")))
        return rc;
    if (n < 1) return fail(OSM_ERR_UNSUPPORTED, "norm: no CTA fits");
    if ((rc = check_cuda(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev), "SM count"))) return rc;
    Setup::Shape& s = su.shapes[dev][su.next[dev]];
    su.next[dev] = (su.next[dev] + 1) % 8;
    s.smem = smem;
    s.threads = threads;
    s.ctas = *ctas = n * sms;
    return OSM_OK;
}

// A launch that may start while the kernel before it on the stream finishes.
template <class K>
int launch(K kern, unsigned grid, unsigned threads, size_t smem, cudaStream_t st, const RowParams& p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid, 1, 1);
    cfg.blockDim = dim3(threads, 1, 1);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return check_cuda(cudaLaunchKernelEx(&cfg, kern, p), "norm launch");
}

template <bool F32, bool HAS_Y, int W, int NS, int WARPS, int MINB>
int launch_tiles(RowParams p, cudaStream_t st) {
    static Setup su;
    auto kern = rows_kernel<F32, HAS_Y, W, NS, WARPS, MINB>;
    const size_t smem = WARPS / W * 2 * W * NS * 4 +
                        static_cast<size_t>((HAS_Y ? 4 : 0) + (p.pre.kind >= 0 ? 4 : 0)) * (p.D / norm::CHUNK) * 16;
    int ctas = 0;
    OSM_TRY(prepare(su, reinterpret_cast<const void*>(kern), 32 * WARPS, smem, &ctas));
    // one tile per CTA: each run is cut into its part of them
    const int64_t cuts = std::max<int64_t>(1, static_cast<int64_t>(ctas) * p.share / p.M);
    p.tile_rows = static_cast<uint32_t>(ceil_div(p.share, cuts));
    p.tiles_per_run = static_cast<uint32_t>(ceil_div(p.share, p.tile_rows));
    p.tiles = static_cast<uint32_t>(ceil_div(p.M, p.share)) * p.tiles_per_run;
    return launch(kern, std::min<uint32_t>(p.tiles, ctas), 32 * WARPS, smem, st, p);
}

template <bool F32, bool HAS_Y, int NS, int MINB>
int launch_single(const RowParams& p, cudaStream_t st) {
    static Setup su;
    auto kern = row_kernel<F32, HAS_Y, NS, MINB>;
    // a warp per segment for few rows; for many, as many segments as a warp can hold
    const int64_t nseg = ceil_div(p.D, norm::SEG);
    const int threads = 32 * static_cast<int>(std::min<int64_t>(16, p.M < 4 * 148 ? nseg : ceil_div(nseg, NS)));
    int ctas = 0;
    OSM_TRY(prepare(su, reinterpret_cast<const void*>(kern), threads, 0, &ctas));
    return launch(kern, std::min<uint32_t>(p.M, ctas), threads, 0, st, p);
}

template <bool F32, bool HAS_Y>
int launch_width(const RowParams& p, cudaStream_t st) {
    // Tiles pay once the rows are more than one round of CTAs with a row each, of
    // up to 16 warps by the row's segments and 32 warps per SM, while a run's
    // coefficients serve a few rows (us, a CTA per row against tiles: 5120 columns,
    // 296 rows 3.8 and 4.4, 400 rows 6.0 and 4.8, 3000 rows 21.7 and 14.8; 1024
    // columns, 1000 rows 3.2 and 3.4, 3000 rows 6.0 and 5.5). The coefficients of
    // 14336 columns (both tables) fill shared memory.
    const int64_t round = 148 * 32 / std::min<int64_t>(16, ceil_div(p.D, norm::SEG));
    const bool tiles = p.M > round && p.share >= 8 && p.D <= 14336;
    if (!tiles) {
        if (p.D <= 8192) return launch_single<F32, HAS_Y, 2, 2>(p, st);
        if (p.D <= 16384) return launch_single<F32, HAS_Y, 4, F32 ? 1 : 2>(p, st);
        return launch_single<F32, HAS_Y, 16, 1>(p, st);
    }
    // Warps per row and per CTA, by what a lane holds of a row (8 columns of each
    // of NS segments: 4 registers for BF16, 8 for FP32, 4 more for y), measured at
    // 2048 and 5120 columns: fewer registers and more warps until the totals'
    // barriers and shuffles cost more than the latency that they hide. 32760 x 5120
    // BF16, back to back, in us: norm_modulate with 1 warp of 20 segments and 16
    // warps per CTA 123.5, 2 x 10 and 16 warps 125, 20 warps 121.0 (85 % of the
    // measured copy rate), 4 x 5 and 24 warps 129, 28 warps 125.6; residual_norm with
    // any of them 227 (90 %). 60000 x 2048 FP32 with a post-norm: 1 x 8 265, 2 x 4
    // 260, 4 x 2 238.
    if (p.D <= 512) return launch_tiles<F32, HAS_Y, 1, 2, 16, 2>(p, st);
    if (p.D <= 2048) {
        if constexpr (HAS_Y && F32) return launch_tiles<F32, HAS_Y, 4, 2, 24, 1>(p, st);
        else if constexpr (HAS_Y) return launch_tiles<F32, HAS_Y, 2, 4, 20, 1>(p, st);
        else return launch_tiles<F32, HAS_Y, 2, 4, 16, 2>(p, st);
    }
    if (p.D <= 5120) {
        if constexpr (F32) return launch_tiles<F32, HAS_Y, HAS_Y ? 4 : 2, HAS_Y ? 5 : 10, 16, 1>(p, st);
        else return launch_tiles<F32, HAS_Y, HAS_Y ? 4 : 2, HAS_Y ? 5 : 10, HAS_Y ? 24 : 20, 1>(p, st);
    }
    constexpr int V = F32 || HAS_Y ? 4 : 2;
    if (p.D <= 8192) return launch_tiles<F32, HAS_Y, V, 32 / V, 16, 1>(p, st);
    constexpr int U = F32 || HAS_Y ? 8 : 4;
    return launch_tiles<F32, HAS_Y, U, 56 / U, 16, 1>(p, st);
}

Spec to_spec(const osm_norm_spec* s) {
    if (!s) return Spec{-1, 1.0f, nullptr, nullptr, nullptr, nullptr, 1, 0};
    return Spec{s->kind, s->eps, s->weight, s->bias, s->scale, s->shift, s->mod_rows > 0 ? s->mod_rows : 1, s->mod_stride};
}

}  // namespace

int launch_norm_rows(const void* X, int x_dtype, int64_t M, int64_t D, const uint16_t* Y, const osm_norm_spec* post,
                     const float* gate, int64_t gate_rows, int64_t gate_stride, float alpha,
                     const osm_norm_spec* pre, void* R_out, uint16_t* H, cudaStream_t st) {
    RowParams p{};
    p.x = X;
    p.y = Y;
    p.r_out = R_out;
    p.h = H;
    p.gate = gate;
    p.gate_stride = gate_stride;
    p.alpha = alpha;
    p.post = to_spec(post);
    p.pre = to_spec(pre);
    p.M = static_cast<uint32_t>(M);
    p.D = static_cast<int>(D);
    // A run of tokens shares its modulation and its gate row; with two runs of
    // different length each row is a run of its own. M < 2^31 and a tile has at
    // most M rows, so row numbers past the end fit 32 bits.
    const int64_t a = pre && (pre->scale || pre->shift) ? std::min(M, pre->mod_rows) : M;
    const int64_t b = gate ? std::min(M, gate_rows) : M;
    p.pre_rows = static_cast<uint32_t>(a);
    p.gate_rows = static_cast<uint32_t>(b);
    p.share = static_cast<uint32_t>(a == M ? b : (b == M || a == b ? a : 1));
    if (Y) return x_dtype == OSM_DT_F32 ? launch_width<true, true>(p, st) : launch_width<false, true>(p, st);
    return x_dtype == OSM_DT_F32 ? launch_width<true, false>(p, st) : launch_width<false, false>(p, st);
}

}  // namespace osm
