// The norms before and after a transformer block's sublayers with their
// modulation, gate and residual:
//   norm_modulate   h = bf16((N(x) w + b) (1 + scale) + shift)
//   residual_norm   r' = r + alpha gate P(y), h = N(r') modulated likewise
// One pass over the rows: each row is read once, its statistics are joined
// across the block (osm_norm.cuh), and the outputs are written from the same
// registers.

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>
#include <map>
#include <mutex>
#include <utility>

#include "osm_internal.h"
#include "osm_norm.cuh"

namespace osm {
namespace {

using norm::Spec;

struct RowParams {
    const void* x;          // [M][D] BF16 or FP32: the rows (norm_modulate) or the residual stream
    const uint16_t* y;      // [M][D] BF16: the sublayer's output (residual_norm)
    void* r_out;            // [M][D] in x's type (residual_norm)
    uint16_t* h;            // [M][D] BF16, or NULL without a pre-norm
    const float* gate;      // [rows / share][gate_stride] or NULL
    int64_t gate_stride;
    float alpha;
    Spec post, pre;         // kind -1: none
    int64_t M, share;       // tokens that share a modulation (and gate) row
    int64_t groups_per_share, groups;
    int64_t gate_rows;
    int D;
    int stages;             // slots of the ring of incoming row groups; 0: rows are loaded directly
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}

// Rows of group g: `rows` (may be <= 0 in a short last share) from `row0` on.
struct Group {
    int64_t row0, mrow;
    int rows;
};
template <int R>
__device__ __forceinline__ Group group_of(const RowParams& p, int64_t g) {
    const int64_t s = g / p.groups_per_share;
    const int64_t off = (g - s * p.groups_per_share) * R;
    const int64_t len = min(p.share, p.M - s * p.share);
    return {s * p.share + off, s, static_cast<int>(min(static_cast<int64_t>(R), len - off))};
}

// Persistent CTAs over groups of R rows. Thread t holds chunks t, t + T, ...
// (V of them) of every row of the group. A thread's chunks come through its
// own slots of a ring in shared memory (16-byte asynchronous copies, waited
// for by the thread that reads them: no barrier, no spinning). With V == 1
// the coefficients of the thread's eight columns stay in registers for all
// rows that share a modulation row.
template <bool F32, bool HAS_Y, int V, int R, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) norm_rows_kernel(const RowParams p) {
    constexpr int XQ = F32 ? 2 : 1;              // 16-byte words of x per chunk
    constexpr int NQ = XQ + (HAS_Y ? 1 : 0);     // words per chunk in the ring
    extern __shared__ __align__(16) uint8_t smem[];
    const int T = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int D = p.D, nchunk = D / norm::CHUNK, nseg = (D + norm::SEG - 1) / norm::SEG;
    const int nw = T >> 5;
    float2* part = reinterpret_cast<float2*>(smem);                 // [2][R][nseg]
    const uint32_t ring = static_cast<uint32_t>(__cvta_generic_to_shared(smem)) + ((2 * R * nseg * 8 + 15) & ~15);
    const uint32_t slot_bytes = static_cast<uint32_t>(R) * NQ * V * T * 16;
    int flip = 0;

    auto slot_addr = [&](int slot, int r, int q, int v) -> uint32_t {
        return ring + slot * slot_bytes + ((((r * NQ) + q) * V + v) * T + tid) * 16;
    };
    auto x_ptr = [&](int64_t row, int c, int q) -> const uint4* {
        return reinterpret_cast<const uint4*>(p.x) + (row * nchunk + c) * XQ + q;
    };
    auto y_ptr = [&](int64_t row, int c) -> const uint4* { return reinterpret_cast<const uint4*>(p.y) + row * nchunk + c; };
    auto fetch = [&](int64_t g, int slot) {
        if (g < p.groups) {
            const Group gr = group_of<R>(p, g);
#pragma unroll
            for (int r = 0; r < R; ++r)
                if (r < gr.rows)
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const int c = tid + v * T;
                        if (c < nchunk) {
#pragma unroll
                            for (int q = 0; q < XQ; ++q) cp_async16(slot_addr(slot, r, q, v), x_ptr(gr.row0 + r, c, q));
                            if constexpr (HAS_Y) cp_async16(slot_addr(slot, r, XQ, v), y_ptr(gr.row0 + r, c));
                        }
                    }
        }
        cp_async_commit();
    };

    // Statistics of R rows whose values the accessor get(r, v, out) gives:
    // one barrier; two copies of `part` so that the next call's writes need none.
    auto statistics = [&](auto get, const Spec& s, float2 (&st)[R]) {
        const bool center = s.kind == OSM_NORM_LAYER;
        float2* pt = part + flip * R * nseg;
        flip ^= 1;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int seg = warp + v * nw;
            if (seg < nseg) {
                float2 val[R][4];
#pragma unroll
                for (int r = 0; r < R; ++r) get(r, v, val[r]);
                norm::segment_stats<R>(val, tid + v * T < nchunk, center, norm::seg_cols(seg, D), lane, pt + seg, nseg);
            }
        }
        __syncthreads();
        norm::join_rows<R>(pt, nseg, nseg, D, center, s.eps, lane, st);
    };

    // coefficients: pre a, b; post (or the bare gate) ga, gb
    float2 ca[V == 1 ? 4 : 1], cb[V == 1 ? 4 : 1], ga[V == 1 ? 4 : 1], gb[V == 1 ? 4 : 1];
    auto pre_coef = [&](int64_t mrow, int j, float2& a, float2& b) { norm::coefficients(p.pre, mrow, j, a, b); };
    auto post_coef = [&](int64_t grow, int j, float2& a, float2& b) {
        float2 g = make_float2(p.alpha, p.alpha);
        if (p.gate) g = __fmul2_rn(g, __ldg(reinterpret_cast<const float2*>(p.gate + grow * p.gate_stride + j)));
        a = g;
        b = make_float2(0.0f, 0.0f);
        if (p.post.weight) a = __fmul2_rn(g, __ldg(reinterpret_cast<const float2*>(p.post.weight + j)));
        if (p.post.bias) b = __fmul2_rn(g, __ldg(reinterpret_cast<const float2*>(p.post.bias + j)));
    };
    int64_t held = -1;

    if (p.stages)
        for (int s = 0; s < p.stages - 1; ++s) fetch(blockIdx.x + static_cast<int64_t>(s) * gridDim.x, s);
    int slot = 0;
    for (int64_t g = blockIdx.x; g < p.groups; g += gridDim.x) {
        const Group gr = group_of<R>(p, g);
        uint4 xq[R][V][XQ], yq[HAS_Y ? R : 1][HAS_Y ? V : 1];
        if (p.stages) {
            int ahead = slot + p.stages - 1;
            if (ahead >= p.stages) ahead -= p.stages;
            fetch(g + static_cast<int64_t>(p.stages - 1) * gridDim.x, ahead);
            if (p.stages == 4) cp_async_wait<3>();
            else if (p.stages == 3) cp_async_wait<2>();
            else cp_async_wait<1>();
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = tid + v * T;
                const bool on = r < gr.rows && c < nchunk;
#pragma unroll
                for (int q = 0; q < XQ; ++q)
                    xq[r][v][q] = !on ? make_uint4(0, 0, 0, 0)
                                      : (p.stages ? lds128(slot_addr(slot, r, q, v)) : *x_ptr(gr.row0 + r, c, q));
                if constexpr (HAS_Y)
                    yq[r][v] = !on ? make_uint4(0, 0, 0, 0)
                                   : (p.stages ? lds128(slot_addr(slot, r, XQ, v)) : *y_ptr(gr.row0 + r, c));
            }
        if (++slot >= p.stages) slot = 0;
        if constexpr (V == 1) {
            if (held != gr.mrow) {
                held = gr.mrow;
                const int j = tid * norm::CHUNK;
                if (tid < nchunk)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (p.pre.kind >= 0) pre_coef(p.pre.scale || p.pre.shift ? gr.row0 / p.pre.mod_rows : 0, j + 2 * i, ca[i], cb[i]);
                        if constexpr (HAS_Y) post_coef(p.gate ? gr.row0 / p.gate_rows : 0, j + 2 * i, ga[i], gb[i]);
                    }
            }
        }
        auto x_get = [&](int r, int v, float2 (&o)[4]) {
            if constexpr (F32) norm::unpack(xq[r][v][0], xq[r][v][1], o);
            else norm::unpack(xq[r][v][0], o);
        };
        if constexpr (HAS_Y) {
            float2 st[R];
            if (p.post.kind >= 0)
                statistics([&](int r, int v, float2 (&o)[4]) { norm::unpack(yq[r][v], o); }, p.post, st);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = tid + v * T;
                if (c >= nchunk) continue;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    if (r >= gr.rows) continue;
                    float2 xv[4], yv[4];
                    x_get(r, v, xv);
                    norm::unpack(yq[r][v], yv);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float2 a, b;
                        if constexpr (V == 1) {
                            a = ga[i];
                            b = gb[i];
                        } else {
                            post_coef(p.gate ? gr.row0 / p.gate_rows : 0, c * norm::CHUNK + 2 * i, a, b);
                        }
                        if (p.post.kind >= 0) yv[i] = norm::normalise(yv[i], st[r]);
                        xv[i] = __fadd2_rn(xv[i], __ffma2_rn(yv[i], a, b));
                    }
                    // rounded to the residual stream's type: the norm reads what is stored
                    if constexpr (F32) {
                        xq[r][v][0] = make_uint4(__float_as_uint(xv[0].x), __float_as_uint(xv[0].y),
                                                 __float_as_uint(xv[1].x), __float_as_uint(xv[1].y));
                        xq[r][v][1] = make_uint4(__float_as_uint(xv[2].x), __float_as_uint(xv[2].y),
                                                 __float_as_uint(xv[3].x), __float_as_uint(xv[3].y));
                    } else {
                        xq[r][v][0] = make_uint4(mx::bf16x2_bits(xv[0].x, xv[0].y), mx::bf16x2_bits(xv[1].x, xv[1].y),
                                                 mx::bf16x2_bits(xv[2].x, xv[2].y), mx::bf16x2_bits(xv[3].x, xv[3].y));
                    }
                    uint4* dst = reinterpret_cast<uint4*>(p.r_out) + ((gr.row0 + r) * nchunk + c) * XQ;
#pragma unroll
                    for (int q = 0; q < XQ; ++q) dst[q] = xq[r][v][q];
                }
            }
        }
        if (!HAS_Y || p.pre.kind >= 0) {
            float2 st[R];
            statistics(x_get, p.pre, st);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const int c = tid + v * T;
                if (c >= nchunk) continue;
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    if (r >= gr.rows) continue;
                    float2 xv[4];
                    x_get(r, v, xv);
                    uint32_t o[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float2 a, b;
                        if constexpr (V == 1) {
                            a = ca[i];
                            b = cb[i];
                        } else {
                            pre_coef(p.pre.scale || p.pre.shift ? gr.row0 / p.pre.mod_rows : 0, c * norm::CHUNK + 2 * i, a, b);
                        }
                        const float2 hv = __ffma2_rn(norm::normalise(xv[i], st[r]), a, b);
                        o[i] = mx::bf16x2_bits(hv.x, hv.y);
                    }
                    reinterpret_cast<uint4*>(p.h)[(gr.row0 + r) * nchunk + c] = make_uint4(o[0], o[1], o[2], o[3]);
                }
            }
        }
    }
    if (p.stages) cp_async_wait<0>();
}

template <bool F32, bool HAS_Y, int V, int R, int MAXT, int MINB>
int launch_rows(RowParams p, cudaStream_t st) {
    auto kern = norm_rows_kernel<F32, HAS_Y, V, R, MAXT, MINB>;
    const int nchunk = p.D / norm::CHUNK, nseg = static_cast<int>(ceil_div(p.D, norm::SEG));
    const int T = static_cast<int>(round_up(ceil_div(nchunk, V), 32));
    const size_t head = (static_cast<size_t>(2) * R * nseg * 8 + 15) & ~size_t(15);
    const size_t slot = static_cast<size_t>(R) * ((F32 ? 2 : 1) + (HAS_Y ? 1 : 0)) * V * T * 16;
    const size_t budget = MINB >= 2 ? 110 * 1024 : 220 * 1024;
    p.stages = head + 4 * slot <= budget ? 4 : (head + 3 * slot <= budget ? 3 : (head + 2 * slot <= budget ? 2 : 0));
    const size_t smem = head + p.stages * slot;
    p.groups_per_share = ceil_div(std::min(p.share, p.M), R);
    p.groups = ceil_div(p.M, p.share) * p.groups_per_share;
    // shared-memory limit, CTAs per SM and SM count: looked up once per device and shape
    struct Setup {
        size_t smem_set = 0;
        std::map<std::pair<size_t, int>, int> per_sm;
        int sms = 0;
    };
    static std::mutex mu;
    static Setup cache[64];
    int dev = 0, per_sm = 0, sms = 0;
    int rc = check_cuda(cudaGetDevice(&dev), "cudaGetDevice");
    if (rc) return rc;
    if (dev < 0 || dev >= 64) return fail(OSM_ERR_UNSUPPORTED, "device index %d", dev);
    {
        std::lock_guard<std::mutex> lk(mu);
        Setup& su = cache[dev];
        if (smem > 48 * 1024 && su.smem_set < smem) {
            if ((rc = check_cuda(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                      static_cast<int>(smem)), "norm smem attribute")))
                return rc;
            su.smem_set = smem;
        }
        auto it = su.per_sm.find({smem, T});
        if (it == su.per_sm.end()) {
            int n = 0;
            if ((rc = check_cuda(cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kern, T, smem), "norm occupancy")))
                return rc;
            it = su.per_sm.emplace(std::make_pair(smem, T), n).first;
        }
        per_sm = it->second;
        if (!su.sms &&
            (rc = check_cuda(cudaDeviceGetAttribute(&su.sms, cudaDevAttrMultiProcessorCount, dev), "SM count")))
            return rc;
        sms = su.sms;
    }
    if (per_sm < 1) return fail(OSM_ERR_UNSUPPORTED, "norm: no CTA fits (D = %d)", p.D);
    const int64_t grid = std::min<int64_t>(p.groups, static_cast<int64_t>(sms) * per_sm);
    kern<<<static_cast<unsigned>(grid), T, smem, st>>>(p);
    return check_cuda(cudaGetLastError(), "norm launch");
}

template <bool F32, bool HAS_Y>
int launch_width(const RowParams& p, bool grouped, cudaStream_t st) {
    if (p.D <= 5120) {
        if (grouped) return launch_rows<F32, HAS_Y, 1, 2, 640, HAS_Y ? 1 : 2>(p, st);
        return launch_rows<F32, HAS_Y, 1, 1, 640, HAS_Y ? 1 : 2>(p, st);
    }
    if (p.D <= 10240) return launch_rows<F32, HAS_Y, 2, 1, 640, 1>(p, st);
    if (p.D <= 20480) return launch_rows<F32, HAS_Y, 4, 1, 640, 1>(p, st);
    return launch_rows<F32, HAS_Y, 8, 1, 1024, 1>(p, st);
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
    p.gate_rows = gate_rows > 0 ? gate_rows : 1;
    p.gate_stride = gate_stride;
    p.alpha = alpha;
    p.post = to_spec(post);
    p.pre = to_spec(pre);
    p.M = M;
    p.D = static_cast<int>(D);
    // Rows are grouped inside the runs of tokens that share their modulation
    // and gate rows; with two runs of different length, or none longer than a
    // token, each row is a group of its own.
    const int64_t a = pre && (pre->scale || pre->shift) ? std::min(M, pre->mod_rows) : M;
    const int64_t b = gate ? std::min(M, gate_rows) : M;
    p.share = a == M ? b : (b == M || a == b ? a : 1);
    const bool grouped = p.share >= 2 && M >= 2 * 148;
    if (Y) return x_dtype == OSM_DT_F32 ? launch_width<true, true>(p, grouped, st) : launch_width<false, true>(p, grouped, st);
    return x_dtype == OSM_DT_F32 ? launch_width<true, false>(p, grouped, st) : launch_width<false, false>(p, grouped, st);
}

}  // namespace osm
