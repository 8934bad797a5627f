// Row statistics and coefficients shared by the kernels that normalise rows
// (norm_modulate, residual_norm, norm_quantize_act).
//
// A row of D values is cut into chunks of 8 consecutive columns and segments
// of 32 chunks (256 columns). A sum over the row is a fixed tree: the eight
// values of a chunk, the 32 chunks of a segment (lanes at distances 1, 2, 4,
// 8, 16), 16 segments (distances 1, 2, 4, 8), then the groups of 16 segments
// in order. The tree does not depend on how a kernel maps rows and segments
// to warps, so every kernel gets the same bits for the same row. The variance
// is the sum of squared deviations from the row's mean, never a difference
// of sums.
#pragma once

#include <cstdint>

#include "osm_mx.cuh"
#include "osm_ptx.cuh"

namespace osm {
namespace norm {

constexpr int CHUNK = 8;              // columns per lane
constexpr int SEG = 32 * CHUNK;       // columns per warp-wide segment

// A norm as a kernel takes it (osm_norm_spec with row counts as 64-bit).
struct Spec {
    int kind;            // OSM_NORM_LAYER, OSM_NORM_RMS, or -1: no norm
    float eps;
    const float* weight; // [D] or NULL
    const float* bias;   // [D] or NULL
    const float* scale;  // [rows / mod_rows][mod_stride] or NULL
    const float* shift;  // likewise
    int64_t mod_rows, mod_stride;
};

// Eight consecutive values of a row, as four pairs.
__device__ __forceinline__ void unpack(const uint4& q, float2 (&v)[4]) {
    v[0] = make_float2(__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xFFFF0000u));
    v[1] = make_float2(__uint_as_float(q.y << 16), __uint_as_float(q.y & 0xFFFF0000u));
    v[2] = make_float2(__uint_as_float(q.z << 16), __uint_as_float(q.z & 0xFFFF0000u));
    v[3] = make_float2(__uint_as_float(q.w << 16), __uint_as_float(q.w & 0xFFFF0000u));
}
__device__ __forceinline__ void unpack(const uint4& lo, const uint4& hi, float2 (&v)[4]) {
    v[0] = make_float2(__uint_as_float(lo.x), __uint_as_float(lo.y));
    v[1] = make_float2(__uint_as_float(lo.z), __uint_as_float(lo.w));
    v[2] = make_float2(__uint_as_float(hi.x), __uint_as_float(hi.y));
    v[3] = make_float2(__uint_as_float(hi.z), __uint_as_float(hi.w));
}

__device__ __forceinline__ float chunk_sum(const float2 (&v)[4]) {
    const float2 s = __fadd2_rn(__fadd2_rn(v[0], v[1]), __fadd2_rn(v[2], v[3]));
    return __fadd_rn(s.x, s.y);
}
// sum (v - mean)^2 (mean 0 for the RMS norm)
__device__ __forceinline__ float chunk_m2(const float2 (&v)[4], float mean) {
    const float2 m = make_float2(-mean, -mean);
    float2 d = __fadd2_rn(v[0], m);
    float2 s = __fmul2_rn(d, d);
#pragma unroll
    for (int i = 1; i < 4; ++i) {
        d = __fadd2_rn(v[i], m);
        s = __ffma2_rn(d, d, s);
    }
    return __fadd_rn(s.x, s.y);
}

// Totals over the warp of N values per lane, part[i * step] = the total of
// s[i]: four at a time, the first two steps halving the values that a lane
// carries (6 exchanges for four totals instead of 20).
template <int N>
__device__ __forceinline__ void warp_totals(const float (&s)[N], int lane, float* part, int step) {
    const bool b0 = lane & 1, b1 = lane & 2;
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const float v0 = s[i], v1 = i + 1 < N ? s[i + 1] : 0.0f, v2 = i + 2 < N ? s[i + 2] : 0.0f,
                    v3 = i + 3 < N ? s[i + 3] : 0.0f;
        float k;
        if (i + 1 < N) {
            // lane bit 0 keeps {v0, v1} or {v2, v3}, bit 1 one of the two
            float k0 = b0 ? v2 : v0, k1 = b0 ? v3 : v1;
            k0 = __fadd_rn(k0, __shfl_xor_sync(0xffffffffu, b0 ? v0 : v2, 1));
            k1 = __fadd_rn(k1, __shfl_xor_sync(0xffffffffu, b0 ? v1 : v3, 1));
            k = __fadd_rn(b1 ? k1 : k0, __shfl_xor_sync(0xffffffffu, b1 ? k0 : k1, 2));
        } else {
            k = __fadd_rn(v0, __shfl_xor_sync(0xffffffffu, v0, 1));
            k = __fadd_rn(k, __shfl_xor_sync(0xffffffffu, k, 2));
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) k = __fadd_rn(k, __shfl_xor_sync(0xffffffffu, k, o));
        const int at = i + 1 < N ? 2 * (lane & 1) + (lane >> 1) : 0;
        if (lane < 4 && i + at < N) part[(i + at) * step] = k;
    }
}

// The row's total from its segments' totals (at most MAX of them), for every
// lane of a warp. Groups of 16 that are not there add zeros. (The trip counts
// are constants: a loop over a run-time count costs three times the
// instructions of its body here.)
template <int MAX>
__device__ __forceinline__ float join_total(const float* part, int nseg, int lane) {
    float sum = 0.0f;
#pragma unroll 1
    for (int s = 0; s < (MAX + 31) / 32 * 32; s += 32) {  // two groups of 16 at a time
        float v = s + lane < nseg ? part[s + lane] : 0.0f;
#pragma unroll
        for (int o = 1; o < 16; o <<= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
        const float w = __shfl_xor_sync(0xffffffffu, v, 16);
        sum = __fadd_rn(sum, lane < 16 ? v : w);
        sum = __fadd_rn(sum, lane < 16 ? w : v);
    }
    return sum;
}
// As join_total for two rows of at most 32 segments at once.
__device__ __forceinline__ float2 join_totals2(const float* part0, const float* part1, int nseg, int lane) {
    const float* part = lane < 16 ? part0 : part1;
    const int s = lane & 15;
    float v = s < nseg ? part[s] : 0.0f, w = s + 16 < nseg ? part[s + 16] : 0.0f;
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) {
        v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, o));
        w = __fadd_rn(w, __shfl_xor_sync(0xffffffffu, w, o));
    }
    v = __fadd_rn(v, w);
    const float other = __shfl_xor_sync(0xffffffffu, v, 16);
    return lane < 16 ? make_float2(v, other) : make_float2(other, v);
}

// The row's mean, sum / D, refined once: with q = sum (1 / D) rounded, the
// residual sum - q D is one fused operation. A constant BF16 row's sum is exact
// (8 bits times at most 65536), the residual of its q exact (a step or two of q
// times D), and the correction gives the constant itself: its deviations are 0.
// (q alone misses it by a step for 95 of the 128 mantissas at 1000 columns, of
// which 1 / sqrt(eps) makes 1e-4 of the constant. A division does the same and
// cost residual_norm with two norms 3 %: 32760 x 5120 BF16, 250 -> 259 us.)
__device__ __forceinline__ float mean_of(float sum, float d, float inv_d) {
    const float q = __fmul_rn(sum, inv_d);
    return __fmaf_rn(__fmaf_rn(-q, d, sum), inv_d, q);
}

// 1 / sqrt(M2 / D + eps), inv_d = 1 / D.
__device__ __forceinline__ float inverse_deviation(float m2, float inv_d, float eps) {
    return rsqrtf(__fmaf_rn(m2, inv_d, eps));
}

// Loads of the rows: each byte is read once, so they bypass L1 (which serves
// the coefficients).
__device__ __forceinline__ uint4 ld_row(const uint4* p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// (x - mean) * rstd on a pair.
__device__ __forceinline__ float2 normalise(float2 x, float2 st) {
    return __fmul2_rn(__fadd2_rn(x, make_float2(-st.x, -st.x)), make_float2(st.y, st.y));
}

// The affine part and the modulation of columns j .. j + 1 as h = n * a + b:
// a = w (1 + scale), b = bias (1 + scale) + shift.
__device__ __forceinline__ void coefficients(const Spec& s, int64_t mrow, int j, float2& a, float2& b) {
    a = make_float2(1.0f, 1.0f);
    if (s.scale) a = __fadd2_rn(a, ptx::ld_f2(s.scale + mrow * s.mod_stride + j));
    b = make_float2(0.0f, 0.0f);
    if (s.bias) b = __fmul2_rn(a, ptx::ld_f2(s.bias + j));
    if (s.shift) b = __fadd2_rn(b, ptx::ld_f2(s.shift + mrow * s.mod_stride + j));
    if (s.weight) a = __fmul2_rn(a, ptx::ld_f2(s.weight + j));
}

// The same for columns j .. j + 3 (j % 4 == 0).
__device__ __forceinline__ void coefficients4(const Spec& s, int64_t mrow, int j, float2 (&a)[2], float2 (&b)[2]) {
    const float2 one = make_float2(1.0f, 1.0f), zero = make_float2(0.0f, 0.0f);
    a[0] = a[1] = one;
    b[0] = b[1] = zero;
    const int64_t at = mrow * s.mod_stride + j;
    if (s.scale) {
        const float4 v = ptx::ld_f4(s.scale + at);
        a[0] = __fadd2_rn(one, make_float2(v.x, v.y));
        a[1] = __fadd2_rn(one, make_float2(v.z, v.w));
    }
    if (s.bias) {
        const float4 v = ptx::ld_f4(s.bias + j);
        b[0] = __fmul2_rn(a[0], make_float2(v.x, v.y));
        b[1] = __fmul2_rn(a[1], make_float2(v.z, v.w));
    }
    if (s.shift) {
        const float4 v = ptx::ld_f4(s.shift + at);
        b[0] = __fadd2_rn(b[0], make_float2(v.x, v.y));
        b[1] = __fadd2_rn(b[1], make_float2(v.z, v.w));
    }
    if (s.weight) {
        const float4 v = ptx::ld_f4(s.weight + j);
        a[0] = __fmul2_rn(a[0], make_float2(v.x, v.y));
        a[1] = __fmul2_rn(a[1], make_float2(v.z, v.w));
    }
}

}  // namespace norm
}  // namespace osm
