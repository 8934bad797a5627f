// Row statistics and coefficients shared by the kernels that normalise rows
// (norm_modulate, residual_norm, norm_quantize_act).
//
// A row of D values is cut into chunks of 8 consecutive columns and segments
// of 32 chunks (256 columns): one lane per chunk, one warp per segment. Each
// segment gives its mean and the sum of squared deviations from that mean,
// and the segments are joined by
//     mean = sum n_s mean_s / D,   M2 = sum M2_s + n_s (mean_s - mean)^2,
// so that the variance never comes from the difference of two large sums and
// the row needs one block barrier. Every addition has a fixed place in the
// tree (lanes joined at distances 1, 2, 4, 8, 16; segments in eight strided
// parts), which does not depend on how a kernel maps segments to warps or
// rows to lanes: all kernels get the same bits for the same row.
#pragma once

#include <cstdint>

#include "osm_mx.cuh"

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

// Sums over the 32 lanes of R values per lane (R = 1, 2 or 4); every lane
// gets all R. With more than one value the first steps halve the values a
// lane carries instead of repeating the exchange for each of them.
template <int R>
__device__ __forceinline__ void warp_sums(float (&s)[R], int lane) {
    if constexpr (R == 1) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) s[0] = __fadd_rn(s[0], __shfl_xor_sync(0xffffffffu, s[0], o));
    } else if constexpr (R == 2) {
        // lane bit 0 = row kept
        const bool odd = lane & 1;
        float k = odd ? s[1] : s[0];
        k = __fadd_rn(k, __shfl_xor_sync(0xffffffffu, odd ? s[0] : s[1], 1));
#pragma unroll
        for (int o = 2; o < 32; o <<= 1) k = __fadd_rn(k, __shfl_xor_sync(0xffffffffu, k, o));
        const float other = __shfl_xor_sync(0xffffffffu, k, 1);
        s[0] = odd ? other : k;
        s[1] = odd ? k : other;
    } else {
        static_assert(R == 4, "1, 2 or 4 rows");
        const bool b0 = lane & 1, b1 = lane & 2;
        // lane bit 0 selects rows {0, 1} or {2, 3}, bit 1 the row of the two
        float k0 = b0 ? s[2] : s[0], k1 = b0 ? s[3] : s[1];
        k0 = __fadd_rn(k0, __shfl_xor_sync(0xffffffffu, b0 ? s[0] : s[2], 1));
        k1 = __fadd_rn(k1, __shfl_xor_sync(0xffffffffu, b0 ? s[1] : s[3], 1));
        float k = b1 ? k1 : k0;
        k = __fadd_rn(k, __shfl_xor_sync(0xffffffffu, b1 ? k0 : k1, 2));
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) k = __fadd_rn(k, __shfl_xor_sync(0xffffffffu, k, o));
        s[0] = __shfl_sync(0xffffffffu, k, 0);
        s[1] = __shfl_sync(0xffffffffu, k, 2);
        s[2] = __shfl_sync(0xffffffffu, k, 1);
        s[3] = __shfl_sync(0xffffffffu, k, 3);
    }
}

// Columns of segment s of a D-column row.
__device__ __forceinline__ int seg_cols(int s, int D) { return min(SEG, D - s * SEG); }

// One segment of R rows: lane `lane` holds chunk `lane` of each row (zeros
// past the end of the row, `live` false there). part[r * stride + seg] =
// (mean, M2) of the segment.
template <int R>
__device__ __forceinline__ void segment_stats(const float2 (&v)[R][4], bool live, bool center, int n, int lane,
                                              float2* part, int stride) {
    float mean[R], m2[R];
    if (center) {
#pragma unroll
        for (int r = 0; r < R; ++r) mean[r] = chunk_sum(v[r]);
        warp_sums<R>(mean, lane);
        const float inv = __frcp_rn(static_cast<float>(n));
#pragma unroll
        for (int r = 0; r < R; ++r) mean[r] = __fmul_rn(mean[r], inv);
    } else {
#pragma unroll
        for (int r = 0; r < R; ++r) mean[r] = 0.0f;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) m2[r] = live ? chunk_m2(v[r], mean[r]) : 0.0f;
    warp_sums<R>(m2, lane);
    if (lane < R) {
        float a = mean[0], b = m2[0];
#pragma unroll
        for (int r = 1; r < R; ++r) {
            a = lane == r ? mean[r] : a;
            b = lane == r ? m2[r] : b;
        }
        part[lane * stride] = make_float2(a, b);
    }
}

// Mean and 1 / sqrt(M2 / D + eps) of one row from its segments (called by
// all lanes of a warp; each group of eight lanes joins a row of its own,
// lanes 8g .. 8g + 7 the segments of `part`, which may differ by group).
__device__ __forceinline__ float2 join_segments(const float2* part, int nseg, int D, bool center, float eps,
                                                int lane) {
    const int p = lane & 7;
    float mean = 0.0f;
    if (center) {
        for (int s = p; s < nseg; s += 8)
            mean = __fmaf_rn(static_cast<float>(seg_cols(s, D)), part[s].x, mean);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) mean = __fadd_rn(mean, __shfl_xor_sync(0xffffffffu, mean, o));
        mean = __fdiv_rn(mean, static_cast<float>(D));
    }
    float m2 = 0.0f;
    for (int s = p; s < nseg; s += 8) {
        const float2 e = part[s];
        const float d = __fadd_rn(e.x, -mean);
        m2 = __fadd_rn(m2, __fmaf_rn(__fmul_rn(d, d), static_cast<float>(seg_cols(s, D)), e.y));
    }
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) m2 = __fadd_rn(m2, __shfl_xor_sync(0xffffffffu, m2, o));
    return make_float2(mean, __frsqrt_rn(__fadd_rn(__fdiv_rn(m2, static_cast<float>(D)), eps)));
}

// Statistics of R rows (<= 4) for every lane: rows in groups of eight lanes.
template <int R>
__device__ __forceinline__ void join_rows(const float2* part, int stride, int nseg, int D, bool center, float eps,
                                          int lane, float2 (&st)[R]) {
    const int row = (lane >> 3) % R;
    const float2 mine = join_segments(part + row * stride, nseg, D, center, eps, lane);
#pragma unroll
    for (int r = 0; r < R; ++r)
        st[r] = make_float2(__shfl_sync(0xffffffffu, mine.x, 8 * r), __shfl_sync(0xffffffffu, mine.y, 8 * r));
}

// (x - mean) * rstd on a pair.
__device__ __forceinline__ float2 normalise(float2 x, float2 st) {
    return __fmul2_rn(__fadd2_rn(x, make_float2(-st.x, -st.x)), make_float2(st.y, st.y));
}

// The affine part and the modulation of columns j .. j + 1 as h = n * a + b:
// a = w (1 + scale), b = bias (1 + scale) + shift.
__device__ __forceinline__ void coefficients(const Spec& s, int64_t mrow, int j, float2& a, float2& b) {
    a = make_float2(1.0f, 1.0f);
    if (s.scale) a = __fadd2_rn(a, __ldg(reinterpret_cast<const float2*>(s.scale + mrow * s.mod_stride + j)));
    b = make_float2(0.0f, 0.0f);
    if (s.bias) b = __fmul2_rn(a, __ldg(reinterpret_cast<const float2*>(s.bias + j)));
    if (s.shift) b = __fadd2_rn(b, __ldg(reinterpret_cast<const float2*>(s.shift + mrow * s.mod_stride + j)));
    if (s.weight) a = __fmul2_rn(a, __ldg(reinterpret_cast<const float2*>(s.weight + j)));
}

}  // namespace norm
}  // namespace osm
