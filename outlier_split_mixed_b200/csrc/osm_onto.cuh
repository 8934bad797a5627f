// The end of a product in tensor memory: scaled, biased, activated, gated,
// added to the residual stream and rounded once, for the GEMM kernels whose
// epilogue warps hold 32 rows x 128 columns of a tile as two slabs of 16 rows
// (tcgen05.ld 16x256b: thread t has rows t / 4 and t / 4 + 8 and, of each
// 8-column block j, columns 2 (t % 4) and the next in registers 4j .. 4j + 3).
//
// Where a warp's 32 rows share a gate row (or there is none), nothing of the
// store loop waits on global memory: the residual words of a slab are in
// registers before its accumulator, those of the second slab loaded as the
// first one's are used up, and bias and gate are in shared memory. The first
// slab's words are loaded while the tile's MMAs still run, except by
// pair_kernel<true> (osm_linear.cu), whose registers are full of sums until
// then. Loaded in the store loop instead they doubled dual_gemm's time at
// 4096 x 5120 x 5120 (104 -> 201 us).
// Where the 32 rows have several gate rows, the store loop loads them from
// global memory: four blocks' at a time in the EACH form, which dual_gemm onto
// BF16 takes for gate rows of fewer than 32 tokens, one at a time in the
// others (4096 x 5120 x 5120, a gate row per token against one for all:
// dual_gemm BF16 95 and 71 us, FP32 123 and 84; linear_hp, which has no EACH
// form, BF16 197 and 181, FP32 318 and 272).
#pragma once

#include <cstdint>
#include <type_traits>

#include "osm_internal.h"
#include "osm_mx.cuh"
#include "osm_ptx.cuh"

namespace osm {
namespace onto {

struct Params {
    int64_t M, N;
    const float* bias;   // [N] or NULL
    void* Y;             // [M][N]; may be onto.r: a thread reads each word of r before it writes that word of Y
    Onto onto;
    float scale;         // of the accumulator (used by SCALED kernels)
    int act;             // OSM_ACT_* (used by ACT kernels)
};

// x / (1 + 2^z) with z = -x log2(e), 2^z and the reciprocal on the special-
// function unit. Where 2^z overflows the reciprocal is 0 and the result -0.
__device__ __forceinline__ float2 silu2(float2 x) {
    const float2 z = __fmul2_rn(x, make_float2(-1.44269504f, -1.44269504f));
    const float2 d = __fadd2_rn(make_float2(mx::ex2_approx(z.x), mx::ex2_approx(z.y)), make_float2(1.0f, 1.0f));
    return __fmul2_rn(x, make_float2(mx::rcp_approx(d.x), mx::rcp_approx(d.y)));
}
__device__ __forceinline__ float2 activate2(float2 v, int act) {
    if (act == OSM_ACT_GELU) return mx::gelu2(v);
    if (act == OSM_ACT_SILU) return silu2(v);
    return v;
}

template <bool F32>
using Word = typename std::conditional<F32, float2, uint32_t>::type;  // two values of the stream

template <bool F32>
__device__ __forceinline__ Word<F32> to_word(float2 v) {
    if constexpr (F32) return v;
    else return mx::bf16x2_bits(v.x, v.y);
}
template <bool F32>
__device__ __forceinline__ float2 from_word(Word<F32> w) {
    if constexpr (F32) return w;
    else return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

// Bias and gate of a warp's 128 columns, when all its rows share a gate row.
struct Vectors {
    float4 bias[32], gate[32];
};

// One warp's part of a tile: rows y0 .. y0 + 31, columns x0 .. x0 + 127. EACH
// (BF16): there is a gate row for every few rows, which is never staged.
template <bool F32, bool EACH = false>
struct Tile {
    int64_t y0, x0;
    int nj;              // 8-column blocks that exist (N % 32 == 0)
    bool staged;         // gate (if any) is in Vectors
    Word<F32> w[32];     // residual words of the slab at hand

    __device__ __forceinline__ static Word<F32>* at(const void* base, const Params& p, int64_t row, int64_t col) {
        return static_cast<Word<F32>*>(const_cast<void*>(base)) + row * (p.N >> 1) + (col >> 1);
    }
    // To be called before the wait for the accumulator.
    __device__ __forceinline__ void prepare(const Params& p, int64_t row0, int64_t col0, int lane, Vectors& v) {
        y0 = row0;
        x0 = col0;
        nj = static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(16), (p.N - x0) >> 3)));
        staged = !EACH;
        if (y0 >= p.M || nj == 0) return;
        uint32_t group = 0;
        if (!EACH && p.onto.gate) {
            const uint32_t share = static_cast<uint32_t>(p.onto.gate_rows);
            group = static_cast<uint32_t>(y0) / share;
            staged = static_cast<uint32_t>(min(y0 + 31, p.M - 1)) / share == group;
        }
        __syncwarp();  // the last tile's readers are done
        const int64_t c = x0 + 4 * lane;
        if (c < p.N) {
            if (p.bias) v.bias[lane] = ptx::ld_f4(p.bias + c);
            if (!EACH && p.onto.gate && staged)
                v.gate[lane] = ptx::ld_f4(p.onto.gate + group * p.onto.gate_stride + c);
        }
        __syncwarp();
        // the residual words are read later: bring them into L2
        const int64_t row = y0 + lane;
        if (p.onto.r && row < p.M) {
            const char* from = reinterpret_cast<const char*>(at(p.onto.r, p, row, x0));
            for (int o = 0; o < nj * 8 * (F32 ? 4 : 2); o += 128)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(from + o));
        }
    }
    // The first slab's residual words; before the wait for the accumulator
    // where the registers allow.
    __device__ __forceinline__ void load_first(const Params& p, int lane) {
        const int64_t ra = y0 + (lane >> 2), rb = ra + 8, col = x0 + 2 * (lane & 3);
        const Word<F32> *pa = at(p.onto.r, p, ra, col), *pb = at(p.onto.r, p, rb, col);
        const int last = p.onto.r ? nj : 0;
        // every word is set, so that none occupies a register before
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            w[2 * j] = j < last && ra < p.M ? pa[4 * j] : Word<F32>{};
            w[2 * j + 1] = j < last && rb < p.M ? pb[4 * j] : Word<F32>{};
        }
    }
    // Slab sl (0, 1) from its 64 accumulator registers, which are used up: four
    // 8-column blocks per turn of a rolled loop, after which registers and
    // residual words move down (they cannot be indexed at run time). Unrolled,
    // the loop's code took several microseconds to fetch the first time (a
    // 256-token F32 call: 7 of its 13 us).
    template <bool SCALED, bool ACT>
    __device__ __forceinline__ void store(const Params& p, int sl, int lane, const Vectors& v, uint32_t* r) {
        const int64_t ra = y0 + 16 * sl + (lane >> 2), rb = ra + 8, c0 = x0 + 2 * (lane & 3);
        const bool on_a = ra < p.M, on_b = rb < p.M, more = p.onto.r != nullptr && sl == 0;
        const bool next_a = more && ra + 16 < p.M, next_b = more && rb + 16 < p.M;
        const float *gate_a = nullptr, *gate_b = nullptr;
        if (EACH || !staged) {  // rows past M read the last row's gate
            const uint32_t last = static_cast<uint32_t>(p.M - 1), share = static_cast<uint32_t>(p.onto.gate_rows);
            gate_a = p.onto.gate + (min(static_cast<uint32_t>(ra), last) / share) * p.onto.gate_stride + c0;
            gate_b = p.onto.gate + (min(static_cast<uint32_t>(rb), last) / share) * p.onto.gate_stride + c0;
        }
        const Word<F32>* na = at(p.onto.r, p, ra + 16, c0);
        const int64_t step = 4 * p.N;  // words between rows 8 apart
        Word<F32>* oa = at(p.Y, p, ra, c0);
        const float2* vb = reinterpret_cast<const float2*>(v.bias) + (lane & 3);
        const float2* vg = reinterpret_cast<const float2*>(v.gate) + (lane & 3);
#pragma unroll 1
        for (int j0 = 0; j0 < nj; j0 += 4) {  // nj is a multiple of 4 (N % 32 == 0)
            float2 ga[4], gb[4];  // EACH: four blocks' gates at once (89 us where one at a time takes 111)
            if constexpr (EACH) {
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    ga[i] = ptx::ld_f2(gate_a + 8 * i);
                    gb[i] = ptx::ld_f2(gate_b + 8 * i);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float2 a = make_float2(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]));
                float2 b = make_float2(__uint_as_float(r[4 * i + 2]), __uint_as_float(r[4 * i + 3]));
                if constexpr (SCALED) {
                    a = __fmul2_rn(a, make_float2(p.scale, p.scale));
                    b = __fmul2_rn(b, make_float2(p.scale, p.scale));
                }
                if (p.bias) {
                    a = __fadd2_rn(a, vb[4 * i]);
                    b = __fadd2_rn(b, vb[4 * i]);
                }
                if constexpr (ACT) {
                    a = activate2(a, p.act);
                    b = activate2(b, p.act);
                }
                if constexpr (EACH) {
                    a = __fmul2_rn(a, ga[i]);
                    b = __fmul2_rn(b, gb[i]);
                } else if (p.onto.gate) {
                    a = __fmul2_rn(a, staged ? vg[4 * i] : ptx::ld_f2(gate_a + 8 * i));
                    b = __fmul2_rn(b, staged ? vg[4 * i] : ptx::ld_f2(gate_b + 8 * i));
                }
                if (p.onto.r) {
                    a = __fadd2_rn(from_word<F32>(w[2 * i]), a);
                    b = __fadd2_rn(from_word<F32>(w[2 * i + 1]), b);
                }
                if (on_a) oa[4 * i] = to_word<F32>(a);
                if (on_b) oa[step + 4 * i] = to_word<F32>(b);
            }
#pragma unroll
            for (int e = 0; e < 48; ++e) r[e] = r[e + 16];
            if (p.onto.r) {
#pragma unroll
                for (int e = 0; e < 24; ++e) w[e] = w[e + 8];
#pragma unroll
                for (int i = 0; i < 4; ++i) {  // the next slab's words of these blocks queue up behind
                    w[24 + 2 * i] = next_a ? na[4 * i] : Word<F32>{};
                    w[25 + 2 * i] = next_b ? na[step + 4 * i] : Word<F32>{};
                }
            }
            oa += 16;
            na += 16;
            vb += 16;
            vg += 16;
            gate_a += 32;
            gate_b += 32;
        }
        // a slab of fewer blocks leaves the queue's head in the wrong place
        if (more)
            for (int j = nj; j < 16; j += 4)
#pragma unroll
                for (int e = 0; e < 24; ++e) w[e] = w[e + 8];
    }
};

}  // namespace onto
}  // namespace osm
