// C ABI of what stands around the layers of a transformer block: the norms
// with their modulation, the gated residual, the products that add to the
// residual stream, and the FFN sublayer made of them. Argument checks only;
// the kernels are in osm_norm.cu, osm_quant.cu, osm_gemm.cu and
// osm_linear.cu.

#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <exception>
#include <new>

#include "osm_internal.h"

namespace osm {
namespace {

bool dtype_ok(int d) { return d == OSM_DT_BF16 || d == OSM_DT_F32; }

// Modulation or gate rows: `rows` tokens share one, rows `stride` floats apart.
int check_rows(const char* who, const char* what, int64_t M, int64_t D, int64_t rows, int64_t stride) {
    OSM_REQUIRE(rows >= 1, "%s: %s needs at least one token per row (%lld)", who, what, (long long)rows);
    OSM_REQUIRE(rows >= M || (stride >= D && stride % 4 == 0 && stride <= (int64_t(1) << 40)),
                "%s: rows of %s are %lld floats apart; need a multiple of 4, at least %lld", who, what,
                (long long)stride, (long long)D);
    return OSM_OK;
}

int check_spec(const char* who, const char* what, const osm_norm_spec* s, int64_t M, int64_t D) {
    OSM_REQUIRE(s->kind == OSM_NORM_LAYER || s->kind == OSM_NORM_RMS, "%s: unknown kind %d of %s", who, s->kind, what);
    OSM_REQUIRE(std::isfinite(s->eps) && s->eps > 0.0f, "%s: eps of %s must be finite and > 0", who, what);
    OSM_REQUIRE(aligned16(s->weight) && aligned16(s->bias) && aligned16(s->scale) && aligned16(s->shift),
                "%s: vectors of %s must be 16-byte aligned", who, what);
    if (s->scale || s->shift) return check_rows(who, what, M, D, s->mod_rows, s->mod_stride);
    return OSM_OK;
}

int check_shape(const char* who, int64_t M, int64_t D) {
    OSM_REQUIRE(M >= 1 && M <= (int64_t(1) << 31) - 1, "%s: need 1 <= M < 2^31", who);
    OSM_REQUIRE(D >= 8 && D <= 65536 && D % 8 == 0, "%s: need 8 <= D <= 65536, D %% 8 == 0 (D=%lld)", who,
                (long long)D);
    return OSM_OK;
}

int check_gate(const char* who, const float* gate, int64_t M, int64_t N, int64_t rows, int64_t stride) {
    if (!gate) return OSM_OK;
    OSM_REQUIRE(aligned16(gate), "%s: gate must be 16-byte aligned", who);
    return check_rows(who, "gate", M, N, rows, stride);
}

// Nothing is thrown across the C boundary.
template <class F>
int guarded(F body) {
    try {
        return body();
    } catch (const std::bad_alloc&) {
        return fail(OSM_ERR_NOMEM, "host allocation failed");
    } catch (const std::exception& e) {
        return fail(OSM_ERR_CUDA, "%s", e.what());
    }
}

Onto onto_of(const void* R, const float* gate, int64_t gate_rows, int64_t gate_stride, int64_t M) {
    return Onto{R, gate, gate ? std::min(gate_rows, M) : M, gate_stride};
}

}  // namespace
}  // namespace osm

using namespace osm;

extern "C" {

int osm_norm_modulate(const void* X, int x_dtype, int64_t M, int64_t D, const osm_norm_spec* spec, uint16_t* H,
                      void* stream) {
    set_error("%s", "");
    OSM_TRY(check_shape("norm_modulate", M, D));
    OSM_REQUIRE(dtype_ok(x_dtype), "norm_modulate: unknown type %d of X", x_dtype);
    OSM_REQUIRE(spec, "norm_modulate: norm is NULL");
    OSM_TRY(check_spec("norm_modulate", "norm", spec, M, D));
    OSM_REQUIRE(X && aligned16(X) && H && aligned16(H), "norm_modulate: X / H null or misaligned");
    OSM_REQUIRE(x_dtype == OSM_DT_BF16 || X != H, "norm_modulate: an FP32 X cannot be normalised in place");
    OSM_TRY(check_device());
    return guarded([&] {
        return launch_norm_rows(X, x_dtype, M, D, nullptr, nullptr, nullptr, 0, 0, 1.0f, spec, nullptr, H,
                                static_cast<cudaStream_t>(stream));
    });
}

int osm_residual_norm(const void* R, int r_dtype, const uint16_t* Y, int64_t M, int64_t D, const osm_norm_spec* post,
                      const float* gate, int64_t gate_rows, int64_t gate_stride, float alpha,
                      const osm_norm_spec* pre, void* R_out, uint16_t* H, void* stream) {
    set_error("%s", "");
    OSM_TRY(check_shape("residual_norm", M, D));
    OSM_REQUIRE(dtype_ok(r_dtype), "residual_norm: unknown type %d of R", r_dtype);
    OSM_REQUIRE(std::isfinite(alpha), "residual_norm: alpha must be finite");
    if (post) {
        OSM_REQUIRE(!post->scale && !post->shift, "residual_norm: post takes no modulation (the gate scales it)");
        OSM_TRY(check_spec("residual_norm", "post", post, M, D));
    }
    if (pre) OSM_TRY(check_spec("residual_norm", "pre", pre, M, D));
    OSM_TRY(check_gate("residual_norm", gate, M, D, gate_rows, gate_stride));
    OSM_REQUIRE(R && aligned16(R) && Y && aligned16(Y) && R_out && aligned16(R_out),
                "residual_norm: R / Y / R_out null or misaligned");
    OSM_REQUIRE(pre ? (H && aligned16(H)) : !H, "residual_norm: H goes with pre (16-byte aligned)");
    OSM_REQUIRE(static_cast<const void*>(H) != R_out && (!H || static_cast<const void*>(H) != R) &&
                    static_cast<const void*>(Y) != R_out,
                "residual_norm: R_out may be R and H may be Y, nothing else");
    OSM_TRY(check_device());
    return guarded([&] {
        return launch_norm_rows(R, r_dtype, M, D, Y, post, gate, gate_rows, gate_stride, alpha, pre, R_out, H,
                                static_cast<cudaStream_t>(stream));
    });
}

int osm_norm_quantize_act(const osm_plan* p, const void* X, int x_dtype, int64_t M, const osm_norm_spec* spec,
                          uint8_t* a_codes, uint8_t* a_scales, uint16_t* a_hp, void* stream) {
    set_error("%s", "");
    OSM_TRY(check_plan(p));
    OSM_TRY(check_shape("norm_quantize_act", M, p->K));
    OSM_REQUIRE(dtype_ok(x_dtype), "norm_quantize_act: unknown type %d of X", x_dtype);
    OSM_REQUIRE(spec, "norm_quantize_act: norm is NULL");
    OSM_TRY(check_spec("norm_quantize_act", "norm", spec, M, p->K));
    OSM_REQUIRE(X && aligned16(X), "norm_quantize_act: X must be a 16-byte aligned device pointer");
    OSM_REQUIRE(p->Kbp == 0 || (a_codes && aligned16(a_codes) && a_scales && aligned16(a_scales)),
                "norm_quantize_act: a_codes / a_scales null or misaligned");
    OSM_REQUIRE(p->kp == 0 || (a_hp && aligned16(a_hp)), "norm_quantize_act: a_hp null or misaligned");
    return guarded([&] {
        return launch_norm_quantize(p, X, x_dtype, M, spec, a_codes, a_scales, a_hp, static_cast<cudaStream_t>(stream));
    });
}

int osm_dual_gemm_residual(const osm_plan* p, const uint8_t* a_codes, const uint8_t* a_scales, const uint16_t* a_hp,
                           int64_t M, const uint8_t* w_codes, const uint8_t* w_scales, const uint16_t* w_hp,
                           const float* bias, const float* gate, int64_t gate_rows, int64_t gate_stride,
                           const void* R, int r_dtype, void* Y, void* stream) {
    set_error("%s", "");
    OSM_TRY(check_plan(p));
    OSM_REQUIRE(M >= 1 && M <= (int64_t(1) << 31) - 1, "dual_gemm_residual: need 1 <= M < 2^31");
    OSM_REQUIRE(dtype_ok(r_dtype), "dual_gemm_residual: unknown type %d of R", r_dtype);
    OSM_REQUIRE(R && aligned16(R) && Y && aligned16(Y), "dual_gemm_residual: R / Y null or misaligned");
    OSM_REQUIRE(!bias || aligned16(bias), "dual_gemm_residual: bias must be 16-byte aligned");
    OSM_TRY(check_gate("dual_gemm_residual", gate, M, p->N, gate_rows, gate_stride));
    OSM_REQUIRE(p->Kbp == 0 || (a_codes && aligned16(a_codes) && a_scales && aligned16(a_scales) && w_codes &&
                                aligned16(w_codes) && w_scales && aligned16(w_scales)),
                "dual_gemm_residual: bulk operands null or misaligned");
    OSM_REQUIRE(p->kp == 0 || (a_hp && aligned16(a_hp) && w_hp && aligned16(w_hp)),
                "dual_gemm_residual: outlier operands null or misaligned");
    OSM_TRY(check_device());
    const Onto onto = onto_of(R, gate, gate_rows, gate_stride, M);
    // gate rows shorter than the 32 rows of an epilogue warp are not staged (4096 x
    // 5120 x 5120 onto BF16, a gate row per token: 89 us, through the staging kernel 111;
    // FP32 rows leave no registers for the form that loads several at once)
    const int epi = r_dtype == OSM_DT_F32 ? EPI_ONTO_F32 : (gate && gate_rows < 32 && M > gate_rows ? EPI_ONTO_EACH : EPI_ONTO_BF16);
    return guarded([&] {
        return launch_dual_gemm(p, a_codes, a_scales, a_hp, M, w_codes, w_scales, w_hp, bias,
                                epi, Y, nullptr, nullptr, nullptr, nullptr, static_cast<cudaStream_t>(stream), &onto);
    });
}

int osm_linear_hp(const osm_plan* p, const uint16_t* X, int64_t M, const uint16_t* w_hp, const float* bias, int act,
                  const float* gate, int64_t gate_rows, int64_t gate_stride, const void* R, void* Y, int y_dtype,
                  void* stream) {
    set_error("%s", "");
    OSM_TRY(check_plan(p));
    OSM_REQUIRE(p->k == p->K && p->unit_s, "linear_hp: needs a plan with k = K and s = 1 (k=%lld, K=%lld)",
                (long long)p->k, (long long)p->K);
    OSM_REQUIRE(!p->hp_fp16, "linear_hp: needs the BF16 outlier branch");
    // an NVFP4 plan's packed slots are w 2^-g_w, and X here is not scaled
    OSM_REQUIRE(p->fmt == OSM_FMT_MXFP4 || p->g_w == 0, "linear_hp: the weights of an NVFP4 plan must be unscaled (g_w = %d)",
                p->g_w);
    OSM_REQUIRE(M >= 1 && M <= (int64_t(1) << 31) - 1, "linear_hp: need 1 <= M < 2^31");
    OSM_REQUIRE(act == OSM_ACT_NONE || act == OSM_ACT_GELU || act == OSM_ACT_SILU, "linear_hp: unknown activation %d",
                act);
    OSM_REQUIRE(dtype_ok(y_dtype), "linear_hp: unknown type %d of Y", y_dtype);
    OSM_REQUIRE(X && aligned16(X) && w_hp && aligned16(w_hp) && Y && aligned16(Y),
                "linear_hp: X / w_hp / Y null or misaligned");
    OSM_REQUIRE(static_cast<const void*>(X) != Y, "linear_hp: Y cannot be X");
    OSM_REQUIRE(aligned16(bias) && aligned16(R), "linear_hp: bias / R misaligned");
    OSM_TRY(check_gate("linear_hp", gate, M, p->N, gate_rows, gate_stride));
    OSM_TRY(check_device());
    return guarded([&] {
        return launch_linear_hp(p, X, M, w_hp, bias, act, onto_of(R, gate, gate_rows, gate_stride, M), Y, y_dtype,
                                static_cast<cudaStream_t>(stream));
    });
}

int osm_ffn_sublayer(const osm_plan* up, const osm_plan* down, const osm_norm_spec* pre, const void* R, int r_dtype,
                     int64_t M, const uint8_t* wu_codes, const uint8_t* wu_scales, const uint16_t* wu_hp,
                     const uint8_t* wd_codes, const uint8_t* wd_scales, const uint16_t* wd_hp, const float* bias_down,
                     const float* gate, int64_t gate_rows, int64_t gate_stride, void* R_out, void* workspace,
                     size_t workspace_bytes, void* stream) {
    set_error("%s", "");
    OSM_TRY(check_plan(up));
    OSM_TRY(check_plan(down));
    OSM_REQUIRE(up->N == down->K, "ffn_sublayer: up->N (%lld) must equal down->K (%lld)", (long long)up->N,
                (long long)down->K);
    OSM_REQUIRE(down->N == up->K, "ffn_sublayer: down->N (%lld) must equal up->K (%lld)", (long long)down->N,
                (long long)up->K);
    OSM_REQUIRE(M >= 1 && M <= (int64_t(1) << 31) - 1, "ffn_sublayer: need 1 <= M < 2^31");
    // what the last call would refuse is refused before the first one runs
    OSM_REQUIRE(dtype_ok(r_dtype), "ffn_sublayer: unknown type %d of R", r_dtype);
    OSM_REQUIRE(R_out && aligned16(R_out), "ffn_sublayer: R_out null or misaligned");
    OSM_REQUIRE(aligned16(bias_down), "ffn_sublayer: bias_down must be 16-byte aligned");
    OSM_TRY(check_gate("ffn_sublayer", gate, M, down->N, gate_rows, gate_stride));
    OSM_REQUIRE(up->fmt == OSM_FMT_MXFP4 && down->fmt == OSM_FMT_MXFP4, "ffn_sublayer: needs MXFP4 plans");
    OSM_REQUIRE((up->Kbp == 0 || (wu_codes && aligned16(wu_codes) && wu_scales && aligned16(wu_scales))) &&
                    (up->kp == 0 || (wu_hp && aligned16(wu_hp))) &&
                    (down->Kbp == 0 || (wd_codes && aligned16(wd_codes) && wd_scales && aligned16(wd_scales))) &&
                    (down->kp == 0 || (wd_hp && aligned16(wd_hp))),
                "ffn_sublayer: packed weights null or misaligned");
    const size_t need = osm_ffn_workspace_size(up, down, M);
    OSM_REQUIRE(workspace && aligned16(workspace) && workspace_bytes >= need,
                "ffn_sublayer: workspace needs %zu bytes", need);
    size_t cu, su, hu, cd, sd, hd;
    osm_plan_sizes(up, M, &cu, &su, &hu);
    osm_plan_sizes(down, M, &cd, &sd, &hd);
    auto align256 = [](size_t x) { return (x + 255) & ~size_t(255); };
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    uint8_t* a_codes = ws;
    ws += align256(cu);
    uint8_t* a_scales = ws;
    ws += align256(su);
    uint16_t* a_hp = reinterpret_cast<uint16_t*>(ws);
    ws += align256(hu);
    uint8_t* h_codes = ws;
    ws += align256(cd);
    uint8_t* h_scales = ws;
    ws += align256(sd);
    uint16_t* h_hp = reinterpret_cast<uint16_t*>(ws);
    OSM_TRY(osm_norm_quantize_act(up, R, r_dtype, M, pre, a_codes, a_scales, a_hp, stream));
    OSM_TRY(osm_dual_gemm(up, a_codes, a_scales, a_hp, M, wu_codes, wu_scales, wu_hp, nullptr, OSM_EPI_GELU_REQUANT,
                          nullptr, down, h_codes, h_scales, h_hp, stream));
    return osm_dual_gemm_residual(down, h_codes, h_scales, h_hp, M, wd_codes, wd_scales, wd_hp, bias_down, gate,
                                  gate_rows, gate_stride, R, r_dtype, R_out, stream);
}

}  // extern "C"
