"""B200 (sm_100a) smoothed, outlier-split W4A4 linear layer.

Python binding of libosm (``include/osm.h``): each function below marshals
torch tensors / numpy arrays into the C entry point of the same name
(``osm_<name>``) and raises :class:`OsmError` on a non-zero return code.
There is no fallback: every computation runs in the CUDA library, and a
missing library raises at first use.

Method: "W4A4 Quantization for Inference on Wan2.2-I2V-A14B" -- SmoothQuant
smoothing (Eq. (1), (2)), a static top-k outlier split (Eq. (4), (5)) and a
dual-branch GEMM whose bulk branch is MXFP4 (E2M1 + E8M0 per 32) and whose
outlier branch is BF16 (Eq. (3)).
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import threading

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libosm.so")

OK = 0
ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_CUDA, ERR_TIMEOUT, ERR_NONFINITE, ERR_NOMEM = 1, 2, 3, 4, 5, 6
STATUS_TIMEOUT = 1
HP_BF16, HP_FP16 = 0, 1
FMT_MXFP4, FMT_NVFP4 = 0, 1
STATUS_NONFINITE = 2
DEBUG_STARVE_QUANTIZE, DEBUG_STARVE_LINEAR = 1, 2
WSCALE_1x32, WSCALE_TILE32x32, WSCALE_STRIP128x1 = 0, 1, 2
EPI_F32, EPI_BF16, EPI_GELU_REQUANT, EPI_GELU_BF16 = 0, 1, 2, 3
DT_BF16, DT_F32 = 0, 1
NORM_LAYER, NORM_RMS = 0, 1
ACT_NONE, ACT_GELU, ACT_SILU = 0, 1, 2

# Every entry point declared in include/osm.h, with its ctypes signature.
_P, _I64, _I, _U64, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_uint64, ctypes.c_size_t
_SIGNATURES = {
    "osm_act_amax_accumulate": (_I, [_P, _I64, _I64, _P, _P]),
    "osm_weight_amax": (_I, [_P, _I64, _I64, _P, _P]),
    "osm_calibrate_finalize": (_I, [_P, _P, _I64, ctypes.c_float, _I64, _P, _P, _P]),
    "osm_plan_create": (_I, [_I64, _I64, _I64, _P, _P, _I, ctypes.POINTER(_P)]),
    "osm_plan_destroy": (_I, [_P]),
    "osm_plan_sizes": (_I, [_P, _I64, ctypes.POINTER(_SZ), ctypes.POINTER(_SZ), ctypes.POINTER(_SZ)]),
    "osm_plan_dims": (_I, [_P] + [ctypes.POINTER(_I64)] * 6),
    "osm_plan_status": (_I, [_P, _P, ctypes.POINTER(ctypes.c_uint32), _I]),
    "osm_plan_set_wait_limit": (_I, [_P, _U64]),
    "osm_plan_set_debug": (_I, [_P, ctypes.c_uint32]),
    "osm_plan_set_outlier_dtype": (_I, [_P, _I]),
    "osm_plan_set_format": (_I, [_P, _I, _I, _I]),
    "osm_nvfp4_tensor_exponent": (_I, [ctypes.c_float, ctypes.POINTER(_I)]),
    "osm_nvfp4_plan_exponents": (_I, [_P, _P, _P, _P, _P, _I64, _I64, ctypes.POINTER(_I), ctypes.POINTER(_I)]),
    "osm_plan_refresh": (_I, [_P, _P, _P, ctypes.c_float, _P]),
    "osm_plan_refresh_scored": (_I, [_P, _P, _P, _P, ctypes.c_float, _P]),
    "osm_act_percentile": (_I, [_P, _I64, _I64, ctypes.c_float, _P, _P]),
    "osm_error_norms": (_I, [_P, _P, _I64, _P, _P]),
    "osm_calibrate_finalize_scored": (_I, [_P, _P, _P, _I64, ctypes.c_float, _I64, _P, _P, _P]),
    "osm_plan_tables": (_I, [_P, _P, _P, _P]),
    "osm_pack_weights": (_I, [_P, _P, _P, _P, _P, _P]),
    "osm_pack_weights_for_next": (_I, [_P, _P, _P, _P, _P, _P, _P]),
    "osm_plan_channel_order": (_I, [_P, _P]),
    "osm_quantize_act": (_I, [_P, _P, _I64, _P, _P, _P, _P]),
    "osm_dual_gemm": (_I, [_P, _P, _P, _P, _I64, _P, _P, _P, _P, _I, _P, _P, _P, _P, _P, _P]),
    "osm_linear_workspace_size": (_SZ, [_P, _I64, _I]),
    "osm_linear_host": (_I, [_P, _P, _I64, _P, _P, _P, _P, _I, _P, _P, _SZ, _P]),
    "osm_scales_to_logical": (_I, [_P, _I64, _I64, _P]),
    "osm_linear_noalloc": (_I, [_P, _P, _I64, _P, _P, _P, _P, _I, _P, _P]),
    "osm_gelu_f32": (_I, [_P, _P, _I64, _P]),
    "osm_ffn_workspace_size": (_SZ, [_P, _P, _I64]),
    "osm_ffn_host_workspace_size": (_SZ, [_P, _P, _I64]),
    "osm_ffn_block": (_I, [_P, _P, _P, _I64, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "osm_ffn_block_host": (_I, [_P, _P, _P, _I64, _P, _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "osm_norm_modulate": (_I, [_P, _I, _I64, _I64, _P, _P, _P]),
    "osm_residual_norm": (_I, [_P, _I, _P, _I64, _I64, _P, _P, _I64, _I64, ctypes.c_float, _P, _P, _P, _P]),
    "osm_norm_quantize_act": (_I, [_P, _P, _I, _I64, _P, _P, _P, _P, _P]),
    "osm_dual_gemm_residual": (_I, [_P, _P, _P, _P, _I64, _P, _P, _P, _P, _P, _I64, _I64, _P, _I, _P, _P]),
    "osm_linear_hp": (_I, [_P, _P, _I64, _P, _P, _I, _P, _I64, _I64, _P, _P, _I, _P]),
    "osm_ffn_sublayer": (_I, [_P, _P, _P, _P, _I, _I64, _P, _P, _P, _P, _P, _P, _P, _P, _I64, _I64, _P, _P, _SZ, _P]),
    "osm_last_error": (ctypes.c_char_p, []),
}

_lock = threading.Lock()
_lib = None


class OsmError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"libosm error {code}: {msg}")
        self.code = code


def lib():
    """The loaded libosm (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(LIB_PATH):
                raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                                   "`python -m outlier_split_mixed_b200.build` (nvcc, sm_100a)")
            L = ctypes.CDLL(LIB_PATH)
            for name, (res, args) in _SIGNATURES.items():
                fn = getattr(L, name)
                fn.restype = res
                fn.argtypes = args
            _lib = L
    return _lib


def last_error() -> str:
    v = lib().osm_last_error()
    return v.decode() if v else ""


def _check(rc: int):
    if rc != OK:
        raise OsmError(rc, last_error())


def _allocating_for(stream, device):
    """A context in which tensors are allocated for the stream that uses them: freed inside the call that uses them there,
    their memory goes to that stream's next allocation, which waits for that use; the current stream's would not."""
    if stream is None:
        return contextlib.nullcontext()
    import torch
    return torch.cuda.stream(torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream)


_raw_stream = None  # torch's current stream of a device, as its address


def _stream(stream):
    global _raw_stream
    if stream is None:
        if _raw_stream is None:
            import torch
            torch.cuda.init()
            _raw_stream = (torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice)
        return _raw_stream[0](_raw_stream[1]())
    return stream if isinstance(stream, int) else stream.cuda_stream


def _ptr(t, name, dtypes=None, numel=None, allow_none=False):
    """Device pointer of a contiguous CUDA tensor (or None)."""
    if (t is not None and t.is_cuda and t.is_contiguous() and (dtypes is None or t.dtype in dtypes)
            and (numel is None or t.nbytes >= numel)):
        return t.data_ptr()
    if t is None:
        if allow_none:
            return None
        raise ValueError(f"{name} is required")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtypes is not None and t.dtype not in dtypes:
        raise ValueError(f"{name} has dtype {t.dtype}, expected one of {dtypes}")
    if numel is not None and t.numel() * t.element_size() < numel:
        raise ValueError(f"{name} holds {t.numel() * t.element_size()} bytes, needs {numel}")
    return t.data_ptr()


def _host_ptr(a: np.ndarray):
    assert a.flags["C_CONTIGUOUS"]
    return ctypes.c_void_p(a.ctypes.data)


_types = {}


def _bf16_types():
    if "bf16" not in _types:
        import torch
        _types["bf16"] = (torch.bfloat16, torch.int16, torch.uint16)
    return _types["bf16"]


def _u8_types():
    if "u8" not in _types:
        import torch
        _types["u8"] = (torch.uint8,)
    return _types["u8"]


# ----------------------------------------------------------------- plans

class Plan:
    """An osm_plan: K, N, k, the smoothing vector s, the outlier set O and
    the weight block-scale mode, with its device tables; optionally the FP16
    outlier branch (hp_fp16) or the NVFP4 bulk format (fmt = FMT_NVFP4 with
    the per-tensor exponents g_act, g_w)."""

    def __init__(self, K: int, N: int, k: int, s: np.ndarray, O: np.ndarray, wscale_mode: int = WSCALE_1x32,
                 hp_fp16: bool = False, fmt: int = FMT_MXFP4, g_act: int = 0, g_w: int = 0):
        s = np.ascontiguousarray(s, dtype=np.float32)
        O = np.ascontiguousarray(O, dtype=np.int32)
        if s.shape != (K,) or O.shape != (k,):
            raise ValueError("s must have shape (K,) and O shape (k,)")
        h = ctypes.c_void_p()
        _check(lib().osm_plan_create(K, N, k, _host_ptr(s), _host_ptr(O) if k else None, int(wscale_mode),
                                     ctypes.byref(h)))
        self._h = h
        self._sizes = {}
        self.s, self.O, self.wscale_mode = s, O, int(wscale_mode)
        d = [ctypes.c_int64() for _ in range(6)]
        _check(lib().osm_plan_dims(self._h, *[ctypes.byref(x) for x in d]))
        self.K, self.N, self.k, self.Kb, self.Kbp, self.kp = (int(x.value) for x in d)
        self.hp_fp16 = bool(hp_fp16)
        if hp_fp16:
            _check(lib().osm_plan_set_outlier_dtype(self._h, HP_FP16))
        self.fmt, self.g_act, self.g_w = FMT_MXFP4, 0, 0
        if fmt != FMT_MXFP4:
            self.set_format(fmt, g_act, g_w)

    def set_format(self, fmt: int, g_act: int = 0, g_w: int = 0):
        """osm_plan_set_format: the 4-bit block format of the bulk branch."""
        _check(lib().osm_plan_set_format(self._h, int(fmt), int(g_act), int(g_w)))
        self.fmt = int(fmt)
        self.g_act, self.g_w = (int(g_act), int(g_w)) if fmt == FMT_NVFP4 else (0, 0)

    @property
    def nblocks(self) -> int:
        """Scale blocks per row: Kbp/32 (MXFP4) or Kbp/16 (NVFP4)."""
        return self.Kbp // (16 if self.fmt == FMT_NVFP4 else 32)

    @property
    def handle(self):
        return self._h

    def sizes(self, rows: int):
        """(codes_bytes, scales_bytes, hp_bytes) for `rows` rows."""
        key = (rows, self.fmt)
        got = self._sizes.get(key)
        if got is None:
            c, s, h = ctypes.c_size_t(), ctypes.c_size_t(), ctypes.c_size_t()
            _check(lib().osm_plan_sizes(self._h, rows, ctypes.byref(c), ctypes.byref(s), ctypes.byref(h)))
            got = int(c.value), int(s.value), int(h.value)
            if len(self._sizes) < 64:
                self._sizes[key] = got
        return got

    def status(self, clear: bool = True, stream=None) -> int:
        v = ctypes.c_uint32()
        _check(lib().osm_plan_status(self._h, _stream(stream), ctypes.byref(v), int(clear)))
        return int(v.value)

    def channel_order(self) -> np.ndarray:
        """[J ascending | O ascending] (osm_plan_channel_order)."""
        out = np.empty(self.K, np.int32)
        _check(lib().osm_plan_channel_order(self._h, _host_ptr(out)))
        return out

    def set_wait_limit(self, ns: int):
        _check(lib().osm_plan_set_wait_limit(self._h, int(ns)))

    def set_debug(self, flags: int):
        _check(lib().osm_plan_set_debug(self._h, int(flags)))

    def refresh(self, amax, wmax, alpha: float, stream=None):
        """Re-calibrate on the device from device statistics (osm_plan_refresh):
        s, inv_s, O and the routing tables are rebuilt; pack the weights again."""
        import torch
        _check(lib().osm_plan_refresh(self._h, _ptr(amax, "amax", (torch.float32,), self.K * 4),
                                      _ptr(wmax, "wmax", (torch.float32,), self.K * 4), float(alpha),
                                      _stream(stream)))

    def refresh_scored(self, amax, score, wmax, alpha: float, stream=None):
        """As refresh, with the top-k by `score` (osm_plan_refresh_scored)."""
        import torch
        f32 = (torch.float32,)
        _check(lib().osm_plan_refresh_scored(self._h, _ptr(amax, "amax", f32, self.K * 4),
                                             _ptr(score, "score", f32, self.K * 4),
                                             _ptr(wmax, "wmax", f32, self.K * 4), float(alpha), _stream(stream)))

    def tables(self):
        """(s, inv_s, O) copied to host numpy arrays (osm_plan_tables)."""
        s = np.empty(self.K, np.float32)
        inv_s = np.empty(self.K, np.float32)
        O = np.empty(max(self.k, 1), np.int32)
        _check(lib().osm_plan_tables(self._h, _host_ptr(s), _host_ptr(inv_s), _host_ptr(O)))
        return s, inv_s, O[:self.k].copy()

    def alloc_packed(self, rows: int, device="cuda"):
        """Allocate (codes, scales, hp) torch buffers for `rows` rows."""
        import torch
        cb, sb, hb = self.sizes(rows)
        codes = torch.empty(max(cb, 16), dtype=torch.uint8, device=device)[:cb]
        scales = torch.empty(max(sb, 16), dtype=torch.uint8, device=device)[:sb]
        hp = torch.empty(max(hb // 2, 8), dtype=torch.bfloat16, device=device)[:hb // 2]
        return codes, scales, hp

    def close(self):
        if getattr(self, "_h", None):
            lib().osm_plan_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ----------------------------------------------------------------- calibration

def act_amax_accumulate(X, amax, stream=None):
    """amax = max(amax, max_t |X[t]|) on the device (osm_act_amax_accumulate)."""
    T, K = X.shape
    import torch
    _check(lib().osm_act_amax_accumulate(_ptr(X, "X", _bf16_types()), T, K,
                                         _ptr(amax, "amax", (torch.float32,), K * 4), _stream(stream)))


def act_percentile(X, q: float, score, stream=None):
    """score[j] = nearest-rank q-percentile of |X[:, j]| on the device (osm_act_percentile)."""
    T, K = X.shape
    import torch
    _check(lib().osm_act_percentile(_ptr(X, "X", _bf16_types()), T, K, float(q),
                                    _ptr(score, "score", (torch.float32,), K * 4), _stream(stream)))


def error_norms(Y, Yref, stream=None):
    """(sum (Y - Yref)^2, sum Yref^2) in FP64 on the device (osm_error_norms)."""
    import torch
    if Y.shape != Yref.shape:
        raise ValueError("Y and Yref differ in shape")
    with _allocating_for(stream, Y.device):
        out = torch.zeros(2, dtype=torch.float64, device=Y.device)
        _check(lib().osm_error_norms(_ptr(Y, "Y", (torch.float32,)), _ptr(Yref, "Yref", (torch.float32,)), Y.numel(),
                                     _ptr(out, "out", (torch.float64,)), _stream(stream)))
        e, n = out.cpu().tolist()
    return e, n


def gelu_f32(x, y=None, stream=None):
    """The FFN epilogues' FP32 GELU routine element-wise (osm_gelu_f32)."""
    import torch
    if y is None:
        with _allocating_for(stream, x.device):
            y = torch.empty_like(x)
    if x.dtype != torch.float32 or y.dtype != torch.float32 or x.numel() != y.numel():
        raise ValueError("x and y must be float32 tensors of one size")
    _check(lib().osm_gelu_f32(_ptr(x, "x"), _ptr(y, "y"), x.numel(), _stream(stream)))
    return y


def weight_amax(W, wmax, stream=None):
    """wmax[j] = max_n |W[j][n]| (osm_weight_amax)."""
    K, N = W.shape
    import torch
    _check(lib().osm_weight_amax(_ptr(W, "W", _bf16_types()), K, N, _ptr(wmax, "wmax", (torch.float32,), K * 4),
                                 _stream(stream)))


def calibrate_finalize(amax_host: np.ndarray, wmax_host: np.ndarray, alpha: float, k: int):
    """Eq. (2) and Eq. (4) on host statistics -> (s, inv_s, O) (osm_calibrate_finalize)."""
    amax_host = np.ascontiguousarray(amax_host, dtype=np.float32)
    wmax_host = np.ascontiguousarray(wmax_host, dtype=np.float32)
    K = amax_host.shape[0]
    s = np.empty(K, np.float32)
    inv_s = np.empty(K, np.float32)
    O = np.empty(max(k, 1), np.int32)
    _check(lib().osm_calibrate_finalize(_host_ptr(amax_host), _host_ptr(wmax_host), K, float(alpha), int(k),
                                        _host_ptr(s), _host_ptr(inv_s), _host_ptr(O)))
    return s, inv_s, O[:k].copy()


def nvfp4_tensor_exponent(amax: float) -> int:
    """osm_nvfp4_tensor_exponent: smallest g in [-100, 100] with amax <= 6 * 448 * 2^g."""
    g = ctypes.c_int()
    _check(lib().osm_nvfp4_tensor_exponent(float(amax), ctypes.byref(g)))
    return int(g.value)


def nvfp4_plan_exponents(amax_host, wmax_host, s, inv_s, O):
    """osm_nvfp4_plan_exponents: (g_act, g_w) from the calibration statistics."""
    a = np.ascontiguousarray(amax_host, dtype=np.float32)
    w = np.ascontiguousarray(wmax_host, dtype=np.float32)
    s = np.ascontiguousarray(s, dtype=np.float32)
    inv_s = np.ascontiguousarray(inv_s, dtype=np.float32)
    O = np.ascontiguousarray(O, dtype=np.int32)
    ga, gw = ctypes.c_int(), ctypes.c_int()
    _check(lib().osm_nvfp4_plan_exponents(_host_ptr(a), _host_ptr(w), _host_ptr(s), _host_ptr(inv_s),
                                          _host_ptr(O) if O.size else None, a.shape[0], O.shape[0],
                                          ctypes.byref(ga), ctypes.byref(gw)))
    return int(ga.value), int(gw.value)


def calibrate_finalize_scored(amax_host: np.ndarray, score_host: np.ndarray, wmax_host: np.ndarray, alpha: float,
                              k: int):
    """Eq. (2) from amax, Eq. (4)'s top-k by score -> (s, inv_s, O) (osm_calibrate_finalize_scored)."""
    amax_host = np.ascontiguousarray(amax_host, dtype=np.float32)
    score_host = np.ascontiguousarray(score_host, dtype=np.float32)
    wmax_host = np.ascontiguousarray(wmax_host, dtype=np.float32)
    K = amax_host.shape[0]
    s = np.empty(K, np.float32)
    inv_s = np.empty(K, np.float32)
    O = np.empty(max(k, 1), np.int32)
    _check(lib().osm_calibrate_finalize_scored(_host_ptr(amax_host), _host_ptr(score_host), _host_ptr(wmax_host), K,
                                               float(alpha), int(k), _host_ptr(s), _host_ptr(inv_s), _host_ptr(O)))
    return s, inv_s, O[:k].copy()


# ----------------------------------------------------------------- layer path

def pack_weights(plan: Plan, W, w_codes, w_scales, w_hp, stream=None):
    """Fold s into W and pack it (osm_pack_weights). W: [K][N] BF16."""
    cb, sb, hb = plan.sizes(plan.N)
    if tuple(W.shape) != (plan.K, plan.N):
        raise ValueError("W must have shape (K, N)")
    _check(lib().osm_pack_weights(plan.handle, _ptr(W, "W", _bf16_types()),
                                  _ptr(w_codes, "w_codes", _u8_types(), cb, allow_none=cb == 0),
                                  _ptr(w_scales, "w_scales", _u8_types(), sb, allow_none=sb == 0),
                                  _ptr(w_hp, "w_hp", _bf16_types(), hb, allow_none=hb == 0), _stream(stream)))


def pack_weights_for_next(plan: Plan, next_plan: Plan, W, w_codes, w_scales, w_hp, stream=None):
    """Pack W with its output columns in next_plan's channel order
    (osm_pack_weights_for_next), for OSM_EPI_GELU_REQUANT."""
    cb, sb, hb = plan.sizes(plan.N)
    if tuple(W.shape) != (plan.K, plan.N):
        raise ValueError("W must have shape (K, N)")
    _check(lib().osm_pack_weights_for_next(plan.handle, next_plan.handle, _ptr(W, "W", _bf16_types()),
                                           _ptr(w_codes, "w_codes", _u8_types(), cb, allow_none=cb == 0),
                                           _ptr(w_scales, "w_scales", _u8_types(), sb, allow_none=sb == 0),
                                           _ptr(w_hp, "w_hp", _bf16_types(), hb, allow_none=hb == 0), _stream(stream)))


def quantize_act(plan: Plan, X, a_codes, a_scales, a_hp, stream=None):
    """Smooth, split and MXFP4-encode activations (osm_quantize_act). X: [M][K] BF16."""
    M, K = X.shape
    if K != plan.K:
        raise ValueError("X must have K columns")
    cb, sb, hb = plan.sizes(M)
    _check(lib().osm_quantize_act(plan.handle, _ptr(X, "X", _bf16_types()), M,
                                  _ptr(a_codes, "a_codes", _u8_types(), cb, allow_none=cb == 0),
                                  _ptr(a_scales, "a_scales", _u8_types(), sb, allow_none=sb == 0),
                                  _ptr(a_hp, "a_hp", _bf16_types(), hb, allow_none=hb == 0), _stream(stream)))


def dual_gemm(plan: Plan, a_codes, a_scales, a_hp, M: int, w_codes, w_scales, w_hp, Y, bias=None,
              epi: int = EPI_F32, stream=None, next_plan: Plan | None = None, next_buffers=None):
    """Eq. (5) on packed operands (osm_dual_gemm). Y: [M][N] float32 or BF16.
    With epi=EPI_GELU_REQUANT, Y and bias are None and next_buffers are the
    (codes, scales, hp) of next_plan for M rows."""
    import torch
    cbm, sbm, hbm = plan.sizes(M)
    cbn, sbn, hbn = plan.sizes(plan.N)
    if epi == EPI_GELU_REQUANT:
        if next_plan is None or next_buffers is None or Y is not None or bias is not None:
            raise ValueError("GELU_REQUANT needs next_plan and next_buffers, and no Y or bias")
        ncb, nsb, nhb = next_plan.sizes(M)
        nc, ns, nh = next_buffers
        _check(lib().osm_dual_gemm(plan.handle,
                                   _ptr(a_codes, "a_codes", _u8_types(), cbm, allow_none=cbm == 0),
                                   _ptr(a_scales, "a_scales", _u8_types(), sbm, allow_none=sbm == 0),
                                   _ptr(a_hp, "a_hp", _bf16_types(), hbm, allow_none=hbm == 0), M,
                                   _ptr(w_codes, "w_codes", _u8_types(), cbn, allow_none=cbn == 0),
                                   _ptr(w_scales, "w_scales", _u8_types(), sbn, allow_none=sbn == 0),
                                   _ptr(w_hp, "w_hp", _bf16_types(), hbn, allow_none=hbn == 0),
                                   None, int(epi), None, next_plan.handle,
                                   _ptr(nc, "next_codes", _u8_types(), ncb, allow_none=ncb == 0),
                                   _ptr(ns, "next_scales", _u8_types(), nsb, allow_none=nsb == 0),
                                   _ptr(nh, "next_hp", _bf16_types(), nhb, allow_none=nhb == 0), _stream(stream)))
        return
    ybytes = M * plan.N * (4 if epi == EPI_F32 else 2)
    u8, bf = _u8_types(), _bf16_types()
    ytypes = (torch.float32,) if epi == EPI_F32 else bf
    _check(lib().osm_dual_gemm(plan.handle,
                               _ptr(a_codes, "a_codes", u8, cbm, allow_none=cbm == 0),
                               _ptr(a_scales, "a_scales", u8, sbm, allow_none=sbm == 0),
                               _ptr(a_hp, "a_hp", bf, hbm, allow_none=hbm == 0), M,
                               _ptr(w_codes, "w_codes", u8, cbn, allow_none=cbn == 0),
                               _ptr(w_scales, "w_scales", u8, sbn, allow_none=sbn == 0),
                               _ptr(w_hp, "w_hp", bf, hbn, allow_none=hbn == 0),
                               _ptr(bias, "bias", (torch.float32,), plan.N * 4, allow_none=True), int(epi),
                               _ptr(Y, "Y", ytypes, ybytes), None, None, None, None, _stream(stream)))


def linear_workspace_size(plan: Plan, M: int, epi: int = EPI_F32) -> int:
    return int(lib().osm_linear_workspace_size(plan.handle, M, int(epi)))


def linear_host(plan: Plan, X_host, M: int, w_codes, w_scales, w_hp, Y_host, workspace, bias=None,
                epi: int = EPI_F32, stream=None):
    """Host X -> device quantize + dual GEMM -> host Y (osm_linear_host).
    X_host / Y_host: pinned CPU torch tensors; the caller synchronises."""
    import torch
    for t, n in ((X_host, "X_host"), (Y_host, "Y_host")):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous host tensor")
    cbn, sbn, hbn = plan.sizes(plan.N)
    _check(lib().osm_linear_host(plan.handle, ctypes.c_void_p(X_host.data_ptr()), M,
                                 _ptr(w_codes, "w_codes", _u8_types(), cbn, allow_none=cbn == 0),
                                 _ptr(w_scales, "w_scales", _u8_types(), sbn, allow_none=sbn == 0),
                                 _ptr(w_hp, "w_hp", _bf16_types(), hbn, allow_none=hbn == 0),
                                 _ptr(bias, "bias", (torch.float32,), plan.N * 4, allow_none=True), int(epi),
                                 ctypes.c_void_p(Y_host.data_ptr()), _ptr(workspace, "workspace"),
                                 workspace.numel() * workspace.element_size(), _stream(stream)))


def ffn_workspace_size(up: Plan, down: Plan, M: int) -> int:
    """Device bytes osm_ffn_block needs for M tokens (both layers' packed activations)."""
    return int(lib().osm_ffn_workspace_size(up.handle, down.handle, M))


def ffn_host_workspace_size(up: Plan, down: Plan, M: int) -> int:
    """Device bytes osm_ffn_block_host needs for M tokens."""
    return int(lib().osm_ffn_host_workspace_size(up.handle, down.handle, M))


def _ffn_weight_ptrs(up: Plan, down: Plan, wu, wd):
    cu, su, hu = up.sizes(up.N)
    cd, sd, hd = down.sizes(down.N)
    return (_ptr(wu[0], "wu_codes", _u8_types(), cu, allow_none=cu == 0),
            _ptr(wu[1], "wu_scales", _u8_types(), su, allow_none=su == 0),
            _ptr(wu[2], "wu_hp", _bf16_types(), hu, allow_none=hu == 0),
            _ptr(wd[0], "wd_codes", _u8_types(), cd, allow_none=cd == 0),
            _ptr(wd[1], "wd_scales", _u8_types(), sd, allow_none=sd == 0),
            _ptr(wd[2], "wd_hp", _bf16_types(), hd, allow_none=hd == 0))


def ffn_block(up: Plan, down: Plan, X, wu, wd, Y, workspace, bias_down=None, stream=None):
    """One FFN block on the device (osm_ffn_block): quantize_act(up), the
    up-projection with the fused GELU + smoothing + requantisation epilogue,
    the down-projection to BF16. wu = (codes, scales, hp) packed by
    pack_weights_for_next(up, down), wd packed by pack_weights(down).
    X: [M][up.K] BF16, Y: [M][down.N] BF16, both CUDA tensors."""
    import torch
    M, K = X.shape
    if K != up.K or tuple(Y.shape) != (M, down.N):
        raise ValueError("X must be [M][up.K] and Y [M][down.N]")
    _check(lib().osm_ffn_block(up.handle, down.handle, _ptr(X, "X", _bf16_types()), M,
                               *_ffn_weight_ptrs(up, down, wu, wd),
                               _ptr(bias_down, "bias_down", (torch.float32,), down.N * 4, allow_none=True),
                               _ptr(Y, "Y", _bf16_types(), M * down.N * 2), _ptr(workspace, "workspace"),
                               workspace.numel() * workspace.element_size(), _stream(stream)))


def ffn_block_host(up: Plan, down: Plan, X_host, wu, wd, Y_host, workspace, bias_down=None, stream=None):
    """osm_ffn_block_host: host (pinned) X in, the block on the device, host
    Y out, all enqueued on `stream`; the caller synchronises."""
    import torch
    for t, n in ((X_host, "X_host"), (Y_host, "Y_host")):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{n} must be a contiguous host tensor")
    M, K = X_host.shape
    if K != up.K or tuple(Y_host.shape) != (M, down.N):
        raise ValueError("X_host must be [M][up.K] and Y_host [M][down.N]")
    _check(lib().osm_ffn_block_host(up.handle, down.handle, ctypes.c_void_p(X_host.data_ptr()), M,
                                    *_ffn_weight_ptrs(up, down, wu, wd),
                                    _ptr(bias_down, "bias_down", (torch.float32,), down.N * 4, allow_none=True),
                                    ctypes.c_void_p(Y_host.data_ptr()), _ptr(workspace, "workspace"),
                                    workspace.numel() * workspace.element_size(), _stream(stream)))


NOALLOC_SCRATCH_BYTES = 16 << 20


def linear_noalloc(plan: Plan, X, w_codes, w_scales, w_hp, Y, bias=None, epi: int = EPI_F32, stream=None):
    """quantize_act + dual_gemm with the packed activations in the library's
    static scratch (osm_linear_noalloc): nothing is allocated, for callers
    that cannot allocate device memory at run time (a runtime whose pool
    owns the GPU's memory, a plug-in handed only tensors and a stream).
    Calls that overlap on the GPU race on the shared scratch; the first call
    on a device looks up the scratch address and should precede any stream
    capture."""
    import torch
    M, K = X.shape
    if K != plan.K:
        raise ValueError("X must have K columns")
    cbn, sbn, hbn = plan.sizes(plan.N)
    ybytes = M * plan.N * (4 if epi == EPI_F32 else 2)
    ytypes = (torch.float32,) if epi == EPI_F32 else _bf16_types()
    _check(lib().osm_linear_noalloc(plan.handle, _ptr(X, "X", _bf16_types()), M,
                                    _ptr(w_codes, "w_codes", _u8_types(), cbn, allow_none=cbn == 0),
                                    _ptr(w_scales, "w_scales", _u8_types(), sbn, allow_none=sbn == 0),
                                    _ptr(w_hp, "w_hp", _bf16_types(), hbn, allow_none=hbn == 0),
                                    _ptr(bias, "bias", (torch.float32,), plan.N * 4, allow_none=True), int(epi),
                                    _ptr(Y, "Y", ytypes, ybytes), _stream(stream)))


def scales_to_logical(swizzled: np.ndarray, rows: int, nblocks: int) -> np.ndarray:
    """Un-swizzle a scales buffer into [rows][nblocks] (osm_scales_to_logical)."""
    swizzled = np.ascontiguousarray(swizzled, dtype=np.uint8)
    out = np.zeros((rows, nblocks), np.uint8)
    if rows and nblocks:
        _check(lib().osm_scales_to_logical(_host_ptr(swizzled), rows, nblocks, _host_ptr(out)))
    return out


# ----------------------------------------------------------------- around the layers

class _NormSpec(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("eps", ctypes.c_float), ("weight", _P), ("bias", _P), ("scale", _P),
                ("shift", _P), ("mod_rows", _I64), ("mod_stride", _I64)]


def _device() -> int:
    """The current device, where the kernels are launched."""
    if _raw_stream is None:
        _stream(None)
    return _raw_stream[1]()


def _operand(t, name, dtypes, shape, dev):
    """Address of a contiguous tensor of this type and shape on device `dev`."""
    if t.get_device() == dev and t.dtype in dtypes and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    _ptr(t, name, dtypes)
    if t.get_device() != dev:
        raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")
    raise ValueError(f"{name} has shape {tuple(t.shape)}, needs {tuple(shape)}")


def _stream_types():
    """The types a residual stream can have, with their DT_* codes."""
    if "stream" not in _types:
        import torch
        _types["stream"] = {torch.bfloat16: DT_BF16, torch.float32: DT_F32}
        _types["f32"], _types["bf16 alone"] = (torch.float32,), (torch.bfloat16,)
    return _types["stream"]


def _stream_type(t, name):
    code = _stream_types().get(t.dtype)
    if code is None:
        raise ValueError(f"{name} has dtype {t.dtype}, expected torch.bfloat16 or torch.float32")
    return code


def _vector(t, name, D, dev):
    return None if t is None else _operand(t, name, _types["f32"], (D,), dev)


def _shared_rows(t, name, M, D, rows, dev):
    """(address, rows, stride) of modulation or gate rows: [D] (one row), or [B][D] whose rows may lie apart (a slice
    of a wider tensor); `rows` tokens share a row (default: M tokens in B equal parts)."""
    if t is None:
        return None, 1, 0
    s = t.shape
    if len(s) not in (1, 2) or t.dtype not in _types["f32"] or t.get_device() != dev:
        if t.is_cuda and t.dtype in _types["f32"] and len(s) in (1, 2):
            raise ValueError(f"{name} is on {t.device}, the current device is cuda:{dev}")
        raise ValueError(f"{name} must be a float32 CUDA tensor [D] or [B][D]")
    stride = t.stride()
    if s[-1] != D or stride[-1] != 1:
        raise ValueError(f"{name} needs {D} contiguous columns")
    B, step = (1, D) if len(s) == 1 else (s[0], stride[0])
    if rows is None:
        if B < 1 or M % B:
            raise ValueError(f"{name} has {B} rows for {M} tokens: say how many tokens share one")
        rows = M // B
    if rows < 1 or -(-M // rows) > B:
        raise ValueError(f"{name} has {B} rows, {M} tokens by {rows} need {-(-M // max(rows, 1))}")
    return t.data_ptr(), rows, step


class Norm:
    """A norm (NORM_LAYER or NORM_RMS) with its affine part (weight, bias: [D] float32) and its modulation (scale,
    shift: [D] or [B][D] float32, `mod_rows` tokens to a row): osm_norm_spec. Holds its tensors."""

    def __init__(self, kind: int = NORM_LAYER, eps: float = 1e-6, weight=None, bias=None, scale=None, shift=None,
                 mod_rows: int | None = None):
        self.kind, self.eps, self.weight, self.bias = kind, eps, weight, bias
        self.scale, self.shift, self.mod_rows = scale, shift, mod_rows

    def spec(self, M: int, D: int, dev: int | None = None) -> _NormSpec:
        _stream_types()
        if dev is None:
            dev = self._any_device()
        a, b = self.scale, self.shift
        scale, rows, stride = _shared_rows(a, "scale", M, D, self.mod_rows, dev)
        if b is None:
            shift = None
        elif a is not None and b.shape == a.shape and b.stride() == a.stride() and b.dtype == a.dtype and b.device == a.device:
            shift = b.data_ptr()
        else:
            shift, rows2, stride2 = _shared_rows(b, "shift", M, D, self.mod_rows, dev)
            if a is None:
                rows, stride = rows2, stride2
            elif rows2 != rows or (rows < M and stride2 != stride):
                raise ValueError("scale and shift must have the same rows and row stride")
        return _NormSpec(self.kind, self.eps, _vector(self.weight, "weight", D, dev), _vector(self.bias, "bias", D, dev),
                         scale, shift, rows, stride)

    def _any_device(self) -> int:
        for t in (self.scale, self.shift, self.weight, self.bias):
            if t is not None and t.is_cuda:
                return t.get_device()
        return -2  # no device: tensors of the host are refused


def _new(shape, dtype, like, stream):
    """An output tensor, allocated for the stream that will write it."""
    import torch
    with _allocating_for(stream, like.device):
        return torch.empty(shape, dtype=dtype, device=like.device)


def norm_modulate(X, norm: Norm, out=None, stream=None):
    """H = bf16(norm(X)) (osm_norm_modulate). X: [M][D] BF16 or float32; out: [M][D] BF16 (may be X)."""
    M, D = shape = X.shape
    code = _stream_type(X, "X")
    dev = _device() if X.is_cuda else -2
    bf = _types["bf16 alone"]
    x = _operand(X, "X", _types["stream"], shape, dev)
    if out is None:
        out = _new(shape, bf[0], X, stream)
    _check(lib().osm_norm_modulate(x, code, M, D,
                                   ctypes.byref(norm.spec(M, D, dev)), _operand(out, "out", bf, shape, dev),
                                   _stream(stream)))
    return out


def residual_norm(R, Y, gate=None, gate_rows: int | None = None, alpha: float = 1.0, post: Norm | None = None,
                  pre: Norm | None = None, out=None, h=None, stream=None):
    """(R + alpha * gate * post(Y), pre of it in BF16 or None) (osm_residual_norm). R: [M][D] BF16 or float32, Y: [M][D]
    BF16; out may be R, h may be Y."""
    M, D = shape = R.shape
    code = _stream_type(R, "R")
    if pre is None and h is not None:
        raise ValueError("h goes with pre")
    dev = _device() if R.is_cuda else -2
    own, bf = (R.dtype,), _types["bf16 alone"]
    r = _operand(R, "R", own, shape, dev)
    if out is None:
        out = _new(shape, R.dtype, R, stream)
    if pre is not None and h is None:
        h = _new(shape, bf[0], R, stream)
    g, rows, stride = _shared_rows(gate, "gate", M, D, gate_rows, dev)
    _check(lib().osm_residual_norm(r, code, _operand(Y, "Y", bf, shape, dev), M, D,
                                   None if post is None else ctypes.byref(post.spec(M, D, dev)), g, rows, stride, alpha,
                                   None if pre is None else ctypes.byref(pre.spec(M, D, dev)),
                                   _operand(out, "out", own, shape, dev),
                                   None if h is None else _operand(h, "h", bf, shape, dev), _stream(stream)))
    return out, h


def _packed_ptrs(plan: Plan, rows: int, codes, scales, hp, which: str, dev: int):
    """Addresses of packed operands, with their sizes checked."""
    cb, sb, hb = plan.sizes(rows)
    u8, bf = _u8_types(), _bf16_types()
    if cb and hb:  # the usual layer: bulk and outlier channels
        got = _ptr(codes, f"{which}_codes", u8, cb), _ptr(scales, f"{which}_scales", u8, sb), _ptr(hp, f"{which}_hp", bf, hb)
        if codes.get_device() == dev and scales.get_device() == dev and hp.get_device() == dev:
            return got
    got = []
    for t, n, types, name in ((codes, cb, u8, "codes"), (scales, sb, u8, "scales"), (hp, hb, bf, "hp")):
        if n == 0 and (t is None or t.numel() == 0):
            got.append(None)
            continue
        p = _ptr(t, f"{which}_{name}", types, n)
        if t.get_device() != dev:
            raise ValueError(f"{which}_{name} is on {t.device}, the current device is cuda:{dev}")
        got.append(p)
    return got


def norm_quantize_act(plan: Plan, X, norm: Norm, a_codes, a_scales, a_hp, stream=None):
    """quantize_act of norm_modulate(X) in one pass (osm_norm_quantize_act). X: [M][plan.K] BF16 or float32. With more
    than 5120 columns and many rows the two calls are faster."""
    M, K = X.shape[0], plan.K
    code = _stream_type(X, "X")
    dev = _device()
    _check(lib().osm_norm_quantize_act(plan.handle, _operand(X, "X", _types["stream"], (M, K), dev), code, M,
                                       ctypes.byref(norm.spec(M, K, dev)),
                                       *_packed_ptrs(plan, M, a_codes, a_scales, a_hp, "a", dev), _stream(stream)))


def dual_gemm_residual(plan: Plan, a_codes, a_scales, a_hp, M: int, w_codes, w_scales, w_hp, R, out=None, bias=None,
                       gate=None, gate_rows: int | None = None, stream=None):
    """R + gate * (the dual-branch product + bias) (osm_dual_gemm_residual). R: [M][N] BF16 or float32; out may be R."""
    N = plan.N
    shape, code, own, dev = (M, N), _stream_type(R, "R"), (R.dtype,), _device()
    if out is None:
        out = _new(shape, R.dtype, R, stream)
    g, rows, stride = _shared_rows(gate, "gate", M, N, gate_rows, dev)
    _check(lib().osm_dual_gemm_residual(plan.handle, *_packed_ptrs(plan, M, a_codes, a_scales, a_hp, "a", dev), M,
                                        *_packed_ptrs(plan, N, w_codes, w_scales, w_hp, "w", dev),
                                        _vector(bias, "bias", N, dev), g, rows, stride,
                                        _operand(R, "R", own, shape, dev), code, _operand(out, "out", own, shape, dev),
                                        _stream(stream)))
    return out


def hp_plan(K: int, N: int) -> Plan:
    """The plan of a layer kept in BF16: every channel on the outlier branch (k = K), no smoothing (s = 1)."""
    return Plan(K, N, K, np.ones(K, np.float32), np.arange(K, dtype=np.int32))


def linear_hp(plan: Plan, X, w_hp, bias=None, act: int = ACT_NONE, gate=None, gate_rows: int | None = None,
              residual=None, out=None, dtype=None, stream=None):
    """[residual +] [gate *] act(X W + bias) in BF16 (osm_linear_hp). plan: hp_plan(K, N); X: [M][K] BF16; w_hp: packed
    by pack_weights; the output is BF16 or float32 (out's type, residual's, or dtype; BF16 by default). out may be
    residual."""
    M, N = X.shape[0], plan.N
    shape, bf = (M, N), _bf16_types()
    _stream_types()
    if out is None:
        out = _new(shape, residual.dtype if residual is not None else dtype or _types["bf16 alone"][0], X, stream)
    if dtype is not None and out.dtype != dtype:
        raise ValueError(f"the output has dtype {out.dtype}, dtype says {dtype}")
    code, own, dev = _stream_type(out, "out"), (out.dtype,), _device()
    if M < 1:
        raise ValueError("X has no rows")
    g, rows, stride = _shared_rows(gate, "gate", M, N, gate_rows, dev)
    w = _ptr(w_hp, "w_hp", bf, plan.sizes(N)[2])
    if w_hp.get_device() != dev:
        raise ValueError(f"w_hp is on {w_hp.device}, the current device is cuda:{dev}")
    _check(lib().osm_linear_hp(plan.handle, _operand(X, "X", bf, (M, plan.K), dev), M, w, _vector(bias, "bias", N, dev),
                               act, g, rows, stride,
                               None if residual is None else _operand(residual, "residual", own, shape, dev),
                               _operand(out, "out", own, shape, dev), code, _stream(stream)))
    return out


def ffn_sublayer(up: Plan, down: Plan, R, norm: Norm, wu, wd, workspace, out=None, bias_down=None, gate=None,
                 gate_rows: int | None = None, stream=None):
    """R + gate * (FFN(norm(R)) + bias_down) (osm_ffn_sublayer): the weights and the workspace of ffn_block. R: [M][D]
    BF16 or float32; out may be R."""
    M, D = shape = R.shape
    if D != up.K:
        raise ValueError("R must have up.K columns")
    code, own, dev = _stream_type(R, "R"), (R.dtype,), _device()
    if out is None:
        out = _new(shape, R.dtype, R, stream)
    if workspace.get_device() != dev:
        raise ValueError(f"workspace is on {workspace.device}, the current device is cuda:{dev}")
    g, rows, stride = _shared_rows(gate, "gate", M, D, gate_rows, dev)
    _check(lib().osm_ffn_sublayer(up.handle, down.handle, ctypes.byref(norm.spec(M, D, dev)),
                                  _operand(R, "R", own, shape, dev), code, M, *_packed_ptrs(up, up.N, *wu, "wu", dev),
                                  *_packed_ptrs(down, down.N, *wd, "wd", dev),
                                  _vector(bias_down, "bias_down", down.N, dev), g, rows, stride,
                                  _operand(out, "out", own, shape, dev), _ptr(workspace, "workspace"),
                                  workspace.numel() * workspace.element_size(), _stream(stream)))
    return out


# ----------------------------------------------------------------- composition

def calibrate(X_batches, W, alpha: float, k: int, stream=None):
    """Per-channel statistics over calibration batches (device kernels),
    then Eq. (2)/(4) on the host: returns (s, inv_s, O, amax, wmax)."""
    import torch
    K = W.shape[0]
    with _allocating_for(stream, W.device):
        amax = torch.zeros(K, dtype=torch.float32, device=W.device)
        wmax = torch.empty(K, dtype=torch.float32, device=W.device)
    for X in X_batches:
        act_amax_accumulate(X, amax, stream)
    weight_amax(W, wmax, stream)
    with _allocating_for(stream, W.device):  # the copies to the host wait for that stream
        a, w = amax.cpu().numpy(), wmax.cpu().numpy()
    s, inv_s, O = calibrate_finalize(a, w, alpha, k)
    return s, inv_s, O, a, w


class QuantLinear:
    """A packed layer: plan + resident packed weights. `forward(X)` runs
    quantize_act and dual_gemm on `stream` (default: the current one); with
    `norm` the rows are normalised on the way (norm_quantize_act), with
    `residual` the product is gated and added to it and has its type: EPI_F32
    and EPI_BF16 are the same there, every other epi is refused
    (dual_gemm_residual)."""

    def __init__(self, plan: Plan, W, bias=None, device="cuda"):
        self.plan = plan
        self.w_codes, self.w_scales, self.w_hp = plan.alloc_packed(plan.N, device)
        pack_weights(plan, W, self.w_codes, self.w_scales, self.w_hp)
        self.bias = bias

    def forward(self, X, epi: int = EPI_F32, out=None, act_buffers=None, stream=None, norm: Norm | None = None,
                residual=None, gate=None, gate_rows: int | None = None):
        import torch
        M = X.shape[0]
        if residual is None and gate is not None:
            raise ValueError("gate goes with residual")
        if residual is not None and epi not in (EPI_F32, EPI_BF16):
            raise ValueError("the product onto a residual takes no activation: epi with GELU does not go with residual")
        a = act_buffers
        if a is None:
            with _allocating_for(stream, X.device):
                a = self.plan.alloc_packed(M, X.device)
        if norm is not None:
            norm_quantize_act(self.plan, X, norm, *a, stream=stream)
        else:
            quantize_act(self.plan, X, *a, stream=stream)
        if residual is not None:
            return dual_gemm_residual(self.plan, *a, M, self.w_codes, self.w_scales, self.w_hp, residual, out=out,
                                      bias=self.bias, gate=gate, gate_rows=gate_rows, stream=stream)
        if out is None:
            out = _new((M, self.plan.N), torch.float32 if epi == EPI_F32 else torch.bfloat16, X, stream)
        dual_gemm(self.plan, *a, M, self.w_codes, self.w_scales, self.w_hp, out, bias=self.bias, epi=epi,
                  stream=stream)
        return out


class HpLinear:
    """A layer kept in BF16: plan + resident packed weights W [K][N]. `forward(X)` runs linear_hp on the current
    stream."""

    def __init__(self, W, bias=None):
        K, N = W.shape
        self.plan = hp_plan(K, N)
        codes, scales, self.w_hp = self.plan.alloc_packed(N, W.device)
        pack_weights(self.plan, W, codes, scales, self.w_hp)
        self.bias = bias

    def forward(self, X, act: int = ACT_NONE, gate=None, gate_rows=None, residual=None, out=None, dtype=None,
                stream=None):
        return linear_hp(self.plan, X, self.w_hp, self.bias, act, gate, gate_rows, residual, out, dtype, stream)
