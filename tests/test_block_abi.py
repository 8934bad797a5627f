"""The entry points around the layers (norms, gated residual, products onto
the residual stream, BF16 layers, FFN sublayer): what they refuse, before any
device is touched. Pointers here are never dereferenced."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

import outlier_split_mixed_b200 as osm  # noqa: E402

P = 4096  # an aligned stand-in for a device pointer


@pytest.fixture(scope="module", autouse=True)
def built():
    from outlier_split_mixed_b200 import build
    build.build()


def _spec(**kw):
    f = dict(kind=osm.NORM_LAYER, eps=1e-6, weight=None, bias=None, scale=None, shift=None, mod_rows=1, mod_stride=0)
    f.update(kw)
    return osm._NormSpec(*f.values())


def _norm(M=4, D=64, x=P, h=P * 2, dt=osm.DT_BF16, spec=None, **kw):
    s = _spec(**kw) if spec is None else spec
    return osm.lib().osm_norm_modulate(x, dt, M, D, ctypes.byref(s) if s else None, h, None)


@pytest.mark.parametrize("bad, says", [
    (dict(M=0), "M"), (dict(M=-1), "M"), (dict(M=1 << 31), "M"), (dict(D=0), "D"), (dict(D=12), "D"),
    (dict(D=65544), "D"), (dict(dt=2), "type"), (dict(x=None), "null"), (dict(h=None), "null"),
    (dict(x=P + 8), "misaligned"), (dict(h=P + 2), "misaligned"), (dict(spec=False), "NULL"),
    (dict(kind=2), "kind"), (dict(eps=0.0), "eps"), (dict(eps=-1.0), "eps"), (dict(eps=float("nan")), "eps"),
    (dict(eps=float("inf")), "eps"), (dict(weight=P + 4), "aligned"), (dict(scale=P + 4, mod_rows=4), "aligned"),
    (dict(scale=P, mod_rows=0), "per row"), (dict(shift=P, mod_rows=2, mod_stride=32), "apart"),
    (dict(scale=P, mod_rows=1, mod_stride=66), "apart"), (dict(dt=osm.DT_F32, h=P), "in place"),
])
def test_norm_modulate_refuses(bad, says):
    assert _norm(**bad) == osm.ERR_INVALID_ARG
    assert says in osm.last_error(), osm.last_error()


def _residual(M=4, D=64, r=P, dt=osm.DT_F32, y=2 * P, post=None, gate=None, rows=4, stride=64, alpha=1.0, pre=None,
              out=3 * P, h=None):
    ref = lambda s: ctypes.byref(s) if s is not None else None  # noqa: E731
    return osm.lib().osm_residual_norm(r, dt, y, M, D, ref(post), gate, rows, stride, alpha, ref(pre), out, h, None)


@pytest.mark.parametrize("bad, says", [
    (dict(M=0), "M"), (dict(D=4), "D"), (dict(dt=7), "type"), (dict(r=None), "null"), (dict(y=None), "null"),
    (dict(out=None), "null"), (dict(out=P + 4), "misaligned"), (dict(alpha=float("nan")), "alpha"),
    (dict(gate=P + 4), "aligned"), (dict(gate=P, rows=0), "per row"), (dict(gate=P, rows=1, stride=60), "apart"),
    (dict(h=4 * P), "pre"), (dict(pre=_spec()), "pre"), (dict(pre=_spec(eps=0.0), h=4 * P), "eps"),
    (dict(post=_spec(scale=P, mod_rows=4)), "modulation"), (dict(post=_spec(kind=-1)), "kind"),
    (dict(out=2 * P), "R_out may be R"), (dict(pre=_spec(), h=3 * P), "R_out may be R"),
    (dict(pre=_spec(), h=P), "R_out may be R"),
])
def test_residual_norm_refuses(bad, says):
    assert _residual(**bad) == osm.ERR_INVALID_ARG
    assert says in osm.last_error(), osm.last_error()


def test_plan_entry_points_refuse_a_missing_plan():
    L = osm.lib()
    s = _spec()
    assert L.osm_norm_quantize_act(None, P, 0, 4, ctypes.byref(s), P, P, P, None) == osm.ERR_INVALID_ARG
    assert L.osm_dual_gemm_residual(None, P, P, P, 4, P, P, P, None, None, 1, 0, P, 0, P, None) == osm.ERR_INVALID_ARG
    assert L.osm_linear_hp(None, P, 4, P, None, 0, None, 1, 0, None, P, 0, None) == osm.ERR_INVALID_ARG
    assert L.osm_ffn_sublayer(None, None, ctypes.byref(s), P, 0, 4, *([P] * 6), None, None, 1, 0, P, P, 1 << 20,
                              None) == osm.ERR_INVALID_ARG
    assert "plan" in osm.last_error()


def test_the_binding_refuses_host_tensors_and_wrong_types():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        osm.norm_modulate(x, osm.Norm(), out=torch.empty_like(x))
    with pytest.raises(ValueError, match="dtype"):
        osm.norm_modulate(x.half(), osm.Norm())
    with pytest.raises(ValueError, match="float32 CUDA"):
        osm.Norm(scale=torch.zeros(64)).spec(4, 64)
    with pytest.raises(ValueError, match="CUDA"):
        osm.Norm(weight=torch.zeros(64)).spec(4, 64, 0)
    with pytest.raises(ValueError, match="pre"):
        osm.residual_norm(x, x, out=x, h=x)
    with pytest.raises(ValueError, match="dtype"):
        osm.residual_norm(x.double(), x)
