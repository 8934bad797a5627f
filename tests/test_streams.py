"""Which stream a layer's own buffers are allocated for (no GPU: streams,
plans and kernels are stand-ins)."""
import contextlib

import pytest

torch = pytest.importorskip("torch")

import outlier_split_mixed_b200 as osm  # noqa: E402


@pytest.fixture
def allocations(monkeypatch):
    """Lists the stream of each allocation, "current" where none was chosen."""
    at, seen = ["current"], []

    @contextlib.contextmanager
    def on(stream):
        at.append(stream)
        yield
        at.pop()

    empty = torch.empty

    def recorded(*args, **kw):
        seen.append(at[-1])
        return empty(*args, **kw)

    monkeypatch.setattr(torch.cuda, "stream", on)
    monkeypatch.setattr(torch, "empty", recorded)
    for name in ("quantize_act", "norm_quantize_act", "dual_gemm"):
        monkeypatch.setattr(osm, name, lambda *a, **kw: None)
    monkeypatch.setattr(osm, "dual_gemm_residual", lambda *a, **kw: kw["out"])
    return seen


class Packed:
    N = 64

    @staticmethod
    def alloc_packed(rows, device):
        return tuple(torch.empty(rows, device=device) for _ in range(3))


def layer():
    lin = object.__new__(osm.QuantLinear)
    lin.plan, lin.bias = Packed(), None
    lin.w_codes = lin.w_scales = lin.w_hp = None
    return lin


@pytest.mark.parametrize("norm", [None, osm.Norm()])
@pytest.mark.parametrize("residual", [False, True])
def test_a_layers_buffers_belong_to_the_stream_of_its_kernels(allocations, norm, residual):
    x = torch.zeros(4, 32, dtype=torch.bfloat16)
    r = torch.zeros(4, 64) if residual else None
    layer().forward(x, stream="side", norm=norm, residual=r)
    assert len(allocations) == (3 if residual else 4) and set(allocations) == {"side"}
    allocations.clear()
    layer().forward(x, norm=norm, residual=r)
    assert set(allocations) == {"current"}


@pytest.mark.parametrize("stream", ["side", None])
def test_statistics_are_cleared_and_read_on_the_stream_of_their_kernels(allocations, monkeypatch, stream):
    cleared, read = [], []
    zeros, cpu = torch.zeros, torch.Tensor.cpu
    on = lambda: (torch.empty(1), allocations.pop())[1]  # noqa: E731

    def recorded_zeros(*args, **kw):
        cleared.append(on())
        return zeros(*args, **kw)

    def recorded_cpu(t):
        read.append(on())
        return cpu(t)

    class Library:
        osm_error_norms = staticmethod(lambda *a: 0)
        osm_gelu_f32 = staticmethod(lambda *a: 0)

    for name in ("act_amax_accumulate", "weight_amax"):
        monkeypatch.setattr(osm, name, lambda *a: None)
    monkeypatch.setattr(osm, "calibrate_finalize", lambda *a: (None, None, None))
    monkeypatch.setattr(osm, "_ptr", lambda *a: None)
    monkeypatch.setattr(osm, "_stream", lambda s: s)
    monkeypatch.setattr(osm, "lib", Library)
    monkeypatch.setattr(torch, "zeros", recorded_zeros)
    monkeypatch.setattr(torch.Tensor, "cpu", recorded_cpu)
    x, w = torch.ones(4, 32), torch.ones(32, 8)
    osm.calibrate([x], w, 0.5, 4, stream=stream)
    osm.error_norms(x, x, stream=stream)
    where = stream or "current"
    assert cleared == [where] * 2 and read == [where] * 3 and allocations == [where]
    monkeypatch.setattr(torch, "empty_like", lambda t: (allocations.append(on()), t.clone())[1])
    osm.gelu_f32(x, stream=stream)
    assert allocations[-1] == where
