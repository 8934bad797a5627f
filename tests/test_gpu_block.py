"""The operators around the layers on the GPU: norm_modulate, residual_norm,
norm_quantize_act, dual_gemm_residual, linear_hp and ffn_sublayer, against
their formulas in 64 bits, and (bit for bit) against the entry points that
they combine.

Tolerances. u = 2^-24 is half an FP32 step, 2^-8 half a BF16 step (relative).
 * norm: the mean is a tree of at most 2 + 1 + 5 + 32 + 3 additions (eight
   values of a lane, 32 lanes, up to 32 segments of a part, eight parts), so
   its error is at most 43 u mean|x|; M2 likewise, which 1 / sqrt halves; the
   subtraction, two products, the affine part and its folding into (1 + scale)
   add eight roundings. With n = (x - mean) rstd and h = n a + b this bounds
   the FP32 error by 64 u (|a| (rstd (mean|x| + |x|) + |n|) + |b| + |bias (1 + scale)|).
 * products: one rounding toward zero per accumulation of 16 BF16 values:
   (K / 16 + 2) 2^-23 sum |x w|, the bias counted as one more.
"""
import itertools

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import outlier_split_mixed_b200 as osm  # noqa: E402

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    osm.lib()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def rand(g, *n, dtype=F32, scale=1.0, shift=0.0):
    return (torch.randn(*n, generator=g, device="cuda") * scale + shift).to(dtype)


def bits(t):
    return t.contiguous().view({2: torch.int16, 4: torch.int32, 1: torch.uint8}[t.element_size()])


def same(a, b):
    assert a.dtype == b.dtype and a.shape == b.shape
    d = bits(a) != bits(b)
    assert not bool(d.any()), f"{int(d.sum())} of {d.numel()} values differ, first at {d.nonzero()[0].tolist()}"


def within(got, ref, tol):
    err = (got.double() - ref).abs()
    assert bool(torch.isfinite(got.double()).all())
    bad = err > tol
    if bool(bad.any()):
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{int(bad.sum())} values off; first {i}: {got[i].item()} for {ref[i].item()}, "
                             f"tolerance {tol[i].item():.3g}; worst {float((err / tol).max()):.3g} of it")


def modulation(g, M, D, mode, parts):
    """(vectors, tokens per row): none, one row, three samples (the last shorter), a row per token -- as slices of
    one wider tensor."""
    if mode == "none":
        return [None] * parts, None
    share = {"one": M, "batch": -(-M // 3), "token": 1}[mode]
    e = rand(g, -(-M // share), parts, D, scale=0.3)
    return [e[:, i] for i in range(parts)], share


def norm64(x, n, tokens):
    """(norm(x), its FP32 error bound) in 64 bits."""
    x = x.double()
    D = x.shape[1]
    mean = x.mean(1, keepdim=True) if n.kind == osm.NORM_LAYER else torch.zeros(x.shape[0], 1, device="cuda").double()
    rstd = 1 / torch.sqrt(((x - mean) ** 2).mean(1, keepdim=True) + n.eps)
    v = (x - mean) * rstd
    group = torch.arange(x.shape[0], device="cuda") // tokens
    a = torch.ones_like(v) if n.scale is None else 1 + n.scale.double().reshape(-1, D)[group]
    w = 1.0 if n.weight is None else n.weight.double()
    b = torch.zeros_like(v) if n.bias is None else n.bias.double() * a
    s = torch.zeros_like(v) if n.shift is None else n.shift.double().reshape(-1, D)[group]
    h = v * w * a + b + s
    e = 64 * U * ((w * a).abs() * (rstd * (x.abs().mean(1, keepdim=True) + x.abs()) + v.abs()) + b.abs() + s.abs())
    return h, e


def make_norm(g, M, D, kind, affine, mode):
    (scale, shift), share = modulation(g, M, D, mode, 2)
    w = rand(g, D, scale=0.2, shift=1.0) if affine else None
    b = rand(g, D, scale=0.1) if affine and kind == osm.NORM_LAYER else None
    return osm.Norm(kind, eps=1e-6, weight=w, bias=b, scale=scale, shift=shift, mod_rows=share), share or M


# ------------------------------------------------------------ norm_modulate

WIDTHS = [8, 64, 248, 256, 264, 512, 1016, 5120, 5128, 10240, 10248, 13824, 20488, 65536]


@pytest.mark.parametrize("D", WIDTHS)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", [osm.NORM_LAYER, osm.NORM_RMS])
def test_norm_modulate_widths(D, dtype, kind):
    for i, (M, mode) in enumerate([(1, "one"), (7, "token"), (301, "batch")] + ([(2053, "none")] if D <= 10240 else [])):
        g = gen(D + i)
        x = rand(g, M, D, dtype=dtype, scale=2.0, shift=0.7)
        n, share = make_norm(g, M, D, kind, i != 1, mode)
        h = osm.norm_modulate(x, n)
        ref, e = norm64(x, n, share)
        within(h, ref, e + 2.0 ** -8 * (ref.abs() + e) + 1e-37)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norm_of_rows_far_from_zero(dtype):
    # mean 1000 times the deviation: a difference of large sums would lose the variance
    g = gen(5)
    x = rand(g, 64, 2048, dtype=dtype, scale=0.05, shift=50.0)
    n = osm.Norm()
    ref, e = norm64(x, n, 64)
    within(osm.norm_modulate(x, n), ref, e + 2.0 ** -8 * (ref.abs() + e))


def test_norm_of_constant_rows_and_nonfinite_rows():
    g = gen(6)
    x = rand(g, 9, 520, dtype=BF)
    x[2] = 3.0
    x[3] = 0.0
    clean = osm.norm_modulate(x, osm.Norm())
    assert bool((clean[3] == 0).all())
    ref, e = norm64(x, osm.Norm(), 9)
    within(clean, ref, e + 2.0 ** -8 * (ref.abs() + e) + 1e-30)
    x[4, 17] = float("nan")
    x[5, 519] = float("inf")
    dirty = osm.norm_modulate(x, osm.Norm())
    for r in range(9):
        if r in (4, 5):
            assert bool(torch.isnan(dirty[r]).all())
        else:
            same(dirty[r], clean[r])


def test_norm_modulate_in_place_and_rows_behind_the_last():
    g = gen(7)
    x = rand(g, 700, 1024, dtype=BF)
    n, _ = make_norm(g, 600, 1024, osm.NORM_LAYER, True, "batch")
    want = osm.norm_modulate(x[:600], n)
    y = x.clone()
    osm.norm_modulate(y[:600], n, out=y[:600])
    same(y[:600], want)
    same(y[600:], x[600:])


# ------------------------------------------------------------ residual_norm

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("post, pre", list(itertools.product([None, osm.NORM_LAYER, osm.NORM_RMS], repeat=2)))
def test_residual_norm(dtype, post, pre):
    for i, (M, D, mode, alpha) in enumerate([(1, 512, "one", 1.0), (77, 8, "none", 0.5), (599, 5120, "batch", 1.0),
                                             (5, 5128, "token", 0.25), (310, 1032, "token", 1.0), (3, 13824, "one", 1.0),
                                             (2, 40960, "token", 1.0)]):
        g = gen(100 + i)
        r, y = rand(g, M, D, dtype=dtype, scale=2.0), rand(g, M, D, dtype=BF, shift=0.2)
        (gate,), share = modulation(g, M, D, mode, 1)
        p = None if post is None else make_norm(g, M, D, post, True, "none")[0]
        n, tokens = (None, M) if pre is None else make_norm(g, M, D, pre, i % 2 == 0, mode)
        out, h = osm.residual_norm(r, y, gate=gate, gate_rows=share, alpha=alpha, post=p, pre=n)
        t, e = (y.double(), torch.zeros(M, D, device="cuda").double()) if p is None else norm64(y, p, M)
        gd = alpha * (1.0 if gate is None else gate.double()[torch.arange(M, device="cuda") // share])
        ref = r.double() + gd * t
        e = e * (gd.abs() if gate is not None else alpha) + 4 * U * (r.double().abs() + 2 * (gd * t).abs())
        within(out, ref, e + HALF[dtype] * (ref.abs() + e))
        if n is not None:
            href, he = norm64(out, n, tokens)
            within(h, href, he + 2.0 ** -8 * (href.abs() + he) + 1e-37)
            # the norm reads the rounded sum: the same bits as a norm of what was stored
            same(h, osm.norm_modulate(out, n))
        else:
            assert h is None


@pytest.mark.parametrize("dtype", [BF, F32])
def test_residual_norm_in_place(dtype):
    g = gen(31)
    r, y = rand(g, 900, 1024, dtype=dtype), rand(g, 900, 1024, dtype=BF)
    n, share = make_norm(g, 900, 1024, osm.NORM_LAYER, False, "batch")
    gate = rand(g, 3, 1024)
    want, hw = osm.residual_norm(r, y, gate=gate, gate_rows=300, pre=n, post=osm.Norm(osm.NORM_RMS))
    out, h = osm.residual_norm(r, y, gate=gate, gate_rows=300, pre=n, post=osm.Norm(osm.NORM_RMS), out=r, h=y)
    assert out is r and h is y
    same(r, want)
    same(y, hw)


def test_gate_and_modulation_rows_of_different_length():
    g = gen(32)
    M, D = 400, 256
    r, y = rand(g, M, D), rand(g, M, D, dtype=BF)
    gate, e = rand(g, 4, D), rand(g, 2, 2, D, scale=0.3)
    n = osm.Norm(scale=e[:, 0], shift=e[:, 1], mod_rows=250)
    out, h = osm.residual_norm(r, y, gate=gate, gate_rows=100, pre=n)
    ref = r.double() + gate.double().repeat_interleave(100, 0) * y.double()
    within(out, ref, 4 * U * (r.double().abs() + ref.abs()) + 1e-30)
    same(h, osm.norm_modulate(out, n))


# ------------------------------------------------------------ norm_quantize_act

def make_plan(g, K, N, k, fmt="mx"):
    s = torch.exp(0.3 * torch.randn(K, generator=g, device="cuda")).cpu().numpy()
    O = torch.randperm(K, generator=g, device="cuda")[:k].sort().values.int().cpu().numpy()
    if fmt == "nv":
        return osm.Plan(K, N, k, s, O, fmt=osm.FMT_NVFP4, g_act=-6, g_w=-8)
    return osm.Plan(K, N, k, s, O, hp_fp16=fmt == "f16")


def guarded(plan, M):
    """Packed buffers with 256 bytes behind each that have to stay as they are."""
    out = []
    for n, dt in zip(plan.sizes(M), (torch.uint8, torch.uint8, BF)):
        b = torch.full((n + 256,), 0xA5, dtype=torch.uint8, device="cuda")
        out.append((b, b[:n].view(dt) if n else torch.empty(0, dtype=dt, device="cuda"), n))
    return out


@pytest.mark.parametrize("fmt", ["mx", "f16", "nv"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K, k", [(32, 0), (32, 32), (256, 3), (512, 16), (1056, 64), (2048, 0), (5120, 128), (5152, 128),
                                  (13824, 256)])
def test_norm_quantize_act_writes_what_the_two_calls_write(fmt, dtype, K, k):
    for i, (M, mode, kind) in enumerate([(1, "one", osm.NORM_LAYER), (130, "batch", osm.NORM_RMS),
                                         (257, "token", osm.NORM_LAYER), (1283, "one", osm.NORM_LAYER)]):
        if M * K > 6_000_000 and fmt != "mx":
            continue
        g = gen(K + 7 * i + k)
        plan = make_plan(g, K, 32, k, fmt)
        x = rand(g, M, K, dtype=dtype, scale=1.5, shift=0.3)
        n, _ = make_norm(g, M, K, kind, i % 2 == 0, mode)
        want = plan.alloc_packed(M)
        osm.quantize_act(plan, osm.norm_modulate(x, n), *want)
        got = guarded(plan, M)
        osm.norm_quantize_act(plan, x, n, *[v for _, v, _ in got])
        for (b, v, size), w, name in zip(got, want, ("codes", "scales", "hp")):
            d = (b[:size] != w.reshape(-1).view(torch.uint8)).nonzero()
            assert d.numel() == 0, f"{name}: {d.numel()} bytes differ, first at {d[0].item()} (M={M})"
            assert bool((b[size:] == 0xA5).all()), f"{name}: bytes behind the buffer were written"
        assert plan.status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("K", [512, 2048, 5120])
@pytest.mark.parametrize("M, run", [(149, 1), (301, 2), (1000, 3), (1283, 7), (1283, 15), (1283, 16), (148, 3)])
def test_norm_quantize_act_of_short_runs(dtype, K, M, run):
    g = gen(K + M + run)
    plan = make_plan(g, K, 32, 16)
    x, e = rand(g, M, K, dtype=dtype, scale=1.5, shift=0.3), rand(g, -(-M // run), 2 * K + 8, scale=0.3)
    n = osm.Norm(weight=rand(g, K), bias=rand(g, K), scale=e[:, :K], shift=e[:, K:2 * K], mod_rows=run)
    want = plan.alloc_packed(M)
    osm.quantize_act(plan, osm.norm_modulate(x, n), *want)
    got = guarded(plan, M)
    osm.norm_quantize_act(plan, x, n, *[v for _, v, _ in got])
    for (b, v, size), w in zip(got, want):
        assert torch.equal(b[:size], w.reshape(-1).view(torch.uint8)) and bool((b[size:] == 0xA5).all())


# ------------------------------------------------------------ dual_gemm_residual

def operands(g, plan, M, N):
    a, w = plan.alloc_packed(M), plan.alloc_packed(N)
    osm.quantize_act(plan, rand(g, M, plan.K, dtype=BF), *a)
    osm.pack_weights(plan, rand(g, plan.K, N, dtype=BF, scale=0.05), *w)
    return a, w


@pytest.mark.parametrize("fmt", ["mx", "f16", "nv"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M, K, N, k", [(1, 256, 32, 8), (255, 512, 256, 16), (300, 128, 416, 0), (513, 352, 544, 352),
                                        (2100, 1024, 1312, 64)])
def test_dual_gemm_residual(fmt, dtype, M, K, N, k):
    for i, mode in enumerate(["none", "one", "batch", "token"]):
        if mode == "batch" and M < 3:
            continue
        g = gen(M + i)
        plan = make_plan(g, K, N, k, fmt)
        a, w = operands(g, plan, M, N)
        r = rand(g, M, N, dtype=dtype, scale=2.0)
        (gate,), share = modulation(g, M, N, mode, 1)
        bias = rand(g, N) if i % 2 else None
        y = torch.empty(M, N, device="cuda")
        osm.dual_gemm(plan, *a, M, *w, y, bias=bias, epi=osm.EPI_F32)
        # the same accumulator, then the epilogue's FP32 operations one by one: the same bits
        if gate is not None:
            y = y * gate[torch.arange(M, device="cuda") // share]
        want = (r.float() + y).to(dtype)
        out = torch.full((M + 1, N), 7.0, dtype=dtype, device="cuda")
        got = osm.dual_gemm_residual(plan, *a, M, *w, r, out=out[:M], bias=bias, gate=gate, gate_rows=share)
        same(got, want)
        assert bool((out[M:] == 7.0).all())
        rr = r.clone()
        osm.dual_gemm_residual(plan, *a, M, *w, rr, out=rr, bias=bias, gate=gate, gate_rows=share)
        same(rr, want)
        assert plan.status() == 0


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M, share", [(2, 1), (33, 31), (259, 3), (700, 16), (700, 31), (700, 32), (700, 33)])
def test_dual_gemm_residual_short_gate_rows(fmt, dtype, M, share):
    g = gen(M + share)
    plan = make_plan(g, 256, 416, 16, fmt)
    a, w = operands(g, plan, M, 416)
    r, gates, bias = rand(g, M, 416, dtype=dtype, scale=2.0), rand(g, -(-M // share), 424), rand(g, 416)
    y = torch.empty(M, 416, device="cuda")
    osm.dual_gemm(plan, *a, M, *w, y, bias=bias, epi=osm.EPI_F32)
    want = (r.float() + y * gates[torch.arange(M, device="cuda") // share, :416]).to(dtype)
    same(osm.dual_gemm_residual(plan, *a, M, *w, r, bias=bias, gate=gates[:, :416], gate_rows=share), want)
    assert plan.status() == 0


# ------------------------------------------------------------ linear_hp

def act64(y, act):
    if act == osm.ACT_GELU:
        return 0.5 * y * (1 + torch.tanh(np.sqrt(2 / np.pi) * (y + 0.044715 * y ** 3)))
    return y * torch.sigmoid(y) if act == osm.ACT_SILU else y


def check_linear(seed, M, K, N, dtype, act, bias, mode, residual):
    g = gen(seed)
    x = rand(g, M, K, dtype=BF)
    W = rand(g, K, N, dtype=BF, scale=1 / np.sqrt(K))
    b = rand(g, N) if bias else None
    lin = osm.HpLinear(W, b)
    (gate,), share = modulation(g, M, N, mode, 1)
    r = rand(g, M, N, dtype=dtype, scale=2.0) if residual else None
    out = torch.full((M + 1, N), 7.0, dtype=dtype, device="cuda")
    got = lin.forward(x, act=act, gate=gate, gate_rows=share, residual=r, out=out[:M])
    assert lin.plan.status() == 0
    assert bool((out[M:] == 7.0).all())
    y = x.double() @ W.double() + (0 if b is None else b.double())
    T = x.double().abs() @ W.double().abs() + (0 if b is None else b.double().abs())
    e = (K / 16 + 2) * 2 * U * T
    v = act64(y, act)
    if act == osm.ACT_GELU:    # |GELU'| <= 1.13, and the routine's own bound
        e = 1.13 * e + 5e-7 * v.abs() + 2e-8 * y.abs()
    elif act == osm.ACT_SILU:  # |SiLU'| <= 1.1; 2^z to 2^-22 with z off by 2 u |z|, the reciprocal to 2^-23, a sum
        e = 1.1 * e + v.abs() * (8 * U + 4 * U * y.abs()) + 1e-37
    if gate is not None:
        gd = gate.double()[torch.arange(M, device="cuda") // share]
        e, v = e * gd.abs() + U * (gd * v).abs(), v * gd
    if r is not None:
        v = r.double() + v
        e = e + U * v.abs()
    within(got, v, e + HALF[dtype] * (v.abs() + e) + 1e-37)
    if residual:
        rr = r.clone()
        lin.forward(x, act=act, gate=gate, gate_rows=share, residual=rr, out=rr)
        same(rr, got)


SHAPES = [(1, 32, 32), (1, 5120, 5120), (2, 96, 160), (16, 512, 128), (17, 1504, 4128), (32, 64, 96), (33, 2048, 256),
          (64, 13824, 160), (65, 512, 1024), (100, 160, 2080), (128, 4096, 512), (129, 1024, 1056), (255, 288, 544),
          (256, 512, 512), (257, 320, 5120), (700, 1504, 1056), (1001, 1504, 4128), (2300, 544, 2336), (5000, 96, 992)]


@pytest.mark.parametrize("M, K, N", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_linear_hp_shapes(M, K, N, dtype):
    mode = ["none", "one", "batch", "token"][(M + N // 32) % 4] if M >= 3 else "one"
    check_linear(M + K + N, M, K, N, dtype, osm.ACT_NONE, True, mode, True)
    check_linear(M + K + N + 1, M, K, N, dtype, osm.ACT_NONE, False, "none", False)


@pytest.mark.parametrize("M", [1, 40, 300, 3000])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", [osm.ACT_NONE, osm.ACT_GELU, osm.ACT_SILU])
@pytest.mark.parametrize("bias, mode, residual", [(True, "none", False), (False, "one", True), (True, "token", False),
                                                  (True, "token", True)])
def test_linear_hp_epilogues(M, dtype, act, bias, mode, residual):
    check_linear(M, M, 480, 2080, dtype, act, bias, mode, residual)


def test_linear_hp_twice_gives_the_same_bits():
    g = gen(3)
    for M in (1, 90, 1300):
        lin = osm.HpLinear(rand(g, 2048, 1536, dtype=BF, scale=0.02))
        x = rand(g, M, 2048, dtype=BF)
        same(lin.forward(x, dtype=F32), lin.forward(x, dtype=F32))


def test_linear_hp_refuses_other_plans():
    x = torch.zeros(4, 64, dtype=BF, device="cuda")
    ones, every = np.ones(64, np.float32), np.arange(64, dtype=np.int32)
    w = torch.zeros(64 * 64, dtype=BF, device="cuda")
    smoothed = osm.Plan(64, 64, 64, 2 * ones, every)
    split = osm.Plan(64, 64, 32, ones, every[:32])
    f16 = osm.Plan(64, 64, 64, ones, every, hp_fp16=True)
    for plan in (smoothed, split, f16):
        with pytest.raises(osm.OsmError) as e:
            osm.linear_hp(plan, x, w)
        assert e.value.code == osm.ERR_INVALID_ARG
    plan = osm.hp_plan(64, 64)
    stats = torch.ones(64, device="cuda")
    plan.refresh(stats, stats, 0.5)  # s may be anything now
    with pytest.raises(osm.OsmError):
        osm.linear_hp(plan, x, w)


@pytest.mark.parametrize("M", [1, 100, 2000])
def test_linear_hp_reports_a_wait_that_runs_out(M):
    # the pipeline gives up at once, reports it and returns; the next call works again
    g = gen(4)
    lin = osm.HpLinear(rand(g, 4096, 2560, dtype=BF, scale=0.02))
    x = rand(g, M, 4096, dtype=BF)
    want = lin.forward(x)
    lin.plan.set_wait_limit(1000)
    lin.forward(x)
    status = lin.plan.status()
    lin.plan.set_wait_limit(2_000_000_000)
    assert status in (0, osm.STATUS_TIMEOUT)
    same(lin.forward(x), want)
    assert lin.plan.status() == 0


def test_linear_hp_keeps_nonfinite_rows_to_themselves():
    g = gen(8)
    lin = osm.HpLinear(rand(g, 512, 384, dtype=BF, scale=0.05), rand(g, 384))
    for M in (7, 300, 3000):
        x, r = rand(g, M, 512, dtype=BF), rand(g, M, 384)
        clean = lin.forward(x, act=osm.ACT_SILU, residual=r)
        bad = [1, M - 2]
        x[bad[0], 5], x[bad[1], 511] = float("nan"), float("inf")
        r[2, 7] = float("inf")
        dirty = lin.forward(x, act=osm.ACT_SILU, residual=r)
        keep = torch.ones(M, dtype=torch.bool, device="cuda")
        keep[bad + [2]] = False
        same(dirty[keep], clean[keep])
        assert not bool(torch.isfinite(dirty[bad]).all(1).any()) and bool(torch.isinf(dirty[2, 7]))
        same(dirty[2, :7], clean[2, :7])


def test_silu_and_gelu_at_the_ends_of_their_range():
    v = torch.tensor([0.0, -0.0, 1e-38, -1e-38, 1.0, -1.0, -20.0, -87.0, -88.8, -104.0, 104.0, -1e4, 1e4, 3e38, -3e38],
                     device="cuda").bfloat16()
    x = torch.zeros(64, 32, dtype=BF, device="cuda")
    x[:v.numel(), 0] = v
    W = torch.eye(32, device="cuda").bfloat16()
    y = osm.HpLinear(W).forward(x, act=osm.ACT_SILU, dtype=F32)[:v.numel(), 0].double()
    ref = v.double() * torch.sigmoid(v.double())
    # relative as derived at check_linear; below 2^-126 results flush to zero
    assert bool(((y - ref).abs() <= ref.abs() * (8 * U + 4 * U * v.double().abs().clamp_max(200)) + 2.0 ** -119).all())
    y = osm.HpLinear(W).forward(x, act=osm.ACT_GELU, dtype=F32)[:v.numel() - 1, 0].double()
    ref = act64(v.double(), osm.ACT_GELU)[:-1]
    assert bool(((y - ref).abs() <= 5e-7 * ref.abs() + 2e-8 * v[:-1].double().abs()).all())


# ------------------------------------------------------------ more than 2^32 values

def room(gib):
    free, _ = torch.cuda.mem_get_info()
    if free < gib << 30:
        pytest.skip(f"needs {gib} GiB of free device memory")


def filled(M, D, dtype):
    """[M][D] values that differ from row to row, without a second buffer of that size."""
    x = torch.empty(M, D, dtype=dtype, device="cuda")
    base = rand(gen(1), 4096, D, dtype=dtype)
    for i in range(0, M, 4096):
        n = min(4096, M - i)
        x[i:i + n] = base[:n].roll(i % D, 1)
    return x


def test_norms_past_32_bit_offsets():
    room(60)
    M, D = 320_001, 14336
    x = filled(M, D, BF)
    at = torch.tensor([0, 1, M // 2, 299_594, M - 2, M - 1], device="cuda")
    n = osm.Norm(scale=rand(gen(2), D, scale=0.3), shift=rand(gen(3), D))
    h = osm.norm_modulate(x, n)
    same(h[at], osm.norm_modulate(x[at], n))
    out, h = osm.residual_norm(x, h, gate=rand(gen(4), D), pre=n, h=h)
    few, fh = osm.residual_norm(x[at], osm.norm_modulate(x[at], n), gate=rand(gen(4), D), pre=n)
    same(out[at], few)
    same(h[at], fh)


def test_norm_quantize_act_past_32_bit_offsets():
    room(40)
    M, K = 900_003, 5120
    plan = make_plan(gen(5), K, 32, 128)
    x = filled(M, K, BF)
    n = osm.Norm()
    a = plan.alloc_packed(M)
    osm.norm_quantize_act(plan, x, n, *a)
    at = torch.tensor([0, M // 2, 838_861, M - 1], device="cuda")
    few = plan.alloc_packed(4)
    osm.norm_quantize_act(plan, x[at], n, *few)
    same(a[0].view(M, -1)[at], few[0].view(4, -1))
    same(a[2].view(M, -1)[at], few[2].view(4, -1))


def test_linear_hp_past_32_bit_offsets():
    room(40)
    M, K, N = 1_100_003, 64, 4096
    g = gen(6)
    x, W = filled(M, K, BF), rand(g, K, N, dtype=BF, scale=0.1)
    y = filled(M, N, BF)
    at = torch.tensor([0, 1_048_575, 1_048_577, M - 1], device="cuda")
    r = y[at]
    osm.HpLinear(W).forward(x, residual=y, out=y)
    ref = r.double() + x[at].double() @ W.double()
    T = x[at].double().abs() @ W.double().abs()
    e = (K / 16 + 2) * 2 * U * T + U * ref.abs()
    within(y[at], ref, e + 2.0 ** -8 * (ref.abs() + e))


# ------------------------------------------------------------ together

def ffn(g, D, F, k):
    up, down = make_plan(g, D, F, k), make_plan(g, F, D, k)
    wu, wd = up.alloc_packed(F), down.alloc_packed(D)
    osm.pack_weights_for_next(up, down, rand(g, D, F, dtype=BF, scale=1 / np.sqrt(D)), *wu)
    osm.pack_weights(down, rand(g, F, D, dtype=BF, scale=1 / np.sqrt(F)), *wd)
    return up, down, wu, wd


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M, D, F, k, mode", [(1, 256, 512, 8, "one"), (300, 512, 1024, 16, "batch"), (129, 1056, 2080, 0, "token"),
                                              (1500, 1024, 1536, 64, "none")])
def test_ffn_sublayer_is_its_parts(dtype, M, D, F, k, mode):
    g = gen(M + D)
    up, down, wu, wd = ffn(g, D, F, k)
    r = rand(g, M, D, dtype=dtype, scale=1.5)
    n, _ = make_norm(g, M, D, osm.NORM_LAYER, True, mode)
    (gate,), share = modulation(g, M, D, mode, 1)
    bias = rand(g, D, scale=0.1)
    ws = torch.empty(osm.ffn_workspace_size(up, down, M), dtype=torch.uint8, device="cuda")
    got = osm.ffn_sublayer(up, down, r, n, wu, wd, ws, bias_down=bias, gate=gate, gate_rows=share)
    a, h = up.alloc_packed(M), down.alloc_packed(M)
    osm.quantize_act(up, osm.norm_modulate(r, n), *a)
    osm.dual_gemm(up, *a, M, *wu, None, epi=osm.EPI_GELU_REQUANT, next_plan=down, next_buffers=h)
    y = torch.empty(M, D, device="cuda")
    osm.dual_gemm(down, *h, M, *wd, y, bias=bias, epi=osm.EPI_F32)
    if gate is not None:
        y = y * gate[torch.arange(M, device="cuda") // share]
    want = (r.float() + y).to(dtype)
    same(got, want)
    osm.ffn_sublayer(up, down, r, n, wu, wd, ws, out=r, bias_down=bias, gate=gate, gate_rows=share)
    same(r, want)
    assert up.status() == 0 and down.status() == 0


def block(x, parts, e, share):
    """A transformer block's FFN half and the BF16 layer behind it, as a model would run them."""
    up, down, wu, wd, ws, lin, qlin = parts
    n1 = osm.Norm(scale=e[:, 0], shift=e[:, 1], mod_rows=share)
    x = osm.ffn_sublayer(up, down, x, n1, wu, wd, ws, gate=e[:, 2], gate_rows=share)
    y = lin.forward(osm.norm_modulate(x, osm.Norm(osm.NORM_RMS)), act=osm.ACT_SILU)
    x, h = osm.residual_norm(x, y, gate=e[:, 2], gate_rows=share, pre=n1, post=osm.Norm(osm.NORM_RMS))
    return qlin.forward(h, residual=x, norm=osm.Norm(), gate=e[:, 0], gate_rows=share)


def test_a_block_captured_replayed_and_on_another_stream():
    g = gen(77)
    M, D, F = 600, 512, 1024
    up, down, wu, wd = ffn(g, D, F, 16)
    ws = torch.empty(osm.ffn_workspace_size(up, down, M), dtype=torch.uint8, device="cuda")
    lin = osm.HpLinear(rand(g, D, D, dtype=BF, scale=0.05), rand(g, D))
    qlin = osm.QuantLinear(make_plan(g, D, D, 16), rand(g, D, D, dtype=BF, scale=0.05))
    parts = (up, down, wu, wd, ws, lin, qlin)
    xs = [rand(g, M, D, dtype=BF) for _ in range(3)]
    es = [rand(g, 2, 3, D, scale=0.3) for _ in range(3)]
    want = [block(x, parts, e, 300) for x, e in zip(xs, es)]
    torch.cuda.synchronize()
    x, e = xs[0].clone(), es[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = block(x, parts, e, 300)
    for i in (1, 2, 0):
        x.copy_(xs[i])
        e.copy_(es[i])
        graph.replay()
        same(out, want[i])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = block(xs[1], parts, es[1], 300)
    torch.cuda.current_stream().wait_stream(side)
    same(got, want[1])
    for p in (up, down, lin.plan, qlin.plan):
        assert p.status() == 0


def test_two_streams_at_once():
    g = gen(78)
    lins = [osm.HpLinear(rand(g, 1024, 2048, dtype=BF, scale=0.03)) for _ in range(2)]
    xs = [rand(g, m, 1024, dtype=BF) for m in (5, 900)]
    n = osm.Norm()
    want = [li.forward(osm.norm_modulate(x, n)) for li, x in zip(lins, xs)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            h = osm.norm_modulate(xs[i], n, stream=streams[i])
            got[i].append((h, lins[i].forward(h, stream=streams[i])))
    torch.cuda.synchronize()
    for i in range(2):
        for _, y in got[i]:
            same(y, want[i])


@pytest.mark.parametrize("M, B", [(2, 2), (40, 1), (1200, 3)])
def test_modulation_written_by_the_kernel_before(M, B):
    """Modulation and gate rows come from linear_hp's call just before the norm and the products that read them, in one
    buffer that the next step overwrites: each step gets the bits of a run that waits after every call."""
    g = gen(M + B)
    D, steps = 512, 12
    embed = osm.HpLinear(rand(g, 256, 3 * D, dtype=BF, scale=0.05), rand(g, 3 * D, scale=0.1))
    lin = osm.HpLinear(rand(g, D, D, dtype=BF, scale=0.05))
    qlin = osm.QuantLinear(make_plan(g, D, D, 16), rand(g, D, D, dtype=BF, scale=0.05))
    es = [rand(g, B, 256, dtype=BF) for _ in range(steps)]
    xs = [rand(g, M, D, dtype=BF, scale=1.5) for _ in range(steps)]
    mod, h, a = torch.empty(B, 3 * D, device="cuda"), torch.empty(M, D, dtype=BF, device="cuda"), qlin.plan.alloc_packed(M)
    shift, scale, gate = mod[:, :D], mod[:, D:2 * D], mod[:, 2 * D:]
    n = osm.Norm(scale=scale, shift=shift)

    def step(i, out, wait):
        embed.forward(es[i], out=mod)
        wait()
        osm.norm_modulate(xs[i], n, out=h)
        wait()
        lin.forward(h, gate=gate, residual=xs[i], out=out)
        wait()
        embed.forward(es[i - 1], out=mod)
        wait()
        osm.residual_norm(out, h, gate=gate, pre=n, out=out, h=h)
        wait()
        embed.forward(es[i], out=mod)
        wait()
        qlin.forward(out, norm=n, residual=out, gate=gate, out=out, act_buffers=a)
        wait()

    want = [torch.empty(M, D, dtype=BF, device="cuda") for _ in range(steps)]
    for i in range(steps):
        step(i, want[i], torch.cuda.synchronize)
    got = [torch.zeros(M, D, dtype=BF, device="cuda") for _ in range(steps)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for i in range(steps):
            step(i, got[i], lambda: None)
    for _ in range(5):
        graph.replay()
        for i in range(steps):
            same(got[i], want[i])
            got[i].zero_()
    for i in range(steps):
        step(i, got[i], lambda: None)
    for i in range(steps):
        same(got[i], want[i])
    assert embed.plan.status() == 0 and lin.plan.status() == 0 and qlin.plan.status() == 0
