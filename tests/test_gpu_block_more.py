"""Further cases of the operators around the layers on the GPU: layers on
several streams at once, plans of other formats, waits that run
out, rows in tiles at every width. Tolerances as in test_gpu_block.py."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

import outlier_split_mixed_b200 as osm  # noqa: E402
from test_gpu_block import (BF, F32, HALF, U, gen, make_norm, make_plan, modulation, norm64, operands, rand,  # noqa: E402
                            same, within)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    osm.lib()


@pytest.mark.parametrize("as_address", [False, True])
def test_quantised_layers_on_two_streams_at_once(as_address):
    # each call packs its activations into buffers of its own, which are free again when it returns
    g = gen(81)
    K, N, M = 2048, 512, 3000
    plan = make_plan(g, K, N, 64)
    lin = osm.QuantLinear(plan, rand(g, K, N, dtype=BF, scale=0.03))
    n = osm.Norm(scale=rand(g, K, scale=0.3), shift=rand(g, K))
    xs = [rand(g, M, K, dtype=BF) for _ in range(2)]
    rs = [rand(g, M, N) for _ in range(2)]
    calls = [dict(), dict(epi=osm.EPI_BF16), dict(norm=n), dict(norm=n, residual=True)]

    def call(i, kw, stream):
        kw = dict(kw, residual=rs[i]) if "residual" in kw else kw
        return lin.forward(xs[i], stream=stream, **kw)

    want = [[call(i, kw, None) for kw in calls] for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for j, kw in enumerate(calls):
            for i in range(2):
                got[i].append((j, call(i, kw, streams[i].cuda_stream if as_address else streams[i])))
    torch.cuda.synchronize()
    for i in range(2):
        for j, y in got[i]:
            same(y, want[i][j])
    assert plan.status() == 0


def test_calibration_on_another_stream():
    # the statistics are complete when they are read, whatever the current stream does
    g = gen(82)
    x, w = rand(g, 20000, 4096, dtype=BF), rand(g, 4096, 2048, dtype=BF)
    want = osm.calibrate([x, 2 * x], w, 0.5, 32)
    y = rand(g, 5000, 4096)
    norms, act = osm.error_norms(y, 2 * y), osm.gelu_f32(y)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    twice, double = 2 * x, 2 * y
    torch.cuda.synchronize()
    for _ in range(5):
        got = osm.calibrate([x, twice], w, 0.5, 32, stream=side)
        assert all((a == b).all() for a, b in zip(got, want))
        # CTAs (148 x 8 at most) add their FP64 sums in any order: none is negative, so each order is within
        # 1184 roundings of 2^-53 of the exact sum and any two orders within twice that
        assert all(abs(a - b) <= 2 * 1184 * 2.0 ** -53 * b for a, b in zip(osm.error_norms(y, double, stream=side), norms))
        z = osm.gelu_f32(y, stream=side)
        side.synchronize()
        same(z, act)


def test_linear_hp_of_nvfp4_plans():
    # packed slots hold w 2^-g_w and X is not scaled: with g_w = 0 it is the product, anything else is refused
    g = gen(83)
    ones, every = np.ones(64, np.float32), np.arange(64, dtype=np.int32)
    x, W = rand(g, 40, 64, dtype=BF), rand(g, 64, 96, dtype=BF, scale=0.1)
    want = osm.HpLinear(W).forward(x)
    for g_act, g_w in ((-6, 0), (0, 0), (-6, -8), (0, 3)):
        plan = osm.Plan(64, 96, 64, ones, every, fmt=osm.FMT_NVFP4, g_act=g_act, g_w=g_w)
        w = plan.alloc_packed(96)
        osm.pack_weights(plan, W, *w)
        if g_w == 0:
            same(osm.linear_hp(plan, x, w[2]), want)
            assert plan.status() == 0
        else:
            with pytest.raises(osm.OsmError, match="g_w") as e:
                osm.linear_hp(plan, x, w[2])
            assert e.value.code == osm.ERR_INVALID_ARG


# Few tokens with and without K splits, and CTA pairs (every call above 4096 tokens; 2000 by the estimate of both times).
STARVED = [(1, 128, 512), (1, 4096, 128), (48, 512, 256), (128, 128, 512), (100, 4096, 256), (2000, 4096, 2560),
           (4352, 512, 512)]


@pytest.mark.parametrize("M, K, N", STARVED)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_linear_hp_starved_of_its_copies_reports_it(M, K, N, dtype):
    # the first K-step of every CTA expects bytes that no copy brings: its wait runs out after 1 ms, the status says so,
    # and the next call gets the same bits as before
    g = gen(84)
    lin = osm.HpLinear(rand(g, K, N, dtype=BF, scale=0.02))
    x = rand(g, M, K, dtype=BF)
    want = lin.forward(x, dtype=dtype)
    assert lin.plan.status() == 0
    lin.plan.set_wait_limit(1_000_000)
    lin.plan.set_debug(osm.DEBUG_STARVE_LINEAR)
    lin.forward(x, dtype=dtype)
    assert lin.plan.status() == osm.STATUS_TIMEOUT
    lin.plan.set_debug(0)
    lin.plan.set_wait_limit(2_000_000_000)
    same(lin.forward(x, dtype=dtype), want)
    assert lin.plan.status() == 0
    with pytest.raises(osm.OsmError):
        lin.plan.set_debug(4)


@pytest.mark.parametrize("dtype, share", [(BF, 1024), (F32, 1024), (BF, 1)])
def test_dual_gemm_residual_reports_a_wait_that_runs_out(dtype, share):
    # a limit of 1 us is far below the time of a tile's MMAs and of an epilogue's end (the three epilogues: BF16, FP32, a
    # gate row per token onto BF16)
    g = gen(85)
    M, K, N = 1024, 5120, 13824
    plan = make_plan(g, K, N, 128)
    a, w = operands(g, plan, M, N)
    r, gate = rand(g, M, N, dtype=dtype), rand(g, M // share, N)
    call = lambda: osm.dual_gemm_residual(plan, *a, M, *w, r, gate=gate, gate_rows=share)  # noqa: E731
    want = call()
    assert plan.status() == 0
    plan.set_wait_limit(1000)
    call()
    assert plan.status() == osm.STATUS_TIMEOUT
    plan.set_wait_limit(2_000_000_000)
    same(call(), want)
    assert plan.status() == 0


def constants(M, D, dtype):
    """Rows of one value each: the 128 BF16 mantissas by powers of two from 2^-9 on, both signs."""
    r = torch.arange(M, device="cuda")
    c = (128 + r % 128) * 2.0 ** (r // 128 % 16 - 9) * (1 - 2 * (r // 7 % 2))
    return c.to(dtype)[:, None].expand(M, D).contiguous()


# Widths whose reciprocal in FP32, times the exact sum, misses most constants: a CTA per row and tiles of rows
@pytest.mark.parametrize("D, M", [(480, 128), (480, 2560), (960, 1280), (2016, 640), (3840, 256), (3840, 384), (6080, 384),
                                  (14344, 128)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_constant_rows_have_no_deviation(D, M, dtype):
    # the sum of D equal BF16 values is exact in FP32 in any order, and so is its quotient by D: N(x) = 0 to the bit
    g = gen(86)
    x, shift = constants(M, D, dtype), rand(g, D)
    n = osm.Norm(weight=rand(g, D), scale=rand(g, D, scale=0.3), shift=shift)
    want = shift.to(BF).expand(M, D)
    h = osm.norm_modulate(x, n)
    same(h, want)
    r, bias = rand(g, M, D, dtype=dtype), rand(g, D)
    out, h = osm.residual_norm(r, x.to(BF), post=osm.Norm(weight=rand(g, D), bias=bias), pre=n)
    same(out, (r.float() + bias).to(dtype))
    plan = make_plan(g, D // 32 * 32, 32, 16)
    xq = x[:, :plan.K].contiguous()
    nq = osm.Norm(shift=shift[:plan.K].clone())
    a, b = plan.alloc_packed(M), plan.alloc_packed(M)
    osm.norm_quantize_act(plan, xq, nq, *a)
    osm.quantize_act(plan, shift[:plan.K].to(BF).expand(M, plan.K).contiguous(), *b)
    for got, ref in zip(a, b):
        same(got, ref)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M, D", [(3, 512), (5, 5120), (400, 5120), (2, 20480)])
def test_rows_beyond_the_range_of_their_statistics(M, D, dtype):
    g = gen(91)
    shift = rand(g, D)
    n = osm.Norm(shift=shift)
    x = rand(g, M, D, dtype=dtype)
    want = osm.norm_modulate(x, n)
    x[0] = rand(g, D, scale=1e19, dtype=dtype)  # squares of 1e38, hundreds of them: the sum of squares is infinite
    x[1] = 3e38                                 # the sum itself is
    h = osm.norm_modulate(x, n)
    same(h[0], shift.to(BF))
    assert bool(torch.isnan(h[1]).all())
    same(h[2:], want[2:])


# Just over the rows from which each width is cut into tiles (148 SMs x 32 warps over the warps of a row), as far as the
# widest; with one run of rows and with three
@pytest.mark.parametrize("M, D", [(6000, 64), (5000, 256), (2500, 504), (1300, 1016), (1300, 1024), (600, 2040), (600, 2048),
                                  (400, 5128), (400, 8184), (400, 8192), (400, 13816), (400, 14336)])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("mode", ["one", "batch"])
@pytest.mark.parametrize("post", [None, osm.NORM_RMS])
def test_rows_in_tiles(M, D, dtype, mode, post):
    g = gen(87)
    x, y = rand(g, M, D, dtype=dtype, scale=2.0, shift=0.7), rand(g, M, D, dtype=BF, shift=0.2)
    n, tokens = make_norm(g, M, D, osm.NORM_LAYER, True, mode)
    href, he = norm64(x, n, tokens)
    within(osm.norm_modulate(x, n), href, he + 2.0 ** -8 * (href.abs() + he) + 1e-37)
    p = None if post is None else make_norm(g, M, D, post, True, "none")[0]
    (gate,), share = modulation(g, M, D, mode, 1)
    out, h = osm.residual_norm(x, y, gate=gate, gate_rows=share, alpha=0.5, post=p, pre=n)
    t, e = (y.double(), torch.zeros(M, D, device="cuda").double()) if p is None else norm64(y, p, M)
    gd = 0.5 * gate.double()[torch.arange(M, device="cuda") // share]
    ref = x.double() + gd * t
    e = e * gd.abs() + 4 * U * (x.double().abs() + 2 * (gd * t).abs())
    within(out, ref, e + HALF[dtype] * (ref.abs() + e))
    href, he = norm64(out, n, tokens)
    within(h, href, he + 2.0 ** -8 * (href.abs() + he) + 1e-37)
    same(h, osm.norm_modulate(out, n))
    alone, none = osm.residual_norm(x, y, gate=gate, gate_rows=share, alpha=0.5, post=p)
    assert none is None
    same(alone, out)
    # in place, with rows behind the last that stay
    xx, yy = torch.cat([x, x[:3]]), torch.cat([y, y[:3]])
    osm.residual_norm(xx[:M], yy[:M], gate=gate, gate_rows=share, alpha=0.5, post=p, pre=n, out=xx[:M], h=yy[:M])
    same(xx[:M], out)
    same(yy[:M], h)
    same(xx[M:], x[:3])
    same(yy[M:], y[:3])


def scale_bytes(buf, rows, nblocks, at):
    """E8M0 bytes of the rows `at`, from the layout's definition: 512-byte atoms of 128 rows x 4 blocks, atoms of one row
    group beside one another, row r and block b at 16 (r % 32) + 4 (r % 128 // 32) + b % 4."""
    r, b = at[:, None], torch.arange(nblocks, device=buf.device)[None]
    return buf[((r // 128) * (nblocks // 4) + b // 4) * 512 + r % 32 * 16 + r % 128 // 32 * 4 + b % 4]


def test_norm_quantize_act_scales_past_32_bit_offsets():
    free, _ = torch.cuda.mem_get_info()
    if free < 40 << 30:
        pytest.skip("needs 40 GiB of free device memory")
    M, K = 900_003, 5120
    plan = make_plan(gen(88), K, 32, 128)
    base = rand(gen(89), 4099, K, dtype=BF)
    x = torch.empty(M, K, dtype=BF, device="cuda")
    for i in range(0, M, 4099):
        n = min(4099, M - i)
        x[i:i + n] = base[:n] * (1 + i % 7)
    a = plan.alloc_packed(M)
    norm = osm.Norm(osm.NORM_RMS, shift=rand(gen(90), K))
    osm.norm_quantize_act(plan, x, norm, *a)
    at = torch.tensor([0, 1, 127, 128, M // 2, 838_860, 838_861, M - 130, M - 2, M - 1], device="cuda")
    few = plan.alloc_packed(at.numel())
    osm.norm_quantize_act(plan, x[at], norm, *few)
    every = torch.arange(at.numel(), device="cuda")
    same(scale_bytes(a[1], M, plan.Kbp // 32, at), scale_bytes(few[1], at.numel(), plan.Kbp // 32, every))
    # the rows that pad the last group of 128 have scale 0
    pad = torch.arange(M, (M + 127) // 128 * 128, device="cuda")
    assert bool((scale_bytes(a[1], M, plan.Kbp // 32, pad) == 0).all())
    assert plan.status() == 0


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("M, K, N", [(300, 512, 1024), (8000, 5120, 64), (700, 5152, 64)])
def test_normed_products_repeat_their_bits(M, K, N, dtype):
    # nothing waits between the passes, and every second one is followed by another layer's on the same stream
    g = gen(92)
    lins = [osm.QuantLinear(make_plan(g, K, N, 64), rand(g, K, N, dtype=BF, scale=0.02)) for _ in range(2)]
    xs = [rand(g, M, K, dtype=dtype, scale=1.5, shift=0.3) for _ in range(2)]
    ns = [osm.Norm(scale=rand(g, K, scale=0.3), shift=rand(g, K)) for _ in range(2)]
    acts = [lin.plan.alloc_packed(M) for lin in lins]
    call = lambda i: lins[i].forward(xs[i], epi=osm.EPI_BF16, norm=ns[i], act_buffers=acts[i])  # noqa: E731
    want = call(0)
    packed = [t.clone() for t in acts[0]]
    torch.cuda.synchronize()
    got = []
    for i in range(50):
        got.append(call(0))
        if i % 2:
            call(1)
    for y in got:
        same(y, want)
    for a, p in zip(acts[0], packed):
        same(a, p)
    assert lins[0].plan.status() == 0
