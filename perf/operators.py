"""The operators around the W4A4 layers of a transformer block, as cases to be measured: the norm with its
modulation, the gated residual with the norms on both sides of it, the norm that hands its rows to a W4A4 product
already quantised, the W4A4 product that adds to the residual stream, and the BF16 product with its epilogue.

Each case has a plain form (elementary torch operations in 32 bits) and the framework's own calls (`own`)."""
import math

import torch

own = False

# E2M1 codes 0..15: three magnitude bits, then the sign
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


# ------------------------------------------------------------------ cases

def listed():
    return [
        # one token's norm in front of the FFN: latency
        {"name": "norm_row", "op": "norm", "M": 1, "D": 5120, "dtype": "bf16", "kind": "layer", "affine": False, "mod": "shared", "groups": 1},
        # the norm in front of the FFN of a whole video's tokens (the FFN block's configuration)
        {"name": "norm_tokens", "op": "norm", "M": 32760, "D": 5120, "dtype": "bf16", "kind": "layer", "affine": False, "mod": "shared", "groups": 1},
        # a short text's tokens, gated residual alone: latency
        {"name": "residual_small", "op": "residual", "M": 77, "D": 512, "dtype": "bf16", "post": "none", "pre": "none", "mod": "shared", "groups": 1, "alpha": 1.0},
        # the step from one sublayer to the next: gated residual, then the next sublayer's modulated norm
        {"name": "residual_norm_tokens", "op": "residual", "M": 32760, "D": 5120, "dtype": "bf16", "post": "none", "pre": "layer", "mod": "shared", "groups": 1, "alpha": 1.0},
        # norms on both sides of the block, FP32 residual stream, three samples of which the last is shorter
        {"name": "residual_sandwich", "op": "residual", "M": 8191, "D": 2048, "dtype": "f32", "post": "rms", "pre": "rms", "mod": "batch", "groups": 3, "alpha": 0.5},
        # the norm in front of a W4A4 layer, quantised on the way: the tiny layer's widths, two samples, FP32 stream
        {"name": "normed_small", "op": "normed", "M": 300, "K": 512, "N": 1024, "k": 16, "dtype": "f32", "kind": "rms", "affine": True, "mod": "batch", "groups": 2},
        # a whole video's tokens normed into a narrow output layer: norm and quantisation are what costs
        {"name": "normed_tokens", "op": "normed", "M": 32760, "K": 5120, "N": 64, "k": 128, "dtype": "bf16", "kind": "layer", "affine": False, "mod": "shared", "groups": 1},
        # the tiny layer's widths, FP32 residual stream
        {"name": "w4a4_residual_small", "op": "w4a4", "M": 256, "K": 1024, "N": 512, "k": 16, "dtype": "f32", "bias": True, "mod": "shared", "groups": 1},
        # the FFN down-projection onto the residual stream
        {"name": "w4a4_residual_down", "op": "w4a4", "M": 32760, "K": 13824, "N": 5120, "k": 256, "dtype": "bf16", "bias": True, "mod": "shared", "groups": 1},
        # a layer kept in BF16, one token: the weights are what is read
        {"name": "linear_row", "op": "linear", "M": 1, "K": 5120, "N": 5120, "dtype": "bf16", "bias": True, "act": "none", "mod": "none", "groups": 1, "residual": False},
        # a short batch through a layer kept in BF16, odd sizes, GELU, FP32 out
        {"name": "linear_ragged", "op": "linear", "M": 1001, "K": 1504, "N": 4128, "dtype": "f32", "bias": True, "act": "gelu", "mod": "none", "groups": 1, "residual": False},
        # an output projection kept in BF16, gated onto the residual stream, a whole video's tokens
        {"name": "linear_tokens", "op": "linear", "M": 32760, "K": 5120, "N": 5120, "dtype": "bf16", "bias": True, "act": "none", "mod": "shared", "groups": 1, "residual": True},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("norm", "residual", "normed", "w4a4", "linear"))
    dtype = rng.choice(("bf16", "f32"))
    mod = rng.choice(("none", "shared", "batch", "token"))
    case = {"op": op, "dtype": dtype, "mod": mod, "groups": 1}
    if op in ("norm", "residual"):
        D = 8 * _log_int(rng, 8, 1728)
        M = _log_int(rng, 1, min(40000, 160_000_000 // D))
        case |= {"M": M, "D": D}
        if op == "norm":
            case |= {"kind": rng.choice(("layer", "rms")), "affine": rng.random() < 0.5}
        else:
            case |= {"post": rng.choice(("none", "layer", "rms")), "pre": rng.choice(("none", "layer", "rms")), "alpha": rng.choice((1.0, 0.5))}
    else:
        K, N = 32 * _log_int(rng, 4, 432), 32 * _log_int(rng, 1, 432)
        M = _log_int(rng, 1, max(1, min(32768, 1_000_000_000_000 // (K * N))))
        case |= {"M": M, "K": K, "N": N}
        if op == "linear":
            case |= {"bias": rng.random() < 0.5, "act": rng.choice(("none", "gelu", "silu")), "residual": rng.random() < 0.7}
        elif op == "w4a4":
            case |= {"bias": rng.random() < 0.5, "k": rng.randint(0, min(K, 256))}
        else:
            case |= {"k": rng.randint(0, min(K, 256)), "kind": rng.choice(("layer", "rms")), "affine": rng.random() < 0.5}
    if mod == "token" and case["M"] * max(case.get(n, 0) for n in "DKN") > 20_000_000:
        case["mod"] = "shared"  # a modulation row for each token is for short inputs
    if case["mod"] == "batch":
        case["groups"] = rng.randint(1, min(4, case["M"]))
    return case


def _rows(case):
    """(modulation rows, tokens that share one)"""
    M = case["M"]
    if case["mod"] == "token":
        return M, 1
    if case["mod"] == "batch":
        share = -(-M // case["groups"])
        return -(-M // share), share
    return 1, M


def _up(n, to):
    return -(-n // to) * to


def work(case):
    M, op = case["M"], case["op"]
    rb = 2 if case["dtype"] == "bf16" else 4
    mrows = 0 if case["mod"] == "none" else _rows(case)[0]
    packed = lambda rows, K, k: rows * (_up(K - k, 128) * 17 // 32 + 2 * _up(k, 64))  # noqa: E731
    if op == "norm":
        D = case["D"]
        return {"bytes": M * D * (rb + 2) + 4 * D * (2 * mrows + 2 * case["affine"]), "flops": 10 * M * D}
    if op == "residual":
        D = case["D"]
        pre = case["pre"] != "none"
        return {"bytes": M * D * (2 * rb + 2 + 2 * pre) + 4 * D * (mrows * (1 + 2 * pre) + 2 * (case["post"] != "none")), "flops": 20 * M * D}
    if op == "w4a4":
        K, N, k = case["K"], case["N"], case["k"]
        return {"bytes": packed(M, K, k) + packed(N, K, k) + 2 * rb * M * N + 4 * N * (case["bias"] + mrows), "flops": 2 * M * N * K}
    if op == "linear":
        K, N = case["K"], case["N"]
        return {"bytes": 2 * (M * K + N * K) + rb * M * N * (1 + case["residual"]) + 4 * N * (case["bias"] + mrows), "flops": 2 * M * N * K}
    K, N = case["K"], case["N"]
    return {"bytes": rb * M * K + packed(N, K, case["k"]) + 2 * M * N + 4 * K * (2 * mrows + 2 * case["affine"]), "flops": 2 * M * N * K}


# ------------------------------------------------------------------ inputs

def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _stream_of(g, M, D, dtype):
    """A residual stream: channels of different widths and means, one in a hundred far wider."""
    width = torch.exp(0.4 * torch.randn(D, generator=g, device="cuda"))
    width = torch.where(torch.rand(D, generator=g, device="cuda") < 0.01, 6 * width, width)
    x = torch.randn(M, D, generator=g, device="cuda") * width + 0.3 * torch.randn(D, generator=g, device="cuda")
    return x.to(dtype)


def _modulation(g, case, n, parts):
    """`parts` vectors of n values for each modulation row, beside one another as the embedding's projection leaves them."""
    if case["mod"] == "none":
        return [None] * parts
    e = 0.3 * torch.randn(_rows(case)[0], parts, n, generator=g, device="cuda")
    return [e[:, i] for i in range(parts)]


def _affine(g, D):
    return 1 + 0.2 * torch.randn(D, generator=g, device="cuda"), 0.1 * torch.randn(D, generator=g, device="cuda")


def _split(g, K, k):
    """Smoothing vector and outlier channels of a layer: s, 1 / s, O ascending, J its complement."""
    s = torch.exp(0.3 * torch.randn(K, generator=g, device="cuda"))
    perm = torch.randperm(K, generator=g, device="cuda")
    return s, 1 / s, perm[:k].sort().values, perm[k:].sort().values


def _times2(v, X):
    """v * 2^X in 32 bits, exactly (X in [-127, 127]): the factor is put together from its exponent's bits."""
    return v * torch.where(X > -127, (X + 127) << 23, torch.full_like(X, 0x400000)).view(torch.float32)


def _codes(v):
    """MXFP4 codes and exponents (X + 127) of [R][n] values, n a multiple of 32: E2M1 with ties to the even code."""
    b = v.float().reshape(v.shape[0], -1, 32)
    amax = b.abs().amax(2)
    X = (torch.frexp(amax).exponent - 3).clamp(-127, 127)
    X = torch.where(amax == 0, torch.full_like(X, -127), X)
    a = _times2(b, -X[..., None])
    m = a.abs()
    code = ((m > 0.25).to(torch.uint8) + (m >= 0.75) + (m > 1.25) + (m >= 1.75) + (m > 2.5) + (m >= 3.5) + (m > 5.0)).to(torch.uint8)
    return (code | (torch.signbit(b).to(torch.uint8) << 3)).reshape(v.shape[0], -1), X


def _packed(v, J, O):
    """[R][K] smoothed BF16 values as packed operands: codes, scales in 128 x 4 atoms, outlier slots."""
    R, Kb, k = v.shape[0], J.numel(), O.numel()
    Kbp, kp, Rp = _up(Kb, 128), _up(k, 64), _up(R, 128)
    hp = torch.zeros(R, kp, dtype=torch.bfloat16, device="cuda")
    hp[:, :k] = v[:, O]
    if not Kb:
        return torch.empty(0, dtype=torch.uint8, device="cuda"), torch.empty(0, dtype=torch.uint8, device="cuda"), hp.reshape(-1)
    bulk = torch.zeros(R, Kbp, dtype=torch.bfloat16, device="cuda")
    bulk[:, :Kb] = v[:, J]
    c, X = _codes(bulk)
    codes = c[:, 0::2] | (c[:, 1::2] << 4)
    sc = torch.zeros(Rp, Kbp // 32, dtype=torch.uint8, device="cuda")
    real = _up(Kb, 32) // 32
    sc[:R, :real] = (X[:, :real] + 127).to(torch.uint8)
    sc = sc.view(Rp // 128, 4, 32, Kbp // 128, 4).permute(0, 3, 2, 1, 4)
    return codes.reshape(-1), sc.reshape(-1), hp.reshape(-1)


def _norm_state(g, case, D, st, name, kind, affine, scale, shift):
    st[name] = {"kind": kind, "eps": 1e-6, "w": None, "b": None, "scale": scale, "shift": shift, "share": _rows(case)[1]}
    if affine:
        st[name]["w"], st[name]["b"] = _affine(g, D)
        if kind == "rms":
            st[name]["b"] = None


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    M, op, dt = case["M"], case["op"], _type(case)
    st = {"case": case, "share": _rows(case)[1]}
    rand = lambda *n: torch.randn(*n, generator=g, device="cuda")  # noqa: E731
    if op == "norm":
        D = case["D"]
        st["x"] = _stream_of(g, M, D, dt)
        shift, scale = _modulation(g, case, D, 2)
        _norm_state(g, case, D, st, "norm", case["kind"], case["affine"], scale, shift)
        st["h"] = torch.empty(M, D, dtype=torch.bfloat16, device="cuda")
    elif op == "residual":
        D = case["D"]
        st["r"] = _stream_of(g, M, D, dt)
        st["y"] = (0.5 * rand(M, D)).bfloat16()
        st["gate"], shift, scale = _modulation(g, case, D, 3)
        st["post"] = st["pre"] = None
        if case["post"] != "none":
            _norm_state(g, case, D, st, "post", case["post"], True, None, None)
        if case["pre"] != "none":
            _norm_state(g, case, D, st, "pre", case["pre"], False, scale, shift)
        st["out"] = torch.empty(M, D, dtype=dt, device="cuda")
        st["h"] = torch.empty(M, D, dtype=torch.bfloat16, device="cuda") if st["pre"] else None
    elif op == "w4a4":
        K, N, k = case["K"], case["N"], case["k"]
        s, inv_s, O, J = _split(g, K, k)
        wide = torch.ones(K, device="cuda")
        wide[O] = 6.0
        x = torch.randn(M, K, generator=g, device="cuda").mul_(0.3 * wide).bfloat16()
        st["a"] = _packed(x, J, O)
        del x
        st["w"] = _packed((0.02 * rand(N, K)).bfloat16(), J, O)
        st["r"] = _stream_of(g, M, N, dt)
        st["bias"] = 0.1 * rand(N) if case["bias"] else None
        st["gate"], = _modulation(g, case, N, 1)
        st["out"] = torch.empty(M, N, dtype=dt, device="cuda")
        st["Kb"] = K - k
        if own:
            import outlier_split_mixed_b200 as osm
            st["plan"] = osm.Plan(K, N, k, s.cpu().numpy(), O.int().cpu().numpy())
    elif op == "linear":
        K, N = case["K"], case["N"]
        st["x"] = _stream_of(g, M, K, torch.bfloat16)
        st["w"] = torch.zeros(N, _up(K, 64), dtype=torch.bfloat16, device="cuda")  # a plan's packed BF16 weights
        st["w"][:, :K] = rand(N, K) / math.sqrt(K)
        st["r"] = _stream_of(g, M, N, dt) if case["residual"] else None
        st["bias"] = 0.1 * rand(N) if case["bias"] else None
        st["gate"], = _modulation(g, case, N, 1)
        st["out"] = torch.empty(M, N, dtype=dt, device="cuda")
        if own:
            import outlier_split_mixed_b200 as osm
            st["plan"] = osm.hp_plan(K, N)
    else:
        K, N, k = case["K"], case["N"], case["k"]
        st["x"] = _stream_of(g, M, K, dt)
        shift, scale = _modulation(g, case, K, 2)
        _norm_state(g, case, K, st, "norm", case["kind"], case["affine"], scale, shift)
        s, st["inv_s"], st["O"], st["J"] = _split(g, K, k)
        st["w"] = _packed((rand(N, K) / math.sqrt(K) * s).bfloat16(), st["J"], st["O"])
        st["out"] = torch.empty(M, N, dtype=torch.bfloat16, device="cuda")
        if own:
            import outlier_split_mixed_b200 as osm
            st["plan"] = osm.Plan(K, N, k, s.cpu().numpy(), st["O"].int().cpu().numpy())
            st["a"] = st["plan"].alloc_packed(M)
    return st


# ------------------------------------------------------------------ plain forms

def _each(v, share, M):
    """A modulation vector for each token: row t takes row t // share (one row is left to broadcast)."""
    return v if v.shape[0] == 1 else v.repeat_interleave(share, 0)[:M]


def _norm(x, n):
    """The norm with its affine part and its modulation, in 32 bits."""
    x = x.float()
    if n["kind"] == "layer":
        x = x - x.mean(1, keepdim=True)
    v = x * torch.rsqrt((x * x).mean(1, keepdim=True) + n["eps"])
    if n["w"] is not None:
        v = v * n["w"]
    if n["b"] is not None:
        v = v + n["b"]
    if n["scale"] is not None:
        v = v * (1 + _each(n["scale"], n["share"], x.shape[0])) + _each(n["shift"], n["share"], x.shape[0])
    return v


def _values(ops, rows, Kb):
    """Packed operands as the values that they stand for: [rows][bulk positions, then outlier slots]."""
    codes, sc, hp = ops
    hp = hp.view(rows, -1).float()
    if not Kb:
        return hp
    Kbp = _up(Kb, 128)
    lut = torch.tensor(E2M1, device="cuda")
    c = codes.view(rows, -1, 1)
    v = lut[torch.cat([c & 15, c >> 4], 2).int()].view(rows, Kbp // 32, 32)
    e = sc.view(-1, Kbp // 128, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, Kbp // 32)[:rows].int() - 127
    v = _times2(v, e[..., None]).view(rows, Kbp)
    return torch.cat([v, hp], 1)


def _quantised(h, inv_s, J, O):
    """Smoothed and split activations as the values that their packed form stands for."""
    v = (h.float() * inv_s).bfloat16()
    bulk = torch.zeros(h.shape[0], _up(J.numel(), 128), dtype=torch.bfloat16, device="cuda")
    bulk[:, :J.numel()] = v[:, J]
    hp = torch.zeros(h.shape[0], _up(O.numel(), 64), device="cuda")
    hp[:, :O.numel()] = v[:, O].float()
    if not J.numel():
        return hp
    c, X = _codes(bulk)
    q = torch.tensor(E2M1, device="cuda")[c.int()].view(h.shape[0], -1, 32)
    return torch.cat([_times2(q, X[..., None]).view(h.shape[0], -1), hp], 1)


def _gelu(x):
    return x / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x * x * x)))


def _act(x, act):
    return _gelu(x) if act == "gelu" else x / (1 + torch.exp(-x)) if act == "silu" else x


def _onto(y, st):
    """The end of a sublayer: gated, onto the residual stream, in its type."""
    if st["gate"] is not None:
        y = y * _each(st["gate"], st["share"], y.shape[0])
    if st["r"] is not None:
        y = st["r"].float() + y
    return y.to(st["out"].dtype)


def _plain(st):
    case, op = st["case"], st["case"]["op"]
    if op == "norm":
        return _norm(st["x"], st["norm"]).bfloat16()
    if op == "residual":
        y = _norm(st["y"], st["post"]) if st["post"] else st["y"].float()
        r = _onto(case["alpha"] * y, st)
        return {"r": r, "h": _norm(r, st["pre"]).bfloat16()} if st["pre"] else {"r": r}
    if op == "w4a4":
        y = _values(st["a"], case["M"], st["Kb"]) @ _values(st["w"], case["N"], st["Kb"]).T
        return _onto(y if st["bias"] is None else y + st["bias"], st)
    if op == "linear":
        y = st["x"].float() @ st["w"][:, :case["K"]].float().T
        return _onto(_act(y if st["bias"] is None else y + st["bias"], case["act"]), st)
    a = _quantised(_norm(st["x"], st["norm"]).bfloat16(), st["inv_s"], st["J"], st["O"])
    return (a @ _values(st["w"], case["N"], case["K"] - case["k"]).T).bfloat16()


# ------------------------------------------------------------------ one pass

def _spec(osm, n):
    if n is None:
        return None
    return osm.Norm(osm.NORM_LAYER if n["kind"] == "layer" else osm.NORM_RMS, eps=n["eps"], weight=n["w"], bias=n["b"],
                    scale=n["scale"], shift=n["shift"], mod_rows=n["share"])


def run(st):
    if not own:
        return _plain(st)
    import outlier_split_mixed_b200 as osm
    case, op = st["case"], st["case"]["op"]
    if op == "norm":
        return osm.norm_modulate(st["x"], _spec(osm, st["norm"]), out=st["h"])
    if op == "residual":
        r, h = osm.residual_norm(st["r"], st["y"], gate=st["gate"], gate_rows=st["share"], alpha=case["alpha"],
                                 post=_spec(osm, st["post"]), pre=_spec(osm, st["pre"]), out=st["out"], h=st["h"])
        return {"r": r, "h": h} if st["pre"] else {"r": r}
    if op == "w4a4":
        return osm.dual_gemm_residual(st["plan"], *st["a"], case["M"], *st["w"], st["r"], out=st["out"], bias=st["bias"],
                                      gate=st["gate"], gate_rows=st["share"])
    if op == "linear":
        act = {"none": osm.ACT_NONE, "gelu": osm.ACT_GELU, "silu": osm.ACT_SILU}[case["act"]]
        return osm.linear_hp(st["plan"], st["x"], st["w"], bias=st["bias"], act=act, gate=st["gate"], gate_rows=st["share"],
                             residual=st["r"], out=st["out"])
    osm.norm_quantize_act(st["plan"], st["x"], _spec(osm, st["norm"]), *st["a"])
    osm.dual_gemm(st["plan"], *st["a"], case["M"], *st["w"], st["out"], epi=osm.EPI_BF16)
    return st["out"]


# ------------------------------------------------------------------ the definition in 64 bits

def _norm64(x, n, group):
    x = x.double()
    c = x - x.sum(1, keepdim=True) / x.shape[1] if n["kind"] == "layer" else x
    v = c / torch.sqrt(c.square().sum(1, keepdim=True) / x.shape[1] + n["eps"])
    v = v * n["w"].double() if n["w"] is not None else v
    v = v + n["b"].double() if n["b"] is not None else v
    return v if n["scale"] is None else v * (1 + n["scale"].double()[group]) + n["shift"].double()[group]


def _pow64(e):
    """2^e in 64 bits, e whole numbers in [-160, 160], from a table."""
    return torch.tensor([2.0 ** i for i in range(-160, 161)], dtype=torch.float64, device="cuda")[e.long() + 160]


def _floor_log2(x):
    return torch.frexp(x).exponent - 1


def _decoded64(ops, rows, Kb):
    """Each value from its own place in the packed buffers: code byte p // 2 of the row, scale byte of its atom."""
    codes, sc, hp = ops
    if not Kb:
        return hp.view(rows, -1).double()
    half = _up(Kb, 128) // 2
    byte = codes.view(rows, half)
    nib = torch.stack([byte & 15, byte >> 4], 2).view(rows, -1)[:, :Kb].long()
    mag, sign = nib & 7, 1 - 2 * (nib >> 3)
    e, m = mag >> 1, mag & 1
    v = sign * torch.where(e > 0, (2 + m).double() * _pow64(e - 2), m.double() / 2)
    r, b = torch.arange(rows, device="cuda")[:, None], torch.arange(-(-Kb // 32), device="cuda")[None]
    at = ((r // 128) * (half // 64) + b // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4
    v = v * _pow64(sc[at].int() - 127).repeat_interleave(32, 1)[:, :Kb]
    return torch.cat([v, hp.view(rows, -1).double()], 1)


def _encoded64(x, J, O):
    """Smoothed values [R][K] as the values of their MXFP4 blocks and outlier slots (the slots padded)."""
    R = x.shape[0]
    slots = torch.zeros(R, _up(O.numel(), 64), dtype=torch.float64, device="cuda")
    slots[:, :O.numel()] = x[:, O]
    if not J.numel():
        return slots
    v = torch.zeros(R, _up(J.numel(), 32), dtype=torch.float64, device="cuda")
    v[:, :J.numel()] = x[:, J]
    v = v.view(R, -1, 32)
    top = v.abs().amax(2, keepdim=True).clamp_min(2.0 ** -125)
    unit = _pow64(_floor_log2(top) - 2)
    u = v / unit
    step = _pow64(_floor_log2(u.abs().clamp_min(1.0)) - 1)  # half below 2, one below 4, two above
    q = (torch.round(u / step) * step).clamp(-6, 6) * unit
    return torch.cat([q.view(R, -1)[:, :J.numel()], slots], 1)


def _gelu64(x):
    return 0.5 * x * (1 + torch.tanh(math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)))


def exact(case, seed):
    st = prepare(case, seed)
    op, M = case["op"], case["M"]
    group = torch.arange(M, device="cuda") // st["share"]

    def end(y):
        y = y if st["gate"] is None else y * st["gate"].double()[group]
        return y if st["r"] is None else st["r"].double() + y

    if op == "norm":
        return _norm64(st["x"], st["norm"], group)
    if op == "residual":
        r = end(case["alpha"] * (_norm64(st["y"], st["post"], group) if st["post"] else st["y"].double()))
        return {"r": r, "h": _norm64(r.to(_type(case)), st["pre"], group)} if st["pre"] else {"r": r}
    if op == "w4a4":
        Kb = case["K"] - case["k"]
        y = _decoded64(st["a"], M, Kb) @ _decoded64(st["w"], case["N"], Kb).T
        return end(y if st["bias"] is None else y + st["bias"].double())
    if op == "linear":
        y = torch.mm(st["x"].double(), st["w"].double()[:, :case["K"]].t())
        y = y if st["bias"] is None else y + st["bias"].double()
        y = _gelu64(y) if case["act"] == "gelu" else y * torch.sigmoid(y) if case["act"] == "silu" else y
        return end(y)
    x = _norm64(st["x"], st["norm"], group).bfloat16().double() * st["inv_s"].double()
    return _encoded64(x.bfloat16().double(), st["J"], st["O"]) @ _decoded64(st["w"], case["N"], case["K"] - case["k"]).T
