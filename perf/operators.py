"""Measured cases of the 4-bit (microscaled) linear layer and of the fused
norm/residual step around it.

Operators, by a case's ``"op"``:

``quant``   rows of x to E2M1 codes with microscales, and read back as values
``linear``  y = q(x) q(W)^T: x quantised per call, W quantised once
``decode``  y = prune(x) q(W)^T for 1..16 tokens, x unquantised
``norm``    r' = a r + gate (y/rms(y) w_post), h = r'/rms(r') w_pre
``block``   the norm step whose h goes as codes into the product

Formats: ``mx`` is E2M1 in blocks of 32 channels with an E8M0 scale, ``nv``
E2M1 in blocks of 16 with an E4M3 scale and one power-of-two float32 scale per
row.  Codes are two per byte (even channel in the low nibble); scale bytes are
in tiles of 128 rows by 4 blocks, row r and block c of a tile at byte
16*(r % 32) + 4*(r // 32) + c.
"""
import math

import torch

own = False

_BLOCK = {"mx": 32, "nv": 16}
_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode token's hidden state, quantised for a 4-bit product
        dict(name="quant_token", op="quant", fmt="nv", dtype="bf16", rows=1, K=4096),
        # a projection's float32 master weights
        dict(name="quant_weights_f32", op="quant", fmt="mx", dtype="f32", rows=4096, K=11008),
        # the FFN activations of a 4096-token prompt
        dict(name="quant_prompt", op="quant", fmt="nv", dtype="bf16", rows=4096, K=14336),
        # key/value projection of a short prompt
        dict(name="linear_kv_short", op="linear", fmt="nv", dtype="bf16", out="bf16", T=40, K=4096, n_out=1024),
        # down projection of a ragged prompt, float32 output
        dict(name="linear_down_ragged", op="linear", fmt="mx", dtype="bf16", out="f32", T=777, K=11008, n_out=4096),
        # down projection of a whole prompt
        dict(name="linear_down_prompt", op="linear", fmt="nv", dtype="bf16", out="bf16", T=4096, K=14336,
             n_out=4096),
        # the layer's headline decode: one token, 8:16 weight-aware with the token shift
        dict(name="decode_one", op="decode", fmt="nv", dtype="bf16", out="bf16", T=1, K=11008, n_out=4096,
             sel="nm", n=8, m=16, keep=0.0, score="weight", dpts=True),
        # gate/up projection of three tokens, per-token top-k, float32 output
        dict(name="decode_topk", op="decode", fmt="nv", dtype="f32", out="f32", T=3, K=4096, n_out=14336,
             sel="topk", n=0, m=0, keep=0.5, score="mag", dpts=False),
        # down projection of a full decode batch
        dict(name="decode_batch", op="decode", fmt="mx", dtype="bf16", out="bf16", T=16, K=14336, n_out=4096,
             sel="nm", n=8, m=16, keep=0.0, score="mag", dpts=False),
        # between two blocks, one token
        dict(name="norm_token", op="norm", T=1, D=4096, rdt="bf16", ydt="bf16", hdt="bf16", gate="channel"),
        # between two blocks of a long prompt, float32 residual stream, gate of every token and channel
        dict(name="norm_prompt", op="norm", T=8192, D=8192, rdt="f32", ydt="bf16", hdt="bf16", gate="token"),
        # the norm step feeding the query projection in 4 bits
        dict(name="block_prompt", op="block", fmt="nv", out="bf16", T=1000, D=4096, n_out=4096, rdt="bf16",
             ydt="bf16", gate="channel"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["quant", "linear", "linear", "decode", "decode", "norm", "block"])
    fmt, odd = rng.choice(["mx", "nv"]), rng.random() < 0.5
    if op == "quant":
        K = 32 * _log(rng, 2, 448)
        return dict(op=op, fmt=fmt, dtype=rng.choice(["bf16", "f32"]), rows=_log(rng, 1, 4096), K=K)
    if op == "linear":
        return dict(op=op, fmt=fmt, dtype=rng.choice(["bf16", "bf16", "f32"]), out=rng.choice(["bf16", "f32"]),
                    T=_log(rng, 1, 4096), K=(32 if odd else 256) * _log(rng, 2, 448 if odd else 56),
                    n_out=(8 if odd else 128) * _log(rng, 8, 512 if odd else 32))
    if op == "decode":
        # K limited so that a call costs no more than the full decode batch
        K, n_out = 32 * _log(rng, 4, 448), 8 * _log(rng, 16, 512)
        sel = rng.choice(["nm", "nm", "topk", "all"])
        m = rng.choice([4, 8, 16, 32])
        return dict(op=op, fmt=fmt, dtype=rng.choice(["bf16", "bf16", "f32"]), out=rng.choice(["bf16", "f32"]),
                    T=rng.randint(1, 16), K=K, n_out=n_out, sel=sel, n=m // 2 if sel == "nm" else 0,
                    m=m if sel == "nm" else 0, keep=round(rng.uniform(0.4, 0.7), 3) if sel == "topk" else 0.0,
                    score=rng.choice(["mag", "weight"]), dpts=rng.random() < 0.5)
    rdt, ydt = rng.choice(["bf16", "f32"]), rng.choice(["bf16", "f32"])
    gate = rng.choice(["none", "channel", "token"])
    if op == "norm":
        return dict(op=op, T=_log(rng, 1, 4096), D=8 * _log(rng, 8, 1024), rdt=rdt, ydt=ydt,
                    hdt=rng.choice(["bf16", "f32"]), gate=gate)
    # bf16 output: a float32 norm next to a rounding border of the codes may go either way
    return dict(op=op, fmt=fmt, out="bf16", T=_log(rng, 1, 2048), D=32 * _log(rng, 8, 256),
                n_out=8 * _log(rng, 16, 512), rdt=rdt, ydt=ydt, gate=gate)


def _size(name):
    return 2 if name == "bf16" else 4


def _codes_bytes(rows, K, fmt):
    return rows * K // 2 + rows * K // _BLOCK[fmt] + (4 * rows if fmt == "nv" else 0)


def work(case):
    op = case["op"]
    if op == "quant":  # the codes are written and read back, the values written
        n = case["rows"] * case["K"]
        return {"bytes": 2 * n * _size(case["dtype"]) + 2 * _codes_bytes(case["rows"], case["K"], case["fmt"]),
                "flops": 4 * n}
    if op == "linear":
        T, K, n = case["T"], case["K"], case["n_out"]
        return {"bytes": T * K * _size(case["dtype"]) + _codes_bytes(n, K, case["fmt"]) + T * n * _size(case["out"]),
                "flops": 2 * T * K * n}
    if op == "decode":
        T, K, n = case["T"], case["K"], case["n_out"]
        f = {"nm": case["n"] / max(case["m"], 1), "topk": case["keep"], "all": 1.0}[case["sel"]]
        union = 1.0 - (1.0 - f) ** T  # expected share of channels that some token keeps
        by = int(union * K * n / 2) + K * n // _BLOCK[case["fmt"]] + T * K * _size(case["dtype"])
        by += T * n * _size(case["out"]) + 4 * n + (4 * K if case["score"] == "weight" else 0)
        return {"bytes": by + (4 * n if case["dpts"] else 0), "flops": int(2 * T * f * K * n)}
    T, D = case["T"], case["D"]
    gate = {"none": 0, "channel": 4 * D, "token": 4 * T * D}[case["gate"]]
    by = T * D * (_size(case["ydt"]) + 2 * _size(case["rdt"])) + gate + 8 * D
    if op == "norm":
        return {"bytes": by + T * D * _size(case["hdt"]), "flops": 10 * T * D}
    n = case["n_out"]
    return {"bytes": by + _codes_bytes(n, D, case["fmt"]) + T * n * _size(case["out"]), "flops": 2 * T * D * n}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _laplace(g, *shape):
    u = torch.rand(*shape, generator=g, device="cuda") - 0.5
    return -torch.sign(u) * torch.log1p(-2.0 * u.abs().clamp(max=0.4999999))


def _activations(g, T, K):
    """Laplace(0, 0.3) with 1 % outlier channels twenty times as large."""
    x = 0.3 * _laplace(g, T, K)
    hot = torch.rand(K, generator=g, device="cuda") < 0.01
    return torch.where(hot, 20.0 * x, x)


def _weights(g, n_out, K):
    return torch.randn(n_out, K, generator=g, device="cuda") * 0.02


def _inputs(case, seed):
    """The case's float inputs, the same for every side."""
    g, op, d = _gen(seed), case["op"], {}
    if op == "quant":
        x = _activations(g, case["rows"], case["K"])
        x = torch.where(torch.rand(case["rows"], case["K"] // 32, 1, generator=g, device="cuda") < 0.02, 0.0,
                        x.view(case["rows"], -1, 32)).view(case["rows"], case["K"])  # blocks of natural zeros
        d["x"] = x.to(_DT[case["dtype"]])
    elif op in ("linear", "decode"):
        d["x"] = _activations(g, case["T"], case["K"]).to(_DT[case["dtype"]])
        d["W"] = _weights(g, case["n_out"], case["K"])
    else:
        T, D = case["T"], case["D"]
        d["r"] = _activations(g, T, D).to(_DT[case["rdt"]])
        d["y"] = (2.0 * torch.randn(T, D, generator=g, device="cuda")).to(_DT[case["ydt"]])
        d["post_w"] = 1.0 + 0.1 * torch.randn(D, generator=g, device="cuda")
        d["pre_w"] = 1.0 + 0.1 * torch.randn(D, generator=g, device="cuda")
        if case["gate"] == "channel":
            d["gate"] = 0.5 + 0.1 * torch.randn(D, generator=g, device="cuda")
        elif case["gate"] == "token":
            d["gate"] = 0.5 + 0.1 * torch.randn(T, D, generator=g, device="cuda")
        else:
            d["gate"] = None
        if op == "block":
            d["W"] = _weights(g, case["n_out"], D)
    return d


_EPS, _ALPHA = 1e-6, 0.9


# --------------------------------------------------- plain forms: the format
def _pow2(e):
    return torch.ldexp(torch.ones_like(e, dtype=torch.float64), e.to(torch.int32))


def _round_e2m1(a):
    """Nearest E2M1 magnitude of a >= 0, ties to the even code, at most 6."""
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0)).to(a.dtype)
    return (torch.round(a / step) * step).clamp(max=6.0)


def _round_e4m3(a):
    """Nearest E4M3 value of 0 <= a <= 448, ties to even."""
    _, ex = torch.frexp(a.clamp(min=2.0 ** -6))
    step = _pow2(ex - 4)
    return torch.round(a / step) * step


def _quant(x, fmt):
    """Signed E2M1 values [R, K], block scales [R, K/B], row scale [R] (float64:
    quotients lie next to rounding borders)."""
    R, K = x.shape
    v = x.to(torch.float64).view(R, -1, _BLOCK[fmt])
    amax = v.abs().amax(-1)
    if fmt == "mx":
        _, ex = torch.frexp(amax)
        s = _pow2((ex - 3).clamp(min=-127))
        s = torch.where(amax > 0, s, 1.0)
        S = torch.ones(R, dtype=torch.float64, device=x.device)
        div = s
    else:
        top = amax.amax(-1)
        m, ex = torch.frexp(top)
        e = torch.where(m <= 0.65625, ex - 12, ex - 11).clamp(min=-126)
        S = torch.where(top > 0, _pow2(e), 1.0)
        s = _round_e4m3(amax / (6.0 * S[:, None]))
        div = s * S[:, None]
    q = _round_e2m1(v.abs() / torch.where(div > 0, div, 1.0)[..., None])
    q = torch.where((div > 0)[..., None], torch.copysign(q, v), 0.0)
    return q.view(R, K).float(), s.float(), S.float()


def _pack_codes(q):
    """E2M1 values [R, K] -> bytes [R, K/2]."""
    mag = torch.bucketize(q.abs(), torch.tensor(_E2M1, device=q.device))
    code = (mag + 8 * torch.signbit(q)).to(torch.uint8)
    return (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous()


def _unpack_codes(b):
    lut = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), device=b.device)
    return torch.stack([lut[(b & 15).long()], lut[(b >> 4).long()]], -1).view(b.shape[0], -1)


def _scale_byte(s, fmt):
    if fmt == "mx":
        return (torch.frexp(s)[1] - 1 + 127).to(torch.uint8)
    m, ex = torch.frexp(s.clamp(min=2.0 ** -6))
    normal = (((ex - 1 + 7) << 3) + torch.round((2 * m - 1) * 8).to(torch.int32)).to(torch.uint8)
    return torch.where(s >= 2.0 ** -6, normal, torch.round(s * 512.0).to(torch.uint8))


def _scale_value(b, fmt):
    b = b.to(torch.int32)
    if fmt == "mx":
        return torch.ldexp(torch.ones_like(b, dtype=torch.float32), b - 127)
    e, m = b >> 3, (b & 7).float()
    return torch.where(e > 0, torch.ldexp(1.0 + m / 8, e - 7), m / 512.0)


def _tile_scales(b):
    """Scale bytes [R, C] -> the tiled buffer (padding zero)."""
    R, C = b.shape
    rt, ct = (R + 127) // 128, (C + 3) // 4
    p = torch.zeros(rt * 128, ct * 4, dtype=torch.uint8, device=b.device)
    p[:R, :C] = b
    return p.view(rt, 4, 32, ct, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)


def _untile_scales(t, R, C):
    rt, ct = (R + 127) // 128, (C + 3) // 4
    return t.view(rt, ct, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(rt * 128, ct * 4)[:R, :C]


def _values(q, s):
    """Codes times block scales, float32 (exact)."""
    R, K = q.shape
    return (q.view(R, s.shape[1], -1) * s[..., None]).view(R, K)


def _stored_values(st):
    """Values of a stored weight: codes x block scale (the row scale apart)."""
    q = _unpack_codes(st["Wq"])
    s = _scale_value(_untile_scales(st["w_sf"], q.shape[0], q.shape[1] // _BLOCK[st["fmt"]]), st["fmt"])
    return _values(q, s)


# ------------------------------------------------------------------ prepare
def prepare(case, seed):
    op = case["op"]
    st = _inputs(case, seed)
    st.update(op=op, case=case, fmt=case.get("fmt"))
    if "W" in st:  # quantised once, kept in the format's layout
        q, s, S = _quant(st.pop("W"), case["fmt"])
        st["Wq"], st["w_sf"], st["w_scale"] = _pack_codes(q), _tile_scales(_scale_byte(s, case["fmt"])), S
    if op == "decode":
        w = _values(q, s).double() * S.double()[:, None]
        st["g"] = torch.sqrt(torch.sqrt((w * w).sum(0))).float()  # column norm to the power 1/2
        st["rowsum"] = w.sum(1).float()
        del w
        st["keep"] = int(case["keep"] * case["K"] + 0.5)
    if own:
        _prepare_own(case, st)
    return st


def _empty_codes(sl, rows, K, fmt):
    return dict(q=torch.empty(rows, K // 2, dtype=torch.uint8, device="cuda"),
                sf=torch.empty(sl.as_fp4_sf_bytes(rows, K, fmt), dtype=torch.uint8, device="cuda"),
                scale=torch.empty(rows, dtype=torch.float32, device="cuda") if fmt == sl.AS_FP4_NV else None)


def _prepare_own(case, st):
    import sparse_linear_b200 as sl
    from sparse_linear_b200.layer import workspace
    op = case["op"]
    st["sl"] = sl
    if "fmt" in case:
        fmt = st["cfmt"] = sl.AS_FP4_NV if case["fmt"] == "nv" else sl.AS_FP4_MX
    if op == "quant":
        st["codes"] = _empty_codes(sl, case["rows"], case["K"], fmt)
        st["out"] = torch.empty_like(st["x"])
    elif op in ("linear", "block"):
        T, K = case["T"], case["K"] if op == "linear" else case["D"]
        st["codes"] = _empty_codes(sl, T, K, fmt)
        st["out"] = torch.empty(T, case["n_out"], dtype=_DT[case["out"]], device="cuda")
    elif op == "decode":
        T, K, n_out = case["T"], case["K"], case["n_out"]
        sel = {"nm": sl.AS_SEL_NM, "topk": sl.AS_SEL_TOPK, "all": sl.AS_SEL_ALL}[case["sel"]]
        st["cfg"] = sl.config(score=sl.AS_SCORE_WEIGHT if case["score"] == "weight" else sl.AS_SCORE_MAG, sel=sel,
                              n=case["n"], m=case["m"], k_keep=st["keep"], dpts=case["dpts"],
                              out_dtype=sl.AS_BF16 if case["out"] == "bf16" else sl.AS_F32)
        st["Wd"] = torch.empty(sl.as_fp4_decode_bytes(n_out, K, fmt), dtype=torch.uint8, device="cuda")
        sl.as_weight_prep_fp4(st["Wq"], st["w_sf"], st["Wd"], w_scale=st["w_scale"], fmt=fmt)
        st["ws"] = workspace(sl.as_workspace_size(sl.AS_OP_DECODE_FP4, T, K, n_out, st["cfg"]), "cuda")
        st["out"] = torch.empty(T, n_out, dtype=_DT[case["out"]], device="cuda")
    if op in ("norm", "block"):
        st["r_out"] = torch.empty_like(st["r"])
        if op == "norm":
            st["h"] = torch.empty(case["T"], case["D"], dtype=_DT[case["hdt"]], device="cuda")


# ------------------------------------------------------------------ run
def run(st):
    return (_run_own if own else _run_plain)(st)


def _run_own(st):
    sl, op, case = st["sl"], st["op"], st["case"]
    if op == "quant":
        c, fmt = st["codes"], st["cfmt"]
        sl.as_quant_fp4(st["x"], c["q"], c["sf"], c["scale"], fmt=fmt)
        sl.as_dequant_fp4(c["q"], c["sf"], st["out"], c["scale"], fmt=fmt)
        return st["out"]
    if op == "linear":
        c, fmt = st["codes"], st["cfmt"]
        sl.as_quant_fp4(st["x"], c["q"], c["sf"], c["scale"], fmt=fmt)
        sl.as_linear_prefill_fp4(c["q"], c["sf"], st["Wq"], st["w_sf"], st["out"], x_scale=c["scale"],
                                 w_scale=st["w_scale"], fmt=fmt)
        return st["out"]
    if op == "decode":
        sl.as_linear_decode_fp4(st["x"], st["Wd"], st["cfg"], st["out"], fmt=st["cfmt"],
                                g=st["g"] if case["score"] == "weight" else None,
                                rowsum=st["rowsum"] if case["dpts"] else None, workspace=st["ws"])
        return st["out"]
    norm = dict(y=st["y"], post_w=st["post_w"], gate=st["gate"], pre_w=st["pre_w"], r_out=st["r_out"],
                res_scale=_ALPHA, eps=_EPS, post_norm=True)
    if op == "norm":
        sl.as_norm_residual(st["r"], h=st["h"], **norm)
        return st["r_out"], st["h"]
    c, fmt = st["codes"], st["cfmt"]
    sl.as_norm_residual(st["r"], h_q=c["q"], h_sf=c["sf"], h_scale=c["scale"], fmt=fmt, **norm)
    sl.as_linear_prefill_fp4(c["q"], c["sf"], st["Wq"], st["w_sf"], st["out"], x_scale=c["scale"],
                             w_scale=st["w_scale"], fmt=fmt)
    return st["r_out"], st["out"]


def _product(x, st, out):
    q, s, S = _quant(x, st["fmt"])
    acc = _values(q, s) @ _stored_values(st).T
    return (acc * S[:, None] * st["w_scale"]).to(out)


def _norm(st):
    y = st["y"].float()
    u = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + _EPS) * st["post_w"]
    if st["gate"] is not None:
        u = u * st["gate"]
    f = _ALPHA * st["r"].float() + u
    return f.to(st["r"].dtype), f * torch.rsqrt((f * f).mean(-1, keepdim=True) + _EPS) * st["pre_w"]


def _kept(x, st):
    """Kept values of every token (zeros where dropped) and the token shift."""
    case = st["case"]
    xf = x.float()
    eta = xf.double().mean(-1).float() if case["dpts"] else None
    if eta is not None:
        xf = xf - eta[:, None]
    sc = xf.abs() * st["g"] if case["score"] == "weight" else xf.abs()
    if case["sel"] == "all":
        return xf, eta
    n, blk = (case["n"], sc.view(sc.shape[0], -1, case["m"])) if case["sel"] == "nm" else (st["keep"], sc[:, None])
    order = torch.sort(blk, dim=-1, descending=True, stable=True)[1]  # ties to the lower channel
    mask = torch.zeros_like(blk).scatter_(-1, order[..., :n], 1.0)
    return xf * mask.view_as(xf), eta


def _run_plain(st):
    op, case = st["op"], st["case"]
    if op == "quant":
        q, s, S = _quant(st["x"], st["fmt"])
        return (_values(q, s) * S[:, None]).to(st["x"].dtype)
    if op == "linear":
        return _product(st["x"], st, _DT[case["out"]])
    if op == "decode":
        xk, eta = _kept(st["x"], st)
        y = (xk @ _stored_values(st).T) * st["w_scale"]
        if eta is not None:
            y = y + eta[:, None] * st["rowsum"]
        return y.to(_DT[case["out"]])
    r, h = _norm(st)
    if op == "norm":
        return r, h.to(_DT[case["hdt"]])
    return r, _product(h, st, _DT[case["out"]])


# ------------------------------------------------------------------ exact
_MID = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)  # borders between E2M1 magnitudes


def _exact_quant(x, fmt):
    """Values (codes x all scales) of the format's definition in 64 bits: the
    code is the count of borders passed, a tie counting where the code above
    is even."""
    R, K = x.shape
    B = _BLOCK[fmt]
    v = x.double().reshape(R, K // B, B)
    a = v.abs()
    amax = a.amax(-1, keepdim=True)
    one = torch.ones_like(amax)
    if fmt == "mx":
        e = torch.floor(torch.log2(torch.where(amax > 0, amax, one)))
        e = torch.where(torch.exp2(e) > amax, e - 1, e)
        e = torch.where(torch.exp2(e + 1) <= amax, e + 1, e)
        scale = torch.where(amax > 0, torch.exp2((e - 2).clamp(min=-127)), one)
    else:
        top = amax.amax(1, keepdim=True)
        t = torch.where(top > 0, top, torch.ones_like(top))
        e = torch.ceil(torch.log2(t / 2688.0))
        e = torch.where(2688.0 * torch.exp2(e - 1) >= t, e - 1, e)
        e = torch.where(2688.0 * torch.exp2(e) < t, e + 1, e)
        row = torch.where(top > 0, torch.exp2(e.clamp(min=-126)), torch.ones_like(top))
        grid = torch.tensor([m / 512.0 for m in range(8)]
                            + [(1 + m / 8.0) * 2.0 ** (k - 7) for k in range(1, 16) for m in range(8)][:-1],
                            dtype=torch.float64, device=x.device)
        want = (amax / (6.0 * row)).contiguous()
        hi = torch.bucketize(want, grid).clamp(max=len(grid) - 1)  # first grid value >= want
        lo = (hi - 1).clamp(min=0)
        dl, dh = want - grid[lo], grid[hi] - want
        pick = torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
        scale = grid[pick] * row
    count = torch.zeros_like(a)
    for i, mid in enumerate(_MID):
        border = mid * scale
        count += (a >= border) if (i + 1) % 2 == 0 else (a > border)
    val = torch.tensor(_E2M1, dtype=torch.float64, device=x.device)[count.long()] * scale
    return torch.where(scale > 0, torch.copysign(val, v), torch.zeros_like(val)).reshape(R, K)


def exact(case, seed):
    d, op = _inputs(case, seed), case["op"]
    if op == "quant":
        return _exact_quant(d["x"], case["fmt"])
    if op == "linear":
        return _exact_quant(d["x"], case["fmt"]) @ _exact_quant(d["W"], case["fmt"]).T
    if op == "decode":
        w = _exact_quant(d["W"], case["fmt"])
        x = d["x"].double()
        # the selection compares float32 scores
        xs, eta = d["x"].float(), None
        if case["dpts"]:
            eta = (x.sum(1) / case["K"]).float()
            xs = xs - eta[:, None]
        g = torch.sqrt(torch.sqrt((w * w).sum(0))).float() if case["score"] == "weight" else None
        sc = xs.abs() if g is None else xs.abs() * g
        keep = torch.ones_like(sc, dtype=torch.bool)
        if case["sel"] != "all":
            k = int(case["keep"] * case["K"] + 0.5) if case["sel"] == "topk" else case["n"]
            width = case["K"] if case["sel"] == "topk" else case["m"]
            b = sc.view(case["T"], -1, width)
            rank = torch.argsort(torch.argsort(-b, dim=-1, stable=True), dim=-1)
            keep = (rank < k).view_as(sc)
        y = torch.where(keep, xs.double(), 0.0) @ w.T
        return y if eta is None else y + eta.double()[:, None] * w.sum(1)
    y, r = d["y"].double(), d["r"].double()
    u = y / torch.sqrt((y ** 2).mean(1, keepdim=True) + _EPS) * d["post_w"].double()
    if d["gate"] is not None:
        u = u * d["gate"].double()
    new = _ALPHA * r + u
    h = new / torch.sqrt((new ** 2).mean(1, keepdim=True) + _EPS) * d["pre_w"].double()
    if op == "norm":
        return new, h
    return new, _exact_quant(h, case["fmt"]) @ _exact_quant(d["W"], case["fmt"]).T
