"""More of the calls that the 4-bit operators and the norm step allow: calls in a
row without a wait, non-finite values, many output tiles, the persistent norm
kernel's limits, repeated runs.  Tolerances as in test_gpu_fp4."""
import numpy as np
import pytest
import torch

import synth
from gpu_util import f32, unpack_bitmask
from oracle import fp4 as o
from test_gpu_fp4 import (Guarded, check_decode, check_norm, check_product, decode_case, dev, ok, prep,  # noqa: F401
                          quantise, random_operand, rng, sl)

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ decode
@pytest.mark.parametrize("sel", ["nm", "topk"])
@pytest.mark.parametrize("T", [1, 7, 16])
def test_decodes_in_a_row_on_one_workspace(sl, T, sel):  # noqa: F811
    """Programmatic launches: the next call's staging must not overtake the columns
    that this call still reads."""
    K, n_out, fmt = 4096, 1032, o.NV
    cfg = (sl.config(sel=sl.AS_SEL_NM, n=8, m=16, out_dtype=sl.AS_F32) if sel == "nm" else
           sl.config(sel=sl.AS_SEL_TOPK, k_keep=1500, out_dtype=sl.AS_F32))
    _, wc, wb, wS = decode_case(3, T, K, n_out, fmt, torch.bfloat16)
    Wd = prep(sl, wc, wb, wS, fmt)
    xs = [synth.random_layer(T, K, 8, seed=70 + i)[0].cuda() for i in range(8)]
    ws = torch.empty(sl.as_workspace_size(sl.AS_OP_DECODE_FP4, T, K, n_out, cfg), dtype=torch.uint8, device="cuda")
    want, got = [[torch.empty(T, n_out, device="cuda") for _ in xs] for _ in range(2)]
    for x, y in zip(xs, want):
        sl.as_linear_decode_fp4(x, Wd, cfg, y, fmt=fmt, workspace=ws)
        ok(sl)
    for _ in range(5):
        for x, y in zip(xs, got):
            sl.as_linear_decode_fp4(x, Wd, cfg, y, fmt=fmt, workspace=ws)
    ok(sl)
    assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("fmt", [o.MX, o.NV])
@pytest.mark.parametrize("bad", [np.inf, -np.inf, np.nan])
def test_decode_non_finite_x(sl, fmt, bad):  # noqa: F811
    """A kept value that is not finite makes its token's outputs NaN; a dropped one
    does nothing."""
    T, K, n_out = 4, 1024, 264
    x, wc, wb, wS = decode_case(5, T, K, n_out, fmt, torch.bfloat16)
    Wd = prep(sl, wc, wb, wS, fmt)
    x[2, 77] = bad

    def run(cfg):
        y = torch.empty(T, n_out, device="cuda")
        mask = torch.empty(T, K // 32, dtype=torch.int32, device="cuda")
        ws = torch.empty(sl.as_workspace_size(sl.AS_OP_DECODE_FP4, T, K, n_out, cfg), dtype=torch.uint8, device="cuda")
        sl.as_linear_decode_fp4(x.cuda(), Wd, cfg, y, fmt=fmt, mask_out=mask, workspace=ws,
                                g=g, rowsum=torch.zeros(n_out, device="cuda"))
        ok(sl)
        word = int(mask[2, 77 // 32].item()) & 0xFFFFFFFF
        return f32(y), bool((word >> (77 % 32)) & 1)

    g = torch.ones(K, device="cuda")
    y, _ = run(sl.config(sel=sl.AS_SEL_ALL, out_dtype=sl.AS_F32))
    assert np.isnan(y[2]).all() and np.isfinite(np.delete(y, 2, 0)).all()
    g[77] = 0.0  # an infinite |x| times 0 is NaN: whatever the selection does with it, the outputs follow the mask
    for cfg in (sl.config(sel=sl.AS_SEL_NM, n=8, m=16, out_dtype=sl.AS_F32),
                sl.config(score=sl.AS_SCORE_WEIGHT, sel=sl.AS_SEL_NM, n=8, m=16, out_dtype=sl.AS_F32),
                sl.config(sel=sl.AS_SEL_TOPK, k_keep=100, out_dtype=sl.AS_F32),
                sl.config(sel=sl.AS_SEL_THRESH, tau=0.3, out_dtype=sl.AS_F32)):
        y, kept = run(cfg)
        assert np.isnan(y[2]).all() if kept else np.isfinite(y[2]).all()
        assert np.isfinite(np.delete(y, 2, 0)).all()


@pytest.mark.parametrize("fmt", [o.MX, o.NV])
@pytest.mark.parametrize("T,K,n_out,odt", [(1, 1024, 14336, "f"), (3, 544, 20008, "b"), (16, 800, 20008, "f"),
                                           (9, 320, 38000, "b")])
def test_decode_many_output_tiles(sl, T, K, n_out, odt, fmt):  # noqa: F811
    """More tiles than clusters of the device, and than SMs."""
    g = rng(T, K, n_out, fmt)
    wc = g.integers(0, 256, (n_out, K // 2), dtype=np.uint8)
    wb = (g.integers(118, 134, (n_out, K // o.BLOCK[fmt])) if fmt == o.MX else
          g.integers(0, 100, (n_out, K // o.BLOCK[fmt]))).astype(np.uint8)
    wS = np.exp(g.standard_normal(n_out)).astype(np.float32)
    x = torch.from_numpy(g.standard_normal((T, K)).astype(np.float32)).bfloat16()
    cfg = sl.config(sel=sl.AS_SEL_NM, n=8, m=16, dpts=T % 2, out_dtype=sl.AS_BF16 if odt == "b" else sl.AS_F32)
    check_decode(sl, x, wc, wb, wS, fmt, cfg)


def decode_single_precision_blocks(seed, T, K):
    """x whose blocks of 32 hold one value 1000 times the others, and weights whose
    codes there are zero: outputs are made of the others alone."""
    g = rng(seed, T, K)
    x = g.standard_normal((T, K))
    hot = np.arange(0, K, 32) + 5
    x[:, hot] *= 1000.0
    return torch.from_numpy(x.astype(np.float32)).bfloat16(), hot


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", [o.MX, o.NV])
def test_decode_outlier_channels_that_no_weight_reads(sl, fmt, out):  # noqa: F811
    T, K, n_out = 4, 2048, 264
    x, hot = decode_single_precision_blocks(7, T, K)
    W = rng(8, n_out, K).standard_normal((n_out, K)) * 0.05
    W[:, hot] = 0.0
    wc, wb, wS = o.quant(W.astype(np.float32), fmt)
    Wd = prep(sl, wc, wb, wS.astype(np.float32), fmt)
    cfg = sl.config(sel=sl.AS_SEL_ALL, out_dtype=sl.AS_BF16 if out == torch.bfloat16 else sl.AS_F32)
    y = torch.empty(T, n_out, dtype=out, device="cuda")
    ws = torch.empty(sl.as_workspace_size(sl.AS_OP_DECODE_FP4, T, K, n_out, cfg), dtype=torch.uint8, device="cuda")
    sl.as_linear_decode_fp4(x.cuda(), Wd, cfg, y, fmt=fmt, workspace=ws)
    ok(sl)
    xf, w = x.double().numpy(), o.values(wc, wb, wS, fmt)
    ref, mag = xf @ w.T, np.abs(xf) @ np.abs(w).T
    # what the parts leave of a value: at most 2^-22 (float32: 2^-28) of its block's largest
    B = o.BLOCK[fmt]
    top = np.repeat(np.abs(xf).reshape(T, -1, B).max(-1), B, axis=1)
    left = (2.0 ** -22 if out == torch.bfloat16 else 2.0 ** -28) * (top @ np.abs(w).T)
    tol = left + (3 * K / 16 / 64 + 27) * 2.0 ** -22 * mag + (2.0 ** -8 if out == torch.bfloat16 else 0) * np.abs(ref)
    assert (np.abs(f32(y) - ref) <= tol).all()


@pytest.mark.parametrize("T,dpts", [(1, 0), (5, 1), (16, 1)])
def test_decode_then_rsparse(sl, T, dpts):  # noqa: F811
    """The compensation of the dropped channels behind a 4-bit decode, by the call's
    own mask and means, without a wait between the two."""
    K, n_out, r = 1056, 264, 64
    x, wc, wb, wS = decode_case(11, T, K, n_out, o.NV, torch.bfloat16)
    g = rng(12, T)
    B = torch.from_numpy(g.standard_normal((K, r)).astype(np.float32) * 0.1).bfloat16()
    A = torch.from_numpy(g.standard_normal((n_out, r)).astype(np.float32) * 0.1).bfloat16()
    w = o.values(wc, wb, wS, o.NV)
    rowsum = w.sum(1).astype(np.float32)
    Wd = prep(sl, wc, wb, wS, o.NV)
    cfg = sl.config(sel=sl.AS_SEL_NM, n=8, m=16, dpts=dpts, out_dtype=sl.AS_F32)
    ws = torch.empty(sl.as_workspace_size(sl.AS_OP_DECODE_FP4, T, K, n_out, cfg), dtype=torch.uint8, device="cuda")
    wr = torch.empty(sl.as_rsparse_workspace(T, K, r), dtype=torch.uint8, device="cuda")
    xd, Bd, Ad, rs = x.cuda(), B.cuda(), A.cuda(), dev(rowsum)
    outs = []
    for _ in range(4):
        y = torch.empty(T, n_out, device="cuda")
        mask = torch.zeros(T, K // 32, dtype=torch.int32, device="cuda")
        eta = torch.zeros(T, device="cuda")
        sl.as_linear_decode_fp4(xd, Wd, cfg, y, fmt=o.NV, rowsum=rs, mask_out=mask, eta_out=eta, workspace=ws)
        sl.as_rsparse_decode(xd, mask, Bd, Ad, y, eta=eta if dpts else None, workspace=wr)
        outs.append((y, mask, eta))
    ok(sl)
    y, mask, eta = outs[0]
    assert all(torch.equal(y, other[0]) for other in outs)
    xf = x.float().numpy()
    m = unpack_bitmask(mask, K)
    e = f32(eta)[:, None] if dpts else np.zeros((T, 1), np.float32)
    xh = (xf - e).astype(np.float32).astype(np.float64)
    Bf, Af = B.double().numpy(), A.double().numpy()
    ref = (xh * m) @ w.T + e.astype(np.float64) * rowsum + ((xh * (m == 0)) @ Bf) @ Af.T
    mag = np.abs(xh) @ np.abs(w).T + np.abs(e * rowsum) + (np.abs(xh) @ np.abs(Bf)) @ np.abs(Af).T
    # the decode's bound, and sums of up to 16 + K / 128 + r float32 steps in the two factors' products
    assert (np.abs(f32(y) - ref) <= ((3 * K / 16 / 64 + 27) + 16 + K / 128 + r) * 2.0 ** -22 * mag).all()


# ------------------------------------------------------------------ product
@pytest.mark.parametrize("fmt", [o.MX, o.NV])
@pytest.mark.parametrize("T,K,n_out", [(1, 288, 20008), (30, 544, 20008), (64, 1056, 38000)])
def test_few_tokens_many_tiles(sl, T, K, n_out, fmt):  # noqa: F811
    check_product(sl, T, K, n_out, fmt, torch.float32 if T % 2 else torch.bfloat16)


@pytest.mark.parametrize("fmt", [o.MX, o.NV])
@pytest.mark.parametrize("T", [3, 200, 1300])
def test_quantise_and_multiply_non_finite_rows(sl, T, fmt):  # noqa: F811
    """The quantiser's form of a non-finite block (zero codes, NaN scale) through
    the three product kernels: NaN in its row (of x) or column (of W) only."""
    K, n_out = 416, 2056
    g = rng(T, fmt)
    x = torch.from_numpy(g.standard_normal((T, K)).astype(np.float32))
    W = torch.from_numpy(g.standard_normal((n_out, K)).astype(np.float32))
    x[1, 40], W[9, 415] = np.inf, np.nan
    xq, xsf, xS = quantise(sl, x, fmt)
    wq, wsf, wS = quantise(sl, W, fmt)
    y = Guarded(T, n_out, dtype=torch.float32)
    sl.as_linear_prefill_fp4(xq, xsf, wq, wsf, y.t, x_scale=xS, w_scale=wS, fmt=fmt)
    ok(sl)
    y.check()
    want = np.zeros((T, n_out), bool)
    want[1], want[:, 9] = True, True
    np.testing.assert_array_equal(np.isnan(f32(y.t)), want)


@pytest.mark.parametrize("T", [3, 200, 1300])
@pytest.mark.parametrize("xb,wb", [(0, 254), (254, 0), (1, 253), (0, 120), (50, 57), (254, 100)])
def test_product_extreme_mx_scales(sl, T, xb, wb):  # noqa: F811
    """E8M0 scales of 2^-127 and 2^127, sums among the subnormal numbers: the
    products of 64 channels are whole multiples of 2^(xb + wb - 256), at most 2^14
    of them, and exact."""
    K, n_out = 64, 2056
    xc, xbytes, _, _ = random_operand(31, T, K, o.MX, False)
    wc, wbytes, _, _ = random_operand(32, n_out, K, o.MX, False)
    xbytes[:], wbytes[:] = xb, wb
    y = torch.empty(T, n_out, device="cuda")
    sl.as_linear_prefill_fp4(dev(xc), dev(o.tile_scales(xbytes, o.MX)), dev(wc), dev(o.tile_scales(wbytes, o.MX)), y,
                             fmt=o.MX)
    ok(sl)
    np.testing.assert_array_equal(f32(y), o.values(xc, xbytes, None, o.MX) @ o.values(wc, wbytes, None, o.MX).T)


# ------------------------------------------------------------------ norm
@pytest.mark.parametrize("T", [296, 300, 443, 445])
@pytest.mark.parametrize("D,types,gate,fmt", [(2080, "fbf", "token", o.NV), (4096, "bbb", "channel", None),
                                              (4128, "fff", "none", o.MX), (8192, "ffb", "token", None)])
def test_norm_few_rows_per_sm(sl, T, D, types, gate, fmt):  # noqa: F811
    """Around the row count from which the persistent kernel runs; some of its CTAs
    have no row."""
    check_norm(sl, T, D, *types, gate=gate, fmt=fmt)


@pytest.mark.parametrize("D", [8200, 16392])
def test_norm_many_long_rows(sl, D):  # noqa: F811
    check_norm(sl, 300, D, "f", "b", "b", "token")


@pytest.mark.parametrize("fmt", [o.MX, o.NV])
@pytest.mark.parametrize("T,D", [(3, 4096), (300, 4096), (300, 8192), (443, 2080)])
def test_norm_parts_of_the_outputs(sl, T, D, fmt):  # noqa: F811
    """r' alone, the 4-bit operand alone: the bits of the call that writes all."""
    g = torch.Generator(device="cuda").manual_seed(T + D)
    r = torch.randn(T, D, generator=g, device="cuda")
    y = torch.randn(T, D, generator=g, device="cuda").bfloat16()
    gate = torch.randn(D, generator=g, device="cuda")
    pre = torch.randn(D, generator=g, device="cuda")

    def outputs():
        return dict(r_out=Guarded(T, D, dtype=torch.float32), h=Guarded(T, D, dtype=torch.float32),
                    h_q=Guarded(T, D // 2, dtype=torch.uint8),
                    h_sf=Guarded(sl.as_fp4_sf_bytes(T, D, fmt), dtype=torch.uint8), h_scale=Guarded(T, dtype=torch.float32))

    def run(names):
        b = outputs()
        sl.as_norm_residual(r, y=y, gate=gate, pre_w=pre, post_norm=True, res_scale=0.5, fmt=fmt,
                            **{n: b[n].t for n in names})
        ok(sl)
        for v in b.values():
            v.check()
        return {n: b[n].t for n in names}

    whole = run(["r_out", "h", "h_q", "h_sf", "h_scale"])
    for names in (["r_out"], ["h"], ["h_q", "h_sf", "h_scale"], ["r_out", "h_q", "h_sf", "h_scale"]):
        for n, v in run(names).items():
            assert torch.equal(v, whole[n]), n
    codes, byte, S = o.quant(f32(whole["h"]), fmt)
    np.testing.assert_array_equal(whole["h_q"].cpu().numpy(), codes)
    np.testing.assert_array_equal(whole["h_sf"].cpu().numpy(), o.tile_scales(byte, fmt))
    np.testing.assert_array_equal(f32(whole["h_scale"]), S)


@pytest.mark.parametrize("fmt", [o.MX, o.NV])
@pytest.mark.parametrize("T,D", [(5, 1024), (300, 4096)])
def test_norm_non_finite(sl, T, D, fmt):  # noqa: F811
    """A NaN makes its row NaN.  An infinity in r makes r' infinite there and h zero
    elsewhere (1 / inf) and NaN there; in y, under the post norm, r' = r elsewhere.
    The codes are those of that h: NaN scale for its block, zeros for the rest."""
    g = rng(T, D)
    r, y = g.standard_normal((T, D)).astype(np.float32), g.standard_normal((T, D)).astype(np.float32)
    r[0, 3], r[1, 40], y[2, 7], y[3, 9] = np.nan, np.inf, np.nan, -np.inf
    t = lambda v: torch.from_numpy(v).cuda()  # noqa: E731
    R, H = Guarded(T, D, dtype=torch.float32), Guarded(T, D, dtype=torch.float32)
    q, sf = Guarded(T, D // 2, dtype=torch.uint8), Guarded(sl.as_fp4_sf_bytes(T, D, fmt), dtype=torch.uint8)
    S = Guarded(T, dtype=torch.float32)
    sl.as_norm_residual(t(r), y=t(y), r_out=R.t, h=H.t, post_norm=True, h_q=q.t, h_sf=sf.t, h_scale=S.t, fmt=fmt)
    ok(sl)
    for b in (R, H, q, sf, S):
        b.check()
    with np.errstate(invalid="ignore"):
        r64, h64 = o.norm_residual(r, y, True)
    # the float64 formula sees the same infinities (inf / inf, inf * 0 are NaN, finite / inf is 0)
    np.testing.assert_array_equal(np.isnan(f32(R.t)), np.isnan(r64))
    np.testing.assert_array_equal(np.isinf(f32(R.t)), np.isinf(r64))
    np.testing.assert_array_equal(np.isnan(f32(H.t)), np.isnan(h64))
    np.testing.assert_allclose(f32(H.t), h64, rtol=1e-5, atol=1e-5)
    codes, byte, rs = o.quant(f32(H.t), fmt)
    np.testing.assert_array_equal(q.t.cpu().numpy(), codes)
    np.testing.assert_array_equal(sf.t.cpu().numpy(), o.tile_scales(byte, fmt))
    np.testing.assert_array_equal(f32(S.t), rs)


# ------------------------------------------------------------------ repeats
def test_repeated_runs_give_the_same_bits(sl):  # noqa: F811
    """A full decode batch, a long prompt's norm step and the norm step into the
    product: the sums' orders are fixed."""
    g = torch.Generator(device="cuda").manual_seed(1)
    T, K, n_out, fmt = 16, 14336, 4096, sl.AS_FP4_MX
    W = torch.randn(n_out, K, generator=g, device="cuda") * 0.02
    q, sf, S = quantise(sl, W.cpu(), fmt)
    Wd = torch.empty(sl.as_fp4_decode_bytes(n_out, K, fmt), dtype=torch.uint8, device="cuda")
    sl.as_weight_prep_fp4(q, sf, Wd, w_scale=S, fmt=fmt)
    cfg = sl.config(sel=sl.AS_SEL_NM, n=8, m=16)
    x = torch.randn(T, K, generator=g, device="cuda").bfloat16()
    ws = torch.empty(sl.as_workspace_size(sl.AS_OP_DECODE_FP4, T, K, n_out, cfg), dtype=torch.uint8, device="cuda")
    ys = [torch.empty(T, n_out, dtype=torch.bfloat16, device="cuda") for _ in range(20)]
    for y in ys:
        sl.as_linear_decode_fp4(x, Wd, cfg, y, fmt=fmt, workspace=ws)
    ok(sl)
    assert all(torch.equal(y, ys[0]) for y in ys)

    T, D = 8192, 8192
    r = torch.randn(T, D, generator=g, device="cuda")
    y = torch.randn(T, D, generator=g, device="cuda").bfloat16()
    gate = torch.randn(T, D, generator=g, device="cuda")
    first = None
    for _ in range(4):
        out, h = torch.empty_like(r), torch.empty(T, D, dtype=torch.bfloat16, device="cuda")
        sl.as_norm_residual(r, y=y, r_out=out, h=h, gate=gate, post_norm=True)
        first = first or (out, h)
        assert torch.equal(out, first[0]) and torch.equal(h, first[1])
    del out, h, first, gate

    T, D, n_out, fmt = 1000, 4096, 4096, sl.AS_FP4_NV
    wq, wsf, wS = quantise(sl, W[:, :D].contiguous().cpu(), fmt)
    r, y = r[:T, :D].contiguous(), y[:T, :D].contiguous()
    hq, hsf = torch.empty(T, D // 2, dtype=torch.uint8, device="cuda"), torch.empty(
        sl.as_fp4_sf_bytes(T, D, fmt), dtype=torch.uint8, device="cuda")
    hs = torch.empty(T, device="cuda")
    ps = [torch.empty(T, n_out, dtype=torch.bfloat16, device="cuda") for _ in range(6)]
    for p in ps:
        sl.as_norm_residual(r, y=y, post_norm=True, h_q=hq, h_sf=hsf, h_scale=hs, fmt=fmt)
        sl.as_linear_prefill_fp4(hq, hsf, wq, wsf, p, x_scale=hs, w_scale=wS, fmt=fmt)
    ok(sl)
    assert all(torch.equal(p, ps[0]) for p in ps)


# ------------------------------------------------------------------ first calls
FIRST_CALLS = """
import sys
sys.path.insert(0, {root!r})
import torch
import sparse_linear_b200 as sl
from sparse_linear_b200.layer import Fp4Linear, SparseLinear
g = torch.Generator(device="cuda").manual_seed(0)
W = torch.randn(1032, 2048, generator=g, device="cuda") * 0.02
x = torch.randn(300, 2048, generator=g, device="cuda").bfloat16()
r = torch.randn(600, 4096, generator=g, device="cuda")
y = torch.randn(600, 4096, generator=g, device="cuda")
cfg = sl.config(score=sl.AS_SCORE_CLACT, sel=sl.AS_SEL_NM, n=8, m=16, out_dtype=sl.AS_F32)
L, S = Fp4Linear(W, cfg), SparseLinear(W.bfloat16(), cfg)


def calls():
    h, o = torch.empty_like(r), torch.empty_like(r)
    sl.as_norm_residual(r, y=y, r_out=o, h=h, post_norm=True)
    return [L.decode(x[:1]), L.decode(x[:16]), L.prefill(x[:20]), L.prefill(x), S.decode(x[:2]), S.prefill(x)[0], h, o]


torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    captured = calls()
eager = calls()  # before the graph has run
torch.cuda.synchronize()
for _ in range(2):
    graph.replay()
    torch.cuda.synchronize()
    assert sl.as_stream_status() == sl.AS_OK
    for i, (a, b) in enumerate(zip(captured, eager)):
        assert torch.equal(a, b), i
"""


def test_first_calls_of_a_process_are_captured():
    """A graph captured by a process that has called nothing before, then the same
    calls outside it, then its replays."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", FIRST_CALLS.format(root=root)], capture_output=True, text=True,
                         timeout=300)
    assert out.returncode == 0, out.stdout + out.stderr


@pytest.mark.parametrize("fmt", [o.MX, o.NV])
def test_decode_longest_rows(sl, fmt):  # noqa: F811
    x, *w = decode_case(9, 2, 131072, 136, fmt, torch.bfloat16)
    check_decode(sl, x, *w, fmt, sl.config(sel=sl.AS_SEL_NM, n=8, m=16, dpts=True, out_dtype=sl.AS_F32))
