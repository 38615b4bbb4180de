"""Microscaled 4-bit operators and the norm/residual step on a B200, against
the float64 oracle.

Codes, scale bytes and row scales are compared bit for bit: they are defined
by real arithmetic.  Products and sums are held to bounds of float32
arithmetic: every step of an accumulation errs by at most 2^-22 of the sum of
magnitudes (one float32 step, doubled for sums that truncate), and the output
is rounded once, by at most eps/2 of the value.
"""
import numpy as np
import pytest
import torch

import oracle
import synth
from gpu_util import f32, unpack_bitmask
from oracle import fp4 as o

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}  # eps / 2
SENTINEL = {torch.uint8: 0xA5, torch.float32: 123.25, torch.bfloat16: 123.0, torch.int32: -559038737}


@pytest.fixture(scope="module")
def sl():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import sparse_linear_b200 as m
    return m


class Guarded:
    """A buffer with 256 elements of a known value behind it."""

    def __init__(self, *shape, dtype):
        n = int(np.prod(shape))
        self.flat = torch.full((n + 256,), SENTINEL[dtype], dtype=dtype, device="cuda")
        self.t = self.flat[:n].view(*shape)

    def check(self):
        assert (self.flat[self.t.numel():] == SENTINEL[self.flat.dtype]).all(), "write past the end"


def rng(*seed):
    return np.random.default_rng(list(seed))


def rows(seed, R, K, dtype):
    """Rows with outliers, zero blocks, one zero row and widely spread rows."""
    g = rng(seed, R, K)
    x = g.laplace(0, 0.3, (R, K)) * np.where(g.random(K) < 0.02, 20.0, 1.0)
    x *= np.exp2(g.integers(-12, 12, (R, 1)))
    x.reshape(R, -1, 16)[g.random((R, K // 16)) < 0.1] = 0.0
    if R > 2:
        x[R // 2] = 0.0
    return torch.from_numpy(x.astype(np.float32)).to(dtype)


def quantise(sl, x, fmt):
    R, K = x.shape
    q = Guarded(R, K // 2, dtype=torch.uint8)
    sf = Guarded(sl.as_fp4_sf_bytes(R, K, fmt), dtype=torch.uint8)
    sc = Guarded(R, dtype=torch.float32)
    sl.as_quant_fp4(x.cuda(), q.t, sf.t, sc.t, fmt=fmt)
    torch.cuda.synchronize()
    for b in (q, sf, sc):
        b.check()
    return q.t, sf.t, sc.t


def ok(sl):
    torch.cuda.synchronize()
    assert sl.as_stream_status() == sl.AS_OK


def check_quant(sl, x, fmt):
    q, sf, sc = quantise(sl, x, fmt)
    codes, byte, S = o.quant(x.float().numpy(), fmt)
    np.testing.assert_array_equal(f32(sc), S)
    np.testing.assert_array_equal(sf.cpu().numpy(), o.tile_scales(byte, fmt))
    np.testing.assert_array_equal(q.cpu().numpy(), codes)
    v = o.values(codes, byte, S, fmt)
    for dt in (torch.float32, torch.bfloat16):
        out = Guarded(*x.shape, dtype=dt)
        sl.as_dequant_fp4(q, sf, out.t, sc, fmt=fmt)
        ok(sl)
        out.check()
        want = torch.from_numpy(v).float().to(dt)  # exact in float32
        assert torch.equal(torch.nan_to_num(out.t.cpu(), 7.0), torch.nan_to_num(want, 7.0))


# ------------------------------------------------------------------ quantiser
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", [o.MX, o.NV])
@pytest.mark.parametrize("R,K", [(1, 32), (1, 4096), (3, 96), (31, 64), (33, 160), (127, 32), (128, 256), (129, 288),
                                 (300, 2080), (5, 20000), (2, 14368)])
def test_quant(sl, R, K, fmt, dtype):
    check_quant(sl, rows(1, R, K, dtype), fmt)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", [o.MX, o.NV])
def test_quant_borders(sl, fmt, dtype):
    """Values on, just under and just over every border between codes, for
    every E4M3 mantissa as the block scale, and the same for the scales' own
    borders."""
    step = 2.0 ** -7 if dtype == torch.bfloat16 else 2.0 ** -23
    border = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    x = np.zeros((16, 256))
    x[:, 0] = 2688.0
    for r in range(16):
        s = (1 + (r % 8) / 8) * 2.0 ** (r // 8 * 3 - 3)  # the block scale wanted
        b = x[r].reshape(-1, 16)
        for k in range(1, 16):
            b[k, 0] = 6 * s
            t = np.tile(border * s, 3)[:15]
            b[k, 1:] = (t * np.repeat([1.0, 1.0 - step, 1.0 + step], 7)[:15]) * (-1.0) ** k
            b[k, 8:] = (border * s * (1 + step if k % 2 else 1 - step))[np.arange(8) % 7]
    check_quant(sl, torch.from_numpy(x.astype(np.float32)).to(dtype), fmt)
    # block maxima around 6 * S * every border of the E4M3 grid
    mid = 6 * (o.E4M3[:-1] + o.E4M3[1:]) / 2
    y = np.zeros((3, 128, 16))
    for i, f in enumerate((1.0, 1 - step, 1 + step)):
        y[i, :126, 3] = mid * f
        y[i, 127, 0] = 2688.0
    check_quant(sl, torch.from_numpy(y.reshape(3, -1).astype(np.float32)).to(dtype), fmt)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", [o.MX, o.NV])
def test_quant_extremes(sl, fmt, dtype):
    big, tiny = float(torch.finfo(dtype).max), 2.0 ** -126
    x = np.zeros((12, 64))
    x[0, ::3], x[1, ::3] = big, -big
    x[2, ::5], x[3, :] = tiny, 2.0 ** -133
    x[4, 0], x[4, 32:] = big, 1.0
    x[5, :] = np.where(np.arange(64) % 2, 1.0, -0.0)
    x[6, 7], x[7, 40], x[8, 3], x[8, 50] = np.inf, np.nan, -np.inf, np.nan
    x[9, :], x[10, 0], x[11, 63] = 1.3125 * 2048, 1.3125 * 2048 * (1 + 2.0 ** -7), 3.0
    x[6, 32:], x[7, :32] = 2.0, -2.0
    check_quant(sl, torch.from_numpy(x).to(torch.float32).to(dtype), fmt)


# ------------------------------------------------------------------ product
def random_operand(seed, R, K, fmt, row_scale=True):
    """Codes, tiled scales and row scales drawn directly (every code and many
    scales), with the values they stand for."""
    g = rng(seed, R, K, fmt)
    codes = g.integers(0, 256, (R, K // 2), dtype=np.uint8)
    nb = K // o.BLOCK[fmt]
    byte = (g.integers(118, 134, (R, nb)) if fmt == o.MX else g.integers(0, 100, (R, nb))).astype(np.uint8)
    S = np.exp(g.standard_normal(R)).astype(np.float32) if row_scale else None
    v = o.values(codes, byte, None, fmt)
    return codes, byte, S, v


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def check_product(sl, T, K, n_out, fmt, dtype, scales=True):
    xc, xb, xS, xv = random_operand(11, T, K, fmt, scales)
    wc, wb, wS, wv = random_operand(12, n_out, K, fmt, scales)
    y = Guarded(T, n_out, dtype=dtype)
    sl.as_linear_prefill_fp4(dev(xc), dev(o.tile_scales(xb, fmt)), dev(wc), dev(o.tile_scales(wb, fmt)), y.t,
                             x_scale=dev(xS), w_scale=dev(wS), fmt=fmt)
    ok(sl)
    y.check()
    s = 1.0 if not scales else xS.astype(np.float64)[:, None] * wS.astype(np.float64)[None, :]
    ref, mag = (xv @ wv.T) * s, (np.abs(xv) @ np.abs(wv).T) * s
    # one step per instruction of 64 channels, eight CTAs' sums, two row scales
    tol = (K / 64 + 12) * 2.0 ** -22 * mag + HALF[dtype] * np.abs(ref)
    err = np.abs(f32(y.t).astype(np.float64) - ref)
    assert (err <= tol).all(), (float((err / np.maximum(tol, 1e-300)).max()), np.argwhere(err > tol)[:4])


PRODUCT = [(1, 32, 8), (1, 4096, 1024), (2, 64, 136), (16, 96, 128), (17, 256, 120), (33, 288, 520), (64, 2048, 264),
           (65, 1056, 136), (128, 64, 128), (129, 4128, 136), (256, 544, 256), (257, 32, 264), (300, 4096, 520),
           (513, 992, 248), (40, 14336, 128), (1, 131072, 8)]


@pytest.mark.parametrize("fmt", [o.MX, o.NV])
@pytest.mark.parametrize("T,K,n_out", PRODUCT)
def test_product(sl, T, K, n_out, fmt):
    check_product(sl, T, K, n_out, fmt, torch.float32)


@pytest.mark.parametrize("T,K,n_out,fmt", [(5, 512, 264, o.MX), (700, 512, 264, o.NV), (260, 1312, 72, o.MX)])
def test_product_bf16_no_row_scales(sl, T, K, n_out, fmt):
    check_product(sl, T, K, n_out, fmt, torch.bfloat16, scales=False)


@pytest.mark.parametrize("fmt", [o.MX, o.NV])
@pytest.mark.parametrize("T", [3, 300])
def test_product_nan_scale_stays_in_its_row(sl, T, fmt):
    K, n_out = 320, 136
    xc, xb, _, xv = random_operand(5, T, K, fmt, False)
    wc, wb, _, wv = random_operand(6, n_out, K, fmt, False)
    xb[1, 2], wb[7, 1] = (255, 255) if fmt == o.MX else (127, 127)
    y = torch.empty(T, n_out, device="cuda")
    sl.as_linear_prefill_fp4(dev(xc), dev(o.tile_scales(xb, fmt)), dev(wc), dev(o.tile_scales(wb, fmt)), y, fmt=fmt)
    ok(sl)
    nan = torch.isnan(y).cpu().numpy()
    want = np.zeros((T, n_out), bool)
    want[1], want[:, 7] = True, True
    np.testing.assert_array_equal(nan, want)


# more than one wave of 128 x 128 tiles: CTA pairs, ragged on every side, one
# and several tiles per pair, K from half a stage to more than the ring
PAIRS = [(1300, 416, 1960), (200, 1312, 9992), (2500, 32, 1032), (777, 2080, 4104), (257, 4128, 8200),
         (3000, 256, 3208)]


@pytest.mark.parametrize("fmt", [o.MX, o.NV])
@pytest.mark.parametrize("T,K,n_out", PAIRS)
def test_product_pairs(sl, T, K, n_out, fmt):
    check_product(sl, T, K, n_out, fmt, torch.float32 if T % 2 else torch.bfloat16)


@pytest.mark.parametrize("T,K,n_out,fmt", [
    (1024, 4096, 128, o.NV), (1000, 544, 1032, o.MX), (1111, 1056, 1024, o.NV), (384, 2048, 768, o.MX),
    (260, 800, 4096, o.NV)])
def test_product_one_wave(sl, T, K, n_out, fmt):
    """128 x 128 tiles at many tokens, clusters of 8 down to 1."""
    check_product(sl, T, K, n_out, fmt, torch.float32)
    check_product(sl, T, K, n_out, fmt, torch.bfloat16, scales=False)


def test_product_pairs_nan_and_deterministic(sl):
    T, K, n_out, fmt = 1300, 320, 2056, o.NV
    xc, xb, xS, _ = random_operand(5, T, K, fmt)
    wc, wb, wS, _ = random_operand(6, n_out, K, fmt)
    xb[1, 2], wb[7, 1] = 127, 127
    ys = []
    for _ in range(2):
        y = torch.empty(T, n_out, device="cuda")
        sl.as_linear_prefill_fp4(dev(xc), dev(o.tile_scales(xb, fmt)), dev(wc), dev(o.tile_scales(wb, fmt)), y,
                                 x_scale=dev(xS), w_scale=dev(wS), fmt=fmt)
        ys.append(y)
    ok(sl)
    want = torch.zeros(T, n_out, dtype=torch.bool)
    want[1], want[:, 7] = True, True
    assert torch.equal(torch.isnan(ys[0]).cpu(), want)
    assert torch.equal(ys[0].nan_to_num(1e30), ys[1].nan_to_num(1e30))


@pytest.mark.parametrize("T", [1, 40, 777])
def test_product_deterministic(sl, T):
    K, n_out, fmt = 2048, 512, o.NV
    xc, xb, xS, _ = random_operand(1, T, K, fmt)
    wc, wb, wS, _ = random_operand(2, n_out, K, fmt)
    args = (dev(xc), dev(o.tile_scales(xb, fmt)), dev(wc), dev(o.tile_scales(wb, fmt)))
    ys = []
    for _ in range(3):
        y = torch.empty(T, n_out, device="cuda")
        sl.as_linear_prefill_fp4(*args, y, x_scale=dev(xS), w_scale=dev(wS), fmt=fmt)
        ys.append(y)
    ok(sl)
    assert torch.equal(ys[0], ys[1]) and torch.equal(ys[0], ys[2])


# ------------------------------------------------------------------ decode
def prep(sl, wc, wb, wS, fmt):
    n_out, K = wc.shape[0], 2 * wc.shape[1]
    Wd = Guarded(sl.as_fp4_decode_bytes(n_out, K, fmt), dtype=torch.uint8)
    sl.as_weight_prep_fp4(dev(wc), dev(o.tile_scales(wb, fmt)), Wd.t, w_scale=dev(wS), fmt=fmt)
    ok(sl)
    Wd.check()
    return Wd.t


def check_decode(sl, x, wc, wb, wS, fmt, cfg, wd=None, eta_static=None):
    T, K = x.shape
    n_out = wc.shape[0]
    w = o.values(wc, wb, wS, fmt)
    g = np.sqrt(np.sqrt((w * w).sum(0))).astype(np.float32)
    rowsum = w.sum(1).astype(np.float32)
    Wd = prep(sl, wc, wb, wS, fmt) if wd is None else wd
    dt = torch.bfloat16 if cfg.out_dtype == sl.AS_BF16 else torch.float32
    y = Guarded(T, n_out, dtype=dt)
    mask = Guarded(T, (K + 31) // 32, dtype=torch.int32)
    eta, col = Guarded(T, dtype=torch.float32), Guarded(K, dtype=torch.float32)
    ws = torch.full((sl.as_workspace_size(sl.AS_OP_DECODE_FP4, T, K, n_out, cfg),), 0xEE, dtype=torch.uint8,
                    device="cuda")
    kw = dict(fmt=fmt, g=dev(g), rowsum=dev(rowsum), workspace=ws)
    sl.as_linear_decode_fp4(x.cuda(), Wd, cfg, y.t, mask_out=mask.t, eta_out=eta.t, colnorm_out=col.t, **kw)
    ok(sl)
    for b in (y, mask, eta, col):
        b.check()
    y2 = torch.empty_like(y.t)
    sl.as_linear_decode_fp4(x.cuda(), Wd, cfg, y2, **kw)  # nothing reported: same result
    ok(sl)
    assert torch.equal(torch.nan_to_num(y.t, 7.0), torch.nan_to_num(y2, 7.0))

    xf = x.float().numpy()
    e = f32(eta.t) if cfg.dpts else None
    if cfg.dpts == sl.AS_PTS_DYNAMIC:
        np.testing.assert_allclose(e, oracle.token_mean(xf), atol=1e-6 * np.abs(xf).mean(), rtol=1e-6)
    f = {sl.AS_SCORE_MAG: None, sl.AS_SCORE_WEIGHT: g, sl.AS_SCORE_CLACT: f32(col.t)}[cfg.score]
    s = oracle.score(xf, eta=e, f=f)
    if cfg.sel == sl.AS_SEL_NM:
        m = oracle.select_nm(s, cfg.n, cfg.m)
    elif cfg.sel == sl.AS_SEL_TOPK:
        m = oracle.select_topk(s, cfg.k_keep)
    elif cfg.sel == sl.AS_SEL_THRESH:
        m = oracle.select_thresh(s, cfg.tau)
    else:
        m = np.ones_like(xf, np.uint8)
    np.testing.assert_array_equal(unpack_bitmask(mask.t, K), m)
    xh = (xf if e is None else (xf - e[:, None]).astype(np.float32)).astype(np.float64) * (m != 0)
    ref, mag = xh @ w.T, np.abs(xh) @ np.abs(w).T
    if e is not None:
        ref = ref + e.astype(np.float64)[:, None] * rowsum.astype(np.float64)
        mag = mag + np.abs(e.astype(np.float64)[:, None] * rowsum)
    # float32 sums: a step per 16 channels and part, the parts, eight CTAs,
    # factor and shift.  A bf16 output takes x in 7 four-bit parts, which leave
    # at most 6^-7 / 3 = 2^-19.6 of a block's largest value; kept values are
    # more than a fifth of it on average, which makes at most 2^-17 of mag.
    # (float32: 10 parts, 6^-10 / 3 = 2^-27.4, inside the first term.)
    tol = ((3 * K / 16 / 64 + 24 + 3) * 2.0 ** -22 + (2.0 ** -17 if dt == torch.bfloat16 else 0)) * mag
    tol = tol + HALF[dt] * np.abs(ref)
    err = np.abs(f32(y.t).astype(np.float64) - ref)
    assert (err <= tol).all(), (float((err / np.maximum(tol, 1e-300)).max()), np.argwhere(err > tol)[:4])
    return y.t


def decode_case(seed, T, K, n_out, fmt, dtype, ties=0):
    x, W = synth.random_layer(T, K, n_out, seed=seed, dtype=torch.float32, ties=ties)
    wc, wb, wS = o.quant(W.numpy(), fmt)
    return x.to(dtype), wc, wb, wS.astype(np.float32)


@pytest.mark.parametrize("fmt", [o.MX, o.NV])
@pytest.mark.parametrize("T,K,n_out,n,m,score,dpts,xdt,odt", [
    (1, 32, 8, 2, 4, 0, 0, "b", "f"), (1, 4096, 520, 8, 16, 1, 1, "b", "b"), (2, 1056, 136, 16, 32, 2, 0, "b", "f"),
    (3, 2080, 264, 8, 16, 1, 1, "f", "f"), (8, 96, 128, 1, 2, 0, 1, "b", "b"), (9, 1056, 136, 2, 4, 2, 1, "b", "f"),
    (16, 4128, 392, 8, 16, 0, 0, "b", "b"), (16, 2048, 136, 4, 8, 1, 1, "f", "b"), (5, 8224, 72, 8, 16, 0, 0, "f", "f"),
    (13, 20000, 136, 16, 32, 1, 1, "b", "f"), (1, 20000, 8, 1, 16, 0, 0, "b", "b"), (4, 1024, 2056, 1, 1, 0, 0, "b", "f"),
])
def test_decode_nm(sl, T, K, n_out, n, m, score, dpts, xdt, odt, fmt):
    x, *w = decode_case(T * 1000 + K, T, K, n_out, fmt, torch.bfloat16 if xdt == "b" else torch.float32, ties=T % 3)
    cfg = sl.config(score=score, sel=sl.AS_SEL_NM, n=n, m=m, dpts=dpts,
                    out_dtype=sl.AS_BF16 if odt == "b" else sl.AS_F32)
    check_decode(sl, x, *w, fmt, cfg)


@pytest.mark.parametrize("fmt", [o.MX, o.NV])
@pytest.mark.parametrize("T,kk,dpts", [(1, 0, 0), (3, 0, 1), (3, 1, 1), (2, 500, 0), (16, 1023, 1), (5, 1024, 0)])
def test_decode_topk(sl, T, kk, dpts, fmt):
    x, *w = decode_case(kk + T, T, 1024, 264, fmt, torch.bfloat16, ties=2)
    cfg = sl.config(sel=sl.AS_SEL_TOPK, k_keep=kk, dpts=dpts, out_dtype=sl.AS_F32)
    y = check_decode(sl, x, *w, fmt, cfg)
    if kk == 0 and not dpts:
        assert not y.any()


@pytest.mark.parametrize("T,K,n_out,dpts,xdt", [(1, 64, 8, 0, "b"), (4, 2080, 136, 0, "f"), (16, 1024, 136, 1, "b"),
                                                (16, 4096, 1032, 0, "b")])
def test_decode_all_and_threshold(sl, T, K, n_out, dpts, xdt):
    x, *w = decode_case(T, T, K, n_out, o.NV, torch.bfloat16 if xdt == "b" else torch.float32)
    check_decode(sl, x, *w, o.NV, sl.config(sel=sl.AS_SEL_ALL, dpts=dpts, out_dtype=sl.AS_F32))
    check_decode(sl, x, *w, o.NV, sl.config(sel=sl.AS_SEL_THRESH, tau=0.3, dpts=dpts, out_dtype=sl.AS_BF16))
    check_decode(sl, x, *w, o.NV, sl.config(sel=sl.AS_SEL_THRESH, tau=1e30, dpts=dpts, out_dtype=sl.AS_F32))
    eta = torch.linspace(-0.2, 0.3, T).cuda()
    check_decode(sl, x, *w, o.NV, sl.config(sel=sl.AS_SEL_NM, n=8, m=16, dpts=sl.AS_PTS_STATIC, eta_static=eta,
                                            out_dtype=sl.AS_F32))


@pytest.mark.parametrize("fmt", [o.MX, o.NV])
def test_decode_every_code_and_scale(sl, fmt):
    """Weights drawn as codes and scale bytes: every E4M3 scale with its
    subnormals and zero, E8M0 scales over 60 binades, row scales apart."""
    K, n_out = 1024, 264
    g = rng(77, fmt)
    wc = g.integers(0, 256, (n_out, K // 2), dtype=np.uint8)
    wb = (g.integers(0, 127, (n_out, K // 16)) if fmt == o.NV else
          g.integers(97, 157, (n_out, 1)) - g.integers(0, 40, (n_out, K // 32))).astype(np.uint8)
    wS = np.exp(g.standard_normal(n_out)).astype(np.float32)
    x = torch.from_numpy(g.standard_normal((3, K)).astype(np.float32)).bfloat16()
    check_decode(sl, x, wc, wb, wS, fmt, sl.config(sel=sl.AS_SEL_NM, n=8, m=16, out_dtype=sl.AS_F32))


@pytest.mark.parametrize("fmt", [o.MX, o.NV])
def test_decode_extreme_scales_and_nan(sl, fmt):
    K, n_out = 256, 136
    g = rng(78, fmt)
    wc = g.integers(0, 256, (n_out, K // 2), dtype=np.uint8)
    wb = np.full((n_out, K // o.BLOCK[fmt]), 127 if fmt == o.MX else 56, np.uint8)
    if fmt == o.MX:
        wb[0], wb[1] = 250, 3
    else:
        wb[0], wb[1] = 126, 1
    wb[2, 1] = 255 if fmt == o.MX else 127
    x = torch.from_numpy(g.standard_normal((2, K)).astype(np.float32)).bfloat16()
    Wd = prep(sl, wc, wb, None, fmt)
    y = torch.empty(2, n_out, device="cuda")
    cfg = sl.config(sel=sl.AS_SEL_ALL, out_dtype=sl.AS_F32)
    ws = torch.empty(sl.as_workspace_size(sl.AS_OP_DECODE_FP4, 2, K, n_out, cfg), dtype=torch.uint8, device="cuda")
    sl.as_linear_decode_fp4(x.cuda(), Wd, cfg, y, fmt=fmt, workspace=ws)
    ok(sl)
    y = f32(y).astype(np.float64)
    assert np.isnan(y[:, 2]).all() and np.isfinite(np.delete(y, 2, 1)).all()
    w = o.values(wc, wb, None, fmt)
    w[2] = 0
    xf = x.double().numpy()
    tol = 40 * 2.0 ** -22 * (np.abs(xf) @ np.abs(w).T) + 2.0 ** -148
    assert (np.abs(np.delete(y - xf @ w.T, 2, 1)) <= np.delete(tol, 2, 1)).all()


# ------------------------------------------------------------------ norm
def check_norm(sl, T, D, rdt, ydt, hdt, gate, fmt=None, post=True, weights=True, inplace=False, scale=0.9, off=0.0,
               eps=1e-6):
    g = rng(T, D, 3)
    t = {"b": torch.bfloat16, "f": torch.float32}
    r = torch.from_numpy((g.laplace(0, 1, (T, D)) * 3).astype(np.float32)).to(t[rdt])
    y = torch.from_numpy((g.standard_normal((T, D)) * np.exp(g.standard_normal((T, 1)))).astype(np.float32)).to(t[ydt])
    pw, qw = [torch.from_numpy((1 + 0.2 * g.standard_normal(D)).astype(np.float32)) if weights else None
              for _ in range(2)]
    gt = {"none": None, "channel": (D,), "token": (T, D)}[gate]
    gt = None if gt is None else torch.from_numpy((0.5 + g.standard_normal(gt)).astype(np.float32))
    R, H = Guarded(T, D, dtype=t[rdt]), Guarded(T, D, dtype=t[hdt])
    rd = r.cuda()
    if inplace:
        R.t.copy_(rd)
        rd = R.t
    kw = {}
    if fmt is not None:
        bufs = (Guarded(T, D // 2, dtype=torch.uint8), Guarded(sl.as_fp4_sf_bytes(T, D, fmt), dtype=torch.uint8),
                Guarded(T, dtype=torch.float32))
        kw = dict(h_q=bufs[0].t, h_sf=bufs[1].t, h_scale=bufs[2].t, fmt=fmt)
    c = lambda v: None if v is None else v.cuda()
    sl.as_norm_residual(rd, y=y.cuda(), r_out=R.t, h=H.t, post_w=c(pw) if post else None, pre_w=c(qw), gate=c(gt),
                        res_scale=scale, eps=eps, w_offset=off, post_norm=post, **kw)
    ok(sl)
    R.check(), H.check()
    n = lambda v: None if v is None else v.double().numpy()
    r64, h64 = o.norm_residual(n(r), n(y), post, n(pw) if post else None, n(gt), n(qw), scale, eps, off)
    # r': the mean square errs by at most D/NT + tree steps (at most 48) of
    # 2^-24, halved by the root; four more factors and one sum.  40 in all.
    E = 40 * 2.0 ** -24
    er = E * (np.abs(scale * n(r)) + np.abs(r64 - scale * n(r)))
    err = np.abs(f32(R.t).astype(np.float64) - r64)
    assert (err <= er + HALF[t[rdt]] * np.abs(r64)).all()
    rms = np.sqrt((r64 * r64).mean(-1, keepdims=True) + eps)
    w = 1.0 if qw is None else np.abs(off + n(qw))
    eh = er / rms * w + (E + np.sqrt((er * er).mean(-1, keepdims=True)) / rms) * np.abs(h64)
    err = np.abs(f32(H.t).astype(np.float64) - h64)
    assert (err <= eh + HALF[t[hdt]] * np.abs(h64)).all()
    if fmt is not None and hdt == "f":  # the codes are those of the float32 h, bit for bit
        for b in bufs:
            b.check()
        codes, byte, S = o.quant(f32(H.t), fmt)
        np.testing.assert_array_equal(f32(bufs[2].t), S)
        np.testing.assert_array_equal(bufs[1].t.cpu().numpy(), o.tile_scales(byte, fmt))
        np.testing.assert_array_equal(bufs[0].t.cpu().numpy(), codes)


@pytest.mark.parametrize("T,D", [(1, 8), (1, 4096), (3, 1000), (2, 1032), (5, 2048), (4, 2056), (7, 4104), (3, 8192),
                                 (2, 8200), (3, 16384), (2, 16392), (2, 32768), (600, 264)])
@pytest.mark.parametrize("types", ["bbb", "fbf", "bff", "ffb"])
def test_norm(sl, T, D, types):
    check_norm(sl, T, D, *types, gate=("none", "channel", "token")[(T + D // 8) % 3])


@pytest.mark.parametrize("fmt", [o.MX, o.NV])
@pytest.mark.parametrize("T,D", [(1, 32), (3, 96), (129, 1056), (33, 4096), (2, 8224), (2, 32768), (300, 64)])
def test_norm_fp4(sl, T, D, fmt):
    check_norm(sl, T, D, "f", "b", "f", "channel", fmt=fmt)


@pytest.mark.parametrize("T,D,types,gate,fmt", [
    (1300, 2056, "bbb", "channel", None), (1300, 2080, "fbf", "token", o.NV), (1201, 4096, "fff", "token", None),
    (1500, 4128, "bbf", "none", o.MX), (1184, 8192, "ffb", "token", None), (1185, 8192, "bfb", "channel", None)])
def test_norm_many_rows(sl, T, D, types, gate, fmt):
    """Enough rows for the persistent kernel."""
    check_norm(sl, T, D, *types, gate=gate, fmt=fmt)


def test_norm_many_rows_options(sl):
    check_norm(sl, 1300, 4096, "b", "b", "b", "token", inplace=True)
    check_norm(sl, 1300, 5000, "f", "b", "f", "channel", post=False, scale=-1.5)
    check_norm(sl, 1300, 4096, "f", "f", "f", "none", weights=False, off=1.0)


def test_norm_options(sl):
    check_norm(sl, 5, 1024, "b", "b", "b", "token", inplace=True)
    check_norm(sl, 5, 1024, "f", "f", "f", "channel", post=False, scale=-1.5)
    check_norm(sl, 5, 1024, "f", "b", "f", "none", weights=False, eps=0.0)
    check_norm(sl, 5, 1024, "f", "b", "f", "none", off=1.0, scale=0.0, eps=0.1)


def test_norm_alone_and_parts(sl):
    """Without a block output: h = norm(r); with one but without h: r' only."""
    g = rng(9)
    r = torch.from_numpy(g.standard_normal((3, 264)).astype(np.float32))
    w = torch.from_numpy(g.standard_normal(264).astype(np.float32))
    h = torch.empty(3, 264, device="cuda")
    sl.as_norm_residual(r.cuda(), h=h, pre_w=w.cuda())
    _, want = o.norm_residual(r.numpy(), pre_w=w.numpy())
    np.testing.assert_allclose(f32(h), want, rtol=40 * 2.0 ** -24)
    out = torch.empty(3, 264, device="cuda")
    sl.as_norm_residual(r.cuda(), y=r.cuda(), r_out=out, res_scale=2.0)
    ok(sl)
    np.testing.assert_allclose(f32(out), 3 * r.numpy(), rtol=2.0 ** -22)
    z = torch.zeros(2, 64, device="cuda")  # a zero row: zeros, no division by zero
    hz = torch.full_like(z, 5.0)
    sl.as_norm_residual(z, h=hz)
    ok(sl)
    assert not hz.any()


# ------------------------------------------------------------------ together
def test_block_chain_on_a_side_stream_and_in_a_graph(sl):
    """norm step -> 4-bit operand -> product, and a decode of the same layer,
    eager on a side stream and as a replayed graph with new inputs."""
    T, D, n_out, fmt = 12, 1056, 264, sl.AS_FP4_NV
    g = rng(4)
    W = torch.from_numpy((g.standard_normal((n_out, D)) * 0.05).astype(np.float32)).cuda()
    r = torch.from_numpy(g.standard_normal((T, D)).astype(np.float32)).cuda()
    y = torch.from_numpy(g.standard_normal((T, D)).astype(np.float32)).cuda()
    wq, wsf, ws = quantise(sl, W, fmt)
    Wd = torch.empty(sl.as_fp4_decode_bytes(n_out, D, fmt), dtype=torch.uint8, device="cuda")
    cfg = sl.config(sel=sl.AS_SEL_NM, n=8, m=16, dpts=True, out_dtype=sl.AS_F32)
    rowsum = torch.from_numpy(o.values(*[a.cpu().numpy() for a in (wq,)], o.quant(f32(W), fmt)[1], f32(ws), fmt)
                              .sum(1).astype(np.float32)).cuda()
    work = torch.empty(sl.as_workspace_size(sl.AS_OP_DECODE_FP4, T, D, n_out, cfg), dtype=torch.uint8, device="cuda")
    b = dict(h=torch.empty(T, D, device="cuda"), r_out=torch.empty(T, D, device="cuda"),
             q=torch.empty(T, D // 2, dtype=torch.uint8, device="cuda"),
             sf=torch.empty(sl.as_fp4_sf_bytes(T, D, fmt), dtype=torch.uint8, device="cuda"),
             sc=torch.empty(T, device="cuda"), p=torch.empty(T, n_out, device="cuda"),
             d=torch.empty(T, n_out, device="cuda"))

    def step():
        sl.as_norm_residual(r, y=y, r_out=b["r_out"], h=b["h"], post_norm=True, h_q=b["q"], h_sf=b["sf"],
                            h_scale=b["sc"], fmt=fmt)
        sl.as_linear_prefill_fp4(b["q"], b["sf"], wq, wsf, b["p"], x_scale=b["sc"], w_scale=ws, fmt=fmt)
        sl.as_linear_decode_fp4(b["h"], Wd, cfg, b["d"], fmt=fmt, rowsum=rowsum, workspace=work)

    def expect():
        _, h = o.norm_residual(f32(r), f32(y), post_norm=True)
        np.testing.assert_allclose(f32(b["h"]), h, rtol=1e-5, atol=1e-5)
        hv = o.values(*o.quant(f32(b["h"]), fmt), fmt)
        wv = o.values(wq.cpu().numpy(), o.quant(f32(W), fmt)[1], f32(ws), fmt)
        mag = np.abs(hv) @ np.abs(wv).T
        assert (np.abs(f32(b["p"]) - hv @ wv.T) <= (D / 64 + 12) * 2.0 ** -22 * mag + 2.0 ** -22 * mag).all()
        hf = f32(b["h"])
        eta = oracle.token_mean(hf).astype(np.float32)
        xh = (hf - eta[:, None]).astype(np.float32)
        m = oracle.select_nm(oracle.score(hf, eta=eta), 8, 16)
        ref = (xh.astype(np.float64) * m) @ wv.T + eta[:, None] * f32(rowsum)
        assert np.linalg.norm(f32(b["d"]) - ref) <= 1e-5 * np.linalg.norm(ref)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        sl.as_weight_prep_fp4(wq, wsf, Wd, w_scale=ws, fmt=fmt)
        step()
    s.synchronize()
    expect()
    eager = {k: v.clone() for k, v in b.items()}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        step()
    for v in b.values():
        v.zero_()
    graph.replay()
    ok(sl)
    for k, v in b.items():
        assert torch.equal(v, eager[k]), k
    r.copy_(torch.from_numpy(g.standard_normal((T, D)).astype(np.float32)))
    y.mul_(-0.5)
    graph.replay()
    ok(sl)
    expect()


@pytest.mark.parametrize("fmt", [o.MX, o.NV])
def test_layer(sl, fmt):
    """Fp4Linear: quantises W, decodes and prefills with the same weights; the
    prefill prunes before it quantises."""
    from sparse_linear_b200.layer import Fp4Linear
    T, K, n_out = 20, 1056, 264
    x, W = synth.random_layer(T, K, n_out, seed=8)
    cfg = sl.config(score=sl.AS_SCORE_WEIGHT, sel=sl.AS_SEL_NM, n=8, m=16, out_dtype=sl.AS_F32)
    L = Fp4Linear(W.cuda(), cfg, alpha=0.5, fmt=fmt)
    wv = o.values(*o.quant(W.float().numpy(), fmt), fmt)
    assert np.array_equal(f32(L.weight.values()), wv)
    g, rs = oracle.weight_prep(wv, 0.5)
    np.testing.assert_allclose(f32(L.g), g, rtol=1e-6)
    np.testing.assert_allclose(f32(L.rowsum), rs, rtol=1e-6, atol=1e-6)
    xf = x.float().numpy()
    m = oracle.select_nm(oracle.score(xf, f=f32(L.g)), 8, 16)
    xk = xf * m
    y = L.decode(x[:16].cuda())
    ok(sl)
    mag = np.abs(xk) @ np.abs(wv).T
    assert (np.abs(f32(y) - xk[:16] @ wv.T) <= 30 * 2.0 ** -22 * mag[:16]).all()
    y = L.prefill(x.cuda())
    ok(sl)
    q = o.values(*o.quant(xk, fmt), fmt)
    assert (np.abs(f32(y) - q @ wv.T) <= (K / 64 + 12) * 2.0 ** -22 * (np.abs(q) @ np.abs(wv).T)).all()
    with pytest.raises(ValueError):
        Fp4Linear(W.cuda(), sl.config(dpts=True, n=8, m=16), fmt=fmt).prefill(x.cuda())


def test_layer_on_a_side_stream(sl):
    """What the layer allocates within a call belongs to the call's stream: work
    that the current stream starts meanwhile does not get its memory."""
    from sparse_linear_b200.layer import Fp4Linear
    T, K, n_out = 64, 2048, 264
    x, W = (t.cuda() for t in synth.random_layer(T, K, n_out, seed=9))
    cfg = sl.config(score=sl.AS_SCORE_WEIGHT, sel=sl.AS_SEL_NM, n=8, m=16, out_dtype=sl.AS_F32)
    L, M = Fp4Linear(W, cfg, alpha=0.5), Fp4Linear(W, cfg, alpha=0.5)
    want = [L.prefill(x), L.decode(x[:16]), L.weight.values()]
    s = torch.cuda.Stream()
    big = torch.ones(4096, 4096, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        for _ in range(20):  # keeps the side stream busy
            big = big @ big * 2.0 ** -12
    got = [M.prefill(x, stream=s), M.decode(x[:16], stream=s.cuda_stream), M.weight.values(stream=s)]
    junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda")
            for n in (T * K * 2, T * K // 2, sl.as_fp4_sf_bytes(T, K), T * 4) for _ in range(4)]
    torch.cuda.synchronize()
    ok(sl)
    assert len(junk) == 16
    for a, b in zip(want, got):
        assert torch.equal(a, b)
