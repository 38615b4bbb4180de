"""Microscaled 4-bit operators without a GPU: the float64 oracle pinned by
hand-worked blocks and exhaustive nearest-value searches, and the library's
refusals (which launch nothing)."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

from oracle import fp4 as o


@pytest.fixture(scope="module")
def lib():
    import sparse_linear_b200 as sl
    return sl


# ------------------------------------------------------------------ oracle
def test_e4m3_table_is_torchs():
    bits = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(bits, o.E4M3)


def test_mx_block_by_hand():
    x = np.zeros((1, 32))
    x[0, :10] = [6.0, -0.25, 0.26, 0.75, -1.25, 1.75, 2.5, 3.5, 5.0, 0.2]
    codes, byte, S = o.quant(x, o.MX)
    assert byte[0, 0] == 127 and S[0] == 1            # floor(log2 6) - 2 = 0
    want = [6.0, -0.0, 0.5, 1.0, -1.0, 2.0, 2.0, 4.0, 4.0, 0.0]
    np.testing.assert_array_equal(o.values(codes, byte, S, o.MX)[0, :10], want)
    assert codes[0, 0] == 7 | (8 << 4)                # channel 0 low, channel 1 (-0) high
    # 7.9 saturates to 6; twice 7.9 moves the scale
    x[0, 0] = 7.9
    assert o.values(*o.quant(x, o.MX), o.MX)[0, 0] == 6
    x[0, 0] = 15.8
    codes, byte, _ = o.quant(x, o.MX)
    assert byte[0, 0] == 128 and o.values(codes, byte, None, o.MX)[0, 0] == 12
    # zero block, smallest and largest float32
    z = np.zeros((1, 32))
    assert o.quant(z, o.MX)[1][0, 0] == 127
    z[0, 3] = 2.0 ** -149
    assert o.quant(z, o.MX)[1][0, 0] == 0
    z[0, 3] = float(np.finfo(np.float32).max)
    assert o.quant(z, o.MX)[1][0, 0] == 252


def test_nv_row_by_hand():
    x = np.zeros((2, 32))
    x[0, 0], x[0, 16] = 2688.0, 6.0
    codes, byte, S = o.quant(x, o.NV)
    assert S[0] == 1 and byte[0].tolist() == [126, 56] and S[1] == 1   # 448 and 1.0
    np.testing.assert_array_equal(o.values(codes, byte, S, o.NV)[0, [0, 16]], [2688.0, 6.0])
    x[0, 0] = 2689.0
    assert o.quant(x, o.NV)[2][0] == 2
    x[0, 0], x[0, 16] = 2688.0, 6.0 * 2.0 ** -10   # half the smallest scale: a tie, to the even zero
    codes, byte, S = o.quant(x, o.NV)
    assert byte[0, 1] == 0 and not o.values(codes, byte, S, o.NV)[0, 16:].any()


@pytest.mark.parametrize("fmt", [o.MX, o.NV])
def test_quant_is_nearest(fmt):
    """No other code of the block's scale is nearer (float64 search over all)."""
    rng = np.random.default_rng(3)
    x = (rng.standard_normal((5, 96)) * np.exp(rng.standard_normal((5, 96)))).astype(np.float32)
    codes, byte, S = o.quant(x, fmt)
    B = o.BLOCK[fmt]
    v = o.values(codes, byte, S, fmt)
    s = np.repeat(o.scale_value(byte, fmt) * S[:, None], B, axis=1)
    best = np.min(np.abs(np.abs(x)[..., None] - o.E2M1 * s[..., None]), -1)
    np.testing.assert_array_equal(np.abs(x - v), best)
    if fmt == o.MX:
        amax = np.abs(x.reshape(5, -1, B)).max(-1)
        assert ((amax >= 4 * o.scale_value(byte, fmt)) & (amax < 8 * o.scale_value(byte, fmt))).all()


def test_non_finite_blocks():
    x = np.ones((1, 64), np.float32)
    x[0, 5], x[0, 40] = np.inf, np.nan
    for fmt, bad, nan in ((o.MX, [0, 1], 255), (o.NV, [0, 2], 127)):
        codes, byte, S = o.quant(x, fmt)
        assert (byte[0, bad] == nan).all() and np.isfinite(S).all()
        v = o.values(codes, byte, S, fmt).reshape(-1, o.BLOCK[fmt])
        assert np.isnan(v[bad]).all() and np.isnan(v).any(-1).sum() == 2


def test_scale_tiles():
    byte = np.arange(130 * 5, dtype=np.uint32).reshape(130, 5).astype(np.uint8)
    t = o.tile_scales(byte, o.NV)
    assert t.size == 2 * 2 * 512
    assert t[16 * 7 + 4 * 1 + 2] == byte[39, 2]             # row 39 = 32 + 7, block 2
    assert t[512 + 16 * 7 + 4] == byte[39, 4]               # second tile along K
    assert t[2 * 512 + 16 * 1] == byte[129, 0]              # second tile of rows
    assert t[512 + 1] == 0


def test_norm_residual_by_hand():
    r, y = np.array([[1.0, 1.0, 1.0, 1.0]]), np.array([[3.0, -4.0, 0.0, 0.0]])
    r2, h = o.norm_residual(r, y, post_norm=True, gate=np.full(4, 2.0), res_scale=0.5, eps=0.0)
    np.testing.assert_allclose(r2, [[0.5 + 2.4, 0.5 - 3.2, 0.5, 0.5]])
    np.testing.assert_allclose((h * h).mean(), 1.0)
    _, h = o.norm_residual(r, pre_w=np.array([1.0, 2.0, 3.0, 4.0]), w_offset=1.0, eps=3.0)
    np.testing.assert_allclose(h, [[1.0, 1.5, 2.0, 2.5]])


# ------------------------------------------------------------------ refusals
FAKE = 1 << 20  # aligned and never dereferenced: a launch would fail here


def test_sizes(lib):
    assert lib.as_fp4_sf_bytes(1, 32, lib.AS_FP4_NV) == 512
    assert lib.as_fp4_sf_bytes(129, 4096, lib.AS_FP4_NV) == 2 * 64 * 512
    assert lib.as_fp4_sf_bytes(128, 4096 + 32, lib.AS_FP4_MX) == 33 * 512
    assert lib.as_fp4_decode_bytes(136, 544, lib.AS_FP4_NV) == 2 * 3 * (16384 + 2048) + 2 * 128 * 4
    assert lib.as_fp4_decode_bytes(128, 64, lib.AS_FP4_MX) == 16384 + 1024 + 128 * 4
    for rows, K, fmt in ((0, 64, 0), (1, 48, 1), (1, 0, 1), (1, 131072 + 32, 1), (1, 64, 2)):
        with pytest.raises(lib.ASError):
            lib.as_fp4_sf_bytes(rows, K, fmt)
    for n_out, K in ((4, 64), (0, 64), (8, 40)):
        with pytest.raises(lib.ASError):
            lib.as_fp4_decode_bytes(n_out, K, 0)
    cfg = lib.config(sel=lib.AS_SEL_NM, n=8, m=16)
    assert lib.as_workspace_size(lib.AS_OP_DECODE_FP4, 16, 4096, 64, cfg) >= 16 * 512 + 64
    with pytest.raises(lib.ASError):
        lib.as_workspace_size(lib.AS_OP_DECODE_FP4, 17, 4096, 64, cfg)


def test_sizes_of_any_number_of_lengths(lib):
    """What the size queries remember stays bounded."""
    for f in (lib.as_fp4_sf_bytes, lib.as_fp4_decode_bytes):
        for rows in range(8, 8 * 3000, 8):
            f(rows, 64, lib.AS_FP4_NV)
        assert f.cache_info().currsize <= 2000


def test_quant_refusals(lib):
    f = lib._lib.as_quant_fp4

    def call(x=FAKE, dt=lib.AS_BF16, rows=4, K=64, fmt=lib.AS_FP4_NV, q=FAKE, sf=FAKE, rs=FAKE):
        return f(x, dt, rows, K, fmt, q, sf, rs, None)

    for kw in (dict(x=None), dict(q=None), dict(sf=None), dict(rs=None), dict(rows=0), dict(rows=-1), dict(fmt=2),
               dict(fmt=-1)):
        assert call(**kw) == lib.AS_ERR_INVALID_ARG, kw
    assert call(dt=2) == lib.AS_ERR_DTYPE
    for K in (0, -32, 16, 72, 131104):
        assert call(K=K) == lib.AS_ERR_SHAPE
    for kw in (dict(x=FAKE + 8), dict(q=FAKE + 4), dict(sf=FAKE + 1), dict(rs=FAKE + 4)):
        assert call(**kw) == lib.AS_ERR_ALIGN
    g = lib._lib.as_dequant_fp4
    assert g(None, FAKE, None, 4, 64, 0, lib.AS_F32, FAKE, None) == lib.AS_ERR_INVALID_ARG
    assert g(FAKE, FAKE, None, 4, 64, 0, lib.AS_F32, None, None) == lib.AS_ERR_INVALID_ARG
    assert g(FAKE, FAKE, None, 4, 64, 3, lib.AS_F32, FAKE, None) == lib.AS_ERR_INVALID_ARG
    assert g(FAKE, FAKE, None, 4, 64, 0, 5, FAKE, None) == lib.AS_ERR_DTYPE
    assert g(FAKE, FAKE, None, 4, 40, 0, lib.AS_F32, FAKE, None) == lib.AS_ERR_SHAPE
    assert g(FAKE, FAKE, None, 4, 64, 0, lib.AS_F32, FAKE + 4, None) == lib.AS_ERR_ALIGN


def test_product_refusals(lib):
    f = lib._lib.as_linear_prefill_fp4

    def call(xq=FAKE, xs=FAKE, T=4, K=64, n=16, wq=FAKE, ws=FAKE, fmt=1, dt=lib.AS_F32, y=FAKE, sx=None, sw=None):
        return f(xq, xs, sx, T, K, n, wq, ws, sw, fmt, dt, y, None)

    for kw in (dict(xq=None), dict(xs=None), dict(wq=None), dict(ws=None), dict(y=None), dict(T=0), dict(n=0),
               dict(fmt=2)):
        assert call(**kw) == lib.AS_ERR_INVALID_ARG, kw
    assert call(dt=3) == lib.AS_ERR_DTYPE
    for kw in (dict(K=48), dict(K=0), dict(n=12)):
        assert call(**kw) == lib.AS_ERR_SHAPE
    for kw in (dict(xq=FAKE + 8), dict(ws=FAKE + 8), dict(y=FAKE + 2), dict(sx=FAKE + 4), dict(sw=FAKE + 4)):
        assert call(**kw) == lib.AS_ERR_ALIGN


def test_decode_refusals(lib):
    f, p = lib._lib.as_linear_decode_fp4, lib._lib.as_weight_prep_fp4
    ok = lib.config(sel=lib.AS_SEL_NM, n=8, m=16)

    def call(x=FAKE, dt=lib.AS_BF16, T=1, K=64, n=16, Wd=FAKE, fmt=1, g=None, rs=None, cfg=ok, y=FAKE, ws=FAKE,
             wb=1 << 20):
        return f(x, dt, T, K, n, Wd, fmt, g, rs, ctypes.byref(cfg), y, None, None, None, ws, wb, None)

    for kw in (dict(x=None), dict(Wd=None), dict(y=None), dict(fmt=2), dict(cfg=lib.config(dpts=True)),
               dict(cfg=lib.config(score=lib.AS_SCORE_WEIGHT))):
        assert call(**kw) == lib.AS_ERR_INVALID_ARG, kw
    for kw in (dict(T=0), dict(T=17), dict(K=48), dict(K=40), dict(n=12), dict(cfg=lib.config(n=5, m=4)),
               dict(cfg=lib.config(sel=lib.AS_SEL_TOPK, k_keep=65))):
        assert call(**kw) == lib.AS_ERR_SHAPE, kw
    assert call(dt=4) == lib.AS_ERR_DTYPE
    assert call(cfg=lib.config(var=True)) == lib.AS_ERR_UNSUPPORTED
    for kw in (dict(x=FAKE + 2), dict(Wd=FAKE + 8), dict(y=FAKE + 8), dict(ws=FAKE + 8)):
        assert call(**kw) == lib.AS_ERR_ALIGN
    assert call(ws=None) == lib.AS_ERR_WORKSPACE
    assert call(wb=8) == lib.AS_ERR_WORKSPACE
    assert p(None, FAKE, None, 16, 64, 0, FAKE, None) == lib.AS_ERR_INVALID_ARG
    assert p(FAKE, FAKE, None, 16, 64, 7, FAKE, None) == lib.AS_ERR_INVALID_ARG
    assert p(FAKE, FAKE, None, 12, 64, 0, FAKE, None) == lib.AS_ERR_SHAPE
    assert p(FAKE, FAKE, None, 16, 48, 0, FAKE, None) == lib.AS_ERR_SHAPE
    assert p(FAKE, FAKE, FAKE + 4, 16, 64, 0, FAKE, None) == lib.AS_ERR_ALIGN


def test_norm_refusals(lib):
    f = lib._lib.as_norm_residual
    base = dict(r=FAKE, y=FAKE, r_out=FAKE, h=FAKE, post_w=FAKE, pre_w=FAKE, gate=FAKE, gate_rows=1, post_norm=1,
                r_dtype=1, y_dtype=1, h_dtype=1, res_scale=1.0, eps=1e-6, fmt=1)

    def call(T=4, D=64, **kw):
        return f(ctypes.byref(lib.as_norm_args(**{**base, **kw})), T, D, None)

    alone = dict(y=None, r_out=None, gate=None, post_w=None, post_norm=0)
    assert f(None, 4, 64, None) == lib.AS_ERR_INVALID_ARG
    for kw in (dict(r=None), dict(T=0), dict(D=0), dict(r_out=None, h=None), dict(gate_rows=3), dict(gate_rows=0),
               dict(post_norm=2), dict(post_norm=0), dict(eps=-1.0), dict(eps=float("nan")), dict(y=None),
               {**alone, "gate": FAKE}, {**alone, "r_out": FAKE}, {**alone, "post_norm": 1}, dict(h_q=FAKE),
               dict(h_sf=FAKE), dict(h_scale=FAKE), dict(h_q=FAKE, h_sf=FAKE),
               dict(h_q=FAKE, h_sf=FAKE, h_scale=FAKE, fmt=2)):
        assert call(**kw) == lib.AS_ERR_INVALID_ARG, kw
    for kw in (dict(r_dtype=2), dict(y_dtype=-1), dict(h_dtype=9)):
        assert call(**kw) == lib.AS_ERR_DTYPE, kw
    for kw in (dict(D=60), dict(D=32768 + 8), dict(D=40, h_q=FAKE, h_sf=FAKE, h_scale=FAKE)):
        assert call(**kw) == lib.AS_ERR_SHAPE, kw
    for name in ("r", "y", "r_out", "h", "post_w", "pre_w", "gate"):
        assert call(**{name: FAKE + 8}) == lib.AS_ERR_ALIGN, name


def test_binding_refuses_wrong_tensors(lib):
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    q, sf, s = torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), torch.zeros(4)
    for bad in itertools.product(*[[0, 1]] * 3):
        if not any(bad):
            continue
        with pytest.raises(ValueError):
            lib.as_quant_fp4(x, q[:3] if bad[0] else q, sf[:511] if bad[1] else sf, s[:2] if bad[2] else s)
    with pytest.raises(ValueError):  # CPU tensors
        lib.as_quant_fp4(x, q, sf, s)
    with pytest.raises(ValueError):
        lib.as_linear_prefill_fp4(q, sf, q, sf, torch.zeros(4, 3))
    with pytest.raises(ValueError):
        lib.as_norm_residual(x, y=x[:2], r_out=x)
    with pytest.raises(ValueError):
        lib.as_norm_residual(x, h=x, pre_w=torch.zeros(64, dtype=torch.bfloat16))


def test_missing_buffers_are_refused(lib):
    with pytest.raises(ValueError):
        lib._bytes("sf", None, 4, 0)
    from sparse_linear_b200.layer import Fp4Linear
    layer = object.__new__(Fp4Linear)
    layer.Wd = None
    with pytest.raises(ValueError):
        layer.decode(torch.zeros(1, 64))
