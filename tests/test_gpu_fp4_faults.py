"""Cases of the 4-bit operators and the norm step that once went wrong or had no
test, against the float64 oracle; tolerances as in test_gpu_fp4."""
import numpy as np
import pytest
import torch

import synth
from gpu_util import f32
from oracle import fp4 as o
from test_gpu_fp4 import dev, ok, random_operand, sl  # noqa: F401  (sl is a fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", [o.MX, o.NV])
def test_pair_products_back_to_back(sl, fmt):  # noqa: F811
    """One K block per tile, so that a CTA pair leaves right after its last
    commit, and the next launch takes its place: 200 launches, one result."""
    T, K, n_out = 2500, 32, 1032
    xc, xb, xS, _ = random_operand(21, T, K, fmt)
    wc, wb, wS, _ = random_operand(22, n_out, K, fmt)
    args = (dev(xc), dev(o.tile_scales(xb, fmt)), dev(wc), dev(o.tile_scales(wb, fmt)))
    kw = dict(x_scale=dev(xS), w_scale=dev(wS), fmt=fmt)
    first = torch.empty(T, n_out, device="cuda")
    sl.as_linear_prefill_fp4(*args, first, **kw)
    ys = [torch.empty_like(first) for _ in range(4)]
    for i in range(200):
        sl.as_linear_prefill_fp4(*args, ys[i % 4], **kw)
    ok(sl)
    assert np.isfinite(f32(first)).all()
    assert all(torch.equal(y, first) for y in ys)


def busy(stream, n=12):
    """Keeps a stream occupied for some milliseconds."""
    with torch.cuda.stream(stream):
        a = torch.ones(4096, 4096, device="cuda")
        for _ in range(n):
            a = a @ a * 2.0 ** -12


@pytest.mark.parametrize("sel", ["nm", "topk", "clact"])
def test_one_layer_on_two_streams(sl, sel):  # noqa: F811
    """Decodes and prefills of one layer, equal T and different tokens, on two
    streams that are both behind other work."""
    from sparse_linear_b200.layer import Fp4Linear
    T, K, n_out = 8, 2048, 520
    cfg = {"nm": sl.config(sel=sl.AS_SEL_NM, n=8, m=16, dpts=True, out_dtype=sl.AS_F32),
           "topk": sl.config(sel=sl.AS_SEL_TOPK, k_keep=900, out_dtype=sl.AS_F32),
           "clact": sl.config(score=sl.AS_SCORE_CLACT, sel=sl.AS_SEL_NM, n=8, m=16, out_dtype=sl.AS_F32)}[sel]
    _, W = synth.random_layer(T, K, n_out, seed=31)
    L = Fp4Linear(W.cuda(), cfg)
    xs = [synth.random_layer(T, K, n_out, seed=40 + i)[0].cuda() for i in range(8)]
    calls = [L.decode] if cfg.dpts else [L.decode, L.prefill]
    want = [[f(x) for f in calls] for x in xs]
    ok(sl)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        busy(s)
    got = [[f(x, stream=streams[i % 2]) for f in calls] for i, x in enumerate(xs)]
    ok(sl)
    for w, g in zip(want, got):
        assert all(torch.equal(a, b) for a, b in zip(w, g))


def test_two_graphs_of_one_layer_at_once(sl):  # noqa: F811
    """Two graphs captured on one stream from one layer, replayed on two streams."""
    from sparse_linear_b200.layer import Fp4Linear
    T, K, n_out = 16, 4096, 264
    cfg = sl.config(sel=sl.AS_SEL_NM, n=8, m=16, out_dtype=sl.AS_F32)
    _, W = synth.random_layer(T, K, n_out, seed=32)
    L = Fp4Linear(W.cuda(), cfg)
    xs = [synth.random_layer(T, K, n_out, seed=50 + i)[0].cuda() for i in range(2)]
    want = [L.decode(x) for x in xs]
    s = torch.cuda.Stream()
    graphs, ys = [torch.cuda.CUDAGraph() for _ in xs], [[], []]
    for g, x, y in zip(graphs, xs, ys):
        with torch.cuda.graph(g, stream=s):
            for _ in range(20):
                y.append(L.decode(x))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    for _ in range(3):
        for g, t in zip(graphs, streams):
            with torch.cuda.stream(t):
                g.replay()
        ok(sl)
        for w, y in zip(want, ys):
            assert all(torch.equal(v, w) for v in y)


def test_layer_with_another_configuration(sl):  # noqa: F811
    """Output type and score changed between two calls at one T."""
    from sparse_linear_b200.layer import Fp4Linear
    T, K, n_out = 16, 1024, 136
    x, W = (t.cuda() for t in synth.random_layer(T, K, n_out, seed=33))
    cfgs = [sl.config(score=score, sel=sl.AS_SEL_NM, n=8, m=16, out_dtype=out)
            for score in (sl.AS_SCORE_MAG, sl.AS_SCORE_CLACT) for out in (sl.AS_BF16, sl.AS_F32)]
    L = Fp4Linear(W, cfgs[0])
    for cfg in cfgs:
        L.cfg = cfg
        assert torch.equal(L.decode(x), Fp4Linear(W, cfg).decode(x))
        assert torch.equal(L.prefill(x), Fp4Linear(W, cfg).prefill(x))
    ok(sl)


def test_one_sparse_layer_on_two_streams(sl):  # noqa: F811
    """SparseLinear: decode and prefill of different tokens on two streams behind
    other work, and the mode switch, which reads a result back."""
    from sparse_linear_b200.layer import SparseLinear
    T, K, n_out = 8, 2048, 520
    _, W = synth.random_layer(T, K, n_out, seed=34)
    xs = [synth.random_layer(T, K, n_out, seed=60 + i)[0].cuda() for i in range(8)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    for cfg, calls in ((sl.config(sel=sl.AS_SEL_NM, n=8, m=16, dpts=True, out_dtype=sl.AS_F32), ("decode", "prefill")),
                       (sl.config(score=sl.AS_SCORE_CLACT, sel=sl.AS_SEL_NM, n=8, m=16), ("decode", "prefill")),
                       (sl.config(sel=sl.AS_SEL_TOPK, k_keep=900), ("decode",)),
                       (sl.config(sel=sl.AS_SEL_NM, n=2, m=4), ("prefill_auto",))):
        L = SparseLinear(W.cuda(), cfg)

        def run(i, **kw):
            out = [getattr(L, c)(xs[i], **kw) for c in calls]
            return [v[0] if isinstance(v, tuple) else v for v in out]

        want = [run(i) for i in range(8)]
        ok(sl)
        for s in streams:
            busy(s)
        got = [run(i, stream=streams[i % 2]) for i in range(8)]
        ok(sl)
        for w, g in zip(want, got):
            assert all(torch.equal(a, b) for a, b in zip(w, g))


# ------------------------------------------------- how decode holds x
def one_hot(K, fmt, code=2, byte=None, w_scale=1.0):
    """Weights [K, K] whose row o reads channel o only: every output is one
    value of x times (E2M1 of code) * scale * w_scale."""
    q = np.zeros((K, K), np.uint8)
    q[np.arange(K), np.arange(K)] = code
    b = np.full((K, K // o.BLOCK[fmt]), byte if byte is not None else (127 if fmt == o.MX else 56), np.uint8)
    return q[:, 0::2] | (q[:, 1::2] << 4), b, np.full(K, w_scale, np.float32)


def decode_values(sl, x, fmt, out, w=None, cfg=None):  # noqa: F811
    """prune(x) as the decode holds it, through one-hot weights."""
    T, K = x.shape
    wc, wb, wS = w or one_hot(K, fmt)
    Wd = torch.empty(sl.as_fp4_decode_bytes(K, K, fmt), dtype=torch.uint8, device="cuda")
    sl.as_weight_prep_fp4(dev(wc), dev(o.tile_scales(wb, fmt)), Wd, w_scale=dev(wS), fmt=fmt)
    cfg = cfg or sl.config(sel=sl.AS_SEL_ALL, out_dtype=sl.AS_F32 if out == torch.float32 else sl.AS_BF16)
    y = torch.empty(T, K, dtype=out, device="cuda")
    ws = torch.empty(sl.as_workspace_size(sl.AS_OP_DECODE_FP4, T, K, K, cfg), dtype=torch.uint8, device="cuda")
    sl.as_linear_decode_fp4(x.cuda(), Wd, cfg, y, fmt=fmt, workspace=ws)
    ok(sl)
    return f32(y).astype(np.float64)


HELD = {torch.bfloat16: 2.0 ** -22, torch.float32: 2.0 ** -28}


def check_held(x, y, fmt, out, factor=1.0):
    """A kept value errs by HELD of its block's largest (NV: or of 2^-17 of its
    token's largest, if more), by a few float32 roundings of itself (the parts'
    sum, the factor) and by the output's rounding, which among subnormal numbers
    is half of 2^-133 (bf16) or of 2^-149."""
    v = x.double().numpy()
    top = np.repeat(np.abs(v).reshape(v.shape[0], -1, o.BLOCK[fmt]).max(-1), o.BLOCK[fmt], axis=1)
    if fmt == o.NV:
        top = np.maximum(top, 2.0 ** -17 * np.abs(v).max(-1, keepdims=True))
    half = 2.0 ** -8 if out == torch.bfloat16 else 0.0
    tol = HELD[out] * top * factor + (3 * 2.0 ** -24 + half) * np.abs(v) * factor
    tol = tol + (2.0 ** -134 if out == torch.bfloat16 else 2.0 ** -149)
    err = np.abs(y - v * factor)
    assert (err <= tol).all(), (float((err / tol).max()), np.argwhere(err > tol)[:4])


def held_rows(K, dtype):
    g = np.random.default_rng(91)
    rows = [g.laplace(0, 0.3, K)]
    for big in (1e3, 1e4, 1e6):  # one value of a block of 16 above the others
        r = g.standard_normal(K)
        r[g.integers(0, 16, K // 16) + 16 * np.arange(K // 16)] *= big
        rows.append(r)
    # values that leave the most after every part: 0.5 of its last place each
    # time, in either direction, and one part too many for the last
    for ratio in (6.0, 8.0):
        for lead, last in ((4.0, 4.999), (2.5, 2.4999), (3.5, 3.4999), (0.25, 0.2499)):
            v = last
            for _ in range(9):
                v = lead + v / ratio
            rows.append(v * np.exp2(g.integers(-3, 4, K // 16)).repeat(16) * np.where(np.arange(K) % 2, 1.0, -1.0))
            rows[-1][::16] = 4.0 * np.abs(rows[-1][1::16])
    rows.append(g.standard_normal(K) * np.exp2(g.integers(-40, 40, K)))
    return torch.from_numpy(np.array(rows).astype(np.float32)).to(dtype)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", [o.MX, o.NV])
def test_decode_holds_x(sl, fmt, out, dtype):  # noqa: F811
    x = held_rows(512, dtype)
    check_held(x, decode_values(sl, x, fmt, out), fmt, out)
    for t in (0, 3):  # one token takes another column count
        check_held(x[t:t + 1], decode_values(sl, x[t:t + 1], fmt, out), fmt, out)


@pytest.mark.parametrize("out", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("fmt", [o.MX, o.NV])
def test_decode_tiny_and_huge_tokens(sl, fmt, out):  # noqa: F811
    """Tokens near both ends of float32, pruned and not."""
    g = np.random.default_rng(92)
    K = 256
    base = g.standard_normal((8, K)) * (g.random((8, K)) < 0.7)
    scale = np.exp2(np.array([-149.0, -140, -127, -120, -100, 100, 120, 125]))[:, None]
    x = torch.from_numpy((base * scale).clip(-3.4e38, 3.4e38).astype(np.float32))
    check_held(x, decode_values(sl, x, fmt, out), fmt, out)
    cfg = sl.config(sel=sl.AS_SEL_NM, n=2, m=4, out_dtype=sl.AS_F32)
    y = decode_values(sl, x, fmt, torch.float32, cfg=cfg)
    kept = np.where(y != 0, x.double().numpy(), 0.0)
    assert (np.count_nonzero(y, axis=1) <= K // 2).all()
    check_held(torch.from_numpy(kept), y, fmt, torch.float32)


def test_decode_sums_do_not_overflow_before_the_row_scale(sl):  # noqa: F811
    """Weights are stored 2688 times their row scale: a large x times them stays
    finite when the output is."""
    x = torch.from_numpy((np.random.default_rng(93).uniform(1, 3, (2, 256)) * 1e38).astype(np.float32))
    w = one_hot(256, o.NV, code=7, byte=126, w_scale=2.0 ** -12)
    y = decode_values(sl, x, o.NV, torch.float32, w=w)
    check_held(x, y, o.NV, torch.float32, factor=2688 * 2.0 ** -12)


def test_decode_mx_rows_of_far_apart_scales(sl):  # noqa: F811
    """Rows with block scales up to 2^123 beside blocks of down to 2^-122: every
    block keeps its own scale, whichever of them x reaches."""
    K = 512
    wc, wb, wS = one_hot(K, o.MX)
    own = np.arange(K) // 32
    small = np.array([5, 40, 100, 120, 134, 136, 200, 250])[np.arange(K) % 8]
    wb[np.arange(K), (own + 1) % (K // 32)] = 250   # codes zero there
    wb[np.arange(K), own] = small
    x = torch.from_numpy(np.random.default_rng(94).uniform(1, 2, (3, K)).astype(np.float32))
    y = decode_values(sl, x, o.MX, torch.float32, w=(wc, wb, wS))
    want = x.double().numpy() * np.exp2(small - 127.0)
    assert (np.abs(y - want) <= (2.0 ** -27 + 3 * 2.0 ** -24) * np.abs(want)).all()  # block within a factor of 2
    # and the large blocks beside them
    q = np.zeros((K, K), np.uint8)
    q[np.arange(K), (np.arange(K) + 32) % K] = 2
    x = x * 2.0 ** -100
    y = decode_values(sl, x, o.MX, torch.float32, w=(q[:, 0::2] | (q[:, 1::2] << 4), wb, wS))
    want = np.roll(x.double().numpy(), -32, axis=1) * 2.0 ** 123
    assert (np.abs(y - want) <= (2.0 ** -27 + 3 * 2.0 ** -24) * np.abs(want)).all()


def test_norm_step_from_many_threads(sl):  # noqa: F811
    """Calls of one kernel that need different shared memory, from host threads
    that start together (a new process would meet them as its first calls)."""
    import threading
    g = torch.Generator(device="cuda").manual_seed(5)
    cases = []
    for i, (D, rdt, ydt) in enumerate([(2056, torch.bfloat16, torch.bfloat16), (4096, torch.float32, torch.float32),
                                       (2080, torch.bfloat16, torch.float32), (4096, torch.float32, torch.bfloat16)]):
        r = torch.randn(600, D, generator=g, device="cuda").to(rdt)
        y = torch.randn(600, D, generator=g, device="cuda").to(ydt)
        gate = torch.randn(600, D, generator=g, device="cuda") if i % 2 else None
        cases.append((r, y, gate))
    got, errors = [None] * 8, []
    gate_open = threading.Barrier(8)
    streams = [torch.cuda.Stream() for _ in range(8)]
    torch.cuda.synchronize()

    def work(i):
        r, y, gate = cases[i % 4]
        try:
            with torch.cuda.stream(streams[i]):
                out = torch.empty_like(r)
                h = torch.empty(r.shape, device="cuda")
                gate_open.wait(30)
                for _ in range(20):
                    sl.as_norm_residual(r, y=y, r_out=out, h=h, gate=gate, post_norm=True)
            got[i] = (out, h)
        except Exception as e:  # noqa: BLE001 (reported below)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    ok(sl)
    assert not errors, errors
    for i in range(4):
        assert all(torch.equal(a, b) for a, b in zip(got[i], got[i + 4]))
        n = lambda v: None if v is None else v.double().cpu().numpy()  # noqa: E731
        r, y, gate = cases[i]
        _, h = o.norm_residual(n(r), n(y), True, None, n(gate))
        assert np.abs(f32(got[i][1]) - h).max() <= 1e-4  # |h| < 8: its roundings are below 40 * 2^-24 * 8 = 2e-5
