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
