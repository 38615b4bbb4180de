"""Cases of the 4-bit operators and the norm step that once went wrong or had no
test, against the float64 oracle; tolerances as in test_gpu_fp4."""
import numpy as np
import pytest
import torch

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
