"""The index-checked build of the library on small cases of the 4-bit and norm
kernels: their oracle comparisons hold and no index left its buffer."""
import pytest
import torch

import test_gpu_fp4 as F
from oracle import fp4 as o
from test_gpu_checked_build import sl_checked  # noqa: F401  (the checked library as a fixture)

pytestmark = pytest.mark.gpu

CASES = [
    (F.test_quant, dict(R=33, K=160, fmt=o.NV, dtype=torch.bfloat16)),
    (F.test_quant, dict(R=129, K=288, fmt=o.MX, dtype=torch.float32)),
    (F.test_product, dict(T=17, K=256, n_out=120, fmt=o.NV)),
    (F.test_product, dict(T=257, K=32, n_out=264, fmt=o.MX)),
    (F.test_product_pairs, dict(T=1300, K=416, n_out=1960, fmt=o.NV)),
    (F.test_product_pairs, dict(T=200, K=1312, n_out=9992, fmt=o.MX)),
    (F.test_product_one_wave, dict(T=1000, K=544, n_out=1032, fmt=o.MX)),
    (F.test_decode_topk, dict(T=16, kk=1023, dpts=1, fmt=o.NV)),
    (F.test_decode_all_and_threshold, dict(T=4, K=2080, n_out=136, dpts=0, xdt="f")),
    (F.test_norm, dict(T=3, D=1000, types="bff")),
    (F.test_norm_fp4, dict(T=129, D=1056, fmt=o.MX)),
    (F.test_norm_many_rows, dict(T=1300, D=2080, types="fbf", gate="token", fmt=o.NV)),
]


@pytest.mark.parametrize("i", range(len(CASES)), ids=[f"{f.__name__}-{j}" for j, (f, _) in enumerate(CASES)])
def test_checked_build(sl_checked, i):  # noqa: F811
    fn, kw = CASES[i]
    try:
        fn(sl_checked, **kw)
        torch.cuda.synchronize()
        assert sl_checked.as_stream_status() == sl_checked.AS_OK
    finally:
        line = sl_checked.as_checked_line()
        assert line == 0, f"index check failed at source line {line}"
