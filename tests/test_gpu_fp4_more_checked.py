"""More cases of the 4-bit decode, its staged columns and the norm step's scale
tiles on the index-checked build."""
import pytest
import torch

import test_gpu_fp4 as F
import test_gpu_fp4_faults as G
import test_gpu_fp4_more as M
from oracle import fp4 as o
from test_gpu_checked_build import sl_checked  # noqa: F401  (the checked library as a fixture)

pytestmark = pytest.mark.gpu

CASES = [
    (F.test_decode_nm, dict(T=16, K=4128, n_out=392, n=8, m=16, score=0, dpts=0, xdt="b", odt="b", fmt=o.NV)),
    (F.test_decode_nm, dict(T=13, K=20000, n_out=136, n=16, m=32, score=1, dpts=1, xdt="b", odt="f", fmt=o.MX)),
    (F.test_decode_nm, dict(T=1, K=32, n_out=8, n=2, m=4, score=0, dpts=0, xdt="b", odt="f", fmt=o.NV)),
    (G.test_decode_holds_x, dict(fmt=o.MX, out=torch.float32, dtype=torch.float32)),
    (G.test_decode_mx_rows_of_far_apart_scales, {}),
    (M.test_decode_many_output_tiles, dict(T=3, K=544, n_out=20008, odt="b", fmt=o.MX)),
    (M.test_few_tokens_many_tiles, dict(T=30, K=544, n_out=20008, fmt=o.NV)),
    (M.test_norm_few_rows_per_sm, dict(T=443, D=2080, types="fbf", gate="token", fmt=o.NV)),
    (M.test_norm_parts_of_the_outputs, dict(T=300, D=4096, fmt=o.MX)),
    (F.test_norm_fp4, dict(T=300, D=64, fmt=o.NV)),
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
