"""The layers' buffer management without a GPU: the library's calls are replaced
by recorders, so that only the Python side runs."""
import pytest
import torch

import sparse_linear_b200.layer as layer
import sparse_linear_b200 as sl

CALLS = ("as_quant_fp4", "as_dequant_fp4", "as_weight_prep", "as_weight_prep_fp4", "as_linear_decode_fp4",
         "as_linear_prefill_fp4", "as_select", "as_linear_decode", "as_linear_prefill")


@pytest.fixture
def calls(monkeypatch):
    """[(name, workspace or None)] of every call, buffers kept alive."""
    seen = []

    def recorder(name):
        return lambda *a, **kw: seen.append((name, kw.get("workspace")))

    for name in CALLS:
        monkeypatch.setattr(layer, name, recorder(name))
    monkeypatch.setattr(layer, "select_out", lambda **kw: None)  # it takes device tensors only
    return seen


def fp4_layer(cfg):
    return layer.Fp4Linear(torch.zeros(16, 64), cfg)


def given(calls, name):
    return [w for n, w in calls if n == name]


def test_fp4_calls_share_no_scratch(calls):
    """Two decodes (prefills) of one layer at one T may be on two streams or in
    two graphs that run at the same time: no buffer in common."""
    L = fp4_layer(sl.config(score=sl.AS_SCORE_CLACT, sel=sl.AS_SEL_NM, n=8, m=16))
    for _ in range(2):
        L.decode(torch.zeros(2, 64))
        L.prefill(torch.zeros(20, 64))
    for name in ("as_linear_decode_fp4", "as_select"):
        a, b = given(calls, name)
        assert a.numel() and a.data_ptr() != b.data_ptr(), name


def test_fp4_scratch_follows_the_configuration(calls):
    """A configuration that needs more scratch than the one before it gets it."""
    L = fp4_layer(sl.config(sel=sl.AS_SEL_NM, n=8, m=16, out_dtype=sl.AS_BF16))
    L.decode(torch.zeros(16, 64))
    for cfg in (sl.config(sel=sl.AS_SEL_NM, n=8, m=16, out_dtype=sl.AS_F32),
                sl.config(score=sl.AS_SCORE_CLACT, sel=sl.AS_SEL_NM, n=8, m=16, out_dtype=sl.AS_F32)):
        L.cfg = cfg
        L.decode(torch.zeros(16, 64))
        need = sl.as_workspace_size(sl.AS_OP_DECODE_FP4, 16, 64, 16, cfg)
        assert given(calls, "as_linear_decode_fp4")[-1].numel() >= need


def test_sparse_workspaces_belong_to_a_stream(calls, monkeypatch):
    """Kept per stream, and not kept when a capture fills them with zeros."""
    now = [1]
    monkeypatch.setattr(layer, "_current_stream", lambda: now[0], raising=False)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: now[0] == 3)
    L = layer.SparseLinear(torch.zeros(16, 64), sl.config(score=sl.AS_SCORE_CLACT, n=8, m=16))
    for stream in (1, 2, 1, 3, 3):
        now[0] = stream
        L.decode(torch.zeros(2, 64))
        L.prefill(torch.zeros(20, 64))
    for name in ("as_linear_decode", "as_select", "as_linear_prefill"):
        one, two, again, captured, next_captured = [w.data_ptr() for w in given(calls, name)]
        assert one == again and len({one, two, captured, next_captured}) == 4, name
