"""Host side of the layer with bias, activation and residual: refusals before any launch, workspace sizes, plans.  No GPU."""
import ctypes
import os
import re

import pytest
import torch

import segmented_gather_matvec_amd as sg
from tests.test_block_host import OnSecond, on
from tests.test_layer_host import FAKE, HEADER, ODD, good

FORWARD, BACKWARD = sg.SGMV_DENSE_ACT_FORWARD, sg.SGMV_DENSE_ACT_BACKWARD
INVALID, UNSUPPORTED, WORKSPACE = sg.SGMV_ERR_INVALID_ARG, sg.SGMV_ERR_UNSUPPORTED, sg.SGMV_ERR_WORKSPACE


def call(op, problem=None, ws_bytes=1 << 40, **kw):
    a = dict(X=FAKE, W=FAKE, Y=0x10000, A=0x10000, B=0x10000, ranks=None, scales=None, bias=FAKE, act=sg.SGMV_ACT_SILU, R=FAKE,
             Z=FAKE, dY=FAKE, dX=FAKE, dW=None, dA=None, dB=None, db=FAKE, acc=0, seg=FAKE, ids=FAKE, ws=FAKE)
    assert set(kw) <= set(a)
    a.update(kw)
    lib, p = sg.load_library(), ctypes.byref(problem or good())
    pj = ctypes.byref(sg.sgmv_projection_t(a["A"], a["B"], a["Y"], a["ranks"], a["scales"]))
    tail = (a["seg"], a["ids"], a["ws"], ws_bytes, None)
    if op == FORWARD:
        return lib.sgmv_dense_act_lora_apply(p, a["X"], a["W"], pj, a["bias"], a["act"], a["R"], a["Z"], *tail)
    g = ctypes.byref(sg.sgmv_projection_grad_t(a["dW"], a["dA"], a["dB"]))
    return lib.sgmv_dense_act_lora_backward(p, a["X"], a["W"], pj, a["act"], a["Z"], a["dY"], a["dX"], g, a["db"], a["acc"], *tail)


def test_values_match_the_header():
    src = open(HEADER).read()
    for name in ("SGMV_ACT_SILU", "SGMV_ACT_GELU_TANH", "SGMV_ACT_NONE", "SGMV_ACT_RELU", "SGMV_ACT_GELU",
                 "SGMV_DENSE_ACT_FORWARD", "SGMV_DENSE_ACT_BACKWARD"):
        assert int(re.search(rf"\b{name} = (\d+)", src).group(1)) == getattr(sg, name)
    ops = open(os.path.join(os.path.dirname(sg.__file__), "csrc", "sgmv_layer_ops.h")).read()
    codes = re.search(r"kActSilu = (\d), kActGeluTanh = (\d), kActNone = (\d), kActRelu = (\d), kActGelu = (\d);", ops).groups()
    assert [int(v) for v in codes] == [sg.SGMV_ACT_SILU, sg.SGMV_ACT_GELU_TANH, sg.SGMV_ACT_NONE, sg.SGMV_ACT_RELU, sg.SGMV_ACT_GELU]


@pytest.mark.parametrize("op", [FORWARD, BACKWARD])
@pytest.mark.parametrize("kw,status", [
    (dict(X=None), INVALID), (dict(W=None), INVALID), (dict(A=None), INVALID), (dict(B=None), INVALID), (dict(seg=None), INVALID),
    (dict(ids=None), INVALID), (dict(act=5), INVALID), (dict(act=-1), INVALID), (dict(X=ODD), UNSUPPORTED), (dict(W=ODD), UNSUPPORTED),
    (dict(Z=ODD), UNSUPPORTED), (dict(A=0x10004), UNSUPPORTED), (dict(ranks=0x10002), UNSUPPORTED), (dict(ws=None), WORKSPACE),
    (dict(ws=ODD), UNSUPPORTED)])
def test_refusals_of_both(op, kw, status):
    assert call(op, **kw) == status


@pytest.mark.parametrize("op,kw,status", [
    (FORWARD, dict(Y=None), INVALID), (FORWARD, dict(Y=0x10008), UNSUPPORTED), (FORWARD, dict(bias=ODD), UNSUPPORTED),
    (FORWARD, dict(R=ODD), UNSUPPORTED), (BACKWARD, dict(dY=None), INVALID), (BACKWARD, dict(Z=None), INVALID),
    (BACKWARD, dict(acc=2), INVALID), (BACKWARD, dict(dY=ODD), UNSUPPORTED), (BACKWARD, dict(dX=ODD), UNSUPPORTED),
    (BACKWARD, dict(db=ODD), UNSUPPORTED), (BACKWARD, dict(dW=0x10008), UNSUPPORTED), (BACKWARD, dict(dA=0x10004), UNSUPPORTED)])
def test_refusals_of_one(op, kw, status):
    assert call(op, **kw) == status


@pytest.mark.parametrize("op", [FORWARD, BACKWARD])
@pytest.mark.parametrize("kw", [dict(rank=24), dict(h_in=4), dict(h_out=1 << 21), dict(n_rows=-1), dict(dtype=2),
                                dict(n_rows=(1 << 30) + 1, num_segs=0, max_seg_len=0)])
def test_bad_problems(op, kw):
    assert call(op, good(**kw)) != sg.SGMV_OK
    with pytest.raises(sg.SgmvError):
        sg.sgmv_layer_workspace_bytes(good(**kw), op)


def test_workspaces():
    """The query's size holds for every activation and part; with a byte less the call that needs most is refused."""
    for kw in (dict(), dict(dtype="bf16"), dict(n_rows=5000, max_seg_len=3000), dict(n_rows=200, num_segs=0, max_seg_len=0)):
        p = good(**kw)
        need = sg.sgmv_layer_workspace_bytes(p, BACKWARD)
        assert need >= sg.sgmv_layer_workspace_bytes(p, sg.SGMV_DENSE_BACKWARD) + p.h_out * 4
        assert call(BACKWARD, p, ws_bytes=need - 1) == WORKSPACE
        fwd = sg.sgmv_layer_workspace_bytes(p, FORWARD)
        assert fwd == sg.sgmv_layer_workspace_bytes(p, sg.SGMV_DENSE_FORWARD)
        if fwd:
            assert call(FORWARD, p, ws_bytes=fwd - 1) == WORKSPACE


def test_nothing_to_do():
    p = good(n_rows=0, num_segs=0, max_seg_len=0)
    assert call(FORWARD, p, ws_bytes=0, X=None, W=None, Y=None, seg=None, ids=None, ws=None) == sg.SGMV_OK
    assert call(BACKWARD, p, ws_bytes=0, X=None, W=None, seg=None, ids=None, ws=None, Z=None, dY=None, db=None, acc=1) == sg.SGMV_OK


def test_gated_calls_keep_their_activations():
    lib, p = sg.load_library(), ctypes.byref(good())
    pj = ctypes.byref(sg.sgmv_projection_t(0x10000, 0x10000, 0x10000, None, None))
    for act in (sg.SGMV_ACT_NONE, sg.SGMV_ACT_RELU, sg.SGMV_ACT_GELU):
        assert lib.sgmv_gated_lora_apply(p, FAKE, FAKE, FAKE, pj, pj, act, FAKE, FAKE, FAKE, FAKE, 1 << 40, None) == INVALID


def test_binding_checks():
    p = good(n_rows=4, h_in=16, h_out=24, max_seg_len=2)
    h = torch.float16
    X, W, Y = on(torch.zeros(4, 16, dtype=h)), on(torch.zeros(16, 24, dtype=h)), on(torch.zeros(4, 24, dtype=h))
    for kw, why in ((dict(bias=on(torch.zeros(16, dtype=h))), r"bias must be \[24\]"), (dict(residual=X), r"residual must be \[4, 24\]"),
                    (dict(Z=on(Y.float())), "Z must be torch.float16"), (dict(bias=on(torch.zeros(24, dtype=h), OnSecond)), "on X's device")):
        with pytest.raises(ValueError, match=why):
            sg.sgmv_dense_act_lora_apply(p, X, W, (None, None, Y), None, None, None, **kw)
    with pytest.raises(ValueError, match=r"dbias must be \[24\]"):
        sg.sgmv_dense_act_lora_backward(p, X, W, (None, None), Y, None, None, None, dbias=on(torch.zeros(23, dtype=h)))
