"""Host side of the entry points around a layer (rows sorted by LoRA and back, layer norm): refusals before any launch,
workspace sizes, plans under the sanitizers, the binding's checks.  No GPU: every call is refused or has nothing to do."""
import ctypes
import os
import re

import pytest
import torch

import segmented_gather_matvec_amd as sg
from tests.test_host_sanitizers import ROOT, SAN, _build_and_run, _tool

HEADER = open(os.path.join(ROOT, "include", "sgmv.h")).read()
FAKE, ODD = 0x10000, 0x10004
OK, INVALID, UNSUPPORTED, WORKSPACE = sg.SGMV_OK, sg.SGMV_ERR_INVALID_ARG, sg.SGMV_ERR_UNSUPPORTED, sg.SGMV_ERR_WORKSPACE
MOST_TOP_K = int(re.search(r"#define SGMV_MAX_TOP_K (\d+)", HEADER).group(1))
MOST_LORAS = int(re.search(r"#define SGMV_MAX_ROUTE_LORAS (\d+)", HEADER).group(1))
MOST_ROWS = 1 << int(re.search(r"#define SGMV_MAX_LAYER_ROWS \(1 << (\d+)\)", HEADER).group(1))

def test_limits_match_the_header():
    assert (sg.SGMV_MAX_TOP_K, sg.SGMV_MAX_ROUTE_LORAS) == (MOST_TOP_K, MOST_LORAS)


ARGS = {
    "sgmv_route_rows": dict(n=6000, k=2, P=40, ids=FAKE, perm=FAKE, slots=FAKE, seg=FAKE, idx=FAKE, ws=FAKE, bytes=1 << 40),
    "sgmv_dispatch_rows": dict(dtype=0, n=10, k=2, w=64, X=FAKE, slots=FAKE, Xs=FAKE),
    "sgmv_combine_rows": dict(dtype=0, n=10, k=2, w=64, Ys=FAKE, slots=FAKE, weights=FAKE, R=FAKE, Y=FAKE),
    "sgmv_combine_rows_backward": dict(dtype=0, n=10, k=2, w=64, dY=FAKE, Ys=FAKE, slots=FAKE, weights=FAKE, dYs=FAKE, dw=FAKE),
    "sgmv_layer_norm_apply": dict(dtype=0, n=10, w=64, X=FAKE, g=FAKE, b=FAKE, eps=1e-5, Y=FAKE, mean=FAKE, rstd=FAKE),
    "sgmv_layer_norm_backward": dict(dtype=0, n=10, w=64, X=FAKE, g=FAKE, mean=FAKE, rstd=FAKE, dY=FAKE, past=FAKE, dX=FAKE,
                                     dg=FAKE, db=FAKE, acc=0, ws=FAKE, bytes=1 << 40),
}


def call(name, **kw):
    args = dict(ARGS[name])
    assert set(kw) <= set(args)
    args.update(kw)
    return getattr(sg.load_library(), name)(*args.values(), None)


ROWS = [n for n in ARGS if n != "sgmv_route_rows"]
CHOICES = ["sgmv_dispatch_rows", "sgmv_combine_rows", "sgmv_combine_rows_backward"]


@pytest.mark.parametrize("name", ROWS)
@pytest.mark.parametrize("kw,status", [
    (dict(dtype=2), UNSUPPORTED), (dict(dtype=-1), UNSUPPORTED), (dict(n=-1), INVALID), (dict(w=0), INVALID), (dict(w=-8), INVALID),
    (dict(w=60), UNSUPPORTED), (dict(w=(1 << 20) + 8), UNSUPPORTED), (dict(n=(1 << 30) + 1), UNSUPPORTED)])
def test_refusals_of_every_call_on_rows(name, kw, status):
    assert call(name, **kw) == status


@pytest.mark.parametrize("name", CHOICES + ["sgmv_route_rows"])
@pytest.mark.parametrize("kw,status", [(dict(k=0), INVALID), (dict(k=-1), INVALID), (dict(k=MOST_TOP_K + 1), UNSUPPORTED),
                                       (dict(n=MOST_ROWS // 2 + 1, k=2), UNSUPPORTED), (dict(n=-1), INVALID)])
def test_refusals_of_choices(name, kw, status):
    assert call(name, **kw) == status


@pytest.mark.parametrize("name,needed", [
    ("sgmv_route_rows", ["ids"]), ("sgmv_dispatch_rows", ["X", "slots", "Xs"]), ("sgmv_combine_rows", ["Ys", "slots", "Y"]),
    ("sgmv_combine_rows_backward", ["dY", "Ys", "slots"]), ("sgmv_layer_norm_apply", ["X", "Y"]),
    ("sgmv_layer_norm_backward", ["X", "mean", "rstd", "dY"])])
def test_null_arguments(name, needed):
    for arg in needed:
        assert call(name, **{arg: None}) == INVALID


@pytest.mark.parametrize("name", list(ARGS))
def test_misaligned_arguments(name):
    """Rows and parameters at 16 bytes, counters, weights and moments at 4."""
    words = {"ids", "perm", "slots", "seg", "idx", "weights", "dw", "mean", "rstd"}
    for arg, v in ARGS[name].items():
        if v != FAKE:
            continue
        assert call(name, **{arg: FAKE + 2 if arg in words else ODD}) == UNSUPPORTED, arg


def test_values_outside_their_range():
    for acc in (-1, 2):
        assert call("sgmv_layer_norm_backward", acc=acc) == INVALID
    for eps in (-1e-9, float("nan"), float("inf")):
        assert call("sgmv_layer_norm_apply", eps=eps) == INVALID
    for P, status in ((0, INVALID), (-3, INVALID), (MOST_LORAS + 1, UNSUPPORTED)):
        assert call("sgmv_route_rows", P=P) == status


def test_nothing_to_do():
    none = dict(n=0)
    assert call("sgmv_dispatch_rows", X=None, slots=None, Xs=None, **none) == OK
    assert call("sgmv_combine_rows", Ys=None, slots=None, Y=None, **none) == OK
    assert call("sgmv_combine_rows_backward", dY=None, slots=None, Ys=None, **none) == OK
    assert call("sgmv_layer_norm_apply", X=None, Y=None, **none) == OK
    assert call("sgmv_layer_norm_backward", X=None, mean=None, rstd=None, dY=None, dg=None, db=None, ws=None, bytes=0, **none) == OK
    assert call("sgmv_layer_norm_backward", X=None, mean=None, rstd=None, dY=None, acc=1, ws=None, bytes=0, **none) == OK


def test_workspaces_are_checked_to_the_byte():
    need = sg.sgmv_route_workspace_bytes(6000, 2, 40)
    assert need > 0 and sg.sgmv_route_workspace_bytes(0, 1, 1) == 0
    assert call("sgmv_route_rows", bytes=need - 1) == WORKSPACE and call("sgmv_route_rows", ws=None) == WORKSPACE
    assert call("sgmv_route_rows", ws=FAKE + 8) == UNSUPPORTED
    need = sg.sgmv_layer_norm_workspace_bytes(10, 64)
    assert call("sgmv_layer_norm_backward", bytes=need - 1) == WORKSPACE
    assert call("sgmv_layer_norm_backward", ws=None) == WORKSPACE
    lib, out = sg.load_library(), ctypes.c_size_t(0)
    assert lib.sgmv_route_workspace_bytes(1, 1, 1, None) == INVALID
    assert lib.sgmv_layer_norm_workspace_bytes(1, 8, None) == INVALID
    assert lib.sgmv_layer_norm_workspace_bytes(1, 12, ctypes.byref(out)) == UNSUPPORTED
    assert lib.sgmv_route_workspace_bytes(1, 1, MOST_LORAS + 1, ctypes.byref(out)) == UNSUPPORTED


def test_block_plans_under_sanitizers(tmp_path):
    csrc = os.path.join(ROOT, "segmented_gather_matvec_amd", "csrc")
    exe = str(tmp_path / "block_checks")
    cmd = [_tool("g++"), "-std=c++17"] + SAN + [
        "-I", os.path.join(ROOT, "include"), "-I", csrc, os.path.join(ROOT, "tests", "sanitize", "block_checks.cpp"),
        os.path.join(csrc, "sgmv_host.cpp"), os.path.join(csrc, "sgmv_block_host.cpp"), "-o", exe]
    assert "block checks ok" in _build_and_run(cmd, exe, tmp_path)


class On(torch.Tensor):
    """A CPU tensor that says it is on a device: the binding's checks come before any launch."""
    index = 0
    is_cuda = property(lambda self: True)
    get_device = lambda self: self.index  # noqa: E731


class OnSecond(On):
    index = 1
    device = property(lambda self: torch.device("cuda", 1))


def on(t, cls=On):
    return t.as_subclass(cls)


def test_binding_checks_types_shapes_and_devices():
    h, f = torch.float16, torch.float32
    X, Xs, slots, w = (on(torch.zeros(4, 16, dtype=h)), on(torch.zeros(8, 16, dtype=h)), on(torch.zeros(8, dtype=torch.int32)),
                       on(torch.zeros(8, dtype=f)))
    g, m = on(torch.zeros(16, dtype=h)), on(torch.zeros(4, dtype=f))
    refused = [
        (lambda: sg.sgmv_dispatch_rows(torch.zeros(4, 16).half(), slots, Xs), "X must be a device tensor"),
        (lambda: sg.sgmv_dispatch_rows(on(torch.zeros(4, 16)), slots, Xs), "X must be torch.float16 or torch.bfloat16"),
        (lambda: sg.sgmv_dispatch_rows(X, slots, on(torch.zeros(7, 16, dtype=h))), "Xs must have a whole number of rows"),
        (lambda: sg.sgmv_dispatch_rows(X, slots, on(torch.zeros(8, 24, dtype=h))), r"Xs must be \[8, 16\]"),
        (lambda: sg.sgmv_dispatch_rows(X, on(torch.zeros(7, dtype=torch.int32)), Xs), "slots must hold 8 entries, got 7"),
        (lambda: sg.sgmv_dispatch_rows(X, on(torch.zeros(8, dtype=torch.int64)), Xs), "slots must be torch.int32"),
        (lambda: sg.sgmv_dispatch_rows(on(X.t()), slots, Xs), "X must be contiguous"),
        (lambda: sg.sgmv_dispatch_rows(X, on(slots, OnSecond), Xs), "slots must be on X's device"),
        (lambda: sg.sgmv_combine_rows(on(Xs.bfloat16()), slots, X), "Ys must be torch.float16"),
        (lambda: sg.sgmv_combine_rows(Xs, slots, X, weights=on(w.half())), "weights must be torch.float32"),
        (lambda: sg.sgmv_combine_rows(Xs, slots, X, residual=Xs), r"residual must be \[4, 16\]"),
        (lambda: sg.sgmv_combine_rows_backward(X, on(torch.zeros(4, 16, dtype=h)), slots, dweights=w), r"Ys must be \[8, 16\]"),
        (lambda: sg.sgmv_combine_rows_backward(X, Xs, slots, dweights=on(torch.zeros(4, dtype=f))), "dweights must hold 8"),
        (lambda: sg.sgmv_layer_norm_apply(X, on(torch.zeros(8, dtype=h)), None, X), r"gamma must be \[16\]"),
        (lambda: sg.sgmv_layer_norm_apply(X, g, None, Xs), r"Y must be \[4, 16\]"),
        (lambda: sg.sgmv_layer_norm_apply(X, g, None, X, mean=on(m.half())), "mean must be torch.float32"),
        (lambda: sg.sgmv_layer_norm_apply(on(torch.zeros(16, dtype=h)), g, None, X), "X must be a 2-D"),
        (lambda: sg.sgmv_layer_norm_backward(X, g, m, m, Xs, None), r"dY must be \[4, 16\]"),
        (lambda: sg.sgmv_layer_norm_backward(X, g, m, None, X, None, dgamma=on(torch.zeros(4, dtype=h))), r"dgamma must be \[16\]"),
        (lambda: sg.sgmv_route_rows(on(torch.zeros(2, 2, 2, dtype=torch.int32)), 3, slots, slots, None, None, None), "ids must be a"),
        (lambda: sg.sgmv_route_rows(on(torch.zeros(9, dtype=torch.int32)), 3, slots, None, None, None, None), "perm must hold 9"),
        (lambda: sg.sgmv_route_rows(slots, 8, None, None, slots, None, None), "seg_indptr must hold 9 entries"),
    ]
    for attempt, why in refused:
        with pytest.raises(ValueError, match=why):
            attempt()
