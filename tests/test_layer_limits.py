"""The layer entry points' own limits: rows, blocks of rows, and nothing of what sgmv_check_problem keeps for the kernels
of the other entry points (arrival counters, variants, splits)."""
import os
import re

import pytest

import segmented_gather_matvec_amd as sg
from tests.test_layer_host import HEADER, OPS, Raw, good
from tests.test_host_sanitizers import ROOT, SAN, _build_and_run, _tool

MOST_UNITS = (1 << int(re.search(r"#define SGMV_MAX_LAYER_UNITS \(\(1 << (\d+)\) - 1\)", open(HEADER).read()).group(1))) - 1
SMALL = dict(h_in=8, h_out=8, rank=16)


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("kw", [
    dict(n_rows=3_000_000, num_segs=1, max_seg_len=3_000_000),      # one long segment
    dict(n_rows=1 << 30, num_segs=2, max_seg_len=(1 << 29) - 64),   # the most rows
    dict(n_rows=400_000, num_segs=400_000, max_seg_len=1),          # a row each
    dict(n_rows=MOST_UNITS, num_segs=MOST_UNITS, max_seg_len=64),   # the most blocks
    dict(n_rows=1000, num_segs=200_000, max_seg_len=500),           # mostly empty segments
])
def test_rows_and_segments_that_a_layer_takes(op, kw):
    p = good(**{**SMALL, **kw})
    assert sg.sgmv_check_problem(p) == sg.SGMV_ERR_UNSUPPORTED      # the other kernels' counters
    assert sg.sgmv_layer_workspace_bytes(p, op) > 0
    assert Raw(p).call(op, ws_bytes=0) == sg.SGMV_ERR_WORKSPACE     # past the problem's checks


@pytest.mark.parametrize("op", OPS)
@pytest.mark.parametrize("kw", [
    dict(n_rows=MOST_UNITS + 1, num_segs=MOST_UNITS + 1, max_seg_len=1),
    dict(n_rows=1 << 30, num_segs=(1 << 31) - 1, max_seg_len=1 << 30),
    dict(n_rows=(1 << 30) + 1, num_segs=1, max_seg_len=1 << 30),
    dict(n_rows=1000, num_segs=(1 << 18) + 1, max_seg_len=65),
])
def test_more_is_refused(op, kw):
    p = good(**{**SMALL, **kw})
    assert Raw(p).call(op) == sg.SGMV_ERR_UNSUPPORTED
    with pytest.raises(sg.SgmvError):
        sg.sgmv_layer_workspace_bytes(p, op)


@pytest.mark.parametrize("op", OPS)
def test_variant_and_splits_are_not_used(op):
    want = sg.sgmv_layer_workspace_bytes(good(rank=8), op)
    for kw in (dict(variant=sg.SGMV_VARIANT_MFMA), dict(variant=17), dict(splits=-3), dict(splits=9)):
        assert sg.sgmv_layer_workspace_bytes(good(rank=8, **kw), op) == want


def test_layer_limits_under_sanitizers(tmp_path):
    """Plans at and beyond the limits, and the area of the rows' powers, with the address and undefined-behaviour sanitizers."""
    csrc = os.path.join(ROOT, "segmented_gather_matvec_amd", "csrc")
    exe = str(tmp_path / "layer_limits")
    cmd = [_tool("g++"), "-std=c++17"] + SAN + [
        "-I", os.path.join(ROOT, "include"), "-I", csrc, os.path.join(ROOT, "tests", "sanitize", "layer_limits.cpp"),
        os.path.join(csrc, "sgmv_host.cpp"), os.path.join(csrc, "sgmv_layer_host.cpp"), "-o", exe]
    assert "layer limits ok" in _build_and_run(cmd, exe, tmp_path)
