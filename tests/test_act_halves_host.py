"""Host side of SGMV_DZ_HALVES: workspace sizes and refusals before any launch, and the plans under the sanitizers.  No GPU."""
import os
import re

import pytest

import segmented_gather_matvec_amd as sg
from tests.test_act_host import BACKWARD, FORWARD, INVALID, UNSUPPORTED, WORKSPACE, call
from tests.test_host_sanitizers import ROOT, SAN, _build_and_run, _tool
from tests.test_layer_host import HEADER, good

HALVES = sg.SGMV_DZ_HALVES


def test_value_matches_the_header():
    assert int(re.search(r"#define SGMV_DZ_HALVES (0x\d+)", open(HEADER).read()).group(1), 16) == HALVES


def test_workspaces():
    for kw in (dict(), dict(dtype="bf16"), dict(n_rows=5000, max_seg_len=3000), dict(n_rows=200, num_segs=0, max_seg_len=0)):
        p = good(**kw)
        plain, need = (sg.sgmv_layer_workspace_bytes(p, BACKWARD | f) for f in (0, HALVES))
        few = p.n_rows <= 128 and p.n_rows * p.h_out <= 1 << 18
        assert need == plain if few else need >= plain + p.n_rows * p.h_out * 2
        assert call(BACKWARD, p, ws_bytes=need - 1, act=sg.SGMV_ACT_GELU | HALVES) == WORKSPACE


@pytest.mark.parametrize("act", [sg.SGMV_ACT_GELU + 1 + HALVES, -1 & ~HALVES, -1, 2 * HALVES, 3 * HALVES])
def test_acts_that_are_none(act):
    assert call(BACKWARD, act=act) == INVALID


def test_only_the_backward_call_takes_it():
    assert call(FORWARD, act=sg.SGMV_ACT_SILU | HALVES) == INVALID
    for op in (FORWARD, sg.SGMV_DENSE_BACKWARD, sg.SGMV_GATED_BACKWARD):
        with pytest.raises(sg.SgmvError):
            sg.sgmv_layer_workspace_bytes(good(), op | HALVES)


def test_most_rows():
    kw = dict(num_segs=0, max_seg_len=0, h_in=8, h_out=8)
    assert sg.sgmv_layer_workspace_bytes(good(n_rows=1 << 29, **kw), BACKWARD | HALVES) > 0
    p = good(n_rows=(1 << 29) + 1, **kw)
    assert call(BACKWARD, p, act=sg.SGMV_ACT_RELU | HALVES) == UNSUPPORTED
    with pytest.raises(sg.SgmvError):
        sg.sgmv_layer_workspace_bytes(p, BACKWARD | HALVES)
    assert sg.sgmv_layer_workspace_bytes(p, BACKWARD) > 0


def test_plans_under_sanitizers(tmp_path):
    csrc = os.path.join(ROOT, "segmented_gather_matvec_amd", "csrc")
    exe = str(tmp_path / "halves_checks")
    cmd = [_tool("g++"), "-std=c++17"] + SAN + [
        "-I", os.path.join(ROOT, "include"), "-I", csrc, os.path.join(ROOT, "tests", "sanitize", "halves_checks.cpp"),
        os.path.join(csrc, "sgmv_host.cpp"), os.path.join(csrc, "sgmv_layer_host.cpp"), "-o", exe]
    assert "halves checks ok" in _build_and_run(cmd, exe, tmp_path)


