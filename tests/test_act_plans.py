"""Plans of the layer calls with an activation under the address and undefined-behaviour sanitizers (CPU only), and that the
sizes of the GPU tests of 128 x 256 tiles (tests/test_gpu_act_wide.py) do reach them."""
import os
import subprocess

import pytest

from tests.test_host_sanitizers import ROOT, SAN, _build_and_run, _tool

CSRC = os.path.join(ROOT, "segmented_gather_matvec_amd", "csrc")
WIDE = 5


@pytest.fixture(scope="module")
def driver(tmp_path_factory):
    tmp = tmp_path_factory.mktemp("act")
    exe = str(tmp / "act_checks")
    cmd = [_tool("g++"), "-std=c++17"] + SAN + [
        "-I", os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(ROOT, "tests", "sanitize", "act_checks.cpp"),
        os.path.join(CSRC, "sgmv_host.cpp"), os.path.join(CSRC, "sgmv_layer_host.cpp"), "-o", exe]
    assert "act checks ok" in _build_and_run(cmd, exe, tmp)
    return exe


def test_act_plans_under_sanitizers(driver):
    assert os.path.exists(driver)


def test_sizes_of_the_wide_tiles(driver):
    from tests.test_gpu_act_wide import FORWARD, BACKWARD
    for cases, column in ((FORWARD, 0), (BACKWARD, 1)):
        args = [str(v) for c in cases for v in c]
        lines = subprocess.run([driver] + args, capture_output=True, text=True, check=True).stdout.split("\n")
        for case, line in zip(cases, lines):
            assert int(line.split()[column]) == WIDE, case


def test_sizes_of_the_shared_term(driver):
    from tests.test_gpu_act_wide import SHARED
    lines = subprocess.run([driver] + [str(v) for c in SHARED for v in c], capture_output=True, text=True, check=True).stdout.split("\n")
    for case, line in zip(SHARED, lines):
        assert line.split()[3] == "1", case
