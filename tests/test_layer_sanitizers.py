"""The layer entry points' host plans under the address and undefined-behaviour sanitizers (CPU only):
tests/sanitize/layer_checks.cpp with the library's host-only sources, over seeded random and extreme problems."""
import os

from tests.test_host_sanitizers import ROOT, SAN, _build_and_run, _tool

CSRC = os.path.join(ROOT, "segmented_gather_matvec_amd", "csrc")


def test_layer_plans_under_sanitizers(tmp_path):
    exe = str(tmp_path / "layer_checks")
    cmd = [_tool("g++"), "-std=c++17"] + SAN + [
        "-I", os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(ROOT, "tests", "sanitize", "layer_checks.cpp"),
        os.path.join(CSRC, "sgmv_host.cpp"), os.path.join(CSRC, "sgmv_layer_host.cpp"), "-o", exe]
    assert "layer checks ok" in _build_and_run(cmd, exe, tmp_path)
