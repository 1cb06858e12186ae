"""Positions of strided gradients as the kernels compute them, against row and
column, under AddressSanitizer and UBSan (host code only)."""
import os

from test_sanitizers_cpu import ROOT, SAN, _build_and_run


def test_positions_of_strided_gradients(tmp_path):
    exe = tmp_path / "list_positions"
    csrc = os.path.join(ROOT, "quantized_momentum_newton_amd", "csrc")
    cmd = ["g++", "-std=c++17", *SAN, "-I", os.path.join(ROOT, "include"), "-I", csrc,
           os.path.join(ROOT, "tests", "sanitize", "list_positions.cpp"), os.path.join(csrc, "list_plan.cpp"),
           os.path.join(csrc, "plan.cpp"), "-o", str(exe)]
    out = _build_and_run(cmd, exe, ["2000"], tmp_path)
    assert " 0 failed checks" in out, out
