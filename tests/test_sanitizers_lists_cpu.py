"""The tensor-list encoder under AddressSanitizer and UBSan (host code only):
random lists, valid and not, and a walk of the task tables that the kernels
read."""
import os

from test_sanitizers_cpu import ROOT, SAN, _build_and_run


def test_list_encoder_under_asan_ubsan(tmp_path):
    exe = tmp_path / "list_fuzz"
    csrc = os.path.join(ROOT, "quantized_momentum_newton_amd", "csrc")
    cmd = ["g++", "-std=c++17", *SAN, "-I", os.path.join(ROOT, "include"), "-I", csrc,
           os.path.join(ROOT, "tests", "sanitize", "list_fuzz.cpp"), os.path.join(csrc, "list_plan.cpp"),
           os.path.join(csrc, "plan.cpp"), "-o", str(exe)]
    out = _build_and_run(cmd, exe, ["4000"], tmp_path)
    assert " 0 failed checks" in out, out
