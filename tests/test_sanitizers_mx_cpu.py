"""Sanitizer build of the MXFP4 and routing argument checks (CPU only), like
test_sanitizers_cpu.py's of the GEMM entry points."""
import os

from test_sanitizers_cpu import ROOT, SAN, _build_and_run, pytestmark  # noqa: F401


def test_api_mx_validation_under_sanitizers(tmp_path):
    out = _build_and_run(tmp_path, "api_mx_san",
                         [os.path.join(ROOT, "block_scaled_fp4_gemm_amd", "csrc", "api_mx.cpp"),
                          os.path.join(SAN, "api_mx_driver.cpp")],
                         ["-I" + os.path.join(SAN, "hip_stub"), "-I" + os.path.join(ROOT, "include")])
    assert "api_mx sanitizer driver: ok" in out
