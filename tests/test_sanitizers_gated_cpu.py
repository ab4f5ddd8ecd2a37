"""Sanitizer build of the gated block's argument checks and tile choice (CPU
only), like test_sanitizers_cpu.py's of the GEMM entry points."""
import os

from test_sanitizers_cpu import ROOT, SAN, _build_and_run, pytestmark  # noqa: F401


def test_api_gated_validation_under_sanitizers(tmp_path):
    out = _build_and_run(tmp_path, "api_gated_san",
                         [os.path.join(ROOT, "block_scaled_fp4_gemm_amd", "csrc", "api_gated.cpp"),
                          os.path.join(SAN, "api_gated_driver.cpp")],
                         ["-I" + os.path.join(SAN, "hip_stub"), "-I" + os.path.join(ROOT, "include")])
    assert "api_gated sanitizer driver: ok" in out
