"""The launch variants that the shapes of the GPU tests take
(CPU only), checked in a sanitizer build of the argument layer."""
import os

from test_sanitizers_cpu import ROOT, SAN, _build_and_run, pytestmark  # noqa: F401


def test_plans_of_the_tested_shapes(tmp_path):
    out = _build_and_run(tmp_path, "gated_plan",
                         [os.path.join(ROOT, "block_scaled_fp4_gemm_amd", "csrc", "api_gated.cpp"),
                          os.path.join(SAN, "gated_plan_driver.cpp")],
                         ["-I" + os.path.join(SAN, "hip_stub"), "-I" + os.path.join(ROOT, "include")])
    assert "gated plan driver: ok" in out
