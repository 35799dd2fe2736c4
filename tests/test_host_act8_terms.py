"""Width of the dX GEMM's adapter operands on the CPU (g++):
tests/host/act8_terms_check.cpp with the planning sources."""

import shutil

import pytest


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_adapter_operands_of_the_dx_gemm(tmp_path):
    from test_host_sanitizers import _build_and_run
    _build_and_run(tmp_path, "act8_terms_check.cpp", "act8_plan.cpp")
