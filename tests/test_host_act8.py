"""Host C++ of the 8-bit checkpoint path on the CPU (g++):
tests/host/act8_check.cpp with the planning sources under AddressSanitizer and
UndefinedBehaviorSanitizer."""

import shutil

import pytest


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_act8_plans_layout_and_quotient(tmp_path):
    from test_host_sanitizers import _build_and_run
    _build_and_run(tmp_path, "act8_check.cpp", "act8_plan.cpp")
