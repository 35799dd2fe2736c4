"""Host C++ of the head's loss on the CPU (g++): tests/host/head_check.cpp with
the planning source under AddressSanitizer and UndefinedBehaviorSanitizer."""

import shutil

import pytest


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_head_plans_and_deal(tmp_path):
    from test_host_sanitizers import _build_and_run
    _build_and_run(tmp_path, "head_check.cpp", "head_plan.cpp")
