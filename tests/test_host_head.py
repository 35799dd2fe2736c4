"""Host C++ of the head's loss and of the orthogonalised updates on the CPU (g++):
tests/host/head_check.cpp and muon_check.cpp with the planning sources under
AddressSanitizer and UndefinedBehaviorSanitizer."""

import shutil

import pytest


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_head_plans_and_deal(tmp_path):
    from test_host_sanitizers import _build_and_run
    _build_and_run(tmp_path, "head_check.cpp", "head_plan.cpp")


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_groups_of_matrices(tmp_path):
    from test_host_sanitizers import _build_and_run
    _build_and_run(tmp_path, "muon_check.cpp", "muon_plan.cpp")
