"""The head's plans for the sizes of tests/test_gpu_head_paths.py, on the CPU (g++)."""

import shutil

import pytest


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_sizes_go_the_ways_they_are_there_for(tmp_path):
    from test_host_sanitizers import _build_and_run
    _build_and_run(tmp_path, "head_paths_check.cpp", "head_plan.cpp")
