"""The quotient behind an 8-bit checkpoint's codes on the CPU (g++) at the
values next to every half step: tests/host/act8_code_check.cpp with the header
that the kernel uses."""

import shutil

import pytest


@pytest.mark.skipif(shutil.which("g++") is None, reason="g++ not available")
def test_codes_next_to_half_steps(tmp_path):
    from test_host_sanitizers import _build_and_run
    _build_and_run(tmp_path, "act8_code_check.cpp", None)
