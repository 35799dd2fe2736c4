"""The hash that a profile carries covers every source that shapes a kernel or
its launches: a change to any of them changes the hash of the kernels it is
behind and of no other's."""

import os
import shutil

import pytest

from bit_nf4_quantized_14_amd import profiling

BEHIND = {"act8_plan.cpp": {"k_adapter_rows"}, "act8_plan.h": {"k_adapter_rows"},
          "act8_linear.hip": {"k_adapter_rows"}, "adapter8.hip": {"k_adapter_rows"},
          "act8_host.h": {"k_adapter_rows", "k_act8_encode"},
          "act8_code.h": {"k_act8_encode"}, "act8.hip": {"k_act8_encode"},
          "pref.hip": {"k_seq_rows"}, "gemm.hip": {"k_gemm"}, "rank.hip": {"k_rank_finish"}}
KERNELS = ("k_adapter_rows", "k_act8_encode", "k_seq_rows", "k_gemm", "k_rank_finish", "k_quantize")


@pytest.mark.parametrize("changed", [*BEHIND, *profiling.COMMON_SOURCES])
def test_a_changed_source_changes_its_kernels_hashes(changed, tmp_path, monkeypatch):
    before = {k: profiling.source_sha(k) for k in KERNELS}
    copy = tmp_path / "csrc"
    shutil.copytree(profiling.CSRC, copy)
    monkeypatch.setattr(profiling, "CSRC", str(copy))
    assert {k: profiling.source_sha(k) for k in KERNELS} == before
    with open(copy / changed, "a") as f:
        f.write("// changed\n")
    after = {k: profiling.source_sha(k) for k in KERNELS}
    assert {k for k in KERNELS if after[k] != before[k]} == BEHIND.get(changed, set(KERNELS))


def test_every_source_is_behind_some_kernel():
    named = {f for _, *own in profiling.KERNEL_SOURCES for f in own} | set(profiling.COMMON_SOURCES)
    # the codebook's levels are kernel arguments, not code
    assert {f for f in os.listdir(profiling.CSRC)} - named == {"codebook.cpp"}
