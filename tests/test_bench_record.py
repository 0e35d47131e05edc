"""The counter record that bench.py reports goes by the code it was taken on:
the kernels' sources with the headers they are written in."""
import os
import shutil

import pytest

import bench

CSRC = bench.CSRC


def test_sources_take_their_headers_along():
    names = [os.path.basename(p) for p in bench.with_headers(bench.KERNEL_SRC)]
    assert names[0] == "tgemm_kernels.hip" and len(names) == len(set(names))
    assert {"tgemm_kernel.hpp", "tgemm_shapes.hpp", "tgemm_internal.hpp"} <= set(names)
    # (Headers of other folders, the C ABI's among them, are no kernel code.)
    assert all(os.path.dirname(p) == CSRC for p in bench.with_headers(bench.KERNEL_SRC))
    assert [os.path.basename(p) for p in bench.with_headers(bench.QUANT_SRC)][0] == "tgemm_quant.hip"


@pytest.mark.parametrize("changed", ["tgemm_kernels.hip", "tgemm_kernel.hpp", "tgemm_shapes.hpp"])
def test_a_change_of_code_ends_a_record_and_one_of_comments_does_not(tmp_path, changed):
    copy = tmp_path / "csrc"
    shutil.copytree(CSRC, copy)
    src = str(copy / os.path.basename(bench.KERNEL_SRC))
    assert bench.kernel_source_hash(src=src) == bench.kernel_source_hash()
    with open(copy / changed, "a") as f:
        f.write("\n\n// a comment\n/* another\n   one */\n")
    assert bench.kernel_source_hash(src=src) == bench.kernel_source_hash()
    with open(copy / changed, "a") as f:
        f.write("constexpr int kOneMore = 1;\n")
    assert bench.kernel_source_hash(src=src) != bench.kernel_source_hash()
