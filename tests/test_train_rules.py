"""The host-side rules of the optimiser's launches, compiled from the
library's own header with the host's compiler and run on the CPU."""
import os
import subprocess

import pytest

from sparse_tree_structured_amd import build as hipbuild

PROGRAM = """
#include <cstdio>
#include <cstdlib>
#include "launch_train.hpp"
int main(int, char** v) {
  std::printf("%d", int(fff::adamw_streams(std::atoi(v[1]), std::atoi(v[2]), v[3][0] == '1', v[4][0] == '1')));
}
"""


@pytest.fixture(scope="module")
def program(tmp_path_factory):
    where = tmp_path_factory.mktemp("rules")
    src, exe = where / "rules.cpp", where / "rules"
    src.write_text(PROGRAM)
    rocm = os.path.dirname(os.path.dirname(os.path.realpath(hipbuild.hipcc())))
    # (a sanitizer of arithmetic: an overflow ends the program with an error)
    subprocess.run(["g++", "-std=c++17", "-fsanitize=signed-integer-overflow", "-fno-sanitize-recover=all",
                    "-D__HIP_PLATFORM_AMD__", "-I", os.path.join(rocm, "include"),
                    "-I", hipbuild.CSRC, "-w", str(src), "-o", str(exe)], check=True)

    def run(blocks, param, grad_bf16, state_e4m3):
        r = subprocess.run([str(exe), str(blocks), str(param), str(int(grad_bf16)), str(int(state_e4m3))],
                           check=True, capture_output=True, text=True)
        return r.stdout == "1"
    return run


# (a param's kind: 0 float32, 1 bf16, 2 bf16 with a master; bytes of an element that a step reads and writes)
EACH = {(0, False, False): 28, (1, False, False): 24, (2, False, False): 30, (2, True, False): 28,
        (0, False, True): 16, (1, True, True): 10, (2, False, True): 18}


@pytest.mark.parametrize("kind", EACH, ids=str)
def test_a_large_launch_streams_whatever_its_size(program, kind):
    """160 MB and more: up to the most workgroups of a launch, of 2048
    elements each.  2^20 of them have 2^31 elements."""
    edge = -(-(160 << 20) // (2048 * EACH[kind]))
    assert not program(1, *kind) and not program(edge - 1, *kind) and program(edge, *kind)
    for blocks in ((1 << 20) - 1, 1 << 20, (1 << 20) + 1, (1 << 21) - 1, 1 << 21, (1 << 21) + 1, 3 << 20, 1 << 23,
                   (1 << 24) - 1):
        assert program(blocks, *kind), blocks
