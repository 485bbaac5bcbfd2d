"""The host-side rules of the optimiser, on the CPU: those of its launches,
compiled from the library's own header with the host's compiler, and the
formulas that the public header states."""
import math
import os
import re
import subprocess

import numpy as np
import pytest

import train_oracle as O
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


def test_the_headers_formulas_give_the_step_its_bits():
    """The four lines that fff.h writes for an AdamW step, evaluated as they
    stand in 32 bits, give the bits of the form the GPU's are compared with."""
    with open(os.path.join(hipbuild.INCLUDE, "fff.h")) as f:
        text = f.read()
    text = text[text.index("AdamW (decoupled weight decay)"):]
    found = re.findall(r"^ \*   (\w+) = (.*)$", text, re.M)
    lines = [(k, v) for k, v in found[:4]]
    consts = [(k, v) for k, v in found[4:7]]
    assert [k for k, _ in lines] == ["g", "m", "v", "p"]
    assert [k for k, _ in consts] == ["decay", "step_size", "root"]

    kw = dict(lr=3e-3, beta1=0.9, beta2=0.99, eps=1e-8, wd=0.1, step=7)
    names = {"lr": kw["lr"], "weight_decay": kw["wd"], "sqrt": math.sqrt,
             **{k: kw[k] for k in ("beta1", "beta2", "step")}}
    at = {k: np.float32(eval(v.replace("^", "**"), {}, names)) for k, v in consts}
    at.update({k: np.float32(kw[k]) for k in ("beta1", "beta2", "eps")})
    at.update(one_beta1=np.float32(1 - kw["beta1"]), one_beta2=np.float32(1 - kw["beta2"]), sqrt=np.sqrt)

    rng = np.random.default_rng(5)
    n = 100_000
    p, grad, m = (rng.normal(size=n).astype(np.float32) for _ in range(3))
    v = rng.random(n).astype(np.float32)
    want = O.adamw(p, grad, m, v, gs=0.37, **kw)
    at.update(p=p, grad=grad, m=m, v=v, grad_scale=np.float32(0.37))
    for k, line in lines:
        line = line.replace("(1 - beta1)", "one_beta1").replace("(1 - beta2)", "one_beta2")
        at[k] = eval(line, {}, at)
        assert at[k].dtype == np.float32
    for k in "pmv":
        assert np.array_equal(at[k], want[k]), k
