"""How many digits the backward of the product of codes holds dz in, and that the
GPU tests' sizes reach every tile with either number of them."""
import os
import subprocess

import pytest
import token_plan_cases as P
import torch

from quantized_convolution_amd import token_ops as T

HERE = os.path.dirname(os.path.abspath(__file__))
F32, BF = torch.float32, torch.bfloat16


@pytest.fixture(scope="module")
def shapes(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("digits") / "token_digits_shapes")
    subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", os.path.join(HERE, "token_digits_shapes.cpp"), "-o", exe], check=True)

    def run(cases, dtype, round_dz):
        lines = "".join(f"{m} {k} {n} {int(dtype == 'bf16')} {int(round_dz)}\n" for m, k, n in cases)
        out = subprocess.run([exe], input=lines, capture_output=True, text=True, check=True).stdout.splitlines()
        assert len(out) == len(cases)
        return {w for line in out for w in line.split()}

    return run


@pytest.mark.parametrize("dtype,round_dz,planes", [("f32", False, 4), ("f32", True, 4), ("bf16", False, 4), ("bf16", True, 2)])
def test_every_tile_with_its_digits(shapes, dtype, round_dz, planes):
    got = shapes(P.BACKWARD[dtype], dtype, round_dz)
    assert not P.BACKWARD_INSTANCES - got
    assert {w for w in got if w.startswith("planes")} == {f"planes={planes}"}


def test_fewer_digits_only_where_asked_for():
    size = lambda **kw: T.Q8LinearPlan(500, 300, 200, **kw).backward_workspace_bytes  # noqa: E731
    assert not T.Q8LinearPlan(5, 3, 2, x_dtype=BF).round_dz and T.Q8LinearPlan(5, 3, 2, x_dtype=BF, round_dz=True).round_dz
    assert size(x_dtype=F32) == size(x_dtype=F32, round_dz=True) == size(x_dtype=BF) == size(x_dtype=BF, y_dtype=F32)
    assert size(x_dtype=BF, round_dz=True) < size(x_dtype=BF)
