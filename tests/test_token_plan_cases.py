"""The GPU tests' sizes reach every kernel instance of the operators on 8-bit
codes: the launch shapes come from the plans' own source, built with the host
compiler."""
import os
import subprocess

import pytest
import token_plan_cases as P

HERE = os.path.dirname(os.path.abspath(__file__))


@pytest.fixture(scope="module")
def shapes(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "token_plan_shapes")
    subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", os.path.join(HERE, "token_plan_shapes.cpp"), "-o", exe], check=True)

    def run(lines):
        r = subprocess.run([exe], input="".join(line + "\n" for line in lines), capture_output=True, text=True, check=True)
        out = r.stdout.splitlines()
        assert len(out) == len(lines)
        return out

    return run


def test_forward_cases_reach_every_instance(shapes):
    got = {line.split()[0][2:] for line in shapes([f"q8linear {m} {k} {n} 1" for m, k, n in P.FORWARD])}
    assert not P.FORWARD_INSTANCES - got


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_backward_cases_reach_every_instance(shapes, dtype):
    lines = shapes([f"q8linear {m} {k} {n} {int(dtype == 'bf16')}" for m, k, n in P.BACKWARD[dtype]])
    assert not P.BACKWARD_INSTANCES - {w for line in lines for w in line.split()[1:]}


def test_row_cases_reach_every_instance(shapes):
    got = {w for line in shapes([f"rows 5 {c}" for c in P.ROWS]) for w in line.split()}
    assert not P.ROWS_INSTANCES - got
