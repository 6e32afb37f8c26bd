"""The GPU tests' sizes reach every kernel instance that they are meant to: the
launch shapes come from the plan's own source, built with the host compiler."""
import os
import subprocess

import pytest

import plan_cases as P

HERE = os.path.dirname(os.path.abspath(__file__))
TYPES = ("f32", "bf16")


@pytest.fixture(scope="module")
def shapes(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "plan_shapes")
    subprocess.run([os.environ.get("CXX", "g++"), "-O1", "-std=c++17", os.path.join(HERE, "plan_shapes.cpp"), "-o", exe], check=True)

    def run(lines):
        r = subprocess.run([exe], input="".join(line + "\n" for line in lines), capture_output=True, text=True, check=True)
        out = r.stdout.splitlines()
        assert len(out) == len(lines)
        return out

    return run


def wanted(instances):
    return {f"{t} {k}" for types, names in instances.items() for t in types.split() for k in names}


def test_norm_cases_reach_every_instance(shapes):
    got = set()
    for c, line in zip(P.NORM, shapes(["norm " + " ".join(map(str, c)) for c in P.NORM])):
        words = line.split()
        for name, batches, parts in (words[:3], words[3:]):
            more = "one" if batches == "batches=1" else "more"
            got.add(f"{TYPES[c[5]]}->{TYPES[c[6]]} {name} {more}{'' if parts == 'J=1' else ' J'}")
    assert not wanted(P.NORM_INSTANCES) - got


def test_linear_cases_reach_every_instance(shapes):
    got = set()
    lines = [f"linear {m} {k} {n} {act} {xt} {yt} 0 0 {r}" for m, k, n, act, xt, yt, r in P.LINEAR]
    for c, line in zip(P.LINEAR, shapes(lines)):
        f, dw, dx, planes = line.split()
        got |= {f"{TYPES[c[4]]} {f}", f"{TYPES[c[4]]} {dw} {planes}", f"{TYPES[c[4]]} {dx} {planes}"}
    assert not wanted(P.LINEAR_INSTANCES) - got
