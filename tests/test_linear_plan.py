"""CPU checks of the linear layer's planner (csrc/linear_plan.hpp, compiled
for the host): the sizes that the GPU tests run take the tiles, splits and
launch forms that they are there for, and every form is among them."""
import os
import subprocess

import pytest

from linear_tile_shapes import BACKWARD, FEW_ROWS, FORWARD

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixture_experts_grouped_router_amd", "csrc")
TILES = [(256, 256), (128, 128), (64, 128), (64, 64)]


@pytest.fixture(scope="module")
def plans(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "linear_plan_dump")
    src = os.path.join(ROOT, "tests", "native", "linear_plan_dump.cpp")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-I",
                    CSRC, src, "-o", exe], check=True)
    sizes = [*FORWARD, *BACKWARD, *FEW_ROWS]
    out = subprocess.run([exe], input="\n".join("%d %d %d" % s
                                                for s in sizes),
                         capture_output=True, text=True, check=True).stdout
    lines = out.splitlines()
    assert len(lines) == len(sizes)
    return {s: [int(v) for v in l.split()]
            for s, l in zip(sizes, lines)}


@pytest.mark.parametrize("size", FORWARD)
def test_forward(plans, size):
    v = plans[size]
    assert not v[0] and tuple(v[1:4]) == FORWARD[size]


@pytest.mark.parametrize("size", BACKWARD)
def test_backward(plans, size):
    v = plans[size]
    assert (bool(v[4]), tuple(v[6:9]), tuple(v[9:12])) == BACKWARD[size]
    # one gradient alone: the same tile and split
    assert v[12:15] == v[6:9] and v[15:18] == v[9:12]


@pytest.mark.parametrize("size", FEW_ROWS)
def test_few_rows(plans, size):
    assert bool(plans[size][0]) == FEW_ROWS[size]


def test_every_form_is_there():
    f = {(p[:2], p[2] > 1) for p in FORWARD.values()}
    assert f == {(t, s) for t in TILES for s in (False, True)}
    b = {(x[:2], j) for j, x, _ in BACKWARD.values()}
    assert b == {(t, j) for t in TILES for j in (False, True)}
    for t in TILES:   # split partials of dx and of dW next to the others
        joint = [(x[2] > 1, w[2] > 1) for j, x, w in BACKWARD.values()
                 if j and x[:2] == t]
        assert any(x for x, _ in joint) and any(w for _, w in joint), t
    w = {p[:2] for j, _, p in BACKWARD.values() if not j}
    assert w == set(TILES)
