"""CPU checks of the few-token layer's choice of kernels (csrc/few_plan.hpp,
compiled for the host): the sizes that the GPU tests run take the kernels that
they are there for."""
import os
import subprocess

import pytest

from few_layer_shapes import PICKS

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "mixture_experts_grouped_router_amd", "csrc")


@pytest.fixture(scope="module")
def plan(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("plan") / "few_plan_dump")
    src = os.path.join(ROOT, "tests", "native", "few_plan_dump.cpp")
    subprocess.run(["g++", "-O2", "-std=c++17", "-Wall", "-Werror", "-I",
                    CSRC, src, "-o", exe], check=True)

    def ask(lines):
        out = subprocess.run([exe], input="\n".join(lines),
                             capture_output=True, text=True, check=True)
        return [[int(v) for v in l.split()] for l in out.stdout.splitlines()]
    return ask


def test_picks(plan):
    got = plan(["%d %d" % s[:2] for s in PICKS])
    assert [bool(g[0]) for g in got] == list(PICKS.values())


def test_picking_costs_no_more_than_was_timed(plan):
    """A token's pick compares E logits with E: no size is fused whose
    comparisons exceed those of the largest that gained (2 x 256 experts)."""
    sizes = [(T, E) for T in range(1, 65) for E in range(1, 1025)]
    got = plan(["%d %d" % s for s in sizes])
    assert all(T * E * E <= 2 * 256 * 256
               for (T, E), g in zip(sizes, got) if g[0])
