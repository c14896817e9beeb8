"""CPU checks of the few-token layer's choice of kernels (csrc/few_plan.hpp,
compiled for the host): the sizes that the GPU tests run take the kernels that
they are there for."""
import os
import subprocess

import pytest

from few_layer_shapes import FORMS, PICKS

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
    got = plan(["pick %d %d" % s[:2] for s in PICKS])
    assert [bool(g[0]) for g in got] == list(PICKS.values())


def test_picking_costs_no_more_than_was_timed(plan):
    """A token's pick compares E logits with E: no size is fused whose
    comparisons exceed those of the largest that gained (2 x 256 experts)."""
    sizes = [(T, E) for T in range(1, 65) for E in range(1, 1025)]
    got = plan(["pick %d %d" % s for s in sizes])
    assert all(T * E * E <= 2 * 256 * 256
               for (T, E), g in zip(sizes, got) if g[0])


def ask_forms(plan, sizes):
    return plan(["form %d %d %d %d %d %d %d" %
                 (*s[:5], s[5] == "mxfp4", s[6]) for s in sizes])


def test_forms(plan):
    got = ask_forms(plan, FORMS)
    assert {s: (bool(g[0]), g[1], g[2], bool(g[3]))
            for s, g in zip(FORMS, got)} == FORMS


def test_every_form_is_there(plan):
    """Of all the sizes that the entry point takes (a sample), none has a form
    that FORMS lacks."""
    sizes = [(T, H, F, E, k, fmt, True)
             for T in (1, 2, 3, 5, 8, 16, 17, 31, 33, 48, 64)
             for H in (96, 128) for F in (32, 128, 800, 4096, 16384)
             for E in (1, 2, 8, 40, 128, 1024)
             for k in (1, 2, 8, 32) if k <= E
             for fmt in ("bf16", "mxfp4")]
    key = lambda s, g: (s[5], *[int(v) for v in g[:4]])
    have = {key(s, v) for s, v in FORMS.items()}
    assert {key(s, g) for s, g in zip(sizes, ask_forms(plan, sizes))} == have
    # every instance of layer_few.hip's table; bf16 with one column set has
    # no form with a wave per item
    assert len(have) == 2 * 4 + 2 * 2 + 5


def test_work_groups(plan):
    """One round of what the chip holds at once, at most an item each."""
    for s, g in zip(FORMS, ask_forms(plan, FORMS)):
        T, _, F, E, k, fmt, _ = s
        cols = 16 if fmt == "mxfp4" else 8
        items = min(T * k, E) * -(-F // cols)
        full = g[1] * g[2] == (16 if fmt == "mxfp4" else 32)
        assert g[4] == min(items, 256 * (2 if g[3] or full else 3))
