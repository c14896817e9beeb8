"""CPU check of the persistent kernels whose grids are whole rounds of what a
compute unit holds: the compiler reports that many waves per SIMD (a work-group
of four waves is one wave on each of a unit's four SIMDs), without scratch."""
import os
import re
import shutil
import subprocess

import pytest

from mixture_experts_grouped_router_amd import build

pytestmark = pytest.mark.skipif(
    shutil.which(build.HIPCC) is None and not os.path.exists(build.HIPCC),
    reason="no hipcc")


def kernels(name):
    """{kernel with its template arguments: (waves per SIMD, scratch bytes)}"""
    src = os.path.join(build.CSRC, name)
    r = subprocess.run([build.HIPCC, *build.COMMON, *build.DEVICE_FLAGS,
                        "--cuda-device-only", "-S",
                        "-Rpass-analysis=kernel-resource-usage", src, "-o",
                        os.devnull], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr[-2000:]
    out = {}
    for b in r.stderr.split("Function Name: ")[1:]:
        n = subprocess.run(["c++filt", b.split()[0]], capture_output=True,
                           text=True, check=True).stdout.strip()
        n = re.sub(r"^void |moe::|\(anonymous namespace\)::", "", n)
        num = lambda key: int(re.search(re.escape(key) + r": (\d+)",
                                        b).group(1))
        out[n.split("(")[0]] = (num("Occupancy [waves/SIMD]"),
                                num("ScratchSize [bytes/lane]"))
    return out


def test_mxfp4_few_rows():
    k = kernels("mxfp4_few_rows.hip")
    for ns in (1, 2):
        for name, per_cu in (("true, 8", 2), ("false, 4", 3)):
            waves, scratch = k["mx4_few_rows_kernel<%s, %d>" % (name, ns)]
            assert waves >= per_cu and scratch == 0, (name, ns)


def test_layer_few():
    """The gate/up kernels: three work-groups per unit, two with a wave per
    item or with the most columns (few_per_cu of few_plan.hpp)."""
    k = {n: v for n, v in kernels("layer_few.hip").items()
         if n.startswith("few_gate_up_kernel")}
    assert len(k) == 17
    for name, (waves, scratch) in k.items():
        fmt, ct, ns, _, ks, _ = [a.strip() for a in
                                 name[name.index("<") + 1:-1].rsplit(",", 5)]
        full = int(ct) * int(ns) == (32 if "Bf16" in fmt else 16)
        assert scratch == 0 and waves >= (2 if ks == "1" or full else 3), name
