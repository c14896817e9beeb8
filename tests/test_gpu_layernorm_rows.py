"""Layer norm with more rows than one round of the grid, in each width of rows
and type: waves and work-groups that take several, loaded ahead of the
reductions.  Bounds as in test_gpu_layernorm.py."""
import pytest
import torch

from test_gpu_layernorm import check_bwd, check_fwd, dev, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mixture_experts_grouped_router_amd as mod
    mod.load_library()
    return mod


# a round is 4096 rows up to H = 1024, 1024 up to 4096, 512 up to 8192, else
# 256 forward; at most 2048, 512, 256 and 256 backward (1024 for H 513..1024)
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,H", [(9001, 8), (9001, 96), (8193, 501),
                                 (5000, 768), (4100, 1023), (2300, 1040),
                                 (2100, 2304), (1100, 4095), (600, 5001),
                                 (530, 8192), (270, 8200), (513, 16384)])
def test_several_rounds(m, T, H, f32):
    d = make(T, H, f32, T)
    got = check_fwd(m, d)
    check_bwd(m, d, got)
    # a row's results do not depend on the rows before it
    one = m.moe_layernorm_fwd(dev(d["x"][-1:]), dev(d["w"]), dev(d["b"]))
    assert torch.equal(got["y"][-1:], one["y"])
