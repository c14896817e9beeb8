"""The MXFP4 expert MLP around the border between its kernels for few rows and
its tiled ones (sixteen rows per expert on average)."""
import pytest
import torch

from oracle import moe_oracle as O
from test_gpu_mxfp4 import host, make, oracle, run

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mixture_experts_grouped_router_amd as mod
    mod.load_library()
    return mod


# entries that are full, hold one row more, or none; on both sides of the
# border, the last K step whole and half
@pytest.mark.parametrize("sizes,H,F", [
    ([16] * 6, 256, 384), ([15, 17, 16, 0, 32], 384, 128), ([13] * 5, 128, 640),
    ([16, 16, 15, 17], 2048, 256), ([0, 33, 31, 0], 640, 768),
    ([96, 0, 0, 0, 0, 0], 384, 256), ([17] * 3, 256, 128),
    ([16, 17, 16], 384, 384), ([49, 0, 0], 128, 256)])
def test_mlp(m, sizes, H, F):
    """As test_gpu_mxfp4.py: 5e-3 is one bf16 rounding and the few elements of
    a that fall on the other side of a rounding border."""
    d = make(sizes, H, F, H + F)
    ref = oracle(d)["z"]
    z = [run(m, d, mode)["z"] for mode in ("bf16 weights", "weight codes",
                                           "codes")]
    assert O.rel_err(host(z[0]), ref) < 5e-3
    assert torch.equal(z[0], z[1]) and torch.equal(z[0], z[2])
    tiled = run(m, d, "codes", save=True)["z"]
    assert O.rel_err(host(tiled), ref) < 5e-3


def test_misaligned_workspace_is_refused(m):
    d = make([3, 40], 256, 128, 3)
    ref = run(m, d, "codes")["z"]
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    for at in (1, 4, 8):
        with pytest.raises(m.MoEError):
            run(m, d, "codes", ws=ws[at:])
    assert torch.equal(run(m, d, "codes", ws=ws[16:])["z"], ref)
