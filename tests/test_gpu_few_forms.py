"""The few-token layer's forms on the GPU: each choice of kernels that
csrc/few_plan.hpp makes, at the sizes of few_layer_shapes.py."""
import numpy as np
import pytest
import torch

from few_layer_shapes import PICKS
from oracle import moe_oracle as O
from test_gpu_layer_few import bf, check, make, up, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mixture_experts_grouped_router_amd as mod
    mod.load_library()
    return mod


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("T,E,k", PICKS)
def test_picked_experts(m, T, E, k, renorm):
    """Experts and weights against the oracle on the separate entry point's
    logits, and the layer's outputs; with equal logits too: experts share
    rows of the router, and one token's are all equal."""
    d = make(T, 64, 32, E, k, 100 * T + E)
    check(m, d, "bf16", router=True, renorm=renorm, bias=True)
    d["wr"][E // 2:] = d["wr"][:E - E // 2]
    d["x"][T - 1] = 0
    kw, _, _ = weights(m, d, "bf16")
    r = m.moe_layer_few(bf(d["x"]), w_r=bf(d["wr"]), k=k, renormalize=renorm,
                        **kw)
    lg = m.moe_router_logits(bf(d["x"]), bf(d["wr"])).cpu().numpy()
    idx, w = O.route_topk(lg, k, renorm)
    np.testing.assert_array_equal(r["topk_idx"].cpu().numpy(), idx)
    assert list(idx[T - 1]) == list(range(k))
    np.testing.assert_allclose(r["topk_w"].cpu().numpy(), w, rtol=2.0 ** -23)
    assert m.check_device_status() == 0
    given = m.moe_layer_few(bf(d["x"]), topk_idx=r["topk_idx"],
                            topk_w=r["topk_w"], **kw)
    assert torch.equal(r["y"], given["y"])
