"""The few-token layer's forms on the GPU: each choice of kernels that
csrc/few_plan.hpp makes, at the sizes of few_layer_shapes.py."""
import numpy as np
import pytest
import torch

from few_layer_shapes import FORMS, PICKS
from oracle import moe_oracle as O
import test_gpu_layer_few as few
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


@pytest.mark.parametrize("T,H,F,E,k,fmt,dwords", FORMS)
def test_forms(m, T, H, F, E, k, fmt, dwords, monkeypatch):
    """Experts as drawn, then with most pairs on one of them (it makes several
    entries), one named twice by a token and one id that is none."""
    d = make(T, H, F, E, k, 7 * T + F)
    kw, gu, dn = weights(m, d, fmt)
    if not dwords:
        for n in ("w_gu_q", "w_dn_q"):
            c, s = kw[n]
            buf = torch.empty(s.numel() + 1, dtype=torch.uint8, device="cuda")
            buf[1:] = s.reshape(-1)
            kw[n] = (c, buf[1:].view(s.shape))
    # (the oracle's weights once)
    monkeypatch.setattr(few, "weights", lambda m, d, fmt: (dict(kw), gu, dn))
    check(m, d, fmt)
    d["idx"][: T // 2 + 1, 0] = E // 2
    if k > 1:
        d["idx"][T - 1, :2] = 0
        d["idx"][T // 2, 1] = -1
        d["w"][T // 2, 1] = np.nan
    check(m, d, fmt, res=False)
    assert m.check_device_status() == (1 if k > 1 else 0)
