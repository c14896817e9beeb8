"""The logit gradient where a slot's expert id is outside [0, E): the slot
contributes nothing, whatever its weight gradient holds."""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mixture_experts_grouped_router_amd as mod
    mod.load_library()
    return mod


@pytest.mark.parametrize("ren", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(12, 4), (200, 8), (300, 9), (1024, 32)])
def test_slots_that_name_no_expert(m, E, k, score, ren):
    rng = np.random.default_rng(E + k)
    T = 9
    lg = rng.standard_normal((T, E)).astype(np.float32)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    idx = B.route_scored(lg, k, score=score)[0]
    bad = np.zeros((T, k), bool)
    bad[1, 0] = bad[4, k - 1] = bad[5, 1] = True
    bad[7, ::2] = True
    bad[8] = True                          # nothing is left of this token
    ids = np.array([-1, E, 2 ** 31 - 1, -2 ** 31], np.int32)
    junk = np.array([np.nan, np.inf, -np.inf, 1.0], np.float32)
    n = int(bad.sum())
    idx_b, dw_b = idx.copy(), dw.copy()
    idx_b[bad] = np.resize(ids, n)
    dw_b[bad] = np.resize(junk, n)
    got = m.moe_route_scored_bwd(
        torch.from_numpy(lg).cuda(), torch.from_numpy(idx_b).cuda(),
        torch.from_numpy(dw_b).cuda(),
        score={"softmax": 0, "sigmoid": 1}[score],
        renormalize=ren).cpu().numpy()
    assert m.check_device_status() == 1
    for t in range(T):
        keep = ~bad[t]
        want = np.zeros(E) if not keep.any() else B.route_scored_bwd(
            lg[t:t + 1], idx[t:t + 1, keep], dw[t:t + 1, keep], score, ren)[0]
        # float64 inside, one rounding to float32; the gradients are
        # differences of terms of dw's size
        assert np.all(np.abs(got[t] - want) <= 2.0 ** -23 * np.abs(want) +
                      1e-13 * np.abs(dw).max()), t
