"""Softmax keys far below the largest logit, against the float64 oracle.

With a bias or sums of two scores per group the selection goes by the scores
themselves, and e^(l - max) is a float64 number down to l - max = -745: below
-708.4 it is subnormal, not 0.  The logits here are 1 or more apart, so that
two neighbouring scores differ by a factor of e and stay different where only
a few bits of a subnormal are left (e^-744 is two units of the last place).
"""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B

pytestmark = pytest.mark.gpu
SC = {"softmax": 0, "sigmoid": 1}
GS = {"max": 0, "top2": 1}


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mixture_experts_grouped_router_amd as mod
    mod.load_library()
    return mod


def check(m, lg, k, bias=None, score="softmax", n_group=1, topk_group=1,
          group_score="max", renormalize=True):
    b = None if bias is None else torch.from_numpy(bias).cuda()
    idx, w = m.moe_route_scored(
        torch.from_numpy(lg).cuda(), k, bias=b, score=SC[score],
        n_group=n_group, topk_group=topk_group, group_score=GS[group_score],
        renormalize=renormalize)
    ridx, rw = B.route_scored(lg, k, bias, score, n_group, topk_group,
                              group_score, renormalize)
    np.testing.assert_array_equal(idx.cpu().numpy(), ridx)
    # float64 inside, one rounding to float32 (half an ulp: 2^-24)
    np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=2.0 ** -23,
                               atol=1e-44)
    assert m.check_device_status() == 0
    return ridx


# 16 lanes per token (4, 8 and 16 experts per lane), one wave per token
SIZES = [8, 64, 100, 256, 300, 1024]


@pytest.mark.parametrize("ren", [True, False])
@pytest.mark.parametrize("E", SIZES)
def test_zero_bias(m, E, ren):
    lg = np.full((5, E), -5000, np.float32)
    lg[0, :4] = [0, -720, -712, -730]
    lg[1, :5] = [0, -740, -730, -720, -712]
    lg[2, -4:] = [-715, -711, -743, 0]
    lg[3] = -np.arange(E) * 100
    lg[4, ::2] = [-709 - i % 36 for i in range(E // 2)]
    lg[4, 1] = 0
    z = np.zeros(E, np.float32)
    got = check(m, lg, 2, bias=z, renormalize=ren)
    assert list(got[0]) == [0, 2]
    check(m, lg, 3, bias=z, renormalize=ren)
    check(m, lg, 8, bias=z, renormalize=ren)


@pytest.mark.parametrize("E", SIZES)
def test_masked_largest_logit(m, E):
    """The expert of the largest logit is masked: every other score is
    subnormal and the weights are a softmax over those that are chosen."""
    rng = np.random.default_rng(E)
    lg = np.full((20, E), -5000, np.float32)
    for t in range(20):
        at = rng.permutation(np.arange(1, E))[:7]
        lg[t, at] = -711 - 4 * rng.permutation(7)
    lg[:, 0] = 0
    bias = np.zeros(E, np.float32)
    bias[0] = -np.inf
    for k in (1, 2, 5):
        check(m, lg, k, bias=bias)


@pytest.mark.parametrize("E,k", [(64, 16), (256, 12), (300, 20), (1024, 32)])
def test_every_step_of_the_subnormal_range(m, E, k):
    """One logit per unit from -744 up to -700 in random places, one or two
    zeros above them."""
    rng = np.random.default_rng(k)
    for zeros in (1, 2):
        lg = np.full((30, E), -5000, np.float32)
        for t in range(30):
            p = rng.permutation(E)
            lo = 700 + rng.integers(0, 44)
            run = -np.arange(lo, 745, dtype=np.float32)
            lg[t, p[:run.size]] = run
            lg[t, p[-zeros:]] = 0
        check(m, lg, min(k, 1 + zeros), bias=np.zeros(E, np.float32))
        # (-5000 gives zeros, which tie: down to the lowest ids)
        check(m, lg, k, bias=np.zeros(E, np.float32))


@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("E,G", [(8, 4), (64, 4), (60, 5), (256, 16),
                                 (300, 5), (1024, 64)])
def test_groups_of_two_largest(m, E, G, bias):
    """Groups whose two largest scores are subnormal."""
    per = E // G
    lg = np.full((3, E), -5000, np.float32)
    lg[:, 0] = 0
    for g in range(1, G):
        for t in range(3):
            # best group: the last, the second, one in the middle
            d = [G - g, g, abs(g - G // 2)][t]
            lg[t, g * per:g * per + 2] = [-711 - 0.5 * d, -720 - 0.5 * d]
    b = np.zeros(E, np.float32) if bias else None
    for tg in (2, 3):
        check(m, lg, 4, bias=b, n_group=G, topk_group=tg, group_score="top2")


@pytest.mark.parametrize("E", [8, 128, 300])
def test_sigmoid_at_its_limit(m, E):
    """1 / (1 + e^-l) up to the largest e^-l that is a float64 number, 0
    behind it."""
    lg = np.full((2, E), -5000, np.float32)
    lg[0, :5] = [-709.79, -709.7825, -709.78, -709.5, -709]
    lg[1, -5:] = [-708, -709.7826, -709.77, -709.79, -720]
    for k in (2, 4):
        check(m, lg, k, bias=np.zeros(E, np.float32), score="sigmoid")
