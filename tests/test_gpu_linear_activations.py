"""The activations and their derivatives at every finite bf16 value, relative
to their size, against float64.

A layer of one output whose weights are (1, 0, ...): y is act(z) and dx[:, 0]
act'(z), each rounded to bf16 once (the product with 1 is exact).  The
derivative is the sum of two float32 terms, e.g. Phi(z) and z phi(z), each a product that starts
from an exponential of an argument of up to 104.  With u = 2^-24, rounding that
argument (and its multiple of log2 e) is off by 2 u of it, which multiplies the
exponential by 1 +- 2 * 104 u; the cubic of the tanh form has four roundings
more (6 * 104 u); the other factors add less than 32 u: 2^-14 of each term is
more than all of it.  Where both terms are below the normal float32 numbers
(2^-126, times |z| up to 104) nothing is asked of them: hardware reciprocals
flush there.
"""
import numpy as np
import pytest
import torch
from scipy.special import ndtr

from oracle import block_oracle as B
from synthetic import bf16_to_f64

pytestmark = pytest.mark.gpu
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
HALF = 2.0 ** -8 * 1.01
FLUSHED = 2.0 ** -126 * 105


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mixture_experts_grouped_router_amd as mod
    mod.load_library()
    return mod


def terms(act, z):
    """Sum of the sizes of the derivative's two terms."""
    if act == "gelu":
        return ndtr(z) + np.abs(z) * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    if act == "gelu_tanh":
        c = 2 * np.sqrt(2 / np.pi)
        s, r = (B.scores_of(f * c * (z + 0.044715 * z ** 3)) for f in (1, -1))
        return s + np.abs(z) * s * r * c * (1 + 3 * 0.044715 * z * z)
    s = B.scores_of(z)
    return s * (1 + np.abs(z) * (1 - s))


@pytest.mark.parametrize("act", ACTS[1:])
def test_every_bf16_value(m, act):
    bits = np.arange(1 << 16, dtype=np.uint16)
    with np.errstate(invalid="ignore"):   # signalling NaN patterns
        z = bf16_to_f64(bits)
    bits = bits[np.isfinite(z)]
    z = z[np.isfinite(z)]
    M = bits.size
    zt = torch.from_numpy(bits.view(np.int16)).view(torch.bfloat16).cuda()
    one = torch.ones((M, 1), dtype=torch.bfloat16, device="cuda")
    w = torch.zeros((1, 8), dtype=torch.bfloat16, device="cuda")
    w[0, 0] = 1
    # the activation itself: one term
    y = m.moe_linear_fwd(torch.nn.functional.pad(zt.view(M, 1), (0, 7)), w,
                         act=ACTS.index(act))["y"][:, 0]
    want = B.act(act, z)
    tol = HALF * np.abs(want) + 1.01 * 2.0 ** -14 * np.abs(want) + FLUSHED
    bad = ~(np.abs(y.double().cpu().numpy() - want) <= tol)
    assert not bad.any(), [(z[i], float(y[i]), want[i]) for i in
                           np.nonzero(bad)[0][:8]]
    got = m.moe_linear_bwd(one, None, w, act=ACTS.index(act),
                           z=zt.view(M, 1), want_dw=False)["dx"]
    assert bool((got[:, 1:] == 0).all())
    got = got[:, 0].double().cpu().numpy()
    with np.errstate(over="ignore", invalid="ignore", under="ignore"):
        want = B.act_grad(act, z)
        size = np.abs(want) if act == "relu" else terms(act, z)
    # beyond |z| = 200 the formulas overflow in float64: 0 or 1
    far = np.abs(z) > 200
    want[far] = z[far] > 0
    size[far] = want[far]
    tol = HALF * np.abs(want) + 1.01 * 2.0 ** -14 * size + FLUSHED
    bad = ~(np.abs(got - want) <= tol)
    assert not bad.any(), [(z[i], got[i], want[i]) for i in
                           np.nonzero(bad)[0][:8]]
