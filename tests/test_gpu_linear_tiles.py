"""Every tile, split and launch form of the dense linear layer on the GPU, at
sizes that end inside a tile (test_linear_plan.py asserts which form each size
takes), against the formulas in float64 torch operations.

Element-wise bounds, u = 2^-24, a bf16 rounding off by at most 2^-8:
 * z: exact float32 products, K + 1 additions and up to 16 of split partials
   or K groups, each off by u of a partial sum of at most A = sum |x w| + |b|;
 * y: z's error times the activation's slope (below 1.13), 2^-18 |z| for the
   activation itself (hardware exponential and reciprocal), one addition of
   the residual, one bf16 rounding;
 * dz: exact without an activation; else 2^-18 |dy| (1 + |z|) from the
   derivative and its bf16 rounding; db sums the unrounded values;
 * dx, dW: dz's error times the other operand, u per addition, one rounding.
"""
import math

import pytest
import torch

from linear_tile_shapes import BACKWARD, FEW_ROWS, FORWARD

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = 2.0 ** -8 * 1.01
NONE, RELU, GELU, GELU_TANH, SILU = range(5)


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mixture_experts_grouped_router_amd as mod
    mod.load_library()
    return mod


def act64(act, z):
    """(activation, derivative) in float64."""
    if act == NONE:
        return z, torch.ones_like(z)
    if act == RELU:
        return z.clamp(min=0), (z > 0).double()
    if act == GELU:
        c = torch.special.ndtr(z)
        return z * c, c + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    if act == GELU_TANH:
        c = 2 * math.sqrt(2 / math.pi)
        s = torch.sigmoid(c * (z + 0.044715 * z ** 3))
        r = torch.sigmoid(-c * (z + 0.044715 * z ** 3))
        return z * s, s + z * s * r * c * (1 + 3 * 0.044715 * z * z)
    s = torch.sigmoid(z)
    return z * s, s * (1 + z * (1 - s))


def inputs(M, N, K, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(shape, std=1.0):
        return torch.randn(shape, generator=g, device="cuda") * std
    return {"x": normal((M, K)).bfloat16(),
            "w": normal((N, K), K ** -0.5).bfloat16(), "b": normal((N,)),
            "r": normal((M, N)).bfloat16(), "dy": normal((M, N)).bfloat16(),
            "z": normal((M, N), 1.5).bfloat16()}


def within(got, want, tol, what):
    bad = (got.double() - want).abs() > tol
    n = int(bad.sum())
    assert n == 0 and bool(torch.isfinite(got).all()), \
        (what, n, torch.nonzero(bad)[:4].tolist())


def product64(d):
    """x W^T and sum |x w|."""
    x, wt = d["x"].double(), d["w"].double().t().contiguous()
    return x @ wt, x.abs() @ wt.abs()


def check_forward(m, d, zp, A, act, bias, res, save):
    K = d["x"].shape[1]
    z = zp + d["b"].double() if bias else zp
    ez = (K + 17) * U * (A + d["b"].double().abs() if bias else A)
    y = act64(act, z)[0]
    ey = 1.13 * ez
    if act not in (NONE, RELU):
        ey = ey + 2.0 ** -18 * z.abs()
    if res:
        r = d["r"].double()
        y = y + r
        ey = ey + U * (y.abs() + r.abs())
    out = m.moe_linear_fwd(d["x"], d["w"], bias=d["b"] if bias else None,
                           act=act, residual=d["r"] if res else None,
                           save=save)
    within(out["y"], y, HALF * y.abs() + 1.01 * ey, "y")
    if save:
        within(out["z"], z, HALF * z.abs() + 1.01 * ez, "z")
    return out


@pytest.mark.parametrize("M,N,K", FORWARD)
def test_forward(m, M, N, K):
    d = inputs(M, N, K, M + N)
    zp, A = product64(d)
    for act in range(5):
        check_forward(m, d, zp, A, act, bias=True, res=True, save=True)
        check_forward(m, d, zp, A, act, bias=act % 2 == 0, res=act % 2 == 1,
                      save=act == GELU)
    check_forward(m, d, zp, A, NONE, bias=False, res=False, save=False)


@pytest.mark.parametrize("M,N,K", FEW_ROWS)
def test_few_rows(m, M, N, K):
    """Dot products of one and two rows, a wave or a work-group per row of W,
    and the matrix form up to 16 rows: rows of W that end inside a block, K
    tails in the first, a later and the last trip, and the sizes just past
    what these forms take."""
    d = inputs(M, N, K, M * 3 + N)
    zp, A = product64(d)
    for act in range(5):
        check_forward(m, d, zp, A, act, bias=True, res=True, save=True)
    check_forward(m, d, zp, A, SILU, bias=False, res=False, save=False)
    # in place on the residual
    want = check_forward(m, d, zp, A, GELU, True, True, False)["y"]
    r = d["r"].clone()
    m.moe_linear_fwd(d["x"], d["w"], bias=d["b"], act=GELU, residual=r, out=r)
    assert torch.equal(r, want)


def check_backward(m, d, act):
    M, N = d["dy"].shape
    dy, z = d["dy"].double(), d["z"].double()
    dz = dy * act64(act, z)[1]
    e = torch.zeros_like(dz) if act in (NONE, RELU) else \
        2.0 ** -18 * dy.abs() * (1 + z.abs())
    adz = dz.abs()
    edz = e if act == NONE else e + HALF * (adz + e)
    x, w = d["x"].double(), d["w"].double()
    g = m.moe_linear_bwd(d["dy"], d["x"], d["w"], act=act,
                         z=None if act == NONE else d["z"], want_db=True)
    s = 1.02 * U * (adz + edz)
    ref = dz @ w
    within(g["dx"], ref, HALF * ref.abs() +
           (1.01 * edz + (N + 17) * s) @ w.abs(), "dx")
    ref = dz.t().contiguous() @ x
    within(g["dw"], ref, HALF * ref.abs() +
           (1.01 * edz + (M + 17) * s).t().contiguous() @ x.abs(), "dw")
    within(g["db"], dz.sum(0), 1.01 * e.sum(0) +
           (M + 17) * U * (adz + e).sum(0), "db")
    return g


@pytest.mark.parametrize("act", [NONE, SILU])
@pytest.mark.parametrize("M,N,K", BACKWARD)
def test_backward(m, M, N, K, act):
    """Without an activation nothing but the sums is rounded, so that a lost
    K tail shows; and with one."""
    d = inputs(M, N, K, M * 5 + N)
    g = check_backward(m, d, act)
    # each gradient alone: the same bits
    z = None if act == NONE else d["z"]
    dx = m.moe_linear_bwd(d["dy"], None, d["w"], act=act, z=z,
                          want_dw=False)["dx"]
    dw = m.moe_linear_bwd(d["dy"], d["x"], None, act=act, z=z,
                          want_dx=False)["dw"]
    assert torch.equal(dx, g["dx"]) and torch.equal(dw, g["dw"])


def inside(t, fill=float("nan")):
    """A copy of t cut out of a larger buffer full of NaN."""
    buf = torch.full((t.numel() + 8192,), fill, dtype=t.dtype, device="cuda")
    v = buf[4096:4096 + t.numel()].view(t.shape)
    v.copy_(t)
    return buf, v


@pytest.mark.parametrize("M,N,K", [(909, 12569, 424), (909, 12544, 424),
                                   (587, 6699, 4632), (1500, 2100, 1032),
                                   (1500, 2048, 1032), (2779, 137, 4936)])
def test_forward_neighbours(m, M, N, K):
    """Large tiles: nothing behind the inputs is read into a result, nothing
    around the outputs is written, the output may be the residual, and a NaN
    row of x or W stays in its own row or column."""
    d = inputs(M, N, K, 9)
    base = m.moe_linear_fwd(d["x"], d["w"], bias=d["b"], act=SILU,
                            residual=d["r"], save=True)
    buf, r = inside(d["r"], 3.0)
    got = m.moe_linear_fwd(inside(d["x"])[1], inside(d["w"])[1], bias=d["b"],
                           act=SILU, residual=r, save=True, out=r)
    assert torch.equal(got["y"], base["y"]) and torch.equal(got["z"],
                                                            base["z"])
    assert bool((buf[:4096] == 3).all()) and bool((buf[-4096:] == 3).all())
    i, j = M - 2, N - 2
    d["x"][i] = float("nan")
    d["w"][j] = float("inf")
    y = m.moe_linear_fwd(d["x"], d["w"], bias=d["b"], act=SILU,
                         residual=d["r"])["y"]
    keep = torch.ones((M, N), dtype=torch.bool, device="cuda")
    keep[i] = False
    keep[:, j] = False
    assert torch.equal(y[keep], base["y"][keep])
    assert bool(torch.isnan(y[i]).all())


@pytest.mark.parametrize("M,N,K", [(1537, 8193, 520), (10157, 651, 536),
                                   (3665, 4521, 392), (4443, 543, 520),
                                   (769, 12817, 1032), (10491, 555, 1416)])
def test_backward_neighbours(m, M, N, K):
    """Large tiles: inputs inside buffers of NaN and a workspace that held
    NaN give the same gradients."""
    d = inputs(M, N, K, 10)
    for act in (NONE, GELU_TANH):
        z = None if act == NONE else d["z"]
        want = m.moe_linear_bwd(d["dy"], d["x"], d["w"], act=act, z=z,
                                want_db=True)
        ws = torch.full((1 << 29,), 255, dtype=torch.uint8, device="cuda")
        got = m.moe_linear_bwd(inside(d["dy"])[1], inside(d["x"])[1],
                               inside(d["w"])[1], act=act,
                               z=None if z is None else inside(z)[1],
                               want_db=True, ws=ws)
        for n in want:
            assert torch.equal(got[n], want[n]), (n, act)


def whole_numbers(M, N, K, seed):
    """Operands from -2 to 2: every sum below 2^24 is exact in float32, so the
    outputs are the exact values rounded to bf16 once, whatever the order, and
    a single lost or doubled term shows."""
    g = torch.Generator(device="cuda").manual_seed(seed)

    def some(shape, dtype=torch.bfloat16):
        return torch.randint(-2, 3, shape, generator=g,
                             device="cuda").to(dtype)
    return {"x": some((M, K)), "w": some((N, K)), "dy": some((M, N)),
            "r": some((M, N)), "b": some((N,), torch.float32)}


@pytest.mark.parametrize("M,N,K", [*FORWARD, *FEW_ROWS])
def test_forward_exact(m, M, N, K):
    d = whole_numbers(M, N, K, M + K)
    z = d["x"].double() @ d["w"].double().t().contiguous() + d["b"].double()
    got = m.moe_linear_fwd(d["x"], d["w"], bias=d["b"], act=RELU,
                           residual=d["r"], save=True)
    y = z.clamp(min=0) + d["r"].double()
    assert float(z.abs().max()) < 2 ** 23
    assert torch.equal(got["z"], z.float().bfloat16())
    assert torch.equal(got["y"], y.float().bfloat16())


@pytest.mark.parametrize("M,N,K", [*BACKWARD])
def test_backward_exact(m, M, N, K):
    d = whole_numbers(M, N, K, N + K)
    dy = d["dy"].double()
    got = m.moe_linear_bwd(d["dy"], d["x"], d["w"], want_db=True)
    dx = dy @ d["w"].double()
    dw = dy.t().contiguous() @ d["x"].double()
    assert float(dx.abs().max()) < 2 ** 23 > float(dw.abs().max())
    assert torch.equal(got["dx"], dx.float().bfloat16())
    assert torch.equal(got["dw"], dw.float().bfloat16())
    assert torch.equal(got["db"], dy.sum(0).float())
