"""The dense linear layer on the GPU against the float64 oracle.

Element-wise bounds, from the arithmetic (u = 2^-24; a bf16 rounding is off
by at most 2^-8 of the value):
 * z: K products are exact in float32, their sum and the bias are K + 1
   additions, each off by u of a partial sum, at most u (K + 1) A with
   A = sum |x w| + |b|; the split partials are additions of the same kind.
 * y: z's error times the activation's slope (below 1.13), the activation's
   own error (2^-18 of |z|: hardware exponential and reciprocal of an
   argument up to about 90), one residual addition, one bf16 rounding.
 * dz: 2^-18 |dy| (1 + |z|) from the derivative, plus its bf16 rounding where
   it feeds dx and dw; db sums the unrounded float32 values.
 * dx, dw: the operands' errors times the other operand, the additions'
   rounding, one bf16 rounding.
"""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B
from synthetic import bf16_bits, bf16_to_f64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = 2.0 ** -8 * 1.01
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mixture_experts_grouped_router_amd as mod
    mod.load_library()
    return mod


def dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(
        torch.bfloat16).cuda()


def host(t):
    return bf16_to_f64(t.cpu().view(torch.int16).numpy().view(np.uint16))


def normal(rng, shape, std=1.0):
    return bf16_bits((rng.standard_normal(shape) * std).astype(np.float32))


def make(M, N, K, seed):
    rng = np.random.default_rng(seed)
    return {"x": normal(rng, (M, K)), "w": normal(rng, (N, K), K ** -0.5),
            "b": rng.standard_normal(N).astype(np.float32),
            "r": normal(rng, (M, N)), "dy": normal(rng, (M, N)),
            "z": normal(rng, (M, N), 1.5)}


def check_fwd(m, d, act, bias, res, save, **kw):
    out = m.moe_linear_fwd(dev(d["x"]), dev(d["w"]),
                           bias=torch.from_numpy(d["b"]).cuda() if bias
                           else None, act=ACTS.index(act),
                           residual=dev(d["r"]) if res else None, save=save,
                           **kw)
    o = B.linear_fwd(d["x"], d["w"], d["b"] if bias else None, act,
                     d["r"] if res else None)
    K = d["x"].shape[1]
    A = np.abs(bf16_to_f64(d["x"])) @ np.abs(bf16_to_f64(d["w"])).T
    if bias:
        A = A + np.abs(d["b"])
    ez = (K + 17) * U * A
    if save:
        z = host(out["z"])
        assert np.all(np.abs(z - o["z"]) <= HALF * np.abs(o["z"]) + 1.01 * ez)
    ey = 1.13 * ez
    if act not in ("none", "relu"):
        ey = ey + 2.0 ** -18 * np.abs(o["z"])
    if res:
        ey = ey + U * (np.abs(o["y"]) + np.abs(bf16_to_f64(d["r"])))
    y = host(out["y"])
    bad = np.abs(y - o["y"]) > HALF * np.abs(o["y"]) + 1.01 * ey
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4])
    return out


def check_bwd(m, d, act, **kw):
    M, N = d["dy"].shape
    K = d["x"].shape[1]
    g = m.moe_linear_bwd(dev(d["dy"]), dev(d["x"]), dev(d["w"]),
                         act=ACTS.index(act),
                         z=None if act == "none" else dev(d["z"]),
                         want_db=True, **kw)
    o = B.linear_bwd(d["dy"], d["x"], d["w"], act, d["z"])
    dy, z = np.abs(bf16_to_f64(d["dy"])), np.abs(bf16_to_f64(d["z"]))
    e = np.zeros((M, N)) if act in ("none", "relu") else \
        2.0 ** -18 * dy * (1 + z)
    adz = np.abs(o["dz"])
    edz = e if act == "none" else e + HALF * (adz + e)
    aw, ax = np.abs(bf16_to_f64(d["w"])), np.abs(bf16_to_f64(d["x"]))
    tdx = HALF * np.abs(o["dx"]) + 1.01 * (edz @ aw) + \
        (N + 17) * U * 1.02 * ((adz + edz) @ aw)
    tdw = HALF * np.abs(o["dw"]) + 1.01 * (edz.T @ ax) + \
        (M + 17) * U * 1.02 * ((adz + edz).T @ ax)
    tdb = e.sum(0) + (M + 17) * U * (adz + e).sum(0)
    assert np.all(np.abs(host(g["dx"]) - o["dx"]) <= tdx + 1e-30)
    assert np.all(np.abs(host(g["dw"]) - o["dw"]) <= tdw + 1e-30)
    assert np.all(np.abs(g["db"].cpu().numpy() - o["db"]) <= 1.01 * tdb)
    return g


# M, N, K: one value, single rows, tile edges +- 1, odd N, K tails of a step
SHAPES = [(1, 1, 8), (1, 1000, 4096), (2, 3, 16), (3, 129, 72), (15, 8, 64),
          (16, 512, 256), (17, 31, 56), (33, 257, 200), (64, 64, 128),
          (65, 100, 1032), (127, 128, 64), (128, 255, 120), (129, 256, 192),
          (200, 1, 2048), (255, 129, 136), (256, 256, 512), (257, 300, 64),
          (300, 77, 1000), (513, 384, 88), (40, 2000, 2056)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_forward(m, M, N, K):
    d = make(M, N, K, M * 7 + N * 3 + K)
    for i, act in enumerate(ACTS):
        check_fwd(m, d, act, bias=i % 2 == 0, res=i % 3 != 1, save=i != 2)
    check_fwd(m, d, "gelu", bias=False, res=False, save=False)
    check_fwd(m, d, "none", bias=True, res=False, save=True)


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_backward(m, M, N, K):
    d = make(M, N, K, M * 5 + N * 2 + K)
    for act in ACTS:
        check_bwd(m, d, act)


@pytest.mark.parametrize("M,N,K", [
    (1500, 2100, 1032),     # 256 tiles, ragged
    (2048, 768, 2048),      # wgrad: few tiles, long reduction (split)
    (70, 300, 14336),       # forward: few tiles, long K (split)
    (5000, 64, 96), (64, 9000, 128)])
def test_larger(m, M, N, K):
    d = make(M, N, K, 3)
    check_fwd(m, d, "silu", bias=True, res=True, save=True)
    check_bwd(m, d, "gelu_tanh")


@pytest.mark.parametrize("M,N,K", [
    (1, 9000, 264), (16, 4100, 4104), (7, 5, 14336), (32, 16401, 72),
    (17, 400, 4096), (33, 16500, 64), (64, 1000, 2056), (48, 20000, 520)])
def test_few_rows(m, M, N, K):
    """Every wave count and row-block form of the one-pass kernel, with
    ragged weight rows and K tails inside and between its trips."""
    d = make(M, N, K, 5)
    check_fwd(m, d, "gelu", bias=True, res=True, save=True)
    check_fwd(m, d, "none", bias=False, res=False, save=False)


@pytest.mark.parametrize("want", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 0)])
def test_partial_gradients(m, want):
    d = make(100, 90, 64, 4)
    full = check_bwd(m, d, "silu")
    dx, dw, db = want
    g = m.moe_linear_bwd(dev(d["dy"]), dev(d["x"]) if dw else None,
                         dev(d["w"]) if dx else None, act=4, z=dev(d["z"]),
                         want_dx=bool(dx), want_dw=bool(dw),
                         want_db=bool(db))
    assert set(g) == {n for n, f in zip(("dx", "dw", "db"), want) if f}
    for n in g:
        assert torch.equal(g[n], full[n])


@pytest.mark.parametrize("M,N,K", [(5, 700, 64), (40, 513, 136),
                                   (250, 90, 64), (700, 260, 72)])
def test_bias_gradient_with_either_product(m, M, N, K):
    """db is summed next to both products, or after one, or alone: the same
    bits, for every way its partial sums are dealt (1, 5, 32 and 88 chunks of
    rows)."""
    d = make(M, N, K, 8)
    full = check_bwd(m, d, "gelu")
    for dx, dw in ((1, 0), (0, 1), (0, 0)):
        g = m.moe_linear_bwd(dev(d["dy"]), dev(d["x"]), dev(d["w"]), act=2,
                             z=dev(d["z"]), want_dx=bool(dx),
                             want_dw=bool(dw), want_db=True)
        for n in g:
            assert torch.equal(g[n], full[n]), (n, dx, dw)


@pytest.mark.parametrize("act", ACTS[1:])
def test_activation_range(m, act):
    """Every magnitude of z through the activation and its derivative: K = 8
    with one non-zero weight, so z is exact."""
    v = np.concatenate([np.linspace(-12, 12, 2001), -np.logspace(-20, 1.9, 400),
                        np.logspace(-20, 30, 400), [0.0, -0.0, 60, -60, 100,
                                                    -100, 1e4, -1e4]])
    zb = bf16_bits(v.astype(np.float32))
    M = zb.size
    x = np.zeros((M, 8), np.uint16)
    x[:, 0] = zb
    w = np.zeros((1, 8), np.uint16)
    w[0, 0] = bf16_bits(np.ones(1, np.float32))[0]
    y = host(m.moe_linear_fwd(dev(x), dev(w), act=ACTS.index(act))["y"])[:, 0]
    z = bf16_to_f64(zb)
    want = B.act(act, z)
    # relative where the exact value is a normal number, down to the float32
    # exponential's underflow
    tol = HALF * np.abs(want) + 2.0 ** -14 * np.abs(want) + 1e-30
    assert np.all(np.abs(y - want) <= tol), \
        [(z[i], y[i], want[i]) for i in np.argwhere(
            np.abs(y - want) > tol)[:5, 0]]
    one = bf16_bits(np.ones((M, 1), np.float32))
    g = m.moe_linear_bwd(dev(one), None, None, act=ACTS.index(act),
                         z=dev(zb.reshape(M, 1)), want_dx=False,
                         want_dw=False, want_db=True)["db"]
    # one derivative at a time, through db of a single row
    keep = np.abs(z) < 1e4
    for i in np.nonzero(keep)[0][::37]:
        g = m.moe_linear_bwd(dev(one[:1]), None, None, act=ACTS.index(act),
                             z=dev(zb[i:i + 1].reshape(1, 1)), want_dx=False,
                             want_dw=False, want_db=True)["db"]
        ref = B.act_grad(act, z[i:i + 1])[0]
        assert abs(float(g[0]) - ref) <= 2.0 ** -18 * (1 + abs(z[i])), z[i]


@pytest.mark.parametrize("act", ACTS[1:])
def test_activation_extremes(m, act):
    """Derivatives of the largest magnitudes (0 or 1 exactly: the other terms
    vanish) and NaN, which stays NaN in both directions."""
    v = np.array([1e10, 1e19, 3e19, 1e25, 3e38], np.float32)
    zb = bf16_bits(np.concatenate([v, -v, [np.nan]]).astype(np.float32))
    n = zb.size
    one = bf16_bits(np.ones((1, n), np.float32))
    g = m.moe_linear_bwd(dev(one), None, None, act=ACTS.index(act),
                         z=dev(zb.reshape(1, n)), want_dx=False,
                         want_dw=False, want_db=True)["db"].cpu().numpy()
    ref = B.act_grad(act, bf16_to_f64(zb[:-1]))
    assert np.all(ref == np.repeat([1.0, 0.0], 5))
    assert np.all(g[:-1] == ref) and np.isnan(g[-1])
    for M in (1, 5, 70):
        x = torch.full((M, 8), float("nan"), dtype=torch.bfloat16,
                       device="cuda")
        w = torch.ones((9, 8), dtype=torch.bfloat16, device="cuda")
        y = m.moe_linear_fwd(x, w, act=ACTS.index(act))["y"]
        assert bool(torch.isnan(y).all())
        dx = m.moe_linear_bwd(torch.ones_like(y), x, w, act=ACTS.index(act),
                              z=y, want_dw=False)["dx"]
        assert bool(torch.isnan(dx).all())


def test_rows_are_isolated(m):
    """A NaN row of x or W reaches its own output row or column only, also
    through K tails (the bytes behind a row's end are the next row's)."""
    for M, N, K in ((40, 70, 72), (300, 300, 200), (20, 33, 8),
                    (1, 300, 1032), (7, 64, 4104)):
        d = make(M, N, K, 6)
        ref = check_fwd(m, d, "silu", True, False, False)["y"]
        x, w = dev(d["x"]), dev(d["w"])
        i, j = M // 2, N // 2
        x[i] = float("nan")
        w[j] = float("inf")
        y = m.moe_linear_fwd(x, w, bias=torch.from_numpy(d["b"]).cuda(),
                             act=4)["y"]
        keep = torch.ones((M, N), dtype=torch.bool, device="cuda")
        keep[i] = False
        keep[:, j] = False
        assert torch.equal(y[keep], ref[keep])
        assert bool(torch.isnan(y[i]).all())


def test_inputs_inside_nan_buffers_and_output_neighbours(m):
    """Tensors cut out of larger buffers full of NaN: nothing behind them is
    read into a result, nothing around the outputs is written."""
    nan = float("nan")

    def inside(bits):
        t = dev(bits)
        buf = torch.full((t.numel() + 8192,), nan, dtype=t.dtype,
                         device="cuda")
        v = buf[4096:4096 + t.numel()].view(t.shape)
        v.copy_(t)
        return v
    for M, N, K in ((33, 100, 72), (257, 130, 1000), (3, 257, 200),
                    (130, 37, 64), (1, 513, 1032)):
        d = make(M, N, K, 9)
        base = check_fwd(m, d, "gelu", True, True, True)
        buf = torch.full((M * N + 8192,), 3.0, dtype=torch.bfloat16,
                         device="cuda")
        out = buf[4096:4096 + M * N].view(M, N)
        r = m.moe_linear_fwd(inside(d["x"]), inside(d["w"]),
                             bias=torch.from_numpy(d["b"]).cuda(), act=2,
                             residual=inside(d["r"]), save=True, out=out)
        assert torch.equal(r["y"], base["y"]) and torch.equal(r["z"],
                                                              base["z"])
        assert bool((buf[:4096] == 3).all())
        assert bool((buf[4096 + M * N:] == 3).all())
        g0 = check_bwd(m, d, "silu")
        # the workspace may hold anything
        ws = torch.full((1 << 24,), 255, dtype=torch.uint8, device="cuda")
        g = m.moe_linear_bwd(inside(d["dy"]), inside(d["x"]), inside(d["w"]),
                             act=4, z=inside(d["z"]), want_db=True, ws=ws)
        for n in g:
            assert torch.equal(g[n], g0[n]), n


def test_residual_in_place(m):
    for M, N, K in ((130, 264, 64), (5, 33, 4096), (70, 300, 14336)):
        d = make(M, N, K, 2)
        want = check_fwd(m, d, "relu", True, True, False)["y"]
        r = dev(d["r"])
        y = m.moe_linear_fwd(dev(d["x"]), dev(d["w"]),
                             bias=torch.from_numpy(d["b"]).cuda(), act=1,
                             residual=r, out=r)["y"]
        assert y.data_ptr() == r.data_ptr() and torch.equal(y, want)


def test_zero_rows(m):
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    w = torch.ones((10, 64), dtype=torch.bfloat16, device="cuda")
    r = m.moe_linear_fwd(x, w, save=True)
    assert r["y"].shape == (0, 10) and r["z"].shape == (0, 10)
    dy = torch.empty((0, 10), dtype=torch.bfloat16, device="cuda")
    g = m.moe_linear_bwd(dy, x, w, act=4, z=dy, want_db=True)
    assert g["dx"].shape == (0, 64)
    assert bool((g["dw"] == 0).all()) and bool((g["db"] == 0).all())


def test_rows_past_32_bit_offsets(m):
    """x of 4.9 GB: the last rows lie past 2^32 bytes."""
    M, N, K = 300001, 40, 8192
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    x = torch.zeros((M, K), dtype=torch.bfloat16, device="cuda")
    d = make(4, N, K, 12)
    x[-4:] = dev(d["x"])
    w = dev(d["w"])
    y = m.moe_linear_fwd(x, w)["y"]
    o = B.linear_fwd(d["x"], d["w"])
    A = np.abs(bf16_to_f64(d["x"])) @ np.abs(bf16_to_f64(d["w"])).T
    assert np.all(np.abs(host(y[-4:]) - o["y"]) <=
                  HALF * np.abs(o["y"]) + 1.01 * (K + 17) * U * A)
    assert bool((y[:-4] == 0).all())
    dy = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    dy[-4:] = dev(d["dy"])
    g = m.moe_linear_bwd(dy, x, w, want_db=True)
    o = B.linear_bwd(d["dy"], d["x"], d["w"])
    ady = np.abs(bf16_to_f64(d["dy"]))
    assert np.all(np.abs(host(g["dw"]) - o["dw"]) <= HALF * np.abs(o["dw"]) +
                  32 * U * (ady.T @ np.abs(bf16_to_f64(d["x"]))))
    assert np.all(np.abs(host(g["dx"][-4:]) - o["dx"]) <=
                  HALF * np.abs(o["dx"]) +
                  64 * U * (ady @ np.abs(bf16_to_f64(d["w"]))))
    assert bool((g["dx"][:-4] == 0).all())
