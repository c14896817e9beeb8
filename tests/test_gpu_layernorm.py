"""Layer norm on the GPU against the float64 oracle.

Element-wise bounds, from the arithmetic (u = 2^-24; a bf16 rounding is off
by at most 2^-8 of the value).  A sum over a row takes at most 32 values in a
lane, six steps across a wave, 16 across waves and a few more: 60 roundings,
each at most u of a partial sum, so at most 60 u times the sum of magnitudes.
 * mean: em = 61 u mean|x|;  x - mean: em + u |x - mean|.
 * variance: relative 2 em mean|d| / var + em^2 / var + 64 u, rstd half of
   that and 4 u (square root, division, the addition of eps).
 * y: the pieces times |w|, two products and one addition, one rounding.
 * dx: xh and g are off by 2 u and u, the row sums by 62 u of their
   magnitudes, the last steps by 4 u; one addition; one rounding.
 * dw, db: xh's 2 u, and one rounding per addition: a lane's rows, the waves,
   the work-groups' sums.
"""
import numpy as np
import pytest
import torch

from oracle import prenorm_oracle as P
from synthetic import bf16_bits, bf16_to_f64

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF = 2.0 ** -8


@pytest.fixture(scope="module")
def m():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    import mixture_experts_grouped_router_amd as mod
    mod.load_library()
    return mod


def dev(a):
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        return torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).cuda()
    return torch.from_numpy(a).cuda()


def host(t):
    if t.dtype == torch.bfloat16:
        return bf16_to_f64(t.cpu().view(torch.int16).numpy().view(np.uint16))
    return t.cpu().numpy().astype(np.float64)


def stored(a, f32):
    a = np.asarray(a, np.float32)
    return a if f32 else bf16_bits(a)


def make(T, H, f32, seed, spread=1.0, shift=0.5):
    rng = np.random.default_rng(seed)
    x = rng.standard_normal((T, H)) * spread * np.exp(
        0.5 * rng.standard_normal(H)) + shift * rng.standard_normal(H)
    return {"x": stored(x, f32),
            "w": (1 + 0.2 * rng.standard_normal(H)).astype(np.float32),
            "b": (0.2 * rng.standard_normal(H)).astype(np.float32),
            "dy": bf16_bits(rng.standard_normal((T, H)).astype(np.float32)),
            "r": stored(rng.standard_normal((T, H)), f32)}


def as64(a):
    return bf16_to_f64(a) if a.dtype == np.uint16 else a.astype(np.float64)


def row(v):
    return v[:, None]


def check_fwd(m, d, w=True, b=True, eps=1e-5, out=None):
    wt, bt = (d["w"] if w else None), (d["b"] if b else None)
    got = m.moe_layernorm_fwd(dev(d["x"]), None if wt is None else dev(wt),
                              None if bt is None else dev(bt), eps=eps,
                              save=True, out=out)
    ref = P.layernorm_fwd(d["x"], wt, bt, eps)
    x = as64(d["x"])
    dd = np.abs(x - row(ref["mean"]))
    em = 61 * U * np.abs(x).mean(axis=1)
    var = 1.0 / ref["rstd"] ** 2
    er = 0.5 * ((2 * em * dd.mean(axis=1) + em ** 2) / var + 64 * U) + 4 * U
    assert np.all(np.abs(host(got["mean"]) - ref["mean"]) <=
                  1.01 * em + U * np.abs(ref["mean"]))
    assert np.all(np.abs(host(got["rstd"]) - ref["rstd"]) <=
                  1.01 * er * ref["rstd"])
    wa = 1.0 if wt is None else np.abs(as64(wt))
    ey = wa * row(ref["rstd"]) * (row(em) + dd * (row(er) + 4 * U))
    ey = ey + U * (np.abs(ref["y"]) + (0 if bt is None else np.abs(as64(bt))))
    y = host(got["y"])
    bad = np.abs(y - ref["y"]) > HALF * (np.abs(ref["y"]) + ey) + 1.01 * ey
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4])
    return got


def check_bwd(m, d, got, w=True, res=True, rows=None, **kw):
    wt = d["w"] if w else None
    g = m.moe_layernorm_bwd(dev(d["dy"]), dev(d["x"]), got["mean"],
                            got["rstd"], None if wt is None else dev(wt),
                            dresidual=dev(d["r"]) if res else None, **kw)
    mean, rstd = host(got["mean"]), host(got["rstd"])
    ref = P.layernorm_bwd(d["dy"], d["x"], mean, rstd, wt,
                          d["r"] if res else None)
    dy, x = as64(d["dy"]), as64(d["x"])
    T, H = x.shape
    xh = np.abs((x - row(mean)) * row(rstd))
    gm = np.abs(dy * (1.0 if wt is None else as64(wt)))
    s1, s2 = gm.mean(axis=1, keepdims=True), (gm * xh).mean(axis=1,
                                                            keepdims=True)
    e = row(np.abs(rstd)) * (5 * U * (gm + s1 + 3 * xh * s2) + 62 * U * s1 +
                             xh * 66 * U * s2)
    if res:
        e = e + U * (np.abs(ref["dx"]) + np.abs(as64(d["r"])))
    if "dx" in g:
        half = HALF if d["x"].dtype == np.uint16 else U
        bad = np.abs(host(g["dx"]) - ref["dx"]) > \
            half * (np.abs(ref["dx"]) + e) + 1.01 * e
        assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4])
    n = min(T, T // 256 + 100) + 4   # additions on the way to one column
    if "dw" in g:
        ew = (n + 4) * U * (np.abs(dy) * xh).sum(axis=0)
        assert np.all(np.abs(host(g["dw"]) - ref["dw"]) <= 1.01 * ew)
    if "db" in g:
        assert np.all(np.abs(host(g["db"]) - ref["db"]) <=
                      1.01 * n * U * np.abs(dy).sum(axis=0))
    return g


# widths: below a chunk, odd, each count of values per lane and of waves per
# row, both access widths, the largest
WIDTHS = [1, 2, 7, 8, 33, 64, 511, 512, 520, 1024, 1032, 1035, 2040, 2047,
          2048, 2056, 2049, 4096, 4104, 5001, 8192, 8185, 8200, 9001, 12288,
          16384, 16383]


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("H", WIDTHS)
def test_widths(m, H, f32):
    d = make(9, H, f32, H)
    got = check_fwd(m, d)
    check_bwd(m, d, got)


# rows: none idle, a part of a work-group, more than one round of them
@pytest.mark.parametrize("T,H", [(1, 2048), (2, 2048), (3, 5000), (5, 64),
                                 (2051, 256), (5000, 1024), (4099, 72),
                                 (1500, 2304), (700, 8200), (2500, 31)])
def test_rows(m, T, H):
    d = make(T, H, False, T)
    got = check_fwd(m, d)
    check_bwd(m, d, got)


@pytest.mark.parametrize("H", [96, 2500])
def test_optional_arguments(m, H):
    d = make(37, H, False, 5)
    for w in (False, True):
        for b in (False, True):
            check_fwd(m, d, w, b)
    got = check_fwd(m, d)
    for want in [(1, 0, 0), (0, 1, 0), (0, 0, 1), (0, 1, 1), (1, 1, 0)]:
        g = check_bwd(m, d, got, w=bool(want[1]), res=bool(want[0]),
                      want_dx=bool(want[0]), want_dw=bool(want[1]),
                      want_db=bool(want[2]))
        assert sorted(g) == sorted(n for n, q in zip(("dx", "dw", "db"), want)
                                   if q)
    # dx over dresidual, y and workspace of the caller
    r = dev(d["r"])
    a = m.moe_layernorm_bwd(dev(d["dy"]), dev(d["x"]), got["mean"],
                            got["rstd"], dev(d["w"]), dresidual=r)
    ws = torch.empty(1 << 22, dtype=torch.uint8, device="cuda")
    b = m.moe_layernorm_bwd(dev(d["dy"]), dev(d["x"]), got["mean"],
                            got["rstd"], dev(d["w"]), dresidual=r, out=r,
                            ws=ws)
    assert b["dx"] is r
    for n in ("dx", "dw", "db"):
        assert torch.equal(a[n], b[n]), n


def test_far_mean_and_small_spread(m):
    """A mean 1000 times the spread: the variance is that of the deviations."""
    d = make(16, 1024, True, 11, spread=1.0, shift=0.0)
    d["x"] = (d["x"] + 1000.0).astype(np.float32)
    got = check_fwd(m, d)
    check_bwd(m, d, got)


def test_constant_and_extreme_rows(m):
    x = np.zeros((4, 256), np.float32)
    x[1] = 3.0
    x[2] = 1e15 * np.random.default_rng(0).standard_normal(256)
    x[3, 5] = np.inf
    got = m.moe_layernorm_fwd(dev(x), save=True)
    y = host(got["y"])
    assert np.all(y[:2] == 0)
    np.testing.assert_allclose(host(got["rstd"])[:2], 1e-5 ** -0.5,
                               rtol=8 * U)
    ref = P.layernorm_fwd(x[2:3])["y"]
    assert np.abs(y[2] - ref[0]).max() <= HALF * np.abs(ref).max() * 1.01
    assert np.all(np.isnan(y[3]))     # and no other row


def test_no_rows(m):
    z = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    s = torch.empty(0, device="cuda")
    assert m.moe_layernorm_fwd(z)["y"].shape == (0, 64)
    g = m.moe_layernorm_bwd(z, z, s, s)
    assert g["dx"].shape == (0, 64)
    assert not g["dw"].any() and not g["db"].any()


def test_gradient_against_differences(m):
    """The float32 path's gradients against central differences of the
    oracle's forward (the formula is checked in the oracle's own tests)."""
    d = make(3, 40, True, 17)
    got = m.moe_layernorm_fwd(dev(d["x"]), dev(d["w"]), dev(d["b"]), save=True)
    g = m.moe_layernorm_bwd(dev(d["dy"]), dev(d["x"]), got["mean"],
                            got["rstd"], dev(d["w"]))
    dy, x = as64(d["dy"]), as64(d["x"])
    dx = host(g["dx"])
    for t, h in [(0, 0), (1, 17), (2, 39), (2, 8)]:
        h0 = 1e-4
        e = np.zeros_like(x)
        e[t, h] = h0
        f = lambda q: (P.layernorm_fwd(q, d["w"], d["b"])["y"] * dy).sum()
        num = (f(x + e) - f(x - e)) / (2 * h0)
        # differences h0^2 (third derivatives of order 10 rstd^3), float32
        # statistics and row sums 2^-16 of values of order 1
        scale = np.abs(dy[t]).max() * host(got["rstd"])[t]
        assert abs(num - dx[t, h]) <= 1e-4 * max(scale, 1.0) * 4


def test_repeats_are_bit_equal_and_streams_do_not_matter(m):
    d = make(3001, 768, False, 23)
    t = {k: dev(v) for k, v in d.items()}

    def call():
        f = m.moe_layernorm_fwd(t["x"], t["w"], t["b"], save=True)
        g = m.moe_layernorm_bwd(t["dy"], t["x"], f["mean"], f["rstd"], t["w"],
                                dresidual=t["r"])
        return [f["y"], g["dx"], g["dw"], g["db"]]
    ref = call()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in streams:
        with torch.cuda.stream(s):
            outs.append(call())
    torch.cuda.synchronize()
    for o in outs:
        for a, b in zip(o, ref):
            assert torch.equal(a, b)
