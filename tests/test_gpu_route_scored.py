"""Scored routing on the GPU against the float64 oracle.

Expert ids are compared exactly.  Weights and gradients are float64 inside
and rounded to float32 once: half an ulp is 2^-24 of the value; 2^-23 leaves
room for the float64 arithmetic, and gradients, which are differences, get
1e-13 of their terms' size on top (float64 sums of a few hundred terms).
"""
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


SC = {"softmax": 0, "sigmoid": 1}
GS = {"max": 0, "top2": 1}


def run(m, lg, k, bias=None, score="softmax", n_group=1, topk_group=1,
        group_score="max", renormalize=True, scale=1.0):
    t = lg if isinstance(lg, torch.Tensor) else torch.from_numpy(lg).cuda()
    b = None if bias is None else torch.from_numpy(bias).cuda()
    idx, w = m.moe_route_scored(
        t, k, bias=b, score=SC[score], n_group=n_group, topk_group=topk_group,
        group_score=GS[group_score], renormalize=renormalize, scale=scale)
    return idx, w


def check(m, lg, k, dw_seed=0, **o):
    idx, w = run(m, lg, k, **o)
    ridx, rw = B.route_scored(lg, k, **o)
    np.testing.assert_array_equal(idx.cpu().numpy(), ridx)
    np.testing.assert_allclose(w.cpu().numpy(), rw, rtol=2.0 ** -23,
                               atol=1e-44)
    bw = {n: o[n] for n in ("score", "renormalize", "scale") if n in o}
    dw = np.random.default_rng(dw_seed).standard_normal(
        (lg.shape[0], k)).astype(np.float32)
    a = dict(bw)
    if "score" in a:
        a["score"] = SC[a["score"]]
    dl = m.moe_route_scored_bwd(torch.from_numpy(lg).cuda(), idx,
                                torch.from_numpy(dw).cuda(), **a)
    want = B.route_scored_bwd(lg, ridx, dw, **bw)
    err = np.abs(dl.cpu().numpy() - want)
    assert np.all(err <= 2.0 ** -23 * np.abs(want) +
                  1e-13 * abs(o.get("scale", 1.0)) * np.abs(dw).max() + 1e-44)
    assert m.check_device_status() == 0


# T, E, k, n_group, topk_group: both kernels, every registers-per-lane form,
# groups in whole lanes (128 / 8, 256 / 8, 64 / 4, 16 / 8, 256 / 2), groups
# through LDS (60 / 3, 96 / 4, 300 / 5, 1024 / 16, 20 / 10, 40 / 1)
SHAPES = [
    (1, 1, 1, 1, 1), (3, 2, 2, 1, 1), (17, 8, 2, 1, 1), (5, 16, 16, 1, 1),
    (33, 16, 4, 8, 3), (257, 40, 6, 1, 1), (65, 60, 6, 3, 2),
    (16, 64, 8, 4, 2), (31, 96, 8, 4, 1), (130, 128, 8, 8, 4),
    (1, 128, 8, 1, 1), (9, 255, 7, 5, 2), (67, 256, 8, 8, 4),
    (20, 256, 16, 2, 1), (6, 256, 17, 8, 8), (7, 20, 3, 10, 2),
    (11, 300, 9, 5, 3), (5, 1024, 32, 16, 4), (3, 1024, 8, 64, 8),
    (4, 100, 20, 4, 1), (2, 513, 5, 27, 5),
    # lists of 2, 8 and 16 over 4, 8 and 16 experts per lane
    (50, 100, 2, 1, 1), (50, 200, 1, 1, 1), (50, 256, 2, 16, 3),
    (50, 128, 12, 8, 3), (50, 130, 16, 1, 1), (50, 64, 13, 1, 1),
]


@pytest.mark.parametrize("T,E,k,G,tg", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_scored(m, T, E, k, G, tg, score):
    rng = np.random.default_rng(T * 1000 + E)
    lg = (rng.standard_normal((T, E)) * 2).astype(np.float32)
    bias = (rng.standard_normal(E) * 0.1).astype(np.float32)
    for gs in (["max", "top2"] if E // G >= 2 else ["max"]):
        for b in (None, bias):
            for ren, sc in ((True, 2.5), (False, 1.0)):
                check(m, lg, k, bias=b, score=score, n_group=G, topk_group=tg,
                      group_score=gs, renormalize=ren, scale=sc)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k,G,tg", [(128, 8, 8, 4), (60, 6, 3, 2),
                                      (300, 9, 5, 3), (8, 8, 1, 1)])
def test_ties_and_signed_zeros(m, score, E, k, G, tg):
    """Coarse logits and biases: most keys and group scores are equal."""
    rng = np.random.default_rng(E)
    lg = rng.integers(-1, 2, (64, E)).astype(np.float32)
    lg[0] = 0.0
    lg[1] = -0.0
    lg[2, ::2] = -0.0
    lg[2, 1::2] = 0.0
    bias = (rng.integers(0, 2, E) * 0.25).astype(np.float32)
    for b in (None, bias):
        for gs in ("max", "top2") if G > 1 else ("max",):
            check(m, lg, k, bias=b, score=score, n_group=G, topk_group=tg,
                  group_score=gs)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_extreme_logits(m, score):
    """Masked logits at the type's lowest value, saturated scores, rows whose
    scores all underflow."""
    lo = np.finfo(np.float32).min
    lg = np.full((6, 32), lo, np.float32)
    lg[0, 3] = 1.0
    lg[1] = -np.arange(32) * 100
    lg[2] = np.arange(32) * 50
    lg[3] = lo                      # nothing is left: lowest ids, no NaN
    lg[4, 5:9] = [1e30, 1e30, -5, 2]
    lg[5] = -800 - np.arange(32)
    for ren in (True, False):
        for G, tg in ((1, 1), (4, 2)):
            check(m, lg, 4, score=score, n_group=G, topk_group=tg,
                  renormalize=ren)
    idx, w = run(m, lg, 4, score=score)
    assert bool(torch.isfinite(w).all())


@pytest.mark.parametrize("E,k,G,tg", [(128, 8, 1, 1), (128, 8, 8, 4),
                                      (40, 6, 1, 1), (60, 6, 3, 2),
                                      (256, 16, 8, 4), (300, 9, 5, 3)])
def test_scores_that_differ_in_their_last_bits(m, E, k, G, tg):
    """Saturated sigmoids: keys that agree in their upper 42 bits and differ
    (or do not) below, in every token and in one token of many."""
    rng = np.random.default_rng(E)
    lg = (24 + 13 * rng.random((48, E))).astype(np.float32)
    mixed = rng.standard_normal((48, E)).astype(np.float32)
    mixed[17] = lg[17]
    for a in (lg, mixed):
        for bias in (np.zeros(E, np.float32),
                     (rng.integers(0, 2, E) * 2.0 ** -44).astype(np.float32)):
            for gs in ("max", "top2") if G > 1 else ("max",):
                check(m, a, k, bias=bias, score="sigmoid", n_group=G,
                      topk_group=tg, group_score=gs)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k,G,tg", [
    (50, 192, 8, 8, 4), (50, 192, 16, 4, 2), (50, 160, 2, 5, 3),
    (50, 145, 7, 1, 1), (50, 130, 8, 2, 1), (50, 176, 12, 16, 5),
    (50, 189, 6, 63, 20), (50, 240, 8, 60, 31), (50, 190, 1, 38, 17)])
def test_twelve_experts_per_lane_and_many_groups(m, T, E, k, G, tg, score):
    """Lists of 2, 8 and 16 over 12 experts per lane; groups in whole lanes,
    through LDS, and more groups than lanes."""
    test_route_scored(m, T, E, k, G, tg, score)
    test_ties_and_signed_zeros(m, score, E, k, G, tg)
    test_scores_that_differ_in_their_last_bits(m, E, k, G, tg)


@pytest.mark.parametrize("E,G,tg", [(128, 1, 1), (64, 4, 2), (60, 3, 2),
                                    (512, 8, 2)])
def test_masked_experts(m, E, G, tg):
    """A bias of -infinity masks an expert; where too few others are left the
    masked ones follow by id."""
    rng = np.random.default_rng(E)
    lg = rng.standard_normal((20, E)).astype(np.float32)
    bias = np.zeros(E, np.float32)
    bias[rng.permutation(E)[: E // 2]] = -np.inf
    check(m, lg, 8, bias=bias, score="sigmoid", n_group=G, topk_group=tg)
    bias[2:] = -np.inf
    check(m, lg, 8, bias=bias, score="sigmoid", n_group=G, topk_group=tg)


@pytest.mark.parametrize("E,k", [(12, 4), (16, 16), (128, 8), (300, 9)])
def test_non_finite_inputs_are_reported(m, E, k):
    rng = np.random.default_rng(E)
    lg = rng.standard_normal((40, E)).astype(np.float32)
    good = lg.copy()
    lg[3, 1], lg[7, E - 1], lg[9] = np.nan, np.inf, np.nan
    idx, _ = run(m, lg, k, score="sigmoid")
    assert m.check_device_status() == 3
    i = idx.cpu().numpy()
    assert i.min() >= 0 and i.max() < E
    rest = [t for t in range(40) if t not in (3, 7, 9)]
    np.testing.assert_array_equal(
        i[rest], B.route_scored(good, k, score="sigmoid")[0][rest])
    bias = np.zeros(E, np.float32)
    bias[E // 2] = np.nan
    idx, _ = run(m, good, k, bias=bias, score="sigmoid")
    assert m.check_device_status() == 3
    i = idx.cpu().numpy()
    assert i.min() >= 0 and i.max() < E


@pytest.mark.parametrize("E,k", [(12, 4), (300, 9), (200, 8)])
def test_bwd_bad_and_repeated_ids(m, E, k):
    """An id outside [0, E) contributes nothing; one named twice adds."""
    rng = np.random.default_rng(E)
    lg = rng.standard_normal((9, E)).astype(np.float32)
    dw = rng.standard_normal((9, k)).astype(np.float32)
    idx = B.route_scored(lg, k)[0]
    idx[1, 1] = idx[1, 0]
    args = [torch.from_numpy(a).cuda() for a in (lg, idx, dw)]
    for sc in ("softmax", "sigmoid"):
        for ren in (True, False):
            got = m.moe_route_scored_bwd(*args, score=SC[sc],
                                         renormalize=ren).cpu().numpy()
            want = B.route_scored_bwd(lg, idx, dw, sc, ren)
            # the two contributions are rounded to float32 and then added
            assert np.all(np.abs(got - want) <= 2.0 ** -22 *
                          (np.abs(want) + np.abs(dw).max()))
    assert m.check_device_status() == 0
    bad = idx.copy()
    bad[4, 0], bad[5, 1] = -1, E
    got = m.moe_route_scored_bwd(args[0], torch.from_numpy(bad).cuda(),
                                 args[2], score=SC["sigmoid"],
                                 renormalize=False).cpu().numpy()
    assert m.check_device_status() == 1
    keep = B.route_scored_bwd(lg, idx, dw, "sigmoid", False)
    keep[4, idx[4, 0]] = 0.0
    keep[5, idx[5, 1]] = 0.0
    assert np.all(np.abs(got - keep) <= 2.0 ** -22 *
                  (np.abs(keep) + np.abs(dw).max()))


def test_unaligned_rows_and_neighbours(m):
    """Inputs and outputs that start off 16-byte boundaries inside larger
    buffers; nothing around the outputs changes."""
    rng = np.random.default_rng(8)
    for T, E, k in ((37, 128, 8), (5, 61, 3), (9, 256, 8)):
        lg = rng.standard_normal((T, E)).astype(np.float32)
        buf = torch.full((T * E + 9,), float("nan"), device="cuda")
        view = buf[1:1 + T * E].view(T, E)
        view.copy_(torch.from_numpy(lg))
        idx, w = run(m, view, k, score="sigmoid")
        ridx, _ = B.route_scored(lg, k, score="sigmoid")
        np.testing.assert_array_equal(idx.cpu().numpy(), ridx)
        dw = rng.standard_normal((T, k)).astype(np.float32)
        out = torch.full((T * E + 9,), 7.0, device="cuda")
        lib = m.load_library()
        import ctypes
        o = m._RouteOpts(1, 1, 1, 0, 1, 1.0)
        dwt = torch.from_numpy(dw).cuda()
        m._check(lib.moe_route_scored_bwd(
            m._context(view.device), view.data_ptr(), idx.data_ptr(),
            dwt.data_ptr(), T, E, k, ctypes.byref(o), out[1:].data_ptr(),
            m._stream()))
        o = out.cpu().numpy()
        assert o[0] == 7.0 and np.all(o[1 + T * E:] == 7.0)
        want = B.route_scored_bwd(lg, ridx, dw, "sigmoid")
        assert np.all(np.abs(o[1:1 + T * E].reshape(T, E) - want) <=
                      2.0 ** -23 * np.abs(want) + 1e-12)


def test_zero_tokens(m):
    lg = torch.empty((0, 16), device="cuda")
    idx, w = m.moe_route_scored(lg, 2)
    assert idx.shape == (0, 2) and w.shape == (0, 2)
    dl = m.moe_route_scored_bwd(lg, idx, w)
    assert dl.shape == (0, 16)
    x = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    wr = torch.ones((16, 64), dtype=torch.bfloat16, device="cuda")
    g = m.moe_router_proj_bwd(lg, x, wr)
    assert g["dx"].shape == (0, 64) and bool((g["dw_r"] == 0).all())


def test_agrees_with_route_topk_and_router_bwd(m):
    """The plain softmax form is that of the existing entry points."""
    rng = np.random.default_rng(12)
    T, E, k, H = 300, 128, 8, 64
    lg = torch.from_numpy(rng.standard_normal((T, E)).astype(np.float32)) \
        .cuda()
    x = torch.randn(T, H, device="cuda").bfloat16()
    wr = torch.randn(E, H, device="cuda").bfloat16()
    dw = torch.randn(T, k, device="cuda")
    for ren in (True, False):
        i0, w0 = m.moe_route_topk(lg, k, ren)
        i1, w1 = m.moe_route_scored(lg, k, renormalize=ren)
        assert torch.equal(i0, i1)
        torch.testing.assert_close(w0, w1, rtol=2.0 ** -22, atol=0)
        g = m.moe_router_bwd(lg, i0, dw, x, wr, renormalize=ren)
        dl = m.moe_route_scored_bwd(lg, i1, dw, renormalize=ren)
        torch.testing.assert_close(dl, g["dlogits"], rtol=2.0 ** -22,
                                   atol=1e-12)
        p = m.moe_router_proj_bwd(g["dlogits"], x, wr)
        assert torch.equal(p["dw_r"], g["dw_r"])
        assert torch.equal(p["dx"], g["dx"])
