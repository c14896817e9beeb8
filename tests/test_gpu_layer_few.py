"""The whole layer for a few tokens on the GPU against the float64 oracle.

Element-wise bound (made by the oracle next to the value): the first
product's sums are off by u (H + 16) of the magnitudes' sum, which reaches a
through the SwiGLU's slopes; a's exponential and reciprocal by 2^-18, its
bf16 rounding by 2^-8; the second product's sums by u (F + 32) of their
magnitudes; then the k experts' additions, the residual's and the rounding
of y.  Routing outputs are compared exactly (indices) and to one float32
rounding (weights)."""
import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
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


def bf(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).view(
        torch.bfloat16).cuda()


def up(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def host(t):
    return bf16_to_f64(t.cpu().view(torch.int16).numpy().view(np.uint16))


def make(T, H, F, E, k, seed):
    rng = np.random.default_rng(seed)
    n = lambda shape, s: bf16_bits((rng.standard_normal(shape) * s)
                                   .astype(np.float32))
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]) if T else \
        np.zeros((0, k))
    return {"x": n((T, H), 1.0), "gu": n((E, 2 * F, H), H ** -0.5),
            "dn": n((E, H, F), F ** -0.5), "res": n((T, H), 1.0),
            "wr": n((E, H), H ** -0.5),
            "bias": (0.1 * rng.standard_normal(E)).astype(np.float32),
            "idx": idx.astype(np.int32),
            "w": rng.random((T, k)).astype(np.float32)}


def weights(m, d, fmt):
    """(keyword arguments, float64 gate/up, float64 down)"""
    if fmt == "bf16":
        return dict(w_gu=bf(d["gu"]), w_dn=bf(d["dn"])), O._as_f64(d["gu"]), \
            O._as_f64(d["dn"])
    return dict(w_gu_q=m.mxfp4_quantize(bf(d["gu"])),
                w_dn_q=m.mxfp4_quantize(bf(d["dn"])),
                precision=m.PREC_MXFP4), \
        P._round_trip(d["gu"]), P._round_trip(d["dn"])


def check(m, d, fmt, router=False, res=True, renorm=True, bias=False, **more):
    kw, gu, dn = weights(m, d, fmt)
    k = d["idx"].shape[1]
    okw = {}
    if router:
        kw.update(w_r=bf(d["wr"]), k=k, renormalize=renorm)
        okw.update(w_r=d["wr"], k=k, renormalize=renorm)
        if bias:
            kw["router_bias"] = up(d["bias"])
            okw["router_bias"] = d["bias"]
    else:
        kw.update(topk_idx=up(d["idx"]), topk_w=up(d["w"]))
        okw.update(topk_idx=d["idx"], topk_w=d["w"])
    got = m.moe_layer_few(bf(d["x"]), residual=bf(d["res"]) if res else None,
                          **kw, **more)
    ref = P.layer_few(d["x"], gu, dn, residual=d["res"] if res else None,
                      **okw)
    if router:
        np.testing.assert_array_equal(got["topk_idx"].cpu().numpy(),
                                      ref["topk_idx"])
        np.testing.assert_allclose(got["topk_w"].cpu().numpy(),
                                   ref["topk_w"], rtol=2.0 ** -23)
    y, tol = host(got["y"]), 1.05 * ref["bound"]
    mag = np.abs(ref["y"]) + (np.abs(bf16_to_f64(d["res"])) if res else 0)
    tol = tol + (k + 2) * U * mag + HALF * (np.abs(ref["y"]) + tol)
    bad = ~(np.abs(y - ref["y"]) <= tol)
    assert not bad.any(), (int(bad.sum()), np.argwhere(bad)[:4])
    # two independent bf16 roundings in the mean square: 2 x 0.0017^2
    if ref["y"].size > 500:
        assert O.rel_err(y, ref["y"]) < 4e-3
    return got


FMTS = ["bf16", "mxfp4"]


# tokens: one, each number of column sets, past one pass of an expert
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [1, 2, 3, 7, 8, 9, 16, 17, 31, 33, 64])
def test_tokens(m, T, fmt):
    check(m, make(T, 128, 96, 8, 2, T), fmt)


# sizes: the smallest, odd multiples, K tails of every kind, few and many
# experts, pairs above and below the number of experts, one expert
@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,H,F,E,k", [
    (1, 32, 32, 1, 1), (5, 64, 32, 1, 1), (3, 96, 160, 3, 3),
    (4, 1056, 224, 130, 5), (2, 2048, 768, 128, 8), (40, 160, 64, 64, 6),
    (64, 64, 64, 4, 4), (9, 352, 1376, 5, 2), (64, 32, 32, 2, 1),
    (6, 4096, 64, 4, 2), (3, 64, 4128, 4, 2), (1, 64, 64, 1024, 32),
    (64, 32, 64, 40, 32), (1, 128, 128, 4, 2), (3, 384, 640, 5, 2),
    (20, 2048, 256, 6, 2), (8, 128, 1408, 200, 3), (2, 4096, 128, 3, 1)])
def test_sizes(m, T, H, F, E, k, fmt):
    check(m, make(T, H, F, E, k, H + F), fmt)


@pytest.mark.parametrize("H,F", [(8, 8), (24, 40), (136, 72), (1000, 1048)])
def test_sizes_in_steps_of_eight(m, H, F):
    check(m, make(5, H, F, 6, 2, H), "bf16")


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,E,k,renorm,bias", [
    (1, 128, 8, True, False), (1, 128, 8, False, True), (5, 8, 2, True, True),
    (64, 300, 20, True, False), (17, 60, 4, False, False), (3, 1, 1, True,
                                                            False)])
def test_router(m, T, E, k, renorm, bias, fmt):
    check(m, make(T, 256, 64, E, k, T + E), fmt, router=True, renorm=renorm,
          bias=bias)


def test_router_equals_the_separate_entry_points(m):
    d = make(33, 512, 32, 128, 8, 3)
    kw, _, _ = weights(m, d, "bf16")
    r = m.moe_layer_few(bf(d["x"]), w_r=bf(d["wr"]), k=8,
                        router_bias=up(d["bias"]), **kw)
    lg = m.moe_router_logits(bf(d["x"]), bf(d["wr"]), up(d["bias"]))
    idx, w = m.moe_route_topk(lg, 8)
    assert torch.equal(r["topk_idx"], idx) and torch.equal(r["topk_w"], w)


@pytest.mark.parametrize("fmt", FMTS)
def test_no_residual_and_in_place(m, fmt):
    d = make(4, 96, 64, 6, 2, 1)
    check(m, d, fmt, res=False)
    kw, _, _ = weights(m, d, fmt)
    kw.update(topk_idx=up(d["idx"]), topk_w=up(d["w"]))
    r = bf(d["res"])
    a = m.moe_layer_few(bf(d["x"]), residual=r, **kw)["y"]
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    b = m.moe_layer_few(bf(d["x"]), residual=r, out=r, ws=ws, **kw)["y"]
    assert b is r and torch.equal(a, b)
    c = m.moe_layer_few(bf(d["x"][:0]), w_r=bf(d["wr"]), k=2,
                        **weights(m, d, fmt)[0])
    assert c["y"].shape == (0, 96)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [1, 12, 64])
def test_repeated_and_bad_ids(m, T, fmt):
    """An expert named twice (or four times) by a token counts as often; ids
    outside [0, E) are skipped and reported."""
    d = make(T, 128, 64, 9, 4, 40 + T)
    d["idx"][0] = [3, 5, 3, 5]
    if T > 1:
        d["idx"][1] = [7, 7, 7, 7]
        d["idx"][T - 1] = [5, 0, 1, 5]
    check(m, d, fmt)
    assert m.check_device_status() == 0
    d["idx"][T // 2] = [9, -1, 2, 2 ** 30]
    check(m, d, fmt)
    assert m.check_device_status() == 1
    d["idx"][:] = -5
    check(m, d, fmt)
    assert m.check_device_status() == 1


@pytest.mark.parametrize("fmt", FMTS)
def test_weights_of_skipped_pairs_are_not_used(m, fmt):
    """Padding by ids outside [0, E), whose weights may be anything."""
    d = make(7, 64, 64, 5, 3, 19)
    d["idx"][2] = [-1, 4, 5]
    d["w"][2] = [np.nan, 0.5, np.inf]
    d["idx"][5] = -1
    d["w"][5] = [np.inf, -np.inf, np.nan]
    y = check(m, d, fmt)["y"]
    assert torch.equal(y[5], bf(d["res"])[5])
    assert m.check_device_status() == 1


def test_infinite_and_nan_weights_stay_with_their_tokens(m):
    d = make(6, 64, 64, 5, 1, 9)
    d["idx"][:, 0] = [0, 1, 2, 0, 1, 3]
    gu, dn = d["gu"].copy(), d["dn"].copy()
    gu[1, 3, 7] = 0x7f80       # infinity
    dn[2, 5, 6] = 0x7fc0       # NaN
    dn[1, 9, 9] = 0xff80
    clean = m.moe_layer_few(bf(d["x"]), bf(d["gu"]), bf(d["dn"]),
                            up(d["idx"]), up(d["w"]))["y"]
    got = m.moe_layer_few(bf(d["x"]), bf(gu), bf(dn), up(d["idx"]),
                          up(d["w"]))["y"]
    for t in (0, 3, 5):
        assert torch.equal(got[t], clean[t])
    same = [h for h in range(64) if h != 5]
    assert torch.equal(got[2][same], clean[2][same])
    assert torch.isnan(got[2][5])
    x = d["x"].copy()
    x[4] = 0x7fc0
    got = m.moe_layer_few(bf(x), bf(d["gu"]), bf(d["dn"]), up(d["idx"]),
                          up(d["w"]))["y"]
    for t in (0, 1, 2, 3, 5):
        assert torch.equal(got[t], clean[t])
    assert torch.isnan(got[4]).all()


def test_two_streams_and_graph(m):
    """Calls on two streams at once, and a captured one replayed with other
    inputs between eager calls, each with its own workspace."""
    d = make(5, 256, 128, 16, 4, 77)
    kw, _, _ = weights(m, d, "mxfp4")
    kw.update(w_r=bf(d["wr"]), k=4, residual=bf(d["res"]))
    x = [bf(d["x"]), bf(d["x"][::-1].copy())]
    ref = [m.moe_layer_few(v, **kw)["y"].clone() for v in x]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for v, s in zip(x, streams):
        with torch.cuda.stream(s):
            outs.append([m.moe_layer_few(v, **kw)["y"] for _ in range(10)])
    torch.cuda.synchronize()
    for o, r in zip(outs, ref):
        assert all(torch.equal(y, r) for y in o)
    buf = x[0].clone()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        m.moe_layer_few(buf, **kw)
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = m.moe_layer_few(buf, **kw)["y"]
    for i in (1, 0, 1, 1, 0):
        buf.copy_(x[i])
        y.view(torch.uint8).fill_(0xA5)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref[i]), i
        m.moe_layer_few(x[1 - i], **kw)
        torch.cuda.synchronize()
