"""Pins of oracle/prenorm_oracle.py: hand cases, an independent decoding,
central differences, and agreement with the grouped path's oracle."""
import numpy as np
import pytest

from oracle import moe_oracle as O
from oracle import prenorm_oracle as P
from synthetic import bf16_bits


def test_layernorm_hand_case():
    x = np.array([[1.0, 2.0, 3.0, 6.0], [5.0, 5.0, 5.0, 5.0]])
    r = P.layernorm_fwd(x, np.array([1.0, 2.0, 1.0, 1.0]),
                        np.array([0.0, 0.0, 0.0, 1.0]), eps=0.5)
    # mean 3, variance (4 + 1 + 0 + 9) / 4 = 3.5: rstd 0.5
    np.testing.assert_allclose(r["mean"], [3, 5])
    np.testing.assert_allclose(r["rstd"], [0.5, np.sqrt(2)])
    np.testing.assert_allclose(r["y"], [[-1, -1, 0, 2.5], [0, 0, 0, 1]],
                               atol=1e-15)


def test_layernorm_bwd_is_the_gradient():
    rng = np.random.default_rng(3)
    T, H = 3, 7
    x, dy = rng.standard_normal((T, H)), rng.standard_normal((T, H))
    w, b = rng.standard_normal(H), rng.standard_normal(H)

    def loss(x, w, b):
        return (P.layernorm_fwd(x, w, b)["y"] * dy).sum()

    f = P.layernorm_fwd(x, w, b)
    g = P.layernorm_bwd(dy, x, f["mean"], f["rstd"], w)
    for name, v, args in (("dx", x, lambda q: (q, w, b)),
                          ("dw", w, lambda q: (x, q, b)),
                          ("db", b, lambda q: (x, w, q))):
        num = np.zeros_like(v)
        for i in np.ndindex(v.shape):
            d = np.zeros_like(v)
            d[i] = 1e-5
            num[i] = (loss(*args(v + d)) - loss(*args(v - d))) / 2e-5
        # central differences: h^2 times a third derivative of order 10
        np.testing.assert_allclose(g[name], num, rtol=1e-6, atol=1e-8)
    r = rng.standard_normal((T, H))
    g2 = P.layernorm_bwd(dy, x, f["mean"], f["rstd"], w, dresidual=r)
    np.testing.assert_allclose(g2["dx"], g["dx"] + r)


def test_mxfp4_hand_case():
    v = np.zeros(64)
    # amax 8 = 2^3: s = 1, elements v / 2
    v[:9] = [8.0, -3.0, 0.5, 1.5, 2.5, 3.5, 5.0, 7.0, -0.0]
    codes, scales = P.mxfp4_quantize(v[None])
    n = np.stack([codes[0] & 15, codes[0] >> 4], 1).reshape(-1)
    assert scales.tolist() == [[128, 0]]
    # 4, -1.5, 0.25 -> 0 (tie to even), 0.75 -> 1 (tie), 1.25 -> 1 (tie),
    # 1.75 -> 2 (tie), 2.5 -> 2 (tie), 3.5 -> 4 (tie), -0
    assert n[:9].tolist() == [6, 8 + 3, 0, 2, 2, 4, 4, 6, 8]
    v[0] = 15.0   # s = 1, 7.5: beyond 6
    codes, _ = P.mxfp4_quantize(v[None])
    assert codes[0, 0] & 15 == 7


def test_mxfp4_dequantize_every_code():
    codes = np.arange(256, dtype=np.uint8).reshape(16, 16)
    scales = np.arange(16, dtype=np.uint8)[:, None] * 17
    got = P.mxfp4_dequantize(codes, scales)
    for r in range(16):
        for c in range(16):
            for half in range(2):
                n = (int(codes[r, c]) >> (4 * half)) & 15
                e, m = (n >> 1) & 3, n & 1
                mag = 0.5 * m if e == 0 else (1 + 0.5 * m) * 2.0 ** (e - 1)
                want = (-1) ** (n >> 3) * mag * 2.0 ** (17 * r - 127)
                assert got[r, 2 * c + half] == want


def test_mxfp4_round_trip_is_idempotent_and_close():
    rng = np.random.default_rng(5)
    v = rng.standard_normal((50, 96)) * np.exp(3 * rng.standard_normal((50, 1)))
    q = P._round_trip(v)
    np.testing.assert_array_equal(P._round_trip(q), q)
    amax = np.abs(v.reshape(50, 3, 32)).max(-1).repeat(32, 1).reshape(50, 96)
    # steps are at most 2 2^s with 2^s <= amax / 4, values past 6 2^s up to
    # 8 2^s come back as 6 2^s
    assert np.all(np.abs(q - v) <= amax / 4 * 2)
    # amax < 8 2^s, so these are below 3 2^s, where steps are at most 2^s and
    # a rounding is off by at most 2^s / 2 <= amax / 8
    inside = np.abs(v) < 1.5 * amax / 4
    assert np.all(np.abs(q - v)[inside] <= amax[inside] / 8)


def test_layer_few_equals_the_grouped_layer():
    rng = np.random.default_rng(7)
    T, H, F, E, k = 5, 64, 64, 6, 3
    x = bf16_bits(rng.standard_normal((T, H)).astype(np.float32))
    gu = bf16_bits((0.1 * rng.standard_normal((E, 2 * F, H))).astype(np.float32))
    dn = bf16_bits((0.1 * rng.standard_normal((E, H, F))).astype(np.float32))
    lg = rng.standard_normal((T, E)).astype(np.float32)
    ref = O.layer_fwd(x, lg, gu, dn, k)
    got = P.layer_few(x, O._as_f64(gu), O._as_f64(dn), ref["topk_idx"],
                      O.route_topk(lg, k)[1])
    np.testing.assert_allclose(got["y"], ref["y"], rtol=1e-5, atol=1e-9)


def test_layer_few_skips_bad_ids_and_takes_a_repeated_one_twice():
    rng = np.random.default_rng(8)
    x = rng.standard_normal((1, 8))
    gu, dn = rng.standard_normal((2, 16, 8)), rng.standard_normal((2, 8, 8))
    one = P.layer_few(x, gu, dn, np.array([[1]]), np.array([[0.75]]))["y"]
    two = P.layer_few(x, gu, dn, np.array([[1, 5, 1]]),
                      np.array([[0.5, 9.0, 0.25]]))["y"]
    np.testing.assert_allclose(one, two, rtol=1e-12)
