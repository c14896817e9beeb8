"""Pins of oracle/block_oracle.py: hand cases, published outputs of the
counter-based generator, central differences of every backward."""
import numpy as np
import pytest

from oracle import block_oracle as B
from oracle import moe_oracle as O


def test_philox_published_vectors():
    """The known answers published with the Random123 generators."""
    u = lambda *v: [np.array([x], np.uint64) for x in v]
    cases = [
        ((0, 0, 0, 0), (0, 0),
         (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
        ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2,
         (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
        ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344),
         (0xA4093822, 0x299F31D0),
         (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
    ]
    for ctr, key, want in cases:
        got = B.philox4x32_10(*u(*ctr), *key)
        assert tuple(int(g[0]) for g in got) == want


def test_dropout_factor_share_and_words():
    M = B.dropout_factor(512, 64, 0.25, 1234567890123456789, 77)
    kept = M > 0
    # 32768 draws: five standard deviations
    assert abs(kept.mean() - 0.75) < 5 * np.sqrt(0.25 * 0.75 / M.size)
    assert np.all(M[kept] == 65536 / (65536 - 16384))
    # value 9 is bits 16..31 of group 1
    u = lambda v: np.array([v], np.uint64)
    w = B.philox4x32_10(u(1), u(0), u(77), u(0), 1234567890123456789 &
                        0xFFFFFFFF, 1234567890123456789 >> 32)
    assert (M.reshape(-1)[9] > 0) == ((int(w[0][0]) >> 16) >= 16384)
    assert np.all(B.dropout_factor(4, 8, 1.0, 1, 1) == 0)
    assert np.all(B.dropout_factor(4, 8, 0.0, 1, 1) == 1)


def test_route_scored_hand_case():
    # two groups of three; the bias promotes expert 5, group 0 wins by max
    lg = np.log(np.array([[3.0, 1, 1, 1, 1, 2]], np.float32) / 9)
    idx, w = B.route_scored(lg, 2, renormalize=False)
    assert idx.tolist() == [[0, 5]]
    np.testing.assert_allclose(w, [[3 / 9, 2 / 9]], rtol=1e-6)
    idx, w = B.route_scored(lg, 2, n_group=2, topk_group=1)
    assert idx.tolist() == [[0, 1]]
    np.testing.assert_allclose(w, [[0.75, 0.25]], rtol=1e-6)
    bias = np.array([0, 0, 0, 0, 0, 0.5], np.float32)
    idx, w = B.route_scored(lg, 2, bias=bias, scale=2.0)
    assert idx.tolist() == [[5, 0]]
    np.testing.assert_allclose(w, [[0.8, 1.2]], rtol=1e-6)
    # sums of two largest: 4/9 against 3/9
    idx, _ = B.route_scored(lg, 1, n_group=2, topk_group=1,
                            group_score="top2")
    assert idx.tolist() == [[0]]


def test_route_scored_reduces_to_route_topk():
    rng = np.random.default_rng(1)
    lg = np.round(rng.standard_normal((50, 24)) * 2).astype(np.float32)
    for ren in (True, False):
        i0, w0 = O.route_topk(lg, 5, ren)
        i1, w1 = B.route_scored(lg, 5, renormalize=ren)
        np.testing.assert_array_equal(i0, i1)
        np.testing.assert_allclose(w1, w0, rtol=1e-6)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_scored_bwd_differences(score, renorm):
    """With the selection held fixed; logits stepped as float32 values whose
    step is exact, so the quotient uses the step that was taken."""
    rng = np.random.default_rng(2)
    T, E, k = 3, 10, 4
    lg = (np.round(rng.standard_normal((T, E)) * 64) / 64).astype(np.float32)
    dw = rng.standard_normal((T, k))
    idx, _ = B.route_scored(lg, k, score=score)

    def weights(l):
        s = B.scores(l, score)
        w = np.take_along_axis(s, idx.astype(np.int64), 1)
        return 1.7 * (w / w.sum(1, keepdims=True) if renorm else w)
    dl = B.route_scored_bwd(lg, idx, dw, score, renorm, 1.7)
    h = np.float32(2.0 ** -10)
    for t in range(T):
        for e in range(E):
            a, b = lg.copy(), lg.copy()
            a[t, e] += h
            b[t, e] -= h
            fd = ((weights(a) - weights(b)) * dw).sum() / (2 * float(h))
            # central difference: h^2 / 6 times a third derivative below 20
            assert abs(fd - dl[t, e]) < 2.0 ** -20 / 6 * 20


@pytest.mark.parametrize("name", ["none", "relu", "gelu", "gelu_tanh",
                                  "silu"])
def test_linear_bwd_differences(name):
    rng = np.random.default_rng(3)
    M, N, K = 3, 4, 5
    x, w = rng.standard_normal((M, K)), rng.standard_normal((N, K))
    b, dy = rng.standard_normal(N), rng.standard_normal((M, N))
    f = B.linear_fwd(x, w, b, name)
    g = B.linear_bwd(dy, x, w, name, f["z"])

    def loss(x, w, b):
        return (B.linear_fwd(x, w, b, name)["y"] * dy).sum()
    h = 1e-6
    for arr, grad, at in ((x, g["dx"], 0), (w, g["dw"], 1), (b, g["db"], 2)):
        for i in np.ndindex(arr.shape):
            args = [x, w, b]
            hi, lo = arr.copy(), arr.copy()
            hi[i] += h
            lo[i] -= h
            args[at] = hi
            up = loss(*args)
            args[at] = lo
            fd = (up - loss(*args)) / (2 * h)
            assert abs(fd - grad[i]) < 1e-7 * max(1.0, abs(fd)), (name, at, i)


def test_unpermute_dropout_bwd_differences():
    rng = np.random.default_rng(4)
    T, H, k = 3, 8, 2
    rm = rng.permutation(T * k)
    rm[1] = -1
    z, cw = rng.standard_normal((T * k, H)), rng.standard_normal((T, k))
    r, dy = rng.standard_normal((T, H)), rng.standard_normal((T, H))
    a = (rm, k, 0.3, 99, 5)
    g = B.unpermute_dropout_bwd(dy, *a, topk_w=cw, z_perm=z)

    def loss(z, cw):
        return (B.unpermute_dropout(z, *a, topk_w=cw, residual=r)["y"] *
                dy).sum()
    h = 1e-6
    for arr, grad, at in ((z, np.nan_to_num(g["dz"]), 0),
                          (cw, g["dtopk_w"], 1)):
        for i in np.ndindex(arr.shape):
            args = [z, cw]
            hi, lo = arr.copy(), arr.copy()
            hi[i] += h
            lo[i] -= h
            args[at] = hi
            up = loss(*args)
            args[at] = lo
            fd = (up - loss(*args)) / (2 * h)
            assert abs(fd - grad[i]) < 1e-7 * max(1.0, abs(fd))
