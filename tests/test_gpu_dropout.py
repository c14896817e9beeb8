"""The combine with dropout and residual on the GPU against the float64
oracle.

The mask is compared exactly through which outputs are zero or equal to the
residual.  Bounds, derived from the arithmetic: a bf16 rounding is off by at
most 2^-8 of the value; the float32 sum of k products, the scale and the
residual are k + 3 roundings of 2^-24 of the terms' sizes, the scale itself
is rounded once more; a dot product over H values has H + 4 of them.
"""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B
from synthetic import bf16_bits, bf16_to_f64

pytestmark = pytest.mark.gpu


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


def make(T, H, k, seed, holes=False):
    rng = np.random.default_rng(seed)
    d = {"z": bf16_bits(rng.standard_normal((T * k, H)).astype(np.float32)),
         "r": bf16_bits(rng.standard_normal((T, H)).astype(np.float32)),
         "dy": bf16_bits(rng.standard_normal((T, H)).astype(np.float32)),
         "cw": rng.random((T, k)).astype(np.float32),
         "map": rng.permutation(T * k).astype(np.int32)}
    if holes:
        d["map"][rng.integers(0, T * k, max(1, T * k // 5))] = -1
        d["map"][0] = T * k           # past the end: ignored as well
        d["map"][-1] = np.iinfo(np.int32).min
    return d


def check_fwd(m, d, k, p, seed, off, routed, weighted, res, **kw):
    rm = d["map"] if routed else None
    cw = d["cw"] if weighted else None
    y = m.moe_unpermute_dropout(
        dev(d["z"]), None if rm is None else torch.from_numpy(rm).cuda(), k,
        p, seed, off, topk_w=None if cw is None else
        torch.from_numpy(cw).cuda(), residual=dev(d["r"]) if res else None,
        **kw)
    o = B.unpermute_dropout(d["z"], rm, k, p, seed, off, cw,
                            d["r"] if res else None)
    got = host(y)
    assert np.all(np.abs(got - o["y"]) <= 2.0 ** -8 * np.abs(o["y"]) * 1.01 +
                  (k + 4) * 2.0 ** -24 * 1.01 * o["mag"])
    M = B.dropout_factor(*d["r"].shape, p, seed, off)
    base = bf16_to_f64(d["r"]) if res else 0.0 * got
    assert np.all(got[M == 0] == base[M == 0])
    return y


def check_bwd(m, d, k, p, seed, off, routed, weighted, dots):
    rm = d["map"] if routed else None
    cw = d["cw"] if weighted else None
    T, H = d["dy"].shape
    out = torch.full((T * k, H), -3.0, dtype=torch.bfloat16, device="cuda")
    g = m.moe_unpermute_dropout_bwd(
        dev(d["dy"]), None if rm is None else torch.from_numpy(rm).cuda(), k,
        p, seed, off, topk_w=None if cw is None else
        torch.from_numpy(cw).cuda(), z_perm=dev(d["z"]) if dots else None,
        out=out)
    o = B.unpermute_dropout_bwd(d["dy"], rm, k, p, seed, off, cw,
                                d["z"] if dots else None)
    dz = host(g["dz"])
    hole = np.isnan(o["dz"])
    assert np.all(dz[hole] == -3.0)        # left as they were
    want = np.where(hole, -3.0, o["dz"])
    assert np.all(np.abs(dz - want) <= np.abs(want) * (2.0 ** -8 * 1.01))
    if dots:
        dw = g["dtopk_w"].cpu().numpy()
        assert np.all(np.abs(dw - o["dtopk_w"]) <=
                      (H + 5) * 2.0 ** -24 * 1.01 * o["dtopk_mag"])


# vectors per row: 1, 2, 3, 7, 33, 64, 65, 128, 200, 256, 300, 520
SHAPES = [(1, 8, 1), (1, 4096, 2), (5, 16, 3), (300, 8, 2), (77, 24, 1),
          (33, 56, 4), (10, 264, 8), (9, 512, 5), (7, 520, 2), (6, 1024, 8),
          (5, 1600, 9), (4, 2048, 8), (3, 2400, 17), (3, 4160, 32)]


@pytest.mark.parametrize("T,H,k", SHAPES)
@pytest.mark.parametrize("p", [0.0, 0.1, 0.5])
def test_routed(m, T, H, k, p):
    d = make(T, H, k, T + H + k, holes=T * k > 6)
    seed, off = 0xDEADBEEF12345678, (1 << 63) + T
    for weighted in (False, True):
        for res in (False, True):
            check_fwd(m, d, k, p, seed, off, True, weighted, res)
        for dots in (False, True):
            check_bwd(m, d, k, p, seed, off, True, weighted, dots)


@pytest.mark.parametrize("T,H", [(1, 8), (3, 1000), (130, 64), (6, 2056),
                                 (2, 8192)])
def test_dense_rows(m, T, H):
    d = make(T, H, 1, T + H)
    for p in (0.05, 1.0, 2.0 ** -18, 1 - 2.0 ** -16):
        for weighted in (False, True):
            check_fwd(m, d, 1, p, 7, 0, False, weighted, True)
            check_bwd(m, d, 1, p, 7, 0, False, weighted, True)


def test_residual_in_place_and_neighbours(m):
    T, H, k = 37, 264, 2
    d = make(T, H, k, 1)
    want = check_fwd(m, d, k, 0.1, 3, 4, True, False, True)
    buf = torch.full((T + 2, H), 5.0, dtype=torch.bfloat16, device="cuda")
    r = buf[1:T + 1]
    r.copy_(dev(d["r"]))
    y = m.moe_unpermute_dropout(dev(d["z"]), torch.from_numpy(d["map"]).cuda(),
                                k, 0.1, 3, 4, residual=r, out=r)
    assert y.data_ptr() == r.data_ptr() and torch.equal(y, want)
    assert bool((buf[0] == 5).all()) and bool((buf[T + 1] == 5).all())


def test_non_finite_values_in_dropped_places(m):
    """Whatever stands in a dropped place, the output is the residual there
    and the gradient is zero."""
    T, H, k, p, seed, off = 16, 256, 2, 0.5, 11, 12
    d = make(T, H, k, 2)
    M = B.dropout_factor(T, H, p, seed, off)
    z = bf16_to_f64(d["z"])
    dy = bf16_to_f64(d["dy"])
    t, h = np.nonzero(M == 0)
    for j in range(k):
        z[d["map"][t * k + j], h] = [np.inf, np.nan][j]
    dy[t, h] = np.nan
    d["z"], d["dy"] = bf16_bits(z.astype(np.float32)), \
        bf16_bits(dy.astype(np.float32))
    check_fwd(m, d, k, p, seed, off, True, True, True)
    g = m.moe_unpermute_dropout_bwd(
        dev(d["dy"]), torch.from_numpy(d["map"]).cuda(), k, p, seed, off,
        topk_w=torch.from_numpy(d["cw"]).cuda(), z_perm=dev(d["z"]))
    assert bool(torch.isfinite(g["dz"]).all())
    assert bool(torch.isfinite(g["dtopk_w"]).all())
    check_bwd(m, d, k, p, seed, off, True, True, True)


def test_step_is_added_to_the_offset(m):
    T, H = 20, 128
    d = make(T, H, 1, 3)
    z = dev(d["z"])
    step = torch.tensor([5], dtype=torch.int64, device="cuda")
    a = m.moe_unpermute_dropout(z, None, 1, 0.3, 9, 100, step=step)
    b = m.moe_unpermute_dropout(z, None, 1, 0.3, 9, 105)
    c = m.moe_unpermute_dropout(z, None, 1, 0.3, 9, 100)
    assert torch.equal(a, b) and not torch.equal(a, c)
    ga = m.moe_unpermute_dropout_bwd(z, None, 1, 0.3, 9, 100, step=step)["dz"]
    assert torch.equal(ga, a)     # the same mask and scale on the same values


def test_zero_tokens(m):
    z = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    rm = torch.empty(0, dtype=torch.int32, device="cuda")
    assert m.moe_unpermute_dropout(z, rm, 4, 0.1, 1).shape == (0, 64)
    g = m.moe_unpermute_dropout_bwd(z, rm, 4, 0.1, 1, z_perm=z)
    assert g["dz"].shape == (0, 64) and g["dtopk_w"].shape == (0, 4)


def test_rows_past_32_bit_offsets(m):
    """z_perm of 5.2 GB: the last rows lie past 2^32 bytes."""
    T, H, k, p = 40000, 8192, 8, 0.25
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    z = torch.zeros((T * k, H), dtype=torch.bfloat16, device="cuda")
    rm = torch.arange(T * k, dtype=torch.int32, device="cuda")
    z[-k:] = torch.randn(k, H, device="cuda").bfloat16()
    y = m.moe_unpermute_dropout(z, rm, k, p, 1, 2)
    u = np.uint64
    g0 = (T - 1) * H // 8
    i = np.arange(g0, g0 + H // 8, dtype=np.uint64)
    w = B.philox4x32_10(i & u(0xFFFFFFFF), i >> u(32), np.full_like(i, 2),
                        np.full_like(i, 0), 1, 0)
    r = np.stack([h for x in w for h in (x & u(0xFFFF), x >> u(16))], 1)
    keep = r.reshape(-1) >= 16384
    s = host(z[-k:]).sum(0)
    want = np.where(keep, s * (65536 / 49152), 0.0)
    mag = np.abs(host(z[-k:])).sum(0) * (65536 / 49152)
    got = host(y[-1])
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * 1.01 * np.abs(want) +
                  12 * 2.0 ** -24 * 1.01 * mag)
    assert bool((y[:-1] == 0).all())
