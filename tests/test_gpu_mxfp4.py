"""MXFP4 on the GPU: codes and scales bit for bit against the oracle over
every finite bf16 value near every block exponent, every code and scale back,
and the 4-bit expert MLP.

The MLP is compared with the oracle running the same algorithm.  Bars: the
first product is exact where the test makes it so; z is one bf16 rounding
(at most 2^-8, 0.0017 in the mean square) and the few elements of a whose
float32 value falls on the other side of a rounding border (a share of about
1e-5, each by a third to a half of itself: 0.002), so 5e-3 normwise."""
import numpy as np
import pytest
import torch

from oracle import moe_oracle as O
from oracle import prenorm_oracle as P
from synthetic import bf16_bits, bf16_to_f64

pytestmark = pytest.mark.gpu


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


def check_quant(m, bits):
    codes, scales = m.mxfp4_quantize(bf(bits))
    rc, rs = P.mxfp4_quantize(bits)
    np.testing.assert_array_equal(scales.cpu().numpy(), rs)
    np.testing.assert_array_equal(codes.cpu().numpy(), rc)
    back = m.mxfp4_dequantize(codes, scales)
    want = bf16_bits(P.mxfp4_dequantize(rc, rs).astype(np.float32))
    got = back.cpu().view(torch.int16).numpy().view(np.uint16)
    np.testing.assert_array_equal(got, want.reshape(got.shape))


def test_every_value_near_every_block_exponent(m):
    rows = []
    for e in range(0, 255):
        # the block's largest value, and all magnitudes of the exponents
        # that do not round to zero in it (and two below)
        lo = max(0, (e - 5) * 128)
        mags = np.arange(lo, (e + 1) * 128, dtype=np.uint16)
        vals = np.concatenate([mags, mags | 0x8000])
        pad = -len(vals) % 31
        vals = np.concatenate([vals, np.zeros(pad, np.uint16)]).reshape(-1, 31)
        top = np.full((len(vals), 1), e * 128 + 127, np.uint16)
        rows.append(np.concatenate([vals, top], axis=1))
    check_quant(m, np.concatenate(rows))


@pytest.mark.parametrize("shape", [(1, 32), (3, 64), (257, 4096), (5, 7, 96),
                                   (1, 2, 3, 32), (64,), (4097, 32)])
def test_shapes(m, shape):
    rng = np.random.default_rng(sum(shape))
    v = rng.standard_normal(shape) * np.exp(2 * rng.standard_normal(shape))
    v[..., :2] = 0
    check_quant(m, bf16_bits(v.astype(np.float32)))


def test_zero_blocks_and_empty(m):
    bits = np.zeros((2, 64), np.uint16)
    bits[0, 3] = 0x8000
    check_quant(m, bits)
    for shape in [(0, 64), (4, 0)]:
        c, s = m.mxfp4_quantize(torch.empty(shape, dtype=torch.bfloat16,
                                            device="cuda"))
        assert c.shape == (shape[0], shape[1] // 2)
        assert m.mxfp4_dequantize(c, s).shape == shape


def test_every_code_and_scale_back(m):
    codes = np.tile(np.arange(256, dtype=np.uint8), (255, 1))
    scales = np.tile(np.arange(255, dtype=np.uint8)[:, None], (1, 16))
    got = host(m.mxfp4_dequantize(up(codes), up(scales)))
    want = P.mxfp4_dequantize(codes, scales)
    with np.errstate(over="ignore"):
        want = bf16_to_f64(bf16_bits(want.astype(np.float32)))
    np.testing.assert_array_equal(got, want)


def test_large_tensor_grid(m):
    """More chunks than one round of the grid."""
    n = 65536 * 1024 * 8 + 4096
    t = torch.randn(n // 64, dtype=torch.float32, device="cuda").bfloat16()
    t = t.repeat(64)[: n // 32 * 32].view(-1, 32)
    c, s = m.mxfp4_quantize(t)
    c1, s1 = m.mxfp4_quantize(t[-4096:].contiguous())
    assert torch.equal(c[-4096:], c1) and torch.equal(s[-4096:], s1)
    b = m.mxfp4_dequantize(c, s)
    assert torch.equal(b[-4096:], m.mxfp4_dequantize(c1, s1))


# ---- the expert MLP ---------------------------------------------------------
def make(sizes, H, F, seed, std=0.05):
    rng = np.random.default_rng(seed)
    E, rows = len(sizes), sum(sizes)
    n = lambda shape, s: bf16_bits((rng.standard_normal(shape) * s)
                                   .astype(np.float32))
    return {"x": n((rows, H), 1.0), "gu": n((E, 2 * F, H), std),
            "dn": n((E, H, F), std),
            "w": rng.random(rows).astype(np.float32),
            "off": np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)}


def oracle(d, weighted=True):
    return P.mlp_mxfp4(d["x"], P.mxfp4_quantize(d["gu"]),
                       P.mxfp4_quantize(d["dn"]),
                       d["w"] if weighted else None, d["off"])


def run(m, d, mode, weighted=True, **kw):
    kw["w_perm"] = up(d["w"]) if weighted else None
    if mode == "bf16 weights":
        a = (bf(d["gu"]), bf(d["dn"]))
    else:
        a = (None, None)
        kw["w_gu_q"] = m.mxfp4_quantize(bf(d["gu"]))
        kw["w_dn_q"] = m.mxfp4_quantize(bf(d["dn"]))
    x = bf(d["x"])
    if mode == "codes":
        x, kw["x_perm_scale"] = m.mxfp4_quantize(x)
    return m.moe_grouped_mlp_fwd(x, *a, up(d["off"]),
                                 precision=m.PREC_MXFP4, **kw)


CASES = [([1], 128, 128), ([3, 0, 70, 1], 256, 384), ([300, 5], 384, 256),
         ([256, 257], 512, 640), ([17] * 5, 1280, 128), ([33, 600], 128, 1408),
         ([40, 1, 0, 9], 2048, 768)]


@pytest.mark.parametrize("sizes,H,F", CASES)
def test_mlp(m, sizes, H, F):
    d = make(sizes, H, F, H + F)
    ref = oracle(d)
    z = [run(m, d, mode)["z"] for mode in ("bf16 weights", "weight codes",
                                           "codes")]
    assert O.rel_err(host(z[0]), ref["z"]) < 5e-3
    assert torch.equal(z[0], z[1]) and torch.equal(z[0], z[2])


# at most twelve rows per expert on average: the kernels for few rows, with
# entries of up to eight (five and fewer) or sixteen rows, experts that need
# several entries, one expert, every K tail
FEW = [([1], 128, 128), ([5, 0, 1, 12], 256, 384), ([8] * 16, 384, 256),
       ([1] * 40, 512, 640), ([64] + [0] * 15, 1280, 128),
       ([0, 3, 0, 61, 0, 0, 0, 0], 128, 1408), ([9, 16, 17, 1, 0, 5, 7, 8],
                                                2048, 768),
       ([2, 40, 0, 0, 0, 0, 1, 0], 640, 384), ([7], 256, 128), ([8], 128, 256),
       ([12] * 5, 256, 256), ([0, 33, 3], 384, 128)]


@pytest.mark.parametrize("sizes,H,F", FEW)
def test_mlp_few_rows(m, sizes, H, F):
    d = make(sizes, H, F, H + F)
    ref = oracle(d)
    z = [run(m, d, mode)["z"] for mode in ("bf16 weights", "weight codes",
                                           "codes")]
    assert O.rel_err(host(z[0]), ref["z"]) < 5e-3
    assert torch.equal(z[0], z[1]) and torch.equal(z[0], z[2])
    # without a weight; and the tiled kernels, which run with the saves
    a = run(m, d, "codes", weighted=False)["z"]
    assert O.rel_err(host(a), oracle(d, weighted=False)["z"]) < 5e-3
    b = run(m, d, "codes", weighted=False, save=True)["z"]
    assert O.rel_err(host(a), host(b)) < 5e-3


def test_mlp_rows_behind_the_last_are_untouched(m):
    """Outputs of a larger buffer past the rows keep what they held."""
    for sizes in ([3, 1, 9, 2], [200, 30]):
        d = make(sizes, 256, 128, 6)
        rows = sum(sizes)
        buf = torch.full((rows + 40, 256), 7.0, dtype=torch.bfloat16,
                         device="cuda")
        z = run(m, d, "codes", out=buf[:rows])["z"]
        assert z.data_ptr() == buf.data_ptr()
        assert bool((buf[rows:] == 7.0).all())
        assert O.rel_err(host(z), oracle(d)["z"]) < 5e-3


def test_mlp_saves_and_no_weight(m):
    d = make([50, 0, 3], 256, 256, 2)
    ref = oracle(d, weighted=False)
    r = run(m, d, "weight codes", weighted=False, save=True)
    assert O.rel_err(host(r["z"]), ref["z"]) < 5e-3
    # float32 sums of exact products, one bf16 rounding
    x = np.abs(P._round_trip(d["x"]))
    gu = np.abs(P._round_trip(d["gu"]))
    for e in range(3):
        q = slice(d["off"][e], d["off"][e + 1])
        tol = 2.0 ** -8 * np.abs(ref["h1"][q]) + 258 * 2.0 ** -24 * \
            (x[q] @ gu[e].T) * 1.01
        assert np.all(np.abs(host(r["h1"])[q] - ref["h1"][q]) <= tol)
    assert O.rel_err(host(r["a"]), ref["a"]) < 3e-3


@pytest.mark.parametrize("H", [256, 384, 768])
def test_operand_layout_exactly(m, H):
    """Few non-zero elements with a scale of their own per block: every sum
    fits bf16, so a misplaced element, half-byte or scale shows."""
    rng = np.random.default_rng(H)
    E, F, rows = 2, 128, 300
    def sparse(shape):
        n = np.zeros(shape[:-1] + (shape[-1],), np.uint8)
        hit = rng.random(n.shape) < 3.0 / H
        n[hit] = rng.integers(1, 16, hit.sum())
        codes = n[..., 0::2] | (n[..., 1::2] << 4)
        scales = rng.integers(126, 129, shape[:-1] + (shape[-1] // 32,))
        return codes.astype(np.uint8), scales.astype(np.uint8)
    x, gu, dn = sparse((rows, H)), sparse((E, 2 * F, H)), sparse((E, H, F))
    off = np.array([0, 37, rows], np.int32)
    r = m.moe_grouped_mlp_fwd(up(x[0]), None, None, up(off),
                              precision=m.PREC_MXFP4,
                              x_perm_scale=up(x[1]),
                              w_gu_q=(up(gu[0]), up(gu[1])),
                              w_dn_q=(up(dn[0]), up(dn[1])), save=True)
    ref = P.mlp_mxfp4(x[0], gu, dn, None, off, x_scale=x[1])
    want = bf16_to_f64(bf16_bits(ref["h1"].astype(np.float32)))
    np.testing.assert_array_equal(host(r["h1"]), want)
    assert O.rel_err(host(r["z"]), ref["z"]) < 5e-3


def test_mlp_empty_and_bad_offsets(m):
    d = make([0, 0], 128, 128, 1)
    assert run(m, d, "weight codes")["z"].shape == (0, 128)
    for sizes in ([4, 4], [40, 4]):
        d = make(sizes, 128, 128, 1)
        d["off"][1] = 60
        run(m, d, "weight codes")
        assert m.check_device_status() == 2
        assert m.check_device_status() == 0
