"""NaN and infinity through MXFP4: a block that holds one gets the scale byte
255, reads back as NaN, and makes every product with it NaN, in the block's
own row and nowhere else (bit for bit)."""
import numpy as np
import pytest
import torch

from synthetic import bf16_bits

pytestmark = pytest.mark.gpu
NAN, INF, NINF = 0x7fc0, 0x7f80, 0xff80


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


def normal(rng, shape, std=1.0):
    return bf16_bits((rng.standard_normal(shape) * std).astype(np.float32))


# quiet and signalling patterns, both signs, next to zeros and large values
@pytest.mark.parametrize("bad", [NAN, 0x7f81, 0xffff, INF, NINF])
@pytest.mark.parametrize("at", [0, 13, 31])
def test_quantise_and_back(m, bad, at):
    v = normal(np.random.default_rng(at), (9, 192))
    v[5, 64:96] = 0
    v[8, 0] = 0x7f7f
    c0, s0 = m.mxfp4_quantize(bf(v))
    b0 = m.mxfp4_dequantize(c0, s0)
    hit = [(0, 0), (2, 5), (5, 2), (8, 0)]   # (row, block)
    for r, b in hit:
        v[r, 32 * b + at] = bad
    c1, s1 = m.mxfp4_quantize(bf(v))
    b1 = m.mxfp4_dequantize(c1, s1)
    clean = torch.ones((9, 6), dtype=torch.bool, device="cuda")
    for r, b in hit:
        clean[r, b] = False
    assert bool((s1[~clean] == 255).all())
    assert torch.equal(s1[clean], s0[clean])
    blocks = lambda t, n: t.view(9, 6, n)
    assert torch.equal(blocks(c1, 16)[clean], blocks(c0, 16)[clean])
    assert torch.equal(blocks(b1, 32)[clean], blocks(b0, 32)[clean])
    assert bool(torch.isnan(blocks(b1, 32)[~clean]).all())


def test_scale_255_reads_back_as_nan_under_every_code(m):
    codes = np.arange(256, dtype=np.uint8).reshape(16, 16)
    scales = np.full((16, 1), 255, np.uint8)
    assert bool(torch.isnan(m.mxfp4_dequantize(up(codes), up(scales))).all())


# ---- the expert MLP: the kernels for few rows (one and two column sets) and
# the tiled ones, whole and half last K steps
MLP = [([3, 0, 5, 1], 256, 384), ([9, 11, 8, 4], 384, 256),
       ([70, 3, 0, 41], 384, 256), ([300, 17, 5, 1], 512, 128)]


def mlp(m, d, mode, save=False):
    x, kw = bf(d["x"]), {}
    gu, dn = bf(d["gu"]), bf(d["dn"])
    if mode == "codes":
        x, kw["x_perm_scale"] = m.mxfp4_quantize(x)
        kw["w_gu_q"], kw["w_dn_q"] = m.mxfp4_quantize(gu), m.mxfp4_quantize(dn)
        gu = dn = None
    return m.moe_grouped_mlp_fwd(x, gu, dn, up(d["off"]), w_perm=up(d["w"]),
                                 precision=m.PREC_MXFP4, save=save, **kw)["z"]


def make(sizes, H, F):
    rng = np.random.default_rng(H + F)
    E, rows = len(sizes), sum(sizes)
    return {"x": normal(rng, (rows, H)),
            "gu": normal(rng, (E, 2 * F, H), 0.05),
            "dn": normal(rng, (E, H, F), 0.05),
            "w": rng.random(rows).astype(np.float32),
            "off": np.concatenate([[0], np.cumsum(sizes)]).astype(np.int32)}


def same_but(got, clean, rows, cols=None):
    """NaN in got[rows, cols], clean's bits elsewhere."""
    bad = torch.zeros(got.shape, dtype=torch.bool, device="cuda")
    for r in rows:
        if cols is None:
            bad[r] = True
        else:
            bad[r, cols] = True
    assert bool(torch.isnan(got[bad]).all())
    assert torch.equal(got[~bad], clean[~bad])


@pytest.mark.parametrize("mode", ["bf16", "codes"])
@pytest.mark.parametrize("sizes,H,F", MLP)
def test_mlp(m, sizes, H, F, mode):
    d = make(sizes, H, F)
    off, rows = d["off"], sum(sizes)
    e = int(np.argmax(sizes))
    mine = list(range(off[e], off[e + 1]))
    for save in (False, True):   # (the saves come with the tiled kernels)
        clean = mlp(m, d, mode, save)
        assert bool(torch.isfinite(clean).all())
        for bad in (NAN, INF, NINF):
            # activations: the first, a middle and the last row
            x = d["x"].copy()
            hit = sorted({0, rows // 2, rows - 1})
            for i, r in enumerate(hit):
                x[r, (37 * i + H - 1) % H] = bad
            same_but(mlp(m, dict(d, x=x), mode, save), clean, hit)
        gu, dn = d["gu"].copy(), d["dn"].copy()
        gu[e, F - 1, 5] = NAN
        same_but(mlp(m, dict(d, gu=gu), mode, save), clean, mine)
        gu = d["gu"].copy()
        gu[e, F + 3, H - 1] = INF
        same_but(mlp(m, dict(d, gu=gu), mode, save), clean, mine)
        dn[e, 7, F - 1] = NINF
        dn[e, H - 1, 0] = NAN
        same_but(mlp(m, dict(d, dn=dn), mode, save), clean, mine, [7, H - 1])


@pytest.mark.parametrize("sizes,H,F", MLP)
def test_activations_that_overflow(m, sizes, H, F):
    """A beyond float32, and routing weights that are no numbers."""
    d = make(sizes, H, F)
    rows = sum(sizes)
    x = d["x"].copy()
    x[0] = 0x7f00          # 2^127: gate times up passes 2^128
    hit, w = [0], d["w"].copy()
    for r, v in ((1, np.nan), (rows // 2, np.inf), (rows - 1, -np.inf)):
        w[r] = v
        hit.append(r)
    for save in (False, True):
        clean = mlp(m, d, "bf16", save)
        same_but(mlp(m, dict(d, x=x, w=w), "bf16", save), clean, hit)


# ---- the layer for a few tokens over MXFP4 weights: byte and dword scales,
# column sets of two and of eight tokens
@pytest.mark.parametrize("T,H,F,k", [(1, 96, 64, 1), (5, 96, 64, 1),
                                     (1, 256, 128, 1), (7, 256, 128, 1),
                                     (12, 256, 128, 3), (40, 128, 256, 2)])
def test_layer_few(m, T, H, F, k):
    rng = np.random.default_rng(T)
    E = 6
    x, gu, dn = normal(rng, (T, H)), normal(rng, (E, 2 * F, H), 0.05), \
        normal(rng, (E, H, F), 0.05)
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    w = rng.random((T, k)).astype(np.float32)
    idx[0, 0] = 2

    def run(gu, dn):
        return m.moe_layer_few(
            bf(x), topk_idx=up(idx), topk_w=up(w), precision=m.PREC_MXFP4,
            w_gu_q=m.mxfp4_quantize(bf(gu)),
            w_dn_q=m.mxfp4_quantize(bf(dn)))["y"]
    clean = run(gu, dn)
    assert bool(torch.isfinite(clean).all())
    hit = [t for t in range(T) if 2 in idx[t]]
    for bad in (NAN, INF):
        g = gu.copy()
        g[2, F + 9, H - 1] = bad
        same_but(run(g, dn), clean, hit)
        g = gu.copy()
        g[2, 9, 0] = bad
        same_but(run(g, dn), clean, hit)
        n = dn.copy()
        n[2, H - 2, F - 1] = bad
        n[2, 3, 31] = bad
        same_but(run(gu, n), clean, hit, [3, H - 2])


@pytest.mark.parametrize("T,H,F,k", [(2, 96, 64, 2), (2, 256, 128, 3),
                                     (9, 128, 256, 2), (12, 256, 128, 1),
                                     (40, 128, 256, 2)])
def test_layer_few_keeps_tokens_apart(m, T, H, F, k):
    """NaN in one token's activations, next to others in its
    column sets."""
    rng = np.random.default_rng(T + F)
    E = 6
    x = normal(rng, (T, H))
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)]).astype(np.int32)
    q = [m.mxfp4_quantize(bf(normal(rng, s, 0.05)))
         for s in ((E, 2 * F, H), (E, H, F))]
    w = up(rng.random((T, k)).astype(np.float32))

    def run(x):
        return m.moe_layer_few(bf(x), topk_idx=up(idx), topk_w=w,
                               precision=m.PREC_MXFP4, w_gu_q=q[0],
                               w_dn_q=q[1])["y"]
    clean = run(x)
    for t in sorted({0, T // 2, T - 1}):
        bad = x.copy()
        bad[t] = NAN
        same_but(run(bad), clean, [t])
        bad = x.copy()
        bad[t, H - 3] = NAN
        same_but(run(bad), clean, [t])
