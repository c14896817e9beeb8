"""The pre-norm half of a transformer block as it runs: layer norm, router,
experts, residual stream.

Training: norm, routing, permutation, expert MLP and back to the gradients of
the norm's input, weight and bias.  Prompts: the same with the experts in
MXFP4.  Decoding: layers of norm and moe_layer_few over the same MXFP4
weights.  Against the float64 oracle (bf16 bars: 2e-2 normwise; routing is
exact on the norm's own output), captured and replayed, and on two streams.
"""
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


def dev(a):
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        return torch.from_numpy(a.view(np.int16)).view(torch.bfloat16).cuda()
    return torch.from_numpy(a).cuda()


def bits(t):
    return t.cpu().view(torch.int16).numpy().view(np.uint16)


def host(t):
    return bf16_to_f64(bits(t)) if t.dtype == torch.bfloat16 else \
        t.cpu().numpy().astype(np.float64)


def make(T, H, F, E, seed):
    rng = np.random.default_rng(seed)
    n = lambda shape, s: bf16_bits((rng.standard_normal(shape) * s)
                                   .astype(np.float32))
    return {"h": (2 * rng.standard_normal((T, H)) + 0.5).astype(np.float32),
            "g": (1 + 0.2 * rng.standard_normal(H)).astype(np.float32),
            "b": (0.2 * rng.standard_normal(H)).astype(np.float32),
            "w_r": n((E, H), H ** -0.5), "w_gu": n((E, 2 * F, H), H ** -0.5),
            "w_dn": n((E, H, F), F ** -0.5), "dy": n((T, H), 1.0)}


T, H, F, E, K = 300, 128, 192, 16, 3


def train(m, g):
    """Residual stream in float32, as its gradient is."""
    s = m.moe_layernorm_fwd(g["h"], g["g"], g["b"], save=True)
    x = s["y"]
    lg = m.moe_router_logits(x, g["w_r"])
    idx, w = m.moe_route_topk(lg, K)
    p = m.moe_permute(x, idx, E, topk_w=w)
    r = m.moe_grouped_mlp_fwd(p["x_perm"], g["w_gu"], g["w_dn"],
                              p["offsets"], w_perm=p["w_perm"], save=True)
    out = {"x": x, "idx": idx,
           "y": m.moe_unpermute(r["z"], p["row_map"], K).float() + g["h"]}
    dz = m.moe_gather_rows(g["dy"], p["row_map"], K)
    e = m.moe_grouped_mlp_bwd(dz, p["x_perm"], g["w_gu"], g["w_dn"],
                              p["offsets"], r["h1"], r["a"],
                              w_perm=p["w_perm"])
    dw = m.moe_unpermute_probs_grad(e["dw_perm"], p["row_map"], K)
    q = m.moe_router_bwd(lg, idx, dw, x, g["w_r"])
    dx = (m.moe_unpermute(e["dx_perm"], p["row_map"], K).float() +
          q["dx"]).bfloat16()
    n = m.moe_layernorm_bwd(dx, g["h"], s["mean"], s["rstd"], g["g"],
                            dresidual=g["dy"].float())
    out.update(dw_gu=e["dw_gu"], dw_dn=e["dw_dn"], dw_r=q["dw_r"], **n)
    return out


def train_oracle(d, x_bits, idx):
    """From the norm's output as the GPU rounded it."""
    lg = O.router_logits(x_bits, d["w_r"])
    ri, w = O.route_topk(lg, K)
    np.testing.assert_array_equal(idx, ri)
    pm = O.permute_index(ri, E)
    X = bf16_to_f64(x_bits)
    xp, wp = X[pm["src_row"] // K], w.reshape(-1)[pm["src_row"]]
    f = O.grouped_mlp_fwd(xp, d["w_gu"], d["w_dn"], wp, pm["offsets"])
    y = O.unpermute(f["z"], pm["row_map"], K) + d["h"].astype(np.float64)
    dy = bf16_to_f64(d["dy"])
    dz = dy[pm["src_row"] // K]
    g = O.grouped_mlp_bwd(dz, xp, d["w_gu"], d["w_dn"], wp, pm["offsets"])
    dw = O.probs_grad(g["dw_perm"], pm["row_map"], K)
    dl = O.router_bwd(lg, ri, dw)
    dw_r, dxr = O.router_weight_grads(dl, x_bits, d["w_r"])
    dx = O.unpermute(g["dx_perm"], pm["row_map"], K) + dxr
    st = P.layernorm_fwd(d["h"], d["g"], d["b"])
    n = P.layernorm_bwd(dx, d["h"], st["mean"], st["rstd"], d["g"], dy)
    return dict(y=y, dw_gu=g["dw_gu"], dw_dn=g["dw_dn"], dw_r=dw_r, **n)


def replay_equals_eager(run, change, reps=4):
    """Captured once; every replay equals the eager call on that replay's
    inputs, with eager work between the replays."""
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run()
    seen = []
    for rep in range(reps):
        change(rep)
        for v in got.values():
            v.view(torch.uint8).fill_(0xA5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        kept = {n: v.clone() for n, v in got.items()}
        want = run()
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(kept[n].view(torch.uint8),
                               want[n].view(torch.uint8)), (rep, n)
        seen.append(kept["y"])
    assert not torch.equal(seen[0], seen[1])


def test_training(m):
    d = make(T, H, F, E, 1)
    out = train(m, {n: dev(v) for n, v in d.items()})
    assert m.check_device_status() == 0
    x = P.layernorm_fwd(d["h"], d["g"], d["b"])["y"]
    assert O.rel_err(host(out["x"]), x) < 4e-3
    ref = train_oracle(d, bits(out["x"]), out["idx"].cpu().numpy())
    for n, v in ref.items():
        assert O.rel_err(host(out[n]), v) < 2e-2, n


def test_training_graph(m):
    g = {n: dev(v) for n, v in make(T, H, F, E, 2).items()}
    other = [dev(make(T, H, F, E, 10 + r)["h"]) for r in range(4)]
    replay_equals_eager(lambda: train(m, g),
                        lambda rep: g["h"].copy_(other[rep]))


def serving(m, d):
    g = {n: dev(d[n]) for n in ("h", "g", "b", "w_r")}
    g["gu"] = m.mxfp4_quantize(dev(d["w_gu"]))
    g["dn"] = m.mxfp4_quantize(dev(d["w_dn"]))
    return g


def prompt(m, g, k):
    x = m.moe_layernorm_fwd(g["h"], g["g"], g["b"])["y"]
    idx, w = m.moe_route_topk(m.moe_router_logits(x, g["w_r"]), k)
    p = m.moe_permute(x, idx, g["w_r"].shape[0], topk_w=w)
    z = m.moe_grouped_mlp_fwd(p["x_perm"], None, None, p["offsets"],
                              w_perm=p["w_perm"], precision=m.PREC_MXFP4,
                              w_gu_q=g["gu"], w_dn_q=g["dn"])["z"]
    return {"y": m.moe_unpermute(z, p["row_map"], k), "x": x, "idx": idx}


def decode(m, g, k, layers=3):
    h = g["h"].bfloat16()
    out = {}
    for i in range(layers):
        x = m.moe_layernorm_fwd(h, g["g"], g["b"])["y"]
        r = m.moe_layer_few(x, w_r=g["w_r"], k=k, w_gu_q=g["gu"],
                            w_dn_q=g["dn"], precision=m.PREC_MXFP4,
                            residual=h)
        out.update({f"h{i}": h, f"x{i}": x, f"idx{i}": r["topk_idx"]})
        h = r["y"]
    out["y"] = h
    return out


# few rows per expert and many (the tiled kernels)
@pytest.mark.parametrize("T,F,E,k", [(21, 256, 16, 3), (300, 384, 6, 2)])
def test_prompt(m, T, F, E, k):
    d = make(T, 256, F, E, T)
    g = serving(m, d)
    r = prompt(m, g, k)
    lg = O.router_logits(bits(r["x"]), d["w_r"])
    idx, w = O.route_topk(lg, k)
    np.testing.assert_array_equal(r["idx"].cpu().numpy(), idx)
    pm = O.permute_index(idx, E)
    xp = bits(r["x"])[pm["src_row"] // k]
    f = P.mlp_mxfp4(xp, P.mxfp4_quantize(d["w_gu"]),
                    P.mxfp4_quantize(d["w_dn"]),
                    w.reshape(-1)[pm["src_row"]], pm["offsets"])
    assert O.rel_err(host(r["y"]), O.unpermute(f["z"], pm["row_map"], k)) \
        < 2e-2
    other = [dev(make(T, 256, 32, E, 50 + i)["h"]) for i in range(4)]
    replay_equals_eager(lambda: prompt(m, g, k),
                        lambda rep: g["h"].copy_(other[rep]))


@pytest.mark.parametrize("T,E,k", [(1, 32, 4), (5, 8, 2), (40, 16, 2)])
def test_decode(m, T, E, k):
    d = make(T, 256, 128, E, 60 + T)
    g = serving(m, d)
    r = decode(m, g, k)
    gu, dn = P._round_trip(d["w_gu"]), P._round_trip(d["w_dn"])
    for i in range(3):                  # each layer from its own input
        h = bits(r[f"h{i}"])
        x = P.layernorm_fwd(h, d["g"], d["b"])["y"]
        assert O.rel_err(host(r[f"x{i}"]), x) < 4e-3
        ref = P.layer_few(bits(r[f"x{i}"]), gu, dn, w_r=d["w_r"], k=k,
                          residual=h)
        np.testing.assert_array_equal(r[f"idx{i}"].cpu().numpy(),
                                      ref["topk_idx"])
        y = r["y"] if i == 2 else r[f"h{i + 1}"]
        assert O.rel_err(host(y), ref["y"]) < 4e-3
    other = [dev(make(T, 256, 32, E, 70 + i)["h"]) for i in range(4)]
    replay_equals_eager(lambda: decode(m, g, k),
                        lambda rep: g["h"].copy_(other[rep]))


def test_prompt_and_decode_on_two_streams(m):
    """A prompt and a decode step in flight at once over the same weights."""
    gp = serving(m, make(77, 256, 256, 32, 5))
    gd = dict(gp, h=dev(make(9, 256, 32, 32, 6)["h"]))
    want_p, want_d = prompt(m, gp, 4), decode(m, gd, 4)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    for st in (a, b):
        st.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(4):
        with torch.cuda.stream(a):
            p = prompt(m, gp, 4)
        with torch.cuda.stream(b):
            got.append((p, decode(m, gd, 4)))
    torch.cuda.synchronize()
    for p, q in got:
        for n in want_p:
            assert torch.equal(p[n], want_p[n]), n
        for n in want_d:
            assert torch.equal(q[n], want_d[n]), n
