"""Scored routing, the dense linear layer and the combine with dropout run
together with the expert MLP, as a transformer block's feed-forward half
does: a shared dense branch, routed experts, dropout on their combine, the
residual stream.  Forward and backward against the float64 oracle (bf16
bars: 2e-2 normwise), and the whole step captured in a HIP graph.
"""
import numpy as np
import pytest
import torch

from oracle import block_oracle as B
from oracle import moe_oracle as O
from synthetic import bf16_bits, bf16_to_f64, generate

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


T, H, F, E, K = 300, 128, 192, 16, 3
D = 200                       # width of the shared dense branch
P, SEED, OFF = 0.15, 1234567, 99
OPTS = dict(score="sigmoid", n_group=4, topk_group=2, group_score="top2",
            scale=2.5)


def make():
    d = generate(T, H, F, E, K, seed=4, want=("x", "w_r", "w_gu", "w_dn",
                                              "dy"))
    rng = np.random.default_rng(9)
    d["bias_r"] = (rng.standard_normal(E) * 0.05).astype(np.float32)
    d["w1"] = bf16_bits((rng.standard_normal((D, H)) * 0.05)
                        .astype(np.float32))
    d["b1"] = (rng.standard_normal(D) * 0.1).astype(np.float32)
    d["w2"] = bf16_bits((rng.standard_normal((H, D)) * 0.05)
                        .astype(np.float32))
    d["b2"] = (rng.standard_normal(H) * 0.1).astype(np.float32)
    return d


def to_gpu(d):
    g = {n: dev(d[n]) for n in ("x", "w_r", "w_gu", "w_dn", "dy", "w1", "w2")}
    g.update({n: torch.from_numpy(d[n]).cuda() for n in ("bias_r", "b1",
                                                         "b2")})
    return g


def forward(m, g, step=None):
    o = dict(score=m.SCORE_SIGMOID, n_group=4, topk_group=2,
             group_score=m.GROUP_TOP2, scale=2.5)
    s = {}
    s["logits"] = m.moe_router_logits(g["x"], g["w_r"])
    s["idx"], s["w"] = m.moe_route_scored(s["logits"], K, bias=g["bias_r"],
                                          **o)
    s["p"] = m.moe_permute(g["x"], s["idx"], E, topk_w=s["w"])
    s["r"] = m.moe_grouped_mlp_fwd(s["p"]["x_perm"], g["w_gu"], g["w_dn"],
                                   s["p"]["offsets"],
                                   w_perm=s["p"]["w_perm"], save=True)
    s["h"] = m.moe_linear_fwd(g["x"], g["w1"], bias=g["b1"], act=m.ACT_GELU,
                              save=True)
    s["shared"] = m.moe_linear_fwd(s["h"]["y"], g["w2"], bias=g["b2"],
                                   residual=g["x"])["y"]
    s["y"] = m.moe_unpermute_dropout(s["r"]["z"], s["p"]["row_map"], K, P,
                                     SEED, OFF, step=step,
                                     residual=s["shared"])
    return s


def backward(m, g, s, step=None):
    dy = g["dy"]
    out = {}
    dz = m.moe_unpermute_dropout_bwd(dy, s["p"]["row_map"], K, P, SEED, OFF,
                                     step=step)["dz"]
    e = m.moe_grouped_mlp_bwd(dz, s["p"]["x_perm"], g["w_gu"], g["w_dn"],
                              s["p"]["offsets"], s["r"]["h1"], s["r"]["a"],
                              w_perm=s["p"]["w_perm"])
    out["dw_gu"], out["dw_dn"] = e["dw_gu"], e["dw_dn"]
    out["dx_experts"] = m.moe_unpermute(e["dx_perm"], s["p"]["row_map"], K)
    out["dw"] = m.moe_unpermute_probs_grad(e["dw_perm"], s["p"]["row_map"], K)
    out["dl"] = m.moe_route_scored_bwd(s["logits"], s["idx"], out["dw"],
                                       score=m.SCORE_SIGMOID, scale=2.5)
    r = m.moe_router_proj_bwd(out["dl"], g["x"], g["w_r"])
    out["dw_r"], out["dx_router"] = r["dw_r"], r["dx"]
    a = m.moe_linear_bwd(dy, s["h"]["y"], g["w2"], want_db=True)
    out["dw2"], out["db2"] = a["dw"], a["db"]
    b = m.moe_linear_bwd(a["dx"], g["x"], g["w1"], act=m.ACT_GELU,
                         z=s["h"]["z"], want_db=True)
    out["dw1"], out["db1"], out["dx_shared"] = b["dw"], b["db"], b["dx"]
    return out


def oracle(d):
    X = bf16_to_f64(d["x"])
    logits = O.router_logits(d["x"], d["w_r"])
    idx, w = B.route_scored(logits, K, bias=d["bias_r"], **OPTS)
    pm = O.permute_index(idx, E)
    xp = X[pm["src_row"] // K]
    wp = w.reshape(-1)[pm["src_row"]]
    f = O.grouped_mlp_fwd(xp, d["w_gu"], d["w_dn"], wp, pm["offsets"])
    h = B.linear_fwd(d["x"], d["w1"], d["b1"], "gelu")
    sh = B.linear_fwd(h["y"], bf16_to_f64(d["w2"]), d["b2"], "none", X)["y"]
    y = B.unpermute_dropout(f["z"], pm["row_map"], K, P, SEED, OFF,
                            residual=sh)["y"]
    dy = bf16_to_f64(d["dy"])
    dz = B.unpermute_dropout_bwd(dy, pm["row_map"], K, P, SEED, OFF)["dz"]
    g = O.grouped_mlp_bwd(dz, xp, d["w_gu"], d["w_dn"], wp, pm["offsets"])
    dw = O.probs_grad(g["dw_perm"], pm["row_map"], K)
    dl = B.route_scored_bwd(logits, idx, dw, "sigmoid", True, 2.5)
    dw_r, dxr = O.router_weight_grads(dl, d["x"], d["w_r"])
    a = B.linear_bwd(dy, h["y"], bf16_to_f64(d["w2"]))
    b = B.linear_bwd(a["dx"], X, bf16_to_f64(d["w1"]), "gelu", h["z"])
    return {"idx": idx, "w": w, "y": y, "dw_gu": g["dw_gu"],
            "dw_dn": g["dw_dn"],
            "dx_experts": O.unpermute(g["dx_perm"], pm["row_map"], K),
            "dw": dw, "dl": dl, "dw_r": dw_r, "dx_router": dxr,
            "dw2": a["dw"], "db2": a["db"], "dw1": b["dw"], "db1": b["db"],
            "dx_shared": b["dx"]}


def test_block_forward_backward(m):
    d = make()
    g = to_gpu(d)
    s = forward(m, g)
    out = backward(m, g, s)
    assert m.check_device_status() == 0
    ref = oracle(d)
    np.testing.assert_array_equal(s["idx"].cpu().numpy(), ref["idx"])
    assert O.rel_err(s["w"].cpu().numpy(), ref["w"]) < 1e-6
    assert O.rel_err(host(s["y"]), ref["y"]) < 2e-2
    for n, v in out.items():
        got = host(v) if v.dtype == torch.bfloat16 else v.cpu().numpy()
        assert O.rel_err(got, ref[n]) < 2e-2, n


def test_block_graph_replay(m):
    """The step captured once: every replay equals the eager step with that
    replay's dropout counter, with eager work between the replays."""
    g = to_gpu(make())
    step = torch.zeros(1, dtype=torch.int64, device="cuda")

    def run():
        s = forward(m, g, step)
        out = backward(m, g, s, step)
        out["y"] = s["y"]
        return out
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
    for rep in range(4):
        step.fill_(rep)
        for v in got.values():
            v.view(torch.uint8).fill_(0xA5)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        kept = {n: v.clone() for n, v in got.items()}
        want = run()                    # eager, same step
        torch.cuda.synchronize()
        for n in want:
            assert torch.equal(kept[n].view(torch.uint8),
                               want[n].view(torch.uint8)), (rep, n)
        seen.append(kept["y"])
    assert not torch.equal(seen[0], seen[1])   # another mask every replay


def test_two_streams_at_once(m):
    """The same calls in flight on two streams give what each gives alone."""
    g = to_gpu(make())
    want = forward(m, g)
    want_b = backward(m, g, want)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    res = []
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for st in streams:
            with torch.cuda.stream(st):
                s = forward(m, g)
                res.append((s["y"], backward(m, g, s)))
    torch.cuda.synchronize()
    for y, b in res:
        assert torch.equal(y, want["y"])
        for n in b:
            assert torch.equal(b[n], want_b[n]), n


def test_split_products_on_two_streams(m):
    """Products whose K range is split hold their partials in the call's own
    workspace."""
    x = torch.randn(70, 14336, device="cuda").bfloat16()
    w = torch.randn(300, 14336, device="cuda").bfloat16()
    want = m.moe_linear_fwd(x, w)["y"]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    res = []
    for _ in range(4):
        for st in streams:
            with torch.cuda.stream(st):
                res.append(m.moe_linear_fwd(x, w)["y"])
    torch.cuda.synchronize()
    for y in res:
        assert torch.equal(y, want)
