"""Cases and plain forms of the operators that serve and train a pre-norm
mixture-of-experts block around its expert MLP.

* the whole layer for a few tokens (``moe_layer_few``): router logits, top-k,
  the chosen experts' gate/up, SwiGLU and down products and the combine with
  the residual, with bf16 or MXFP4 weights;
* MXFP4 (E2M1 elements, one E8M0 scale per 32 consecutive values):
  ``mxfp4_quantize`` / ``mxfp4_dequantize`` and the expert MLP on 4-bit
  operands (``moe_grouped_mlp_fwd`` with ``PREC_MXFP4``);
* layer norm, forward and backward (``moe_layernorm_fwd`` /
  ``moe_layernorm_bwd``), with the gradients of weight and bias and the
  residual stream's gradient added to that of the input.

``run`` computes the plain form with elementary torch operations where ``own``
is false, and calls the framework where it is true.
"""
import math

import torch

own = False

DEV = "cuda"


# --------------------------------------------------------------------------
# cases
def listed():
    return [
        # one generated token through the Qwen3-shaped layer, router and
        # residual included: a decode step, latency and weight reading
        dict(name="layer_one_token", op="few", T=1, H=2048, F=768, E=128, k=8,
             fmt="bf16", router=True, renorm=True, residual=True),
        # a decode batch over the same layer with 4-bit weights, routed
        # beforehand by the scored routing
        dict(name="layer_few_mxfp4", op="few", T=16, H=2048, F=768, E=128,
             k=8, fmt="mxfp4", router=False, renorm=True, residual=True),
        # five tokens (a drafted run being checked) through the
        # Mixtral-shaped layer: few experts, large weights
        dict(name="layer_few_large", op="few", T=5, H=4096, F=14336, E=8,
             k=2, fmt="bf16", router=True, renorm=True, residual=False),
        # a short prompt through the Qwen3-shaped experts in 4 bits: a
        # handful of rows per expert
        dict(name="mlp_mxfp4_prompt", op="mlp", T=77, H=2048, F=768, E=128,
             k=8, zipf=0.0),
        # a batch through the Mixtral-shaped experts in 4 bits
        dict(name="mlp_mxfp4_large", op="mlp", T=8192, H=4096, F=14336, E=8,
             k=2, zipf=0.0),
        # a batch through the Qwen3-shaped experts, skewed, some empty
        dict(name="mlp_mxfp4_skewed", op="mlp", T=16384, H=2048, F=768,
             E=128, k=8, zipf=1.2),
        # activations of a small ragged batch in 4 bits and back
        dict(name="mxfp4_rows", op="quant", E=1, rows=257, cols=4096),
        # the Qwen3-shaped down projections of all experts, quantised after
        # a weight update and read back
        dict(name="mxfp4_weights", op="quant", E=128, rows=2048, cols=768),
        # one token's norm ahead of the router: pure latency
        dict(name="norm_one_token", op="ln_fwd", T=1, H=2048, f32=False,
             bias=True, save=False),
        # the pre-norm of a training batch, statistics kept
        dict(name="norm_batch", op="ln_fwd", T=16384, H=2048, f32=False,
             bias=True, save=True),
        # its gradients over a long-sequence batch, the residual stream's
        # gradient joined in
        dict(name="norm_bwd_batch", op="ln_bwd", T=32768, H=2048, f32=False,
             dres=True),
        # gradients over a ragged batch with a float32 residual stream and
        # an odd width
        dict(name="norm_bwd_ragged", op="ln_bwd", T=1001, H=1035, f32=True,
             dres=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["few", "few", "mlp", "quant", "ln_fwd", "ln_bwd"])
    if op == "few":
        E = _log(rng, 1, 256)
        k = rng.randint(1, min(E, 8))
        T = _log(rng, 1, 64)
        fmt = rng.choice(["bf16", "mxfp4"])
        step = 8 if fmt == "bf16" else 32
        while True:
            H, F = step * _log(rng, 1, 4096 // step), \
                step * _log(rng, 1, 14336 // step)
            # the experts' weights, and the plain form's copies of them
            if E * F * H <= 8 * 4096 * 14336 and T * k * F * H <= 2 ** 32:
                break
        return dict(op=op, T=T, H=H, F=F, E=E, k=k, fmt=fmt,
                    router=rng.random() < 0.5, renorm=rng.random() < 0.7,
                    residual=rng.random() < 0.5)
    if op == "mlp":
        E = _log(rng, 1, 128)
        k = rng.randint(1, min(E, 8))
        while True:
            T = _log(rng, 1, 16384)
            H, F = 128 * _log(rng, 1, 32), 128 * _log(rng, 1, 112)
            if E * F * H <= 8 * 4096 * 14336 and \
                    T * k * F * H <= 16384 * 4096 * 14336:
                break
        return dict(op=op, T=T, H=H, F=F, E=E, k=k,
                    zipf=rng.choice([0.0, 0.6, 1.2]))
    if op == "quant":
        E = rng.choice([1, 1, 2, 8, 31])
        cols = 32 * _log(rng, 1, 448)
        rows = _log(rng, 1, max(2, min(65536, 2 ** 27 // (E * cols))))
        return dict(op=op, E=E, rows=rows, cols=cols)
    H = _log(rng, 1, 16384)
    if rng.random() < 0.6:
        H = max(8, H // 8 * 8)
    T = _log(rng, 1, max(2, min(32768, 32768 * 1024 // H)))
    case = dict(op=op, T=T, H=H, f32=rng.random() < 0.4)
    if op == "ln_fwd":
        case.update(bias=rng.random() < 0.7, save=rng.random() < 0.5)
    else:
        case.update(dres=rng.random() < 0.5)
    return case


# --------------------------------------------------------------------------
# inputs
def _gen(seed, salt):
    g = torch.Generator(device=DEV)
    g.manual_seed((int(seed) * 1000003 + salt) & 0x7FFFFFFFFFFFFFFF)
    return g


def _normal(shape, g, std=1.0):
    return torch.randn(shape, generator=g, device=DEV).mul_(std)


def _weights(shape, g, fmt):
    """Expert weights, N(0, 0.02): a bf16 tensor, or the (codes, scales) that
    a program with 4-bit weights keeps."""
    if fmt == "bf16":
        return _normal(shape, g, 0.02).bfloat16()
    codes = torch.empty(shape[:-1] + (shape[-1] // 2,), dtype=torch.uint8,
                        device=DEV)
    scales = torch.empty(shape[:-1] + (shape[-1] // 32,), dtype=torch.uint8,
                         device=DEV)
    for e in range(shape[0]):
        w = _normal(shape[1:], g, 0.02).bfloat16().float()
        mag, exp = _to_mxfp4(w)
        nib = mag | (torch.signbit(w).to(torch.uint8) << 3)
        codes[e] = nib[..., 0::2] | (nib[..., 1::2] << 4)
        scales[e] = (exp + 127).to(torch.uint8)
    return codes, scales


def _inputs(case, seed):
    op = case["op"]
    if op in ("few", "mlp"):
        g = _gen(seed, 41 if op == "few" else 43)
        T, H, F, E, k = (case[n] for n in ("T", "H", "F", "E", "k"))
        fmt = case.get("fmt", "mxfp4")
        s = {"x": _normal((T, H), g).bfloat16(),
             "w_gu": _weights((E, 2 * F, H), g, fmt),
             "w_dn": _weights((E, H, F), g, fmt)}
        if op == "few" and case["router"]:
            s["w_r"] = _normal((E, H), g, 0.02).bfloat16()
        else:
            # a router's choice: distinct experts per token, a skewed share
            rank = torch.arange(1, E + 1, device=DEV).float()
            z = _normal((T, E), g, 0.8) - case.get("zipf", 0.3) * torch.log(
                rank)
            idx = torch.sort(z, dim=1, descending=True,
                             stable=True).indices[:, :k]
            w = torch.softmax(torch.gather(z, 1, idx), dim=1)
            s["idx"] = idx.to(torch.int32).contiguous()
            s["w"] = w.contiguous()
        if op == "few":
            if case["residual"]:
                s["res"] = _normal((T, H), g).bfloat16()
            return s
        # rows in expert order, with the counts that the program made
        e = s["idx"].long().reshape(-1)
        order = torch.sort(e, stable=True).indices
        n = torch.bincount(e, minlength=E)
        s["x_perm"] = s["x"][order // k].contiguous()
        s["w_perm"] = s["w"].reshape(-1)[order].contiguous()
        off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
        off[1:] = torch.cumsum(n, 0)
        s["offsets"] = off
        s["sizes"] = n.tolist()
        return s
    if op == "quant":
        g = _gen(seed, 47)
        E, R, C = case["E"], case["rows"], case["cols"]
        spread = torch.exp(_normal((E, R, 1), g, 0.5))
        return {"src": (_normal((E, R, C), g, 0.02) * spread).bfloat16()}
    g = _gen(seed, 53)
    T, H = case["T"], case["H"]
    # a residual stream: channels of their own mean and spread, a few large
    mean = _normal((H,), g, 0.5)
    std = torch.exp(_normal((H,), g, 0.7))
    x = _normal((T, H), g) * std + mean
    s = {"x": x if case["f32"] else x.bfloat16(),
         "weight": 1.0 + _normal((H,), g, 0.1)}
    if op == "ln_fwd":
        if case["bias"]:
            s["bias"] = _normal((H,), g, 0.1)
        return s
    x64 = s["x"].double()
    mu = x64.mean(dim=1, keepdim=True)
    var = ((x64 - mu) ** 2).mean(dim=1)
    s["mean"] = mu[:, 0].float()
    s["rstd"] = (1.0 / torch.sqrt(var + EPS)).float()
    s["dy"] = _normal((T, H), g).bfloat16()
    if case["dres"]:
        r = _normal((T, H), g)
        s["dres"] = r if case["f32"] else r.bfloat16()
    return s


EPS = 1e-5


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    return s


# --------------------------------------------------------------------------
# plain forms
_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _pow2(exp, dtype=torch.float32):
    """2^exp (-128 to 128), exact where a power function may not be."""
    lut = torch.tensor([2.0 ** i for i in range(-128, 129)],
                       dtype=torch.float64, device=exp.device).to(dtype)
    return lut[exp.long() + 128]


def _to_mxfp4(v):
    """(E2M1 magnitude codes uint8 of v's shape, block exponents int32
    [.., n / 32]) of float32 values: the exponent is floor(log2 amax) - 2,
    magnitudes round to nearest even and saturate at 6."""
    b = v.reshape(v.shape[:-1] + (-1, 32)).abs()
    amax = b.amax(dim=-1, keepdim=True)
    exp = torch.frexp(amax).exponent - 3        # amax = m 2^e, m in [.5, 1)
    exp = torch.where(amax > 0, exp, torch.full_like(exp, -127))
    exp = exp.clamp(-127, 127)
    a = b * _pow2(-exp)
    mag = (a > 0.25).to(torch.uint8)
    for border, up in ((0.75, True), (1.25, False), (1.75, True),
                       (2.5, False), (3.5, True), (5.0, False)):
        mag += (a >= border) if up else (a > border)
    return mag.reshape(v.shape), exp[..., 0]


def _mxfp4_values(v):
    """Float32 values after a round trip through MXFP4."""
    mag, exp = _to_mxfp4(v)
    lut = torch.tensor(_E2M1, device=v.device)
    q = lut[mag.long()].reshape(v.shape[:-1] + (-1, 32))
    q = (q * _pow2(exp.unsqueeze(-1))).reshape(v.shape)
    return torch.where(torch.signbit(v), -q, q)


def _decode(cs):
    """Float32 values of (codes, scales)."""
    codes, scales = cs
    lut = torch.tensor(_E2M1 + tuple(-x for x in _E2M1), device=DEV)
    q = torch.stack([lut[(codes & 15).long()], lut[(codes >> 4).long()]],
                    dim=-1)
    q = q.reshape(scales.shape + (32,))
    q = q * _pow2(scales.to(torch.int32).unsqueeze(-1) - 127)
    return q.reshape(codes.shape[:-1] + (-1,))


def _take(w, e):
    """Float32 weights of expert(s) e."""
    if isinstance(w, tuple):
        return _decode((w[0][e], w[1][e]))
    return w[e].float()


def _silu(z):
    return z / (1.0 + torch.exp(-z))


def _plain_few(s):
    case = s["case"]
    T, H, F, k = case["T"], case["H"], case["F"], case["k"]
    x = s["x"].float()
    if case["router"]:
        # the logits in 64 bits, rounded once: they decide a selection
        logits = (s["x"].double() @ s["w_r"].double().t()).float().double()
        idx = torch.sort(logits, dim=1, descending=True,
                         stable=True).indices[:, :k]
        top = torch.gather(logits, 1, idx)
        ref = top if case["renorm"] else logits
        peak = logits.max(dim=1, keepdim=True).values
        w = torch.exp(top - peak) / torch.exp(ref - peak).sum(dim=1,
                                                              keepdim=True)
        w = w.float()
    else:
        idx, w = s["idx"].long(), s["w"]
    e = idx.reshape(-1)
    tok = torch.arange(T, device=DEV).repeat_interleave(k)
    z = torch.empty((T * k, H), device=DEV)
    step = max(1, 2 ** 30 // (2 * F * H))       # pairs whose weights fit
    for p in range(0, T * k, step):
        q = slice(p, p + step)
        h = torch.bmm(_take(s["w_gu"], e[q]), x[tok[q]].unsqueeze(2))[:, :, 0]
        a = _silu(h[:, :F]) * h[:, F:] * w.reshape(-1)[q].unsqueeze(1)
        z[q] = torch.bmm(_take(s["w_dn"], e[q]), a.unsqueeze(2))[:, :, 0]
    y = z.view(T, k, H).sum(dim=1)
    if case["residual"]:
        y = y + s["res"].float()
    out = [y.bfloat16()]
    if case["router"]:
        out += [idx.to(torch.int32), w]
    return out


def _plain_mlp(s):
    case = s["case"]
    H, F = case["H"], case["F"]
    x = _mxfp4_values(s["x_perm"].float())
    z = torch.empty((x.shape[0], H), dtype=torch.bfloat16, device=DEV)
    r = 0
    for e, n in enumerate(s["sizes"]):
        if n == 0:
            continue
        h = x[r:r + n] @ _take(s["w_gu"], e).t()
        a = _silu(h[:, :F]) * h[:, F:] * s["w_perm"][r:r + n].unsqueeze(1)
        z[r:r + n] = (_mxfp4_values(a) @ _take(s["w_dn"], e).t()).bfloat16()
        r += n
    return [z]


def _plain_quant(s):
    return [torch.stack([_mxfp4_values(w.float()).bfloat16()
                         for w in s["src"]])]


def _plain_ln_fwd(s):
    case = s["case"]
    x = s["x"].float()
    mu = x.mean(dim=1, keepdim=True)
    d = x - mu
    rstd = 1.0 / torch.sqrt((d * d).mean(dim=1, keepdim=True) + EPS)
    y = d * rstd * s["weight"]
    if case["bias"]:
        y = y + s["bias"]
    out = [y.bfloat16()]
    return out + [mu[:, 0], rstd[:, 0]] if case["save"] else out


def _plain_ln_bwd(s):
    case = s["case"]
    dy = s["dy"].float()
    xh = (s["x"].float() - s["mean"].unsqueeze(1)) * s["rstd"].unsqueeze(1)
    g = dy * s["weight"]
    c1 = g.mean(dim=1, keepdim=True)
    c2 = (g * xh).mean(dim=1, keepdim=True)
    dx = (g - c1 - xh * c2) * s["rstd"].unsqueeze(1)
    if case["dres"]:
        dx = dx + s["dres"].float()
    return [dx.to(s["x"].dtype), (dy * xh).sum(dim=0), dy.sum(dim=0)]


_PLAIN = {"few": _plain_few, "mlp": _plain_mlp, "quant": _plain_quant,
          "ln_fwd": _plain_ln_fwd, "ln_bwd": _plain_ln_bwd}


# --------------------------------------------------------------------------
# the framework's calls
def _own(s):
    import mixture_experts_grouped_router_amd as m
    case = s["case"]
    op = case["op"]
    if op == "few":
        kw = {}
        if case["fmt"] == "bf16":
            kw.update(w_gu=s["w_gu"], w_dn=s["w_dn"])
        else:
            kw.update(w_gu_q=s["w_gu"], w_dn_q=s["w_dn"],
                      precision=m.PREC_MXFP4)
        if case["router"]:
            kw.update(w_r=s["w_r"], k=case["k"], renormalize=case["renorm"])
        else:
            kw.update(topk_idx=s["idx"], topk_w=s["w"])
        r = m.moe_layer_few(s["x"], residual=s.get("res"), **kw)
        return [r["y"]] + ([r["topk_idx"], r["topk_w"]] if case["router"]
                           else [])
    if op == "mlp":
        return [m.moe_grouped_mlp_fwd(
            s["x_perm"], None, None, s["offsets"], w_perm=s["w_perm"],
            precision=m.PREC_MXFP4, w_gu_q=s["w_gu"], w_dn_q=s["w_dn"])["z"]]
    if op == "quant":
        return [m.mxfp4_dequantize(*m.mxfp4_quantize(s["src"]))]
    if op == "ln_fwd":
        r = m.moe_layernorm_fwd(s["x"], s["weight"], s.get("bias"), eps=EPS,
                                save=case["save"])
        return [r["y"]] + ([r["mean"], r["rstd"]] if case["save"] else [])
    r = m.moe_layernorm_bwd(s["dy"], s["x"], s["mean"], s["rstd"],
                            s["weight"], dresidual=s.get("dres"))
    return [r["dx"], r["dw"], r["db"]]


def run(state):
    if own:
        return _own(state)
    return _PLAIN[state["case"]["op"]](state)


# --------------------------------------------------------------------------
# what a pass cannot do without
def _w_bytes(n, fmt):
    return 2 * n if fmt == "bf16" else n // 2 + n // 32


def work(case):
    op = case["op"]
    if op == "few":
        T, H, F, E, k = (case[n] for n in ("T", "H", "F", "E", "k"))
        # experts that T tokens reach, on average
        hit = E * (1.0 - (1.0 - k / E) ** T)
        b = int(hit * _w_bytes(3 * F * H, case["fmt"])) + 4 * T * H
        b += 2 * E * H + 8 * T * k if case["router"] else 8 * T * k
        b += 2 * T * H if case["residual"] else 0
        f = 6 * T * k * F * H + (2 * T * E * H if case["router"] else 0)
        return {"bytes": b, "flops": f}
    if op == "mlp":
        T, H, F, E, k = (case[n] for n in ("T", "H", "F", "E", "k"))
        hit = E * (1.0 - (1.0 - k / E) ** T)
        b = int(hit * _w_bytes(3 * F * H, "mxfp4")) + T * k * (4 * H + 4)
        return {"bytes": b, "flops": 6 * T * k * F * H}
    if op == "quant":
        n = case["E"] * case["rows"] * case["cols"]
        return {"bytes": 4 * n + 2 * _w_bytes(n, "mxfp4"), "flops": 4 * n}
    T, H = case["T"], case["H"]
    x = 4 if case["f32"] else 2
    if op == "ln_fwd":
        b = T * H * (x + 2) + (8 if case["bias"] else 4) * H
        return {"bytes": b + (8 * T if case["save"] else 0),
                "flops": 8 * T * H}
    b = T * H * (2 * x + 2 + (x if case["dres"] else 0)) + 8 * T + 12 * H
    return {"bytes": b, "flops": 14 * T * H}


# --------------------------------------------------------------------------
# the definitions in 64 bits
def _exact_mxfp4(v):
    """Float64 values after a round trip through MXFP4: each magnitude to the
    nearest multiple of its quantum (ties to the even one), at most 6."""
    b = v.reshape(-1, 32)
    amax = b.abs().max(dim=1, keepdim=True).values
    lg = torch.floor(torch.log2(torch.where(amax > 0, amax,
                                            torch.ones_like(amax))))
    two = torch.float64
    # log2 next to a power of two
    lg = torch.where(_pow2(lg.clamp(-128, 127), two) > amax, lg - 1, lg)
    lg = torch.where(_pow2(lg.clamp(-128, 127) + 1, two) <= amax, lg + 1, lg)
    s = torch.where(amax > 0, lg - 2, torch.full_like(lg, -127))
    scale = _pow2(s.clamp(-127, 127), two)
    a = b / scale
    quantum = torch.where(a.abs() < 2, 0.5 * torch.ones_like(a),
                          torch.where(a.abs() < 4, torch.ones_like(a),
                                      2 * torch.ones_like(a)))
    q = (torch.round(a / quantum) * quantum).clamp(-6, 6)
    return (q * scale).reshape(v.shape)


def _exact_weights(w, e):
    """Float64 weights of expert e."""
    if not isinstance(w, tuple):
        return w[e].double()
    codes, scales = w[0][e], w[1][e]
    rows = codes.shape[0]
    nib = torch.empty((rows, 2 * codes.shape[1]), dtype=torch.int64,
                      device=codes.device)
    nib[:, 0::2] = (codes & 0xF).long()
    nib[:, 1::2] = (codes // 16).long()
    exp, man = (nib >> 1) & 3, nib & 1
    mag = torch.where(exp == 0, 0.5 * man.double(),
                      (1.0 + 0.5 * man.double()) *
                      _pow2(exp - 1, torch.float64))
    val = torch.where(nib >= 8, -mag, mag).reshape(rows, -1, 32)
    scale = _pow2(scales.int() - 127, torch.float64)
    return (val * scale.unsqueeze(2)).reshape(rows, -1)


def _exact_expert(x, gu, dn, w, quantised):
    """z [n, H] of one expert's rows, everything float64."""
    F = gu.shape[0] // 2
    h = torch.matmul(x, gu.t().contiguous())
    a = h[:, :F] * torch.sigmoid(h[:, :F]) * h[:, F:] * w.unsqueeze(1)
    if quantised:
        a = _exact_mxfp4(a)
    return torch.matmul(a, dn.t().contiguous())


def _exact_few(case, s):
    T, H, E, k = case["T"], case["H"], case["E"], case["k"]
    x = s["x"].double()
    if case["router"]:
        l = (x.unsqueeze(1) * s["w_r"].double()).sum(dim=2)
        l = l.float().double().cpu()
        idx = torch.tensor([sorted(range(E), key=lambda e: (-row[e], e))[:k]
                            for row in l.tolist()])
        sel = torch.gather(l, 1, idx)
        if case["renorm"]:
            w = torch.softmax(sel, dim=1)
        else:
            w = torch.gather(torch.softmax(l, dim=1), 1, idx)
        extra = [idx.to(torch.int32), w]
        idx, w = idx.to(x.device), w.to(x.device)
    else:
        idx, w, extra = s["idx"].long(), s["w"].double(), []
    y = torch.zeros((T, H), dtype=torch.float64, device=x.device)
    for e in sorted(set(idx.reshape(-1).tolist())):
        t, j = (idx == e).nonzero(as_tuple=True)
        y.index_add_(0, t, _exact_expert(
            x[t], _exact_weights(s["w_gu"], e), _exact_weights(s["w_dn"], e),
            w[t, j], False))
    if case["residual"]:
        y += s["res"].double()
    return [y.cpu()] + extra


def _exact_mlp(case, s):
    x = s["x_perm"].double()
    z, r = [], 0
    for e, n in enumerate(s["sizes"]):
        if n:
            z.append(_exact_expert(_exact_mxfp4(x[r:r + n]),
                                   _exact_weights(s["w_gu"], e),
                                   _exact_weights(s["w_dn"], e),
                                   s["w_perm"][r:r + n].double(), True).cpu())
        r += n
    return [torch.cat(z)]


def _exact_ln(case, s):
    x = s["x"].double()
    if case["op"] == "ln_fwd":
        var, mu = torch.var_mean(x, dim=1, unbiased=False)
        rstd = torch.rsqrt(var + EPS)
        y = (x - mu.unsqueeze(1)) * (rstd.unsqueeze(1) * s["weight"].double())
        if case["bias"]:
            y += s["bias"].double()
        return [y.cpu()] + ([mu.cpu(), rstd.cpu()] if case["save"] else [])
    H = x.shape[1]
    mu, rstd = s["mean"].double(), s["rstd"].double()
    dy, w = s["dy"].double(), s["weight"].double()
    xh = (x - mu.unsqueeze(1)) * rstd.unsqueeze(1)
    # H dxhat - sum(dxhat) - xhat sum(dxhat xhat), over H sigma
    dxh = dy * w
    dx = H * dxh - dxh.sum(dim=1, keepdim=True) - \
        xh * (dxh * xh).sum(dim=1, keepdim=True)
    dx = dx * (rstd / H).unsqueeze(1)
    if case["dres"]:
        dx += s["dres"].double()
    return [dx.cpu(), torch.einsum("th,th->h", dy, xh).cpu(),
            dy.sum(dim=0).cpu()]


def exact(case, seed):
    s = _inputs(case, seed)
    if case["op"] == "few":
        return _exact_few(case, s)
    if case["op"] == "mlp":
        return _exact_mlp(case, s)
    if case["op"] == "quant":
        return [torch.stack([_exact_mxfp4(w.double()).cpu()
                             for w in s["src"]])]
    return _exact_ln(case, s)
