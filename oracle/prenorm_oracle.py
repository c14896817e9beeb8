"""CPU oracle of the operators of a pre-norm mixture-of-experts block -- TEST
INFRASTRUCTURE ONLY: layer norm forward and backward, MXFP4, the 4-bit expert
MLP and the whole layer for a few tokens.

Plain numpy in float64 from the definitions in include/moe.h; shares no code
with the GPU library.  Pinned by tests/test_prenorm_oracle.py (hand cases,
central differences, an independent decoding of every code).
"""
from __future__ import annotations

from typing import Dict, Optional, Tuple

import numpy as np

from .moe_oracle import _as_f64, route_topk

f64 = np.float64


# --------------------------------------------------------------------------
# layer norm
# --------------------------------------------------------------------------
def layernorm_fwd(x, weight=None, bias=None, eps: float = 1e-5
                  ) -> Dict[str, np.ndarray]:
    x = _as_f64(x)
    mean = x.mean(axis=1)
    d = x - mean[:, None]
    rstd = 1.0 / np.sqrt((d * d).mean(axis=1) + f64(np.float32(eps)))
    y = d * rstd[:, None]
    if weight is not None:
        y = y * _as_f64(weight)
    if bias is not None:
        y = y + _as_f64(bias)
    return {"y": y, "mean": mean, "rstd": rstd}


def layernorm_bwd(dy, x, mean, rstd, weight=None, dresidual=None
                  ) -> Dict[str, np.ndarray]:
    dy, x = _as_f64(dy), _as_f64(x)
    mean, rstd = _as_f64(mean)[:, None], _as_f64(rstd)[:, None]
    xh = (x - mean) * rstd
    g = dy if weight is None else dy * _as_f64(weight)
    H = x.shape[1]
    dx = rstd * (g - g.sum(axis=1, keepdims=True) / H -
                 xh * (g * xh).sum(axis=1, keepdims=True) / H)
    if dresidual is not None:
        dx = dx + _as_f64(dresidual)
    return {"dx": dx, "dw": (dy * xh).sum(axis=0), "db": dy.sum(axis=0)}


# --------------------------------------------------------------------------
# MXFP4
# --------------------------------------------------------------------------
E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def mxfp4_quantize(v) -> Tuple[np.ndarray, np.ndarray]:
    """(codes uint8 [.., n / 2], scale bytes uint8 [.., n / 32])."""
    v = _as_f64(v)
    b = v.reshape(v.shape[:-1] + (-1, 32))
    amax = np.abs(b).max(axis=-1)
    _, e = np.frexp(amax)                      # amax = m 2^e, m in [.5, 1)
    s = np.where(amax > 0, e - 1 - 2, -127)
    s = np.clip(s, -127, 127)
    a = np.abs(b) * np.ldexp(1.0, -s)[..., None]
    # nearest value; halfway, the even code
    hi = np.searchsorted(E2M1, np.minimum(a, 6.0), side="left")
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - E2M1[lo], E2M1[hi] - a
    code = np.where(dl < dh, lo, np.where(dl > dh, hi,
                                          np.where(lo % 2 == 0, lo, hi)))
    code = np.where(a >= 6.0, 7, code).astype(np.uint8)
    code |= (np.signbit(b).astype(np.uint8) << 3)
    code = code.reshape(v.shape)
    return (code[..., 0::2] | (code[..., 1::2] << 4),
            (s + 127).astype(np.uint8))


def mxfp4_dequantize(codes, scales) -> np.ndarray:
    codes = np.asarray(codes)
    n = np.empty(codes.shape[:-1] + (2 * codes.shape[-1],), np.uint8)
    n[..., 0::2] = codes & 15
    n[..., 1::2] = codes >> 4
    v = E2M1[n & 7] * np.where(n & 8, -1.0, 1.0)
    v = v.reshape(v.shape[:-1] + (-1, 32))
    v = np.ldexp(v, np.asarray(scales).astype(np.int32)[..., None] - 127)
    return v.reshape(n.shape)


def _round_trip(v) -> np.ndarray:
    return mxfp4_dequantize(*mxfp4_quantize(v))


def _swiglu(h, w):
    F = h.shape[1] // 2
    g, u = h[:, :F], h[:, F:]
    with np.errstate(over="ignore"):
        return w[:, None] * (g / (1.0 + np.exp(-g))) * u


def mlp_mxfp4(x_perm, gu_q, dn_q, w_perm, offsets, x_scale=None
              ) -> Dict[str, np.ndarray]:
    """z, (g, u) and the unquantised a of the 4-bit expert MLP.  x_perm: bf16
    bits, or codes with x_scale; gu_q, dn_q: (codes, scales)."""
    x = _round_trip(x_perm) if x_scale is None else \
        mxfp4_dequantize(x_perm, x_scale)
    off = np.asarray(offsets)
    E, F2 = gu_q[0].shape[:2]
    rows, H = x.shape
    z = np.zeros((rows, H))
    h1 = np.zeros((rows, F2))
    a = np.zeros((rows, F2 // 2))
    w = np.ones(rows) if w_perm is None else _as_f64(w_perm)
    for e in range(E):
        r = slice(off[e], off[e + 1])
        if off[e + 1] == off[e]:
            continue
        h1[r] = x[r] @ mxfp4_dequantize(gu_q[0][e], gu_q[1][e]).T
        a[r] = _swiglu(h1[r], w[r])
        z[r] = _round_trip(a[r]) @ mxfp4_dequantize(dn_q[0][e], dn_q[1][e]).T
    return {"z": z, "h1": h1, "a": a}


# --------------------------------------------------------------------------
# the whole layer for a few tokens
# --------------------------------------------------------------------------
def layer_few(x, w_gu, w_dn, topk_idx=None, topk_w=None, w_r=None, k=0,
              router_bias=None, renormalize=True, residual=None
              ) -> Dict[str, np.ndarray]:
    """w_gu, w_dn: float64 weights.  Also returns "bound", the sum of
    |W_dn| |error of a| and of the products' magnitudes that the GPU tests'
    tolerances are made of."""
    x = _as_f64(x)
    T, H = x.shape
    E, F2 = w_gu.shape[:2]
    F = F2 // 2
    if w_r is not None:
        l = x @ _as_f64(w_r).T
        if router_bias is not None:
            l = l + _as_f64(router_bias)
        topk_idx, topk_w = route_topk(l.astype(np.float32), k, renormalize)
    y = np.zeros((T, H))
    bound = np.zeros((T, H))
    u24 = 2.0 ** -24
    for t in range(T):
        for j in range(topk_idx.shape[1]):
            e = int(topk_idx[t, j])
            if not 0 <= e < E:
                continue
            w = f64(topk_w[t, j])
            h = w_gu[e] @ x[t]
            eh = (H + 16) * u24 * (np.abs(w_gu[e]) @ np.abs(x[t]))
            g, u = h[:F], h[F:]
            with np.errstate(over="ignore"):
                sg = g / (1.0 + np.exp(-g))
            a = sg * u
            # slope of silu below 1.1; exponential and reciprocal 2^-18; one
            # bf16 rounding
            ea = 1.1 * eh[:F] * np.abs(u) + np.abs(sg) * eh[F:] + \
                1.1 * eh[:F] * eh[F:] + 2.0 ** -18 * np.abs(a)
            ea = ea + 2.0 ** -8 * (np.abs(a) + ea)
            y[t] += w * (w_dn[e] @ a)
            bound[t] += np.abs(w) * (np.abs(w_dn[e]) @ (
                ea + (F + 32) * u24 * (np.abs(a) + ea)))
    if residual is not None:
        y = y + _as_f64(residual)
    return {"y": y, "topk_idx": topk_idx, "topk_w": topk_w, "bound": bound}
