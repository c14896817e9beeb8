"""CPU oracle of the operators around the expert MLP -- TEST INFRASTRUCTURE
ONLY: scored routing, the dense linear layer, the combine with dropout, each
forward and backward.

Plain numpy in float64 from the definitions in include/moe.h; shares no code
with the GPU library.  Pinned by tests/test_block_oracle.py (hand cases,
published generator outputs, central differences).
"""
from __future__ import annotations

from typing import Dict, Optional, Tuple

import numpy as np
from scipy.special import ndtr

from .moe_oracle import _as_f64

f64 = np.float64


# --------------------------------------------------------------------------
# scored routing
# --------------------------------------------------------------------------
def scores(logits: np.ndarray, score: str) -> np.ndarray:
    l = np.asarray(logits, np.float32).astype(f64)
    if score == "softmax":
        e = np.exp(l - l.max(axis=1, keepdims=True))
        return e / e.sum(axis=1, keepdims=True)
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-l))


def route_scored(logits, k: int, bias=None, score: str = "softmax",
                 n_group: int = 1, topk_group: int = 1,
                 group_score: str = "max", renormalize: bool = True,
                 scale: float = 1.0) -> Tuple[np.ndarray, np.ndarray]:
    """(topk_idx int32 [T, k], topk_w float64 [T, k]); one token at a time."""
    lg = np.asarray(logits, np.float32).astype(f64) + 0.0
    s = scores(logits, score)
    T, E = lg.shape
    gsz = E // n_group
    idx = np.empty((T, k), np.int64)
    w = np.empty((T, k), f64)
    b = None if bias is None else np.asarray(bias, np.float32).astype(f64)
    for t in range(T):
        key = lg[t] if b is None else s[t] + b
        allowed = range(E)
        if n_group > 1:
            gs = []
            for g in range(n_group):
                run = slice(g * gsz, (g + 1) * gsz)
                if group_score == "max":
                    gs.append(key[run].max())
                else:
                    c = np.sort(s[t, run] if b is None else key[run])
                    gs.append(c[-1] + c[-2])
            kept = sorted(range(n_group), key=lambda g: (-gs[g], g))
            kept = set(kept[:topk_group])
            allowed = [e for e in range(E) if e // gsz in kept]
        order = sorted(allowed, key=lambda e: (-key[e], e))[:k]
        idx[t] = order
        if not renormalize:
            w[t] = s[t, order]
        elif score == "softmax":
            ex = np.exp(lg[t, order] - lg[t, order].max())
            w[t] = ex / ex.sum()
        else:
            tot = s[t, order].sum()
            w[t] = s[t, order] / tot if tot > 0 else 0.0
    return idx.astype(np.int32), w * scale


def route_scored_bwd(logits, topk_idx, dtopk_w, score: str = "softmax",
                     renormalize: bool = True, scale: float = 1.0
                     ) -> np.ndarray:
    """dlogits float64 [T, E]."""
    l = np.asarray(logits, np.float32).astype(f64)
    s = scores(logits, score)
    idx = np.asarray(topk_idx, np.int64)
    g = np.asarray(dtopk_w, f64) * scale
    T, E = l.shape
    dl = np.zeros((T, E), f64)
    for t in range(T):
        S = idx[t]
        if renormalize:
            if score == "softmax":
                ex = np.exp(l[t, S] - l[t, S].max())
                h = ex / ex.sum()
            else:
                tot = s[t, S].sum()
                h = s[t, S] / tot if tot > 0 else np.zeros(len(S))
            v = h * (g[t] - (h * g[t]).sum())
        else:
            v = s[t, S] * g[t]
        if score == "sigmoid":
            with np.errstate(over="ignore"):
                v = v / (1.0 + np.exp(l[t, S]))
        np.add.at(dl[t], S, v)
        if score == "softmax" and not renormalize:
            dl[t] -= s[t] * v.sum()
    return dl


# --------------------------------------------------------------------------
# dense linear layer
# --------------------------------------------------------------------------
def act(name: str, z: np.ndarray) -> np.ndarray:
    if name == "relu":
        return np.where(z > 0, z, 0.0)
    if name == "gelu":
        return z * ndtr(z)
    if name == "gelu_tanh":
        # 0.5 (1 + tanh u) = sigmoid(2 u), without the cancellation
        return z * scores_of(2 * np.sqrt(2 / np.pi) *
                             (z + 0.044715 * z ** 3))
    if name == "silu":
        return z * scores_of(z)
    return z


def scores_of(z):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-z))


def act_grad(name: str, z: np.ndarray) -> np.ndarray:
    if name == "relu":
        return (z > 0).astype(f64)
    if name == "gelu":
        return ndtr(z) + z * np.exp(-z * z / 2) / np.sqrt(2 * np.pi)
    if name == "gelu_tanh":
        c = np.sqrt(2 / np.pi)
        u2 = 2 * c * (z + 0.044715 * z ** 3)
        return scores_of(u2) + 2 * z * scores_of(u2) * scores_of(-u2) * c * \
            (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        s = scores_of(z)
        return s * (1 + z * (1 - s))
    return np.ones_like(z)


def linear_fwd(x, w, bias=None, act_name: str = "none", residual=None
               ) -> Dict[str, np.ndarray]:
    z = _as_f64(x) @ _as_f64(w).T
    if bias is not None:
        z = z + np.asarray(bias, f64)
    y = act(act_name, z)
    if residual is not None:
        y = y + _as_f64(residual)
    return {"y": y, "z": z}


def linear_bwd(dy, x, w, act_name: str = "none", z=None
               ) -> Dict[str, np.ndarray]:
    dz = _as_f64(dy)
    if act_name != "none":
        dz = dz * act_grad(act_name, _as_f64(z))
    return {"dz": dz, "dx": dz @ _as_f64(w), "dw": dz.T @ _as_f64(x),
            "db": dz.sum(axis=0)}


# --------------------------------------------------------------------------
# combine with dropout
# --------------------------------------------------------------------------
def philox4x32_10(c0, c1, c2, c3, k0: int, k1: int):
    """Ten rounds on arrays of 32-bit counter words (as uint64 arrays)."""
    u, low = np.uint64, np.uint64(0xFFFFFFFF)
    for _ in range(10):
        a, b = c0 * u(0xD2511F53), c2 * u(0xCD9E8D57)
        c0, c1, c2, c3 = ((b >> u(32)) ^ c1 ^ u(k0), b & low,
                          (a >> u(32)) ^ c3 ^ u(k1), a & low)
        k0 = (k0 + 0x9E3779B9) & 0xFFFFFFFF
        k1 = (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c0, c1, c2, c3


def dropout_factor(T: int, H: int, p: float, seed: int, offset: int
                   ) -> np.ndarray:
    """M float64 [T, H]: 0 where dropped, 65536 / (65536 - thr) elsewhere."""
    thr = int(np.floor(p * 65536.0 + 0.5))
    u = np.uint64
    i = np.arange(T * H // 8, dtype=np.uint64)
    offset &= (1 << 64) - 1
    words = philox4x32_10(i & u(0xFFFFFFFF), i >> u(32),
                          np.full_like(i, offset & 0xFFFFFFFF),
                          np.full_like(i, offset >> 32),
                          seed & 0xFFFFFFFF, seed >> 32)
    r = np.empty((i.size, 8), np.int64)
    for n, wd in enumerate(words):
        r[:, 2 * n] = (wd & u(0xFFFF)).astype(np.int64)
        r[:, 2 * n + 1] = (wd >> u(16)).astype(np.int64)
    keep = r.reshape(T, H) >= thr
    return np.where(keep, 65536.0 / (65536 - thr) if thr < 65536 else 0.0, 0.0)


def unpermute_dropout(z_perm, row_map, k: int, p: float, seed: int,
                      offset: int, topk_w=None, residual=None
                      ) -> Dict[str, np.ndarray]:
    """{"y", "mag"}: mag is sum_j |c_j z| M + |residual|, the size of the
    terms, for error bounds.  Dropped values are 0 whatever z holds."""
    z = _as_f64(z_perm)
    R, H = z.shape
    T = R // k
    rm = (np.arange(R) if row_map is None else
          np.asarray(row_map, np.int64)).reshape(T, k)
    M = dropout_factor(T, H, p, seed, offset)
    s = np.zeros((T, H), f64)
    mag = np.zeros((T, H), f64)
    for t in range(T):
        for j in range(k):
            if 0 <= rm[t, j] < R:
                c = 1.0 if topk_w is None else float(topk_w[t, j])
                s[t] += c * z[rm[t, j]]
                mag[t] += np.abs(c * z[rm[t, j]])
    y = np.where(M > 0, s * M, 0.0)
    mag = np.where(M > 0, mag * M, 0.0)
    if residual is not None:
        y = y + _as_f64(residual)
        mag = mag + np.abs(_as_f64(residual))
    return {"y": y, "mag": mag}


def unpermute_dropout_bwd(dy, row_map, k: int, p: float, seed: int,
                          offset: int, topk_w=None, z_perm=None
                          ) -> Dict[str, np.ndarray]:
    """dz [T*k, H] (NaN in rows no pair maps to), and with z_perm dtopk_w
    [T, k] and the size of its terms, dtopk_mag."""
    d = _as_f64(dy)
    T, H = d.shape
    R = T * k
    rm = (np.arange(R) if row_map is None else
          np.asarray(row_map, np.int64)).reshape(T, k)
    M = dropout_factor(T, H, p, seed, offset)
    g = np.where(M > 0, d * M, 0.0)
    dz = np.full((R, H), np.nan)
    out = {"dz": dz}
    if z_perm is not None:
        z = _as_f64(z_perm)
        out["dtopk_w"] = np.zeros((T, k), f64)
        out["dtopk_mag"] = np.zeros((T, k), f64)
    for t in range(T):
        for j in range(k):
            r = rm[t, j]
            if not 0 <= r < R:
                continue
            c = 1.0 if topk_w is None else float(topk_w[t, j])
            dz[r] = c * g[t]
            if z_perm is not None:
                pr = np.where(M[t] > 0, z[r], 0.0) * g[t]
                out["dtopk_w"][t, j] = pr.sum()
                out["dtopk_mag"][t, j] = np.abs(pr).sum()
    return out
