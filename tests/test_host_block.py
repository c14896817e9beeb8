"""CPU checks of the scored routing, linear and dropout entry points: every
argument is validated on the host before the context and the device are
touched, so bad arguments are refused (and good ones get as far as the null
context) without a GPU."""
import ctypes

import pytest

import mixture_experts_grouped_router_amd as m

OK_PTR = 4096        # 16-byte aligned, never dereferenced on these paths
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    return m.load_library()


def reaches_context(lib, status):
    return status == INVALID and b"null context" in lib.moe_last_error()


def route(lib, T=4, E=8, k=2, bwd=False, logits=OK_PTR, idx=OK_PTR,
          w=OK_PTR, dl=OK_PTR, null_opts=False, **o):
    d = dict(score=0, n_group=1, topk_group=1, group_score=0, renormalize=1,
             scale=1.0)
    d.update(o)
    opts = m._RouteOpts(**d)
    ref = None if null_opts else ctypes.byref(opts)
    if bwd:
        return lib.moe_route_scored_bwd(None, logits, idx, w, T, E, k, ref,
                                        dl, None)
    return lib.moe_route_scored(None, logits, None, T, E, k, ref, idx, w,
                                None)


@pytest.mark.parametrize("bwd", [False, True])
def test_route_scored_refusals(lib, bwd):
    good = [dict(), dict(T=0, logits=None, idx=None, w=None, dl=None),
            dict(E=64, n_group=8, topk_group=4, group_score=1, k=8),
            dict(E=1024, k=32), dict(E=1, k=1), dict(score=1, scale=0.0)]
    for a in good:
        assert reaches_context(lib, route(lib, bwd=bwd, **a)), a
    bad = [dict(T=-1), dict(E=0, k=0), dict(k=0), dict(k=9), dict(score=2),
           dict(score=-1), dict(group_score=2), dict(n_group=0),
           dict(n_group=3), dict(n_group=2, topk_group=3),
           dict(topk_group=0), dict(n_group=4, topk_group=1, k=3),
           dict(n_group=8, topk_group=4, group_score=1),
           dict(scale=float("nan")), dict(scale=float("inf")),
           dict(null_opts=True), dict(logits=None), dict(idx=None),
           dict(w=None)]
    if bwd:
        bad.append(dict(dl=None))
    for a in bad:
        st = route(lib, bwd=bwd, **a)
        assert st == INVALID and not reaches_context(lib, st), a
    for a in [dict(E=1025, k=2), dict(E=64, k=33), dict(T=1 << 25),
              dict(E=130, n_group=65, topk_group=1)]:
        assert route(lib, bwd=bwd, **a) == UNSUPPORTED, a


def linear(lib, bwd=False, M=4, N=8, K=16, act=0, **p):
    cls = m._LinearBwdArgs if bwd else m._LinearFwdArgs
    a = cls()
    a.M, a.N, a.K, a.act = M, N, K, act
    names = ("dy", "x", "w", "z", "dx", "dw", "db") if bwd else \
        ("x", "w", "y")
    for n in names:
        setattr(a, n, OK_PTR)
    a.ws, a.ws_bytes = OK_PTR, 1 << 40
    for n, v in p.items():
        setattr(a, n, v)
    fn = lib.moe_linear_bwd if bwd else lib.moe_linear_fwd
    return fn(None, ctypes.byref(a), None)


@pytest.mark.parametrize("bwd", [False, True])
def test_linear_refusals(lib, bwd):
    good = [dict(), dict(M=0), dict(M=1, N=1, K=8), dict(N=1001),
            dict(M=100000, N=14336, K=4096), dict(act=4)]
    good += [dict(dx=None, w=None), dict(dw=None, x=None),
             dict(act=0, z=None), dict(dx=None, dw=None, db=None)] if bwd \
        else [dict(residual=OK_PTR, bias=OK_PTR + 4, z_save=OK_PTR)]
    for a in good:
        assert reaches_context(lib, linear(lib, bwd, **a)), a
    bad = [dict(M=-1), dict(N=0), dict(K=0), dict(act=5), dict(act=-1)]
    bad += [dict(dy=None), dict(x=None), dict(w=None),
            dict(act=2, z=None)] if bwd else \
        [dict(x=None), dict(w=None), dict(y=None)]
    for a in bad:
        st = linear(lib, bwd, **a)
        assert st == INVALID and not reaches_context(lib, st), a
    un = [dict(K=12), dict(K=1), dict(K=(1 << 22) + 8), dict(N=(1 << 22) + 1),
          dict(M=1 << 40), dict(M=1 << 30, N=4096), dict(x=OK_PTR + 2),
          dict(w=OK_PTR + 8)]
    un += [dict(dy=OK_PTR + 4), dict(z=OK_PTR + 2), dict(dx=OK_PTR + 2),
           dict(dw=OK_PTR + 2)] if bwd else \
        [dict(y=OK_PTR + 2), dict(residual=OK_PTR + 2),
         dict(z_save=OK_PTR + 2)]
    for a in un:
        assert linear(lib, bwd, **a) == UNSUPPORTED, a
    # a workspace that is missing, short or misaligned
    big = dict(M=768, N=768, K=16384) if not bwd else dict(M=16384, N=768,
                                                           K=768)
    big["act"] = 4
    assert linear(lib, bwd, ws=None, ws_bytes=0, **big) == WORKSPACE
    assert linear(lib, bwd, ws_bytes=16, **big) == WORKSPACE
    assert linear(lib, bwd, ws=OK_PTR + 8, **big) == UNSUPPORTED


def test_linear_null_args(lib):
    n = ctypes.c_size_t()
    for f in (lib.moe_linear_fwd_workspace_size,
              lib.moe_linear_bwd_workspace_size):
        assert f(None, ctypes.byref(n)) == INVALID
    assert lib.moe_linear_fwd(None, None, None) == INVALID
    assert lib.moe_linear_bwd(None, None, None) == INVALID


def drop(lib, bwd=False, T=4, H=16, k=2, p=0.1, row_map=OK_PTR, w=OK_PTR,
         z=OK_PTR, res=OK_PTR, out=OK_PTR, step=None, dw=OK_PTR):
    if bwd:
        return lib.moe_unpermute_dropout_bwd(None, out, row_map, w, z, T, H,
                                             k, p, 1, 2, step, OK_PTR, dw,
                                             None)
    return lib.moe_unpermute_dropout(None, z, row_map, w, res, T, H, k, p, 1,
                                     2, step, out, None)


@pytest.mark.parametrize("bwd", [False, True])
def test_dropout_refusals(lib, bwd):
    good = [dict(), dict(T=0, z=None, out=None, row_map=None),
            dict(k=1, row_map=None), dict(p=0.0), dict(p=1.0),
            dict(w=None, res=None), dict(H=8), dict(k=32),
            dict(step=OK_PTR + 8)]
    if bwd:
        good.append(dict(dw=None, z=None))
    for a in good:
        assert reaches_context(lib, drop(lib, bwd, **a)), a
    bad = [dict(T=-1), dict(H=0), dict(k=0), dict(p=-0.1), dict(p=1.5),
           dict(p=float("nan")), dict(row_map=None), dict(z=None),
           dict(out=None)]
    for a in bad:
        st = drop(lib, bwd, **a)
        assert st == INVALID and not reaches_context(lib, st), a
    for a in [dict(H=12), dict(k=33), dict(T=1 << 30),
              dict(T=1 << 24, H=4096, k=1), dict(z=OK_PTR + 2),
              dict(out=OK_PTR + 8), dict(step=OK_PTR + 4)]:
        assert drop(lib, bwd, **a) == UNSUPPORTED, a
    if not bwd:
        assert drop(lib, res=OK_PTR + 4) == UNSUPPORTED


def test_router_proj_bwd_refusals(lib):
    def go(dl=OK_PTR, x=OK_PTR, w=OK_PTR, T=4, H=64, E=8, dw=OK_PTR,
           dx=OK_PTR, ws=OK_PTR, nb=1 << 40):
        return lib.moe_router_proj_bwd(None, dl, x, w, T, H, E, dw, dx, ws,
                                       nb, None)
    for a in [dict(), dict(T=0, dl=None, x=None, w=None),
              dict(dw=None, x=None), dict(dx=None, w=None)]:
        assert reaches_context(lib, go(**a)), a
    for a in [dict(T=-1), dict(H=0), dict(E=0), dict(dl=None), dict(x=None),
              dict(w=None)]:
        st = go(**a)
        assert st == INVALID and not reaches_context(lib, st), a
    assert go(E=1025) == UNSUPPORTED
    assert go(T=64 * 65535 + 1) == UNSUPPORTED
    assert go(T=100000, H=4096, ws=None, nb=0) == WORKSPACE


def test_binding_refuses_host_tensors_and_bad_numbers():
    import torch
    bf = torch.zeros(4, 16, dtype=torch.bfloat16)
    f = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        m.moe_route_scored(f, 2)
    with pytest.raises(TypeError):
        m.moe_route_scored(f.double(), 2)
    with pytest.raises(ValueError):
        m.moe_linear_fwd(bf, bf)
    with pytest.raises(ValueError):
        m.moe_linear_bwd(bf, None, None)
    with pytest.raises(ValueError):
        m.moe_unpermute_dropout(bf, None, 3, 0.1, 1)
    with pytest.raises(ValueError):
        m._u64(-1, "seed")
    with pytest.raises(ValueError):
        m._u64(1 << 64, "seed")
