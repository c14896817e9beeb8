"""CPU checks of the layer norm, MXFP4 and few-token entry points: every
argument is validated on the host before the context and the device are
touched, so bad arguments are refused (and good ones get as far as the null
context) without a GPU."""
import ctypes

import pytest
import torch

import mixture_experts_grouped_router_amd as m

OK_PTR = 4096        # 16-byte aligned, never dereferenced on these paths
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3
BIG = 1 << 40        # a workspace that is never too small


@pytest.fixture(scope="module")
def lib():
    return m.load_library()


def reaches_context(lib, status):
    return status == INVALID and b"null context" in lib.moe_last_error()


def check(lib, call, good, invalid, unsupported, workspace=()):
    for a in good:
        assert reaches_context(lib, call(**a)), (a, lib.moe_last_error())
    for a in invalid:
        st = call(**a)
        assert st == INVALID and not reaches_context(lib, st), a
    for a in unsupported:
        assert call(**a) == UNSUPPORTED, a
    for a in workspace:
        assert call(**a) == WORKSPACE, a


def test_layernorm_fwd(lib):
    def call(x=OK_PTR, f32=0, w=OK_PTR, b=OK_PTR, T=4, H=64, eps=1e-5,
             y=OK_PTR, mean=OK_PTR, rstd=OK_PTR):
        return lib.moe_layernorm_fwd(None, x, f32, w, b, T, H, eps, y, mean,
                                     rstd, None)
    check(lib, call,
          [dict(), dict(w=None, b=None, mean=None, rstd=None), dict(H=1),
           dict(T=0, x=None, y=None), dict(H=16384, f32=1), dict(eps=0.0),
           dict(mean=4100)],
          [dict(T=-1), dict(H=0), dict(x=None), dict(y=None),
           dict(eps=-1e-5), dict(eps=float("nan")), dict(eps=float("inf"))],
          [dict(H=16385), dict(T=1 << 57), dict(x=4104), dict(y=4100),
           dict(w=4100), dict(b=4108)])


def test_layernorm_bwd(lib):
    def call(dy=OK_PTR, x=OK_PTR, mean=OK_PTR, rstd=OK_PTR, w=OK_PTR,
             r=OK_PTR, T=5000, H=64, dx=OK_PTR, dw=OK_PTR, db=OK_PTR,
             ws=OK_PTR, n=BIG):
        return lib.moe_layernorm_bwd(None, dy, x, 0, mean, rstd, w, r, T, H,
                                     dx, dw, db, ws, n, None)
    check(lib, call,
          [dict(), dict(w=None, r=None), dict(dx=None), dict(dw=None),
           dict(dw=None, db=None, ws=None, n=0), dict(T=1, ws=None, n=0),
           dict(T=0, dy=None, x=None, mean=None, rstd=None, ws=None, n=0)],
          [dict(T=-1), dict(H=0), dict(dy=None), dict(x=None),
           dict(mean=None), dict(rstd=None)],
          [dict(H=16385), dict(dy=4100), dict(x=4100), dict(w=4100),
           dict(r=4100), dict(dx=4100), dict(dw=4100), dict(db=4100),
           dict(ws=4100)],
          [dict(ws=None), dict(n=0), dict(n=64)])
    b = ctypes.c_size_t(0)
    size = lambda T, H, want: (
        lib.moe_layernorm_bwd_workspace_size(T, H, want, ctypes.byref(b)),
        b.value)
    assert size(1, 64, 1) == (0, 0) and size(0, 64, 1) == (0, 0)
    assert size(5000, 64, 0) == (0, 0) and size(5000, 64, 1)[1] > 0
    # bounded however many rows
    assert size(1 << 40, 64, 1)[1] <= 256 * 4 * 2 * 64 * 4
    assert size(5, 16385, 1)[0] == UNSUPPORTED
    assert lib.moe_layernorm_bwd_workspace_size(1, 1, 1, None) == INVALID


def test_mxfp4(lib):
    def quant(src=OK_PTR, rows=3, cols=64, codes=OK_PTR, scales=OK_PTR):
        return lib.mxfp4_quantize(None, src, rows, cols, codes, scales, None)

    def back(src=OK_PTR, rows=3, cols=64, codes=OK_PTR, scales=OK_PTR):
        return lib.mxfp4_dequantize(None, codes, scales, rows, cols, src, None)
    for call in (quant, back):
        check(lib, call,
              [dict(), dict(rows=0, src=None), dict(cols=0, codes=None),
               dict(scales=4097)],
              [dict(rows=-1), dict(cols=-32), dict(src=None),
               dict(codes=None), dict(scales=None)],
              [dict(cols=48), dict(cols=1), dict(src=4104),
               dict(codes=4100), dict(rows=1 << 60)])


def mlp(lib, **o):
    d = dict(E=2, H=128, F=256, rows=8, precision=3, x_perm=OK_PTR,
             w_gu=OK_PTR, w_dn=OK_PTR, offsets=OK_PTR, z_perm=OK_PTR,
             ws=OK_PTR, ws_bytes=BIG)
    d.update(o)
    a = m._FwdArgs()
    for k, v in d.items():
        setattr(a, k, v)
    n = ctypes.c_size_t(0)
    return lib.moe_grouped_mlp_fwd_workspace_size(ctypes.byref(a),
                                                  ctypes.byref(n)), n.value


def test_mlp_mxfp4_sizes(lib):
    st, full = mlp(lib)
    assert st == 0 and full > 0
    codes = dict(w_gu=None, w_dn=None, w_gu_q=OK_PTR, w_gu_s=OK_PTR,
                 w_dn_q=OK_PTR, w_dn_s=OK_PTR)
    st, less = mlp(lib, **codes)
    assert st == 0 and full - less >= 2 * (256 * 128 + 128 * 128) // 2
    st, least = mlp(lib, x_perm_scale=OK_PTR, **codes)
    assert st == 0 and least < less
    for bad in [dict(H=64), dict(F=192), dict(E=1025)]:
        assert mlp(lib, **bad)[0] == UNSUPPORTED, bad
    assert mlp(lib, precision=4)[0] == INVALID
    b = m._BwdArgs()
    b.E, b.H, b.F, b.rows, b.precision = 2, 128, 256, 8, 3
    n = ctypes.c_size_t(0)
    assert lib.moe_grouped_mlp_bwd_workspace_size(
        ctypes.byref(b), ctypes.byref(n)) == UNSUPPORTED


def few(lib, **o):
    d = dict(T=4, H=64, F=96, E=8, k=2, precision=0, renormalize=1, x=OK_PTR,
             topk_idx=OK_PTR, topk_w=OK_PTR, w_gu=OK_PTR, w_dn=OK_PTR,
             y=OK_PTR, ws=OK_PTR, ws_bytes=BIG)
    d.update(o)
    a = m._LayerFewArgs()
    for k, v in d.items():
        setattr(a, k, v)
    return lib.moe_layer_few(None, ctypes.byref(a), None)


def test_layer_few(lib):
    q4 = dict(precision=3, w_gu=None, w_dn=None, w_gu_q=OK_PTR,
              w_gu_s=4097, w_dn_q=OK_PTR, w_dn_s=4099)
    check(lib, lambda **a: few(lib, **a),
          [dict(), q4, dict(T=0, x=None, y=None, topk_idx=None, topk_w=None,
                            ws=None, ws_bytes=0),
           dict(w_r=OK_PTR, router_bias=4100), dict(T=64, E=1024, k=32),
           dict(H=8, F=24), dict(residual=OK_PTR), dict(E=1, k=1)],
          [dict(T=-1), dict(H=0), dict(F=0), dict(E=0), dict(k=0),
           dict(k=9), dict(precision=9), dict(x=None), dict(y=None),
           dict(topk_idx=None), dict(topk_w=None), dict(w_gu=None),
           dict(w_dn=None), dict(router_bias=OK_PTR), dict(w_gu_q=OK_PTR)] +
          [dict(q4, **{n: None}) for n in ("w_gu_q", "w_gu_s", "w_dn_q",
                                           "w_dn_s")],
          [dict(T=65), dict(E=1025), dict(E=64, k=33), dict(precision=1),
           dict(precision=2), dict(H=12), dict(F=20), dict(q4, H=48),
           dict(q4, F=40), dict(H=1 << 20, F=1 << 12), dict(x=4104),
           dict(w_gu=4104), dict(w_dn=4100), dict(y=4098), dict(ws=4104),
           dict(residual=4100), dict(w_r=4104), dict(q4, w_gu_q=4100),
           dict(E=1024, H=8, F=1 << 18)],
          [dict(ws=None), dict(ws_bytes=16), dict(ws_bytes=0)])
    assert lib.moe_layer_few(None, None, None) == INVALID


WIDE = (1 << 32) + 8
BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8


def t(dtype, *shape):
    return torch.empty(shape, dtype=dtype, device="meta")


@pytest.mark.parametrize("call", [
    lambda: m.moe_layernorm_fwd(t(BF, 1, WIDE)),
    lambda: m.moe_layernorm_bwd(t(BF, 1, WIDE), t(BF, 1, WIDE), t(F32, 1),
                                t(F32, 1)),
    lambda: m.moe_layer_few(t(BF, 1, 8), t(BF, 2, 16, 8), t(BF, 2, 8, 8),
                            w_r=t(BF, 2, 8), k=WIDE),
    lambda: m.moe_layer_few(t(BF, 1, WIDE), t(BF, 2, 16, WIDE),
                            t(BF, 2, WIDE, 8), w_r=t(BF, 2, WIDE), k=1)])
def test_binding_refuses_wide_sizes(call):
    with pytest.raises(ValueError):
        call()


@pytest.mark.parametrize("call", [
    lambda: m.mxfp4_quantize(t(BF, 4, 40)),
    lambda: m.mxfp4_dequantize(t(U8, 4, 24), t(U8, 4, 1)),
    lambda: m.moe_layer_few(t(BF, 1, 8)),
    lambda: m.moe_layer_few(t(BF, 1, 8), t(BF, 2, 16, 8)),
    lambda: m.moe_layer_few(t(BF, 1, 8), t(BF, 2, 16, 8), t(BF, 2, 8, 8)),
    lambda: m.moe_layer_few(t(BF, 1, 32), precision=m.PREC_MXFP4,
                            w_gu_q=(t(U8, 2, 64, 16), t(U8, 2, 64, 1))),
    lambda: m.moe_grouped_mlp_fwd(t(BF, 4, 128), None, None, t(I32, 3)),
    lambda: m.moe_grouped_mlp_fwd(t(BF, 4, 128), None, None, t(I32, 3),
                                  precision=m.PREC_MXFP4),
    lambda: m.moe_layernorm_fwd(t(BF, 4, 4, 8)),
])
def test_binding_refuses_missing_or_misshapen(call):
    with pytest.raises((ValueError, TypeError)):
        call()


def test_binding_refuses_other_types():
    with pytest.raises(TypeError):
        m.moe_layernorm_fwd(t(torch.float16, 4, 8))
    with pytest.raises(TypeError):
        m.mxfp4_quantize(t(F32, 4, 32))
