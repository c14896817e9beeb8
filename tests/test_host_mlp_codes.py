"""CPU checks of what moe_grouped_mlp_fwd's binding hands to the library:
quantised weights that replace bf16 ones have the sizes that the kernels read.
Meta tensors stand for device tensors; the library is replaced by a
recorder."""
import ctypes

import pytest
import torch

import mixture_experts_grouped_router_amd as m

BF, F32, I32, U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
E, H, F, ROWS, NEED = 2, 128, 256, 8, 1000


def t(dtype, *shape):
    return torch.empty(shape, dtype=dtype, device="meta")


class Recorder:
    def __init__(self):
        self.args = None

    def moe_grouped_mlp_fwd_workspace_size(self, args, n):
        n._obj.value = NEED
        return 0

    def moe_grouped_mlp_fwd(self, ctx, args, stream):
        self.args = args._obj
        return 0


@pytest.fixture
def lib(monkeypatch):
    def need(t, dtype, shape, name):
        if t.dtype != dtype:
            raise TypeError(name)
        if tuple(t.shape) != tuple(shape) or not t.is_contiguous():
            raise ValueError(name)
    rec = Recorder()
    monkeypatch.setattr(m, "_need", need)
    monkeypatch.setattr(m, "load_library", lambda path=None: rec)
    monkeypatch.setattr(m, "_context", lambda dev: 1)
    monkeypatch.setattr(m, "_stream", lambda: 0)
    return rec


def codes(per_byte, gu=(E, 2 * F, H), dn=(E, H, F), sgu=None, sdn=None):
    q = lambda s, sc: (t(U8, s[0], s[1], s[2] // per_byte),
                       sc if sc is not None else t(U8, s[0], s[1],
                                                   s[2] // 32))
    return {"w_gu_q": q(gu, sgu), "w_dn_q": q(dn, sdn)}


WEIGHTS = {"gu": t(BF, E, 2 * F, H), "dn": t(BF, E, H, F)}
GIVEN = [(None, None), ("gu", None), (None, "dn")]


def call(prec, given, q, **kw):
    return m.moe_grouped_mlp_fwd(
        t(BF, ROWS, H), *[None if g is None else WEIGHTS[g] for g in given],
        t(I32, E + 1), precision=prec, **q, **kw)


@pytest.mark.parametrize("given", GIVEN)
@pytest.mark.parametrize("prec,per", [(m.PREC_MXFP8, 1), (m.PREC_MXFP4, 2)])
def test_codes_in_place_of_weights(lib, prec, per, given):
    call(prec, given, codes(per))
    assert lib.args is not None
    lib.args = None
    for bad in (codes(per, dn=(E, H, F // 2)), codes(per, dn=(1, H, F)),
                codes(per, sgu=t(U8, E, 2 * F, H // 64)),
                codes(per, sdn=t(U8, E, H, 1)),
                codes(per, sgu=t(F32, E, 2 * F, H // 32)),
                codes(per, dn=(E, H, 2 * F))):
        with pytest.raises((ValueError, TypeError)):
            call(prec, given, bad)
    assert lib.args is None
