"""CPU checks of what the expert MLP's binding hands to the library:
quantised weights that replace bf16 ones have the sizes that the kernels read,
and a workspace is the caller's only where it can serve as one.  Meta tensors
stand for device tensors; the library is replaced by a recorder."""
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

    moe_expert_loop_mlp_fwd_workspace_size = \
        moe_grouped_mlp_bwd_workspace_size = moe_grouped_mlp_fwd_workspace_size

    def moe_grouped_mlp_fwd(self, ctx, args, stream):
        self.args = args._obj
        return 0

    moe_expert_loop_mlp_fwd = moe_grouped_mlp_bwd = moe_grouped_mlp_fwd


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


X, OFF = t(BF, ROWS, H), t(I32, E + 1)
CALLS = {
    "mxfp4": lambda ws: call(m.PREC_MXFP4, (None, None), codes(2), ws=ws),
    "bf16": lambda ws: call(m.PREC_BF16, ("gu", "dn"), {}, ws=ws),
    "loop": lambda ws: m.moe_expert_loop_mlp_fwd(
        X, WEIGHTS["gu"], WEIGHTS["dn"], OFF, ws=ws),
    "backward": lambda ws: m.moe_grouped_mlp_bwd(
        X, X, WEIGHTS["gu"], WEIGHTS["dn"], OFF, t(BF, ROWS, 2 * F),
        t(BF, ROWS, F), ws=ws)}


@pytest.mark.parametrize("entry", CALLS)
@pytest.mark.parametrize("ws", [
    t(U8, NEED - 1), t(U8, 2 * NEED)[::2], t(F32, NEED),
    torch.empty(2 * NEED, dtype=U8)])
def test_unfit_workspaces_are_not_used(lib, monkeypatch, ws, entry):
    """Too small, strided, of another type, on another device: another one
    takes its place."""
    sent = []
    monkeypatch.setattr(m, "_ptr", lambda x: sent.append(x) or 0)
    CALLS[entry](ws)
    assert not any(x is ws for x in sent)
    assert lib.args.ws_bytes >= NEED


@pytest.mark.parametrize("entry", CALLS)
def test_a_fitting_workspace_is_used(lib, monkeypatch, entry):
    sent = []
    monkeypatch.setattr(m, "_ptr", lambda x: sent.append(x) or 0)
    ws = t(U8, NEED)
    CALLS[entry](ws)
    assert any(x is ws for x in sent) and lib.args.ws_bytes == NEED
