"""CPU checks of the binding: sizes and choices that do not fit the C
interface's 32-bit integers are refused, not cut to their low 32 bits (which
would run a call of another size).  Meta tensors have a shape and no memory."""
import pytest
import torch

import mixture_experts_grouped_router_amd as m

WIDE = (1 << 32) + 8         # its low 32 bits are 8
BF, F32, I32 = torch.bfloat16, torch.float32, torch.int32


def t(dtype, *shape):
    return torch.empty(shape, dtype=dtype, device="meta")


CALLS = {
    "scored E": lambda: m.moe_route_scored(t(F32, 1, WIDE), 2),
    "scored k": lambda: m.moe_route_scored(t(F32, 1, 8), WIDE),
    "scored score": lambda: m.moe_route_scored(t(F32, 1, 8), 2,
                                               score=1 << 32),
    "scored n_group": lambda: m.moe_route_scored(
        t(F32, 1, 8), 2, n_group=(1 << 32) + 2, topk_group=2),
    "scored topk_group": lambda: m.moe_route_scored(
        t(F32, 1, 8), 2, n_group=2, topk_group=(1 << 32) + 2),
    "scored group_score": lambda: m.moe_route_scored(
        t(F32, 1, 8), 2, group_score=-(1 << 32)),
    "scored bwd E": lambda: m.moe_route_scored_bwd(
        t(F32, 1, WIDE), t(I32, 1, 2), t(F32, 1, 2)),
    "scored bwd k": lambda: m.moe_route_scored_bwd(
        t(F32, 1, 8), t(I32, 1, WIDE), t(F32, 1, WIDE)),
    "scored bwd score": lambda: m.moe_route_scored_bwd(
        t(F32, 1, 8), t(I32, 1, 2), t(F32, 1, 2), score=(1 << 32) + 1),
    "proj E": lambda: m.moe_router_proj_bwd(t(F32, 1, WIDE), t(BF, 1, 8),
                                            t(BF, WIDE, 8)),
    "proj H": lambda: m.moe_router_proj_bwd(t(F32, 1, 8), t(BF, 1, WIDE),
                                            t(BF, 8, WIDE)),
    "dropout H": lambda: m.moe_unpermute_dropout(t(BF, 1, WIDE), None, 1, 0.1,
                                                 1),
    "dropout k": lambda: m.moe_unpermute_dropout(t(BF, WIDE, 8),
                                                 t(I32, WIDE), WIDE, 0.1, 1),
    "dropout bwd H": lambda: m.moe_unpermute_dropout_bwd(
        t(BF, 1, WIDE), None, 1, 0.1, 1),
    "dropout bwd k": lambda: m.moe_unpermute_dropout_bwd(
        t(BF, 1, 8), t(I32, WIDE), WIDE, 0.1, 1),
    "linear N": lambda: m.moe_linear_fwd(t(BF, 1, 8), t(BF, WIDE, 8)),
    "linear K": lambda: m.moe_linear_fwd(t(BF, 1, WIDE), t(BF, 8, WIDE)),
    "linear act": lambda: m.moe_linear_fwd(t(BF, 1, 8), t(BF, 8, 8),
                                           act=1 << 32),
    "linear bwd N": lambda: m.moe_linear_bwd(t(BF, 1, WIDE), t(BF, 1, 8),
                                             t(BF, WIDE, 8)),
    "linear bwd K": lambda: m.moe_linear_bwd(t(BF, 1, 8), t(BF, 1, WIDE),
                                             t(BF, 8, WIDE)),
    "linear bwd act": lambda: m.moe_linear_bwd(t(BF, 1, 8), t(BF, 1, 8),
                                               t(BF, 8, 8), act=-(1 << 32)),
}


@pytest.mark.parametrize("name", CALLS)
def test_refused(name):
    with pytest.raises(ValueError, match="32 bits"):
        CALLS[name]()


def test_limits():
    m._need_i32(0, -1, (1 << 31) - 1, -(1 << 31))
    for v in (1 << 31, -(1 << 31) - 1):
        with pytest.raises(ValueError, match="32 bits"):
            m._need_i32(3, v)


def test_whole_floats_are_still_taken():
    o = m._route_opts(1.0, 8.0, 4.0, 1.0, True, 2.5)
    assert (o.score, o.n_group, o.topk_group, o.group_score) == (1, 8, 4, 1)
    with pytest.raises(ValueError, match="device tensor"):
        m.moe_linear_fwd(t(BF, 1, 8), t(BF, 8, 8), act=2.0)
    with pytest.raises(ValueError, match="device tensor"):
        m.moe_linear_bwd(t(BF, 1, 8), t(BF, 1, 8), t(BF, 8, 8), act=2.0)
