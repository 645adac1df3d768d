"""GPU tests of the per-token forward at the ends of its ranges, against 64-bit
values: magnitudes whose squares underflow, rows of zeros, activations far below
zero, long sums, launches that give up."""
import numpy as np
import pytest
import torch

from weight_merge_b200 import binding as Bnd

from . import forward_ref as ref
from .test_gpu_forward import (ACT, BF, F32, SCORE, built, check, gen, make_routes, model, route_check,  # noqa: F401
                               rows, stream, workspace)

pytestmark = pytest.mark.gpu


# --------------------------------------------------------------------------
# routing to experts

def border_router(g, d, E):
    """Columns that differ in their last bits: 32-bit sums cannot order them."""
    base = torch.randn((d, 1), generator=g, device="cuda") * 0.05
    step = torch.randint(-1, 2, (d, E), generator=g, device="cuda").float() * 2.0 ** -23
    return (base * (1 + step)).contiguous()


def test_route_two_columns_whose_squares_underflow():
    _, sw = model(8, 8, E=2)
    h = torch.tensor([[1.0, 2.0 ** -30, 0.0, 0.0]], device="cuda")
    Wr = torch.zeros((4, 2), device="cuda")
    Wr[0], Wr[1, 1] = 2.0 ** -80, 2.0 ** -80     # column 1 is larger by 2^-30 of it
    for score in ("softmax", "sigmoid"):
        idx, _ = route_check(sw, h, Wr, 2, score=score, k=1)
        assert idx[0, 0] == 1


# powers of two on h and Wr: squares below fp32's range, below its normal range,
# the values themselves below it, and both sides of 2^-40
@pytest.mark.parametrize("hs,ws", [(-80, 0), (0, -80), (-68, 0), (0, -60), (-50, -50), (-36, -36), (-40, -45),
                                   (-120, 0), (0, -120), (-140, 0), (0, -140), (60, -80), (-100, 100)])
@pytest.mark.parametrize("E,dtype", [(8, F32), (16, BF), (24, F32), (64, F32)])
def test_route_decides_in_64_bits_at_any_magnitude(E, dtype, hs, ws):
    T, d = 60, 2048
    _, sw = model(8, 8, E=E)
    g = gen(9)
    h = (rows(g, T, d, F32) * 2.0 ** hs).to(dtype)
    Wr = border_router(g, d, E) * 2.0 ** ws
    k = min(E, 8)
    route_check(sw, h, Wr, 8, score="softmax", k=k)
    route_check(sw, h, Wr, 8, score="sigmoid", k=k)
    if hs + ws <= -60:   # scores that 64 bits cannot tell apart: groups and a bias see ties
        b = torch.randn((E,), generator=g, device="cuda").round()
        for score in ("softmax", "sigmoid"):
            route_check(sw, h, Wr, 8, score=score, k=k, bias=b)
            route_check(sw, h, Wr, 8, score=score, k=k, n_groups=4, top_groups=3, group_top=2)


def test_route_rows_and_columns_of_any_magnitude_together():
    """Tokens from 2^-140 to 2^60 in one batch, and one expert's column far below
    the others."""
    T, d, E = 90, 516, 12
    _, sw = model(8, 8, E=E)
    g = gen(3)
    h = rows(g, T, d, F32).contiguous()
    h *= 2.0 ** torch.randint(-140, 61, (T, 1), generator=g, device="cuda").float()
    Wr = border_router(g, d, E)
    route_check(sw, h, Wr, 8, score="softmax", k=8)
    Wr[:, 3] *= 2.0 ** -90
    Wr[:, 7] *= 2.0 ** -90
    route_check(sw, h, Wr, 8, score="softmax", k=8)
    Wr[:, :] *= 2.0 ** -70
    route_check(sw, h, Wr, 8, score="softmax", k=8)
