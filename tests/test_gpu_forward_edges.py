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


def test_route_with_a_gating_built_directly():
    T, d, E = 20, 64, 8
    _, sw = model(8, 8, E=E)
    g = gen(2)
    h, Wr = rows(g, T, d, F32), torch.randn((d, E), generator=g, device="cuda")
    b = torch.randn((E,), generator=g, device="cuda")
    for bias in (None, b):
        made = Bnd.make_gating(score=SCORE["sigmoid"], k=2, n_groups=2, bias=bias)
        direct = Bnd.Gating(SCORE["sigmoid"], 2, 2, 1, 1, 1, 1.0, None if bias is None else bias.data_ptr())
        got = [torch.zeros((T, 4), dtype=torch.int32, device="cuda") for _ in range(2)]
        sw.route_experts(h, Wr, made, got[0], stream())
        sw.route_experts(h, Wr, direct, got[1], stream())
        torch.cuda.synchronize()
        assert torch.equal(*got)


ZERO_ROWS = [
    # T, d, E, score, k, groups, top, group_top, bias
    (1, 64, 8, "softmax", 2, 1, 1, 1, None), (1, 64, 64, "sigmoid", 8, 8, 3, 2, "equal"),
    (40, 512, 8, "softmax", 2, 4, 2, 1, None), (70, 512, 16, "sigmoid", 4, 4, 2, 2, "random"),
    (70, 516, 16, "softmax", 3, 1, 1, 1, "equal"), (300, 1028, 64, "softmax", 8, 8, 3, 1, None),
    (300, 256, 64, "sigmoid", 8, 8, 4, 2, "few"), (2500, 64, 12, "softmax", 6, 3, 2, 2, "few"),
    (4600, 64, 24, "sigmoid", 4, 2, 1, 2, "few"),
]


@pytest.mark.parametrize("T,d,E,score,k,G,top,gt,bias", ZERO_ROWS)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_route_rows_of_zeros(T, d, E, score, k, G, top, gt, bias, dtype):
    """Padded rows of a batch: every logit 0 (of either sign), picks by bias, group
    and index."""
    _, sw = model(8, 8, E=E)
    g = gen(T + E)
    h = rows(g, T, d, dtype, pad=8)
    Wr = torch.randn((d, E), generator=g, device="cuda") * 0.05
    b = None
    if bias is not None:
        b = torch.randn((E,), generator=g, device="cuda")
        b = torch.full_like(b, 0.25) if bias == "equal" else b.round() if bias == "few" else b
    kw = dict(score=score, k=k, n_groups=G, top_groups=top, group_top=gt, bias=b)
    some = torch.rand((T,), generator=g, device="cuda") < 0.5
    h[some] = 0.0
    h[some, ::3] = -0.0
    route_check(sw, h, Wr, 8, **kw)
    route_check(sw, h, torch.zeros_like(Wr), 8, **kw)
    # 0 * inf and 0 * nan are no logits; a row of zeros but for one is none of zeros
    h[0] = 0.0
    h[T // 2, d - 1] = 2.0 ** -100
    route_check(sw, h, Wr, 8, **kw)
    Wr[d // 2, E // 2] = float("inf")
    with np.errstate(invalid="ignore"):
        idx, _ = route_check(sw, h, Wr, 8, **kw)
    assert np.all(idx[0] == -1)


def device_us(fn, n=25):
    """The median device time of a call, with the host ahead."""
    for _ in range(3):
        fn()
    took = []
    for _ in range(n):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        torch.cuda._sleep(100000)
        a.record()
        fn()
        b.record()
        torch.cuda.synchronize()
        took.append(a.elapsed_time(b) * 1e3)
    return sorted(took)[n // 2]


@pytest.mark.parametrize("T,d,E,k,G,bias", [(2048, 4096, 8, 2, 1, False), (777, 4096, 64, 8, 8, False),
                                            (1024, 4096, 16, 4, 4, True), (64, 4096, 8, 2, 1, False)])
def test_route_rows_of_zeros_cost_no_more(T, d, E, k, G, bias):
    """A padded batch takes as long as a full one: where each row of zeros was
    summed in fp64, these took four to eight times as long."""
    _, sw = model(8, 8, E=E)
    g = gen(1)
    h = rows(g, T, d, F32).contiguous()
    Wr = torch.randn((d, E), generator=g, device="cuda") * 0.05
    gating = Bnd.make_gating(k=k, n_groups=G, top_groups=max(G // 2, 1),
                             bias=torch.zeros((E,), device="cuda") if bias else None)
    slots = 2 if k <= 2 else 4 if k <= 4 else 8
    rt = torch.zeros((T, 2 * slots), dtype=torch.int32, device="cuda")

    def us(x, w):
        return device_us(lambda: sw.route_experts(x, w, gating, rt, stream()))

    full = us(h, Wr)
    last, every = h.clone(), h.clone()
    last[T // 2:] = 0
    every[::2] = 0
    for x, w in ((last, Wr), (every, Wr), (torch.zeros_like(h), Wr), (h, torch.zeros_like(Wr))):
        assert us(x, w) < 2 * full


# --------------------------------------------------------------------------
# the product with its epilogue

def act_exact(v, name):
    """The activation in 64 bits, in forms that do not cancel, and how far 32
    bits may be from it, relative to it, in units of u = 2^-24.

    gelu = v h below 0, v (1 - h) above, h = t p(t) e^w with w = -v^2 / 2: w is off
    by 3u |w| (square, constant, product), e^w by as much and 2 ulp (4u); t by 3u
    (sum, 2 ulp of its inverse), p by 1.5e-7 (2.5u) and 2u of its evaluation, three
    products: 1.5 v^2 + 15, and 1 for 1 - h.  gelu_tanh = v / (1 + e^w): w off by
    4u |w| (square, two constants or their sum, product), e^w by as much and 2 ulp
    (4u), the sum 1u, the division 2 ulp (4u).  silu the same with w = -v exact and a
    rounded division."""
    if name == "gelu":
        return 0.5 * v * torch.special.erfc(-v / np.sqrt(2.0)), 1.5 * v * v + 16
    if name == "gelu_tanh":
        w = -2 * np.sqrt(2 / np.pi) * (v + 0.044715 * v ** 3)
        return v / (1 + torch.exp(w)), 4 * w.abs() + 9
    if name == "silu":
        return v / (1 + torch.exp(-v)), torch.full_like(v, 4 + 2)
    return torch.where(v < 0, 0.0, v), torch.zeros_like(v)


@pytest.mark.parametrize("T,inn,out", [(1, 64, 1024), (8, 64, 1024), (40, 128, 1032), (300, 128, 520), (700, 64, 2056)])
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu", "relu"])
def test_activations_keep_their_digits_far_below_zero(T, inn, out, act):
    """Arguments that the product gives exactly (each row of x picks a column of
    W), from -8 to 8, the result times a large factor."""
    m, sw = model(out, inn, E=1, r=8)
    g = gen(T)
    m.W[0].copy_((torch.rand((out, inn), generator=g, device="cuda") * 16 - 8).to(BF))
    pick = torch.randint(0, inn, (T,), generator=g, device="cuda")
    x = torch.zeros((T, inn), dtype=BF, device="cuda")
    x[torch.arange(T, device="cuda"), pick] = 1.0
    mul = torch.randn((T, out), generator=g, device="cuda") * 1e6
    v = m.W[0].double().t()[pick]
    for factor in (None, mul):
        y = torch.empty((T, out), dtype=F32, device="cuda")
        sw.linear(0, 0, x, y, activation=ACT[act], mul=factor, stream=stream())
        torch.cuda.synchronize()
        want, units = act_exact(v, act)
        if factor is not None:
            want, units = want * factor.double(), units + 1
        check(y, want.cpu(), (units * 2.0 ** -24 * want.abs() + 1e-37).cpu())


@pytest.mark.parametrize("T", [1, 40, 300])
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu", "relu"])
def test_activations_of_huge_arguments(T, act):
    inf, nan, top = float("inf"), float("nan"), 3.4e38
    bias = torch.tensor([inf, nan, 1e30, -1e30, top, -top, 100.0, -300.0], device="cuda")
    m, sw = model(8, 64, E=1, r=8)
    x = torch.zeros((T, 64), dtype=BF, device="cuda")
    y = torch.empty((T, 8), dtype=F32, device="cuda")
    sw.linear(0, 0, x, y, bias=bias, activation=ACT[act], stream=stream())
    torch.cuda.synchronize()
    want = torch.tensor([inf, nan, bias[2], 0.0, bias[4], 0.0, 100.0, 0.0], device="cuda")
    assert torch.equal(y.nan_to_num(nan=-7.0, posinf=-8.0), want.nan_to_num(nan=-7.0, posinf=-8.0).expand(T, 8))


# --------------------------------------------------------------------------
# every token's own experts

@pytest.mark.parametrize("r", [4, 8, 12, 20, 63])
def test_workspace_of_few_tokens_holds_no_copy_of_b(r):
    """Up to 8 tokens read B as it lies: their workspace is x A^T in fp32 alone, and
    is enough."""
    E, inn, out = 4, 128, 4096
    m, sw = model(out, inn, E=E, r=r, seed=r)
    g = gen(r)
    rp = (r + 7) // 8 * 8
    for T in (0, 1, 8):
        assert sw.linear_workspace(0, 0, T, True) == (T * E * rp * 4 + 255) // 256 * 256
    for T in (1, 8, 9):
        n = sw.linear_workspace(0, 0, T, True)
        x, rt = rows(g, T, inn), make_routes(g, T, E, 2, 2)
        y = torch.zeros((T, out), device="cuda")
        ws = torch.full((n + 512,), 0x5a, dtype=torch.uint8, device="cuda")
        sw.linear_routed(0, 0, x, rt, y, ws[:n], stream=stream())
        torch.cuda.synchronize()
        check(y, *ref.product(x, m.W[0], routes=rt, slots=2, A=m.A[0], B=m.B[0], s=2.0, out_dtype=F32))
        assert (ws[n:] == 0x5a).all()


# --------------------------------------------------------------------------
# launches that give up

def held(y, want, tol):
    """y's elements that are as they were (7); the others must be right."""
    old = (y == 7.0).cpu()
    check(torch.where(old, want.to(y.dtype), y.cpu()), want, tol)
    return old


STALLED = [
    # T, in, out: clusters of CTAs that share a tile, single CTAs, CTA pairs
    (40, 4096, 256, BF), (100, 2048, 1032, F32), (90, 136, 20000, BF), (600, 1024, 8192, F32), (1500, 520, 4096, BF),
]


@pytest.mark.parametrize("T,inn,out,dtype", STALLED)
def test_a_product_that_gives_up_stores_only_finished_values(T, inn, out, dtype):
    """The hook keeps the first CTA (pair) waiting until its bound (1 s): its
    tile stays as it was, the other tiles hold the product, and the next call is
    right everywhere."""
    m, sw = model(out, inn, E=4, r=8, seed=T)
    x = rows(gen(T), T, inn)
    want, tol = ref.product(x, m.W[0], out_dtype=dtype)
    y = torch.full((T, out), 7.0, dtype=dtype, device="cuda")
    Bnd.adafuse_debug_stall_next_product(sw.ctx, 1)
    sw.linear(0, 0, x, y, stream=stream())
    assert sw.status(stream()) == Bnd.ADAFUSE_STATUS_TIMEOUT
    old = held(y, want, tol)
    assert old[0, 0] and not old[-1, -1]
    sw.linear(0, 0, x, y, stream=stream())
    assert sw.status(stream()) == 0
    check(y, want, tol)


@pytest.mark.parametrize("T,inn,out,dtype", STALLED)
@pytest.mark.parametrize("launch", [1, 2])
def test_a_routed_product_that_gives_up_stores_only_finished_values(T, inn, out, dtype, launch):
    """The same in either launch of a routed product: what the second one would
    make of an incomplete x A^T is not stored either."""
    E, r = 16, 32
    m, sw = model(out, inn, E=E, r=r, seed=T)
    g = gen(T)
    x, rt = rows(g, T, inn), make_routes(g, T, E, 2, 2)
    want, tol = ref.product(x, m.W[0], routes=rt, slots=2, A=m.A[0], B=m.B[0], s=2.0, out_dtype=dtype)
    y = torch.full((T, out), 7.0, dtype=dtype, device="cuda")
    ws = workspace(sw, T, dtype == F32)
    Bnd.adafuse_debug_stall_next_product(sw.ctx, launch)
    sw.linear_routed(0, 0, x, rt, y, ws, stream=stream())
    assert sw.status(stream()) == Bnd.ADAFUSE_STATUS_TIMEOUT
    old = held(y, want, tol)
    assert old.all() if launch == 1 else old[0, 0] and not old[-1, -1]
    sw.linear_routed(0, 0, x, rt, y, ws, stream=stream())
    assert sw.status(stream()) == 0
    check(y, want, tol)


def test_a_timeout_that_nobody_read_stops_the_next_routed_product():
    T, inn, out, E = 40, 512, 256, 4
    m, sw = model(out, inn, E=E, r=8)
    g = gen(1)
    x, rt = rows(g, T, inn), make_routes(g, T, E, 2, 2)
    y = torch.full((T, out), 7.0, dtype=BF, device="cuda")
    ws = workspace(sw, T, False)
    Bnd.adafuse_debug_stall_next_product(sw.ctx, 1)
    sw.linear(0, 0, x, torch.empty_like(y), stream=stream())
    sw.linear_routed(0, 0, x, rt, y, ws, stream=stream())
    assert sw.status(stream()) == Bnd.ADAFUSE_STATUS_TIMEOUT
    assert (y == 7.0).all()
    sw.linear_routed(0, 0, x, rt, y, ws, stream=stream())
    assert sw.status(stream()) == 0
    check(y, *ref.product(x, m.W[0], routes=rt, slots=2, A=m.A[0], B=m.B[0], s=2.0))


def test_the_product_hook_refuses_a_launch_number_below_one():
    _, sw = model(64, 64)
    with pytest.raises(Bnd.AdafuseError):
        Bnd.adafuse_debug_stall_next_product(sw.ctx, 0)


# --------------------------------------------------------------------------
# long sums

LONG = [
    # T, in, out: W streamed past the tensor cores; clusters and single CTAs whose
    # accumulators are emptied; CTA pairs, one and several tiles each
    (1, 11008, 512), (8, 14336, 1024), (61, 11008, 4096), (100, 11008, 11008), (128, 14336, 14336),
    (128, 8192, 19200), (700, 11008, 2048), (2048, 11008, 4096), (2050, 14336, 1032),
]


def one_sided(g, n, k):
    """Values of one sign: every partial sum grows, so each step's loss shows."""
    return (torch.rand((n, k), generator=g, device="cuda") + 0.5).to(BF)


@pytest.mark.parametrize("T,inn,out", LONG)
@pytest.mark.parametrize("signs", ["mixed", "one"])
@pytest.mark.parametrize("routed", [False, True])
def test_fp32_outputs_of_long_sums(T, inn, out, signs, routed):
    """The relative norm of the error of fp32 outputs over long contractions.

    A tensor-core accumulator cuts what a 16-deep piece adds below its last bit:
    on average half a unit of 2^-23 of itself, a piece; n pieces on one lose
    n / 2 units of a sum that grows evenly to its end, half of that of the end's
    value: n 2^-25.  With 48 pieces at most 48 / 2^25 = 1.4e-6 if every sum grows
    evenly (signs of one kind), and its square root's share of it if they wander;
    2^-24 sqrt(20) = 2.7e-7 for the fp32 additions that join up to 20 parts, and
    2^-24 for the rest: 1.8e-6.  One chain of 688 pieces would leave 2e-5 (one sign).
    Mixed signs: sums that wander are on average 2/3 of their end, 0.95e-6: 1.3e-6.
    V as two bf16 terms: each within 2^-18 of its value, independently: 2^-18 of
    the adapters' part."""
    E, r = 4, 8
    m, sw = model(out, inn, E=E, r=r, seed=T)
    g = gen(inn + T)
    x = rows(g, T, inn).contiguous()
    if signs == "one":
        x = one_sided(g, T, inn)
        m.W[0].copy_(one_sided(g, out, inn))
    y = torch.empty((T, out), dtype=F32, device="cuda")
    xd = x.double()
    want = xd @ m.W[0].double().t()
    tol = (1.8e-6 if signs == "one" else 1.3e-6) * want.norm()
    if routed:
        rt = make_routes(g, T, E, 2, 2)
        gates = ref.dense_gates(rt, 2, E).cuda()
        part = torch.zeros_like(want)
        for e in range(E):
            part += (2.0 * gates[:, e:e + 1] * (xd @ m.A[0][e].double().t())) @ m.B[0][e].double().t()
        want += part
        tol += (2.0 ** -18 + 1.8e-6) * part.norm()
        sw.linear_routed(0, 0, x, rt, y, workspace(sw, T, True), stream=stream())
    else:
        sw.linear(0, 0, x, y, stream=stream())
    torch.cuda.synchronize()
    off = (y.double() - want).norm()
    assert off <= tol, (off / want.norm()).item()


# --------------------------------------------------------------------------
# operands that the call before wrote

@pytest.mark.parametrize("T", [4, 40, 300])
def test_every_operand_may_come_from_the_call_before(T):
    """Bias, router, balance bias, weight and adapters made by a product right
    before the call that reads them, in one graph without a gap, over buffers
    that held something else before."""
    n, E, r = 256, 8, 16
    src, made = model(n, n, E=E, r=r, seed=5)                  # makes the operands
    g = gen(T)
    W, A, B = (torch.zeros(s, dtype=BF, device="cuda") for s in ((n, n), (E, r, n), (E, n, r)))
    sw = Bnd.Switcher([W], [A], [B], 1, 1, E, r, 2.0 * r, device=torch.cuda.current_device())
    shapes = {"bias": (1, n), "W": (n, n), "A": (E * r, n), "Bt": (E * n * r // n, n), "Wr": (n * E // n, n)}
    seeds = {k: rows(g, v[0], n).contiguous() for k, v in shapes.items()}
    x, h = rows(g, T, n), rows(g, T, n)
    bias, bal = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    Wr = torch.zeros((n, E), device="cuda")
    rt = make_routes(g, T, E, 2, 2)
    rec = torch.zeros((T, 4), dtype=torch.int32, device="cuda")
    ys = [torch.zeros((T, n), device="cuda") for _ in range(3)]
    ws = workspace(sw, T, True)
    gating = Bnd.make_gating(k=2, bias=bal[:E])
    torch.cuda.synchronize()

    def calls(s):
        made.linear(0, 0, seeds["bias"], bias.view(1, n), stream=s)
        sw.linear(0, 0, x, ys[0], bias=bias, stream=s)
        made.linear(0, 0, seeds["W"], W, stream=s)
        sw.linear(0, 0, x, ys[1], stream=s)
        made.linear(0, 0, seeds["A"], A.view(-1, n), stream=s)
        made.linear(0, 0, seeds["Bt"], B.view(-1, n), stream=s)
        sw.linear_routed(0, 0, x, rt, ys[2], ws, stream=s)
        made.linear(0, 0, seeds["Wr"], Wr.view(-1, n), stream=s)
        made.linear(0, 0, seeds["bias"], bal.view(1, n), stream=s)
        sw.route_experts(h, Wr, gating, rec, s)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        calls(torch.cuda.current_stream().cuda_stream)
    for _ in range(3):
        for k in seeds:
            seeds[k].copy_(torch.randn(seeds[k].shape, generator=g, device="cuda"))
        old_W = W.clone()
        graph.replay()
        torch.cuda.synchronize()
        check(bias.view(1, n), *ref.product(seeds["bias"], src.W[0], out_dtype=F32))
        check(W, *ref.product(seeds["W"], src.W[0]))
        check(ys[0], *ref.product(x, old_W, bias=bias, out_dtype=F32))
        check(ys[1], *ref.product(x, W, out_dtype=F32))
        check(ys[2], *ref.product(x, W, routes=rt, slots=2, A=A, B=B, s=2.0, out_dtype=F32))
        idx, _, _ = ref.route(h, Wr, score="softmax", k=2, bias=bal[:E])
        assert np.array_equal(rec[:, :2].cpu().numpy(), idx)
