"""GPU tests of the per-token forward against 64-bit values: routing to
experts, the product with its epilogue, and the product with every token's own
experts, alone and run together."""
import numpy as np
import pytest
import torch

from weight_merge_b200 import binding as Bnd
from weight_merge_b200 import workloads as wl

from . import forward_ref as ref

pytestmark = pytest.mark.gpu

ACT = {"none": Bnd.ADAFUSE_ACT_NONE, "relu": Bnd.ADAFUSE_ACT_RELU, "gelu": Bnd.ADAFUSE_ACT_GELU,
       "gelu_tanh": Bnd.ADAFUSE_ACT_GELU_TANH, "silu": Bnd.ADAFUSE_ACT_SILU}
SCORE = {"softmax": Bnd.ADAFUSE_SCORE_SOFTMAX, "sigmoid": Bnd.ADAFUSE_SCORE_SIGMOID}
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    from weight_merge_b200 import build
    build.build()
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"


def stream():
    return torch.cuda.current_stream().cuda_stream


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rows(g, T, n, dtype=BF, pad=0, std=1.0):
    """[T, n] rows, pad elements apart; the gaps hold a pattern."""
    full = (torch.randn((T, n + pad), generator=g, device="cuda") * std).to(dtype)
    return full[:, :n]


def model(out, inn, E=4, r=8, seed=1, layers=1):
    cfg = wl.custom("f", layers, [("q", out, inn)], n_experts=E, rank=r, alpha=2.0 * r, n_tokens=1)
    m = wl.make_model(cfg, device="cuda", seed=seed)
    for b in m.B:       # adapters that weigh as much as the product itself
        b.mul_(16)
    sw = Bnd.Switcher(m.W, m.A, m.B, layers, 1, E, r, cfg.alpha, device=torch.cuda.current_device())
    return m, sw


def make_routes(g, T, E, k, slots, empty=0.0):
    z = torch.randn((T, E), generator=g, device="cuda") * 2
    top = torch.topk(z, k, dim=1)
    idx = torch.full((T, slots), -1, dtype=torch.int32, device="cuda")
    gate = torch.zeros((T, slots), device="cuda")
    idx[:, :k] = top.indices.int()
    gate[:, :k] = torch.softmax(top.values, dim=1)
    idx[torch.rand((T,), generator=g, device="cuda") < empty] = -1
    return torch.cat([idx, gate.view(torch.int32)], dim=1).contiguous()


def check(y, want, tol):
    d = (y.detach().double().cpu() - want).abs()
    bad = ~(d <= tol)
    if bad.any():
        i = np.unravel_index(int(torch.argmax(torch.where(bad, d / tol, 0.0).nan_to_num(1e30))), d.shape)
        raise AssertionError(f"{int(bad.sum())} of {d.numel()} off; worst at {i}: "
                             f"{y[i].item()} for {want[i].item()}, tol {tol[i].item()}")


def workspace(sw, T, f32):
    return torch.full((max(sw.linear_workspace(0, 0, T, f32), 1),), 0xff, dtype=torch.uint8, device="cuda")


# --------------------------------------------------------------------------
# routing to experts

ROUTE = [
    # T, d, E, score, k, groups, top, group_top, bias, renorm, dtype, pad
    (1, 4096, 8, "softmax", 2, 1, 1, 1, False, True, F32, 0),
    (1, 4, 1, "softmax", 2, 1, 1, 1, False, True, F32, 0),
    (1, 4096, 64, "sigmoid", 8, 8, 4, 2, True, True, BF, 0),
    (2, 260, 3, "sigmoid", 3, 3, 2, 2, True, False, BF, 0),
    (3, 12, 64, "softmax", 8, 64, 8, 2, False, True, BF, 4),
    (7, 1024, 16, "softmax", 4, 4, 2, 1, True, False, F32, 8),
    (33, 5120, 12, "sigmoid", 6, 4, 1, 2, False, True, F32, 0),
    (64, 4096, 8, "softmax", 4, 2, 1, 1, False, False, BF, 0),
    (257, 516, 40, "sigmoid", 7, 5, 3, 1, True, True, BF, 0),
    (300, 2052, 17, "softmax", 5, 1, 1, 1, True, True, F32, 4),
    (1025, 256, 64, "sigmoid", 8, 8, 3, 2, True, True, F32, 0),
    (515, 128, 32, "softmax", 1, 2, 2, 2, True, False, BF, 8),
]


def route_run(sw, h, Wr, slots, **kw):
    bias = kw.get("bias")
    g = Bnd.make_gating(score=SCORE[kw["score"]], k=kw["k"], n_groups=kw.get("n_groups", 1),
                        top_groups=kw.get("top_groups", 1), group_top=kw.get("group_top", 1),
                        renorm=kw.get("renorm", True), scale=kw.get("scale", 1.0), bias=bias)
    rt = torch.full((h.shape[0] + 1, 2 * slots), 0x5a5a5a5a, dtype=torch.int32, device="cuda")
    sw.route_experts(h, Wr, g, rt[:h.shape[0]], stream())
    torch.cuda.synchronize()
    assert (rt[-1] == 0x5a5a5a5a).all()     # the record behind the last token
    rt = rt[:-1]
    return rt[:, :slots].cpu().numpy(), rt[:, slots:].contiguous().view(F32).double().cpu().numpy()


def route_check(sw, h, Wr, slots, **kw):
    idx, gate = route_run(sw, h, Wr, slots, **kw)
    want_i, want_g, z = ref.route(h, Wr, slots=slots, **kw)
    assert np.array_equal(idx, want_i), np.argwhere(idx != want_i)[:4]
    # gates move by at most twice the logits' error each way, numerator and
    # denominator: a logit of d products summed in fp32 over chains of at most
    # d / 128 + 24 additions
    d = h.shape[1]
    mag = (h.double().abs().cpu().numpy() @ Wr.double().abs().cpu().numpy())
    mag = np.where(np.isfinite(mag), mag, 0.0).max(axis=1, keepdims=True)
    dz = (d / 128 + 24) * 2.0 ** -24 * mag
    tol = np.abs(want_g) * (np.expm1(np.minimum(4 * dz, 1.0)) + 2.0 ** -21) + 1e-37
    assert np.all(np.abs(gate - want_g) <= tol), np.max(np.abs(gate - want_g) / tol)
    return idx, gate


@pytest.mark.parametrize("T,d,E,score,k,G,top,gt,bias,renorm,dtype,pad", ROUTE)
def test_route_experts(T, d, E, score, k, G, top, gt, bias, renorm, dtype, pad):
    _, sw = model(8, 8, E=E)
    g = gen(T * 7 + E)
    h = rows(g, T, d, dtype, pad)
    Wr = torch.randn((d, E), generator=g, device="cuda") * 0.05
    b = torch.randn((E,), generator=g, device="cuda") * 0.1 if bias else None
    for slots in [s for s in (2, 4, 8) if s >= k]:
        route_check(sw, h, Wr, slots, score=score, k=k, n_groups=G, top_groups=top, group_top=gt,
                    renorm=renorm, scale=2.5, bias=b)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T", [1, 5, 300])
def test_route_equal_columns_go_to_the_lower_index(score, T):
    E, d = 16, 512
    _, sw = model(8, 8, E=E)
    g = gen(3)
    h = rows(g, T, d, F32)
    Wr = (torch.randn((d, 4), generator=g, device="cuda") * 0.05).repeat(1, 4).contiguous()
    idx, _ = route_check(sw, h, Wr, 8, score=score, k=8)
    assert np.all(idx[:, 0] < 4)
    route_check(sw, h, Wr, 8, score=score, k=6, n_groups=4, top_groups=2, group_top=2)
    route_check(sw, h, Wr, 4, score=score, k=4, bias=torch.zeros(E, device="cuda"))
    # one column all over: every logit equal, picks 0..k-1
    idx, gate = route_check(sw, h, Wr[:, :1].repeat(1, E).contiguous(), 8, score=score, k=8)
    assert np.array_equal(idx, np.tile(np.arange(8), (T, 1)))
    assert np.allclose(gate, 1 / 8, rtol=1e-6, atol=0)


@pytest.mark.parametrize("E", [8, 64])
def test_route_decides_in_64_bits_next_to_a_border(E):
    # columns that differ in their last bits: 32-bit sums cannot order them
    T, d = 200, 4096
    _, sw = model(8, 8, E=E)
    g = gen(9)
    h = rows(g, T, d, F32)
    base = torch.randn((d, 1), generator=g, device="cuda") * 0.05
    step = torch.randint(-1, 2, (d, E), generator=g, device="cuda").float() * 2.0 ** -23
    Wr = (base * (1 + step)).contiguous()
    for score in ("softmax", "sigmoid"):
        route_check(sw, h, Wr, 8, score=score, k=8)
        route_check(sw, h, Wr, 8, score=score, k=5, bias=torch.zeros(E, device="cuda"))
        route_check(sw, h, Wr, 8, score=score, k=8, n_groups=E // 2, top_groups=E // 2 - 1, group_top=2)


def test_route_bias_disables_and_forces_experts():
    E, d, T = 8, 256, 40
    _, sw = model(8, 8, E=E)
    g = gen(4)
    h = rows(g, T, d, BF)
    Wr = torch.randn((d, E), generator=g, device="cuda") * 0.05
    inf = float("inf")
    b = torch.tensor([0, -inf, 0.1, float("nan"), -inf, 0, inf, -3.4e38], device="cuda")
    for score in ("softmax", "sigmoid"):
        idx, _ = route_check(sw, h, Wr, 8, score=score, k=8, bias=b)
        assert np.all(idx[:, 0] == 6) and np.all(idx[:, 4] == 7) and np.all(idx[:, 5:] == -1)
        # a kept group whose experts are all disabled, and a token left with nothing
        b2 = torch.full((E,), -inf, device="cuda")
        idx, gate = route_check(sw, h, Wr, 4, score=score, k=3, bias=b2)
        assert np.all(idx == -1) and np.all(gate == 0)
        b2[5] = 0
        idx, gate = route_check(sw, h, Wr, 4, score=score, k=3, bias=b2, n_groups=4, top_groups=3, group_top=2)
        assert np.all(idx[:, 0] == 5) and np.all(idx[:, 1:] == -1) and np.allclose(gate[:, 0], 1)


def test_route_saturated_scores_and_non_finite_rows():
    E, d, T = 8, 64, 12
    _, sw = model(8, 8, E=E)
    g = gen(5)
    h = rows(g, T, d, F32)
    Wr = torch.randn((d, E), generator=g, device="cuda")
    for f in (30.0, 1000.0):        # sigmoid near 0 and 1, softmax underflow
        for renorm in (True, False):
            for score in ("softmax", "sigmoid"):
                idx, gate = route_check(sw, h * f, Wr, 4, score=score, k=4, renorm=renorm)
                if renorm:
                    assert np.allclose(gate.sum(axis=1), 1, rtol=1e-6)
    neg = -h[:, :1].abs().repeat(1, d).contiguous() * 50     # every logit far below zero
    route_check(sw, neg, Wr.abs().contiguous(), 4, score="sigmoid", k=3)
    h = h.clone()
    h[1, 3], h[4, 0], h[7, 63], h[9] = float("nan"), float("inf"), -float("inf"), 3e38
    idx, gate = route_check(sw, h, Wr, 4, score="sigmoid", k=3)
    for t in (1, 4, 7, 9):
        assert np.all(idx[t] == -1) and np.all(gate[t] == 0)
    assert np.all(idx[0] != [-1, -1, -1, 0])


def test_route_experts_top2_picks_what_pregate_picks():
    T, d, E = 300, 4096, 8
    _, sw = model(8, 8, E=E)
    g = gen(6)
    h = rows(g, T, d, F32)
    Wr = torch.randn((d, E), generator=g, device="cuda") * 0.05
    a = torch.zeros((T, 4), dtype=torch.int32, device="cuda")
    b = torch.zeros((T, 4), dtype=torch.int32, device="cuda")
    sw.pregate(h, Wr, a, stream())
    sw.route_experts(h, Wr, Bnd.make_gating(k=2), b, stream())
    torch.cuda.synchronize()
    assert torch.equal(a[:, :2], b[:, :2])
    torch.testing.assert_close(a[:, 2:].view(F32), b[:, 2:].view(F32), rtol=1e-5, atol=0)


@pytest.mark.parametrize("E", [8, 48, 64])
@pytest.mark.parametrize("T", [1, 70])
def test_route_zero_router(T, E):
    """A router before its first update: every logit 0, so the order is the
    index's, or the bias's."""
    d = 1032
    _, sw = model(8, 8, E=E)
    g = gen(2)
    h, Wr = rows(g, T, d, BF), torch.zeros((d, E), device="cuda")
    bias = torch.randn((E,), generator=g, device="cuda")
    for score in ("softmax", "sigmoid"):
        idx, _ = route_check(sw, h, Wr, 8, score=score, k=8)
        assert np.array_equal(idx, np.tile(np.arange(8), (T, 1)))
        route_check(sw, h, Wr, 8, score=score, k=8, bias=bias)
        route_check(sw, h, Wr, 4, score=score, k=4, n_groups=4, top_groups=2, group_top=2)
        route_check(sw, h, Wr, 4, score=score, k=4, n_groups=4, top_groups=3, group_top=2, bias=bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_groups_next_to_a_border(score):
    """Groups whose worth differs in the last bits of their columns only, and
    whose members are far apart."""
    T, d, E, G = 130, 2052, 32, 4
    _, sw = model(8, 8, E=E)
    g = gen(9)
    h = rows(g, T, d, F32)
    base = torch.randn((d, E // G), generator=g, device="cuda") * 0.05
    step = torch.randint(-1, 2, (d, E), generator=g, device="cuda").float() * 2.0 ** -23
    Wr = (base.repeat(1, G) * (1 + step)).contiguous()
    for top in (1, 2, 3):
        for gt in (1, 2):
            route_check(sw, h, Wr, 8, score=score, k=8, n_groups=G, top_groups=top, group_top=gt)
            route_check(sw, h, Wr, 4, score=score, k=3, n_groups=G, top_groups=top, group_top=gt,
                        bias=torch.zeros(E, device="cuda"))


@pytest.mark.parametrize("T", [1, 9, 100])
@pytest.mark.parametrize("d", [4, 60, 124, 132, 380, 1028])
@pytest.mark.parametrize("E", [5, 37, 63])
def test_route_any_alignment(T, d, E):
    """Wr on a 4-byte boundary with rows of any length, h with rows that no
    16-byte vector divides, and a short last part of d."""
    _, sw = model(8, 8, E=E)
    g = gen(T + d)
    Wr = (torch.randn((d * E + 1,), generator=g, device="cuda") * 0.05)[1:].view(d, E)
    assert Wr.data_ptr() % 8 == 4
    for dtype in (BF, F32):
        route_check(sw, rows(g, T, d, dtype, pad=4), Wr, 8, score="sigmoid", k=min(E, 8))


def test_route_refusals():
    _, sw = model(8, 8, E=8)
    h = torch.zeros((4, 64), device="cuda")
    Wr = torch.zeros((64, 8), device="cuda")
    rt = torch.full((4, 16), 7, dtype=torch.int32, device="cuda")
    L = Bnd.lib()
    import ctypes

    def call(h=h.data_ptr(), dt=1, T=4, d=64, ldh=64, Wr=Wr.data_ptr(), slots=8, route=rt.data_ptr(), **kw):
        g = Bnd.Gating(kw.get("score", 0), kw.get("k", 2), kw.get("n_groups", 1), kw.get("top_groups", 1),
                       kw.get("group_top", 1), 1, kw.get("scale", 1.0), kw.get("bias", None))
        return L.adafuse_route_experts(sw.ctx, h, dt, T, d, ldh, Wr, ctypes.byref(g), slots, route, stream())

    for bad in (dict(h=None), dict(h=h.data_ptr() + 4), dict(dt=2), dict(dt=-1), dict(T=-1), dict(d=62),
                dict(d=0), dict(d=2 ** 31, ldh=2 ** 31), dict(ldh=60), dict(ldh=66), dict(Wr=None), dict(Wr=Wr.data_ptr() + 2),
                dict(slots=3), dict(slots=16), dict(slots=0), dict(route=None), dict(route=rt.data_ptr() + 8),
                dict(score=2), dict(k=0), dict(k=9), dict(slots=2, k=3), dict(n_groups=3), dict(n_groups=0),
                dict(n_groups=16), dict(n_groups=2, top_groups=3), dict(top_groups=0), dict(group_top=0),
                dict(group_top=3), dict(scale=float("nan")), dict(scale=float("inf")), dict(bias=2)):
        assert call(**bad) == Bnd.ADAFUSE_ERR_INVALID_ARG, bad
    assert L.adafuse_route_experts(sw.ctx, h.data_ptr(), 1, 4, 64, 64, Wr.data_ptr(), None, 8,
                                   rt.data_ptr(), None) == Bnd.ADAFUSE_ERR_INVALID_ARG
    assert call(T=0, h=None) == Bnd.ADAFUSE_OK
    torch.cuda.synchronize()
    assert (rt == 7).all()
    with pytest.raises(TypeError):
        sw.route_experts(h.half(), Wr, Bnd.make_gating(), rt, stream())
    with pytest.raises(ValueError):
        sw.route_experts(h, Wr[:, :4], Bnd.make_gating(), rt, stream())
    with pytest.raises(ValueError):
        sw.route_experts(h, Wr, Bnd.make_gating(bias=torch.zeros(4, device="cuda")), rt, stream())
    with pytest.raises(ValueError):
        Bnd.make_gating(bias=torch.zeros((2, 4), device="cuda"))


# --------------------------------------------------------------------------
# the product with its epilogue

SHAPES = [(1, 8, 8), (1, 4096, 256), (2, 64, 136), (3, 72, 1024), (5, 1000, 264), (8, 4096, 128),
          (16, 512, 2056), (17, 136, 128), (31, 256, 384), (33, 4104, 72), (64, 1024, 512), (65, 320, 200),
          (127, 64, 128), (128, 128, 128), (129, 2048, 264), (200, 192, 1032), (256, 256, 256),
          (257, 88, 512), (300, 1096, 392), (511, 128, 776), (700, 520, 136), (1030, 264, 512)]


@pytest.mark.parametrize("T,inn,out", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_linear_shapes(T, inn, out, dtype):
    m, sw = model(out, inn, seed=T + inn)
    g = gen(T + out)
    x = rows(g, T, inn)
    y = torch.full((T + 1, out), 7.0, dtype=dtype, device="cuda")
    sw.linear(0, 0, x, y[:T], stream=stream())
    torch.cuda.synchronize()
    assert (y[T] == 7).all()
    check(y[:T], *ref.product(x, m.W[0], out_dtype=dtype))
    assert sw.status(stream()) == 0


@pytest.mark.parametrize("T", [2, 9, 40, 130, 300])
@pytest.mark.parametrize("inn,out,E,r", [(8, 8, 1, 1), (8, 40, 5, 8), (24, 8, 2, 16), (56, 16, 64, 2), (72, 8, 3, 64)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_weights_smaller_than_any_tile(T, inn, out, E, r, dtype):
    m, sw = model(out, inn, E=E, r=r, seed=T)
    g = gen(T + inn)
    x, rt = rows(g, T, inn, BF, pad=8), make_routes(g, T, E, min(E, 2), 2)
    full = torch.full((T + 1, out + 8), 3.0, dtype=dtype, device="cuda")
    y = full[:T, :out]
    sw.linear(0, 0, x, y, stream=stream())
    torch.cuda.synchronize()
    check(y, *ref.product(x, m.W[0], out_dtype=dtype))
    sw.linear_routed(0, 0, x, rt, y, workspace(sw, T, dtype == F32), stream=stream())
    torch.cuda.synchronize()
    check(y, *ref.product(x, m.W[0], routes=rt, slots=2, A=m.A[0], B=m.B[0], s=2.0, out_dtype=dtype))
    assert (full[:, out:] == 3).all() and (full[T] == 3).all()


@pytest.mark.parametrize("T", [1, 6, 40, 150, 600])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("act", list(ACT))
@pytest.mark.parametrize("bias,mul,residual", [(1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 1)])
def test_linear_epilogue_and_strides(T, dtype, act, bias, mul, residual):
    inn, out = 264, 328
    m, sw = model(out, inn, seed=T)
    g = gen(T * 5 + bias + 2 * mul)
    x = rows(g, T, inn, BF, pad=24)
    kw = dict(bias=torch.randn((out,), generator=g, device="cuda") if bias else None,
              mul=rows(g, T, out, dtype, pad=8) if mul else None,
              residual=rows(g, T, out, dtype, pad=16) if residual else None)
    full = torch.full((T, out + 8), 3.0, dtype=dtype, device="cuda")
    sw.linear(0, 0, x, full[:, :out], activation=ACT[act], stream=stream(), **kw)
    torch.cuda.synchronize()
    assert (full[:, out:] == 3).all()        # the gaps between rows stay
    check(full[:, :out], *ref.product(x, m.W[0], activation=act, out_dtype=dtype, **kw))


@pytest.mark.parametrize("T", [1, 40, 300])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_linear_in_place_over_its_residual_and_mul(T, dtype):
    m, sw = model(264, 512, seed=2)
    g = gen(T)
    x, y = rows(g, T, 512), rows(g, T, 264, dtype)
    before = y.clone()
    sw.linear(0, 0, x, y, residual=y, stream=stream())
    torch.cuda.synchronize()
    check(y, *ref.product(x, m.W[0], residual=before, out_dtype=dtype))
    before = y.clone()
    sw.linear(0, 0, x, y, mul=y, activation=ACT["silu"], stream=stream())
    torch.cuda.synchronize()
    check(y, *ref.product(x, m.W[0], mul=before, activation="silu", out_dtype=dtype))


@pytest.mark.parametrize("T", [4, 100, 400])
def test_non_finite_rows_stay_in_their_rows(T):
    m, sw = model(264, 512, E=3, r=8, seed=2)
    g = gen(T)
    x = rows(g, T, 512).contiguous()
    x[1] = float("nan")
    x[3, 5] = float("inf")
    rt = make_routes(g, T, 3, 2, 2)
    y = torch.empty((T, 264), dtype=BF, device="cuda")
    ok = torch.ones(T, dtype=torch.bool)
    ok[1] = ok[3] = False
    for routed in (False, True):
        if routed:
            sw.linear_routed(0, 0, x, rt, y, workspace(sw, T, False), stream=stream())
            want, tol = ref.product(x[ok], m.W[0], routes=rt[ok.cuda()], slots=2, A=m.A[0], B=m.B[0], s=2.0)
        else:
            sw.linear(0, 0, x, y, stream=stream())
            want, tol = ref.product(x[ok], m.W[0])
        torch.cuda.synchronize()
        check(y[ok], want, tol)
        assert torch.isnan(y[1]).all() and not torch.isfinite(y[3]).any()


def test_linear_long_rows_accumulate_in_fp32():
    # one long row: tensor-core accumulators lose low bits on every step, so
    # fp32 outputs are held to a bound no single chain of 700 steps meets
    T, inn, out = 150, 11008, 256
    m, sw = model(out, inn, seed=3)
    x = rows(gen(1), T, inn)
    y = torch.empty((T, out), dtype=F32, device="cuda")
    sw.linear(0, 0, x, y, stream=stream())
    torch.cuda.synchronize()
    want, _ = ref.product(x, m.W[0], out_dtype=F32)
    rel = ((y.double().cpu() - want).norm() / want.norm()).item()
    assert rel < 5e-6, rel


# --------------------------------------------------------------------------
# every token's own experts

ROUTED = [
    # T, in, out, E, r, k, slots, empty
    (1, 8, 8, 1, 1, 1, 2, 0.0), (1, 4096, 264, 8, 8, 2, 2, 0.0), (2, 64, 136, 4, 3, 3, 4, 0.0),
    (5, 512, 1032, 5, 12, 2, 2, 0.2), (8, 1096, 128, 64, 4, 8, 8, 0.0), (16, 256, 256, 16, 64, 2, 2, 0.0),
    (17, 264, 520, 3, 7, 2, 2, 0.5), (33, 256, 384, 8, 16, 2, 2, 0.1), (64, 520, 264, 2, 24, 2, 2, 0.0),
    (65, 128, 200, 7, 20, 4, 4, 0.1), (128, 512, 512, 8, 8, 2, 2, 0.0), (200, 264, 136, 12, 40, 6, 8, 0.3),
    (257, 192, 1032, 4, 32, 3, 4, 0.0), (300, 512, 256, 16, 64, 2, 2, 0.1), (513, 72, 264, 9, 5, 2, 2, 0.0),
    (600, 320, 520, 64, 64, 8, 8, 0.0), (1025, 256, 384, 8, 8, 2, 2, 1.0),
    (150, 2048, 1032, 8, 8, 2, 2, 0.0), (250, 2048, 1024, 8, 16, 2, 2, 0.1), (333, 2048, 4104, 4, 4, 3, 4, 0.1),
]


@pytest.mark.parametrize("T,inn,out,E,r,k,slots,empty", ROUTED)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_linear_routed(T, inn, out, E, r, k, slots, empty, dtype):
    m, sw = model(out, inn, E=E, r=r, seed=T + r)
    g = gen(T + out)
    x = rows(g, T, inn, BF, pad=8)
    rt = make_routes(g, T, E, k, slots, empty)
    y = torch.full((T + 1, out), 7.0, dtype=dtype, device="cuda")
    W0 = m.W[0].clone()
    sw.linear_routed(0, 0, x, rt, y[:T], workspace(sw, T, dtype == F32), stream=stream())
    torch.cuda.synchronize()
    assert (y[T] == 7).all() and torch.equal(m.W[0], W0)
    check(y[:T], *ref.product(x, m.W[0], routes=rt, slots=slots, A=m.A[0], B=m.B[0], s=2.0, out_dtype=dtype))
    assert sw.status(stream()) == 0


@pytest.mark.parametrize("T", [1, 20, 130, 400])
@pytest.mark.parametrize("act", ["gelu", "silu"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_linear_routed_epilogue(T, act, dtype):
    inn, out, E, r = 512, 328, 8, 16
    m, sw = model(out, inn, E=E, r=r, seed=T)
    g = gen(T)
    x = rows(g, T, inn)
    rt = make_routes(g, T, E, 2, 4, 0.1)
    kw = dict(bias=torch.randn((out,), generator=g, device="cuda"), mul=rows(g, T, out, dtype, pad=8),
              residual=rows(g, T, out, dtype))
    full = torch.full((T, out + 8), 3.0, dtype=dtype, device="cuda")
    sw.linear_routed(0, 0, x, rt, full[:, :out], workspace(sw, T, dtype == F32), activation=ACT[act],
                     stream=stream(), **kw)
    torch.cuda.synchronize()
    assert (full[:, out:] == 3).all()
    check(full[:, :out], *ref.product(x, m.W[0], activation=act, routes=rt, slots=4, A=m.A[0], B=m.B[0],
                                      s=2.0, out_dtype=dtype, **kw))


@pytest.mark.parametrize("T", [3, 70, 300])
def test_routed_repeated_and_bad_slots(T):
    inn, out, E, r = 256, 264, 4, 8
    m, sw = model(out, inn, E=E, r=r, seed=3)
    g = gen(8)
    x = rows(g, T, inn)
    rt = make_routes(g, T, E, 2, 4)
    rt[:, 2] = rt[:, 0]                                   # the same expert a second time
    rt[:, 6] = torch.full((T,), 0.25, device="cuda").view(torch.int32)
    y = torch.empty((T, out), dtype=BF, device="cuda")
    ws = workspace(sw, T, False)
    sw.linear_routed(0, 0, x, rt, y, ws, stream=stream())
    torch.cuda.synchronize()
    assert sw.status(stream()) == 0
    check(y, *ref.product(x, m.W[0], routes=rt, slots=4, A=m.A[0], B=m.B[0], s=2.0))
    for col, val, bit in ((0, E, Bnd.ADAFUSE_STATUS_BAD_EXPERT), (1, -2, Bnd.ADAFUSE_STATUS_BAD_EXPERT),
                          (4, 0x7fc00000, Bnd.ADAFUSE_STATUS_BAD_GATE), (5, 0x7f800000, Bnd.ADAFUSE_STATUS_BAD_GATE),
                          (0, 0x7fffffff, Bnd.ADAFUSE_STATUS_BAD_EXPERT)):
        b = rt.clone()
        b[T - 1, col] = val
        sw.linear_routed(0, 0, x, b, y, ws, stream=stream())
        torch.cuda.synchronize()
        assert sw.status(stream()) == bit
        check(y, *ref.product(x, m.W[0], routes=b, slots=4, A=m.A[0], B=m.B[0], s=2.0))
    e = rt.clone()                                       # a bad gate in an empty slot is not read
    e[0, 0], e[0, 4] = -1, 0x7fc00000
    sw.linear_routed(0, 0, x, e, y, ws, stream=stream())
    torch.cuda.synchronize()
    assert sw.status(stream()) == 0


@pytest.mark.parametrize("T", [2, 100, 300])
def test_base_weight_while_w_is_merged(T):
    inn, out, E, r = 256, 264, 4, 8
    m, sw = model(out, inn, E=E, r=r, seed=3)
    g = gen(8)
    x = rows(g, T, inn)
    y = torch.empty((T, out), dtype=F32, device="cuda")
    with pytest.raises(Bnd.AdafuseError):
        sw.linear(0, 0, x, y, base=True, stream=stream())
    W0 = m.W[0].clone()
    sw.set_base([W0])
    one = make_routes(g, 1, E, 2, 2)
    sw.switch(None, one.data_ptr(), stream())
    rt = make_routes(g, T, E, 2, 2)
    sw.linear(0, 0, x, y, stream=stream())
    torch.cuda.synchronize()
    assert not torch.equal(m.W[0], W0)
    check(y, *ref.product(x, m.W[0], out_dtype=F32))
    sw.linear_routed(0, 0, x, rt, y, workspace(sw, T, True), base=True, stream=stream())
    torch.cuda.synchronize()
    check(y, *ref.product(x, W0, routes=rt, slots=2, A=m.A[0], B=m.B[0], s=2.0, out_dtype=F32))


@pytest.mark.parametrize("T", [1, 24, 200, 520])
def test_router_products_and_merge_together(T):
    """As they are used: one decision per token, a gated block of three
    products with the tokens' own experts, captured into a graph and replayed
    on new inputs; and for one token the same as merging its experts."""
    d, ffn, E, r = 512, 1032, 8, 8
    cfg = wl.custom("b", 2, [("gate", ffn, d), ("up", ffn, d), ("down", d, ffn)], n_experts=E, rank=r,
                    alpha=16.0, n_tokens=1, d=d)
    m = wl.make_model(cfg, device="cuda", seed=5)
    sw = Bnd.Switcher(m.W, m.A, m.B, 2, 3, E, r, 16.0, device=torch.cuda.current_device())
    g = gen(T)
    h = torch.empty((T, d), dtype=BF, device="cuda")
    x = torch.empty((T, d), dtype=BF, device="cuda")
    res = torch.empty((T, d), dtype=F32, device="cuda")
    rt = torch.zeros((T, 8), dtype=torch.int32, device="cuda")
    up = torch.empty((T, ffn), dtype=BF, device="cuda")
    hid = torch.empty((T, ffn), dtype=BF, device="cuda")
    y = torch.empty((T, d), dtype=F32, device="cuda")
    need = max(sw.linear_workspace(1, k, T, f) for k, f in ((0, False), (1, False), (2, True)))
    ws = torch.empty((need,), dtype=torch.uint8, device="cuda")
    gating = Bnd.make_gating(score=SCORE["sigmoid"], k=3, n_groups=4, top_groups=2, group_top=2,
                             bias=torch.randn((E,), generator=g, device="cuda") * 0.1)

    def fill(seed):
        q = gen(seed)
        h.copy_(torch.randn((T, d), generator=q, device="cuda"))
        x.copy_(torch.randn((T, d), generator=q, device="cuda"))
        res.copy_(torch.randn((T, d), generator=q, device="cuda"))

    def block(s):
        sw.route_experts(h, m.Wr, gating, rt, s)
        sw.linear_routed(1, 1, x, rt, up, ws, stream=s)
        sw.linear_routed(1, 0, x, rt, hid, ws, activation=ACT["silu"], mul=up, stream=s)
        sw.linear_routed(1, 2, hid, rt, y, ws, residual=res, stream=s)

    def verify():
        idx, gate, _ = ref.route(h, m.Wr, score="sigmoid", k=3, n_groups=4, top_groups=2, group_top=2,
                                 bias=gating._keep, slots=4)
        assert np.array_equal(rt[:, :4].cpu().numpy(), idx)
        kw = dict(routes=rt, slots=4, s=2.0)
        w = lambda k: dict(A=m.A[3 + k], B=m.B[3 + k], **kw)
        check(up, *ref.product(x, m.W[4], **w(1)))
        check(hid, *ref.product(x, m.W[3], activation="silu", mul=up, **w(0)))
        check(y, *ref.product(hid, m.W[5], residual=res, out_dtype=F32, **w(2)))

    side = torch.cuda.Stream()
    fill(1)
    torch.cuda.synchronize()
    block(side.cuda_stream)
    side.synchronize()
    verify()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        block(torch.cuda.current_stream().cuda_stream)
    for seed in (2, 3):
        fill(seed)
        ws.fill_(0xff)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        verify()
    assert sw.status(stream()) == 0
    if T == 1:
        # merged form: W <- W + its experts, then the plain product
        y2 = torch.empty_like(up)
        sw.linear_routed(1, 1, x, rt, up, ws, stream=stream())
        sw.switch_topk(None, rt.data_ptr(), stream())
        sw.linear(1, 1, x, y2, stream=stream())
        torch.cuda.synchronize()
        # W' is rounded to bf16: 2^-8 of every |x w'| beside both outputs' own rounding
        tol = 2.0 ** -8 * (x.double().abs() @ m.W[4].double().abs().t()) + 2.0 ** -7 * up.double().abs()
        assert ((up.double() - y2.double()).abs() <= tol).all()


def test_calls_on_two_streams_at_once():
    T, inn, out, E, r = 300, 1024, 512, 8, 8
    m, sw = model(out, inn, E=E, r=r, seed=3)
    g = gen(8)
    jobs = []
    for i in range(2):
        x, rt = rows(g, T, inn), make_routes(g, T, E, 2, 2)
        jobs.append((torch.cuda.Stream(), x, rt, torch.empty((T, out), dtype=BF, device="cuda"),
                     workspace(sw, T, False)))
    torch.cuda.synchronize()
    for _ in range(10):
        for st, x, rt, y, ws in jobs:
            sw.linear_routed(0, 0, x, rt, y, ws, stream=st.cuda_stream)
    torch.cuda.synchronize()
    for st, x, rt, y, ws in jobs:
        check(y, *ref.product(x, m.W[0], routes=rt, slots=2, A=m.A[0], B=m.B[0], s=2.0))


@pytest.mark.parametrize("T", [1, 40, 300, 600])
def test_same_bits_every_time(T):
    inn, out, E, r = 2048, 520, 8, 16
    m, sw = model(out, inn, E=E, r=r, seed=3)
    g = gen(8)
    x, rt = rows(g, T, inn), make_routes(g, T, E, 2, 2)
    ws = workspace(sw, T, True)
    y = [torch.empty((T, out), dtype=F32, device="cuda") for _ in range(6)]
    for t in y[:3]:
        sw.linear_routed(0, 0, x, rt, t, ws, stream=stream())
    for t in y[3:]:
        sw.linear(0, 0, x, t, stream=stream())
    torch.cuda.synchronize()
    assert torch.equal(y[0], y[1]) and torch.equal(y[0], y[2])
    assert torch.equal(y[3], y[4]) and torch.equal(y[3], y[5])


def test_offsets_past_32_bits():
    T, inn, out = 300, 64, 72
    m, sw = model(out, inn, E=2, r=8, seed=3)
    ld = 8 * 1024 * 1024
    xs = torch.empty((T, ld), dtype=BF, device="cuda")      # 5 GB: row starts past 2^31 elements
    ys = torch.empty((T, ld), dtype=BF, device="cuda")
    x, y = xs[:, 8:8 + inn], ys[:, ld - out:]
    x.copy_(torch.randn((T, inn), generator=gen(1), device="cuda"))
    rt = make_routes(gen(2), T, 2, 1, 2)
    sw.linear(0, 0, x, y, stream=stream())
    torch.cuda.synchronize()
    check(y, *ref.product(x, m.W[0]))
    sw.linear_routed(0, 0, x, rt, y, workspace(sw, T, False), residual=x.new_zeros((T, out)), stream=stream())
    torch.cuda.synchronize()
    check(y, *ref.product(x, m.W[0], routes=rt, slots=2, A=m.A[0], B=m.B[0], s=2.0))


# More tokens than small tiles serve well: every width a tile of 256 tokens
# takes, ends of tiles in tokens and columns, contractions with a tail, of one
# accumulation and of several, and every layout of the adapters' ranks.
WIDE = [
    # T, in, out, E, r
    (2048, 128, 1296, 8, 8), (2047, 200, 1440, 5, 16), (1900, 72, 1584, 3, 32), (1793, 264, 1720, 4, 64),
    (2030, 136, 1872, 16, 24), (1801, 64, 2008, 8, 5), (1290, 128, 3360, 64, 8), (2041, 192, 2040, 7, 12),
    (1025, 1608, 4104, 4, 16), (2000, 3208, 2048, 2, 40),
]


@pytest.mark.parametrize("T,inn,out,E,r", WIDE)
@pytest.mark.parametrize("dtype", [BF, F32])
def test_many_tokens(T, inn, out, E, r, dtype):
    m, sw = model(out, inn, E=E, r=r, seed=T)
    g = gen(T + inn)
    x = rows(g, T, inn, BF, pad=16)
    k = min(E, 2)
    rt = make_routes(g, T, E, k, 2, 0.1)
    kw = dict(bias=torch.randn((out,), generator=g, device="cuda"), mul=rows(g, T, out, dtype, pad=8),
              residual=rows(g, T, out, dtype))
    full = torch.full((T + 1, out + 16), 3.0, dtype=dtype, device="cuda")
    y = full[:T, :out]
    sw.linear(0, 0, x, y, activation=ACT["gelu"], stream=stream(), **kw)
    torch.cuda.synchronize()
    assert (full[:, out:] == 3).all() and (full[T] == 3).all()
    check(y, *ref.product(x, m.W[0], activation="gelu", out_dtype=dtype, **kw))
    ws = workspace(sw, T, dtype == F32)
    guard = torch.full((ws.numel() + 256,), 0x5a, dtype=torch.uint8, device="cuda")
    sw.linear_routed(0, 0, x, rt, y, guard[:ws.numel()], stream=stream(), residual=kw["residual"])
    torch.cuda.synchronize()
    assert (full[:, out:] == 3).all() and (full[T] == 3).all() and (guard[ws.numel():] == 0x5a).all()
    check(y, *ref.product(x, m.W[0], routes=rt, slots=2, A=m.A[0], B=m.B[0], s=2.0, out_dtype=dtype,
                          residual=kw["residual"]))
    assert sw.status(stream()) == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_more_tokens_than_one_launch_takes(dtype):
    T, inn, out, E, r = 2 ** 17 + 21, 64, 72, 4, 8
    m, sw = model(out, inn, E=E, r=r, seed=2)
    g = gen(1)
    x, rt = rows(g, T, inn, BF, pad=8), make_routes(g, T, E, 2, 4, 0.1)
    kw = dict(mul=rows(g, T, out, dtype, pad=8), residual=rows(g, T, out, dtype))
    full = torch.full((T, out + 8), 3.0, dtype=dtype, device="cuda")
    y = full[:, :out]
    sw.linear(0, 0, x, y, stream=stream(), **kw)
    torch.cuda.synchronize()
    check(y, *ref.product(x, m.W[0], out_dtype=dtype, **kw))
    f32 = dtype == F32
    assert sw.linear_workspace(0, 0, T, f32) == sw.linear_workspace(0, 0, 2 ** 17, f32)
    sw.linear_routed(0, 0, x, rt, y, workspace(sw, T, f32), stream=stream(), **kw)
    torch.cuda.synchronize()
    assert (full[:, out:] == 3).all()
    check(y, *ref.product(x, m.W[0], routes=rt, slots=4, A=m.A[0], B=m.B[0], s=2.0, out_dtype=dtype, **kw))


@pytest.mark.parametrize("T", [3, 40, 300])
@pytest.mark.parametrize("r", [4, 8, 12])
def test_adapters_changed_in_place(T, r):
    inn, out, E = 256, 264, 4
    m, sw = model(out, inn, E=E, r=r, seed=3)
    g = gen(8)
    x, rt = rows(g, T, inn), make_routes(g, T, E, 2, 2)
    y, ws = torch.empty((T, out), dtype=BF, device="cuda"), workspace(sw, T, False)
    for f in (1.0, -2.0):
        m.A[0].mul_(f)
        m.B[0].mul_(0.5 * f)
        Bnd.adafuse_refresh_adapters(sw.ctx, stream())
        sw.linear_routed(0, 0, x, rt, y, ws, stream=stream())
        torch.cuda.synchronize()
        check(y, *ref.product(x, m.W[0], routes=rt, slots=2, A=m.A[0], B=m.B[0], s=2.0))


@pytest.mark.parametrize("T", [5, 40, 300])
def test_two_graphs_at_once(T):
    """Two captured calls with workspaces of their own, replayed on two streams
    together, on inputs that change between replays."""
    inn, out, E, r = 1024, 512, 8, 8
    m, sw = model(out, inn, E=E, r=r, seed=3)
    jobs = []
    for i in range(2):
        x = torch.empty((T, inn), dtype=BF, device="cuda")
        rt = make_routes(gen(i), T, E, 2, 2)
        y, ws, st = torch.empty((T, out), dtype=F32, device="cuda"), workspace(sw, T, True), torch.cuda.Stream()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            for _ in range(3):
                sw.linear_routed(0, 0, x, rt, y, ws, stream=torch.cuda.current_stream().cuda_stream)
        jobs.append((st, graph, x, rt, y))
    for seed in (5, 6):
        for i, (_, _, x, rt, _) in enumerate(jobs):
            x.copy_(torch.randn((T, inn), generator=gen(seed + 10 * i), device="cuda"))
            rt.copy_(make_routes(gen(seed + 20 * i), T, E, 2, 2))
        torch.cuda.synchronize()
        for _ in range(4):
            for st, graph, *_ in jobs:
                with torch.cuda.stream(st):
                    graph.replay()
        torch.cuda.synchronize()
        for _, _, x, rt, y in jobs:
            check(y, *ref.product(x, m.W[0], routes=rt, slots=2, A=m.A[0], B=m.B[0], s=2.0, out_dtype=F32))
    assert sw.status(stream()) == 0


@pytest.mark.parametrize("T", [2, 8, 30, 200])
def test_chain_of_calls_over_one_buffer(T):
    """Calls that follow each other without a gap, each reading what the one
    before wrote in place: residual and factor, then x, then the router's rows."""
    n, E, r = 264, 8, 4
    m, sw = model(n, n, E=E, r=r, seed=T)
    g = gen(T)
    Wr = torch.randn((n, E), generator=g, device="cuda") * 0.05
    x, rt = rows(g, T, n), make_routes(g, T, E, 2, 2)
    ws = workspace(sw, T, False)
    first = rows(g, T, n).contiguous()
    steps = 12
    hist = [[torch.empty_like(first) for _ in range(2)] for _ in range(steps)]
    recs = torch.zeros((steps, T, 4), dtype=torch.int32, device="cuda")
    a, b = first.clone(), first.clone()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=side):
        s = torch.cuda.current_stream().cuda_stream
        for i in range(steps):
            sw.linear(0, 0, x, a, residual=a, stream=s)                     # a <- a + x W
            hist[i][0].copy_(a)
            sw.linear_routed(0, 0, a, rt, b, ws, residual=b, stream=s)      # b <- b + a W'
            sw.route_experts(b, Wr, Bnd.make_gating(k=2), recs[i], s)
            hist[i][1].copy_(b)
            sw.linear(0, 0, b, a, activation=ACT["relu"], mul=a, stream=s)  # a <- a relu(b W)
            sw.linear_routed(0, 0, x, recs[i], a, ws, stream=s)             # a <- x W''
    for _ in range(2):
        a.copy_(first)
        b.copy_(first)
        graph.replay()
        torch.cuda.synchronize()
    pa, pb = first, first
    kw = dict(slots=2, A=m.A[0], B=m.B[0], s=2.0)
    for i in range(steps):
        check(hist[i][0], *ref.product(x, m.W[0], residual=pa))
        check(hist[i][1], *ref.product(hist[i][0], m.W[0], residual=pb, routes=rt, **kw))
        pb = hist[i][1]
        idx, _, _ = ref.route(pb, Wr, score="softmax", k=2)
        assert np.array_equal(recs[i, :, :2].cpu().numpy(), idx)
        pa = torch.empty_like(first)
        sw.linear_routed(0, 0, x, recs[i], pa, ws, stream=stream())
        torch.cuda.synchronize()
        check(pa, *ref.product(x, m.W[0], routes=recs[i], **kw))
    check(a, *ref.product(x, m.W[0], routes=recs[-1], **kw))


def test_linear_refusals():
    import ctypes
    inn, out, T = 64, 72, 4
    m, sw = model(out, inn, E=2, r=8, seed=3)
    L = Bnd.lib()
    x = torch.zeros((T, inn), dtype=BF, device="cuda")
    y = torch.full((T, out), 7.0, dtype=F32, device="cuda")
    rt = make_routes(gen(2), T, 2, 1, 2)
    ws = torch.zeros((4096,), dtype=torch.uint8, device="cuda")

    def args(**kw):
        a = Bnd.LinearArgs(0, 0, 0, 0, Bnd.ADAFUSE_DTYPE_F32, T, x.data_ptr(), inn, None, None, 0, None, 0,
                           y.data_ptr(), out)
        for k, v in kw.items():
            setattr(a, k, v)
        return a

    def both(a):
        p = ctypes.byref(a)
        return {L.adafuse_linear(sw.ctx, p, stream()),
                L.adafuse_linear_routed(sw.ctx, p, rt.data_ptr(), 2, ws.data_ptr(), 4096, stream())}

    bad = {Bnd.ADAFUSE_ERR_INVALID_ARG}
    for kw in (dict(layer=1), dict(layer=-1), dict(target=1), dict(target=-1), dict(weight=2), dict(weight=1),
               dict(activation=5), dict(activation=-1), dict(io_dtype=2), dict(T=-1), dict(x=None),
               dict(x=x.data_ptr() + 2), dict(ldx=60), dict(ldx=68), dict(ldx=-64), dict(y=None),
               dict(y=y.data_ptr() + 8), dict(ldy=64), dict(ldy=73), dict(bias=2), dict(mul=y.data_ptr()),
               dict(mul=y.data_ptr() + 4, ldmul=out), dict(residual=y.data_ptr(), ldres=70),
               dict(residual=y.data_ptr() + 4, ldres=out), dict(ldx=2 ** 62), dict(ldy=2 ** 61)):
        assert both(args(**kw)) == bad, kw
    assert both(args(T=2 ** 31)) == {Bnd.ADAFUSE_ERR_UNSUPPORTED_SHAPE}
    assert both(args(T=0, x=None, y=None)) == {Bnd.ADAFUSE_OK}
    p = ctypes.byref(args())
    n = sw.linear_workspace(0, 0, T, True)
    for rp, sl, w, nb in ((None, 2, ws.data_ptr(), 4096), (rt.data_ptr() + 8, 2, ws.data_ptr(), 4096),
                          (rt.data_ptr(), 3, ws.data_ptr(), 4096), (rt.data_ptr(), 2, None, 4096),
                          (rt.data_ptr(), 2, ws.data_ptr() + 16, 4080), (rt.data_ptr(), 2, ws.data_ptr(), n - 1)):
        assert L.adafuse_linear_routed(sw.ctx, p, rp, sl, w, nb, stream()) == Bnd.ADAFUSE_ERR_INVALID_ARG
    assert L.adafuse_linear(sw.ctx, None, stream()) == Bnd.ADAFUSE_ERR_INVALID_ARG
    b = ctypes.c_int64()
    for a in ((1, 0, T, 1), (0, -1, T, 1), (0, 0, -1, 1), (0, 0, T, 2)):
        assert L.adafuse_linear_workspace(sw.ctx, *a, ctypes.byref(b)) == Bnd.ADAFUSE_ERR_INVALID_ARG
    torch.cuda.synchronize()
    assert (y == 7).all()
    sizes = [sw.linear_workspace(0, 0, t, f) for f in (False, True) for t in (0, 1, 7, 64, 300, 5000)]
    assert all(v % 256 == 0 for v in sizes) and sizes[:6] == sorted(sizes[:6]) and sizes[6:] == sorted(sizes[6:])
    with pytest.raises(TypeError):
        sw.linear(0, 0, x.float(), y, stream=stream())
    with pytest.raises(ValueError):
        sw.linear(0, 0, x[:, :32], y, stream=stream())
    with pytest.raises(ValueError):
        sw.linear(0, 0, x, y, residual=y[:2], stream=stream())
    with pytest.raises(ValueError):
        sw.linear(0, 1, x, y, stream=stream())
