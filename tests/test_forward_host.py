"""Host checks of the per-token forward: the 64-bit statement the GPU tests
compare with, pinned by hand and by library routines, and refusals that need no
device."""
import ctypes
import math

import numpy as np
import torch

from weight_merge_b200 import binding as Bnd

from . import forward_ref as ref


def test_calls_without_a_context_are_refused():
    L = Bnd.lib()
    g = Bnd.Gating(0, 2, 1, 1, 1, 1, 1.0, None)
    a = Bnd.LinearArgs()
    n = ctypes.c_int64()
    bad = Bnd.ADAFUSE_ERR_INVALID_ARG
    assert L.adafuse_route_experts(None, None, 1, 1, 8, 8, None, ctypes.byref(g), 2, None, None) == bad
    assert L.adafuse_linear(None, ctypes.byref(a), None) == bad
    assert L.adafuse_linear_routed(None, ctypes.byref(a), None, 2, None, 0, None) == bad
    assert L.adafuse_linear_workspace(None, 0, 0, 1, 0, ctypes.byref(n)) == bad


def test_structs_have_the_c_layout():
    assert ctypes.sizeof(Bnd.Route8) == 64
    assert ctypes.sizeof(Bnd.Gating) == 40 and Bnd.Gating.bias.offset == 32
    assert ctypes.sizeof(Bnd.LinearArgs) == 104 and Bnd.LinearArgs.T.offset == 24
    fields = (1, 2, 3, 4, 5, 2 ** 40, 2 ** 62 + 1, 7, 8, 9, 10, 11, 12, 13, 14)
    assert Bnd._pack_linear_args(*fields) == bytes(Bnd.LinearArgs(*fields))


def test_a_gating_built_directly_keeps_no_tensor():
    assert Bnd.Gating(0, 2, 1, 1, 1, 1, 1.0, None)._keep is None
    assert Bnd.make_gating(k=3)._keep is None


def test_route_by_hand():
    # logits 2, 1, 0, 3 for one token
    h = torch.tensor([[1.0, 0.0]])
    Wr = torch.tensor([[2.0, 1.0, 0.0, 3.0], [0.0, 0.0, 0.0, 0.0]])
    idx, gate, z = ref.route(h, Wr, score="softmax", k=2)
    e = [math.exp(v) for v in (2, 1, 0, 3)]
    assert list(idx[0]) == [3, 0]
    np.testing.assert_allclose(gate[0], [e[3] / (e[3] + e[0]), e[0] / (e[3] + e[0])])
    idx, gate, _ = ref.route(h, Wr, score="softmax", k=2, renorm=False, scale=2.0)
    np.testing.assert_allclose(gate[0], [2 * e[3] / sum(e), 2 * e[0] / sum(e)])
    # groups {0, 1} and {2, 3}: by best expert the second, by the best two too
    # (sigmoid: .88 + .73 against .5 + .95); a bias on expert 1 turns it round
    assert list(ref.route(h, Wr, score="sigmoid", k=2, n_groups=2, group_top=1)[0][0]) == [3, 2]
    assert list(ref.route(h, Wr, score="sigmoid", k=2, n_groups=2, group_top=2)[0][0]) == [0, 1]
    b = torch.tensor([0.0, 1.0, 0.0, 0.0])
    idx, gate, _ = ref.route(h, Wr, score="sigmoid", k=1, renorm=False, bias=b)
    assert idx[0, 0] == 1                                # picked by its bias ...
    np.testing.assert_allclose(gate[0, 0], 1 / (1 + math.exp(-1)))   # ... gated by its score
    b = torch.tensor([-math.inf, 0.0, 0.0, -math.inf])
    assert list(ref.route(h, Wr, score="sigmoid", k=3, bias=b, slots=4)[0][0]) == [1, 2, -1, -1]
    assert list(ref.route(h * math.nan, Wr, score="sigmoid", k=2)[0][0]) == [-1, -1]


def test_product_by_hand_and_by_library():
    torch.manual_seed(0)
    x, W = torch.randn(5, 16).bfloat16(), torch.randn(8, 16).bfloat16()
    A, B = torch.randn(3, 2, 16).bfloat16(), torch.randn(3, 8, 2).bfloat16()
    idx = torch.tensor([[0, 2], [1, -1], [2, 2], [-1, -1], [7, 0]], dtype=torch.int32)
    gate = torch.tensor([[.75, .25], [1.0, 9.0], [.5, .25], [1.0, 1.0], [.5, .5]])
    routes = torch.cat([idx, gate.view(torch.int32)], dim=1)
    y, tol = ref.product(x, W, routes=routes, slots=2, A=A, B=B, s=2.0, activation="gelu")
    eff = [{0: .75, 2: .25}, {1: 1.0}, {2: .75}, {}, {0: .5}]
    for t, sel in enumerate(eff):
        Wt = W.double() + sum((2.0 * g * (B[e].double() @ A[e].double()) for e, g in sel.items()),
                              torch.zeros(8, 16, dtype=torch.float64))
        want = torch.nn.functional.gelu(x[t].double() @ Wt.t())
        torch.testing.assert_close(y[t], want, rtol=1e-12, atol=1e-12)
    for name, fn in (("silu", torch.nn.functional.silu), ("relu", torch.relu),
                     ("gelu_tanh", lambda v: torch.nn.functional.gelu(v, approximate="tanh"))):
        torch.testing.assert_close(ref.act(y, name), fn(y), rtol=1e-12, atol=1e-12)
    # the bound notices a planted mistake: one gate dropped, one bf16 step and a half
    off, _ = ref.product(x, W, routes=torch.where(routes == routes[0, 0], -1, routes), slots=2, A=A, B=B,
                         s=2.0, activation="gelu")
    assert ((off - y).abs() > tol).any()
    y, tol = ref.product(x, W, activation="gelu")
    big = y.abs() > 1
    assert big.any() and ((y * (1 + 1.5 * 2.0 ** -7) - y).abs() > tol)[big].all()
