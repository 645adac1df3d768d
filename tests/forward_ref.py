"""The per-token forward in 64 bits, written plainly: routing to experts, the
product with its epilogue, and the product with every token's own experts.
Test infrastructure only; shares no code with the library."""
import math

import numpy as np
import torch


def route(h, Wr, *, score, k, n_groups=1, top_groups=1, group_top=1, renorm=True, scale=1.0,
          bias=None, slots=None):
    """h [T, d], Wr [d, E] (any float type) -> idx [T, slots] int32, gate
    [T, slots] fp64, logits [T, E] fp64.  score: "softmax" or "sigmoid"."""
    h = h.detach().double().cpu().numpy()
    Wr = Wr.detach().double().cpu().numpy()
    T, E = h.shape[0], Wr.shape[1]
    slots = slots or (2 if k <= 2 else 4 if k <= 4 else 8)
    # column by column, so that equal columns give equal logits
    with np.errstate(all="ignore"):
        z = np.stack([(h * Wr[:, e]).sum(axis=1) for e in range(E)], axis=1)
    b = None if bias is None else bias.detach().double().cpu().numpy()
    idx = np.full((T, slots), -1, np.int32)
    gate = np.zeros((T, slots))
    per = E // n_groups
    fmax = float(torch.finfo(torch.float32).max)
    for t in range(T):
        zt = z[t]
        if not np.all(np.abs(zt) <= fmax):
            continue
        if score == "softmax":
            s = [math.exp(v - max(zt)) for v in zt]
            tot = sum(s)
            s = [v / tot for v in s]
        else:
            s = [1 / (1 + math.exp(-v)) if v > -700 else 0.0 for v in zt]
        on = [b is None or b[e] > -math.inf for e in range(E)]
        q = [s[e] + (0.0 if b is None else b[e]) for e in range(E)]
        key = list(zt) if b is None else q
        if n_groups > 1:
            def worth(g):
                v = sorted((q[e] for e in range(g * per, (g + 1) * per) if on[e]), reverse=True)
                return sum(v[:group_top]) if v else -math.inf
            w = [worth(g) for g in range(n_groups)]
            kept = sorted(range(n_groups), key=lambda g: (-w[g], g))[:top_groups]
            on = [on[e] and e // per in kept for e in range(E)]
        picks = sorted((e for e in range(E) if on[e]), key=lambda e: (-key[e], e))[:k]
        if not picks:
            continue
        if renorm:
            zm = max(zt[e] for e in picks)
            if score == "softmax":
                x = [math.exp(zt[e] - zm) for e in picks]
            else:
                x = [math.exp(min(zt[e], 0) - min(zm, 0)) / (1 + math.exp(-abs(zt[e]))) for e in picks]
            g = [v / sum(x) for v in x]
        else:
            g = [s[e] for e in picks]
        idx[t, :len(picks)] = picks
        gate[t, :len(picks)] = [scale * v for v in g]
    return idx, gate, z


def act(v, name):
    if name == "relu":
        return torch.where(v < 0, torch.zeros_like(v), v)
    if name == "gelu":
        return 0.5 * v * (1 + torch.erf(v / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    if name == "silu":
        return v / (1 + torch.exp(-v))
    return v


def dense_gates(routes, slots, E):
    """int32 [T, 2 * slots] records -> [T, E] fp64 gates, bad and empty slots left out."""
    idx = routes[:, :slots].cpu()
    gate = routes[:, slots:].contiguous().view(torch.float32).cpu().double()
    ok = (idx >= 0) & (idx < E) & torch.isfinite(gate)
    d = torch.zeros((routes.shape[0], E), dtype=torch.float64)
    d.scatter_add_(1, torch.where(ok, idx, 0).long(), torch.where(ok, gate, 0.0))
    return d


def product(x, W, *, bias=None, activation="none", mul=None, residual=None, routes=None, slots=0,
            A=None, B=None, s=0.0, out_dtype=torch.bfloat16):
    """-> (y fp64, tol fp64): the exact value of every element, and how far a
    kernel of the documented arithmetic may be from it.

    The bound, with u(t) = finfo(t).eps / 2:
      products     the tensor cores add 16 products at a time onto an fp32
                   accumulator without rounding to nearest: at most 2^-22 of
                   the terms' magnitude M = sum |x w| for each of in / 16
                   steps and 16 more for joining partial sums;
      adapters     u = x A^T the same way, gated and rounded to bf16 (2^-8 of
                   each term) or, for fp32 outputs, to two bf16 terms (2^-16),
                   then summed over the experts' ranks;
      activation   slopes at most 1.13; evaluated to 2^-20 (1 + |v|);
      epilogue     three fp32 roundings and the last one, u(out_dtype) |y|."""
    d = lambda t: t.detach().double().cpu()
    x, W = d(x), d(W)
    v = x @ W.t()
    steps = x.shape[1] / 16 + 16
    M = x.abs() @ W.abs().t()
    err = steps * 2.0 ** -22 * M
    if routes is not None:
        E, r, _ = A.shape
        gates = dense_gates(routes, slots, E)
        A, B = d(A), d(B)
        fine = 2.0 ** -8 if out_dtype == torch.bfloat16 else 2.0 ** -16
        for e in range(E):
            rows = torch.nonzero(gates[:, e] != 0).flatten()
            if not rows.numel():
                continue
            c = s * gates[rows, e][:, None]
            u = c * (x[rows] @ A[e].t())
            mu = c.abs() * (x[rows].abs() @ A[e].abs().t())
            v[rows] += u @ B[e].t()
            mag = u.abs() @ B[e].abs().t()
            err[rows] += fine * mag + (steps * 2.0 ** -22 * mu) @ B[e].abs().t()
            err[rows] += (r * E / 16 + 16) * 2.0 ** -22 * mag + 2.0 ** -22 * M[rows]
    if bias is not None:
        v = v + d(bias)
        err = err + 2.0 ** -24 * v.abs()
    y = act(v, activation)
    err = 1.13 * err + 2.0 ** -20 * (1 + v.abs()) if activation != "none" else err
    if mul is not None:
        err = err * d(mul).abs()
        y = y * d(mul)
        err = err + 2.0 ** -23 * y.abs()
    if residual is not None:
        err = err + 2.0 ** -23 * (y.abs() + d(residual).abs())
        y = y + d(residual)
    tol = err + (torch.finfo(out_dtype).eps / 2) * (y.abs() + err) + 1e-37
    return y, tol
