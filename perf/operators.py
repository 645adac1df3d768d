"""The forward pass of tokens that carry their own experts: three operators, as
they are measured.

route   routing to experts.  logits z = h Wr; scores = softmax or sigmoid of z;
        selection by score (+ a balance bias per expert) inside the best groups
        of experts; k picks, lower index first among equals; gates = the picks'
        scores, renormalised if asked, times a factor.
linear  y = residual + mul * act(x W^T + bias) on one weight of the model.
routed  the same with every token's own gated experts, W left as it is:
        y = residual + mul * act(x W^T + bias + s sum_j g_j (x A_e^T) B_e^T).

Sizes are those of the repository's workloads (Llama-2-7B, 13B and Llama-3-8B
shapes, E = 8 or 16, ranks 4 to 64) and generic ones between them.
"""
import math

import numpy as np
import torch

own = False

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def listed():
    return [
        # the router on one decoded token, top-2 of 8
        dict(name="route-token", op="route", T=1, d=4096, E=8, score="softmax", k=2, groups=1,
             top_groups=1, group_top=1, bias=False, renorm=True, scale=1.0, f32=True, pad=0),
        # a prompt of 4096 tokens, 16 experts in 4 groups, balanced by a bias
        dict(name="route-prompt", op="route", T=4096, d=4096, E=16, score="sigmoid", k=4, groups=4,
             top_groups=2, group_top=2, bias=True, renorm=True, scale=2.5, f32=False, pad=0),
        # an odd batch over many experts at the 13B width
        dict(name="route-odd", op="route", T=777, d=5120, E=64, score="softmax", k=8, groups=8,
             top_groups=3, group_top=1, bias=False, renorm=False, scale=1.0, f32=True, pad=8),
        # one decoded token through the gated half of a feed-forward block
        dict(name="linear-token", op="linear", T=1, inn=4096, out=11008, bias=False, act="silu",
             mul=True, residual=False, f32=False, pad=0),
        # a decode batch through the block's last product, onto an fp32 residual stream
        dict(name="linear-batch", op="linear", T=61, inn=11008, out=4096, bias=False, act="none",
             mul=False, residual=True, f32=True, pad=0),
        # an odd prompt through a grouped key projection with a bias
        dict(name="linear-odd", op="linear", T=1037, inn=4096, out=1024, bias=True, act="gelu_tanh",
             mul=False, residual=False, f32=False, pad=8),
        # a full prompt through the gate product of a feed-forward block
        dict(name="linear-prompt", op="linear", T=4096, inn=4096, out=14336, bias=False, act="silu",
             mul=True, residual=False, f32=False, pad=0),
        # one decoded token that keeps W unmerged
        dict(name="routed-token", op="routed", T=1, inn=4096, out=4096, E=8, rank=8, k=2, slots=2,
             bias=False, act="none", mul=False, residual=True, f32=False, pad=0, empty=0.0),
        # a decode batch in which every sequence has its own experts
        dict(name="routed-batch", op="routed", T=24, inn=5120, out=13824, E=8, rank=16, k=2, slots=2,
             bias=False, act="silu", mul=True, residual=False, f32=False, pad=0, empty=0.1),
        # an odd batch on a small rank, three experts a token, some tokens with none
        dict(name="routed-odd", op="routed", T=333, inn=4096, out=1024, E=4, rank=4, k=3, slots=4,
             bias=True, act="none", mul=False, residual=False, f32=False, pad=8, empty=0.2),
        # a full prompt through the last product of a block, onto an fp32 residual stream
        dict(name="routed-prompt", op="routed", T=4096, inn=11008, out=4096, E=8, rank=8, k=2, slots=2,
             bias=False, act="none", mul=False, residual=True, f32=True, pad=0, empty=0.0),
        # a long prompt on 16 experts of rank 64
        dict(name="routed-rank64", op="routed", T=2048, inn=4096, out=4096, E=16, rank=64, k=2, slots=2,
             bias=False, act="none", mul=False, residual=False, f32=False, pad=0, empty=0.0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "linear", "routed"])
    T = _log(rng, 1, 4096)
    if op == "route":
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * rng.randint(1 if groups > 1 else 2, 64 // groups)
        top_groups = rng.randint(1, groups)
        return dict(op=op, T=T, d=4 * _log(rng, 64, 1280), E=E, score=rng.choice(["softmax", "sigmoid"]),
                    k=rng.randint(1, min(8, E)), groups=groups, top_groups=top_groups,
                    group_top=rng.choice([1, 2]), bias=rng.random() < 0.5, renorm=rng.random() < 0.5,
                    scale=rng.choice([1.0, 2.5]), f32=rng.random() < 0.5, pad=rng.choice([0, 8]))
    inn, out = 8 * _log(rng, 32, 1792), 8 * _log(rng, 32, 1792)
    T = max(1, min(T, 4096 * 4096 * 14336 // (2 * inn * out)))
    c = dict(op=op, T=T, inn=inn, out=out, bias=rng.random() < 0.5, act=rng.choice(ACTS),
             mul=rng.random() < 0.3, residual=rng.random() < 0.5, f32=rng.random() < 0.4,
             pad=rng.choice([0, 8, 24]))
    if op == "routed":
        E = rng.choice([2, 3, 4, 8, 8, 12, 16, 16])
        k = rng.randint(1, min(8, E, 4 if rng.random() < 0.8 else 8))
        c.update(E=E, rank=rng.choice([1, 2, 4, 8, 8, 12, 16, 16, 20, 24, 32, 64]), k=k,
                 slots=2 if k <= 2 else 4 if k <= 4 else 8, empty=rng.choice([0.0, 0.1, 0.5]))
    return c


def _rows(g, T, n, pad, dtype, std=1.0):
    """[T, n] rows, `pad` elements apart from the next row's start."""
    full = torch.empty((T, n + pad), dtype=torch.float32, device="cuda").normal_(0.0, std, generator=g)
    return full.to(dtype)[:, :n]


def _inputs(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 1000003 + 17)
    c = case
    if c["op"] == "route":
        s = dict(h=_rows(g, c["T"], c["d"], c["pad"], torch.float32 if c["f32"] else torch.bfloat16),
                 Wr=torch.empty((c["d"], c["E"]), device="cuda").normal_(0.0, 0.05, generator=g),
                 bias=None)
        if c["bias"]:
            s["bias"] = torch.empty((c["E"],), device="cuda").normal_(0.0, 0.1, generator=g)
        return s
    io = torch.float32 if c["f32"] else torch.bfloat16
    T, inn, out = c["T"], c["inn"], c["out"]
    s = dict(x=_rows(g, T, inn, c["pad"], torch.bfloat16), W=_rows(g, out, inn, 0, torch.bfloat16, 0.02),
             bias=None, mul=None, residual=None)
    if c["bias"]:
        s["bias"] = torch.empty((out,), device="cuda").normal_(0.0, 0.5, generator=g)
    if c["mul"]:
        s["mul"] = _rows(g, T, out, c["pad"], io)
    if c["residual"]:
        s["residual"] = _rows(g, T, out, c["pad"], io)
    if c["op"] == "routed":
        E, r, k = c["E"], c["rank"], c["k"]
        s["A"] = torch.empty((E, r, inn), device="cuda").normal_(0.0, inn ** -0.5, generator=g).to(torch.bfloat16)
        s["B"] = torch.empty((E, out, r), device="cuda").normal_(0.0, 0.01, generator=g).to(torch.bfloat16)
        s["factor"] = 2.0
        # records as a router writes them: k experts in order of their gates, idx then gate
        z = torch.empty((T, E), device="cuda").normal_(0.0, 2.0, generator=g)
        top = torch.topk(z, k, dim=1)
        idx = torch.full((T, c["slots"]), -1, dtype=torch.int32, device="cuda")
        gate = torch.zeros((T, c["slots"]), device="cuda")
        idx[:, :k] = top.indices.to(torch.int32)
        gate[:, :k] = torch.softmax(top.values, dim=1)
        none = torch.rand((T,), device="cuda", generator=g) < c["empty"]
        idx[none] = -1
        s["routes"] = torch.cat([idx, gate.view(torch.int32)], dim=1).contiguous()
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    c = s["case"] = dict(case)
    if own:
        from weight_merge_b200 import binding as B
        if c["op"] == "route":
            w = torch.zeros((8, 8), dtype=torch.bfloat16, device="cuda")
            a = torch.zeros((c["E"], 8, 8), dtype=torch.bfloat16, device="cuda")
            s["sw"] = B.Switcher([w], [a], [a], 1, 1, c["E"], 8, 16.0)
            s["gating"] = B.make_gating(
                score=B.ADAFUSE_SCORE_SOFTMAX if c["score"] == "softmax" else B.ADAFUSE_SCORE_SIGMOID,
                k=c["k"], n_groups=c["groups"], top_groups=c["top_groups"], group_top=c["group_top"],
                renorm=c["renorm"], scale=c["scale"], bias=s["bias"])
            s["slots"] = 2 if c["k"] <= 2 else 4 if c["k"] <= 4 else 8
            s["routes"] = torch.empty((c["T"], 2 * s["slots"]), dtype=torch.int32, device="cuda")
            return s
        routed = c["op"] == "routed"
        A = s["A"] if routed else torch.zeros((1, 8, c["inn"]), dtype=torch.bfloat16, device="cuda")
        Bm = s["B"] if routed else torch.zeros((1, c["out"], 8), dtype=torch.bfloat16, device="cuda")
        r = A.shape[1]
        s["sw"] = B.Switcher([s["W"]], [A], [Bm], 1, 1, A.shape[0], r, 2.0 * r)
        s["act"] = getattr(B, "ADAFUSE_ACT_" + c["act"].upper())
        s["y"] = torch.empty((c["T"], c["out"]), dtype=torch.float32 if c["f32"] else torch.bfloat16,
                             device="cuda")
        if routed:
            n = s["sw"].linear_workspace(0, 0, c["T"], c["f32"])
            s["workspace"] = torch.empty((max(n, 1),), dtype=torch.uint8, device="cuda")
    return s


def _act(v, name):
    if name == "relu":
        return torch.clamp(v, min=0.0)
    if name == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * math.sqrt(0.5)))
    if name == "gelu_tanh":
        return 0.5 * v * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v * v * v)))
    if name == "silu":
        return v / (1.0 + torch.exp(-v))
    return v


def _plain_route(s):
    c = s["case"]
    T, E, G, k = c["T"], c["E"], c["groups"], c["k"]
    # picks are decided in 64 bits: 32 lose the order of scores next to each other
    z = s["h"].double() @ s["Wr"].double()
    if c["score"] == "softmax":
        e = torch.exp(z - z.max(dim=1, keepdim=True).values)
        score = e / e.sum(dim=1, keepdim=True)
    else:
        score = 1.0 / (1.0 + torch.exp(-z))
    by = score + s["bias"].double() if c["bias"] else score
    key = by if c["bias"] else z
    if G > 1:
        best = torch.sort(by.view(T, G, E // G), dim=2, descending=True).values
        of_group = best[:, :, :c["group_top"]].sum(dim=2)
        order = torch.sort(of_group, dim=1, descending=True, stable=True).indices
        kept = torch.zeros((T, G), dtype=torch.bool, device=z.device)
        kept.scatter_(1, order[:, :c["top_groups"]], True)
        key = torch.where(kept.repeat_interleave(E // G, dim=1), key, -math.inf)
    val, idx = torch.sort(key, dim=1, descending=True, stable=True)
    idx, there = idx[:, :k], val[:, :k] > -math.inf
    gate = torch.where(there, torch.gather(score, 1, idx), 0.0)
    if c["renorm"]:
        gate = gate / gate.sum(dim=1, keepdim=True)
    gate = gate * c["scale"]
    slots = 2 if k <= 2 else 4 if k <= 4 else 8
    oi = torch.full((T, slots), -1, dtype=torch.int32, device=z.device)
    og = torch.zeros((T, slots), device=z.device)
    oi[:, :k] = torch.where(there, idx, -1).to(torch.int32)
    og[:, :k] = gate.float()
    return {"idx": oi, "gate": og}


def _plain_linear(s):
    c = s["case"]
    v = s["x"].float() @ s["W"].float().t()
    if c["bias"]:
        v = v + s["bias"]
    if c["op"] == "routed":
        E, r, n = c["E"], c["rank"], c["slots"]
        idx, gate = s["routes"][:, :n], s["routes"][:, n:].view(torch.float32)
        dense = torch.zeros((c["T"], E), device=v.device)
        dense.scatter_add_(1, idx.clamp(min=0).long(), torch.where(idx >= 0, gate, 0.0))
        u = (s["x"].float() @ s["A"].float().view(E * r, -1).t()).view(-1, E, r)
        u = (u * (s["factor"] * dense).unsqueeze(2)).view(-1, E * r)
        v = v + u @ s["B"].float().permute(0, 2, 1).reshape(E * r, -1)
    v = _act(v, c["act"])
    if c["mul"]:
        v = v * s["mul"].float()
    if c["residual"]:
        v = v + s["residual"].float()
    return v if c["f32"] else v.to(torch.bfloat16)


def run(state):
    s = state
    op = s["case"]["op"]
    if not own:
        return _plain_route(s) if op == "route" else {"y": _plain_linear(s)}
    stream = torch.cuda.current_stream().cuda_stream
    if op == "route":
        s["sw"].route_experts(s["h"], s["Wr"], s["gating"], s["routes"], stream)
        n = s["slots"]
        return {"idx": s["routes"][:, :n], "gate": s["routes"][:, n:].view(torch.float32)}
    more = dict(bias=s["bias"], activation=s["act"], mul=s["mul"], residual=s["residual"], stream=stream)
    if op == "linear":
        s["sw"].linear(0, 0, s["x"], s["y"], **more)
    else:
        s["sw"].linear_routed(0, 0, s["x"], s["routes"], s["y"], s["workspace"], **more)
    return {"y": s["y"]}


def work(case):
    c = case
    T = c["T"]
    if c["op"] == "route":
        slots = 2 if c["k"] <= 2 else 4 if c["k"] <= 4 else 8
        return {"bytes": T * c["d"] * (4 if c["f32"] else 2) + 4 * c["d"] * c["E"] + 8 * slots * T
                + (4 * c["E"] if c["bias"] else 0),
                "flops": 2 * T * c["d"] * c["E"]}
    inn, out, io = c["inn"], c["out"], 4 if c["f32"] else 2
    moved = 2 * inn * out + 2 * T * inn + io * T * out * (1 + c["mul"] + c["residual"]) + (4 * out if c["bias"] else 0)
    flops = 2 * T * inn * out
    if c["op"] == "routed":
        picks = T * (1.0 - c["empty"]) * c["k"]
        used = c["E"] * (1.0 - (1.0 - c["k"] / c["E"]) ** (T * (1.0 - c["empty"])))
        moved += int(used * c["rank"] * (inn + out) * 2) + 8 * c["slots"] * T
        flops += int(2 * picks * c["rank"] * (inn + out))
    return {"bytes": moved, "flops": flops}


def _exact_route(c, s):
    """Token by token, in 64 bits: the definition, pick by pick."""
    z_all = (s["h"].double().cpu().numpy() @ s["Wr"].double().cpu().numpy())
    bias = s["bias"].double().cpu().numpy() if c["bias"] else None
    T, E, G, k = c["T"], c["E"], c["groups"], c["k"]
    slots = 2 if k <= 2 else 4 if k <= 4 else 8
    oi, og = np.full((T, slots), -1, np.int32), np.zeros((T, slots))
    per = E // G
    for t in range(T):
        z = z_all[t]
        if c["score"] == "softmax":
            p = np.exp(z - z.max())
            p /= p.sum()
        else:
            p = np.where(z >= 0, 1 / (1 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1 + np.exp(-np.abs(z))))
        q = p if bias is None else p + bias
        rank_by = z if bias is None else q
        allowed = list(range(E))
        if G > 1:
            worth = [sum(sorted(q[g * per:(g + 1) * per], reverse=True)[:c["group_top"]]) for g in range(G)]
            best = sorted(range(G), key=lambda g: (-worth[g], g))[:c["top_groups"]]
            allowed = [e for e in allowed if e // per in best]
        picks = sorted(allowed, key=lambda e: (-rank_by[e], e))[:k]
        w = p[picks]
        if c["renorm"]:
            w = w / w.sum()
        oi[t, :len(picks)] = picks
        og[t, :len(picks)] = w * c["scale"]
    return {"idx": torch.from_numpy(oi), "gate": torch.from_numpy(og)}


def exact(case, seed):
    c, s = case, _inputs(case, seed)
    if c["op"] == "route":
        return _exact_route(c, s)
    x = s["x"].to(torch.float64)
    v = torch.nn.functional.linear(x, s["W"].to(torch.float64))
    if c["bias"]:
        v += s["bias"].to(torch.float64)
    if c["op"] == "routed":
        n = c["slots"]
        idx, gate = s["routes"][:, :n], s["routes"][:, n:].view(torch.float32).to(torch.float64)
        for e in range(c["E"]):
            g = torch.where(idx == e, gate, 0.0).sum(dim=1)
            rows = torch.nonzero(g != 0).flatten()
            if rows.numel():
                low = torch.nn.functional.linear(x[rows], s["A"][e].to(torch.float64))
                v[rows] += s["factor"] * g[rows, None] * torch.nn.functional.linear(low, s["B"][e].to(torch.float64))
    if c["act"] == "relu":
        v = torch.where(v > 0, v, 0.0)
    elif c["act"] == "gelu":
        v = v * 0.5 * torch.erfc(-v / math.sqrt(2.0))
    elif c["act"] == "gelu_tanh":
        v = v / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    elif c["act"] == "silu":
        v = v * torch.sigmoid(v)
    if c["mul"]:
        v = v * s["mul"].to(torch.float64)
    if c["residual"]:
        v = v + s["residual"].to(torch.float64)
    return {"y": v}
