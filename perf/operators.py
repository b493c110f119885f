"""The operators of a routed expert layer around the grouped FP8 GEMMs, as cases to be measured.

Four kinds of pass, each a dict with "op":

  route     scores of E experts -> the top_k of each token with their weights (and, with "grad", the
            gradient of the router's logits);
  dispatch  the expert order of the routed rows (the plan), then every token's row quantised in that
            order: the 1x128 codes and, with "both", the ragged 128x1 transposed ones of the weight
            gradient;
  combine   the experts' output rows back to tokens, weighted (and, with "grad", the backward pass:
            the gradient of the weights and the quantised gradient of the rows);
  swiglu    a = silu(gate) * up quantised for the next GEMM, with the 8-bit checkpoint of its input
            (and, with "grad", the backward pass from that checkpoint).

With ``own`` false ``run`` computes them from elementary torch operations; with ``own`` true it makes
the calls of fp8_fine_grained_fp8q_b200.ops.
"""
import math

import torch

own = False

G = 128            # elements of a quantisation group
TOP = 448.0        # largest finite E4M3 value
FLOOR = 2.0 ** -100
F8 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------------------------- #
# Cases
# ---------------------------------------------------------------------------------------------- #

def listed():
    route = dict(op="route", E=256, k=8, groups=8, keep=4, score="sigmoid", bias=True, renorm=True, scale=2.5,
                 dtype="fp32", masked=0)
    return [
        # One token being decoded: the latency of the call is all there is.
        dict(route, name="route_step", T=1, grad=False),
        # A training batch of 8192 tokens over 256 experts, forward and backward.
        dict(route, name="route_train", T=8192, grad=True),
        # Softmax scores without groups or a bias, bf16 logits, an odd batch, three experts switched off.
        dict(name="route_softmax", op="route", T=5003, E=96, k=4, groups=1, keep=1, score="softmax", bias=False,
             renorm=False, scale=1.0, dtype="bf16", masked=3, grad=True),
        # A small odd batch being served: codes of the rows only.
        dict(name="dispatch_serve", op="dispatch", T=37, E=256, k=8, C=7168, both=False),
        # The training batch: both operand forms, for the experts' Fprop and Wgrad.
        dict(name="dispatch_train", op="dispatch", T=8192, E=256, k=8, C=7168, both=True),
        # One token's eight expert rows summed.
        dict(name="combine_step", op="combine", T=1, E=256, k=8, C=7168, weighted=True, add=False, grad=False),
        # The training batch, onto the output of an expert that every token shares.
        dict(name="combine_train", op="combine", T=8192, E=256, k=8, C=7168, weighted=True, add=True, grad=False),
        # Its backward pass: the weights' gradient, and the rows' in both operand forms.
        dict(name="combine_grad", op="combine", T=8192, E=256, k=8, C=7168, weighted=True, add=False, grad=True),
        # One token's rows in eight experts.
        dict(name="swiglu_step", op="swiglu", M=8, I=2048, E=0, keep=False, grad=False),
        # The training batch's 65536 expert rows, with the checkpoint.
        dict(name="swiglu_train", op="swiglu", M=65536, I=2048, E=0, keep=True, grad=False),
        # Its backward pass, rows grouped by expert.
        dict(name="swiglu_grad", op="swiglu", M=65536, I=2048, E=256, keep=True, grad=True),
        # The backward pass of one dense feed-forward layer, an odd number of tokens.
        dict(name="swiglu_grad_dense", op="swiglu", M=3001, I=1408, E=0, keep=True, grad=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "dispatch", "combine", "swiglu"])
    T = _log(rng, 1, 8192)
    if op == "route":
        score = rng.choice(["sigmoid", "softmax"])
        groups = rng.choice([1, 1, 2, 4, 8])
        E = groups * _log(rng, 4, 256 // groups)
        keep = rng.randint(max(1, groups // 2), groups)
        return dict(op=op, T=T, E=E, k=rng.randint(1, min(8, keep * (E // groups))), groups=groups, keep=keep,
                    score=score, bias=rng.random() < 0.6, renorm=rng.random() < 0.6, scale=rng.choice([1.0, 2.5]),
                    dtype=rng.choice(["fp32", "bf16"]), masked=rng.choice([0, 0, 1]), grad=rng.random() < 0.6)
    E = _log(rng, 8, 256)
    k = rng.randint(1, 8)
    C = G * rng.randint(4, 56)
    if op == "dispatch":
        return dict(op=op, T=T, E=E, k=k, C=C, both=rng.random() < 0.6)
    if op == "combine":
        return dict(op=op, T=T, E=E, k=k, C=C, weighted=rng.random() < 0.7, add=rng.random() < 0.5,
                    grad=rng.random() < 0.5)
    grad = rng.random() < 0.6
    return dict(op=op, M=_log(rng, 1, 65536), I=G * rng.randint(2, 16), E=E if grad and rng.random() < 0.7 else 0,
                keep=grad or rng.random() < 0.6, grad=grad)


def _capacity(M, E):
    """Padded token columns that suffice for M rows over E experts (E = 0: one sequence of rows)."""
    return G * (-(-M // G) + E)


def work(case):
    c, op = case, case["op"]
    if op == "route":
        T, E, k = c["T"], c["E"], c["k"]
        e = 4 if c["dtype"] == "fp32" else 2
        nbytes = T * E * e + T * k * 8 + (4 * E if c["bias"] else 0)
        if c["grad"]:
            nbytes += T * E * e + T * k * 4
        return {"bytes": nbytes, "flops": T * E * 8}
    if op == "swiglu":
        M, I = c["M"], c["I"]
        if not c["grad"]:
            nbytes = 4 * M * I + M * I + M * I // 32
            nbytes += (2 * M * I + M * I // 16) if c["keep"] else 0
            return {"bytes": nbytes, "flops": 12 * M * I}
        nbytes = 2 * M * I + 2 * M * I + M * I // 16            # da, the checkpoint
        nbytes += 2 * M * I + M * I // 16 + 3 * M * I + 3 * M * I // 32
        return {"bytes": nbytes, "flops": 30 * M * I}
    T, k, C = c["T"], c["k"], c["C"]
    M = T * k
    row = C + C // 32                                          # a quantised row: codes and scales
    if op == "dispatch":
        return {"bytes": 4 * M * 3 + 2 * T * C + M * row * (2 if c["both"] else 1), "flops": 4 * M * C}
    if not c["grad"]:
        return {"bytes": 2 * M * C + 2 * T * C + 8 * M + (2 * T * C if c["add"] else 0), "flops": 2 * M * C}
    nbytes = 2 * T * C + 8 * M + 2 * M * row
    if c["weighted"]:
        nbytes += 2 * M * C + 8 * M
    return {"bytes": nbytes, "flops": 6 * M * C}


# ---------------------------------------------------------------------------------------------- #
# Inputs
# ---------------------------------------------------------------------------------------------- #

def _routing(g, T, E, k):
    """Distinct experts for each token, of uneven popularity; some of them get no token."""
    popular = -1.1 * torch.log(1.0 + torch.randperm(E, generator=g, device="cuda").float())
    popular[torch.randperm(E, generator=g, device="cuda")[: max(0, min(E // 32, E - k))]] = -1e4
    u = torch.rand(T, E, generator=g, device="cuda").clamp_(1e-7, 1.0 - 1e-7)
    return torch.topk(popular - torch.log(-torch.log(u)), k, dim=-1).indices.to(torch.int32).contiguous()


def _activations(g, M, C):
    """N(0, 1) with one channel in a thousand a hundred times as large."""
    x = torch.randn(M, C, generator=g, device="cuda")
    x[:, torch.randperm(C, generator=g, device="cuda")[: max(1, C // 1000)]] *= 100.0
    return x.to(torch.bfloat16)


def _grads(g, M, C):
    """N(0, 1e-3) with a heavy tail: one entry in a hundred is the quotient of two normals."""
    y = torch.randn(M, C, generator=g, device="cuda")
    t = torch.rand(M, C, generator=g, device="cuda")
    y = torch.where(t < 0.01, y / (0.05 + 100.0 * t), y)
    return (1e-3 * y).to(torch.bfloat16)


def _rows_buffers(M, C):
    return torch.zeros(M, C, dtype=torch.uint8, device="cuda"), torch.zeros(C // G, M, device="cuda")


def _cols_buffers(C, cap):
    return torch.zeros(C, cap, dtype=torch.uint8, device="cuda"), torch.zeros(cap // G, C, device="cuda")


def prepare(case, seed):
    c, op = case, case["op"]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if op == "route":
        T, E, k = c["T"], c["E"], c["k"]
        logits = torch.randn(T, E, generator=g, device="cuda") + 0.7 * torch.randn(E, generator=g, device="cuda")
        if c["masked"]:
            logits[:, torch.randperm(E, generator=g, device="cuda")[: min(c["masked"], E - k)]] = -math.inf
        logits = logits.to(torch.float32 if c["dtype"] == "fp32" else torch.bfloat16)
        bias = 0.05 * torch.randn(E, generator=g, device="cuda") if c["bias"] else None
        return dict(case=c, logits=logits, bias=bias, dw=1e-2 * torch.randn(T, k, generator=g, device="cuda"))
    if op == "swiglu":
        M, I = c["M"], c["I"]
        h = torch.randn(M, 2 * I, generator=g, device="cuda").to(torch.bfloat16)
        if not c["grad"]:
            return dict(case=c, h=h)
        q, s = _quant_rows(h.float())
        offsets, cap = None, _capacity(M, 0)
        if c["E"]:
            e = torch.sort(_routing(g, M, c["E"], 1).reshape(-1)).values
            offsets = torch.searchsorted(e, torch.arange(c["E"] + 1, device="cuda", dtype=torch.int32)).to(torch.int32)
            cap = _capacity(M, c["E"])
        return dict(case=c, da=_grads(g, M, I), hq=q.view(torch.uint8), hs=s, offsets=offsets, cap=cap,
                    rows=_rows_buffers(M, 2 * I), cols=_cols_buffers(2 * I, cap), acts=_cols_buffers(I, cap))
    T, E, k, C = c["T"], c["E"], c["k"], c["C"]
    E = max(E, k)
    M, cap = T * k, _capacity(T * k, E)
    idx = _routing(g, T, E, k)
    state = dict(case=c, E=E, cap=cap)
    if op == "dispatch":
        state.update(idx=idx, x=_activations(g, T, C), rows=_rows_buffers(M, C))
        if c["both"]:
            state["cols"] = _cols_buffers(C, cap)
        return state
    w = torch.rand(T, k, generator=g, device="cuda") + 0.05
    state.update(zip(("offsets", "slots", "back"), _plan(idx, E)))
    state["w"] = 2.5 * w / w.sum(-1, keepdim=True) if c["weighted"] else None
    if c["grad"]:
        state.update(dout=_grads(g, T, C), rows=_rows_buffers(M, C), cols=_cols_buffers(C, cap))
    if c["weighted"] or not c["grad"]:
        state["y"] = torch.randn(M, C, generator=g, device="cuda").to(torch.bfloat16)
    state["add"] = torch.randn(T, C, generator=g, device="cuda").to(torch.bfloat16) if c["add"] else None
    return state


# ---------------------------------------------------------------------------------------------- #
# One pass
# ---------------------------------------------------------------------------------------------- #

def run(state):
    if own:
        return _run_own(state)
    return {"route": _plain_route, "dispatch": _plain_dispatch, "combine": _plain_combine,
            "swiglu": _plain_swiglu}[state["case"]["op"]](state)


def _run_own(st):
    from fp8_fine_grained_fp8q_b200 import ops

    c, op = st["case"], st["case"]["op"]
    if op == "route":
        idx, w = ops.moe_route(st["logits"], c["k"], bias=st["bias"], score=c["score"], n_group=c["groups"],
                               topk_group=c["keep"], renormalize=c["renorm"], scale=c["scale"])
        if not c["grad"]:
            return [idx, w]
        return [idx, w, ops.moe_route_backward(st["dw"], w, idx, st["logits"], score=c["score"],
                                               renormalize=c["renorm"], scale=c["scale"])]
    if op == "dispatch":
        plan = ops.moe_plan(st["idx"], st["E"])
        q, s = st["rows"]
        qt, t = st["cols"] if c["both"] else (None, None)
        ops.moe_dispatch(st["x"], plan, transposed=c["both"], q=q, s=s, qt=qt, st=t)
        out = [plan.offsets, plan.slots, plan.rows, q.view(F8), s]
        return out + [qt.view(F8), t] if c["both"] else out
    if op == "combine":
        plan = ops.MoePlan(st["offsets"], st["slots"], st["back"])
        if not c["grad"]:
            return ops.moe_combine(st["y"], plan, weights=st["w"], add=st["add"])
        (q, s), (qt, t) = st["rows"], st["cols"]
        ops.moe_dispatch(st["dout"], plan, weights=st["w"], transposed=True, q=q, s=s, qt=qt, st=t)
        out = [q.view(F8), s, qt.view(F8), t]
        return out + [ops.moe_combine_dweight(st["dout"], st["y"], plan)] if c["weighted"] else out
    if not c["grad"]:
        q, s, hq, hs = ops.swiglu_quant(st["h"], checkpoint=c["keep"])
        return [q.view(F8), s] + ([hq.view(F8), hs] if c["keep"] else [])
    (q, s), (qt, t), (aqt, at) = st["rows"], st["cols"], st["acts"]
    ops.swiglu_backward_quant(st["da"], st["hq"], st["hs"], offsets=st["offsets"], q=q, s=s, qt=qt, st=t, aqt=aqt,
                              ast=at)
    return [q.view(F8), s, qt.view(F8), t, aqt.view(F8), at]


# ---------------------------------------------------------------------------------------------- #
# The plain forms
# ---------------------------------------------------------------------------------------------- #

def _codes(v, a):
    """E4M3 codes and the scale of groups whose largest magnitude is `a` (broadcast against v): IEEE
    divisions (a tensor by a tensor), one product, one rounding."""
    a = a.clamp_min(FLOOR)
    top = torch.full_like(a, TOP)
    return (v * (top / a)).clamp(-TOP, TOP).to(F8), a / top


def _quant_rows(v):
    """1x128 groups: v [M, C] fp32 -> codes [M, C], scales [C/128, M]."""
    M, C = v.shape
    v = v.view(M, C // G, G)
    q, s = _codes(v, v.abs().amax(-1, keepdim=True))
    return q.view(M, C), s.view(M, C // G).t().contiguous()


def _places(offsets, M):
    """Padded column of each row, and the number of padded groups."""
    counts = offsets[1:] - offsets[:-1]
    groups = (counts + (G - 1)) // G
    first = torch.cumsum(groups, 0) - groups
    e = torch.searchsorted(offsets[1:].contiguous(), torch.arange(M, device="cuda", dtype=torch.int32), right=True)
    return torch.arange(M, device="cuda") - offsets[e] + G * first[e], groups.sum()


def _quant_cols(v, offsets, cap):
    """128x1 groups over each expert's own rows, transposed: v [M, C] fp32 -> [C, cap], [cap/128, C].
    What lies behind the last group stays zero."""
    M, C = v.shape
    if offsets is None:
        at, groups = torch.arange(M, device="cuda"), -(-M // G)
    else:
        at, groups = _places(offsets, M)
    padded = v.new_zeros(cap, C)
    padded[at] = v
    padded = padded.view(cap // G, G, C)
    q, s = _codes(padded, padded.abs().amax(1, keepdim=True))
    s = s.view(cap // G, C) * (torch.arange(cap // G, device="cuda") < groups)[:, None]
    return q.view(torch.uint8).view(cap, C).t().contiguous().view(F8), s


def _plan(idx, E):
    """Rows ordered by expert, then by slot: offsets [E+1], the slot of each row, the row of each slot."""
    flat = idx.reshape(-1)
    e, slots = torch.sort(flat, stable=True)
    offsets = torch.searchsorted(e, torch.arange(E + 1, device="cuda", dtype=torch.int32))
    back = torch.empty_like(slots)
    back[slots] = torch.arange(slots.numel(), device="cuda")
    return offsets.to(torch.int32), slots.to(torch.int32), back.to(torch.int32).view(idx.shape)


def _plain_route(st):
    c, l, bias = st["case"], st["logits"].double(), st["bias"]
    T, E = l.shape
    k, groups = c["k"], c["groups"]
    if c["score"] == "sigmoid":
        s = torch.sigmoid(l)
    else:
        s = torch.exp(l - l.amax(-1, keepdim=True))
        s = s / s.sum(-1, keepdim=True)
    key = l if bias is None else s + bias.double()
    key = key.masked_fill(torch.isinf(l), -1e300)
    if groups > 1:
        per = key.view(T, groups, E // groups)
        best = per.topk(min(2, E // groups), dim=-1).values if bias is not None else per.amax(-1, keepdim=True)
        best = best.masked_fill(best == -1e300, 0.0).sum(-1).masked_fill(per.amax(-1) == -1e300, -1e300)
        kept = torch.sort(best, dim=-1, descending=True, stable=True).indices[:, : c["keep"]]
        allowed = torch.zeros(T, groups, dtype=torch.bool, device="cuda").scatter_(1, kept, True)
        key = per.masked_fill(~allowed[:, :, None], -math.inf).view(T, E)
    idx = torch.sort(key, dim=-1, descending=True, stable=True).indices[:, :k]
    p = s.gather(1, idx)
    if c["renorm"]:
        p, r = p / p.sum(-1, keepdim=True), p
    else:
        r = p
    w = p * c["scale"]
    out = [idx.to(torch.int32), w.float()]
    if not c["grad"]:
        return out
    g = st["dw"].double()
    if c["renorm"]:
        g = w * (g - (g * p).sum(-1, keepdim=True))
    else:
        g = w * g
    if c["score"] == "sigmoid":
        d = torch.zeros_like(l).scatter_(1, idx, g * (1.0 - r))
    else:
        d = torch.zeros_like(l).scatter_(1, idx, g)
        if not c["renorm"]:
            d = d - s * g.sum(-1, keepdim=True)
    return out + [d.to(st["logits"].dtype)]


def _plain_dispatch(st):
    c = st["case"]
    offsets, slots, back = _plan(st["idx"], st["E"])
    v = st["x"][(slots // c["k"]).long()].float()
    out = [offsets, slots, back, *_quant_rows(v)]
    return out + [*_quant_cols(v, offsets, st["cap"])] if c["both"] else out


def _plain_combine(st):
    c, w = st["case"], st["w"]
    if not c["grad"]:
        y = st["y"][st["back"].long()].float()
        out = (y if w is None else y * w[:, :, None]).sum(1)
        if st["add"] is not None:
            out = out + st["add"].float()
        return out.to(torch.bfloat16)
    v = st["dout"][(st["slots"] // c["k"]).long()].float()
    if w is not None:
        v = v * w.reshape(-1)[st["slots"].long()][:, None]
    out = [*_quant_rows(v), *_quant_cols(v, st["offsets"], st["cap"])]
    if w is None:
        return out
    return out + [(st["y"][st["back"].long()].float() * st["dout"].float()[:, None, :]).sum(-1)]


def _plain_swiglu(st):
    c = st["case"]
    I = c["I"]
    if not c["grad"]:
        h = st["h"].float()
        g, u = h[:, :I], h[:, I:]
        out = [*_quant_rows(g * torch.sigmoid(g) * u)]
        return out + [*_quant_rows(h)] if c["keep"] else out
    h = st["hq"].view(F8).float().view(-1, 2 * I // G, G) * st["hs"].t()[:, :, None]
    h = h.view(-1, 2 * I)
    g, u, da = h[:, :I], h[:, I:], st["da"].float()
    r = torch.sigmoid(g)
    a = g * r
    dh = torch.cat([da * u * (r + a * (1.0 - r)), da * a], 1)
    return [*_quant_rows(dh), *_quant_cols(dh, st["offsets"], st["cap"]),
            *_quant_cols(a * u, st["offsets"], st["cap"])]


# ---------------------------------------------------------------------------------------------- #
# The same in 64 bits.  A code stands here for the value that was to be rounded to it.
# ---------------------------------------------------------------------------------------------- #

def _exact_rows(v):
    M, C = v.shape
    s = v.abs().reshape(M, -1, G).amax(2).clamp(min=FLOOR) / TOP
    return v / s.repeat_interleave(G, 1), s.T.contiguous()


def _exact_cols(v, offsets, cap):
    """Expert by expert, as the definition has it."""
    M, C = v.shape
    bounds = [0, M] if offsets is None else offsets.tolist()
    q, s, at = v.new_zeros(C, cap), v.new_zeros(cap // G, C), 0
    for lo, hi in zip(bounds[:-1], bounds[1:]):
        n = -(-(hi - lo) // G)
        if n:
            rows = torch.cat([v[lo:hi], v.new_zeros(n * G - (hi - lo), C)])
            s[at : at + n] = rows.abs().reshape(n, G, C).amax(1).clamp(min=FLOOR) / TOP
            q[:, G * at : G * (at + n)] = (rows / s[at : at + n].repeat_interleave(G, 0)).T
            at += n
    return q, s


def exact(case, seed):
    st = prepare(case, seed)
    c, op = case, case["op"]
    if op == "route":
        l = st["logits"].double()
        bias = torch.zeros(c["E"], device="cuda", dtype=torch.float64) if st["bias"] is None else st["bias"].double()
        p = 1.0 / (1.0 + torch.exp(-l)) if c["score"] == "sigmoid" else torch.softmax(l, -1)
        key = (l if st["bias"] is None else p + bias).masked_fill(l == -math.inf, -1e300)
        n = c["E"] // c["groups"]
        by = key.unflatten(1, (c["groups"], n)).sort(dim=-1, descending=True).values
        two = by[..., 0] if st["bias"] is None or n == 1 else by[..., 0] + by[..., 1].clamp(min=-1e150) * (by[..., 1] > -1e300)
        rank = torch.argsort(torch.argsort(two, dim=1, descending=True, stable=True), dim=1, stable=True)
        key = key.masked_fill((rank >= c["keep"]).repeat_interleave(n, 1), -math.inf)
        idx = torch.argsort(key, dim=1, descending=True, stable=True)[:, : c["k"]]
        chosen = torch.zeros_like(l, dtype=torch.bool).scatter_(1, idx, True)
        total = (p * chosen).sum(1, keepdim=True) if c["renorm"] else torch.ones_like(l[:, :1])
        w = c["scale"] * (p / total).gather(1, idx)
        if not c["grad"]:
            return [None, w]
        # d(loss)/d(score), over all experts, then through the scores' own derivative.
        up = c["scale"] * torch.zeros_like(l).scatter_(1, idx, st["dw"].double()) / total
        if c["renorm"]:
            near = idx[:, :, None] == idx[:, None, :]
            dw, r = st["dw"].double(), (p / total).gather(1, idx)
            off = ((dw[:, :, None] - dw[:, None, :]) * r[:, None, :]).masked_fill(near, 0.0).sum(2)
            up = torch.zeros_like(l).scatter_(1, idx, c["scale"] * off) / total
        return [None, w, up * p * (1.0 - p) if c["score"] == "sigmoid" else p * (up - (up * p).sum(1, keepdim=True))]
    if op == "swiglu":
        I = c["I"]
        if not c["grad"]:
            h = st["h"].double()
            a = h[:, :I] / (1.0 + torch.exp(-h[:, :I])) * h[:, I:]
            return [*_exact_rows(a), *(_exact_rows(h) if c["keep"] else ())]
        h = st["hq"].view(F8).double() * st["hs"].double().T.repeat_interleave(G, 1)
        gate, up, da = h[:, :I], h[:, I:], st["da"].double()
        z = 1.0 + torch.exp(-gate)
        dh = torch.empty_like(h)
        dh[:, :I] = da * up / z * (1.0 + gate * (z - 1.0) / z)
        dh[:, I:] = da * gate / z
        return [*_exact_rows(dh), *_exact_cols(dh, st["offsets"], st["cap"]),
                *_exact_cols(gate * up / z, st["offsets"], st["cap"])]
    k = c["k"]
    if op == "dispatch":
        e = st["idx"].flatten()
        order = torch.argsort(e, stable=True)
        v = st["x"].double()[order // k]
        if not c["both"]:
            return [None, None, None, *_exact_rows(v)]
        offsets = torch.cat([e.new_zeros(1), torch.bincount(e, minlength=st["E"]).cumsum(0).to(e.dtype)])
        return [None, None, None, *_exact_rows(v), *_exact_cols(v, offsets, st["cap"])]
    w = torch.ones_like(st["back"], dtype=torch.float64) if st["w"] is None else st["w"].double()
    if not c["grad"]:
        out = torch.zeros(c["T"], c["C"], device="cuda", dtype=torch.float64)
        if st["add"] is not None:
            out += st["add"].double()
        for j in range(k):
            out += w[:, j : j + 1] * st["y"][st["back"][:, j].long()].double()
        return out
    token = (st["slots"] // k).long()
    dout = st["dout"].double()
    v = dout[token] * w.flatten()[st["slots"].long()][:, None]
    out = [*_exact_rows(v), *_exact_cols(v, st["offsets"], st["cap"])]
    del v
    if not c["weighted"]:
        return out
    dw = torch.stack([(st["y"][st["back"][:, j].long()].double() * dout).sum(1) for j in range(k)], 1)
    return out + [dw]
