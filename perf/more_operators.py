"""Performance cases of the linear layer in 8-bit integers (scales per token and
per channel: forward, gradient, the products of a MoE layer's experts) and of the
router with sigmoid or softmax scores, a selection bias and groups of experts,
forward and backward.

own == False: the plain form in elementary torch operations, fp32 inside (the
codes' quotients and the router's selection values in 64 bits: both stand next
to borders), rounded once at the end.  own == True: the library's entry points.

Definitions:
  codes      S = fp32(max|v| / 127) of a row (or column), q = the integer nearest
             to v / S (ties to even); S = 0 and q = 0 where all values are 0
  linear     y[t, o] = sx[t] sw[o] sum_i qx[t, i] qw[o, i]: x bf16 with codes per
             token, weights as codes and scales per output channel
  linear_grad  dx = dy w and dw = dy^T x in the same arithmetic: dy's codes per
             token and w's per input channel; dy's per output channel and x's per
             input channel, both over the tokens
  grouped    c[r, n] = s[t] sw[g, n] sum_k q[t, k] qw[g, n, k] for row r of
             expert g, t = row_token[r]
  route      s = sigmoid(z) or softmax(z), v = s + bias; a group's value is its
             largest v or the sum of its two largest; the best `keep` groups stay
             (ties: lower group), of their experts the k largest v are taken
             (ties: lower expert); w_j = scale s_j / (sum of the taken s + 1e-20),
             or scale s_j; counts, offsets and rows of the stable (expert, token)
             order; balance = E sum_e f_e P_e with f_e = counts_e / sum(counts)
             and P_e the mean over tokens of p_e = s_e / (sum_e s_e + 1e-20);
             z = mean(lse^2) with softmax scores, 0 with sigmoid ones; total is
             lse, or sum_e s_e, and -inf for a token that is not routed.  Masked
             tokens and experts whose logit is -inf are not assigned.
  route_grad the gradient of the weights and of both losses at the logits
"""
import math

import torch

own = False

EPS = 1e-20


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one new token of one sequence (rollout decode) through the up projection
        {"name": "linear 1x2560 to 9728 decode", "op": "linear", "rows": 1, "cols": 2560, "out": 9728},
        # a decode batch of 64 sequences through the down projection
        {"name": "linear 64x9728 to 2560 decode", "op": "linear", "rows": 64, "cols": 9728, "out": 2560},
        # the same layer over a prompt or a training batch of 4096 tokens
        {"name": "linear 4096x2560 to 9728", "op": "linear", "rows": 4096, "cols": 2560, "out": 9728},
        # a ragged batch through a layer whose widths fill no whole tile
        {"name": "linear 333x1000 to 1512 ragged", "op": "linear", "rows": 333, "cols": 1000, "out": 1512},
        # the up projection's backward pass at 4096 tokens
        {"name": "linear_grad 4096x2560 to 9728", "op": "linear_grad", "rows": 4096, "cols": 2560, "out": 9728},
        # a short odd batch's backward pass
        {"name": "linear_grad 205x1000 to 1512", "op": "linear_grad", "rows": 205, "cols": 1000, "out": 1512},
        # a decode batch of 32 tokens through 128 experts' gate and up projections
        {"name": "grouped 256 rows of 128 experts", "op": "grouped", "tokens": 32, "experts": 128, "top_k": 8,
         "cols": 2048, "out": 1536, "pad": 0},
        # the same layer at 16384 tokens, 131072 expert rows
        {"name": "grouped 131072 rows", "op": "grouped", "tokens": 16384, "experts": 128, "top_k": 8, "cols": 2048,
         "out": 1536, "pad": 0},
        # routing of a decode batch: sigmoid scores, a bias, half of eight groups
        {"name": "route 32x128 top8 decode", "op": "route", "tokens": 32, "experts": 128, "top_k": 8, "groups": 8,
         "keep": 4, "score": "sigmoid", "group_score": "top2", "bias": True, "logits32": True, "renorm": True,
         "scale": 2.5, "pad": 0, "disabled": 0},
        # routing of a training batch over 256 experts
        {"name": "route 16384x256 top8", "op": "route", "tokens": 16384, "experts": 256, "top_k": 8, "groups": 8,
         "keep": 4, "score": "sigmoid", "group_score": "top2", "bias": True, "logits32": True, "renorm": True,
         "scale": 2.5, "pad": 0, "disabled": 0},
        # its gradient
        {"name": "route_grad 16384x256 top8", "op": "route_grad", "tokens": 16384, "experts": 256, "top_k": 8,
         "groups": 8, "keep": 4, "score": "sigmoid", "group_score": "top2", "bias": True, "logits32": True,
         "renorm": True, "scale": 2.5, "pad": 0, "disabled": 0},
        # a padded bf16 batch over an odd number of experts in groups, four of them
        # disabled, softmax scores and the groups' largest value
        {"name": "route_grad 1000x60 top4 padded", "op": "route_grad", "tokens": 1000, "experts": 60, "top_k": 4,
         "groups": 4, "keep": 2, "score": "softmax", "group_score": "max", "bias": False, "logits32": False,
         "renorm": False, "scale": 1.0, "pad": 77, "disabled": 4},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear_grad", "grouped", "route", "route_grad"])
    if op in ("linear", "linear_grad"):
        cols, out = 8 * _spread(rng, 16, 1216), 8 * _spread(rng, 16, 1216)
        rows = _spread(rng, 1, min(4096, 4096 * 2560 * 9728 // (cols * out)))
        return {"op": op, "rows": rows, "cols": cols, "out": out}
    if op == "grouped":
        experts, top_k = _spread(rng, 4, 128), rng.randint(1, 4)
        cols, out = 16 * _spread(rng, 8, 128), 8 * _spread(rng, 16, 192)
        tokens = _spread(rng, 1, 16384)
        return {"op": op, "tokens": tokens, "experts": experts, "top_k": top_k, "cols": cols, "out": out,
                "pad": rng.choice([0, rng.randint(0, tokens // 4)])}
    groups = rng.choice([1, 2, 4, 4, 8, 8, 6, 16])
    per = _spread(rng, 4, min(64, 512 // groups))
    keep = rng.randint((groups + 1) // 2, groups)
    experts = groups * per
    tokens = _spread(rng, 1, min(16384, 16384 * 256 // experts))
    return {"op": op, "tokens": tokens, "experts": experts, "top_k": rng.randint(1, min(8, keep * per)),
            "groups": groups, "keep": keep, "score": "sigmoid" if groups == 1 else rng.choice(["sigmoid", "softmax"]),
            "group_score": rng.choice(["top2", "max"]), "bias": rng.random() < 0.7, "logits32": rng.random() < 0.6,
            "renorm": rng.random() < 0.6, "scale": rng.choice([1.0, 2.5, round(rng.uniform(0.5, 3.0), 3)]),
            "pad": rng.randint(0, tokens // 4), "disabled": rng.choice([0, rng.randint(0, per // 4)])}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(1000033 * (int(seed) + 1))


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _acts(g, rows, cols, outliers=20.0):
    """Activations: N(0, 1) with 0.1% of the values larger by `outliers`."""
    v = _normal(g, rows, cols)
    v[torch.rand((rows, cols), generator=g, device="cuda") < 1e-3] *= outliers
    return v.to(torch.bfloat16)


def _weight_codes(g, *shape):
    """Codes [..., padded columns] and scales of normal weights: what a serving
    program keeps.  Codes are padded with zeros to a multiple of 16 columns."""
    w = 0.02 * _normal(g, *shape)
    s = w.abs().amax(dim=-1) / torch.full((), 127.0, device="cuda")
    q = torch.zeros(shape[:-1] + (-(-shape[-1] // 16) * 16,), dtype=torch.int8, device="cuda")
    q[..., :shape[-1]] = torch.round(w / s[..., None]).clamp(-127, 127).to(torch.int8)
    return q, s


def _rows_of(experts, E):
    """offsets [E + 1], row_token [T k], token_rows and counts of experts [T, k]
    (-1: none) in the stable (expert, token) order."""
    T, k = experts.shape
    flat = experts.reshape(-1).long()
    key = torch.where(flat >= 0, flat, torch.full_like(flat, E))
    order = key.sort(stable=True).indices
    counts = (key[:, None] == torch.arange(E, device=key.device)[None, :]).sum(dim=0)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=key.device)
    offsets[1:] = counts.cumsum(0)
    place = torch.empty_like(order)
    place[order] = torch.arange(T * k, device=key.device)
    token_rows = torch.where(flat >= 0, place, torch.full_like(place, -1))
    row_token = torch.where(key[order] < E, order // k, torch.zeros_like(order))
    i32 = lambda t: t.to(torch.int32)
    return i32(offsets), i32(row_token), i32(token_rows).view(T, k), i32(counts)


def _route_inputs(c, g):
    T, E = c["tokens"], c["experts"]
    popular = 0.7 * _normal(g, E)            # an unbalanced router, and a bias that has begun to balance it
    z = _normal(g, T, E) + popular
    bias = None
    if c["bias"]:
        bias = (-0.08 * popular + 0.02 * _normal(g, E)) * (1.0 if c["score"] == "sigmoid" else 8.0 / E)
    if c["disabled"]:
        z[:, torch.randperm(E, generator=g, device="cuda")[:c["disabled"]]] = -math.inf
    mask = None
    if c["pad"]:
        mask = torch.ones(T, dtype=torch.bool, device="cuda")
        mask[T - c["pad"]:] = False
        z[T - c["pad"]:] = math.nan          # whatever the padding holds is not read
    return {"logits": z.to(torch.float32 if c["logits32"] else torch.bfloat16), "mask": mask, "bias": bias}


def prepare(case, seed):
    c, g = case, _gen(seed)
    op = c["op"]
    if op == "linear":
        st = {"x": _acts(g, c["rows"], c["cols"])}
        st["qw"], st["sw"] = _weight_codes(g, c["out"], c["cols"])
    elif op == "linear_grad":
        st = {"x": _acts(g, c["rows"], c["cols"]), "w": (0.02 * _normal(g, c["out"], c["cols"])).to(torch.bfloat16),
              "dy": (1e-2 * _normal(g, c["rows"], c["out"])).to(torch.bfloat16)}
    elif op == "grouped":
        T, E, k = c["tokens"], c["experts"], c["top_k"]
        z = _normal(g, T, E) + 0.5 * _normal(g, E)
        experts = z.sort(dim=1, descending=True, stable=True).indices[:, :k]
        experts[T - c["pad"]:] = -1
        st = {}
        st["offsets"], st["row_token"], _, counts = _rows_of(experts, E)
        st["q"], st["s"] = _codes(_acts(g, T, c["cols"]), 1)
        st["qw"], st["sw"] = _weight_codes(g, E, c["out"], c["cols"])
        st["most"] = int(counts.max())       # rows of the largest expert: the plain form's batch size
    else:
        st = _route_inputs(c, g)
        if op == "route_grad":
            saved = _plain_route(c, st)      # what the forward pass saved
            st.update({n: saved[n] for n in ("experts", "counts", "total")})
            st["dweights"] = _normal(g, c["tokens"], c["top_k"])
            st["dloss"] = torch.tensor([1e-2, 1e-3], device="cuda")
    st["case"] = c
    return st


# ------------------------------------------------------------- plain forms
def _codes(x, dim):
    """int8 codes and fp32 scales of the rows (dim 1) or columns (dim 0) of x."""
    s = x.float().abs().amax(dim=dim, keepdim=True) / torch.full((), 127.0, device=x.device)
    q = torch.round(x.double() / torch.where(s > 0, s, torch.ones_like(s)).double())
    return q.clamp(-127, 127).to(torch.int8), s.view(-1)


def _plain_linear(c, st):
    q, s = _codes(st["x"], 1)
    acc = q.float() @ st["qw"][:, :c["cols"]].float().t().contiguous()
    return (acc * s[:, None] * st["sw"][None, :]).to(torch.bfloat16)


def _plain_linear_grad(c, st):
    (qdy, sdy), (qw, sw) = _codes(st["dy"], 1), _codes(st["w"], 0)
    (qdyt, sdyt), (qx, sx) = _codes(st["dy"], 0), _codes(st["x"], 0)
    dx = (qdy.float() @ qw.float()) * sdy[:, None] * sw[None, :]
    dw = (qdyt.float().t().contiguous() @ qx.float()) * sdyt[:, None] * sx[None, :]
    return {"dx": dx, "dw": dw}


def _plain_grouped(c, st):
    E, cols = c["experts"], c["cols"]
    live = (c["tokens"] - c["pad"]) * c["top_k"]
    if live == 0:
        return torch.zeros((0, c["out"]), dtype=torch.bfloat16, device="cuda")
    row = torch.arange(live, device="cuda")
    expert = torch.searchsorted(st["offsets"][1:].long(), row, right=True)
    slot = row - st["offsets"].long()[expert]
    token = st["row_token"][:live].long()
    a = torch.zeros((E, st["most"], cols), dtype=torch.float32, device="cuda")
    a[expert, slot] = st["q"][token].float()
    acc = torch.bmm(a, st["qw"].float().transpose(1, 2).contiguous())[expert, slot]
    return (acc * st["s"][token][:, None] * st["sw"][expert]).to(torch.bfloat16)


def _scores(c, z):
    """Scores and total of logits without masked tokens (all -inf: 0 and -inf)."""
    some = (z > -math.inf).any(dim=1, keepdim=True)
    if c["score"] == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-z))
        return s, torch.where(some[:, 0], s.sum(dim=1), torch.full_like(s[:, 0], -math.inf))
    m = torch.where(some, z.amax(dim=1, keepdim=True), torch.zeros_like(z[:, :1]))
    e = torch.exp(z - m)
    full = e.sum(dim=1, keepdim=True)
    return torch.where(some, e / full, torch.zeros_like(e)), (m + torch.log(full))[:, 0]


def _live_logits(st):
    z = st["logits"].float()
    return z if st["mask"] is None else torch.where(st["mask"][:, None], z, torch.full_like(z, -math.inf))


def _plain_route(c, st):
    E, k, G = c["experts"], c["top_k"], c["groups"]
    z = _live_logits(st)
    T = z.shape[0]
    # the selection in 64 bits: two experts' values may be nearer than an fp32 step
    v = _scores(c, z.double())[0]
    if st["bias"] is not None:
        v = v + st["bias"].double()
    v = torch.where(z > -math.inf, v, torch.full_like(v, -math.inf))
    by_group = v.view(T, G, E // G).sort(dim=2, descending=True).values
    value = by_group[:, :, 0]
    if c["group_score"] == "top2":
        value = value + torch.where(by_group[:, :, 1] > -math.inf, by_group[:, :, 1], torch.zeros_like(value))
    order = value.sort(dim=1, descending=True, stable=True).indices[:, :c["keep"]]
    kept = torch.zeros((T, G), dtype=torch.bool, device=z.device).scatter_(1, order, True)
    v = torch.where(kept.repeat_interleave(E // G, dim=1), v, torch.full_like(v, -math.inf))
    top, idx = v.sort(dim=1, descending=True, stable=True)
    used, idx = top[:, :k] > -math.inf, idx[:, :k]
    s, total = _scores(c, z)
    taken = torch.where(used, s.gather(1, idx), torch.zeros_like(s[:, :k]))
    weights = c["scale"] * (taken / (taken.sum(dim=1, keepdim=True) + EPS) if c["renorm"] else taken)
    experts = torch.where(used, idx, torch.full_like(idx, -1)).to(torch.int32)
    offsets, row_token, token_rows, counts = _rows_of(experts, E)
    live = total > -math.inf
    p = s if c["score"] == "softmax" else s / (s.sum(dim=1, keepdim=True) + EPS)
    n = live.sum()
    some = n.clamp(min=1).float()
    f = counts.float() / counts.sum().clamp(min=1).float()
    balance = E * (f * (torch.where(live[:, None], p, torch.zeros_like(p)).sum(dim=0) / some)).sum()
    zloss = torch.zeros_like(balance)
    if c["score"] == "softmax":
        zloss = torch.where(live, total * total, torch.zeros_like(total)).sum() / some
    return {"experts": experts, "weights": weights, "counts": torch.cat([counts, n.view(1).to(torch.int32)]),
            "offsets": offsets, "row_token": row_token, "token_rows": token_rows, "total": total,
            "loss": torch.stack([balance, zloss])}


def _plain_route_grad(c, st):
    E = c["experts"]
    live = st["total"] > -math.inf
    z = torch.where(live[:, None], st["logits"].float(), torch.full_like(st["logits"].float(), -math.inf))
    s, _ = _scores(c, z)
    used = st["experts"] >= 0
    at = st["experts"].long().clamp(min=0)
    taken = torch.where(used, s.gather(1, at), torch.zeros_like(s[:, :c["top_k"]]))
    dw = c["scale"] * torch.where(used, st["dweights"], torch.zeros_like(taken))
    if c["renorm"]:
        norm = taken.sum(dim=1, keepdim=True) + EPS
        dw = (dw - (taken / norm * dw).sum(dim=1, keepdim=True)) / norm
    ds = torch.zeros((z.shape[0], E + 1), dtype=torch.float32, device=z.device)
    ds.scatter_(1, torch.where(used, at, torch.full_like(at, E)), dw)
    ds = ds[:, :E]
    n = st["counts"][E].clamp(min=1).float()
    f = st["counts"][:E].float() / st["counts"][:E].sum().clamp(min=1).float()
    g = st["dloss"]
    if c["score"] == "sigmoid":
        norm = s.sum(dim=1, keepdim=True) + EPS
        ds = ds + g[0] * E / n * (f - (s / norm * f).sum(dim=1, keepdim=True)) / norm
        d = ds * s * (1.0 - s)
    else:
        ds = ds + g[0] * E / n * f
        total = torch.where(live, st["total"], torch.zeros_like(st["total"]))
        d = s * (ds - (s * ds).sum(dim=1, keepdim=True) + (2.0 * g[1] / n * total)[:, None])
    return torch.where(live[:, None], d, torch.zeros_like(d)).to(st["logits"].dtype)


# -------------------------------------------------------------------- run
def _route_options(c, st):
    return {"score": c["score"], "bias": st["bias"], "groups": c["groups"], "keep_groups": c["keep"],
            "group_score": c["group_score"], "renorm": c["renorm"], "scale": c["scale"]}


def _own(c, st):
    from fp8_block_scaled_x128_amd import ops
    op, out = c["op"], st.get("out")
    if op == "linear":
        st["out"] = ops.i8_linear(st["x"], st["qw"], st["sw"], out=out)
        return st["out"].y
    if op == "linear_grad":
        st["out"] = ops.i8_linear_backward(st["dy"], (st["w"], st["x"]), out=out)
        return {"dx": st["out"].dx, "dw": st["out"].dw}
    if op == "grouped":
        st["out"] = ops.i8_grouped_gemm(st["q"], st["s"], st["qw"], st["sw"], st["offsets"], st["row_token"], out=out)
        # rows behind the last assignment are not written
        return st["out"][:(c["tokens"] - c["pad"]) * c["top_k"]]
    if op == "route":
        r = ops.moe_route_grouped(st["logits"], c["top_k"], mask=st["mask"], out=out, **_route_options(c, st))
        st["out"] = r
        return {"experts": r.experts, "weights": r.weights, "counts": r.counts, "offsets": r.offsets,
                "row_token": r.row_token, "token_rows": r.token_rows, "total": r.lse, "loss": r.loss}
    st["out"] = ops.moe_route_grouped_backward(st["logits"], st["experts"], st["counts"], st["total"],
                                               dweights=st["dweights"], dloss=st["dloss"], score=c["score"],
                                               renorm=c["renorm"], scale=c["scale"], out=out)
    return st["out"]


_PLAIN = {"linear": _plain_linear, "linear_grad": _plain_linear_grad, "grouped": _plain_grouped,
          "route": _plain_route, "route_grad": _plain_route_grad}


def run(state):
    c = state["case"]
    return _own(c, state) if own else _PLAIN[c["op"]](c, state)


# ------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] in ("linear", "linear_grad"):
        T, K, N = c["rows"], c["cols"], c["out"]
        if c["op"] == "linear":
            return {"bytes": 2 * T * K + N * K + 4 * N + 2 * T * N, "flops": 2 * T * K * N}
        return {"bytes": 2 * (T * N + T * K + N * K) + 4 * (T * K + N * K), "flops": 4 * T * K * N}
    T, k, E = c["tokens"], c["top_k"], c["experts"]
    live = T - c["pad"]
    if c["op"] == "grouped":
        K, N, rows = c["cols"], c["out"], live * k
        used = E * (1.0 - (1.0 - 1.0 / E) ** rows)          # experts with rows, were all as popular
        return {"bytes": int(live * (K + 4) + used * N * (K + 4) + rows * (2 * N + 4)), "flops": 2 * rows * K * N}
    z = 4 if c["logits32"] else 2
    if c["op"] == "route":
        return {"bytes": live * E * z + T * (16 * k + 4) + 8 * E + 8 + 4 * E * c["bias"] + T * bool(c["pad"]),
                "flops": live * E * (6 + k)}
    return {"bytes": live * E * z + T * E * z + T * (8 * k + 4) + 4 * E, "flops": live * E * 12}


# ------------------------------------------------- the definitions, 64 bits
def _exact_codes(v):
    """(codes, scales) of the rows of v as 64-bit numbers; scales are fp32 values."""
    v = v.to(torch.float64)
    s = (v.abs().max(dim=1).values / 127.0).to(torch.float32).to(torch.float64)
    low = torch.floor(v / s.clamp(min=1e-300)[:, None])
    rest = v - low * s[:, None]              # exact: both terms have few bits
    half = 0.5 * s[:, None]
    up = (rest > half) | ((rest == half) & (torch.remainder(low, 2.0) == 1.0))
    return (low + up.to(torch.float64)) * (s > 0)[:, None], s


def _exact_product(a, b):
    (qa, sa), (qb, sb) = a, b
    return torch.outer(sa, sb) * (qa @ qb.t().contiguous())


def _exact_route_parts(c, st):
    """Logits in 64 bits, which tokens are routed, scores, normalised scores and
    the total, through torch's own sigmoid and softmax."""
    z = st["logits"].to(torch.float64)
    if st["mask"] is not None:
        z = z.masked_fill(~st["mask"][:, None], -math.inf)
    live = z.amax(dim=1) > -math.inf
    safe = z.masked_fill(~live[:, None], 0.0)
    if c["score"] == "sigmoid":
        s = torch.sigmoid(safe) * live[:, None]
        total = s.sum(dim=1)
        return z, live, s, s / (total[:, None] + EPS), total.masked_fill(~live, -math.inf)
    s = torch.softmax(safe, dim=1) * live[:, None]
    return z, live, s, s, torch.logsumexp(safe, dim=1).masked_fill(~live, -math.inf)


def _exact_route(c, st):
    z, live, s, p, total = _exact_route_parts(c, st)
    E, k, G = c["experts"], c["top_k"], c["groups"]
    v = s if st["bias"] is None else s + st["bias"].to(torch.float64)
    v = v.masked_fill(z == -math.inf, -math.inf)
    best = v.view(-1, G, E // G).topk(min(2, E // G), dim=2).values
    value = best[..., 0] if c["group_score"] == "max" else best.masked_fill(
        (best == -math.inf) & (best[..., :1] > -math.inf), 0.0).sum(dim=2)
    cut = value.sort(dim=1, descending=True, stable=True).indices[:, c["keep"]:]
    v = v.view(-1, G, E // G).scatter(1, cut[..., None].expand(-1, -1, E // G), -math.inf).view(-1, E)
    chosen = v.sort(dim=1, descending=True, stable=True)
    hit = chosen.values[:, :k] > -math.inf
    w = s.gather(1, chosen.indices[:, :k]) * hit
    if c["renorm"]:
        w = w / (w.sum(dim=1, keepdim=True) + EPS)
    hits = torch.zeros_like(s).scatter_(1, chosen.indices[:, :k], hit.double())
    f = hits.sum(dim=0) / hits.sum().clamp(min=1.0)
    n = live.sum().clamp(min=1).double()
    zl = total[live].square().sum() / n if c["score"] == "softmax" else torch.zeros((), device="cuda").double()
    return {"experts": None, "weights": c["scale"] * w, "counts": None, "offsets": None, "row_token": None,
            "token_rows": None, "total": total, "loss": torch.stack([E * torch.dot(f, p.sum(dim=0) / n), zl])}


def _exact_route_grad(c, st):
    """Through autograd in 64 bits: the scalar sum(w dweights) + dloss . loss."""
    E = c["experts"]
    live = st["total"] > -math.inf
    z = st["logits"].to(torch.float64).masked_fill(~live[:, None], 0.0).requires_grad_(True)
    s = (torch.sigmoid(z) if c["score"] == "sigmoid" else torch.softmax(z, dim=1)) * live[:, None]
    p = s / (s.sum(dim=1, keepdim=True) + EPS) if c["score"] == "sigmoid" else s
    w = s.gather(1, st["experts"].long().clamp(min=0)) * (st["experts"] >= 0)
    if c["renorm"]:
        w = w / (w.sum(dim=1, keepdim=True) + EPS)
    counts, g = st["counts"].to(torch.float64), st["dloss"].to(torch.float64)
    n = counts[E].clamp(min=1.0)
    f = counts[:E] / counts[:E].sum().clamp(min=1.0)
    total = c["scale"] * (w * st["dweights"].to(torch.float64)).sum() + g[0] * E * torch.dot(f, p.sum(dim=0)) / n
    if c["score"] == "softmax":
        total = total + g[1] * torch.logsumexp(z, dim=1)[live].square().sum() / n
    d, = torch.autograd.grad(total, (z,))
    return d * live[:, None]


def exact(case, seed):
    c = case
    st = prepare(c, seed)
    if c["op"] == "linear":
        return _exact_product(_exact_codes(st["x"]), (st["qw"][:, :c["cols"]].double(), st["sw"].double()))
    if c["op"] == "linear_grad":
        across = lambda t: _exact_codes(t.t().contiguous())
        return {"dx": _exact_product(_exact_codes(st["dy"]), across(st["w"])),
                "dw": _exact_product(across(st["dy"]), across(st["x"]))}
    if c["op"] == "grouped":
        ends = st["offsets"].tolist()
        out = torch.zeros((ends[-1], c["out"]), dtype=torch.float64, device="cuda")
        for e in range(c["experts"]):
            at = st["row_token"][ends[e]:ends[e + 1]].long()
            if at.numel():
                out[ends[e]:ends[e + 1]] = _exact_product((st["q"][at].double(), st["s"][at].double()),
                                                          (st["qw"][e].double(), st["sw"][e].double()))
        return out
    return (_exact_route if c["op"] == "route" else _exact_route_grad)(c, st)
