"""The operators between the FP8 GEMMs of a transformer block, forward and
backward, as performance cases: the norms before and after a block fused with
its gate, residual scale and 1x128 quantization; top-k routing with per-expert
counts, expert-sorted rows and the balance loss; the gradients of both; the
gradient of the MoE combine.

own == False: the plain form in elementary torch operations, fp32 inside,
rounded once at the end.  own == True: the library's entry points.

Definitions (v * rsqrt(mean(v^2) + eps) * w is N(v; w)):
  norm       h = residual + scale * gate * N(x; w_post);  y = N(h; w_pre);
             1x128 groups of the fp32 y: S = max|y| / 448, codes E4M3(y / S)
  norm_grad  the gradients of h and y with respect to x, residual, gate,
             w_post and w_pre, at the saved h and x
  route      the k largest logits of each token (ties: lower expert), their
             softmax weights, counts, and the stable (expert, token) order;
             balance = E sum_e f_e P_e with f_e = counts_e / sum(counts) and
             P_e the mean probability; z = mean(lse^2).  Masked tokens and
             experts whose logit is -inf are not assigned (-1, weight 0).
  route_grad the gradient of the weights and of both losses at the logits
  combine_grad  out[t] = sum_j w_tj y[row_tj]: dy[row_tj] = w_tj dout[t] and
             dw_tj = <dout[t], y[row_tj]>
"""
import math

import torch

own = False

EPS = 1e-6
GROUP = 128


# ------------------------------------------------------------------- cases
def listed():
    return [
        # one new token of one sequence (rollout decode), hidden 2560: the
        # block's output norm, the residual add and the next block's input norm
        {"name": "norm 1x2560 decode", "op": "norm", "kind": "both", "rows": 1, "cols": 2560, "res32": False,
         "w32": False, "gate_rows": 0, "scale": 1.0, "quant": True, "y": False},
        # the trainer's block boundary at 4096 tokens: bf16 y is kept for wgrad
        {"name": "norm 4096x2560 train", "op": "norm", "kind": "both", "rows": 4096, "cols": 2560, "res32": False,
         "w32": False, "gate_rows": 0, "scale": 1.0, "quant": True, "y": True},
        # fp32 residual stream, a gate per sequence and channel, depth-scaled residual
        {"name": "norm 16384x2048 gated fp32", "op": "norm", "kind": "both", "rows": 16384, "cols": 2048,
         "res32": True, "w32": True, "gate_rows": 2048, "scale": 0.35, "quant": True, "y": True},
        # backward of the trainer's block boundary
        {"name": "norm_grad 4096x2560", "op": "norm_grad", "kind": "both", "rows": 4096, "cols": 2560,
         "res32": False, "w32": False, "gate_rows": 0, "scale": 1.0, "dy32": True},
        # the same over an fp32 stream with the per-sequence gate's gradient
        {"name": "norm_grad 16384x2048 gated fp32", "op": "norm_grad", "kind": "both", "rows": 16384, "cols": 2048,
         "res32": True, "w32": True, "gate_rows": 2048, "scale": 0.35, "dy32": False},
        # a short ragged batch, a width that fills no whole 128-group, a gate per token
        {"name": "norm_grad 333x1000 ragged", "op": "norm_grad", "kind": "both", "rows": 333, "cols": 1000,
         "res32": False, "w32": False, "gate_rows": 1, "scale": 0.5, "dy32": False},
        # a decode batch of 32 tokens over 128 experts
        {"name": "route 32x128 top8 decode", "op": "route", "tokens": 32, "experts": 128, "top_k": 8,
         "logits32": True, "renorm": True, "pad": 0, "disabled": 0},
        # a training batch over 128 experts with both losses
        {"name": "route 16384x128 top8", "op": "route", "tokens": 16384, "experts": 128, "top_k": 8,
         "logits32": True, "renorm": True, "pad": 0, "disabled": 0},
        # its gradient
        {"name": "route_grad 16384x128 top8", "op": "route_grad", "tokens": 16384, "experts": 128, "top_k": 8,
         "logits32": True, "renorm": True, "pad": 0, "disabled": 0},
        # a padded bf16 batch over an odd number of experts, four of them disabled
        {"name": "route_grad 1000x60 top4 padded", "op": "route_grad", "tokens": 1000, "experts": 60, "top_k": 4,
         "logits32": False, "renorm": False, "pad": 77, "disabled": 4},
        # the combine's gradient of a small padded batch
        {"name": "combine_grad 512x256 top2", "op": "combine_grad", "tokens": 512, "cols": 256, "experts": 8,
         "top_k": 2, "pad": 33, "dout32": False},
        # the combine's gradient at 16384 tokens, 131072 expert rows of 2048
        {"name": "combine_grad 16384x2048 top8", "op": "combine_grad", "tokens": 16384, "cols": 2048,
         "experts": 128, "top_k": 8, "pad": 0, "dout32": False},
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "route", "route_grad", "combine_grad"])
    if op in ("norm", "norm_grad"):
        cols = 8 * _spread(rng, 16, 1280)
        rows = _spread(rng, 1, min(16384, 16384 * 2048 // cols))
        c = {"op": op, "kind": rng.choice(["both", "both", "pre", "post"]), "rows": rows, "cols": cols,
             "res32": rng.random() < 0.4, "w32": rng.random() < 0.4,
             "gate_rows": rng.choice([0, 1, _spread(rng, 1, max(2, rows))]),
             "scale": rng.choice([1.0, 0.5, round(rng.uniform(0.1, 1.5), 3)])}
        if op == "norm":
            c["quant"] = rng.random() < 0.7
            c["y"] = not c["quant"] or rng.random() < 0.5
        else:
            c["dy32"] = rng.random() < 0.4
        return c
    experts = _spread(rng, 8, 512)
    top_k = rng.randint(1, min(8, experts))
    if op == "combine_grad":
        cols = 8 * _spread(rng, 16, 1024)
        tokens = _spread(rng, 1, min(16384, 16384 * 2048 * 8 // (cols * top_k)))
        return {"op": op, "tokens": tokens, "cols": cols, "experts": experts, "top_k": top_k,
                "pad": rng.randint(0, tokens // 4), "dout32": rng.random() < 0.4}
    tokens = _spread(rng, 1, 16384)
    return {"op": op, "tokens": tokens, "experts": experts, "top_k": top_k, "logits32": rng.random() < 0.6,
            "renorm": rng.random() < 0.6, "pad": rng.randint(0, tokens // 4),
            "disabled": rng.choice([0, rng.randint(0, experts // 4)])}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(1000003 * (int(seed) + 1))


def _normal(g, *shape):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)


def _acts(g, rows, cols, dtype, outliers=20.0):
    """Activations: N(0, 1) with 0.1% of the values larger by `outliers`."""
    v = _normal(g, rows, cols)
    v[torch.rand((rows, cols), generator=g, device="cuda") < 1e-3] *= outliers
    return v.to(dtype)


def _stream_type(c):
    return torch.float32 if c["res32"] else torch.bfloat16


def _norm_inputs(c, g):
    rows, cols = c["rows"], c["cols"]
    wt = torch.float32 if c["w32"] else torch.bfloat16
    st = {"x": None, "w_post": None, "gate": None, "w_pre": None, "rows_per_gate": max(1, c["gate_rows"])}
    if c["kind"] != "pre":
        st["x"] = _acts(g, rows, cols, torch.bfloat16)
        st["w_post"] = (1.0 + 0.2 * _normal(g, cols)).to(wt)
        if c["gate_rows"]:
            n = -(-rows // c["gate_rows"])
            st["gate"] = (0.5 + 0.3 * _normal(g, n, cols)).to(torch.bfloat16)
    if c["kind"] != "post":
        st["w_pre"] = (1.0 + 0.2 * _normal(g, cols)).to(wt)
    return st


def _route_inputs(c, g):
    T, E = c["tokens"], c["experts"]
    # an unbalanced router: experts differ in popularity
    z = _normal(g, T, E) + 0.7 * _normal(g, E)
    if c["disabled"]:
        z[:, torch.randperm(E, generator=g, device="cuda")[:c["disabled"]]] = -math.inf
    mask = None
    if c["pad"]:
        mask = torch.ones(T, dtype=torch.bool, device="cuda")
        mask[T - c["pad"]:] = False
        z[T - c["pad"]:] = math.nan          # whatever the padding holds is not read
    return z.to(torch.float32 if c["logits32"] else torch.bfloat16), mask


def prepare(case, seed):
    c, g = case, _gen(seed)
    op = c["op"]
    if op == "norm":
        st = _norm_inputs(c, g)
        st["residual"] = (3.0 * _acts(g, c["rows"], c["cols"], torch.float32)).to(_stream_type(c))
    elif op == "norm_grad":
        st = _norm_inputs(c, g)
        rows, cols = c["rows"], c["cols"]
        st["dh"] = (1e-2 * _normal(g, rows, cols)).to(_stream_type(c))
        st["h"] = st["dy"] = None
        if c["kind"] != "post":
            st["h"] = (3.0 * _acts(g, rows, cols, torch.float32)).to(_stream_type(c))
            st["dy"] = (1e-2 * _normal(g, rows, cols)).to(torch.float32 if c["dy32"] else torch.bfloat16)
    elif op == "route":
        z, mask = _route_inputs(c, g)
        st = {"logits": z, "mask": mask}
    elif op == "route_grad":
        z, mask = _route_inputs(c, g)
        st = {"logits": z, "mask": mask}
        st.update(_plain_route(c, st))       # what the forward pass saved
        st["dweights"] = _normal(g, c["tokens"], c["top_k"])
        st["dloss"] = torch.tensor([1e-2, 1e-3], device="cuda")
    else:
        T, k, E, H = c["tokens"], c["top_k"], c["experts"], c["cols"]
        live = T - c["pad"]
        z = _normal(g, T, E) + 0.7 * _normal(g, E)
        experts = z.sort(dim=1, descending=True, stable=True).indices[:, :k].to(torch.int32)
        experts[live:] = -1
        rows = T * k
        st = {"token_rows": _expert_order(experts, E)[3],
              "weights": torch.softmax(_normal(g, T, k), dim=1) * (experts >= 0)}
        st["y"] = _acts(g, rows, H, torch.bfloat16)
        st["dout"] = (1e-2 * _normal(g, T, H)).to(torch.float32 if c["dout32"] else torch.bfloat16)
    st["case"] = c
    return st


# ------------------------------------------------------------- plain forms
def _unit(v):
    """v * rsqrt(mean(v^2) + eps) by rows, and the factor."""
    r = torch.rsqrt((v * v).mean(dim=1, keepdim=True) + EPS)
    return v * r, r


def _gate_rows(st, rows):
    return st["gate"].float().repeat_interleave(st["rows_per_gate"], dim=0)[:rows]


def _plain_norm(c, st):
    rows, cols = c["rows"], c["cols"]
    h = st["residual"].float()
    if st["x"] is not None:
        n = _unit(st["x"].float())[0] * st["w_post"].float()
        if st["gate"] is not None:
            n = n * _gate_rows(st, rows)
        h = h + c["scale"] * n
    out = {}
    if st["x"] is not None:
        out["h"] = h.to(_stream_type(c))
    if st["w_pre"] is None:
        return out
    y = _unit(h)[0] * st["w_pre"].float()
    if c["y"]:
        out["y"] = y.to(torch.bfloat16)
    if c["quant"]:
        groups = -(-cols // GROUP)
        yg = torch.zeros((rows, groups * GROUP), dtype=torch.float32, device=y.device)
        yg[:, :cols] = y
        yg = yg.view(rows, groups, GROUP)
        s = yg.abs().amax(dim=2) / 448.0
        q = torch.where(s[:, :, None] > 0, yg / s[:, :, None], torch.zeros_like(yg)).clamp(-448.0, 448.0)
        out["q"] = q.view(rows, groups * GROUP)[:, :cols].to(torch.float8_e4m3fn)
        out["s"] = s
    return out


def _plain_norm_grad(c, st):
    rows, cols = c["rows"], c["cols"]
    out = {}
    dh = st["dh"].float()
    if st["w_pre"] is not None:
        hh, r = _unit(st["h"].float())
        dy = st["dy"].float()
        out["dw_pre"] = (dy * hh).sum(dim=0)
        g = dy * st["w_pre"].float()
        dh = dh + r * (g - hh * (g * hh).mean(dim=1, keepdim=True))
    if st["w_pre"] is not None:
        out["dres"] = dh.to(_stream_type(c))
    if st["x"] is not None:
        xh, r = _unit(st["x"].float())
        dn = c["scale"] * dh
        if st["gate"] is not None:
            R, n = st["rows_per_gate"], st["gate"].shape[0]
            dg = torch.zeros((n * R, cols), dtype=torch.float32, device=dh.device)
            dg[:rows] = dn * (xh * st["w_post"].float())
            dg = dg.view(n, R, cols).sum(dim=1)
            out["dgate"] = dg if R > 1 else dg.to(torch.bfloat16)
            dn = dn * _gate_rows(st, rows)
        out["dw_post"] = (dn * xh).sum(dim=0)
        g = dn * st["w_post"].float()
        out["dx"] = (r * (g - xh * (g * xh).mean(dim=1, keepdim=True))).to(torch.bfloat16)
    return out


def _expert_order(experts, E):
    """counts, offsets, row_token, token_rows of the stable (expert, token)
    order; unassigned slots (-1) have no row, and row_token is 0 behind the
    last row."""
    T, k = experts.shape
    flat = experts.reshape(-1).long()
    key = torch.where(flat >= 0, flat, torch.full_like(flat, E))
    # slots are in (token, slot) order and a token has an expert once: a
    # stable sort by expert is the (expert, token) order
    order = key.sort(stable=True).indices
    counts = (key[:, None] == torch.arange(E, device=key.device)[None, :]).sum(dim=0)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=key.device)
    offsets[1:] = counts.cumsum(0)
    place = torch.empty_like(order)
    place[order] = torch.arange(T * k, device=key.device)
    token_rows = torch.where(flat >= 0, place, torch.full_like(place, -1))
    row_token = torch.where(key[order] < E, order // k, torch.zeros_like(order))
    i32 = lambda t: t.to(torch.int32)
    return i32(counts), i32(offsets), i32(row_token), i32(token_rows).view(T, k)


def _plain_route(c, st):
    E, k = c["experts"], c["top_k"]
    z = st["logits"].float()
    live = torch.ones(z.shape[0], dtype=torch.bool, device=z.device) if st["mask"] is None else st["mask"]
    z = torch.where(live[:, None], z, torch.full_like(z, -math.inf))
    live = live & (z > -math.inf).any(dim=1)
    top, idx = z.sort(dim=1, descending=True, stable=True)
    top, idx = top[:, :k], idx[:, :k]
    m = torch.where(live, top[:, 0], torch.zeros_like(top[:, 0]))[:, None]
    full = torch.exp(z - m).sum(dim=1, keepdim=True)
    lse = (m + torch.log(full))[:, 0]                     # -inf where nothing is left
    e = torch.exp(top - m)
    norm = e.sum(dim=1, keepdim=True) if c["renorm"] else full
    used = top > -math.inf
    weights = torch.where(used, e / norm, torch.zeros_like(e))
    experts = torch.where(used, idx, torch.full_like(idx, -1)).to(torch.int32)
    counts, offsets, row_token, token_rows = _expert_order(experts, E)
    p = torch.where(live[:, None], torch.exp(z - m) / full, torch.zeros_like(z))
    n = live.sum()
    some = n.clamp(min=1).float()
    f = counts.float() / counts.sum().clamp(min=1).float()
    balance = E * (f * (p.sum(dim=0) / some)).sum()
    zloss = torch.where(live, lse * lse, torch.zeros_like(lse)).sum() / some
    return {"experts": experts, "weights": weights, "counts": torch.cat([counts, n.view(1).to(torch.int32)]),
            "offsets": offsets, "row_token": row_token, "token_rows": token_rows, "lse": lse,
            "loss": torch.stack([balance, zloss])}


def _plain_route_grad(c, st):
    E, k = c["experts"], c["top_k"]
    z = st["logits"].float()
    lse, w, dw, counts = st["lse"], st["weights"], st["dweights"], st["counts"]
    live = lse > -math.inf
    p = torch.where(live[:, None], torch.exp(z - torch.where(live, lse, torch.zeros_like(lse))[:, None]),
                    torch.zeros_like(z))
    n = counts[E].clamp(min=1).float()
    f = counts[:E].float() / counts[:E].sum().clamp(min=1).float()
    g = st["dloss"]
    d = p * (g[0] * E / n * (f - (p * f).sum(dim=1, keepdim=True)))
    d = d + p * (2.0 * g[1] / n * torch.where(live, lse, torch.zeros_like(lse)))[:, None]
    used = st["experts"] >= 0
    dot = (w * dw).sum(dim=1, keepdim=True)
    if c["renorm"]:
        part = torch.where(used, w * (dw - dot), torch.zeros_like(w))
    else:
        part = torch.where(used, w * dw, torch.zeros_like(w))
        d = d - p * dot
    wide = torch.zeros((z.shape[0], E + 1), dtype=torch.float32, device=z.device)
    wide.scatter_(1, torch.where(used, st["experts"].long(), torch.full_like(st["experts"].long(), E)), part)
    return (d + wide[:, :E]).to(st["logits"].dtype)


def _plain_combine_grad(c, st):
    T, k, H = c["tokens"], c["top_k"], c["cols"]
    pos, w = st["token_rows"].reshape(-1).long(), st["weights"]
    live = pos >= 0
    src, slot = pos[live], torch.nonzero(live)[:, 0]
    dout = st["dout"].float()
    dy = torch.zeros((T * k, H), dtype=torch.float32, device=dout.device)
    dy[src] = w.reshape(-1)[slot][:, None] * dout[slot // k]
    dw = torch.zeros(T * k, dtype=torch.float32, device=dout.device)
    dw[slot] = (st["y"][src].float() * dout[slot // k]).sum(dim=1)
    return {"dy": dy[:src.numel()].to(torch.bfloat16), "dweights": dw.view(T, k)}


# -------------------------------------------------------------------- run
def _own(c, st):
    from fp8_block_scaled_x128_amd import ops
    op, out = c["op"], st.get("out")
    if op == "norm":
        r = ops.block_norm(st["residual"], st["x"], w_pre=st["w_pre"], w_post=st["w_post"], gate=st["gate"],
                           rows_per_gate=st["rows_per_gate"], scale=c["scale"], eps=EPS, h=st["x"] is not None,
                           y=st["w_pre"] is not None and c["y"], quant=st["w_pre"] is not None and c["quant"],
                           out=out)
        st["out"] = r
        got = {"h": r.h, "y": r.y, "s": r.s}
        if r.q is not None:
            got["q"] = r.q.view(torch.float8_e4m3fn)
        return {k: v for k, v in got.items() if v is not None}
    if op == "norm_grad":
        r = ops.block_norm_backward(st["dy"], st["dh"], st["h"], st["x"], w_pre=st["w_pre"], w_post=st["w_post"],
                                    gate=st["gate"], rows_per_gate=st["rows_per_gate"], scale=c["scale"], eps=EPS,
                                    dres=st["w_pre"] is not None,
                                    dgate_dtype=torch.float32 if st["rows_per_gate"] > 1 else torch.bfloat16,
                                    out=out)
        st["out"] = r
        got = {"dres": r.dres, "dx": r.dx, "dgate": r.dgate, "dw_pre": r.dw_pre, "dw_post": r.dw_post}
        return {k: v for k, v in got.items() if v is not None}
    if op == "route":
        r = ops.moe_route(st["logits"], c["top_k"], renorm=c["renorm"], mask=st["mask"], out=out)
        st["out"] = r
        return {"experts": r.experts, "weights": r.weights, "counts": r.counts, "offsets": r.offsets,
                "row_token": r.row_token, "token_rows": r.token_rows, "lse": r.lse, "loss": r.loss}
    if op == "route_grad":
        r = ops.moe_route_backward(st["logits"], st["experts"], st["weights"], st["counts"], st["lse"],
                                   dweights=st["dweights"], dloss=st["dloss"], renorm=c["renorm"], out=out)
        st["out"] = r
        return r
    dy, dw = ops.moe_combine_backward(st["dout"], st["y"], st["token_rows"], st["weights"], out=out)
    st["out"] = (dy, dw)
    # rows behind the last assignment are not written
    return {"dy": dy[:(c["tokens"] - c["pad"]) * c["top_k"]], "dweights": dw}


_PLAIN = {"norm": _plain_norm, "norm_grad": _plain_norm_grad, "route": _plain_route, "route_grad": _plain_route_grad,
          "combine_grad": _plain_combine_grad}


def run(state):
    c = state["case"]
    return _own(c, state) if own else _PLAIN[c["op"]](c, state)


# ------------------------------------------------------------------- work
def work(case):
    c = case
    if c["op"] in ("norm", "norm_grad"):
        n, rows, cols = c["rows"] * c["cols"], c["rows"], c["cols"]
        st, w = (4 if c["res32"] else 2), (4 if c["w32"] else 2)
        pre, post = c["kind"] != "post", c["kind"] != "pre"
        gate = (-(-rows // c["gate_rows"]) * cols) if post and c["gate_rows"] else 0
        b = cols * w * (pre + post) + 2 * gate
        if c["op"] == "norm":
            b += n * st + (n * (2 + st) if post else 0)
            if pre:
                b += 2 * n * c["y"] + c["quant"] * (n + 4 * rows * -(-cols // GROUP))
            return {"bytes": b, "flops": n * (6 * post + 9 * pre)}
        b += n * st + 4 * cols * (pre + post) + gate * (4 if c["gate_rows"] > 1 else 2)
        if pre:
            b += n * (2 * st + (4 if c["dy32"] else 2))
        if post:
            b += 4 * n
        return {"bytes": b, "flops": n * (12 * pre + 14 * post)}
    T, k = c["tokens"], c["top_k"]
    live = T - c["pad"]
    if c["op"] == "combine_grad":
        H = c["cols"]
        return {"bytes": live * H * (4 if c["dout32"] else 2) + live * k * H * 4 + T * k * 12,
                "flops": 3 * live * k * H}
    E, z = c["experts"], (4 if c["logits32"] else 2)
    if c["op"] == "route":
        return {"bytes": live * E * z + T * (16 * k + 4) + 8 * E + 8 + T * bool(c["pad"]), "flops": live * E * (4 + k)}
    return {"bytes": live * E * z + T * E * z + T * (12 * k + 4) + 4 * E, "flops": live * E * 8}


# ------------------------------------------------- the definitions, 64 bits
def _d(t):
    return None if t is None else t.to(torch.float64)


def _e4m3(v):
    """The E4M3 value nearest to v (ties to even), |v| <= 448."""
    a = v.abs()
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -6))).clamp(min=-6.0)
    e = torch.where(torch.ldexp(torch.ones_like(e), e.int()) > a.clamp(min=2.0 ** -6), e - 1, e).clamp(min=-6.0)
    step = torch.ldexp(torch.ones_like(e), (e - 3).int())
    return torch.sign(v) * torch.round(a / step) * step


def _exact_norm(c, st):
    rows, cols = c["rows"], c["cols"]
    h, out = _d(st["residual"]), {}
    if st["x"] is not None:
        x = _d(st["x"])
        branch = x / torch.sqrt(torch.linalg.vector_norm(x, dim=1, keepdim=True) ** 2 / cols + EPS) * _d(st["w_post"])
        if st["gate"] is not None:
            at = torch.arange(rows, device=x.device) // st["rows_per_gate"]
            branch = branch * _d(st["gate"])[at]
        h = torch.add(h, branch, alpha=c["scale"])
        out["h"] = h
    if st["w_pre"] is None:
        return out
    y = h / torch.sqrt(torch.linalg.vector_norm(h, dim=1, keepdim=True) ** 2 / cols + EPS) * _d(st["w_pre"])
    if c["y"]:
        out["y"] = y
    if c["quant"]:
        parts = [y[:, g:g + GROUP] for g in range(0, cols, GROUP)]
        scales = [p.abs().max(dim=1, keepdim=True).values / 448.0 for p in parts]
        out["q"] = torch.cat([_e4m3(p / s.clamp(min=1e-300)) for p, s in zip(parts, scales)], dim=1)
        out["s"] = torch.cat(scales, dim=1)
    return out


def _exact_norm_grad(c, st):
    """By the chain rule through autograd in 64 bits, from the forward's
    definition at the saved h and x."""
    rows, cols = c["rows"], c["cols"]
    leaf = lambda t: None if t is None else _d(t).requires_grad_(True)
    out = {}
    dh = _d(st["dh"])
    if st["w_pre"] is not None:
        h, w = leaf(st["h"]), leaf(st["w_pre"])
        y = h / torch.sqrt((h * h).sum(dim=1, keepdim=True) / cols + EPS) * w
        gh, out["dw_pre"] = torch.autograd.grad((y * _d(st["dy"])).sum(), (h, w))
        dh = dh + gh
        out["dres"] = dh
    if st["x"] is not None:
        x, w, gate = leaf(st["x"]), leaf(st["w_post"]), leaf(st["gate"])
        n = x / torch.sqrt((x * x).sum(dim=1, keepdim=True) / cols + EPS) * w
        if gate is not None:
            n = n * gate[torch.arange(rows, device=x.device) // st["rows_per_gate"]]
        leaves = [x, w] + ([gate] if gate is not None else [])
        grads = torch.autograd.grad((c["scale"] * n * dh).sum(), leaves)
        out["dx"], out["dw_post"] = grads[0], grads[1]
        if gate is not None:
            out["dgate"] = grads[2]
    return out


def _exact_probs(z, mask):
    z = _d(z)
    if mask is not None:
        z = z.masked_fill(~mask[:, None], -math.inf)
    lse = torch.logsumexp(z, dim=1)
    live = lse > -math.inf
    p = torch.softmax(z.masked_fill(~live[:, None], 0.0), dim=1) * live[:, None]
    return z, lse, live, p


def _exact_route(c, st):
    z, lse, live, p = _exact_probs(st["logits"], st["mask"])
    E, k = c["experts"], c["top_k"]
    chosen = z.sort(dim=1, descending=True, stable=True)
    top, idx = chosen.values[:, :k], chosen.indices[:, :k]
    w = p.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-300)
    hits = torch.zeros(z.shape[0], E, dtype=torch.float64, device=z.device)
    hits.scatter_(1, idx, (top > -math.inf).double())
    f = hits.sum(dim=0) / hits.sum().clamp(min=1.0)
    n = live.sum().clamp(min=1).double()
    loss = torch.stack([E * torch.dot(f, p.sum(dim=0) / n), lse[live].square().sum() / n])
    return {"experts": None, "weights": w, "counts": None, "offsets": None, "row_token": None, "token_rows": None,
            "lse": lse, "loss": loss}


def _exact_route_grad(c, st):
    """Through autograd in 64 bits: the scalar sum(w dweights) + dloss . loss."""
    E, k = c["experts"], c["top_k"]
    live = st["lse"] > -math.inf
    z = _d(st["logits"]).masked_fill(~live[:, None], 0.0).requires_grad_(True)
    lse = torch.logsumexp(z, dim=1)
    p = torch.softmax(z, dim=1) * live[:, None]
    used = st["experts"] >= 0
    w = p.gather(1, st["experts"].long().clamp(min=0)) * used
    if c["renorm"]:
        w = w / w.sum(dim=1, keepdim=True).clamp(min=1e-300)
    counts = _d(st["counts"])
    n = counts[E].clamp(min=1.0)
    f = counts[:E] / counts[:E].sum().clamp(min=1.0)
    g = _d(st["dloss"])
    total = (w * _d(st["dweights"])).sum() + g[0] * E * torch.dot(f, p.sum(dim=0)) / n
    total = total + g[1] * torch.where(live, lse, torch.zeros_like(lse)).square().sum() / n
    d, = torch.autograd.grad(total, (z,))
    return d * live[:, None]


def _exact_combine_grad(c, st):
    T, k, H = c["tokens"], c["top_k"], c["cols"]
    rows = (T - c["pad"]) * k
    owner = torch.zeros(rows, dtype=torch.int64, device="cuda")
    weight = torch.zeros(rows, dtype=torch.float64, device="cuda")
    dw = torch.zeros((T, k), dtype=torch.float64, device="cuda")
    dout = _d(st["dout"])
    live = T - c["pad"]
    for j in range(k):
        at = st["token_rows"][:live, j].long()
        owner[at] = torch.arange(live, device="cuda")
        weight[at] = _d(st["weights"])[:live, j]
        dw[:live, j] = torch.linalg.vecdot(_d(st["y"][at]), dout[:live])
    return {"dy": dout[owner] * weight[:, None], "dweights": dw}


def exact(case, seed):
    st = prepare(case, seed)
    return {"norm": _exact_norm, "norm_grad": _exact_norm_grad, "route": _exact_route,
            "route_grad": _exact_route_grad, "combine_grad": _exact_combine_grad}[case["op"]](case, st)
