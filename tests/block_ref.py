"""64-bit references of the block norm, the router and the combine's gradient
(plain torch on the CPU), with the magnitudes the tests' error bounds use.

fp32 bounds count roundings of U = 2^-24 (finfo(float32).eps / 2) on the sum
of the magnitudes of the terms that enter a value."""
import torch

U = torch.finfo(torch.float32).eps / 2
HALF = {torch.float32: U, torch.bfloat16: torch.finfo(torch.bfloat16).eps / 2}


def d(t):
    return None if t is None else t.detach().cpu().double()


def rms(v, eps):
    return 1.0 / torch.sqrt((v * v).mean(dim=1, keepdim=True) + eps)


def spread(gate, R, rows):
    return gate[torch.arange(rows) // R]


def norm(residual, x, w_pre, w_post, gate, R, scale, eps):
    """(h, |h| terms, y, |y| terms) in 64 bits."""
    residual, x, w_pre, w_post, gate = map(d, (residual, x, w_pre, w_post, gate))
    rows, cols = (x if residual is None else residual).shape
    h = torch.zeros(rows, cols, dtype=torch.float64) if residual is None else residual
    mag = h.abs()
    if x is not None:
        b = x if w_post is None else x * rms(x, eps) * w_post
        b = scale * b
        if gate is not None:
            b = b * spread(gate, R, rows)
        h, mag = h + b, mag + b.abs()
    if w_pre is None:
        return h, mag, None, None
    r = rms(h, eps)
    return h, mag, h * r * w_pre, mag * r * w_pre.abs()


def norm_grad(dy, dh, h, x, w_pre, w_post, gate, R, scale, eps):
    """dict of name -> (value, terms' magnitude) in 64 bits."""
    dy, dh, h, x, w_pre, w_post, gate = map(d, (dy, dh, h, x, w_pre, w_post, gate))
    rows, cols = (dh if dh is not None else h).shape
    out = {}
    dH = torch.zeros(rows, cols, dtype=torch.float64) if dh is None else dh
    mH = dH.abs()
    if w_pre is not None:
        r = rms(h, eps)
        hh, g = h * r, dy * w_pre
        out["dw_pre"] = ((dy * hh).sum(0), (dy * hh).abs().sum(0))
        dH = dH + r * (g - hh * (g * hh).mean(1, keepdim=True))
        mH = mH + r * (g.abs() + hh.abs() * (g * hh).abs().mean(1, keepdim=True))
    out["dres"] = (dH, mH)
    if x is None:
        return out
    r = rms(x, eps) if w_post is not None else torch.ones(rows, 1, dtype=torch.float64)
    xh = x * r
    dn, mn = scale * dH, abs(scale) * mH
    if gate is not None:
        n = xh if w_post is None else xh * w_post
        G = gate.shape[0]
        s = lambda v: torch.zeros(G, cols, dtype=torch.float64).index_add_(0, torch.arange(rows) // R, v)
        out["dgate"] = (s(dn * n), s(mn * n.abs()))
        dn, mn = dn * spread(gate, R, rows), mn * spread(gate, R, rows).abs()
    if w_post is not None:
        out["dw_post"] = ((dn * xh).sum(0), (mn * xh.abs()).sum(0))
        g, mg = dn * w_post, mn * w_post.abs()
        out["dx"] = (r * (g - xh * (g * xh).mean(1, keepdim=True)),
                     r * (mg + xh.abs() * (mg * xh.abs()).mean(1, keepdim=True)))
    else:
        out["dx"] = (dn, mn)
    return out


def close(got, ref, mag, c, what):
    """|got - ref| <= c U mag + half a step of got's type (+ the smallest
    fp32 / bf16 subnormal steps)."""
    g = d(got)
    bound = c * U * mag + HALF[got.dtype] * torch.maximum(g.abs(), ref.abs()) + 1e-38
    err = (g - ref).abs()
    assert torch.isfinite(g).all(), "%s: not finite" % what
    worst = float((err / bound).max()) if err.numel() else 0.0
    assert worst <= 1.0, "%s: %.3g times the bound" % (what, worst)


E4M3 = torch.arange(0, 0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).double()   # 0 .. 448


def check_codes(q, s, y, mag, c, what):
    """Scales within c U of max|y| / 448 by terms; each code's value is at a
    distance from y / s no larger than the nearest code's plus twice the fp32
    error of the quotient."""
    rows, cols = y.shape
    ng = (cols + 127) // 128
    pad = lambda v: torch.nn.functional.pad(v, (0, ng * 128 - cols)).view(rows, ng, 128)
    yg, mg = pad(y), pad(mag)
    sref = yg.abs().amax(2) / 448.0
    s = d(s)
    assert ((s - sref).abs() <= c * U * mg.amax(2) / 448.0 + 1e-45).all(), "%s: scales" % what
    v = pad(q.cpu().view(torch.float8_e4m3fn).double())
    assert (v[(sref == 0)[:, :, None].expand_as(v)] == 0).all(), "%s: codes of a zero group" % what
    safe = torch.where(s > 0, s, torch.ones_like(s))[:, :, None]
    t = yg / safe
    tol = c * U * mg / safe + 4 * U * t.abs()
    a = t.abs().clamp(max=448.0)
    i = torch.searchsorted(E4M3, a.contiguous()).clamp(1, E4M3.numel() - 1)
    best = torch.minimum((E4M3[i] - a).abs(), (E4M3[i - 1] - a).abs())
    over = (v - t.clamp(-448.0, 448.0)).abs() - best - 2 * tol
    over = torch.where((s > 0)[:, :, None], over, torch.zeros_like(over))
    assert (over <= 0).all(), "%s: a code is not the nearest (by %.3g)" % (what, float(over.max()))


# ------------------------------------------------------------------ router
def route(logits, k, renorm, mask):
    """Selection, row maps (exact) and weights, lse, losses in 64 bits.  NaN
    is the largest logit; -inf and masked tokens take nothing."""
    z = d(logits)
    T, E = z.shape
    live = torch.ones(T, dtype=torch.bool) if mask is None else mask.cpu().bool()
    z = torch.where(live[:, None], z, torch.full_like(z, -torch.inf))
    key = torch.where(torch.isnan(z), torch.full_like(z, torch.inf), z)
    nan = torch.isnan(z).double()
    order = torch.arange(E).expand(T, E)
    # by (NaN first, value descending, index)
    idx = torch.argsort(-key, dim=1, stable=True)
    idx = idx.gather(1, torch.argsort(-nan.gather(1, idx), dim=1, stable=True))[:, :k]
    del order
    top = z.gather(1, idx)
    used = ~(top == -torch.inf)
    live = live & used.any(1)
    experts = torch.where(used, idx, torch.full_like(idx, -1))
    lse = torch.logsumexp(z, 1)
    # not exp(z - lse): at logits of a type's lowest value lse rounds to them
    p = torch.softmax(torch.where(live[:, None], z, torch.zeros_like(z)), dim=1) * live[:, None]
    m = top[:, :1]
    e = torch.where(used, torch.exp(top - torch.where(live[:, None], m, torch.zeros_like(m))), torch.zeros_like(top))
    w = e / e.sum(1, keepdim=True) if renorm else p.gather(1, idx)
    w = torch.where(used, w, torch.zeros_like(w))
    flat = experts.reshape(-1)
    key2 = torch.where(flat >= 0, flat, torch.full_like(flat, E))
    perm = torch.argsort(key2, stable=True)
    counts = torch.bincount(key2, minlength=E + 1)[:E]
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
    total = int(offsets[-1])
    row_token = torch.zeros(T * k, dtype=torch.int64)
    row_token[:total] = perm[:total] // k
    token_rows = torch.full((T * k,), -1, dtype=torch.int64)
    token_rows[perm[:total]] = torch.arange(total)
    n = int(live.sum())
    f = counts.double() / max(1, int(counts.sum()))
    balance = E * float((f * p.sum(0)).sum()) / max(1, n)
    zl = float((lse[live] ** 2).sum()) / max(1, n)
    return {"experts": experts, "weights": w, "counts": torch.cat([counts, torch.tensor([n])]), "offsets": offsets,
            "row_token": row_token, "token_rows": token_rows.view(T, k), "lse": lse,
            "loss": torch.tensor([balance, zl], dtype=torch.float64), "p": p, "live": live, "f": f, "z": z}


def route_grad(ref, k, renorm, dweights, dloss):
    """(dlogits, terms' magnitude) in 64 bits from route()'s result."""
    p, live, f, w, lse = ref["p"], ref["live"], ref["f"], ref["weights"], ref["lse"]
    T, E = p.shape
    n = max(1, int(live.sum()))
    g0, g1 = (0.0, 0.0) if dloss is None else [float(v) for v in d(dloss)]
    dot = (p * f).sum(1, keepdim=True)
    l = torch.where(live, lse, torch.zeros_like(lse))[:, None]
    out = p * (g0 * E / n * (f - dot) + 2 * g1 / n * l)
    mag = p * (abs(g0) * E / n * (f + dot) + 2 * abs(g1) / n * l.abs())
    if dweights is not None:
        used = ref["experts"] >= 0
        dw = torch.where(used, d(dweights), torch.zeros_like(w))
        wd, wm = (w * dw).sum(1, keepdim=True), (w * dw).abs().sum(1, keepdim=True)
        part, pm = w * dw, (w * dw).abs()
        if renorm:
            part, pm = part - w * wd, pm + w * wm
        else:
            out, mag = out - p * wd, mag + p * wm
        at = ref["experts"].clamp(min=0)
        out = out.scatter_add(1, at, torch.where(used, part, torch.zeros_like(part)))
        mag = mag.scatter_add(1, at, torch.where(used, pm, torch.zeros_like(pm)))
    return out * live[:, None], mag * live[:, None]
