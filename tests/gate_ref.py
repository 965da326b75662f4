"""64-bit reference of the router with scores, a selection bias and groups (CPU),
with the magnitudes that the tests' error bounds use."""
import torch

EPS = 1e-20


def d(t):
    return None if t is None else t.detach().cpu().double()


def scores(z, sigmoid):
    """(s, p, total, live): logits with -inf in every place of a token that is not
    routed."""
    live = ~(z == -torch.inf).all(dim=1)
    safe = torch.where(live[:, None], z, torch.zeros_like(z))
    on = live[:, None].double()
    if sigmoid:
        s = torch.sigmoid(safe) * on
        sum_ = s.sum(dim=1)
        return s, s / (sum_ + EPS)[:, None], torch.where(live, sum_, torch.full_like(sum_, -torch.inf)), live
    s = torch.softmax(safe, dim=1) * on
    total = torch.logsumexp(safe, dim=1)
    return s, s, torch.where(live, total, torch.full_like(total, -torch.inf)), live


def select(z, v, groups, keep, top2, k):
    """Experts of one token, by comparing values one by one: nothing but the
    definition.  z, v: lists of 64-bit numbers."""
    E, per = len(v), len(v) // groups
    rank = lambda x: (1, 0.0) if x != x else (0, x)         # NaN is the largest
    there = [not (z[e] == float("-inf") or v[e] == float("-inf")) for e in range(E)]
    if keep < groups:
        value = []
        for g in range(groups):
            best = sorted((v[e] for e in range(g * per, (g + 1) * per) if there[e]), key=rank, reverse=True)
            value.append(sum(best[:2 if top2 else 1]) if best else float("-inf"))
        kept = set(sorted(range(groups), key=lambda g: (rank(value[g])[0], rank(value[g])[1], -g), reverse=True)[:keep])
        there = [there[e] and e // per in kept for e in range(E)]
    left = [e for e in range(E) if there[e]]
    left.sort(key=lambda e: (rank(v[e])[0], rank(v[e])[1], -e), reverse=True)
    return left[:k]


def route(z, k, *, sigmoid, bias=None, groups=1, keep=None, top2=True, renorm=True, scale=1.0, mask=None):
    keep = groups if keep is None else keep
    T, E = z.shape
    z = d(z)
    if mask is not None:
        z = torch.where(mask.cpu().bool()[:, None], z, torch.full_like(z, -torch.inf))
    s, p, total, live = scores(z, sigmoid)
    v = s if bias is None else s + d(bias)
    if bias is None:                     # the scores are monotone: where two agree in 64 bits, logits decide
        order = z
    experts = torch.full((T, k), -1, dtype=torch.int64)
    zl, vl = z.tolist(), v.tolist()
    for t in range(T):
        if not live[t]:
            continue
        if bias is None:
            # groups by value, experts inside by logits
            if keep < groups:
                per = E // groups
                all_ = select(zl[t], vl[t], groups, keep, top2, E) if top2 else select(zl[t], zl[t], groups, keep, False, E)
                kept = {e // per for e in all_}
                row = [x if e // per in kept else float("-inf") for e, x in enumerate(order[t].tolist())]
            else:
                row = order[t].tolist()
            at = select(row, row, 1, 1, False, k)
        else:
            at = select(zl[t], vl[t], groups, keep, top2, k)
        experts[t, :len(at)] = torch.tensor(at, dtype=torch.int64)
    used = experts >= 0
    w = torch.where(used, s.gather(1, experts.clamp(min=0)), torch.zeros(T, k, dtype=torch.float64))
    if renorm:
        w = w / (w.sum(dim=1, keepdim=True) + EPS)
    flat = experts.reshape(-1)
    row_of = torch.nonzero(flat >= 0)[:, 0]
    order = row_of[flat[row_of].sort(stable=True).indices]
    row_token = torch.zeros(T * k, dtype=torch.int64)
    row_token[:order.numel()] = order // k
    token_rows = torch.full((T * k,), -1, dtype=torch.int64)
    token_rows[order] = torch.arange(order.numel())
    counts = torch.bincount(flat[row_of], minlength=E)
    offsets = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
    n = max(1, int(live.sum()))
    f = counts.double() / max(1, int(counts.sum()))
    loss = torch.stack([E * (f * p.sum(0) / n).sum(),
                        torch.zeros((), dtype=torch.float64) if sigmoid else (total[live] ** 2).sum() / n])
    return {"z": z, "s": s, "p": p, "total": total, "live": live, "experts": experts, "weights": scale * w,
            "counts": torch.cat([counts, torch.tensor([int(live.sum())])]), "offsets": offsets, "row_token": row_token,
            "token_rows": token_rows.view(T, k), "loss": loss, "f": f, "n": n}


def objective(ref, z, dw, dl, *, sigmoid, renorm, scale):
    """sum(weights dw) + dl . loss at logits z, with ref's selection and counts."""
    s, p, total, live = scores(z, sigmoid)
    used = ref["experts"] >= 0
    w = torch.where(used, s.gather(1, ref["experts"].clamp(min=0)), torch.zeros_like(dw))
    if renorm:
        w = w / (w.sum(dim=1, keepdim=True) + EPS)
    out = scale * (w * torch.where(used, dw, torch.zeros_like(dw))).sum() + dl[0] * z.shape[1] * (ref["f"] * p.sum(0)).sum() / ref["n"]
    return out if sigmoid else out + dl[1] * (total[live] ** 2).sum() / ref["n"]


def grad(ref, dw, dl, *, sigmoid, renorm, scale):
    """(gradient at the logits, magnitude of its terms) by the formulas."""
    z, s, p, live = ref["z"], ref["s"], ref["p"], ref["live"]
    T, E = z.shape
    dw, dl = d(dw), d(dl)
    used = ref["experts"] >= 0
    at = ref["experts"].clamp(min=0)
    a, m = torch.zeros(T, E + 1, dtype=torch.float64), torch.zeros(T, E + 1, dtype=torch.float64)
    if dw is not None:
        g = scale * torch.where(used, dw, torch.zeros_like(dw))
        mg = g.abs()
        taken = torch.where(used, s.gather(1, at), torch.zeros_like(g))
        if renorm:
            norm = taken.sum(1, keepdim=True) + EPS
            mean, mmean = (taken / norm * g).sum(1, keepdim=True), (taken / norm * mg).sum(1, keepdim=True)
            g, mg = (g - mean) / norm, (mg + mmean) / norm
        idx = torch.where(used, at, torch.full_like(at, E))
        a.scatter_(1, idx, g)
        m.scatter_(1, idx, mg)
    a, m = a[:, :E], m[:, :E]
    g0, g1 = (0.0, 0.0) if dl is None else (float(dl[0]), float(dl[1]))
    f = g0 * E / ref["n"] * ref["f"]
    if sigmoid:
        sum_ = s.sum(1, keepdim=True) + EPS
        a = a + (f - (f * p).sum(1, keepdim=True)) / sum_
        m = m + (f.abs() + (f.abs() * p).sum(1, keepdim=True)) / sum_
        out, mag = a * s * (1 - s), m * s * (1 - s)
    else:
        tot = torch.where(live, ref["total"], torch.zeros_like(ref["total"]))[:, None] * (2 * g1 / ref["n"])
        a, m = a + f, m + f.abs()
        out = p * (a - (p * a).sum(1, keepdim=True) + tot)
        mag = p * (m + (p * m).sum(1, keepdim=True) + tot.abs())
    zero = torch.zeros_like(out)
    return torch.where(live[:, None], out, zero), torch.where(live[:, None], mag, zero)
