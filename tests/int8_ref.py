"""64-bit references of the linear layers in 8-bit integers (CPU)."""
import torch

U = 2.0 ** -24                               # half a step of fp32, relative


def codes(x):
    """(codes, scales) of the rows of x by the definition, from exact integers:
    x / S is compared with the half-way points through x - q S, which 64 bits hold
    exactly for bf16 x and fp32 S.  Non-finite rows: codes 0."""
    x = x.to(torch.float64)
    amax = x.abs().amax(dim=1) if x.shape[1] else torch.zeros(x.shape[0], dtype=torch.float64)
    amax = torch.where(torch.isnan(x).any(dim=1), torch.full_like(amax, torch.nan), amax)
    s = (amax / 127.0).to(torch.float32).to(torch.float64)
    fine = torch.isfinite(s) & (s > 0)
    d = torch.where(fine, s, torch.ones_like(s))[:, None]
    v = torch.where(fine[:, None], x, torch.zeros_like(x))
    q = torch.round(v / d)
    for _ in range(2):
        r = v - q * d
        out = (r.abs() > d / 2) | ((r.abs() == d / 2) & (torch.remainder(q, 2) == 1))
        q = torch.where(out, q + torch.sign(r), q)
    return q, s


def pad(q):
    """Codes as int8 with zero columns up to a multiple of 16."""
    out = torch.zeros((q.shape[0], (q.shape[1] + 15) // 16 * 16), dtype=torch.int8)
    out[:, :q.shape[1]] = q.to(torch.int8)
    return out


def product(qa, sa, qb, sb):
    """The product in 64 bits: codes' sums are exact (below 2^53)."""
    d = lambda t: t.detach().cpu().to(torch.float64)
    return d(sa)[:, None] * d(sb)[None, :] * (d(qa) @ d(qb).t().contiguous())


def check_product(c, ref):
    """Three fp32 roundings (the sum's conversion, two products), then half a step
    of the output's type; and a result of 0 where the sum or a scale is 0.  Below
    the type's normal numbers a step is absolute."""
    c = c.detach().cpu()
    half = torch.finfo(c.dtype).eps / 2 if c.dtype != torch.float32 else 0.0
    lim = ref.abs() * (3.01 * U + half * 1.01) + 2.0 ** -133
    err = (c.to(torch.float64) - ref).abs()
    assert (err <= lim).all(), "worst ratio %.3g" % float((err / lim).max())


def silu_h(gu):
    """h = bf16(silu(gate) up), through float32 only where that is exact: rounds the
    64-bit value to bf16 by its own spacing."""
    gu = gu.to(torch.float64)
    I = gu.shape[1] // 2
    g, u = gu[:, :I], gu[:, I:]
    v = g / (1.0 + torch.exp(-g)) * u
    a = v.abs()
    e = torch.floor(torch.log2(a.clamp(min=2.0 ** -126)))
    e = torch.where(torch.exp2(e) > a.clamp(min=2.0 ** -126), e - 1, e).clamp(min=-126)
    step = torch.exp2(e - 7)
    return (torch.round(v / step) * step).to(torch.bfloat16)
