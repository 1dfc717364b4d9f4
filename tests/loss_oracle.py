"""Routing and distillation in 64 bits on the CPU, straight from their
formulas, and how far 32-bit kernels may be from them.

Tolerances.  u = 2^-24 is fp32's unit roundoff.  A kernel's probability is
2^((x - m) log2(e) / tau) / Z: the difference, the product and the constant
round once each (3 u relative to the exponent, so 3 u |x - m| / tau relative
to the result), the hardware's 2^x is good to 2 u, and Z is a sum of at most a
few hundred partial roundings on top of terms that are themselves off by
3 u D e^-D <= 1.2 u, so p is off by less than (4 D + 64) u relative, with
D = |x - m| / tau.  A gradient is scale (p - q) with both off by that much
(and the scale by 4 u), then rounded once to its type.  Products below 1e-37
may be flushed."""
import torch

U = 2.0 ** -24
STEP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
LEAST = {torch.float32: 1e-37, torch.float16: 2.0 ** -24, torch.bfloat16: 1e-37}


def assert_within(got, want, tol, what=""):
    # a result past its type's range is an infinity of that type; one whose tolerance reaches past it may be
    most = torch.finfo(got.dtype).max
    got = got.detach().cpu().double()
    past = (want.abs() > most) | ((want.abs() + tol > most) & torch.isinf(got))
    want = torch.where(past, want.sign() * torch.inf, want.double())
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan), f"{what}: NaN in other places"
    inf = torch.isinf(want)
    assert torch.equal(got[inf], want[inf]), f"{what}: infinities differ"
    ok = ~(nan | inf)
    off = (got - want).abs()
    bad = ok & ~(off <= tol)
    if bad.any():
        i = torch.nonzero(bad)[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} values off, first at {i}: got "
                             f"{got[tuple(i)].item()!r}, want {want[tuple(i)].item()!r}")


# ---- routing ----------------------------------------------------------------------
def _gate(x, keep):
    live = ~torch.isneginf(x).all(1)
    if keep is not None:
        live &= keep.bool()
    y = torch.where(live[:, None], x, 0.0)
    m = torch.where(torch.isnan(y), -torch.inf, y).amax(1, keepdim=True)
    e = torch.exp(y - m)
    p = e / e.sum(1, keepdim=True)
    return torch.where(live[:, None], p, 0.0), live, (m - y).abs()


def route(x, topk, keep, normalize):
    """(chosen, weights, counts, prob_sums, relative tolerance of weights, of p)"""
    x = x.double()
    t, e = x.shape
    p, live, far = _gate(x, keep)
    can = live[:, None] & ~torch.isneginf(x) & ~torch.isnan(x)
    chosen = torch.full((t, topk), -1, dtype=torch.int32)
    for r in range(t):
        order = sorted((i for i in range(e) if can[r, i]), key=lambda i: (-x[r, i].item(), i))[:topk]
        chosen[r, :len(order)] = torch.tensor(order, dtype=torch.int32)
    at = chosen.clamp(min=0).long()
    w = torch.where(chosen >= 0, p.gather(1, at), 0.0)
    if normalize:
        w = torch.where(chosen >= 0, w / w.sum(1, keepdim=True), 0.0)
        bad = torch.isnan(p).any(1, keepdim=True)
        w = torch.where((chosen >= 0) & bad, torch.nan, w)
    counts = torch.zeros(e + 1, dtype=torch.int32)
    for i in range(e):
        counts[i] = (chosen == i).sum()
    counts[e] = live.sum()
    wide = torch.where(torch.isfinite(far), far, 0.0)
    rel = (4 * wide.gather(1, at) + 64) * U
    return chosen, w, counts, p.sum(0), 2 * rel * w.abs() + 1e-37, ((4 * wide + 64) * U * p).sum(0) + t * U * p.sum(0)


def balance_loss(x, counts, prob_sums, topk, coef):
    """The scalar that sim_route_grad reports."""
    e = counts.numel() - 1
    n = float(counts[e])
    if n == 0:
        return torch.zeros((), dtype=torch.float64)
    f = counts[:e].double() * e / (topk * n)
    return coef * (f * prob_sums.double()).sum() / n


def route_objective(x, chosen, dweights, counts, coef, keep, normalize):
    """What sim_route_grad's dlogits is the gradient of, for a double x."""
    e = x.shape[1]
    p, live, _ = _gate(x, keep)
    total = torch.zeros((), dtype=torch.float64)
    if counts is not None and float(counts[e]) > 0:
        n = float(counts[e])
        total = total + coef / n * (p * (counts[:e].double() * e / (chosen.shape[1] * n))).sum()
    if dweights is not None:
        ok = (chosen >= 0) & (chosen < e) & live[:, None]
        w = torch.where(ok, p.gather(1, torch.where(ok, chosen, 0).long()), 0.0)
        if normalize:
            s = w.sum(1, keepdim=True)
            w = w / torch.where(s == 0, 1.0, s)
        total = total + (torch.where(ok, dweights.double(), 0.0) * w).sum()
    return total


def route_grad(x, chosen, dweights, counts, coef, keep, normalize):
    """(gradient, absolute tolerance before the rounding to its type)"""
    y = x.double()
    p, live, far = _gate(y, keep)
    t, e = y.shape
    g = torch.zeros(t, e, dtype=torch.float64)
    if counts is not None and float(counts[e]) > 0:
        n = float(counts[e])
        g += coef / n * counts[:e].double() * e / (chosen.shape[1] * n)
    u = torch.zeros(t, e + 1, dtype=torch.float64)
    hot = torch.zeros(t, e + 1, dtype=torch.float64)
    if dweights is not None:
        ok = (chosen >= 0) & (chosen < e)
        at = torch.where(ok, chosen, e).long()
        u.scatter_(1, at, dweights.double())
        hot.scatter_(1, at, 1.0)
    u, hot = u[:, :e], hot[:, :e]
    rel = (4 * torch.where(torch.isfinite(far), far, 0.0).clamp(max=200.0) + 64 + e) * U
    if not normalize:
        g = g + u
    d = p * (g - (p * g).sum(1, keepdim=True))
    tol = 4 * rel * p * (g.abs() + (p * g.abs()).sum(1, keepdim=True))
    if normalize:
        w = p * hot
        s = w.sum(1, keepdim=True)
        w = w / torch.where(s == 0, 1.0, s)
        d = d + w * (u - (w * u).sum(1, keepdim=True))
        tol = tol + 4 * rel * w * (u.abs() + (w * u.abs()).sum(1, keepdim=True))
    return torch.where(live[:, None], d, 0.0), tol + 1e-37


# ---- distillation -------------------------------------------------------------------
def teacher(ids, z, tau, vocab):
    """(valid, q, log q, live row)"""
    ok = (ids >= 0) & (ids < vocab)
    y = torch.where(ok, z.double() / tau, -torch.inf)
    live = (ok & ~torch.isneginf(y)).any(1)
    top = torch.where(live[:, None], torch.where(torch.isnan(y), -torch.inf, y).amax(1, keepdim=True), 0.0)
    e = torch.exp(y - top)
    s = torch.where(live[:, None], e.sum(1, keepdim=True), 1.0)
    return ok, e / s, y - top - torch.log(s), live


def distill_loss(x, ids, z, tau):
    """Loss of each row for a double x."""
    ok, q, logq, live = teacher(ids, z, tau, x.shape[1])
    y = x / tau
    m = torch.where(torch.isnan(y), -torch.inf, y).amax(1, keepdim=True)
    logs = torch.log(torch.exp(y - m).sum(1, keepdim=True))
    logp = (y.gather(1, torch.where(ok, ids, 0).long()) - m) - logs
    return torch.where(live, torch.where(ok & (q != 0), q * (logq - logp), 0.0).sum(1), 0.0)


def distill(x, ids, z, tau, row_scale, coef):
    """(loss, its tolerance, gradient, its tolerance before the rounding to its type)"""
    x = x.double()
    t, v = x.shape
    ok, q, logq, live = teacher(ids, z, tau, v)
    y = x / tau
    m = torch.where(torch.isnan(y), -torch.inf, y).amax(1, keepdim=True)
    e = torch.exp(y - m)
    s = e.sum(1, keepdim=True)
    p = e / s
    loss = distill_loss(x, ids, z, tau)
    far = torch.where(torch.isfinite(m - y), (m - y).abs(), 0.0)
    target = torch.zeros(t, v + 1, dtype=torch.float64).scatter_add_(1, torch.where(ok, ids, v).long(), q)[:, :v]
    scale = (torch.ones(t, dtype=torch.float64) if row_scale is None else row_scale.double()) * (coef / tau)
    d = torch.where(live[:, None], scale[:, None] * (p - target), 0.0)
    tol = scale.abs()[:, None] * U * ((4 * far.clamp(max=200.0) + 64) * p + (4 * 64 + 64) * target) + 1e-37
    at = torch.where(ok, ids, 0).long()
    size = 16 + torch.where(ok & (q > 0), logq.abs() + far.gather(1, at), 0.0).amax(1)
    return loss, 8 * U * size, d, torch.where(torch.isnan(tol), 0.0, tol)


def rounded(tol, want, dtype):
    """A tolerance before the rounding to `dtype`, with that rounding."""
    return tol + STEP[dtype] * want.abs() + LEAST[dtype]
