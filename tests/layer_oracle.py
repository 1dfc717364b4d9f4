"""Norm, expert dispatch and clipping in 64 bits on the CPU, straight from
their formulas, and how far 32-bit kernels may be from them.

Tolerances.  u = 2^-24 is fp32's unit roundoff.
Norm: h = x + residual rounds once.  A sum over a row goes over at most 32
elements of a thread, then over at most 10 levels of pairs, so the sum of
squares is off by less than 44 u relative and r = 1 / sqrt(mean + eps) by less
than 22 u + 4 u; y = g h r has three more roundings: 32 u.  A sum of products
that may cancel is off by less than 48 u times the sum of their sizes.
Combine: topk fused multiply-adds, topk u times the sum of the sizes.
Products over a row: a lane adds cols / 64 + 8 terms where one wave takes a token,
less where two to eight waves share it, then 6 to 9 levels: products_tolerance().  Up
to 2,200 columns of one wave, and for all shared rows, that is within the (40 + cols /
256) u of combine_grad below.  Clipping: squares in 64 bits, of halves eight at a time in 32 (8 u, so
4 u of the norm), the norm rounds once, the factor once, the product once."""
import torch

from tests.loss_oracle import STEP, U, assert_within, rounded  # noqa: F401

E4M3 = torch.float8_e4m3fn


# ---- norm ---------------------------------------------------------------------------
def norm(x, gain, residual, eps):
    """(h, r, y)"""
    h = x.double() if residual is None else x.double() + residual.double()
    r = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    g = torch.ones(x.shape[1], dtype=torch.float64) if gain is None else gain.double()
    return h, r, g * h * r


def check_norm(got, total, x, gain, residual, eps, what=""):
    h, _, y = norm(x, gain, residual, eps)
    assert_within(got, y, rounded(64 * U * y.abs(), y, got.dtype), f"{what} y")
    if total is not None:
        assert_within(total, h, rounded(U * h.abs(), h, total.dtype), f"{what} total")


def check_quant(q, scales, total, x, gain, residual, eps, group, what=""):
    """q and scales against y / scale and max |y| / 448; e4m3 rounds by at most 2^-4 of the value, or half of its
    smallest step 2^-9."""
    h, _, y = norm(x, gain, residual, eps)
    n, c = y.shape
    k = -(-c // group)
    parts = torch.nn.functional.pad(y, (0, k * group - c)).view(n, k, group)
    top = parts.abs().amax(2)
    assert_within(scales, top / 448, 64 * U * top / 448 + 1e-37, f"{what} scales")
    t = torch.where(top[:, :, None] > 0, parts / torch.where(top > 0, top, 1.0)[:, :, None] * 448, 0.0)
    t = t.reshape(n, k * group)[:, :c]
    got = q.cpu().float().double()
    off = (got - t).abs()
    tol = torch.clamp(t.abs() * 2.0 ** -4, min=2.0 ** -10) * (1 + 64 * U) + 64 * U * t.abs()
    assert got.shape == t.shape and not (off > tol).any(), f"{what} q: off by {(off / tol).max().item()} tolerances"
    if total is not None:
        assert_within(total, h, rounded(U * h.abs(), h, total.dtype), f"{what} total")


def norm_grad(h, gain, dy, dtotal, eps):
    """(dx, its tolerance before its rounding, dgain, its tolerance)"""
    h, d = h.double(), dy.double()
    n, c = h.shape
    g = torch.ones(c, dtype=torch.float64) if gain is None else gain.double()
    r = 1.0 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    u, dg = h * r, d * g
    mean = (dg * u).mean(1, keepdim=True)
    s = torch.zeros_like(h) if dtotal is None else dtotal.double()
    dx = r * (dg - u * mean) + s
    size = (dg * u).abs().mean(1, keepdim=True)
    tol = U * (r * (40 * dg.abs() + u.abs() * (64 * mean.abs() + 80 * size)) + 4 * s.abs() + 4 * dx.abs()) + 1e-37
    terms = (d * u).abs().sum(0)
    return dx, tol, (d * u).sum(0), (500 + n / 200) * U * terms + 1e-37


def norm_objective(x, gain, residual, eps, dy, dtotal):
    """What norm_grad's results are the gradients of."""
    h, _, y = norm(x, gain, residual, eps)
    return (y * dy).sum() + (0.0 if dtotal is None else (h * dtotal).sum())


# ---- experts ------------------------------------------------------------------------
def places(chosen, experts):
    """(place, offsets) by a sort of Python's."""
    t, k = chosen.shape
    slots = sorted((int(e), i) for i, e in enumerate(chosen.reshape(-1).tolist()) if 0 <= e < experts)
    place = torch.full((t * k,), -1, dtype=torch.int32)
    counts = [0] * (experts + 1)
    for n, (e, i) in enumerate(slots):
        place[i] = n
        counts[e + 1] += 1
    return place.view(t, k), torch.tensor(counts).cumsum(0).int()


def combine(rows, place, weights):
    """(out, tolerance before its rounding)"""
    t, k = place.shape
    out = torch.zeros(t, rows.shape[1], dtype=torch.float64)
    size = torch.zeros_like(out)
    for j in range(k):
        for i in range(t):
            p = int(place[i, j])
            if 0 <= p < rows.shape[0]:
                v = (1.0 if weights is None else weights[i, j].double()) * rows[p].double()
                out[i] += v
                size[i] += v.abs()
    return out, (k + 1) * U * size


def combine_grad(dy, rows, place, weights):
    """(drows with NaN where nothing is written, dweights, its tolerance)"""
    t, k = place.shape
    m, c = rows.shape
    drows = torch.full((m, c), torch.nan, dtype=torch.float64)
    dw, tol = torch.zeros(t, k, dtype=torch.float64), torch.zeros(t, k, dtype=torch.float64)
    for j in range(k):
        for i in range(t):
            p = int(place[i, j])
            if 0 <= p < m:
                d = dy[i].double()
                drows[p] = (1.0 if weights is None else weights[i, j].double()) * d
                dw[i, j] = (d * rows[p].double()).sum()
                tol[i, j] = (40 + c / 256) * U * (d * rows[p].double()).abs().sum()
    return drows, dw, tol + 1e-37


def products_tolerance(terms):
    """Of a sum over the last dimension of these products, in 32 bits by one wave."""
    return (terms.shape[-1] / 64 + 17) * U * terms.abs().sum(-1) + 1e-37


# ---- clipping ------------------------------------------------------------------------
def norm_of(grads):
    return torch.sqrt(sum(((g.double() ** 2).sum() for g in grads), torch.zeros((), dtype=torch.float64)))


def check_clip(norm, got, grads, max_norm, total=None):
    """total: the norm of all ranks' gradients, where grads are one rank's."""
    want = norm_of(grads) if total is None else total
    assert_within(norm.reshape(()), want, 8 * U * want + 1e-44, "norm")
    factor = 1.0 if want <= max_norm else max_norm / want
    for i, (a, g) in enumerate(zip(got, grads)):
        w = g.double() * factor
        assert_within(a, w, rounded(12 * U * w.abs(), w, a.dtype), f"gradient {i}")
