"""Seeded random calls of the norm, expert and clipping operators over their
whole ranges of sizes, types and strides, against the 64-bit formulas on the
GPU."""
import random

import pytest
import torch

from tests import layer_oracle as oracle

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.float16, torch.bfloat16]
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def lib():
    import all_reduce_reduction_amd as sim
    sim.sim_init(0, 16, 0)
    yield sim


def log(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def matrix(rng, gen, n, c, dtype, factor=1.0):
    """n x c inside wider rows, from any column on; (view, whether the rest stayed)"""
    wide = torch.full((n, c + rng.choice((0, 0, 1, 7, 64))), 7.0, dtype=dtype)
    first = rng.randint(0, wide.shape[1] - c)
    wide[:, first:first + c] = (torch.randn(n, c, generator=gen) * factor).to(dtype)
    wide = wide.cuda()

    def stayed():
        return bool((wide[:, :first] == 7).all() and (wide[:, first + c:] == 7).all())

    return wide[:, first:first + c], stayed


@pytest.mark.parametrize("seed", range(40))
def test_norm(lib, seed):
    rng, gen = random.Random(seed), torch.Generator().manual_seed(seed)
    dtype, gt = rng.choice(DTYPES), rng.choice(DTYPES + [None])
    c = log(rng, 1, 32768)
    n = log(rng, 1, min(5000, max(2, (1 << 22) // c)))
    gain = None if gt is None else (1 + 0.2 * torch.randn(c, generator=gen)).to(gt)
    gd = None if gain is None else gain.cuda()
    x, _ = matrix(rng, gen, n, c, dtype)
    residual = matrix(rng, gen, n, c, dtype, 2.0)[0] if rng.random() < 0.6 else None
    rc = None if residual is None else residual.cpu()
    (y, y_ok), (total, t_ok) = matrix(rng, gen, n, c, dtype), matrix(rng, gen, n, c, dtype)
    lib.norm(x, gd, residual=residual, eps=EPS, out=(y, total if residual is not None else None))
    oracle.check_norm(y, total if residual is not None else None, x.cpu(), gain, rc, EPS)
    assert y_ok() and t_ok()
    group = rng.choice((32, 64, 128, c))
    q, s, t = lib.norm_quant(x, gd, residual=residual, eps=EPS, group=group)
    oracle.check_quant(q, s, t, x.cpu(), gain, rc, EPS, group)
    dy, _ = matrix(rng, gen, n, c, dtype)
    dtotal = matrix(rng, gen, n, c, dtype)[0] if rng.random() < 0.5 else None
    (dx, d_ok) = matrix(rng, gen, n, c, dtype)
    dgain = torch.empty(c, device="cuda")
    lib.norm_grad(x, gd, dy, dtotal=dtotal, eps=EPS, out=(dx, dgain))
    want, tol, wg, gtol = oracle.norm_grad(x.cpu(), gain, dy.cpu(), None if dtotal is None else dtotal.cpu(), EPS)
    oracle.assert_within(dx, want, oracle.rounded(tol, want, dtype), "dx")
    oracle.assert_within(dgain, wg, gtol, "dgain")
    assert d_ok()


@pytest.mark.parametrize("seed", range(40))
def test_experts(lib, seed):
    rng, gen = random.Random(100 + seed), torch.Generator().manual_seed(100 + seed)
    dtype = rng.choice(DTYPES)
    e, k, c = log(rng, 1, 1024), rng.randint(1, 32), log(rng, 1, 6000)
    t = log(rng, 1, min(9000, max(2, (1 << 23) // (k * c))))
    chosen = torch.randint(-2, e + 1, (t, k), generator=gen, dtype=torch.int32).cuda()
    x, _ = matrix(rng, gen, t, c, dtype)
    groups = rng.choice((0, 0, 1, 5, 700))
    scales = torch.rand(t, groups, generator=gen).cuda() if groups else None
    rows, place, offsets, row_scales = lib.dispatch(x, chosen, e, scales=scales)
    flat = chosen.reshape(-1).long()
    key = torch.where((flat >= 0) & (flat < e), flat, e)
    order = torch.sort(key, stable=True).indices
    m = int((key < e).sum())
    at = torch.full_like(flat, -1)
    at[order[:m]] = torch.arange(m, device="cuda")
    assert torch.equal(place.reshape(-1).long(), at)
    assert torch.equal(offsets[1:].long(), torch.bincount(key, minlength=e + 1)[:e].cumsum(0)) and offsets[0] == 0
    assert torch.equal(rows[:m], x[order[:m] // k])
    if groups:
        assert torch.equal(row_scales[:m], scales[order[:m] // k])
    # back, and the gradient, by the same places
    (src, s_ok), (out, o_ok) = matrix(rng, gen, t * k, c, dtype), matrix(rng, gen, t, c, dtype)
    w = torch.randn(t, k, generator=gen).cuda() if rng.random() < 0.7 else None
    lib.combine(src, place, w, out=out)
    full = (at >= 0).view(t, k)
    picked = src[at.clamp(min=0)].view(t, k, c).double()
    ww = full.double() if w is None else torch.where(full, w.double(), 0.0)
    terms = picked * ww[:, :, None]
    want = terms.sum(1)
    oracle.assert_within(out.cpu(), want.cpu(), oracle.rounded((k + 1) * oracle.U * terms.abs().sum(1), want, dtype).cpu(), "out")
    dy, _ = matrix(rng, gen, t, c, dtype)
    drows, d_ok = matrix(rng, gen, t * k, c, dtype)
    before = drows.clone()
    dw = torch.empty(t, k, device="cuda")
    lib.combine_grad(dy, src, place, w, out=(drows, dw))
    prods = dy.double()[:, None] * picked
    oracle.assert_within(dw.cpu(), torch.where(full, prods.sum(2), 0.0).cpu(),
                         ((40 + c / 256) * oracle.U * prods.abs().sum(2) + 1e-37).cpu(), "dweights")
    up = dy.float()[:, None].expand(t, k, c) if w is None else dy.float()[:, None] * w[:, :, None]
    before[at[full.view(-1)]] = up.reshape(t * k, c)[full.view(-1)].to(dtype)
    assert torch.equal(drows, before) and s_ok() and o_ok() and d_ok()


@pytest.mark.parametrize("seed", range(30))
def test_clip(lib, seed):
    rng, gen = random.Random(200 + seed), torch.Generator().manual_seed(200 + seed)
    n = log(rng, 1, 400)
    factor = rng.choice((1.0, 1.0, 1e-3, 100.0))
    types = rng.choice(([torch.bfloat16], [torch.float32], DTYPES))
    host = [(torch.randn(log(rng, 1, rng.choice((10, 3000, 100000))), generator=gen) * factor).to(rng.choice(types)) for _ in range(n)]
    grads = [g.cuda() for g in host]
    most = oracle.norm_of(host).item() * rng.choice((0.01, 0.5, 2.0))
    out = [torch.empty_like(g) for g in grads] if rng.random() < 0.5 else None
    if out is not None and rng.random() < 0.3:
        out[0] = grads[0]  # some in place, some not
    norm = lib.clip_grads(grads, most, out=out)
    oracle.check_clip(norm, grads if out is None else out, host, most)
