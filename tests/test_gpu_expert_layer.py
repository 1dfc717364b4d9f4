"""An expert layer's training step on simulated ranks with every operator around
it: norm of the residual sum, routing, dispatch, the experts' products, combine;
back through all of them; the gradients reduced over the ranks and clipped.
Against automatic differentiation of all ranks' tokens at once, in 64 bits.

Tolerance, of a tensor's 2-norm: about a dozen operations follow each other, each
rounding at most 96 times (sums of 64 terms, exponents of at most 8) with errors of
either sign, 2 sqrt(96) u of its terms' sizes, which cancellation lets grow past the
results' by less than 30: 12 * 20 * 30 u = 4.3e-4.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
RANKS, TOKENS, COLS, EXPERTS, TOPK, EPS = 4, 96, 64, 8, 2, 1e-5


@pytest.fixture(scope="module", autouse=True)
def lib():
    import all_reduce_reduction_amd as sim
    sim.sim_init(0, 16, 0)
    yield sim


def near(got, want, what):
    off = (got.cpu().double() - want).norm() / want.norm()
    assert off < 4.3e-4, f"{what}: {off}"


def reference(x, res, gain, wr, we, g, chosen, keep):
    x, res, gain, wr, we = (t.double().requires_grad_(True) for t in (x, res, gain, wr, we))
    h = x + res
    y = gain * h / torch.sqrt((h * h).mean(1, keepdim=True) + EPS)
    p = torch.softmax(y @ wr, 1).gather(1, chosen.clamp(min=0).long())
    w = p / p.sum(1, keepdim=True)
    parts = torch.einsum("tc,tkcd->tkd", y, we[chosen.clamp(min=0).long()])
    out = h + torch.where(keep[:, None], (w[:, :, None] * parts).sum(1), 0.0)
    (out * g.double()).sum().backward()
    return out.detach(), x.grad, gain.grad, wr.grad, we.grad


@pytest.mark.parametrize("captured", [False, True])
def test_a_step_of_an_expert_layer(lib, captured):
    gen = torch.Generator().manual_seed(1)

    def rand(*shape, factor=1.0):
        return torch.randn(shape, generator=gen) * factor

    x, res, g = (rand(RANKS * TOKENS, COLS) for _ in range(3))
    gain, wr, we = 1 + 0.1 * rand(COLS), rand(COLS, EXPERTS, factor=0.3), rand(EXPERTS, COLS, COLS, factor=0.1)
    keep = torch.rand(RANKS * TOKENS, generator=gen) < 0.9  # padding tokens reach no expert
    dense, experts = [], []
    outs, dxs, chosens = [], [], []
    wrd, wed, gaind = wr.cuda(), we.cuda(), gain.cuda()
    for r in range(RANKS):
        mine = slice(r * TOKENS, (r + 1) * TOKENS)
        xd, rd, gd, kd = x[mine].cuda(), res[mine].cuda(), g[mine].cuda(), keep[mine].cuda()
        y, total = lib.norm(xd, gaind, residual=rd, eps=EPS)
        logits = y @ wrd
        chosen, weights, counts, sums = lib.route(logits, TOPK, keep=kd)
        rows, place, offsets, _ = lib.dispatch(y, chosen, EXPERTS)
        at = offsets.tolist()
        assert at[EXPERTS] == int(kd.sum()) * TOPK and torch.equal(offsets[1:] - offsets[:-1], counts[:EXPERTS])
        done = torch.zeros_like(rows)
        for e in range(EXPERTS):
            done[at[e]:at[e + 1]] = rows[at[e]:at[e + 1]] @ wed[e]
        outs.append(total + lib.combine(done, place, weights))
        # backward
        drows, dweights = lib.combine_grad(gd, done, place, weights)
        drows[at[EXPERTS]:] = 0  # (not written)
        dwe, back = torch.zeros_like(wed), torch.zeros_like(drows)
        for e in range(EXPERTS):
            part = slice(at[e], at[e + 1])
            dwe[e] = rows[part].t() @ drows[part]
            back[part] = drows[part] @ wed[e].t()
        _, dlogits = lib.route_grad(logits, chosen, dweights, keep=kd)
        dy = lib.dispatch_grad(back, place) + dlogits @ wrd.t()
        dx, dgain = lib.norm_grad(total, gaind, dy, dtotal=gd, eps=EPS)
        dense.append([dgain, y.t() @ dlogits])
        experts.append(dwe)
        dxs.append(dx)
        chosens.append(chosen.cpu())
    out, dx, dgain, dwr, dwe = reference(x, res, gain, wr, we, g, torch.cat(chosens), keep)
    near(torch.cat(outs), out, "out")
    near(torch.cat(dxs), dx, "dx")
    # every rank: the dense gradients' sum, and the sum of the experts that are its own
    for i, want in enumerate((dgain, dwr)):
        lib.allreduce([d[i] for d in dense])
        near(dense[0][i], want, "reduced")
    each = EXPERTS // RANKS
    own = [torch.empty(each, COLS, COLS, device="cuda") for _ in range(RANKS)]
    lib.reduce_scatter(experts, own)
    near(torch.cat(own), dwe, "experts")
    # the experts' norm over all ranks, the dense gradients' on each; both clipped
    total = dwe.norm()
    gathered = [torch.empty(RANKS, device="cuda") for _ in range(RANKS)]
    before = [o.clone() for o in own]

    def clip():
        lib.all_gather([lib.grad_norm([o]) for o in own], gathered)
        return ([lib.clip_grads([o], total.item() / 2, parts=p) for o, p in zip(own, gathered)],
                [lib.clip_grads(d, 1e6) for d in dense])

    if captured:
        clip()  # (the collectives' first calls allocate)
        for o, b in zip(own, before):
            o.copy_(b)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            norms, whole = clip()
        for _ in range(3):
            for o, b in zip(own, before):
                o.copy_(b)
            graph.replay()
            torch.cuda.synchronize()
            near(torch.cat(own), dwe / 2, "clipped")
    else:
        norms, whole = clip()
    near(torch.cat(own), dwe / 2, "clipped")
    for n, w, d in zip(norms, whole, dense):
        near(n, total.reshape(1), "norm")
        near(w, torch.stack([dgain.norm(), dwr.norm()]).norm().reshape(1), "dense norm")
        near(d[0], dgain, "not clipped")


def test_8_bit_activations_to_their_experts(lib):
    """The norm's e4m3 rows and scales, dispatched, are the token's own."""
    x = torch.randn(300, 700, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    chosen = torch.randint(-1, 12, (300, 4), generator=torch.Generator().manual_seed(4), dtype=torch.int32).cuda()
    q, scales, _ = lib.norm_quant(x)
    rows, place, offsets, row_scales = lib.dispatch(q, chosen, 12, scales=scales)
    y, _ = lib.norm(x)
    n = int(offsets[12])
    full = place.reshape(-1) >= 0
    at, token = place.reshape(-1)[full].long(), torch.arange(1200, device="cuda")[full] // 4
    assert n == int(full.sum()) and torch.equal(rows.view(torch.uint8)[at], q.view(torch.uint8)[token])
    assert torch.equal(row_scales[at], scales[token])
    # as numbers: within e4m3's and bf16's roundings, or half of e4m3's smallest step of the group's scale
    whole = (rows[at].float() * row_scales[at].repeat_interleave(128, 1)[:, :700]).double()
    want = y[token].double()
    tol = want.abs() * (2.0 ** -4 + 2.0 ** -8 + 2.0 ** -11) + 2.0 ** -10 * row_scales[at].repeat_interleave(128, 1)[:, :700].double()
    assert ((whole - want).abs() <= tol).all()
