"""The operators around an expert layer as measured work: listed and drawn
cases, their inputs, one pass through each operator, and what a pass has to
read, write and compute.

  norm          root-mean-square norm of activation plus residual; the sum, and
                the norm in the activations' type or in e4m3 with a scale for
                each group of columns
  norm_grad     its gradient: for the sum (with the residual path's own
                gradient added) and for the gain
  dispatch      tokens sorted by their experts: the place of each (token,
                slot), where each expert's rows start, the rows themselves
  combine       the experts' rows back to their tokens, weighted (without
                weights: the gradient of dispatch)
  combine_grad  the gradient of combine for the rows and the weights
  clip          the norm over all gradients, and the gradients scaled down to
                a largest norm

With `own` false, run() computes them in plain torch operations in 32 bits;
with `own` true it calls the library.
"""
from __future__ import annotations

import torch

own = False

DTYPES = {"fp32": torch.float32, "fp16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
BYTES = {"fp32": 4, "fp16": 2, "bf16": 2, "e4m3": 1}
E4M3_MAX = 448.0
EPS = 1e-6


# ---- cases -----------------------------------------------------------------------
def listed():
    return [
        # the all-reduced activation of one decoded token, on its way into the experts in 8 bits: latency alone
        dict(name="norm_one", op="norm", rows=1, cols=8192, dtype="bf16", residual=True, group=128, gap=0),
        # a long prompt or a training batch of the same activations
        dict(name="norm_batch", op="norm", rows=16384, cols=8192, dtype="bf16", residual=True, group=128, gap=0),
        # fp32 activations of an odd width, column slices of a wider buffer, no residual path
        dict(name="norm_grad_ragged", op="norm_grad", rows=1003, cols=2261, dtype="fp32", residual=False, gap=27),
        # the backward pass of a training batch
        dict(name="norm_grad_batch", op="norm_grad", rows=16384, cols=8192, dtype="bf16", residual=True, gap=0),
        # one decoded token to its eight experts
        dict(name="dispatch_one", op="dispatch", tokens=1, cols=8192, experts=256, topk=8, dtype="bf16", group=0, empty=0.0),
        # a batch of 8-bit activations with their scales
        dict(name="dispatch_batch", op="dispatch", tokens=16384, cols=4096, experts=256, topk=8, dtype="e4m3", group=128, empty=0.0),
        # half precision, padding tokens without experts; without weights, as in the backward pass of a dispatch
        dict(name="combine_ragged", op="combine", tokens=1003, cols=1501, experts=60, topk=4, dtype="fp16", weighted=False, empty=0.1),
        # the experts' outputs of a batch
        dict(name="combine_batch", op="combine", tokens=16384, cols=4096, experts=256, topk=8, dtype="bf16", weighted=True, empty=0.0),
        # few tokens, fp32, padding among them
        dict(name="combine_grad_ragged", op="combine_grad", tokens=333, cols=2263, experts=60, topk=6, dtype="fp32", empty=0.2),
        # the backward pass of a batch
        dict(name="combine_grad_batch", op="combine_grad", tokens=16384, cols=4096, experts=256, topk=8, dtype="bf16", empty=0.0),
        # one small layer, odd sizes, nothing to clip
        dict(name="clip_small", op="clip", layers=1, hidden=509, inner=1021, dtype="fp16", over=0.5),
        # four large layers: 16-bit matrices beside fp32 gains
        dict(name="clip_batch", op="clip", layers=4, hidden=4096, inner=11008, dtype="bf16", over=3.0),
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))

    op = rng.choice(("norm", "norm_grad", "dispatch", "combine", "combine_grad", "clip"))
    dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
    if op == "clip":
        hidden = log(64, 4096)
        return dict(op=op, layers=rng.randint(1, 2 if dtype == "fp32" else 4), hidden=hidden, inner=log(hidden, min(4 * hidden, 8192)), dtype=dtype,
                    over=rng.choice((0.5, 1.5, 10.0)))
    if op in ("norm", "norm_grad"):
        cols = log(64, 16384)
        case = dict(op=op, rows=log(1, min(16384, (1 << 26) // cols)), cols=cols, dtype=dtype, residual=rng.random() < 0.7,
                    gap=rng.choice((0, 0, 1, 64)))
        if op == "norm":
            case["group"] = rng.choice((0, 32, 64, 128, cols))  # 0: in the activations' type; cols: a scale for a row
        return case
    if op == "dispatch":
        dtype = rng.choice(("bf16", "fp16", "fp32", "e4m3"))
    experts = log(4, 512)
    topk, cols = rng.randint(1, min(16, experts // 2)), log(64, 8192)
    case = dict(op=op, tokens=log(1, max(1, min(16384, (1 << 28) // (topk * cols)))), cols=cols, experts=experts, topk=topk, dtype=dtype,
                empty=rng.choice((0.0, 0.1, 0.5)))
    if op == "dispatch":
        case["group"] = 128 if dtype == "e4m3" else 0
    if op == "combine":
        case["weighted"] = rng.random() < 0.7
    return case


def groups(case):
    """Scales of a row."""
    return -(-case["cols"] // case["group"]) if case["group"] else 0


def shapes(case):
    """A layer's matrices and its two gains, all layers."""
    h, i = case["hidden"], case["inner"]
    return [(h, h)] * 4 + [(h, i)] * 2 + [(i, h)], [(h,)] * 2


def work(case):
    es, op = BYTES[case["dtype"]], case["op"]
    if op == "clip":
        mats, gains = shapes(case)
        n, m = sum(a * b for a, b in mats) * case["layers"], sum(a for a, in gains) * case["layers"]
        return {"bytes": 2 * (n * es + m * 4) + 4, "flops": 3 * (n + m)}
    if op in ("norm", "norm_grad"):
        n = case["rows"] * case["cols"]
        if op == "norm":
            out = n + 4 * case["rows"] * groups(case) if case["group"] else n * es
            return {"bytes": n * es * (3 if case["residual"] else 1) + out + 4 * case["cols"], "flops": 6 * n}
        return {"bytes": n * es * (4 if case["residual"] else 3) + 8 * case["cols"], "flops": 10 * n}
    # (on average; the empty slots are drawn with the inputs)
    t, k, row = case["tokens"], case["topk"], case["cols"] * es
    slots = t * k * (1.0 - case["empty"])
    if op == "dispatch":
        row += 4 * groups(case)
        return {"bytes": t * row + slots * row + 8 * t * k + 4 * (case["experts"] + 1), "flops": 0}
    if op == "combine":
        return {"bytes": t * row + slots * row + (8 if case["weighted"] else 4) * t * k, "flops": 2 * slots * case["cols"]}
    return {"bytes": t * row + 2 * slots * row + 12 * t * k, "flops": 3 * slots * case["cols"]}


# ---- inputs ----------------------------------------------------------------------
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device=dev)

    def uniform(*shape):
        return torch.rand(shape, generator=gen, device=dev)

    op, dt = case["op"], DTYPES[case["dtype"]]
    scale = 1024.0 if case["dtype"] == "fp16" else 1.0  # half-precision training runs under a loss scale
    s = {"case": case}
    if op == "clip":
        mats, gains = shapes(case)
        s["cuts"] = [(a * b, (a, b)) for _ in range(case["layers"]) for a, b in mats], [(a, (a,)) for _ in range(case["layers"]) for a, in gains]
        # gradients lie in one buffer per type, as an all-reduce over the ranks leaves them
        flat = [torch.empty(sum(n for n, _ in cut), dtype=t, device=dev) for cut, t in zip(s["cuts"], (dt, torch.float32))]
        for f in flat:
            f.normal_(0.0, 1.0, generator=gen).mul_(0.01)
        s["max_norm"] = 0.01 * sum(f.numel() for f in flat) ** 0.5 / case["over"]
        s["flat_out"] = [torch.zeros_like(f) for f in flat]
        s["grads"], s["out"] = ([p.view(shape) for f, cut in zip(buffers, s["cuts"]) for p, (_, shape) in zip(f.split([n for n, _ in cut]), cut)]
                                for buffers in (flat, s["flat_out"]))
        s["norm"] = torch.empty(1, device=dev)
        return s

    def matrix(rows, cols, factor=1.0):
        wide = torch.zeros(rows, cols + case.get("gap", 0), dtype=dt, device=dev)
        wide[:, :cols] = normal(rows, cols) * factor
        return wide[:, :cols]

    if op in ("norm", "norm_grad"):
        n, c = case["rows"], case["cols"]
        s["gain"] = (1.0 + 0.2 * normal(c)).to(dt)
        # some columns are far larger than the others, as in trained models
        loud = 1.0 + 20.0 * (uniform(c) < 0.003)
        if op == "norm":
            s["x"] = matrix(n, c, 0.5)
            s["residual"] = matrix(n, c, loud) if case["residual"] else None
            total = torch.empty(n, c, dtype=dt, device=dev) if case["residual"] else None
            if case["group"]:
                s["out"] = (torch.empty(n, c, dtype=DTYPES["e4m3"], device=dev), torch.empty(n, groups(case), device=dev), total)
            else:
                s["out"] = (torch.empty(n, c, dtype=dt, device=dev), total)
            return s
        s["total"] = matrix(n, c, loud)
        s["dout"] = matrix(n, c, scale / max(1, n) ** 0.5)
        s["dtotal"] = matrix(n, c, scale / max(1, n) ** 0.5) if case["residual"] else None
        s["out"] = (torch.empty(n, c, dtype=dt, device=dev), torch.empty(c, device=dev))
        return s

    t, k, e, c = case["tokens"], case["topk"], case["experts"], case["cols"]
    # some experts are liked more than others; padding tokens have none
    chosen = torch.topk(normal(t, e) + 0.7 * normal(e), k, dim=1).indices.int()
    chosen[uniform(t) < case["empty"]] = -1
    if op == "dispatch":
        x = normal(t, c)
        s["chosen"] = chosen
        s["x"] = (60.0 * x).clamp(-E4M3_MAX, E4M3_MAX).to(dt) if case["dtype"] == "e4m3" else x.to(dt)
        s["scales"] = 0.01 + uniform(t, groups(case)) if case["group"] else None
        s["out"] = (torch.zeros(t * k, c, dtype=torch.uint8 if case["dtype"] == "e4m3" else dt, device=dev).view(dt),
                    torch.empty(t, k, dtype=torch.int32, device=dev), torch.empty(e + 1, dtype=torch.int32, device=dev),
                    torch.zeros(t * k, groups(case), device=dev) if case["group"] else None)
        return s
    s["place"] = _places(chosen, e)[0]
    s["rows"] = normal(t * k, c).to(dt)
    w = uniform(t, k) + 0.05
    s["weights"] = w / w.sum(1, keepdim=True) if case.get("weighted", True) else None
    if op == "combine":
        s["out"] = torch.empty(t, c, dtype=dt, device=dev)
        return s
    s["dout"] = (normal(t, c) * scale / max(1, t) ** 0.5).to(dt)
    s["out"] = (torch.zeros(t * k, c, dtype=dt, device=dev), torch.empty(t, k, device=dev))
    return s


# ---- plain forms -----------------------------------------------------------------
def _norm(x, residual, gain, group, eps):
    h = x.float() if residual is None else x.float() + residual.float()
    r = torch.rsqrt(h.square().mean(1, keepdim=True) + eps)
    y = h * r * gain.float()
    total = None if residual is None else h.to(x.dtype)
    if not group:
        return y.to(x.dtype), total
    n, c = y.shape
    g = -(-c // group)
    y = torch.nn.functional.pad(y, (0, g * group - c)).view(n, g, group)
    scales = y.abs().amax(2) / E4M3_MAX
    q = torch.where(scales[:, :, None] > 0, y / scales[:, :, None], y)
    return q.view(n, g * group)[:, :c].to(DTYPES["e4m3"]), scales, total


def _norm_grad(total, gain, dout, dtotal, eps):
    h, d, g = total.float(), dout.float(), gain.float()
    r = torch.rsqrt(h.square().mean(1, keepdim=True) + eps)
    u = h * r
    dg = d * g
    dx = r * (dg - u * (dg * u).mean(1, keepdim=True))
    if dtotal is not None:
        dx = dx + dtotal.float()
    return dx.to(total.dtype), (d * u).sum(0)


def _places(chosen, experts):
    t, k = chosen.shape
    flat = chosen.reshape(-1).long()
    valid = (flat >= 0) & (flat < experts)
    key = torch.where(valid, flat, experts)
    order = torch.sort(key, stable=True).indices
    at = torch.empty_like(order).scatter_(0, order, torch.arange(t * k, device=order.device))
    counts = torch.zeros(experts + 1, dtype=torch.int64, device=flat.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.cumsum(counts, 0) - counts
    return torch.where(valid, at, -1).view(t, k).int(), offsets.int()


def _dispatch(x, scales, chosen, experts):
    t, k = chosen.shape
    place, offsets = _places(chosen, experts)
    at = torch.where(place >= 0, place, t * k).reshape(-1).long()
    from_token = torch.arange(t, device=x.device).repeat_interleave(k)

    def move(m):
        out = torch.zeros(t * k + 1, m.shape[1], dtype=m.dtype, device=m.device)
        return out.index_copy_(0, at, m[from_token])[:t * k]

    rows = move(x.view(torch.uint8)).view(x.dtype) if x.dtype == DTYPES["e4m3"] else move(x)
    return rows, place, offsets, None if scales is None else move(scales)


def _combine(rows, place, weights):
    full = place >= 0
    got = rows[place.clamp(min=0).long()].float()
    w = full.float() if weights is None else torch.where(full, weights, 0.0)
    return torch.where(full[:, :, None], got * w[:, :, None], 0.0).sum(1).to(rows.dtype)


def _combine_grad(dout, rows, place, weights):
    full = place >= 0
    t, k = place.shape
    d = dout.float()
    dw = torch.where(full, (rows[place.clamp(min=0).long()].float() * d[:, None]).sum(2), 0.0)
    at = torch.where(full, place, rows.shape[0]).reshape(-1).long()
    out = torch.zeros(rows.shape[0] + 1, rows.shape[1], dtype=rows.dtype, device=rows.device)
    out.index_copy_(0, at, (d[:, None] * weights[:, :, None]).to(rows.dtype).view(t * k, -1))
    return out[:-1], dw


def _clip(grads, cuts, max_norm):
    # the squares of a tensor in 32 bits, all tensors' together in 64
    norm = torch.stack([g.float().square().sum() for g in grads]).double().sum().sqrt()
    coef = torch.clamp(max_norm / norm, max=1.0).float()
    scaled = [(g.float() * coef).to(g.dtype).reshape(-1) for g in grads]
    n = len(cuts[0])
    return norm.float().reshape(1), torch.cat(scaled[:n]), torch.cat(scaled[n:])


# ---- one pass --------------------------------------------------------------------
_library = None


def _sim():
    global _library
    if _library is None:
        import all_reduce_reduction_amd
        all_reduce_reduction_amd.sim_init(0)
        _library = all_reduce_reduction_amd
    return _library


def run(s):
    case = s["case"]
    op = case["op"]
    if op == "norm":
        if own and case["group"]:
            return _sim().norm_quant(s["x"], s["gain"], residual=s["residual"], eps=EPS, group=case["group"], out=s["out"])
        if own:
            return _sim().norm(s["x"], s["gain"], residual=s["residual"], eps=EPS, out=s["out"])
        return _norm(s["x"], s["residual"], s["gain"], case["group"], EPS)
    if op == "norm_grad":
        if own:
            return _sim().norm_grad(s["total"], s["gain"], s["dout"], dtotal=s["dtotal"], eps=EPS, out=s["out"])
        return _norm_grad(s["total"], s["gain"], s["dout"], s["dtotal"], EPS)
    if op == "dispatch":
        if own:
            return _sim().dispatch(s["x"], s["chosen"], case["experts"], scales=s["scales"], out=s["out"])
        return _dispatch(s["x"], s["scales"], s["chosen"], case["experts"])
    if op == "combine":
        if own:
            return _sim().combine(s["rows"], s["place"], s["weights"], out=s["out"])
        return _combine(s["rows"], s["place"], s["weights"])
    if op == "combine_grad":
        if own:
            return _sim().combine_grad(s["dout"], s["rows"], s["place"], s["weights"], out=s["out"])
        return _combine_grad(s["dout"], s["rows"], s["place"], s["weights"])
    if own:
        return [_sim().clip_grads(s["grads"], s["max_norm"], out=s["out"], norm=s["norm"])] + s["flat_out"]
    return list(_clip(s["grads"], s["cuts"], s["max_norm"]))


# ---- the definition in 64 bits ---------------------------------------------------
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        got = [_exact_norm(s, slice(a, a + 2048)) for a in range(0, case["rows"], 2048)]
        return [None if p[0] is None else torch.cat(p) for p in zip(*got)]
    if op == "norm_grad":
        parts = [_exact_norm_grad(s, slice(a, a + 2048)) for a in range(0, case["rows"], 2048)]
        return torch.cat([p[0] for p in parts]), torch.stack([p[1] for p in parts]).sum(0)
    if op == "dispatch":
        # each pair's place by counting, for the pairs of one expert at a time
        t, k = s["chosen"].shape
        flat = s["chosen"].reshape(-1)
        place = torch.full((t * k,), -1, dtype=torch.int32, device=flat.device)
        rows = torch.zeros(t * k, case["cols"], dtype=torch.float64, device=flat.device)
        scales = torch.zeros(t * k, groups(case), device=flat.device) if case["group"] else None
        offsets, start = [], 0
        for e in range(case["experts"]):
            mine = torch.nonzero(flat == e).reshape(-1)
            end = start + mine.numel()
            place[mine] = torch.arange(start, end, dtype=torch.int32, device=flat.device)
            rows[start:end] = s["x"].view(torch.uint8)[mine // k].view(DTYPES["e4m3"]).double() if case["dtype"] == "e4m3" else s["x"][mine // k].double()
            if scales is not None:
                scales[start:end] = s["scales"][mine // k]
            offsets.append(start)
            start = end
        return rows, place.view(t, k), torch.tensor(offsets + [start], dtype=torch.int32), None if scales is None else scales.double()
    if op == "clip":
        squares = sum(torch.dot(v, v) for g in s["grads"] for v in [g.double().reshape(-1)])
        norm = torch.sqrt(squares)
        factor = min(1.0, s["max_norm"] / norm.item())
        n = len(s["cuts"][0])
        flat = [torch.cat([g.reshape(-1) for g in part]).double().mul_(factor) for part in (s["grads"][:n], s["grads"][n:])]
        return [norm.reshape(1)] + flat
    t, k = s["place"].shape
    rows, place = s["rows"], s["place"].long()
    y = torch.zeros(t, case["cols"], dtype=torch.float64, device=rows.device)
    drows = torch.zeros(rows.shape, dtype=torch.float64, device=rows.device) if op == "combine_grad" else None
    dw = torch.zeros(t, k, dtype=torch.float64, device=rows.device)
    for j in range(k):
        some = torch.nonzero(place[:, j] >= 0).reshape(-1)
        at = place[some, j]
        w = torch.ones(some.numel(), 1, dtype=torch.float64, device=rows.device) if s["weights"] is None else s["weights"][some, j, None].double()
        part = rows[at].double()
        if op == "combine":
            y.index_add_(0, some, w * part)
        else:
            d = s["dout"][some].double()
            dw[some, j] = torch.linalg.vecdot(d, part)
            drows[at] = w * d
    return y if op == "combine" else (drows, dw)


def _exact_norm(s, rows):
    case, x = s["case"], s["x"][rows].double()
    h = x if s["residual"] is None else x + s["residual"][rows].double()
    y = h / torch.sqrt((h * h).sum(1, keepdim=True) / case["cols"] + EPS) * s["gain"].double()
    total = None if s["residual"] is None else h
    if not case["group"]:
        return y, total
    parts = y.split(case["group"], 1)
    top = torch.stack([p.abs().max(1).values for p in parts], 1)
    q = torch.cat([p * (E4M3_MAX / m[:, None].clamp(min=1e-300)) for p, m in zip(parts, top.unbind(1))], 1)
    return q, top / E4M3_MAX, total


def _exact_norm_grad(s, rows):
    h, d, g = s["total"][rows].double(), s["dout"][rows].double(), s["gain"].double()
    inv = 1.0 / torch.sqrt((h * h).sum(1, keepdim=True) / s["case"]["cols"] + EPS)
    dot = (d * g * h).sum(1, keepdim=True) / s["case"]["cols"]
    dx = inv * d * g - inv ** 3 * dot * h
    if s["dtotal"] is not None:
        dx = dx + s["dtotal"][rows].double()
    return dx, (d * h * inv).sum(0)
