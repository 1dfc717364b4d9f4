"""Distillation from a teacher's top logits against its formulas in 64 bits:
whole rows and vocabulary shards, ragged sizes, empty rows, infinities and
NaN, strides, streams, graphs, refusals."""
import pytest
import torch

from tests import loss_oracle as oracle

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.float16, torch.bfloat16]
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def lib():
    import all_reduce_reduction_amd as sim
    sim.sim_init(0, 16, 0)
    yield sim


def case(t, v, k, dtype, tdtype, seed, holes=True):
    g = torch.Generator().manual_seed(seed)
    x = 2.0 * torch.randn(t, v, generator=g)
    ids = torch.randint(0, v, (t, k), generator=g, dtype=torch.int32)  # the same id may come twice
    z = 6.0 * torch.rand(t, k, generator=g)
    x.scatter_add_(1, ids.long(), 0.5 * z)
    if holes and k > 1:
        ids[torch.rand(t, k, generator=g) < 0.2] = -1
    if holes and t > 3:
        ids[t // 2] = -1
    return x.to(dtype), ids, z.to(tdtype), torch.rand(t, generator=g) + 0.5


def check(x, ids, z, tau, scale, coef, loss, d, what=""):
    want, ltol, dwant, dtol = oracle.distill(x, ids, z, tau, scale, coef)
    oracle.assert_within(loss, want, ltol, what + " loss")
    oracle.assert_within(d, dwant, oracle.rounded(dtol, dwant, x.dtype), what + " dlogits")


def step(sim, x, ids, z, tau=1.0, scale=None, coef=1.0, xd=None, **kw):
    xd = x.cuda() if xd is None else xd
    return sim.distill_step(xd, ids.cuda(), z.cuda(), temperature=tau, coef=coef,
                            row_scale=None if scale is None else scale.cuda(), **kw)


SIZES = [(1, 1, 1), (1, 7, 3), (1, 32768, 32), (2, 50021, 256), (5, 1000, 8), (33, 4097, 64), (700, 1003, 20),
         (600, 8192, 65), (3, 131072, 64), (513, 2050, 1), (300, 16385, 7), (1, 200003, 128), (520, 65, 130)]


@pytest.mark.parametrize("t,v,k", SIZES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_step_sizes(lib, t, v, k, dtype):
    tau = (1.0, 2.0, 0.7)[k % 3]
    x, ids, z, scale = case(t, v, k, dtype, (torch.float32, dtype)[t % 2], t + v)
    coef = 4096.0 if dtype == torch.float16 else 0.25
    scale = scale / t
    loss, d = step(lib, x, ids, z, tau, scale, coef)
    check(x, ids, z, tau, scale, coef, loss, d)


@pytest.mark.parametrize("v", [30011, 65536, 70000, 131072, 131080, 140001])
@pytest.mark.parametrize("dtype", DTYPES)
def test_step_long_rows(lib, v, dtype):
    """Enough rows that one workgroup takes a row, on both sides of every length at which a row is held otherwise."""
    t = 520
    x, ids, z, scale = case(8, v, 40, dtype, torch.float32, v)
    pick = torch.arange(t) % 8
    loss, d = lib.distill_step(x.cuda()[pick.cuda()], ids.cuda()[pick.cuda()], z.cuda()[pick.cuda()], coef=512.0)
    check(x, ids, z, 1.0, None, 512.0, loss[:8], d[:8])
    for r in range(8, t, 8):
        n = min(8, t - r)
        assert torch.equal(d[r:r + n], d[:n]) and torch.equal(loss[r:r + n], loss[:n])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t", [12, 600])
def test_empty_rows_and_special_values(lib, dtype, t):
    v, k = 3001, 9
    x, ids, z, scale = case(t, v, k, dtype, torch.float32, 77, holes=False)
    ids[0] = -1                       # no slot: nothing of the row counts
    x[0] = NAN
    ids[1] = v + 5                    # ids outside the vocabulary are empty slots
    x[1] = INF
    z[2] = -INF                       # a teacher without mass
    z[3, 1:] = -INF                   # all mass on one slot
    ids[4, 3:] = -2
    z[4, 3:] = NAN                    # empty slots hold anything
    x[5, 100:] = -INF                 # columns that are switched off
    ids[5] = torch.arange(k)
    x[6] = -INF                       # no finite logit: NaN
    x[7, 12] = NAN
    x[8, 13] = INF
    x[9, ids[9, 0].long()] = -INF     # the teacher asks for a column that is switched off
    z[10, 2] = NAN                    # a teacher's NaN stays in its row
    x[11] = torch.finfo(dtype).min    # the type's lowest value is a logit like any other
    x[11, 5] = torch.finfo(dtype).min / 2
    for tau in (1.0, 3.0):
        loss, d = step(lib, x, ids, z, tau, scale, 2.0)
        check(x, ids, z, tau, scale, 2.0, loss, d)
    assert torch.equal(loss[:3].cpu(), torch.zeros(3)) and not d[:3].any()
    assert torch.isinf(loss[9]) and torch.isnan(loss[[6, 7, 8, 10]]).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t", [5, 600])
def test_logits_at_the_ends_of_the_type(lib, dtype, t):
    """Rows whose logits are all so large that logit / temperature overflows, beside ordinary ones."""
    v, k = 2100, 7
    x, ids, z, _ = case(t, v, k, dtype, torch.float32, 78, holes=False)
    low, high = torch.finfo(dtype).min, torch.finfo(dtype).max
    x[0] = low                    # masked everywhere: the softmax is even
    x[1] = high
    x[2, :v - 50] = low           # masked by the type's lowest value, ordinary elsewhere
    x[3, 40:] = low
    x[3, :40] = -INF
    x[4, 100] = high
    ids[2, 0] = v - 1
    for tau in (1.0, 0.25, 1e-3):
        loss, d = step(lib, x, ids, z, tau)
        check(x, ids, z, tau, None, 1.0, loss, d, f"tau {tau}")
        loss, d, _ = shards(lib, x, ids, z, tau, None, 1.0, 2)
        check(x, ids, z, tau, None, 1.0, loss, d, f"shards, tau {tau}")


def test_repeated_ids_add_up(lib):
    x, ids, z, _ = case(40, 500, 16, torch.float32, torch.float32, 5, holes=False)
    ids[:, 8:] = ids[:, :8]
    ids[7] = 3
    loss, d = step(lib, x, ids, z)
    check(x, ids, z, 1.0, None, 1.0, loss, d)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,v,first,wide", [(6, 9000, 1, 9011), (530, 1234, 3, 1301), (530, 40001, 5, 40013),
                                            (4, 33333, 0, 33333)])
def test_column_slices(lib, dtype, t, v, first, wide):
    """Rows at any alignment, the gradient at another."""
    x, ids, z, scale = case(t, v, 12, dtype, dtype, 21)
    big = torch.full((t, wide), 5.0, dtype=dtype, device="cuda")
    part = big[:, first:first + v]
    part.copy_(x)
    out = torch.full((t, wide + 3), 7.0, dtype=dtype, device="cuda")
    loss, d = step(lib, x, ids, z, 1.0, scale, 64.0, xd=part,
                   out=(torch.empty(t, device="cuda"), out[:, 2:2 + v]))
    check(x, ids, z, 1.0, scale, 64.0, loss, d)
    assert (out[:, :2] == 7).all() and (out[:, 2 + v:] == 7).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,v", [(3, 20011), (600, 5003), (520, 66000), (260, 131072)])
def test_in_place(lib, dtype, t, v):
    x, ids, z, scale = case(t, v, 33, dtype, torch.float32, 22)
    want = step(lib, x, ids, z, 1.0, scale, 16.0)
    y = x.cuda()
    got = step(lib, x, ids, z, 1.0, scale, 16.0, xd=y, out=(torch.empty(t, device="cuda"), y))
    assert torch.equal(got[0], want[0]) and torch.equal(y, want[1])


def shards(sim, x, ids, z, tau, scale, coef, p, even=False):
    v, t = x.shape[1], x.shape[0]
    cut = [r * v // p for r in range(p + 1)]
    xs = [x[:, a:b].contiguous().cuda() for a, b in zip(cut, cut[1:])]
    i, y = ids.cuda(), z.cuda()
    parts = [sim.distill_parts(s, i, y, temperature=tau, first=a, vocab=v) for s, a in zip(xs, cut)]
    if p > 1:
        gathered = [torch.empty(p, 4, t, device="cuda") for _ in range(p)]
        sim.all_gather(parts, gathered)
    else:
        gathered = [parts[0][None]]
    joined = [sim.distill_join(g, i, y, temperature=tau, vocab=v) for g in gathered]
    for loss, norm in joined[1:]:
        assert torch.equal(loss.nan_to_num(9.0), joined[0][0].nan_to_num(9.0))
    sc = None if scale is None else scale.cuda()
    d = [sim.distill_grad(s, i, y, n, temperature=tau, row_scale=sc, coef=coef, first=a, vocab=v)
         for s, a, (_, n) in zip(xs, cut, joined)]
    return joined[0][0], torch.cat(d, 1), parts


@pytest.mark.parametrize("p", [1, 2, 3, 8])
@pytest.mark.parametrize("t,v,k", [(1, 40, 5), (9, 4001, 30), (530, 1003, 17), (4, 100003, 200)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_shards(lib, p, t, v, k, dtype):
    tau = 1.5 if t % 2 else 1.0
    x, ids, z, scale = case(t, v, k, dtype, (dtype, torch.float32)[t % 2], 31)
    loss, d, _ = shards(lib, x, ids, z, tau, scale, 1024.0, p)
    check(x, ids, z, tau, scale, 1024.0, loss, d)


def test_shards_with_special_values(lib):
    t, v, k = 8, 900, 6
    x, ids, z, _ = case(t, v, k, torch.float32, torch.float32, 32, holes=False)
    x[0, :450] = -INF            # one shard has nothing, and a slot in it
    ids[0, 0] = 5
    x[1, :300] = -INF            # one shard has nothing, and no slot in it
    ids[1] = torch.arange(500, 500 + k)
    x[2] = -INF
    x[3, 700] = NAN
    x[4, 2] = INF
    ids[5] = -1
    x[5] = NAN
    loss, d, parts = shards(lib, x, ids, z, 1.0, None, 1.0, 3)
    check(x, ids, z, 1.0, None, 1.0, loss, d)
    assert torch.isinf(loss[0]) and loss[5] == 0


def test_parts_hold_what_they_say(lib):
    t, v, first, total = 21, 5000, 700, 9000
    x, _, z, _ = case(t, v, 11, torch.float32, torch.float32, 33)
    ids = torch.randint(-50, total + 50, (t, 11), generator=torch.Generator().manual_seed(1), dtype=torch.int32)
    tau = 2.0
    got = lib.distill_parts(x.cuda(), ids.cuda(), z.cuda(), temperature=tau, first=first, vocab=total)
    ok, q, _, live = oracle.teacher(ids, z, tau, total)
    assert live.all()
    y = x.double()
    m = y.amax(1)
    here = ok & (ids >= first) & (ids < first + v)
    at = torch.where(here, ids - first, 0).long()
    far = (y.gather(1, at) - m[:, None]) / tau
    s = torch.exp((y - m[:, None]) / tau).sum(1)
    oracle.assert_within(got[0], m, torch.zeros(t), "largest")
    oracle.assert_within(got[1], s, 100 * oracle.U * s, "sum")
    mass = torch.where(here, q, 0.0).sum(1)
    oracle.assert_within(got[2], mass, 100 * oracle.U * torch.ones(t), "mass")
    dot = torch.where(here, q * far, 0.0).sum(1)
    oracle.assert_within(got[3], dot, 100 * oracle.U * (1 + dot.abs()), "dot")


def test_gradient_against_differences(lib):
    t, v, k, tau = 4, 50, 6, 1.3
    x, ids, z, scale = case(t, v, k, torch.float32, torch.float32, 41)
    _, d = step(lib, x, ids, z, tau, scale, 1.0)
    g = torch.Generator().manual_seed(4)
    h = 1e-5
    for _ in range(20):
        w = torch.randn(t, v, generator=g, dtype=torch.float64)
        f = [(oracle.distill_loss(x.double() + s * h * w, ids, z, tau) * scale.double()).sum() for s in (1, -1)]
        slope = (f[0] - f[1]).item() / (2 * h)
        dot = d.cpu().double() * w
        assert abs(slope - dot.sum().item()) <= 1e-5 * dot.abs().sum().item() + 1e-8


def test_the_same_bits_every_time(lib):
    for t, v in ((3, 70001), (600, 9001)):
        x, ids, z, _ = case(t, v, 20, torch.bfloat16, torch.bfloat16, 42)
        a, b = step(lib, x, ids, z), step(lib, x, ids, z)
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("t,v", [(2, 60000), (600, 3001)])
def test_other_stream_and_graph(lib, t, v):
    x, ids, z, _ = case(t, v, 20, torch.bfloat16, torch.float32, 43)
    xd, i, y = x.cuda(), ids.cuda(), z.cuda()
    want = lib.distill_step(xd, i, y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lib.distill_step(xd, i, y, stream=side)
    side.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    out = (torch.empty(t, device="cuda"), torch.empty_like(xd))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.distill_step(xd, i, y, out=out)
    for _ in range(3):
        out[0].zero_()
        out[1].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_offsets_past_32_bits(lib):
    v, rows, ld = 2000, 5, 1 << 30
    big = torch.empty(4 * ld + v, dtype=torch.bfloat16, device="cuda")
    part = big.as_strided((rows, v), (ld, 1))
    x, ids, z, scale = case(rows, v, 9, torch.bfloat16, torch.float32, 44)
    part.copy_(x)
    loss, d = step(lib, x, ids, z, 1.0, scale, 1.0, xd=part, out=(torch.empty(rows, device="cuda"), part))
    check(x, ids, z, 1.0, scale, 1.0, loss, d)


def test_no_rows(lib):
    x = torch.empty(0, 100, dtype=torch.bfloat16, device="cuda")
    i, z = torch.empty(0, 4, dtype=torch.int32, device="cuda"), torch.empty(0, 4, device="cuda")
    loss, d = lib.distill_step(x, i, z)
    parts = lib.distill_parts(x, i, z)
    loss2, norm = lib.distill_join(parts[None], i, z, vocab=100)
    assert lib.distill_grad(x, i, z, norm).shape == (0, 100) and loss.shape == (0,) and loss2.shape == (0,)


def test_refusals(lib):
    t, v, k = 4, 64, 3
    x = torch.zeros(t, v, dtype=torch.bfloat16, device="cuda")
    d = torch.zeros_like(x)
    i = torch.zeros(t, k, dtype=torch.int32, device="cuda")
    z = torch.zeros(t, k, device="cuda")
    loss, norm, parts = torch.zeros(t, device="cuda"), torch.zeros(2, t, device="cuda"), torch.zeros(4, t, device="cuda")
    need = lib.sim_distill_work(t, v, "bf16")
    work = torch.zeros(max(need, 4), dtype=torch.uint8, device="cuda")
    common = dict(dtype="bf16", rows=t, ids=i.data_ptr(), teacher=z.data_ptr(), teacher_dtype="fp32", topk=k,
                  temperature=1.0, stream=0)
    good = dict(common, logits=x.data_ptr(), row_stride=v, vocab=v, row_scale=None, coef=1.0, dlogits=d.data_ptr(),
                drow_stride=v, loss=loss.data_ptr(), work=work.data_ptr(), work_bytes=need)
    assert lib.sim_distill_step(**good) == 0
    for change, status in ((dict(dtype="int32"), -1), (dict(teacher_dtype="int32"), -1), (dict(topk=0), -1),
                           (dict(topk=257), -1), (dict(temperature=0.0), -1), (dict(temperature=-1.0), -1),
                           (dict(temperature=INF), -1), (dict(temperature=NAN), -1), (dict(rows=-1), -1),
                           (dict(vocab=0), -1), (dict(vocab=2 ** 31), -1), (dict(row_stride=v - 1), -1),
                           (dict(drow_stride=v - 1), -1), (dict(logits=None), -1), (dict(ids=None), -1),
                           (dict(loss=None), -1), (dict(logits=x.data_ptr() + 1), -3), (dict(ids=i.data_ptr() + 2), -3),
                           (dict(dlogits=x.data_ptr() + 2), -4), (dict(dlogits=x.data_ptr(), drow_stride=v + 1), -4),
                           (dict(loss=z.data_ptr()), -4), (dict(row_stride=2 ** 60), -1)):
        assert lib.sim_distill_step(**{**good, **change}) == status, change
    if need:
        assert lib.sim_distill_step(**{**good, "work": None}) == -1
        assert lib.sim_distill_step(**{**good, "work_bytes": need - 1}) == -5
    shard = dict(common, logits=x.data_ptr(), row_stride=v, columns=v, first=0, vocab=2 * v)
    part = dict(shard, parts=parts.data_ptr(), work=work.data_ptr(), work_bytes=need)
    assert lib.sim_distill_parts(**part) == 0
    for change, status in ((dict(first=-1), -1), (dict(first=v + 1), -1), (dict(columns=0), -1), (dict(parts=None), -1),
                           (dict(parts=x.data_ptr()), -4)):
        assert lib.sim_distill_parts(**{**part, **change}) == status, change
    join = dict(parts=parts.data_ptr(), nparts=1, rows=t, vocab=v, ids=i.data_ptr(), teacher=z.data_ptr(),
                teacher_dtype="fp32", topk=k, temperature=1.0, loss=loss.data_ptr(), norm=norm.data_ptr(), stream=0)
    assert lib.sim_distill_join(**join) == 0
    for change, status in ((dict(nparts=0), -1), (dict(norm=None), -1), (dict(norm=parts.data_ptr()), -4),
                           (dict(loss=norm.data_ptr()), -4)):
        assert lib.sim_distill_join(**{**join, **change}) == status, change
    grad = dict(shard, norm=norm.data_ptr(), row_scale=None, coef=1.0, dlogits=d.data_ptr(), drow_stride=v)
    assert lib.sim_distill_grad(**grad) == 0
    for change, status in ((dict(norm=None), -1), (dict(dlogits=None), -1), (dict(first=v + 1), -1),
                           (dict(dlogits=x.data_ptr() + 4), -4)):
        assert lib.sim_distill_grad(**{**grad, **change}) == status, change
    with pytest.raises(ValueError):
        lib.distill_step(x.t(), i, z)
    with pytest.raises(ValueError):
        lib.distill_step(x, i.long(), z)
    with pytest.raises(ValueError):
        lib.distill_step(x, i[:2], z[:2])
    with pytest.raises(ValueError):
        lib.distill_step(x, i, z, out=(loss, d[:, :32]))
    with pytest.raises(lib.SimError):
        lib.distill_step(x, i, z, temperature=0.0)
    torch.cuda.synchronize()


def test_both_forms_of_the_tensor_checks_agree(lib):
    """The checks in C and their Python forms return or refuse the same."""
    f32, i32 = (torch.float32,), (torch.int32,)
    x = torch.zeros(6, 40, device="cuda")
    same = [x, x.half(), x.bfloat16(), x[:, 3:9], x[::2], x[:1], x[:0], x[:, :1], x.t(), x[0], x.int(), x.double(), x.cpu(),
            x.view(2, 3, 40), x[:, ::2]]
    ids = torch.zeros(6, 3, dtype=torch.int32, device="cuda")
    rows = [(t, "t", like) for t in same for like in (None, lib._rows_py(x, "x", None))]
    vecs = [(t, "t", f32, 0, *shape) for t in same + [None] for shape in ((6, 40), (6,), (2, 3, 40))]
    slots = [(i, z, i32, n, 0) for i in (ids, ids[:5], ids.long(), ids[0], ids.cpu(), ids[:, :2])
             for z in (ids.float(), ids.half(), ids, ids[:, :2].float(), ids.float().cpu()) for n in (6, 5)]
    for c, py, calls in ((lib._rows, lib._rows_py, rows), (lib._vec, lib._vec_py, vecs), (lib._slots, lib._slots_py, slots)):
        assert c is not py
        for args in calls:
            got = []
            for f in (c, py):
                try:
                    got.append(f(*args))
                except ValueError:
                    got.append("refused")
            assert got[0] == got[1], args


@pytest.mark.parametrize("t", [40, 300])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_step_row_lengths(lib, dtype, t):
    """Every number of vectors per thread that small rows are held in, one column before it, at it and after it."""
    vec = 16 // dtype.itemsize
    lengths = sorted({threads * r * vec + d for threads in (64, 256, 1024) for r in range(1, 9)
                      if threads * r <= 2048 for d in (-1, 0, 1)})
    for v in lengths:
        x, ids, z, scale = case(4, v, 10, dtype, torch.float32, v)
        pick = (torch.arange(t) % 4).cuda()
        loss, d = lib.distill_step(x.cuda()[pick], ids.cuda()[pick], z.cuda()[pick], coef=64.0)
        check(x, ids, z, 1.0, None, 64.0, loss[:4], d[:4], "%d columns" % v)
        assert torch.equal(d.view(-1, 4, v), d[:4].expand(t // 4, 4, v)), v


@pytest.mark.parametrize("t,v", [(3, 70), (300, 3001), (2, 140001)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_many_slots_with_one_id(lib, dtype, t, v):
    """Rows of one id alone, of a few ids many times, and padded with one id of no mass."""
    k = 200
    x, ids, z, scale = case(t, v, k, dtype, torch.float32, 5, holes=False)
    ids[0] = v // 2
    ids[1] = torch.arange(k, dtype=torch.int32) % 3 * (v // 4)
    ids[-1, 20:] = 0
    z[-1, 20:] = -INF
    loss, d = step(lib, x, ids, z, 2.0, scale, 64.0)
    check(x, ids, z, 2.0, scale, 64.0, loss, d)
    again = step(lib, x, ids, z, 2.0, scale, 64.0)
    assert torch.equal(again[0], loss) and torch.equal(again[1], d)
    loss, d, _ = shards(lib, x, ids, z, 2.0, scale, 64.0, 2)
    check(x, ids, z, 2.0, scale, 64.0, loss, d)


@pytest.mark.parametrize("dtype", DTYPES)
def test_shards_of_many_rows(lib, dtype):
    """Short runs of many rows: around every number of chunks of a wave, with odd starts of rows too."""
    t, vec = 1040, 16 // dtype.itemsize
    for n in (1, 2, 8):
        for d in (-1, 0, 1, 33):
            v = 256 * vec * n + d
            x, ids, z, scale = case(8, v, 12, dtype, torch.float32, v)
            pick = torch.arange(t) % 8
            loss, grad, _ = shards(lib, x[pick], ids[pick], z[pick], 1.5, None, 64.0, 2 if d == 33 else 1)
            check(x, ids, z, 1.5, None, 64.0, loss[:8], grad[:8], "%d columns" % v)
            assert torch.equal(grad.view(-1, 8, v), grad[:8].expand(t // 8, 8, v)), v


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t", [6, 600])
def test_logits_at_both_ends_of_the_type(lib, dtype, t):
    """The type's lowest value beside its highest: their distance is past fp32's range, over the temperature it is not."""
    v, k = 2100, 5
    x, ids, z, _ = case(t, v, k, dtype, torch.float32, 79, holes=False)
    low, high = torch.finfo(dtype).min, torch.finfo(dtype).max
    ids[:5] = torch.arange(k, dtype=torch.int32) * 400 + 7
    x[0, 100], x[0, 7] = high, low           # in one shard
    x[1, 2000], x[1, 407] = high, low        # in two
    x[2, :1050], x[2, 2000] = low, high      # a shard of the lowest value alone
    x[3, 1050:], x[3, 3] = low, high
    x[4], x[4, 1:3] = low, high              # all of a row at one end or the other
    for tau in (3.0, 1e4, 1e15):
        loss, d = step(lib, x, ids, z, tau)
        check(x, ids, z, tau, None, 1.0, loss, d, f"tau {tau}")
        assert torch.isfinite(loss).all()
        for p in (2, 3):
            loss, d, _ = shards(lib, x, ids, z, tau, None, 1.0, p)
            check(x, ids, z, tau, None, 1.0, loss, d, f"{p} shards, tau {tau}")


def test_shards_have_to_be_told_the_whole_vocabulary(lib):
    """One shard cannot know which ids are slots of the row: a size of its own would drop those of later shards."""
    x, ids, z, _ = case(6, 90, 4, torch.bfloat16, torch.float32, 80, holes=False)
    ids[:, 0] = 80
    xs, i, y = [x[:, :50].contiguous().cuda(), x[:, 50:].contiguous().cuda()], ids.cuda(), z.cuda()
    parts = lib.distill_parts(xs[0], i, y, vocab=90)
    gathered = torch.stack([parts, lib.distill_parts(xs[1], i, y, first=50, vocab=90)])
    _, norm = lib.distill_join(gathered, i, y, vocab=90)
    for call in (lambda: lib.distill_parts(xs[0], i, y), lambda: lib.distill_parts(xs[1], i, y, first=50),
                 lambda: lib.distill_join(gathered, i, y), lambda: lib.distill_grad(xs[0], i, y, norm)):
        with pytest.raises(ValueError, match="vocab"):
            call()


def test_more_rows_than_a_launch_has_threads_for(lib):
    """Refused as the caller's error, before anything is enqueued; one row fewer runs."""
    t = 1 << 26  # 64 threads a row
    x, d = (torch.zeros(t, 1, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    ids = torch.zeros(t, 1, dtype=torch.int32, device="cuda")
    z = torch.zeros(t, 1, dtype=torch.bfloat16, device="cuda")
    loss = torch.full((t,), 7.0, device="cuda")
    norm = torch.full((2, t), 7.0, device="cuda")
    parts = torch.full((4, t), 7.0, device="cuda")
    need = lib.sim_distill_work(t, 1, "bf16")
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    common = dict(rows=t, vocab=1, ids=ids.data_ptr(), teacher=z.data_ptr(), teacher_dtype="bf16", topk=1, temperature=1.0)
    shard = dict(common, logits=x.data_ptr(), row_stride=1, dtype="bf16", columns=1, first=0)
    step = dict(common, logits=x.data_ptr(), row_stride=1, dtype="bf16", row_scale=None, coef=1.0, dlogits=d.data_ptr(),
                drow_stride=1, loss=loss.data_ptr(), work=work.data_ptr(), work_bytes=need)
    assert lib.sim_distill_step(**step) == -1
    assert lib.sim_distill_parts(**shard, parts=parts.data_ptr(), work=work.data_ptr(), work_bytes=need) == -1
    assert lib.sim_distill_grad(**shard, norm=norm.data_ptr(), row_scale=None, coef=1.0, dlogits=d.data_ptr(),
                                drow_stride=1) == -1
    assert lib.sim_distill_join(**common, parts=parts.data_ptr(), nparts=1, loss=loss.data_ptr(),
                                norm=norm.data_ptr()) == -1
    torch.cuda.synchronize()
    assert (loss == 7).all() and (norm == 7).all() and (parts == 7).all() and not d.any()
    assert lib.sim_distill_step(**{**step, "rows": t - 64}) == 0
    torch.cuda.synchronize()
    assert not loss[:t - 64].any() and (loss[t - 64:] == 7).all()


@pytest.mark.parametrize("dtype", DTYPES)
def test_gradients_into_other_columns_of_the_same_buffer(lib, dtype):
    """Logits and gradient are slices of one wide buffer, side by side, in either order, of several widths."""
    for t, v, gap, wide in ((7, 1001, 0, 2002), (7, 1001, 3, 2010), (300, 333, 1, 700), (1, 40, 0, 80)):
        x, ids, z, scale = case(t, v, 9, dtype, torch.float32, 81)
        for at, to in ((0, v + gap), (v + gap, 0)):
            big = torch.full((t, wide), 7.0, dtype=dtype, device="cuda")
            big[:, at:at + v] = x.cuda()
            part, out = big[:, at:at + v], big[:, to:to + v]
            _, want = step(lib, x, ids, z, 1.0, scale, 16.0, xd=part)
            step(lib, x, ids, z, 1.0, scale, 16.0, xd=part, out=(torch.empty(t, device="cuda"), out))
            assert torch.equal(out, want)
            out.fill_(7.0)
            i, y = ids.cuda(), z.cuda()
            loss, norm = lib.distill_join(lib.distill_parts(part, i, y, vocab=v)[None], i, y, vocab=v)
            lib.distill_grad(part, i, y, norm, row_scale=scale.cuda(), coef=16.0, vocab=v, out=out)
            check(x, ids, z, 1.0, scale, 16.0, loss, out)
            assert torch.equal(part.cpu(), x)
            rest = torch.ones(wide, dtype=torch.bool)
            rest[at:at + v] = rest[to:to + v] = False
            assert (big[:, rest.cuda()] == 7).all()


def test_gradients_into_shared_columns_are_refused(lib):
    big = torch.zeros(5, 200, dtype=torch.bfloat16, device="cuda")
    ids, z = torch.zeros(5, 2, dtype=torch.int32, device="cuda"), torch.zeros(5, 2, device="cuda")
    loss = torch.zeros(5, device="cuda")
    for a, b, shared in ((big[:, :90], big[:, 89:179], True), (big[:, 89:179], big[:, :90], True),
                         (big[:, :90], big[:, 90:180], False), (big[:, 110:], big[:, 19:109], False),
                         (big[:4, 100:190], big[1:, 50:140], True), (big[1:, 50:140], big[:4, 100:190], True),
                         (big[:4, 100:190], big[1:, 10:100], False), (big[1:, 110:200], big[:4, 10:100], False),
                         (big.view(-1)[:900].view(5, 180)[:, :80], big[:, 90:170], True)):  # rows at other distances
        n = a.shape[0]
        call = lambda: lib.distill_step(a, ids[:n], z[:n], out=(loss[:n], b))
        if shared:
            with pytest.raises(lib.SimError):
                call()
        else:
            call()
    torch.cuda.synchronize()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,v,first,wide", [(6, 9000, 1, 9011), (530, 1234, 3, 1301), (530, 20001, 5, 20013),
                                            (1040, 500, 1, 503), (4, 33333, 0, 33333)])
def test_shards_inside_wider_rows(lib, dtype, t, v, first, wide):
    """Shards are column slices of one buffer, at any alignment, their gradients slices of another."""
    x, ids, z, scale = case(t, v, 12, dtype, dtype, 82)
    big = torch.full((t, wide), 5.0, dtype=dtype, device="cuda")
    big[:, first:first + v] = x.cuda()
    out = torch.full((t, wide + 3), 7.0, dtype=dtype, device="cuda")
    i, y, sc = ids.cuda(), z.cuda(), scale.cuda()
    cut = [0, v // 3, v // 3 + 8, v]
    xs = [big[:, first + a:first + b] for a, b in zip(cut, cut[1:])]
    ds = [out[:, 2 + a:2 + b] for a, b in zip(cut, cut[1:])]
    parts = [lib.distill_parts(s, i, y, temperature=1.5, first=a, vocab=v) for s, a in zip(xs, cut)]
    loss, norm = lib.distill_join(torch.stack(parts), i, y, temperature=1.5, vocab=v)
    for s, a, d in zip(xs, cut, ds):
        lib.distill_grad(s, i, y, norm, temperature=1.5, row_scale=sc, coef=64.0, first=a, vocab=v, out=d)
    check(x, ids, z, 1.5, scale, 64.0, loss, out[:, 2:2 + v])
    assert (out[:, :2] == 7).all() and (out[:, 2 + v:] == 7).all()
    for s, a, d in zip(xs, cut, ds):  # over its logits
        lib.distill_grad(s, i, y, norm, temperature=1.5, row_scale=sc, coef=64.0, first=a, vocab=v, out=s)
        assert torch.equal(s, d)
    assert (big[:, :first] == 5).all() and (big[:, first + v:] == 5).all()


def test_shards_with_offsets_past_32_bits(lib):
    v, rows, ld = 2001, 5, (1 << 30) + 1  # rows at either alignment
    big = torch.empty(4 * ld + v, dtype=torch.bfloat16, device="cuda")
    part = big.as_strided((rows, v), (ld, 1))
    x, ids, z, scale = case(rows, v, 9, torch.bfloat16, torch.float32, 83)
    part.copy_(x)
    i, y = ids.cuda(), z.cuda()
    loss, norm = lib.distill_join(lib.distill_parts(part, i, y, vocab=v)[None], i, y, vocab=v)
    lib.distill_grad(part, i, y, norm, row_scale=scale.cuda(), coef=4.0, vocab=v, out=part)
    check(x, ids, z, 1.0, scale, 4.0, loss, part)


@pytest.mark.parametrize("tdtype", DTYPES)
@pytest.mark.parametrize("t", [8, 600])
def test_an_infinite_teacher_stays_in_its_row(lib, tdtype, t):
    v, k = 3001, 9
    x, ids, z, scale = case(t, v, k, torch.bfloat16, tdtype, 84, holes=False)
    z[0, 3] = INF
    z[1] = INF
    z[2, 4], z[2, 5] = INF, -INF
    z[3, 2], z[3, 6] = INF, NAN
    ids[4, 1], z[4, 1] = -1, INF       # an empty slot holds anything
    z[5, :] = -INF
    z[5, 0] = INF
    loss, d = step(lib, x, ids, z, 1.5, scale, 2.0)
    check(x, ids, z, 1.5, scale, 2.0, loss, d)
    assert torch.isnan(loss[[0, 1, 2, 3, 5]]).all() and torch.isfinite(loss[[4, 6, 7]]).all()
    for p in (1, 3):
        loss, d, _ = shards(lib, x, ids, z, 1.5, scale, 2.0, p)
        check(x, ids, z, 1.5, scale, 2.0, loss, d)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t", [6, 600])
def test_a_slot_of_little_mass_on_a_masked_logit(lib, dtype, t):
    """The slot's mass brings a distance over the temperature that is past fp32's range back into it."""
    v, k = 2100, 5
    x, ids, z, _ = case(t, v, k, dtype, torch.float32, 85, holes=False)
    low = torch.finfo(dtype).min
    ids[:4] = torch.arange(k, dtype=torch.int32) * 400 + 7
    x[0, 7] = low                            # one masked logit with a slot
    z[0, 0] = z[0].max() - 12.0
    x[1, :1050] = low                        # masked up to the middle
    z[1, :3] = z[1].max() - 14.0
    x[2, 407] = low
    z[2, 1] = z[2].max() - 25.0
    x[3, 1050:] = low
    z[3, 3:] = z[3].max() - 16.0
    for tau in (0.9, 0.5, 0.3):
        loss, d = step(lib, x, ids, z, tau)
        check(x, ids, z, tau, None, 1.0, loss, d, f"tau {tau}")
        assert torch.isfinite(loss).all()
        for p in (1, 2, 3):
            loss, d, _ = shards(lib, x, ids, z, tau, None, 1.0, p)
            check(x, ids, z, tau, None, 1.0, loss, d, f"{p} shards, tau {tau}")
