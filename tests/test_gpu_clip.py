"""The norm over lists of gradients and clipping against their formulas in 64
bits: sizes, types, extreme values, overlaps, several ranks' parts, streams,
graphs, refusals."""
import pytest
import torch

from tests import layer_oracle as oracle

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.float16, torch.bfloat16]
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def lib():
    import all_reduce_reduction_amd as sim
    sim.sim_init(0, 16, 0)
    yield sim


def make(sizes, dtypes, seed, factor=1.0):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * factor).to(dtypes[i % len(dtypes)]) for i, n in enumerate(sizes)]


def check(lib, grads, max_norm, outs=None):
    mine = [g.cuda() for g in grads]
    norm = lib.clip_grads(mine, max_norm, out=outs)
    oracle.check_clip(norm, mine if outs is None else outs, grads, max_norm)
    if outs is not None:
        assert all(torch.equal(a.cpu().view(torch.uint8), b.view(torch.uint8)) for a, b in zip(mine, grads))
    return norm


LISTS = [[1], [7], [8], [9], [255, 3, 0, 5], [16383], [16384], [16385], [0], [0, 0, 1], [100000, 1, 16384, 32768, 5, 2047, 4096],
         [3] * 119, [5] * 120, [9] * 121, [11] * 500, [70000] * 130, [2500001, 3, 800000]]


@pytest.mark.parametrize("sizes", LISTS, ids=lambda s: f"{len(s)}x{s[0]}")
@pytest.mark.parametrize("dtypes", [[d] for d in DTYPES] + [DTYPES], ids=["fp32", "fp16", "bf16", "mixed"])
def test_sizes(lib, sizes, dtypes):
    grads = make(sizes, dtypes, len(sizes) + sizes[0])
    n = oracle.norm_of(grads).item()
    for most in (n / 3, n * 2):
        check(lib, grads, most)
        check(lib, grads, most, outs=[torch.full_like(g, 7.0, device="cuda") for g in grads])
    oracle.assert_within(lib.grad_norm([g.cuda() for g in grads]).reshape(()), oracle.norm_of(grads), 8 * oracle.U * n, "norm")


def test_no_tensors(lib):
    assert lib.clip_grads([], 1.0).item() == 0 and lib.grad_norm([]).item() == 0
    assert lib.clip_grads([torch.empty(0, device="cuda")], 1.0).item() == 0


@pytest.mark.parametrize("dtype", DTYPES)
def test_zero_gradients_and_a_zero_norm(lib, dtype):
    z = [torch.zeros(50, dtype=dtype)]
    check(lib, z, 1.0)
    check(lib, z, 0.0)
    norm = check(lib, [torch.ones(50, dtype=dtype)], 0.0)  # scaled to nothing
    assert norm.item() > 7
    check(lib, [torch.ones(64, dtype=dtype)], 8.0)  # the norm is the largest allowed
    check(lib, [torch.ones(64, dtype=dtype)], INF)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size", [1e-30, 1e-22, 1e18, 1e25, 1e34])
def test_values_whose_squares_are_past_fp32(lib, dtype, size):
    grads = make([1000, 70], [dtype], 3, size)
    n = oracle.norm_of(grads).item()
    check(lib, grads, n / 5)
    check(lib, grads, n * 5)


def test_halves_at_the_ends_of_their_range(lib):
    check(lib, [torch.full((100000,), 65504.0).half(), torch.full((999,), -65504.0).half()], 10.0)
    check(lib, [torch.full((100000,), 2.0 ** -24).half()], 1e-6)


@pytest.mark.parametrize("dtype", DTYPES)
def test_nan_and_infinity(lib, dtype):
    g = make([300, 20], [dtype], 4)
    for value, finite in ((NAN, NAN), (INF, 0.0), (-INF, 0.0)):
        grads = [t.clone() for t in g]
        grads[1][7] = value
        mine = [t.cuda() for t in grads]
        norm = lib.clip_grads(mine, 1.0)
        assert torch.isnan(norm).item() == (value != value) and (value != value or norm.item() == INF)
        assert torch.isnan(mine[1][7])
        rest = torch.cat([mine[0], mine[1][:7], mine[1][8:]])
        assert torch.isnan(rest).all() if finite != finite else not rest.any()
        assert torch.isnan(lib.grad_norm([t.cuda() for t in grads])).item() == (value != value)


def test_a_norm_past_fp32_is_infinite(lib):
    g = torch.full((4,), 3e38, device="cuda")
    assert lib.clip_grads([g], 1.0).item() == INF and not g.any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_starts_at_any_element(lib, dtype):
    """Views into one buffer, one after the other, some moved by single elements; what lies between stays."""
    base = make([200000], [dtype], 6)[0].cuda()
    keep = base.clone()
    cuts = [(0, 1), (1, 8), (11, 1000), (1011, 7), (1019, 30000), (40001, 65536), (105539, 3)]
    views = [base[a:a + n] for a, n in cuts]
    grads = [v.cpu().clone() for v in views]
    n = oracle.norm_of(grads).item()
    norm = lib.clip_grads(views, n / 2)
    oracle.check_clip(norm, views, grads, n / 2)
    other = torch.ones(200000, dtype=torch.bool, device="cuda")
    for a, m in cuts:
        other[a:a + m] = False
    assert torch.equal(base[other], keep[other])
    shifted = torch.zeros(200010, dtype=dtype, device="cuda")
    outs = [shifted[a + 5:a + 5 + m] for a, m in cuts]
    lib.clip_grads(views, n / 5, out=outs)
    now = [v.cpu() for v in views]
    oracle.check_clip(oracle.norm_of(now).float(), outs, now, n / 5)


def test_shapes_and_parameters(lib):
    p = torch.nn.Parameter(torch.randn(30, 40, device="cuda"))
    p.grad = torch.randn(30, 40, device="cuda")
    want = p.grad.cpu().clone()
    norm = lib.clip_grads((q.grad for q in [p]), 1.0)
    oracle.check_clip(norm, [p.grad], [want], 1.0)


@pytest.mark.parametrize("p", [2, 8])
def test_parts_of_several_ranks(lib, p):
    """Each rank's norm, gathered; every rank scales its own gradients by the norm of all."""
    ranks = [make([1000 * (r + 1), 33, 20000], DTYPES, 10 + r) for r in range(p)]
    mine = [[g.cuda() for g in gs] for gs in ranks]
    parts = [lib.grad_norm(gs) for gs in mine]
    gathered = [torch.empty(p, device="cuda") for _ in range(p)]
    lib.all_gather(parts, gathered)
    total = oracle.norm_of([g for gs in ranks for g in gs])
    for gs, theirs, g in zip(ranks, mine, gathered):
        norm = lib.clip_grads(theirs, total.item() / 4, parts=g)
        oracle.check_clip(norm, theirs, gs, total.item() / 4, total)
    many = [torch.ones(4, device="cuda") for _ in range(150)]
    norm = lib.clip_grads(many, 1.0, parts=torch.tensor([3.0, 4.0], device="cuda"))
    assert abs(norm.item() - 5.0) < 1e-6 and all(torch.allclose(t, torch.full_like(t, 0.2)) for t in many)


def test_parts_of_many_ranks_and_of_one(lib):
    parts = torch.rand(1000, generator=torch.Generator().manual_seed(1))
    want = (parts.double() ** 2).sum().sqrt()
    g = torch.ones(5, device="cuda")
    norm = lib.clip_grads([g], 1.0, parts=parts.cuda())
    oracle.assert_within(norm.reshape(()), want, 8 * oracle.U * want, "norm")
    oracle.assert_within(g, torch.full((5,), 1.0).double() / want, 12 * oracle.U / want, "gradient")
    for n in (3, 0):  # one rank's norm is all of it, whatever it is
        g = [torch.ones(5, device="cuda") for _ in range(n)]
        assert lib.clip_grads(g, 1.0, parts=torch.tensor([4.0], device="cuda")).item() == 4.0
        assert all((t == 0.25).all() for t in g)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("size,most", [(1e37, 1.0), (1e37, 1e-4), (1e37, 1e-7), (1e30, 1e-13), (1e20, 1e-26), (1e37, 1e-37), (1e25, 1e-30)])
def test_factors_below_the_normal_numbers(lib, dtype, size, most):
    """fp32: the factor and the product round by at most u; below the normal numbers what is multiplied with the factor
    and the product by half a step of 2^-149 each."""
    grads = make([90, 5000 if size < 1e36 else 30], [dtype], 5, size)
    want = oracle.norm_of(grads).item()
    most = torch.tensor(most, dtype=torch.float32).item()
    for outs in (None, [torch.full_like(g, 7.0, device="cuda") for g in grads]):
        mine = [g.cuda() for g in grads]
        lib.clip_grads(mine, most, out=outs)
        for a, g in zip(mine if outs is None else outs, grads):
            w = g.double() * (most / want)
            tol = (2 + 2.0 ** -16) * oracle.U * w.abs() + 2.0 ** -149
            oracle.assert_within(a, w, oracle.rounded(tol, w, dtype) if dtype != torch.float32 else tol, f"{size} {most}")


@pytest.mark.parametrize("sizes", [[5000], [700, 4000, 33], [40] * 130, [9000000]], ids=lambda s: f"{len(s)}x{s[0]}")
def test_the_factor_is_formed_of_the_norm_in_64_bits(lib, sizes):
    """One rounding of the factor and one of the product, u = 2^-24 each; the sums in 64 bits are off by far less than
    2^-16 u.  Whatever the norm's own rounding would add is common to all elements."""
    worst = 0.0
    for seed in range(100 if sum(sizes) < 10000 else 4):
        grads = [(torch.rand(n, generator=torch.Generator("cuda").manual_seed(seed), device="cuda") + 0.5) for n in sizes]
        want = torch.cat([g.double() for g in grads])
        norm = want.square().sum().sqrt().item()
        most = torch.tensor(norm / (1.3 + seed / 30)).item()
        lib.clip_grads(grads, most)
        want *= torch.tensor(most, dtype=torch.float32).double().item() / norm
        worst = max(worst, ((torch.cat([g.double() for g in grads]) - want).abs() / want).max().item())
    assert worst <= (2 + 2.0 ** -16) * oracle.U, worst / oracle.U


@pytest.mark.parametrize("tensors,n", [(3, 1000), (130, 50), (1, 40000000)])
def test_ranks_with_the_same_parts_have_the_same_factor(lib, tensors, n):
    """Whichever launches a rank's own list takes; factor and norm are those of the fp32 norm[0]."""
    for seed in range(20):
        parts = (torch.rand(8, generator=torch.Generator().manual_seed(seed)) + 1.0).cuda()
        few, own = [torch.ones(16, device="cuda")], [torch.ones(n, device="cuda") for _ in range(tensors)]
        a, b = lib.clip_grads(few, 0.7, parts=parts), lib.clip_grads(own, 0.7, parts=parts)
        factor = (torch.tensor(0.7).double() / a.double().cpu()).float()
        assert torch.equal(a, b) and (few[0].cpu() == factor).all() and all((g == few[0][0]).all() for g in own)


def test_the_same_bits_every_time(lib):
    grads = [g.cuda() for g in make([500001, 77, 40000], DTYPES, 20)]
    a, b = ([torch.empty_like(g) for g in grads] for _ in range(2))
    n, m = lib.clip_grads(grads, 1.0, out=a), lib.clip_grads(grads, 1.0, out=b)
    assert torch.equal(n, m) and all(torch.equal(i, j) for i, j in zip(a, b)) and torch.equal(lib.grad_norm(grads), n)


def test_more_elements_than_32_bits_count(lib):
    """One tensor of 2^32 + 5 elements."""
    n = (1 << 32) + 5
    g = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g[-3:] = 3.0
    g[0] = 4.0
    g[1 << 31] = 2.0
    norm = lib.clip_grads([g], 1.0)
    want = (3 * 9 + 16 + 4) ** 0.5
    assert abs(norm.item() - want) < 1e-5
    for i, v in ((0, 4.0), (1 << 31, 2.0), (n - 3, 3.0), (n - 1, 3.0)):
        assert abs(g[i].item() - v / want) < 2.0 ** -8 * v / want
    assert torch.count_nonzero(g).item() == 5


def test_streams_and_graphs(lib):
    grads = [g.cuda() for g in make([30000, 5, 999] + [20] * 130, DTYPES, 30)]
    want = [torch.empty_like(g) for g in grads]
    n = lib.clip_grads(grads, 1.0, out=want).clone()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [[torch.zeros_like(g) for g in grads] for _ in streams]
    torch.cuda.synchronize()
    norms = [[lib.clip_grads(grads, 1.0, out=o, stream=s) for s, o in zip(streams, got)] for _ in range(5)]
    parts = [lib.grad_norm(grads, stream=s) for s in streams]
    torch.cuda.synchronize()
    assert all(torch.equal(m, n) for row in norms for m in row) and all(torch.equal(m, n) for m in parts)
    assert all(torch.equal(a, b) for o in got for a, b in zip(o, want))
    out, norm = [torch.zeros_like(g) for g in grads], torch.zeros(1, device="cuda")
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for g in graphs:
        with torch.cuda.graph(g):
            lib.clip_grads(grads, 1.0, out=out, norm=norm)
    for g in graphs + graphs:
        for o in out:
            o.zero_()
        norm.zero_()
        g.replay()
        lib.clip_grads(grads, 2.0, out=got[0])
        torch.cuda.synchronize()
        assert torch.equal(norm, n) and all(torch.equal(a, b) for a, b in zip(out, want))


def test_both_forms_of_the_tensor_checks_agree(lib):
    """The checks in C++ and their Python forms return or refuse the same, for tensors of any kind."""
    x = torch.zeros(6, 40, device="cuda")
    some = [x, x.half(), x.bfloat16(), x[:, 3:9], x[::2], x[:1], x[:0], x[:, :1], x[:, :0], x.t(), x[0], x.int(), x.double(),
            x.cpu(), x.view(2, 3, 40), x[:, ::2], x.to(torch.float8_e4m3fn), torch.nn.Parameter(x), x.expand(6, 40), x[:1].expand(6, 40)]
    mine = lib._rows_py(x, "x", None)
    lists = [[], [x], [x, x.half()], [x.half(), x], [x, x.t()], [x.cpu()], [x.int()], [x[:0], x[1]], (x,), [x.view(-1)]]
    likes = [None] + [lib._tensors_py(ts, "l", 0, None) for ts in ([], [x], [x, x.half()])]
    pairs = [(lib._raw, lib._raw_py, [(t, "t", d) for t in some for d in (None, torch.float32, torch.float8_e4m3fn)]),
             (lib._like, lib._like_py, [(t, "t", mine) for t in some + [None]]),
             (lib._rows, lib._rows_py, [(t, "t", w) for t in some for w in (None, mine)]),
             (lib._gain, lib._gain_py, [(t, n, 0) for t in some + [None, x.view(-1)] for n in (40, 240)]),
             (lib._vec, lib._vec_py, [(t, "t", (torch.float32,), 0, 6, 40) for t in some + [None]]),
             (lib._tensors, lib._tensors_py, [(ts, "l", 0, w) for ts in lists for w in likes])]
    for c, py, calls in pairs:
        assert c is not py
        for args in calls:
            got = []
            for f in (c, py):
                try:
                    got.append(f(*args))
                except ValueError as e:
                    got.append(type(e))
            assert got[0] == got[1], (py.__name__, args)


def test_refusals(lib):
    a, b = torch.ones(10, device="cuda"), torch.ones(6, 4, device="cuda")
    for f in (lambda: lib.clip_grads([a, b.t()], 1.0), lambda: lib.clip_grads([a, b.cpu()], 1.0), lambda: lib.clip_grads([a.cpu()], 1.0),
              lambda: lib.clip_grads([a.double()], 1.0), lambda: lib.clip_grads([a.int()], 1.0), lambda: lib.clip_grads([a], 1.0, out=[b]),
              lambda: lib.clip_grads([a], 1.0, out=[a.bfloat16()]), lambda: lib.clip_grads([a, b], 1.0, out=[a]),
              lambda: lib.clip_grads([a], 1.0, norm=b), lambda: lib.clip_grads([a], 1.0, parts=b.double().view(-1)),
              lambda: lib.grad_norm([b.t()]), lambda: lib.grad_norm([a], out=b)):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: lib.clip_grads([a, a], 1.0), lambda: lib.clip_grads([a], -1.0), lambda: lib.clip_grads([a], NAN),
              lambda: lib.clip_grads([a, a[5:]], 1.0), lambda: lib.clip_grads([a], 1.0, norm=a[:1]),
              lambda: lib.clip_grads([b], 1.0, parts=torch.empty(0, device="cuda")),
              lambda: lib.clip_grads([b.view(-1)[:12], a], 1.0, out=[b.view(-1)[6:18], a])):
        with pytest.raises(lib.SimError):
            f()
    torch.cuda.synchronize()
    assert (a == 1).all() and (b == 1).all()
