"""Root-mean-square norm with residual and 8-bit output, and its gradient,
against their formulas in 64 bits: sizes, types, strides, overlaps, rows of
special values, streams, graphs, refusals."""
import pytest
import torch

from tests import layer_oracle as oracle

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.float16, torch.bfloat16]
INF, NAN = float("inf"), float("nan")
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def lib():
    import all_reduce_reduction_amd as sim
    sim.sim_init(0, 16, 0)
    yield sim


def rand(n, c, dtype, seed, factor=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(n, c, generator=g) * factor).to(dtype)


def gains(c, dtype, seed):
    return None if dtype is None else (1 + 0.3 * torch.randn(c, generator=torch.Generator().manual_seed(seed))).to(dtype)


def cuda(t):
    return None if t is None else t.cuda()


# one column, rows shorter than a vector, ends inside a vector, every number of threads and vectors a row is held in
SIZES = [(1, 1), (3, 3), (6, 5), (2, 8), (9, 64), (33, 100), (130, 511), (5, 513), (7, 1000), (4, 1023), (3, 2047),
         (2, 2261), (1, 4096), (3, 5001), (1, 8192), (2, 8200), (2, 12289), (1, 16384), (2, 16390), (1, 32768), (3, 30011)]
# as many rows as the narrow workgroups of long rows want
MANY = [(1030, 1000), (1100, 2000), (1025, 3500), (1030, 6000), (1040, 8190), (4100, 70)]


@pytest.mark.parametrize("n,c", SIZES + MANY)
@pytest.mark.parametrize("dtype", DTYPES)
def test_sizes(lib, n, c, dtype):
    x, res = rand(n, c, dtype, n + c), rand(n, c, dtype, n + c + 1, 3.0)
    for k, (residual, gt) in enumerate(((None, dtype), (res, torch.float32), (res, torch.bfloat16), (res, torch.float16), (None, None))):
        if n > 1000 and k not in (0, 1):
            continue
        gain = gains(c, gt, c)
        y, total = lib.norm(x.cuda(), cuda(gain), residual=cuda(residual), eps=EPS)
        oracle.check_norm(y, total, x, gain, residual, EPS, f"{gt}")
        assert (total is None) == (residual is None) and y.dtype == dtype


@pytest.mark.parametrize("n,c", SIZES + MANY)
@pytest.mark.parametrize("dtype", DTYPES)
def test_quant_sizes(lib, n, c, dtype):
    x, res = rand(n, c, dtype, n + c + 2), rand(n, c, dtype, n + c + 3, 2.0)
    for k, (group, residual, gt) in enumerate(((128, res, dtype), (64, None, torch.float32), (32, res, torch.bfloat16), (c, res, dtype))):
        if n > 1000 and k not in (0, 3):
            continue
        gain = gains(c, gt, c)
        q, scales, total = lib.norm_quant(x.cuda(), cuda(gain), residual=cuda(residual), eps=EPS, group=group)
        assert q.dtype == oracle.E4M3 and scales.shape == (n, -(-c // group))
        oracle.check_quant(q, scales, total, x, gain, residual, EPS, group, f"group {group}")


# both sides of where one workgroup takes all rows, and of where each takes one row, two, and up to four
SHARED = [(64, 300), (65, 300), (4, 1500), (5, 1500), (2, 9000), (3, 9000), (255, 4112), (256, 4112), (513, 2300), (1027, 1100),
          (120, 10000)]


@pytest.mark.parametrize("n,c", SIZES + MANY + SHARED)
@pytest.mark.parametrize("dtype", DTYPES)
def test_grad_sizes(lib, n, c, dtype):
    h, dy, ds = rand(n, c, dtype, n + c + 4, 2.0), rand(n, c, dtype, n + c + 5), rand(n, c, dtype, n + c + 6)
    for dtotal, gt in ((None, dtype), (ds, torch.float32), (ds, None)):
        gain = gains(c, gt, c)
        dx, dg = lib.norm_grad(h.cuda(), cuda(gain), dy.cuda(), dtotal=cuda(dtotal), eps=EPS)
        want, tol, wg, gtol = oracle.norm_grad(h, gain, dy, dtotal, EPS)
        oracle.assert_within(dx, want, oracle.rounded(tol, want, dtype), "dx")
        oracle.assert_within(dg, wg, gtol, "dgain")
        only, none = lib.norm_grad(h.cuda(), cuda(gain), dy.cuda(), dtotal=cuda(dtotal), eps=EPS, out=(torch.empty_like(dx), None))
        assert none is None and torch.equal(only, dx)


def test_gradient_against_differences_of_the_forward(lib):
    """Central differences of the fp32 forward: step 2^-6 of unit rows leaves an error of the third derivative, below
    step^2 / 6 times 20 |v|^3 / n, and of the results' rounding, 64 u sqrt(n c) / step."""
    n, c, step = 4, 96, 2.0 ** -6
    h, dy, v = (rand(n, c, torch.float32, s) for s in (1, 2, 3))
    gain = gains(c, torch.float32, 4)
    dx, dg = lib.norm_grad(h.cuda(), gain.cuda(), dy.cuda(), eps=EPS)

    def value(h, g):
        return (lib.norm(h.cuda(), g.cuda(), eps=EPS)[0].double().cpu() * dy.double()).sum()

    for got, ends in (((dx.cpu().double() * v).sum(), [value(h + s * step * v, gain) for s in (1, -1)]),
                      ((dg.cpu().double() * v[0]).sum(), [value(h, gain + s * step * v[0]) for s in (1, -1)])):
        diff = (ends[0] - ends[1]) / (2 * step)
        bound = step ** 2 / 6 * 20 * v.norm() ** 3 / c ** 0.5 + 64 * oracle.U * (n * c) ** 0.5 * 8 / step
        assert abs(diff - got) < bound, (diff, got, bound)


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_of_special_values(lib, dtype):
    n, c = 40, 300
    x = rand(n, c, dtype, 20)
    big, tiny = torch.finfo(dtype).max, torch.finfo(dtype).tiny
    x[0] = 0
    x[1] = -0.0
    x[2] = tiny
    x[3, 5] = NAN
    x[4] = NAN
    x[5, 7] = INF
    x[6, 7:9] = -INF
    x[7, :] = 0
    x[7, 11] = 1.0
    x[8] = torch.finfo(dtype).smallest_normal
    if dtype == torch.float16:  # (its largest values' squares are within fp32's range)
        x[9] = big
        x[10] = -big
        x[11, ::2] = big
    gain = gains(c, dtype, 3)
    y, _ = lib.norm(x.cuda(), gain.cuda(), eps=EPS)
    h, r, want = oracle.norm(x, gain, None, EPS)
    # an infinity: r is 0, so that finite values become 0 and infinite ones NaN
    for row in (5, 6):
        inf = torch.isinf(x[row])
        assert torch.isnan(y[row].cpu()[inf]).all() and (y[row].cpu()[~inf] == 0).all()
    rest = [i for i in range(n) if i not in (5, 6)]
    oracle.assert_within(y[rest], want[rest], oracle.rounded(64 * oracle.U * want[rest].abs(), want[rest], dtype), "y")
    assert torch.isnan(y[3]).all() and torch.isnan(y[4]).all() and not y[0].any() and not y[1].any()
    for group in (32, 128, c):
        q, s, _ = lib.norm_quant(x.cuda(), gain.cuda(), eps=EPS, group=group)
        sane = [i for i in range(n) if i not in (3, 4, 5, 6)]
        oracle.check_quant(q[sane], s[sane], None, x[sane], gain, None, EPS, group)
        assert (s[0] == 0).all() and not q[0].float().any() and torch.isnan(s[3]).all() and torch.isnan(s[4]).all()
        k = 7 // group if group < c else 0
        assert torch.isnan(s[5, k]) and (s[5].cpu()[torch.arange(s.shape[1]) != k] == 0).all()
    # gradients of the same rows: those of NaN and infinities stay in their rows, and make dgain NaN
    dy = rand(n, c, dtype, 21)
    dx, dg = lib.norm_grad(x.cuda(), gain.cuda(), dy.cuda(), eps=EPS)
    want, tol, wg, gtol = oracle.norm_grad(x[rest], gain, dy[rest], None, EPS)
    oracle.assert_within(dx[rest], want, oracle.rounded(tol, want, dtype), "dx")
    assert torch.isnan(dg).all()
    ok = [i for i in rest if i not in (3, 4)]
    _, dg = lib.norm_grad(x[ok].cuda(), gain.cuda(), dy[ok].cuda(), eps=EPS)
    _, _, wg, gtol = oracle.norm_grad(x[ok], gain, dy[ok], None, EPS)
    oracle.assert_within(dg, wg, gtol, "dgain")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_small_groups_of_small_values(lib, dtype):
    """448 over a group's largest value may lie past fp32's range; a group of zeros stays one."""
    x = rand(6, 256, dtype, 30)
    x[:, 32:64] *= 1e-36
    x[:, 64:96] = 0
    x[:, 96:128] *= 1e-38
    for group in (32, 64):
        q, s, _ = lib.norm_quant(x.cuda(), None, eps=EPS, group=group)
        oracle.check_quant(q, s, None, x, None, None, EPS, group)


def nearest_codes(t):
    """e4m3 values nearest to t in 64 bits, of two equally near ones the even one."""
    e = (torch.frexp(t)[1] - 1).clamp(min=-6)
    step = torch.exp2(e.double() - 3)
    return (torch.round(t / step) * step).clamp(-448, 448)


@pytest.mark.parametrize("dtype", DTYPES)
def test_halfway_between_two_codes(lib, dtype):
    """g h * 448 / m halfway between two codes becomes the even one.  Every value here is a product of integers of at
    most 8 bits and a power of two, and so is exact in every type and in the sums of products."""
    odd = [n + 0.5 for n in range(8, 16)]  # between codes of one power of two
    t = torch.tensor([448.0] + [v * 2.0 ** k for k in range(-3, 5) for v in odd] + [(n + 0.5) * 2.0 ** -9 for n in range(8)] + [2.0 ** -10])
    t = torch.cat([t, torch.zeros(128 - len(t))]).repeat(2).double()
    for top in (448.0, 7.0, 0.875, 224.0, 448.0 * 2 ** -12, 3.5 * 2 ** 20 if dtype != torch.float16 else 3.5 * 2 ** 10):
        x = t * top / 448
        keep = x.to(dtype).double() == x  # (what a half's denormal numbers cannot hold is left out)
        x = torch.where(keep, x, 0.0)
        want = nearest_codes(torch.where(keep, t, 0.0))
        x = torch.stack([x, -x]).to(dtype).cuda()
        for group in (128, 256):
            for gain in (None, torch.full((len(t),), 4.0, dtype=dtype, device="cuda")):
                q, _, _ = lib.norm_quant(x, gain, group=group)
                assert torch.equal(q.cpu().double(), torch.stack([want, -want])), (top, group)


@pytest.mark.parametrize("n,c", [(37, 40), (64, 128), (50, 300), (20, 1000), (9, 2500), (8, 8192), (6, 20000)])
@pytest.mark.parametrize("group", [32, 128, 0])
def test_codes_of_16_bit_values_are_the_nearest(lib, n, c, group):
    """Of bf16 values x and gain, g x and m are integers a, b < 2^16 times powers of two, and a halfway value is an odd
    integer T < 2^5 times one.  448 a / b is equal to T, or relative to it at least 1 / (T b) > 2^-21 away, more than
    what one rounding to fp32 moves it: the codes are those of the quotient in 64 bits."""
    x, gain = rand(n, c, torch.bfloat16, n + c), gains(c, torch.bfloat16, c)
    q, _, _ = lib.norm_quant(x.cuda(), gain.cuda(), eps=EPS, group=group or c)
    gx = gain.double() * x.double()
    g = group or c
    k = -(-c // g)
    parts = torch.nn.functional.pad(gx, (0, k * g - c)).view(n, k, g)
    t = (parts * 448 / parts.abs().amax(2, keepdim=True)).view(n, k * g)[:, :c]
    assert torch.equal(q.cpu().double(), nearest_codes(t))


# (size of x, of the gain, eps): g h past fp32's range, in numbers that it holds with few bits, below it, all with
# values of y that it holds
FAR = [(1e10, 1e30, 1e-6), (1e15, 1e37, 1e-6), (1e15, 1e24, 1e-6), (1e-20, 1e-20, 1e-30), (1e-17, 1e-30, 1e-30), (1e-30, 1e-16, 1e-30),
       (1e-15, 1e-24, 1e-30)]


@pytest.mark.parametrize("size,factor,eps", FAR)
@pytest.mark.parametrize("n,c", [(3, 3), (5, 61), (9, 300), (3, 900), (2, 5001), (2, 20000)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_products_of_gain_and_value_near_the_ends_of_the_range(lib, size, factor, eps, n, c, dtype):
    x, gain = rand(n, c, dtype, n + c, size), (gains(c, torch.float32, c) * factor).to(dtype)
    eps = torch.tensor(eps, dtype=torch.float32).item()
    y, _ = lib.norm(x.cuda(), gain.cuda(), eps=eps)
    oracle.check_norm(y, None, x, gain, None, eps)
    for group in (32, 128, c):
        q, s, _ = lib.norm_quant(x.cuda(), gain.cuda(), eps=eps, group=group)
        oracle.check_quant(q, s, None, x, gain, None, eps, group, f"group {group}")
        y = oracle.norm(x, gain, None, eps)[2]
        assert (s > 0).all() and (q.float().abs().amax(1) == 448).all() and y.abs().max() < 3e38


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("c", [96, 500, 3000])
def test_groups_at_both_ends_of_the_range_beside_each_other(lib, dtype, c):
    """Each group has its own way, whatever lanes of its wave take another one; so has each row with one scale."""
    x, gain = rand(12, c, dtype, c), gains(c, dtype, c)
    gain[:32] *= 1e30
    gain[32:64] *= 1e-30
    x[1:] *= 1e10
    x[2:, 32:64] *= 1e-25
    x[3] = 0
    x[4] *= 1e-18
    x[5, 64:] = 0
    for group in (32, 64, c):
        q, s, _ = lib.norm_quant(x.cuda(), gain.cuda(), eps=EPS, group=group)
        oracle.check_quant(q, s, None, x, gain, None, EPS, group, f"group {group}")
        for row in range(12):  # alone
            a, b, _ = lib.norm_quant(x[row:row + 1].cuda(), gain.cuda(), eps=EPS, group=group)
            assert torch.equal(a.view(torch.uint8), q[row:row + 1].view(torch.uint8)) and torch.equal(b, s[row:row + 1])


def test_eps_is_all_that_a_row_of_zeros_has(lib):
    x = torch.full((3, 70), 1e-15)
    for eps in (1e-30, 1.0, 1e30):
        y, _ = lib.norm(x.cuda(), None, eps=eps)
        oracle.check_norm(y, None, x, None, None, torch.tensor(eps, dtype=torch.float32).double())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("first,c,wide", [(0, 60, 77), (1, 64, 65), (3, 513, 600), (5, 1500, 1511), (7, 2055, 2070)])
def test_column_slices(lib, dtype, first, c, wide):
    n = 21
    x, res, dy = (rand(n, wide, dtype, s).cuda() for s in (40, 41, 42))
    gain = gains(wide, dtype, 43).cuda()
    cut = slice(first, first + c)
    part = [t[:, cut] for t in (x, res, dy)]
    outs = [torch.full((n, wide), 7.0, dtype=dtype, device="cuda") for _ in range(3)]
    lib.norm(part[0], gain[cut].clone(), residual=part[1], eps=EPS, out=(outs[0][:, cut], outs[1][:, cut]))
    oracle.check_norm(outs[0][:, cut], outs[1][:, cut], part[0].cpu(), gain[cut].cpu(), part[1].cpu(), EPS)
    q = torch.full((n, wide), 0x33, dtype=torch.uint8, device="cuda").view(oracle.E4M3)
    s = torch.empty(n, -(-c // 32), device="cuda")
    lib.norm_quant(part[0], gain[cut].clone(), residual=part[1], eps=EPS, group=32, out=(q[:, cut], s, None))
    oracle.check_quant(q[:, cut], s, None, part[0].cpu(), gain[cut].cpu(), part[1].cpu(), EPS, 32)
    dg = torch.empty(c, device="cuda")
    lib.norm_grad(part[0], gain[cut].clone(), part[2], dtotal=part[1], eps=EPS, out=(outs[2][:, cut], dg))
    want, tol, wg, gtol = oracle.norm_grad(part[0].cpu(), gain[cut].cpu(), part[2].cpu(), part[1].cpu(), EPS)
    oracle.assert_within(outs[2][:, cut], want, oracle.rounded(tol, want, dtype), "dx")
    oracle.assert_within(dg, wg, gtol, "dgain")
    outside = torch.ones(wide, dtype=torch.bool, device="cuda")
    outside[cut] = False
    assert all((o[:, outside] == 7).all() for o in outs) and (q.view(torch.uint8)[:, outside] == 0x33).all()
    # between the inputs' own columns
    if 2 * c <= wide - first:
        keep = x.clone()
        lib.norm(x[:, cut], None, eps=EPS, out=(x[:, first + c:first + 2 * c], None))
        oracle.check_norm(x[:, first + c:first + 2 * c], None, keep[:, cut].cpu(), None, None, EPS)


@pytest.mark.parametrize("n,c", [(5, 3), (700, 77), (1300, 1001), (9, 5003), (3, 20001)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_in_place(lib, n, c, dtype):
    x, res, dy = (rand(n, c, dtype, s).cuda() for s in (50, 51, 52))
    gain = gains(c, dtype, 53).cuda()
    y, total = lib.norm(x, gain, residual=res, eps=EPS)
    for where in ("total on residual", "total on x", "y on x", "y on residual", "y on x, total on residual"):
        a, b = x.clone(), res.clone()
        out = {"total on residual": (torch.empty_like(x), b), "total on x": (torch.empty_like(x), a), "y on x": (a, torch.empty_like(x)),
               "y on residual": (b, None), "y on x, total on residual": (a, b)}[where]
        lib.norm(a, gain, residual=b, eps=EPS, out=out)
        assert torch.equal(out[0], y) and (out[1] is None or torch.equal(out[1], total)), where
    a = x.clone()
    lib.norm(a, gain, eps=EPS, out=(a, None))
    assert torch.equal(a, lib.norm(x, gain, eps=EPS)[0])
    q, s, total = lib.norm_quant(x, gain, residual=res, eps=EPS)
    b = res.clone()
    got = lib.norm_quant(x, gain, residual=b, eps=EPS, out=(torch.empty_like(q), torch.empty_like(s), b))
    assert torch.equal(got[0].view(torch.uint8), q.view(torch.uint8)) and torch.equal(got[1], s) and torch.equal(b, total)
    dx, dg = lib.norm_grad(x, gain, dy, dtotal=res, eps=EPS)
    for k in range(3):
        t = [x.clone(), dy.clone(), res.clone()]
        got = lib.norm_grad(t[0], gain, t[1], dtotal=t[2], eps=EPS, out=(t[k], torch.empty_like(dg)))
        assert torch.equal(t[k], dx) and torch.equal(got[1], dg), k


def test_no_rows(lib):
    x = torch.empty(0, 50, device="cuda")
    y, total = lib.norm(x, None, residual=x)
    assert y.shape == (0, 50) and total.shape == (0, 50)
    q, s, _ = lib.norm_quant(x)
    assert q.shape == (0, 50) and s.shape == (0, 1)
    dx, dg = lib.norm_grad(x, None, x, out=(torch.empty_like(x), torch.full((50,), 3.0, device="cuda")))
    assert dx.shape == (0, 50) and not dg.any()


@pytest.mark.parametrize("n,c", [(2100000 * 4 + 3, 2), (2100003, 300)])
def test_more_rows_than_the_grid_takes_at_once(lib, n, c):
    base = 41
    x, dy = rand(base, c, torch.bfloat16, 60), rand(base, c, torch.bfloat16, 61)
    on = torch.arange(n, device="cuda") % base
    xd = x.cuda()[on]
    y, _ = lib.norm(xd, None, eps=EPS)
    oracle.check_norm(y[:base], None, x, None, None, EPS)
    assert torch.equal(y, y[:base][on])
    dyd = dy.cuda()[on]
    dx, dg = lib.norm_grad(xd, None, dyd, eps=EPS)
    want, tol, wg, _ = oracle.norm_grad(x, None, dy, None, EPS)
    oracle.assert_within(dx[:base], want, oracle.rounded(tol, want, torch.bfloat16), "dx")
    assert torch.equal(dx, dx[:base][on])
    reps = torch.bincount(on, minlength=base).cpu().double()[:, None]
    h, r, _ = oracle.norm(x, None, None, EPS)
    terms = dy.double() * h * r
    oracle.assert_within(dg, (reps * terms).sum(0), (500 + n / 200) * oracle.U * (reps * terms.abs()).sum(0), "dgain")


def test_offsets_past_32_bits(lib):
    c, n, ld = 200, 5, 1 << 30
    big = torch.empty(4 * ld + c, dtype=torch.bfloat16, device="cuda")
    part = big.as_strided((n, c), (ld, 1))
    x, res, dy = (rand(n, c, torch.bfloat16, s) for s in (70, 71, 72))
    gain = gains(c, torch.bfloat16, 73)
    part.copy_(x)
    y, total = lib.norm(part, gain.cuda(), residual=res.cuda(), eps=EPS)
    oracle.check_norm(y, total, x, gain, res, EPS)
    dx, _ = lib.norm_grad(part, gain.cuda(), dy.cuda(), eps=EPS, out=(part, None))
    want, tol, _, _ = oracle.norm_grad(x, gain, dy, None, EPS)
    oracle.assert_within(part, want, oracle.rounded(tol, want, torch.bfloat16), "dx")
    q8 = torch.empty(4 * ld + c, dtype=torch.uint8, device="cuda")
    q = q8.as_strided((n, c), (ld, 1)).view(oracle.E4M3)
    s = torch.empty(n, 2, device="cuda")
    lib.norm_quant(x.cuda(), gain.cuda(), eps=EPS, out=(q, s, None))
    oracle.check_quant(q, s, None, x, gain, None, EPS, 128)


def test_streams_and_graphs(lib):
    n, c = 300, 1111
    x, res, dy = (rand(n, c, torch.bfloat16, s).cuda() for s in (80, 81, 82))
    gain = gains(c, torch.float32, 83).cuda()
    y, total = lib.norm(x, gain, residual=res, eps=EPS)
    q, s, _ = lib.norm_quant(x, gain, residual=res, eps=EPS)
    dx, dg = lib.norm_grad(total, gain, dy, dtotal=res, eps=EPS)
    want = [y, total, q.view(torch.uint8), s, dx, dg]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    a = lib.norm(x, gain, residual=res, eps=EPS, stream=side)
    b = lib.norm_quant(x, gain, residual=res, eps=EPS, stream=side)
    d = lib.norm_grad(a[1], gain, dy, dtotal=res, eps=EPS, stream=side)
    side.synchronize()
    assert all(torch.equal(i, j) for i, j in zip([*a, b[0].view(torch.uint8), b[1], *d], want))
    outs = [torch.empty_like(t) for t in want]
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for g in graphs:
        with torch.cuda.graph(g):
            lib.norm(x, gain, residual=res, eps=EPS, out=(outs[0], outs[1]))
            lib.norm_quant(x, gain, residual=res, eps=EPS, out=(outs[2].view(oracle.E4M3), outs[3], None))
            lib.norm_grad(outs[1], gain, dy, dtotal=res, eps=EPS, out=(outs[4], outs[5]))
    for g in graphs + graphs:
        for o in outs:
            o.zero_()
        g.replay()
        again = lib.norm_grad(total, gain, dy, dtotal=res, eps=EPS)
        torch.cuda.synchronize()
        assert all(torch.equal(i, j) for i, j in zip(outs, want)) and torch.equal(again[1], dg)


def test_refusals(lib):
    x = torch.zeros(4, 64, dtype=torch.bfloat16, device="cuda")
    gain = torch.ones(64, device="cuda")
    for f in (lambda: lib.norm(x.t()), lambda: lib.norm(x[0]), lambda: lib.norm(x, gain[:5]), lambda: lib.norm(x, gain.cpu()),
              lambda: lib.norm(x, gain.double()), lambda: lib.norm(x, residual=x.float()), lambda: lib.norm(x, residual=x[:2]),
              lambda: lib.norm(x.double()), lambda: lib.norm(x, out=(x.float(), None)), lambda: lib.norm(x, out=(x[:, :8], None)),
              lambda: lib.norm_quant(x, out=(x, gain, None)), lambda: lib.norm_grad(x, gain, x.float()),
              lambda: lib.norm_grad(x, gain, x, out=(torch.empty_like(x), gain.bfloat16())),
              lambda: lib.norm_quant(x, group=16), lambda: lib.norm_quant(x, group=0), lambda: lib.norm_quant(x, group=-64),
              lambda: lib.norm_quant(x, group=256), lambda: lib.norm_grad(x, gain, x, dtotal=x[:1])):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: lib.norm(x, eps=0.0), lambda: lib.norm(x, out=(torch.empty_like(x), torch.empty_like(x))),
              lambda: lib.norm(torch.zeros(2, 40000, device="cuda")), lambda: lib.norm(x, residual=x.clone(), out=(x, x)),
              lambda: lib.norm_grad(x, gain, x, out=(torch.empty_like(x), gain))):
        with pytest.raises(lib.SimError):
            f()
    torch.cuda.synchronize()
