"""Tokens sorted by their experts and back with weights, and the gradients,
against plain loops in 64 bits: places, moved rows of every type, empty slots
and tokens, strides, overlaps, streams, graphs, refusals."""
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


def choose(t, k, e, seed, empty=0.2, distinct=False):
    g = torch.Generator().manual_seed(seed)
    if distinct:
        c = torch.rand(t, e, generator=g).argsort(1)[:, :k].int()
    else:
        c = (torch.rand(t, k, generator=g) ** 2 * e).int()  # low experts are liked more; a token may name one twice
    odd = torch.rand(t, k, generator=g)
    c[odd < empty / 2] = -1
    c[(odd >= empty / 2) & (odd < empty * 0.75)] = e
    c[(odd >= empty * 0.75) & (odd < empty)] = -2 ** 31
    if t > 3:
        c[t // 2] = -1  # a token without any
    return c


def check_dispatch(lib, x, chosen, e, scales=None, **more):
    t, k = chosen.shape
    place, offsets = oracle.places(chosen, e)
    bits = torch.uint8 if x.element_size() == 1 else torch.int16 if x.element_size() == 2 else torch.int32
    fill = torch.full((t * k, x.shape[1]), 0x35, dtype=bits, device="cuda")
    out = (fill.clone().view(x.dtype), torch.full((t, k), -9, dtype=torch.int32, device="cuda"),
           torch.full((e + 1,), -9, dtype=torch.int32, device="cuda"),
           None if scales is None else torch.full((t * k, scales.shape[1]), 5.0, device="cuda"))
    lib.dispatch(x.cuda(), chosen.cuda(), e, scales=None if scales is None else scales.cuda(), out=out, **more)
    torch.cuda.synchronize()
    assert torch.equal(out[1].cpu(), place) and torch.equal(out[2].cpu(), offsets)
    want = fill.cpu().clone()
    full = place.reshape(-1) >= 0
    at = place.reshape(-1)[full].long()
    token = (torch.arange(t * k) // k)[full]
    want[at] = x.view(bits)[token]
    assert torch.equal(out[0].view(bits).cpu(), want)
    if scales is not None:
        s = torch.full((t * k, scales.shape[1]), 5.0)
        s[at] = scales[token]
        assert torch.equal(out[3].cpu(), s)
    return out


# (tokens, slots, experts, columns): one token, few and many slots on both sides of 4,096, 8,192 and 16,384, few and
# many experts there, chunks that end inside
SIZES = [(1, 1, 1, 1), (1, 8, 256, 100), (5, 3, 7, 33), (64, 8, 64, 40), (511, 8, 300, 9), (512, 8, 256, 4), (513, 8, 60, 5),
         (1366, 3, 1024, 3), (4097, 1, 2, 7), (129, 32, 1000, 2), (3000, 7, 33, 3), (70, 32, 32, 300), (2500, 16, 96, 2),
         (1024, 8, 32, 3), (1025, 8, 32, 3), (1000, 8, 31, 3), (700, 9, 1024, 2), (8000, 1, 33, 1),
         (2048, 8, 32, 1), (2049, 8, 32, 1), (4100, 2, 3, 1)]


@pytest.mark.parametrize("t,k,e,c", SIZES)
@pytest.mark.parametrize("dtype", DTYPES + [oracle.E4M3, torch.int32])
def test_dispatch_sizes(lib, t, k, e, c, dtype):
    g = torch.Generator().manual_seed(t + c)
    x = torch.randint(-2 ** 31, 2 ** 31 - 1, (t, c), generator=g, dtype=torch.int32)
    x = x if dtype == torch.int32 else x.view(torch.uint8)[:, :c].contiguous().view(dtype) if dtype == oracle.E4M3 else (x % 1000).to(dtype)
    check_dispatch(lib, x, choose(t, k, e, t + k, 0.2 if t % 2 else 0.0), e, scales=torch.rand(t, 3, generator=g) if c % 2 else None)


# few slots that many workgroups would read: both sides of where they are placed by a launch of their own
@pytest.mark.parametrize("t,k,e,c", [(2172, 1, 5, 7), (2173, 1, 5, 7), (48, 32, 9, 300), (49, 32, 9, 300), (341, 9, 30, 5),
                                     (342, 9, 30, 5), (4096, 1, 1024, 40), (1500, 1, 9, 2122), (1365, 3, 16, 1030),
                                     (128, 32, 8, 5000), (455, 9, 64, 4500)])
@pytest.mark.parametrize("dtype", [torch.float32, oracle.E4M3])
def test_dispatch_of_few_slots_to_be_read_often(lib, t, k, e, c, dtype):
    g = torch.Generator().manual_seed(t + c)
    x = torch.randint(0, 256, (t, c), generator=g, dtype=torch.uint8)
    x = x.float() if dtype == torch.float32 else x.view(dtype)
    check_dispatch(lib, x, choose(t, k, e, t + k, 0.2 if t % 2 else 0.0), e, scales=torch.rand(t, 3, generator=g) if t % 3 else None)
    chosen = choose(t, k, e, t, 0.1)
    rows, place, offsets, _ = lib.dispatch(torch.empty(t, 0, device="cuda"), chosen.cuda(), e)
    want = oracle.places(chosen, e)
    assert torch.equal(place.cpu(), want[0]) and torch.equal(offsets.cpu(), want[1])


@pytest.mark.parametrize("c", [1, 15, 16, 17, 255, 257, 2047, 2049, 4096, 5000])
@pytest.mark.parametrize("t", [37, 700])
def test_dispatch_row_lengths(lib, t, c):
    x = torch.randint(0, 256, (t, c), generator=torch.Generator().manual_seed(c), dtype=torch.uint8)
    check_dispatch(lib, x.view(oracle.E4M3), choose(t, 8, 40, c), 40, scales=torch.rand(t, -(-c // 128)))


@pytest.mark.parametrize("t", [37, 700])
@pytest.mark.parametrize("c,groups", [(8, 300), (700, 900), (3000, 1), (1, 65), (2049, 2049)])
def test_scales_of_any_length_beside_rows_of_any_length(lib, t, c, groups):
    x = torch.randint(0, 256, (t, c), generator=torch.Generator().manual_seed(c), dtype=torch.uint8)
    check_dispatch(lib, x, choose(t, 8, 40, groups), 40, scales=torch.rand(t, groups))


@pytest.mark.parametrize("t", [37, 700])
def test_the_places_alone(lib, t):
    chosen = choose(t, 8, 40, t)
    rows, place, offsets, _ = lib.dispatch(torch.empty(t, 0, device="cuda"), chosen.cuda(), 40)
    want = oracle.places(chosen, 40)
    assert rows.shape == (t * 8, 0) and torch.equal(place.cpu(), want[0]) and torch.equal(offsets.cpu(), want[1])


def test_no_slot_has_an_expert(lib):
    t, k = 30, 3
    place = torch.full((t, k), -1, dtype=torch.int32, device="cuda")
    w = torch.full((t, k), NAN, device="cuda")
    for c in (5, 64, 2000):
        rows = torch.full((t * k, c), NAN, device="cuda")
        assert not lib.combine(rows, place, w).any()
        keep = torch.full_like(rows, 7.0)
        _, dw = lib.combine_grad(torch.ones(t, c, device="cuda"), rows, place, w, out=(keep, torch.empty(t, k, device="cuda")))
        assert (keep == 7).all() and not dw.any()


@pytest.mark.parametrize("t", [100, 2000, 5000])
def test_all_to_one_expert_none_and_the_last(lib, t):
    x = torch.randn(t, 24)
    for chosen in (torch.full((t, 4), 5), torch.full((t, 4), -1), torch.full((t, 4), 63), torch.full((t, 4), 64)):
        check_dispatch(lib, x, chosen.int(), 64)


def test_no_tokens(lib):
    rows, place, offsets, none = lib.dispatch(torch.empty(0, 8, device="cuda"), torch.empty(0, 4, dtype=torch.int32, device="cuda"), 5)
    assert rows.shape == (0, 8) and place.shape == (0, 4) and none is None and offsets.tolist() == [0] * 6
    y = lib.combine(rows, place)
    assert y.shape == (0, 8)
    drows, dw = lib.combine_grad(y, rows, place)
    assert drows.shape == (0, 8) and dw.shape == (0, 4)
    some = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    drows, dw = lib.combine_grad(torch.ones(3, 8, device="cuda"), rows, some)
    assert drows.shape == (0, 8) and dw.shape == (3, 2) and not dw.any()
    lib.combine_grad(torch.ones(3, 8, device="cuda"), rows, some, out=(drows, None))
    y = lib.combine(rows, torch.zeros(3, 2, dtype=torch.int32, device="cuda"))  # tokens without rows
    assert y.shape == (3, 8) and not y.any()


def test_large_batches_place_every_slot(lib):
    """Chunks of more than the least size, all experts, against a sort by torch."""
    for t, k, e in ((200000, 8, 256), (50001, 32, 1024), (1100003, 1, 77)):
        g = torch.Generator("cuda").manual_seed(t)
        chosen = (torch.rand(t, k, device="cuda", generator=g) ** 2 * (e + 1)).int()  # e: empty
        x = torch.arange(t, device="cuda", dtype=torch.int32)[:, None].contiguous()
        rows, place, offsets, _ = lib.dispatch(x, chosen, e)
        flat = chosen.reshape(-1).long()
        order = torch.sort(flat, stable=True).indices
        n = int((flat < e).sum())
        at = torch.full_like(flat, -1)
        at[order[:n]] = torch.arange(n, device="cuda")
        assert torch.equal(place.reshape(-1).long(), at)
        assert torch.equal(offsets.long(), torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), torch.bincount(flat, minlength=e + 1)[:e].cumsum(0)]))
        assert torch.equal(rows[:n, 0].long(), order[:n] // k)


@pytest.mark.parametrize("t,k,e", [(16384, 16, 512), (16384, 32, 1024), (16400, 8, 1024), (65537, 8, 256), (300001, 4, 1000)])
def test_many_slots_of_many_experts(lib, t, k, e):
    """Chunks of more slots than the least because of the experts, against a sort by torch."""
    g = torch.Generator("cuda").manual_seed(t + e)
    chosen = torch.randint(-1, e, (t, k), device="cuda", generator=g, dtype=torch.int32)
    x = torch.arange(t, device="cuda", dtype=torch.int32)[:, None].contiguous()
    rows, place, offsets, _ = lib.dispatch(x, chosen, e)
    flat = chosen.reshape(-1).long()
    key = torch.where(flat >= 0, flat, e)
    order = torch.sort(key, stable=True).indices
    n = int((flat >= 0).sum())
    at = torch.full_like(flat, -1)
    at[order[:n]] = torch.arange(n, device="cuda")
    assert torch.equal(place.reshape(-1).long(), at)
    assert offsets[0] == 0 and torch.equal(offsets[1:].long(), torch.bincount(key, minlength=e + 1)[:e].cumsum(0))
    assert torch.equal(rows[:n, 0].long(), order[:n] // k)


@pytest.mark.parametrize("dtype", [torch.bfloat16, oracle.E4M3])
def test_dispatch_slices(lib, dtype):
    t, k, e, c = 50, 4, 9, 37
    wide = torch.randint(0, 100, (t, 64), generator=torch.Generator().manual_seed(1)).to(torch.uint8).view(dtype) if dtype == oracle.E4M3 \
        else torch.randn(t, 64).to(dtype)
    x = wide.cuda()[:, 5:5 + c]
    chosen = choose(t, k, e, 2)
    big = torch.zeros(t * k, 50, dtype=torch.uint8 if dtype == oracle.E4M3 else dtype, device="cuda").view(dtype)
    out = (big[:, 3:3 + c], torch.empty(t, k, dtype=torch.int32, device="cuda"), torch.empty(e + 1, dtype=torch.int32, device="cuda"), None)
    lib.dispatch(x, chosen.cuda(), e, out=out)
    want = check_dispatch(lib, x.contiguous().cpu(), chosen, e)
    n = int(out[2][e])
    assert torch.equal(out[0][:n].float(), want[0][:n].float()) and torch.equal(out[1], want[1])
    assert not big.float()[:, :3].any() and not big.float()[:, 3 + c:].any() and not big.float()[n:].any()


COMBINE = [(1, 1, 1), (1, 8, 8192), (7, 3, 5), (65, 8, 64), (40, 8, 129), (33, 9, 520), (20, 32, 1025), (9, 17, 2049), (5, 4, 5003), (300, 2, 8),
           (19, 11, 500), (23, 14, 1024), (18, 7, 1031), (16, 5, 2048)]


def expert_case(t, k, c, dtype, seed, spare=3):
    g = torch.Generator().manual_seed(seed)
    place, offsets = oracle.places(choose(t, k, 10, seed), 10)
    rows = torch.randn(t * k + spare, c, generator=g).to(dtype)
    w = torch.randn(t, k, generator=g)
    dy = torch.randn(t, c, generator=g).to(dtype)
    used = torch.zeros(t * k + spare, dtype=torch.bool)
    used[place[place >= 0].long()] = True
    rows[~used] = NAN  # what no place names is not looked at
    w[place < 0] = NAN
    return place, rows, w, dy, used


@pytest.mark.parametrize("t,k,c", COMBINE)
@pytest.mark.parametrize("dtype", DTYPES)
def test_combine_sizes(lib, t, k, c, dtype):
    place, rows, w, _, _ = expert_case(t, k, c, dtype, t + c)
    for weights in (w, None):
        got = lib.combine(rows.cuda(), place.cuda(), None if weights is None else weights.cuda())
        want, tol = oracle.combine(rows, place, weights)
        oracle.assert_within(got, want, oracle.rounded(tol, want, dtype), "out")
    assert torch.equal(lib.dispatch_grad(rows.cuda(), place.cuda()), got)


@pytest.mark.parametrize("t,k,c", COMBINE)
@pytest.mark.parametrize("dtype", DTYPES)
def test_combine_grad_sizes(lib, t, k, c, dtype):
    place, rows, w, dy, used = expert_case(t, k, c, dtype, t + c + 1)
    for weights in (w, None):
        wd = None if weights is None else weights.cuda()
        out = (torch.full((rows.shape[0], c), 7.0, dtype=dtype, device="cuda"), torch.full((t, k), 7.0, device="cuda"))
        lib.combine_grad(dy.cuda(), rows.cuda(), place.cuda(), wd, out=out)
        want, ww, wtol = oracle.combine_grad(dy, rows, place, weights)
        oracle.assert_within(out[0][used.cuda()], want[used], oracle.rounded(oracle.U * want[used].abs(), want[used], dtype), "drows")
        oracle.assert_within(out[1], ww, wtol, "dweights")
        assert (out[0][~used.cuda()] == 7).all() and (out[1].cpu()[place < 0] == 0).all()
        over = rows.cuda()
        _, dw = lib.combine_grad(dy.cuda(), over, place.cuda(), wd, out=(over, torch.empty_like(out[1])))
        assert torch.equal(over[used.cuda()], out[0][used.cuda()]) and torch.equal(dw, out[1])
        alone = torch.full_like(out[0], 7.0)
        assert lib.combine_grad(dy.cuda(), rows.cuda(), place.cuda(), wd, out=(alone, None))[1] is None
        _, dw = lib.combine_grad(dy.cuda(), rows.cuda(), place.cuda(), wd, out=(None, torch.empty_like(out[1])))
        assert torch.equal(alone, out[0]) and torch.equal(dw, out[1])


@pytest.mark.parametrize("t,k,c,dtype", [(6500, 8, 2051, torch.bfloat16), (13000, 4, 1025, torch.float32), (3400, 32, 1030, torch.float16)])
def test_combine_grad_of_more_rows_than_the_caches_hold(lib, t, k, c, dtype):
    """There the weights' gradient and the rows' are found one after the other."""
    g = torch.Generator("cuda").manual_seed(t)
    chosen = torch.randint(-1, 40, (t, k), device="cuda", generator=g, dtype=torch.int32)
    _, place, offsets, _ = lib.dispatch(torch.empty(t, 1, device="cuda"), chosen, 40)
    n = int(offsets[40])
    rows = torch.randn(t * k, c, device="cuda", generator=g).to(dtype)
    dy = torch.randn(t, c, device="cuda", generator=g).to(dtype)
    w = torch.rand(t, k, device="cuda", generator=g)
    out = (torch.full((t * k, c), 7.0, dtype=dtype, device="cuda"), torch.empty(t, k, device="cuda"))
    lib.combine_grad(dy, rows, place, w, out=out)
    full = place.reshape(-1) >= 0
    at, token = place.reshape(-1)[full].long(), torch.arange(t * k, device="cuda")[full] // k
    want = torch.full_like(out[0], 7.0)
    want[at] = (w.reshape(-1)[full][:, None] * dy[token].float()).to(dtype)  # one product, rounded once more
    assert torch.equal(out[0], want)
    for a in range(0, n, 8000):
        i, d = at[a:a + 8000], dy[token[a:a + 8000]].double()
        terms = d * rows[i].double()
        oracle.assert_within(out[1].reshape(-1)[full][a:a + 8000].cpu(), terms.sum(1).cpu(),
                             (40 + c / 256) * oracle.U * terms.abs().sum(1).cpu() + 1e-37, "dweights")
    assert not out[1].reshape(-1)[~full].any()
    dw = torch.empty_like(out[1])
    lib.combine_grad(dy, rows, place, w, out=(rows, dw))
    assert torch.equal(rows[:n], out[0][:n]) and torch.equal(dw, out[1])


@pytest.mark.parametrize("t,k,c,dtype", [(21000, 8, 1001, torch.bfloat16), (30000, 6, 1024, torch.bfloat16), (9000, 9, 1061, torch.float32),
                                         (13000, 7, 1000, torch.float32), (7000, 16, 1550, torch.float16), (20000, 5, 1700, torch.float16)])
def test_combine_of_more_rows_than_the_caches_hold(lib, t, k, c, dtype):
    g = torch.Generator("cuda").manual_seed(t)
    chosen = torch.randint(-1, 40, (t, k), device="cuda", generator=g, dtype=torch.int32)
    _, place, offsets, _ = lib.dispatch(torch.empty(t, 1, device="cuda"), chosen, 40)
    rows = torch.randn(t * k, c, device="cuda", generator=g).to(dtype)
    rows[int(offsets[40]):] = NAN
    w = torch.randn(t, k, device="cuda", generator=g)
    w[place < 0] = NAN
    got = lib.combine(rows, place, w)
    for a in range(0, t, 3000):
        full = (place[a:a + 3000] >= 0)[:, :, None]
        picked = rows[place[a:a + 3000].clamp(min=0).long()].double()
        terms = torch.where(full, picked * w[a:a + 3000, :, None].double(), 0.0)
        want = terms.sum(1)
        oracle.assert_within(got[a:a + 3000].cpu(), want.cpu(), oracle.rounded((k + 1) * oracle.U * terms.abs().sum(1), want, dtype).cpu(), "out")


# (a wave takes a token, and its columns in several turns: rows that start on a line, whose loads stream, and others;
# weights and rows in one launch, and in two where the rows are more than the caches hold)
@pytest.mark.parametrize("t,k,c,dtype", [(6500, 8, 2048, torch.bfloat16), (5000, 2, 2048, torch.bfloat16), (5000, 2, 2051, torch.bfloat16),
                                         (5000, 3, 2048, torch.float16), (4100, 3, 1024, torch.float32), (4100, 1, 1029, torch.float32),
                                         (4097, 9, 1536, torch.bfloat16), (13000, 2, 5120, torch.bfloat16)])
def test_combine_grad_of_batches(lib, t, k, c, dtype):
    g = torch.Generator("cuda").manual_seed(t + c)
    chosen = torch.randint(-1, 40, (t, k), device="cuda", generator=g, dtype=torch.int32)
    _, place, offsets, _ = lib.dispatch(torch.empty(t, 1, device="cuda"), chosen, 40)
    n = int(offsets[40])
    rows = torch.randn(t * k, c, device="cuda", generator=g).to(dtype)
    dy = torch.randn(t, c, device="cuda", generator=g).to(dtype)
    w = torch.rand(t, k, device="cuda", generator=g) + 0.1
    full = place.reshape(-1) >= 0
    at, token = place.reshape(-1)[full].long(), torch.arange(t * k, device="cuda")[full] // k
    drows = torch.full((t * k, c), 7.0, dtype=dtype, device="cuda")
    want = drows.clone()
    want[at] = (w.reshape(-1)[full][:, None] * dy[token].float()).to(dtype)  # one product, rounded once more
    _, dw = lib.combine_grad(dy, rows, place, w, out=(drows, torch.empty(t, k, device="cuda")))
    assert torch.equal(drows, want)
    for a in range(0, n, 8000):
        terms = dy[token[a:a + 8000]].double() * rows[at[a:a + 8000]].double()
        oracle.assert_within(dw.reshape(-1)[full][a:a + 8000].cpu(), terms.sum(1).cpu(), oracle.products_tolerance(terms).cpu(), "dweights")
    assert not dw.reshape(-1)[~full].any()
    alone = lib.combine_grad(dy, rows, place, w, out=(None, torch.empty_like(dw)))[1]
    over, twice = rows.clone(), torch.empty_like(dw)
    lib.combine_grad(dy, over, place, w, out=(over, twice))
    assert torch.equal(over[:n], want[:n]) and torch.equal(over[n:], rows[n:]) and torch.equal(twice, dw) and torch.equal(alone, dw)
    # without weights: the rows are dy itself
    lib.combine_grad(dy, rows, place, out=(over, twice))
    assert torch.equal(over[at], dy[token]) and torch.equal(twice, dw)


def test_places_outside_the_rows_are_empty_slots(lib):
    rows = torch.randn(6, 70)
    place = torch.tensor([[0, 6, -1], [2 ** 31 - 1, -2 ** 31, 5], [7, 100, -7]], dtype=torch.int32)
    w, dy = torch.rand(3, 3), torch.randn(3, 70)
    got = lib.combine(rows.cuda(), place.cuda(), w.cuda())
    want, tol = oracle.combine(rows, place, w)
    oracle.assert_within(got, want, oracle.rounded(tol, want, torch.float32))
    out = (torch.full((6, 70), 7.0, device="cuda"), torch.empty(3, 3, device="cuda"))
    lib.combine_grad(dy.cuda(), rows.cuda(), place.cuda(), w.cuda(), out=out)
    _, ww, wtol = oracle.combine_grad(dy, rows, place, w)
    oracle.assert_within(out[1], ww, wtol)
    assert (out[0][1:5] == 7).all() and not (out[0][[0, 5]] == 7).any()


@pytest.mark.parametrize("dtype", DTYPES)
def test_infinities_and_nan_stay_in_their_tokens(lib, dtype):
    place, rows, w, dy, _ = expert_case(20, 4, 66, dtype, 9)
    full = torch.nonzero(place >= 0)
    (i, j), (m, n) = full[0].tolist(), full[-1].tolist()
    rows[place[i, j], 3] = INF
    rows[place[m, n], 4] = NAN
    got = lib.combine(rows.cuda(), place.cuda(), w.cuda())
    want, tol = oracle.combine(rows, place, w)
    oracle.assert_within(got, want, oracle.rounded(torch.nan_to_num(tol), want, dtype))
    dy[i, 5] = NAN
    drows, dw = lib.combine_grad(dy.cuda(), rows.cuda(), place.cuda(), w.cuda())
    assert torch.isnan(dw[i].cpu()[place[i] >= 0]).all() and torch.isnan(dw[m, n])
    clean = (place >= 0)
    clean[i] = False
    clean[m, n] = False
    _, ww, wtol = oracle.combine_grad(dy, rows, place, w)
    oracle.assert_within(dw.cpu()[clean], ww[clean], wtol[clean])


@pytest.mark.parametrize("dtype", DTYPES)
def test_slices(lib, dtype):
    t, k, c = 31, 5, 301
    place, rows, w, dy, used = expert_case(t, k, c, dtype, 11)
    wide = torch.full((rows.shape[0], c + 40), 7.0, dtype=dtype, device="cuda")
    wide[:, 3:3 + c] = rows.cuda()
    out = torch.full((t, c + 9), 7.0, dtype=dtype, device="cuda")
    lib.combine(wide[:, 3:3 + c], place.cuda(), w.cuda(), out=out[:, 1:1 + c])
    want, tol = oracle.combine(rows, place, w)
    oracle.assert_within(out[:, 1:1 + c], want, oracle.rounded(tol, want, dtype))
    assert (out[:, :1] == 7).all() and (out[:, 1 + c:] == 7).all()
    out[:, 2:2 + c] = dy.cuda()
    dw = torch.empty(t, k, device="cuda")
    lib.combine_grad(out[:, 2:2 + c], wide[:, 3:3 + c], place.cuda(), w.cuda(), out=(wide[:, 3:3 + c], dw))
    want, ww, wtol = oracle.combine_grad(dy, rows, place, w)
    got = wide[:, 3:3 + c][used.cuda()]
    oracle.assert_within(got, want[used], oracle.rounded(oracle.U * want[used].abs(), want[used], dtype))
    oracle.assert_within(dw, ww, wtol)
    assert (wide[:, :3] == 7).all() and (wide[:, 3 + c:] == 7).all()


def test_offsets_past_32_bits(lib):
    c, m, ld = 40, 5, 1 << 30
    big = torch.zeros(4 * ld + c, dtype=torch.bfloat16, device="cuda")
    rows = big.as_strided((m, c), (ld, 1))
    x = torch.randn(m, c).bfloat16()
    rows.copy_(x)
    place = torch.tensor([[4, 0], [3, 1]], dtype=torch.int32)
    got = lib.combine(rows, place.cuda())
    want, tol = oracle.combine(x, place, None)
    oracle.assert_within(got, want, oracle.rounded(tol, want, torch.bfloat16))
    dy = torch.randn(2, c).bfloat16()
    _, dw = lib.combine_grad(dy.cuda(), rows, place.cuda(), out=(rows, torch.empty(2, 2, device="cuda")))
    want, ww, wtol = oracle.combine_grad(dy, x, place, None)
    oracle.assert_within(dw, ww, wtol)
    assert torch.equal(rows[[4, 0, 3, 1]].cpu(), dy[[0, 0, 1, 1]]) and torch.equal(rows[2].cpu(), x[2])
    chosen = torch.tensor([[1], [0], [1], [-1], [0]], dtype=torch.int32)
    rows.copy_(x)
    out = (torch.empty(5, c, dtype=torch.bfloat16, device="cuda"), torch.empty(5, 1, dtype=torch.int32, device="cuda"),
           torch.empty(3, dtype=torch.int32, device="cuda"), None)
    lib.dispatch(rows, chosen.cuda(), 2, out=out)
    assert torch.equal(out[0][:4].cpu(), x[[1, 4, 0, 2]])
    lib.dispatch(x.cuda(), chosen.cuda(), 2, out=(rows, *out[1:]))
    assert torch.equal(rows[:4].cpu(), x[[1, 4, 0, 2]])


def test_many_tokens(lib):
    """More tokens than one grid's workgroups take at once."""
    for t, c in ((140007, 2100), (9000001, 4)):
        base, k = 50, 2
        x = torch.randn(base, c).bfloat16().cuda()
        on = torch.arange(t, device="cuda") % base
        place = torch.stack([on, (on + 1) % base], 1).int()
        got = lib.combine(x, place)
        assert torch.equal(got[:base], lib.combine(x, place[:base].contiguous())) and torch.equal(got, got[:base][on])
        del got
        dy = x.flip(0)[on]
        _, dw = lib.combine_grad(dy, x, place, out=(None, torch.empty(t, k, device="cuda")))
        assert torch.equal(dw, dw[:base][on])


@pytest.mark.parametrize("t", [60, 1000])
def test_streams_and_graphs(lib, t):
    k, e, c = 8, 40, 520
    chosen = choose(t, k, e, 3).cuda()
    x = torch.randn(t, c, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    w = torch.rand(t, k, generator=torch.Generator().manual_seed(5)).cuda()

    def all_of(rows, place, offsets, y, drows, dw, stream=None):
        lib.dispatch(x, chosen, e, out=(rows, place, offsets, None), stream=stream)
        lib.combine(rows, place, w, out=y, stream=stream)
        lib.combine_grad(y, rows, place, w, out=(drows, dw), stream=stream)

    def outs():
        return [torch.zeros(t * k, c, dtype=torch.bfloat16, device="cuda"), torch.zeros(t, k, dtype=torch.int32, device="cuda"),
                torch.zeros(e + 1, dtype=torch.int32, device="cuda"), torch.zeros(t, c, dtype=torch.bfloat16, device="cuda"),
                torch.zeros(t * k, c, dtype=torch.bfloat16, device="cuda"), torch.zeros(t, k, device="cuda")]

    want = outs()
    all_of(*want)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [outs() for _ in streams]
    torch.cuda.synchronize()
    for _ in range(5):
        for s, o in zip(streams, got):
            all_of(*o, stream=s)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for o in got for a, b in zip(o, want))
    res = outs()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for g in graphs:
        with torch.cuda.graph(g):
            all_of(*res)
    for g in graphs + graphs:
        for o in res:
            o.zero_()
        g.replay()
        all_of(*got[0])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(res, want))


def test_refusals(lib):
    x = torch.zeros(4, 16, device="cuda")
    chosen = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    place = torch.arange(8, dtype=torch.int32, device="cuda").view(4, 2)
    rows = torch.zeros(8, 16, device="cuda")
    w = torch.zeros(4, 2, device="cuda")
    for f in (lambda: lib.dispatch(x.t(), chosen, 4), lambda: lib.dispatch(x, chosen.long(), 4), lambda: lib.dispatch(x, chosen[:3], 4),
              lambda: lib.dispatch(x, chosen[:, 0], 4), lambda: lib.dispatch(x, chosen, 4, scales=w[:2]),
              lambda: lib.dispatch(x, chosen, 4, out=(rows.bfloat16(), place, place[0], None)),
              lambda: lib.dispatch(x, chosen, 4, out=(rows[:7], place, chosen.view(-1)[:5], None)),
              lambda: lib.dispatch(x, chosen, 4, out=(rows, place, chosen.view(-1)[:5], w)),
              lambda: lib.combine(rows, place.long()), lambda: lib.combine(rows, place[0]), lambda: lib.combine(rows, place, w[:2]),
              lambda: lib.combine(rows.int(), place), lambda: lib.combine(rows, place, out=torch.zeros(4, 15, device="cuda")),
              lambda: lib.combine_grad(x, rows.bfloat16(), place), lambda: lib.combine_grad(x, rows[:, :8], place),
              lambda: lib.combine_grad(x, rows, place[:2]), lambda: lib.combine_grad(x, rows, place, out=(rows[:4], w)),
              lambda: lib.combine_grad(x, rows, place, out=(None, w[:, :1]))):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: lib.dispatch(x, chosen, 0, out=(rows, place, chosen[0, :1], None)), lambda: lib.dispatch(x, chosen, 2000),
              lambda: lib.dispatch(x, torch.zeros(4, 33, dtype=torch.int32, device="cuda"), 64),
              lambda: lib.dispatch(rows[:4], chosen, 4, out=(rows, place, torch.zeros(5, dtype=torch.int32, device="cuda"), None)),
              lambda: lib.dispatch(x, chosen, 4, out=(rows, chosen, torch.zeros(5, dtype=torch.int32, device="cuda"), None)),
              lambda: lib.combine(rows, place, out=rows[:4]), lambda: lib.combine_grad(rows[:4], rows, place, out=(rows, None)),
              lambda: lib.combine_grad(x, rows, place, out=(None, None))):
        with pytest.raises(lib.SimError):
            f()
    torch.cuda.synchronize()
