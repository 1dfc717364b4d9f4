"""Softmax gate with per-expert statistics, and the balance loss's gradient,
against their formulas in 64 bits: ragged sizes, ties, masked and dead rows,
strides, streams, graphs, refusals."""
import pytest
import torch

from tests import loss_oracle as oracle

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.float16, torch.bfloat16]
INF = float("inf")


@pytest.fixture(scope="module", autouse=True)
def lib():
    import all_reduce_reduction_amd as sim
    sim.sim_init(0, 16, 0)
    yield sim


def logits(t, e, dtype, seed, coarse=False):
    g = torch.Generator().manual_seed(seed)
    x = 2.0 * torch.randn(t, e, generator=g)
    return ((x * 2).round() / 2 if coarse else x).to(dtype)


def check_route(sim, x, topk, keep, normalize, xd=None):
    xd = x.cuda() if xd is None else xd
    got = sim.route(xd, topk, keep=None if keep is None else keep.cuda(), normalize=normalize)
    chosen, w, counts, sums, wtol, stol = oracle.route(x, topk, keep, normalize)
    assert torch.equal(got[0].cpu(), chosen)
    assert torch.equal(got[2].cpu(), counts)
    oracle.assert_within(got[1], w, wtol, "weights")
    oracle.assert_within(got[3], sums, stol + 1e-37, "prob_sums")
    return got


SIZES = [(0, 8, 2), (1, 1, 1), (1, 256, 8), (3, 5, 5), (7, 64, 1), (130, 65, 7), (257, 256, 8), (2049, 60, 4),
         (300, 1024, 32), (63, 100, 16), (5, 1000, 3), (1, 513, 32), (9, 17, 2), (70, 128, 32), (4100, 16, 2)]


@pytest.mark.parametrize("t,e,k", SIZES)
@pytest.mark.parametrize("dtype", DTYPES)
def test_route_sizes(lib, t, e, k, dtype):
    check_route(lib, logits(t, e, dtype, t + e), k, None, (t + k) % 2 == 0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("e,k", [(8, 8), (64, 6), (96, 8), (256, 8), (300, 20)])
def test_ties_go_to_the_lowest_index(lib, dtype, e, k):
    x = logits(200, e, dtype, 3, coarse=True)
    x[0] = 0.0
    x[1, ::2] = -0.0  # equal to +0
    x[1, 1::2] = 0.0
    check_route(lib, x, k, None, True)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("normalize", [False, True])
def test_masked_and_dead_rows(lib, dtype, normalize):
    t, e, k = 90, 40, 6
    x = logits(t, e, dtype, 5)
    keep = torch.rand(t, generator=torch.Generator().manual_seed(1)) < 0.6
    x[~keep] = torch.tensor([float("nan"), INF, -INF, 1.0]).repeat(e // 4).to(dtype)  # masked rows hold anything
    x[3] = -INF  # nothing to choose
    x[4] = -INF
    x[4, 7] = 1.0  # fewer than k
    x[5, 2:] = torch.finfo(dtype).min  # the type's lowest value is a logit like any other
    x[6, :] = torch.finfo(dtype).max
    x[8, :e - 2] = -INF
    keep[[3, 4, 5, 6, 8]] = True
    check_route(lib, x, k, keep, normalize)
    check_route(lib, x, k, keep.to(torch.uint8) * 3, normalize)
    check_route(lib, x, k, torch.zeros(t, dtype=torch.bool), normalize)


@pytest.mark.parametrize("dtype", DTYPES)
def test_nan_and_infinity_stay_in_their_rows(lib, dtype):
    x = logits(20, 30, dtype, 6)
    x[2, 4] = float("nan")
    x[7] = float("nan")
    x[9, 3] = INF
    got = check_route(lib, x, 4, None, True)
    assert torch.isnan(got[3]).all() and not torch.isnan(got[1][[0, 1, 3, 8, 10]]).any()
    check_route(lib, x, 4, None, False)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("first,e,wide", [(0, 60, 77), (1, 64, 65), (3, 256, 300), (5, 100, 111)])
def test_column_slices(lib, dtype, first, e, wide):
    big = logits(150, wide, dtype, 8).cuda()
    part = big[:, first:first + e]
    check_route(lib, part.cpu(), 4, None, True, xd=part)
    chosen, _, counts, sums = lib.route(part, 4)
    out = torch.full((150, wide), 7.0, dtype=dtype, device="cuda")
    dw = torch.randn(150, 4, device="cuda")
    lib.route_grad(part, chosen, dw, counts, sums, 0.5, out=(torch.empty(1, device="cuda"), out[:, first:first + e]))
    check_grad_values(part.cpu(), chosen.cpu(), dw.cpu(), counts.cpu(), 0.5, None, True, out[:, first:first + e])
    assert (out[:, :first] == 7).all() and (out[:, first + e:] == 7).all()


def test_the_same_bits_every_time(lib):
    x = logits(5000, 200, torch.bfloat16, 9).cuda()
    a, b = lib.route(x, 8), lib.route(x, 8)
    assert all(torch.equal(i, j) for i, j in zip(a, b))


def check_grad_values(x, chosen, dw, counts, coef, keep, normalize, got):
    want, tol = oracle.route_grad(x, chosen, dw, counts, coef, keep, normalize)
    oracle.assert_within(got, want, oracle.rounded(tol, want, x.dtype), "dlogits")


@pytest.mark.parametrize("t,e,k", SIZES)
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("normalize", [False, True])
def test_grad_sizes(lib, t, e, k, dtype, normalize):
    x = logits(t, e, dtype, t + e + 1)
    keep = (torch.arange(t) % 5 != 2) if t % 2 else None
    kd = None if keep is None else keep.cuda()
    chosen, _, counts, sums = lib.route(x.cuda(), k, keep=kd, normalize=normalize)
    dw = torch.randn(t, k, generator=torch.Generator().manual_seed(2))
    counts2, sums2 = counts * 3, sums * 3  # three ranks with the same tokens
    coef = 40.0
    for use_dw, use_counts in ((True, True), (True, False), (False, True)):
        loss, d = lib.route_grad(x.cuda(), chosen, dw.cuda() if use_dw else None, counts2 if use_counts else None,
                                 sums2 if use_counts else None, coef, keep=kd, normalize=normalize)
        check_grad_values(x, chosen.cpu(), dw if use_dw else None, counts2.cpu() if use_counts else None, coef, keep,
                          normalize, d)
        want = oracle.balance_loss(x, counts2.cpu(), sums2.cpu(), k, coef) if use_counts else torch.zeros(())
        oracle.assert_within(loss, want.reshape(1).double(), (e + 16) * oracle.U * want.abs() + 1e-37, "loss")


@pytest.mark.parametrize("normalize", [False, True])
def test_grad_against_differences(lib, normalize):
    t, e, k, coef = 6, 24, 3, 2.0
    x = logits(t, e, torch.float32, 11)
    chosen, _, counts, sums = (v.cpu() for v in lib.route(x.cuda(), k, normalize=normalize))
    dw = torch.randn(t, k, generator=torch.Generator().manual_seed(3))
    _, d = lib.route_grad(x.cuda(), chosen.cuda(), dw.cuda(), counts.cuda(), sums.cuda(), coef, normalize=normalize)
    g = torch.Generator().manual_seed(4)
    h = 1e-5
    for _ in range(20):
        v = torch.randn(t, e, generator=g, dtype=torch.float64)
        f = [oracle.route_objective(x.double() + s * h * v, chosen, dw, counts, coef, None, normalize) for s in (1, -1)]
        slope = (f[0] - f[1]).item() / (2 * h)
        dot = (d.cpu().double() * v).sum().item()
        # the difference quotient is off by h^2 of the third derivative and 1e-16 / h; the kernel by 1e-5 of the terms
        assert abs(slope - dot) <= 1e-5 * (d.cpu().double() * v).abs().sum().item() + 1e-8


@pytest.mark.parametrize("dtype", DTYPES)
def test_grad_of_masked_rows_and_odd_slots(lib, dtype):
    t, e, k = 40, 33, 4
    x = logits(t, e, dtype, 12)
    keep = torch.arange(t) % 3 != 0
    x[~keep] = float("nan")
    x[1] = -INF
    x[2, 3:] = -INF
    chosen, _, counts, sums = lib.route(x.cuda(), k, keep=keep.cuda())
    dw = torch.randn(t, k)
    dw[chosen.cpu() < 0] = float("nan")  # empty slots hold anything
    for normalize in (False, True):
        _, d = lib.route_grad(x.cuda(), chosen, dw.cuda(), counts, sums, 1.0, keep=keep.cuda(), normalize=normalize)
        clean = torch.where(chosen.cpu() < 0, 0.0, dw)
        check_grad_values(x, chosen.cpu(), clean, counts.cpu(), 1.0, keep, normalize, d)
    odd = chosen.cpu().clone()
    odd[5] = torch.tensor([e, -7, 2 ** 31 - 1, 4], dtype=torch.int32)  # only 4 is an expert
    _, d = lib.route_grad(x.cuda(), odd.cuda(), clean.cuda(), counts, sums, 1.0, keep=keep.cuda())
    check_grad_values(x, odd, clean, counts.cpu(), 1.0, keep, True, d)


def test_grad_in_place_and_without_tokens(lib):
    x = logits(500, 70, torch.bfloat16, 13).cuda()
    chosen, _, counts, sums = lib.route(x, 4)
    dw = torch.randn(500, 4, device="cuda")
    _, want = lib.route_grad(x, chosen, dw, counts, sums, 1.0)
    y = x.clone()
    lib.route_grad(y, chosen, dw, counts, sums, 1.0, out=(torch.empty(1, device="cuda"), y))
    assert torch.equal(y, want)
    # a rank without tokens still reports the loss; nothing routed anywhere gives loss 0
    none = torch.empty(0, 70, dtype=torch.bfloat16, device="cuda")
    loss, _ = lib.route_grad(none, chosen[:0], None, counts, sums, 1.0)
    oracle.assert_within(loss, oracle.balance_loss(None, counts.cpu(), sums.cpu(), 4, 1.0).reshape(1), 1e-5)
    loss, d = lib.route_grad(x, chosen, None, torch.zeros_like(counts), torch.zeros_like(sums), 1.0)
    assert loss.item() == 0 and not d.any()


def test_other_stream_and_graph(lib):
    x = logits(3000, 128, torch.bfloat16, 14).cuda()
    want = [v.clone() for v in lib.route(x, 8)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = lib.route(x, 8, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = tuple(torch.empty_like(v) for v in want)
    dw = torch.randn(3000, 8, device="cuda")
    res = (torch.empty(1, device="cuda"), torch.empty_like(x))
    ref = lib.route_grad(x, want[0], dw, want[2], want[3], 0.1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.route(x, 8, out=out)
        lib.route_grad(x, out[0], dw, out[2], out[3], 0.1, out=res)
    for _ in range(3):
        for v in out + res:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)) and all(torch.equal(a, b) for a, b in zip(res, ref))


def test_offsets_past_32_bits(lib):
    e, rows, ld = 64, 5, 1 << 30
    big = torch.empty(4 * ld + e, dtype=torch.bfloat16, device="cuda")
    part = big.as_strided((rows, e), (ld, 1))
    x = logits(rows, e, torch.bfloat16, 15)
    part.copy_(x)
    got = check_route(lib, x, 6, None, True, xd=part)
    dw = torch.randn(rows, 6, device="cuda")
    lib.route_grad(part, got[0], dw, got[2], got[3], 1.0, out=(torch.empty(1, device="cuda"), part))
    check_grad_values(x, got[0].cpu(), dw.cpu(), got[2].cpu(), 1.0, None, True, part)


def test_refusals(lib):
    x = torch.zeros(4, 16, dtype=torch.bfloat16, device="cuda")
    c = torch.zeros(4, 2, dtype=torch.int32, device="cuda")
    w = torch.zeros(4, 2, device="cuda")
    n = torch.zeros(17, dtype=torch.int32, device="cuda")
    s = torch.zeros(16, device="cuda")
    good = dict(logits=x.data_ptr(), row_stride=16, dtype="bf16", keep=None, tokens=4, experts=16, topk=2, normalize=1,
                chosen=c.data_ptr(), weights=w.data_ptr(), counts=n.data_ptr(), prob_sums=s.data_ptr(), work=None,
                work_bytes=0, stream=0)
    assert lib.sim_route(**good) == 0
    for change, status in ((dict(dtype="int32"), -1), (dict(dtype=9), -1), (dict(experts=0), -1),
                           (dict(experts=1025, row_stride=1025), -1), (dict(topk=0), -1), (dict(topk=17), -1),
                           (dict(topk=33, experts=40, row_stride=40), -1), (dict(tokens=-1), -1),
                           (dict(row_stride=15), -1), (dict(logits=None), -1), (dict(counts=None), -1),
                           (dict(weights=None), -1), (dict(logits=x.data_ptr() + 1), -3),
                           (dict(chosen=c.data_ptr() + 2), -3), (dict(chosen=x.data_ptr()), -4),
                           (dict(weights=c.data_ptr()), -4), (dict(tokens=2 ** 31), -1),
                           (dict(row_stride=2 ** 60), -1)):
        assert lib.sim_route(**{**good, **change}) == status, change
    need = lib.sim_route_work(100000, 16, 2, "bf16")
    assert need > 0
    many = torch.zeros(100000, 16, dtype=torch.bfloat16, device="cuda")
    mc, mw = torch.zeros(100000, 2, dtype=torch.int32, device="cuda"), torch.zeros(100000, 2, device="cuda")
    work = torch.zeros(need, dtype=torch.uint8, device="cuda")
    big = {**good, "logits": many.data_ptr(), "tokens": 100000, "chosen": mc.data_ptr(), "weights": mw.data_ptr()}
    assert lib.sim_route(**big) == -1
    assert lib.sim_route(**{**big, "work": work.data_ptr(), "work_bytes": need - 1}) == -5
    assert lib.sim_route(**{**big, "work": work.data_ptr(), "work_bytes": need}) == 0
    d = torch.zeros_like(x)
    one = torch.zeros(1, device="cuda")
    grad = dict(logits=x.data_ptr(), row_stride=16, dtype="bf16", keep=None, tokens=4, experts=16, topk=2, normalize=1,
                chosen=c.data_ptr(), dweights=w.data_ptr(), counts=n.data_ptr(), prob_sums=s.data_ptr(), coef=1.0,
                dlogits=d.data_ptr(), drow_stride=16, loss=one.data_ptr(), stream=0)
    assert lib.sim_route_grad(**grad) == 0
    for change, status in ((dict(prob_sums=None), -1), (dict(loss=None), -1), (dict(dlogits=None), -1),
                           (dict(chosen=None), -1), (dict(drow_stride=8), -1), (dict(dlogits=x.data_ptr() + 2), -4),
                           (dict(dlogits=x.data_ptr(), drow_stride=17), -4), (dict(loss=s.data_ptr()), -4),
                           (dict(dlogits=d.data_ptr() + 1), -3)):
        assert lib.sim_route_grad(**{**grad, **change}) == status, change
    assert lib.sim_route_grad(**{**grad, "dlogits": x.data_ptr()}) == 0
    with pytest.raises(ValueError):
        lib.route(x.t(), 2)
    with pytest.raises(ValueError):
        lib.route(x.cpu(), 2)
    with pytest.raises(ValueError):
        lib.route(x, 2, keep=torch.ones(3, dtype=torch.bool, device="cuda"))
    with pytest.raises(lib.SimError):
        lib.route(x, 40)
    torch.cuda.synchronize()


@pytest.mark.parametrize("t,e,k", [(96, 8, 2), (97, 256, 8), (700, 100, 16), (1024, 256, 8), (2048, 64, 8), (2049, 64, 8),
                                   (512, 512, 4)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_sums_of_a_graph_have_the_bits_of_a_call(lib, t, e, k, dtype):
    """A captured call adds up its workgroups' sums in a launch of its own."""
    x = logits(t, e, dtype, 23).cuda()
    want = [v.clone() for v in lib.route(x, k)]
    out = tuple(torch.empty_like(v) for v in want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.route(x, k, out=out)
    for _ in range(3):
        for v in out:
            v.zero_()
        graph.replay()
        again = lib.route(x, k)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) and torch.equal(c, b) for a, b, c in zip(out, want, again))


def test_small_calls_on_several_streams_at_once(lib):
    t = 1500
    xs = [logits(t, 64, torch.bfloat16, 30 + i).cuda() for i in range(6)]
    want = [[v.clone() for v in lib.route(x, 6)] for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in xs]
    got = [[] for _ in xs]
    for _ in range(20):
        for x, s, g in zip(xs, streams, got):
            g.append(lib.route(x, 6, stream=s))
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(a, b) for call in g for a, b in zip(call, w))


def test_more_streams_than_counters(lib):
    import ctypes
    hip = ctypes.CDLL("libamdhip64.so")
    x = logits(500, 32, torch.float16, 41).cuda()
    want = [v.clone() for v in lib.route(x, 4)]
    torch.cuda.synchronize()
    raw = []
    try:
        for _ in range(70):
            s = ctypes.c_void_p()
            assert hip.hipStreamCreate(ctypes.byref(s)) == 0
            raw.append(s)
        out = [tuple(torch.empty_like(v) for v in want) for _ in raw]
        torch.cuda.synchronize()
        for s, o in zip(raw, out):
            lib.route(x, 4, out=o, stream=torch.cuda.ExternalStream(s.value))
        torch.cuda.synchronize()
    finally:
        for s in raw:
            hip.hipStreamDestroy(s)
    assert all(torch.equal(a, b) for o in out for a, b in zip(o, want))


@pytest.mark.parametrize("e,k", [(16, 5), (32, 32), (60, 8), (128, 20), (256, 8), (500, 16), (1000, 32)])
def test_fp32_logits_a_bit_apart(lib, e, k):
    """Neighbouring values, of either sign and below the smallest normal number, are told apart to the last bit."""
    g = torch.Generator().manual_seed(e)
    order = torch.rand(200, e, generator=g).argsort(1).float()
    x = 1.0 + order * 2.0 ** -23
    x[50:100] = -1.0 - order[50:100] * 2.0 ** -23
    x[100:150] = (order[100:150] - e // 2) * 2.0 ** -149
    x[150:] = torch.where(order[150:] < e // 2, 2.0 * order[150:] / e, x[150:])
    check_route(lib, x, k, None, True)
    check_route(lib, x, k, None, False)


def nan_with_the_sign_set(dtype):
    bits, as_int = {torch.float32: (-0x400000, torch.int32), torch.float16: (-0x200, torch.int16),
                    torch.bfloat16: (-0x40, torch.int16)}[dtype]
    v = torch.tensor([bits], dtype=as_int).view(dtype)
    assert torch.isnan(v).all() and torch.signbit(v).all()
    return v


@pytest.mark.parametrize("e,k", [(4, 2), (30, 4), (32, 20), (64, 8), (100, 6), (256, 8), (256, 12), (500, 8), (1000, 32)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_nan_with_the_sign_set(lib, dtype, e, k):
    """Such a NaN orders below -inf; its row is live and not a number all the same, forward and backward."""
    nan = nan_with_the_sign_set(dtype)
    dw = torch.randn(70, k, generator=torch.Generator().manual_seed(7))
    for rows in ("nan", "nan and -inf", "one nan", "one nan among -inf"):
        x = logits(70, e, dtype, 50 + e)
        if rows in ("nan and -inf", "one nan among -inf"):
            x[[0, 33]] = -INF
        x[[0, 33], (slice(None) if rows == "nan" else slice(1, e, 2) if rows == "nan and -inf" else e // 2)] = nan
        for normalize in (True, False):
            got = check_route(lib, x, k, None, normalize)
            assert got[2][e].item() == 70 and torch.isnan(got[3]).all(), rows
            _, d = lib.route_grad(x.cuda(), got[0], dw.cuda(), got[2], torch.ones(e, device="cuda"), 1.0,
                                  normalize=normalize)
            check_grad_values(x, got[0].cpu(), dw, got[2].cpu(), 1.0, None, normalize, d)


@pytest.mark.parametrize("normalize", [False, True])
@pytest.mark.parametrize("dtype", DTYPES)
def test_empty_rows_get_zeros_whatever_their_slots_and_coef_hold(lib, dtype, normalize):
    t, e, k = 300, 40, 4
    x = logits(t, e, dtype, 60)
    keep = torch.arange(t) % 4 != 1
    x[2] = -INF
    empty = ~keep
    empty[2] = True
    chosen, _, counts, sums = lib.route(x.cuda(), k, normalize=normalize)  # every row has slots
    chosen[2] = torch.arange(k, dtype=torch.int32, device="cuda")
    dw = torch.randn(t, k, generator=torch.Generator().manual_seed(8))
    odd = dw.clone()
    odd[empty] = torch.tensor([float("nan"), INF, -INF, 1.0])
    _, d = lib.route_grad(x.cuda(), chosen, odd.cuda(), counts, sums, 1.0, keep=keep.cuda(), normalize=normalize)
    assert not d[empty.cuda()].any()
    check_grad_values(x, chosen.cpu(), torch.where(empty[:, None], 0.0, dw), counts.cpu(), 1.0, keep, normalize, d)
    for coef in (INF, float("nan")):
        _, d = lib.route_grad(x.cuda(), chosen, dw.cuda(), counts, sums, coef, keep=keep.cuda(), normalize=normalize)
        assert not d[empty.cuda()].any() and torch.isnan(d[~empty.cuda()]).all()


def test_streams_that_come_and_go_keep_the_one_launch_form(lib):
    """However many streams a process has made, a small call's workgroups add up their own sums."""
    import ctypes
    hip = ctypes.CDLL("libamdhip64.so")
    x = logits(500, 32, torch.bfloat16, 61).cuda()
    want = [v.clone() for v in lib.route(x, 4)]
    out = tuple(torch.empty_like(v) for v in want)
    torch.cuda.synchronize()
    for _ in range(150):
        s = ctypes.c_void_p()
        assert hip.hipStreamCreate(ctypes.byref(s)) == 0
        try:
            lib.route(x, 4, out=out, stream=torch.cuda.ExternalStream(s.value))
            assert lib.sim_debug_get("route_launches") == 1
        finally:
            torch.cuda.synchronize()
            hip.hipStreamDestroy(s)
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        for v in out:
            v.zero_()


def test_many_small_calls_in_a_row(lib):
    """More calls than the library has counters, waited for and not; a captured call takes none."""
    x = logits(700, 24, torch.float32, 62).cuda()
    want = [v.clone() for v in lib.route(x, 3)]
    out = tuple(torch.empty_like(v) for v in want)
    for n in (1, 500, 4096, 5000, 9000):
        for v in out:
            v.zero_()
        for _ in range(n):
            lib.route(x, 3, out=out)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)), n
    lib.route(x, 3, out=out)
    assert lib.sim_debug_get("route_launches") == 1
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        lib.route(x, 3, out=out)
        assert lib.sim_debug_get("route_launches") == 2
    for _ in range(3):
        for v in out:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_the_per_thread_stream(lib):
    t, e, k = 900, 48, 5
    x = logits(t, e, torch.bfloat16, 63).cuda()
    want = lib.route(x, k)
    out = tuple(torch.zeros_like(v) for v in want)
    need = lib.sim_route_work(t, e, k, "bf16")
    work = torch.empty(need, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert lib.sim_route(x.data_ptr(), e, "bf16", None, t, e, k, 1, *(v.data_ptr() for v in out), work.data_ptr(), need,
                         stream=2) == 0  # hipStreamPerThread
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("t,e,k", [(40003, 256, 8), (9001, 1024, 32), (70001, 100, 12), (140007, 32, 4)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("normalize", [False, True])
def test_more_rows_than_the_grid_takes_at_once(lib, dtype, normalize, t, e, k):
    """Every workgroup goes over its rows several times: a few distinct rows over and over, each repeat with the bits
    of the first."""
    n = 37
    x = logits(n, e, dtype, 70 + e)
    x[5] = -INF
    keep = torch.arange(n) % 7 != 3
    x[~keep] = float("nan")
    pick = torch.arange(t) % n
    reps = torch.bincount(pick, minlength=n)
    on = pick.cuda()
    xd, kd = x.cuda()[on], keep.cuda()[on]
    chosen, w, counts, sums = lib.route(xd, k, keep=kd, normalize=normalize)
    want, ww, _, _, wtol, _ = oracle.route(x, k, keep, normalize)
    assert torch.equal(chosen[:n].cpu(), want)
    oracle.assert_within(w[:n], ww, wtol, "weights")
    assert torch.equal(chosen, chosen[:n][on]) and torch.equal(w, w[:n][on])
    each = [oracle.route(x[i:i + 1], k, keep[i:i + 1], normalize) for i in range(n)]
    assert torch.equal(counts.cpu().long(), sum(int(reps[i]) * r[2].long() for i, r in enumerate(each)))
    total = sum(int(reps[i]) * r[3] for i, r in enumerate(each))
    oracle.assert_within(sums, total, sum(int(reps[i]) * r[5] for i, r in enumerate(each)) + t * oracle.U * total, "prob_sums")
    dw = torch.randn(n, k, generator=torch.Generator().manual_seed(9))
    dwd = dw.cuda()[on]
    loss, d = lib.route_grad(xd, chosen, dwd, counts, sums, 30.0, keep=kd, normalize=normalize)
    check_grad_values(x, want, dw, counts.cpu(), 30.0, keep, normalize, d[:n])
    assert torch.equal(d, d[:n][on])
    oracle.assert_within(loss, oracle.balance_loss(None, counts.cpu(), sums.cpu(), k, 30.0).reshape(1),
                         (e + 16) * oracle.U * loss.abs().cpu().double())
    lib.route_grad(xd, chosen, dwd, counts, sums, 30.0, keep=kd, normalize=normalize, out=(loss, xd))  # over its logits
    assert torch.equal(xd, d)
