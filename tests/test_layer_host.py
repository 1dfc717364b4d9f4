"""Norm, expert dispatch and clipping without a GPU: the entry points' own
argument checks (compiled for the host, with stand-ins for the launches), the
entry points before sim_init, the 64-bit oracle of the GPU tests against
automatic differentiation and differences."""
import ctypes
import os
import shutil
import subprocess

import pytest
import torch

from tests import layer_oracle as oracle

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "all_reduce_reduction_amd", "csrc")
HIP = os.environ.get("ROCM_PATH", "/opt/rocm")
INVALID, ALIGN, ALIAS, NOMEM = -1, -3, -4, -5
NAMES = ("sim_norm", "sim_norm_grad_work", "sim_norm_grad", "sim_dispatch_work", "sim_dispatch", "sim_combine",
         "sim_combine_grad", "sim_clip_work", "sim_clip_norm", "sim_clip")


@pytest.fixture(scope="module")
def checks(tmp_path_factory):
    """The entry points over stand-ins; a call's launches are counted, not made."""
    import all_reduce_reduction_amd as sim
    cxx = shutil.which("g++")
    if cxx is None or not os.path.isdir(os.path.join(HIP, "include", "hip")):
        pytest.skip("no g++ or no HIP headers")
    out = str(tmp_path_factory.mktemp("layer") / "checks.so")
    subprocess.run([cxx, "-std=c++17", "-O1", "-Wall", "-shared", "-fPIC", "-D__HIP_PLATFORM_AMD__",
                    "-I", os.path.join(HIP, "include"), "-I", os.path.join(ROOT, "include"), "-I", CSRC,
                    os.path.join(ROOT, "tests", "layer_checks_stub.cpp"), os.path.join(CSRC, "api_layer.cpp"),
                    os.path.join(CSRC, "layer_sizes.cpp"), "-o", out], check=True, capture_output=True, text=True)
    lib = ctypes.CDLL(out)
    for name in NAMES:
        getattr(lib, name).argtypes = getattr(sim.lib, name).argtypes
        getattr(lib, name).restype = ctypes.c_int
    return lib


A, B, C, D, E, F = (0x10000000 * (i + 1) for i in range(6))  # addresses of arrays that are never touched
FP32, FP16, BF16 = 1, 2, 3


def run(checks, name, good, change, status):
    before = checks.stub_launches()
    assert getattr(checks, name)(*{**good, **change}.values()) == status, (name, change)
    assert (checks.stub_launches() > before) == (status == 0), (name, change)
    assert checks.stub_bad() == 0, (name, change)


def test_norm_checks(checks):
    good = dict(x=A, x_stride=100, dtype=BF16, residual=B, residual_stride=100, rows=7, columns=100, gain=C, gain_dtype=FP32,
                eps=1e-6, sum=D, sum_stride=100, out=E, out_stride=100, scales=None, group=0, stream=None)
    for change in ({}, dict(gain=None), dict(sum=None), dict(residual=None, sum=None), dict(sum=A), dict(sum=B), dict(out=A),
                   dict(out=B), dict(sum=B, out=A), dict(dtype=FP32, gain_dtype=BF16), dict(scales=F, group=0),
                   dict(scales=F, group=32), dict(scales=F, group=128, out=E + 1), dict(columns=32768, x_stride=32768, residual_stride=32768,
                   sum_stride=32768, out_stride=32768), dict(x_stride=200, out=A + 200, out_stride=200),
                   dict(group=77)):  # (without scales there is no group)
        run(checks, "sim_norm", good, change, 0)
    for change, status in ((dict(dtype=0), INVALID), (dict(dtype=4), INVALID), (dict(gain_dtype=0), INVALID),
                           (dict(eps=0.0), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
                           (dict(eps=1e38), INVALID), (dict(rows=-1), INVALID), (dict(rows=2 ** 31), INVALID),
                           (dict(columns=0), INVALID), (dict(columns=32769, x_stride=40000), INVALID),
                           (dict(x_stride=99), INVALID), (dict(residual_stride=99), INVALID), (dict(sum_stride=99), INVALID),
                           (dict(out_stride=99), INVALID), (dict(x_stride=2 ** 60), INVALID), (dict(x=None), INVALID),
                           (dict(out=None), INVALID), (dict(residual=None), INVALID), (dict(scales=F, group=16), INVALID),
                           (dict(scales=F, group=-1), INVALID), (dict(scales=F, group=256), INVALID),
                           (dict(x=A + 1), ALIGN), (dict(gain=C + 2), ALIGN), (dict(scales=F + 2, group=32), ALIGN),
                           (dict(out=A + 2), ALIAS), (dict(sum=A, out=A), ALIAS), (dict(sum=E), ALIAS), (dict(out=C), ALIAS),
                           (dict(sum=B, sum_stride=101), ALIAS), (dict(out=A, scales=F, group=32), ALIAS),
                           (dict(scales=A, group=32), ALIAS), (dict(scales=E, group=32), ALIAS), (dict(sum=C), ALIAS)):
        run(checks, "sim_norm", good, change, status)
    assert checks.sim_norm(*{**good, "rows": 0, "x": None, "out": None}.values()) == 0


def test_norm_grad_checks(checks):
    need = ctypes.c_size_t()
    assert checks.sim_norm_grad_work(7, 2000, BF16, ctypes.byref(need)) == 0 and need.value == 7 * 2000 * 4
    assert checks.sim_norm_grad_work(1, 100, BF16, ctypes.byref(need)) == 0 and need.value == 0
    for bad in ((-1, 100, BF16), (7, 0, BF16), (7, 40000, BF16), (7, 100, 0)):
        assert checks.sim_norm_grad_work(*bad, ctypes.byref(need)) == INVALID
    assert checks.sim_norm_grad_work(7, 100, BF16, None) == INVALID
    good = dict(h=A, h_stride=2000, dtype=BF16, rows=7, columns=2000, gain=B, gain_dtype=BF16, eps=1e-6, dy=C, dy_stride=2000,
                dsum=D, dsum_stride=2000, dx=E, dx_stride=2000, dgain=F, work=F + 0x10000, work_bytes=56000, stream=None)
    for change in ({}, dict(dsum=None), dict(gain=None), dict(dgain=None, work=None, work_bytes=0), dict(dx=A), dict(dx=C),
                   dict(dx=D), dict(rows=1, work=None, work_bytes=0), dict(rows=0, h=None, dy=None, dx=None, work=None)):
        run(checks, "sim_norm_grad", good, change, 0)
    for change, status in ((dict(h=None), INVALID), (dict(dy=None), INVALID), (dict(dx=None), INVALID), (dict(work=None), INVALID),
                           (dict(work_bytes=55999), NOMEM), (dict(work=F + 0x10002), ALIGN), (dict(dgain=F + 1), ALIGN),
                           (dict(dx=B), ALIAS), (dict(dgain=A), ALIAS), (dict(dgain=E), ALIAS), (dict(work=F), ALIAS),
                           (dict(dx=A, dx_stride=2001), ALIAS), (dict(dx=C + 2), ALIAS), (dict(dy_stride=5), INVALID),
                           (dict(dsum_stride=5), INVALID), (dict(eps=0.0), INVALID), (dict(dtype=7), INVALID)):
        run(checks, "sim_norm_grad", good, change, status)


def test_dispatch_checks(checks):
    need = ctypes.c_size_t()
    assert checks.sim_dispatch_work(512, 8, 256, ctypes.byref(need)) == 0 and need.value == 0
    assert checks.sim_dispatch_work(20000, 8, 256, ctypes.byref(need)) == 0 and need.value > 0 and need.value % (256 * 4) == 0
    for bad in ((-1, 8, 8), (1, 0, 8), (1, 33, 64), (1, 1, 0), (1, 1, 1025), (2 ** 28, 8, 8)):
        assert checks.sim_dispatch_work(*bad, ctypes.byref(need)) == INVALID
    assert checks.sim_dispatch_work(40000, 4, 16, ctypes.byref(need)) == 0
    many = need.value
    good = dict(x=A, x_pitch=200, row_bytes=200, scales=None, groups=0, chosen=B, tokens=10, topk=4, experts=16, rows=C,
                rows_pitch=200, row_scales=None, place=D, offsets=E, work=None, work_bytes=0, stream=None)
    for change in ({}, dict(x=A + 1, rows=C + 3), dict(row_bytes=0, x=None, rows=None, x_pitch=0, rows_pitch=0),
                   dict(scales=F, groups=3, row_scales=F + 0x1000), dict(tokens=0, x=None, rows=None, chosen=None, place=None),
                   dict(tokens=40000, work=F, work_bytes=many), dict(x_pitch=600, rows=A + 200, rows_pitch=600),
                   dict(experts=1024, topk=32)):
        run(checks, "sim_dispatch", good, change, 0)
    for change, status in ((dict(tokens=-1), INVALID), (dict(topk=0), INVALID), (dict(topk=33), INVALID), (dict(experts=0), INVALID),
                           (dict(experts=1025), INVALID), (dict(tokens=2 ** 30), INVALID), (dict(x_pitch=199), INVALID),
                           (dict(rows_pitch=199), INVALID), (dict(row_bytes=-1), INVALID), (dict(x=None), INVALID),
                           (dict(rows=None), INVALID), (dict(chosen=None), INVALID), (dict(place=None), INVALID),
                           (dict(offsets=None), INVALID), (dict(groups=3, scales=F), INVALID), (dict(groups=-1), INVALID),
                           (dict(groups=3, row_scales=F), INVALID), (dict(tokens=40000), INVALID),
                           (dict(tokens=40000, work=F, work_bytes=many - 1), NOMEM), (dict(chosen=B + 2), ALIGN),
                           (dict(place=D + 1), ALIGN), (dict(offsets=E + 2), ALIGN), (dict(rows=A), ALIAS), (dict(place=B), ALIAS),
                           (dict(offsets=D), ALIAS), (dict(rows=D), ALIAS), (dict(x=C + 7999), ALIAS),
                           (dict(scales=F, groups=3, row_scales=F + 8), ALIAS)):
        run(checks, "sim_dispatch", good, change, status)


def test_combine_checks(checks):
    good = dict(rows=A, rows_stride=50, dtype=FP16, nrows=40, columns=50, place=B, weights=C, tokens=10, topk=4, out=D,
                out_stride=50, stream=None)
    for change in ({}, dict(weights=None), dict(nrows=0, rows=None), dict(columns=2 ** 30, rows_stride=2 ** 30, out_stride=2 ** 30, nrows=1,
                                                                         tokens=1, rows=A, out=2 ** 44, place=2 ** 45, weights=2 ** 46)):
        run(checks, "sim_combine", good, change, 0)
    assert checks.sim_combine(*{**good, "tokens": 0, "out": None}.values()) == 0
    for change, status in ((dict(dtype=0), INVALID), (dict(nrows=-1), INVALID), (dict(columns=0), INVALID), (dict(rows=None), INVALID),
                           (dict(place=None), INVALID), (dict(out=None), INVALID), (dict(topk=33), INVALID), (dict(tokens=-5), INVALID),
                           (dict(rows_stride=49), INVALID), (dict(out_stride=49), INVALID), (dict(columns=2 ** 31, rows_stride=2 ** 31), INVALID),
                           (dict(rows=A + 1), ALIGN), (dict(place=B + 2), ALIGN), (dict(weights=C + 1), ALIGN), (dict(out=A), ALIAS),
                           (dict(out=B), ALIAS), (dict(out=C), ALIAS)):
        run(checks, "sim_combine", good, change, status)


def test_combine_grad_checks(checks):
    good = dict(dy=A, dy_stride=50, dtype=FP32, rows=B, rows_stride=50, nrows=40, columns=50, place=C, weights=D, tokens=10,
                topk=4, drows=E, drows_stride=50, dweights=F, stream=None)
    for change in ({}, dict(weights=None), dict(drows=None), dict(dweights=None), dict(dweights=None, rows=None), dict(drows=B),
                   dict(nrows=0, rows=None)):
        run(checks, "sim_combine_grad", good, change, 0)
    assert checks.sim_combine_grad(*{**good, "tokens": 0, "dy": None}.values()) == 0
    for change, status in ((dict(drows=None, dweights=None), INVALID), (dict(dy=None), INVALID), (dict(place=None), INVALID),
                           (dict(rows=None), INVALID), (dict(dtype=0), INVALID), (dict(dy_stride=1), INVALID),
                           (dict(rows_stride=1), INVALID), (dict(drows_stride=1), INVALID), (dict(topk=0), INVALID),
                           (dict(dy=A + 2), ALIGN), (dict(drows=A), ALIAS), (dict(drows=B + 4), ALIAS), (dict(drows=B, drows_stride=51), ALIAS),
                           (dict(dweights=D), ALIAS), (dict(dweights=C), ALIAS), (dict(dweights=E), ALIAS), (dict(dweights=F + 2), ALIGN)):
        run(checks, "sim_combine_grad", good, change, status)


def lists(ptrs, counts, dtypes):
    return ((ctypes.c_void_p * len(ptrs))(*ptrs), (ctypes.c_int64 * len(counts))(*counts), (ctypes.c_int * len(dtypes))(*dtypes))


def test_clip_checks(checks):
    need = ctypes.c_size_t()

    def work(counts, dtypes):
        _, c, d = lists([], counts, dtypes)
        assert checks.sim_clip_work(c, d, len(counts), ctypes.byref(need)) == 0
        return need.value

    assert work([], []) == 0 and work([0, 0], [FP32, BF16]) == 0
    assert work([1], [FP32]) == 8 and work([4096], [FP32]) == 8 and work([4097, 5], [FP32, BF16]) == 24
    assert work([2 ** 30], [BF16]) == 8 * 2048
    assert work([1] * 1000, [FP32] * 1000) == 8000
    _, c, d = lists([], [1, -1], [FP32, FP32])
    assert checks.sim_clip_work(c, d, 2, ctypes.byref(need)) == INVALID
    _, c, d = lists([], [1], [0])
    assert checks.sim_clip_work(c, d, 1, ctypes.byref(need)) == INVALID
    assert checks.sim_clip_work(None, None, 1, ctypes.byref(need)) == INVALID
    assert checks.sim_clip_work(c, d, 70000, ctypes.byref(need)) == INVALID

    def clip(ptrs, counts, dtypes, outs=None, n=None, parts=None, nparts=0, max_norm=1.0, norm=F, work=E, work_bytes=1 << 20):
        p, c, d = lists(ptrs, counts, dtypes)
        o = None if outs is None else (ctypes.c_void_p * len(outs))(*outs)
        before = checks.stub_launches()
        rc = checks.sim_clip(p, o, c, d, len(ptrs) if n is None else n, parts, nparts, max_norm, norm, work, work_bytes, None)
        assert (checks.stub_launches() > before) == (rc == 0) and checks.stub_bad() == 0
        only = checks.sim_clip_norm(p, c, d, len(ptrs) if n is None else n, norm, work, work_bytes, None)
        assert checks.stub_bad() == 0
        return rc, only

    two = ([A, B], [1000, 77], [BF16, FP32])
    assert clip(*two) == (0, 0) and clip([], [], []) == (0, 0) and clip(*two, max_norm=float("inf")) == (0, 0)
    assert clip([A, None], [5, 0], [FP16, FP16]) == (0, 0)
    assert clip(*two, outs=[C, D]) == (0, 0) and clip(*two, outs=[A, D]) == (0, 0) and clip(*two, outs=[A, B]) == (0, 0)
    assert clip(*two, parts=C, nparts=8, work=None, work_bytes=0)[0] == 0
    many = ([A + 64 * i for i in range(1000)], [16] * 1000, [FP32] * 1000)
    assert clip(*many) == (0, 0) and clip(*many, parts=C, nparts=8)[0] == 0
    assert clip(*many[:2], [BF16] * 1000, outs=[A + 64 * i + 32 for i in range(1000)]) == (0, 0)  # between each other
    assert clip([A] * 3, [10] * 3, [BF16] * 3) == (ALIAS, 0)  # scaled once for each time it is listed
    assert clip([A, A + 1998], [1000, 10], [BF16] * 2) == (ALIAS, 0)
    assert clip([A, A + 2000], [1000, 10], [BF16] * 2) == (0, 0)
    assert clip(*two, outs=[C, C + 100])[0] == ALIAS and clip(*two, outs=[B, D])[0] == ALIAS and clip(*two, outs=[A + 2, D])[0] == ALIAS
    assert clip(*two, norm=A) == (ALIAS, ALIAS) and clip(*two, work=A) == (ALIAS, ALIAS) and clip(*two, norm=E) == (ALIAS, ALIAS)
    assert clip(*two, outs=[C, D], norm=C)[0] == ALIAS and clip(*two, parts=F, nparts=2)[0] == ALIAS
    assert clip(*two, parts=A, nparts=2)[0] == ALIAS
    assert clip([A + 1, B], *two[1:]) == (ALIGN, ALIGN) and clip([A, B + 2], *two[1:]) == (ALIGN, ALIGN)
    assert clip(*two, outs=[C, D + 2])[0] == ALIGN and clip(*two, norm=F + 2) == (ALIGN, ALIGN)
    assert clip(*two, work=E + 4) == (ALIGN, ALIGN) and clip(*two, parts=C + 1, nparts=1)[0] == ALIGN
    assert clip([None, B], *two[1:]) == (INVALID, INVALID) and clip(*two, outs=[C, None])[0] == INVALID
    assert clip([A, B], [1000, 77], [BF16, 0]) == (INVALID, INVALID) and clip([A, B], [-1, 77], two[2]) == (INVALID, INVALID)
    assert clip(*two, n=-1) == (INVALID, INVALID) and clip(*two, norm=None) == (INVALID, INVALID)
    assert clip(*two, max_norm=-1.0)[0] == INVALID and clip(*two, max_norm=float("nan"))[0] == INVALID
    assert clip(*two, parts=C, nparts=0)[0] == INVALID and clip(*two, parts=None, nparts=2)[0] == INVALID
    assert clip(*two, work=None) == (INVALID, INVALID) and clip(*two, work_bytes=15) == (NOMEM, NOMEM)
    assert checks.sim_clip(None, None, None, None, 3, None, 0, 1.0, F, E, 1 << 20, None) == INVALID


def test_refused_before_init():
    import all_reduce_reduction_amd as sim
    sim.sim_finalize()
    assert sim.sim_norm(None, 8, "bf16", None, 8, 0, 8, None, "bf16", 1e-6, None, 8, None, 8, None, 0) == -9
    assert sim.sim_norm_grad(None, 8, "bf16", 0, 8, None, "bf16", 1e-6, None, 8, None, 8, None, 8, None, None, 0) == -9
    assert sim.sim_dispatch(None, 8, 8, None, 0, None, 0, 1, 8, None, 8, None, None, None, None, 0) == -9
    assert sim.sim_combine(None, 8, "bf16", 0, 8, None, None, 0, 1, None, 8) == -9
    assert sim.sim_combine_grad(None, 8, "bf16", None, 8, 0, 8, None, None, 0, 1, None, 8, None) == -9
    assert sim.sim_clip_norm([], [], [], None, None, 0) == -9
    assert sim.sim_clip([], None, [], [], None, 0, 1.0, None, None, 0) == -9
    for f in (lambda: sim.sim_norm_grad_work(1, 8, "bf16"), lambda: sim.sim_dispatch_work(1, 8, 8),
              lambda: sim.sim_clip_work([1], ["bf16"])):
        with pytest.raises(sim.SimError):
            f()


def test_helpers_refuse_host_tensors():
    import all_reduce_reduction_amd as sim
    x, i = torch.zeros(4, 8), torch.zeros(2, 2, dtype=torch.int32)
    for f in (lambda: sim.norm(x), lambda: sim.norm_quant(x), lambda: sim.norm_grad(x, None, x), lambda: sim.dispatch(x, i, 4),
              lambda: sim.combine(x, i), lambda: sim.dispatch_grad(x, i), lambda: sim.combine_grad(x, x, i),
              lambda: sim.grad_norm([x]), lambda: sim.clip_grads([x], 1.0)):
        with pytest.raises(ValueError):
            f()


def test_tensor_extension_is_built_and_survives_what_is_no_tensor():
    import all_reduce_reduction_amd as sim
    assert sim._pytensor is not None, "the tensor extension is not built"
    for call in (lambda: sim._rows(3, "x", None), lambda: sim._raw("x", "x", None), lambda: sim._rows(torch.zeros(2, 2), "x"),
                 lambda: sim._vec([1], "x", (torch.float32,), 0, 1), lambda: sim._vec(torch.zeros(1), "x", 7, 0, 1),
                 lambda: sim._gain(1.0, 2, 0), lambda: sim._gain(torch.zeros(2), "two", 0), lambda: sim._like(None, "x", (1, 2)),
                 lambda: sim._tensors([1, 2], "l", 0, None), lambda: sim._tensors(None, "l", 0, None),
                 lambda: sim._slots(None, None, (), 1, 0), lambda: sim._slots(torch.zeros(1, 1), 5, (torch.float32,), 1, 0)):
        with pytest.raises(TypeError):
            call()
    meta = torch.zeros(2, 3, device="meta")
    for call in (lambda: sim._rows(meta, "x", None), lambda: sim._vec(meta, "x", (torch.float32,), 0, 2, 3),
                 lambda: sim._tensors([meta], "l", 0, None), lambda: sim._rows(torch.zeros(2, 3).to_sparse(), "x", None)):
        with pytest.raises(ValueError):
            call()


def test_limits_match_the_header():
    import re

    import all_reduce_reduction_amd as sim
    text = open(os.path.join(ROOT, "include", "simar.h")).read()
    for name in ("NORM_MAX_COLUMNS", "CLIP_MAX_TENSORS"):
        assert getattr(sim, name) == int(re.search(rf"#define SIM_{name} (\d+)", text).group(1))


@pytest.mark.parametrize("with_residual", [False, True])
def test_norm_gradient_is_that_of_the_objective(with_residual):
    g = torch.Generator().manual_seed(1)
    x, res, dy, dt = (torch.randn(5, 12, generator=g, dtype=torch.float64) for _ in range(4))
    gain = 1 + 0.1 * torch.randn(12, generator=g, dtype=torch.float64)
    res, dt = (res, dt) if with_residual else (None, None)
    x.requires_grad_(True)
    gain.requires_grad_(True)
    oracle.norm_objective(x, gain, res, 1e-3, dy, dt).backward()
    h = oracle.norm(x.detach(), None, res, 1e-3)[0]
    dx, _, dg, _ = oracle.norm_grad(h, gain.detach(), dy, dt, 1e-3)
    assert torch.allclose(x.grad, dx, rtol=1e-12, atol=1e-13) and torch.allclose(gain.grad, dg, rtol=1e-12, atol=1e-13)
    # by differences: the error of a central difference is of the order of step^2
    with torch.no_grad():
        for got, at in ((dx, x), (dg, gain)):
            v = torch.randn(at.shape, generator=g, dtype=torch.float64)
            ends = []
            for sign in (1, -1):
                moved = at + sign * 1e-5 * v
                ends.append(oracle.norm_objective(*((moved, gain) if at is x else (x, moved)), res, 1e-3, dy, dt))
            assert abs((ends[0] - ends[1]) / 2e-5 - (got * v).sum()) < 1e-7


def test_expert_gradients_are_those_of_the_objective():
    g = torch.Generator().manual_seed(2)
    t, k, e, c = 9, 3, 5, 4
    chosen = torch.randint(-1, e + 1, (t, k), generator=g, dtype=torch.int32)
    place, offsets = oracle.places(chosen, e)
    m = int(offsets[e])
    assert sorted(p for p in place.reshape(-1).tolist() if p >= 0) == list(range(m)) and m < t * k
    x = torch.randn(t, c, generator=g, dtype=torch.float64, requires_grad=True)
    w = torch.rand(t, k, generator=g, dtype=torch.float64, requires_grad=True)
    scale = torch.randn(t * k, c, generator=g, dtype=torch.float64)  # stands for the experts
    dy = torch.randn(t, c, generator=g, dtype=torch.float64)

    def objective(x, w):
        total = 0.0
        for i in range(t):
            for j in range(k):
                p = int(place[i, j])
                if p >= 0:
                    total = total + (w[i, j] * x[i] * scale[p] * dy[i]).sum()
        return total

    objective(x, w).backward()
    rows = torch.zeros(t * k, c, dtype=torch.float64)
    for i in range(t):
        for j in range(k):
            if place[i, j] >= 0:
                rows[place[i, j]] = x.detach()[i] * scale[place[i, j]]
    y, _ = oracle.combine(rows, place, w.detach())
    assert abs((y * dy).sum() - objective(x, w).detach()) < 1e-12
    drows, dw, _ = oracle.combine_grad(dy, rows, place, w.detach())
    dx, _ = oracle.combine(torch.nan_to_num(drows) * scale, place, None)
    assert torch.allclose(w.grad, dw, rtol=1e-12, atol=1e-13) and torch.allclose(x.grad, dx, rtol=1e-12, atol=1e-13)
    assert torch.isnan(drows[m:]).all() and not torch.isnan(drows[:m]).any()
    with torch.no_grad():
        v, u = torch.randn(t, c, generator=g, dtype=torch.float64), torch.randn(t, k, generator=g, dtype=torch.float64)
        ends = [objective(x + s * 1e-5 * v, w + s * 1e-5 * u) for s in (1, -1)]
        assert abs((ends[0] - ends[1]) / 2e-5 - (dx * v).sum() - (dw * u).sum()) < 1e-8


# ---- the tensor extension -----------------------------------------------------------
def build_script():
    import importlib.util
    spec = importlib.util.spec_from_file_location("build_script", os.path.join(ROOT, "all_reduce_reduction_amd", "_build.py"))
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


@pytest.mark.parametrize("missing", ["headers", "torch"])
def test_a_build_without_torch_headers_leaves_the_tensor_extension_out(tmp_path, monkeypatch, missing):
    """The package treats it as optional, and so does the build; one that is there already is of another build."""
    import sys
    import sysconfig
    if missing == "headers":
        import torch.utils.cpp_extension as ext
        monkeypatch.setattr(ext, "include_paths", lambda *a, **k: [str(tmp_path)])
    else:
        monkeypatch.setitem(sys.modules, "torch", None)
    old = tmp_path / ("_pytensor" + sysconfig.get_config_var("EXT_SUFFIX"))
    old.write_bytes(b"of an earlier build")
    assert build_script().build_pytensor(str(tmp_path)) is None and not old.exists()


@pytest.mark.parametrize("version", [None, "1.0.0"])
def test_the_tensor_extension_is_of_the_torch_that_runs(version):
    """One that was built with another torch's headers may read tensors by the wrong layout: it is not used."""
    import sys
    import all_reduce_reduction_amd as sim
    if sim._pytensor is None:
        pytest.skip("the tensor extension is not built")
    code = ("import torch\n" + (f"torch.__version__ = {version!r}\n" if version else "") +
            "import all_reduce_reduction_amd as sim\n"
            "print(sim._pytensor is not None, sim._rows is sim._rows_py, sim._tensors is sim._tensors_py, sim._vec is sim._vec_py)")
    got = subprocess.run([sys.executable, "-c", code], cwd=ROOT, check=True, capture_output=True, text=True).stdout.split()
    assert got == (["False"] + ["True"] * 3 if version else ["True"] + ["False"] * 3)


def test_counts_read_by_all_chunks_do_not_grow_with_their_square(checks):
    """Each chunk's workgroup reads all chunks' counts, which are dispatch's scratch: at most 64 for each of its slots, with
    no fewer than half as many chunks as that allows."""
    for tokens, topk, experts in ((16384, 8, 256), (16384, 8, 1024), (16384, 16, 512), (65536, 8, 256), (16384, 32, 1024), (65536, 32, 1024),
                                  (1 << 20, 32, 1024), ((1 << 31) - 1, 1, 1024), (60000000, 32, 4), (4097, 4, 1024)):
        n = ctypes.c_size_t(0)
        assert checks.sim_dispatch_work(tokens, topk, experts, ctypes.byref(n)) == 0
        chunks = n.value // (4 * experts)
        assert chunks * (chunks - 1) * experts <= 64 * tokens * topk, (tokens, topk, experts, chunks)
        assert chunks >= min(tokens * topk // 1024, 256, (64 * tokens * topk / experts) ** 0.5 / 2.01), (tokens, topk, experts, chunks)
        at = [(i + 1) << 36 for i in range(4)]
        before = checks.stub_bad()
        assert checks.sim_dispatch(None, 0, 0, None, 0, at[0], tokens, topk, experts, None, 0, None, at[1], at[2], at[3], n.value, None) == 0
        assert checks.stub_bad() == before


def test_without_a_gains_gradient_rows_share_workgroups_only_where_the_gpu_is_full(checks):
    """What one workgroup for few rows, or several rows each, saves is the launch that adds up the gain's gradient."""
    of = checks._ZN5simar20norm_grad_workgroupsEllib
    of.argtypes, of.restype = [ctypes.c_int64, ctypes.c_int64, ctypes.c_int, ctypes.c_bool], ctypes.c_int
    for dtype in (FP32, BF16):
        for rows, cols in ((2, 4096), (4, 4096), (8, 5000), (250, 10000), (4, 2000), (256, 32768)):
            assert of(rows, cols, dtype, False) == rows >= of(rows, cols, dtype, True)
        for rows, cols, turns in ((512, 30, 8), (64, 250, 4), (60, 130, 2), (1, 64, 1)):
            assert of(rows, cols, dtype, False) >= turns and of(rows, cols, dtype, True) == 1
        assert of(0, 64, dtype, True) == of(0, 64, dtype, False) == 1
