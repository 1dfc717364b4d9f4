"""Python binding of libsimar.so (argument marshalling only).

Every function named ``sim_*`` here calls the C function of the same name in
``include/simar.h`` through ctypes and raises :class:`SimError` on a
non-zero status.  All work of the all-reduce path runs in the HIP kernels of
the library; there is no Python or CPU fallback -- if the library is missing
the import fails.

The ``allreduce`` / ``reduce_scatter`` / ``all_gather`` helpers take lists of
torch device tensors (PyTorch is used for device memory and streams only)
and pass their pointers and the current HIP stream to the library.
"""
from __future__ import annotations

import ctypes
import functools
import os
from typing import List, Optional, Sequence

try:  # load torch's HIP runtime first so the library and torch share it
    import torch  # noqa: F401
except Exception:  # pragma: no cover - the host-only tests work without torch
    torch = None

_HERE = os.path.dirname(os.path.abspath(__file__))
# SIMAR_LIB selects another build of the same library (e.g. a variant
# compiled with different cache-policy flags); the default is the in-tree one.
LIBPATH = os.environ.get("SIMAR_LIB") or os.path.join(_HERE, "libsimar.so")

SIM_OK = 0
STATUS = {0: "SIM_OK", -1: "SIM_ERR_INVALID_ARG", -2: "SIM_ERR_UNSUPPORTED", -3: "SIM_ERR_ALIGN",
          -4: "SIM_ERR_ALIAS", -5: "SIM_ERR_NOMEM", -6: "SIM_ERR_HIP", -7: "SIM_ERR_TIMEOUT",
          -8: "SIM_ERR_VERIFY", -9: "SIM_ERR_NOT_INIT"}
STATUS_CODE = {v: k for k, v in STATUS.items()}
DTYPES = {"int32": 0, "fp32": 1, "fp16": 2, "bf16": 3}
OPS = {"sum": 0, "prod": 1, "min": 2, "max": 3, "avg": 4}
ALGOS = {"auto": 0, "ring": 1, "allpairs": 2, "oneshot": 3, "oneshot_ll": 4, "ring_fifo": 5,
         "tree": 6, "rexch": 7, "hier": 8, "hier_large": 9, "allpairs_persistent": 10}
TOPOLOGY_ALGOS = ("tree", "rexch", "hier", "hier_large")
ALGO_NAMES = {v: k for k, v in ALGOS.items()}
ESIZE = {"int32": 4, "fp32": 4, "fp16": 2, "bf16": 2}
XFER_KINDS = {0: "REDUCE", 1: "REDUCE_POST", 2: "COPY", 3: "GATHER_REDUCE", 4: "FANOUT", 5: "ONESHOT",
              6: "GATHER", 7: "GATHER_POST", 8: "EXCH", 9: "EXCH_POST", 10: "MCAST"}
CONFIG = {"ranks_per_node": 0, "radix": 1, "max_workgroups": 2}
DEBUG = {"epoch": 0, "spin_limit": 1, "ll_wait_skew": 2, "fill_ll": 3, "log": 4, "workgroups": 5,
         "unroll": 6, "fifo_channels": 7, "fifo_slots": 8, "fifo_withhold": 9, "fifo_vecs": 10,
         "ptr_table": 11, "ptr_sets": 12, "ring_ll_max": 13,
              "phased": 14, "phased_min": 15, "phased_expired": 16, "phased_last": 17,
         "phased_layout": 18, "phased_whole_last": 19, "route_launches": 20}
MAX_RANKS = 16
ROUTE_MAX_EXPERTS, ROUTE_MAX_TOPK, DISTILL_MAX_TOPK = 1024, 32, 256
NORM_MAX_COLUMNS, CLIP_MAX_TENSORS = 32768, 65536
LL_MAX_BYTES_PER_RANK = 1 << 20


class SimError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)} ({status})")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIBPATH):
        raise ImportError(f"{LIBPATH} is not built; run __graft_entry__.build() "
                          "(hipcc --offload-arch=gfx950) first")
    lib = ctypes.CDLL(LIBPATH)
    vp, sz, i, d = ctypes.c_void_p, ctypes.c_size_t, ctypes.c_int, ctypes.c_double
    i64, f, psz = ctypes.c_int64, ctypes.c_float, ctypes.POINTER(ctypes.c_size_t)
    pp = ctypes.POINTER(ctypes.c_void_p)
    sig = {
        "sim_init": ([i, i, sz], i),
        "sim_finalize": ([], i),
        "sim_allreduce": ([pp, pp, i, sz, i, i, i, vp], i),
        "sim_allreduce_noalloc": ([pp, pp, i, sz, i, i, i, vp], i),
        "sim_reduce_scatter": ([pp, pp, i, sz, i, i, i, vp], i),
        "sim_all_gather": ([pp, pp, i, sz, i, i, vp], i),
        "sim_select": ([i, sz, i, i, ctypes.POINTER(i), ctypes.POINTER(d)], i),
        "sim_last_algo": ([], i),
        "sim_model_load": ([ctypes.c_char_p], i),
        "sim_model_predict": ([i, i, i, d, ctypes.POINTER(d)], i),
        "sim_model_set": ([i, d, d, d, d], i),
        "sim_model_reset": ([], i),
        "sim_model_set_workgroup_rate": ([i, d], i),
        "sim_model_set_host_overlap": ([i, d], i),
        "sim_check_error": ([vp], i),
        "sim_copy_streams": ([pp, pp, i, sz, i, vp], i),
        "sim_config_set": ([i, i], i),
        "sim_config_get": ([i, ctypes.POINTER(i)], i),
        "sim_tree_info": ([i, i, i, i, ctypes.POINTER(i), ctypes.POINTER(i), ctypes.POINTER(i)], i),
        "sim_schedule_info": ([i, i, ctypes.POINTER(i), ctypes.POINTER(i), ctypes.POINTER(i)], i),
        "sim_schedule_xfers": ([i, i, i, ctypes.POINTER(i), i, ctypes.POINTER(i)], i),
        "sim_schedule_state": ([i, i, i, ctypes.POINTER(ctypes.c_uint32)], i),
        "sim_verify_schedule": ([i, i, ctypes.c_char_p, sz], i),
        "sim_verify_custom": ([i, i, i, i, i, ctypes.POINTER(i), ctypes.POINTER(i), ctypes.c_char_p, sz], i),
        "sim_debug_set": ([i, ctypes.c_uint64], i),
        "sim_debug_get": ([i, ctypes.POINTER(ctypes.c_uint64)], i),
        "sim_debug_set_epoch": ([ctypes.c_uint32], i),
        "sim_route_work": ([i64, i, i, i, psz], i),
        "sim_route": ([vp, i64, i, vp, i64, i, i, i, vp, vp, vp, vp, vp, sz, vp], i),
        "sim_route_grad": ([vp, i64, i, vp, i64, i, i, i, vp, vp, vp, vp, f, vp, i64, vp, vp], i),
        "sim_distill_work": ([i64, i64, i, psz], i),
        "sim_distill_step": ([vp, i64, i, i64, i64, vp, vp, i, i, f, vp, f, vp, i64, vp, vp, sz, vp], i),
        "sim_distill_parts": ([vp, i64, i, i64, i64, i64, i64, vp, vp, i, i, f, vp, vp, sz, vp], i),
        "sim_distill_join": ([vp, i, i64, i64, vp, vp, i, i, f, vp, vp, vp], i),
        "sim_distill_grad": ([vp, i64, i, i64, i64, i64, i64, vp, vp, i, i, f, vp, vp, f, vp, i64, vp], i),
        "sim_norm": ([vp, i64, i, vp, i64, i64, i64, vp, i, f, vp, i64, vp, i64, vp, i, vp], i),
        "sim_norm_grad_work": ([i64, i64, i, psz], i),
        "sim_norm_grad": ([vp, i64, i, i64, i64, vp, i, f, vp, i64, vp, i64, vp, i64, vp, vp, sz, vp], i),
        "sim_dispatch_work": ([i64, i, i, psz], i),
        "sim_dispatch": ([vp, i64, i64, vp, i64, vp, i64, i, i, vp, i64, vp, vp, vp, vp, sz, vp], i),
        "sim_combine": ([vp, i64, i, i64, i64, vp, vp, i64, i, vp, i64, vp], i),
        "sim_combine_grad": ([vp, i64, i, vp, i64, i64, i64, vp, vp, i64, i, vp, i64, vp, vp], i),
        "sim_clip_work": ([vp, vp, i, psz], i),
        "sim_clip_norm": ([vp, vp, vp, i, vp, vp, sz, vp], i),
        "sim_clip": ([vp, vp, vp, vp, i, vp, i, f, vp, vp, sz, vp], i),
        "sim_status_string": ([i], ctypes.c_char_p),
        "sim_version": ([], i),
    }
    for name, (args, res) in sig.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


lib = _load()

try:  # the prepared-call object (csrc/pycall.c), built beside the library
    from . import _pycall
except ImportError:  # not built: prepare_allreduce falls back to a ctypes call of the same entry point
    _pycall = None


try:  # tensors' pointers, sizes and types (csrc/pytensor.cpp), built beside it
    from . import _pytensor
    if _pytensor.torch_version != str(torch.__version__):  # another torch may lay its tensors out in another way
        _pytensor = None
except (ImportError, AttributeError):  # not built, or without torch: the same checks in Python
    _pytensor = None


def _check(status: int, what: str) -> int:
    if status != SIM_OK:
        raise SimError(status, what)
    return status


def _ptr_array(ptrs: Sequence[int]):
    return (ctypes.c_void_p * len(ptrs))(*[int(p) for p in ptrs])


def _code(table, v, what):
    if isinstance(v, str):
        if v not in table:
            raise ValueError(f"unknown {what} {v!r}")
        return table[v]
    return int(v)


# The model fitted by calibrate.py on MI355X; sim_init loads it unless the
# SIM_CALIB environment variable names another file (which the C library
# then loads itself).
CALIBRATION = os.path.join(_HERE, "calib", "mi355x.json")


# ---- the C functions, one to one ------------------------------------------------
_device: Optional[int] = None  # the one that sim_init chose


def _forget_sizes() -> None:
    for f in (sim_route_work, sim_distill_work, sim_norm_grad_work, sim_dispatch_work):
        f.cache_clear()


def sim_init(device: int = 0, p_max: int = MAX_RANKS, max_bytes_per_rank: int = 0) -> None:
    global _device
    _forget_sizes()
    _check(lib.sim_init(device, p_max, max_bytes_per_rank), "sim_init")
    _device = device
    if not os.environ.get("SIM_CALIB") and os.path.exists(CALIBRATION):
        sim_model_load(CALIBRATION)


def sim_finalize() -> None:
    global _device
    _forget_sizes()
    _check(lib.sim_finalize(), "sim_finalize")
    _device = None


def sim_allreduce(in_ptrs, out_ptrs, p, n, dtype, op, algo, stream=0) -> int:
    return lib.sim_allreduce(_ptr_array(in_ptrs), _ptr_array(out_ptrs), p, n, _code(DTYPES, dtype, "dtype"),
                             _code(OPS, op, "op"), _code(ALGOS, algo, "algo"), stream or None)


def sim_allreduce_noalloc(in_ptrs, out_ptrs, p, n, dtype, op, algo, stream=0) -> int:
    return lib.sim_allreduce_noalloc(_ptr_array(in_ptrs), _ptr_array(out_ptrs), p, n,
                                     _code(DTYPES, dtype, "dtype"), _code(OPS, op, "op"),
                                     _code(ALGOS, algo, "algo"), stream or None)


NOALLOC_SCRATCH_BYTES = 64 << 20


def prepare_allreduce(in_ptrs, out_ptrs, p, n, dtype, op, algo, stream=0):
    """The same call as sim_allreduce with its arguments marshalled once:
    returns a function of no arguments that calls the C entry point and
    returns its status (for loops that repeat one call, where Python-side
    marshalling would otherwise dominate a few-microsecond call)."""
    f = lib["sim_allreduce"]
    f.restype = ctypes.c_int
    dt, o, a = _code(DTYPES, dtype, "dtype"), _code(OPS, op, "op"), _code(ALGOS, algo, "algo")
    if _pycall is not None:
        # the arguments held as C values and the entry point called directly
        return _pycall.PreparedCall(ctypes.cast(f, ctypes.c_void_p).value, [int(q) for q in in_ptrs],
                                    [int(q) for q in out_ptrs], p, n, dt, o, a, int(stream or 0))
    # a bare function pointer (no argtypes) called with ready-made ctypes
    # objects: no per-call argument conversion
    args = (_ptr_array(in_ptrs), _ptr_array(out_ptrs), ctypes.c_int(p), ctypes.c_size_t(n),
            ctypes.c_int(dt), ctypes.c_int(o), ctypes.c_int(a), ctypes.c_void_p(stream or None))
    return lambda: f(*args)


def sim_reduce_scatter(in_ptrs, out_ptrs, p, n_out_per_rank, dtype, op, algo, stream=0) -> int:
    return lib.sim_reduce_scatter(_ptr_array(in_ptrs), _ptr_array(out_ptrs), p, n_out_per_rank,
                                  _code(DTYPES, dtype, "dtype"), _code(OPS, op, "op"),
                                  _code(ALGOS, algo, "algo"), stream or None)


def sim_all_gather(in_ptrs, out_ptrs, p, n_in_per_rank, dtype, algo, stream=0) -> int:
    return lib.sim_all_gather(_ptr_array(in_ptrs), _ptr_array(out_ptrs), p, n_in_per_rank,
                              _code(DTYPES, dtype, "dtype"), _code(ALGOS, algo, "algo"), stream or None)


def sim_select(p: int, n: int, dtype, op="sum"):
    a, us = ctypes.c_int(0), ctypes.c_double(0)
    _check(lib.sim_select(p, n, _code(DTYPES, dtype, "dtype"), _code(OPS, op, "op"), ctypes.byref(a),
                          ctypes.byref(us)), "sim_select")
    return ALGO_NAMES[a.value], us.value


def sim_last_algo() -> Optional[str]:
    return ALGO_NAMES.get(lib.sim_last_algo())


def sim_model_load(path: str) -> None:
    _check(lib.sim_model_load(path.encode()), f"sim_model_load({path})")


def sim_model_predict(algo, p: int, dtype, bytes_per_rank: float) -> float:
    us = ctypes.c_double(0)
    _check(lib.sim_model_predict(_code(ALGOS, algo, "algo"), p, _code(DTYPES, dtype, "dtype"),
                                 float(bytes_per_rank), ctypes.byref(us)), "sim_model_predict")
    return us.value


def sim_model_set(algo, alpha_us: float, steps: float, bytes_factor: float, gbps: float) -> None:
    _check(lib.sim_model_set(_code(ALGOS, algo, "algo"), alpha_us, steps, bytes_factor, gbps), "sim_model_set")


def sim_model_set_workgroup_rate(algo, gbps_per_workgroup: float) -> None:
    _check(lib.sim_model_set_workgroup_rate(_code(ALGOS, algo, "algo"), float(gbps_per_workgroup)),
           "sim_model_set_workgroup_rate")


def sim_model_set_host_overlap(algo, host_us_per_launch: float) -> None:
    _check(lib.sim_model_set_host_overlap(_code(ALGOS, algo, "algo"), float(host_us_per_launch)),
           "sim_model_set_host_overlap")


def sim_model_reset() -> None:
    _check(lib.sim_model_reset(), "sim_model_reset")


def sim_check_error(stream=0) -> int:
    """Returns the status (SIM_OK or SIM_ERR_TIMEOUT) without raising."""
    return lib.sim_check_error(stream or None)


def sim_copy_streams(src_ptrs, dst_ptrs, k: int, nbytes: int, workgroups: int = 0, stream=0) -> int:
    return lib.sim_copy_streams(_ptr_array(src_ptrs), _ptr_array(dst_ptrs), k, nbytes, workgroups,
                                stream or None)


@functools.lru_cache(maxsize=1024)
def sim_route_work(tokens: int, experts: int, topk: int, dtype) -> int:
    """Workspace bytes of sim_route (they follow from these sizes and the device that sim_init chose)."""
    n = ctypes.c_size_t(0)
    _check(lib.sim_route_work(tokens, experts, topk, _code(DTYPES, dtype, "dtype"), ctypes.byref(n)),
           "sim_route_work")
    return n.value


def sim_route(logits, row_stride, dtype, keep, tokens, experts, topk, normalize, chosen, weights, counts, prob_sums,
              work, work_bytes, stream=0) -> int:
    return lib.sim_route(logits, row_stride, _code(DTYPES, dtype, "dtype"), keep, tokens, experts, topk, normalize,
                         chosen, weights, counts, prob_sums, work, work_bytes, stream or None)


def sim_route_grad(logits, row_stride, dtype, keep, tokens, experts, topk, normalize, chosen, dweights, counts,
                   prob_sums, coef, dlogits, drow_stride, loss, stream=0) -> int:
    return lib.sim_route_grad(logits, row_stride, _code(DTYPES, dtype, "dtype"), keep, tokens, experts, topk,
                              normalize, chosen, dweights, counts, prob_sums, coef, dlogits, drow_stride, loss,
                              stream or None)


@functools.lru_cache(maxsize=1024)
def sim_distill_work(rows: int, columns: int, dtype) -> int:
    """Workspace bytes of sim_distill_step (columns: the vocabulary) and sim_distill_parts."""
    n = ctypes.c_size_t(0)
    _check(lib.sim_distill_work(rows, columns, _code(DTYPES, dtype, "dtype"), ctypes.byref(n)), "sim_distill_work")
    return n.value


def sim_distill_step(logits, row_stride, dtype, rows, vocab, ids, teacher, teacher_dtype, topk, temperature,
                     row_scale, coef, dlogits, drow_stride, loss, work, work_bytes, stream=0) -> int:
    return lib.sim_distill_step(logits, row_stride, _code(DTYPES, dtype, "dtype"), rows, vocab, ids, teacher,
                                _code(DTYPES, teacher_dtype, "dtype"), topk, temperature, row_scale, coef, dlogits,
                                drow_stride, loss, work, work_bytes, stream or None)


def sim_distill_parts(logits, row_stride, dtype, rows, columns, first, vocab, ids, teacher, teacher_dtype, topk,
                      temperature, parts, work, work_bytes, stream=0) -> int:
    return lib.sim_distill_parts(logits, row_stride, _code(DTYPES, dtype, "dtype"), rows, columns, first, vocab, ids,
                                 teacher, _code(DTYPES, teacher_dtype, "dtype"), topk, temperature, parts, work,
                                 work_bytes, stream or None)


def sim_distill_join(parts, nparts, rows, vocab, ids, teacher, teacher_dtype, topk, temperature, loss, norm,
                     stream=0) -> int:
    return lib.sim_distill_join(parts, nparts, rows, vocab, ids, teacher, _code(DTYPES, teacher_dtype, "dtype"), topk,
                                temperature, loss, norm, stream or None)


def sim_distill_grad(logits, row_stride, dtype, rows, columns, first, vocab, ids, teacher, teacher_dtype, topk,
                     temperature, norm, row_scale, coef, dlogits, drow_stride, stream=0) -> int:
    return lib.sim_distill_grad(logits, row_stride, _code(DTYPES, dtype, "dtype"), rows, columns, first, vocab, ids,
                                teacher, _code(DTYPES, teacher_dtype, "dtype"), topk, temperature, norm, row_scale,
                                coef, dlogits, drow_stride, stream or None)


def sim_norm(x, x_stride, dtype, residual, residual_stride, rows, columns, gain, gain_dtype, eps, sum, sum_stride, out,
             out_stride, scales, group, stream=0) -> int:
    return lib.sim_norm(x, x_stride, _code(DTYPES, dtype, "dtype"), residual, residual_stride, rows, columns, gain,
                        _code(DTYPES, gain_dtype, "dtype"), eps, sum, sum_stride, out, out_stride, scales, group,
                        stream or None)


@functools.lru_cache(maxsize=1024)
def sim_norm_grad_work(rows: int, columns: int, dtype) -> int:
    """Workspace bytes of sim_norm_grad with a dgain."""
    n = ctypes.c_size_t(0)
    _check(lib.sim_norm_grad_work(rows, columns, _code(DTYPES, dtype, "dtype"), ctypes.byref(n)), "sim_norm_grad_work")
    return n.value


def sim_norm_grad(h, h_stride, dtype, rows, columns, gain, gain_dtype, eps, dy, dy_stride, dsum, dsum_stride, dx,
                  dx_stride, dgain, work, work_bytes, stream=0) -> int:
    return lib.sim_norm_grad(h, h_stride, _code(DTYPES, dtype, "dtype"), rows, columns, gain,
                             _code(DTYPES, gain_dtype, "dtype"), eps, dy, dy_stride, dsum, dsum_stride, dx, dx_stride,
                             dgain, work, work_bytes, stream or None)


@functools.lru_cache(maxsize=1024)
def sim_dispatch_work(tokens: int, topk: int, experts: int) -> int:
    """Workspace bytes of sim_dispatch."""
    n = ctypes.c_size_t(0)
    _check(lib.sim_dispatch_work(tokens, topk, experts, ctypes.byref(n)), "sim_dispatch_work")
    return n.value


def sim_dispatch(x, x_pitch, row_bytes, scales, groups, chosen, tokens, topk, experts, rows, rows_pitch, row_scales,
                 place, offsets, work, work_bytes, stream=0) -> int:
    return lib.sim_dispatch(x, x_pitch, row_bytes, scales, groups, chosen, tokens, topk, experts, rows, rows_pitch,
                            row_scales, place, offsets, work, work_bytes, stream or None)


def sim_combine(rows, rows_stride, dtype, nrows, columns, place, weights, tokens, topk, out, out_stride,
                stream=0) -> int:
    return lib.sim_combine(rows, rows_stride, _code(DTYPES, dtype, "dtype"), nrows, columns, place, weights, tokens,
                           topk, out, out_stride, stream or None)


def sim_combine_grad(dy, dy_stride, dtype, rows, rows_stride, nrows, columns, place, weights, tokens, topk, drows,
                     drows_stride, dweights, stream=0) -> int:
    return lib.sim_combine_grad(dy, dy_stride, _code(DTYPES, dtype, "dtype"), rows, rows_stride, nrows, columns, place,
                                weights, tokens, topk, drows, drows_stride, dweights, stream or None)


def _host_array(values, ctype):
    """A host array of a C call (None: none)."""
    return None if values is None else (ctype * len(values))(*values)


def sim_clip_work(counts, dtypes) -> int:
    """Workspace bytes of sim_clip_norm, and of sim_clip without parts, over tensors of these sizes and types."""
    n = ctypes.c_size_t(0)
    _check(lib.sim_clip_work(_host_array(counts, ctypes.c_int64),
                             _host_array([_code(DTYPES, d, "dtype") for d in dtypes], ctypes.c_int), len(counts),
                             ctypes.byref(n)), "sim_clip_work")
    return n.value


def sim_clip_norm(grads, counts, dtypes, norm, work, work_bytes, stream=0) -> int:
    return lib.sim_clip_norm(_host_array(grads, ctypes.c_void_p), _host_array(counts, ctypes.c_int64),
                             _host_array([_code(DTYPES, d, "dtype") for d in dtypes], ctypes.c_int), len(grads), norm,
                             work, work_bytes, stream or None)


def sim_clip(grads, outs, counts, dtypes, parts, nparts, max_norm, norm, work, work_bytes, stream=0) -> int:
    return lib.sim_clip(_host_array(grads, ctypes.c_void_p), _host_array(outs, ctypes.c_void_p),
                        _host_array(counts, ctypes.c_int64),
                        _host_array([_code(DTYPES, d, "dtype") for d in dtypes], ctypes.c_int), len(grads), parts,
                        nparts, max_norm, norm, work, work_bytes, stream or None)


def sim_config_set(key, value: int) -> None:
    _check(lib.sim_config_set(_code(CONFIG, key, "config key"), int(value)), "sim_config_set")


def sim_config_get(key) -> int:
    v = ctypes.c_int(0)
    _check(lib.sim_config_get(_code(CONFIG, key, "config key"), ctypes.byref(v)), "sim_config_get")
    return v.value


def sim_tree_info(tree: int, p: int, ranks_per_node: int, rank: int):
    """(parent, [children ascending]) of `rank` in tree 0 or 1."""
    par, nch = ctypes.c_int(0), ctypes.c_int(0)
    ch = (ctypes.c_int * 3)()
    _check(lib.sim_tree_info(tree, p, ranks_per_node, rank, ctypes.byref(par), ch, ctypes.byref(nch)),
           "sim_tree_info")
    return par.value, list(ch[:nch.value])


def sim_schedule_info(algo, p: int):
    """(steps, transfers, chunks) of the lowered all-reduce schedule."""
    ns, nx, nc = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    _check(lib.sim_schedule_info(_code(ALGOS, algo, "algo"), p, ctypes.byref(ns), ctypes.byref(nx),
                                 ctypes.byref(nc)), "sim_schedule_info")
    return ns.value, nx.value, nc.value


def sim_schedule_xfers(algo, p: int, step: int):
    """The step's transfers as (kind, src, dst, chunk, rank set) tuples."""
    cap = 512
    buf = (ctypes.c_int * (5 * cap))()
    cnt = ctypes.c_int(0)
    _check(lib.sim_schedule_xfers(_code(ALGOS, algo, "algo"), p, step, buf, cap, ctypes.byref(cnt)),
           "sim_schedule_xfers")
    return [tuple(buf[5 * k:5 * k + 5]) for k in range(cnt.value)]


def sim_schedule_state(algo, p: int, after_steps: int):
    """masks[r][c] after `after_steps` steps."""
    nch = sim_schedule_info(algo, p)[2]
    m = (ctypes.c_uint32 * (p * nch))()
    _check(lib.sim_schedule_state(_code(ALGOS, algo, "algo"), p, after_steps, m), "sim_schedule_state")
    return [[m[r * nch + c] for c in range(nch)] for r in range(p)]


def sim_verify_schedule(algo, p: int):
    buf = ctypes.create_string_buffer(1024)
    st = lib.sim_verify_schedule(_code(ALGOS, algo, "algo"), p, buf, 1024)
    return st, buf.value.decode()


def sim_verify_custom(algo, p: int, steps: List[List[tuple]], nchunks: Optional[int] = None,
                      rounds: Optional[int] = None):
    """Check a caller-made all-reduce schedule.  Transfers are 5-tuples
    (kind, src, dst, chunk, rank set); 4-tuples get an empty rank set.
    nchunks defaults to p, rounds to the number of steps."""
    steps = [[tuple(x) + (0,) * (5 - len(x)) for x in s] for s in steps]
    counts = (ctypes.c_int * max(1, len(steps)))(*[len(s) for s in steps])
    flat = [v for s in steps for x in s for v in x]
    xf = (ctypes.c_int * max(1, len(flat)))(*flat)
    buf = ctypes.create_string_buffer(1024)
    st = lib.sim_verify_custom(_code(ALGOS, algo, "algo"), p, p if nchunks is None else nchunks,
                               len(steps) if rounds is None else rounds, len(steps), counts, xf, buf, 1024)
    return st, buf.value.decode()


def sim_debug_set(key, value: int) -> None:
    _check(lib.sim_debug_set(_code(DEBUG, key, "debug key"), int(value) & (2 ** 64 - 1)), "sim_debug_set")


def sim_debug_get(key) -> int:
    v = ctypes.c_uint64(0)
    _check(lib.sim_debug_get(_code(DEBUG, key, "debug key"), ctypes.byref(v)), "sim_debug_get")
    return v.value


def sim_debug_set_epoch(epoch: int) -> None:
    _check(lib.sim_debug_set_epoch(int(epoch) & 0xFFFFFFFF), "sim_debug_set_epoch")


def sim_status_string(status: int) -> str:
    return lib.sim_status_string(status).decode()


def sim_version() -> int:
    return lib.sim_version()


# ---- torch tensor helpers (marshalling only) --------------------------------------
def _dtype_name(t) -> str:
    import torch as _t
    m = {_t.int32: "int32", _t.float32: "fp32", _t.float16: "fp16", _t.bfloat16: "bf16"}
    if t.dtype not in m:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return m[t.dtype]


def _stream(stream) -> int:
    import torch as _t
    s = stream if stream is not None else _t.cuda.current_stream()
    return int(s.cuda_stream)


def _ptrs(ts) -> List[int]:
    out = []
    for t in ts:
        if not t.is_cuda or not t.is_contiguous():
            raise ValueError("tensors must be contiguous device tensors")
        out.append(t.data_ptr())
    return out


def allreduce(inputs: Sequence, outputs: Optional[Sequence] = None, op="sum", algo="auto", stream=None):
    """All-reduce p same-shaped device tensors (outputs=None: in place)."""
    outputs = list(inputs) if outputs is None else list(outputs)
    dt = _dtype_name(inputs[0])
    st = sim_allreduce(_ptrs(inputs), _ptrs(outputs), len(inputs), inputs[0].numel(), dt, op, algo,
                       _stream(stream))
    _check(st, "sim_allreduce")
    return outputs


def reduce_scatter(inputs: Sequence, outputs: Sequence, op="sum", algo="auto", stream=None):
    dt = _dtype_name(inputs[0])
    st = sim_reduce_scatter(_ptrs(inputs), _ptrs(outputs), len(inputs), outputs[0].numel(), dt, op, algo,
                            _stream(stream))
    _check(st, "sim_reduce_scatter")
    return outputs


def all_gather(inputs: Sequence, outputs: Sequence, algo="auto", stream=None):
    dt = _dtype_name(inputs[0])
    st = sim_all_gather(_ptrs(inputs), _ptrs(outputs), len(inputs), inputs[0].numel(), dt, algo,
                        _stream(stream))
    _check(st, "sim_all_gather")
    return outputs


# ---- routing and losses (torch tensors; marshalling only) --------------------------
_raw_stream = getattr(getattr(torch, "_C", None), "_cuda_getCurrentRawStream", None)
_TORCH_CODE = {} if torch is None else {torch.float32: 1, torch.float16: 2, torch.bfloat16: 3}
if torch is not None:
    _F32, _I32, _MASK = (torch.float32,), (torch.int32,), (torch.bool, torch.uint8)
    _FLOATS = tuple(_TORCH_CODE)

_ENTRIES = ("route", "route_grad", "distill_step", "distill_parts", "distill_join", "distill_grad", "norm", "norm_grad",
            "dispatch", "combine", "combine_grad", "clip_work", "clip_norm", "clip")


def _vec_py(t, what, dtypes, device, *shape):
    """Pointer of a contiguous device tensor of the given shape and one of the given dtypes (None: None)."""
    if t is None:
        return None
    if t.dtype not in dtypes or t.shape != shape or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous tensor {shape!r} of one of {dtypes!r} on cuda:{device}")
    return t.data_ptr()


def _rows_py(t, what, like):
    """(pointer, row stride, rows, columns, dtype code, device index) of a 2-D device tensor whose rows are
    contiguous; like: None, or the tuple of a tensor whose shape, dtype and device it must have."""
    if t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{what} must be a 2-D device tensor")
    n, c = t.shape
    st = t.stride()
    if st[1] != 1 and c > 1:
        raise ValueError(f"{what}'s rows must be contiguous")
    if t.dtype not in _TORCH_CODE:
        raise ValueError(f"unsupported dtype {t.dtype}")
    got = (t.data_ptr(), st[0] if n > 1 else c, n, c, _TORCH_CODE[t.dtype], t.get_device())
    if like is not None and got[2:] != like[2:]:
        raise ValueError(f"{what} must have the first tensor's shape, dtype and device")
    return got


def _slots_py(ids, teacher, dtypes, rows, device):
    """(ids pointer, teacher pointer, its dtype code, topk)"""
    if ids.dim() != 2:
        raise ValueError("ids must be [rows, topk]")
    k = ids.shape[1]
    return (_vec_py(ids, "ids", dtypes, device, rows, k), _vec_py(teacher, "teacher", _FLOATS, device, rows, k),
            _TORCH_CODE[teacher.dtype], k)


def _like_py(t, what, like):
    """The first two of _rows' for a tensor like another one; of None, None and the columns."""
    return (None, like[3]) if t is None else _rows_py(t, what, like)[:2]


def _gain_py(gain, columns, device):
    """(pointer, type code) of a norm's gain (None: all 1)."""
    if gain is None:
        return None, 1
    return _vec_py(gain, "gain", _FLOATS, device, columns), _TORCH_CODE[gain.dtype]


def _clip_work_py(counts, dtypes, n):
    nb = ctypes.c_size_t(0)
    rc = lib.sim_clip_work(counts, dtypes, n, ctypes.byref(nb))
    return rc or nb.value


def _raw_py(t, what, dtype):
    """(pointer, bytes from row to row, rows, bytes of a row, device index) of a 2-D device tensor of any type whose
    rows are contiguous; dtype: the one it must have, or None."""
    if t.dim() != 2 or not t.is_cuda:
        raise ValueError(f"{what} must be a 2-D device tensor")
    n, c = t.shape
    st = t.stride()
    if st[1] != 1 and c > 1:
        raise ValueError(f"{what}'s rows must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{what} must be of type {dtype}")
    e = t.element_size()
    return t.data_ptr(), (st[0] if n > 1 else c) * e, n, c * e, t.get_device()


def _tensors_py(ts, what, device, like):
    """(pointers, counts, type codes), each an array of the host, of contiguous tensors on that device; like: None, or
    such a tuple whose counts and types they must have."""
    for i, t in enumerate(ts):
        if t.dtype not in _TORCH_CODE or t.get_device() != device or not t.is_contiguous():
            raise ValueError(f"{what}[{i}] must be a contiguous tensor of one of the float types on cuda:{device}")
    got = tuple(bytes(_host_array(v, c)) for v, c in (([t.data_ptr() for t in ts], ctypes.c_void_p),
                                                      ([t.numel() for t in ts], ctypes.c_int64),
                                                      ([_TORCH_CODE[t.dtype] for t in ts], ctypes.c_int)))
    if like is not None and got[1:] != like[1:]:
        raise ValueError(f"{what} must have the gradients' sizes and types")
    return got


if hasattr(_pycall, "clip_work"):
    # arguments converted in C: ctypes took a good half of a small call's time on the host
    for _name in _ENTRIES:
        _pycall.bind(_name, ctypes.cast(lib["sim_" + _name], ctypes.c_void_p).value)
    _entry, _clip_bytes = _pycall, _pycall.clip_work
else:
    import types as _types
    _entry, _clip_bytes = _types.SimpleNamespace(**{n: getattr(lib, "sim_" + n) for n in _ENTRIES}), _clip_work_py
if _pytensor is not None:
    # tensors looked at in C++: five attributes and methods of each took 0.25 us in Python's own calls
    _rows, _like, _raw, _vec, _tensors = _pytensor.rows, _pytensor.like, _pytensor.raw, _pytensor.pointer, _pytensor.tensors
    _gain, _slots = _pytensor.gain, _pytensor.slots
else:
    _rows, _like, _raw, _vec, _tensors = _rows_py, _like_py, _raw_py, _vec_py, _tensors_py
    _gain, _slots = _gain_py, _slots_py


def _on(stream, device):
    """The stream's handle (default: the device's current stream); torch's raw accessor, where there is one, makes no
    stream object for every call (0.1 instead of 2.9 us)."""
    if stream is not None:
        return stream.cuda_stream or None
    if _raw_stream is not None:
        return _raw_stream(device) or None
    return torch.cuda.current_stream(device).cuda_stream or None


def _empty(shape, dtype, device, stream):
    """A new tensor for the call's stream: memory the allocator hands out for one stream may still be in use there, so
    it is taken from the stream the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _work(nbytes, device, stream):
    """A call's scratch: (tensor, pointer)."""
    if nbytes == 0:
        return None, None
    w = _empty(nbytes, torch.uint8, device, stream)
    return w, w.data_ptr()


def route(logits, topk: int, keep=None, normalize: bool = True, out=None, stream=None):
    """Softmax gate of logits [tokens, experts]: (chosen int32 [tokens, topk], weights fp32 [tokens, topk], counts
    int32 [experts + 1], prob_sums fp32 [experts]); ``sim_route`` in include/simar.h says what each holds.  keep:
    bool or uint8 [tokens].  out: the same four tensors, to write into."""
    ptr, ld, n, e, dt, dev = _rows(logits, "logits", None)
    if out is None:
        out = (_empty((n, topk), torch.int32, dev, stream), _empty((n, topk), torch.float32, dev, stream),
               _empty(e + 1, torch.int32, dev, stream), _empty(e, torch.float32, dev, stream))
    chosen, weights, counts, sums = out
    nb = sim_route_work(n, e, topk, dt)
    w, wp = _work(nb, dev, stream)
    _check(_entry.route(ptr, ld, dt, _vec(keep, "keep", _MASK, dev, n), n, e, topk, bool(normalize),
                        _vec(chosen, "chosen", _I32, dev, n, topk), _vec(weights, "weights", _F32, dev, n, topk),
                        _vec(counts, "counts", _I32, dev, e + 1), _vec(sums, "prob_sums", _F32, dev, e), wp, nb,
                        _on(stream, dev)), "sim_route")
    return out


def route_grad(logits, chosen, dweights=None, counts=None, prob_sums=None, coef: float = 0.0, keep=None,
               normalize: bool = True, out=None, stream=None):
    """Balance loss of the (reduced) counts and prob_sums, and the gradient of that loss and of the combine weights
    for the logits: (loss fp32 [1], dlogits); ``sim_route_grad`` in include/simar.h says what each holds.  out: the
    same two tensors, to write into (dlogits may be the logits)."""
    ptr, ld, n, e, dt, dev = mine = _rows(logits, "logits", None)
    topk = chosen.shape[1]
    if out is None:
        out = (_empty(1, torch.float32, dev, stream), _empty((n, e), logits.dtype, dev, stream))
    loss, dlogits = out
    dptr, dld, *_ = _rows(dlogits, "dlogits", mine)
    _check(_entry.route_grad(ptr, ld, dt, _vec(keep, "keep", _MASK, dev, n), n, e, topk,
                             bool(normalize), _vec(chosen, "chosen", _I32, dev, n, topk),
                             _vec(dweights, "dweights", _F32, dev, n, topk), _vec(counts, "counts", _I32, dev, e + 1),
                             _vec(prob_sums, "prob_sums", _F32, dev, e), coef, dptr, dld,
                             _vec(loss, "loss", _F32, dev, 1), _on(stream, dev)), "sim_route_grad")
    return out


def distill_step(logits, ids, teacher, temperature: float = 1.0, row_scale=None, coef: float = 1.0, out=None,
                 stream=None):
    """Distillation of logits [rows, vocab] from a teacher's top logits (ids int32 [rows, topk], teacher [rows,
    topk]): (loss fp32 [rows], dlogits); ``sim_distill_step`` in include/simar.h says what each holds.  out: the same
    two tensors, to write into (dlogits may be the logits)."""
    ptr, ld, n, v, dt, dev = mine = _rows(logits, "logits", None)
    if out is None:
        out = (_empty(n, torch.float32, dev, stream), _empty((n, v), logits.dtype, dev, stream))
    loss, dlogits = out
    dptr, dld, *_ = _rows(dlogits, "dlogits", mine)
    ip, tp, tdt, k = _slots(ids, teacher, _I32, n, dev)
    nb = sim_distill_work(n, v, dt)
    w, wp = _work(nb, dev, stream)
    _check(_entry.distill_step(ptr, ld, dt, n, v, ip, tp, tdt, k, temperature,
                               _vec(row_scale, "row_scale", _F32, dev, n), coef, dptr, dld,
                               _vec(loss, "loss", _F32, dev, n), wp, nb, _on(stream, dev)), "sim_distill_step")
    return out


def _whole(vocab, rows, columns):
    """The whole vocabulary's size.  A teacher's slots are those with an id in it, so parts, join and gradient have to
    be told the same one; no size that one shard could take by itself is right for all of them.  (Without rows there is
    nothing to be told.)"""
    if vocab is not None:
        return vocab
    if rows:
        raise ValueError("vocab must be given: the columns of all shards together")
    return columns


def distill_parts(logits, ids, teacher, temperature: float = 1.0, first: int = 0, vocab: Optional[int] = None,
                  out=None, stream=None):
    """A vocabulary shard's statistics, fp32 [4, rows]: logits hold the columns from `first` on of all `vocab` ones
    (must be given)."""
    ptr, ld, n, c, dt, dev = _rows(logits, "logits", None)
    if out is None:
        out = _empty((4, n), torch.float32, dev, stream)
    ip, tp, tdt, k = _slots(ids, teacher, _I32, n, dev)
    nb = sim_distill_work(n, c, dt)
    w, wp = _work(nb, dev, stream)
    _check(_entry.distill_parts(ptr, ld, dt, n, c, first, _whole(vocab, n, first + c), ip, tp, tdt, k,
                                temperature, _vec(out, "parts", _F32, dev, 4, n), wp, nb, _on(stream, dev)),
           "sim_distill_parts")
    return out


def distill_join(parts, ids, teacher, temperature: float = 1.0, vocab: Optional[int] = None, out=None, stream=None):
    """Loss of all shards' parts [nparts, 4, rows], as all_gather leaves them: (loss fp32 [rows], norm fp32 [2,
    rows]).  vocab: the columns of all shards together (must be given; an id outside it is an empty slot)."""
    if parts.dim() != 3 or not parts.is_cuda:
        raise ValueError("parts must be a device tensor [nparts, 4, rows]")
    p, _, n = parts.shape
    dev = parts.get_device()
    if out is None:
        out = (_empty(n, torch.float32, dev, stream), _empty((2, n), torch.float32, dev, stream))
    loss, norm = out
    ip, tp, tdt, k = _slots(ids, teacher, _I32, n, dev)
    _check(_entry.distill_join(_vec(parts, "parts", _F32, dev, p, 4, n), p, n, _whole(vocab, n, 1),
                               ip, tp, tdt, k, temperature, _vec(loss, "loss", _F32, dev, n),
                               _vec(norm, "norm", _F32, dev, 2, n), _on(stream, dev)), "sim_distill_join")
    return out


def distill_grad(logits, ids, teacher, norm, temperature: float = 1.0, row_scale=None, coef: float = 1.0,
                 first: int = 0, vocab: Optional[int] = None, out=None, stream=None):
    """The gradient of a vocabulary shard's logits, the columns from `first` on of all `vocab` ones (must be given),
    from the joined norm [2, rows].  out: the gradient, to write into (it may be the logits)."""
    ptr, ld, n, c, dt, dev = mine = _rows(logits, "logits", None)
    if out is None:
        out = _empty((n, c), logits.dtype, dev, stream)
    dptr, dld, *_ = _rows(out, "dlogits", mine)
    ip, tp, tdt, k = _slots(ids, teacher, _I32, n, dev)
    _check(_entry.distill_grad(ptr, ld, dt, n, c, first, _whole(vocab, n, first + c), ip, tp,
                               tdt, k, temperature, _vec(norm, "norm", _F32, dev, 2, n),
                               _vec(row_scale, "row_scale", _F32, dev, n), coef, dptr, dld, _on(stream, dev)),
           "sim_distill_grad")
    return out


# ---- around the experts, and before the optimizer (torch tensors; marshalling only) --
_E4M3 = getattr(torch, "float8_e4m3fn", None)


def _here(device):
    """The library works on one device: tensors elsewhere are the caller's error."""
    if _device is not None and device != _device:
        raise ValueError(f"tensors must be on cuda:{_device}, the device that sim_init chose")


def norm(x, gain=None, residual=None, eps: float = 1e-6, out=None, stream=None):
    """Root-mean-square norm of the rows of x (+ residual): (y, x + residual; without a residual None); ``sim_norm`` in
    include/simar.h says what each holds.  out: the same two, to write into (each may be x or residual)."""
    ptr, ld, n, c, dt, dev = mine = _rows(x, "x", None)
    _here(dev)
    if out is None:
        out = (_empty((n, c), x.dtype, dev, stream),
               None if residual is None else _empty((n, c), x.dtype, dev, stream))
    y, total = out
    yp, yld = _like(y, "y", mine)
    rp, rld = _like(residual, "residual", mine)
    tp, tld = _like(total, "total", mine)
    gp, gdt = _gain(gain, c, dev)
    _check(_entry.norm(ptr, ld, dt, rp, rld, n, c, gp, gdt, eps, tp, tld, yp, yld, None, 0, _on(stream, dev)),
           "sim_norm")
    return out


def norm_quant(x, gain=None, residual=None, eps: float = 1e-6, group: int = 128, out=None, stream=None):
    """The same with y in 8 bits: (float8_e4m3fn [rows, columns], scales fp32 [rows, groups], x + residual or None).
    group: the columns of a scale, 32, 64 or 128, or all columns of a row."""
    ptr, ld, n, c, dt, dev = mine = _rows(x, "x", None)
    _here(dev)
    if group not in (32, 64, 128, c):
        raise ValueError("group must be 32, 64, 128 or all columns")
    groups = 1 if group == c else -(-c // group)
    if out is None:
        out = (_empty((n, c), _E4M3, dev, stream), _empty((n, groups), torch.float32, dev, stream),
               None if residual is None else _empty((n, c), x.dtype, dev, stream))
    q, scales, total = out
    qp, qld, qn, qc, qdev = _raw(q, "q", _E4M3)
    if qn != n or qc != c or qdev != dev:
        raise ValueError("q must have x's shape and device")
    rp, rld = _like(residual, "residual", mine)
    tp, tld = _like(total, "total", mine)
    gp, gdt = _gain(gain, c, dev)
    _check(_entry.norm(ptr, ld, dt, rp, rld, n, c, gp, gdt, eps, tp, tld, qp, qld,
                       _vec(scales, "scales", _F32, dev, n, groups), 0 if group == c else group,
                       _on(stream, dev)), "sim_norm")
    return out


def norm_grad(total, gain, dout, dtotal=None, eps: float = 1e-6, out=None, stream=None):
    """Gradient of the norm of `total` (x, or x + residual): (dx, dgain fp32 [columns]); dtotal: the gradient that
    reaches `total` by another way.  out: the same two, to write into (dx may be any of the three inputs; dgain None:
    not wanted)."""
    ptr, ld, n, c, dt, dev = mine = _rows(total, "total", None)
    _here(dev)
    if out is None:
        out = (_empty((n, c), total.dtype, dev, stream), _empty(c, torch.float32, dev, stream))
    dx, dgain = out
    dp, dld = _like(dx, "dx", mine)
    op, old = _like(dout, "dout", mine)
    tp, tld = _like(dtotal, "dtotal", mine)
    gp, gdt = _gain(gain, c, dev)
    nb = 0 if dgain is None else sim_norm_grad_work(n, c, dt)
    w, wp = _work(nb, dev, stream)
    _check(_entry.norm_grad(ptr, ld, dt, n, c, gp, gdt, eps, op, old, tp, tld, dp, dld,
                            _vec(dgain, "dgain", _F32, dev, c), wp, nb, _on(stream, dev)), "sim_norm_grad")
    return out


def dispatch(x, chosen, experts: int, scales=None, out=None, stream=None):
    """The rows of x [tokens, columns] (any type) sorted by the experts of chosen int32 [tokens, topk]: (rows
    [tokens * topk, columns], place int32 [tokens, topk], offsets int32 [experts + 1], the rows' scales fp32
    [tokens * topk, groups]; without scales None); ``sim_dispatch`` in include/simar.h says what each holds.  Rows
    from offsets[experts] on are not written.  scales: fp32 [tokens, groups] of x.  out: the same four, to write into."""
    ptr, pitch, n, nb, dev = _raw(x, "x", None)
    _here(dev)
    if chosen.dim() != 2:
        raise ValueError("chosen must be [tokens, topk]")
    k = chosen.shape[1]
    groups = 0 if scales is None else scales.shape[-1]
    if out is None:
        out = (_empty((n * k, x.shape[1]), x.dtype, dev, stream), _empty((n, k), torch.int32, dev, stream),
               _empty(experts + 1, torch.int32, dev, stream),
               None if scales is None else _empty((n * k, groups), torch.float32, dev, stream))
    rows, place, offsets, row_scales = out
    rp, rpitch, rn, rnb, rdev = _raw(rows, "rows", x.dtype)
    if rn != n * k or rnb != nb or rdev != dev:
        raise ValueError("rows must be [tokens * topk, columns] on x's device")
    if (scales is None) != (row_scales is None):
        raise ValueError("scales and the rows' scales: both or neither")
    wb = sim_dispatch_work(n, k, experts)
    w, wp = _work(wb, dev, stream)
    _check(_entry.dispatch(ptr, pitch, nb, _vec(scales, "scales", _F32, dev, n, groups), groups,
                           _vec(chosen, "chosen", _I32, dev, n, k), n, k, experts, rp, rpitch,
                           _vec(row_scales, "row_scales", _F32, dev, n * k, groups),
                           _vec(place, "place", _I32, dev, n, k), _vec(offsets, "offsets", _I32, dev, experts + 1), wp,
                           wb, _on(stream, dev)), "sim_dispatch")
    return out


def combine(rows, place, weights=None, out=None, stream=None):
    """The experts' rows back to their tokens, [tokens, columns]: the sum over a token's slots of weights fp32 [tokens,
    topk] (None: all 1) times rows[place]; ``sim_combine`` in include/simar.h.  out: the result, to write into."""
    ptr, ld, m, c, dt, dev = _rows(rows, "rows", None)
    _here(dev)
    if place.dim() != 2:
        raise ValueError("place must be [tokens, topk]")
    n, k = place.shape
    if out is None:
        out = _empty((n, c), rows.dtype, dev, stream)
    op, old = _like(out, "out", (None, None, n, c, dt, dev))
    _check(_entry.combine(ptr, ld, dt, m, c, _vec(place, "place", _I32, dev, n, k),
                          _vec(weights, "weights", _F32, dev, n, k), n, k, op, old, _on(stream, dev)), "sim_combine")
    return out


def dispatch_grad(drows, place, out=None, stream=None):
    """The gradient of dispatch for x: combine without weights."""
    return combine(drows, place, out=out, stream=stream)


def combine_grad(dout, rows, place, weights=None, out=None, stream=None):
    """The gradient of combine for the rows and the weights: (drows, dweights fp32 [tokens, topk]); ``sim_combine_grad``
    in include/simar.h says what each holds.  Rows that no place names are not written.  out: the same two, to write
    into (drows may be the rows; either may be None: not wanted)."""
    dp, dld, n, c, dt, dev = _rows(dout, "dout", None)
    _here(dev)
    rp, rld, m, rc, rdt, rdev = theirs = _rows(rows, "rows", None)
    if rc != c or rdt != dt or rdev != dev:
        raise ValueError("rows must have dout's columns, dtype and device")
    if place.dim() != 2:
        raise ValueError("place must be [tokens, topk]")
    k = place.shape[1]
    if out is None:
        out = (_empty((m, c), rows.dtype, dev, stream), _empty((n, k), torch.float32, dev, stream))
    drows, dweights = out
    gp, gld = _like(drows, "drows", theirs)
    _check(_entry.combine_grad(dp, dld, dt, rp, rld, m, c, _vec(place, "place", _I32, dev, n, k),
                               _vec(weights, "weights", _F32, dev, n, k), n, k, gp, gld,
                               _vec(dweights, "dweights", _F32, dev, n, k), _on(stream, dev)), "sim_combine_grad")
    return out


def _list_device(grads):
    if not grads:
        return _device if _device is not None else torch.cuda.current_device()
    if not grads[0].is_cuda:
        raise ValueError("grads must be device tensors")
    return grads[0].get_device()


def _clip_work(lists, n, device, stream):
    """Scratch of a norm over a list: (tensor, pointer, bytes)."""
    nb = _clip_bytes(lists[1], lists[2], n)
    if nb < 0:
        raise SimError(nb, "sim_clip_work")
    return (*_work(nb, device, stream), nb)


def grad_norm(grads, out=None, stream=None):
    """The norm over all elements of a list of gradients, fp32 [1] (``sim_clip_norm`` in include/simar.h): a rank's part
    of clip_grads where each rank holds a part of them.  out: the norm, to write into."""
    grads = list(grads)
    dev = _list_device(grads)
    _here(dev)
    lists = _tensors(grads, "grads", dev, None)
    if out is None:
        out = _empty(1, torch.float32, dev, stream)
    w, wp, nb = _clip_work(lists, len(grads), dev, stream)
    _check(_entry.clip_norm(*lists, len(grads), _vec(out, "norm", _F32, dev, 1), wp, nb, _on(stream, dev)),
           "sim_clip_norm")
    return out


def clip_grads(grads, max_norm: float, parts=None, out=None, norm=None, stream=None):
    """A list of gradients scaled down to a norm of at most max_norm, in place (out: or into tensors of the same sizes
    and types); returns their norm before, fp32 [1] (``sim_clip`` in include/simar.h).  parts: fp32 [ranks], every
    rank's grad_norm, where this rank's list is not all of them.  norm: the norm, to write into."""
    grads = list(grads)
    dev = _list_device(grads)
    _here(dev)
    lists = _tensors(grads, "grads", dev, None)
    outs = None if out is None else _tensors(list(out), "out", dev, lists)[0]
    if norm is None:
        norm = _empty(1, torch.float32, dev, stream)
    w, wp, nb = (None, None, 0) if parts is not None else _clip_work(lists, len(grads), dev, stream)
    nparts = 0 if parts is None else parts.numel()
    _check(_entry.clip(lists[0], outs, lists[1], lists[2], len(grads), _vec(parts, "parts", _F32, dev, nparts), nparts,
                       max_norm, _vec(norm, "norm", _F32, dev, 1), wp, nb, _on(stream, dev)), "sim_clip")
    return norm
