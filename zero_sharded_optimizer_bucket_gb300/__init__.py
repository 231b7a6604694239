"""Python binding of libzs (include/zs.h): the ZeRO-3 per-step shard data
path on one GB300, N virtual ranks in one HBM.

Argument marshalling only.  Every step of the path runs in libzs's CUDA
kernels; this module converts Python values (ints, torch tensors, streams)
to the C arguments and raises ZsError on a non-zero status.  Importing it
fails loudly when libzs.so is missing: there is no fallback.

Functions keep the C names: zs_build_partition, zs_plan_upload,
zs_partition, zs_reduce_scatter, zs_grad_norm, zs_adam_step,
zs_all_gather_coalesced, zs_shard_step, plus the plan queries; and, for
training with little memory, zs_build_tensors / zs_norm_tensors,
zs_clip_tensors, zs_adam_tensors, zs_mx4_quantize, zs_mx4_dequantize,
zs_mx4_matmul, zs_mx4_matvec, and zs_rms_norm, zs_rms_norm_backward, which
take torch tensors and read sizes, strides and types from them.
"""
from __future__ import annotations

import ctypes as C
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libzs.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it first "
        "(python -c 'import __graft_entry__ as g; g.build()'); libzs has no CPU fallback")
_lib = C.CDLL(LIB_PATH)

ZS_OK, ZS_EINVAL, ZS_ENOMEM, ZS_ECUDA, ZS_ESTATE, ZS_ETIMEOUT = 0, -1, -2, -3, -4, -5
ZS_MAX_RANKS = 256
ZS_SKIP_NONFINITE = 1
ZS_DTYPE_BF16, ZS_DTYPE_FP16, ZS_DTYPE_FP32 = 0, 1, 2
ZS_ROUND_NEAREST, ZS_ROUND_STOCHASTIC = 0, 1
ZS_STATE_BLOCK = 256     # elements that share the scales of 8-bit moments
ZS_MATVEC_MAX_TOKENS = 1024
ZS_NOALLOC_NORM_MAX_SCRATCH = 1 << 20
TILE_DTYPE = [("dst", "<i8"), ("src", "<i8"), ("flat", "<i8"), ("win", "<i8"),
              ("len", "<i4"), ("valid", "<i4"), ("flat_len", "<i4"), ("bucket", "<i4")]


class ZsError(RuntimeError):
    def __init__(self, status: int, fn: str, msg: str):
        super().__init__(f"{fn} failed ({status}): {msg}")
        self.status = status


class zs_config(C.Structure):
    _fields_ = [("n_ranks", C.c_int32), ("dtype", C.c_int32),
                ("param_persistence_threshold", C.c_int64), ("reduce_bucket_size", C.c_int64),
                ("prefetch_bucket_size", C.c_int64), ("sub_group_size", C.c_int64),
                ("shard_group_size", C.c_int32), ("reserved", C.c_int32)]


class zs_adam_hparams(C.Structure):
    _fields_ = [("lr", C.c_float), ("beta1", C.c_float), ("beta2", C.c_float),
                ("eps", C.c_float), ("weight_decay", C.c_float), ("adamw", C.c_int32),
                ("bias_correction", C.c_int32)]


class zs_plan_info_t(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("n_ranks", "n_params", "n_reduce_buckets",
                                         "n_gather_buckets", "n_sub_groups", "dtype",
                                         "shard_group_size", "reserved")] + \
               [(n, C.c_int64) for n in ("psi", "shard_elems", "shard_elems_logical",
                                         "persist_elems", "persist_elems_logical", "flat_elems",
                                         "padding_elems", "max_bucket_buf_elems",
                                         "max_gather_elems", "bytes_per_rank", "n_tiles",
                                         "device_table_bytes", "norm_scratch_elems")]


class zs_param_info_t(C.Structure):
    _fields_ = [(n, C.c_int64) for n in ("numel", "ds_id", "partition_size", "padding",
                                         "shard_offset", "persist_offset", "flat_offset",
                                         "input_offset")] + \
               [(n, C.c_int32) for n in ("persistent", "position", "sub_group", "gather_bucket",
                                         "first_reduce_bucket", "n_reduce_buckets")]


class zs_bucket_info_t(C.Structure):
    _fields_ = [("n_entries", C.c_int32), ("reserved", C.c_int32), ("buf_elems", C.c_int64),
                ("grad_elems", C.c_int64), ("first_tile", C.c_int64), ("n_tiles", C.c_int64)]


class zs_gather_bucket_info_t(C.Structure):
    _fields_ = [("n_params", C.c_int32), ("reserved", C.c_int32), ("flat_offset", C.c_int64),
                ("flat_elems", C.c_int64)]


class zs_sub_group_info_t(C.Structure):
    _fields_ = [("n_params", C.c_int32), ("reserved", C.c_int32), ("shard_lo", C.c_int64),
                ("shard_hi", C.c_int64), ("persist_lo", C.c_int64), ("persist_hi", C.c_int64)]


class zs_loss_scaler(C.Structure):
    _fields_ = [("d_scale", C.c_void_p), ("d_good_steps", C.c_void_p), ("scale_factor", C.c_float),
                ("min_scale", C.c_float), ("scale_window", C.c_int32), ("reserved", C.c_int32)]


class zs_shard_state(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("grad_shards", "param_shards", "master", "exp_avg",
                                          "exp_avg_sq", "persist_grads", "persist_params",
                                          "p_master", "p_exp_avg", "p_exp_avg_sq")]


class zs_sched_config(C.Structure):
    _fields_ = [(n, C.c_int64) for n in ("prefetch_bucket_size", "max_live_parameters",
                                         "max_reuse_distance", "arena_elems",
                                         "gather_ctas", "log_limit")]


class zs_sched_stats_t(C.Structure):
    _fields_ = [(n, C.c_int64) for n in ("passes", "gathers", "params_gathered", "elems_gathered",
                                         "elems_prefetched", "fetch_misses", "max_live_elems",
                                         "max_arena_elems", "invalidations")]


class zs_sched_event(C.Structure):
    _fields_ = [("kind", C.c_int32), ("module_pos", C.c_int32), ("op", C.c_int32),
                ("param", C.c_int32), ("offset", C.c_int64), ("aux", C.c_int64)]


class zs_tensors_config(C.Structure):
    _fields_ = [("state_bits", C.c_int32), ("grad_dtype", C.c_int32), ("param_dtype", C.c_int32),
                ("reserved", C.c_int32)]


class zs_tensor(C.Structure):
    _fields_ = [("numel", C.c_int64)] + \
               [(n, C.c_void_p) for n in ("grad", "param", "master", "exp_avg", "exp_avg_sq",
                                          "exp_avg_scale", "exp_avg_sq_scale")]


class zs_tensors_info_t(C.Structure):
    _fields_ = [("n_tensors", C.c_int32), ("state_bits", C.c_int32), ("numel", C.c_int64),
                ("n_chunks", C.c_int64), ("n_blocks", C.c_int64),
                ("device_table_bytes", C.c_int64)]


class zs_mx4_launch(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("cluster", "split", "stages", "shared_bytes", "tmem_columns", "reserved")]


class zs_mx4_matvec_launch(C.Structure):
    _fields_ = [(n, C.c_int32) for n in ("tokens", "warps_n", "warps_k", "split", "units", "stage", "depth", "shared_bytes")]


_P = C.c_void_p
_i32, _i64, _f32 = C.c_int32, C.c_int64, C.c_float


def _sig(name, res, args):
    f = getattr(_lib, name)
    f.restype = res
    f.argtypes = args
    return f


_sig("zs_last_error", C.c_char_p, [])
_sig("zs_version", C.c_char_p, [])
_sig("zs_default_config", None, [C.POINTER(zs_config), _i32])
_sig("zs_build_partition", _i32, [C.POINTER(zs_config), _i32, C.POINTER(_i64), C.POINTER(_i64),
                                  C.POINTER(_P)])
_sig("zs_free_plan", None, [_P])
_sig("zs_plan_info", _i32, [_P, C.POINTER(zs_plan_info_t)])
_sig("zs_param_info", _i32, [_P, _i32, C.POINTER(zs_param_info_t)])
_sig("zs_param_at", _i32, [_P, _i32, C.POINTER(_i32)])
_sig("zs_bucket_info", _i32, [_P, _i32, C.POINTER(zs_bucket_info_t)])
_sig("zs_bucket_entry", _i32, [_P, _i32, _i32, C.POINTER(_i32), C.POINTER(_i64), C.POINTER(_i64),
                               C.POINTER(_i64)])
_sig("zs_gather_bucket_info", _i32, [_P, _i32, C.POINTER(zs_gather_bucket_info_t)])
_sig("zs_gather_bucket_param", _i32, [_P, _i32, _i32, C.POINTER(_i32)])
_sig("zs_sub_group_info", _i32, [_P, _i32, C.POINTER(zs_sub_group_info_t)])
_sig("zs_plan_table", _i32, [_P, _P, _i64])
_sig("zs_plan_upload", _i32, [_P, _P, _i64, _P])
_sig("zs_partition", _i32, [_P, _P, C.POINTER(zs_shard_state), _P])
_sig("zs_reduce_scatter", _i32, [_P, _i32, C.POINTER(_P), _P, _P, _P, _P])
_sig("zs_grad_norm", _i32, [_P, _P, _P, _P, _i32, _f32, _P, _P, _P, _P])
_sig("zs_adam_step", _i32, [_P, _i32, C.POINTER(zs_adam_hparams), _i64, _P, _P,
                            C.POINTER(zs_shard_state), _P])
_sig("zs_all_gather_coalesced", _i32, [_P, _i32, C.POINTER(_i32), _P, _P, _i64, C.POINTER(_i64), _P])
_sig("zs_device_wait_timeouts", _i32, [C.POINTER(_i32), _i32])
_sig("zs_test_wait_timeout", _i32, [_i64, _P])
_sig("zs_reduce_scatter_all", _i32, [_P, _P, _P, _P, _P, _P])
_sig("zs_reduce_scatter_range", _i32, [_P, _i32, _i32, _P, _P, _P, _P, _P])
_sig("zs_adam_gather", _i32, [_P, C.POINTER(zs_adam_hparams), _i64, _P, _P,
                              C.POINTER(zs_shard_state), _P, _P])
_sig("zs_grad_norm_noalloc", _i32, [_P, _P, _P, _f32, _P, _P, _P, _P])
_sig("zs_unscale_and_clip", _i32, [_P, _P, _P, _P, _i32, _f32, C.POINTER(zs_loss_scaler), _P,
                                   _P, _P, _P])
_sig("zs_shard_step_scaled", _i32, [_P, _P, C.POINTER(zs_shard_state), _P,
                                    C.POINTER(zs_adam_hparams), _i64, _f32,
                                    C.POINTER(zs_loss_scaler), _P, _P, _P, _P, _P])
_sig("zs_sched_create", _i32, [_P, _i32, C.POINTER(_i32), C.POINTER(_i32),
                               C.POINTER(zs_sched_config), _P, C.POINTER(_P)])
_sig("zs_sched_destroy", None, [_P])
_sig("zs_sched_fetch", _i32, [_P, _i32, _P, _P, _P])
_sig("zs_sched_release", _i32, [_P, _i32, _P])
_sig("zs_sched_end_pass", _i32, [_P, _P])
_sig("zs_sched_param_offset", _i32, [_P, _i32, C.POINTER(_i64)])
_sig("zs_sched_stats", _i32, [_P, C.POINTER(zs_sched_stats_t)])
_sig("zs_sched_log", _i32, [_P, C.POINTER(zs_sched_event), _i64, C.POINTER(_i64)])
_sig("zs_shard_step", _i32, [_P, _P, C.POINTER(zs_shard_state), _P, C.POINTER(zs_adam_hparams),
                             _i64, _f32, _P, _P, _P, _P, _P])
_sig("zs_build_tensors", _i32, [C.POINTER(zs_tensors_config), _i32, C.POINTER(zs_tensor),
                                C.POINTER(_P)])
_sig("zs_free_tensors", None, [_P])
_sig("zs_tensors_info", _i32, [_P, C.POINTER(zs_tensors_info_t)])
_sig("zs_tensors_upload", _i32, [_P, _P, _i64, _P])
_sig("zs_adam_tensors", _i32, [_P, C.POINTER(zs_adam_hparams), _i64, _i32, C.c_uint64, _P, _P, _P])
_sig("zs_norm_tensors", _i32, [_P, _P, _f32, C.POINTER(zs_loss_scaler), _P, _P, _P, _P])
_sig("zs_clip_tensors", _i32, [_P, _P, _P, _P])
_sig("zs_mx4_sizes", _i32, [_i64, _i64, C.POINTER(_i64), C.POINTER(_i64), C.POINTER(_i64)])
_sig("zs_mx4_quantize", _i32, [_P, _i64, _i64, _i64, _i32, _P, _P, _P, _P, _P])
_sig("zs_mx4_dequantize", _i32, [_P, _P, _i64, _i64, _P, _i64, _i32, _P])
_sig("zs_mx4_matvec", _i32, [_i64, _i64, _i64, _P, _i64, _i32, _P, _P, _P, _i64, _i32, _P])
_sig("zs_rms_norm", _i32, [_P, _i64, _P, _i64, _P, _i32, _i64, _i64, _i32, _f32, _P, _i64, _P, _i64, _P, _P, _P, _P, _P, _P])
_sig("zs_rms_norm_scratch", _i32, [_i64, _i64, C.POINTER(_i64)])
_sig("zs_rms_norm_backward", _i32, [_P, _i64, _P, _i64, _P, _i32, _P, _P, _i64, _i64, _i64, _i32, _P, _i64, _P, _i32, _P, _P, _P,
                                    _P, _P, _P])
_sig("zs_test_late_copy", _i32, [_P, _P, _i64, _i64, _P])
_sig("zs_test_root", _i32, [_P, _P])
_sig("zs_test_give_up", _i32, [_i32])
_sig("zs_test_mx4_launch", _i32, [_i64, _i64, _i64, C.POINTER(zs_mx4_launch)])
_sig("zs_test_mx4_matvec_launch", _i32, [_i64, _i64, _i64, _i32, C.POINTER(zs_mx4_matvec_launch)])
_sig("zs_mx4_matmul", _i32, [_i64, _i64, _i64, _P, _P, _P, _P, _P, _i64, _i32, _P])


def _check(status: int, fn: str) -> None:
    if status != ZS_OK:
        raise ZsError(status, fn, _lib.zs_last_error().decode(errors="replace"))


def _ptr(x):
    """Device/host address of a tensor, an int, or None (NULL)."""
    if x is None:
        return None
    if hasattr(x, "data_ptr"):
        return x.data_ptr()
    return int(x)


def _find_current_stream():
    """The address of torch's current stream; from its second call on, by the
    quickest way that this torch has (the public one takes about 4 us, as long
    as a small kernel)."""
    global _current_stream, _current_device
    try:
        import torch
        if not torch.cuda.is_available():
            return None
        stream = torch.cuda.current_stream().cuda_stream
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
        device = getattr(torch._C, "_cuda_getDevice", None)
        if raw is not None and device is not None and raw(device()) == stream:
            _current_stream = lambda: raw(device())
            if device() == torch.cuda.current_device():
                _current_device = device
        return stream
    except Exception:  # torch without CUDA
        return None


def _find_current_device() -> int:
    """The index of torch's current device (-2: no CUDA); from the first stream
    on by the quickest way, as above."""
    try:
        import torch
        return torch.cuda.current_device() if torch.cuda.is_available() else -2
    except Exception:  # torch without CUDA
        return -2


_current_stream = _find_current_stream
_current_device = _find_current_device


def _stream(s):
    if s is None:
        return _current_stream()
    if hasattr(s, "cuda_stream"):
        return s.cuda_stream
    return int(s)


def _struct(cls, d):
    if isinstance(d, cls):
        return d
    obj = cls()
    for k, v in d.items():
        setattr(obj, k, v)
    return obj


def zs_version() -> str:
    return _lib.zs_version().decode()


def zs_last_error() -> str:
    return _lib.zs_last_error().decode(errors="replace")


def zs_default_config(n_ranks: int) -> zs_config:
    c = zs_config()
    _lib.zs_default_config(C.byref(c), n_ranks)
    return c


class Plan:
    """Owner of a zs_plan* (freed with the object)."""

    def __init__(self, handle: int):
        self._h = handle
        self._table = None   # device buffer the plan was uploaded to (kept alive)

    @property
    def handle(self):
        return self._h

    def __del__(self):
        if getattr(self, "_h", None):
            _lib.zs_free_plan(self._h)
            self._h = None

    def info(self) -> dict:
        return zs_plan_info(self)


def _h(plan):
    return plan.handle if isinstance(plan, Plan) else plan


def zs_build_partition(config, numel, ds_id=None) -> Plan:
    cfg = config if isinstance(config, zs_config) else _struct(zs_config, dict(config))
    n = len(numel)
    arr = (_i64 * max(n, 1))(*[int(x) for x in numel])
    ids = None
    if ds_id is not None:
        ids = (_i64 * max(n, 1))(*[int(x) for x in ds_id])
    out = _P()
    _check(_lib.zs_build_partition(C.byref(cfg), n, arr, ids, C.byref(out)), "zs_build_partition")
    return Plan(out.value)


def zs_free_plan(plan: Plan) -> None:
    if plan._h:
        _lib.zs_free_plan(plan._h)
        plan._h = None


def _to_dict(s):
    return {name: getattr(s, name) for name, _ in s._fields_ if name != "reserved"}


def zs_plan_info(plan) -> dict:
    o = zs_plan_info_t()
    _check(_lib.zs_plan_info(_h(plan), C.byref(o)), "zs_plan_info")
    return _to_dict(o)


def zs_param_info(plan, i: int) -> dict:
    o = zs_param_info_t()
    _check(_lib.zs_param_info(_h(plan), i, C.byref(o)), "zs_param_info")
    return _to_dict(o)


def zs_param_at(plan, position: int) -> int:
    o = _i32()
    _check(_lib.zs_param_at(_h(plan), position, C.byref(o)), "zs_param_at")
    return o.value


def zs_bucket_info(plan, b: int) -> dict:
    o = zs_bucket_info_t()
    _check(_lib.zs_bucket_info(_h(plan), b, C.byref(o)), "zs_bucket_info")
    return _to_dict(o)


def zs_bucket_entry(plan, b: int, q: int):
    p, lo, hi, off = _i32(), _i64(), _i64(), _i64()
    _check(_lib.zs_bucket_entry(_h(plan), b, q, C.byref(p), C.byref(lo), C.byref(hi), C.byref(off)),
           "zs_bucket_entry")
    return p.value, lo.value, hi.value, off.value


def zs_gather_bucket_info(plan, g: int) -> dict:
    o = zs_gather_bucket_info_t()
    _check(_lib.zs_gather_bucket_info(_h(plan), g, C.byref(o)), "zs_gather_bucket_info")
    return _to_dict(o)


def zs_gather_bucket_param(plan, g: int, i: int) -> int:
    o = _i32()
    _check(_lib.zs_gather_bucket_param(_h(plan), g, i, C.byref(o)), "zs_gather_bucket_param")
    return o.value


def zs_sub_group_info(plan, s: int) -> dict:
    o = zs_sub_group_info_t()
    _check(_lib.zs_sub_group_info(_h(plan), s, C.byref(o)), "zs_sub_group_info")
    return _to_dict(o)


def zs_plan_table(plan):
    """Host copy of the work table as a numpy structured array."""
    import numpy as np
    info = zs_plan_info(plan)
    arr = np.zeros(info["n_tiles"], dtype=TILE_DTYPE)
    _check(_lib.zs_plan_table(_h(plan), arr.ctypes.data if arr.size else None, arr.nbytes),
           "zs_plan_table")
    return arr


def zs_plan_launch_order(plan):
    """The reduce-scatter's launch order (int32 per tile: launch position i
    works on tile order[i]), the part of the device table after the tiles."""
    import numpy as np
    info = zs_plan_info(plan)
    n = info["n_tiles"]
    buf = np.zeros(info["device_table_bytes"], dtype=np.uint8)
    _check(_lib.zs_plan_table(_h(plan), buf.ctypes.data if buf.size else None, buf.nbytes),
           "zs_plan_table")
    rec = np.dtype(TILE_DTYPE).itemsize
    return buf[rec * n:(rec + 4) * n].view(np.int32).copy()


def zs_plan_upload(plan, d_table, nbytes: int, stream=None) -> None:
    _check(_lib.zs_plan_upload(_h(plan), _ptr(d_table), int(nbytes), _stream(stream)),
           "zs_plan_upload")
    if isinstance(plan, Plan):
        plan._table = d_table


def make_state(**kw) -> zs_shard_state:
    """zs_shard_state from tensors / addresses given by field name."""
    st = zs_shard_state()
    for name, _ in zs_shard_state._fields_:
        setattr(st, name, _ptr(kw.get(name)))
    return st


def zs_partition(plan, full_params, state: zs_shard_state, stream=None) -> None:
    _check(_lib.zs_partition(_h(plan), _ptr(full_params), C.byref(state), _stream(stream)),
           "zs_partition")


def zs_reduce_scatter(plan, bucket: int, rank_grads, grad_shards, persist_grads,
                      norm_scratch=None, stream=None) -> None:
    ptrs = (_P * max(len(rank_grads), 1))(*[_ptr(x) for x in rank_grads])
    _check(_lib.zs_reduce_scatter(_h(plan), bucket, ptrs, _ptr(grad_shards), _ptr(persist_grads),
                                  _ptr(norm_scratch), _stream(stream)), "zs_reduce_scatter")


def zs_grad_norm(plan, grad_shards, persist_grads, norm_scratch, recompute: bool, max_norm: float,
                 d_norm, d_clip_coef, d_flags, stream=None) -> None:
    _check(_lib.zs_grad_norm(_h(plan), _ptr(grad_shards), _ptr(persist_grads), _ptr(norm_scratch),
                             1 if recompute else 0, float(max_norm), _ptr(d_norm),
                             _ptr(d_clip_coef), _ptr(d_flags), _stream(stream)), "zs_grad_norm")


def _hp(hp) -> zs_adam_hparams:
    if isinstance(hp, zs_adam_hparams):
        return hp
    d = hp if type(hp) is dict else dict(hp)
    return zs_adam_hparams(float(d["lr"]), float(d["beta1"]), float(d["beta2"]), float(d["eps"]),
                           float(d["weight_decay"]), int(d.get("adamw", 1)),
                           int(d.get("bias_correction", 1)))


def zs_adam_step(plan, sub_group: int, hp, step: int, d_clip_coef, d_flags,
                 state: zs_shard_state, stream=None) -> None:
    h = _hp(hp)
    _check(_lib.zs_adam_step(_h(plan), sub_group, C.byref(h), int(step), _ptr(d_clip_coef),
                             _ptr(d_flags), C.byref(state), _stream(stream)), "zs_adam_step")


def zs_all_gather_coalesced(plan, params, param_shards, flat_out, flat_capacity: int,
                            stream=None) -> list:
    n = len(params)
    arr = (_i32 * max(n, 1))(*[int(x) for x in params])
    views = (_i64 * max(n, 1))()
    _check(_lib.zs_all_gather_coalesced(_h(plan), n, arr, _ptr(param_shards), _ptr(flat_out),
                                        int(flat_capacity), views, _stream(stream)),
           "zs_all_gather_coalesced")
    return [views[i] for i in range(n)]


def zs_device_wait_timeouts(reset: bool = False) -> int:
    """Bounded device waits that gave up on the current device (synchronous)."""
    c = _i32()
    st = _lib.zs_device_wait_timeouts(C.byref(c), int(bool(reset)))
    if st != ZS_ETIMEOUT:
        _check(st, "zs_device_wait_timeouts")
    return c.value


def zs_test_wait_timeout(limit_ns: int, stream=None) -> None:
    """Enqueue one bounded wait that runs out after limit_ns (test hook)."""
    _check(_lib.zs_test_wait_timeout(int(limit_ns), _stream(stream)), "zs_test_wait_timeout")


def zs_shard_step(plan, d_rank_grads, state: zs_shard_state, norm_scratch, hp, step: int,
                  max_norm: float, d_norm, d_clip_coef, d_flags, flat_out, stream=None) -> None:
    h = _hp(hp)
    _check(_lib.zs_shard_step(_h(plan), _ptr(d_rank_grads), C.byref(state), _ptr(norm_scratch),
                              C.byref(h), int(step), float(max_norm), _ptr(d_norm),
                              _ptr(d_clip_coef), _ptr(d_flags), _ptr(flat_out), _stream(stream)),
           "zs_shard_step")


def zs_reduce_scatter_all(plan, d_rank_grads, grad_shards, persist_grads, norm_scratch,
                          stream=None) -> None:
    _check(_lib.zs_reduce_scatter_all(_h(plan), _ptr(d_rank_grads), _ptr(grad_shards),
                                      _ptr(persist_grads), _ptr(norm_scratch), _stream(stream)),
           "zs_reduce_scatter_all")


def zs_reduce_scatter_range(plan, first_bucket: int, n_buckets: int, d_rank_grads, grad_shards,
                            persist_grads, norm_scratch, stream=None) -> None:
    _check(_lib.zs_reduce_scatter_range(_h(plan), int(first_bucket), int(n_buckets),
                                        _ptr(d_rank_grads), _ptr(grad_shards), _ptr(persist_grads),
                                        _ptr(norm_scratch), _stream(stream)),
           "zs_reduce_scatter_range")


def zs_adam_gather(plan, hp, step: int, d_clip_coef, d_flags, state: zs_shard_state, flat_out,
                   stream=None) -> None:
    h = _hp(hp)
    _check(_lib.zs_adam_gather(_h(plan), C.byref(h), int(step), _ptr(d_clip_coef), _ptr(d_flags),
                               C.byref(state), _ptr(flat_out), _stream(stream)), "zs_adam_gather")


def zs_grad_norm_noalloc(plan, grad_shards, persist_grads, max_norm: float, d_norm, d_clip_coef,
                         d_flags, stream=None) -> None:
    """zs_grad_norm(recompute=1) with the library's built-in scratch array,
    for callers that cannot allocate device memory."""
    _check(_lib.zs_grad_norm_noalloc(_h(plan), _ptr(grad_shards), _ptr(persist_grads),
                                     float(max_norm), _ptr(d_norm), _ptr(d_clip_coef),
                                     _ptr(d_flags), _stream(stream)), "zs_grad_norm_noalloc")


def make_loss_scaler(d_scale, d_good_steps=None, scale_factor=2.0, min_scale=1.0,
                     scale_window=1000) -> zs_loss_scaler:
    """zs_loss_scaler from device tensors / addresses (float32 scale, int32 count)."""
    return zs_loss_scaler(_ptr(d_scale), _ptr(d_good_steps), float(scale_factor),
                          float(min_scale), int(scale_window), 0)


def zs_unscale_and_clip(plan, grad_shards, persist_grads, norm_scratch, recompute: bool,
                        max_norm: float, scaler: zs_loss_scaler, d_norm, d_clip_coef, d_flags,
                        stream=None) -> None:
    _check(_lib.zs_unscale_and_clip(_h(plan), _ptr(grad_shards), _ptr(persist_grads),
                                    _ptr(norm_scratch), 1 if recompute else 0, float(max_norm),
                                    C.byref(scaler), _ptr(d_norm), _ptr(d_clip_coef),
                                    _ptr(d_flags), _stream(stream)), "zs_unscale_and_clip")


def zs_shard_step_scaled(plan, d_rank_grads, state: zs_shard_state, norm_scratch, hp, step: int,
                         max_norm: float, scaler: zs_loss_scaler, d_norm, d_clip_coef, d_flags,
                         flat_out, stream=None) -> None:
    h = _hp(hp)
    _check(_lib.zs_shard_step_scaled(_h(plan), _ptr(d_rank_grads), C.byref(state),
                                     _ptr(norm_scratch), C.byref(h), int(step), float(max_norm),
                                     C.byref(scaler), _ptr(d_norm), _ptr(d_clip_coef),
                                     _ptr(d_flags), _ptr(flat_out), _stream(stream)),
           "zs_shard_step_scaled")


class Sched:
    """Owner of a zs_sched* (destroyed with the object); keeps the plan alive."""

    def __init__(self, handle, plan, arena):
        self._h, self._plan, self._arena = handle, plan, arena

    @property
    def handle(self):
        return self._h

    def __del__(self):
        if getattr(self, "_h", None):
            _lib.zs_sched_destroy(self._h)
            self._h = None


def zs_sched_create(plan, modules, cfg, d_arena=None) -> Sched:
    """modules: list of lists of parameter indices; cfg: dict or zs_sched_config."""
    c = cfg if isinstance(cfg, zs_sched_config) else _struct(zs_sched_config, dict(cfg))
    offs, flat = [0], []
    for m in modules:
        flat += [int(p) for p in m]
        offs.append(len(flat))
    o = (_i32 * len(offs))(*offs)
    f = (_i32 * max(len(flat), 1))(*flat)
    out = _P()
    _check(_lib.zs_sched_create(_h(plan), len(modules), o, f, C.byref(c), _ptr(d_arena),
                                C.byref(out)), "zs_sched_create")
    return Sched(out.value, plan, d_arena)


def zs_sched_fetch(sched, module: int, param_shards=None, compute_stream=None,
                   gather_stream=None) -> None:
    _check(_lib.zs_sched_fetch(sched.handle, module, _ptr(param_shards),
                               _stream(compute_stream) if sched._arena is not None else None,
                               _stream(gather_stream) if sched._arena is not None else None),
           "zs_sched_fetch")


def zs_sched_release(sched, module: int, compute_stream=None) -> None:
    _check(_lib.zs_sched_release(sched.handle, module,
                                 _stream(compute_stream) if sched._arena is not None else None),
           "zs_sched_release")


def zs_sched_end_pass(sched, compute_stream=None) -> None:
    _check(_lib.zs_sched_end_pass(sched.handle,
                                  _stream(compute_stream) if sched._arena is not None else None),
           "zs_sched_end_pass")


def zs_sched_param_offset(sched, param: int) -> int:
    o = _i64()
    _check(_lib.zs_sched_param_offset(sched.handle, param, C.byref(o)), "zs_sched_param_offset")
    return o.value


def zs_sched_stats(sched) -> dict:
    o = zs_sched_stats_t()
    _check(_lib.zs_sched_stats(sched.handle, C.byref(o)), "zs_sched_stats")
    return {n: getattr(o, n) for n, _ in o._fields_}


def zs_sched_log(sched) -> list:
    n = _i64()
    _check(_lib.zs_sched_log(sched.handle, None, 0, C.byref(n)), "zs_sched_log")
    buf = (zs_sched_event * max(n.value, 1))()
    _check(_lib.zs_sched_log(sched.handle, buf, n.value, C.byref(n)), "zs_sched_log")
    return [(e.kind, e.module_pos, e.op, e.param, e.offset, e.aux) for e in buf[:n.value]]


# ---------------------------------------------- training with little memory --

_DTYPES: dict = {}


def _dtype(t) -> int:
    """ZS_DTYPE_* of a torch tensor."""
    if not _DTYPES:
        import torch
        _DTYPES.update({torch.bfloat16: ZS_DTYPE_BF16, torch.float16: ZS_DTYPE_FP16,
                        torch.float32: ZS_DTYPE_FP32})
    got = _DTYPES.get(t.dtype)
    if got is None:
        raise TypeError(f"bfloat16, float16 or float32 expected, got {t.dtype}")
    return got


def _elsewhere(x, what: str, device: int) -> None:
    """Refuse a torch tensor that is not on the current device, unless the
    device reaches it all the same (pinned host memory) or nothing is in it."""
    if x.numel() == 0 or x.get_device() < 0 and device >= 0 and x.is_pinned():
        return
    raise ValueError(f"{what}: a tensor on " + (f"cuda:{device}" if device >= 0 else "a GPU") + f" expected, got {x.device}")


def _device_address(x, what: str, device: int):
    """The address of a torch tensor on the device, or the address (or None) x."""
    try:
        at = x.data_ptr()
    except AttributeError:
        return None if x is None else int(x)
    if x.get_device() != device:
        _elsewhere(x, what, device)
    return at


class Tensors:
    """Owner of a zs_tensors* (freed with the object); keeps the torch tensors alive."""

    def __init__(self, handle: int, keep):
        self._h, self._keep, self._table = handle, keep, None
        self._device = None              # of the torch tensors, once uploaded
        self._n_chunks = None

    @property
    def handle(self):
        return self._h

    @property
    def n_chunks(self) -> int:
        if self._n_chunks is None:
            self._n_chunks = zs_tensors_info(self)["n_chunks"]
        return self._n_chunks

    def __del__(self):
        if getattr(self, "_h", None):
            _lib.zs_free_tensors(self._h)
            self._h = None


# names of zs_tensor's fields, 8 bytes each, by place
_TENSOR_AT = {name: i for i, (name, _) in enumerate(zs_tensor._fields_)}


def zs_build_tensors(tensors, state_bits: int = 32, grad_dtype=None, param_dtype=None) -> Tensors:
    """tensors: a list of dicts by the names of zs_tensor, of contiguous torch
    tensors (param, and with state_bits 32 the scales, may be left out), or of
    addresses with "numel" and both dtypes given.  Torch tensors give the
    dtypes themselves; all gradients have one, all parameters one."""
    size = {"master": 4, "exp_avg": state_bits // 8, "exp_avg_sq": state_bits // 8,
            "exp_avg_scale": 4, "exp_avg_sq_scale": 4}
    dtypes = {"grad": grad_dtype, "param": param_dtype}
    n = len(tensors)
    rows = []          # the fields of each zs_tensor
    keep = []          # the torch tensors (a caller may put others into its dicts)
    for i, t in enumerate(tensors):
        numel = t.get("numel")
        numel = t["master"].numel() if numel is None else int(numel)
        blocks = -(-numel // ZS_STATE_BLOCK)
        row = [numel, 0, 0, 0, 0, 0, 0, 0]
        for name, x in t.items():
            at = _TENSOR_AT.get(name)
            if at is None:
                raise TypeError(f"tensor {i}: unknown {name}")
            if at == 0 or x is None:
                continue
            try:
                row[at] = x.data_ptr()
            except AttributeError:
                row[at] = int(x)
                continue
            need = blocks if at >= 6 else numel
            if x.numel() < need or not x.is_contiguous():
                raise ValueError(f"tensor {i}: {name} is not {need} contiguous elements")
            if at <= 2:
                d = _dtype(x)
                if dtypes[name] is None:
                    dtypes[name] = d
                elif dtypes[name] != d:
                    raise TypeError(f"tensor {i}: {name} is {x.dtype}, another type than before it")
            elif x.itemsize != size[name]:
                raise TypeError(f"tensor {i}: {name} is {x.dtype}, {size[name]} bytes an element expected")
            keep.append(x)
        rows += row
    flat = (_i64 * max(len(rows), 1))(*[r - (1 << 64) if r >= 1 << 63 else r for r in rows])
    arr = C.cast(flat, C.POINTER(zs_tensor))
    grad_dtype, param_dtype = dtypes["grad"], dtypes["param"]
    cfg = zs_tensors_config(int(state_bits), ZS_DTYPE_BF16 if grad_dtype is None else int(grad_dtype),
                            ZS_DTYPE_BF16 if param_dtype is None else int(param_dtype), 0)
    out = _P()
    _check(_lib.zs_build_tensors(C.byref(cfg), n, arr, C.byref(out)), "zs_build_tensors")
    return Tensors(out.value, keep)


def zs_free_tensors(tensors: Tensors) -> None:
    if tensors._h:
        _lib.zs_free_tensors(tensors._h)
        tensors._h = None


def zs_tensors_info(tensors) -> dict:
    o = zs_tensors_info_t()
    _check(_lib.zs_tensors_info(tensors.handle, C.byref(o)), "zs_tensors_info")
    return _to_dict(o)


def zs_tensors_upload(tensors, d_table, nbytes: int, stream=None) -> None:
    device = _current_device()
    if not {x.get_device() for x in tensors._keep} <= {device}:
        for x in tensors._keep:
            if x.get_device() != device:
                _elsewhere(x, "zs_tensors_upload", device)
    _device_address(d_table, "zs_tensors_upload", device)
    if tensors._keep:
        tensors._device = device
    _check(_lib.zs_tensors_upload(tensors.handle, _ptr(d_table), int(nbytes), _stream(stream)),
           "zs_tensors_upload")
    tensors._table = d_table


_ROUNDING = {"nearest": ZS_ROUND_NEAREST, "stochastic": ZS_ROUND_STOCHASTIC}


def zs_adam_tensors(tensors, hp, step: int, d_clip_coef=None, d_flags=None, rounding="nearest",
                    seed: int = 0, stream=None) -> None:
    h = _hp(hp)
    device = _current_device()
    if tensors._device != device and tensors._device is not None:
        raise ValueError(f"zs_adam_tensors: the list is of cuda:{tensors._device}, the current device is cuda:{device}")
    st = _lib.zs_adam_tensors(tensors.handle, C.byref(h), int(step),
                              _ROUNDING[rounding] if isinstance(rounding, str) else int(rounding),
                              int(seed) & 0xFFFFFFFFFFFFFFFF,
                              None if d_clip_coef is None else _device_address(d_clip_coef, "zs_adam_tensors", device),
                              None if d_flags is None else _device_address(d_flags, "zs_adam_tensors", device),
                              _current_stream() if stream is None else _stream(stream))
    if st:
        _check(st, "zs_adam_tensors")


def _on_list(tensors, fn: str) -> int:
    """The current device, which has to be the list's."""
    device = _current_device()
    if tensors._device != device and tensors._device is not None:
        raise ValueError(f"{fn}: the list is of cuda:{tensors._device}, the current device is cuda:{device}")
    return device


def _scalar(x, what: str, device: int, itemsize: int = 4):
    """The address of a device scalar (an address, or None, as it is)."""
    if x is None:
        return None
    at = _device_address(x, what, device)
    if hasattr(x, "data_ptr") and (x.numel() < 1 or x.itemsize != itemsize):
        raise TypeError(f"{what}: a scalar of {itemsize} bytes expected, got {tuple(x.shape)} of {x.dtype}")
    return at


def zs_norm_tensors(tensors, scratch, max_norm: float, d_norm, d_clip_coef, d_flags, scaler=None,
                    stream=None) -> None:
    """scratch: at least zs_tensors_info's n_chunks float64 (tensor or address);
    scaler: of make_loss_scaler, or None."""
    device = _on_list(tensors, "zs_norm_tensors")
    d_scratch = _device_address(scratch, "scratch", device)
    if hasattr(scratch, "data_ptr"):
        need = 8 * tensors.n_chunks
        if scratch.nbytes < need or not scratch.is_contiguous():
            raise ValueError(f"scratch: {need} contiguous bytes expected, got {tuple(scratch.shape)} of {scratch.dtype}")
    st = _lib.zs_norm_tensors(tensors.handle, d_scratch, max_norm, None if scaler is None else C.byref(scaler),
                              _scalar(d_norm, "d_norm", device), _scalar(d_clip_coef, "d_clip_coef", device),
                              _scalar(d_flags, "d_flags", device), _current_stream() if stream is None else _stream(stream))
    if st:
        _check(st, "zs_norm_tensors")


def zs_clip_tensors(tensors, d_clip_coef, d_flags=None, stream=None) -> None:
    device = _on_list(tensors, "zs_clip_tensors")
    st = _lib.zs_clip_tensors(tensors.handle, _scalar(d_clip_coef, "d_clip_coef", device), _scalar(d_flags, "d_flags", device),
                              _current_stream() if stream is None else _stream(stream))
    if st:
        _check(st, "zs_clip_tensors")


def zs_mx4_sizes(rows: int, cols: int) -> dict:
    r, c, s = _i64(), _i64(), _i64()
    _check(_lib.zs_mx4_sizes(int(rows), int(cols), C.byref(r), C.byref(c), C.byref(s)), "zs_mx4_sizes")
    return dict(row_bytes=r.value, code_bytes=c.value, scale_bytes=s.value)


def _mx4(held, rows: int, cols: int, device: int):
    """(codes, scales) addresses of a dict with "codes" and "scales" (uint8
    tensors on the device, or addresses), whose tensors are large enough for
    rows x cols.  Codes are flat, or a row of the matrix a row: the kernels
    take the distance of rows from cols, so another one is another matrix."""
    if held is None:
        return None, None
    codes, scales = held["codes"], held["scales"]
    try:
        at = codes.data_ptr(), scales.data_ptr()
    except AttributeError:
        return _device_address(codes, "codes", device), _device_address(scales, "scales", device)
    groups = (cols + 31) >> 5
    if (codes.nbytes < 16 * rows * groups or scales.nbytes < ((rows + 127) >> 7) * ((groups + 7) >> 3) << 10
            or codes.itemsize != 1 or scales.itemsize != 1 or not codes.is_contiguous() or not scales.is_contiguous()):
        raise ValueError(f"{16 * rows * groups} and {((rows + 127) >> 7) * ((groups + 7) >> 3) << 10} contiguous bytes expected for "
                         f"{rows} x {cols}, got {tuple(codes.shape)} of {codes.dtype} and {tuple(scales.shape)} of {scales.dtype}")
    if codes.nbytes != 16 * rows * groups and codes.dim() > 1 and codes.shape[-1] != 16 * groups:
        raise ValueError(f"codes are {tuple(codes.shape)}: {16 * groups} bytes a row expected for {cols} columns")
    if codes.get_device() != device or scales.get_device() != device:
        for name, x in (("codes", codes), ("scales", scales)):
            if x.get_device() != device:
                _elsewhere(x, name, device)
    return at


def _matrix(x, what: str):
    """(rows, cols, row stride, dtype) of a 2-D torch tensor whose rows are
    contiguous."""
    shape = x.shape
    if len(shape) != 2:
        raise ValueError(f"{what}: a matrix expected, got {tuple(shape)}")
    rows, cols = shape
    ld, one = x.stride()
    if one != 1 and cols > 1:
        raise ValueError(f"{what}: rows are not contiguous")
    return rows, cols, ld if rows > 1 else cols, _dtype(x)


def zs_mx4_quantize(x, rows=None, cols=None, stream=None) -> None:
    """x: [r, c] torch matrix.  rows: the dict of x held along its rows
    ([r, c]); cols: of the transposed matrix ([c, r]); either may be None."""
    device = _current_device()
    r, c, ld, dtype = _matrix(x, "x")
    rc, rs = _mx4(rows, r, c, device)
    cc, cs = _mx4(cols, c, r, device)
    if x.get_device() != device:
        _elsewhere(x, "x", device)
    st = _lib.zs_mx4_quantize(x.data_ptr(), r, c, ld, dtype, rc, rs, cc, cs, _current_stream() if stream is None else _stream(stream))
    if st:
        _check(st, "zs_mx4_quantize")


def zs_mx4_dequantize(held, out, stream=None):
    """out: [r, c] torch matrix that receives the values; returned."""
    device = _current_device()
    r, c, ld, dtype = _matrix(out, "out")
    hc, hs = _mx4(held, r, c, device)
    if out.get_device() != device:
        _elsewhere(out, "out", device)
    st = _lib.zs_mx4_dequantize(hc, hs, r, c, out.data_ptr(), ld, dtype, _current_stream() if stream is None else _stream(stream))
    if st:
        _check(st, "zs_mx4_dequantize")
    return out


def zs_mx4_matmul(a, b, k: int, out, stream=None):
    """out [m, n] = a [m, k] b [n, k]^T of two held matrices; out is returned."""
    device = _current_device()
    m, n, ld, dtype = _matrix(out, "out")
    ac, as_ = _mx4(a, m, k, device)
    bc, bs = _mx4(b, n, k, device)
    if out.get_device() != device:
        _elsewhere(out, "out", device)
    st = _lib.zs_mx4_matmul(m, n, k, ac, as_, bc, bs, out.data_ptr(), ld, dtype, _current_stream() if stream is None else _stream(stream))
    if st:
        _check(st, "zs_mx4_matmul")
    return out


def zs_mx4_matvec(x, w, out, stream=None):
    """out [m, n] = x [m, k] w [n, k]^T of a torch matrix and a held weight; out is returned."""
    device = _current_device()
    m, k, ldx, dtype = _matrix(x, "x")
    rows, n, ldo, out_dtype = _matrix(out, "out")
    if rows != m:
        raise ValueError(f"out: {m} rows expected, got {rows}")
    wc, ws = _mx4(w, n, k, device)
    if x.get_device() != device or out.get_device() != device:
        for name, y in (("x", x), ("out", out)):
            if y.get_device() != device:
                _elsewhere(y, name, device)
    st = _lib.zs_mx4_matvec(m, n, k, x.data_ptr(), ldx, dtype, wc, ws, out.data_ptr(), ldo, out_dtype,
                            _current_stream() if stream is None else _stream(stream))
    if st:
        _check(st, "zs_mx4_matvec")
    return out


def _like(m, what: str, x, device: int):
    """(address, row stride) of a matrix of x's sizes and type, or of none."""
    if m is None:
        return None, 0
    if m.shape != x.shape or m.dtype != x.dtype:
        raise ValueError(f"{what}: {tuple(x.shape)} of {x.dtype} expected, got {tuple(m.shape)} of {m.dtype}")
    rows, cols = m.shape
    ld, one = m.stride()
    if one != 1 and cols > 1:
        raise ValueError(f"{what}: rows are not contiguous")
    if m.get_device() != device:
        _elsewhere(m, what, device)
    return m.data_ptr(), ld if rows > 1 else cols


def _vector(v, what: str, n: int, device: int, dtype=None):
    """(address, dtype) of a contiguous vector of n elements, or of none."""
    if v is None:
        return None, ZS_DTYPE_FP32
    d = _DTYPES.get(v.dtype)
    if d is None:
        d = _dtype(v)
    if v.dim() != 1 or v.numel() != n or n > 1 and v.stride(0) != 1 or dtype is not None and d != dtype:
        raise ValueError(f"{what}: {n} contiguous elements{' of float32' if dtype == ZS_DTYPE_FP32 else ''} expected, "
                         f"got {tuple(v.shape)} of {v.dtype}")
    if v.get_device() != device:
        _elsewhere(v, what, device)
    return v.data_ptr(), d


def zs_rms_norm(x, weight, eps: float, rstd, residual=None, sum=None, out=None, rows=None, cols=None, stream=None) -> None:
    """x, residual, sum, out: [r, c] torch matrices of one type; weight [c];
    rstd [r] float32.  rows: the dict of the result held along its rows, cols:
    along its columns (of the transposed matrix)."""
    device = _current_device()
    r, c, ldx, dtype = _matrix(x, "x")
    ra, ldr = _like(residual, "residual", x, device)
    sa, lds = _like(sum, "sum", x, device)
    oa, ldo = _like(out, "out", x, device)
    wa, wd = _vector(weight, "weight", c, device)
    rc, rs = _mx4(rows, r, c, device)
    cc, cs = _mx4(cols, c, r, device)
    if x.get_device() != device:
        _elsewhere(x, "x", device)
    st = _lib.zs_rms_norm(x.data_ptr(), ldx, ra, ldr, wa, wd, r, c, dtype, eps, sa, lds, oa, ldo,
                          _vector(rstd, "rstd", r, device, ZS_DTYPE_FP32)[0], rc, rs, cc, cs,
                          _current_stream() if stream is None else _stream(stream))
    if st:
        _check(st, "zs_rms_norm")


def zs_rms_norm_scratch(rows: int, cols: int) -> int:
    n = _i64()
    _check(_lib.zs_rms_norm_scratch(int(rows), int(cols), C.byref(n)), "zs_rms_norm_scratch")
    return n.value


def zs_rms_norm_backward(dy, x, weight, rstd, dx, scratch, residual=None, dw=None, rows=None, cols=None, stream=None) -> None:
    """dy, x, residual, dx: [r, c] torch matrices of one type; weight, dw [c];
    rstd [r] float32; scratch: zs_rms_norm_scratch's bytes.  rows, cols:
    the dicts of dx held along its rows and its columns."""
    device = _current_device()
    r, c, ldx, dtype = _matrix(x, "x")
    ya, ldy = _like(dy, "dy", x, device)
    ra, ldr = _like(residual, "residual", x, device)
    da, ldd = _like(dx, "dx", x, device)
    wa, wd = _vector(weight, "weight", c, device)
    dwa, dwd = _vector(dw, "dw", c, device)
    rc, rs = _mx4(rows, r, c, device)
    cc, cs = _mx4(cols, c, r, device)
    sa = _device_address(scratch, "scratch", device)
    if x.get_device() != device:
        _elsewhere(x, "x", device)
    if hasattr(scratch, "data_ptr") and (scratch.nbytes < zs_rms_norm_scratch(r, c) or not scratch.is_contiguous()):
        raise ValueError(f"scratch: {zs_rms_norm_scratch(r, c)} contiguous bytes expected, got {tuple(scratch.shape)} of {scratch.dtype}")
    st = _lib.zs_rms_norm_backward(ya, ldy, x.data_ptr(), ldx, wa, wd,
                                   _vector(rstd, "rstd", r, device, ZS_DTYPE_FP32)[0], ra, ldr, r, c, dtype, da, ldd, dwa, dwd, sa,
                                   rc, rs, cc, cs, _current_stream() if stream is None else _stream(stream))
    if st:
        _check(st, "zs_rms_norm_backward")


def zs_test_late_copy(dst, src, nbytes: int, delay_ns: int, stream=None) -> None:
    """A kernel that lets the next one begin, and copies src to dst delay_ns later (test hook)."""
    _check(_lib.zs_test_late_copy(_ptr(dst), _ptr(src), int(nbytes), int(delay_ns), _stream(stream)), "zs_test_late_copy")


def zs_test_root(d_count, stream=None) -> None:
    """Counts the floats whose root the 8-bit update would not round correctly (test)."""
    _check(_lib.zs_test_root(_ptr(d_count), _stream(stream)), "zs_test_root")


def zs_test_give_up(at: int = -1) -> None:
    """From now on the waits for stage `at` of the low-memory kernels' operands run out; -1: none (test hook)."""
    _check(_lib.zs_test_give_up(int(at)), "zs_test_give_up")


def zs_test_mx4_launch(m: int, n: int, k: int) -> dict:
    """What a CTA of zs_mx4_matmul's launch asks of its SM (for tests)."""
    o = zs_mx4_launch()
    _check(_lib.zs_test_mx4_launch(int(m), int(n), int(k), C.byref(o)), "zs_test_mx4_launch")
    return _to_dict(o)


def zs_test_mx4_matvec_launch(m: int, n: int, k: int, dtype: int) -> dict:
    """How zs_mx4_matvec shares out a product of these sizes on the current device (for tests)."""
    o = zs_mx4_matvec_launch()
    _check(_lib.zs_test_mx4_matvec_launch(int(m), int(n), int(k), int(dtype), C.byref(o)), "zs_test_mx4_matvec_launch")
    return _to_dict(o)
