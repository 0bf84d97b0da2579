"""GB300-native FSDP FlatParameter shard step.

Python binding of the C ABI in ``include/fsdp.h`` (libfsdp_gb300.so, built
for sm_103a by ``fully_sharded_gb300.build``). The functions below have the
ABI's names and only marshal arguments: tensors become device pointers, lists
become host pointer arrays, the status code becomes an exception. Every step
of the path runs in the CUDA library; there is no other implementation, and
importing this package fails when the library is missing.

Tensors are torch CUDA tensors (contiguous) or raw integer device addresses.
bf16 buffers may be torch.bfloat16, torch.int16 or torch.uint16 (bit patterns).
"""
from __future__ import annotations

import ctypes
import os
from typing import Sequence

from . import build as _build_mod

__all__ = [
    "FsdpError", "Layout", "AdamHyper", "Account", "library_path",
    "fsdp_flatten_layout", "fsdp_pack_flat", "fsdp_unpack_flat", "fsdp_reduce_scatter",
    "fsdp_adam_shard_step", "fsdp_all_gather", "fsdp_shard_step", "fsdp_shard_step_grouped",
    "fsdp_account", "fsdp_status_string", "UnitArgs", "UnitBatch",
    "fsdp_shard_step_grouped_launches", "fsdp_pipeline_step", "PipelineUnit", "PipelineBatch",
    "fsdp_pipeline_step_noalloc", "fsdp_all_gather_state", "fsdp_zero1_step", "fsdp_account_zero",
    "fsdp_shard_step_grouped_plan", "fsdp_device_status", "fsdp_selftest_wait_timeout",
    "fsdp_offload_step", "OffloadUnit", "OffloadBatch", "fsdp_reduce_scatter_ranks",
    "fsdp_adam_shard_step_grouped", "AdamShard",
    "fsdp_rmsnorm", "fsdp_rmsnorm_backward", "fsdp_rmsnorm_backward_workspace",
    "NewtonSchulz", "NewtonSchulzBatch", "fsdp_newton_schulz", "fsdp_newton_schulz_workspace",
    "Muon", "MuonTensor", "MuonUnit", "fsdp_muon_step", "fsdp_muon_workspace",
]

FSDP_OK = 0
FSDP_EINVAL = -1
FSDP_EALIAS = -2
FSDP_ECUDA = -3
FSDP_ENOSPACE = -4
FSDP_EWORKSPACE = -5
NOALLOC_STAGING_BYTES = 64 << 20  # FSDP_NOALLOC_STAGING_BYTES of include/fsdp.h
FSDP_DTYPE_F32 = 0
FSDP_DTYPE_BF16 = 1
FSDP_DTYPE_E4M3 = 2
MAX_WORLD = 64

_c_i32, _c_i64, _c_dbl, _c_p = ctypes.c_int32, ctypes.c_int64, ctypes.c_double, ctypes.c_void_p


class Layout(ctypes.Structure):
    _fields_ = [("numel", _c_i64), ("padded_numel", _c_i64), ("shard_numel", _c_i64),
                ("world_size", _c_i32), ("shard_factor", _c_i32), ("n_tensors", _c_i32)]

    def __repr__(self):
        return ("Layout(numel=%d, padded_numel=%d, shard_numel=%d, world_size=%d, shard_factor=%d, "
                "n_tensors=%d)" % (self.numel, self.padded_numel, self.shard_numel, self.world_size,
                                   self.shard_factor, self.n_tensors))


class AdamHyper(ctypes.Structure):
    _fields_ = [("lr", _c_dbl), ("beta1", _c_dbl), ("beta2", _c_dbl), ("eps", _c_dbl),
                ("weight_decay", _c_dbl), ("step", _c_i64)]

    def __init__(self, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, step=1):
        super().__init__(lr, beta1, beta2, eps, weight_decay, step)


class UnitArgs(ctypes.Structure):
    _fields_ = [("layout", ctypes.POINTER(Layout)), ("grads", _c_p), ("master", _c_p),
                ("exp_avg", _c_p), ("exp_avg_sq", _c_p), ("other_shards", _c_p),
                ("full_out", _c_p)]


class PipelineUnit(ctypes.Structure):
    _fields_ = [("layout", ctypes.POINTER(Layout)), ("grad_slices", _c_p), ("master", _c_p),
                ("exp_avg", _c_p), ("exp_avg_sq", _c_p), ("other_shards", _c_p), ("full_out", _c_p),
                ("shard_out", _c_p)]


class OffloadUnit(ctypes.Structure):
    _fields_ = [("layout", ctypes.POINTER(Layout)), ("grads", _c_p), ("master", _c_p), ("exp_avg", _c_p),
                ("exp_avg_sq", _c_p), ("other_shards", _c_p), ("full_out", _c_p)]


class AdamShard(ctypes.Structure):
    _fields_ = [("master", _c_p), ("exp_avg", _c_p), ("exp_avg_sq", _c_p), ("grad_shard", _c_p),
                ("bf16_shard_out", _c_p), ("n", _c_i64)]


class RmsNormArgs(ctypes.Structure):
    _fields_ = [("rows", _c_i64), ("cols", _c_i64), ("x_stride", _c_i64), ("residual_stride", _c_i64),
                ("h_stride", _c_i64), ("y_stride", _c_i64), ("dtype", _c_i32), ("gain_dtype", _c_i32),
                ("y_dtype", _c_i32), ("group", _c_i32), ("eps", _c_dbl)]


class RmsNormBackwardArgs(ctypes.Structure):
    _fields_ = [("rows", _c_i64), ("cols", _c_i64), ("dy_stride", _c_i64), ("h_stride", _c_i64),
                ("dh_stride", _c_i64), ("dx_stride", _c_i64), ("dtype", _c_i32), ("gain_dtype", _c_i32)]


class NewtonSchulz(ctypes.Structure):
    """Parameters of the orthogonalisation. `coefficients`: one (a, b, c) for every step, a list
    of `steps` of them, or None for the default quintic; `terms`: 0, 1 or 3 (see include/fsdp.h)."""
    _fields_ = [("steps", _c_i32), ("terms", _c_i32), ("coefficients", ctypes.POINTER(_c_dbl)), ("eps", _c_dbl)]

    def __init__(self, steps=5, coefficients=None, eps=1e-7, terms=0):
        super().__init__(steps, terms, None, eps)
        if coefficients is not None:
            per_step = [coefficients] * steps if not hasattr(coefficients[0], "__len__") else list(coefficients)
            if len(per_step) != steps or any(len(abc) != 3 for abc in per_step):
                raise ValueError("expected (a, b, c), or one (a, b, c) for each of %d steps" % steps)
            self._values = (_c_dbl * max(1, 3 * steps))(*[v for abc in per_step for v in abc])
            self.coefficients = ctypes.cast(self._values, ctypes.POINTER(_c_dbl))


class MatrixArgs(ctypes.Structure):
    _fields_ = [("source", _c_p), ("out", _c_p), ("rows", _c_i64), ("cols", _c_i64), ("source_stride", _c_i64),
                ("out_stride", _c_i64), ("dtype", _c_i32)]


class MuonTensor(ctypes.Structure):
    """One tensor of a unit: a matrix (rows, cols) whose update is scaled by `scale`, or, with
    cols = 0, a tensor of `rows` elements that Adam updates."""
    _fields_ = [("rows", _c_i64), ("cols", _c_i64), ("scale", _c_dbl)]

    def __init__(self, rows=0, cols=0, scale=1.0):
        super().__init__(rows, cols, scale)


class Muon(ctypes.Structure):
    """Hyper-parameters of the Muon step; `adam` (an AdamHyper, with its own lr and step) serves
    the tensors that are not matrices."""
    _fields_ = [("lr", _c_dbl), ("momentum", _c_dbl), ("weight_decay", _c_dbl), ("nesterov", _c_i32),
                ("newton_schulz", ctypes.POINTER(NewtonSchulz)), ("adam", AdamHyper)]

    def __init__(self, lr=1e-3, momentum=0.95, weight_decay=0.0, nesterov=True, newton_schulz=None, adam=None):
        super().__init__(lr, momentum, weight_decay, 1 if nesterov else 0, None, adam or AdamHyper())
        if newton_schulz is not None:
            self._newton_schulz = newton_schulz
            self.newton_schulz = ctypes.pointer(newton_schulz)


class MuonUnitArgs(ctypes.Structure):
    _fields_ = [("layout", ctypes.POINTER(Layout)), ("tensors", ctypes.POINTER(MuonTensor)), ("grads", _c_p),
                ("master", _c_p), ("exp_avg", _c_p), ("exp_avg_sq", _c_p), ("full_out", _c_p)]


class ZeroAccount(ctypes.Structure):
    _fields_ = [(n, _c_dbl) for n in ("weights_bytes", "grads_bytes", "optimizer_bytes", "total_bytes",
                                      "reduction_vs_ddp", "comm_elems")]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class Account(ctypes.Structure):
    _fields_ = [(n, _c_dbl) for n in (
        "persistent_bytes", "ddp_persistent_bytes", "transient_bytes", "peak_bytes", "comm_elems",
        "comm_elems_ring", "ddp_comm_elems", "ddp_comm_elems_ring", "comm_bytes", "ddp_comm_bytes")]

    def as_dict(self):
        return {n: getattr(self, n) for n, _ in self._fields_}


class FsdpError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__("%s: %s (status %d)" % (fn, fsdp_status_string(status), status))
        self.status = status


def library_path() -> str:
    """The in-tree library, or the file named by FSDP_GB300_LIB (an alternative build)."""
    return os.environ.get("FSDP_GB300_LIB") or _build_mod.SO


def _load():
    so = library_path()
    if not os.path.exists(so):
        raise ImportError("fully_sharded_gb300: CUDA library %s is not built; run "
                          "`python fully_sharded_gb300/build.py` (needs nvcc)" % so)
    lib = ctypes.CDLL(so)
    P = _c_p
    sigs = {
        "fsdp_flatten_layout": [P, _c_i32, _c_i32, _c_i32, P, ctypes.POINTER(Layout)],
        "fsdp_pack_flat": [P, ctypes.POINTER(Layout), P, _c_i32, P, P],
        "fsdp_unpack_flat": [P, ctypes.POINTER(Layout), P, _c_i32, P, P],
        "fsdp_reduce_scatter": [P, ctypes.POINTER(Layout), _c_i32, P, P],
        "fsdp_adam_shard_step": [P, P, P, P, _c_i64, ctypes.POINTER(AdamHyper), P, P],
        "fsdp_reduce_scatter_ranks": [P, ctypes.POINTER(Layout), _c_i32, _c_i32, P, P],
        "fsdp_adam_shard_step_grouped": [ctypes.POINTER(AdamShard), _c_i32, ctypes.POINTER(AdamHyper), P],
        "fsdp_all_gather": [P, ctypes.POINTER(Layout), P, P],
        "fsdp_shard_step": [P, ctypes.POINTER(Layout), _c_i32, _c_i32, P, P, P, P, P,
                            ctypes.POINTER(AdamHyper), P],
        "fsdp_shard_step_grouped": [ctypes.POINTER(UnitArgs), _c_i32, _c_i32, _c_i32,
                                    ctypes.POINTER(AdamHyper), P],
        "fsdp_shard_step_grouped_launches": [ctypes.POINTER(UnitArgs), _c_i32, _c_i32, _c_i32,
                                             ctypes.POINTER(_c_i32)],
        "fsdp_account": [_c_dbl, _c_dbl, _c_i32, _c_i32, _c_i32, ctypes.POINTER(Account)],
        "fsdp_pipeline_step": [ctypes.POINTER(PipelineUnit), _c_i32, _c_i32, P, _c_i64, _c_i32,
                               ctypes.POINTER(AdamHyper), P, P],
        "fsdp_pipeline_step_noalloc": [ctypes.POINTER(PipelineUnit), _c_i32, _c_i32, _c_i32,
                                       ctypes.POINTER(AdamHyper), P, P],
        "fsdp_all_gather_state": [P, ctypes.POINTER(Layout), _c_i32, P, P],
        "fsdp_zero1_step": [P, ctypes.POINTER(Layout), _c_i32, P, P, P, P, P, P, ctypes.POINTER(AdamHyper), P],
        "fsdp_account_zero": [_c_dbl, _c_i32, _c_i32, ctypes.POINTER(ZeroAccount)],
        "fsdp_shard_step_grouped_plan": [ctypes.POINTER(UnitArgs), _c_i32, _c_i32, _c_i32,
                                         ctypes.POINTER(_c_i32), ctypes.POINTER(_c_i32),
                                         ctypes.POINTER(_c_i32)],
        "fsdp_device_status": [_c_i32, ctypes.POINTER(ctypes.c_uint32)],
        "fsdp_selftest_wait_timeout": [P, P, _c_i64, _c_i64, P, ctypes.POINTER(ctypes.c_uint32)],
        "fsdp_offload_step": [ctypes.POINTER(OffloadUnit), _c_i32, _c_i32, P, _c_i64, _c_i32,
                              ctypes.POINTER(AdamHyper), P, P, P],
        "fsdp_rmsnorm": [ctypes.POINTER(RmsNormArgs), P, P, P, P, P, P, P, P],
        "fsdp_rmsnorm_backward": [ctypes.POINTER(RmsNormBackwardArgs), P, P, P, P, P, P, P, P, _c_i64, P],
        "fsdp_rmsnorm_backward_workspace": [_c_i64, _c_i64, ctypes.POINTER(_c_i64)],
        "fsdp_newton_schulz": [ctypes.POINTER(MatrixArgs), _c_i32, ctypes.POINTER(NewtonSchulz), P, _c_i64, P],
        "fsdp_newton_schulz_workspace": [ctypes.POINTER(MatrixArgs), _c_i32, ctypes.POINTER(NewtonSchulz),
                                         ctypes.POINTER(_c_i64)],
        "fsdp_muon_step": [ctypes.POINTER(MuonUnitArgs), ctypes.POINTER(Muon), P, _c_i64, P],
        "fsdp_muon_workspace": [ctypes.POINTER(MuonUnitArgs), ctypes.POINTER(Muon), ctypes.POINTER(_c_i64)],
    }
    for name, args in sigs.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int
    lib.fsdp_status_string.argtypes = [ctypes.c_int]
    lib.fsdp_status_string.restype = ctypes.c_char_p
    return lib


_lib = _load()


# ------------------------------------------------------------- marshalling

def _dptr(x, itemsize: int | None = None) -> int | None:
    """Device address of a contiguous CUDA tensor (or an int address, or None)."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    if not x.is_cuda:
        raise ValueError("expected a CUDA tensor, got one on %s" % x.device)
    if not x.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    if itemsize is not None and x.element_size() != itemsize:
        raise ValueError("expected %d-byte elements, got %s" % (itemsize, x.dtype))
    return x.data_ptr()


def _parray(xs, itemsize=None):
    if xs is None:
        return None
    arr = (_c_p * max(1, len(xs)))()
    for i, x in enumerate(xs):
        arr[i] = _dptr(x, itemsize)
    return arr


def _stream(stream) -> int | None:
    if stream is None:
        import torch
        return torch.cuda.current_stream().cuda_stream if torch.cuda.is_available() else None
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _check(fn: str, status: int):
    if status != FSDP_OK:
        raise FsdpError(fn, status)


def fsdp_status_string(status: int) -> str:
    return _lib.fsdp_status_string(status).decode()


# -------------------------------------------------------------- the calls

def fsdp_flatten_layout(numels: Sequence[int], world_size: int, shard_factor: int | None = None):
    """a1: returns (Layout, offsets list of n+1 ints)."""
    n = len(numels)
    nums = (_c_i64 * max(1, n))(*numels)
    offs = (_c_i64 * (n + 1))()
    lay = Layout()
    F = world_size if shard_factor is None else shard_factor
    _check("fsdp_flatten_layout",
           _lib.fsdp_flatten_layout(nums, n, world_size, F, offs, ctypes.byref(lay)))
    return lay, list(offs)


def _offsets(offsets):
    return (_c_i64 * len(offsets))(*offsets)


def _dtype_of(t) -> int:
    size = t.element_size()
    return FSDP_DTYPE_F32 if size == 4 else FSDP_DTYPE_BF16


def fsdp_pack_flat(tensors, layout: Layout, offsets, flat_out, stream=None):
    """a2: flat_out[offsets[i]:offsets[i+1]] = tensors[i]; pad zeroed."""
    es = flat_out.element_size()
    _check("fsdp_pack_flat", _lib.fsdp_pack_flat(_parray(tensors, es), ctypes.byref(layout),
                                                 _offsets(offsets), _dtype_of(flat_out),
                                                 _dptr(flat_out), _stream(stream)))


def fsdp_unpack_flat(flat, layout: Layout, offsets, tensors_out, stream=None):
    es = flat.element_size()
    _check("fsdp_unpack_flat", _lib.fsdp_unpack_flat(_dptr(flat), ctypes.byref(layout),
                                                     _offsets(offsets), _dtype_of(flat),
                                                     _parray(tensors_out, es), _stream(stream)))


def fsdp_reduce_scatter(grads, layout: Layout, rank: int, grad_shard_out, stream=None):
    """a3: grad_shard_out (fp32 [S]) = fixed-order fp32 mean of the W bf16 rows at rank's slice."""
    _check("fsdp_reduce_scatter", _lib.fsdp_reduce_scatter(
        _parray(grads, 2), ctypes.byref(layout), rank, _dptr(grad_shard_out, 4), _stream(stream)))


def fsdp_adam_shard_step(master, exp_avg, exp_avg_sq, grad_shard, adam: AdamHyper,
                         bf16_shard_out=None, stream=None, n: int | None = None):
    """a4+a5: Adam in place on the fp32 shard; optional bf16 cast out."""
    if n is None:
        n = master.numel()
    _check("fsdp_adam_shard_step", _lib.fsdp_adam_shard_step(
        _dptr(master, 4), _dptr(exp_avg, 4), _dptr(exp_avg_sq, 4), _dptr(grad_shard, 4), n,
        ctypes.byref(adam), _dptr(bf16_shard_out, 2), _stream(stream)))


def fsdp_reduce_scatter_ranks(grads, layout: Layout, rank_begin: int, rank_end: int, grad_shards_out,
                              stream=None):
    """a3 for ranks [rank_begin, rank_end) in one launch: grad_shards_out[r - rank_begin] (fp32 [S])
    receives rank r's reduce-scatter."""
    _check("fsdp_reduce_scatter_ranks", _lib.fsdp_reduce_scatter_ranks(
        _parray(grads, 2), ctypes.byref(layout), rank_begin, rank_end, _parray(grad_shards_out, 4),
        _stream(stream)))


class AdamShardBatch:
    """Marshalled shards for fsdp_adam_shard_step_grouped."""

    def __init__(self, shards):
        self.n = len(shards)
        self.array = (AdamShard * max(1, self.n))()
        for i, s in enumerate(shards):
            a = self.array[i]
            a.master = _dptr(s["master"], 4)
            a.exp_avg = _dptr(s["exp_avg"], 4)
            a.exp_avg_sq = _dptr(s["exp_avg_sq"], 4)
            a.grad_shard = _dptr(s["grad_shard"], 4)
            a.bf16_shard_out = _dptr(s.get("bf16_shard_out"), 2)
            a.n = s["n"] if "n" in s else s["master"].numel()


def fsdp_adam_shard_step_grouped(shards, adam: AdamHyper, stream=None):
    """a4+a5 over several shards in one launch. `shards`: dicts (master, exp_avg, exp_avg_sq,
    grad_shard, optional bf16_shard_out and n) or a prepared AdamShardBatch."""
    batch = shards if isinstance(shards, AdamShardBatch) else AdamShardBatch(shards)
    _check("fsdp_adam_shard_step_grouped", _lib.fsdp_adam_shard_step_grouped(
        batch.array, batch.n, ctypes.byref(adam), _stream(stream)))


def fsdp_all_gather(shards, layout: Layout, full_out, stream=None):
    """a6: full_out[k*S:(k+1)*S] = shards[k]."""
    _check("fsdp_all_gather", _lib.fsdp_all_gather(_parray(shards, 2), ctypes.byref(layout),
                                                   _dptr(full_out, 2), _stream(stream)))


def fsdp_shard_step(grads, layout: Layout, rank_begin: int, rank_end: int, master, exp_avg,
                    exp_avg_sq, other_shards, full_out, adam: AdamHyper, stream=None):
    """a7/a8: fused reduce-scatter -> Adam -> bf16 -> all-gather for ranks [rank_begin, rank_end)."""
    _check("fsdp_shard_step", _lib.fsdp_shard_step(
        _parray(grads, 2), ctypes.byref(layout), rank_begin, rank_end, _parray(master, 4),
        _parray(exp_avg, 4), _parray(exp_avg_sq, 4), _parray(other_shards, 2),
        _parray(full_out, 2), ctypes.byref(adam), _stream(stream)))


class UnitBatch:
    """Marshalled arguments of several units for fsdp_shard_step_grouped (kept alive together)."""

    def __init__(self, units):
        self._keep = []
        self.array = (UnitArgs * max(1, len(units)))()
        self.n = len(units)
        for i, u in enumerate(units):
            lay = u["layout"]
            arrs = dict(grads=_parray(u["grads"], 2), master=_parray(u["master"], 4),
                        exp_avg=_parray(u["exp_avg"], 4), exp_avg_sq=_parray(u["exp_avg_sq"], 4),
                        other_shards=_parray(u.get("other_shards"), 2),
                        full_out=_parray(u["full_out"], 2))
            self._keep.append((lay, arrs))
            a = self.array[i]
            a.layout = ctypes.pointer(lay)
            for k, v in arrs.items():
                setattr(a, k, ctypes.cast(v, _c_p) if v is not None else None)


def fsdp_shard_step_grouped(units, rank_begin: int, rank_end: int, adam: AdamHyper, stream=None):
    """a7 over several units in one launch. `units`: list of dicts (layout, grads, master,
    exp_avg, exp_avg_sq, other_shards, full_out) or a prepared UnitBatch."""
    batch = units if isinstance(units, UnitBatch) else UnitBatch(units)
    _check("fsdp_shard_step_grouped", _lib.fsdp_shard_step_grouped(
        batch.array, batch.n, rank_begin, rank_end, ctypes.byref(adam), _stream(stream)))


def fsdp_shard_step_grouped_launches(units, rank_begin: int, rank_end: int) -> int:
    """Host only: how many kernel launches fsdp_shard_step_grouped makes for these units."""
    batch = units if isinstance(units, UnitBatch) else UnitBatch(units)
    n = _c_i32(0)
    _check("fsdp_shard_step_grouped_launches", _lib.fsdp_shard_step_grouped_launches(
        batch.array, batch.n, rank_begin, rank_end, ctypes.byref(n)))
    return n.value


def _addr(x) -> int | None:
    """Address of a tensor in device or (pinned) host memory, or an int address."""
    if x is None or isinstance(x, int):
        return x
    if not x.is_contiguous():
        raise ValueError("expected a contiguous tensor")
    return x.data_ptr()


class PipelineBatch:
    """Marshalled units for fsdp_pipeline_step (kept alive together)."""

    def __init__(self, units):
        self._keep = []
        self.array = (PipelineUnit * max(1, len(units)))()
        self.n = len(units)
        for i, u in enumerate(units):
            lay = u["layout"]
            oth = _parray(u["other_shards"], 2)
            self._keep.append((lay, oth))
            a = self.array[i]
            a.layout = ctypes.pointer(lay)
            a.grad_slices = _addr(u["grad_slices"])
            a.master = _dptr(u["master"], 4)
            a.exp_avg = _dptr(u["exp_avg"], 4)
            a.exp_avg_sq = _dptr(u["exp_avg_sq"], 4)
            a.other_shards = ctypes.cast(oth, _c_p)
            a.full_out = _dptr(u["full_out"], 2)
            a.shard_out = _addr(u.get("shard_out"))


def fsdp_pipeline_step(units, rank: int, staging, slot_numel: int, n_slots: int, adam: AdamHyper,
                       compute=None, copy=None):
    """Pipelined step of one rank over many units (prefetch = n_slots - 1). `units`: list of
    dicts (layout, grad_slices, master, exp_avg, exp_avg_sq, other_shards, full_out,
    shard_out) or a PipelineBatch; `staging`: device bf16 buffer of n_slots * slot_numel."""
    batch = units if isinstance(units, PipelineBatch) else PipelineBatch(units)
    _check("fsdp_pipeline_step", _lib.fsdp_pipeline_step(
        batch.array, batch.n, rank, _dptr(staging, 2), slot_numel, n_slots, ctypes.byref(adam),
        _stream(compute), _stream(copy)))


class OffloadBatch:
    """Marshalled units for fsdp_offload_step (kept alive together)."""

    def __init__(self, units):
        self._keep = []
        self.array = (OffloadUnit * max(1, len(units)))()
        self.n = len(units)
        for i, u in enumerate(units):
            lay = u["layout"]
            g = _parray(u["grads"], 2)
            oth = _parray(u["other_shards"], 2)
            self._keep.append((lay, g, oth))
            a = self.array[i]
            a.layout = ctypes.pointer(lay)
            a.grads = ctypes.cast(g, _c_p)
            for name in ("master", "exp_avg", "exp_avg_sq"):
                x = u[name]
                if x is not None and not isinstance(x, int) and x.element_size() != 4:
                    raise ValueError("%s: expected fp32, got %s" % (name, x.dtype))
                setattr(a, name, _addr(x))
            a.other_shards = ctypes.cast(oth, _c_p)
            a.full_out = _dptr(u["full_out"], 2)


def fsdp_offload_step(units, rank: int, staging, slot_numel: int, n_slots: int, adam: AdamHyper,
                      compute=None, h2d=None, d2h=None):
    """Staged optimizer-state offload over many units: `units` are dicts (layout, grads,
    master, exp_avg, exp_avg_sq, other_shards, full_out) with master/exp_avg/exp_avg_sq in
    (pinned) host memory, or an OffloadBatch; `staging`: device fp32 buffer of
    n_slots * 3 * slot_numel."""
    batch = units if isinstance(units, OffloadBatch) else OffloadBatch(units)
    _check("fsdp_offload_step", _lib.fsdp_offload_step(
        batch.array, batch.n, rank, _dptr(staging, 4), slot_numel, n_slots, ctypes.byref(adam),
        _stream(compute), _stream(h2d), _stream(d2h)))


def fsdp_pipeline_step_noalloc(units, rank: int, n_slots: int, adam: AdamHyper, compute=None,
                               copy=None):
    """fsdp_pipeline_step without a staging argument, for callers that cannot allocate
    device memory when they step: the pool is a fixed array of NOALLOC_STAGING_BYTES
    inside the library (FsdpError with status FSDP_ENOSPACE if n_slots times the largest
    unit, rounded up to 8 elements, does not fit). Calls on one device share that array,
    so their GPU work must not overlap."""
    batch = units if isinstance(units, PipelineBatch) else PipelineBatch(units)
    _check("fsdp_pipeline_step_noalloc", _lib.fsdp_pipeline_step_noalloc(
        batch.array, batch.n, rank, n_slots, ctypes.byref(adam), _stream(compute), _stream(copy)))


def fsdp_all_gather_state(shards, layout: Layout, full_out, stream=None):
    """Gather per-rank state (fp32 master/m/v, or bf16) into the full flat buffer of a group."""
    es = full_out.element_size()
    _check("fsdp_all_gather_state", _lib.fsdp_all_gather_state(
        _parray(shards, es), ctypes.byref(layout), _dtype_of(full_out), _dptr(full_out), _stream(stream)))


def fsdp_zero1_step(grads, layout: Layout, rank: int, avg_grad_out, master, exp_avg, exp_avg_sq, other_shards,
                    full_out, adam: AdamHyper, stream=None):
    """ZeRO stage 1 step of one rank: full all-reduce average into avg_grad_out, Adam on the
    rank's slice, bf16 shard and gather into full_out."""
    _check("fsdp_zero1_step", _lib.fsdp_zero1_step(
        _parray(grads, 2), ctypes.byref(layout), rank, _dptr(avg_grad_out, 4), _dptr(master, 4),
        _dptr(exp_avg, 4), _dptr(exp_avg_sq, 4), _parray(other_shards, 2), _dptr(full_out, 2),
        ctypes.byref(adam), _stream(stream)))


def fsdp_account_zero(P: float, N: int, stage: int) -> dict:
    """Per-GPU bytes of ZeRO stage 0 (DDP) .. 3 (FSDP) and the communication per step (host only)."""
    out = ZeroAccount()
    _check("fsdp_account_zero", _lib.fsdp_account_zero(float(P), N, stage, ctypes.byref(out)))
    return out.as_dict()


def fsdp_shard_step_grouped_plan(units, rank_begin: int, rank_end: int, interleaved: bool = False):
    """Host only: (launches, launches in the TMA form) of fsdp_shard_step_grouped for these
    units; with interleaved=True also the number of TMA launches that stage their step
    chunks in interleaved quarter-chunk copies."""
    batch = units if isinstance(units, UnitBatch) else UnitBatch(units)
    n, t, i = _c_i32(0), _c_i32(0), _c_i32(0)
    _check("fsdp_shard_step_grouped_plan", _lib.fsdp_shard_step_grouped_plan(
        batch.array, batch.n, rank_begin, rank_end, ctypes.byref(n), ctypes.byref(t), ctypes.byref(i)))
    return (n.value, t.value, i.value) if interleaved else (n.value, t.value)


def fsdp_device_status(clear: bool = False) -> int:
    """The current device's sticky status word (bit 0: a bounded wait of the TMA form ran out)."""
    v = ctypes.c_uint32(0)
    _check("fsdp_device_status", _lib.fsdp_device_status(1 if clear else 0, ctypes.byref(v)))
    return v.value


def fsdp_selftest_wait_timeout(src, dst, wait_limit_ns: int, stream=None) -> int:
    """Diagnostic call of include/fsdp_test.h (not part of the method's interface):
    provokes one bounded-wait timeout on a copy of src into dst; returns the status word seen."""
    v = ctypes.c_uint32(0)
    nbytes = src.numel() * src.element_size()
    _check("fsdp_selftest_wait_timeout", _lib.fsdp_selftest_wait_timeout(
        _dptr(src), _dptr(dst), nbytes, int(wait_limit_ns), _stream(stream), ctypes.byref(v)))
    return v.value


def fsdp_account(P: float, U: float, N: int, F: int | None = None, prefetch: int = 1) -> dict:
    """a9: closed-form memory and communication budget (host only)."""
    out = Account()
    _check("fsdp_account", _lib.fsdp_account(float(P), float(U), N, N if F is None else F,
                                             prefetch, ctypes.byref(out)))
    return out.as_dict()


# ------------------------------------------- operators of the training loop

def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


_torch_module = None


def _cuda_stream(stream, device: int | None = None):
    """The stream's handle; None: the current stream (of `device`, or of the current one)."""
    if stream is None:
        torch = _torch()
        raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)  # 2.8 us less than the Stream object
        if raw is not None:
            return raw(torch.cuda.current_device() if device is None else device)
        return torch.cuda.current_stream().cuda_stream
    return stream if isinstance(stream, int) else stream.cuda_stream


def _float_dtype(t, what: str) -> int:
    torch = _torch()
    dtype = t.dtype
    if dtype is torch.bfloat16:
        return FSDP_DTYPE_BF16
    if dtype is torch.float32:
        return FSDP_DTYPE_F32
    raise ValueError("%s: expected float32 or bfloat16, got %s" % (what, dtype))


def _device(t, what: str) -> int:
    if not t.is_cuda:
        raise ValueError("%s: expected a CUDA tensor, got one on %s" % (what, t.device))
    return t.get_device()


def _current_device(device: int, what: str):
    """Kernels are launched on the current device: the tensors have to lie there."""
    current = _torch().cuda.current_device()
    if device != current:
        raise ValueError("%s: on cuda:%d, but the current device is cuda:%d" % (what, device, current))


def _elsewhere(t, what: str, device: int) -> ValueError:
    return ValueError("%s: expected a CUDA tensor on cuda:%d, got one on %s" % (what, device, t.device))


def _matrix(t, what: str, shape, device: int, dtype=None):
    """(address, row stride) of a matrix of the given shape on `device` whose rows are contiguous."""
    if t.get_device() != device:  # -1: not a CUDA tensor
        raise _elsewhere(t, what, device)
    if t.shape != shape:
        raise ValueError("%s: expected shape %s, got %s" % (what, tuple(shape), tuple(t.shape)))
    if dtype is not None and t.dtype is not dtype:
        raise ValueError("%s: expected %s, got %s" % (what, dtype, t.dtype))
    rows, cols = shape
    row, col = t.stride()
    if col != 1 and cols > 1:
        raise ValueError("%s: expected contiguous rows" % what)
    return t.data_ptr(), (row if rows > 1 else cols)


def _vector(t, what: str, n: int, device: int, dtype=None):
    if t.get_device() != device:
        raise _elsewhere(t, what, device)
    if not t.is_contiguous() or t.numel() != n:
        raise ValueError("%s: expected a contiguous CUDA tensor of %d elements" % (what, n))
    if dtype is not None and t.dtype != dtype:
        raise ValueError("%s: expected %s, got %s" % (what, dtype, t.dtype))
    return t.data_ptr()


def _workspace(t, device: int | None):
    if t is None:
        return None, 0
    if device is not None and t.get_device() != device:
        raise _elsewhere(t, "workspace", device)
    return _dptr(t), t.numel() * t.element_size()


def _shape2(t, what: str):
    shape = t.shape
    if len(shape) != 2:
        raise ValueError("%s: expected a matrix, got shape %s" % (what, tuple(shape)))
    return shape


def fsdp_rmsnorm(x, gain, y, residual=None, h_out=None, scales=None, rstd=None, group: int = 0, eps: float = 1e-6,
                 stream=None):
    """RMS norm of the rows of x (+ residual, the sum written to h_out) into y: y's type is x's,
    or 8 bits (torch.float8_e4m3fn) with fp32 `scales` [rows, groups], one per `group` elements
    (0: per row). rstd (fp32 [rows], optional) is what the backward pass needs."""
    torch = _torch()
    shape = _shape2(x, "x")
    rows, cols = shape
    dtype, y_dtype = x.dtype, y.dtype
    code = _float_dtype(x, "x")
    device = _device(x, "x")
    _current_device(device, "x")
    xp, x_stride = _matrix(x, "x", shape, device)
    rp = hp = sp = None
    r_stride = h_stride = cols
    if residual is not None:
        rp, r_stride = _matrix(residual, "residual", shape, device, dtype)
    if h_out is not None:
        hp, h_stride = _matrix(h_out, "h_out", shape, device, dtype)
    y_code = code
    if y_dtype == torch.float8_e4m3fn:
        y_code = FSDP_DTYPE_E4M3
        if scales is None:
            raise ValueError("scales: needed for an 8-bit y")
        sp = _vector(scales, "scales", rows * (-(-cols // group) if group > 0 else 1), device, torch.float32)
    else:
        if y_dtype != dtype:
            raise ValueError("y: expected %s or torch.float8_e4m3fn, got %s" % (dtype, y_dtype))
        if scales is not None:
            raise ValueError("scales: only for an 8-bit y")
    yp, y_stride = _matrix(y, "y", shape, device)
    dp = _vector(rstd, "rstd", rows, device, torch.float32) if rstd is not None else None
    a = RmsNormArgs(rows, cols, x_stride, r_stride, h_stride, y_stride, code, _float_dtype(gain, "gain"), y_code, group,
                    eps)
    _check("fsdp_rmsnorm", _lib.fsdp_rmsnorm(ctypes.byref(a), xp, rp, _vector(gain, "gain", cols, device), hp, yp, sp, dp,
                                             _cuda_stream(stream, device)))


def fsdp_rmsnorm_backward_workspace(rows: int, cols: int) -> int:
    """Bytes of workspace that fsdp_rmsnorm_backward needs (host only)."""
    n = _c_i64(0)
    _check("fsdp_rmsnorm_backward_workspace", _lib.fsdp_rmsnorm_backward_workspace(rows, cols, ctypes.byref(n)))
    return n.value


def fsdp_rmsnorm_backward(dy, h, gain, rstd, dx, dgain, workspace, dh=None, stream=None):
    """Gradients of fsdp_rmsnorm: dx (of x, and of the residual) from dy, the forward's h and rstd,
    and dh, the gradient that reaches h by the residual path; dgain in gain's type, summed over the rows
    (it may be a view into a rank's gradient row)."""
    shape = _shape2(h, "h")
    rows, cols = shape
    dtype = h.dtype
    device = _device(h, "h")
    _current_device(device, "h")
    hp, h_stride = _matrix(h, "h", shape, device)
    yp, dy_stride = _matrix(dy, "dy", shape, device, dtype)
    xp, dx_stride = _matrix(dx, "dx", shape, device, dtype)
    dhp, dh_stride = _matrix(dh, "dh", shape, device, dtype) if dh is not None else (None, cols)
    a = RmsNormBackwardArgs(rows, cols, dy_stride, h_stride, dh_stride, dx_stride, _float_dtype(h, "h"),
                            _float_dtype(gain, "gain"))
    ws, ws_bytes = _workspace(workspace, device)
    _check("fsdp_rmsnorm_backward", _lib.fsdp_rmsnorm_backward(
        ctypes.byref(a), yp, hp, _vector(gain, "gain", cols, device), _vector(rstd, "rstd", rows, device, _torch().float32),
        dhp, xp, _vector(dgain, "dgain", cols, device, gain.dtype), ws, ws_bytes, _cuda_stream(stream, device)))


class NewtonSchulzBatch:
    """Marshalled matrices for fsdp_newton_schulz: `sources` (float32 or bfloat16) and their bf16
    results `outs`, kept alive together."""

    def __init__(self, sources, outs):
        if len(sources) != len(outs):
            raise ValueError("expected one out for each of %d sources, got %d" % (len(sources), len(outs)))
        self._keep = (list(sources), list(outs))
        self.n = len(sources)
        self.array = (MatrixArgs * max(1, self.n))()
        self.device = _device(sources[0], "source") if self.n else None
        for a, source, out in zip(self.array, sources, outs):
            shape = _shape2(source, "source")
            a.rows, a.cols = shape
            a.dtype = _float_dtype(source, "source")
            a.source, a.source_stride = _matrix(source, "source", shape, self.device)
            a.out, a.out_stride = _matrix(out, "out", shape, self.device, _torch().bfloat16)


def _byref_or_none(x):
    return ctypes.byref(x) if x is not None else None


def fsdp_newton_schulz_workspace(batch: NewtonSchulzBatch, newton_schulz: NewtonSchulz | None = None) -> int:
    """Bytes of workspace that fsdp_newton_schulz needs for these matrices (host only)."""
    n = _c_i64(0)
    _check("fsdp_newton_schulz_workspace", _lib.fsdp_newton_schulz_workspace(
        batch.array, batch.n, _byref_or_none(newton_schulz), ctypes.byref(n)))
    return n.value


def fsdp_newton_schulz(batch: NewtonSchulzBatch, workspace, newton_schulz: NewtonSchulz | None = None, stream=None):
    """Orthogonalises every matrix of the batch into its out by Newton-Schulz products."""
    if batch.device is not None:
        _current_device(batch.device, "batch")
    ws, ws_bytes = _workspace(workspace, batch.device)
    _check("fsdp_newton_schulz", _lib.fsdp_newton_schulz(batch.array, batch.n, _byref_or_none(newton_schulz), ws,
                                                         ws_bytes, _cuda_stream(stream)))


class MuonUnit:
    """Marshalled arguments of one unit for fsdp_muon_step: its tensors in flat order
    (MuonTensor each), the W bf16 gradient rows, the W fp32 shards of the state, the
    gathered bf16 parameters. Kept alive together."""

    def __init__(self, layout: Layout, tensors, grads, master, exp_avg, exp_avg_sq, full_out):
        if len(tensors) != layout.n_tensors:
            raise ValueError("expected %d tensors, got %d" % (layout.n_tensors, len(tensors)))
        world, padded, shard = layout.world_size, layout.padded_numel, layout.shard_numel
        for what, xs, n in (("grads", grads, padded), ("master", master, shard), ("exp_avg", exp_avg, shard),
                            ("exp_avg_sq", exp_avg_sq, shard), ("full_out", [full_out] * world, padded)):
            if len(xs) != world:
                raise ValueError("%s: expected one per rank (%d), got %d" % (what, world, len(xs)))
            for x in xs:
                if x is not None and not isinstance(x, int) and x.numel() != n:
                    raise ValueError("%s: expected %d elements, got %d" % (what, n, x.numel()))
        self.device = None  # of the tensors among the arguments (addresses have none)
        for what, xs in (("grads", grads), ("master", master), ("exp_avg", exp_avg), ("exp_avg_sq", exp_avg_sq),
                         ("full_out", [full_out])):
            for x in xs:
                if x is None or isinstance(x, int):
                    continue
                if self.device is None:
                    self.device = _device(x, what)
                if x.get_device() != self.device:
                    raise _elsewhere(x, what, self.device)
        self._tensors = (MuonTensor * max(1, len(tensors)))(*tensors)
        arrays = dict(grads=_parray(grads, 2), master=_parray(master, 4), exp_avg=_parray(exp_avg, 4),
                      exp_avg_sq=_parray(exp_avg_sq, 4))
        self._keep = (layout, list(grads), list(master), list(exp_avg), list(exp_avg_sq), full_out, arrays)
        self.args = MuonUnitArgs(layout=ctypes.pointer(layout),
                                 tensors=ctypes.cast(self._tensors, ctypes.POINTER(MuonTensor)),
                                 full_out=_dptr(full_out, 2))
        for k, v in arrays.items():
            setattr(self.args, k, ctypes.cast(v, _c_p))


def fsdp_muon_workspace(unit: MuonUnit, muon: Muon | None = None) -> int:
    """Bytes of workspace that fsdp_muon_step needs for this unit (host only)."""
    n = _c_i64(0)
    _check("fsdp_muon_workspace", _lib.fsdp_muon_workspace(ctypes.byref(unit.args), ctypes.byref(muon or Muon()),
                                                           ctypes.byref(n)))
    return n.value


def fsdp_muon_step(unit: MuonUnit, muon: Muon, workspace, stream=None):
    """The Muon step of one unit on all its ranks: reduce-scatter and momentum, every matrix's update
    orthogonalised and applied, the other tensors by Adam, the bf16 cast and the gather."""
    if unit.device is not None:
        _current_device(unit.device, "unit")
    ws, ws_bytes = _workspace(workspace, unit.device)
    _check("fsdp_muon_step", _lib.fsdp_muon_step(ctypes.byref(unit.args), ctypes.byref(muon), ws, ws_bytes,
                                                 _cuda_stream(stream)))
