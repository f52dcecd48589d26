"""ctypes binding of ``include/mla_split.h`` (argument marshalling only).

Every function has the name of the C entry point it calls and does nothing but
convert arguments (torch tensors -> device pointers, streams -> handles) and
turn a non-zero status into ``SplitKVError``. All computation happens in the
CUDA library; there is no fallback: if ``libsplitkv.so`` is missing the first
call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libsplitkv.so")

MLA_OK = 0
MLA_OUT_F32, MLA_OUT_BF16, MLA_OUT_E4M3 = 0, 1, 2
MLA_STATUS_TIMEOUT = 0x1
MLA_STATUS_BAD_SHAPE = 0x2
MLA_STATUS_BAD_INDEX = 0x10
MLA_STATUS_BAD_ALIGN = 0x4
MLA_MAX_SPLITS = 64
MLA_FORCE_BALANCED = -1
SDPA_BF16, SDPA_E4M3, SDPA_E2M1 = 1, 2, 4
KV_PAGES_MAX_BATCH = 16384
MLA_ERR_INVALID_ARG = 1
OUT_DTYPES = {"f32": MLA_OUT_F32, "bf16": MLA_OUT_BF16, "e4m3": MLA_OUT_E4M3}

# Every symbol the header declares (checked by the library-load test).
EXPORTS = [
    "mla_decode_plan", "mla_sparse_decode_split", "mla_split_combine", "mla_sparse_decode_direct",
    "mla_sparse_decode", "mla_sparse_decode_host", "sdpa_fp8_decode_plan", "sdpa_fp8_decode_split",
    "sdpa_split_combine", "sdpa_fp8_decode_direct", "sdpa_fp8_decode", "mla_get_status",
    "mla_selftest_wait_timeout", "mla_status_string", "mla_abi_version", "mla_sparse_decode_noalloc",
    "mla_workspace_init", "mla_set_wait_limit_ns", "mla_plan_set_partials_bf16", "mla_set_index_checks",
    "kv_pages_map", "kv_pages_write", "sdpa_paged_plan", "sdpa_paged", "sdpa_prompt", "kv_pages_write_rotary",
    "kv_pages_read",
]


class SplitKVError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({status_string(status)})")


class MlaPlan(ctypes.Structure):
    _fields_ = [("s_q_max", ctypes.c_int32), ("h_q", ctypes.c_int32), ("d_qk", ctypes.c_int32),
                ("d_v", ctypes.c_int32), ("topk", ctypes.c_int32), ("block_rows", ctypes.c_int32),
                ("num_blocks", ctypes.c_int32), ("num_splits", ctypes.c_int32), ("num_sms", ctypes.c_int32),
                ("balanced_ctas", ctypes.c_int32), ("dim_groups", ctypes.c_int32),
                ("partial_bf16", ctypes.c_int32), ("tail_ctas", ctypes.c_int32), ("o_acc_bytes", ctypes.c_uint64),
                ("lse_acc_offset", ctypes.c_uint64), ("lse_acc_bytes", ctypes.c_uint64),
                ("workspace_bytes", ctypes.c_uint64)]


class SdpaPlan(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("h_q", ctypes.c_int32), ("h_kv", ctypes.c_int32),
                ("d", ctypes.c_int32), ("max_q_per_seq", ctypes.c_int32), ("total_q_max", ctypes.c_int32),
                ("max_kv", ctypes.c_int32), ("key_tile", ctypes.c_int32), ("num_splits", ctypes.c_int32),
                ("num_sms", ctypes.c_int32), ("adaptive_splits", ctypes.c_int32), ("o_acc_bytes", ctypes.c_uint64),
                ("lse_acc_offset", ctypes.c_uint64), ("lse_acc_bytes", ctypes.c_uint64),
                ("workspace_bytes", ctypes.c_uint64)]


class KvPages(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("dtype", ctypes.c_int32),
                ("num_pages", ctypes.c_int32), ("page_size", ctypes.c_int32), ("h_kv", ctypes.c_int32),
                ("d", ctypes.c_int32), ("reserved", ctypes.c_int32), ("page_stride", ctypes.c_int64),
                ("row_stride", ctypes.c_int64), ("head_stride", ctypes.c_int64), ("k_scales", ctypes.c_void_p),
                ("v_scales", ctypes.c_void_p), ("scale_page_stride", ctypes.c_int64), ("scale_head_stride", ctypes.c_int64)]


class SdpaPagedPlan(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("h_q", ctypes.c_int32), ("h_kv", ctypes.c_int32), ("d", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("max_q_per_seq", ctypes.c_int32), ("total_q_max", ctypes.c_int32),
                ("max_kv", ctypes.c_int32), ("num_splits", ctypes.c_int32), ("num_sms", ctypes.c_int32),
                ("adaptive_splits", ctypes.c_int32), ("row_kernel", ctypes.c_int32), ("o_acc_bytes", ctypes.c_uint64),
                ("lse_acc_offset", ctypes.c_uint64), ("lse_acc_bytes", ctypes.c_uint64),
                ("map_offset", ctypes.c_uint64), ("workspace_bytes", ctypes.c_uint64)]


_lib = None
_P = ctypes.c_void_p
_I = ctypes.c_int
_F = ctypes.c_float
_I64 = ctypes.c_int64
_U64 = ctypes.c_uint64

_SIGS = {
    "mla_decode_plan": [_I, _I, _I, _I, _I, _I, _I, _I, ctypes.POINTER(MlaPlan)],
    "mla_sparse_decode_split": [ctypes.POINTER(MlaPlan), _I, _P, _P, _I64, _P, _F, _P, _P],
    "mla_split_combine": [ctypes.POINTER(MlaPlan), _I, _P, _P, _I, _F, _P, _P, _P, _P],
    "mla_sparse_decode_direct": [_I, _I, _P, _P, _I64, _P, _F, _P, _I, _F, _P, _P, _P, _P],
    "mla_sparse_decode": [ctypes.POINTER(MlaPlan), _I, _P, _P, _I64, _P, _F, _P, _I, _F, _P, _P, _P, _P, _P],
    "mla_sparse_decode_host": [ctypes.POINTER(MlaPlan), _I, _P, _P, _P, _I64, _P, _P, _F, _P, _I, _F, _P, _P, _P,
                               _P, _P, _P, _P],
    "sdpa_fp8_decode_plan": [_I, _I, _I, _I, _I, _I, _I, _I, _I, _I, ctypes.POINTER(SdpaPlan)],
    "sdpa_fp8_decode_split": [ctypes.POINTER(SdpaPlan), _I, _I64, _P, _P, _P, _P, _P, _P, _P, _P, _F, _P, _P],
    "sdpa_split_combine": [ctypes.POINTER(SdpaPlan), _I, _P, _I, _F, _P, _P, _P, _P],
    "sdpa_fp8_decode_direct": [_I, _I, _I, _I, _I, _I64, _P, _P, _P, _P, _P, _P, _P, _P, _F, _I, _F, _P, _P, _P,
                               _P],
    "sdpa_fp8_decode": [ctypes.POINTER(SdpaPlan), _I, _I64, _P, _P, _P, _P, _P, _P, _P, _P, _F, _I, _F, _P, _P,
                        _P, _P, _P],
    "mla_get_status": [ctypes.POINTER(ctypes.c_uint32), ctypes.POINTER(ctypes.c_uint32)],
    "mla_selftest_wait_timeout": [_U64, _P],
    "mla_status_string": [_I],
    "mla_abi_version": [],
    "mla_sparse_decode_noalloc": [_I, _I, _P, _P, _I64, _P, _F, _P, _I, _I, _F, _P, _P, _P, _P],
    "mla_workspace_init": [ctypes.POINTER(MlaPlan), _P, _P],
    "mla_set_wait_limit_ns": [_U64],
    "mla_set_index_checks": [_I],
    "mla_plan_set_partials_bf16": [ctypes.POINTER(MlaPlan), _I],
    "kv_pages_map": [_I, _I, _P, _P, _P, _I, _P, _I, _P, _I, _P, _P, _P, _P, _P],
    "kv_pages_write": [ctypes.POINTER(KvPages), _I64, _P, _P, _I64, _I64, _P, _P, _P, _P],
    "kv_pages_write_rotary": [ctypes.POINTER(KvPages), _I64, _I, _P, _I64, _I64, _P, _P, _I64, _I64, _P, _P, _I64, _I, _I, _P,
                              _P, _P, _P, _I, _P, _I64, _I64, _P, _I64, _I64, _P],
    "kv_pages_read": [ctypes.POINTER(KvPages), _I64, _P, _P, _P, _P, _P, _I64, _I64, _P],
    "sdpa_paged_plan": [_I, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I, ctypes.POINTER(SdpaPagedPlan)],
    "sdpa_paged": [ctypes.POINTER(SdpaPagedPlan), _I, _P, _I64, _I64, ctypes.POINTER(KvPages), _P, _I, _P, _P, _P, _P,
                   _P, _F, _I, _F, _P, _P, _P, _P, _P],
    "sdpa_prompt": [_I, _I, _I, _I, _I, _I, _I64, _P, _I64, _I64, _P, _P, _I64, _I64, _P, _P, _P, _P, _P, _F, _I, _F,
                    _P, _P, _P, _P],
}


def lib() -> ctypes.CDLL:
    """Load libsplitkv.so (built in-tree by split_kv_sparse_gb300.build); raise if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is not built; run `python -m split_kv_sparse_gb300.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, args in _SIGS.items():
            fn = getattr(L, name)
            fn.argtypes = args
            fn.restype = ctypes.c_char_p if name == "mla_status_string" else ctypes.c_int
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().mla_status_string(status).decode()


def _ptr(x) -> Optional[int]:
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


def _stream(s) -> Optional[int]:
    if s is None:
        import torch
        return torch.cuda.current_stream().cuda_stream
    if isinstance(s, int):
        return s
    return s.cuda_stream


def _check(st: int, where: str):
    if st != MLA_OK:
        raise SplitKVError(st, where)


def _dtype(out_dtype) -> int:
    return OUT_DTYPES[out_dtype] if isinstance(out_dtype, str) else int(out_dtype)


# ---------------------------------------------------------------------- MLA --

def mla_decode_plan(s_q_max: int, topk: int, *, h_q: int = 64, d_qk: int = 576, d_v: int = 512,
                    num_sms: int = 0, max_splits: int = 0, force_splits: int = 0) -> MlaPlan:
    plan = MlaPlan()
    _check(lib().mla_decode_plan(s_q_max, h_q, d_qk, d_v, topk, num_sms, max_splits, force_splits,
                                 ctypes.byref(plan)), "mla_decode_plan")
    return plan


def mla_plan_set_partials_bf16(plan: MlaPlan, enable: bool = True) -> MlaPlan:
    """Switches the plan's O partials to bf16 (or back to fp32) in place; returns the plan."""
    _check(lib().mla_plan_set_partials_bf16(ctypes.byref(plan), enable if isinstance(enable, int) else int(enable)),
           "mla_plan_set_partials_bf16")
    return plan


def mla_workspace_init(plan: MlaPlan, workspace, stream=None):
    _check(lib().mla_workspace_init(ctypes.byref(plan), _ptr(workspace), _stream(stream)), "mla_workspace_init")


def mla_sparse_decode_split(plan: MlaPlan, s_q: int, q, kv, n_kv: int, idx, sm_scale: float, workspace,
                            stream=None):
    _check(lib().mla_sparse_decode_split(ctypes.byref(plan), s_q, _ptr(q), _ptr(kv), n_kv, _ptr(idx),
                                         sm_scale, _ptr(workspace), _stream(stream)),
           "mla_sparse_decode_split")


def mla_split_combine(plan: MlaPlan, s_q: int, workspace, sink, out_dtype, out_inv_scale: float, out,
                      lse_out=None, amax_out=None, stream=None):
    _check(lib().mla_split_combine(ctypes.byref(plan), s_q, _ptr(workspace), _ptr(sink), _dtype(out_dtype),
                                   out_inv_scale, _ptr(out), _ptr(lse_out), _ptr(amax_out), _stream(stream)),
           "mla_split_combine")


def mla_sparse_decode_direct(s_q: int, topk: int, q, kv, n_kv: int, idx, sm_scale: float, sink, out_dtype,
                             out_inv_scale: float, out, lse_out=None, amax_out=None, stream=None):
    _check(lib().mla_sparse_decode_direct(s_q, topk, _ptr(q), _ptr(kv), n_kv, _ptr(idx), sm_scale, _ptr(sink),
                                          _dtype(out_dtype), out_inv_scale, _ptr(out), _ptr(lse_out),
                                          _ptr(amax_out), _stream(stream)),
           "mla_sparse_decode_direct")


def mla_sparse_decode(plan: MlaPlan, s_q: int, q, kv, n_kv: int, idx, sm_scale: float, sink, out_dtype,
                      out_inv_scale: float, out, lse_out=None, amax_out=None, workspace=None, stream=None):
    _check(lib().mla_sparse_decode(ctypes.byref(plan), s_q, _ptr(q), _ptr(kv), n_kv, _ptr(idx), sm_scale,
                                   _ptr(sink), _dtype(out_dtype), out_inv_scale, _ptr(out), _ptr(lse_out),
                                   _ptr(amax_out), _ptr(workspace), _stream(stream)),
           "mla_sparse_decode")


def mla_sparse_decode_host(plan: MlaPlan, s_q: int, q_host, q_dev, kv, n_kv: int, idx_host, idx_dev,
                           sm_scale: float, sink, out_dtype, out_inv_scale: float, out_dev, out_host,
                           lse_dev=None, lse_host=None, amax_out=None, workspace=None, stream=None):
    """The decode step with q / idx / out / lse in host memory (pinned for asynchronous copies): the
    library copies them through the given device buffers around mla_sparse_decode, on `stream`."""
    _check(lib().mla_sparse_decode_host(ctypes.byref(plan), s_q, _ptr(q_host), _ptr(q_dev), _ptr(kv), n_kv,
                                        _ptr(idx_host), _ptr(idx_dev), sm_scale, _ptr(sink), _dtype(out_dtype),
                                        out_inv_scale, _ptr(out_dev), _ptr(out_host), _ptr(lse_dev),
                                        _ptr(lse_host), _ptr(amax_out), _ptr(workspace), _stream(stream)),
           "mla_sparse_decode_host")


# -------------------------------------------------------------------- dense --

def sdpa_fp8_decode_plan(batch: int, h_q: int, h_kv: int, d: int, max_q_per_seq: int, total_q_max: int,
                         max_kv: int, *, num_sms: int = 0, max_splits: int = 0, force_splits: int = 0) -> SdpaPlan:
    plan = SdpaPlan()
    _check(lib().sdpa_fp8_decode_plan(batch, h_q, h_kv, d, max_q_per_seq, total_q_max, max_kv, num_sms,
                                      max_splits, force_splits, ctypes.byref(plan)), "sdpa_fp8_decode_plan")
    return plan


def sdpa_fp8_decode_split(plan: SdpaPlan, total_q: int, total_kv: int, q, k, v, cu_seqlens_q, cu_seqlens_kv,
                          descale_q, descale_k, descale_v, sm_scale: float, workspace, stream=None):
    _check(lib().sdpa_fp8_decode_split(ctypes.byref(plan), total_q, total_kv, _ptr(q), _ptr(k), _ptr(v),
                                       _ptr(cu_seqlens_q), _ptr(cu_seqlens_kv), _ptr(descale_q), _ptr(descale_k),
                                       _ptr(descale_v), sm_scale, _ptr(workspace), _stream(stream)),
           "sdpa_fp8_decode_split")


def sdpa_split_combine(plan: SdpaPlan, total_q: int, workspace, out_dtype, out_inv_scale: float, out,
                       lse_out=None, amax_out=None, stream=None):
    _check(lib().sdpa_split_combine(ctypes.byref(plan), total_q, _ptr(workspace), _dtype(out_dtype),
                                    out_inv_scale, _ptr(out), _ptr(lse_out), _ptr(amax_out), _stream(stream)),
           "sdpa_split_combine")


def sdpa_fp8_decode_direct(batch: int, h_q: int, h_kv: int, d: int, total_q: int, total_kv: int, q, k, v,
                           cu_seqlens_q, cu_seqlens_kv, descale_q, descale_k, descale_v, sm_scale: float, out_dtype,
                           out_inv_scale: float, out, lse_out=None, amax_out=None, stream=None):
    _check(lib().sdpa_fp8_decode_direct(batch, h_q, h_kv, d, total_q, total_kv, _ptr(q), _ptr(k), _ptr(v),
                                        _ptr(cu_seqlens_q), _ptr(cu_seqlens_kv), _ptr(descale_q),
                                        _ptr(descale_k), _ptr(descale_v), sm_scale, _dtype(out_dtype),
                                        out_inv_scale, _ptr(out), _ptr(lse_out), _ptr(amax_out), _stream(stream)),
           "sdpa_fp8_decode_direct")


def sdpa_fp8_decode(plan: SdpaPlan, total_q: int, total_kv: int, q, k, v, cu_seqlens_q, cu_seqlens_kv, descale_q,
                    descale_k, descale_v, sm_scale: float, out_dtype, out_inv_scale: float, out, lse_out=None,
                    amax_out=None, workspace=None, stream=None):
    _check(lib().sdpa_fp8_decode(ctypes.byref(plan), total_q, total_kv, _ptr(q), _ptr(k), _ptr(v), _ptr(cu_seqlens_q),
                                 _ptr(cu_seqlens_kv), _ptr(descale_q), _ptr(descale_k), _ptr(descale_v), sm_scale,
                                 _dtype(out_dtype), out_inv_scale, _ptr(out), _ptr(lse_out), _ptr(amax_out),
                                 _ptr(workspace), _stream(stream)),
           "sdpa_fp8_decode")


def mla_sparse_decode_noalloc(s_q: int, topk: int, q, kv, n_kv: int, idx, sm_scale: float, sink, num_splits: int,
                              out_dtype, out_inv_scale: float, out, lse_out=None, amax_out=None, stream=None):
    """Decode step whose split workspace is the library's own scratch array (no allocation)."""
    _check(lib().mla_sparse_decode_noalloc(s_q, topk, _ptr(q), _ptr(kv), n_kv, _ptr(idx), sm_scale, _ptr(sink),
                                           num_splits, _dtype(out_dtype), out_inv_scale, _ptr(out), _ptr(lse_out),
                                           _ptr(amax_out), _stream(stream)),
           "mla_sparse_decode_noalloc")


# -------------------------------------------- paged KV cache, prompt attention --

_SDPA_DTYPES = {"bf16": SDPA_BF16, "e4m3": SDPA_E4M3, "e2m1": SDPA_E2M1}


class _Types:
    """torch's types that the calls below take, by what they are used for (made on the first call)."""

    def __init__(self):
        import torch
        self.i32, self.i64, self.f32, self.bf16 = (torch.int32,), (torch.int64,), (torch.float32,), (torch.bfloat16,)
        self.BF, self.I32, self.I64, self.F32 = torch.bfloat16, torch.int32, torch.int64, torch.float32
        self.codes = (torch.uint8, torch.float8_e4m3fn)
        self.data = self.bf16 + self.codes
        self.bytes4 = (torch.uint8,) + ((torch.float4_e2m1fn_x2,) if hasattr(torch, "float4_e2m1fn_x2") else ())
        self.bytes = (torch.uint8, torch.float32)
        self.sdpa = {torch.bfloat16: SDPA_BF16, torch.uint8: SDPA_E4M3, torch.float8_e4m3fn: SDPA_E4M3}
        self.out = {MLA_OUT_F32: self.f32, MLA_OUT_BF16: self.bf16, MLA_OUT_E4M3: self.codes}
        self.device, self.raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream
        self.cuda = torch.cuda


_types = None


def _t() -> _Types:
    global _types
    if _types is None:
        _types = _Types()
    return _types


def _refuse(where: str, what: str):
    raise SplitKVError(MLA_ERR_INVALID_ARG, f"{where}: {what}")


def _device(where: str) -> int:
    """The current CUDA device."""
    t = _t()
    if not t.cuda.is_initialized():
        if not t.cuda.is_available():
            return -2          # no tensor lies on it
        t.cuda.init()
    return t.device()


def _dev(where: str, name: str, x, dtypes, dev: int, numel: int = 0, contiguous: bool = True) -> int:
    """The address of a tensor that lies on the current device, has one of `dtypes`, is contiguous (unless its strides
    are taken) and holds at least `numel` elements; raises for any other."""
    try:
        if x.get_device() == dev and x.dtype in dtypes and x.numel() >= numel and (not contiguous or x.is_contiguous()):
            return x.data_ptr()
    except AttributeError:
        _refuse(where, f"{name} is missing or no tensor")
    if x.get_device() != dev:
        _refuse(where, f"{name} must be a tensor on the current CUDA device")
    if x.dtype not in dtypes:
        _refuse(where, f"{name} has type {x.dtype}, not {' or '.join(map(str, dtypes))}")
    if x.numel() < numel:
        _refuse(where, f"{name} has {x.numel()} elements, fewer than {numel}")
    _refuse(where, f"{name} must be contiguous")


def _opt(where: str, name: str, x, dtypes, dev: int, numel: int = 0):
    return None if x is None else _dev(where, name, x, dtypes, dev, numel)


def _strided(where: str, name: str, x, dims: int):
    """The strides of a tensor whose last dimension is contiguous; a dimension of one element, whose stride
    says nothing, counts as packed."""
    st, shape = x.stride(), x.shape
    if len(shape) != dims or (shape[-1] > 1 and st[-1] != 1):
        _refuse(where, f"{name} must have {dims} dimensions, the last one contiguous")
    if 1 not in shape:
        return st
    st, packed = list(st), 1
    for i in reversed(range(dims)):
        if shape[i] == 1:
            st[i] = packed
        packed *= max(1, shape[i])
    return tuple(st)


def _strided_pair(where: str, names, x, y, dims: int):
    """The strides of two tensors that have to share shape and strides."""
    st, shape = x.stride(), x.shape
    if len(shape) == dims and 1 not in shape and st[-1] == 1 and y.stride() == st and y.shape == shape:
        return st
    st = _strided(where, names[0], x, dims)
    if y.shape != x.shape or (y.stride() != x.stride() and _strided(where, names[1], y, dims) != st):
        _refuse(where, f"{names[0]} and {names[1]} differ in shape or strides")
    return st


def _rows(where: str, pages: KvPages, names, x, y, slot_map, descale_k, descale_v, dev: int):
    """What kv_pages_write and kv_pages_read take of their tensors: addresses, strides, the row count."""
    t = _t()
    F32 = t.F32
    try:   # (the checks of _dev in one go: the call of few rows is the host's time)
        ok = (x.get_device() == dev and y.get_device() == dev and slot_map.get_device() == dev and x.dtype is t.BF and y.dtype is t.BF
              and slot_map.dtype is t.I64 and slot_map.is_contiguous()
              and (descale_k is None or (descale_k.get_device() == dev and descale_k.dtype is F32 and descale_k.numel() == 1))
              and (descale_v is None or (descale_v.get_device() == dev and descale_v.dtype is F32 and descale_v.numel() == 1)))
    except AttributeError:
        ok = False
    if not ok:
        for n, z in zip(names, (x, y)):
            _dev(where, n, z, t.bf16, dev, contiguous=False)
        _dev(where, "slot_map", slot_map, t.i64, dev)
        _opt(where, "descale_k", descale_k, t.f32, dev, 1)
        _opt(where, "descale_v", descale_v, t.f32, dev, 1)
    st = _strided_pair(where, names, x, y, 3)
    rows, h, d = x.shape
    if h != pages.h_kv or d != pages.d:
        _refuse(where, f"{names[0]} and {names[1]} must be [rows, {pages.h_kv}, {pages.d}]")
    if slot_map.numel() < rows:
        _refuse(where, f"slot_map has {slot_map.numel()} elements, fewer than {rows}")
    return (rows, x.data_ptr(), y.data_ptr(), st, slot_map.data_ptr(), None if descale_k is None else descale_k.data_ptr(),
            None if descale_v is None else descale_v.data_ptr())


def _table(where: str, block_table, batch: int, dev: int):
    p = _dev(where, "block_table", block_table, _t().i32, dev, 1)
    if block_table.dim() != 2 or block_table.shape[0] < batch:
        _refuse(where, "block_table must be [batch, table_width]")
    return p, block_table.shape[1]


def _outputs(where: str, out_dtype: int, out, lse_out, amax_out, rows: int, d: int, dev: int):
    t = _t()
    if out_dtype not in t.out:
        _refuse(where, f"unknown output type {out_dtype}")
    return (_dev(where, "out", out, t.out[out_dtype], dev, rows * d), _opt(where, "lse_out", lse_out, t.f32, dev, rows),
            _opt(where, "amax_out", amax_out, t.f32, dev, 1))


def _on(stream, dev: int) -> int:
    return _t().raw_stream(dev) if stream is None else _stream(stream)


def _pages(where: str, pages: KvPages, dev: int):
    """The descriptor by reference; raises where kv_pages made it from tensors on another device than the current one."""
    if getattr(pages, "device", dev) != dev:
        _refuse(where, f"pages lie on CUDA device {pages.device}, the current one is {dev}")
    return ctypes.byref(pages)


def kv_pages(k_cache, v_cache, k_scales=None, v_scales=None) -> KvPages:
    """The C descriptor of a paged cache from views [num_pages, page_size, h_kv, d] of its tensors (bfloat16, or
    uint8 / float8_e4m3fn codes; any strides over a contiguous d, so a [num_pages, h_kv, page_size, d] cache is
    passed as its permute(0, 2, 1, 3)). A cache in 4 bits has views [num_pages, page_size, h_kv, d / 2] of bytes (two e2m1
    codes each, the first in the low half) and, with them, its scales: views [num_pages, page_size, h_kv, d / 16] of e4m3 bytes
    in which the rows of a page and head lie side by side, the permute(0, 2, 1, 3) of [num_pages, h_kv, page_size, d / 16].
    The descriptor keeps the tensors alive; calls that take it want their device to be the current one."""
    where, t = "kv_pages", _t()
    dev = _device(where)
    four = k_scales is not None or v_scales is not None
    k, v = (_dev(where, n, x, t.bytes4 if four else t.data, dev, contiguous=False)
            for n, x in (("k_cache", k_cache), ("v_cache", v_cache)))
    st = _strided(where, "k_cache", k_cache, 4)
    dt = SDPA_E2M1 if four else t.sdpa[k_cache.dtype]
    if (v_cache.shape != k_cache.shape or (not four and t.sdpa[v_cache.dtype] != dt)
            or _strided(where, "v_cache", v_cache, 4) != st):
        _refuse(where, "k_cache and v_cache differ in shape, type or strides")
    n, ps, h, d = k_cache.shape
    if not four:
        pages = KvPages(k, v, dt, n, ps, h, d, 0, st[0], st[1], st[2])
        pages.tensors, pages.device = (k_cache, v_cache), dev
        return pages
    d *= 2
    ks, vs = (_dev(where, name, x, t.codes, dev, contiguous=False) for name, x in (("k_scales", k_scales), ("v_scales", v_scales)))
    ss = _strided(where, "k_scales", k_scales, 4)
    if tuple(k_scales.shape) != (n, ps, h, d // 16) or v_scales.shape != k_scales.shape or _strided(where, "v_scales", v_scales, 4) != ss:
        _refuse(where, f"k_scales and v_scales must be [{n}, {ps}, {h}, {d // 16}], with the same strides")
    if ps > 1 and ss[1] != d // 16:
        _refuse(where, "the scales of a page and head must lie side by side: the permute(0, 2, 1, 3) of [num_pages, h_kv, page_size, d / 16]")
    # (a dimension of one element, whose stride says nothing, counts as packed behind the rows)
    sh = ss[2] if h > 1 else ps * (d // 16)
    sp = ss[0] if n > 1 else ps * (d // 16) * h
    pages = KvPages(k, v, dt, n, ps, h, d, 0, st[0], st[1], st[2], ks, vs, sp, sh)
    pages.tensors, pages.device = (k_cache, v_cache, k_scales, v_scales), dev
    return pages


def kv_pages_map(page_size: int, held_lens, new_lens, cu_seqlens_q, total_q: int, block_table, free_pages, free_in,
                 free_out, slot_map=None, positions=None, stream=None):
    """Block tables and slot maps from request lengths (block_table, free_pages, free_out, slot_map and
    positions are written in place)."""
    where, t = "kv_pages_map", _t()
    i32, dev = t.i32, _device(where)
    held = _dev(where, "held_lens", held_lens, i32, dev, 1)
    batch = held_lens.numel()
    new = _dev(where, "new_lens", new_lens, i32, dev, batch)
    cu = _dev(where, "cu_seqlens_q", cu_seqlens_q, i32, dev, batch + 1)
    table, width = _table(where, block_table, batch, dev)
    free = _dev(where, "free_pages", free_pages, i32, dev, 1)
    fin, fout = _dev(where, "free_in", free_in, i32, dev, 1), _dev(where, "free_out", free_out, i32, dev, 2)
    slots = _opt(where, "slot_map", slot_map, t.i64, dev, total_q)
    pos = _opt(where, "positions", positions, i32, dev, total_q)
    _check(lib().kv_pages_map(batch, page_size, held, new, cu, total_q, table, width, free, free_pages.numel(), fin, fout,
                              slots, pos, _on(stream, dev)), where)


def kv_pages_write(pages: KvPages, k_new, v_new, slot_map, descale_k=None, descale_v=None, stream=None):
    """Rows of k_new and v_new (bfloat16 [rows, h_kv, d], any strides over a contiguous d) into their slots."""
    where = "kv_pages_write"
    dev = _device(where)
    rows, k, v, st, slots, dk, dv = _rows(where, pages, ("k_new", "v_new"), k_new, v_new, slot_map, descale_k, descale_v, dev)
    status = (_lib or lib()).kv_pages_write(_pages(where, pages, dev), rows, k, v, st[0], st[1], slots, dk, dv, _on(stream, dev))
    if status:
        raise SplitKVError(status, where)


def kv_pages_write_rotary(pages: KvPages, q, k_new, v_new, positions, cos_sin, slot_map, q_out=None, k_out=None, *,
                          interleaved: bool = False, descale_q=None, descale_k=None, descale_v=None, stream=None):
    """kv_pages_write with the rows' rotation on the way: q (or None) and k_new turned by the angles of their positions, q into
    q_out (bfloat16, or uint8 / float8_e4m3fn codes; None: in place), k_new into its slots and, rotated, into k_out
    (bfloat16, or None). cos_sin is float32 [num_positions, rotary_dim], cosines then sines."""
    where, t = "kv_pages_write_rotary", _t()
    dev = _device(where)
    BF, F32 = t.BF, t.F32
    try:   # (the checks of _dev in one go: the call of few rows is the host's time)
        ok = (k_new.get_device() == dev and v_new.get_device() == dev and positions.get_device() == dev
              and cos_sin.get_device() == dev and slot_map.get_device() == dev and k_new.dtype is BF and v_new.dtype is BF
              and positions.dtype is t.I32 and cos_sin.dtype is F32 and slot_map.dtype is t.I64
              and positions.is_contiguous() and cos_sin.is_contiguous() and slot_map.is_contiguous()
              and (q is None or (q.get_device() == dev and q.dtype is BF))
              and (q_out is None or (q_out.get_device() == dev and q_out.dtype in t.sdpa))
              and (descale_q is None or (descale_q.get_device() == dev and descale_q.dtype is F32 and descale_q.numel() == 1))
              and (descale_k is None or (descale_k.get_device() == dev and descale_k.dtype is F32 and descale_k.numel() == 1))
              and (descale_v is None or (descale_v.get_device() == dev and descale_v.dtype is F32 and descale_v.numel() == 1)))
    except AttributeError:
        ok = False
    if not ok:
        for n, x, dt, c in (("k_new", k_new, t.bf16, False), ("v_new", v_new, t.bf16, False), ("positions", positions, t.i32, True),
                            ("cos_sin", cos_sin, t.f32, True), ("slot_map", slot_map, t.i64, True)):
            _dev(where, n, x, dt, dev, contiguous=c)
        for n, x, dt in (("q", q, t.bf16), ("q_out", q_out, t.data)):
            if x is not None:
                _dev(where, n, x, dt, dev, contiguous=False)
        for n, x in (("descale_q", descale_q), ("descale_k", descale_k), ("descale_v", descale_v)):
            _opt(where, n, x, t.f32, dev, 1)
    st = _strided_pair(where, ("k_new", "v_new"), k_new, v_new, 3)
    shape = k_new.shape
    rows, h, d = shape
    if h != pages.h_kv or d != pages.d:
        _refuse(where, f"k_new and v_new must be [rows, {pages.h_kv}, {pages.d}]")
    table = cos_sin.shape
    if len(table) != 2:
        _refuse(where, "cos_sin must be [num_positions, rotary_dim]")
    if positions.numel() < rows or slot_map.numel() < rows:
        _refuse(where, f"positions and slot_map must have {rows} elements")
    h_q, qp, qs, qo, qo_dt, os_ = 0, None, (0, 0), None, SDPA_BF16, (0, 0)
    if q is not None:
        qp = q.data_ptr()
        q_shape, qs = q.shape, q.stride()
        if len(q_shape) != 3 or 1 in q_shape or qs[2] != 1:
            qs = _strided(where, "q", q, 3)
        h_q = q_shape[1]
        if q_shape[0] != rows or q_shape[2] != d:
            _refuse(where, f"q must be [{rows}, h_q, {d}]")
        if q_out is None:
            qo, os_ = qp, qs
        else:
            qo, qo_dt, os_ = q_out.data_ptr(), t.sdpa[q_out.dtype], q_out.stride()
            if q_out.shape != q_shape:
                _refuse(where, "q_out must have q's shape")
            if 1 in q_shape or os_[2] != 1:
                os_ = _strided(where, "q_out", q_out, 3)
    elif q_out is not None:
        _refuse(where, "q_out without q")
    ko, ks = None, (0, 0)
    if k_out is not None:
        ko = _dev(where, "k_out", k_out, t.bf16, dev, contiguous=False)
        ks = _strided(where, "k_out", k_out, 3)
        if k_out.shape != shape:
            _refuse(where, "k_out must have k_new's shape")
    dq = None if descale_q is None else descale_q.data_ptr()
    dk = None if descale_k is None else descale_k.data_ptr()
    dv = None if descale_v is None else descale_v.data_ptr()
    status = (_lib or lib()).kv_pages_write_rotary(
        _pages(where, pages, dev), rows, h_q, qp, qs[0], qs[1], k_new.data_ptr(), v_new.data_ptr(), st[0], st[1],
        positions.data_ptr(), cos_sin.data_ptr(), table[0], table[1], 1 if interleaved else 0, slot_map.data_ptr(), dq, dk, dv, qo_dt, qo,
        os_[0], os_[1], ko, ks[0], ks[1], _on(stream, dev))
    if status:
        raise SplitKVError(status, where)


def kv_pages_read(pages: KvPages, slot_map, k_out, v_out, descale_k=None, descale_v=None, stream=None):
    """Rows of a cache of any type into k_out and v_out (bfloat16 [rows, h_kv, d], any strides over a contiguous d)."""
    where = "kv_pages_read"
    dev = _device(where)
    rows, k, v, st, slots, dk, dv = _rows(where, pages, ("k_out", "v_out"), k_out, v_out, slot_map, descale_k, descale_v, dev)
    status = (_lib or lib()).kv_pages_read(_pages(where, pages, dev), rows, slots, dk, dv, k, v, st[0], st[1], _on(stream, dev))
    if status:
        raise SplitKVError(status, where)


def sdpa_paged_plan(batch: int, h_q: int, h_kv: int, d: int, dtype, max_q_per_seq: int, total_q_max: int, max_kv: int,
                    *, num_sms: int = 0, max_splits: int = 0, force_splits: int = 0) -> SdpaPagedPlan:
    plan = SdpaPagedPlan()
    dt = _SDPA_DTYPES[dtype] if isinstance(dtype, str) else int(dtype)
    _check(lib().sdpa_paged_plan(batch, h_q, h_kv, d, dt, max_q_per_seq, total_q_max, max_kv, num_sms, max_splits,
                                 force_splits, ctypes.byref(plan)), "sdpa_paged_plan")
    return plan


def sdpa_paged(plan: SdpaPagedPlan, total_q: int, q, pages: KvPages, block_table, kv_lens, cu_seqlens_q, descale_q,
               descale_k, descale_v, sm_scale: float, out_dtype, out_inv_scale: float, out, lse_out=None, amax_out=None,
               workspace=None, stream=None):
    """Attention of new tokens over a paged cache; q [>= total_q, h_q, d] of the plan's type, any strides over a
    contiguous d."""
    where, t = "sdpa_paged", _t()
    dev = _device(where)
    batch, h_q, d = plan.batch, plan.h_q, plan.d
    q_types = t.codes if plan.dtype == SDPA_E4M3 else t.bf16
    od, F32, I32 = _dtype(out_dtype), t.F32, t.I32
    try:   # (the checks of _dev in one go: a short call is the host's time)
        ok = (q.get_device() == dev and q.dtype in q_types and block_table.get_device() == dev and block_table.dtype is I32
              and block_table.is_contiguous() and block_table.numel() > 0 and kv_lens.get_device() == dev and kv_lens.dtype is I32
              and kv_lens.is_contiguous() and kv_lens.numel() >= batch and cu_seqlens_q.get_device() == dev and cu_seqlens_q.dtype is I32
              and cu_seqlens_q.is_contiguous() and cu_seqlens_q.numel() > batch
              and (descale_q is None or (descale_q.get_device() == dev and descale_q.dtype is F32 and descale_q.numel() == 1))
              and (descale_k is None or (descale_k.get_device() == dev and descale_k.dtype is F32 and descale_k.numel() == 1))
              and (descale_v is None or (descale_v.get_device() == dev and descale_v.dtype is F32 and descale_v.numel() == 1))
              and out.get_device() == dev and out.dtype in t.out[od] and out.is_contiguous() and out.numel() >= total_q * h_q * d
              and (lse_out is None or (lse_out.get_device() == dev and lse_out.dtype is F32 and lse_out.is_contiguous()
                                       and lse_out.numel() >= total_q * h_q))
              and (amax_out is None or (amax_out.get_device() == dev and amax_out.dtype is F32 and amax_out.numel() == 1)))
    except (AttributeError, KeyError):
        ok = False
    if not ok:
        _dev(where, "q", q, q_types, dev, contiguous=False)
        _table(where, block_table, batch, dev)
        _dev(where, "kv_lens", kv_lens, t.i32, dev, batch)
        _dev(where, "cu_seqlens_q", cu_seqlens_q, t.i32, dev, batch + 1)
        for n, x in (("descale_q", descale_q), ("descale_k", descale_k), ("descale_v", descale_v)):
            _opt(where, n, x, t.f32, dev, 1)
        _outputs(where, od, out, lse_out, amax_out, total_q * h_q, d, dev)
    q_shape, st = q.shape, q.stride()
    if len(q_shape) != 3 or 1 in q_shape or st[2] != 1:
        st = _strided(where, "q", q, 3)
    if q_shape[1] != h_q or q_shape[2] != d or q_shape[0] < total_q:
        _refuse(where, f"q must be [{total_q} or more, {h_q}, {d}]")
    shape = block_table.shape
    if len(shape) != 2 or shape[0] < batch:
        _refuse(where, "block_table must be [batch, table_width]")
    ws = None
    if plan.workspace_bytes:
        ws = _dev(where, "workspace", workspace, t.bytes, dev)
        if workspace.nbytes < plan.workspace_bytes:
            _refuse(where, "workspace is smaller than the plan's")
    status = (_lib or lib()).sdpa_paged(
        ctypes.byref(plan), total_q, q.data_ptr(), st[0], st[1], _pages(where, pages, dev), block_table.data_ptr(), shape[1],
        kv_lens.data_ptr(), cu_seqlens_q.data_ptr(), None if descale_q is None else descale_q.data_ptr(),
        None if descale_k is None else descale_k.data_ptr(), None if descale_v is None else descale_v.data_ptr(), sm_scale, od,
        out_inv_scale, out.data_ptr(), None if lse_out is None else lse_out.data_ptr(),
        None if amax_out is None else amax_out.data_ptr(), ws, _on(stream, dev))
    if status:
        raise SplitKVError(status, where)


def sdpa_prompt(batch: int, q, k, v, cu_seqlens_q, cu_seqlens_kv, descale_q, descale_k, descale_v, sm_scale: float,
                out_dtype, out_inv_scale: float, out, lse_out=None, amax_out=None, stream=None):
    """Causal attention over packed prompts; q [total_q, h_q, d], k and v [total_kv, h_kv, d] of one type, any
    strides over a contiguous d (k and v the same)."""
    where, t = "sdpa_prompt", _t()
    dev = _device(where)
    qp, kp, vp = (_dev(where, n, x, t.data, dev, contiguous=False) for n, x in (("q", q), ("k", k), ("v", v)))
    qs, ks = _strided(where, "q", q, 3), _strided(where, "k", k, 3)
    if v.shape != k.shape or _strided(where, "v", v, 3) != ks:
        _refuse(where, "k and v differ in shape or strides")
    dt = t.sdpa[q.dtype]
    total_q, h_q, d = q.shape
    total_kv, h_kv, dk_ = k.shape
    if t.sdpa[k.dtype] != dt or t.sdpa[v.dtype] != dt or dk_ != d:
        _refuse(where, "q, k and v must have one type and one head dim")
    cu = _dev(where, "cu_seqlens_q", cu_seqlens_q, t.i32, dev, batch + 1)
    ck = _dev(where, "cu_seqlens_kv", cu_seqlens_kv, t.i32, dev, batch + 1)
    dq = _opt(where, "descale_q", descale_q, t.f32, dev, 1)
    dk = _opt(where, "descale_k", descale_k, t.f32, dev, 1)
    dv = _opt(where, "descale_v", descale_v, t.f32, dev, 1)
    od = _dtype(out_dtype)
    o, lse, amax = _outputs(where, od, out, lse_out, amax_out, total_q * h_q, d, dev)
    _check(lib().sdpa_prompt(batch, h_q, h_kv, d, dt, total_q, total_kv, qp, qs[0], qs[1], kp, vp, ks[0], ks[1], cu, ck, dq,
                             dk, dv, sm_scale, od, out_inv_scale, o, lse, amax, _on(stream, dev)), where)


# ------------------------------------------------------------------- status --

def mla_get_status():
    """Synchronise the current device, then read and clear its status word: (bits, first site)."""
    st, site = ctypes.c_uint32(0), ctypes.c_uint32(0)
    _check(lib().mla_get_status(ctypes.byref(st), ctypes.byref(site)), "mla_get_status")
    return st.value, site.value


def mla_set_index_checks(enable: bool = True):
    """Report gathered indices outside {-1} and [0, n_kv) (status bit MLA_STATUS_BAD_INDEX) in later calls."""
    _check(lib().mla_set_index_checks(int(enable)), "mla_set_index_checks")


def mla_set_wait_limit_ns(limit_ns: int):
    """Time limit of the decode kernels' pipeline waits for later calls (0 = the 2 s default)."""
    _check(lib().mla_set_wait_limit_ns(limit_ns), "mla_set_wait_limit_ns")


def mla_selftest_wait_timeout(limit_ns: int, stream=None):
    _check(lib().mla_selftest_wait_timeout(limit_ns, _stream(stream)), "mla_selftest_wait_timeout")


def mla_abi_version() -> int:
    return lib().mla_abi_version()
