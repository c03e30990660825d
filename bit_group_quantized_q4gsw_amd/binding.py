"""Thin ctypes binding of libq4gsw.so (include/q4gsw.h).

Argument marshalling only: every step of the computation runs in the HIP
kernels behind the C ABI.  PyTorch provides device memory (output and workspace
tensors) and the current HIP stream.  There is no CPU fallback: importing the
package without the built library raises.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
import re
import struct
import threading
import warnings
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libq4gsw.so")

F32, F16, BF16 = 0, 1, 2
OP_FWD, OP_BWD_INPUT, OP_QKV, OP_DQ8CA = 0, 1, 2, 3
ROUTES = {
    "none": 0, "generic": 1, "gemv": 2, "gemm_fold": 3, "gemm_group": 4, "gemm_split": 5,
    "bwd_gemv": 6, "bwd_fold": 7, "bwd_split": 8, "qkv_fused": 9, "bwd_bsplit": 10, "dq8ca": 11,
}
FLAG_FOLD_F16 = 1
_TORCH_DTYPE = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}


class Q4gswError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {status_str(status)} (status {status})")
        self.status = status


class WeightDesc(ctypes.Structure):
    """Mirror of struct q4gsw_weight."""
    _fields_ = [
        ("magic", ctypes.c_uint32), ("version", ctypes.c_uint32),
        ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("group_size", ctypes.c_int64),
        ("n_pad", ctypes.c_int64), ("k_pad", ctypes.c_int64), ("g_pad", ctypes.c_int64),
        ("scale_dtype", ctypes.c_int32), ("flags", ctypes.c_uint32),
        ("data", ctypes.c_void_p), ("bytes", ctypes.c_uint64),
        ("nibble_offset", ctypes.c_uint64), ("scale_offset", ctypes.c_uint64),
    ]


class PlanInfo(ctypes.Structure):
    """q4gsw_plan_info of include/q4gsw.h."""
    _fields_ = [("route", ctypes.c_int32), ("tile_rows", ctypes.c_int32), ("splits", ctypes.c_int32)]


class Options(ctypes.Structure):
    """q4gsw_options of include/q4gsw.h: a per-call route family, block rows and split count."""
    _fields_ = [("route", ctypes.c_int32), ("tile_rows", ctypes.c_int32), ("splits", ctypes.c_int32)]


class AdamwParams(ctypes.Structure):
    """q4gsw_adamw_params of include/q4gsw.h."""
    _fields_ = [("lr", ctypes.c_float), ("beta1", ctypes.c_float), ("beta2", ctypes.c_float),
                ("eps", ctypes.c_float), ("weight_decay", ctypes.c_float)]


class KvCacheDesc(ctypes.Structure):
    """q4gsw_kv_cache of include/q4gsw.h."""
    _fields_ = [("pages", ctypes.c_int64), ("page_size", ctypes.c_int32), ("heads", ctypes.c_int32),
                ("dim", ctypes.c_int32), ("reserved", ctypes.c_int32), ("data", ctypes.c_void_p),
                ("bytes", ctypes.c_uint64)]


class KvSeqs(ctypes.Structure):
    """q4gsw_kv_seqs of include/q4gsw.h."""
    _fields_ = [("table", ctypes.c_void_p), ("table_ld", ctypes.c_int64), ("table_cols", ctypes.c_int32),
                ("batch", ctypes.c_int32), ("cu", ctypes.c_void_p), ("lens", ctypes.c_void_p),
                ("tokens", ctypes.c_int64)]


class AdaptersDesc(ctypes.Structure):
    """q4gsw_adapters of include/q4gsw.h."""
    _fields_ = [("N", ctypes.c_int64), ("K", ctypes.c_int64), ("slots", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32), ("data", ctypes.c_void_p),
                ("bytes", ctypes.c_uint64)]


class LogitsRules(ctypes.Structure):
    """q4gsw_logits_rules of include/q4gsw.h."""
    _fields_ = [("batch", ctypes.c_int32), ("max_new", ctypes.c_int32), ("cu", ctypes.c_void_p),
                ("history", ctypes.c_void_p), ("history_ld", ctypes.c_int64), ("history_cols", ctypes.c_int32),
                ("bias_cols", ctypes.c_int32), ("history_len", ctypes.c_void_p), ("prompt_len", ctypes.c_void_p),
                ("ids", ctypes.c_void_p), ("parents", ctypes.c_void_p), ("repetition", ctypes.c_void_p),
                ("presence", ctypes.c_void_p), ("frequency", ctypes.c_void_p), ("bias_ids", ctypes.c_void_p),
                ("bias", ctypes.c_void_p), ("bias_ld", ctypes.c_int64), ("mask", ctypes.c_void_p),
                ("mask_ld", ctypes.c_int64)]


class KvPlanInfo(ctypes.Structure):
    """q4gsw_kv_plan_info of include/q4gsw.h."""
    _fields_ = [("kernel", ctypes.c_int32), ("waves", ctypes.c_int32), ("splits", ctypes.c_int32)]


class KvOptions(ctypes.Structure):
    """q4gsw_kv_options of include/q4gsw.h."""
    _fields_ = [("kernel", ctypes.c_int32), ("reserved", ctypes.c_int32)]


KV_KERNELS = {"any": 0, "few_rows": 1, "many_rows": 2, "tree": 3}


# Choices made by forced_route / forced_plan, held per Python thread and handed to each call
# (the library itself keeps no routing state).
class _Local(threading.local):
    opts = None
    kv = None


_local = _Local()


def _opts():
    """The current thread's options, or None (library defaults)."""
    o = _local.opts
    if o is None or (o.route == 0 and o.tile_rows == 0 and o.splits == 0):
        return None
    return ctypes.byref(o)


_lib: Optional[ctypes.CDLL] = None
_host = None            # the module _host: regular serving calls, marshalled in C++ (csrc/host.cpp)


class _Python:
    """In the place of _host where it cannot be loaded: no call is regular, and all are marshalled in Python."""

    @staticmethod
    def _left(*args):
        return None

    attention = append = read = keep = adapters = logits = _left


def _load_host(h: ctypes.CDLL):
    """The module _host, or its stand-in where it was not built or was built for another torch."""
    try:
        from . import _host as host
        if host.torch_version != re.match(r"[0-9.]*[0-9]", torch.__version__).group():      # the headers' has no suffix
            raise ImportError(f"_host was built for torch {host.torch_version}")
        host.open(h._handle, torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream)
        return host
    except (ImportError, AttributeError) as e:
        warnings.warn(f"serving calls are marshalled in Python, which takes longer ({e}); build again with "
                      "python bit_group_quantized_q4gsw_amd/build.py", RuntimeWarning, stacklevel=3)
        return _Python()


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built (no fallback exists)."""
    global _lib, _host
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: build it with python bit_group_quantized_q4gsw_amd/build.py; "
                              "there is no CPU fallback")
        h = ctypes.CDLL(LIB_PATH)
        i32, i64, u64, vp = ctypes.c_int32, ctypes.c_int64, ctypes.c_uint64, ctypes.c_void_p
        pw = ctypes.POINTER(WeightDesc)
        po = ctypes.POINTER(Options)
        ko = ctypes.POINTER(KvOptions)
        pa = ctypes.POINTER(AdaptersDesc)
        pc, ps = ctypes.POINTER(KvCacheDesc), vp       # sequences: a KvSeqs by reference or its packed bytes
        sigs = {
            "q4gsw_packed_bytes": [i64, i64, i64, i32, ctypes.POINTER(u64)],
            "q4gsw_pack": [vp, vp, i32, i64, i64, i64, vp, u64, vp, pw],
            "q4gsw_unpack": [pw, vp, vp, vp],
            "q4gsw_workspace_bytes": [i32, pw, i64, i32, ctypes.POINTER(u64)],
            "q4gsw_qkv_workspace_bytes": [pw, pw, pw, i64, i32, ctypes.POINTER(u64)],
            "q4gsw_workspace_bytes_ex": [i32, pw, i64, i32, po, ctypes.POINTER(u64)],
            "q4gsw_qkv_workspace_bytes_ex": [pw, pw, pw, i64, i32, po, ctypes.POINTER(u64)],
            "q4gsw_linear_fwd": [pw, vp, i32, i64, vp, vp, u64, vp],
            "q4gsw_linear_bwd_input": [pw, vp, i32, i64, vp, vp, u64, vp],
            "q4gsw_qkv_fused": [pw, pw, pw, vp, i32, i64, vp, vp, vp, vp, u64, vp],
            "q4gsw_linear_fwd_ex": [pw, vp, i32, i64, vp, vp, u64, po, vp],
            "q4gsw_linear_fwd_noalloc": [pw, vp, i32, i64, vp, vp],
            "q4gsw_linear_bwd_input_ex": [pw, vp, i32, i64, vp, vp, u64, po, vp],
            "q4gsw_qkv_fused_ex": [pw, pw, pw, vp, i32, i64, vp, vp, vp, vp, u64, po, vp],
            "q4gsw_route": [i32, pw, i64, i32],
            "q4gsw_plan": [i32, pw, pw, pw, i64, i32, po, ctypes.POINTER(PlanInfo)],
            "q4gsw_embedding": [pw, vp, i64, vp, vp],
            "q4gsw_dq8ca_quantize": [vp, i32, i64, i64, vp, vp, vp, vp],
            "q4gsw_linear_dq8ca": [pw, vp, i32, i64, vp, vp, u64, vp],
            "q4gsw_linear_dq8ca_ex": [pw, vp, i32, i64, vp, vp, u64, po, vp],
            "q4gsw_dq8ca_rows_bytes": [i64, i64, ctypes.POINTER(u64)],
            "q4gsw_rmsnorm_dq8ca": [vp, i32, vp, vp, i32, i64, i64, ctypes.c_float, vp, vp, u64, vp, vp],
            "q4gsw_dq8ca_rows_workspace_bytes": [pw, i64, ctypes.POINTER(u64)],
            "q4gsw_linear_dq8ca_rows": [pw, vp, u64, i64, vp, vp, u64, vp],
            "q4gsw_dq8ca_rows_workspace_bytes_ex": [pw, i64, po, ctypes.POINTER(u64)],
            "q4gsw_linear_dq8ca_rows_ex": [pw, vp, u64, i64, vp, vp, u64, po, vp],
            "q4gsw_kv_bytes": [pc, ctypes.POINTER(u64)],
            "q4gsw_kv_append": [pc, ps, vp, i64, vp, i64, i32, vp],
            "q4gsw_kv_read": [pc, ps, vp, vp, vp],
            "q4gsw_kv_attention_workspace_bytes": [pc, i32, i64, i32, i32, i32, ctypes.POINTER(u64)],
            "q4gsw_kv_attention_plan": [pc, i32, i64, i32, i32, i32, i32, i32, ko, ctypes.POINTER(KvPlanInfo)],
            "q4gsw_kv_attention": [pc, ps, vp, i64, i32, i32, i32, i32, i32, ctypes.c_float, vp, vp, u64, vp],
            "q4gsw_kv_attention_ex": [pc, ps, vp, i64, i32, i32, i32, i32, i32, ctypes.c_float, vp, vp, u64, ko, vp],
            "q4gsw_kv_tree_attention_workspace_bytes": [pc, i32, i64, i32, i32, i32, ctypes.POINTER(u64)],
            "q4gsw_kv_tree_attention": [pc, ps, vp, vp, i64, i32, i32, i32, i32, i32, ctypes.c_float, vp, vp, u64, vp],
            "q4gsw_kv_tree_attention_ex": [pc, ps, vp, vp, i64, i32, i32, i32, i32, i32, ctypes.c_float, vp, vp, u64, ko, vp],
            "q4gsw_kv_keep": [pc, i32, ps, vp, vp, i32, vp, vp, vp],
            "q4gsw_adapter_workspace_bytes": [i32, pw, i64, i32, i32, ctypes.POINTER(u64)],
            "q4gsw_adapter_fwd": [pw, vp, i32, i64, vp, vp, i32, ctypes.c_float, vp, vp, vp, u64, vp],
            "q4gsw_adapter_bwd": [pw, vp, vp, i32, i64, vp, vp, i32, ctypes.c_float, vp, vp, vp, vp, vp, u64, vp],
            "q4gsw_logits_adjust": [vp, i32, i64, i64, i64, vp, vp, i64, vp],
            "q4gsw_adapters_bytes": [pa, ctypes.POINTER(u64)],
            "q4gsw_adapters_load": [pa, i32, vp, vp, i32, i32, ctypes.c_float, vp],
            "q4gsw_adapters_workspace_bytes": [pa, pw, i64, i32, ctypes.POINTER(u64)],
            "q4gsw_adapters_add": [pa, vp, i32, i64, vp, vp, vp, vp, u64, vp],
            "q4gsw_adapters_fwd": [pw, pa, vp, i32, i64, vp, vp, vp, u64, vp],
            "q4gsw_adamw_step": [vp, vp, vp, vp, i64, ctypes.POINTER(AdamwParams), i64, vp],
        }
        for name, args in sigs.items():
            fn = getattr(h, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int32
        h.q4gsw_route_name.argtypes = [i32]
        h.q4gsw_route_name.restype = ctypes.c_char_p
        h.q4gsw_status_str.argtypes = [i32]
        h.q4gsw_status_str.restype = ctypes.c_char_p
        h.q4gsw_layout_version.argtypes = []
        h.q4gsw_layout_version.restype = ctypes.c_uint32
        h.q4gsw_build_info.argtypes = []
        h.q4gsw_build_info.restype = ctypes.c_char_p
        _lib, _host = h, _load_host(h)
    return _lib


def status_str(status: int) -> str:
    return lib().q4gsw_status_str(status).decode()


def route_name(route: int) -> str:
    return lib().q4gsw_route_name(route).decode()


def _check(status: int, what: str) -> None:
    if status != 0:
        raise Q4gswError(status, what)


def _done(result, what: str):
    """What a function of _host returned, unless it is the status of a call that the library refused."""
    if type(result) is int:
        raise Q4gswError(result, what)
    return result


def _stream() -> int:
    """The current device's current stream as the integer a stream argument takes (through torch's raw
    accessors: building a Stream object costs more than a small kernel's launch)."""
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _stream_of(dev: int) -> int:
    """The current stream of the device of a call's tensors, which has to be the current device: a kernel is
    launched there."""
    current = torch._C._cuda_getDevice()
    if dev != current:
        raise ValueError(f"the tensors are on cuda:{dev}, the current device is cuda:{current}")
    return torch._C._cuda_getCurrentRawStream(current)


def _dev(t: torch.Tensor, name: str) -> torch.Tensor:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    return t.contiguous()


def _out(out: Optional[torch.Tensor], shape: Tuple[int, ...], device, name: str) -> torch.Tensor:
    """A caller's output tensor, checked against what the kernels write (contiguous fp32 of
    exactly `shape` on `device`), or a new one."""
    if out is None:
        return torch.empty(*shape, dtype=torch.float32, device=device)
    if (out.dtype != torch.float32 or not out.is_contiguous() or tuple(out.shape) != tuple(shape)
            or out.device != device):
        raise ValueError(f"{name} must be a contiguous fp32 tensor of shape {list(shape)} on {device}")
    return out


class PackedWeight:
    """A packed q4gsw weight: the descriptor plus the device buffer it points into."""

    def __init__(self, desc: WeightDesc, buffer: torch.Tensor):
        self.desc = desc
        self.buffer = buffer

    @property
    def N(self) -> int:
        return self.desc.N

    @property
    def K(self) -> int:
        return self.desc.K

    @property
    def group_size(self) -> int:
        return self.desc.group_size

    @property
    def foldable(self) -> bool:
        return bool(self.desc.flags & FLAG_FOLD_F16)

    def ref(self):
        return ctypes.byref(self.desc)


def packed_bytes(N: int, K: int, group_size: int, scale_dtype: torch.dtype) -> int:
    out = ctypes.c_uint64()
    _check(lib().q4gsw_packed_bytes(N, K, group_size, _TORCH_DTYPE[scale_dtype], ctypes.byref(out)),
           "q4gsw_packed_bytes")
    return out.value


def pack(codes: torch.Tensor, scales: torch.Tensor, group_size: int) -> PackedWeight:
    """codes uint8 [N, K] (0..15) and scales [K/group_size, N] (fp16/fp32), both on the GPU."""
    codes = _dev(codes, "codes")
    scales = _dev(scales, "scales")
    if codes.dtype != torch.uint8 or codes.dim() != 2:
        raise ValueError("codes must be uint8 [N, K]")
    N, K = codes.shape
    if scales.dtype not in (torch.float16, torch.float32):
        raise ValueError("scales must be fp16 or fp32")
    if group_size < 1 or K % group_size or tuple(scales.shape) != (K // group_size, N):
        raise ValueError("scales must be [K / group_size, N]")
    nbytes = packed_bytes(N, K, group_size, scales.dtype)
    buf = torch.empty(nbytes, dtype=torch.uint8, device=codes.device)
    desc = WeightDesc()
    _check(lib().q4gsw_pack(codes.data_ptr(), scales.data_ptr(), _TORCH_DTYPE[scales.dtype], N, K, group_size,
                            buf.data_ptr(), nbytes, _stream(), ctypes.byref(desc)), "q4gsw_pack")
    return PackedWeight(desc, buf)


def unpack(w: PackedWeight) -> Tuple[torch.Tensor, torch.Tensor]:
    dev = w.buffer.device
    codes = torch.empty(w.N, w.K, dtype=torch.uint8, device=dev)
    sdt = torch.float16 if w.desc.scale_dtype == F16 else torch.float32
    scales = torch.empty(w.K // w.group_size, w.N, dtype=sdt, device=dev)
    _check(lib().q4gsw_unpack(w.ref(), codes.data_ptr(), scales.data_ptr(), _stream()), "q4gsw_unpack")
    return codes, scales


def _workspace(nbytes: int, device) -> Tuple[Optional[torch.Tensor], int, int]:
    if nbytes == 0:
        return None, 0, 0
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return ws, ws.data_ptr(), nbytes


def workspace_bytes(op: int, w: PackedWeight, M: int, dtype: torch.dtype) -> int:
    out = ctypes.c_uint64()
    _check(lib().q4gsw_workspace_bytes_ex(op, w.ref(), M, _TORCH_DTYPE[dtype], _opts(), ctypes.byref(out)),
           "q4gsw_workspace_bytes")
    return out.value


def _ws_args(need: int, workspace: Optional[torch.Tensor], device):
    """(tensor kept alive, pointer, bytes): the caller's workspace when it is a large enough uint8
    tensor on `device`, else a new one."""
    if workspace is not None and workspace.dtype == torch.uint8 and workspace.is_contiguous() \
            and workspace.device == device and workspace.numel() >= need:
        return workspace, workspace.data_ptr(), workspace.numel()
    return _workspace(need, device)


def linear_fwd(w: PackedWeight, x: torch.Tensor, out: Optional[torch.Tensor] = None,
               workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [M, N] fp32 = x [M, K] . dequant(W)^T."""
    x = _dev(x, "x")
    if x.dim() != 2 or x.shape[1] != w.K:
        raise ValueError("x must be [M, K]")
    M = x.shape[0]
    y = _out(out, (M, w.N), x.device, "out")
    need = workspace_bytes(OP_FWD, w, M, x.dtype)
    ws, wp, wb = _ws_args(need, workspace, x.device)
    _check(lib().q4gsw_linear_fwd_ex(w.ref(), x.data_ptr(), _TORCH_DTYPE[x.dtype], M, y.data_ptr(), wp, wb,
                                     _opts(), _stream()), "q4gsw_linear_fwd")
    return y


def linear_fwd_noalloc(w: PackedWeight, x: torch.Tensor, out: torch.Tensor) -> torch.Tensor:
    """y [M, N] fp32 = x [M, K] . dequant(W)^T into the caller's `out`, through the entry point that
    allocates nothing (its split partials live in the library's per-device scratch; calls that
    overlap on one device race on it).  Raises Q4gswError (E_SCRATCH) when the call would need more
    scratch than the library holds."""
    x = _dev(x, "x")
    if x.dim() != 2 or x.shape[1] != w.K:
        raise ValueError("x must be [M, K]")
    M = x.shape[0]
    if out is None:
        raise ValueError("out is required: this entry point allocates nothing")
    y = _out(out, (M, w.N), x.device, "out")
    _check(lib().q4gsw_linear_fwd_noalloc(w.ref(), x.data_ptr(), _TORCH_DTYPE[x.dtype], M, y.data_ptr(), _stream()),
           "q4gsw_linear_fwd_noalloc")
    return y


def linear_bwd_input(w: PackedWeight, d_out: torch.Tensor, out: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """d_x [M, K] fp32 = d_out [M, N] . dequant(W), contracting over N."""
    d_out = _dev(d_out, "d_out")
    if d_out.dim() != 2 or d_out.shape[1] != w.N:
        raise ValueError("d_out must be [M, N]")
    M = d_out.shape[0]
    dx = _out(out, (M, w.K), d_out.device, "out")
    need = workspace_bytes(OP_BWD_INPUT, w, M, d_out.dtype)
    ws, wp, wb = _ws_args(need, workspace, d_out.device)
    _check(lib().q4gsw_linear_bwd_input_ex(w.ref(), d_out.data_ptr(), _TORCH_DTYPE[d_out.dtype], M,
                                           dx.data_ptr(), wp, wb, _opts(), _stream()), "q4gsw_linear_bwd_input")
    return dx


def dq8ca_quantize(x: torch.Tensor) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Per-row int8 quantisation of x [M, K]: (q int8 [M, K], scale fp32 [M], zero_point int32 [M])."""
    x = _dev(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [M, K]")
    M, K = x.shape
    q = torch.empty(M, K, dtype=torch.int8, device=x.device)
    scale = torch.empty(M, dtype=torch.float32, device=x.device)
    zp = torch.empty(M, dtype=torch.int32, device=x.device)
    _check(lib().q4gsw_dq8ca_quantize(x.data_ptr(), _TORCH_DTYPE[x.dtype], M, K, q.data_ptr(), scale.data_ptr(),
                                      zp.data_ptr(), _stream()), "q4gsw_dq8ca_quantize")
    return q, scale, zp


def linear_dq8ca(w: PackedWeight, x: torch.Tensor, out: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [M, N] fp32 = the forward of x's rows quantised to int8 per row (linear_dq8ca_q4gsw)."""
    x = _dev(x, "x")
    if x.dim() != 2 or x.shape[1] != w.K:
        raise ValueError("x must be [M, K]")
    M = x.shape[0]
    y = _out(out, (M, w.N), x.device, "out")
    need = workspace_bytes(OP_DQ8CA, w, M, x.dtype)
    ws, wp, wb = _ws_args(need, workspace, x.device)
    _check(lib().q4gsw_linear_dq8ca_ex(w.ref(), x.data_ptr(), _TORCH_DTYPE[x.dtype], M, y.data_ptr(), wp, wb,
                                       _opts(), _stream()), "q4gsw_linear_dq8ca")
    return y


class Dq8caRows:
    """M rows of K int8 activations in the int8 linear's layout, written by rmsnorm_dq8ca and read
    by linear_dq8ca_rows: codes, row scales and zero points in one device buffer."""

    def __init__(self, M: int, K: int, buffer: torch.Tensor):
        self.M = M
        self.K = K
        self.buffer = buffer


def dq8ca_rows(M: int, K: int, device="cuda") -> Dq8caRows:
    """An (unwritten) rows buffer for M rows of K columns."""
    out = ctypes.c_uint64()
    _check(lib().q4gsw_dq8ca_rows_bytes(M, K, ctypes.byref(out)), "q4gsw_dq8ca_rows_bytes")
    return Dq8caRows(M, K, torch.empty(out.value, dtype=torch.uint8, device=device))


def rmsnorm_dq8ca(x: torch.Tensor, weight: torch.Tensor, eps: float, residual: Optional[torch.Tensor] = None,
                  rows: Optional[Dq8caRows] = None, h: Optional[torch.Tensor] = None,
                  values: Optional[torch.Tensor] = None):
    """(rows, h, values): h = round(x + residual) in weight's dtype (x itself rounded, without a
    residual), rows = h * weight / sqrt(mean(h^2) + eps) in int8 codes with a scale and a zero point
    per row, for linear_dq8ca_rows.  `h` may be `residual` itself (updated in place); without a
    residual it is written only if given.  `values` (fp32 [M, K]) receives what the rows stand for
    if given."""
    x = _dev(x, "x")
    if x.dim() != 2:
        raise ValueError("x must be [M, K]")
    shape = x.shape
    M, K = shape
    dev = x.get_device()
    dt = weight.dtype
    r_dtype = _TORCH_DTYPE.get(dt)
    if r_dtype is None or weight.dim() != 1 or weight.numel() != K or weight.get_device() != dev:
        raise ValueError(f"weight must be a floating tensor of shape [{K}] on {x.device}")
    weight = weight.contiguous()
    r_ptr = h_ptr = v_ptr = None
    if residual is not None:
        if residual.dtype is not dt or residual.shape != shape or residual.get_device() != dev:
            raise ValueError(f"residual must be {dt} [M, K] on {x.device}")
        residual = residual.contiguous()
        r_ptr = residual.data_ptr()
        if h is None:
            h = torch.empty_like(residual)
    if h is not None:
        if h.dtype is not dt or h.shape != shape or h.get_device() != dev or not h.is_contiguous():
            raise ValueError(f"h must be a contiguous {dt} tensor [M, K] on {x.device}")
        h_ptr = h.data_ptr()
    if rows is None:
        rows = dq8ca_rows(M, K, x.device)
    elif rows.M != M or rows.K != K or rows.buffer.get_device() != dev:
        raise ValueError(f"rows must hold [{M}, {K}] on {x.device}")
    if values is not None:
        if values.dtype is not torch.float32 or values.shape != shape or values.get_device() != dev \
                or not values.is_contiguous():
            raise ValueError(f"values must be a contiguous fp32 tensor of shape {list(shape)} on {x.device}")
        v_ptr = values.data_ptr()
    buf = rows.buffer
    _check(lib().q4gsw_rmsnorm_dq8ca(x.data_ptr(), _TORCH_DTYPE[x.dtype], r_ptr, weight.data_ptr(), r_dtype, M, K, eps,
                                     h_ptr, buf.data_ptr(), buf.numel(), v_ptr, _stream()), "q4gsw_rmsnorm_dq8ca")
    return rows, h, values


def linear_dq8ca_rows(w: PackedWeight, rows: Dq8caRows, out: Optional[torch.Tensor] = None,
                      workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [M, N] fp32 = linear_dq8ca of rows that are quantised already."""
    if rows.K != w.K:
        raise ValueError("rows must have w.K columns")
    dev = rows.buffer.device
    y = _out(out, (rows.M, w.N), dev, "out")
    need = ctypes.c_uint64()
    _check(lib().q4gsw_dq8ca_rows_workspace_bytes_ex(w.ref(), rows.M, _opts(), ctypes.byref(need)),
           "q4gsw_dq8ca_rows_workspace_bytes")
    ws, wp, wb = _ws_args(need.value, workspace, dev)
    _check(lib().q4gsw_linear_dq8ca_rows_ex(w.ref(), rows.buffer.data_ptr(), rows.buffer.numel(), rows.M, y.data_ptr(),
                                            wp, wb, _opts(), _stream()), "q4gsw_linear_dq8ca_rows")
    return y


class KvCache:
    """A paged cache of keys and values in 4 bits: the descriptor and its device buffer."""

    def __init__(self, desc: KvCacheDesc, buffer: torch.Tensor):
        self.desc = desc
        self.buffer = buffer
        self.pages, self.page_size, self.heads, self.dim = desc.pages, desc.page_size, desc.heads, desc.dim
        self._ref = ctypes.byref(desc)
        self._addr = ctypes.addressof(desc)
        self._dev = buffer.get_device()


def _int32(*sizes: int) -> None:
    """ctypes takes integers modulo 2^32 without a word."""
    for n in sizes:
        if n >> 31 not in (0, -1):
            raise ValueError(f"{n} does not fit a 32-bit argument")


def kv_cache(pages: int, page_size: int, heads: int, dim: int, device="cuda") -> KvCache:
    """An empty cache (zeros) of `pages` pages of page_size tokens."""
    _int32(page_size, heads, dim)
    desc = KvCacheDesc(pages, page_size, heads, dim, 0, None, 0)
    out = ctypes.c_uint64()
    _check(lib().q4gsw_kv_bytes(ctypes.byref(desc), ctypes.byref(out)), "q4gsw_kv_bytes")
    buf = torch.zeros(out.value, dtype=torch.uint8, device=device)
    if not buf.is_cuda:
        raise ValueError("a cache lives on a GPU")
    desc.data, desc.bytes = buf.data_ptr(), out.value
    return KvCache(desc, buf)


# q4gsw_kv_seqs as packed bytes: a call's checks and marshalling cost as much as a small kernel, and
# building a Structure four times what packing its fields does.
_pack_seqs = struct.Struct("PqiiPPq").pack


def _kv_seqs(cache: KvCache, table: torch.Tensor, cu: torch.Tensor, lens: torch.Tensor, tokens: int) -> bytes:
    dev, i32 = cache._dev, torch.int32
    if lens.dtype is not i32 or lens.dim() != 1 or lens.get_device() != dev or not lens.is_contiguous() \
            or not lens.numel():
        raise ValueError(f"lens must be a contiguous int32 tensor [batch] on {cache.buffer.device}")
    B = lens.numel()
    if cu.dtype is not i32 or cu.dim() != 1 or cu.numel() != B + 1 or cu.get_device() != dev or not cu.is_contiguous():
        raise ValueError(f"cu must be a contiguous int32 tensor [batch + 1] on {cache.buffer.device}")
    if table.dtype is not i32 or table.dim() != 2 or table.get_device() != dev:
        raise ValueError(f"table must be an int32 tensor [batch, pages per sequence] on {cache.buffer.device}")
    n, cols = table.shape
    ld, step = table.stride()
    if n != B or (cols > 1 and step != 1):
        raise ValueError("table must have a dense row for each sequence")
    if B == 1:
        ld = cols
    elif ld < cols:
        raise ValueError("table's rows must not overlap")
    return _pack_seqs(table.data_ptr(), ld, cols, B, cu.data_ptr(), lens.data_ptr(), tokens)


def _token_rows(t: torch.Tensor, heads: int, cache: KvCache, name: str) -> Tuple[torch.Tensor, int, int, int]:
    """(tensor, its address, token pitch in elements, dtype code): `t` itself where its token rows are
    dense and 16-byte aligned (a slice of a fused projection's output, say), else a copy."""
    dim = cache.dim
    code = _TORCH_DTYPE.get(t.dtype)
    n, th, td = t.shape if t.dim() == 3 else (0, 0, 0)
    if th != heads or td != dim or code is None or t.get_device() != cache._dev:
        raise ValueError(f"{name} must be a floating tensor [tokens, {heads}, {dim}] on {cache.buffer.device}")
    ld, sh, sd = t.stride()
    row = heads * dim
    if n <= 1:
        ld = row
    ptr = t.data_ptr()
    if sd != 1 or (sh != dim and heads > 1) or ld < row or (ptr | ld * (4 if code == F32 else 2)) & 15:
        t = t.clone(memory_format=torch.contiguous_format)
        return t, t.data_ptr(), row, code
    return t, ptr, ld, code


def kv_append(cache: KvCache, k: torch.Tensor, v: torch.Tensor, table: torch.Tensor, cu: torch.Tensor,
              lens: torch.Tensor) -> None:
    """Store the keys and values k, v [tokens, heads, dim] of new tokens: rows cu[b] .. cu[b + 1] - 1
    are the last of sequence b's lens[b] tokens (with them), whose pages are table[b]."""
    done = _host.append(cache._addr, cache._dev, k, v, table, cu, lens)
    if done is not None:
        return _check(done, "q4gsw_kv_append")
    k, kp, k_ld, dt = _token_rows(k, cache.heads, cache, "k")
    v, vp, v_ld, v_dt = _token_rows(v, cache.heads, cache, "v")
    tokens = k.shape[0]
    if v_dt != dt or v.shape[0] != tokens:
        raise ValueError("k and v must have one dtype and one number of tokens")
    _check(lib().q4gsw_kv_append(cache._ref, _kv_seqs(cache, table, cu, lens, tokens), kp, k_ld, vp, v_ld, dt,
                                 _stream()), "q4gsw_kv_append")


def kv_read(cache: KvCache, table: torch.Tensor, cu: torch.Tensor, lens: torch.Tensor, tokens: int,
            out: Optional[Tuple[torch.Tensor, torch.Tensor]] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(k, v) fp32 [tokens, heads, dim]: what the cache stands for at the places kv_append with the
    same table, cu and lens writes."""
    if out is None:
        done = _host.read(cache._addr, cache._dev, table, cu, lens, tokens)
        if done is not None:
            return _done(done, "q4gsw_kv_read")
    seqs = _kv_seqs(cache, table, cu, lens, tokens)
    dev = cache.buffer.device
    shape = (tokens, cache.heads, cache.dim)
    k, v = out if out is not None else (None, None)
    k, v = _out(k, shape, dev, "k"), _out(v, shape, dev, "v")
    _check(lib().q4gsw_kv_read(cache._ref, seqs, k.data_ptr(), v.data_ptr(), _stream()), "q4gsw_kv_read")
    return k, v


def kv_attention_workspace_bytes(cache: KvCache, batch: int, tokens: int, hq: int, max_new: int, max_ctx: int) -> int:
    """Workspace of kv_attention calls with these sizes (any window)."""
    _int32(batch, hq, max_new, max_ctx)
    out = ctypes.c_uint64()
    _check(lib().q4gsw_kv_attention_workspace_bytes(cache._ref, batch, tokens, hq, max_new, max_ctx, ctypes.byref(out)),
           "q4gsw_kv_attention_workspace_bytes")
    return out.value


def kv_attention_plan(cache: KvCache, batch: int, tokens: int, hq: int, max_new: int, max_ctx: int,
                      dtype: torch.dtype, window: int = 0) -> dict:
    """How a kv_attention call with these sizes runs: the kernel ("few_rows" or "many_rows"), waves
    per workgroup and splits of the cache's length."""
    _int32(batch, hq, max_new, max_ctx, window)
    info = KvPlanInfo()
    _check(lib().q4gsw_kv_attention_plan(cache._ref, batch, tokens, hq, max_new, max_ctx, window, _TORCH_DTYPE[dtype],
                                         _local.kv, ctypes.byref(info)), "q4gsw_kv_attention_plan")
    return {"kernel": next(k for k, v in KV_KERNELS.items() if v == info.kernel), "waves": info.waves, "splits": info.splits}


def _per_row(t: torch.Tensor, n: int, dev: int, name: str) -> torch.Tensor:
    """`t` itself, or a dense copy: int32 [n] on the device of that index."""
    if t.dtype is not torch.int32 or t.dim() != 1 or t.numel() != n or t.get_device() != dev:
        raise ValueError(f"{name} must be an int32 tensor [{n}] on cuda:{dev}")
    return t if t.is_contiguous() else t.contiguous()


def _int_out(out: Optional[torch.Tensor], shape: Tuple[int, ...], device, name: str) -> torch.Tensor:
    if out is None:
        return torch.empty(shape, dtype=torch.int32, device=device)
    if out.dtype is not torch.int32 or tuple(out.shape) != shape or out.device != device or not out.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor of shape {list(shape)} on {device}")
    return out


def kv_attention(cache: KvCache, q: torch.Tensor, table: torch.Tensor, cu: torch.Tensor, lens: torch.Tensor,
                 max_new: int, max_ctx: int, window: int = 0, softcap: float = 0.0,
                 out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, parents: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out [tokens, hq, dim] of q's dtype: causal attention of the new tokens q over the cache, which
    holds their own keys and values already.  max_new and max_ctx bound the sequences' new tokens and
    lengths; window > 0 keeps the last `window` keys of each token, softcap > 0 caps the scores.  A row that
    sees no key gives zeros, else one whose query holds a NaN or an infinity gives NaN.  With `parents` the new tokens form a tree
    (kv_tree_attention)."""
    if _local.kv is None:
        done = _host.attention(cache._addr, cache._dev, q, parents, table, cu, lens, max_new, max_ctx, window, softcap, out, workspace)
        if done is not None:
            return _done(done, "q4gsw_kv_attention" if parents is None else "q4gsw_kv_tree_attention")
    if (max_new | max_ctx | window) >> 31:       # negative ones too, of which the library refuses the 32-bit ones
        _int32(max_new, max_ctx, window)
    if q.dim() != 3:
        raise ValueError("q must be [tokens, hq, dim]")
    shape = q.shape
    tokens, hq, _ = shape
    dt = q.dtype
    q, qp, q_ld, code = _token_rows(q, hq, cache, "q")
    if out is None:
        out = torch.empty(shape, dtype=dt, device=q.device)
    elif out.dtype is not dt or out.shape != shape or out.get_device() != cache._dev or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {dt} tensor [tokens, hq, dim] on {cache.buffer.device}")
    seqs = _kv_seqs(cache, table, cu, lens, tokens)
    if parents is not None:
        parents = _per_row(parents, tokens, cache._dev, "parents")
    if workspace is None:
        need = (kv_attention_workspace_bytes if parents is None else kv_tree_attention_workspace_bytes)(
            cache, lens.numel(), tokens, hq, max_new, max_ctx)
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    elif workspace.dtype is not torch.uint8 or workspace.get_device() != cache._dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {cache.buffer.device}")
    if parents is None:
        _check(lib().q4gsw_kv_attention_ex(cache._ref, seqs, qp, q_ld, code, hq, max_new, max_ctx, window, softcap,
                                           out.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                           _local.kv, _stream()), "q4gsw_kv_attention")
    else:
        _check(lib().q4gsw_kv_tree_attention_ex(cache._ref, seqs, parents.data_ptr(), qp, q_ld, code, hq, max_new, max_ctx,
                                                window, softcap, out.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                                _local.kv, _stream_of(cache._dev)), "q4gsw_kv_tree_attention")
    return out


def kv_tree_attention_workspace_bytes(cache: KvCache, batch: int, tokens: int, hq: int, max_new: int, max_ctx: int) -> int:
    """Workspace of kv_tree_attention calls with these sizes (any window)."""
    _int32(batch, hq, max_new, max_ctx)
    out = ctypes.c_uint64()
    _check(lib().q4gsw_kv_tree_attention_workspace_bytes(cache._ref, batch, tokens, hq, max_new, max_ctx, ctypes.byref(out)),
           "q4gsw_kv_tree_attention_workspace_bytes")
    return out.value


def kv_tree_attention(cache: KvCache, q: torch.Tensor, parents: torch.Tensor, table: torch.Tensor, cu: torch.Tensor,
                      lens: torch.Tensor, max_new: int, max_ctx: int, window: int = 0, softcap: float = 0.0,
                      out: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """kv_attention of drafted tokens that form a tree: parents (int32 [tokens]) of the row of a sequence's
    node i is its parent's number in the sequence's new tokens, below i; any other value makes it a root.
    A node sees the tokens before the tree, its ancestors and itself; with window > 0 those whose position
    is above its own - window, a node's position being that of the tree's start + its depth.  max_new is
    at most 512."""
    if parents is None:
        raise ValueError("parents must be given")
    return kv_attention(cache, q, table, cu, lens, max_new, max_ctx, window, softcap, out, workspace, parents)


def kv_keep(caches, parents: torch.Tensor, leaf: torch.Tensor, table: torch.Tensor, cu: torch.Tensor, lens: torch.Tensor,
            max_new: int, kept: Optional[torch.Tensor] = None,
            path: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(kept, path) int32 [batch], [batch, max_new]: the nodes on the way from a root of sequence b's tree to
    node leaf[b] (int32 [batch]; outside the tree: none) move to the places behind the tokens before the tree,
    in `caches` (a KvCache, or a sequence of up to 128 of one shape that share the table).  kept: the tokens
    that each sequence has then; path: the nodes moved, in order, then -1."""
    caches = (caches,) if isinstance(caches, KvCache) else tuple(caches)
    if not caches:
        raise ValueError("caches must hold at least one cache")
    first = caches[0]
    for c in caches:
        if c._dev != first._dev:
            raise ValueError("caches must be on one device")
    done = _host.keep([c._addr for c in caches], first._dev, parents, leaf, table, cu, lens, max_new, kept, path)
    if done is not None:
        return _done(done, "q4gsw_kv_keep")
    _int32(max_new)
    if max_new < 1:
        raise ValueError("max_new must be positive")
    if parents.dim() != 1:
        raise ValueError("parents must be an int32 tensor [tokens]")
    tokens = parents.numel()
    parents = _per_row(parents, tokens, first._dev, "parents")
    seqs = _kv_seqs(first, table, cu, lens, tokens)
    B = lens.numel()
    leaf = _per_row(leaf, B, first._dev, "leaf")
    dev = first.buffer.device
    kept, path = _int_out(kept, (B,), dev, "kept"), _int_out(path, (B, max_new), dev, "path")
    descs = first._ref if len(caches) == 1 else (KvCacheDesc * len(caches))(*[c.desc for c in caches])
    _check(lib().q4gsw_kv_keep(descs, len(caches), seqs, parents.data_ptr(), leaf.data_ptr(), max_new, kept.data_ptr(),
                               path.data_ptr(), _stream_of(first._dev)), "q4gsw_kv_keep")
    return kept, path


# q4gsw_logits_rules as packed bytes, as with the sequences.
_pack_rules = struct.Struct("iiPPqiiPPPPPPPPPqPq").pack


def _table(t: torch.Tensor, dtype: torch.dtype, rows: int, dev: int, name: str) -> Tuple[int, int, int]:
    """(address, row pitch, columns) of a [rows, columns] tensor of dense rows."""
    if t.dtype is not dtype or t.dim() != 2 or t.shape[0] != rows or t.get_device() != dev:
        raise ValueError(f"{name} must be a {dtype} tensor [{rows}, columns] on cuda:{dev}")
    cols = t.shape[1]
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{name} must have dense rows")
    if rows <= 1:
        ld = cols
    elif ld < cols:
        raise ValueError(f"{name}'s rows must not overlap")
    return t.data_ptr(), ld, cols


def logits_adjust(logits: torch.Tensor, cu: Optional[torch.Tensor] = None, max_new: int = 1,
                  history: Optional[torch.Tensor] = None, history_lens: Optional[torch.Tensor] = None,
                  prompt_lens: Optional[torch.Tensor] = None, ids: Optional[torch.Tensor] = None,
                  parents: Optional[torch.Tensor] = None, repetition: Optional[torch.Tensor] = None,
                  presence: Optional[torch.Tensor] = None, frequency: Optional[torch.Tensor] = None,
                  bias_ids: Optional[torch.Tensor] = None, bias: Optional[torch.Tensor] = None,
                  mask: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out [rows, V] of logits' dtype (may be logits itself): x of a token seen so far divided by repetition
    where it is positive, else multiplied; of one generated n times lowered by frequency n + presence; bias
    added; -inf where the mask does not allow it.

    Row r is sequence r's, or with cu (int32 [batch + 1]) rows cu[b] .. cu[b + 1] - 1 are sequence b's, of which
    those past max_new and those of no sequence are left as they are.  Per sequence: history (int32 [batch,
    columns]; the first history_lens[b] tokens, prompt_lens[b] of them only seen), repetition, presence and
    frequency (fp32 [batch]), bias_ids (int32 [batch, columns]) with bias (fp32): of entries with one token the
    last counts.  Per row: ids (int32 [rows]), the rows' own tokens, which count as generated with those of the
    rows before them in the sequence, or with parents (as in kv_tree_attention) with those of their
    ancestors; mask (int32 [rows, ceil(V / 32)]), bit v % 32 of word v // 32 allows token v."""
    done = _host.logits(logits, cu, max_new, history, history_lens, prompt_lens, ids, parents, repetition, presence, frequency,
                        bias_ids, bias, mask, out)
    if done is not None:
        return _done(done, "q4gsw_logits_adjust")
    code = _TORCH_DTYPE.get(logits.dtype)
    dev = logits.get_device()
    if logits.dim() != 2 or code is None or dev < 0:
        raise ValueError("logits must be a floating GPU tensor [rows, V]")
    rows, V = logits.shape
    if out is None:
        out = torch.empty(rows, V, dtype=logits.dtype, device=logits.device)
    elif out.dtype is not logits.dtype or out.shape != logits.shape or out.get_device() != dev:
        raise ValueError(f"out must be a {logits.dtype} tensor [{rows}, {V}] on cuda:{dev}")
    pitches = []
    for t, name in ((logits, "logits"), (out, "out")):
        ld, step = t.stride()
        if rows <= 1:
            ld = V
        if (V > 1 and step != 1) or ld < V:
            raise ValueError(f"{name} must have dense rows")
        pitches.append(ld)
    batch, cp = rows, None
    if cu is not None:
        if cu.dim() != 1 or cu.numel() < 2:
            raise ValueError("cu must be an int32 tensor [batch + 1]")
        batch = cu.numel() - 1
        cu = _per_row(cu, batch + 1, dev, "cu")
        cp = cu.data_ptr()
    _int32(max_new)
    keep = [cu]                                       # dense copies live until the launch
    def one(t, n, name, dtype=torch.int32):
        if t is None:
            return None
        if t.dtype is not dtype or t.dim() != 1 or t.numel() != n or t.get_device() != dev:
            raise ValueError(f"{name} must be a {dtype} tensor [{n}] on cuda:{dev}")
        if not t.is_contiguous():
            t = t.contiguous()
            keep.append(t)
        return t.data_ptr()
    hp = bp = vp = mp = None
    h_ld = h_cols = b_ld = b_cols = m_ld = 0
    if history is not None:
        hp, h_ld, h_cols = _table(history, torch.int32, batch, dev, "history")
        if history_lens is None:
            raise ValueError("history needs history_lens")
    if (bias_ids is None) != (bias is None):
        raise ValueError("bias_ids and bias go together")
    if bias is not None:
        bp, b_ld, b_cols = _table(bias_ids, torch.int32, batch, dev, "bias_ids")
        vp, v_ld, v_cols = _table(bias, torch.float32, batch, dev, "bias")
        if v_cols != b_cols or v_ld != b_ld:
            raise ValueError("bias must have bias_ids' shape and strides")
    if mask is not None:
        mp, m_ld, m_cols = _table(mask, torch.int32, rows, dev, "mask")
        if m_cols < (V + 31) // 32:
            raise ValueError("mask must have a bit for every token")
    if parents is not None and (ids is None or cu is None):
        raise ValueError("parents need ids and cu")
    f32 = torch.float32
    rules = _pack_rules(batch, max_new, cp or 0, hp or 0, h_ld, h_cols, b_cols, one(history_lens, batch, "history_lens") or 0,
                        one(prompt_lens, batch, "prompt_lens") or 0, one(ids, rows, "ids") or 0,
                        one(parents, rows, "parents") or 0, one(repetition, batch, "repetition", f32) or 0,
                        one(presence, batch, "presence", f32) or 0, one(frequency, batch, "frequency", f32) or 0, bp or 0,
                        vp or 0, b_ld, mp or 0, m_ld)
    _check(lib().q4gsw_logits_adjust(logits.data_ptr(), code, rows, V, pitches[0], rules, out.data_ptr(), pitches[1],
                                     _stream_of(dev)), "q4gsw_logits_adjust")
    return out


def adapter_workspace_bytes(op: int, w: PackedWeight, M: int, dtype: torch.dtype, rank: int) -> int:
    out = ctypes.c_uint64()
    _check(lib().q4gsw_adapter_workspace_bytes(op, w.ref(), M, _TORCH_DTYPE[dtype], rank, ctypes.byref(out)),
           "q4gsw_adapter_workspace_bytes")
    return out.value


def _factor(t: torch.Tensor, shape: Tuple[int, int], device, name: str) -> torch.Tensor:
    if t.dtype != torch.float32 or tuple(t.shape) != tuple(shape) or t.device != device:
        raise ValueError(f"{name} must be an fp32 tensor of shape {list(shape)} on {device}")
    return t.contiguous()


def adapter_fwd(w: PackedWeight, x: torch.Tensor, A: torch.Tensor, B: torch.Tensor, alpha: float,
                out: Optional[torch.Tensor] = None, t: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """(y [M, N], t [M, r]) = (x . dequant(W)^T + alpha (x A^T) B^T, x A^T) for the low-rank
    adapter A [r, K], B [N, r] (fp32) beside the frozen weight."""
    x = _dev(x, "x")
    if x.dim() != 2 or x.shape[1] != w.K:
        raise ValueError("x must be [M, K]")
    M, r = x.shape[0], A.shape[0]
    A = _factor(A, (r, w.K), x.device, "A")
    B = _factor(B, (w.N, r), x.device, "B")
    y = _out(out, (M, w.N), x.device, "out")
    t = _out(t, (M, r), x.device, "t")
    need = adapter_workspace_bytes(OP_FWD, w, M, x.dtype, r)
    ws, wp, wb = _ws_args(need, workspace, x.device)
    _check(lib().q4gsw_adapter_fwd(w.ref(), x.data_ptr(), _TORCH_DTYPE[x.dtype], M, A.data_ptr(), B.data_ptr(), r,
                                   float(alpha), y.data_ptr(), t.data_ptr(), wp, wb, _stream()), "q4gsw_adapter_fwd")
    return y, t


def adapter_bwd(w: PackedWeight, x: torch.Tensor, d_out: torch.Tensor, A: torch.Tensor, B: torch.Tensor,
                alpha: float, t: torch.Tensor, d_x: Optional[torch.Tensor] = None,
                d_A: Optional[torch.Tensor] = None, d_B: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(d_x [M, K], d_A [r, K], d_B [N, r]): the gradients of <d_out, y> for the adapter forward of
    the same x (t is its x A^T)."""
    x = _dev(x, "x")
    d_out = _dev(d_out, "d_out")
    if x.dim() != 2 or x.shape[1] != w.K or d_out.shape != (x.shape[0], w.N) or d_out.dtype != x.dtype:
        raise ValueError("x must be [M, K] and d_out [M, N] of x's dtype")
    M, r = x.shape[0], A.shape[0]
    A = _factor(A, (r, w.K), x.device, "A")
    B = _factor(B, (w.N, r), x.device, "B")
    t = _factor(t, (M, r), x.device, "t")
    dx = _out(d_x, (M, w.K), x.device, "d_x")
    dA = _out(d_A, (r, w.K), x.device, "d_A")
    dB = _out(d_B, (w.N, r), x.device, "d_B")
    need = adapter_workspace_bytes(OP_BWD_INPUT, w, M, x.dtype, r)
    ws, wp, wb = _ws_args(need, workspace, x.device)
    _check(lib().q4gsw_adapter_bwd(w.ref(), x.data_ptr(), d_out.data_ptr(), _TORCH_DTYPE[x.dtype], M, A.data_ptr(),
                                   B.data_ptr(), r, float(alpha), t.data_ptr(), dx.data_ptr(), dA.data_ptr(),
                                   dB.data_ptr(), wp, wb, _stream()), "q4gsw_adapter_bwd")
    return dx, dA, dB


class Adapters:
    """Low-rank adapters in the slots of one set: the descriptor and its device buffer."""

    def __init__(self, desc: AdaptersDesc, buffer: torch.Tensor):
        self.desc = desc
        self.buffer = buffer
        self.slots, self.rank, self.N, self.K = desc.slots, desc.rank, desc.N, desc.K
        self._ref = ctypes.byref(desc)
        self._addr = ctypes.addressof(desc)
        self._dev = buffer.get_device()


def adapters(slots: int, rank: int, N: int, K: int, dtype: torch.dtype = torch.bfloat16, device="cuda") -> Adapters:
    """An empty set (no slot adds anything) of `slots` adapters of up to `rank` beside a projection [N, K], its
    factors held in `dtype` (bf16 or fp16)."""
    _int32(slots, rank)
    if dtype not in (torch.float16, torch.bfloat16):
        raise ValueError("dtype must be torch.float16 or torch.bfloat16")
    desc = AdaptersDesc(N, K, slots, rank, _TORCH_DTYPE[dtype], 0, None, 0)
    out = ctypes.c_uint64()
    _check(lib().q4gsw_adapters_bytes(ctypes.byref(desc), ctypes.byref(out)), "q4gsw_adapters_bytes")
    buf = torch.zeros(out.value, dtype=torch.uint8, device=device)
    if not buf.is_cuda:
        raise ValueError("a set of adapters lives on a GPU")
    desc.data, desc.bytes = buf.data_ptr(), out.value
    return Adapters(desc, buf)


def adapters_load(s: Adapters, slot: int, A: torch.Tensor, B: torch.Tensor, alpha: float) -> None:
    """The adapter A [r, K], B [N, r] (r up to the set's rank; rounded once to its type), scaled by alpha, into a
    slot."""
    _int32(slot)
    r = A.shape[0] if A.dim() == 2 else 0
    code = _TORCH_DTYPE.get(A.dtype)
    if tuple(A.shape) != (r, s.K) or tuple(B.shape) != (s.N, r) or code is None or B.dtype is not A.dtype \
            or A.get_device() != s._dev or B.get_device() != s._dev:
        raise ValueError(f"A must be [r, {s.K}] and B [{s.N}, r], of one floating type, on {s.buffer.device}")
    A, B = A.contiguous(), B.contiguous()
    _check(lib().q4gsw_adapters_load(s._ref, slot, A.data_ptr(), B.data_ptr(), code, r, float(alpha), _stream_of(s._dev)),
           "q4gsw_adapters_load")


def adapters_workspace_bytes(s: Adapters, M: int, dtype: torch.dtype, w: Optional[PackedWeight] = None) -> int:
    """Workspace of adapters_fwd with the weight w, or of adapters_add, on M rows of `dtype`."""
    out = ctypes.c_uint64()
    _check(lib().q4gsw_adapters_workspace_bytes(s._ref, w.ref() if w is not None else None, M, _TORCH_DTYPE[dtype],
                                                ctypes.byref(out)), "q4gsw_adapters_workspace_bytes")
    return out.value


def _adapter_rows(x: torch.Tensor, s: Adapters, slots: torch.Tensor) -> Tuple[torch.Tensor, int, torch.Tensor, int]:
    code = _TORCH_DTYPE.get(x.dtype)
    if x.dim() != 2 or x.shape[1] != s.K or code is None or x.get_device() != s._dev:
        raise ValueError(f"x must be a floating tensor [M, {s.K}] on {s.buffer.device}")
    M = x.shape[0]
    return x.contiguous(), code, _per_row(slots, M, s._dev, "slots"), M


def adapters_fwd(w: PackedWeight, x: torch.Tensor, s: Adapters, slots: torch.Tensor, out: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """y [M, N] fp32: y[m] = x[m] . dequant(W)^T + alpha_i (x[m] A_i^T) B_i^T for the adapter in slot i = slots[m]
    (int32 [M]; outside the set's slots: none)."""
    if w.buffer.get_device() != s._dev:
        raise ValueError(f"w must be on {s.buffer.device}")
    done = _host.adapters(ctypes.addressof(w.desc), s._addr, s._dev, x, slots, None, out, workspace)
    if done is not None:
        return _done(done, "q4gsw_adapters_fwd")
    x, code, slots, M = _adapter_rows(x, s, slots)
    y = _out(out, (M, s.N), x.device, "out")
    need = adapters_workspace_bytes(s, M, x.dtype, w)
    ws, wp, wb = _ws_args(need, workspace, x.device)
    _check(lib().q4gsw_adapters_fwd(w.ref(), s._ref, x.data_ptr(), code, M, slots.data_ptr(), y.data_ptr(), wp, wb,
                                    _stream_of(s._dev)), "q4gsw_adapters_fwd")
    return y


def adapters_add(y: torch.Tensor, x: torch.Tensor, s: Adapters, slots: torch.Tensor, out: Optional[torch.Tensor] = None,
                 workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out [M, N] fp32: y[m] (fp32; a projection of the same rows) + alpha_i (x[m] A_i^T) B_i^T for the adapter in
    slot i = slots[m].  `out` may be y itself."""
    done = _host.adapters(None, s._addr, s._dev, x, slots, y, out, workspace)
    if done is not None:
        return _done(done, "q4gsw_adapters_add")
    x, code, slots, M = _adapter_rows(x, s, slots)
    if y.dtype is not torch.float32 or tuple(y.shape) != (M, s.N) or y.get_device() != s._dev:
        raise ValueError(f"y must be an fp32 tensor [{M}, {s.N}] on {s.buffer.device}")
    if out is not y:
        y = y.contiguous()
    out = _out(out, (M, s.N), x.device, "out")
    need = adapters_workspace_bytes(s, M, x.dtype)
    ws, wp, wb = _ws_args(need, workspace, x.device)
    _check(lib().q4gsw_adapters_add(s._ref, x.data_ptr(), code, M, slots.data_ptr(), y.data_ptr(), out.data_ptr(), wp, wb,
                                    _stream_of(s._dev)), "q4gsw_adapters_add")
    return out


def adamw_step(param: torch.Tensor, grad: torch.Tensor, exp_avg: torch.Tensor, exp_avg_sq: torch.Tensor,
               step: int, lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
               weight_decay: float = 0.01) -> None:
    """One AdamW step in place on contiguous fp32 GPU tensors of one size (param, exp_avg and
    exp_avg_sq are updated)."""
    ts = [param, grad, exp_avg, exp_avg_sq]
    n = param.numel()
    for name, tt in zip(("param", "grad", "exp_avg", "exp_avg_sq"), ts):
        if tt.dtype != torch.float32 or not tt.is_contiguous() or tt.numel() != n or tt.device != param.device \
                or not tt.is_cuda:
            raise ValueError(f"{name} must be a contiguous fp32 GPU tensor of {n} elements on {param.device}")
    hp = AdamwParams(lr, beta1, beta2, eps, weight_decay)
    _check(lib().q4gsw_adamw_step(param.data_ptr(), grad.data_ptr(), exp_avg.data_ptr(), exp_avg_sq.data_ptr(), n,
                                  ctypes.byref(hp), int(step), _stream()), "q4gsw_adamw_step")


def embedding(w: PackedWeight, ids: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out [*ids.shape, K] fp32: entry ids[i] gives row ids[i] of dequant(W) (zeros outside [0, N))."""
    ids = _dev(ids, "ids")
    if ids.dtype != torch.int64:
        raise ValueError("ids must be int64")
    T = ids.numel()
    o = out if out is not None else torch.empty(*ids.shape, w.K, dtype=torch.float32, device=ids.device)
    if o.dtype != torch.float32 or not o.is_contiguous() or o.numel() != T * w.K or o.device != ids.device:
        raise ValueError("out must be a contiguous fp32 tensor of ids.numel() * K elements on ids' device")
    _check(lib().q4gsw_embedding(w.ref(), ids.data_ptr(), T, o.data_ptr(), _stream()), "q4gsw_embedding")
    return o


def qkv_workspace_bytes(wq: PackedWeight, wk: PackedWeight, wv: PackedWeight, M: int, dtype: torch.dtype) -> int:
    out = ctypes.c_uint64()
    _check(lib().q4gsw_qkv_workspace_bytes_ex(wq.ref(), wk.ref(), wv.ref(), M, _TORCH_DTYPE[dtype], _opts(),
                                              ctypes.byref(out)), "q4gsw_qkv_workspace_bytes")
    return out.value


def qkv_fused(wq: PackedWeight, wk: PackedWeight, wv: PackedWeight, x: torch.Tensor,
              outs: Optional[Tuple[torch.Tensor, torch.Tensor, torch.Tensor]] = None,
              workspace: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """(q, k, v) fp32 = x . dequant(Wq)^T, x . dequant(Wk)^T, x . dequant(Wv)^T in one call."""
    x = _dev(x, "x")
    if x.dim() != 2 or x.shape[1] != wq.K:
        raise ValueError("x must be [M, K]")
    M = x.shape[0]
    if outs is None:
        outs = (None, None, None)
    if len(outs) != 3:
        raise ValueError("outs must be three tensors (q, k, v)")
    q, k, v = (_out(o, (M, w.N), x.device, name) for o, w, name in zip(outs, (wq, wk, wv), ("q", "k", "v")))
    need = qkv_workspace_bytes(wq, wk, wv, M, x.dtype)
    ws, wp, wb = _ws_args(need, workspace, x.device)
    _check(lib().q4gsw_qkv_fused_ex(wq.ref(), wk.ref(), wv.ref(), x.data_ptr(), _TORCH_DTYPE[x.dtype], M,
                                    q.data_ptr(), k.data_ptr(), v.data_ptr(), wp, wb, _opts(), _stream()),
           "q4gsw_qkv_fused")
    return q, k, v


def route(op: int, w: PackedWeight, M: int, dtype: torch.dtype) -> str:
    """The route a call with these arguments takes (under this thread's forced route, if any).  For
    OP_QKV the route depends on Wq only."""
    o = _opts()
    if o is None:
        return route_name(lib().q4gsw_route(op, w.ref(), M, _TORCH_DTYPE[dtype]))
    info = PlanInfo()
    extra = w.ref() if op == OP_QKV else None
    _check(lib().q4gsw_plan(op, w.ref(), extra, extra, M, _TORCH_DTYPE[dtype], o, ctypes.byref(info)), "q4gsw_plan")
    return route_name(info.route)


def plan(op: int, w: PackedWeight, M: int, dtype: torch.dtype, wk: PackedWeight = None,
         wv: PackedWeight = None) -> dict:
    """How a call runs: route name, MFMA block rows and contraction splits.  For OP_QKV pass wk
    and wv."""
    info = PlanInfo()
    refs = [x.ref() if x is not None else None for x in (wk, wv)]
    _check(lib().q4gsw_plan(op, w.ref(), refs[0], refs[1], M, _TORCH_DTYPE[dtype], _opts(), ctypes.byref(info)),
           "q4gsw_plan")
    return {"route": route_name(info.route), "tile_rows": info.tile_rows, "splits": info.splits}


@contextlib.contextmanager
def _with_options(**fields):
    """Set fields of this thread's per-call options for the calls inside the block."""
    old = _local.opts
    new = Options()
    if old is not None:
        ctypes.memmove(ctypes.byref(new), ctypes.byref(old), ctypes.sizeof(Options))
    for k, v in fields.items():
        setattr(new, k, v)
    _local.opts = new
    try:
        yield
    finally:
        _local.opts = old


@contextlib.contextmanager
def forced_plan(tile_rows: int = 0, splits: int = 0):
    """Pin the forward / QKV MFMA block rows (64 or 128) and the contraction splits (the split
    count also governs the 32x32 input-gradient routes) of the calls made by this thread inside the
    block; 0 leaves a choice per shape.  Out-of-range values raise ValueError."""
    if tile_rows not in (0, 64, 128) or not 0 <= splits <= 64:
        raise ValueError("tile_rows must be 0, 64 or 128 and splits 0..64")
    with _with_options(tile_rows=tile_rows, splits=splits):
        yield


@contextlib.contextmanager
def forced_route(name: str):
    """Send the calls made by this thread inside the block onto one route family (tests and
    benchmarks); a call the family cannot serve raises Q4gswError with E_ROUTE."""
    with _with_options(route=ROUTES[name]):
        yield


@contextlib.contextmanager
def forced_kv_kernel(name: str):
    """Send the kv_attention calls made by this thread inside the block to one kernel, "few_rows" or
    "many_rows", or the kv_tree_attention calls to either or to "tree" (tests and benchmarks); Q4gswError with E_ROUTE where it cannot serve a call."""
    old = _local.kv
    _local.kv = ctypes.pointer(KvOptions(KV_KERNELS[name], 0))
    try:
        yield
    finally:
        _local.kv = old


def build_info() -> str:
    return lib().q4gsw_build_info().decode()
