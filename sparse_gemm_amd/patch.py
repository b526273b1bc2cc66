"""Python binding of libpatch.so (C ABI in include/patch.h).

Argument marshalling only: every step of the hybrid GEMM runs in the HIP
kernels behind the C ABI.  torch provides device memory and the current HIP
stream; nothing here computes on the CPU, and there is no fallback -- if the
library is missing, every call raises.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
import struct
from typing import Optional

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpatch.so")

PATCH_F16, PATCH_BF16, PATCH_F32 = 0, 1, 2
VARIANTS = {"auto": 0, "decode": 1, "prefill": 2, "prefill_w64": 3, "prefill_w128": 4, "prefill_w192": 5,
            "prefill_w256": 6, "prefill_w128_lds": 7, "prefill_w192_lds": 8, "prefill_w256_lds": 9,
            "prefill_w64_lds": 10, "prefill_big": 11, "prefill_big_w128": 12, "prefill_big_w192": 13,
            "prefill_big_w256": 14, "prefill_big8_w128": 15, "prefill_big8_w256": 16}
STATUS = {0: "PATCH_OK", 1: "PATCH_ERR_INVALID_ARG", 2: "PATCH_ERR_SHAPE", 3: "PATCH_ERR_MASK",
          4: "PATCH_ERR_BUFFER_TOO_SMALL", 5: "PATCH_ERR_UNSUPPORTED", 6: "PATCH_ERR_HIP"}

_TORCH_DT = {torch.float16: PATCH_F16, torch.bfloat16: PATCH_BF16, torch.float32: PATCH_F32}
_DT_TORCH = {PATCH_F16: torch.float16, PATCH_BF16: torch.bfloat16, PATCH_F32: torch.float32}


class PatchError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"{STATUS.get(status, status)}: {detail}")
        self.status = status
        self.name = STATUS.get(status, str(status))


class Desc(ctypes.Structure):
    _fields_ = [("version", ctypes.c_uint32), ("dtype", ctypes.c_uint32), ("tile_n", ctypes.c_uint32),
                ("tile_k", ctypes.c_uint32), ("N", ctypes.c_uint32), ("K", ctypes.c_uint32),
                ("nt_n", ctypes.c_uint32), ("nt_k", ctypes.c_uint32), ("n_sparse", ctypes.c_uint32),
                ("n_48", ctypes.c_uint32), ("table_offset", ctypes.c_uint64), ("data_offset", ctypes.c_uint64),
                ("total_bytes", ctypes.c_uint64)]


EXPORTS = ("patch_abi_version", "patch_packed_bytes", "patch_pack", "patch_packed_bytes_q64", "patch_pack_q64",
           "patch_desc_from_header",
           "patch_gemm_workspace_bytes", "patch_dense_gemm_workspace_bytes", "patch_gemm", "patch_gemm_ex",
           "patch_dense_gemm", "patch_dense_gemm_ex", "patch_packed_bytes_gate_up", "patch_pack_gate_up",
           "patch_gemm_swiglu_workspace_bytes", "patch_gemm_swiglu", "patch_dense_gemm_swiglu_workspace_bytes",
           "patch_dense_gemm_swiglu", "patch_packed_bytes_concat", "patch_pack_concat", "patch_sample_mask",
           "patch_exec_tile_map", "patch_apply_fine_mask", "patch_probe_stream_read", "patch_probe_matrix_rate", "patch_probe_copy_rate", "patch_probe_copy_bytes",
           "patch_debug_tail_wait",
           "patch_probe_matrix_flops", "patch_noalloc_scratch_bytes", "patch_gemm_noalloc", "patch_rope_table",
           "patch_rope", "patch_kv_append", "patch_attention_workspace_bytes", "patch_attention", "patch_w4_bytes",
           "patch_w4_quantize", "patch_w4_pack", "patch_w4_gemm", "patch_status_string", "patch_last_error")

_lib = None


def load():
    """Load libpatch.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python -m sparse_gemm_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I64, U64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint64, ctypes.c_int32
    DP = ctypes.POINTER(Desc)
    lib.patch_abi_version.argtypes = []
    lib.patch_abi_version.restype = I32
    lib.patch_packed_bytes.argtypes = [ctypes.c_int, I64, I64, P]
    lib.patch_packed_bytes.restype = U64
    lib.patch_pack.argtypes = [ctypes.c_int, I64, I64, P, P, P, P, U64, DP, P]
    lib.patch_pack.restype = ctypes.c_int
    lib.patch_packed_bytes_q64.argtypes = [ctypes.c_int, I64, I64, P]
    lib.patch_packed_bytes_q64.restype = U64
    lib.patch_pack_q64.argtypes = [ctypes.c_int, I64, I64, P, P, P, P, U64, DP, P]
    lib.patch_pack_q64.restype = ctypes.c_int
    lib.patch_desc_from_header.argtypes = [P, U64, DP]
    lib.patch_desc_from_header.restype = ctypes.c_int
    lib.patch_gemm_workspace_bytes.argtypes = [DP, I64]
    lib.patch_gemm_workspace_bytes.restype = U64
    lib.patch_dense_gemm_workspace_bytes.argtypes = [I64, I64, I64]
    lib.patch_dense_gemm_workspace_bytes.restype = U64
    lib.patch_gemm.argtypes = [DP, P, P, I64, P, ctypes.c_int, P, U64, P]
    lib.patch_gemm.restype = ctypes.c_int
    lib.patch_gemm_ex.argtypes = [DP, P, P, I64, P, ctypes.c_int, P, U64, I32, P]
    lib.patch_gemm_ex.restype = ctypes.c_int
    lib.patch_dense_gemm.argtypes = [ctypes.c_int, I64, I64, I64, P, P, P, ctypes.c_int, P, U64, P]
    lib.patch_dense_gemm.restype = ctypes.c_int
    lib.patch_dense_gemm_ex.argtypes = [ctypes.c_int, I64, I64, I64, P, P, P, ctypes.c_int, P, U64, I32, P]
    lib.patch_dense_gemm_ex.restype = ctypes.c_int
    lib.patch_packed_bytes_gate_up.argtypes = [ctypes.c_int, I64, I64, P, P]
    lib.patch_packed_bytes_gate_up.restype = U64
    lib.patch_pack_gate_up.argtypes = [ctypes.c_int, I64, I64, P, P, P, P, P, P, P, U64, DP, P]
    lib.patch_pack_gate_up.restype = ctypes.c_int
    lib.patch_gemm_swiglu_workspace_bytes.argtypes = [DP, I64]
    lib.patch_gemm_swiglu_workspace_bytes.restype = U64
    lib.patch_gemm_swiglu.argtypes = [DP, P, P, I64, P, ctypes.c_int, P, U64, I32, P]
    lib.patch_gemm_swiglu.restype = ctypes.c_int
    lib.patch_dense_gemm_swiglu_workspace_bytes.argtypes = [I64, I64, I64]
    lib.patch_dense_gemm_swiglu_workspace_bytes.restype = U64
    lib.patch_dense_gemm_swiglu.argtypes = [ctypes.c_int, I64, I64, I64, P, P, P, P, ctypes.c_int, P, U64, I32, P]
    lib.patch_dense_gemm_swiglu.restype = ctypes.c_int
    lib.patch_packed_bytes_concat.argtypes = [ctypes.c_int, I32, P, I64, P]
    lib.patch_packed_bytes_concat.restype = U64
    lib.patch_pack_concat.argtypes = [ctypes.c_int, I32, P, I64, P, P, P, P, U64, DP, P]
    lib.patch_pack_concat.restype = ctypes.c_int
    lib.patch_sample_mask.argtypes = [I64, I64, P, P, P, P, ctypes.c_float, P, P, P, P]
    lib.patch_sample_mask.restype = ctypes.c_int
    lib.patch_exec_tile_map.argtypes = [I64, I64, I64, I64, P, P, ctypes.POINTER(I64)]
    lib.patch_exec_tile_map.restype = ctypes.c_int
    lib.patch_apply_fine_mask.argtypes = [ctypes.c_int, I64, I64, I64, I64, P, P, P, P, P]
    lib.patch_apply_fine_mask.restype = ctypes.c_int
    lib.patch_probe_stream_read.argtypes = [P, U64, P, U64, P]
    lib.patch_probe_stream_read.restype = ctypes.c_int
    lib.patch_probe_matrix_rate.argtypes = [I32, I32, I32, P, P]
    lib.patch_probe_matrix_rate.restype = ctypes.c_int
    lib.patch_probe_matrix_flops.argtypes = [I32, I32, I32]
    lib.patch_probe_matrix_flops.restype = U64
    lib.patch_probe_copy_rate.argtypes = [P, U64, U64, I32, I32, P, U64, P]
    lib.patch_probe_copy_rate.restype = ctypes.c_int
    lib.patch_probe_copy_bytes.argtypes = [I32, I32]
    lib.patch_probe_copy_bytes.restype = U64
    lib.patch_debug_tail_wait.argtypes = [I32]
    lib.patch_debug_tail_wait.restype = None
    lib.patch_noalloc_scratch_bytes.argtypes = []
    lib.patch_noalloc_scratch_bytes.restype = U64
    lib.patch_gemm_noalloc.argtypes = [DP, P, P, I64, P, ctypes.c_int, P]
    lib.patch_gemm_noalloc.restype = ctypes.c_int
    F64 = ctypes.c_double
    lib.patch_rope_table.argtypes = [I64, I64, F64, I32, F64, F64, F64, F64, F64, P, P]
    lib.patch_rope_table.restype = ctypes.c_int
    lib.patch_rope.argtypes = [P, P]
    lib.patch_rope.restype = ctypes.c_int
    lib.patch_kv_append.argtypes = [P, P, P]
    lib.patch_kv_append.restype = ctypes.c_int
    lib.patch_attention_workspace_bytes.argtypes = [I64, I64, I64, I64, I64]
    lib.patch_attention_workspace_bytes.restype = U64
    lib.patch_attention.argtypes = [P, P, P, U64, P]
    lib.patch_attention.restype = ctypes.c_int
    lib.patch_w4_bytes.argtypes = [I64, I64, I64, I32]
    lib.patch_w4_bytes.restype = U64
    lib.patch_w4_quantize.argtypes = [ctypes.c_int, I64, I64, I64, P, P, P, P, P]
    lib.patch_w4_quantize.restype = ctypes.c_int
    lib.patch_w4_pack.argtypes = [ctypes.c_int, I64, I64, I64, P, P, P, P, U64, P]
    lib.patch_w4_pack.restype = ctypes.c_int
    lib.patch_w4_gemm.argtypes = [ctypes.c_int, I64, I64, I64, I32, P, U64, P, I64, P, ctypes.c_int, P]
    lib.patch_w4_gemm.restype = ctypes.c_int
    lib.patch_status_string.argtypes = [ctypes.c_int]
    lib.patch_status_string.restype = ctypes.c_char_p
    lib.patch_last_error.argtypes = []
    lib.patch_last_error.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _check(rc: int):
    if rc != 0:
        raise PatchError(rc, load().patch_last_error().decode())


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(device_index: Optional[int] = None) -> int:
    """The current HIP stream of the device, as an integer handle."""
    if _raw_stream is not None:
        return _raw_stream(torch.cuda.current_device() if device_index is None else device_index)
    return torch.cuda.current_stream().cuda_stream


def _ptr(t: Optional[torch.Tensor]) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def _dt(dtype: torch.dtype) -> int:
    if dtype not in _TORCH_DT:
        raise TypeError(f"unsupported dtype {dtype}")
    return _TORCH_DT[dtype]


def _need(cond: bool, msg: str):
    if not cond:
        raise ValueError(msg)


def _check_dev(t: torch.Tensor, name: str, dtype=None, shape=None, on_device: bool = True):
    """A contiguous (device) tensor of the given dtype and shape: the C ABI
    takes raw pointers and cannot check any of this itself.  Type, dtype,
    shape and layout are checked before the device, so every one of these
    errors can be raised without a GPU."""
    _need(isinstance(t, torch.Tensor), f"{name} must be a torch tensor")
    if dtype is not None:
        _need(t.dtype == dtype, f"{name} must be {dtype}, not {t.dtype}")
    if shape is not None:
        _need(tuple(t.shape) == tuple(shape), f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    _need(t.is_contiguous(), f"{name} must be contiguous")
    if on_device:
        _need(t.is_cuda, f"{name} must be a device tensor")


def _check_out(out: Optional[torch.Tensor], shape, dtype):
    if out is not None:
        _check_dev(out, "out", dtype, shape, on_device=False)


def _same_device(X: torch.Tensor, *others):
    """Every tensor on X's device (after the shape checks)."""
    _need(X.is_cuda, "X must be a device tensor")
    for name, t in others:
        if t is not None:
            _need(t.is_cuda and t.device == X.device, f"{name} must be on the same device as X")


def _host_map(tile_map) -> np.ndarray:
    if isinstance(tile_map, torch.Tensor):
        tile_map = tile_map.detach().cpu().numpy()
    return np.ascontiguousarray(tile_map, dtype=np.uint8)


@dataclasses.dataclass
class PackedWeight:
    blob: torch.Tensor  # uint8, device
    desc: Desc

    @property
    def N(self) -> int:
        return self.desc.N

    @property
    def K(self) -> int:
        return self.desc.K

    @property
    def dtype(self) -> torch.dtype:
        return _DT_TORCH[self.desc.dtype]

    @property
    def n_sparse(self) -> int:
        """Compressed (2:4 and 4:8) tiles."""
        return self.desc.n_sparse

    @property
    def n_48(self) -> int:
        """4:8 tiles among the compressed ones."""
        return self.desc.n_48

    @property
    def nbytes(self) -> int:
        return self.desc.total_bytes


def packed_bytes(dtype: torch.dtype, N: int, K: int, tile_map) -> int:
    tm = _host_map(tile_map)
    return int(load().patch_packed_bytes(_dt(dtype), N, K, tm.ctypes.data_as(ctypes.c_void_p)))


def pack(W: torch.Tensor, tile_map, mask: torch.Tensor, out: Optional[torch.Tensor] = None) -> PackedWeight:
    """Pack W (N x K, f16/bf16, device), a host tile map (0 dense, 1 2:4,
    2 4:8) and a device byte mask (nonzero = keep) into a blob (patch_pack)."""
    lib = load()
    _need(isinstance(W, torch.Tensor) and W.dim() == 2, "W must be a 2-D tensor (N x K)")
    _need(W.dtype in (torch.float16, torch.bfloat16), "W must be float16 or bfloat16")
    N, K = W.shape
    _check_dev(W, "W", on_device=False)
    _check_dev(mask, "mask", torch.uint8, (N, K), on_device=False)
    tm = _host_map(tile_map)
    _need(tm.shape == (N // 128, K // 128) or N % 128 or K % 128, f"tile map must have shape {(N // 128, K // 128)}")
    if out is not None:
        _check_dev(out, "out", torch.uint8, on_device=False)
    _need(W.is_cuda and mask.is_cuda and (out is None or out.is_cuda), "W, mask and out must be device tensors")
    nbytes = packed_bytes(W.dtype, N, K, tm)
    if nbytes == 0:
        # let the library name what is wrong (it checks before the buffer size)
        probe = torch.empty(16, dtype=torch.uint8, device=W.device)
        _check(lib.patch_pack(_dt(W.dtype), N, K, _ptr(W), tm.ctypes.data_as(ctypes.c_void_p), _ptr(mask),
                              _ptr(probe), 0, ctypes.byref(Desc()), _stream()))
        raise PatchError(2, f"invalid arguments for pack: {tuple(W.shape)} {W.dtype}")
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
    desc = Desc()
    _check(lib.patch_pack(_dt(W.dtype), N, K, _ptr(W), tm.ctypes.data_as(ctypes.c_void_p), _ptr(mask), _ptr(out),
                          out.numel(), ctypes.byref(desc), _stream()))
    return PackedWeight(out, desc)


def packed_bytes_q64(dtype: torch.dtype, N: int, K: int, quad_map) -> int:
    """Blob size for 64 x 64 execution tiles (format 4) and a (N/64, K/64)
    quadrant map (0 dense, 1 2:4); 0 for invalid arguments."""
    qm = _host_map(quad_map)
    if qm.shape != (N // 64, K // 64):
        return 0
    return int(load().patch_packed_bytes_q64(_dt(dtype), N, K, qm.ctypes.data_as(ctypes.c_void_p)))


def pack_q64(W: torch.Tensor, quad_map, mask: torch.Tensor, out: Optional[torch.Tensor] = None) -> PackedWeight:
    """Pack W (N x K, f16/bf16, device), a host quadrant map ((N/64) x (K/64):
    0 dense, 1 2:4) and a device byte mask into a blob of 64 x 64 execution
    tiles (patch_pack_q64)."""
    lib = load()
    _need(isinstance(W, torch.Tensor) and W.dim() == 2, "W must be a 2-D tensor (N x K)")
    _need(W.dtype in (torch.float16, torch.bfloat16), "W must be float16 or bfloat16")
    N, K = W.shape
    _check_dev(W, "W", on_device=False)
    _check_dev(mask, "mask", torch.uint8, (N, K), on_device=False)
    qm = _host_map(quad_map)
    _need(qm.shape == (N // 64, K // 64) or N % 128 or K % 128, f"quadrant map must have shape {(N // 64, K // 64)}")
    if out is not None:
        _check_dev(out, "out", torch.uint8, on_device=False)
    _need(W.is_cuda and mask.is_cuda and (out is None or out.is_cuda), "W, mask and out must be device tensors")
    nbytes = packed_bytes_q64(W.dtype, N, K, qm)
    if nbytes == 0:
        probe = torch.empty(16, dtype=torch.uint8, device=W.device)
        _check(lib.patch_pack_q64(_dt(W.dtype), N, K, _ptr(W), qm.ctypes.data_as(ctypes.c_void_p), _ptr(mask),
                                  _ptr(probe), 0, ctypes.byref(Desc()), _stream()))
        raise PatchError(2, f"invalid arguments for pack_q64: {tuple(W.shape)} {W.dtype}")
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=W.device)
    desc = Desc()
    _check(lib.patch_pack_q64(_dt(W.dtype), N, K, _ptr(W), qm.ctypes.data_as(ctypes.c_void_p), _ptr(mask),
                              _ptr(out), out.numel(), ctypes.byref(desc), _stream()))
    return PackedWeight(out, desc)


def desc_from_header(header: bytes) -> Desc:
    buf = (ctypes.c_uint8 * len(header)).from_buffer_copy(header)
    d = Desc()
    _check(load().patch_desc_from_header(ctypes.cast(buf, ctypes.c_void_p), len(header), ctypes.byref(d)))
    return d


_WS_BYTES = {}


def _ws_bytes(kind: str, M: int, N: int, K: int, dev: int, query) -> int:
    """The library's workspace query, remembered per shape (it is a pure
    function of the shape on a given device)."""
    key = (kind, M, N, K, dev)
    nb = _WS_BYTES.get(key)
    if nb is None:
        nb = int(query())
        if len(_WS_BYTES) > 4096:
            _WS_BYTES.clear()
        _WS_BYTES[key] = nb
    return nb


def _check_x(X: torch.Tensor, dtype: torch.dtype, K: int):
    _need(isinstance(X, torch.Tensor) and X.dim() == 2, "X must be a 2-D tensor (M x K)")
    _need(X.shape[1] == K, f"X must have K = {K} columns, not {X.shape[1]}")
    _check_dev(X, "X", dtype, on_device=False)


def _check_out_dtype(od: torch.dtype, xd: torch.dtype):
    _need(od in (xd, torch.float32), f"out_dtype must be {xd} or torch.float32, not {od}")


def _workspace(nbytes: int, workspace, device):
    """workspace="auto": a fresh buffer of the size the library asks for
    (from torch's caching allocator) on every call; None: no workspace; a
    tensor: used as given.  Callers that run the same shapes repeatedly keep
    one buffer per call site (sized by patch_gemm_workspace_bytes) and pass
    it: with the per-call allocation a step of two tail-split GEMMs measured
    up to 3% slower."""
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError(f"workspace must be 'auto', None or a tensor, not {workspace!r}")
        return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes > 0 else None
    if workspace is not None:
        _check_dev(workspace, "workspace")
        _need(workspace.device == device, "workspace must be on the same device as X")
    return workspace


def gemm(X: torch.Tensor, packed: PackedWeight, out_dtype: Optional[torch.dtype] = None, variant: str = "auto",
         out: Optional[torch.Tensor] = None, workspace="auto") -> torch.Tensor:
    """Y = X (W o E)^T from a packed blob (patch_gemm_ex)."""
    lib = _lib or load()
    _check_x(X, packed.dtype, packed.K)
    _check_dev(packed.blob, "packed blob", torch.uint8, on_device=False)
    _need(packed.blob.numel() >= packed.nbytes, "packed blob is smaller than its descriptor's total_bytes")
    M = X.shape[0]
    od = out_dtype or X.dtype
    _check_out_dtype(od, X.dtype)
    _check_out(out, (M, packed.N), od)
    _same_device(X, ("packed blob", packed.blob), ("out", out))
    dev = X.get_device()
    if out is None:
        out = torch.empty((M, packed.N), dtype=od, device=X.device)
    ws, nb = None, 0
    if workspace is not None:
        nb = _ws_bytes("packed", M, packed.N, packed.K, dev,
                       lambda: lib.patch_gemm_workspace_bytes(ctypes.byref(packed.desc), M))
        ws = _workspace(nb, workspace, X.device)
        nb = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib.patch_gemm_ex(ctypes.byref(packed.desc), packed.blob.data_ptr(), X.data_ptr(), M, out.data_ptr(),
                             _dt(od), None if ws is None else ws.data_ptr(), nb, VARIANTS[variant],
                             _stream(dev)))
    return out


def gemm_noalloc(X: torch.Tensor, packed: PackedWeight, out: torch.Tensor,
                 out_dtype: Optional[torch.dtype] = None) -> torch.Tensor:
    """Y = X (W o E)^T into a caller-supplied `out` with the library's own
    device scratch (patch_gemm_noalloc): nothing is allocated, by the
    library or here."""
    lib = _lib or load()
    _check_x(X, packed.dtype, packed.K)
    _check_dev(packed.blob, "packed blob", torch.uint8, on_device=False)
    _need(packed.blob.numel() >= packed.nbytes, "packed blob is smaller than its descriptor's total_bytes")
    od = out_dtype or out.dtype
    _check_out_dtype(od, X.dtype)
    _check_out(out, (X.shape[0], packed.N), od)
    _same_device(X, ("packed blob", packed.blob), ("out", out))
    _check(lib.patch_gemm_noalloc(ctypes.byref(packed.desc), packed.blob.data_ptr(), X.data_ptr(), X.shape[0],
                                  out.data_ptr(), _dt(od), _stream(X.get_device())))
    return out


def dense_gemm(X: torch.Tensor, W: torch.Tensor, out_dtype: Optional[torch.dtype] = None, variant: str = "auto",
               out: Optional[torch.Tensor] = None, workspace="auto") -> torch.Tensor:
    """Same-shape dense baseline Y = X W^T from row-major W (patch_dense_gemm_ex)."""
    lib = _lib or load()
    _need(W.dim() == 2, "W must be 2-D (N x K)")
    _check_x(X, W.dtype, W.shape[1])
    _check_dev(W, "W", X.dtype, on_device=False)
    M, K = X.shape
    N = W.shape[0]
    od = out_dtype or X.dtype
    _check_out_dtype(od, X.dtype)
    _check_out(out, (M, N), od)
    _same_device(X, ("W", W), ("out", out))
    dev = X.get_device()
    if out is None:
        out = torch.empty((M, N), dtype=od, device=X.device)
    ws, nb = None, 0
    if workspace is not None:
        nb = _ws_bytes("dense", M, N, K, dev, lambda: lib.patch_dense_gemm_workspace_bytes(M, N, K))
        ws = _workspace(nb, workspace, X.device)
        nb = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib.patch_dense_gemm_ex(_dt(X.dtype), M, N, K, X.data_ptr(), W.data_ptr(), out.data_ptr(), _dt(od),
                                   None if ws is None else ws.data_ptr(), nb, VARIANTS[variant], _stream(dev)))
    return out


def pack_gate_up(Wg: torch.Tensor, Wu: torch.Tensor, map_g, map_u, mask_g: torch.Tensor, mask_u: torch.Tensor,
                 out: Optional[torch.Tensor] = None) -> PackedWeight:
    """Pack gate and up weights (F x K each, device) into one blob of their
    row-block interleave (patch_pack_gate_up)."""
    lib = load()
    F, K = Wg.shape
    if tuple(Wu.shape) != (F, K) or Wu.dtype != Wg.dtype:
        raise ValueError("gate and up weights must have the same shape and dtype")
    tg, tu = _host_map(map_g), _host_map(map_u)
    nbytes = int(lib.patch_packed_bytes_gate_up(_dt(Wg.dtype), F, K, tg.ctypes.data_as(ctypes.c_void_p),
                                                tu.ctypes.data_as(ctypes.c_void_p)))
    if nbytes == 0:
        raise PatchError(2, f"invalid shape/dtype for pack_gate_up: {tuple(Wg.shape)} {Wg.dtype}")
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=Wg.device)
    desc = Desc()
    _check(lib.patch_pack_gate_up(_dt(Wg.dtype), F, K, _ptr(Wg), _ptr(Wu), tg.ctypes.data_as(ctypes.c_void_p),
                                  tu.ctypes.data_as(ctypes.c_void_p), _ptr(mask_g), _ptr(mask_u), _ptr(out),
                                  out.numel(), ctypes.byref(desc), _stream()))
    return PackedWeight(out, desc)


def gemm_swiglu(X: torch.Tensor, packed: PackedWeight, out_dtype: Optional[torch.dtype] = None,
                variant: str = "auto", out: Optional[torch.Tensor] = None, workspace="auto") -> torch.Tensor:
    """H = SiLU(X Wg^T) * (X Wu^T) from a gate/up blob (patch_gemm_swiglu)."""
    lib = _lib or load()
    _check_x(X, packed.dtype, packed.K)
    _check_dev(packed.blob, "packed blob", torch.uint8, on_device=False)
    _need(packed.blob.numel() >= packed.nbytes, "packed blob is smaller than its descriptor's total_bytes")
    M = X.shape[0]
    F = packed.N // 2
    od = out_dtype or X.dtype
    _check_out_dtype(od, X.dtype)
    _check_out(out, (M, F), od)
    _same_device(X, ("packed blob", packed.blob), ("out", out))
    dev = X.get_device()
    if out is None:
        out = torch.empty((M, F), dtype=od, device=X.device)
    ws, nb = None, 0
    if workspace is not None:
        nb = _ws_bytes("swiglu", M, packed.N, packed.K, dev,
                       lambda: lib.patch_gemm_swiglu_workspace_bytes(ctypes.byref(packed.desc), M))
        ws = _workspace(nb, workspace, X.device)
        nb = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib.patch_gemm_swiglu(ctypes.byref(packed.desc), packed.blob.data_ptr(), X.data_ptr(), M, out.data_ptr(),
                                 _dt(od), None if ws is None else ws.data_ptr(), nb, VARIANTS[variant], _stream(dev)))
    return out


def dense_gemm_swiglu(X: torch.Tensor, Wg: torch.Tensor, Wu: torch.Tensor, out_dtype: Optional[torch.dtype] = None,
                      variant: str = "auto", out: Optional[torch.Tensor] = None, workspace="auto") -> torch.Tensor:
    """Same-shape dense baseline of gemm_swiglu from row-major Wg, Wu (patch_dense_gemm_swiglu)."""
    lib = _lib or load()
    _need(Wg.dim() == 2, "Wg must be 2-D (F x K)")
    _check_x(X, Wg.dtype, Wg.shape[1])
    _check_dev(Wg, "Wg", X.dtype, on_device=False)
    _check_dev(Wu, "Wu", X.dtype, tuple(Wg.shape), on_device=False)
    M, K = X.shape
    F = Wg.shape[0]
    od = out_dtype or X.dtype
    _check_out_dtype(od, X.dtype)
    _check_out(out, (M, F), od)
    _same_device(X, ("Wg", Wg), ("Wu", Wu), ("out", out))
    dev = X.get_device()
    if out is None:
        out = torch.empty((M, F), dtype=od, device=X.device)
    ws, nb = None, 0
    if workspace is not None:
        nb = _ws_bytes("dense_swiglu", M, F, K, dev, lambda: lib.patch_dense_gemm_swiglu_workspace_bytes(M, F, K))
        ws = _workspace(nb, workspace, X.device)
        nb = 0 if ws is None else ws.numel() * ws.element_size()
    _check(lib.patch_dense_gemm_swiglu(_dt(X.dtype), M, F, K, X.data_ptr(), Wg.data_ptr(), Wu.data_ptr(),
                                       out.data_ptr(), _dt(od), None if ws is None else ws.data_ptr(), nb,
                                       VARIANTS[variant], _stream(dev)))
    return out


def pack_concat(Ws, tile_maps, masks, out: Optional[torch.Tensor] = None) -> PackedWeight:
    """Pack the row-concatenation of several weights with the same K (device
    tensors, host tile maps, device masks) into one blob (patch_pack_concat):
    one GEMM on it returns the projections side by side."""
    lib = load()
    n = len(Ws)
    if not (len(tile_maps) == len(masks) == n) or n < 1:
        raise ValueError("one tile map and one mask per weight")
    K = Ws[0].shape[1]
    if any(W.dtype != Ws[0].dtype or W.shape[1] != K for W in Ws):
        raise ValueError("the weights must share dtype and K")
    Ns = (ctypes.c_int64 * n)(*[int(W.shape[0]) for W in Ws])
    maps = [_host_map(t) for t in tile_maps]
    mp = (ctypes.c_void_p * n)(*[m.ctypes.data for m in maps])
    wp = (ctypes.c_void_p * n)(*[W.data_ptr() for W in Ws])
    kp = (ctypes.c_void_p * n)(*[m.data_ptr() for m in masks])
    nbytes = int(lib.patch_packed_bytes_concat(_dt(Ws[0].dtype), n, Ns, K, mp))
    if nbytes == 0:
        raise PatchError(2, "invalid shapes for pack_concat")
    if out is None:
        out = torch.empty(nbytes, dtype=torch.uint8, device=Ws[0].device)
    desc = Desc()
    _check(lib.patch_pack_concat(_dt(Ws[0].dtype), n, Ns, K, wp, mp, kp, _ptr(out), out.numel(), ctypes.byref(desc),
                                 _stream()))
    return PackedWeight(out, desc)


def sample_mask(tile_logits: torch.Tensor, tile_u: torch.Tensor, pat_logits: torch.Tensor, pat_u: torch.Tensor,
                tau: float, soft: bool = True, out=None):
    """Forward hybrid-mask sampler (patch_sample_mask) on device float32
    tensors: tile_logits, tile_u [N/128, K/128, 2]; pat_logits, pat_u
    [N, K/4, 6].  Returns (tile_map uint8 [N/128, K/128], mask uint8 [N, K],
    soft float32 [N, K] or None); out = (tile_map, mask, soft) reuses
    buffers."""
    lib = load()
    N, G = int(pat_logits.shape[0]), int(pat_logits.shape[1])
    K = 4 * G
    for t, shape in ((tile_logits, (N // 128, K // 128, 2)), (tile_u, (N // 128, K // 128, 2)),
                     (pat_logits, (N, G, 6)), (pat_u, (N, G, 6))):
        if t.dtype != torch.float32 or tuple(t.shape) != shape or not t.is_contiguous() or not t.is_cuda:
            raise ValueError(f"expected a contiguous float32 device tensor of shape {shape}")
    dev = pat_logits.device
    if out is None:
        out = (torch.empty((N // 128, K // 128), dtype=torch.uint8, device=dev),
               torch.empty((N, K), dtype=torch.uint8, device=dev),
               torch.empty((N, K), dtype=torch.float32, device=dev) if soft else None)
    tmap, mask, sf = out
    _check(lib.patch_sample_mask(N, K, _ptr(tile_logits), _ptr(tile_u), _ptr(pat_logits), _ptr(pat_u), float(tau),
                                 _ptr(tmap), _ptr(mask), _ptr(sf) if soft else ctypes.c_void_p(0),
                                 _stream(dev.index)))
    return tmap, mask, (sf if soft else None)


def exec_tile_map(N: int, K: int, fine_map, b1: int, b2: int) -> np.ndarray:
    """128 x 128 execution tile map from a fine tile map of b1 x b2 tiles
    (patch_exec_tile_map): 1 where every fine tile is 2:4."""
    fm = _host_map(fine_map)
    if fm.shape != (N // b1, K // b2):
        raise ValueError(f"fine map must be {(N // b1, K // b2)}")
    out = np.zeros((N // 128, K // 128), dtype=np.uint8)
    n = ctypes.c_int64(0)
    _check(load().patch_exec_tile_map(N, K, b1, b2, fm.ctypes.data, out.ctypes.data, ctypes.byref(n)))
    return out


def apply_fine_mask(W: torch.Tensor, fine_map: torch.Tensor, mask: torch.Tensor, b1: int, b2: int,
                    out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """W o E_fine on the device (patch_apply_fine_mask): fine_map uint8
    [N/b1, K/b2] and mask uint8 [N, K] device tensors."""
    N, K = W.shape
    if out is None:
        out = torch.empty_like(W)
    _check(load().patch_apply_fine_mask(_dt(W.dtype), N, K, b1, b2, _ptr(W), _ptr(fine_map), _ptr(mask), _ptr(out),
                                        _stream(W.device.index)))
    return out


def pack_fine(W: torch.Tensor, fine_map, mask: torch.Tensor, b1: int, b2: int) -> PackedWeight:
    """Pack a layer whose mask was learnt on b1 x b2 tiles: execution map by
    the all-2:4 policy, dense execution tiles from W o E_fine."""
    N, K = W.shape
    fm_host = _host_map(fine_map)
    emap = exec_tile_map(N, K, fm_host, b1, b2)
    Wm = apply_fine_mask(W, torch.from_numpy(fm_host).to(W.device), mask, b1, b2)
    return pack(Wm, emap, mask)


def probe_stream_read(src: torch.Tensor, sink: torch.Tensor) -> None:
    """Read every byte of src once (patch_probe_stream_read); time it around
    the call.  sink: a device scratch tensor (its bytes bound the grid)."""
    _check_dev(src, "src")
    _check_dev(sink, "sink")
    nb = src.numel() * src.element_size()
    _check(load().patch_probe_stream_read(_ptr(src), nb - nb % 16, _ptr(sink), sink.numel() * sink.element_size(),
                                          _stream(src.device.index)))


def probe_matrix_rate(kind: int, iters: int, workgroups: int, sink: torch.Tensor) -> int:
    """Launch the matrix-instruction rate probe (patch_probe_matrix_rate);
    returns the flops it executes (dense-equivalent for the sparse kinds)."""
    _check_dev(sink, "sink")
    _need(sink.numel() * sink.element_size() >= 4 * workgroups, "sink needs 4 bytes a workgroup")
    lib = load()
    _check(lib.patch_probe_matrix_rate(kind, iters, workgroups, _ptr(sink), _stream(sink.device.index)))
    return int(lib.patch_probe_matrix_flops(kind, iters, workgroups))


def debug_tail_wait(polls: int) -> None:
    """For tests of the tail split's bounded wait (patch_debug_tail_wait):
    polls > 0 makes the first K range of every left-over block wait for a
    flag value no range stores, give up after that many polls and mark its
    block's outputs NaN; polls <= 0 restores normal launches."""
    (_lib or load()).patch_debug_tail_wait(int(polls))


def probe_copy_rate(src: torch.Tensor, window_bytes: int, iters: int, workgroups: int, sink: torch.Tensor) -> int:
    """Launch the global -> LDS copy-rate probe (patch_probe_copy_rate) over
    src (its size a multiple of window_bytes); returns the bytes it copies."""
    _check_dev(src, "src")
    _check_dev(sink, "sink")
    lib = load()
    _check(lib.patch_probe_copy_rate(_ptr(src), src.numel() * src.element_size(), window_bytes, iters, workgroups,
                                     _ptr(sink), sink.numel() * sink.element_size(), _stream(src.device.index)))
    return int(lib.patch_probe_copy_bytes(iters, workgroups))


# ---------------------------------------------------------------------------- decoder-layer operators
# Their C structures are 8-byte fields in order: packed here with struct.
_ROPE_ARGS = struct.Struct("16q")
_APPEND_ARGS = struct.Struct("25q")
_ATTENTION_ARGS = struct.Struct("7qd11q")
_CACHE_ARGS = struct.Struct("8q")
_LAYOUTS = {"half": 0, "interleaved": 1}
_HALVES = {torch.float16: PATCH_F16, torch.bfloat16: PATCH_BF16}
_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "by_parts": 3}


_get_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device


def _call(index: int, fn, *args):
    """A library call on the current stream of device `index`, which is made
    the current device for it: a launch goes to the current device."""
    if index == _get_device():
        rc = fn(*args, _stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _stream(index))
    if rc:
        _check(rc)


# The checks below build their messages only where they fail: a decode step's
# calls last a few microseconds each.
def _heads(t, name: str, dtype, T, H, D, index):
    """A [tokens, heads, dim] tensor on device `index` whose elements of a
    head are contiguous: its address, other strides, and heads (H None: any)."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch tensor")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, not {t.dtype}")
    s = t.shape
    if len(s) != 3 or s[0] != T or s[2] != D or (H is not None and s[1] != H):
        raise ValueError(f"{name} must have shape {(T, 'heads' if H is None else H, D)}, not {tuple(s)}")
    st = t.stride()
    if st[2] != 1 and D > 1:
        raise ValueError(f"{name}: the elements of a head must be contiguous")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on device {index}, not {t.device}")
    return t.data_ptr(), st[0], st[1], s[1]


def _rows_out(t, name: str, dtype, T, H, D, index):
    """_heads of a tensor that is written."""
    p, st, sh, _ = _heads(t, name, dtype, T, H, D, index)
    if (st == 0 and T > 1) or (sh == 0 and H > 1):
        raise ValueError(f"{name} overlaps itself")
    return p, st, sh


def _index(t, name: str, n: int, index):
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or t.dim() != 1 or t.shape[0] != n or (
            n > 1 and not t.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous int32 tensor of {n}")
    if t.get_device() != index:
        raise ValueError(f"{name} must be on device {index}, not {t.device}")
    return t.data_ptr()


def _device_of(t, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a torch tensor")
    return t.get_device()


def _need_device(index: int):
    if index < 0:
        raise ValueError("tensors must be on the device")


def rope_table(positions: int, rot: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
               original: float = 0.0, low: float = 1.0, high: float = 32.0, magnitude: float = 1.0, device="cuda",
               out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """cos and sin of every position's angles, float32 [positions, rot]
    (patch_rope_table).  scaling: "none", "linear", "ntk" or "by_parts", for
    contexts `factor` times the `original` one."""
    lib = _lib or load()
    _need(scaling in _SCALINGS, f"scaling must be one of {sorted(_SCALINGS)}, not {scaling!r}")
    _check_out(out, (positions, rot), torch.float32)
    if out is None:
        _need(positions >= 1 and rot >= 2, f"positions={positions} and rot={rot} must be positive")
        out = torch.empty((positions, rot), dtype=torch.float32, device=device)
    _need_device(out.get_device())
    _call(out.get_device(), lib.patch_rope_table, positions, rot, base, _SCALINGS[scaling], factor, original, low, high,
          magnitude, out.data_ptr())
    return out


def _table_of(table: Optional[torch.Tensor], index):
    if table is None:
        return 0, 0, 0
    if not isinstance(table, torch.Tensor) or table.dtype is not torch.float32 or table.dim() != 2 or \
            not table.is_contiguous():
        raise ValueError("table must be a contiguous float32 tensor (positions, rot)")
    if table.get_device() != index:
        raise ValueError(f"table must be on device {index}, not {table.device}")
    n, rot = table.shape
    return table.data_ptr(), n, rot


def rope(x: torch.Tensor, positions: torch.Tensor, table: torch.Tensor, layout: str = "half", inverse: bool = False,
         out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x [tokens, heads, dim] (float16, bfloat16 or float32; any token and
    head stride) turned by each token's position, int32 [tokens]
    (patch_rope).  inverse=True turns back: the gradient of x from that of
    the result.  out may be x."""
    lib = _lib or load()
    if layout not in _LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(_LAYOUTS)}, not {layout!r}")
    if not isinstance(x, torch.Tensor) or x.dim() != 3:
        raise ValueError("x must be a 3-D tensor (tokens, heads, dim)")
    dt, dtype, index = x.dtype, _dt(x.dtype), x.get_device()
    T, H, D = x.shape
    xp, xt, xh, _ = _heads(x, "x", dt, T, H, D, index)
    pos = _index(positions, "positions", T, index)
    tp, context, rot = _table_of(table, index)
    if not rot:
        raise ValueError("table must be a tensor with rot > 0 columns")
    if out is None:
        _need_device(index)
        out = torch.empty((T, H, D), dtype=dt, device=x.device)
    op, ot, oh = _rows_out(out, "out", dt, T, H, D, index)
    _need_device(index)
    _call(index, lib.patch_rope,
          _ROPE_ARGS.pack(dtype, _LAYOUTS[layout], bool(inverse), T, H, D, rot, context, xp, xt, xh, op, ot, oh, pos, tp))
    return out


@dataclasses.dataclass(frozen=True)
class KVCache:
    """The pages of a paged 8-bit cache (patch_kv_cache): k, v [pages,
    kv_heads, page, dim] of torch.float8_e4m3fn (or uint8 bits), k_scale,
    v_scale float32 [pages, kv_heads]; all contiguous on one device.  Checked
    here once; the tensors stay the caller's."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor

    def __post_init__(self):
        k = self.k
        _need(isinstance(k, torch.Tensor) and k.dim() == 4, "k must be a 4-D tensor (pages, kv_heads, page, dim)")
        _need(k.dtype in (torch.float8_e4m3fn, torch.uint8), "k must be float8_e4m3fn or uint8")
        _check_dev(k, "k", on_device=False)
        _check_dev(self.v, "v", k.dtype, tuple(k.shape), on_device=False)
        _check_dev(self.k_scale, "k_scale", torch.float32, tuple(k.shape[:2]), on_device=False)
        _check_dev(self.v_scale, "v_scale", torch.float32, tuple(k.shape[:2]), on_device=False)
        pages, heads, page, dim = k.shape
        _need(page in (16, 32, 64, 128), f"pages must hold 16, 32, 64 or 128 tokens, not {page}")
        _need(dim % 16 == 0 and 16 <= dim <= 256, f"dim must be a multiple of 16 up to 256, not {dim}")
        _need_device(k.get_device())
        for name in ("v", "k_scale", "v_scale"):
            _need(getattr(self, name).device == k.device, f"{name} must be on {k.device}")
        object.__setattr__(self, "_args", _CACHE_ARGS.pack(
            k.data_ptr(), self.v.data_ptr(), self.k_scale.data_ptr(), self.v_scale.data_ptr(), pages, heads, page, dim))
        object.__setattr__(self, "_shape", (pages, heads, page, dim))
        object.__setattr__(self, "_index", k.get_device())


def kv_cache(pages: int, kv_heads: int, dim: int, page: int = 64, device="cuda") -> KVCache:
    """A new, empty cache of `pages` pages of `page` tokens."""
    kv = [torch.zeros((pages, kv_heads, page, dim), dtype=torch.uint8, device=device).view(torch.float8_e4m3fn)
          for _ in range(2)]
    scales = [torch.zeros((pages, kv_heads), dtype=torch.float32, device=device) for _ in range(2)]
    return KVCache(kv[0], kv[1], scales[0], scales[1])


def _pages_of(page_table: torch.Tensor, index):
    if not isinstance(page_table, torch.Tensor) or page_table.dtype is not torch.int32 or page_table.dim() != 2:
        raise ValueError("page_table must be an int32 tensor (sequences, pages)")
    S, n = page_table.shape
    st = page_table.stride()
    if st[1] != 1 and n > 1:
        raise ValueError("page_table: each row must be contiguous")
    if page_table.get_device() != index:
        raise ValueError(f"page_table must be on device {index}, not {page_table.device}")
    return page_table.data_ptr(), S, n, st[0] if S > 1 else n


def _cache_of(cache, index):
    if not isinstance(cache, KVCache):
        raise ValueError("cache must be a KVCache")
    if cache._index != index:
        raise ValueError(f"cache must be on device {index}, not {cache.k.device}")
    return cache._shape


def kv_append(k: torch.Tensor, v: torch.Tensor, cache: KVCache, page_table: torch.Tensor, kv_lens: torch.Tensor,
              cu_new: torch.Tensor, table: Optional[torch.Tensor] = None, layout: str = "half",
              q: Optional[torch.Tensor] = None, q_out: Optional[torch.Tensor] = None) -> Optional[torch.Tensor]:
    """Rotate the newest tokens' keys (and q), round keys and values to 8 bits
    and put them into the cache (patch_kv_append).  k, v [tokens, kv_heads,
    dim]; q [tokens, heads, dim] or None; page_table int32 [sequences,
    pages]; kv_lens int32 [sequences], lengths with the new tokens; cu_new
    int32 [sequences + 1], where each sequence's tokens begin; table of
    rope_table, or None for no rotation.  Returns the rotated q (q_out,
    which may be q), or None."""
    lib = _lib or load()
    if layout not in _LAYOUTS:
        raise ValueError(f"layout must be one of {sorted(_LAYOUTS)}, not {layout!r}")
    index = _device_of(k, "k")
    _, hk, _, D = _cache_of(cache, index)
    dt = k.dtype
    if dt not in _HALVES or k.dim() != 3:
        raise ValueError("k must be a float16 or bfloat16 3-D tensor (tokens, kv_heads, dim)")
    T = k.shape[0]
    kp, kt, kh, _ = _heads(k, "k", dt, T, hk, D, index)
    vp, vt, vh, _ = _heads(v, "v", dt, T, hk, D, index)
    pp, S, max_pages, row = _pages_of(page_table, index)
    lens, cu = _index(kv_lens, "kv_lens", S, index), _index(cu_new, "cu_new", S + 1, index)
    tp, context, rot = _table_of(table, index)
    qp = qt = qh = op = ot = oh = heads = 0
    if q is not None:
        qp, qt, qh, heads = _heads(q, "q", dt, T, None, D, index)
        if q_out is None:
            q_out = torch.empty((T, heads, D), dtype=dt, device=k.device)
        op, ot, oh = _rows_out(q_out, "q_out", dt, T, heads, D, index)
    elif q_out is not None:
        raise ValueError("q_out without q")
    _call(index, lib.patch_kv_append,
          _APPEND_ARGS.pack(_HALVES[dt], _LAYOUTS[layout], T, S, heads, rot, context, max_pages, kp, kt, kh, vp, vt, vh, qp,
                            qt, qh, op, ot, oh, pp, row, lens, cu, tp), cache._args)
    return q_out


def attention_workspace_bytes(tokens: int, sequences: int, heads: int, kv_heads: int, dim: int) -> int:
    """Scratch that lets attention split long sequences (patch_attention_workspace_bytes)."""
    return int((_lib or load()).patch_attention_workspace_bytes(tokens, sequences, heads, kv_heads, dim))


def attention(q: torch.Tensor, cache: KVCache, page_table: torch.Tensor, kv_lens: torch.Tensor, cu_new: torch.Tensor,
              scale: Optional[float] = None, window: int = 0, out_dtype: Optional[torch.dtype] = None,
              out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, workspace="auto") -> torch.Tensor:
    """softmax(scale q k^T) v over the cache for every sequence's newest
    tokens, which were appended before (patch_attention): q [tokens, heads,
    dim], heads a multiple of the cache's; page_table, kv_lens and cu_new as
    for kv_append.  A token sees the keys up to its own position, with window
    > 0 the last `window` of them.  scale: 1 / sqrt(dim) if not given.  lse:
    float32 [tokens, heads] to take the logarithm of each softmax's sum.
    workspace as for gemm."""
    lib = _lib or load()
    index = _device_of(q, "q")
    _, hk, _, D = _cache_of(cache, index)
    dt = q.dtype
    if dt not in _HALVES or q.dim() != 3:
        raise ValueError("q must be a float16 or bfloat16 3-D tensor (tokens, heads, dim)")
    T, H, _ = q.shape
    qp, qt, qh, _ = _heads(q, "q", dt, T, H, D, index)
    pp, S, max_pages, row = _pages_of(page_table, index)
    lens, cu = _index(kv_lens, "kv_lens", S, index), _index(cu_new, "cu_new", S + 1, index)
    od = out_dtype or dt
    if od is not dt:
        _check_out_dtype(od, dt)
    if out is None:
        out = torch.empty((T, H, D), dtype=od, device=q.device)
    op, ot, oh = _rows_out(out, "out", od, T, H, D, index)
    lp = 0
    if lse is not None:
        _check_dev(lse, "lse", torch.float32, (T, H))
        _need(lse.get_device() == index, f"lse must be on device {index}")
        lp = lse.data_ptr()
    wp, nb = None, 0
    if workspace is not None:
        nb = _ws_bytes("attention", (T, S), (H, hk), D, index, lambda: lib.patch_attention_workspace_bytes(T, S, H, hk, D))
        ws = _workspace(nb, workspace, q.device)
        if ws is not None:
            wp, nb = ws.data_ptr(), ws.numel() * ws.element_size()
    _call(index, lib.patch_attention,
          _ATTENTION_ARGS.pack(_HALVES[dt], _TORCH_DT[od], T, S, H, max_pages, window, D ** -0.5 if scale is None else scale,
                               qp, qt, qh, op, ot, oh, lp, pp, row, lens, cu),
          cache._args, wp, nb)
    return out


@dataclasses.dataclass(frozen=True)
class W4Weight:
    """A weight of 4-bit values and group scales, laid out for w4_gemm."""
    packed: torch.Tensor  # uint8, device
    dtype: torch.dtype    # of the scales and of X
    N: int
    K: int
    group: int
    with_zero: bool


def w4_quantize(W: torch.Tensor, group: int = 128, zero: bool = False):
    """W (N x K, float16 or bfloat16) rounded to 4 bits a group of `group`
    columns (patch_w4_quantize): returns q uint8 [N, K / 2], scale [N, K /
    group] of W's type, and with zero=True the zeros uint8 [N, K / group],
    else None."""
    lib = _lib or load()
    _need(isinstance(W, torch.Tensor) and W.dim() == 2, "W must be a 2-D tensor (N x K)")
    _need(W.dtype in (torch.float16, torch.bfloat16), "W must be float16 or bfloat16")
    _check_dev(W, "W", on_device=False)
    N, K = W.shape
    _need(group in (32, 64, 128) and K % group == 0 and N > 0 and K > 0, f"K={K} must be a multiple of the group ({group}: 32, 64 or 128)")
    _need_device(W.get_device())
    q = torch.empty((N, K // 2), dtype=torch.uint8, device=W.device)
    scale = torch.empty((N, K // group), dtype=W.dtype, device=W.device)
    z = torch.empty((N, K // group), dtype=torch.uint8, device=W.device) if zero else None
    _call(W.get_device(), lib.patch_w4_quantize, _HALVES[W.dtype], N, K, group, W.data_ptr(), q.data_ptr(), scale.data_ptr(),
          None if z is None else z.data_ptr())
    return q, scale, z


def w4_pack(q: torch.Tensor, scale: torch.Tensor, zero: Optional[torch.Tensor], group: int) -> W4Weight:
    """Lay 4-bit weights out for w4_gemm (patch_w4_pack): q uint8 [N, K / 2],
    the even column in a byte's low half; scale [N, K / group]; zero uint8
    [N, K / group], or None for 8 everywhere."""
    lib = _lib or load()
    _need(isinstance(q, torch.Tensor) and q.dim() == 2, "q must be a 2-D tensor (N x K / 2)")
    _check_dev(q, "q", torch.uint8, on_device=False)
    N, K = q.shape[0], 2 * q.shape[1]
    _need(group in (32, 64, 128) and K % group == 0 and N > 0 and K > 0, f"K={K} must be a multiple of the group ({group}: 32, 64 or 128)")
    _check_dev(scale, "scale", shape=(N, K // group), on_device=False)
    _need(scale.dtype in (torch.float16, torch.bfloat16), "scale must be float16 or bfloat16")
    if zero is not None:
        _check_dev(zero, "zero", torch.uint8, (N, K // group), on_device=False)
    _need_device(q.get_device())
    _need(scale.device == q.device and (zero is None or zero.device == q.device), "scale and zero must be on q's device")
    packed = torch.empty(int(lib.patch_w4_bytes(N, K, group, zero is not None)), dtype=torch.uint8, device=q.device)
    _call(q.get_device(), lib.patch_w4_pack, _HALVES[scale.dtype], N, K, group, q.data_ptr(), scale.data_ptr(),
          None if zero is None else zero.data_ptr(), packed.data_ptr(), packed.numel())
    return W4Weight(packed, scale.dtype, N, K, group, zero is not None)


def w4_gemm(X: torch.Tensor, weight: W4Weight, out_dtype: Optional[torch.dtype] = None,
            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y = X W^T with 4-bit weights (patch_w4_gemm)."""
    lib = _lib or load()
    if not isinstance(weight, W4Weight):
        raise ValueError("weight must be a W4Weight (w4_pack)")
    dt, N, K, index = weight.dtype, weight.N, weight.K, _device_of(X, "X")
    if X.dtype is not dt or X.dim() != 2 or X.shape[1] != K or not X.is_contiguous():
        raise ValueError(f"X must be a contiguous {dt} tensor (M, {K}), not {X.dtype} {tuple(X.shape)}")
    M = X.shape[0]
    od = out_dtype or dt
    if od is not dt:
        _check_out_dtype(od, dt)
    packed = weight.packed
    if packed.get_device() != index:
        raise ValueError(f"weight must be on device {index}, not {packed.device}")
    _need_device(index)
    if out is None:
        out = torch.empty((M, N), dtype=od, device=X.device)
    else:
        _check_out(out, (M, N), od)
        _need(out.get_device() == index, f"out must be on device {index}")
    _call(index, lib.patch_w4_gemm, _HALVES[dt], N, K, weight.group, weight.with_zero, packed.data_ptr(), packed.numel(),
          X.data_ptr(), M, out.data_ptr(), _TORCH_DT[od])
    return out
