"""gemm_rtn_sym_gb300 — symmetric INT4 group-128 RTN quantiser and W4A16 matmul
for NVIDIA GB300 (sm_103a).

A thin ctypes binding over the C ABI in include/w4.h (libw4.so, built in-tree by
``gemm_rtn_sym_gb300.build``; calls whose kernels last microseconds go through a
compiled module, csrc/binding.cpp, where their tensors are what they should be).  The functions here only check and marshal
arguments: torch tensors provide device memory and the current CUDA stream;
every step of the computation runs in the library's CUDA kernels.  There is no
CPU fallback: if libw4.so is missing or a CUDA device is absent, calls raise.
"""
from __future__ import annotations

import ctypes
import importlib
import os
import threading

import torch

__all__ = [
    "load", "library_path", "W4Error",
    "w4_quantize_rtn", "w4_quantize_rtn_scaled", "w4_scale_activations", "w4_quantize_rtn_asym",
    "w4_gemm", "w4_gemm_ex", "w4_gemm_affine", "w4_gemm_path_for", "w4_zeros_bytes", "GROUPS",
    "w4_gptq_factor", "w4_gptq_quantize", "w4_gptq_workspace_bytes", "w4_gptq_factor_workspace_bytes",
    "W4_ERR_NUMERIC",
    "w4_packed_bytes", "w4_scales_bytes", "w4_last_device_status", "w4_wait_probe",
    "w4_status_string", "W4_PATH_AUTO", "W4_PATH_SMALL_M", "W4_PATH_TENSOR", "GROUP",
    "GroupedPlan", "w4_grouped_plan", "w4_gemm_grouped", "w4_gemm_grouped_noalloc",
    "w4_kv_pages", "w4_kv_append", "w4_attn_decode", "w4_attn_decode_workspace_bytes",
    "w4_kv_append_norm", "w4_kv_fork", "w4_kv_copy", "w4_kv_compact",
    "w4_attn_decode_shared", "w4_attn_decode_shared_workspace_bytes",
]

GROUP = 128
GROUPS = (32, 64, 128)
W4_OK, W4_ERR_INVALID_ARG, W4_ERR_UNSUPPORTED, W4_ERR_MISALIGNED, W4_ERR_CUDA, W4_ERR_TIMEOUT, W4_ERR_NUMERIC = range(7)
W4_PATH_AUTO, W4_PATH_SMALL_M, W4_PATH_TENSOR = 0, 1, 2

_PKG = os.path.dirname(os.path.abspath(__file__))
_lib = None
_fast = _fast_error = None
_lock = threading.Lock()

_i64, _i32, _vp, _sz = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t


class _Problem(ctypes.Structure):
    """w4_gemm_problem of include/w4.h."""
    _fields_ = [("x", _vp), ("M", _i64), ("N", _i64), ("K", _i64), ("packed", _vp), ("scales", _vp), ("y", _vp)]


class _Plan(ctypes.Structure):
    """w4_grouped_plan of include/w4.h."""
    _fields_ = [("device_plan", _vp), ("bytes", _sz), ("count", _i32), ("device", _i32), ("items", _i32),
                ("ctas", _i32), ("token_rows", _i32), ("tc_items", _i32), ("tc_ctas", _i32), ("tc_max_bm", _i32),
                ("tc_offset", _sz), ("format", _i32)]

_SIGNATURES = {
    "w4_packed_bytes": (_sz, [_i64, _i64]),
    "w4_scales_bytes": (_sz, [_i64, _i64, _i32]),
    "w4_quantize_rtn": (ctypes.c_int, [_vp, _i64, _i64, _i32, _vp, _vp, _vp]),
    "w4_quantize_rtn_scaled": (ctypes.c_int, [_vp, _i64, _i64, _i32, _vp, _vp, _vp, _vp]),
    "w4_quantize_rtn_asym": (ctypes.c_int, [_vp, _i64, _i64, _i32, _vp, _vp, _vp, _vp]),
    "w4_zeros_bytes": (_sz, [_i64, _i64, _i32]),
    "w4_gptq_factor_workspace_bytes": (_sz, [_i64]),
    "w4_gptq_factor": (ctypes.c_int, [_vp, _i64, ctypes.c_double, _vp, _vp, _sz, _vp]),
    "w4_gptq_workspace_bytes": (_sz, [_i64, _i64]),
    "w4_gptq_quantize": (ctypes.c_int, [_vp, _i64, _i64, _i32, _vp, _vp, _vp, _vp, _sz, _vp]),
    "w4_gemm_affine": (ctypes.c_int, [_vp, _i64, _i64, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _i32]),
    "w4_scale_activations": (ctypes.c_int, [_vp, _i64, _i64, _vp, _vp, _vp]),
    "w4_gemm": (ctypes.c_int, [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp]),
    "w4_gemm_ex": (ctypes.c_int, [_vp, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _i32]),
    "w4_gemm_path_for": (ctypes.c_int, [_i64, _i64, _i64]),
    "w4_last_device_status": (ctypes.c_int, [_vp]),
    "w4_wait_probe": (ctypes.c_int, [_i64, _i32, _vp]),
    "w4_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "w4_grouped_plan_bytes": (_sz, [_i32, ctypes.POINTER(_Problem)]),
    "w4_grouped_plan_init": (ctypes.c_int, [ctypes.POINTER(_Plan), _vp, _sz, _i32, ctypes.POINTER(_Problem)]),
    "w4_gemm_grouped": (ctypes.c_int, [ctypes.POINTER(_Plan), _vp]),
    "w4_gemm_grouped_noalloc": (ctypes.c_int, [_i32, ctypes.POINTER(_Problem), _vp]),
    "w4_grouped_plan_bytes_affine": (_sz, [_i32, ctypes.POINTER(_Problem), _i32, ctypes.POINTER(_vp)]),
    "w4_grouped_plan_init_affine": (ctypes.c_int, [ctypes.POINTER(_Plan), _vp, _sz, _i32, ctypes.POINTER(_Problem),
                                                   _i32, ctypes.POINTER(_vp)]),
}


class _KvCache(ctypes.Structure):
    """w4_kv_cache of include/w4.h."""
    _fields_ = [("k", _vp), ("v", _vp), ("k_scales", _vp), ("v_scales", _vp), ("pages", _i64), ("page_stride", _i64),
                ("token_stride", _i64), ("head_stride", _i64), ("page_size", _i32), ("kv_heads", _i32),
                ("head_dim", _i32), ("format", _i32)]


class _Rows(ctypes.Structure):
    """w4_rows of include/w4.h."""
    _fields_ = [("data", _vp), ("token_stride", _i64), ("head_stride", _i64)]


class _Rope(ctypes.Structure):
    """w4_rope of include/w4.h."""
    _fields_ = [("positions", _vp), ("axis_stride", _i64), ("cos", _vp), ("sin", _vp), ("rows", _i64),
                ("rotary", _i32), ("axes", _i32), ("sections", _i32 * 4), ("cycled", _i32), ("paired", _i32)]


class _Norm(ctypes.Structure):
    """w4_norm of include/w4.h."""
    _fields_ = [("q_weight", _vp), ("k_weight", _vp), ("format", _i32), ("eps", ctypes.c_float), ("unit_offset", _i32)]


_SIGNATURES.update({
    "w4_kv_pages_held_workspace_bytes": (_sz, [_i32, _i32, _i64]),
    "w4_kv_pages_held": (ctypes.c_int, [_vp, _vp, _i32, _i32, _vp, _i64, _vp, _vp, _i64, _i32, _i64, _vp, _vp, _vp, _vp,
                                        _vp, _vp, _vp, _sz, _vp]),
    "w4_kv_fork": (ctypes.c_int, [_vp, _vp, _vp, _i32, _i32, _vp, _i64, _i32, _vp, _vp, _i64, _vp, _vp, _vp, _vp, _vp]),
    "w4_kv_compact": (ctypes.c_int, [_vp, _i32, _i32, _vp, _i64, _i32, _vp, _i64, _vp, _vp, _i64, _vp, _vp, _vp, _vp,
                                     _vp]),
    "w4_kv_copy": (ctypes.c_int, [ctypes.POINTER(_KvCache), _vp, _i32, _vp]),
    "w4_kv_append_norm": (ctypes.c_int, [ctypes.POINTER(_KvCache), ctypes.POINTER(_Rope), ctypes.POINTER(_Norm), _i64,
                                         _i32, ctypes.POINTER(_Rows), ctypes.POINTER(_Rows), ctypes.POINTER(_Rows),
                                         ctypes.POINTER(_Rows), _vp, _vp]),
    "w4_attn_decode_shared_workspace_bytes": (_sz, [ctypes.POINTER(_KvCache), _i32, _i64, _i32, _i32]),
    "w4_attn_decode_shared": (ctypes.c_int, [ctypes.POINTER(_KvCache), _i32, _i64, _i32, ctypes.POINTER(_Rows),
                                             ctypes.POINTER(_Rows), _vp, _i64, _i32, _vp, _vp, _i32, _vp, _vp, _i64,
                                             _i32, _vp, ctypes.c_float, _vp, _sz, _vp]),
    "w4_kv_pages": (ctypes.c_int, [_vp, _vp, _i32, _i32, _vp, _i64, _vp, _vp, _i64, _i32, _i64, _vp, _vp, _vp, _vp,
                                   _vp, _vp]),
    "w4_kv_append": (ctypes.c_int, [ctypes.POINTER(_KvCache), ctypes.POINTER(_Rope), _i64, _i32, ctypes.POINTER(_Rows),
                                    ctypes.POINTER(_Rows), ctypes.POINTER(_Rows), ctypes.POINTER(_Rows), _vp, _vp]),
    "w4_attn_decode_workspace_bytes": (_sz, [ctypes.POINTER(_KvCache), _i32, _i64, _i32]),
    "w4_attn_decode": (ctypes.c_int, [ctypes.POINTER(_KvCache), _i32, _i64, _i32, ctypes.POINTER(_Rows),
                                      ctypes.POINTER(_Rows), _vp, _i64, _i32, _vp, _vp, ctypes.c_float, _i64, _vp, _sz,
                                      _vp]),
})


class W4Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {w4_status_string(status)}")


def library_path() -> str:
    return os.path.join(_PKG, "libw4.so")


def load() -> ctypes.CDLL:
    """Load libw4.so (built by gemm_rtn_sym_gb300.build), raises if absent, and the compiled module beside it, whose calls
    raise where it cannot be imported."""
    global _lib, _fast, _fast_error
    with _lock:
        if _lib is None:
            path = library_path()
            if not os.path.exists(path):
                raise RuntimeError(
                    f"{path} is missing: build it with `python -m gemm_rtn_sym_gb300.build` "
                    "(there is no CPU fallback)")
            lib = ctypes.CDLL(path)
            for name, (res, args) in _SIGNATURES.items():
                fn = getattr(lib, name)
                fn.restype, fn.argtypes = res, args
            try:
                _fast = importlib.import_module("._binding", __name__)
            except ImportError as e:
                _fast_error = e
            _lib = lib
    return _lib


def w4_status_string(status: int) -> str:
    return load().w4_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != W4_OK:
        raise W4Error(status, where)


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _cuda_tensor(t: torch.Tensor, name: str, dtype: torch.dtype, ndim: int) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {ndim}-D tensor")


def w4_packed_bytes(N: int, K: int) -> int:
    return load().w4_packed_bytes(N, K)


def w4_scales_bytes(N: int, K: int, group: int = GROUP) -> int:
    return load().w4_scales_bytes(N, K, group)


def w4_zeros_bytes(N: int, K: int, group: int = GROUP) -> int:
    return load().w4_zeros_bytes(N, K, group)


def w4_gemm_path_for(M: int, N: int, K: int) -> int:
    r = load().w4_gemm_path_for(M, N, K)
    if r < 0:
        raise W4Error(-r, "w4_gemm_path_for")
    return r


def _quant_outputs(W, group, packed, scales, where):
    _cuda_tensor(W, "W", torch.bfloat16, 2)
    N, K = W.shape
    if group not in GROUPS or K % GROUP:
        raise W4Error(W4_ERR_UNSUPPORTED, where)
    if packed is None:
        packed = torch.empty((N, K // 2), dtype=torch.uint8, device=W.device)
    if scales is None:
        scales = torch.empty((N, K // group), dtype=torch.bfloat16, device=W.device)
    _cuda_tensor(packed, "packed", torch.uint8, 2)
    _cuda_tensor(scales, "scales", torch.bfloat16, 2)
    if tuple(packed.shape) != (N, K // 2) or tuple(scales.shape) != (N, K // group):
        raise ValueError("packed / scales have the wrong shape")
    return N, K, packed, scales


def w4_quantize_rtn(W: torch.Tensor, group: int = GROUP, packed: torch.Tensor | None = None,
                    scales: torch.Tensor | None = None):
    """RTN symmetric INT4 of W (bf16 [N, K]) -> (packed u8 [N, K/2], scales bf16 [N, K/group])."""
    N, K, packed, scales = _quant_outputs(W, group, packed, scales, "w4_quantize_rtn")
    with torch.cuda.device(W.device):
        _check(load().w4_quantize_rtn(W.data_ptr(), N, K, group, packed.data_ptr(),
                                      scales.data_ptr(), _stream(W.device)), "w4_quantize_rtn")
    return packed, scales


def w4_quantize_rtn_asym(W: torch.Tensor, group: int = GROUP, packed: torch.Tensor | None = None,
                         scales: torch.Tensor | None = None, zeros: torch.Tensor | None = None):
    """RTN asymmetric INT4 of W -> (packed u8 [N, K/2], scales bf16 [N, K/group],
    zeros int8 [N, K/group])."""
    N, K, packed, scales = _quant_outputs(W, group, packed, scales, "w4_quantize_rtn_asym")
    if zeros is None:
        zeros = torch.empty((N, K // group), dtype=torch.int8, device=W.device)
    _cuda_tensor(zeros, "zeros", torch.int8, 2)
    if tuple(zeros.shape) != (N, K // group):
        raise ValueError("zeros has the wrong shape")
    with torch.cuda.device(W.device):
        _check(load().w4_quantize_rtn_asym(W.data_ptr(), N, K, group, packed.data_ptr(), scales.data_ptr(),
                                           zeros.data_ptr(), _stream(W.device)), "w4_quantize_rtn_asym")
    return packed, scales, zeros


def _channel_scales(s: torch.Tensor, K: int) -> None:
    _cuda_tensor(s, "s", torch.float32, 1)
    if s.shape[0] != K:
        raise ValueError("s must hold one scale per input channel (K)")


def w4_quantize_rtn_scaled(W: torch.Tensor, s: torch.Tensor, group: int = GROUP,
                           packed: torch.Tensor | None = None, scales: torch.Tensor | None = None):
    """RTN of the channel-scaled weights W' = bf16(W · s) (s fp32 [K], finite, > 0)
    -> (packed u8 [N, K/2], scales bf16 [N, K/128])."""
    _cuda_tensor(W, "W", torch.bfloat16, 2)
    N, K = W.shape
    _channel_scales(s, K)
    if group != GROUP or K % GROUP:
        raise W4Error(W4_ERR_UNSUPPORTED, "w4_quantize_rtn_scaled")
    if packed is None:
        packed = torch.empty((N, K // 2), dtype=torch.uint8, device=W.device)
    if scales is None:
        scales = torch.empty((N, K // GROUP), dtype=torch.bfloat16, device=W.device)
    _cuda_tensor(packed, "packed", torch.uint8, 2)
    _cuda_tensor(scales, "scales", torch.bfloat16, 2)
    if tuple(packed.shape) != (N, K // 2) or tuple(scales.shape) != (N, K // GROUP):
        raise ValueError("packed / scales have the wrong shape")
    with torch.cuda.device(W.device):
        _check(load().w4_quantize_rtn_scaled(W.data_ptr(), N, K, group, s.data_ptr(), packed.data_ptr(),
                                             scales.data_ptr(), _stream(W.device)), "w4_quantize_rtn_scaled")
    return packed, scales


def w4_scale_activations(x: torch.Tensor, s: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """x' = bf16(x / s): x bf16 [M, K], s fp32 [K] -> bf16 [M, K]; out may be x (in place)."""
    _cuda_tensor(x, "x", torch.bfloat16, 2)
    M, K = x.shape
    _channel_scales(s, K)
    if out is None:
        out = torch.empty_like(x)
    _cuda_tensor(out, "out", torch.bfloat16, 2)
    if tuple(out.shape) != (M, K):
        raise ValueError("out has the wrong shape")
    with torch.cuda.device(x.device):
        _check(load().w4_scale_activations(x.data_ptr(), M, K, s.data_ptr(), out.data_ptr(),
                                           _stream(x.device)), "w4_scale_activations")
    return out


def w4_gptq_factor(H: torch.Tensor, damp: float = 0.01, U: torch.Tensor | None = None,
                   workspace: torch.Tensor | None = None) -> torch.Tensor:
    """U (fp64 [K, K], upper triangle) with Uᵀ U = (H + λI)⁻¹, λ = damp·mean(diag H)."""
    _cuda_tensor(H, "H", torch.float32, 2)
    K = H.shape[0]
    if tuple(H.shape) != (K, K):
        raise ValueError("H must be square")
    if U is None:
        U = torch.empty((K, K), dtype=torch.float64, device=H.device)
    _cuda_tensor(U, "U", torch.float64, 2)
    if tuple(U.shape) != (K, K):
        raise ValueError("U must be [K, K]")
    with torch.cuda.device(H.device):
        need = load().w4_gptq_factor_workspace_bytes(K)
        if need == 0:
            raise W4Error(W4_ERR_UNSUPPORTED, "w4_gptq_factor_workspace_bytes")
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=H.device)
        _cuda_tensor(workspace, "workspace", torch.uint8, 1)
        _check(load().w4_gptq_factor(H.data_ptr(), K, float(damp), U.data_ptr(), workspace.data_ptr(),
                                     workspace.numel(), _stream(H.device)), "w4_gptq_factor")
    return U


def w4_gptq_quantize(W: torch.Tensor, U: torch.Tensor, group: int = GROUP, packed: torch.Tensor | None = None,
                     scales: torch.Tensor | None = None, workspace: torch.Tensor | None = None):
    """GPTQ of W (bf16 [N, K]) given U from w4_gptq_factor -> (packed u8 [N, K/2],
    scales bf16 [N, K/group]), the RTN storage."""
    N, K, packed, scales = _quant_outputs(W, group, packed, scales, "w4_gptq_quantize")
    _cuda_tensor(U, "U", torch.float64, 2)
    if tuple(U.shape) != (K, K):
        raise ValueError("U must be [K, K]")
    with torch.cuda.device(W.device):
        need = load().w4_gptq_workspace_bytes(N, K)
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=W.device)
        _cuda_tensor(workspace, "workspace", torch.uint8, 1)
        _check(load().w4_gptq_quantize(W.data_ptr(), N, K, group, U.data_ptr(), packed.data_ptr(),
                                       scales.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                       _stream(W.device)), "w4_gptq_quantize")
    return packed, scales


def w4_gptq_workspace_bytes(N: int, K: int) -> int:
    return load().w4_gptq_workspace_bytes(N, K)


def w4_gptq_factor_workspace_bytes(K: int) -> int:
    return load().w4_gptq_factor_workspace_bytes(K)


def w4_gemm_ex(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
               out: torch.Tensor | None = None, path: int = W4_PATH_AUTO) -> torch.Tensor:
    """y = Ŵ x: x bf16 [M, K], packed u8 [N, K/2], scales bf16 [N, K/128] -> y bf16 [M, N]."""
    _cuda_tensor(x, "x", torch.bfloat16, 2)
    _cuda_tensor(packed, "packed", torch.uint8, 2)
    _cuda_tensor(scales, "scales", torch.bfloat16, 2)
    M, K = x.shape
    N = packed.shape[0]
    if tuple(packed.shape) != (N, K // 2) or tuple(scales.shape) != (N, K // GROUP) or K % GROUP:
        raise ValueError("x / packed / scales shapes disagree")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _cuda_tensor(out, "out", torch.bfloat16, 2)
    if tuple(out.shape) != (M, N):
        raise ValueError("out has the wrong shape")
    with torch.cuda.device(x.device):
        _check(load().w4_gemm_ex(x.data_ptr(), M, N, K, packed.data_ptr(), scales.data_ptr(),
                                 out.data_ptr(), _stream(x.device), path), "w4_gemm")
    return out


def w4_gemm(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor,
            out: torch.Tensor | None = None) -> torch.Tensor:
    return w4_gemm_ex(x, packed, scales, out, W4_PATH_AUTO)


def w4_gemm_affine(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor | None = None,
                   group: int = GROUP, out: torch.Tensor | None = None, path: int = W4_PATH_AUTO) -> torch.Tensor:
    """y = Ŵ x with ŵ = d·(code − zero) per group of ``group`` (zeros int8 [N, K/group] or None)."""
    _cuda_tensor(x, "x", torch.bfloat16, 2)
    _cuda_tensor(packed, "packed", torch.uint8, 2)
    _cuda_tensor(scales, "scales", torch.bfloat16, 2)
    M, K = x.shape
    N = packed.shape[0]
    if group not in GROUPS:
        raise W4Error(W4_ERR_UNSUPPORTED, "w4_gemm_affine")
    if tuple(packed.shape) != (N, K // 2) or K % GROUP or tuple(scales.shape) != (N, K // group):
        raise ValueError("x / packed / scales shapes disagree")
    if zeros is not None:
        _cuda_tensor(zeros, "zeros", torch.int8, 2)
        if tuple(zeros.shape) != (N, K // group):
            raise ValueError("zeros has the wrong shape")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _cuda_tensor(out, "out", torch.bfloat16, 2)
    if tuple(out.shape) != (M, N):
        raise ValueError("out has the wrong shape")
    with torch.cuda.device(x.device):
        _check(load().w4_gemm_affine(x.data_ptr(), M, N, K, group, packed.data_ptr(), scales.data_ptr(),
                                     zeros.data_ptr() if zeros is not None else None, out.data_ptr(),
                                     _stream(x.device), path), "w4_gemm_affine")
    return out


class GroupedPlan:
    """A built grouped-matmul plan: the device memory holding it (a torch
    tensor) and the C descriptor.  Keeps the problems' tensors referenced, since
    the plan records their addresses."""

    def __init__(self, memory: torch.Tensor, plan: _Plan, tensors: list):
        self.memory = memory
        self.plan = plan
        self.tensors = tensors

    @property
    def items(self) -> int:
        return self.plan.items + self.plan.tc_items


def w4_grouped_plan(problems, group: int = GROUP, zeros=None) -> GroupedPlan:
    """Plan for many matmuls y_i = Ŵ_i x_i run by one w4_gemm_grouped call.
    problems: sequence of (x, packed, scales, y) CUDA tensors with the shapes
    of w4_gemm, all on one device.  For the affine formats of w4_gemm_affine:
    group (32, 64 or 128; scales [N, K/group]) and zeros, None or one entry
    per problem (an int8 [N, K/group] tensor, or None for symmetric codes)."""
    problems = list(problems)
    arr, n, device = _problem_array(problems, group)
    tensors = [t for p in problems for t in p]
    affine = group != GROUP or zeros is not None
    zarr = None
    if zeros is not None:
        zeros = list(zeros)
        if len(zeros) != n:
            raise ValueError("zeros needs one entry per problem")
        zarr = (_vp * n)()
        for i, (z, (x, packed, _, _)) in enumerate(zip(zeros, problems)):
            if z is None:
                continue
            _cuda_tensor(z, "zeros", torch.int8, 2)
            if tuple(z.shape) != (packed.shape[0], x.shape[1] // group) or z.device != device:
                raise ValueError(f"problem {i}: zeros must be int8 [N, K/group] on the problems' device")
            zarr[i] = z.data_ptr()
            tensors.append(z)
    with torch.cuda.device(device):
        if affine:
            nbytes = load().w4_grouped_plan_bytes_affine(n, arr, int(group), zarr)
        else:
            nbytes = load().w4_grouped_plan_bytes(n, arr)
        size = max(nbytes, 128)
        memory = torch.empty(size + 128, dtype=torch.uint8, device=device)
        off = (-memory.data_ptr()) % 128
        plan = _Plan()
        if affine:
            status = load().w4_grouped_plan_init_affine(ctypes.byref(plan), memory.data_ptr() + off, nbytes, n, arr,
                                                        int(group), zarr)
        else:
            status = load().w4_grouped_plan_init(ctypes.byref(plan), memory.data_ptr() + off, nbytes, n, arr)
        if status == W4_OK and nbytes == 0:
            status = W4_ERR_INVALID_ARG
        _check(status, "w4_grouped_plan_init")
    return GroupedPlan(memory, plan, tensors)


def _problem_array(problems, group: int = GROUP):
    """The w4_gemm_problem array of (x, packed, scales, y) tuples, after the
    shape, dtype and device checks (scales [N, K/group]); returns (array,
    count, device)."""
    problems = list(problems)
    if not problems:
        raise ValueError("no problems")
    arr = (_Problem * len(problems))()
    device = problems[0][0].device
    for i, (x, packed, scales, y) in enumerate(problems):
        _cuda_tensor(x, "x", torch.bfloat16, 2)
        _cuda_tensor(packed, "packed", torch.uint8, 2)
        _cuda_tensor(scales, "scales", torch.bfloat16, 2)
        _cuda_tensor(y, "y", torch.bfloat16, 2)
        M, K = x.shape
        N = packed.shape[0]
        if tuple(packed.shape) != (N, K // 2) or tuple(scales.shape) != (N, K // group) or tuple(y.shape) != (M, N):
            raise ValueError(f"problem {i}: x / packed / scales / y shapes disagree")
        if x.device != device or packed.device != device or scales.device != device or y.device != device:
            raise ValueError("all tensors of a grouped call must be on one device")
        arr[i] = _Problem(x.data_ptr(), M, N, K, packed.data_ptr(), scales.data_ptr(), y.data_ptr())
    return arr, len(problems), device


def w4_gemm_grouped_noalloc(problems) -> None:
    """Every problem (x, packed, scales, y) through the library's static plan
    buffer (no caller memory, no allocation; see w4.h for its race rules)."""
    arr, n, device = _problem_array(problems)
    with torch.cuda.device(device):
        _check(load().w4_gemm_grouped_noalloc(n, arr, _stream(device)), "w4_gemm_grouped_noalloc")


def w4_gemm_grouped(plan: GroupedPlan) -> None:
    """Runs every problem of the plan on the current stream of its device."""
    device = torch.device("cuda", plan.plan.device)
    with torch.cuda.device(device):
        _check(load().w4_gemm_grouped(ctypes.byref(plan.plan), _stream(device)), "w4_gemm_grouped")


def w4_last_device_status(device=None) -> int:
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(device):
        return load().w4_last_device_status(_stream(device))


def w4_wait_probe(limit_ns: int, arrive: bool, device=None) -> None:
    device = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(device):
        _check(load().w4_wait_probe(int(limit_ns), int(bool(arrive)), _stream(device)), "w4_wait_probe")


# The cache's calls come many to a step and their kernels last microseconds: their checks take each tensor's type, device
# (one integer) and strides once, and the device is switched only where it is another.
def _device_index(t: torch.Tensor, name: str) -> int:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _typed(t: torch.Tensor, name: str, dtype: torch.dtype, index: int) -> None:
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index:
        return
    if not isinstance(t, torch.Tensor) or t.get_device() < 0:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype is not dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    raise ValueError(f"{name} must be on cuda:{index}")


def _vector(t: torch.Tensor, name: str, dtype: torch.dtype, n: int, index: int) -> int:
    """Address of a contiguous tensor of n values."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != index:
        _typed(t, name, dtype, index)
    if t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous tensor of {n} values")
    return t.data_ptr()


def _strides(t: torch.Tensor, name: str, dtype: torch.dtype, ndim: int, index: int):
    """Strides of a tensor with unit stride in its last dimension."""
    if not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != index:
        _typed(t, name, dtype, index)
    strides = t.stride()
    if len(strides) != ndim or (strides[-1] != 1 and t.shape[-1] > 1 and t.numel() > 0):
        raise ValueError(f"{name} must be a {ndim}-D tensor with unit stride in its last dimension")
    return strides


def _rows(t: torch.Tensor, name: str, shape, index: int) -> _Rows:
    strides = _strides(t, name, torch.bfloat16, 3, index)
    if t.shape != shape:
        raise ValueError(f"{name} must be {shape}, got {tuple(t.shape)}")
    return _Rows(t.data_ptr(), strides[0], strides[1])


def _kv_cache(k_cache, v_cache, k_scales, v_scales, index) -> _KvCache:
    """The w4_kv_cache of key and value pages [pages, page_size, kv_heads, head_dim]
    (bf16, or int8 with scales bf16 [pages, kv_heads, page_size])."""
    dtype = k_cache.dtype if isinstance(k_cache, torch.Tensor) else None
    if dtype is not torch.bfloat16 and dtype is not torch.int8:
        raise TypeError("k_cache must be a bfloat16 or int8 CUDA tensor")
    strides = _strides(k_cache, "k_cache", dtype, 4, index)
    shape = k_cache.shape
    if _strides(v_cache, "v_cache", dtype, 4, index) != strides or v_cache.shape != shape:
        raise ValueError("k_cache and v_cache must have one shape and the same strides")
    pages, page_size, heads, dim = shape
    k_scale = v_scale = None
    if dtype is torch.int8:
        for t, name in ((k_scales, "k_scales"), (v_scales, "v_scales")):
            _typed(t, name, torch.bfloat16, index)
            if t.shape != (pages, heads, page_size) or not t.is_contiguous():
                raise ValueError(f"{name} must be a contiguous [pages, kv_heads, page_size] tensor")
        k_scale, v_scale = k_scales.data_ptr(), v_scales.data_ptr()
    elif k_scales is not None or v_scales is not None:
        raise ValueError("a bfloat16 cache has no scales")
    return _KvCache(k_cache.data_ptr(), v_cache.data_ptr(), k_scale, v_scale, pages, strides[0], strides[1], strides[2],
                    page_size, heads, dim, 16 if k_scale is None else 8)


# The address of a device's current stream (what torch.cuda.current_stream(i).cuda_stream gives, without the objects).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)
# (where a tensor is on the GPU, CUDA has been set up)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
# Memory of the caching allocator without a tensor around it, for the time of a call (a tensor costs 2 µs more).
_raw_alloc = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_alloc", None)
_raw_delete = getattr(torch._C, "_cuda_cudaCachingAllocator_raw_delete", None)


def _call(name: str, index: int, *args) -> None:
    """Runs a library function on the current stream of the device."""
    fn = getattr(_lib or load(), name)
    if _current_device() == index:
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status != W4_OK:
        raise W4Error(status, name)


def _compiled():
    """The compiled module: its functions return NotImplemented where a call is not the usual one."""
    if _fast is None:
        load()
        if _fast is None:
            raise RuntimeError(f"{_PKG}/_binding.so cannot be loaded: build it with `python -m gemm_rtn_sym_gb300.build`") from _fast_error
    return _fast


def _result(done, name: str):
    """What a compiled function returned; a status (an int) is an error that came up at a launch."""
    if type(done) is int:
        raise W4Error(done, name)
    return done


def w4_kv_pages(lens: torch.Tensor, target: torch.Tensor, block_table: torch.Tensor, free_pages: torch.Tensor,
                free_range: torch.Tensor, page_size: int, tokens: int, new_lens: torch.Tensor | None = None,
                starts: torch.Tensor | None = None, slots: torch.Tensor | None = None,
                positions: torch.Tensor | None = None, free_range_out: torch.Tensor | None = None,
                holders: torch.Tensor | None = None):
    """Moves requests from `lens` to `target` tokens (int32 [B]): takes pages from, and gives them back to, the
    ring free_pages (int32 [pages]; entries free_range[0] to free_range[1], int64 [2]), updates block_table (int32
    [B, width]) and returns (new_lens int32 [B], starts int32 [B + 1], slots int64 [tokens], positions int32
    [tokens], free_range_out int64 [2]).  `tokens`: the new tokens of all requests together.  holders (int32 [pages],
    in and out): the table entries that each page stands in, where requests share pages (w4_kv_fork); a page goes back to
    the ring when its last holder lets go."""
    if holders is not None:
        done = _compiled().kv_pages_held(lens, target, block_table, free_pages, free_range, page_size, tokens, holders,
                                        new_lens, starts, slots, positions, free_range_out)
        if done is not NotImplemented:
            return _result(done, "w4_kv_pages_held")
    index = _device_index(block_table, "block_table")
    stride = _strides(block_table, "block_table", torch.int32, 2, index)[0]
    B, width = block_table.shape
    dev = block_table.device
    i32, i64 = torch.int32, torch.int64
    outs, addresses = [], []
    for t, name, dtype, n in ((new_lens, "new_lens", i32, B), (starts, "starts", i32, B + 1), (slots, "slots", i64, tokens),
                              (positions, "positions", i32, tokens), (free_range_out, "free_range_out", i64, 2)):
        if t is None:
            t = torch.empty(n, dtype=dtype, device=dev)
            addresses.append(t.data_ptr())
        else:
            addresses.append(_vector(t, name, dtype, n, index))
        outs.append(t)
    pages = free_pages.numel()
    args = (_vector(lens, "lens", i32, B, index), _vector(target, "target", i32, B, index), B, page_size,
            _vector(free_pages, "free_pages", i32, pages, index), pages, _vector(free_range, "free_range", i64, 2, index),
            block_table.data_ptr(), stride, width, tokens)
    if holders is None:
        _call("w4_kv_pages", index, *args, *addresses)
    else:
        size = load().w4_kv_pages_held_workspace_bytes(B, width, pages)
        scratch = torch.empty(size, dtype=torch.uint8, device=dev)
        _call("w4_kv_pages_held", index, *args, _vector(holders, "holders", i32, pages, index), *addresses,
              scratch.data_ptr(), size)
    return tuple(outs)


def _outputs(outs, index: int, dev):
    """Tensors and addresses of outputs (tensor or None, name, dtype, shape): contiguous, made where they are None."""
    tensors, addresses = [], []
    for t, name, dtype, shape in outs:
        if t is None:
            t = torch.empty(shape, dtype=dtype, device=dev)
        elif not isinstance(t, torch.Tensor) or t.dtype is not dtype or t.get_device() != index:
            _typed(t, name, dtype, index)
        if t.shape != shape or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous tensor of shape {shape}")
        tensors.append(t)
        addresses.append(t.data_ptr())
    return tensors, addresses


def w4_kv_fork(lens: torch.Tensor, source: torch.Tensor, keep: torch.Tensor, block_table: torch.Tensor,
               holders: torch.Tensor, free_pages: torch.Tensor, free_range: torch.Tensor, page_size: int,
               new_lens: torch.Tensor | None = None, copies: torch.Tensor | None = None,
               free_range_out: torch.Tensor | None = None):
    """Lets requests of length 0 begin as the first keep[b] tokens of request source[b] (int32 [B]; −1: none): full pages
    are shared, with one more holder (int32 [pages]) each; a page filled in part gets a page of its own from the ring,
    to be copied.  Updates block_table (int32 [B, width]) and holders, and returns (new_lens int32 [B], copies int32
    [3, B] for w4_kv_copy, free_range_out int64 [2])."""
    done = _compiled().kv_fork(lens, source, keep, block_table, holders, free_pages, free_range, page_size, new_lens, copies,
                              free_range_out)
    if done is not NotImplemented:
        return _result(done, "w4_kv_fork")
    index = _device_index(block_table, "block_table")
    stride = _strides(block_table, "block_table", torch.int32, 2, index)[0]
    B, width = block_table.shape
    i32, i64 = torch.int32, torch.int64
    outs, addresses = _outputs(((new_lens, "new_lens", i32, (B,)), (copies, "copies", i32, (3, B)),
                                (free_range_out, "free_range_out", i64, (2,))), index, block_table.device)
    pages = free_pages.numel()
    _call("w4_kv_fork", index, _vector(lens, "lens", i32, B, index), _vector(source, "source", i32, B, index),
          _vector(keep, "keep", i32, B, index), B, page_size, block_table.data_ptr(), stride, width,
          _vector(holders, "holders", i32, pages, index), _vector(free_pages, "free_pages", i32, pages, index), pages,
          _vector(free_range, "free_range", i64, 2, index), *addresses)
    return tuple(outs)


def w4_kv_compact(lens: torch.Tensor, block_table: torch.Tensor, holders: torch.Tensor, free_range: torch.Tensor,
                  page_size: int, new_table: torch.Tensor | None = None, new_holders: torch.Tensor | None = None,
                  free_pages: torch.Tensor | None = None, free_range_out: torch.Tensor | None = None,
                  copies: torch.Tensor | None = None):
    """Moves the pages in use (holders above 0) to the lowest ids.  Returns (new_table int32 [B, width], new_holders and
    the ring free_pages int32 [pages], free_range_out int64 [2], copies int32 [3, pages // 2] for w4_kv_copy)."""
    done = _compiled().kv_compact(lens, block_table, holders, free_range, page_size, new_table, new_holders, free_pages,
                                 free_range_out, copies)
    if done is not NotImplemented:
        return _result(done, "w4_kv_compact")
    index = _device_index(block_table, "block_table")
    stride = _strides(block_table, "block_table", torch.int32, 2, index)[0]
    B, width = block_table.shape
    i32, i64 = torch.int32, torch.int64
    pages = holders.numel()
    outs, addresses = _outputs(((new_table, "new_table", i32, (B, width)), (new_holders, "new_holders", i32, (pages,)),
                                (free_pages, "free_pages", i32, (pages,)), (free_range_out, "free_range_out", i64, (2,)),
                                (copies, "copies", i32, (3, pages // 2))), index, block_table.device)
    _call("w4_kv_compact", index, _vector(lens, "lens", i32, B, index), B, page_size, block_table.data_ptr(), stride, width,
          _vector(holders, "holders", i32, pages, index), pages, _vector(free_range, "free_range", i64, 2, index),
          addresses[0], width, *addresses[1:])
    return tuple(outs)


def w4_kv_copy(k_cache: torch.Tensor, v_cache: torch.Tensor, copies: torch.Tensor, k_scales: torch.Tensor | None = None,
               v_scales: torch.Tensor | None = None) -> None:
    """Copies the first copies[2][i] tokens of page copies[0][i] to page copies[1][i] (int32 [3, n]; −1, −1: nothing), keys,
    values and scales."""
    if _result(_compiled().kv_copy(k_cache, v_cache, copies, k_scales, v_scales), "w4_kv_copy") is None:
        return
    index = _device_index(k_cache, "k_cache")
    cache = _kv_cache(k_cache, v_cache, k_scales, v_scales, index)
    _typed(copies, "copies", torch.int32, index)
    if copies.dim() != 2 or copies.shape[0] != 3 or not copies.is_contiguous():
        raise ValueError("copies must be a contiguous [3, n] tensor")
    _call("w4_kv_copy", index, cache, copies.data_ptr(), copies.shape[1])


def _append(name, q, k, v, positions, cos, sin, k_cache, v_cache, slots, sections, cycled, paired, k_scales, v_scales, q_out,
            norm=None):
    index = _device_index(k, "k")
    cache = _kv_cache(k_cache, v_cache, k_scales, v_scales, index)
    T = k.shape[0]
    dim = cache.head_dim
    kv_shape = (T, cache.kv_heads, dim)
    if cos is None:
        rope = _Rope()
    else:
        _typed(cos, "cos", torch.float32, index)
        _typed(sin, "sin", torch.float32, index)
        rows = cos.shape
        if len(rows) != 2 or sin.shape != rows or not cos.is_contiguous() or not sin.is_contiguous():
            raise ValueError("cos and sin must be contiguous [rows, rotary / 2] tensors of one shape")
        sections = (rows[1],) if sections is None else tuple(sections)
        axes = len(sections)
        _typed(positions, "positions", torch.int32, index)
        shape, strides = positions.shape, positions.stride()
        if not 1 <= axes <= 4 or (shape != (axes, T) and shape != (T,)) or (strides[-1] != 1 and T > 1):
            raise ValueError("positions must be [T], or [axes, T] with one section for each of 1 to 4 axes, with unit "
                             "stride in the last dimension")
        rope = _Rope(positions.data_ptr(), strides[0] if len(shape) == 2 else 0, cos.data_ptr(), sin.data_ptr(), rows[0],
                     2 * rows[1], axes, sections, cycled, paired)
    rows_q = rows_out = None
    q_heads = 0
    if q is not None:
        q_heads = q.shape[1]
        shape = (T, q_heads, dim)
        if q_out is None:
            q_out = torch.empty(shape, dtype=torch.bfloat16, device=k.device)
        rows_q, rows_out = _rows(q, "q", shape, index), _rows(q_out, "q_out", shape, index)
    args = (T, q_heads, rows_q, rows_out, _rows(k, "k", kv_shape, index), _rows(v, "v", kv_shape, index),
            _vector(slots, "slots", torch.int64, T, index))
    if norm is None:
        _call(name, index, cache, rope, *args)
    else:
        q_weight, k_weight, eps, unit_offset = norm
        dtype = k_weight.dtype if isinstance(k_weight, torch.Tensor) else None
        if dtype is not torch.bfloat16 and dtype is not torch.float32:
            raise TypeError("k_weight must be a bfloat16 or float32 CUDA tensor")
        weights = _Norm(None if q is None else _vector(q_weight, "q_weight", dtype, dim, index),
                        _vector(k_weight, "k_weight", dtype, dim, index), 16 if dtype is torch.bfloat16 else 32, eps,
                        unit_offset)
        _call(name, index, cache, rope, weights, *args)
    return q_out


def w4_kv_append(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor | None,
                 cos: torch.Tensor | None, sin: torch.Tensor | None, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 slots: torch.Tensor, sections=None, cycled: bool = False, paired: bool = False,
                 k_scales: torch.Tensor | None = None, v_scales: torch.Tensor | None = None,
                 q_out: torch.Tensor | None = None) -> torch.Tensor | None:
    """Rotates q (bf16 [T, q_heads, head_dim]) and k ([T, kv_heads, head_dim]) by the rows of cos and sin (fp32
    [rows, rotary / 2]) at positions (int32 [T], or [axes, T] with `sections` frequencies per axis) and writes k
    and v to their slots (int64 [T], −1: none) of the cache.  Returns the rotated queries (q_out; may be q).
    cos None: no rotation; q None: keys and values only."""
    return _append("w4_kv_append", q, k, v, positions, cos, sin, k_cache, v_cache, slots, sections, cycled, paired,
                   k_scales, v_scales, q_out)


def w4_kv_append_norm(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, q_weight: torch.Tensor | None,
                      k_weight: torch.Tensor, positions: torch.Tensor | None, cos: torch.Tensor | None,
                      sin: torch.Tensor | None, k_cache: torch.Tensor, v_cache: torch.Tensor, slots: torch.Tensor,
                      eps: float = 1e-6, unit_offset: bool = False, sections=None, cycled: bool = False,
                      paired: bool = False, k_scales: torch.Tensor | None = None, v_scales: torch.Tensor | None = None,
                      q_out: torch.Tensor | None = None) -> torch.Tensor | None:
    """w4_kv_append of queries and keys normalised head by head before they turn: x · (mean(x²) + eps)^−½ · w over each
    row's head_dim values, with q_weight and k_weight (bf16 or fp32 [head_dim]; unit_offset: w = 1 + weight) for all
    heads; one rounding in all."""
    done = _compiled().kv_append_norm(q, k, v, q_weight, k_weight, positions, cos, sin, k_cache, v_cache, slots, eps,
                                     unit_offset, sections, cycled, paired, k_scales, v_scales, q_out)
    if done is not NotImplemented:
        return _result(done, "w4_kv_append_norm")[0]
    return _append("w4_kv_append_norm", q, k, v, positions, cos, sin, k_cache, v_cache, slots, sections, cycled, paired,
                   k_scales, v_scales, q_out, (q_weight, k_weight, eps, unit_offset))


def w4_attn_decode_workspace_bytes(q: torch.Tensor, k_cache: torch.Tensor, requests: int) -> int:
    """Bytes of workspace of w4_attn_decode for these queries, cache pages and number of requests."""
    cache = _KvCache(kv_heads=k_cache.shape[2], head_dim=k_cache.shape[3], format=8 if k_cache.dtype == torch.int8 else 16)
    return load().w4_attn_decode_workspace_bytes(cache, requests, q.shape[0], q.shape[1])


def w4_attn_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                   lens: torch.Tensor, starts: torch.Tensor | None = None, k_scales: torch.Tensor | None = None,
                   v_scales: torch.Tensor | None = None, scale: float | None = None, window: int = 0,
                   out: torch.Tensor | None = None, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """Attention of the newest tokens q (bf16 [T, q_heads, head_dim]) of each request over its pages (block_table
    int32 [B, width]; lens int32 [B], the new tokens counted) -> bf16 like q.  Rows starts[b] to starts[b + 1] − 1
    (int32 [B + 1]) are request b's; without starts, T / B each.  scale: 1/√head_dim by default; window: tokens
    each row sees, its own counted (0: all); out may be q."""
    index = _device_index(q, "q")
    cache = _kv_cache(k_cache, v_cache, k_scales, v_scales, index)
    stride = _strides(block_table, "block_table", torch.int32, 2, index)[0]
    B, width = block_table.shape
    if q.dim() != 3:
        raise ValueError("q must be a 3-D tensor")
    T, q_heads, dim = q.shape
    shape = (T, q_heads, cache.head_dim)
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=q.device)
    rows_q, rows_out = _rows(q, "q", shape, index), _rows(out, "out", shape, index)
    args = (cache, B, T, q_heads, rows_q, rows_out, block_table.data_ptr(), stride, width,
            _vector(lens, "lens", torch.int32, B, index),
            None if starts is None else _vector(starts, "starts", torch.int32, B + 1, index),
            dim ** -0.5 if scale is None else scale, window)
    _attend("w4_attn_decode", index, args, workspace, q.device,
            lambda: (_lib or load()).w4_attn_decode_workspace_bytes(cache, B, T, q_heads))
    return out


def _attend(name: str, index: int, args, workspace, dev, bytes_needed) -> None:
    """Runs a library function with the caller's workspace, or one for the time of the call."""
    if workspace is not None:
        size = workspace.numel()
        _call(name, index, *args, _vector(workspace, "workspace", torch.uint8, size, index), size)
        return
    size = bytes_needed()
    if size and _raw_alloc and _raw_delete and _current_device() == index:
        scratch = _raw_alloc(size, _raw_stream(index))
        try:
            _call(name, index, *args, scratch, size)
        finally:
            _raw_delete(scratch)  # the stream's next allocations may have it
    else:
        scratch = torch.empty(size, dtype=torch.uint8, device=dev)  # (a name keeps it until the launch)
        _call(name, index, *args, scratch.data_ptr(), size)


def w4_attn_decode_shared_workspace_bytes(q: torch.Tensor, k_cache: torch.Tensor, requests: int, groups: int) -> int:
    """Bytes of workspace of w4_attn_decode_shared for these queries, cache pages and numbers of requests and groups."""
    cache = _KvCache(kv_heads=k_cache.shape[2], head_dim=k_cache.shape[3], format=8 if k_cache.dtype == torch.int8 else 16)
    return load().w4_attn_decode_shared_workspace_bytes(cache, requests, q.shape[0], q.shape[1], groups)


def w4_attn_decode_shared(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_table: torch.Tensor,
                          lens: torch.Tensor, group_starts: torch.Tensor, prefix_table: torch.Tensor,
                          prefix_lens: torch.Tensor, starts: torch.Tensor | None = None,
                          k_scales: torch.Tensor | None = None, v_scales: torch.Tensor | None = None,
                          scale: float | None = None, out: torch.Tensor | None = None,
                          workspace: torch.Tensor | None = None) -> torch.Tensor:
    """w4_attn_decode of requests that share prefixes.  Requests group_starts[g] to group_starts[g + 1] − 1 (int32
    [groups + 1]) begin with the prefix_lens[g] tokens (int32 [groups]) in the pages prefix_table[g] (int32 [groups,
    width]), which are read once for all of them; what follows is in their own pages, at the places that block_table has
    for it.  lens counts the prefix.  Requests outside of the groups, and those whose new tokens do not all lie behind the
    prefix, are attended over their own pages.  Few requests behind a short prefix are faster by w4_attn_decode (w4.h)."""
    if workspace is None:
        done = _compiled().attn_decode_shared(q, k_cache, v_cache, block_table, lens, group_starts, prefix_table, prefix_lens,
                                             starts, k_scales, v_scales, scale, out)
        if done is not NotImplemented:
            return _result(done, "w4_attn_decode_shared")[0]
    index = _device_index(q, "q")
    cache = _kv_cache(k_cache, v_cache, k_scales, v_scales, index)
    stride = _strides(block_table, "block_table", torch.int32, 2, index)[0]
    prefix_stride = _strides(prefix_table, "prefix_table", torch.int32, 2, index)[0]
    B, width = block_table.shape
    groups, prefix_width = prefix_table.shape
    if q.dim() != 3:
        raise ValueError("q must be a 3-D tensor")
    T, q_heads, dim = q.shape
    shape = (T, q_heads, cache.head_dim)
    if out is None:
        out = torch.empty(shape, dtype=torch.bfloat16, device=q.device)
    rows_q, rows_out = _rows(q, "q", shape, index), _rows(out, "out", shape, index)
    i32 = torch.int32
    args = (cache, B, T, q_heads, rows_q, rows_out, block_table.data_ptr(), stride, width, _vector(lens, "lens", i32, B, index),
            None if starts is None else _vector(starts, "starts", i32, B + 1, index), groups,
            _vector(group_starts, "group_starts", i32, groups + 1, index), prefix_table.data_ptr(), prefix_stride,
            prefix_width, _vector(prefix_lens, "prefix_lens", i32, groups, index), dim ** -0.5 if scale is None else scale)
    _attend("w4_attn_decode_shared", index, args, workspace, q.device,
            lambda: (_lib or load()).w4_attn_decode_shared_workspace_bytes(cache, B, T, q_heads, groups))
    return out
