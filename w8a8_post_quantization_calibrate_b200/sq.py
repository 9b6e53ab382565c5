"""Thin Python binding of libsq (include/sq.h): argument marshalling only.

Every function has the name of the C entry point it calls. Tensors are torch
CUDA tensors (device memory and the current stream come from PyTorch); outputs
not supplied by the caller are allocated with torch. All computation happens in
libsq's kernels: importing this module loads libsq.so and raises if it has not
been built -- there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
import re
import struct
import typing

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# SQ_LIBRARY=debug loads the -DSQ_DEBUG build (index checks in the kernels)
LIB_PATH = os.path.join(_PKG, "libsq_debug.so" if os.environ.get("SQ_LIBRARY") == "debug" else "libsq.so")
HEADER = os.path.join(os.path.dirname(_PKG), "include", "sq.h")

SQ_OK, SQ_ERR_INVALID_ARG, SQ_ERR_UNSUPPORTED, SQ_ERR_CUDA, SQ_ERR_TIMEOUT, SQ_ERR_BOUNDS = 0, 1, 2, 3, 4, 5
SQ_F32, SQ_BF16, SQ_I32 = 0, 1, 2
STATUS_NAMES = {0: "SQ_OK", 1: "SQ_ERR_INVALID_ARG", 2: "SQ_ERR_UNSUPPORTED", 3: "SQ_ERR_CUDA",
                4: "SQ_ERR_TIMEOUT", 5: "SQ_ERR_BOUNDS"}


class SqError(RuntimeError):
    def __init__(self, status: int, where: str, message: str):
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}: {message}")
        self.status = status


if not os.path.exists(LIB_PATH):
    raise ImportError(f"{os.path.basename(LIB_PATH)} is not built ({LIB_PATH}); run "
                      "`python -m w8a8_post_quantization_calibrate_b200.build`"
                      + (" --debug" if LIB_PATH.endswith("_debug.so") else ""))

_lib = ctypes.CDLL(LIB_PATH)
_vp, _i64, _f32, _sz, _int = ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t, ctypes.c_int

_SIGS = {
    "sq_version": ([], _int),
    "sq_calibrate_absmax": ([_vp, _int, _i64, _i64, _vp, _vp], _int),
    "sq_smooth_factors": ([_vp, _vp, _i64, _f32, _f32, _vp, _vp], _int),
    "sq_fold_quant_weights": ([_vp, _int, _i64, _i64, _vp, _vp, _vp, _vp], _int),
    "sq_smooth_quant_act": ([_vp, _int, _i64, _i64, _vp, _vp, _vp, _vp], _int),
    "sq_calibrate_absmax_pair": ([_vp, _i64, _vp, _i64, _int, _i64, _vp, _vp, _vp], _int),
    "sq_fold_smooth_quant_pair": ([_vp, _i64, _vp, _i64, _int, _i64, _vp, _vp, _vp, _vp, _vp, _vp], _int),
    "sq_fold_smooth_quant_pair_e4m3": ([_vp, _i64, _vp, _i64, _int, _i64, _vp, _vp, _vp, _vp, _vp, _vp], _int),
    "sq_fold_quant_weights_e4m3": ([_vp, _int, _i64, _i64, _vp, _vp, _vp, _vp], _int),
    "sq_smooth_quant_act_e4m3": ([_vp, _int, _i64, _i64, _vp, _vp, _vp, _vp], _int),
    "sq_w8a8_gemm_e4m3": ([_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _int, _vp], _int),
    "sq_tensor_absmax": ([_vp, _int, _i64, _i64, _vp, _vp, _vp], _int),
    "sq_quant_act_per_tensor": ([_vp, _int, _i64, _i64, _vp, _vp, _vp, _vp, _vp], _int),
    "sq_fold_norm_gain": ([_vp, _int, _i64, _vp, _vp, _vp], _int),
    "sq_rmsnorm_quant_act": ([_vp, _int, _i64, _i64, _vp, _f32, _vp, _vp, _vp, _vp], _int),
    "sq_outlier_split": ([_vp, _i64, _f32, _vp, _vp, _vp, _vp], _int),
    "sq_quant_bulk": ([_vp, _int, _i64, _i64, _vp, _vp, _vp, _vp], _int),
    "sq_gather_columns": ([_vp, _int, _i64, _i64, _vp, _i64, _i64, _vp, _vp], _int),
    "sq_w8a8_gemm_split": ([_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _vp, _i64, _vp, _int, _vp, _sz, _vp],
                           _int),
    "sq_alpha_search_workspace_size": ([_i64, _i64, _i64, _i64], _sz),
    "sq_alpha_search": ([_vp, _vp, _int, _i64, _i64, _i64, _vp, _i64, _f32, _vp, _vp, _vp, _sz, _vp], _int),
    "sq_w8a8_gemm_workspace_size": ([_i64, _i64, _i64], _sz),
    "sq_w8a8_gemm": ([_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _int, _vp, _sz, _vp], _int),
    "sq_w8a8_gemm_noalloc": ([_vp, _vp, _vp, _vp, _i64, _i64, _i64, _vp, _int, _vp], _int),
    "sq_linear_workspace_size": ([_i64, _i64, _i64, _int, _int], _sz),
    "sq_linear_workspace_offsets": ([_i64, _i64, _i64, _int, _int, _vp], _int),
    "sq_linear": ([_vp, _vp, _int, _i64, _i64, _i64, _f32, _f32, _vp, _int, _vp, _sz, _vp], _int),
    "sq_rope_table": ([_vp, _i64, _i64, _i64, ctypes.c_double, _vp, _vp], _int),
    "sq_rope_kv_append": ([_vp, _vp, _i64, _vp, _vp, _i64, _i64, _vp, _i64, _i64, _vp, _i64, _vp, _i64, _int, _vp, _i64,
                           _i64, _int, _vp, _vp, _vp], _int),
    "sq_kv_read": ([_vp, _vp, _i64, _vp, _vp, _i64, _i64, _vp, _vp, _int, _vp], _int),
    "sq_kv_attention_workspace_size": ([_vp, _i64, _i64, _i64], _sz),
    "sq_kv_attention": ([_vp, _i64, _int, _vp, _vp, _i64, _vp, _i64, _i64, _i64, _f32, _vp, _vp, _vp, _sz, _vp], _int),
    "sq_prompt_attention": ([_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i64, _i64, _i64, _i64, _f32, _int, _vp, _vp,
                             _vp], _int),
    "sq_get_status": ([_vp], _int),
    "sq_last_status_site": ([], ctypes.c_uint),
    "sq_last_error_string": ([], ctypes.c_char_p),
    "sq_set_wait_timeout_ms": ([_i64], _int),
    "sq_selftest_wait_timeout": ([_i64, _vp], _int),
    "sq_selftest_dirty_noalloc_scratch": ([_vp], _int),
    "sq_probe_tensor_int8": ([_i64, _vp, _vp, _vp], _int),
}
for _name, (_args, _res) in _SIGS.items():
    _fn = getattr(_lib, _name)
    _fn.argtypes = _args
    _fn.restype = _res


def header_functions() -> list[str]:
    """Names of the functions include/sq.h declares."""
    with open(HEADER) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(sq_[a-z0-9_]+)\s*\(", text)))


def _check(status: int, where: str) -> None:
    if status != SQ_OK:
        msg = _lib.sq_last_error_string().decode(errors="replace")
        raise SqError(status, where, msg)


def _stream(stream) -> int:
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return SQ_F32
    if t.dtype == torch.bfloat16:
        return SQ_BF16
    if t.dtype == torch.int32:
        return SQ_I32
    raise TypeError(f"unsupported dtype {t.dtype}")


def _torch_dtype(code: int):
    return {SQ_F32: torch.float32, SQ_BF16: torch.bfloat16, SQ_I32: torch.int32}[code]


def _dev(t: torch.Tensor, name: str) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def sq_version() -> int:
    return _lib.sq_version()


def sq_calibrate_absmax(x: torch.Tensor, absmax: torch.Tensor, stream=None) -> torch.Tensor:
    """Running per-column max |x| into `absmax` (float32 [cols], in/out)."""
    rows, cols = x.shape
    _check(_lib.sq_calibrate_absmax(_dev(x, "x"), _dt(x), rows, cols, _dev(absmax, "absmax"),
                                    _stream(stream)), "sq_calibrate_absmax")
    return absmax


def sq_smooth_factors(xmax: torch.Tensor, wmax: torch.Tensor, alpha: float, eps: float = 1e-8,
                      s: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    K = xmax.shape[0]
    if s is None:
        s = torch.empty(K, dtype=torch.float32, device=xmax.device)
    _check(_lib.sq_smooth_factors(_dev(xmax, "xmax"), _dev(wmax, "wmax"), K, float(alpha), float(eps),
                                  _dev(s, "s"), _stream(stream)), "sq_smooth_factors")
    return s


def sq_fold_quant_weights(w: torch.Tensor, s: torch.Tensor, wq: torch.Tensor | None = None,
                          w_scale: torch.Tensor | None = None, stream=None):
    N, K = w.shape
    if wq is None:
        wq = torch.empty((N, K), dtype=torch.int8, device=w.device)
    if w_scale is None:
        w_scale = torch.empty(N, dtype=torch.float32, device=w.device)
    _check(_lib.sq_fold_quant_weights(_dev(w, "w"), _dt(w), N, K, _dev(s, "s"), _dev(wq, "wq"),
                                      _dev(w_scale, "w_scale"), _stream(stream)), "sq_fold_quant_weights")
    return wq, w_scale


def sq_smooth_quant_act(x: torch.Tensor, s: torch.Tensor, xq: torch.Tensor | None = None,
                        x_scale: torch.Tensor | None = None, stream=None):
    T, K = x.shape
    if xq is None:
        xq = torch.empty((T, K), dtype=torch.int8, device=x.device)
    if x_scale is None:
        x_scale = torch.empty(T, dtype=torch.float32, device=x.device)
    _check(_lib.sq_smooth_quant_act(_dev(x, "x"), _dt(x), T, K, _dev(s, "s"), _dev(xq, "xq"),
                                    _dev(x_scale, "x_scale"), _stream(stream)), "sq_smooth_quant_act")
    return xq, x_scale


def sq_calibrate_absmax_pair(x: torch.Tensor, w: torch.Tensor, xmax: torch.Tensor, wmax: torch.Tensor,
                             stream=None):
    """Running column maxima of x into xmax and of w into wmax, one launch."""
    T, K = x.shape
    N = w.shape[0]
    if x.dtype != w.dtype:
        raise TypeError("x and w must have the same dtype")
    _check(_lib.sq_calibrate_absmax_pair(_dev(x, "x"), T, _dev(w, "w"), N, _dt(x), K, _dev(xmax, "xmax"),
                                         _dev(wmax, "wmax"), _stream(stream)), "sq_calibrate_absmax_pair")
    return xmax, wmax


def sq_fold_smooth_quant_pair(w: torch.Tensor, x: torch.Tensor, s: torch.Tensor, wq=None, w_scale=None, xq=None,
                              x_scale=None, stream=None):
    """a3 on w and a4 on x with the same s, in one launch where possible ->
    (wq, w_scale, xq, x_scale)."""
    N, K = w.shape
    T = x.shape[0]
    if x.dtype != w.dtype:
        raise TypeError("x and w must have the same dtype")
    if wq is None:
        wq = torch.empty((N, K), dtype=torch.int8, device=w.device)
    if w_scale is None:
        w_scale = torch.empty(N, dtype=torch.float32, device=w.device)
    if xq is None:
        xq = torch.empty((T, K), dtype=torch.int8, device=x.device)
    if x_scale is None:
        x_scale = torch.empty(T, dtype=torch.float32, device=x.device)
    _check(_lib.sq_fold_smooth_quant_pair(_dev(w, "w"), N, _dev(x, "x"), T, _dt(w), K, _dev(s, "s"), _dev(wq, "wq"),
                                          _dev(w_scale, "w_scale"), _dev(xq, "xq"), _dev(x_scale, "x_scale"),
                                          _stream(stream)), "sq_fold_smooth_quant_pair")
    return wq, w_scale, xq, x_scale


def sq_fold_smooth_quant_pair_e4m3(w: torch.Tensor, x: torch.Tensor, s: torch.Tensor, wq=None, w_scale=None,
                                   xq=None, x_scale=None, stream=None):
    """FP8 E4M3 codes of w (folded) and x (smoothed) in one launch where
    possible -> (wq uint8, w_scale, xq uint8, x_scale)."""
    N, K = w.shape
    T = x.shape[0]
    if x.dtype != w.dtype:
        raise TypeError("x and w must have the same dtype")
    if wq is None:
        wq = torch.empty((N, K), dtype=torch.uint8, device=w.device)
    if w_scale is None:
        w_scale = torch.empty(N, dtype=torch.float32, device=w.device)
    if xq is None:
        xq = torch.empty((T, K), dtype=torch.uint8, device=x.device)
    if x_scale is None:
        x_scale = torch.empty(T, dtype=torch.float32, device=x.device)
    _check(_lib.sq_fold_smooth_quant_pair_e4m3(_dev(w, "w"), N, _dev(x, "x"), T, _dt(w), K, _dev(s, "s"),
                                               _dev(wq, "wq"), _dev(w_scale, "w_scale"), _dev(xq, "xq"),
                                               _dev(x_scale, "x_scale"), _stream(stream)),
           "sq_fold_smooth_quant_pair_e4m3")
    return wq, w_scale, xq, x_scale


def sq_fold_quant_weights_e4m3(w: torch.Tensor, s: torch.Tensor, wq=None, w_scale=None, stream=None):
    """Fold s into W, per-output-channel FP8 E4M3 -> (codes uint8 [N, K], w_scale)."""
    N, K = w.shape
    if wq is None:
        wq = torch.empty((N, K), dtype=torch.uint8, device=w.device)
    if w_scale is None:
        w_scale = torch.empty(N, dtype=torch.float32, device=w.device)
    _check(_lib.sq_fold_quant_weights_e4m3(_dev(w, "w"), _dt(w), N, K, _dev(s, "s"), _dev(wq, "wq"),
                                           _dev(w_scale, "w_scale"), _stream(stream)), "sq_fold_quant_weights_e4m3")
    return wq, w_scale


def sq_smooth_quant_act_e4m3(x: torch.Tensor, s: torch.Tensor, xq=None, x_scale=None, stream=None):
    """Smooth X by s, per-token FP8 E4M3 -> (codes uint8 [T, K], x_scale)."""
    T, K = x.shape
    if xq is None:
        xq = torch.empty((T, K), dtype=torch.uint8, device=x.device)
    if x_scale is None:
        x_scale = torch.empty(T, dtype=torch.float32, device=x.device)
    _check(_lib.sq_smooth_quant_act_e4m3(_dev(x, "x"), _dt(x), T, K, _dev(s, "s"), _dev(xq, "xq"),
                                         _dev(x_scale, "x_scale"), _stream(stream)), "sq_smooth_quant_act_e4m3")
    return xq, x_scale


def sq_w8a8_gemm_e4m3(xq: torch.Tensor, x_scale: torch.Tensor, wq: torch.Tensor, w_scale: torch.Tensor,
                      out_dtype=torch.bfloat16, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    M, K = xq.shape
    N = wq.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype, device=xq.device)
    _check(_lib.sq_w8a8_gemm_e4m3(_dev(xq, "xq"), _dev(x_scale, "x_scale"), _dev(wq, "wq"), _dev(w_scale, "w_scale"),
                                  M, N, K, _dev(y, "y"), _dt(y), _stream(stream)), "sq_w8a8_gemm_e4m3")
    return y


def _opt_dev(t: torch.Tensor | None, name: str):
    return None if t is None else _dev(t, name)


def sq_tensor_absmax(x: torch.Tensor, s: torch.Tensor | None, amax: torch.Tensor | None = None,
                     stream=None) -> torch.Tensor:
    """Running per-tensor max |x / s_j| into `amax` (float32 [1], in/out; a
    fresh zero tensor if not given). s None: max |x|."""
    rows, cols = x.shape
    if amax is None:
        amax = torch.zeros(1, dtype=torch.float32, device=x.device)
    _check(_lib.sq_tensor_absmax(_dev(x, "x"), _dt(x), rows, cols, _opt_dev(s, "s"), _dev(amax, "amax"),
                                 _stream(stream)), "sq_tensor_absmax")
    return amax


def sq_quant_act_per_tensor(x: torch.Tensor, s: torch.Tensor | None, amax: torch.Tensor,
                            xq: torch.Tensor | None = None, x_scale: torch.Tensor | None = None,
                            stream=None):
    T, K = x.shape
    if xq is None:
        xq = torch.empty((T, K), dtype=torch.int8, device=x.device)
    if x_scale is None:
        x_scale = torch.empty(T, dtype=torch.float32, device=x.device)
    _check(_lib.sq_quant_act_per_tensor(_dev(x, "x"), _dt(x), T, K, _opt_dev(s, "s"), _dev(amax, "amax"),
                                        _dev(xq, "xq"), _dev(x_scale, "x_scale"), _stream(stream)),
           "sq_quant_act_per_tensor")
    return xq, x_scale


def sq_fold_norm_gain(gain: torch.Tensor, s: torch.Tensor, gain_folded: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    K = gain.shape[0]
    if gain_folded is None:
        gain_folded = torch.empty(K, dtype=torch.float32, device=gain.device)
    _check(_lib.sq_fold_norm_gain(_dev(gain, "gain"), _dt(gain), K, _dev(s, "s"),
                                  _dev(gain_folded, "gain_folded"), _stream(stream)), "sq_fold_norm_gain")
    return gain_folded


def sq_rmsnorm_quant_act(x: torch.Tensor, gain_folded: torch.Tensor, eps: float,
                         xq: torch.Tensor | None = None, x_scale: torch.Tensor | None = None,
                         inv_rms: torch.Tensor | None = None, want_inv_rms: bool = True, stream=None):
    """RMSNorm with the folded gain, then per-token int8 -> (xq, x_scale, inv_rms or None)."""
    T, K = x.shape
    if xq is None:
        xq = torch.empty((T, K), dtype=torch.int8, device=x.device)
    if x_scale is None:
        x_scale = torch.empty(T, dtype=torch.float32, device=x.device)
    if inv_rms is None and want_inv_rms:
        inv_rms = torch.empty(T, dtype=torch.float32, device=x.device)
    _check(_lib.sq_rmsnorm_quant_act(_dev(x, "x"), _dt(x), T, K, _dev(gain_folded, "gain_folded"),
                                     float(eps), _dev(xq, "xq"), _dev(x_scale, "x_scale"),
                                     _opt_dev(inv_rms, "inv_rms"), _stream(stream)), "sq_rmsnorm_quant_act")
    return xq, x_scale, inv_rms


def sq_w8a8_gemm_workspace_size(M: int, N: int, K: int) -> int:
    return int(_lib.sq_w8a8_gemm_workspace_size(M, N, K))


_ws_cache: dict = {}


def gemm_workspace(M: int, N: int, K: int, device) -> torch.Tensor | None:
    """A zero-filled workspace for sq_w8a8_gemm, cached per (device, size);
    calls that complete leave it zero-filled, as the C API requires."""
    need = sq_w8a8_gemm_workspace_size(M, N, K)
    if need == 0:
        return None
    key = (str(device), need)
    ws = _ws_cache.get(key)
    if ws is None:
        ws = torch.zeros(need, dtype=torch.uint8, device=device)
        _ws_cache[key] = ws
    return ws


def sq_w8a8_gemm(xq: torch.Tensor, x_scale: torch.Tensor | None, wq: torch.Tensor,
                 w_scale: torch.Tensor | None, out_dtype=torch.bfloat16, y: torch.Tensor | None = None,
                 workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    M, K = xq.shape
    N = wq.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype, device=xq.device)
    if workspace is None:
        workspace = gemm_workspace(M, N, K, xq.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(_lib.sq_w8a8_gemm(_dev(xq, "xq"), x_scale.data_ptr() if x_scale is not None else None,
                             _dev(wq, "wq"), w_scale.data_ptr() if w_scale is not None else None,
                             M, N, K, _dev(y, "y"), _dt(y), ws_ptr, ws_bytes, _stream(stream)),
           "sq_w8a8_gemm")
    return y


def sq_w8a8_gemm_noalloc(xq: torch.Tensor, x_scale: torch.Tensor | None, wq: torch.Tensor,
                         w_scale: torch.Tensor | None, out_dtype=torch.bfloat16, y: torch.Tensor | None = None,
                         stream=None) -> torch.Tensor:
    """Decode GEMM (1 <= M <= 16) for callers that cannot allocate device
    memory: libsq keeps the scratch in a fixed array of its own. Only `y`, if
    not given, is allocated here (by torch, for the convenience of Python
    callers); the C call itself allocates nothing."""
    M, K = xq.shape
    N = wq.shape[0]
    for name, t in (("wq", wq), ("x_scale", x_scale), ("w_scale", w_scale), ("y", y)):
        if t is not None and t.device != xq.device:
            raise ValueError(f"{name} is on {t.device}, xq on {xq.device}")
    # the C call takes the scratch of the current device: make it xq's
    with torch.cuda.device(xq.device):
        if y is None:
            y = torch.empty((M, N), dtype=out_dtype, device=xq.device)
        _check(_lib.sq_w8a8_gemm_noalloc(_dev(xq, "xq"), x_scale.data_ptr() if x_scale is not None else None,
                                         _dev(wq, "wq"), w_scale.data_ptr() if w_scale is not None else None,
                                         M, N, K, _dev(y, "y"), _dt(y), _stream(stream)),
               "sq_w8a8_gemm_noalloc")
    return y


def sq_selftest_dirty_noalloc_scratch(stream=None) -> None:
    _check(_lib.sq_selftest_dirty_noalloc_scratch(_stream(stream)), "sq_selftest_dirty_noalloc_scratch")


def sq_outlier_split(xmax: torch.Tensor, threshold: float, keep: torch.Tensor | None = None,
                     idx: torch.Tensor | None = None, count: torch.Tensor | None = None, stream=None):
    """-> (keep float32 [K], idx int32 [K] (first `count` valid), count int32 [1]), all on the device."""
    K = xmax.shape[0]
    if keep is None:
        keep = torch.empty(K, dtype=torch.float32, device=xmax.device)
    if idx is None:
        idx = torch.empty(max(K, 1), dtype=torch.int32, device=xmax.device)
    if count is None:
        count = torch.empty(1, dtype=torch.int32, device=xmax.device)
    _check(_lib.sq_outlier_split(_dev(xmax, "xmax"), K, float(threshold), _dev(keep, "keep"), _dev(idx, "idx"),
                                 _dev(count, "count"), _stream(stream)), "sq_outlier_split")
    return keep, idx, count


def sq_quant_bulk(x: torch.Tensor, keep: torch.Tensor, q: torch.Tensor | None = None,
                  scale: torch.Tensor | None = None, stream=None):
    rows, K = x.shape
    if q is None:
        q = torch.empty((rows, K), dtype=torch.int8, device=x.device)
    if scale is None:
        scale = torch.empty(rows, dtype=torch.float32, device=x.device)
    _check(_lib.sq_quant_bulk(_dev(x, "x"), _dt(x), rows, K, _dev(keep, "keep"), _dev(q, "q"),
                              _dev(scale, "scale"), _stream(stream)), "sq_quant_bulk")
    return q, scale


def sq_gather_columns(x: torch.Tensor, idx: torch.Tensor, n: int, ld: int, out: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    rows, K = x.shape
    if out is None:
        out = torch.empty((rows, ld), dtype=torch.float32, device=x.device)
    _check(_lib.sq_gather_columns(_dev(x, "x"), _dt(x), rows, K, _dev(idx, "idx"), int(n), int(ld),
                                  _dev(out, "out"), _stream(stream)), "sq_gather_columns")
    return out


def sq_w8a8_gemm_split(xq: torch.Tensor, x_scale: torch.Tensor, wq: torch.Tensor, w_scale: torch.Tensor,
                       x_out: torch.Tensor, w_out: torch.Tensor, out_dtype=torch.bfloat16,
                       y: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                       stream=None) -> torch.Tensor:
    M, K = xq.shape
    N = wq.shape[0]
    ld = x_out.shape[1]
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype, device=xq.device)
    if workspace is None:
        workspace = gemm_workspace(M, N, K, xq.device)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(_lib.sq_w8a8_gemm_split(_dev(xq, "xq"), _dev(x_scale, "x_scale"), _dev(wq, "wq"),
                                   _dev(w_scale, "w_scale"), M, N, K, _dev(x_out, "x_out"), _dev(w_out, "w_out"),
                                   ld, _dev(y, "y"), _dt(y), ws_ptr, ws_bytes, _stream(stream)),
           "sq_w8a8_gemm_split")
    return y


def sq_alpha_search_workspace_size(T: int, N: int, K: int, n_alpha: int) -> int:
    return int(_lib.sq_alpha_search_workspace_size(T, N, K, n_alpha))


def sq_alpha_search(x: torch.Tensor, w: torch.Tensor, alphas, eps: float = 1e-8,
                    workspace: torch.Tensor | None = None, stream=None):
    """W8A8 relative output error for each alpha on the calibration batch x
    -> (errors list of float, best alpha). Synchronizes the stream."""
    T, K = x.shape
    N = w.shape[0]
    if x.dtype != w.dtype:
        raise TypeError("x and w must have the same dtype")
    a = (ctypes.c_float * len(alphas))(*[float(v) for v in alphas])
    err = (ctypes.c_double * len(alphas))()
    best = ctypes.c_float(0.0)
    need = sq_alpha_search_workspace_size(T, N, K, len(alphas))
    if workspace is None:
        workspace = torch.zeros(need, dtype=torch.uint8, device=x.device)
    _check(_lib.sq_alpha_search(_dev(x, "x"), _dev(w, "w"), _dt(x), T, N, K, ctypes.cast(a, _vp), len(alphas),
                                float(eps), ctypes.cast(err, _vp), ctypes.cast(ctypes.pointer(best), _vp),
                                workspace.data_ptr(), workspace.numel(), _stream(stream)), "sq_alpha_search")
    return list(err), float(best.value)


def sq_linear_workspace_size(M: int, N: int, K: int, in_dtype=torch.bfloat16, out_dtype=torch.bfloat16) -> int:
    return int(_lib.sq_linear_workspace_size(M, N, K, _dt(torch.empty(0, dtype=in_dtype)),
                                             _dt(torch.empty(0, dtype=out_dtype))))


LINEAR_WORKSPACE_PARTS = ("xmax", "wmax", "s", "xq", "x_scale", "wq", "w_scale")


def sq_linear_workspace_offsets(M: int, N: int, K: int, in_dtype=torch.bfloat16,
                                out_dtype=torch.bfloat16) -> dict:
    """Byte offsets of sq_linear's intermediates inside its workspace."""
    off = (ctypes.c_size_t * len(LINEAR_WORKSPACE_PARTS))()
    _check(_lib.sq_linear_workspace_offsets(M, N, K, _dt(torch.empty(0, dtype=in_dtype)),
                                            _dt(torch.empty(0, dtype=out_dtype)), ctypes.cast(off, _vp)),
           "sq_linear_workspace_offsets")
    return dict(zip(LINEAR_WORKSPACE_PARTS, (int(v) for v in off)))


def sq_linear_workspace_views(workspace: torch.Tensor, M: int, N: int, K: int, in_dtype=torch.bfloat16,
                              out_dtype=torch.bfloat16) -> dict:
    """Tensor views of sq_linear's intermediates (maxima, factors, codes and
    scales) inside a workspace it has used."""
    off = sq_linear_workspace_offsets(M, N, K, in_dtype, out_dtype)
    shapes = {"xmax": ((K,), torch.float32), "wmax": ((K,), torch.float32), "s": ((K,), torch.float32),
              "xq": ((M, K), torch.int8), "x_scale": ((M,), torch.float32),
              "wq": ((N, K), torch.int8), "w_scale": ((N,), torch.float32)}
    views = {}
    for name, (shape, dt) in shapes.items():
        n = 1
        for d in shape:
            n *= d
        nbytes = n * torch.empty(0, dtype=dt).element_size()
        views[name] = workspace[off[name]:off[name] + nbytes].view(dt).view(shape)
    return views


def sq_linear(x: torch.Tensor, w: torch.Tensor, alpha: float, eps: float = 1e-8,
              out_dtype=torch.bfloat16, y: torch.Tensor | None = None,
              workspace: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The whole path (a1..a5) on one batch. x, w and y may be CUDA tensors or
    (pinned) host tensors; host operands are staged through the workspace."""
    M, K = x.shape
    N = w.shape[0]
    if x.dtype != w.dtype:
        raise TypeError("x and w must have the same dtype")
    if not (x.is_contiguous() and w.is_contiguous()):
        raise ValueError("x and w must be contiguous")
    dev = x.device if x.is_cuda else (w.device if w.is_cuda else torch.device("cuda", torch.cuda.current_device()))
    if y is None:
        y = torch.empty((M, N), dtype=out_dtype, device=dev)
    need = sq_linear_workspace_size(M, N, K, x.dtype, y.dtype)
    if workspace is None:
        workspace = torch.zeros(need, dtype=torch.uint8, device=dev)
    _check(_lib.sq_linear(x.data_ptr(), w.data_ptr(), _dt(x), M, N, K, float(alpha), float(eps),
                          y.data_ptr(), _dt(y), workspace.data_ptr(), workspace.numel(), _stream(stream)),
           "sq_linear")
    return y


# C structs as their bytes (host memory that lives for the call)
_ROPE_SCALING = struct.Struct("dddqd")    # sq_rope_scaling
_KV_CACHE = struct.Struct("PPPPqiiii")    # sq_kv_cache


class KvCache(typing.NamedTuple):
    """A paged 8-bit key/value cache (sq_kv_cache): int8 codes k, v [n_pages,
    n_heads, page_size, head_dim] and float32 scales k_scale, v_scale [n_pages,
    n_heads, page_size / scale_block], one per scale_block tokens and head."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor

    @classmethod
    def empty(cls, n_pages: int, n_heads: int, head_dim: int, page_size: int = 64, scale_block: int = 16, device="cuda"):
        """A cache that holds nothing yet (codes and scales uninitialised)."""
        codes = [torch.empty((n_pages, n_heads, page_size, head_dim), dtype=torch.int8, device=device) for _ in range(2)]
        scales = [torch.empty((n_pages, n_heads, page_size // scale_block), dtype=torch.float32, device=device)
                  for _ in range(2)]
        return cls(*codes, *scales)


def _ptr(t: torch.Tensor, dtype, index: int, name: str) -> int:
    """The address of a contiguous tensor of `dtype` on CUDA device `index`."""
    if index < 0 or t.get_device() != index or t.dtype is not dtype or not t.is_contiguous():
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        raise ValueError(f"{name} is on {t.device}, other tensors on cuda:{index}")
    return t.data_ptr()


def _shaped(t: torch.Tensor, shape: tuple, dtype, index: int, name: str) -> int:
    if t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, has {tuple(t.shape)}")
    return _ptr(t, dtype, index, name)


def _cache_bytes(cache: KvCache) -> tuple[bytes, int, int, int]:
    """-> (sq_kv_cache, CUDA device index, n_heads, head_dim)."""
    k, v, ks, vs = cache
    n_pages, n_heads, page_size, head_dim = shape = k.shape
    if v.shape != shape or vs.shape != ks.shape or ks.dim() != 3 or ks.shape[:2] != shape[:2]:
        raise ValueError("cache: k and v, and k_scale and v_scale, must have the same shapes")
    blocks = ks.shape[2]
    if blocks == 0 or page_size % blocks:
        raise ValueError("cache: page_size must be a multiple of the scales per page")
    index = k.get_device()
    if index < 0:
        raise ValueError("cache.k must be a CUDA tensor")
    return (_KV_CACHE.pack(_ptr(k, torch.int8, index, "cache.k"), _ptr(v, torch.int8, index, "cache.v"),
                           _ptr(ks, torch.float32, index, "cache.k_scale"), _ptr(vs, torch.float32, index, "cache.v_scale"),
                           n_pages, n_heads, head_dim, page_size, page_size // blocks), index, n_heads, head_dim)


def _token_rows(t: torch.Tensor, index: int, name: str) -> tuple[int, int]:
    """(address, elements between tokens) of [.., tokens, heads, head_dim] whose
    heads are contiguous and whose tokens are evenly spaced."""
    if t.get_device() != index or index < 0:
        raise ValueError(f"{name} must be a CUDA tensor on the other tensors' device")
    shape, stride = t.shape, t.stride()
    d, heads = shape[-1], shape[-2]
    if t.numel() and ((d > 1 and stride[-1] != 1) or (heads > 1 and stride[-2] != d)):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    step = stride[-3] if shape[-3] > 1 else d * heads
    if len(shape) == 4 and shape[0] > 1:
        if shape[1] == 1:
            step = stride[0]
        elif stride[0] != shape[1] * step:
            raise ValueError(f"{name}: tokens must be evenly spaced")
    return t.data_ptr(), step


def _made(device: torch.device, shape, dtype, stream) -> torch.Tensor:
    """A new tensor that the call on `stream` writes. On another stream than the
    current one its memory is that stream's, which does not wait for what the
    current stream still does with memory freed there; the current stream is
    noted as a reader."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    current = torch.cuda.current_stream(device)
    if not isinstance(stream, torch.cuda.Stream):
        raw = int(stream)
        stream = torch.cuda.ExternalStream(raw, device) if raw else torch.cuda.default_stream(device)
    if stream.cuda_stream == current.cuda_stream:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    t.record_stream(current)
    return t


def _given_or_made(t, like: torch.Tensor, shape, dtype, index: int, stream, name: str):
    """-> (t, its address); a new tensor if t is None."""
    if t is None:
        t = like.new_empty(shape, dtype=dtype) if stream is None else _made(like.device, shape, dtype, stream)
        return t, t.data_ptr()
    return t, _shaped(t, shape, dtype, index, name)


def _on_device(index: int, call, *args):
    if torch.cuda.current_device() == index:
        return call(*args)
    with torch.cuda.device(index):
        return call(*args)


def _launch(index: int, stream, name: str, *args) -> None:
    """Call a C entry point on CUDA device `index`, on `stream` or that device's
    current stream (the last C argument)."""
    call = getattr(_lib, name)
    if stream is None:
        st = torch._C._cuda_getCurrentRawStream(index)
    else:
        st = stream.cuda_stream if isinstance(stream, torch.cuda.Stream) else int(stream)
    status = _on_device(index, call, *args, st)
    if status != SQ_OK:
        _check(status, name)


def sq_rope_table(n_pos: int, rot_dim: int, theta: float = 10000.0, first_pos: int = 0, factor: float = 1.0,
                  low_turns: float = 0.0, high_turns: float = 0.0, original_len: int = 0, magnitude: float = 1.0,
                  table: torch.Tensor | None = None, device=None, stream=None) -> torch.Tensor:
    """cos and sin of the rotary angles, float32 [n_pos, rot_dim / 2, 2];
    frequencies scaled by `factor`, all of them or (high_turns > 0) those that
    make few turns in original_len tokens."""
    shape = (max(n_pos, 0), max(rot_dim, 0) // 2, 2)
    if table is None:
        device = torch.device("cuda" if device is None else device)
        if device.type != "cuda":
            raise ValueError("the table is a CUDA tensor")
        table = _made(device, shape, torch.float32, stream)
    index = table.get_device()
    ptr = _shaped(table, shape, torch.float32, index, "table")
    scaling = _ROPE_SCALING.pack(factor, low_turns, high_turns, original_len, magnitude)
    _launch(index, stream, "sq_rope_table", ptr, first_pos, n_pos, rot_dim, theta, scaling)
    return table


def sq_rope_kv_append(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, cache: KvCache, block_table: torch.Tensor,
                      ctx_len: torch.Tensor, cu_new: torch.Tensor, table: torch.Tensor | None = None,
                      interleaved: bool = False, q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                      want_k: bool = False, stream=None):
    """Rotate q [T, n_q_heads, head_dim] and k, append k and v [T, n_heads,
    head_dim] to the cache -> (rotated q, rotated k or None). The tensors may be
    slices of one QKV output."""
    c, index, heads, d = _cache_bytes(cache)
    dtype = k.dtype
    dt = _dt(k)
    T = k.shape[0]
    if k.shape != (T, heads, d) or v.shape != k.shape:
        raise ValueError(f"k and v must be [T, {heads}, {d}]")
    if v.dtype is not dtype or (q is not None and q.dtype is not dtype):
        raise TypeError("q, k and v must have the same dtype")
    n_seqs, max_pages = block_table.shape
    q_ptr, q_step, hq, qo = None, 0, 0, None
    if q is not None:
        hq = q.shape[1]
        if q.shape != (T, hq, d):
            raise ValueError(f"q must be [{T}, n_q_heads, {d}]")
        q_ptr, q_step = _token_rows(q, index, "q")
        q_out, qo = _given_or_made(q_out, q, (T, hq, d), dtype, index, stream, "q_out")
    elif q_out is not None:
        raise ValueError("q_out is given without q")
    k_ptr, k_step = _token_rows(k, index, "k")
    v_ptr, v_step = _token_rows(v, index, "v")
    ko = None
    if k_out is not None or want_k:
        k_out, ko = _given_or_made(k_out, k, (T, heads, d), dtype, index, stream, "k_out")
    t_ptr, n_pos, rot = None, 0, 0
    if table is not None:
        n_pos, half, _ = table.shape
        rot = 2 * half
        t_ptr = _shaped(table, (n_pos, half, 2), torch.float32, index, "table")
    _launch(index, stream, "sq_rope_kv_append", c, _ptr(block_table, torch.int32, index, "block_table"), max_pages,
            _shaped(ctx_len, (n_seqs,), torch.int32, index, "ctx_len"),
            _shaped(cu_new, (n_seqs + 1,), torch.int32, index, "cu_new"), n_seqs, T, q_ptr, q_step, hq, k_ptr, k_step,
            v_ptr, v_step, dt, t_ptr, n_pos, rot, 1 if interleaved else 0, qo, ko)
    return q_out, k_out


def sq_kv_read(cache: KvCache, block_table: torch.Tensor, first: torch.Tensor, cu_out: torch.Tensor, n_rows: int,
               dtype=torch.bfloat16, k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None, stream=None):
    """The cached tokens from first[b] on of every sequence, packed by cu_out
    into n_rows rows -> (k, v) [n_rows, n_heads, head_dim]."""
    c, index, heads, d = _cache_bytes(cache)
    n_seqs, max_pages = block_table.shape
    shape = (n_rows, heads, d)
    if k_out is not None:
        dtype = k_out.dtype
    elif v_out is not None:
        dtype = v_out.dtype
    k_out, ko = _given_or_made(k_out, cache.k, shape, dtype, index, stream, "k_out")
    v_out, vo = _given_or_made(v_out, cache.k, shape, dtype, index, stream, "v_out")
    _launch(index, stream, "sq_kv_read", c, _ptr(block_table, torch.int32, index, "block_table"), max_pages,
            _shaped(first, (n_seqs,), torch.int32, index, "first"),
            _shaped(cu_out, (n_seqs + 1,), torch.int32, index, "cu_out"), n_seqs, n_rows,
            ko, vo, _dt(k_out))
    return k_out, v_out


def sq_kv_attention_workspace_size(cache: KvCache, n_seqs: int, q_len: int, n_q_heads: int) -> int:
    c, index, _, _ = _cache_bytes(cache)
    return int(_on_device(index, _lib.sq_kv_attention_workspace_size, c, n_seqs, q_len, n_q_heads))


def sq_kv_attention(q: torch.Tensor, cache: KvCache, block_table: torch.Tensor, seq_len: torch.Tensor,
                    scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                    want_lse: bool = False, workspace: torch.Tensor | None = None, stream=None):
    """The newest q_len tokens' q [n_seqs, q_len, n_q_heads, head_dim] over the
    cached tokens of their sequences -> out, or (out, lse) if asked for. `scale`
    is head_dim ** -0.5 if not given."""
    c, index, _, d = _cache_bytes(cache)
    shape = q.shape
    if len(shape) != 4 or shape[3] != d:
        raise ValueError(f"q must be [n_seqs, q_len, n_q_heads, {d}]")
    n_seqs, q_len, hq, _ = shape
    dtype = q.dtype
    dt = _dt(q)
    q_ptr, q_step = _token_rows(q, index, "q")
    max_pages = block_table.shape[1]
    out, o_ptr = _given_or_made(out, q, shape, dtype, index, stream, "out")
    l_ptr = None
    if lse is not None or want_lse:
        lse, l_ptr = _given_or_made(lse, q, (n_seqs, q_len, hq), torch.float32, index, stream, "lse")
    if workspace is None:
        ws_bytes = _on_device(index, _lib.sq_kv_attention_workspace_size, c, n_seqs, q_len, hq)   # by that device's SMs
        workspace, ws = _given_or_made(None, q, (ws_bytes,), torch.uint8, index, stream, "workspace")
    else:
        ws_bytes = workspace.numel()
        ws = _ptr(workspace, torch.uint8, index, "workspace")
    _launch(index, stream, "sq_kv_attention", q_ptr, q_step, dt, c,
            _shaped(block_table, (n_seqs, max_pages), torch.int32, index, "block_table"), max_pages,
            _shaped(seq_len, (n_seqs,), torch.int32, index, "seq_len"), n_seqs, q_len, hq,
            d ** -0.5 if scale is None else scale, o_ptr, l_ptr, ws, ws_bytes)
    return out if lse is None else (out, lse)


def sq_prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, causal: bool = True,
                        scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                        want_lse: bool = False, stream=None):
    """Packed prompts q [T, n_q_heads, head_dim], k, v [T, n_kv_heads, head_dim]
    (bf16; slices of one QKV output may be given) over themselves -> out, or
    (out, lse) if asked for. `scale` is head_dim ** -0.5 if not given."""
    shape = q.shape
    T, hq, d = shape
    heads = k.shape[1]
    if k.shape != (T, heads, d) or v.shape != k.shape:
        raise ValueError("q must be [T, n_q_heads, head_dim], k and v [T, n_kv_heads, head_dim]")
    if q.dtype is not torch.bfloat16 or k.dtype is not torch.bfloat16 or v.dtype is not torch.bfloat16:
        raise TypeError("q, k and v must be bfloat16")
    index = q.get_device()
    (q_ptr, q_step), (k_ptr, k_step), (v_ptr, v_step) = (_token_rows(q, index, "q"), _token_rows(k, index, "k"),
                                                         _token_rows(v, index, "v"))
    n_seqs = cu_seqlens.shape[0] - 1
    out, o_ptr = _given_or_made(out, q, shape, torch.bfloat16, index, stream, "out")
    l_ptr = None
    if lse is not None or want_lse:
        lse, l_ptr = _given_or_made(lse, q, (T, hq), torch.float32, index, stream, "lse")
    _launch(index, stream, "sq_prompt_attention", q_ptr, q_step, k_ptr, k_step, v_ptr, v_step,
            _shaped(cu_seqlens, (n_seqs + 1,), torch.int32, index, "cu_seqlens"), n_seqs, T, hq, heads, d,
            d ** -0.5 if scale is None else scale, 1 if causal else 0, o_ptr, l_ptr)
    return out if lse is None else (out, lse)


def sq_get_status(stream=None) -> int:
    """Synchronize the stream and return (and clear) the device status word."""
    return int(_lib.sq_get_status(_stream(stream)))


def sq_last_status_site() -> int:
    return int(_lib.sq_last_status_site())


def sq_last_error_string() -> str:
    return _lib.sq_last_error_string().decode(errors="replace")


def sq_set_wait_timeout_ms(ms: int) -> None:
    _check(_lib.sq_set_wait_timeout_ms(int(ms)), "sq_set_wait_timeout_ms")


def sq_selftest_wait_timeout(limit_us: int, stream=None) -> None:
    _check(_lib.sq_selftest_wait_timeout(int(limit_us), _stream(stream)), "sq_selftest_wait_timeout")


def sq_probe_tensor_int8(iters: int, clocks: torch.Tensor | None = None, stream=None) -> float:
    """Launch the int8 tensor-core rate probe; returns the int8 operations the
    launch performs (time it with CUDA events on the stream). `clocks`, a
    CUDA int64 tensor of 2 entries if given, receives one SM's cycles and
    nanoseconds over the MMAs."""
    ops = ctypes.c_double(0.0)
    _check(_lib.sq_probe_tensor_int8(int(iters), ctypes.cast(ctypes.pointer(ops), _vp),
                                     None if clocks is None else _dev(clocks, "clocks"), _stream(stream)),
           "sq_probe_tensor_int8")
    return float(ops.value)


def raw_status(fn_name: str, *args) -> int:
    """Call a C entry point with raw ctypes arguments and return its status
    (tests of the host-side argument checks)."""
    return int(getattr(_lib, fn_name)(*args))
