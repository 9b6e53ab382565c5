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


class _RopeScaling(ctypes.Structure):
    _fields_ = [("factor", ctypes.c_double), ("low_turns", ctypes.c_double), ("high_turns", ctypes.c_double),
                ("original_len", _i64), ("magnitude", ctypes.c_double)]


class _KvCacheStruct(ctypes.Structure):
    _fields_ = [("k", _vp), ("v", _vp), ("k_scale", _vp), ("v_scale", _vp), ("n_pages", _i64),
                ("n_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("page_size", ctypes.c_int32),
                ("scale_block", ctypes.c_int32)]


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


def _cache_struct(cache: KvCache) -> _KvCacheStruct:
    k, v, ks, vs = cache
    n_pages, n_heads, page_size, head_dim = k.shape
    if v.shape != k.shape or vs.shape != ks.shape or ks.dim() != 3 or ks.shape[:2] != k.shape[:2]:
        raise ValueError("cache: k and v, and k_scale and v_scale, must have the same shapes")
    blocks = ks.shape[2]
    if blocks == 0 or page_size % blocks:
        raise ValueError("cache: page_size must be a multiple of the scales per page")
    if k.dtype != torch.int8 or v.dtype != torch.int8 or ks.dtype != torch.float32 or vs.dtype != torch.float32:
        raise TypeError("cache: codes are int8, scales float32")
    return _KvCacheStruct(_dev(k, "cache.k"), _dev(v, "cache.v"), _dev(ks, "cache.k_scale"), _dev(vs, "cache.v_scale"),
                          n_pages, n_heads, head_dim, page_size, page_size // blocks)


def _same_device(first: torch.Tensor, *others) -> None:
    for t in others:
        if t is not None and t.device != first.device:
            raise ValueError(f"tensors on {first.device} and {t.device}")


def _i32(t: torch.Tensor, shape: tuple, name: str) -> int:
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, has {tuple(t.shape)}")
    return _dev(t, name)


def _token_rows(t: torch.Tensor, name: str) -> tuple[int, int]:
    """(address, elements between tokens) of [.., tokens, heads, head_dim] whose
    heads are contiguous and whose tokens are evenly spaced."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    shape, stride = t.shape, t.stride()
    if t.numel() and ((shape[-1] > 1 and stride[-1] != 1) or (shape[-2] > 1 and stride[-2] != shape[-1])):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    width = shape[-1] * shape[-2]
    step = stride[-3] if shape[-3] > 1 else width
    if t.dim() == 4 and shape[0] > 1:
        if shape[1] == 1:
            step = stride[0]
        elif stride[0] != shape[1] * step:
            raise ValueError(f"{name}: tokens must be evenly spaced")
    return t.data_ptr(), step


def _made(shape, dtype, device, stream) -> torch.Tensor:
    """A tensor that the call on `stream` writes; known to the allocator as in
    use there when that is not the current stream."""
    t = torch.empty(shape, dtype=dtype, device=device)
    if stream is not None:
        t.record_stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(int(stream), device))
    return t


class _on:
    """Makes `device` current for a call if it is not, and gives its stream."""

    def __init__(self, device: torch.device, stream):
        index = device.index if device.index is not None else torch.cuda.current_device()
        self.guard = torch.cuda.device(index) if index != torch.cuda.current_device() else None
        self.stream = stream

    def __enter__(self) -> int:
        if self.guard is not None:
            self.guard.__enter__()
        return _stream(self.stream)

    def __exit__(self, *args):
        if self.guard is not None:
            self.guard.__exit__(*args)


def sq_rope_table(n_pos: int, rot_dim: int, theta: float = 10000.0, first_pos: int = 0, factor: float = 1.0,
                  low_turns: float = 0.0, high_turns: float = 0.0, original_len: int = 0, magnitude: float = 1.0,
                  table: torch.Tensor | None = None, device=None, stream=None) -> torch.Tensor:
    """cos and sin of the rotary angles, float32 [n_pos, rot_dim / 2, 2];
    frequencies scaled by `factor`, all of them or (high_turns > 0) those that
    make few turns in original_len tokens."""
    device = table.device if table is not None else torch.device("cuda" if device is None else device)
    if device.type != "cuda":
        raise ValueError("the table is a CUDA tensor")
    if table is not None and (tuple(table.shape) != (n_pos, rot_dim // 2, 2) or table.dtype != torch.float32):
        raise ValueError(f"table must be float32 [{n_pos}, {rot_dim // 2}, 2]")
    scaling = _RopeScaling(float(factor), float(low_turns), float(high_turns), int(original_len), float(magnitude))
    with _on(device, stream) as st:
        if table is None:
            table = _made((max(n_pos, 0), max(rot_dim, 0) // 2, 2), torch.float32, device, stream)
        _check(_lib.sq_rope_table(_dev(table, "table"), first_pos, n_pos, rot_dim, float(theta), ctypes.byref(scaling), st),
               "sq_rope_table")
    return table


def sq_rope_kv_append(q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor, cache: KvCache, block_table: torch.Tensor,
                      ctx_len: torch.Tensor, cu_new: torch.Tensor, table: torch.Tensor | None = None,
                      interleaved: bool = False, q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                      want_k: bool = False, stream=None):
    """Rotate q [T, n_q_heads, head_dim] and k, append k and v [T, n_heads,
    head_dim] to the cache -> (rotated q, rotated k or None). The tensors may be
    slices of one QKV output."""
    c = _cache_struct(cache)
    T = k.shape[0]
    if k.shape != v.shape or tuple(k.shape) != (T, c.n_heads, c.head_dim):
        raise ValueError(f"k and v must be [T, {c.n_heads}, {c.head_dim}]")
    if v.dtype != k.dtype or (q is not None and q.dtype != k.dtype):
        raise TypeError("q, k and v must have the same dtype")
    _same_device(k, q, v, *cache, block_table, ctx_len, cu_new, table, q_out, k_out)
    n_seqs, max_pages = block_table.shape
    dt = _dt(k)
    with _on(k.device, stream) as st:
        q_ptr, q_step, hq, qo = None, 0, 0, None
        if q is not None:
            if q.dim() != 3 or q.shape[0] != T or q.shape[2] != c.head_dim:
                raise ValueError(f"q must be [{T}, n_q_heads, {c.head_dim}]")
            hq = q.shape[1]
            q_ptr, q_step = _token_rows(q, "q")
            if q_out is None:
                q_out = _made((T, hq, c.head_dim), q.dtype, q.device, stream)
            elif q_out.shape != q.shape or q_out.dtype != q.dtype:
                raise ValueError("q_out must have q's shape and dtype")
            qo = _dev(q_out, "q_out")
        k_ptr, k_step = _token_rows(k, "k")
        v_ptr, v_step = _token_rows(v, "v")
        if k_out is None and want_k:
            k_out = _made((T, c.n_heads, c.head_dim), k.dtype, k.device, stream)
        elif k_out is not None and (k_out.shape != k.shape or k_out.dtype != k.dtype):
            raise ValueError("k_out must have k's shape and dtype")
        t_ptr, n_pos, rot = None, 0, 0
        if table is not None:
            if table.dim() != 3 or table.shape[2] != 2 or table.dtype != torch.float32:
                raise ValueError("table must be float32 [n_pos, rot_dim / 2, 2]")
            t_ptr, n_pos, rot = _dev(table, "table"), table.shape[0], 2 * table.shape[1]
        _check(_lib.sq_rope_kv_append(ctypes.byref(c), _i32(block_table, (n_seqs, max_pages), "block_table"), max_pages,
                                      _i32(ctx_len, (n_seqs,), "ctx_len"), _i32(cu_new, (n_seqs + 1,), "cu_new"), n_seqs, T,
                                      q_ptr, q_step, hq, k_ptr, k_step, v_ptr, v_step, dt, t_ptr, n_pos, rot,
                                      int(interleaved), qo, _opt_dev(k_out, "k_out"), st), "sq_rope_kv_append")
    return q_out, k_out


def sq_kv_read(cache: KvCache, block_table: torch.Tensor, first: torch.Tensor, cu_out: torch.Tensor, n_rows: int,
               dtype=torch.bfloat16, k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None, stream=None):
    """The cached tokens from first[b] on of every sequence, packed by cu_out
    into n_rows rows -> (k, v) [n_rows, n_heads, head_dim]."""
    c = _cache_struct(cache)
    _same_device(cache.k, *cache[1:], block_table, first, cu_out, k_out, v_out)
    n_seqs, max_pages = block_table.shape
    shape = (n_rows, c.n_heads, c.head_dim)
    with _on(cache.k.device, stream) as st:
        if k_out is None:
            k_out = _made(shape, dtype, cache.k.device, stream)
        if v_out is None:
            v_out = _made(shape, k_out.dtype, cache.k.device, stream)
        if tuple(k_out.shape) != shape or tuple(v_out.shape) != shape or k_out.dtype != v_out.dtype:
            raise ValueError(f"k_out and v_out must be {shape} and of one dtype")
        _check(_lib.sq_kv_read(ctypes.byref(c), _i32(block_table, (n_seqs, max_pages), "block_table"), max_pages,
                               _i32(first, (n_seqs,), "first"), _i32(cu_out, (n_seqs + 1,), "cu_out"), n_seqs, n_rows,
                               _dev(k_out, "k_out"), _dev(v_out, "v_out"), _dt(k_out), st), "sq_kv_read")
    return k_out, v_out


def sq_kv_attention_workspace_size(cache: KvCache, n_seqs: int, q_len: int, n_q_heads: int) -> int:
    with _on(cache.k.device, None):
        return int(_lib.sq_kv_attention_workspace_size(ctypes.byref(_cache_struct(cache)), n_seqs, q_len, n_q_heads))


def sq_kv_attention(q: torch.Tensor, cache: KvCache, block_table: torch.Tensor, seq_len: torch.Tensor,
                    scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                    want_lse: bool = False, workspace: torch.Tensor | None = None, stream=None):
    """The newest q_len tokens' q [n_seqs, q_len, n_q_heads, head_dim] over the
    cached tokens of their sequences -> out, or (out, lse) if asked for. `scale`
    is head_dim ** -0.5 if not given."""
    c = _cache_struct(cache)
    if q.dim() != 4 or q.shape[3] != c.head_dim:
        raise ValueError(f"q must be [n_seqs, q_len, n_q_heads, {c.head_dim}]")
    n_seqs, q_len, hq, d = q.shape
    max_pages = block_table.shape[1]
    _same_device(q, *cache, block_table, seq_len, out, lse, workspace)
    dt = _dt(q)
    with _on(q.device, stream) as st:
        q_ptr, q_step = _token_rows(q, "q")
        if out is None:
            out = _made((n_seqs, q_len, hq, d), q.dtype, q.device, stream)
        elif out.shape != q.shape or out.dtype != q.dtype:
            raise ValueError("out must have q's shape and dtype")
        if lse is None and want_lse:
            lse = _made((n_seqs, q_len, hq), torch.float32, q.device, stream)
        elif lse is not None and (tuple(lse.shape) != (n_seqs, q_len, hq) or lse.dtype != torch.float32):
            raise ValueError("lse must be float32 [n_seqs, q_len, n_q_heads]")
        if workspace is None:
            need = int(_lib.sq_kv_attention_workspace_size(ctypes.byref(c), n_seqs, q_len, hq))
            workspace = _made((need,), torch.uint8, q.device, stream)
        _check(_lib.sq_kv_attention(q_ptr, q_step, dt, ctypes.byref(c), _i32(block_table, (n_seqs, max_pages), "block_table"),
                                    max_pages, _i32(seq_len, (n_seqs,), "seq_len"), n_seqs, q_len, hq,
                                    float(d ** -0.5 if scale is None else scale), _dev(out, "out"), _opt_dev(lse, "lse"),
                                    _dev(workspace, "workspace"), workspace.numel() * workspace.element_size(), st),
               "sq_kv_attention")
    return out if lse is None else (out, lse)


def sq_prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor, causal: bool = True,
                        scale: float | None = None, out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                        want_lse: bool = False, stream=None):
    """Packed prompts q [T, n_q_heads, head_dim], k, v [T, n_kv_heads, head_dim]
    (bf16; slices of one QKV output may be given) over themselves -> out, or
    (out, lse) if asked for. `scale` is head_dim ** -0.5 if not given."""
    if q.dim() != 3 or k.dim() != 3 or k.shape != v.shape or k.shape[0] != q.shape[0] or k.shape[2] != q.shape[2]:
        raise ValueError("q must be [T, n_q_heads, head_dim], k and v [T, n_kv_heads, head_dim]")
    if any(t.dtype != torch.bfloat16 for t in (q, k, v)):
        raise TypeError("q, k and v must be bfloat16")
    _same_device(q, k, v, cu_seqlens, out, lse)
    T, hq, d = q.shape
    n_seqs = cu_seqlens.shape[0] - 1
    (q_ptr, q_step), (k_ptr, k_step), (v_ptr, v_step) = _token_rows(q, "q"), _token_rows(k, "k"), _token_rows(v, "v")
    with _on(q.device, stream) as st:
        if out is None:
            out = _made((T, hq, d), q.dtype, q.device, stream)
        elif out.shape != q.shape or out.dtype != q.dtype:
            raise ValueError("out must have q's shape and dtype")
        if lse is None and want_lse:
            lse = _made((T, hq), torch.float32, q.device, stream)
        elif lse is not None and (tuple(lse.shape) != (T, hq) or lse.dtype != torch.float32):
            raise ValueError("lse must be float32 [T, n_q_heads]")
        _check(_lib.sq_prompt_attention(q_ptr, q_step, k_ptr, k_step, v_ptr, v_step,
                                        _i32(cu_seqlens, (n_seqs + 1,), "cu_seqlens"), n_seqs, T, hq, k.shape[1], d,
                                        float(d ** -0.5 if scale is None else scale), int(causal), _dev(out, "out"),
                                        _opt_dev(lse, "lse"), st), "sq_prompt_attention")
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
