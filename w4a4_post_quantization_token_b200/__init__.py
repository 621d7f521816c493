"""Python binding of libkq, the B200 (sm_100a) W4A4 quantized linear layer.

Argument marshalling only: every step of the layer runs in the CUDA library
(include/kq.h); this module checks tensor placement, dtypes and sizes, passes raw
device pointers and the current CUDA stream, and raises on a non-OK status.
PyTorch is used for device memory and streams. There is no CPU fallback: if the
shared library is missing or cannot be loaded, importing this package raises.
"""
from __future__ import annotations

import ctypes
import functools
import os

import numpy as np

__all__ = ["KQError", "Layer", "lib", "library_path", "weights_bytes", "act_bytes",
           "prepare_ws_bytes", "prepare_weights", "prepare_weights_lp", "debug_encode_lp_f32", "quantize_act", "smooth_quantize_act", "linear",
           "linear_noalloc", "lloydmax_codebook", "CB_MXFP4", "CB_LLOYDMAX",
           "linear_host", "NOALLOC_WORKSPACE_BYTES",
           "gemm", "weights_pack", "weights_unpack", "act_pack", "act_unpack",
           "debug_transform", "debug_encode_f32", "debug_wait_timeout", "last_device_error",
           "status_string", "ERR_DEVICE_TIMEOUT", "ERR_LOWRANK_RANGE",
           "OUT_F32", "OUT_BF16", "SYMBOLS",
           "Fp8Layer", "fp8_weights_bytes", "fp8_act_bytes", "fp8_ffn_bytes",
           "fp8_prepare_weights", "fp8_weights_pack", "fp8_weights_unpack", "fp8_quantize_act",
           "fp8_rmsnorm_act", "fp8_act_pack", "fp8_act_unpack", "fp8_gemm", "fp8_gated_act",
           "fp8_linear", "fp8_ffn", "fp8_last_device_error", "fp8_debug_wait_timeout", "ACT_SILU", "ACT_GELU"]

OUT_F32, OUT_BF16 = 0, 1
ERR_DEVICE_TIMEOUT, ERR_LOWRANK_RANGE = 7, 9
T_NONE, T_KRON, T_RPBH = 0, 1, 2
_KIND = {"none": T_NONE, "kron": T_KRON, "rpbh": T_RPBH}
CB_MXFP4, CB_LLOYDMAX = 0, 1
ACT_SILU, ACT_GELU = 0, 1
_ACTIVATION = {"silu": ACT_SILU, "gelu": ACT_GELU}
_CODEBOOK = {"mxfp4": CB_MXFP4, "lloydmax": CB_LLOYDMAX}

_HERE = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_HERE, "libkq.so")

# every symbol include/kq.h declares
SYMBOLS = ["kq_weights_bytes", "kq_act_bytes", "kq_prepare_ws_bytes", "kq_prepare_weights",
           "kq_quantize_act", "kq_linear", "kq_linear_host", "kq_gemm", "kq_weights_pack",
           "kq_weights_unpack", "kq_act_pack", "kq_act_unpack", "kq_debug_transform",
           "kq_debug_encode_f32", "kq_last_device_error", "kq_status_string", "kq_version",
           "kq_linear_noalloc", "kq_smooth_quantize_act", "kq_prepare_weights_lp",
           "kq_debug_encode_lp_f32", "kq_lloydmax_codebook", "kq_debug_wait_timeout",
           "kq_fp8_weights_bytes", "kq_fp8_act_bytes", "kq_fp8_ffn_bytes",
           "kq_fp8_prepare_weights", "kq_fp8_weights_pack", "kq_fp8_weights_unpack",
           "kq_fp8_quantize_act", "kq_fp8_rmsnorm_act", "kq_fp8_act_pack", "kq_fp8_act_unpack",
           "kq_fp8_gemm", "kq_fp8_gated_act", "kq_fp8_linear", "kq_fp8_ffn",
           "kq_fp8_last_device_error", "kq_fp8_debug_wait_timeout"]


class KQError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {status_string(status)} (status {status})")
        self.status = status


if not os.path.exists(library_path):
    raise ImportError(f"libkq.so not found at {library_path}; build it with "
                      "`python w4a4_post_quantization_token_b200/build.py`")
lib = ctypes.CDLL(library_path)


class _TransformDesc(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("A", ctypes.POINTER(ctypes.c_float)),
                ("a_dim", ctypes.c_int32), ("B", ctypes.POINTER(ctypes.c_float)),
                ("b_dim", ctypes.c_int32), ("perm", ctypes.POINTER(ctypes.c_int32)),
                ("sign", ctypes.POINTER(ctypes.c_int8))]


class _LayerNormDesc(ctypes.Structure):
    _fields_ = [("on", ctypes.c_int32), ("eps", ctypes.c_float),
                ("gamma", ctypes.POINTER(ctypes.c_float)), ("beta", ctypes.POINTER(ctypes.c_float))]


class _LayerDesc(ctypes.Structure):
    _fields_ = [("K", ctypes.c_int32), ("N", ctypes.c_int32), ("rank", ctypes.c_int32),
                ("center", ctypes.c_int32), ("t", _TransformDesc), ("ln", _LayerNormDesc),
                ("codebook", ctypes.c_int32)]


class _Fp8Desc(ctypes.Structure):
    _fields_ = [("K", ctypes.c_int32), ("N", ctypes.c_int32), ("gated", ctypes.c_int32),
                ("activation", ctypes.c_int32)]


_P = ctypes.c_void_p
_D = ctypes.POINTER(_LayerDesc)
_F = ctypes.POINTER(_Fp8Desc)
_I32, _I64, _SZ = ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
_sigs = {
    "kq_weights_bytes": (ctypes.c_size_t, [_D]),
    "kq_act_bytes": (ctypes.c_size_t, [_D, ctypes.c_int32]),
    "kq_prepare_ws_bytes": (ctypes.c_size_t, [_D]),
    "kq_prepare_weights": (ctypes.c_int, [_D, _P, _P, _P, ctypes.c_size_t, _P]),
    "kq_quantize_act": (ctypes.c_int, [_D, _P, _P, ctypes.c_int32, _P, ctypes.c_size_t, _P]),
    "kq_linear": (ctypes.c_int, [_D, _P, _P, ctypes.c_int32, _P, ctypes.c_int32, _P,
                                 ctypes.c_size_t, _P]),
    "kq_prepare_weights_lp": (ctypes.c_int, [_D, ctypes.c_double, _P, _P, _P, ctypes.c_size_t, _P]),
    "kq_debug_encode_lp_f32": (ctypes.c_int, [_P, ctypes.c_int32, ctypes.c_int32, ctypes.c_double,
                                              _P, _P, _P]),
    "kq_smooth_quantize_act": (ctypes.c_int, [_D, _P, _P, ctypes.c_int32, _P, ctypes.c_size_t, _P]),
    "kq_linear_noalloc": (ctypes.c_int, [_D, _P, _P, ctypes.c_int32, _P, ctypes.c_int32, _P]),
    "kq_linear_host": (ctypes.c_int, [_D, _P, _P, _P, ctypes.c_int32, _P, _P, ctypes.c_int32,
                                      _P, ctypes.c_size_t, _P]),
    "kq_gemm": (ctypes.c_int, [_D, _P, _P, ctypes.c_int32, _P, ctypes.c_int32, _P]),
    "kq_weights_pack": (ctypes.c_int, [_D, _P, _P, _P, _P, _P, _P, _P]),
    "kq_weights_unpack": (ctypes.c_int, [_D, _P, _P, _P, _P, _P, _P, _P, _P]),
    "kq_act_pack": (ctypes.c_int, [_D, _P, _P, _P, _P, ctypes.c_int32, _P, ctypes.c_size_t, _P]),
    "kq_act_unpack": (ctypes.c_int, [_D, _P, ctypes.c_int32, _P, _P, _P, _P, _P]),
    "kq_debug_transform": (ctypes.c_int, [_D, _P, _P, ctypes.c_int32, _P, _P, _P]),
    "kq_debug_encode_f32": (ctypes.c_int, [_P, ctypes.c_int32, ctypes.c_int32, _P, _P, _P]),
    "kq_last_device_error": (ctypes.c_int, [_D, _P, ctypes.c_int32, _P]),
    "kq_debug_wait_timeout": (ctypes.c_int, [_D, _P, ctypes.c_int32, ctypes.c_uint32, _P]),
    "kq_lloydmax_codebook": (ctypes.c_int, [_P, _P]),
    "kq_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "kq_version": (ctypes.c_char_p, []),
    "kq_fp8_weights_bytes": (_SZ, [_F]),
    "kq_fp8_act_bytes": (_SZ, [_I32, _I32]),
    "kq_fp8_ffn_bytes": (_SZ, [_F, _F, _I32]),
    "kq_fp8_prepare_weights": (ctypes.c_int, [_F, _P, _P, _P, _P]),
    "kq_fp8_weights_pack": (ctypes.c_int, [_F, _P, _P, _P, _P, _P, _P]),
    "kq_fp8_weights_unpack": (ctypes.c_int, [_F, _P, _P, _P, _P, _P, _P]),
    "kq_fp8_quantize_act": (ctypes.c_int, [_I32, _P, _I64, _I32, _P, _SZ, _P]),
    "kq_fp8_rmsnorm_act": (ctypes.c_int, [_I32, _P, _I64, _P, _I64, _I32, _P, ctypes.c_float, _I32,
                                          _P, _SZ, _P]),
    "kq_fp8_act_pack": (ctypes.c_int, [_I32, _P, _P, _I32, _P, _SZ, _P]),
    "kq_fp8_act_unpack": (ctypes.c_int, [_I32, _P, _I32, _P, _P, _P, _I32, _P]),
    "kq_fp8_gemm": (ctypes.c_int, [_F, _P, _P, _I32, _P, _I64, _I32, _P]),
    "kq_fp8_gated_act": (ctypes.c_int, [_F, _P, _P, _I32, _P, _SZ, _P]),
    "kq_fp8_linear": (ctypes.c_int, [_F, _P, _P, _I64, _I32, _P, _I64, _I32, _P, _SZ, _P]),
    "kq_fp8_ffn": (ctypes.c_int, [_F, _P, _F, _P, _P, _I64, _P, _I64, _I32, _P, ctypes.c_float, _I32,
                                  _P, _I64, _I32, _P, _SZ, _P]),
    "kq_fp8_last_device_error": (ctypes.c_int, [_P, _P]),
    "kq_fp8_debug_wait_timeout": (ctypes.c_int, [_F, _P, _P, _I64, _I32, _P, _I64, _I32, _P, _SZ, _P, _SZ, _I64,
                                                 ctypes.c_uint32, _P]),
}
for _name, (_res, _args) in _sigs.items():
    _f = getattr(lib, _name)
    _f.restype = _res
    _f.argtypes = _args


def lloydmax_codebook() -> tuple[np.ndarray, np.ndarray]:
    """The library's (8 positive levels, 7 thresholds) of its 16-level Lloyd-Max codebook."""
    lv = np.zeros(8, np.float64)
    th = np.zeros(7, np.float64)
    _check(lib.kq_lloydmax_codebook(lv.ctypes.data_as(_P), th.ctypes.data_as(_P)),
           "kq_lloydmax_codebook")
    return lv, th


def status_string(s: int) -> str:
    return lib.kq_status_string(int(s)).decode()


def _check(status: int, where: str) -> None:
    if status != 0:
        raise KQError(status, where)


class Layer:
    """Host description of one linear layer (the C ``kq_layer_desc``).

    ``transform`` is ``{"kind": "kron", "A": 4x4, "B": 8x8}``,
    ``{"kind": "rpbh", "perm": int[K], "sign": +-1[K]}`` or ``{"kind": "none"}``.
    ``layernorm`` (optional) is ``{"gamma": float[K], "beta": float[K], "eps": float}``: the
    fused LayerNorm front-end (needs ``center``).
    ``codebook`` is ``"mxfp4"`` (default) or ``"lloydmax"``: the 16-level Lloyd-Max
    codebook with a per-token sigma (RPBH or no transform; activations reach the fp16
    tensor-core GEMM as decoded fp16 values).
    The host arrays are kept alive by this object."""

    def __init__(self, K: int, N: int, rank: int, center: bool, transform: dict,
                 layernorm: dict | None = None, codebook: str = "mxfp4"):
        self.K, self.N, self.rank, self.center = int(K), int(N), int(rank), bool(center)
        self.transform = transform
        kind = _KIND[transform["kind"]]
        t = _TransformDesc(kind=kind)
        self._keep = []
        if kind == T_KRON:
            A = np.ascontiguousarray(transform["A"], dtype=np.float32)
            B = np.ascontiguousarray(transform["B"], dtype=np.float32)
            self._keep += [A, B]
            t.A = A.ctypes.data_as(ctypes.POINTER(ctypes.c_float))
            t.B = B.ctypes.data_as(ctypes.POINTER(ctypes.c_float))
            t.a_dim, t.b_dim = A.shape[0], B.shape[0]
        elif kind == T_RPBH:
            perm = np.ascontiguousarray(transform["perm"], dtype=np.int32)
            sign = np.ascontiguousarray(transform["sign"], dtype=np.int8)
            self._keep += [perm, sign]
            t.perm = perm.ctypes.data_as(ctypes.POINTER(ctypes.c_int32))
            t.sign = sign.ctypes.data_as(ctypes.POINTER(ctypes.c_int8))
        ln = _LayerNormDesc(on=0)
        self.layernorm = layernorm
        if layernorm is not None:
            g = np.ascontiguousarray(layernorm["gamma"], dtype=np.float32)
            b = np.ascontiguousarray(layernorm["beta"], dtype=np.float32)
            self._keep += [g, b]
            ln.on, ln.eps = 1, float(layernorm.get("eps", 1e-6))
            ln.gamma = g.ctypes.data_as(ctypes.POINTER(ctypes.c_float))
            ln.beta = b.ctypes.data_as(ctypes.POINTER(ctypes.c_float))
        self.codebook = codebook
        self._desc = _LayerDesc(K=self.K, N=self.N, rank=self.rank, center=int(self.center), t=t,
                                ln=ln, codebook=_CODEBOOK[codebook])

    @property
    def desc(self):
        return ctypes.byref(self._desc)


def _ptr(t) -> int | None:
    return None if t is None else int(t.data_ptr())


def _stream(stream=None) -> int:
    import torch
    s = torch.cuda.current_stream() if stream is None else stream
    return int(s.cuda_stream)


def _need(t, dtype, numel: int | None = None, name: str = "tensor", cuda: bool = True):
    import torch
    if t is None:
        raise ValueError(f"{name} is required")
    if cuda and not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name} has {t.numel()} elements, needs {numel}")
    return t


def weights_bytes(layer: Layer) -> int:
    return int(lib.kq_weights_bytes(layer.desc))


def act_bytes(layer: Layer, M: int) -> int:
    return int(lib.kq_act_bytes(layer.desc, int(M)))


def prepare_ws_bytes(layer: Layer) -> int:
    return int(lib.kq_prepare_ws_bytes(layer.desc))


def prepare_weights(layer: Layer, W, weights, ws, stream=None) -> None:
    import torch
    _need(W, torch.bfloat16, layer.K * layer.N, "W")
    _need(weights, torch.uint8, weights_bytes(layer), "weights")
    _need(ws, torch.uint8, None, "ws")
    _check(lib.kq_prepare_weights(layer.desc, _ptr(W), _ptr(weights), _ptr(ws), ws.numel(),
                                  _stream(stream)), "kq_prepare_weights")


def quantize_act(layer: Layer, weights, X, act, stream=None) -> None:
    import torch
    M = X.shape[0]
    _need(X, torch.bfloat16, M * layer.K, "X")
    _need(act, torch.uint8, act_bytes(layer, M), "act")
    _check(lib.kq_quantize_act(layer.desc, _ptr(weights), _ptr(X), M, _ptr(act), act.numel(),
                               _stream(stream)), "kq_quantize_act")


def prepare_weights_lp(layer: Layer, p: float, W, weights, ws, stream=None) -> None:
    """prepare_weights with the robust l_p fit of the residual's block scales."""
    import torch
    _need(W, torch.bfloat16, layer.K * layer.N, "W")
    _need(weights, torch.uint8, weights_bytes(layer), "weights")
    _need(ws, torch.uint8, None, "ws")
    _check(lib.kq_prepare_weights_lp(layer.desc, float(p), _ptr(W), _ptr(weights), _ptr(ws),
                                     ws.numel(), _stream(stream)), "kq_prepare_weights_lp")


def debug_encode_lp_f32(V, p: float, codes, scales, stream=None) -> None:
    M, K = V.shape
    _check(lib.kq_debug_encode_lp_f32(_ptr(V), M, K, float(p), _ptr(codes), _ptr(scales),
                                      _stream(stream)), "kq_debug_encode_lp_f32")


def smooth_quantize_act(layer: Layer, inv_s, X, act, stream=None) -> None:
    """SmoothQuant comparator: per-channel multiply by inv_s (fp32 [K]), then MXFP4."""
    import torch
    M = X.shape[0]
    _need(inv_s, torch.float32, layer.K, "inv_s")
    _need(X, torch.bfloat16, M * layer.K, "X")
    _need(act, torch.uint8, act_bytes(layer, M), "act")
    _check(lib.kq_smooth_quantize_act(layer.desc, _ptr(inv_s), _ptr(X), M, _ptr(act), act.numel(),
                                      _stream(stream)), "kq_smooth_quantize_act")


def linear(layer: Layer, weights, X, Y, act, out_dtype: int = OUT_F32, stream=None) -> None:
    import torch
    M = X.shape[0]
    _need(X, torch.bfloat16, M * layer.K, "X")
    _need(Y, torch.bfloat16 if out_dtype == OUT_BF16 else torch.float32, M * layer.N, "Y")
    _need(act, torch.uint8, act_bytes(layer, M), "act")
    _check(lib.kq_linear(layer.desc, _ptr(weights), _ptr(X), M, _ptr(Y), int(out_dtype), _ptr(act),
                         act.numel(), _stream(stream)), "kq_linear")


def linear_noalloc(layer: Layer, weights, X, Y, out_dtype: int = OUT_F32, stream=None) -> None:
    """kq_linear on the library's built-in workspace: no workspace argument, nothing
    allocated. Calls that can overlap on the GPU share that workspace and race."""
    import torch
    M = X.shape[0]
    _need(X, torch.bfloat16, M * layer.K, "X")
    _need(Y, torch.bfloat16 if out_dtype == OUT_BF16 else torch.float32, M * layer.N, "Y")
    _check(lib.kq_linear_noalloc(layer.desc, _ptr(weights), _ptr(X), M, _ptr(Y), int(out_dtype),
                                 _stream(stream)), "kq_linear_noalloc")


NOALLOC_WORKSPACE_BYTES = 16 << 20


def linear_host(layer: Layer, weights, X_host, X_dev, Y_host, Y_dev, act,
                out_dtype: int = OUT_F32, stream=None) -> None:
    """Host-buffer variant: X_host and Y_host are pinned CPU tensors."""
    import torch
    M = X_host.shape[0]
    _need(X_host, torch.bfloat16, M * layer.K, "X_host", cuda=False)
    _need(X_dev, torch.bfloat16, M * layer.K, "X_dev")
    ydt = torch.bfloat16 if out_dtype == OUT_BF16 else torch.float32
    _need(Y_host, ydt, M * layer.N, "Y_host", cuda=False)
    _need(Y_dev, ydt, M * layer.N, "Y_dev")
    _check(lib.kq_linear_host(layer.desc, _ptr(weights), _ptr(X_host), _ptr(X_dev), M,
                              _ptr(Y_host), _ptr(Y_dev), int(out_dtype), _ptr(act), act.numel(),
                              _stream(stream)), "kq_linear_host")


def gemm(layer: Layer, weights, act, M: int, Y, out_dtype: int = OUT_F32, stream=None) -> None:
    _check(lib.kq_gemm(layer.desc, _ptr(weights), _ptr(act), int(M), _ptr(Y), int(out_dtype),
                       _stream(stream)), "kq_gemm")


def weights_pack(layer: Layer, r_codes, r_scales, L1p, L2, s, weights, stream=None) -> None:
    import torch
    _need(r_codes, torch.uint8, layer.N * layer.K // 2, "r_codes")
    _need(r_scales, torch.uint8, layer.N * layer.K // 32, "r_scales")
    _need(s, torch.float32, layer.N, "s")
    if layer.rank:
        _need(L1p, torch.float32, layer.K * layer.rank, "L1p")
        _need(L2, torch.bfloat16, layer.rank * layer.N, "L2")
    _need(weights, torch.uint8, weights_bytes(layer), "weights")
    _check(lib.kq_weights_pack(layer.desc, _ptr(r_codes), _ptr(r_scales), _ptr(L1p), _ptr(L2),
                               _ptr(s), _ptr(weights), _stream(stream)), "kq_weights_pack")


def weights_unpack(layer: Layer, weights, r_codes=None, r_scales=None, L1p=None, L2=None, c1=None,
                   s=None, stream=None) -> None:
    _check(lib.kq_weights_unpack(layer.desc, _ptr(weights), _ptr(r_codes), _ptr(r_scales),
                                 _ptr(L1p), _ptr(L2), _ptr(c1), _ptr(s), _stream(stream)),
           "kq_weights_unpack")


def act_pack(layer: Layer, codes, scales, mu, U, M: int, act, stream=None) -> None:
    _check(lib.kq_act_pack(layer.desc, _ptr(codes), _ptr(scales), _ptr(mu), _ptr(U), int(M),
                           _ptr(act), act.numel(), _stream(stream)), "kq_act_pack")


def act_unpack(layer: Layer, act, M: int, codes=None, scales=None, mu=None, U=None,
               stream=None) -> None:
    _check(lib.kq_act_unpack(layer.desc, _ptr(act), int(M), _ptr(codes), _ptr(scales), _ptr(mu),
                             _ptr(U), _stream(stream)), "kq_act_unpack")


def debug_transform(layer: Layer, weights, X, Xt, mu, stream=None) -> None:
    _check(lib.kq_debug_transform(layer.desc, _ptr(weights), _ptr(X), X.shape[0], _ptr(Xt),
                                  _ptr(mu), _stream(stream)), "kq_debug_transform")


def debug_encode_f32(V, codes, scales, stream=None) -> None:
    M, K = V.shape
    _check(lib.kq_debug_encode_f32(_ptr(V), M, K, _ptr(codes), _ptr(scales), _stream(stream)),
           "kq_debug_encode_f32")


def last_device_error(layer: Layer, act, M: int, stream=None) -> int:
    """0 if the device error word is clear, else ERR_DEVICE_TIMEOUT (a bounded device wait
    ran out) or ERR_LOWRANK_RANGE (a low-rank activation was saturated to the fp16 range).
    Synchronises the stream and clears the word."""
    return int(lib.kq_last_device_error(layer.desc, _ptr(act), int(M), _stream(stream)))


def debug_wait_timeout(layer: Layer, act, M: int, limit_us: int, stream=None) -> None:
    """Enqueue one warp that waits limit_us on a barrier nothing completes, so that the
    next last_device_error on `act` reports ERR_DEVICE_TIMEOUT."""
    _need(act, __import__("torch").uint8, act_bytes(layer, M), "act")
    _check(lib.kq_debug_wait_timeout(layer.desc, _ptr(act), int(M), int(limit_us), _stream(stream)),
           "kq_debug_wait_timeout")


# ---------------------------------------------------------------- 8-bit operators --------
def _fits(size: int, name: str) -> None:
    """ctypes would pass the low 32 bits of a size to the C ABI without a word."""
    if not -1 << 31 <= size < 1 << 31:
        raise ValueError(f"{name} = {size} is past 32 bits")


class Fp8Layer:
    """One 8-bit linear layer (the C ``kq_fp8_desc``): E4M3 codes with a power-of-two scale for
    each token and 128 features, and for each 128 x 128 piece of a weight. ``gated``: two
    weights and ``activation(X Wgate) * (X Wup)``, ``activation`` ``"silu"`` or ``"gelu"`` (erf)."""

    def __init__(self, K: int, N: int, gated: bool = False, activation: str = "silu"):
        self.K, self.N, self.gated, self.activation = int(K), int(N), bool(gated), activation
        _fits(self.K, "K"), _fits(self.N, "N")
        self._desc = _Fp8Desc(K=self.K, N=self.N, gated=int(self.gated), activation=_ACTIVATION[activation])
        self._ref = ctypes.byref(self._desc)
        self._weights_bytes = fp8_weights_bytes(self)

    @property
    def desc(self):
        return self._ref


class _Names:
    """What the 8-bit calls use of torch, looked up once: a call for one token takes a few
    microseconds on the host, and each lookup on its way counts."""

    def __init__(self):
        import torch
        self.u8, self.f32 = torch.uint8, torch.float32
        self.bf16 = (torch.bfloat16,)
        self.out = {OUT_F32: (torch.float32,), OUT_BF16: (torch.bfloat16,)}
        self.flag = {torch.float32: OUT_F32, torch.bfloat16: OUT_BF16}
        self.raw_stream, self.device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice
        self.guard = torch.cuda.device


@functools.lru_cache(maxsize=None)
def _names() -> _Names:
    return _Names()


def _rows(t, dtypes, rows: int | None, width: int, name: str) -> int:
    """Checks a matrix whose rows may be a pitch apart and returns the pitch."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype not in dtypes:
        raise ValueError(f"{name} must be {' or '.join(map(str, dtypes))}, got {t.dtype}")
    shape = t.shape
    if len(shape) != 2 or shape[1] != width or (rows is not None and shape[0] != rows):
        raise ValueError(f"{name} must be [{'M' if rows is None else rows}, {width}], got {list(shape)}")
    pitch, step = t.stride()
    if step != 1:
        raise ValueError(f"{name} must have contiguous rows")
    # the pitch of a single row is of no consequence, and torch leaves it arbitrary
    return pitch if shape[0] > 1 else width


def _flat(t, dtype, numel: int, name: str):
    """Checks a contiguous tensor of at least numel elements (its device: _fp8_call)."""
    if t is None:
        raise ValueError(f"{name} is required")
    if t.dtype is not dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if t.numel() < numel:
        raise ValueError(f"{name} has {t.numel()} elements, needs {numel}")
    return t


def _fp8_call(fn, where: str, stream, tensors, args) -> None:
    """Calls fn(*args, stream) on the device of `tensors`, which must all be on one CUDA device,
    and on `stream` or that device's current stream."""
    names = _names()
    dev = tensors[0].get_device()
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"{where}: tensors are on different devices")
    if dev < 0:
        raise ValueError(f"{where}: every tensor must be a CUDA tensor")
    if stream is None:
        raw = names.raw_stream(dev)
    elif stream.device_index != dev:
        raise ValueError(f"{where}: the stream is of another device than the tensors")
    else:
        raw = stream.cuda_stream
    if names.device() == dev:
        status = fn(*args, raw)
    else:
        with names.guard(dev):
            status = fn(*args, raw)
    if status:
        raise KQError(status, where)


def fp8_weights_bytes(layer: Fp8Layer) -> int:
    return int(lib.kq_fp8_weights_bytes(layer.desc))


@functools.lru_cache(maxsize=4096)
def fp8_act_bytes(K: int, M: int) -> int:
    """0 for sizes that no call takes."""
    return int(lib.kq_fp8_act_bytes(int(K), int(M))) if 0 < min(K, M) and max(K, M) < 1 << 31 else 0


def fp8_ffn_bytes(gated: Fp8Layer, down: Fp8Layer, M: int) -> int:
    """0 for sizes that no call takes."""
    return int(lib.kq_fp8_ffn_bytes(gated.desc, down.desc, int(M))) if 0 < M < 1 << 31 else 0


def _fp8_pair(layer: Fp8Layer, up, name: str) -> None:
    if (up is not None) != layer.gated:
        raise ValueError(f"{name} goes with gated layers, and with those only")


def _fp8_weights(layer: Fp8Layer, weights):
    if not layer._weights_bytes:
        raise ValueError(f"unsupported 8-bit layer K={layer.K} N={layer.N}")
    return _flat(weights, _names().u8, layer._weights_bytes, "weights")


def _e4m3(t, numel: int, name: str):
    import torch
    if t is not None and t.dtype == torch.float8_e4m3fn:
        t = t.view(torch.uint8)
    return _flat(t, torch.uint8, numel, name)


def fp8_prepare_weights(layer: Fp8Layer, W, weights, W_up=None, stream=None) -> None:
    """Quantize W (bf16 [K, N]; gated layers: W is the gate's and W_up the other) into weights."""
    import torch
    _fp8_pair(layer, W_up, "W_up")
    _fp8_weights(layer, weights)
    for t, name in ((W, "W"), (W_up, "W_up"))[:1 + layer.gated]:
        _flat(t, torch.bfloat16, layer.K * layer.N, name)
    _fp8_call(lib.kq_fp8_prepare_weights, "kq_fp8_prepare_weights", stream, (W, W_up, weights),
              (layer.desc, _ptr(W), _ptr(W_up), _ptr(weights)))


def _fp8_parts(layer: Fp8Layer, codes, scales, up_codes, up_scales, optional: bool):
    import torch
    n, ns = layer.K * layer.N, -(-layer.N // 128) * -(-layer.K // 128)
    parts = [codes, scales, up_codes, up_scales]
    for i, (t, name) in enumerate(zip(parts, ("codes", "scales", "up_codes", "up_scales"))):
        if t is None and (optional or (i > 1 and not layer.gated)):
            continue
        if i > 1 and not layer.gated:
            raise ValueError(f"{name} goes with gated layers only")
        parts[i] = _flat(t, torch.uint8, ns, name) if i % 2 else _e4m3(t, n, name)
    return parts


def fp8_weights_pack(layer: Fp8Layer, codes, scales, weights, up_codes=None, up_scales=None, stream=None) -> None:
    """Write weights from canonical parts: codes [N, K] (uint8 or float8_e4m3fn), scales uint8
    [ceil(N / 128), ceil(K / 128)] (exponent + 127); gated layers take the up_ pair too."""
    _fp8_weights(layer, weights)
    parts = _fp8_parts(layer, codes, scales, up_codes, up_scales, optional=False)
    _fp8_call(lib.kq_fp8_weights_pack, "kq_fp8_weights_pack", stream, (weights, *parts),
              (layer.desc, *map(_ptr, parts), _ptr(weights)))


def fp8_weights_unpack(layer: Fp8Layer, weights, codes=None, scales=None, up_codes=None, up_scales=None,
                   stream=None) -> None:
    _fp8_weights(layer, weights)
    parts = _fp8_parts(layer, codes, scales, up_codes, up_scales, optional=True)
    _fp8_call(lib.kq_fp8_weights_unpack, "kq_fp8_weights_unpack", stream, (weights, *parts),
              (layer.desc, _ptr(weights), *map(_ptr, parts)))


def _fp8_act(act, K: int, M: int, name: str = "act"):
    n = fp8_act_bytes(K, M)
    if not n:
        _fits(K, "K"), _fits(M, "M")
    return _flat(act, _names().u8, n, name)


def fp8_quantize_act(X, act, stream=None) -> None:
    """Quantize X (bf16 [M, K], rows may be a pitch apart) into an activation workspace."""
    M, K = X.shape
    ldx = _rows(X, _names().bf16, None, K, "X")
    _fp8_act(act, K, M)
    _fp8_call(lib.kq_fp8_quantize_act, "kq_fp8_quantize_act", stream, (X, act),
              (K, X.data_ptr(), ldx, M, act.data_ptr(), act.numel()))


def _fp8_norm(gamma, residual, M: int, K: int):
    """(residual address, pitch, dtype) after the checks."""
    names = _names()
    _flat(gamma, names.f32, K, "gamma")
    if residual is None:
        return None, 0, OUT_F32
    ldr = _rows(residual, names.flag, M, K, "residual")
    return residual.data_ptr(), ldr, names.flag[residual.dtype]


def fp8_rmsnorm_act(X, gamma, eps: float, act, residual=None, stream=None) -> None:
    """Root-mean-square norm of X + residual times gamma, quantized into act; residual (bf16 or
    fp32 [M, K]) is replaced by the sum."""
    M, K = X.shape
    ldx = _rows(X, _names().bf16, None, K, "X")
    res, ldr, rdt = _fp8_norm(gamma, residual, M, K)
    _fp8_act(act, K, M)
    _fp8_call(lib.kq_fp8_rmsnorm_act, "kq_fp8_rmsnorm_act", stream, (X, gamma, act, residual),
              (K, X.data_ptr(), ldx, res, ldr, rdt, gamma.data_ptr(), eps, M, act.data_ptr(), act.numel()))


def fp8_act_pack(K: int, codes, scales, M: int, act, stream=None) -> None:
    import torch
    codes = _e4m3(codes, M * K, "codes")
    _flat(scales, torch.uint8, M * -(-K // 128), "scales")
    _fp8_act(act, K, M)
    _fp8_call(lib.kq_fp8_act_pack, "kq_fp8_act_pack", stream, (codes, scales, act),
              (int(K), _ptr(codes), _ptr(scales), int(M), _ptr(act), act.numel()))


def fp8_act_unpack(K: int, act, M: int, codes=None, scales=None, values=None, stream=None) -> None:
    """Read an activation workspace: codes [M, K], scales uint8 [M, ceil(K / 128)], values (bf16
    or fp32 [M, K]) = code * 2^(scale - 127); parts that are None are skipped."""
    names = _names()
    _fp8_act(act, K, M)
    vdt = OUT_F32
    if codes is not None:
        codes = _e4m3(codes, M * K, "codes")
    if scales is not None:
        _flat(scales, names.u8, M * -(-K // 128), "scales")
    if values is not None:
        vdt = names.flag.get(values.dtype, OUT_F32)
        _flat(values, names.out[vdt][0], M * K, "values")
    _fp8_call(lib.kq_fp8_act_unpack, "kq_fp8_act_unpack", stream, (act, codes, scales, values),
              (K, act.data_ptr(), M, _ptr(codes), _ptr(scales), _ptr(values), vdt))


def _fp8_y(Y, M: int, N: int, out_dtype: int) -> int:
    dtypes = _names().out.get(out_dtype)
    if dtypes is None:
        raise ValueError(f"out_dtype must be OUT_F32 or OUT_BF16, got {out_dtype}")
    return _rows(Y, dtypes, M, N, "Y")


def fp8_gemm(layer: Fp8Layer, weights, act, M: int, Y, out_dtype: int = OUT_F32, stream=None) -> None:
    """The layer on a filled activation workspace."""
    _fp8_weights(layer, weights)
    _fp8_act(act, layer.K, M)
    ldy = _fp8_y(Y, M, layer.N, out_dtype)
    _fp8_call(lib.kq_fp8_gemm, "kq_fp8_gemm", stream, (weights, act, Y),
              (layer._ref, weights.data_ptr(), act.data_ptr(), M, Y.data_ptr(), ldy, out_dtype))


def fp8_gated_act(layer: Fp8Layer, weights, act, M: int, out_act, stream=None) -> None:
    """A gated layer whose output is quantized into out_act, the workspace of a following layer."""
    _fp8_weights(layer, weights)
    _fp8_act(act, layer.K, M)
    _fp8_act(out_act, layer.N, M, "out_act")
    _fp8_call(lib.kq_fp8_gated_act, "kq_fp8_gated_act", stream, (weights, act, out_act),
              (layer._ref, weights.data_ptr(), act.data_ptr(), M, out_act.data_ptr(), out_act.numel()))


def fp8_linear(layer: Fp8Layer, weights, X, Y, act, out_dtype: int = OUT_F32, stream=None) -> None:
    """The layer on X (bf16 [M, K]) into Y [M, N]; act is scratch."""
    M, K = X.shape
    _fp8_weights(layer, weights)
    ldx = _rows(X, _names().bf16, None, layer.K, "X")
    ldy = _fp8_y(Y, M, layer.N, out_dtype)
    _fp8_act(act, K, M)
    _fp8_call(lib.kq_fp8_linear, "kq_fp8_linear", stream, (weights, X, Y, act),
              (layer._ref, weights.data_ptr(), X.data_ptr(), ldx, M, Y.data_ptr(), ldy, out_dtype,
               act.data_ptr(), act.numel()))


def fp8_ffn(gated: Fp8Layer, gated_weights, down: Fp8Layer, down_weights, X, gamma, eps: float, Y, ws,
            out_dtype: int = OUT_F32, residual=None, stream=None) -> None:
    """A feed-forward block: rmsnorm of X + residual (gamma None: X as it is), the gated layer,
    the down projection into Y. ws: uint8, fp8_ffn_bytes(gated, down, M)."""
    M = X.shape[0]
    _fp8_weights(gated, gated_weights)
    _fp8_weights(down, down_weights)
    if not gated.gated or down.gated or down.K != gated.N or M < 1:
        raise ValueError("fp8_ffn takes a gated layer and a plain one with K equal to its N, and M >= 1")
    _fits(M, "M")
    _flat(ws, _names().u8, fp8_act_bytes(gated.K, M) + fp8_act_bytes(gated.N, M), "ws")
    ldx = _rows(X, _names().bf16, None, gated.K, "X")
    if gamma is None and residual is not None:
        raise ValueError("residual needs gamma")
    res, ldr, rdt = _fp8_norm(gamma, residual, M, gated.K) if gamma is not None else (None, 0, OUT_F32)
    ldy = _fp8_y(Y, M, down.N, out_dtype)
    _fp8_call(lib.kq_fp8_ffn, "kq_fp8_ffn", stream, (gated_weights, down_weights, X, gamma, residual, Y, ws),
              (gated._ref, gated_weights.data_ptr(), down._ref, down_weights.data_ptr(), X.data_ptr(), ldx, res, ldr,
               rdt, _ptr(gamma), eps, M, Y.data_ptr(), ldy, out_dtype, ws.data_ptr(), ws.numel()))


def fp8_last_device_error(act, stream=None) -> int:
    """0, or ERR_DEVICE_TIMEOUT if a bounded device wait ran out. Synchronises the stream and
    clears the word."""
    import torch
    _need(act, torch.uint8, 256, "act")
    with torch.cuda.device(act.device):
        return int(lib.kq_fp8_last_device_error(_ptr(act), _stream(stream)))


def fp8_debug_wait_timeout(layer: Fp8Layer, weights, act, M: int, k_tile: int, limit_us: int, X=None, Y=None,
                           out_act=None, out_dtype: int = OUT_F32, stream=None) -> None:
    """The product of fp8_gemm, of fp8_linear (with X) or of fp8_gated_act (with out_act instead of Y) in
    which every CTA leaves out the load of the weights of its k_tile-th k-tile and waits limit_us at most."""
    _fp8_weights(layer, weights)
    _fp8_act(act, layer.K, M)
    ldx = 0 if X is None else _rows(X, _names().bf16, M, layer.K, "X")
    ldy = 0 if out_act is not None else _fp8_y(Y, M, layer.N, out_dtype)
    if out_act is not None:
        _fp8_act(out_act, layer.N, M, "out_act")
    _fp8_call(lib.kq_fp8_debug_wait_timeout, "kq_fp8_debug_wait_timeout", stream, (weights, X, Y, act, out_act),
              (layer._ref, _ptr(weights), _ptr(X), ldx, int(M), _ptr(Y), ldy, out_dtype, _ptr(act), act.numel(),
               _ptr(out_act), 0 if out_act is None else out_act.numel(), int(k_tile), int(limit_us)))
