"""Thin ctypes binding of libsparse_ffn.so (declared in include/sparse_ffn.h).

The functions carry the C names and do argument marshalling only: they check that the
torch tensors they are given live on the GPU with the expected dtype and layout, pass
their device pointers and the current stream to the library, and raise on a negative
status. Every step of the computation runs in the library's HIP kernels; PyTorch only
owns the device memory and the stream. Importing this module fails loudly when the
library has not been built (``python -m contextual_activation_sparsity_amd.build``); so do
the paged cache's calls and the norm where their compiled tensor checks have not been.
"""

import ctypes
import os
import re
import sys
from dataclasses import dataclass
from typing import Optional

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
# SFN_LIBRARY names another build of the same library (the host-sanitized one)
LIB_PATH = os.environ.get("SFN_LIBRARY") or os.path.join(_PKG, "libsparse_ffn.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -m contextual_activation_sparsity_amd.build` "
        "(hipcc, gfx950). There is no fallback implementation."
    )
_lib = ctypes.CDLL(LIB_PATH)

SFN_OK, SFN_EINVAL, SFN_ESHAPE, SFN_EDTYPE = 0, -1, -2, -3
SFN_EWORKSPACE, SFN_EALIGN, SFN_EUNSUPPORTED, SFN_EHIP, SFN_ETOOLARGE = -4, -5, -6, -7, -8
SFN_F32, SFN_BF16 = 0, 1
SFN_ACT_SILU, SFN_ACT_RELU = 0, 1
SFN_MAX_BATCH, SFN_MAX_CHUNK = 4, 16
SFN_PIPE_SEQUENTIAL, SFN_PIPE_PARALLEL = 0, 1
SFN_WORKSPACE_HEADER_BYTES, SFN_WORKSPACE_STATUS_OFFSET = 2048, 1024
SFN_STATUS_BALANCER_TIMEOUT, SFN_STATUS_PREDICTOR_TIMEOUT = 1, 2
SFN_NOALLOC_SCRATCH_BYTES = 32 << 20
SFN_MAX_REQUESTS, SFN_MAX_STEP_TOKENS, SFN_MAX_HEADS = 4096, 262144, 1024

EXPORTED = (
    "sparse_ffn_workspace_size",
    "svd_predict_workspace_size",
    "sparse_ffn_strerror",
    "sparse_ffn_calibrate",
    "sparse_ffn_decode",
    "sparse_ffn_decode_noalloc",
    "sparse_ffn_decode_parallel",
    "sparse_ffn_svd_workspace_size",
    "sparse_ffn_decode_svd",
    "svd_predict",
    "ffn_dense_chunk",
    "kv_cache_plan",
    "kv_cache_append",
    "kv_cache_attend_workspace_size",
    "kv_cache_attend",
    "residual_norm",
)


class sfn_ffn(ctypes.Structure):
    _fields_ = [
        ("d", ctypes.c_int32), ("f", ctypes.c_int32), ("wdtype", ctypes.c_int32), ("act", ctypes.c_int32),
        ("w_gate", ctypes.c_void_p), ("w_up", ctypes.c_void_p), ("w_down_t", ctypes.c_void_p),
        ("b_gate", ctypes.c_void_p),
    ]


class sfn_svd(ctypes.Structure):
    _fields_ = [
        ("d", ctypes.c_int32), ("f", ctypes.c_int32), ("r", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("q", ctypes.c_void_p), ("l", ctypes.c_void_p), ("b", ctypes.c_void_p), ("tau", ctypes.c_void_p),
    ]


class sfn_kv(ctypes.Structure):
    _fields_ = [
        ("n_pages", ctypes.c_int32), ("page", ctypes.c_int32), ("h_kv", ctypes.c_int32), ("dh", ctypes.c_int32),
        ("dtype", ctypes.c_int32), ("reserved", ctypes.c_int32), ("k", ctypes.c_void_p), ("v", ctypes.c_void_p),
    ]


class sfn_norm(ctypes.Structure):
    _fields_ = [
        ("d", ctypes.c_int32), ("wdtype", ctypes.c_int32), ("eps", ctypes.c_float), ("scale", ctypes.c_float),
        ("w_post", ctypes.c_void_p), ("w_pre", ctypes.c_void_p),
    ]


_vp, _i32, _sz, _f32 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t, ctypes.c_float
_lib.sparse_ffn_workspace_size.argtypes = [ctypes.POINTER(sfn_ffn), _i32]
_lib.sparse_ffn_workspace_size.restype = _sz
_lib.svd_predict_workspace_size.argtypes = [ctypes.POINTER(sfn_svd)]
_lib.svd_predict_workspace_size.restype = _sz
_lib.sparse_ffn_strerror.argtypes = [ctypes.c_int]
_lib.sparse_ffn_strerror.restype = ctypes.c_char_p
_lib.sparse_ffn_calibrate.argtypes = [ctypes.POINTER(sfn_ffn), _vp, _i32, _f32, _vp, _vp, _vp, _sz, _vp]
_lib.sparse_ffn_calibrate.restype = ctypes.c_int
_lib.sparse_ffn_decode.argtypes = [ctypes.POINTER(sfn_ffn), _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.sparse_ffn_decode.restype = ctypes.c_int
_lib.sparse_ffn_decode_noalloc.argtypes = [ctypes.POINTER(sfn_ffn), _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp]
_lib.sparse_ffn_decode_noalloc.restype = ctypes.c_int
_lib.sparse_ffn_decode_parallel.argtypes = [ctypes.POINTER(sfn_ffn), _vp, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.sparse_ffn_decode_parallel.restype = ctypes.c_int
_lib.sparse_ffn_svd_workspace_size.argtypes = [ctypes.POINTER(sfn_ffn), ctypes.POINTER(sfn_svd)]
_lib.sparse_ffn_svd_workspace_size.restype = _sz
_lib.sparse_ffn_decode_svd.argtypes = [ctypes.POINTER(sfn_ffn), ctypes.POINTER(sfn_svd), _vp, _i32, _vp, _vp, _vp, _vp,
                                       _sz, _vp]
_lib.sparse_ffn_decode_svd.restype = ctypes.c_int
_lib.svd_predict.argtypes = [ctypes.POINTER(sfn_svd), _vp, _vp, _vp, _vp, _vp, _sz, _vp]
_lib.svd_predict.restype = ctypes.c_int
_lib.ffn_dense_chunk.argtypes = [ctypes.POINTER(sfn_ffn), _vp, _i32, _vp, _vp, _sz, _vp]
_lib.ffn_dense_chunk.restype = ctypes.c_int
_i64 = ctypes.c_int64
_lib.kv_cache_plan.argtypes = [ctypes.POINTER(sfn_kv), _i32, _i32, _i32] + [_vp] * 13
_lib.kv_cache_plan.restype = ctypes.c_int
_lib.kv_cache_append.argtypes = [ctypes.POINTER(sfn_kv), _i32, _i32, _vp, _i64, _vp, _i64, _vp, _i64, _vp, _vp, _vp, _i32,
                                 _i32, _vp, _vp]
_lib.kv_cache_append.restype = ctypes.c_int
_lib.kv_cache_attend_workspace_size.argtypes = [ctypes.POINTER(sfn_kv), _i32, _i32, _i32, _i32, _i32]
_lib.kv_cache_attend_workspace_size.restype = _sz
_lib.kv_cache_attend.argtypes = [ctypes.POINTER(sfn_kv), _i32, _i32, _i32, _vp, _i64, _vp, _i32, _vp, _vp, _i32, _i32, _f32,
                                 _i32, _vp, _vp, _sz, _vp]
_lib.kv_cache_attend.restype = ctypes.c_int
_lib.residual_norm.argtypes = [ctypes.POINTER(sfn_norm), _i32, _vp, _i32, _vp, _i32, _vp, _i64, _vp, _vp, _vp]
_lib.residual_norm.restype = ctypes.c_int


class _NoChecks:
    """Stands for the compiled tensor checks where they cannot be had."""

    def __init__(self, why):
        self._why = f"{why}: build it with `python -m contextual_activation_sparsity_amd.build`"

    def __getattr__(self, name):
        raise ImportError(self._why)


def _load_checks():
    """The tensor checks of the paged cache's calls and the norm, compiled (csrc/torch_args.cpp)
    for one torch and one Python. The FFN's calls do without them, so a module that is missing
    or was built for others is reported by the calls that need it."""
    try:
        from . import _torch_args as m

        built = (m.TORCH_VERSION, m.PY_VERSION)
    except (ImportError, AttributeError) as e:
        return _NoChecks(e)
    here = (re.match(r"\d+\.\d+\.\d+|", torch.__version__).group(), "%d.%d" % sys.version_info[:2])
    if built != here:
        return _NoChecks(f"_torch_args.so is for torch {built[0]} and Python {built[1]}, this is torch {here[0]} and Python {here[1]}")
    m.bind(*(ctypes.cast(f, ctypes.c_void_p).value
             for f in (_lib.kv_cache_plan, _lib.kv_cache_append, _lib.kv_cache_attend, _lib.residual_norm)))
    return m


_args = _load_checks()


class SparseFFNError(RuntimeError):
    def __init__(self, status, call):
        self.status = status
        super().__init__(f"{call}: status {status} ({sparse_ffn_strerror(status)})")


def _check(status, call):
    if status != SFN_OK:
        raise SparseFFNError(status, call)


def _ptr(t: Optional[torch.Tensor], name, dtype=None, numel=None):
    if t is None:
        return None
    # the common case first: this runs several times a call, in the time of a short kernel
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.is_contiguous() and (dtype is None or t.dtype is dtype)
            and (numel is None or t.numel() >= numel)):
        return t.data_ptr()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor or None")
    if t.device.type != "cuda":
        raise ValueError(f"{name} must be a GPU tensor (got {t.device})")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if dtype is not None and t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} (got {t.dtype})")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name} holds {t.numel()} elements, needs {numel}")
    return t.data_ptr()


def _stream(stream):
    if stream is None:
        # torch.cuda.current_stream().cuda_stream without building a Stream object (2.8 us)
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


_WDT = {torch.bfloat16: SFN_BF16, torch.float32: SFN_F32}


@dataclass
class FFNLayer:
    """One FFN layer's device tensors, each [f, d] row-major (w_down_t = W_down^T)."""

    w_gate: torch.Tensor
    w_up: Optional[torch.Tensor]
    w_down_t: Optional[torch.Tensor]
    b_gate: Optional[torch.Tensor] = None
    act: int = SFN_ACT_SILU

    def __post_init__(self):
        f, d = self.w_gate.shape
        dt = self.w_gate.dtype
        if dt not in _WDT:
            raise ValueError("weights must be bfloat16 or float32")
        for name in ("w_up", "w_down_t"):
            t = getattr(self, name)
            if t is not None and (tuple(t.shape) != (f, d) or t.dtype != dt):
                raise ValueError(f"{name} must be [{f}, {d}] {dt}")
        if self.b_gate is not None and (self.b_gate.dtype != torch.float32 or self.b_gate.numel() != f):
            raise ValueError("b_gate must be float32 [f]")
        self.d, self.f, self.dtype = d, f, dt
        self.c = sfn_ffn(
            d, f, _WDT[dt], int(self.act),
            _ptr(self.w_gate, "w_gate"), _ptr(self.w_up, "w_up"), _ptr(self.w_down_t, "w_down_t"),
            _ptr(self.b_gate, "b_gate", torch.float32),
        )


@dataclass
class SVDPredictor:
    """Rank-r predictor factors of one layer: q [r, d] bf16, l [f, r] bf16, b and tau [f] fp32."""

    q: torch.Tensor
    l: torch.Tensor
    tau: torch.Tensor
    b: Optional[torch.Tensor] = None

    def __post_init__(self):
        r, d = self.q.shape
        f, r2 = self.l.shape
        if r2 != r or self.q.dtype != torch.bfloat16 or self.l.dtype != torch.bfloat16:
            raise ValueError("q must be [r, d] and l [f, r], both bfloat16")
        self.d, self.f, self.r = d, f, r
        self.c = sfn_svd(d, f, r, 0, _ptr(self.q, "q"), _ptr(self.l, "l"),
                         _ptr(self.b, "b", torch.float32), _ptr(self.tau, "tau", torch.float32, f))


def sparse_ffn_workspace_size(layer: FFNLayer, max_tokens: int) -> int:
    return int(_lib.sparse_ffn_workspace_size(ctypes.byref(layer.c), int(max_tokens)))


def svd_predict_workspace_size(pred: SVDPredictor) -> int:
    return int(_lib.svd_predict_workspace_size(ctypes.byref(pred.c)))


def sparse_ffn_strerror(status: int) -> str:
    return _lib.sparse_ffn_strerror(int(status)).decode()


def workspace_status(ws: torch.Tensor) -> int:
    """The workspace status word (synchronises): 0, or the SFN_STATUS_* code of a bounded
    device-side wait that gave up during a call on this workspace."""
    off = SFN_WORKSPACE_STATUS_OFFSET
    return int(ws[off:off + 4].view(torch.int32).item())


def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """A zero-filled workspace of nbytes (its reserved first 2 KiB must start at zero)."""
    if nbytes <= 0:
        raise ValueError("workspace size query failed (invalid arguments)")
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def sparse_ffn_calibrate(layer: FFNLayer, x_cal: torch.Tensor, k: float, t_out: torch.Tensor,
                         ws: torch.Tensor, scores_out: Optional[torch.Tensor] = None, stream=None):
    n = x_cal.shape[0]
    st = _lib.sparse_ffn_calibrate(
        ctypes.byref(layer.c), _ptr(x_cal, "x_cal", layer.dtype, n * layer.d), int(n), float(k),
        _ptr(t_out, "t_out", torch.float32, 1),
        _ptr(scores_out, "scores_out", torch.float32, n * layer.f),
        _ptr(ws, "ws"), ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "sparse_ffn_calibrate")


def sparse_ffn_decode(layer: FFNLayer, x: torch.Tensor, t: Optional[torch.Tensor], ws: torch.Tensor,
                      y: Optional[torch.Tensor] = None, cand: Optional[torch.Tensor] = None,
                      n_cand: Optional[torch.Tensor] = None, mask_in: Optional[torch.Tensor] = None,
                      active_idx: Optional[torch.Tensor] = None, n_active: Optional[torch.Tensor] = None,
                      stream=None):
    B = x.shape[0] if x.dim() == 2 else 1
    st = _lib.sparse_ffn_decode(
        ctypes.byref(layer.c), _ptr(x, "x", layer.dtype, B * layer.d), int(B),
        _ptr(t, "t", torch.float32, 1), _ptr(cand, "cand", torch.int32), _ptr(n_cand, "n_cand", torch.int32, 1),
        _ptr(mask_in, "mask_in", torch.uint8, B * layer.f), _ptr(y, "y", torch.float32, B * layer.d),
        _ptr(active_idx, "active_idx", torch.int32, B * layer.f), _ptr(n_active, "n_active", torch.int32, B),
        _ptr(ws, "ws"), ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "sparse_ffn_decode")


def sparse_ffn_decode_noalloc(layer: FFNLayer, x: torch.Tensor, t: Optional[torch.Tensor],
                              y: Optional[torch.Tensor] = None, cand: Optional[torch.Tensor] = None,
                              n_cand: Optional[torch.Tensor] = None, mask_in: Optional[torch.Tensor] = None,
                              active_idx: Optional[torch.Tensor] = None, n_active: Optional[torch.Tensor] = None,
                              stream=None):
    B = x.shape[0] if x.dim() == 2 else 1
    st = _lib.sparse_ffn_decode_noalloc(
        ctypes.byref(layer.c), _ptr(x, "x", layer.dtype, B * layer.d), int(B),
        _ptr(t, "t", torch.float32, 1), _ptr(cand, "cand", torch.int32), _ptr(n_cand, "n_cand", torch.int32, 1),
        _ptr(mask_in, "mask_in", torch.uint8, B * layer.f), _ptr(y, "y", torch.float32, B * layer.d),
        _ptr(active_idx, "active_idx", torch.int32, B * layer.f), _ptr(n_active, "n_active", torch.int32, B),
        _stream(stream))
    _check(st, "sparse_ffn_decode_noalloc")


def sparse_ffn_decode_parallel(layer: FFNLayer, x: torch.Tensor, cand: torch.Tensor, n_cand: torch.Tensor,
                               ws: torch.Tensor, y: torch.Tensor, stream=None):
    st = _lib.sparse_ffn_decode_parallel(
        ctypes.byref(layer.c), _ptr(x, "x", layer.dtype, layer.d), _ptr(cand, "cand", torch.int32),
        _ptr(n_cand, "n_cand", torch.int32, 1), _ptr(y, "y", torch.float32, layer.d), _ptr(ws, "ws"),
        ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "sparse_ffn_decode_parallel")


def sparse_ffn_svd_workspace_size(layer: FFNLayer, pred: SVDPredictor) -> int:
    return int(_lib.sparse_ffn_svd_workspace_size(ctypes.byref(layer.c), ctypes.byref(pred.c)))


def sparse_ffn_decode_svd(layer: FFNLayer, pred: SVDPredictor, x: torch.Tensor, ws: torch.Tensor,
                          y: Optional[torch.Tensor] = None, idx: Optional[torch.Tensor] = None,
                          n_idx: Optional[torch.Tensor] = None, pipeline: int = SFN_PIPE_SEQUENTIAL, stream=None):
    st = _lib.sparse_ffn_decode_svd(
        ctypes.byref(layer.c), ctypes.byref(pred.c), _ptr(x, "x", torch.bfloat16, layer.d), int(pipeline),
        _ptr(y, "y", torch.float32, layer.d), _ptr(idx, "idx", torch.int32, layer.f),
        _ptr(n_idx, "n_idx", torch.int32, 1), _ptr(ws, "ws"), ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "sparse_ffn_decode_svd")


def svd_predict(pred: SVDPredictor, x: torch.Tensor, cand_idx: torch.Tensor, n_cand: torch.Tensor,
                ws: torch.Tensor, p_out: Optional[torch.Tensor] = None, stream=None):
    st = _lib.svd_predict(
        ctypes.byref(pred.c), _ptr(x, "x", torch.bfloat16, pred.d), _ptr(cand_idx, "cand_idx", torch.int32, pred.f),
        _ptr(n_cand, "n_cand", torch.int32, 1), _ptr(p_out, "p_out", torch.float32, pred.f),
        _ptr(ws, "ws"), ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "svd_predict")


def ffn_dense_chunk(layer: FFNLayer, x: torch.Tensor, y: torch.Tensor, ws: torch.Tensor, stream=None):
    n = x.shape[0]
    st = _lib.ffn_dense_chunk(
        ctypes.byref(layer.c), _ptr(x, "x", layer.dtype, n * layer.d), int(n),
        _ptr(y, "y", torch.float32, n * layer.d), _ptr(ws, "ws"), ws.numel() * ws.element_size(),
        _stream(stream))
    _check(st, "ffn_dense_chunk")


@dataclass
class KVCache:
    """One layer's paged key/value cache: k and v [n_pages, h_kv, page, dh], bfloat16 or
    float32, page 16, 32, 64, 128 or 256 tokens, dh 64 or 128."""

    k: torch.Tensor
    v: torch.Tensor

    def __post_init__(self):
        if self.k.dim() != 4 or self.k.shape != self.v.shape or self.k.dtype != self.v.dtype:
            raise ValueError("k and v must both be [n_pages, h_kv, page, dh] of one dtype")
        if self.k.dtype not in _WDT:
            raise ValueError("the cache must be bfloat16 or float32")
        self.n_pages, self.h_kv, self.page, self.dh = self.k.shape
        self.dtype = self.k.dtype
        self.c = sfn_kv(self.n_pages, self.page, self.h_kv, self.dh, _WDT[self.dtype], 0, _ptr(self.k, "k"),
                        _ptr(self.v, "v"))
        self.addr = ctypes.addressof(self.c)


@dataclass
class ResidualNorm:
    """Weights of residual_norm, [d] each: w_pre of the norm before the next block, w_post
    (optional) of the norm after the last one, the residual scale and the norms' eps."""

    w_pre: torch.Tensor
    w_post: Optional[torch.Tensor] = None
    eps: float = 1e-5
    scale: float = 1.0

    def __post_init__(self):
        if self.w_pre.dtype not in _WDT:
            raise ValueError("weights must be bfloat16 or float32")
        self.d, self.dtype = self.w_pre.numel(), self.w_pre.dtype
        if self.w_post is not None and self.w_post.numel() != self.d:
            raise ValueError(f"w_post must be [{self.d}]")
        self.c = sfn_norm(self.d, _WDT[self.dtype], float(self.eps), float(self.scale),
                          _ptr(self.w_post, "w_post", self.dtype), _ptr(self.w_pre, "w_pre"))
        self.addr = ctypes.addressof(self.c)


def kv_cache_plan(kv: KVCache, held_len: torch.Tensor, ctx_len: torch.Tensor, new_len: torch.Tensor, table: torch.Tensor,
                  free_pages: torch.Tensor, n_free: torch.Tensor, n_free_out: torch.Tensor, cu: torch.Tensor,
                  kv_len: torch.Tensor, pos: torch.Tensor, slot: torch.Tensor, status: torch.Tensor, stream=None):
    st = _args.plan(kv.addr, held_len, ctx_len, new_len, table, free_pages, n_free, n_free_out, cu, kv_len, pos, slot,
                    status, _stream(stream))
    _check(st, "kv_cache_plan")


def kv_cache_append(kv: KVCache, k: torch.Tensor, v: torch.Tensor, slot: torch.Tensor, q: Optional[torch.Tensor] = None,
                    q_out: Optional[torch.Tensor] = None, pos: Optional[torch.Tensor] = None,
                    rope: Optional[torch.Tensor] = None, stream=None):
    st = _args.append(kv.addr, k, v, slot, q, q_out, pos, rope, _stream(stream))
    _check(st, "kv_cache_append")


def kv_cache_attend_workspace_size(kv: KVCache, R: int, T: int, h_q: int, max_new: int, max_len: int) -> int:
    return int(_lib.kv_cache_attend_workspace_size(kv.c, int(R), int(T), int(h_q), int(max_new), int(max_len)))


def kv_cache_attend(kv: KVCache, q: torch.Tensor, table: torch.Tensor, cu: torch.Tensor, kv_len: torch.Tensor,
                    out: torch.Tensor, ws: torch.Tensor, max_new: int, max_len: int, scale: Optional[float] = None,
                    window: int = 0, stream=None):
    st = _args.attend(kv.addr, q, table, cu, kv_len, out, ws, max_new, max_len, kv.dh ** -0.5 if scale is None else scale,
                      window, _stream(stream))
    _check(st, "kv_cache_attend")


def residual_norm(norm: ResidualNorm, h: torch.Tensor, y: Optional[torch.Tensor], h_out: Optional[torch.Tensor],
                  x_out: Optional[torch.Tensor], gate: Optional[torch.Tensor] = None, stream=None):
    st = _args.norm(norm.addr, h, y, h_out, x_out, gate, _stream(stream))
    _check(st, "residual_norm")


def raw():
    """The loaded ctypes library (for tests of the C-level error conventions)."""
    return _lib
