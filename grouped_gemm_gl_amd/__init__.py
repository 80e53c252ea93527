"""Python binding of the gfx950 grouped-linear library ``libgrouped_linear.so``.

Argument marshalling only: each function takes torch tensors (device memory),
checks that their shapes, dtypes and devices agree with one another, and passes
their addresses plus the current HIP stream to the C entry point of the same name
(declared in ``include/grouped_linear.h``).  Every step of the computation runs in
the library's HIP kernels; nothing here computes, and there is no fallback: if the
library is not built, importing works but the first call raises.

Weights, biases and weight gradients are accepted stacked (one tensor with a
leading group dimension) or per group (a list of tensors); for a list, a device
array of their addresses is built and handed over.
"""
from __future__ import annotations

import collections
import ctypes
import functools
import os
from typing import Optional, Sequence, Union

import torch

__all__ = [
    "GL_F32", "GL_BF16", "GL_F16", "GL_E4M3", "GLError", "library_path", "load", "gl_version",
    "gl_workspace_size", "new_workspace", "workspace_offsets", "gl_offsets", "gl_read_status",
    "gl_forward", "gl_dgrad", "gl_wgrad", "gl_wgrad_bgrad", "gl_bgrad",
    "gl_group_quantize_mxfp8", "gl_colwise_ld", "gl_group_quantize_mxfp8_colwise",
    "gl_group_quantize_mxfp8_rowwise_colwise", "gl_quantize_mxfp8_colwise_weights",
    "gl_offsets_quantize_mxfp8", "gl_offsets_quantize_mxfp8_rowwise_colwise", "gl_quantize_mxfp8_weights",
    "gl_dgrad_mxfp8", "gl_wgrad_mxfp8", "gl_swiglu_forward", "gl_swiglu_backward",
    "gl_grouped_mlp_forward", "gl_grouped_mlp_backward", "WgradQueue", "gl_forward_noalloc",
    "NOALLOC_MAX_GROUPS", "gl_rmsnorm_forward", "gl_rmsnorm_workspace_size", "gl_rmsnorm_backward",
    "GL_SCORE_SOFTMAX", "GL_SCORE_SIGMOID", "gl_route_workspace_size", "gl_route_forward", "gl_route_backward",
    "gl_moe_few_tokens_workspace_size", "gl_moe_few_tokens", "MOE_MAX_TOKENS",
    "GL_GLU_SILU", "GL_GLU_GELU", "GL_GLU_GELU_TANH", "gl_glu_forward", "gl_glu_backward",
    "gl_quantize_int8", "gl_forward_int8", "gl_glu_forward_int8",
]

GL_F32, GL_BF16, GL_F16, GL_E4M3 = 0, 1, 2, 3
NOALLOC_MAX_GROUPS = 16384  # GL_NOALLOC_MAX_GROUPS
GL_SCORE_SOFTMAX, GL_SCORE_SIGMOID = 0, 1
MOE_MAX_TOKENS = 64  # GL_MOE_MAX_TOKENS
GL_GLU_SILU, GL_GLU_GELU, GL_GLU_GELU_TANH = 0, 1, 2
GL_STATUS_NEGATIVE_SPLIT, GL_STATUS_SUM_MISMATCH, GL_STATUS_WORKSPACE = 1, 2, 4

_HERE = os.path.dirname(os.path.abspath(__file__))
# GL_LIBRARY_PATH selects another build of the same library (e.g. the host-sanitized one)
library_path = os.environ.get("GL_LIBRARY_PATH") or os.path.join(_HERE, "libgrouped_linear.so")
_lib = None

Tensor = torch.Tensor
Grouped = Union[Tensor, Sequence[Tensor]]


class GLError(RuntimeError):
    """A non-zero return code of the C library, with its message."""

    def __init__(self, code: int, msg: str):
        super().__init__(f"[{code}] {msg}")
        self.code = code


def load():
    """Load the shared library (once); raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(library_path):
        raise RuntimeError(f"{library_path} is not built; run `python -m grouped_gemm_gl_amd.build`")
    lib = ctypes.CDLL(library_path)
    P, I, I64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64
    sig = {
        "gl_workspace_size": (ctypes.c_size_t, [I]),
        "gl_workspace_offsets": (P, [P]),
        "gl_offsets": (I, [P, I, I64, P, P]),
        "gl_read_status": (I, [P, ctypes.POINTER(ctypes.c_int), P]),
        "gl_forward": (I, [I, I64, I64, I64, I, I, P, P, P, P, P, P, P, P, P, I64, P, P]),
        "gl_dgrad": (I, [I, I64, I64, I64, I, P, P, P, P, I64, P, P]),
        "gl_wgrad": (I, [I, I64, I64, I64, I, I, P, P, P, P, I, P, P]),
        "gl_wgrad_bgrad": (I, [I, I64, I64, I64, I, I, I, P, P, P, P, I, P, P, P, P]),
        "gl_bgrad": (I, [I, I64, I64, I, P, P, P, P, P]),
        "gl_group_quantize_mxfp8": (I, [P, I64, I64, P, P, P]),
        "gl_colwise_ld": (I64, [I, I64]),
        "gl_group_quantize_mxfp8_colwise": (I, [P, I64, I, I64, P, P, P, I64, P]),
        "gl_quantize_mxfp8_colwise_weights": (I, [P, I, I64, I64, P, P, P]),
        "gl_group_quantize_mxfp8_rowwise_colwise": (I, [P, I64, I, I64, P, P, P, P, P, I64, P]),
        "gl_offsets_quantize_mxfp8": (I, [P, I, I64, P, P, I64, P, P, P]),
        "gl_offsets_quantize_mxfp8_rowwise_colwise": (I, [P, I, I64, P, P, I64, P, P, P, P, I64, P]),
        "gl_swiglu_forward": (I, [I64, I64, I, P, P, P]),
        "gl_swiglu_backward": (I, [I64, I64, I, P, P, P, P]),
        "gl_grouped_mlp_forward": (I, [I, I64, I64, I64, I64, I] + [P] * 12 + [I64, P, P]),
        "gl_grouped_mlp_backward": (I, [I, I64, I64, I64, I64, I, I] + [P] * 11 + [I64] + [P] * 8 + [I, P, P]),
        "gl_quantize_mxfp8_weights": (I, [P, I, I64, I64, P, P, P, P, P, P]),
        "gl_dgrad_mxfp8": (I, [I, I64, I64, I64, I, P, P, P, P, P, I64, P, P]),
        "gl_wgrad_mxfp8": (I, [I, I64, I64, I64, I, P, P, P, P, I64, P, P, I, P, P]),
        "gl_wgrad_queue_create": (I, [ctypes.POINTER(P)]),
        "gl_wgrad_queue_destroy": (I, [P]),
        "gl_wgrad_queue_put": (I, [P, I, I64, I64, I64, I, I, I, P, P, P, P, I, P, P, P]),
        "gl_wgrad_queue_put_mxfp8": (I, [P, I, I64, I64, I64, I, P, P, P, P, I64, P, P, I, P]),
        "gl_wgrad_queue_size": (I, [P]),
        "gl_wgrad_queue_run_next": (I, [P, P]),
        "gl_wgrad_queue_flush": (I, [P, P]),
        "gl_wgrad_queue_clear": (I, [P]),
        "gl_forward_noalloc": (I, [I, I64, I64, I64, I, I] + [P] * 10 + [I64, P]),
        "gl_rmsnorm_forward": (I, [I64, I64, I, I, P, P, P, ctypes.c_float, P, P, P, P, P]),
        "gl_rmsnorm_workspace_size": (ctypes.c_size_t, [I64, I64]),
        "gl_rmsnorm_backward": (I, [I64, I64, I, I, P, P, P, P, ctypes.c_float, P, I, P, I, P, P]),
        "gl_route_workspace_size": (ctypes.c_size_t, [I64, I]),
        "gl_route_forward": (I, [I64, I, I, I, I, I] + [P] * 8),
        "gl_route_backward": (I, [I64, I, I, I, I, I] + [P] * 5),
        "gl_moe_few_tokens_workspace_size": (ctypes.c_size_t, [I64, I, I, I64]),
        "gl_moe_few_tokens": (I, [I, I64, I64, I64, I64, I, I, I] + [P] * 17 + [I64, P, P]),
        "gl_glu_forward": (I, [I, I64, I64, I64, I, I] + [P] * 7 + [I64, P, P]),
        "gl_glu_backward": (I, [I, I64, I64, I64, I, I, I] + [P] * 10 + [I64] + [P] * 4 + [I, P, P]),
        "gl_quantize_int8": (I, [I64, I64, I, P, P, P, P]),
        "gl_forward_int8": (I, [I, I64, I64, I64, I] + [P] * 9 + [I64, P, P]),
        "gl_glu_forward_int8": (I, [I, I64, I64, I64, I, I] + [P] * 9 + [I64, P, P]),
        "gl_last_error": (ctypes.c_char_p, []),
        "gl_version": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    _lib = lib
    return lib


def _check(rc: int):
    if rc != 0:
        raise GLError(rc, load().gl_last_error().decode())


def _stream(stream) -> Optional[int]:
    if stream is None:
        if torch.cuda.is_initialized():  # the same handle, without a Stream object (2.4 us a call)
            return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
        return torch.cuda.current_stream().cuda_stream
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _ptr(t: Optional[Tensor]) -> Optional[int]:
    if t is None:
        return None
    if not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous")
    return t.data_ptr() if t.numel() else None


_DT = {torch.float32: GL_F32, torch.bfloat16: GL_BF16, torch.float16: GL_F16, torch.uint8: GL_E4M3}


def _dtype(t: Tensor) -> int:
    if t.dtype not in _DT:
        raise ValueError(f"unsupported dtype {t.dtype}")
    return _DT[t.dtype]


def _record(tensors, stream):
    """Ties tensors' memory to a caller-given stream: torch's caching allocator
    then waits for the work queued on that stream before it reuses the memory
    (without it, a pointer array freed right after an enqueue on another stream
    could be handed out again before the kernel has read it)."""
    if stream is None:
        return
    s = stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(_stream(stream))
    for t in tensors:
        if isinstance(t, Tensor) and t.is_cuda:
            t.record_stream(s)


def _grouped(g: Optional[Grouped], device, stream=None):
    """(stacked pointer, pointer-array pointer, keep-alive) for a stacked tensor or a
    list; the device pointer array of a list is tied to ``stream`` (see _record)."""
    if g is None:
        return None, None, None
    if isinstance(g, Tensor):
        return _ptr(g), None, None
    ptrs = torch.tensor([_ptr(t) or 0 for t in g], dtype=torch.int64, device=device)
    _record([ptrs], stream)
    return None, ptrs.data_ptr(), (ptrs, list(g))


def _first(g: Grouped) -> Tensor:
    return g[0] if not isinstance(g, Tensor) or g.dim() == 3 else g


def gl_version() -> str:
    return load().gl_version().decode()


def gl_workspace_size(num_groups: int) -> int:
    return int(load().gl_workspace_size(num_groups))


def new_workspace(num_groups: int, device="cuda") -> Tensor:
    """Device buffer sized for a call sequence over ``num_groups`` groups."""
    return torch.empty(gl_workspace_size(num_groups), dtype=torch.uint8, device=device)


def gl_offsets(m_splits: Tensor, total_rows: int, workspace: Tensor, stream=None) -> None:
    """Split-offset scan of the device int64 split sizes into ``workspace``."""
    if m_splits.dtype != torch.int64:
        raise ValueError("m_splits must be int64")
    _check(load().gl_offsets(_ptr(m_splits), m_splits.numel(), int(total_rows), _ptr(workspace), _stream(stream)))


def workspace_offsets(workspace: Tensor, num_groups: int) -> Tensor:
    """The int64[G+1] offsets inside a workspace, as a view (no device work); the
    library names where they sit (gl_workspace_offsets)."""
    start = int(load().gl_workspace_offsets(_ptr(workspace))) - workspace.data_ptr()
    return workspace[start: start + 8 * (num_groups + 1)].view(torch.int64)


def gl_read_status(workspace: Tensor, stream=None) -> int:
    """Synchronise the stream and return the workspace status word (0 = valid splits)."""
    st = ctypes.c_int(0)
    _check(load().gl_read_status(_ptr(workspace), ctypes.byref(st), _stream(stream)))
    return st.value


def gl_forward(x: Tensor, w: Grouped, y: Tensor, workspace: Tensor, *, bias: Optional[Grouped] = None,
               x_scale: Optional[Tensor] = None, w_scale: Optional[Grouped] = None, stream=None) -> Tensor:
    """y[:T] = grouped x W_g^T (+ b_g); T = x.shape[0]; rows of y past T are left untouched.

    x: [T, K] float32 / bfloat16, or uint8 E4M3 codes with ``x_scale`` [T, K/32];
    w: [G, N, K] or G tensors [N, K] (uint8 with ``w_scale`` for MXFP8);
    y: [>= T, N] (float32 / bfloat16; for MXFP8 its dtype picks the output type).
    """
    G = w.shape[0] if isinstance(w, Tensor) else len(w)
    w0 = _first(w)
    N, K = w0.shape[-2], w0.shape[-1]
    T = x.shape[0]
    if x.dim() != 2 or x.shape[1] != K:
        raise ValueError(f"x must be [T, {K}], got {tuple(x.shape)}")
    if y.dim() != 2 or y.shape[1] != N:
        raise ValueError(f"y must be [rows >= {T}, {N}], got {tuple(y.shape)}")
    if w0.dtype != x.dtype:
        raise ValueError("x and w must have the same dtype")
    if bias is not None and _first(bias).dtype != y.dtype:
        raise ValueError("bias dtype must equal the output dtype")
    dev = x.device
    wp, wpp, keep_w = _grouped(w, dev, stream)
    bp, bpp, keep_b = _grouped(bias, dev, stream)
    sp, spp, keep_s = _grouped(w_scale, dev, stream)
    _check(load().gl_forward(G, K, N, T, _dtype(x), _dtype(y), _ptr(x), _ptr(x_scale), wp, wpp, sp, spp, bp, bpp,
                             _ptr(y), y.shape[0], _ptr(workspace), _stream(stream)))
    del keep_w, keep_b, keep_s
    return y


def gl_forward_noalloc(m_splits: Tensor, x: Tensor, w: Grouped, y: Tensor, *, bias: Optional[Grouped] = None,
                       x_scale: Optional[Tensor] = None, w_scale: Optional[Grouped] = None, stream=None) -> Tensor:
    """gl_offsets + gl_forward with the library's own fixed device scratch in place of a
    workspace (the C call allocates nothing; the per-group pointer form of ``w`` builds
    its pointer array here, so callers that must not allocate pass stacked tensors).
    At most NOALLOC_MAX_GROUPS groups; calls that overlap on one device race."""
    G = w.shape[0] if isinstance(w, Tensor) else len(w)
    w0 = _first(w)
    N, K = w0.shape[-2], w0.shape[-1]
    T = x.shape[0]
    if m_splits.dtype != torch.int64 or m_splits.numel() != G:
        raise ValueError(f"m_splits must be int64 with {G} entries")
    if x.dim() != 2 or x.shape[1] != K:
        raise ValueError(f"x must be [T, {K}], got {tuple(x.shape)}")
    if y.dim() != 2 or y.shape[1] != N:
        raise ValueError(f"y must be [rows >= {T}, {N}], got {tuple(y.shape)}")
    if w0.dtype != x.dtype:
        raise ValueError("x and w must have the same dtype")
    if bias is not None and _first(bias).dtype != y.dtype:
        raise ValueError("bias dtype must equal the output dtype")
    dev = x.device
    wp, wpp, keep_w = _grouped(w, dev, stream)
    bp, bpp, keep_b = _grouped(bias, dev, stream)
    sp, spp, keep_s = _grouped(w_scale, dev, stream)
    _check(load().gl_forward_noalloc(G, K, N, T, _dtype(x), _dtype(y), _ptr(m_splits), _ptr(x), _ptr(x_scale), wp,
                                     wpp, sp, spp, bp, bpp, _ptr(y), y.shape[0], _stream(stream)))
    del keep_w, keep_b, keep_s
    return y


def gl_dgrad(dy: Tensor, w: Grouped, dx: Tensor, workspace: Tensor, stream=None) -> Tensor:
    """dx[:T] = grouped dy W_g; T = dy.shape[0]; rows of dx past T are left untouched."""
    G = w.shape[0] if isinstance(w, Tensor) else len(w)
    w0 = _first(w)
    N, K = w0.shape[-2], w0.shape[-1]
    T = dy.shape[0]
    if dy.dim() != 2 or dy.shape[1] != N:
        raise ValueError(f"dy must be [T, {N}], got {tuple(dy.shape)}")
    if dx.dim() != 2 or dx.shape[1] != K or dx.dtype != dy.dtype or w0.dtype != dy.dtype:
        raise ValueError("dx must be [rows >= T, K] and dy, w, dx must share one dtype")
    wp, wpp, keep = _grouped(w, dy.device, stream)
    _check(load().gl_dgrad(G, K, N, T, _dtype(dy), _ptr(dy), wp, wpp, _ptr(dx), dx.shape[0], _ptr(workspace),
                           _stream(stream)))
    del keep
    return dx


def gl_wgrad(x: Tensor, dy: Tensor, dw: Grouped, workspace: Tensor, *, accumulate: bool = False,
             stream=None) -> Grouped:
    """dW_g (+)= dy_g^T x_g over each group's rows; dw is [G, N, K] or G tensors [N, K]."""
    G = dw.shape[0] if isinstance(dw, Tensor) else len(dw)
    d0 = _first(dw)
    N, K = d0.shape[-2], d0.shape[-1]
    T = x.shape[0]
    if x.shape != (T, K) or dy.shape != (T, N) or x.dtype != dy.dtype:
        raise ValueError("x must be [T, K] and dy [T, N] with one dtype")
    dp, dpp, keep = _grouped(dw, x.device, stream)
    _check(load().gl_wgrad(G, K, N, T, _dtype(x), _dtype(d0), _ptr(x), _ptr(dy), dp, dpp, int(bool(accumulate)),
                           _ptr(workspace), _stream(stream)))
    del keep
    return dw


def gl_wgrad_bgrad(x: Tensor, dy: Tensor, dw: Grouped, db: Grouped, workspace: Tensor, *, accumulate: bool = False,
                   stream=None):
    """gl_wgrad and the bias gradient of the same dy in one call: db is [G, N] or G
    tensors [N], of dy's dtype or fp32."""
    G = dw.shape[0] if isinstance(dw, Tensor) else len(dw)
    d0 = _first(dw)
    b0 = _first(db)
    N, K = d0.shape[-2], d0.shape[-1]
    T = x.shape[0]
    if x.shape != (T, K) or dy.shape != (T, N) or x.dtype != dy.dtype:
        raise ValueError("x must be [T, K] and dy [T, N] with one dtype")
    if b0.shape[-1] != N or (isinstance(db, Tensor) and db.shape != (G, N)):
        raise ValueError("db must be [G, N] or G tensors [N]")
    dp, dpp, keep = _grouped(dw, x.device, stream)
    bp, bpp, keep_b = _grouped(db, x.device, stream)
    _check(load().gl_wgrad_bgrad(G, K, N, T, _dtype(x), _dtype(d0), _dtype(b0), _ptr(x), _ptr(dy), dp, dpp,
                                 int(bool(accumulate)), bp, bpp, _ptr(workspace), _stream(stream)))
    del keep, keep_b
    return dw, db


def gl_bgrad(dy: Tensor, db: Grouped, workspace: Tensor, stream=None) -> Grouped:
    """db_g = column sums of dy over each group's rows; db is [G, N] or G tensors [N]."""
    G = db.shape[0] if isinstance(db, Tensor) else len(db)
    N = dy.shape[1]
    d0 = db[0] if not isinstance(db, Tensor) else db
    if d0.shape[-1] != N or d0.dtype != dy.dtype:
        raise ValueError("db must have dy's column count and dtype")
    dp, dpp, keep = _grouped(db, dy.device, stream)
    _check(load().gl_bgrad(G, N, dy.shape[0], _dtype(dy), _ptr(dy), dp, dpp, _ptr(workspace), _stream(stream)))
    del keep
    return db


def gl_group_quantize_mxfp8(src: Tensor, data: Tensor, scale: Tensor, stream=None):
    """Rowwise MXFP8 of a bf16 [rows, cols] tensor into uint8 data [rows, cols] and
    uint8 scale [rows, cols/32] (leading dimensions are flattened into rows)."""
    if src.dtype != torch.bfloat16:
        raise ValueError("src must be bfloat16")
    cols = src.shape[-1]
    rows = src.numel() // cols if cols else 0
    if data.numel() != src.numel() or data.dtype != torch.uint8:
        raise ValueError("data must be uint8 with src's element count")
    if scale.numel() != rows * (cols // 32) or scale.dtype != torch.uint8:
        raise ValueError("scale must be uint8 with rows * cols/32 elements")
    _check(load().gl_group_quantize_mxfp8(_ptr(src), rows, cols, _ptr(data), _ptr(scale), _stream(stream)))
    return data, scale


# ------------------------------------------------------------------ MXFP8 backward


def gl_colwise_ld(num_groups: int, total_rows: int) -> int:
    """Row length of the transposed columnwise activation layout that fits any split."""
    return int(load().gl_colwise_ld(int(num_groups), int(total_rows)))


def gl_group_quantize_mxfp8_colwise(src: Tensor, data_t: Tensor, scale_t: Tensor, workspace: Tensor,
                                    num_groups: int, stream=None):
    """Columnwise MXFP8 of bf16 [T, C] per group into data_t [C, ld] / scale_t [C, ld/32]."""
    T, C = src.shape
    ld = data_t.shape[1]
    if src.dtype != torch.bfloat16 or data_t.shape != (C, ld) or scale_t.shape != (C, ld // 32):
        raise ValueError("src must be bf16 [T, C], data_t [C, ld] and scale_t [C, ld/32]")
    _check(load().gl_group_quantize_mxfp8_colwise(_ptr(src), C, int(num_groups), T, _ptr(workspace), _ptr(data_t),
                                                  _ptr(scale_t), ld, _stream(stream)))
    return data_t, scale_t


def gl_group_quantize_mxfp8_rowwise_colwise(src: Tensor, data: Tensor, scale: Tensor, data_t: Tensor,
                                            scale_t: Tensor, workspace: Tensor, num_groups: int, stream=None):
    """Rowwise codes data [T, C] / scale [T, C/32] and per-group columnwise codes
    data_t [C, ld] / scale_t [C, ld/32] of one bf16 tensor [T, C], read once."""
    T, C = src.shape
    ld = data_t.shape[1]
    if src.dtype != torch.bfloat16 or data.shape != (T, C) or scale.shape != (T, C // 32):
        raise ValueError("src must be bf16 [T, C], data [T, C] and scale [T, C/32]")
    if data_t.shape != (C, ld) or scale_t.shape != (C, ld // 32):
        raise ValueError("data_t must be [C, ld] and scale_t [C, ld/32]")
    _check(load().gl_group_quantize_mxfp8_rowwise_colwise(_ptr(src), C, int(num_groups), T, _ptr(workspace),
                                                          _ptr(data), _ptr(scale), _ptr(data_t), _ptr(scale_t), ld,
                                                          _stream(stream)))
    return data, scale, data_t, scale_t


def gl_quantize_mxfp8_colwise_weights(w: Tensor, data_t: Tensor, scale_t: Tensor, stream=None):
    """Columnwise MXFP8 of bf16 weights [G, N, K] into data_t [G, K, N] / scale_t [G, K, N/32]."""
    G, N, K = w.shape
    if w.dtype != torch.bfloat16 or data_t.shape != (G, K, N) or scale_t.shape != (G, K, N // 32):
        raise ValueError("w must be bf16 [G, N, K], data_t [G, K, N] and scale_t [G, K, N/32]")
    _check(load().gl_quantize_mxfp8_colwise_weights(_ptr(w), G, N, K, _ptr(data_t), _ptr(scale_t), _stream(stream)))
    return data_t, scale_t


def gl_offsets_quantize_mxfp8(m_splits: Tensor, x: Tensor, workspace: Tensor, data: Tensor, scale: Tensor,
                              stream=None):
    """One launch: the split-offset scan into ``workspace`` and rowwise MXFP8 of the
    bf16 activations x [T, K] into data [T, K] / scale [T, K/32]."""
    if m_splits.dtype != torch.int64:
        raise ValueError("m_splits must be int64")
    T, K = x.shape
    if x.dtype != torch.bfloat16 or data.shape != (T, K) or scale.shape != (T, K // 32):
        raise ValueError("x must be bf16 [T, K], data [T, K] and scale [T, K/32]")
    _check(load().gl_offsets_quantize_mxfp8(_ptr(m_splits), m_splits.numel(), T, _ptr(workspace), _ptr(x), K,
                                            _ptr(data), _ptr(scale), _stream(stream)))
    return data, scale


def gl_offsets_quantize_mxfp8_rowwise_colwise(m_splits: Tensor, x: Tensor, workspace: Tensor, data: Tensor,
                                              scale: Tensor, data_t: Tensor, scale_t: Tensor, stream=None):
    """The split-offset scan into ``workspace`` and both MXFP8 usages of the bf16
    activations x [T, K]: rowwise data [T, K] / scale [T, K/32] and per-group
    columnwise data_t [K, ld] / scale_t [K, ld/32], x read once."""
    if m_splits.dtype != torch.int64:
        raise ValueError("m_splits must be int64")
    T, K = x.shape
    ld = data_t.shape[1]
    if x.dtype != torch.bfloat16 or data.shape != (T, K) or scale.shape != (T, K // 32):
        raise ValueError("x must be bf16 [T, K], data [T, K] and scale [T, K/32]")
    if data_t.shape != (K, ld) or scale_t.shape != (K, ld // 32):
        raise ValueError("data_t must be [K, ld] and scale_t [K, ld/32]")
    _check(load().gl_offsets_quantize_mxfp8_rowwise_colwise(_ptr(m_splits), m_splits.numel(), T, _ptr(workspace),
                                                            _ptr(x), K, _ptr(data), _ptr(scale), _ptr(data_t),
                                                            _ptr(scale_t), ld, _stream(stream)))
    return data, scale, data_t, scale_t


def gl_quantize_mxfp8_weights(w: Tensor, data: Tensor, scale: Tensor, data_t: Tensor = None, scale_t: Tensor = None,
                              noop_flag: Tensor = None, stream=None):
    """The weights' MXFP8 workspace in one launch: rowwise data [G, N, K] / scale
    [G, N, K/32] and, if given, columnwise data_t [G, K, N] / scale_t [G, K, N/32].
    ``noop_flag`` (device int32, one element): nonzero at run time skips the work."""
    G, N, K = w.shape
    if w.dtype != torch.bfloat16 or data.shape != (G, N, K) or scale.shape != (G, N, K // 32):
        raise ValueError("w must be bf16 [G, N, K], data [G, N, K] and scale [G, N, K/32]")
    if (data_t is None) != (scale_t is None):
        raise ValueError("give both data_t and scale_t, or neither")
    if data_t is not None and (data_t.shape != (G, K, N) or scale_t.shape != (G, K, N // 32)):
        raise ValueError("data_t must be [G, K, N] and scale_t [G, K, N/32]")
    if noop_flag is not None and (noop_flag.dtype != torch.int32 or noop_flag.numel() != 1):
        raise ValueError("noop_flag must be a one-element int32 tensor")
    _check(load().gl_quantize_mxfp8_weights(_ptr(w), G, N, K, _ptr(data), _ptr(scale),
                                            _ptr(data_t) if data_t is not None else None,
                                            _ptr(scale_t) if scale_t is not None else None,
                                            _ptr(noop_flag) if noop_flag is not None else None, _stream(stream)))
    return data, scale


def gl_swiglu_forward(h: Tensor, a: Tensor, stream=None) -> Tensor:
    """a [T, F] = silu(h[:, :F]) * h[:, F:] for h [T, 2F]."""
    T, F2 = h.shape
    if a.shape != (T, F2 // 2) or a.dtype != h.dtype or F2 % 2:
        raise ValueError("h must be [T, 2F] and a [T, F] of h's dtype")
    _check(load().gl_swiglu_forward(T, F2 // 2, _dtype(h), _ptr(h), _ptr(a), _stream(stream)))
    return a


def gl_swiglu_backward(h: Tensor, da: Tensor, dh: Tensor, stream=None) -> Tensor:
    """dh [T, 2F]: the gradient of gl_swiglu_forward at h for the upstream gradient da [T, F]."""
    T, F2 = h.shape
    if da.shape != (T, F2 // 2) or dh.shape != h.shape or not (da.dtype == dh.dtype == h.dtype):
        raise ValueError("h and dh must be [T, 2F] and da [T, F], one dtype")
    _check(load().gl_swiglu_backward(T, F2 // 2, _dtype(h), _ptr(h), _ptr(da), _ptr(dh), _stream(stream)))
    return dh


def gl_grouped_mlp_forward(x: Tensor, w1: Grouped, w2: Grouped, h: Tensor, a: Tensor, y: Tensor, workspace: Tensor,
                           b1: Grouped = None, b2: Grouped = None, stream=None) -> Tensor:
    """y[:T] = FC2(SwiGLU(FC1(x))) per group; h [T, 2F] and a [T, F] receive the
    intermediates (kept for the backward); y may have more rows than T."""
    G = w1.shape[0] if isinstance(w1, Tensor) else len(w1)
    F2, K = _first(w1).shape[-2:]
    N = _first(w2).shape[-2]
    T = x.shape[0]
    if x.shape != (T, K) or h.shape != (T, F2) or a.shape != (T, F2 // 2) or y.dim() != 2 or y.shape[1] != N:
        raise ValueError("shapes: x [T, K], w1 [G, 2F, K], w2 [G, N, F], h [T, 2F], a [T, F], y [rows >= T, N]")
    p1, pp1, k1 = _grouped(w1, x.device, stream)
    p2, pp2, k2 = _grouped(w2, x.device, stream)
    q1, qq1, k3 = _grouped(b1, x.device, stream)
    q2, qq2, k4 = _grouped(b2, x.device, stream)
    _check(load().gl_grouped_mlp_forward(G, K, F2 // 2, N, T, _dtype(x), _ptr(x), p1, pp1, q1, qq1, p2, pp2, q2, qq2,
                                         _ptr(h), _ptr(a), _ptr(y), y.shape[0], _ptr(workspace), _stream(stream)))
    del k1, k2, k3, k4
    return y


def gl_grouped_mlp_backward(x: Tensor, w1: Grouped, w2: Grouped, h: Tensor, a: Tensor, dy: Tensor, da: Tensor,
                            dh: Tensor, dx: Tensor, dw1: Grouped, dw2: Grouped, workspace: Tensor,
                            db1: Grouped = None, db2: Grouped = None, *, accumulate: bool = False, stream=None):
    """Backward of gl_grouped_mlp_forward: dx[:T], dW1, dW2 (of dw1's dtype: the
    input's or fp32, added into them with ``accumulate``), optional db1, db2; da
    [T, F] and dh [T, 2F] are scratch."""
    G = w1.shape[0] if isinstance(w1, Tensor) else len(w1)
    F2, K = _first(w1).shape[-2:]
    N = _first(w2).shape[-2]
    T = x.shape[0]
    if dy.shape != (T, N) or da.shape != (T, F2 // 2) or dh.shape != (T, F2) or dx.dim() != 2 or dx.shape[1] != K:
        raise ValueError("shapes: dy [T, N], da [T, F], dh [T, 2F], dx [rows >= T, K]")
    keep = []
    ptr = {}
    for name, g in (("w1", w1), ("w2", w2), ("dw1", dw1), ("dw2", dw2), ("db1", db1), ("db2", db2)):
        p, pp, k = _grouped(g, x.device, stream)
        ptr[name] = (p, pp)
        keep.append(k)
    _check(load().gl_grouped_mlp_backward(G, K, F2 // 2, N, T, _dtype(x), _dtype(_first(dw1)), _ptr(x), *ptr["w1"],
                                          *ptr["w2"], _ptr(h), _ptr(a), _ptr(dy), _ptr(da), _ptr(dh), _ptr(dx),
                                          dx.shape[0], *ptr["dw1"], *ptr["db1"], *ptr["dw2"], *ptr["db2"],
                                          int(bool(accumulate)), _ptr(workspace), _stream(stream)))
    del keep
    return dx


def gl_dgrad_mxfp8(dy: Tensor, dy_scale: Tensor, w_t: Tensor, w_t_scale: Tensor, dx: Tensor, workspace: Tensor,
                   stream=None) -> Tensor:
    """dx[:T] = grouped deq(dy) deq(W_g) from rowwise dy codes and columnwise weight codes [G, K, N]."""
    G, K, N = w_t.shape
    T = dy.shape[0]
    if dy.shape != (T, N) or dx.dim() != 2 or dx.shape[1] != K:
        raise ValueError("dy must be [T, N] codes and dx [rows >= T, K]")
    _check(load().gl_dgrad_mxfp8(G, K, N, T, _dtype(dx), _ptr(dy), _ptr(dy_scale), _ptr(w_t), _ptr(w_t_scale),
                                 _ptr(dx), dx.shape[0], _ptr(workspace), _stream(stream)))
    return dx


def gl_wgrad_mxfp8(dy_t: Tensor, dy_t_scale: Tensor, x_t: Tensor, x_t_scale: Tensor, dw: Grouped,
                   workspace: Tensor, total_rows: int, *, accumulate: bool = False, stream=None) -> Grouped:
    """dW_g (+)= deq(dy_g)^T deq(x_g) from columnwise codes dy_t [N, ld] and x_t [K, ld]."""
    G = dw.shape[0] if isinstance(dw, Tensor) else len(dw)
    d0 = _first(dw)
    N, ld = dy_t.shape
    K = x_t.shape[0]
    if x_t.shape != (K, ld) or tuple(d0.shape[-2:]) != (N, K):
        raise ValueError("x_t must be [K, ld] and dw [G, N, K] or G tensors [N, K]")
    dp, dpp, keep = _grouped(dw, dy_t.device, stream)
    _check(load().gl_wgrad_mxfp8(G, K, N, int(total_rows), _dtype(d0), _ptr(dy_t), _ptr(dy_t_scale), _ptr(x_t),
                                 _ptr(x_t_scale), ld, dp, dpp, int(bool(accumulate)), _ptr(workspace),
                                 _stream(stream)))
    del keep
    return dw


# -------------------------------------------------------------------- expert block


def _addresses(first: Tensor, *others: Optional[Tensor]):
    """Addresses of ``first`` and of the others (None for None), which must be contiguous and
    on ``first``'s GPU."""
    dev = first.get_device()
    if dev < 0:
        raise ValueError("tensors must be on the GPU")
    out = []
    for t in (first, *others):
        if t is None:
            out.append(None)
            continue
        if t.get_device() != dev:
            raise ValueError(f"tensors must be on one device (got {first.device} and {t.device})")
        if not t.is_contiguous():
            raise ValueError("tensors passed to the library must be contiguous")
        out.append(t.data_ptr())
    return out


def _enough(workspace: Optional[Tensor], size: int) -> None:
    if workspace is None or workspace.numel() * workspace.element_size() < size:
        raise ValueError(f"workspace must hold {size} bytes")


def gl_rmsnorm_forward(x: Tensor, gamma: Tensor, eps: float, *, residual: Optional[Tensor] = None,
                       h: Optional[Tensor] = None, y: Optional[Tensor] = None, data: Optional[Tensor] = None,
                       scale: Optional[Tensor] = None, stream=None) -> None:
    """RMS norm of s = x (+ residual), [T, C]: h = s, y = s rstd gamma, and / or the MXFP8
    codes of y, data [T, C] / scale [T, C/32].  gamma [C] is fp32 or of x's dtype; h may be
    ``x`` or ``residual`` itself."""
    if x.dim() != 2 or gamma.shape != (x.shape[1],):
        raise ValueError("x must be [T, C] and gamma [C]")
    T, C = x.shape
    for t in (residual, h, y):
        if t is not None and (t.shape != x.shape or t.dtype != x.dtype):
            raise ValueError("residual, h and y must have x's shape and dtype")
    if data is not None and (data.shape != x.shape or data.dtype != torch.uint8):
        raise ValueError("data must be uint8 [T, C]")
    if scale is not None and (scale.shape != (T, C // 32) or scale.dtype != torch.uint8):
        raise ValueError("scale must be uint8 [T, C/32]")
    px, pr, pg, ph, py, pd, ps = _addresses(x, residual, gamma, h, y, data, scale)
    _check(load().gl_rmsnorm_forward(T, C, _dtype(x), _dtype(gamma), px, pr, pg, eps, ph, py, pd, ps, _stream(stream)))


def gl_rmsnorm_workspace_size(total_rows: int, features: int) -> int:
    """Bytes of the workspace gl_rmsnorm_backward needs for dgamma."""
    return int(load().gl_rmsnorm_workspace_size(int(total_rows), int(features)))


def gl_rmsnorm_backward(dy: Tensor, h: Tensor, gamma: Tensor, eps: float, dx: Tensor, *,
                        dh: Optional[Tensor] = None, dgamma: Optional[Tensor] = None, accumulate: bool = False,
                        workspace: Optional[Tensor] = None, stream=None) -> Tensor:
    """Gradient of the norm at h, [T, C]: dx (of x and of the residual alike, with dh, the
    gradient arriving at h, added) and dgamma [C] (fp32 or of h's dtype; added into with
    ``accumulate``), which needs ``workspace``."""
    if h.dim() != 2 or gamma.shape != (h.shape[1],):
        raise ValueError("h must be [T, C] and gamma [C]")
    T, C = h.shape
    for t in (dy, dx, dh):
        if t is not None and (t.shape != h.shape or t.dtype != h.dtype):
            raise ValueError("dy, dx and dh must have h's shape and dtype")
    if dgamma is not None:
        if dgamma.shape != (C,):
            raise ValueError("dgamma must be [C]")
        _enough(workspace, gl_rmsnorm_workspace_size(T, C))
    ph, py, pd, pg, px, pw, ws = _addresses(h, dy, dh, gamma, dx, dgamma, workspace)
    _check(load().gl_rmsnorm_backward(T, C, _dtype(h), _dtype(gamma), py, pd, ph, pg, eps, px,
                                      GL_F32 if dgamma is None else _dtype(dgamma), pw, int(bool(accumulate)), ws,
                                      _stream(stream)))
    return dx



def _route_args(logits: Tensor, ids: Tensor, weights: Tensor):
    if logits.dim() != 2 or ids.dim() != 2 or ids.shape[0] != logits.shape[0] or weights.shape != ids.shape:
        raise ValueError("logits must be [T, E], ids and the weights [T, top_k]")
    if ids.dtype != torch.int32 or weights.dtype != torch.float32:
        raise ValueError("ids must be int32 and the weights float32")
    return logits.shape[0], logits.shape[1], ids.shape[1]


def gl_route_workspace_size(total_rows: int, num_experts: int) -> int:
    """Bytes of the workspace a routing plan needs."""
    return int(load().gl_route_workspace_size(int(total_rows), int(num_experts)))


def gl_route_forward(logits: Tensor, ids: Tensor, weights: Tensor, *, score: int = GL_SCORE_SOFTMAX,
                     renormalize: bool = True, m_splits: Optional[Tensor] = None, row_index: Optional[Tensor] = None,
                     slot_index: Optional[Tensor] = None, workspace: Optional[Tensor] = None, stream=None):
    """The top_k experts of each token, ids int32 [T, top_k], and their weights (float32)
    from logits [T, E]; with m_splits (int64 [E]), row_index (int32 [T, top_k]) and
    slot_index (int32 [T * top_k]) also the plan that orders the slots by expert."""
    T, E, k = _route_args(logits, ids, weights)
    if (m_splits is None) != (row_index is None) or (m_splits is None) != (slot_index is None):
        raise ValueError("give m_splits, row_index and slot_index, or none of them")
    if m_splits is not None:
        if m_splits.shape != (E,) or m_splits.dtype != torch.int64:
            raise ValueError("m_splits must be int64 [E]")
        if row_index.shape != (T, k) or slot_index.shape != (T * k,):
            raise ValueError("row_index must be [T, top_k] and slot_index [T * top_k]")
        if row_index.dtype != torch.int32 or slot_index.dtype != torch.int32:
            raise ValueError("row_index and slot_index must be int32")
        _enough(workspace, gl_route_workspace_size(T, E))
    at = _addresses(logits, ids, weights, m_splits, row_index, slot_index, workspace)
    _check(load().gl_route_forward(T, E, k, _dtype(logits), int(score), int(bool(renormalize)), *at, _stream(stream)))
    return ids, weights


def gl_route_backward(logits: Tensor, ids: Tensor, dweights: Tensor, dlogits: Tensor, *,
                      score: int = GL_SCORE_SOFTMAX, renormalize: bool = True, stream=None) -> Tensor:
    """dlogits [T, E]: the gradient of gl_route_forward's weights at its logits and ids."""
    T, E, k = _route_args(logits, ids, dweights)
    if dlogits.shape != logits.shape or dlogits.dtype != logits.dtype:
        raise ValueError("dlogits must have the shape and dtype of logits")
    at = _addresses(logits, ids, dweights, dlogits)
    _check(load().gl_route_backward(T, E, k, _dtype(logits), int(score), int(bool(renormalize)), *at, _stream(stream)))
    return dlogits


def gl_moe_few_tokens_workspace_size(total_rows: int, top_k: int, num_experts: int, ffn_features: int) -> int:
    """Bytes of the workspace gl_moe_few_tokens needs."""
    return int(load().gl_moe_few_tokens_workspace_size(int(total_rows), int(top_k), int(num_experts),
                                                       int(ffn_features)))


def _each_shape(g: Optional[Grouped], G: int, shape, dtype, what: str) -> None:
    """Checks a stacked tensor [G, *shape] or a list of G tensors of that shape."""
    if g is None:
        return
    if isinstance(g, Tensor):
        good = tuple(g.shape) == (G, *shape) and g.dtype == dtype
    else:
        good = len(g) == G and all(tuple(t.shape) == tuple(shape) and t.dtype == dtype for t in g)
    if not good:
        raise ValueError(f"{what} must be [{G}, {', '.join(map(str, shape))}] or {G} tensors, of {dtype}")


def gl_moe_few_tokens(x: Tensor, ids: Tensor, weights: Tensor, w1: Grouped, w2: Grouped, y: Tensor,
                      workspace: Tensor, *, w1_scale: Optional[Grouped] = None, w2_scale: Optional[Grouped] = None,
                      b1: Optional[Grouped] = None, b2: Optional[Grouped] = None,
                      residual: Optional[Tensor] = None, stream=None) -> Tensor:
    """y[t] = residual[t] + sum_j weights[t, j] (W2_e SwiGLU(W1_e x[t] + b1_e) + b2_e) with
    e = ids[t, j], for at most MOE_MAX_TOKENS tokens; slots whose id is outside
    [0, E) take no part.

    x: [T, K]; w1: [E, 2F, K], w2: [E, N, F] stacked or per expert, of x's dtype, or uint8
    E4M3 codes with ``w1_scale`` [E, 2F, K/32] / ``w2_scale`` [E, N, F/32] and bf16 x."""
    E = w1.shape[0] if isinstance(w1, Tensor) else len(w1)
    F2, K = _first(w1).shape[-2:]
    N, F = _first(w2).shape[-2:]
    T, k = ids.shape
    if x.shape != (T, K) or F2 != 2 * F or y.dim() != 2 or y.shape[1] != N:
        raise ValueError("shapes: x [T, K], ids [T, top_k], w1 [E, 2F, K], w2 [E, N, F], y [rows >= T, N]")
    if weights.shape != ids.shape or ids.dtype != torch.int32 or weights.dtype != torch.float32:
        raise ValueError("ids must be int32 and weights float32, both [T, top_k]")
    if y.dtype != x.dtype or (residual is not None and (residual.shape != (T, N) or residual.dtype != x.dtype)):
        raise ValueError("y and residual [T, N] must have x's dtype")
    wd = _first(w1).dtype
    _each_shape(w1, E, (F2, K), wd, "w1")
    _each_shape(w2, E, (N, F), wd, "w2")
    _each_shape(w1_scale, E, (F2, K // 32), torch.uint8, "w1_scale")
    _each_shape(w2_scale, E, (N, F // 32), torch.uint8, "w2_scale")
    _each_shape(b1, E, (F2,), x.dtype, "b1")
    _each_shape(b2, E, (N,), x.dtype, "b2")
    _enough(workspace, gl_moe_few_tokens_workspace_size(T, k, E, F))
    px, pi, pw, pr, py, ws = _addresses(x, ids, weights, residual, y, workspace)
    for g, what, align in ((w1, "w1", 16), (w2, "w2", 16), (w1_scale, "w1_scale", 4), (w2_scale, "w2_scale", 4),
                           (b1, "b1", 1), (b2, "b2", 1)):
        if g is not None:
            at = _addresses(x, *((g,) if isinstance(g, Tensor) else g))[1:]
            if not isinstance(g, Tensor) and any(a % align for a in at):  # the library sees only their array
                raise ValueError(f"every expert's {what} must be {align}-byte aligned")
    p1, pp1, k1 = _grouped(w1, x.device, stream)
    p2, pp2, k2 = _grouped(w2, x.device, stream)
    s1, ss1, k3 = _grouped(w1_scale, x.device, stream)
    s2, ss2, k4 = _grouped(w2_scale, x.device, stream)
    q1, qq1, k5 = _grouped(b1, x.device, stream)
    q2, qq2, k6 = _grouped(b2, x.device, stream)
    _check(load().gl_moe_few_tokens(E, K, F, N, T, k, _dtype(x), _DT[wd] if wd in _DT else -1, px, pi, pw, p1, pp1,
                                    s1, ss1, q1, qq1, p2, pp2, s2, ss2, q2, qq2, pr, py, y.shape[0], ws,
                                    _stream(stream)))
    del k1, k2, k3, k4, k5, k6
    return y


# ------------------------------------------------- gated layer, 8-bit integers
#
# (These are called for single tokens too, where the checks below are most of a call: a stacked tensor
# is looked at once, and nothing is sliced.)


def _here(t: Tensor) -> int:
    """The GPU that ``t`` is on, which has to be the current one: the launch goes there."""
    dev = t.get_device()
    if dev < 0:
        raise ValueError("tensors must be on the GPU")
    if dev != torch._C._cuda_getDevice():
        raise ValueError(f"tensors are on {t.device}, which is not the current device")
    return dev


def _at(dev: int, t: Optional[Tensor]) -> Optional[int]:
    """Address of a contiguous tensor on GPU ``dev``, None for None."""
    if t is None:
        return None
    if t.get_device() != dev:
        raise ValueError(f"tensors must be on one device (cuda:{dev} and {t.device})")
    if not t.is_contiguous():
        raise ValueError("tensors passed to the library must be contiguous")
    return t.data_ptr()


def _group_at(dev: int, g: Optional[Grouped], shape, dtype, what: str, stream, keep: list):
    """(address, pointer array) of a stacked tensor of ``shape`` or a list of shape[0] tensors of
    shape[1:], 16-byte aligned each (scales: 4); the pointer array goes into ``keep``."""
    if g is None:
        return None, None
    if isinstance(g, Tensor):
        if g.shape != shape or g.dtype != dtype:
            raise ValueError(f"{what} must be {list(shape)} or {shape[0]} tensors {list(shape[1:])}, of {dtype}")
        return _at(dev, g), None
    if len(g) != shape[0] or any(t.shape != shape[1:] or t.dtype != dtype for t in g):
        raise ValueError(f"{what} must be {list(shape)} or {shape[0]} tensors {list(shape[1:])}, of {dtype}")
    each = [_at(dev, t) for t in g]
    align = 4 if what == "w_scale" else 16
    if any(a % align for a in each):  # the library sees only their array
        raise ValueError(f"every group's {what} must be {align}-byte aligned")
    ptrs = torch.tensor(each, dtype=torch.int64, device=f"cuda:{dev}")
    _record([ptrs], stream)
    keep.append((ptrs, list(g)))
    return None, ptrs.data_ptr()


@functools.lru_cache(maxsize=None)
def _workspace_bytes(num_groups: int) -> int:
    return gl_workspace_size(num_groups)


def _glu_sizes(x: Tensor, w: Grouped, workspace: Tensor, gated: bool):
    """(T, G, K, N, F) of x [T, K] and w [G, N, K] or G tensors [N, K]."""
    ws = w.shape if isinstance(w, Tensor) else (len(w), *(w[0].shape if len(w) else ()))
    if x.dim() != 2 or len(ws) != 3:
        raise ValueError("x must be [T, K] and w [G, N, K] or G tensors [N, K]")
    G, N, K = ws
    T, k = x.shape
    if k != K or (gated and N % 2):
        raise ValueError(f"x must be [T, {K}], and w have an even number of rows where they are gated")
    if workspace.numel() * workspace.element_size() < _workspace_bytes(G):
        raise ValueError(f"workspace must hold {_workspace_bytes(G)} bytes")
    return T, G, K, N, N // 2 if gated else N


def _matrix(t: Optional[Tensor], rows: int, cols: int, dtype, what: str, more: bool = False) -> None:
    """Checks a tensor [rows, cols] (``more``: or of more rows), None passes."""
    if t is None:
        return
    s = t.shape
    if len(s) != 2 or s[1] != cols or (s[0] < rows if more else s[0] != rows) or t.dtype != dtype:
        raise ValueError(f"{what} must be [{'rows >= ' if more else ''}{rows}, {cols}] of {dtype}")


def gl_glu_forward(x: Tensor, w: Grouped, a: Tensor, workspace: Tensor, *, bias: Optional[Grouped] = None,
                   h: Optional[Tensor] = None, act: int = GL_GLU_SILU, stream=None) -> Tensor:
    """a[:T] = act(h[:, :F]) * h[:, F:] with h = grouped x W_g^T (+ b_g), in one launch.

    x: [T, K]; w: [G, 2F, K] or G tensors [2F, K], the gate's rows first; bias [G, 2F] or G
    tensors [2F]; a: [>= T, F], rows past T are left untouched; h: [T, 2F] to keep for
    ``gl_glu_backward``, or None.  One dtype (float32, bfloat16, float16)."""
    T, G, K, N, F = _glu_sizes(x, w, workspace, True)
    dt = x.dtype
    _matrix(a, T, F, dt, "a", more=True)
    _matrix(h, T, N, dt, "h")
    dev, keep = _here(x), []
    pw, pww = _group_at(dev, w, (G, N, K), dt, "w", stream, keep)
    pb, pbb = _group_at(dev, bias, (G, N), dt, "bias", stream, keep)
    _check(load().gl_glu_forward(G, K, F, T, _dtype(x), int(act), _at(dev, x), pw, pww, pb, pbb, _at(dev, h), _at(dev, a),
                                 a.shape[0], _at(dev, workspace), _stream(stream)))
    del keep
    return a


def gl_glu_backward(x: Tensor, w: Grouped, da: Tensor, dh: Tensor, dx: Optional[Tensor], dw: Grouped,
                    workspace: Tensor, *, h: Optional[Tensor] = None, bias: Optional[Grouped] = None,
                    a: Optional[Tensor] = None, db: Optional[Grouped] = None, act: int = GL_GLU_SILU,
                    accumulate: bool = False, stream=None) -> Optional[Tensor]:
    """Backward of gl_glu_forward for the gradient da [T, F] of a: dh [T, 2F] (the gradient of
    h, a caller's buffer; may be h), dx[:T] (or None), dw (of x's dtype or float32, added into
    with ``accumulate``) and db (of x's dtype).  ``h`` as the forward kept it, or None: computed
    again from x, w and ``bias``.  ``a`` [T, F] receives the forward's output again."""
    T, G, K, N, F = _glu_sizes(x, w, workspace, True)
    dt = x.dtype
    _matrix(da, T, F, dt, "da")
    _matrix(dh, T, N, dt, "dh")
    _matrix(h, T, N, dt, "h")
    _matrix(a, T, F, dt, "a")
    _matrix(dx, T, K, dt, "dx", more=True)
    if not isinstance(dw, Tensor) and len(dw) != G:
        raise ValueError(f"dw must be a tensor or a list of {G}")
    wd = (dw if isinstance(dw, Tensor) else dw[0]).dtype
    if wd not in _DT:
        raise ValueError(f"unsupported dtype {wd}")
    dev, keep = _here(x), []
    pw, pww = _group_at(dev, w, (G, N, K), dt, "w", stream, keep)
    pb, pbb = _group_at(dev, bias, (G, N), dt, "bias", stream, keep)
    pdw, pdww = _group_at(dev, dw, (G, N, K), wd, "dw", stream, keep)
    pdb, pdbb = _group_at(dev, db, (G, N), dt, "db", stream, keep)
    _check(load().gl_glu_backward(G, K, F, T, _dtype(x), _DT[wd], int(act), _at(dev, x), pw, pww, pb, pbb, _at(dev, h),
                                  _at(dev, da), _at(dev, dh), _at(dev, a), _at(dev, dx), 0 if dx is None else dx.shape[0],
                                  pdw, pdww, pdb, pdbb, int(bool(accumulate)), _at(dev, workspace), _stream(stream)))
    del keep
    return dx


def gl_quantize_int8(src: Tensor, data: Tensor, scale: Tensor, stream=None):
    """Rows of src [..., cols] as int8 codes data (src's shape) and float32 scale [...]: a
    token's activations, or with weights [G, N, K] a channel's."""
    s = src.shape
    if len(s) < 1 or data.shape != s or data.dtype != torch.int8:
        raise ValueError("data must be int8 of src's shape")
    if scale.shape != s[:-1] or scale.dtype != torch.float32:
        raise ValueError("scale must be float32 with one value for each row of src")
    cols, dev = s[-1], _here(src)
    _check(load().gl_quantize_int8(src.numel() // cols if cols else 0, cols, _dtype(src), _at(dev, src), _at(dev, data),
                                   _at(dev, scale), _stream(stream)))
    return data, scale


def _int8(name: str, gated: bool, x, x_scale, w, w_scale, y, workspace, bias, act, stream) -> Tensor:
    T, G, K, N, F = _glu_sizes(x, w, workspace, gated)
    if x.dtype != torch.int8 or x_scale.shape != (T,) or x_scale.dtype != torch.float32:
        raise ValueError("x must be int8 [T, K] and x_scale float32 [T]")
    if isinstance(w, Tensor) != isinstance(w_scale, Tensor):
        raise ValueError("w and w_scale must both be stacked or both be lists")
    _matrix(y, T, F, y.dtype, "the output", more=True)
    dev, keep = _here(x), []
    pw, pww = _group_at(dev, w, (G, N, K), torch.int8, "w", stream, keep)
    pc, pcc = _group_at(dev, w_scale, (G, N), torch.float32, "w_scale", stream, keep)
    pb, pbb = _group_at(dev, bias, (G, N), y.dtype, "bias", stream, keep)
    _check(getattr(load(), name)(G, K, F, T, _dtype(y), *((int(act),) if gated else ()), _at(dev, x), _at(dev, x_scale), pw,
                                 pww, pc, pcc, pb, pbb, _at(dev, y), y.shape[0], _at(dev, workspace), _stream(stream)))
    del keep
    return y


def gl_forward_int8(x: Tensor, x_scale: Tensor, w: Grouped, w_scale: Grouped, y: Tensor, workspace: Tensor, *,
                    bias: Optional[Grouped] = None, stream=None) -> Tensor:
    """y[:T] = grouped (x W_g^T) x_scale[t] w_scale_g[n] (+ b_g) from int8 x [T, K] and w
    [G, N, K] (or G tensors [N, K]) with float32 scales x_scale [T] and w_scale [G, N] (or G
    tensors [N]); y [>= T, N] is float32, bfloat16 or float16, the bias of its dtype."""
    return _int8("gl_forward_int8", False, x, x_scale, w, w_scale, y, workspace, bias, 0, stream)


def gl_glu_forward_int8(x: Tensor, x_scale: Tensor, w: Grouped, w_scale: Grouped, a: Tensor, workspace: Tensor, *,
                        bias: Optional[Grouped] = None, act: int = GL_GLU_SILU, stream=None) -> Tensor:
    """gl_glu_forward from int8 x and w (w [G, 2F, K], the gate's rows first) with the scales
    of gl_forward_int8; a [>= T, F] is float32, bfloat16 or float16."""
    return _int8("gl_glu_forward_int8", True, x, x_scale, w, w_scale, a, workspace, bias, act, stream)


def _tensors(obj):
    """Every tensor inside nested tuples / lists."""
    if isinstance(obj, Tensor):
        yield obj
    elif isinstance(obj, (tuple, list)):
        for o in obj:
            yield from _tensors(o)


class WgradQueue:
    """Deferred grouped weight gradients (the ``gl_wgrad_queue_*`` entry points).

    ``put`` / ``put_mxfp8`` take the arguments of ``gl_wgrad_bgrad`` (``db=None``:
    plain ``gl_wgrad``) / ``gl_wgrad_mxfp8``, check them in full and record the
    call without running it; ``run_next`` launches the oldest recorded call and
    ``flush`` all of them, in put order.  The queue holds a reference to every
    tensor of a recorded call until it has been launched, and ties their memory
    to the stream it runs on; the workspace must still hold the same splits' offsets.
    """

    def __init__(self):
        self._q = ctypes.c_void_p()
        _check(load().gl_wgrad_queue_create(ctypes.byref(self._q)))
        self._held = collections.deque()

    def __len__(self) -> int:
        n = load().gl_wgrad_queue_size(self._q)
        if n < 0:
            _check(n)
        return n

    def put(self, x: Tensor, dy: Tensor, dw: Grouped, workspace: Tensor, *, db: Optional[Grouped] = None,
            accumulate: bool = False) -> None:
        G = dw.shape[0] if isinstance(dw, Tensor) else len(dw)
        d0 = _first(dw)
        N, K = d0.shape[-2], d0.shape[-1]
        T = x.shape[0]
        if x.shape != (T, K) or dy.shape != (T, N) or x.dtype != dy.dtype:
            raise ValueError("x must be [T, K] and dy [T, N] with one dtype")
        db_dtype = GL_F32
        if db is not None:
            b0 = _first(db)
            if b0.shape[-1] != N or (isinstance(db, Tensor) and db.shape != (G, N)):
                raise ValueError("db must be [G, N] or G tensors [N]")
            db_dtype = _dtype(b0)
        dp, dpp, keep = _grouped(dw, x.device)
        bp, bpp, keep_b = _grouped(db, x.device)
        _check(load().gl_wgrad_queue_put(self._q, G, K, N, T, _dtype(x), _dtype(d0), db_dtype, _ptr(x), _ptr(dy), dp,
                                         dpp, int(bool(accumulate)), bp, bpp, _ptr(workspace)))
        self._held.append((x, dy, dw, db, workspace, keep, keep_b))

    def put_mxfp8(self, dy_t: Tensor, dy_t_scale: Tensor, x_t: Tensor, x_t_scale: Tensor, dw: Grouped,
                  workspace: Tensor, total_rows: int, *, accumulate: bool = False) -> None:
        G = dw.shape[0] if isinstance(dw, Tensor) else len(dw)
        d0 = _first(dw)
        N, ld = dy_t.shape
        K = x_t.shape[0]
        if x_t.shape != (K, ld) or tuple(d0.shape[-2:]) != (N, K):
            raise ValueError("x_t must be [K, ld] and dw [G, N, K] or G tensors [N, K]")
        dp, dpp, keep = _grouped(dw, dy_t.device)
        _check(load().gl_wgrad_queue_put_mxfp8(self._q, G, K, N, int(total_rows), _dtype(d0), _ptr(dy_t),
                                               _ptr(dy_t_scale), _ptr(x_t), _ptr(x_t_scale), ld, dp, dpp,
                                               int(bool(accumulate)), _ptr(workspace)))
        self._held.append((dy_t, dy_t_scale, x_t, x_t_scale, dw, workspace, keep))

    def _launching(self, held, stream):
        _record(list(_tensors(held)), torch.cuda.current_stream() if stream is None else stream)

    def run_next(self, stream=None) -> None:
        """Launch the oldest recorded call on ``stream`` (torch's current one by default)."""
        if not self._held:
            return
        self._launching(self._held.popleft(), stream)
        _check(load().gl_wgrad_queue_run_next(self._q, _stream(stream)))

    def flush(self, stream=None) -> None:
        """Launch every recorded call, in put order."""
        held, self._held = list(self._held), collections.deque()
        for h in held:
            self._launching(h, stream)
        _check(load().gl_wgrad_queue_flush(self._q, _stream(stream)))

    def clear(self) -> None:
        """Drop the recorded calls without running them."""
        _check(load().gl_wgrad_queue_clear(self._q))
        self._held.clear()

    def close(self) -> None:
        if self._q:
            load().gl_wgrad_queue_destroy(self._q)
            self._q = ctypes.c_void_p()
        self._held.clear()

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
