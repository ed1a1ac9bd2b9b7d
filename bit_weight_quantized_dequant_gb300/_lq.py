"""ctypes binding of the liblq C ABI (include/lq.h).

Tensors are PyTorch CUDA tensors; only their device pointers, the current CUDA
stream and plain sizes cross the boundary.
"""
from __future__ import annotations

import ctypes
import functools
from dataclasses import dataclass
from pathlib import Path

LQ_OK, LQ_ERR_INVALID_ARG, LQ_ERR_UNSUPPORTED, LQ_ERR_ALIGNMENT, LQ_ERR_WORKSPACE, LQ_ERR_CUDA, LQ_ERR_TIMEOUT, \
    LQ_ERR_RANGE, LQ_ERR_INDEX = range(9)
FMT_2BIT, FMT_NF4, FMT_INT4, FMT_NF4_DQ = 1, 2, 3, 4
F32, F16, BF16 = 0, 1, 2
ROPE_HALF, ROPE_INTERLEAVED = 0, 1
_INT_MAX = 0x7fffffff       # (larger numbers would lose their upper bits at the C boundary)

#: every entry point include/lq.h declares
EXPORTED = ("lq_create", "lq_destroy", "lq_status_string", "lq_sync", "lq_dequant", "lq_gemv",
            "lq_anchor_count",
            "lq_gemv_grouped", "lq_gemv_layers", "lq_gemm", "lq_gemm_grouped", "lq_gemv_noalloc",
            "lq_select_anchors", "lq_quantize_2bit", "lq_quantize_nf4",
            "lq_stream_create", "lq_stream_run", "lq_stream_destroy", "lq_stream_run_direct",
            "lq_rope_table", "lq_rope", "lq_kv_tile_bytes", "lq_kv_append", "lq_kv_read", "lq_kv_attention",
            "lq_kv_attention_window", "lq_kv_attention_chunk", "lq_logprobs", "lq_logprobs_grad", "lq_selftest_wait")

_LIB = None


class LQError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        msg = _LIB.lq_status_string(status).decode() if _LIB is not None else str(status)
        super().__init__(f"{where}: {msg} (status {status})")


class lq_problem(ctypes.Structure):
    _fields_ = [
        ("format", ctypes.c_int), ("M", ctypes.c_int), ("N", ctypes.c_int), ("K", ctypes.c_int),
        ("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("offsets", ctypes.c_void_p),
        ("anchor_idx", ctypes.c_void_p), ("anchor_w", ctypes.c_void_p),
        ("A", ctypes.c_int), ("ld_anchor", ctypes.c_int),
        ("x", ctypes.c_void_p), ("x_dtype", ctypes.c_int), ("y", ctypes.c_void_p), ("y_dtype", ctypes.c_int),
        ("batch", ctypes.c_int),
        ("stride_codes", ctypes.c_int64), ("stride_scales", ctypes.c_int64), ("stride_offsets", ctypes.c_int64),
        ("stride_anchor_idx", ctypes.c_int64), ("stride_anchor_w", ctypes.c_int64),
        ("stride_x", ctypes.c_int64), ("stride_y", ctypes.c_int64),
    ]


class lq_rope_config(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int), ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("original_length", ctypes.c_double), ("low_rotations", ctypes.c_double),
                ("high_rotations", ctypes.c_double), ("mscale", ctypes.c_float)]


class lq_rope_args(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("y", ctypes.c_void_p), ("dtype", ctypes.c_int), ("n", ctypes.c_int),
                ("heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("rot_dim", ctypes.c_int),
                ("x_token_stride", ctypes.c_int64), ("x_head_stride", ctypes.c_int64),
                ("y_token_stride", ctypes.c_int64), ("y_head_stride", ctypes.c_int64), ("table", ctypes.c_void_p),
                ("table_rows", ctypes.c_int), ("positions", ctypes.c_void_p), ("layout", ctypes.c_int),
                ("inverse", ctypes.c_int)]


class lq_kv_cache(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("page_size", ctypes.c_int),
                ("kv_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("bits", ctypes.c_int)]


class lq_kv_append_args(ctypes.Structure):
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("q", ctypes.c_void_p), ("q_out", ctypes.c_void_p),
                ("dtype", ctypes.c_int), ("n", ctypes.c_int), ("q_heads", ctypes.c_int),
                ("k_token_stride", ctypes.c_int64), ("v_token_stride", ctypes.c_int64),
                ("q_token_stride", ctypes.c_int64), ("q_out_token_stride", ctypes.c_int64), ("slots", ctypes.c_void_p),
                ("table", ctypes.c_void_p), ("table_rows", ctypes.c_int), ("positions", ctypes.c_void_p),
                ("rot_dim", ctypes.c_int), ("layout", ctypes.c_int)]


class lq_kv_attention_args(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("dtype", ctypes.c_int),
                ("batch", ctypes.c_int), ("tokens", ctypes.c_int), ("q_heads", ctypes.c_int),
                ("q_token_stride", ctypes.c_int64), ("out_token_stride", ctypes.c_int64),
                ("block_table", ctypes.c_void_p), ("block_table_stride", ctypes.c_int64), ("max_pages", ctypes.c_int),
                ("lens", ctypes.c_void_p), ("prefix_table", ctypes.c_void_p), ("prefix_len", ctypes.c_int),
                ("scale", ctypes.c_float)]


class lq_kv_chunk_args(ctypes.Structure):
    _fields_ = [("q", ctypes.c_void_p), ("out", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("dtype", ctypes.c_int),
                ("batch", ctypes.c_int), ("tokens", ctypes.c_int), ("q_heads", ctypes.c_int),
                ("q_token_stride", ctypes.c_int64), ("out_token_stride", ctypes.c_int64), ("starts", ctypes.c_void_p),
                ("block_table", ctypes.c_void_p), ("block_table_stride", ctypes.c_int64), ("max_pages", ctypes.c_int),
                ("lens", ctypes.c_void_p), ("window", ctypes.c_int), ("sinks", ctypes.c_int), ("scale", ctypes.c_float)]


class lq_logprobs_args(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("dtype", ctypes.c_int), ("n", ctypes.c_int), ("vocab", ctypes.c_int),
                ("row_stride", ctypes.c_int64), ("tokens", ctypes.c_void_p), ("logprob", ctypes.c_void_p),
                ("entropy", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("top", ctypes.c_int), ("top_ids", ctypes.c_void_p),
                ("top_logprobs", ctypes.c_void_p), ("lse_rest", ctypes.c_void_p)]


class lq_logprobs_grad_args(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("d_logits", ctypes.c_void_p), ("dtype", ctypes.c_int), ("n", ctypes.c_int),
                ("vocab", ctypes.c_int), ("row_stride", ctypes.c_int64), ("d_row_stride", ctypes.c_int64),
                ("tokens", ctypes.c_void_p), ("lse", ctypes.c_void_p), ("entropy", ctypes.c_void_p),
                ("d_logprob", ctypes.c_void_p), ("d_entropy", ctypes.c_void_p), ("lse_rest", ctypes.c_void_p)]


def library_path() -> Path:
    from .build import LIB
    return LIB


def load_library(build_if_missing: bool = True):
    """Load liblq.so (building it first if asked and needed); raises if it cannot be loaded."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = library_path()
    if build_if_missing:
        from .build import build
        path = build()
    if not path.exists():
        raise RuntimeError(f"liblq.so not built at {path}; run bit_weight_quantized_dequant_gb300.build()")
    L = ctypes.CDLL(str(path))
    P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    L.lq_create.argtypes = [ctypes.POINTER(P), I, S]
    L.lq_create.restype = I
    L.lq_destroy.argtypes = [P]
    L.lq_destroy.restype = I
    L.lq_sync.argtypes = [P]
    L.lq_sync.restype = I
    L.lq_status_string.argtypes = [I]
    L.lq_status_string.restype = ctypes.c_char_p
    L.lq_dequant.argtypes = [P, I, P, P, P, P, P, I, I, P, I, I, I, P]
    L.lq_dequant.restype = I
    L.lq_gemv.argtypes = [P, I, P, P, P, P, P, I, I, P, I, P, I, I, I, I, P]
    L.lq_gemv.restype = I
    L.lq_gemm.argtypes = [P, I, P, P, P, P, P, I, I, P, I, P, I, I, I, I, P]
    L.lq_gemm.restype = I
    L.lq_gemv_noalloc.argtypes = [I, P, P, P, P, P, I, I, P, I, P, I, I, I, I, P]
    L.lq_gemv_noalloc.restype = I
    L.lq_gemv_grouped.argtypes = [P, ctypes.POINTER(lq_problem), I, P]
    L.lq_gemv_grouped.restype = I
    L.lq_gemv_layers.argtypes = [P, ctypes.POINTER(lq_problem), ctypes.POINTER(I), I, P]
    L.lq_gemv_layers.restype = I
    L.lq_gemm_grouped.argtypes = [P, ctypes.POINTER(lq_problem), I, P]
    L.lq_gemm_grouped.restype = I
    L.lq_anchor_count.argtypes = [I]
    L.lq_anchor_count.restype = I
    L.lq_select_anchors.argtypes = [P, P, I, I, P, I, P, P]
    L.lq_select_anchors.restype = I
    L.lq_quantize_2bit.argtypes = [P, P, I, I, P, I, P, P, P, P, I, P]
    L.lq_quantize_2bit.restype = I
    L.lq_quantize_nf4.argtypes = [P, P, I, I, P, P, P]
    L.lq_quantize_nf4.restype = I
    L.lq_stream_create.argtypes = [ctypes.POINTER(P), P, S]
    L.lq_stream_create.restype = I
    L.lq_stream_run.argtypes = [P, P, S, S, I, ctypes.POINTER(lq_problem), I, ctypes.c_int64, P]
    L.lq_stream_run.restype = I
    L.lq_stream_destroy.argtypes = [P]
    L.lq_stream_destroy.restype = I
    L.lq_stream_run_direct.argtypes = [P, P, S, S, I, ctypes.POINTER(lq_problem), I, ctypes.c_int64, P]
    L.lq_stream_run_direct.restype = I
    C = ctypes.POINTER(lq_kv_cache)
    L.lq_rope_table.argtypes = [P, ctypes.POINTER(lq_rope_config), I, I, P, P]
    L.lq_rope_table.restype = I
    L.lq_rope.argtypes = [P, ctypes.POINTER(lq_rope_args), P]
    L.lq_rope.restype = I
    L.lq_kv_tile_bytes.argtypes = [I, I]
    L.lq_kv_tile_bytes.restype = I
    L.lq_kv_append.argtypes = [P, C, ctypes.POINTER(lq_kv_append_args), P]
    L.lq_kv_append.restype = I
    L.lq_kv_read.argtypes = [P, C, P, I, P, P, I, P]
    L.lq_kv_read.restype = I
    L.lq_kv_attention.argtypes = [P, C, ctypes.POINTER(lq_kv_attention_args), P]
    L.lq_kv_attention.restype = I
    L.lq_kv_attention_window.argtypes = [P, C, ctypes.POINTER(lq_kv_attention_args), I, I, P]
    L.lq_kv_attention_window.restype = I
    L.lq_kv_attention_chunk.argtypes = [P, C, ctypes.POINTER(lq_kv_chunk_args), P]
    L.lq_kv_attention_chunk.restype = I
    L.lq_logprobs.argtypes = [P, ctypes.POINTER(lq_logprobs_args), P]
    L.lq_logprobs.restype = I
    L.lq_logprobs_grad.argtypes = [P, ctypes.POINTER(lq_logprobs_grad_args), P]
    L.lq_logprobs_grad.restype = I
    L.lq_selftest_wait.argtypes = [P, ctypes.c_uint, P]
    L.lq_selftest_wait.restype = I
    _LIB = L
    return L


def exported_symbols(path: Path | None = None) -> list[str]:
    """Names from EXPORTED that the library resolves (no GPU needed)."""
    L = ctypes.CDLL(str(path or library_path()))
    return [n for n in EXPORTED if hasattr(L, n)]


def _ptr(t) -> int | None:
    return None if t is None else int(t.data_ptr())


def _dtype_code(t) -> int:
    import torch
    return {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}[t.dtype]


@functools.lru_cache(maxsize=None)
def _torch():
    import torch
    return torch


@functools.lru_cache(maxsize=None)
def _code(dtype) -> int:
    import torch
    codes = {torch.float32: F32, torch.float16: F16, torch.bfloat16: BF16}
    if dtype not in codes:
        raise ValueError(f"dtype {dtype} is not float32, float16 or bfloat16")
    return codes[dtype]


def _stream(stream) -> int | None:
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream) or None


@functools.lru_cache(maxsize=None)
def _rotation():
    """Handle.rope as a differentiable function of x: the gradient is the transpose of what came."""
    import torch

    class Rotation(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x, handle, positions, table, layout, inverse, stream):
            ctx.save_for_backward(positions, table)
            ctx.how = handle, layout, inverse
            return handle.rope(x, positions, table, layout, inverse, stream=stream)

        @staticmethod
        def backward(ctx, g):
            (handle, layout, inverse), (positions, table) = ctx.how, ctx.saved_tensors
            if g.stride(-1) != 1:
                g = g.contiguous()
            return handle.rope(g, positions, table, layout, not inverse), None, None, None, None, None, None

    return Rotation


@functools.lru_cache(maxsize=None)
def _scored():
    """Handle.token_logprobs as a differentiable function of the logits, through the log probabilities and the entropy."""
    import torch

    class Scored(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits, handle, tokens, top, stream):
            logprob, entropy, lse, ids, best = handle._token_logprobs(logits, tokens, top, stream)
            ctx.save_for_backward(logits, tokens, lse, entropy)
            ctx.handle = handle
            ctx.set_materialize_grads(False)
            if ids is not None:
                ctx.mark_non_differentiable(ids, best)
            return logprob, entropy, ids, best

        @staticmethod
        def backward(ctx, d_logprob, d_entropy, *_):
            if torch.is_grad_enabled():     # (a graph of the gradient was asked for)
                raise RuntimeError("token_logprobs has no second derivative")
            if d_logprob is None and d_entropy is None:
                return None, None, None, None, None
            return ctx.handle._token_logprobs_grad(*ctx.saved_tensors, d_logprob, d_entropy), None, None, None, None

    return Scored


@dataclass
class QuantWeights:
    """One quantized matrix W [N][K] in device memory (layouts as in include/lq.h)."""
    format: int
    N: int
    K: int
    codes: object                 # uint8 tensor
    scales: object                # float16 [N][K/32] (2-bit, INT4), float32 [N][K/64] (NF4) or uint8 [N][K/64] (NF4-DQ)
    offsets: object = None        # float16 [N][K/32] (2-bit), int32 permutation [K] (INT4) or float32 second level (NF4-DQ)
    anchor_idx: object = None     # int32 [A]
    anchor_w: object = None       # float16 [N][ld_anchor]
    A: int = 0
    ld_anchor: int = 0

    @staticmethod
    def from_host(packed: dict, fmt: int, device="cuda") -> "QuantWeights":
        """Copy a packed host dict (numpy arrays, bit patterns as uint16) to the device."""
        import numpy as np
        import torch

        def t(a, dtype):
            return torch.from_numpy(np.ascontiguousarray(a)).view(dtype).to(device)
        if fmt in (FMT_2BIT, FMT_INT4):
            A = int(packed["A"])
            off = t(packed["offsets"], torch.float16) if fmt == FMT_2BIT else t(packed["perm"], torch.int32)
            return QuantWeights(fmt, int(packed["N"]), int(packed["K"]), t(packed["codes"], torch.uint8),
                                t(packed["scales"], torch.float16), off,
                                t(packed["anchor_idx"], torch.int32) if A > 0 else None,
                                t(packed["anchor_w"], torch.float16) if A > 0 else None, A, int(packed["ld_anchor"]))
        if fmt == FMT_NF4_DQ:
            return QuantWeights(FMT_NF4_DQ, int(packed["N"]), int(packed["K"]), t(packed["codes"], torch.uint8),
                                t(packed["acodes"], torch.uint8), t(packed["second"], torch.float32))
        return QuantWeights(FMT_NF4, int(packed["N"]), int(packed["K"]), t(packed["codes"], torch.uint8),
                            t(packed["absmax"], torch.float32))

    def args(self):
        return (self.format, _ptr(self.codes), _ptr(self.scales), _ptr(self.offsets), _ptr(self.anchor_idx),
                _ptr(self.anchor_w), int(self.A), int(self.ld_anchor))


class KVCache:
    """A paged low-bit cache of keys and values (layout as in include/lq.h): uint8 pages
    [num_pages][kv_heads][page_size / 16][tile bytes], made here (zeroed) or the caller's."""

    def __init__(self, pages=None, *, page_size: int, kv_heads: int, head_dim: int, bits: int, num_pages: int = 0,
                 device="cuda"):
        import torch
        tile = load_library().lq_kv_tile_bytes(int(bits), int(head_dim))
        if tile == 0:
            raise ValueError(f"no cache with {bits} bits and heads of {head_dim}")
        if page_size < 16 or page_size % 16:
            raise ValueError("page_size must be a multiple of 16")
        if pages is None:
            pages = torch.zeros((num_pages, kv_heads, page_size // 16, tile), dtype=torch.uint8, device=device)
        if (pages.dtype != torch.uint8 or not pages.is_contiguous() or
                tuple(pages.shape[1:]) != (kv_heads, page_size // 16, tile)):
            raise ValueError(f"pages must be contiguous uint8 [num_pages][{kv_heads}][{page_size // 16}][{tile}]")
        self.pages = pages
        self.num_pages, self.page_size, self.kv_heads, self.head_dim, self.bits = \
            pages.shape[0], page_size, kv_heads, head_dim, bits
        self._c = lq_kv_cache(pages.data_ptr(), self.num_pages, page_size, kv_heads, head_dim, bits)
        self._ref = ctypes.byref(self._c)
        self._device = pages.get_device()

    def _on(self, device):
        if self._device != device:
            raise ValueError(f"the cache must be on cuda:{device}")
        return self._ref


class Handle:
    """An lq handle on one CUDA device, with its split-K workspace."""

    def __init__(self, device: int = 0, workspace_bytes: int = 0):
        self._lib = load_library()
        h = ctypes.c_void_p()
        st = self._lib.lq_create(ctypes.byref(h), int(device), int(workspace_bytes))
        if st != LQ_OK:
            raise LQError(st, "lq_create")
        self._h = h
        self.device = device
        self._device = f"cuda:{device}"

    def close(self):
        if getattr(self, "_h", None):
            st = self._lib.lq_destroy(self._h)
            self._h = None
            if st != LQ_OK:
                raise LQError(st, "lq_destroy")

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()

    @property
    def raw(self):
        return self._h

    def sync(self):
        st = self._lib.lq_sync(self._h)
        if st != LQ_OK:
            raise LQError(st, "lq_sync")

    def dequant(self, w: QuantWeights, out=None, out_dtype=None, stream=None):
        import torch
        if out is None:
            out = torch.empty((w.N, w.K), dtype=out_dtype or torch.float32, device=w.codes.device)
        fmt, c, s, o, ai, aw, A, ld = w.args()
        st = self._lib.lq_dequant(self._h, fmt, c, s, o, ai, aw, A, ld, _ptr(out), _dtype_code(out), w.N, w.K,
                                  _stream(stream))
        if st != LQ_OK:
            raise LQError(st, "lq_dequant")
        return out

    def _mm(self, fn, name, w: QuantWeights, x, y=None, y_dtype=None, stream=None):
        import torch
        M = x.shape[0]
        if y is None:
            y = torch.empty((M, w.N), dtype=y_dtype or torch.float32, device=x.device)
        fmt, c, s, o, ai, aw, A, ld = w.args()
        st = fn(self._h, fmt, c, s, o, ai, aw, A, ld, _ptr(x), _dtype_code(x), _ptr(y), _dtype_code(y), M, w.N, w.K,
                _stream(stream))
        if st != LQ_OK:
            raise LQError(st, name)
        return y

    def gemv(self, w: QuantWeights, x, y=None, y_dtype=None, stream=None):
        """y = x * W_eff^T for 1 <= M <= 32 tokens (decode)."""
        return self._mm(self._lib.lq_gemv, "lq_gemv", w, x, y, y_dtype, stream)

    def gemm(self, w: QuantWeights, x, y=None, y_dtype=None, stream=None):
        """y = x * W_eff^T on the tcgen05 tensor-core path (prefill)."""
        return self._mm(self._lib.lq_gemm, "lq_gemm", w, x, y, y_dtype, stream)

    @staticmethod
    def problem(w: QuantWeights, x, y, batch: int = 1, strides: dict | None = None) -> lq_problem:
        """Describe one (batched) product for gemv_grouped; strides are in bytes."""
        p = lq_problem()
        fmt, c, s, o, ai, aw, A, ld = w.args()
        p.format, p.M, p.N, p.K = fmt, int(x.shape[-2]), w.N, w.K
        p.codes, p.scales, p.offsets, p.anchor_idx, p.anchor_w = c, s, o, ai, aw
        p.A, p.ld_anchor = A, ld
        p.x, p.x_dtype, p.y, p.y_dtype = _ptr(x), _dtype_code(x), _ptr(y), _dtype_code(y)
        p.batch = int(batch)
        for k, v in (strides or {}).items():
            setattr(p, "stride_" + k, int(v))
        return p

    @staticmethod
    def prepare(problems):
        """The C array of a list of problems, built once: a decode loop passes it to gemv_grouped
        every token instead of the list (no per-call marshalling)."""
        return (lq_problem * len(problems))(*problems)

    def gemv_grouped(self, problems, stream=None):
        arr = problems if isinstance(problems, ctypes.Array) else (lq_problem * len(problems))(*problems)
        st = self._lib.lq_gemv_grouped(self._h, arr, len(arr), _stream(stream))
        if st != LQ_OK:
            raise LQError(st, "lq_gemv_grouped")

    def gemv_layers(self, layers, stream=None):
        """Consecutive layers (each a list of problems) in one call; a layer may read what the
        layers before it wrote."""
        flat = [p for layer in layers for p in layer]
        arr = (lq_problem * len(flat))(*flat)
        counts = (ctypes.c_int * len(layers))(*[len(layer) for layer in layers])
        st = self._lib.lq_gemv_layers(self._h, arr, counts, len(layers), _stream(stream))
        if st != LQ_OK:
            raise LQError(st, "lq_gemv_layers")

    def selftest_wait(self, limit_us: int, stream=None):
        """Run the bounded-wait self-test: a wait that nothing completes gives up after
        limit_us; the next sync() raises LQError with status LQ_ERR_TIMEOUT."""
        st = self._lib.lq_selftest_wait(self._h, int(limit_us), _stream(stream))
        if st != LQ_OK:
            raise LQError(st, "lq_selftest_wait")

    # ---- rotary positions, the low-bit KV cache and attention over it ----
    # (A decode step calls these once per layer: their checks are few and cheap.)

    def _raw(self, stream):
        """The raw stream of a call."""
        return _torch()._C._cuda_getCurrentRawStream(self.device) if stream is None else stream.cuda_stream

    def _new(self, shape, dtype, stream):
        """A result of a call on `stream`, in memory of that stream: what the current stream's allocator has at hand may
        still be read by work of that stream, which another does not wait for.  Freed, it is not reused before the
        current stream's work so far is done either."""
        torch = _torch()
        with torch.cuda.stream(stream):
            t = torch.empty(shape, dtype=dtype, device=self._device)
        t.record_stream(torch.cuda.current_stream(self.device))
        return t

    def _rows(self, name, t, n, heads, dim, dtype):
        """Token stride of a [n][heads][dim] operand of this device, heads and dimensions contiguous."""
        if t.shape != (n, heads, dim) or t.dtype is not dtype or t.get_device() != self.device:
            raise ValueError(f"{name} must be [{n}][{heads}][{dim}] of {dtype} on cuda:{self.device}")
        s = t.stride()
        if (s[2] != 1 or (s[1] != dim and heads > 1)) and n:
            raise ValueError(f"{name}'s heads and dimensions must be contiguous")
        return s[0] if n > 1 else heads * dim

    def _indices(self, name, t, dtype, n):
        if t is None or t.dtype is not dtype or t.shape != (n,) or not t.is_contiguous() or t.get_device() != self.device:
            raise ValueError(f"{name} must be a contiguous [{n}] tensor of {dtype} on cuda:{self.device}")
        return t.data_ptr()

    def _table(self, table):
        if table.dtype is not _torch().float32 or table.dim() != 2 or not table.is_contiguous() or \
                table.get_device() != self.device:
            raise ValueError(f"table must be a contiguous fp32 [rows][rot_dim] tensor on cuda:{self.device}")
        return table.data_ptr()

    def rope_table(self, count, rot_dim, base=10000.0, first=0, factor=1.0, original_length=0.0, low_rotations=1.0,
                   high_rotations=32.0, mscale=1.0, out=None, stream=None):
        """Rows first .. first + count - 1 of the rotation table, fp32 [count][rot_dim]: cosines, then
        sines.  factor stretches the positions: every frequency (original_length 0) or by parts."""
        if abs(first) > _INT_MAX or abs(count) > _INT_MAX:
            raise ValueError("first and count must be below 2^31")
        if out is None:
            torch, shape = _torch(), (count, rot_dim)
            out = torch.empty(shape, dtype=torch.float32, device=self._device) if stream is None else \
                self._new(shape, torch.float32, stream)
        elif out.shape != (count, rot_dim):
            raise ValueError(f"out must be [{count}][{rot_dim}]")
        c = lq_rope_config(rot_dim, base, factor, original_length, low_rotations, high_rotations, mscale)
        st = self._lib.lq_rope_table(self._h, ctypes.byref(c), first, count, self._table(out), self._raw(stream))
        if st != LQ_OK:
            raise LQError(st, "lq_rope_table")
        return out

    def rope(self, x, positions, table, layout=ROPE_HALF, inverse=False, out=None, stream=None):
        """Rotate the first table.shape[1] dimensions of x [n][heads][dim] (any token and head stride) by
        its int32 positions' table rows; inverse=True applies the transpose (the gradient).  An x that
        requires a gradient gets it through the result (then without out)."""
        torch = _torch()
        if x.requires_grad and torch.is_grad_enabled():
            if out is not None:
                raise ValueError("out cannot take the rotation of an x that requires a gradient")
            return _rotation().apply(x, self, positions, table, layout, inverse, stream)
        n, heads, dim = shape = x.shape
        if n > _INT_MAX or heads > _INT_MAX or dim > _INT_MAX:
            raise ValueError("x has 2^31 or more tokens, heads or dimensions")
        if out is None:
            out = torch.empty(shape, dtype=x.dtype, device=x.device) if stream is None else self._new(shape, x.dtype, stream)
        elif out.shape != shape or out.dtype is not x.dtype or out.get_device() != self.device:
            raise ValueError(f"out must have x's shape and dtype on cuda:{self.device}")
        xs, ys = x.stride(), out.stride()
        if (xs[2] != 1 or ys[2] != 1) and dim > 1:
            raise ValueError("dimensions must be contiguous")
        if x.get_device() != self.device:
            raise ValueError(f"x must be on cuda:{self.device}")
        rows, rot = table.shape
        a = lq_rope_args(x.data_ptr(), out.data_ptr(), _code(x.dtype), n, heads, dim, rot, xs[0], xs[1], ys[0], ys[1],
                         self._table(table), rows, self._indices("positions", positions, torch.int32, n), layout, inverse)
        if n == 0:
            return out
        st = self._lib.lq_rope(self._h, ctypes.byref(a), self._raw(stream))
        if st != LQ_OK:
            raise LQError(st, "lq_rope")
        return out

    def kv_append(self, cache: KVCache, k, v, slots, q=None, table=None, positions=None, layout=ROPE_HALF, q_out=None,
                  stream=None):
        """Quantise k and v [n][kv_heads][dim] into the cache's int64 slots (negative: skipped).  With a
        table, k is rotated first, and so is q [n][q_heads][dim] when given, into the returned tensor."""
        torch = _torch()
        dt, n, dim, hkv = k.dtype, k.shape[0], cache.head_dim, cache.kv_heads
        ks, vs = self._rows("k", k, n, hkv, dim, dt), self._rows("v", v, n, hkv, dim, dt)
        qp = op = tp = pp = None
        hq = qs = os = rows = rot = 0
        if q is not None:
            hq = q.shape[1]
            qs = self._rows("q", q, n, hq, dim, dt)
            if q_out is None:
                q_out = torch.empty((n, hq, dim), dtype=dt, device=q.device) if stream is None else \
                    self._new((n, hq, dim), dt, stream)
                os = hq * dim
            else:
                os = self._rows("q_out", q_out, n, hq, dim, dt)
            qp, op = q.data_ptr(), q_out.data_ptr()
        if table is not None:
            rows, rot = table.shape
            tp, pp = self._table(table), self._indices("positions", positions, torch.int32, n)
        a = lq_kv_append_args(k.data_ptr(), v.data_ptr(), qp, op, _code(dt), n, hq, ks, vs, qs, os,
                              self._indices("slots", slots, torch.int64, n), tp, rows, pp, rot, layout)
        if n == 0:
            return q_out
        st = self._lib.lq_kv_append(self._h, cache._on(self.device), ctypes.byref(a), self._raw(stream))
        if st != LQ_OK:
            raise LQError(st, "lq_kv_append")
        return q_out

    def kv_read(self, cache: KVCache, slots, dtype=None, stream=None):
        """The cached keys and values of int64 slots [n], dense [n][kv_heads][dim] (default bfloat16)."""
        torch = _torch()
        dt, n = dtype or torch.bfloat16, slots.shape[0]
        sp = self._indices("slots", slots, torch.int64, n)
        shape, dev = (n, cache.kv_heads, cache.head_dim), slots.device
        if stream is None:
            k, v = torch.empty(shape, dtype=dt, device=dev), torch.empty(shape, dtype=dt, device=dev)
        else:
            k, v = self._new(shape, dt, stream), self._new(shape, dt, stream)
        if n == 0:
            return k, v
        st = self._lib.lq_kv_read(self._h, cache._on(self.device), sp, n, k.data_ptr(), v.data_ptr(), _code(dt),
                                  self._raw(stream))
        if st != LQ_OK:
            raise LQError(st, "lq_kv_read")
        return k, v

    def _window(self, window, sinks):
        """(window, sinks) as the library takes them; a window of 0 is none."""
        if window is None:
            if sinks:
                raise ValueError("sinks are of a window, and there is none")
            return 0, 0
        if not 1 <= window <= _INT_MAX or not 0 <= sinks <= _INT_MAX:
            raise ValueError("window must be 1 or more, sinks 0 or more, and both below 2^31")
        return window, sinks

    def kv_attention(self, q, cache: KVCache, block_table, lens, scale=None, prefix_table=None, prefix_len=None, out=None,
                     lse=None, stream=None, window=None, sinks=0):
        """Attention of q [batch][tokens][q_heads][dim] (each request's newest tokens, already in the cache)
        over the cache: request b's own tokens in the pages block_table[b] (int32), lens[b] (int32) of
        them, after the prefix_len tokens of prefix_table's pages, which all requests share.  With a window
        (and then no prefix) a row sees the last `window` tokens up to its own, and the request's first
        `sinks`.  Returns out (q's shape and dtype) and the fp32 log-sum-exp [batch][tokens][q_heads]."""
        torch, dev = _torch(), self.device
        B, T, hq, dim = shape = q.shape
        dt, row = q.dtype, hq * dim

        def token_stride(name, t):
            if t.shape != shape or t.dtype is not dt or t.get_device() != dev or dim != cache.head_dim:
                raise ValueError(f"q and out must be [batch][tokens][heads][{cache.head_dim}] of one dtype on cuda:{dev}")
            s = t.stride()
            if s[3] != 1 or (s[2] != dim and hq > 1) or (B > 1 and T > 1 and s[0] != T * s[1]):
                raise ValueError(f"{name} must be rows of contiguous heads with one token stride")
            return s[1] if T > 1 else s[0] if B > 1 else row

        qs = token_stride("q", q)
        if out is None:
            out = torch.empty(shape, dtype=dt, device=q.device) if stream is None else self._new(shape, dt, stream)
            os = row
        else:
            os = token_stride("out", out)
        if lse is None:
            lse = torch.empty((B, T, hq), dtype=torch.float32, device=q.device) if stream is None else \
                self._new((B, T, hq), torch.float32, stream)
        elif lse.shape != (B, T, hq) or lse.dtype is not torch.float32 or not lse.is_contiguous() or lse.get_device() != dev:
            raise ValueError(f"lse must be contiguous fp32 [batch][tokens][heads] on cuda:{dev}")
        if block_table.dtype is not torch.int32 or block_table.dim() != 2 or block_table.get_device() != dev:
            raise ValueError(f"block_table must be int32 [{B}][pages] on cuda:{dev}")
        rows, pages = block_table.shape
        bs = block_table.stride()
        if rows != B or (bs[1] != 1 and pages > 1):
            raise ValueError(f"block_table must be int32 [{B}][pages], rows contiguous")
        pp = None
        if prefix_table is not None:
            n = prefix_table.shape[0]
            pp = self._indices("prefix_table", prefix_table, torch.int32, n)
            room = n * cache.page_size
            if prefix_len is None:
                prefix_len = room
            elif prefix_len > room:
                raise ValueError("prefix_table has too few pages for prefix_len")
        a = lq_kv_attention_args(q.data_ptr(), out.data_ptr(), lse.data_ptr(), _code(dt), B, T, hq, qs, os,
                                 block_table.data_ptr(), bs[0] if B > 1 else pages, pages,
                                 self._indices("lens", lens, torch.int32, B), pp, prefix_len or 0,
                                 dim ** -0.5 if scale is None else scale)
        if window is None and not sinks:
            st = self._lib.lq_kv_attention(self._h, cache._on(dev), ctypes.byref(a), self._raw(stream))
            if st != LQ_OK:
                raise LQError(st, "lq_kv_attention")
            return out, lse
        st = self._lib.lq_kv_attention_window(self._h, cache._on(dev), ctypes.byref(a), *self._window(window, sinks),
                                              self._raw(stream))
        if st != LQ_OK:
            raise LQError(st, "lq_kv_attention_window")
        return out, lse

    def kv_attention_chunk(self, q, cache: KVCache, block_table, lens, starts, scale=None, window=None, sinks=0, out=None,
                           lse=None, stream=None):
        """Attention of chunks of new tokens, as many of each request as there are, over the cache they are in
        already: request b's rows of q [tokens][q_heads][dim] are starts[b] .. starts[b + 1] - 1 (int32
        [batch + 1]), the newest of its lens[b] (int32) tokens in the pages block_table[b] (int32).  Row t sees
        the tokens up to its own; with a window the last `window` of them and the request's first `sinks`.
        Returns out (q's shape and dtype) and the fp32 log-sum-exp [tokens][q_heads]; rows that belong to no
        request are left as they were."""
        torch, dev = _torch(), self.device
        if q.dim() != 3:
            raise ValueError("q must be [tokens][heads][dim]")
        n, hq, dim = shape = q.shape
        if n > _INT_MAX:
            raise ValueError("q has 2^31 or more tokens")
        dt = q.dtype
        if dim != cache.head_dim:
            raise ValueError(f"q must be [tokens][heads][{cache.head_dim}]")
        qs = self._rows("q", q, n, hq, dim, dt)
        if out is None:
            out = torch.empty(shape, dtype=dt, device=q.device) if stream is None else self._new(shape, dt, stream)
            os = hq * dim
        else:
            os = self._rows("out", out, n, hq, dim, dt)
        if lse is None:
            lse = torch.empty((n, hq), dtype=torch.float32, device=q.device) if stream is None else \
                self._new((n, hq), torch.float32, stream)
        elif lse.shape != (n, hq) or lse.dtype is not torch.float32 or not lse.is_contiguous() or lse.get_device() != dev:
            raise ValueError(f"lse must be contiguous fp32 [tokens][heads] on cuda:{dev}")
        if block_table.dtype is not torch.int32 or block_table.dim() != 2 or block_table.get_device() != dev:
            raise ValueError(f"block_table must be int32 [batch][pages] on cuda:{dev}")
        B, pages = block_table.shape
        bs = block_table.stride()
        if bs[1] != 1 and pages > 1:
            raise ValueError("block_table's rows must be contiguous")
        if B > _INT_MAX or pages > _INT_MAX:
            raise ValueError("block_table has 2^31 or more requests or pages")
        a = lq_kv_chunk_args(q.data_ptr(), out.data_ptr(), lse.data_ptr(), _code(dt), B, n, hq, qs, os,
                             self._indices("starts", starts, torch.int32, B + 1), block_table.data_ptr(),
                             bs[0] if B > 1 else pages, pages, self._indices("lens", lens, torch.int32, B),
                             *self._window(window, sinks), dim ** -0.5 if scale is None else scale)
        if n == 0:
            return out, lse
        st = self._lib.lq_kv_attention_chunk(self._h, cache._on(dev), ctypes.byref(a), self._raw(stream))
        if st != LQ_OK:
            raise LQError(st, "lq_kv_attention_chunk")
        return out, lse

    # ---- log probabilities ----

    def _logits(self, name, t, shape=None):
        """Row stride of a [n][vocab] operand of this device, vocabulary contiguous."""
        if t.dim() != 2 or t.get_device() != self.device or (shape is not None and t.shape != shape):
            raise ValueError(f"{name} must be [rows][vocab] on cuda:{self.device}")
        n, V = t.shape
        if n > _INT_MAX or V > _INT_MAX:
            raise ValueError(f"{name} has 2^31 or more rows or tokens")
        s = t.stride()
        if s[1] != 1 and V > 1:
            raise ValueError(f"{name}'s rows must be contiguous")
        return s[0] if n > 1 else V

    def token_logprobs(self, logits, tokens, top=0, stream=None):
        """Log probabilities of the given tokens (int64 [rows]; negative: left out, 0) under logits [rows][vocab] of fp32,
        float16 or bfloat16, the entropy of each row, and its `top` (up to 64) best tokens with theirs.  Returns
        (logprob, entropy, top_ids, top_logprobs): fp32 [rows] twice, int64 and fp32 [rows][top], equal logits by ascending
        id (None both without top).  Logits that require a gradient get it through logprob and entropy, as accurate about
        any offset of a row's logits: a first one only (a backward pass with create_graph is refused); where it is captured
        into a CUDA graph, no graph of operations that was built outside of the capture may hold the same leaves, as for
        any of torch's functions.  Of a Handle's calls this and rope carry gradients."""
        torch = _torch()
        if logits.requires_grad and torch.is_grad_enabled():
            if stream is None:
                return _scored().apply(logits, self, tokens, top, None)
            with torch.cuda.stream(stream):     # (so that the gradient is computed there too)
                out = _scored().apply(logits, self, tokens, top, None)
            for t in out:
                if t is not None:
                    t.record_stream(torch.cuda.current_stream(self.device))
            return out
        logprob, entropy, _, ids, best = self._token_logprobs(logits, tokens, top, stream)
        return logprob, entropy, ids, best

    def _token_logprobs(self, logits, tokens, top, stream):
        torch = _torch()
        rs = self._logits("logits", logits)
        n, V = logits.shape
        if not 0 <= top <= V:
            raise ValueError("top must be from 0 to the vocabulary's size")
        tp = self._indices("tokens", tokens, torch.int64, n)

        def new(shape, dtype):
            return torch.empty(shape, dtype=dtype, device=logits.device) if stream is None else self._new(shape, dtype, stream)
        logprob, entropy = new((n,), torch.float32), new((n,), torch.float32)
        lse = new((2, n), torch.float32)          # (and what its rounding left out)
        ids = best = None
        if top:
            ids, best = new((n, top), torch.int64), new((n, top), torch.float32)
        a = lq_logprobs_args(logits.data_ptr(), _code(logits.dtype), n, V, rs, tp, logprob.data_ptr(), entropy.data_ptr(),
                             lse.data_ptr(), top, _ptr(ids), _ptr(best), lse.data_ptr() + 4 * n)
        if n:
            st = self._lib.lq_logprobs(self._h, ctypes.byref(a), self._raw(stream))
            if st != LQ_OK:
                raise LQError(st, "lq_logprobs")
        return logprob, entropy, lse, ids, best

    def _token_logprobs_grad(self, logits, tokens, lse, entropy, d_logprob, d_entropy):
        torch = _torch()
        n, V = logits.shape
        grads = [None if d is None else d.contiguous() for d in (d_logprob, d_entropy)]
        d_logits = torch.empty((n, V), dtype=logits.dtype, device=logits.device)
        a = lq_logprobs_grad_args(logits.data_ptr(), d_logits.data_ptr(), _code(logits.dtype), n, V,
                                  self._logits("logits", logits), V, tokens.data_ptr(), lse.data_ptr(), entropy.data_ptr(),
                                  _ptr(grads[0]), _ptr(grads[1]), lse.data_ptr() + 4 * n)
        if n:
            st = self._lib.lq_logprobs_grad(self._h, ctypes.byref(a), self._raw(None))
            if st != LQ_OK:
                raise LQError(st, "lq_logprobs_grad")
        return d_logits

    # ---- quantizers (the converter step; include/lq.h gives the definitions) ----

    @staticmethod
    def _weights_arg(W):
        import torch
        if W.dtype != torch.float32 or W.dim() != 2 or not W.is_contiguous() or not W.is_cuda:
            raise ValueError("W must be a contiguous fp32 [N][K] CUDA tensor")
        return W.shape[0], W.shape[1]

    def select_anchors(self, W, A=None, profile=None, stream=None):
        """Anchor columns of W: the A largest ||W[:,c]||_2 * profile_c (ties to the lower
        column), ascending, as an int32 CUDA tensor.  A defaults to the library's
        outlier-anchor count for K (lq_anchor_count); profile is an fp64 [K] CUDA tensor
        (None: all ones)."""
        import torch
        N, K = self._weights_arg(W)
        A = self._lib.lq_anchor_count(K) if A is None else int(A)
        idx = torch.empty(max(A, 0), dtype=torch.int32, device=W.device)
        if profile is not None and (profile.dtype != torch.float64 or profile.numel() != K or not profile.is_contiguous()):
            raise ValueError("profile must be a contiguous fp64 [K] tensor")
        st = self._lib.lq_select_anchors(self._h, _ptr(W), N, K, _ptr(profile), A, _ptr(idx) if A > 0 else None,
                                         _stream(stream))
        if st != LQ_OK:
            raise LQError(st, "lq_select_anchors")
        return idx

    def quantize_2bit(self, W, anchor_idx=None, ld_anchor=None, stream=None) -> QuantWeights:
        """The 2-bit Lloyd-Max G=32 quantizer of W (fp32 [N][K] on the device), with the given
        anchor columns (int32 CUDA tensor, ascending) kept in binary16."""
        import torch
        N, K = self._weights_arg(W)
        A = 0 if anchor_idx is None else int(anchor_idx.numel())
        ld = (int(ld_anchor) if ld_anchor is not None else max(8, (A + 7) // 8 * 8)) if A > 0 else 0
        dev = W.device
        codes = torch.empty((N, K // 4), dtype=torch.uint8, device=dev)
        scales = torch.empty((N, K // 32), dtype=torch.float16, device=dev)
        offsets = torch.empty((N, K // 32), dtype=torch.float16, device=dev)
        anchor_w = torch.empty((N, ld), dtype=torch.float16, device=dev) if A > 0 else None
        st = self._lib.lq_quantize_2bit(self._h, _ptr(W), N, K, _ptr(anchor_idx) if A > 0 else None, A, _ptr(codes),
                                        _ptr(scales), _ptr(offsets), _ptr(anchor_w), ld, _stream(stream))
        if st != LQ_OK:
            raise LQError(st, "lq_quantize_2bit")
        return QuantWeights(FMT_2BIT, N, K, codes, scales, offsets, anchor_idx if A > 0 else None, anchor_w, A, ld)

    def quantize_nf4(self, W, stream=None) -> QuantWeights:
        """The NF4 block-64 quantizer of W (fp32 [N][K] on the device)."""
        import torch
        N, K = self._weights_arg(W)
        codes = torch.empty((N, K // 2), dtype=torch.uint8, device=W.device)
        absmax = torch.empty((N, max(K // 64, 1)), dtype=torch.float32, device=W.device)
        st = self._lib.lq_quantize_nf4(self._h, _ptr(W), N, K, _ptr(codes), _ptr(absmax), _stream(stream))
        if st != LQ_OK:
            raise LQError(st, "lq_quantize_nf4")
        return QuantWeights(FMT_NF4, N, K, codes, absmax)

    def gemm_grouped(self, problems, stream=None):
        """Several prefill products (same format and x dtype) in one tensor-core launch."""
        arr = (lq_problem * len(problems))(*problems)
        st = self._lib.lq_gemm_grouped(self._h, arr, len(problems), _stream(stream))
        if st != LQ_OK:
            raise LQError(st, "lq_gemm_grouped")


# ---- layer streaming (weights in host memory, two device slots) --------------------

def pack_layer(packed: list, fmt: int, align: int = 256):
    """Lay one layer's packed host dicts (the layout of QuantWeights.from_host) out as one
    byte blob.  Returns (blob as uint8 numpy array, per-matrix dict of byte offsets)."""
    import numpy as np
    parts, offs = [], []
    pos = 0

    def add(a):
        nonlocal pos
        b = np.ascontiguousarray(a).view(np.uint8).reshape(-1)
        pad = (-pos) % align
        if pad:
            parts.append(np.zeros(pad, np.uint8))
            pos += pad
        o = pos
        parts.append(b)
        pos += b.nbytes
        return o

    for p in packed:
        d = {"codes": add(p["codes"]), "N": int(p["N"]), "K": int(p["K"]), "A": 0, "ld_anchor": 0}
        if fmt == FMT_2BIT:
            d["scales"] = add(p["scales"])
            d["offsets"] = add(p["offsets"])
            A = int(p["A"])
            d["A"], d["ld_anchor"] = A, (int(p["ld_anchor"]) if A > 0 else 0)
            d["anchor_idx"] = add(p["anchor_idx"]) if A > 0 else 0
            d["anchor_w"] = add(p["anchor_w"]) if A > 0 else 0
        else:
            d["scales"] = add(p["absmax"])
            d["offsets"] = d["anchor_idx"] = d["anchor_w"] = 0
        offs.append(d)
    pad = (-pos) % align
    if pad:
        parts.append(np.zeros(pad, np.uint8))
    return np.concatenate(parts), offs


class LayerStream:
    """A decode pass over a layer stack whose packed weights live in (pinned) host memory:
    layer l+1 is copied into one of two device slots while layer l computes."""

    def __init__(self, handle: Handle, slot_bytes: int):
        self._lib = handle._lib
        self._handle = handle
        s = ctypes.c_void_p()
        st = self._lib.lq_stream_create(ctypes.byref(s), handle.raw, int(slot_bytes))
        if st != LQ_OK:
            raise LQError(st, "lq_stream_create")
        self._s = s

    @staticmethod
    def problem(meta: dict, fmt: int, x, y) -> lq_problem:
        """One matrix of a layer: weight fields are byte offsets from pack_layer's `meta`."""
        p = lq_problem()
        p.format, p.M, p.N, p.K = fmt, int(x.shape[-2]), meta["N"], meta["K"]
        p.codes, p.scales, p.offsets = meta["codes"], meta["scales"], meta["offsets"]
        p.anchor_idx, p.anchor_w = meta["anchor_idx"], meta["anchor_w"]
        p.A, p.ld_anchor = meta["A"], meta["ld_anchor"]
        p.x, p.x_dtype, p.y, p.y_dtype = _ptr(x), _dtype_code(x), _ptr(y), _dtype_code(y)
        p.batch = 1
        return p

    def run(self, host_layers, host_stride: int, layer_bytes: int, L: int, problems, y_layer_stride: int = 0,
            stream=None):
        """host_layers: a uint8 CPU tensor (pinned for overlap) holding L layers at host_stride bytes."""
        arr = (lq_problem * len(problems))(*problems)
        st = self._lib.lq_stream_run(self._s, int(host_layers.data_ptr()), int(host_stride), int(layer_bytes), int(L),
                                     arr, len(problems), int(y_layer_stride), _stream(stream))
        if st != LQ_OK:
            raise LQError(st, "lq_stream_run")

    def run_direct(self, host_layers, host_stride: int, layer_bytes: int, L: int, problems, y_layer_stride: int = 0,
                   stream=None):
        """The same pass with the kernels reading the pinned host bytes directly (no copies)."""
        arr = (lq_problem * len(problems))(*problems)
        st = self._lib.lq_stream_run_direct(self._handle.raw, int(host_layers.data_ptr()), int(host_stride),
                                            int(layer_bytes), int(L), arr, len(problems), int(y_layer_stride),
                                            _stream(stream))
        if st != LQ_OK:
            raise LQError(st, "lq_stream_run_direct")

    def close(self):
        if getattr(self, "_s", None):
            st = self._lib.lq_stream_destroy(self._s)
            self._s = None
            if st != LQ_OK:
                raise LQError(st, "lq_stream_destroy")

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass
