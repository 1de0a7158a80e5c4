"""Python binding of the decoder-layer operators of libw4a8 (the C ABI in
include/w4a8_block.h): what stands between the W4A8 linears of ``w4a8.py``.

    xq, xs, h = rmsnorm_quant_act(x, weight, residual)      # add, norm, rotate, int8 rows
    qkv = w4a8.w4a8_gemm(xq, xs, layer)                     # (or w4a8_gemv for at most 8 rows)
    cache = KVCache8.empty(pages, kv_heads, head_dim)       # paged, 8-bit, a scale a page and head
    q = kv8_append(cache, table, ctx_len, start, max_new, k, v, q=q, pos=pos, rope=rope)
    o = kv8_attention(q, cache, table, kv_len, start, max_new, max_kv)

and for training ``rmsnorm_grad`` and ``rope_axes`` (forward and, with ``inverse``, backward).

Argument marshalling only; there is no fallback: a CPU tensor or a missing library raises.
Activations are bf16 [tokens, columns] or [tokens, heads, head_dim] with dense heads; the
latter may be slices of a wider projection output (any token stride that keeps 16-byte
alignment).
"""

from __future__ import annotations

import ctypes
import math
from dataclasses import dataclass
from typing import Optional, Sequence

import torch

from . import w4a8
from .w4a8 import ROT_BLOCK, _check, _dev

ABI_VERSION = 1
NORM_MAX_K, ROPE_MAX_AXES, ROPE_MAX_HEAD_DIM = 16384, 4, 256
_STREAM_TYPES = {torch.bfloat16: 0, torch.float32: 1}

_P, _I64, _I32, _F32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float


class RopeDesc(ctypes.Structure):
    """Mirror of struct w4a8_rope in include/w4a8_block.h."""
    _fields_ = [("pos", _P), ("pos_stride", _I64), ("inv_freq", _P), ("rotary_dim", _I32), ("axes", _I32),
                ("sections", _I32 * ROPE_MAX_AXES), ("interleaved", _I32)]


class KV8Desc(ctypes.Structure):
    """Mirror of struct w4a8_kv8 in include/w4a8_block.h."""
    _fields_ = [("k", _P), ("v", _P), ("k_scale", _P), ("v_scale", _P), ("pages", _I64), ("heads", _I32),
                ("head_dim", _I32), ("page_tokens", _I32), ("table_stride", _I32), ("table", _P)]


# Symbols declared in include/w4a8_block.h, with their ctypes signatures.
SIGNATURES = {
    "rmsnorm_quant_act": [_P, _P, _I32, _P, _I64, _I64, _F32, _I32, _I32, _P, _P, _P, _P, _P, _P],
    "rmsnorm_grad": [_P, _P, _I32, _P, _P, _P, _I64, _I64, _I32, _P, _P, _P, _I64, _P],
    "rmsnorm_grad_workspace": [_I64, _I64],
    "rope_axes": [_P, _I64, _I32, _I32, _I64, _P, _I32, _P, _I64, _P],
    "kv8_append": [_P, _P, _P, _I64, _I64, _I64, _P, _I64, _P, _I64, _P, _I32, _I64, _P, _P, _I64, _P],
    "kv8_attention": [_P, _I32, _I64, _P, _P, _P, _I64, _I64, _I64, _I64, _F32, _I32, _I64, _P, _I64, _P, _P, _I64, _P],
    "kv8_attention_workspace": [_I64, _I64, _I64, _I64, _I32, _I32, _I32],
    "w4a8_block_abi_version": [],
}

_lib = None


def load() -> ctypes.CDLL:
    """The entries of w4a8_block.h in libw4a8.so (built by __graft_entry__.build())."""
    global _lib
    if _lib is None:
        lib = w4a8.load()
        for name, args in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = ctypes.c_int64 if name.endswith("_workspace") else ctypes.c_int
        if lib.w4a8_block_abi_version() != ABI_VERSION:
            raise ImportError("libw4a8.so: version mismatch of the decoder-layer entries")
        _lib = lib
    return _lib


def call(fn: str, *args) -> int:
    """Call a C entry point with raw arguments (pointers as ints); returns its result."""
    return getattr(load(), fn)(*args)


def _new_or(t, shape, dtype, device, name: str) -> torch.Tensor:
    """A caller's output buffer, checked, or a new one."""
    return torch.empty(shape, dtype=dtype, device=device) if t is None else _is(t, shape, dtype, name)


def _stream(t: torch.Tensor) -> int:
    """The current stream's handle; without building a torch Stream object, which costs as much as half a launch."""
    return torch._C._cuda_getCurrentRawStream(t.device.index)


def _is(t, shape, dtype, name: str) -> torch.Tensor:
    """A given tensor must be on the GPU, dense, and exactly of this shape and type."""
    if t.__class__ is torch.Tensor and t.dtype is dtype and t.shape == shape and t.is_cuda and t.is_contiguous():
        return t
    _dev(t, dtype, name)
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    return t


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _rows(x: torch.Tensor, name: str):
    _dev(x, torch.bfloat16, name)
    if x.dim() != 2:
        raise ValueError(f"{name} must be [rows, columns]")
    return x.shape


def _heads(x: torch.Tensor, name: str, heads: Optional[int] = None, head_dim: Optional[int] = None, rows=None) -> int:
    """Checks a bf16 [tokens, heads, head_dim] tensor with dense heads; its token stride."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda:
        raise ValueError(f"{name} must be a CUDA (HIP) tensor")
    if x.dtype is not torch.bfloat16 or x.dim() != 3:
        raise ValueError(f"{name} must be bfloat16 [tokens, heads, head_dim]")
    t, h, d = x.shape
    if (heads is not None and h != heads) or (head_dim is not None and d != head_dim) or (rows is not None and t != rows):
        raise ValueError(f"{name} has shape {tuple(x.shape)}, expected "
                         f"({'tokens' if rows is None else rows}, {heads or 'heads'}, {head_dim or 'head_dim'})")
    stride = x.stride()
    if (d > 1 and stride[2] != 1) or (h > 1 and stride[1] != d):
        raise ValueError(f"{name} must have dense heads")
    return stride[0] if t > 1 else h * d


def _norm(m, k, x, weight, residual, eps, qmax, h, rstd, y, xq, xs):
    _is(weight, (k,), torch.float32, "weight")
    stream = torch.bfloat16
    if residual is not None:
        stream = residual.dtype
        if stream not in _STREAM_TYPES:
            raise ValueError("residual must be bfloat16 or float32")
        _is(residual, (m, k), stream, "residual")
        h = _new_or(h, (m, k), stream, x.device, "h")
    elif h is not None:
        raise ValueError("h is an output only where there is a residual")
    if rstd is not None:
        _is(rstd, (m,), torch.float32, "rstd")
    _check("rmsnorm_quant_act", load().rmsnorm_quant_act(
        x.data_ptr(), _ptr(residual), _STREAM_TYPES[stream], weight.data_ptr(), m, k, eps, ROT_BLOCK, qmax, _ptr(h),
        _ptr(rstd), _ptr(y), _ptr(xq), _ptr(xs), _stream(x)))
    return x if residual is None else h


def rmsnorm_quant_act(x, weight, residual=None, eps: float = 1e-6, qmax: int = 127, h=None, rstd=None, y=None, xq=None,
                      xs=None):
    """h = residual + x (in the residual's type, bf16 or fp32), RMS norm of h with fp32
    weight [K], then the rotation and int8 rows of rotate_quant_act, in one pass:
    bf16 x [M, K] -> (int8 xq [M, K], float32 xs [M], h).  Without a residual h is x.
    ``h`` may be the residual itself (updated in place).  ``rstd`` float32 [M] and ``y``
    bf16 [M, K] (the normalised rows, unrotated) are written if given."""
    m, k = _rows(x, "x")
    xq = _new_or(xq, (m, k), torch.int8, x.device, "xq")
    xs = _new_or(xs, (m,), torch.float32, x.device, "xs")
    if y is not None:
        _is(y, (m, k), torch.bfloat16, "y")
    return xq, xs, _norm(m, k, x, weight, residual, eps, qmax, h, rstd, y, xq, xs)


def rmsnorm(x, weight, residual=None, eps: float = 1e-6, h=None, rstd=None, y=None):
    """The same norm without the int8 rows (a final norm): (y bf16 [M, K], h)."""
    m, k = _rows(x, "x")
    y = _new_or(y, (m, k), torch.bfloat16, x.device, "y")
    return y, _norm(m, k, x, weight, residual, eps, 127, h, rstd, y, None, None)


def rmsnorm_grad(grad, h, rstd, weight, grad_h=None, rotated: bool = True, dx=None, dweight=None,
                 need_dweight: bool = True, workspace=None):
    """The backward of rmsnorm_quant_act (``rotated``: grad is bf16 with respect to the
    rotated activation, as grad_input gives it) or of rmsnorm: (dx, dweight).  dx, of h's
    type, is the gradient of x and of the residual alike; ``grad_h`` is the gradient that
    reached h on other ways (dx may be the same tensor).  dweight is float32 [K], None
    without need_dweight.  ``workspace``: a uint8 tensor of rmsnorm_grad_workspace(M, K)
    bytes at least, allocated if None."""
    m, k = _rows(grad, "grad")
    _is(weight, (k,), torch.float32, "weight")
    dt = h.dtype
    if dt not in _STREAM_TYPES:
        raise ValueError("h must be bfloat16 or float32")
    _is(h, (m, k), dt, "h")
    _is(rstd, (m,), torch.float32, "rstd")
    if grad_h is not None:
        _is(grad_h, (m, k), dt, "grad_h")
    dx = _new_or(dx, (m, k), dt, grad.device, "dx")
    lib, ws = load(), 0
    if need_dweight:
        dweight = _new_or(dweight, (k,), torch.float32, grad.device, "dweight")
        ws = lib.rmsnorm_grad_workspace(m, k)
        workspace = _workspace(workspace, ws, grad.device)
    elif dweight is not None:
        raise ValueError("dweight is given but not needed")
    _check("rmsnorm_grad", lib.rmsnorm_grad(
        grad.data_ptr(), h.data_ptr(), _STREAM_TYPES[dt], rstd.data_ptr(), weight.data_ptr(), _ptr(grad_h), m, k,
        ROT_BLOCK if rotated else 0, dx.data_ptr(), _ptr(dweight), _ptr(workspace) if ws else None, ws, _stream(grad)))
    return dx, dweight


def _workspace(t, size: int, device):
    if size == 0:
        return None
    if t is None:
        return torch.empty(size, dtype=torch.uint8, device=device)
    _dev(t, torch.uint8, "workspace")
    if t.numel() < size:
        raise ValueError(f"workspace has {t.numel()} bytes, {size} are needed")
    return t


def rmsnorm_grad_workspace(m: int, k: int) -> int:
    """Bytes of workspace of rmsnorm_grad with dweight."""
    return int(load().rmsnorm_grad_workspace(int(m), int(k)))


@dataclass
class Rope:
    """Rotary positions: the frequency of every pair, and how many pairs each axis has
    (sections, one number an axis; all pairs on one axis by default)."""
    inv_freq: torch.Tensor                        # float32 [rotary_dim / 2]
    sections: Optional[Sequence[int]] = None
    interleaved: bool = False

    def desc(self, pos: torch.Tensor, tokens: int) -> RopeDesc:
        _dev(self.inv_freq, torch.float32, "inv_freq")
        n = self.inv_freq.numel()
        sections = [n] if self.sections is None else list(self.sections)
        if not 1 <= len(sections) <= ROPE_MAX_AXES:
            raise ValueError(f"1 to {ROPE_MAX_AXES} axes, got {len(sections)}")
        _is(pos, (len(sections), tokens), torch.int32, "pos")
        return RopeDesc(pos.data_ptr(), tokens, self.inv_freq.data_ptr(), 2 * n, len(sections),
                        (_I32 * ROPE_MAX_AXES)(*sections), int(bool(self.interleaved)))


def rope_axes(x, pos, rope: Rope, inverse: bool = False, out=None):
    """Rotates bf16 x [T, heads, head_dim] by the int32 positions pos [axes, T]; ``inverse``
    turns back (the backward).  ``out`` may be x itself."""
    xs = _heads(x, "x")
    t, h, d = x.shape
    if out is None:
        out = torch.empty(t, h, d, dtype=torch.bfloat16, device=x.device)
    os_ = _heads(out, "out", h, d, t)
    desc = rope.desc(pos, t)
    _check("rope_axes", load().rope_axes(x.data_ptr(), t, h, d, xs, ctypes.addressof(desc), int(bool(inverse)),
                                         out.data_ptr(), os_, _stream(x)))
    return out


@dataclass
class KVCache8:
    """Pages of int8 keys and values with one scale for each page and head."""
    k: torch.Tensor          # int8 [pages, heads, page_tokens, head_dim]
    v: torch.Tensor          # int8 [pages, heads, head_dim, page_tokens]
    k_scale: torch.Tensor    # float32 [pages, heads]
    v_scale: torch.Tensor    # float32 [pages, heads]

    @classmethod
    def empty(cls, pages: int, heads: int, head_dim: int, page_tokens: int = 64, device="cuda"):
        z = lambda *s: torch.zeros(*s, dtype=torch.int8, device=device)
        f = lambda: torch.zeros(pages, heads, dtype=torch.float32, device=device)
        return cls(z(pages, heads, page_tokens, head_dim), z(pages, heads, head_dim, page_tokens), f(), f())

    @property
    def page_tokens(self) -> int:
        return self.k.shape[2]

    def desc(self, table: torch.Tensor, batch: int) -> KV8Desc:
        _dev(self.k, torch.int8, "cache.k")
        if self.k.dim() != 4:
            raise ValueError("cache.k must be [pages, heads, page_tokens, head_dim]")
        pages, heads, tokens, d = self.k.shape
        _is(self.v, (pages, heads, d, tokens), torch.int8, "cache.v")
        _is(self.k_scale, (pages, heads), torch.float32, "cache.k_scale")
        _is(self.v_scale, (pages, heads), torch.float32, "cache.v_scale")
        _dev(table, torch.int32, "table")
        if table.dim() != 2 or table.shape[0] != batch:
            raise ValueError(f"table must be [{batch}, pages of a sequence], got {tuple(table.shape)}")
        return KV8Desc(self.k.data_ptr(), self.v.data_ptr(), self.k_scale.data_ptr(), self.v_scale.data_ptr(), pages,
                       heads, d, tokens, table.shape[1], table.data_ptr())


def kv8_append(cache: KVCache8, table, ctx_len, q_start, max_new: int, k, v, q=None, pos=None, rope: Rope = None,
               q_out=None):
    """Appends the new keys and values bf16 [T, kv_heads, head_dim] of B sequences to their
    pages (table int32 [B, pages of a sequence]), the keys rotated by ``rope`` at ``pos``
    [axes, T].  Rows q_start[b] .. q_start[b + 1] (int32 [B + 1]) belong to sequence b,
    which held ctx_len[b] (int32 [B]) tokens; max_new bounds the new tokens of a sequence.
    With ``q`` bf16 [T, q_heads, head_dim] its rotation is returned (into ``q_out``)."""
    batch = ctx_len.numel()
    desc = cache.desc(table, batch)
    _is(ctx_len, (batch,), torch.int32, "ctx_len")
    _is(q_start, (batch + 1,), torch.int32, "q_start")
    heads, d = cache.k.shape[1], cache.k.shape[3]
    ks = _heads(k, "k", heads, d)
    t = k.shape[0]
    vs = _heads(v, "v", heads, d, t)
    qh = qs = os_ = 0
    if q is not None:
        qs = _heads(q, "q", None, d, t)
        qh = q.shape[1]
        if q_out is None:
            q_out = torch.empty(t, qh, d, dtype=torch.bfloat16, device=q.device)
        os_ = _heads(q_out, "q_out", qh, d, t)
    elif q_out is not None:
        raise ValueError("q_out without q")
    if (rope is None) != (pos is None):
        raise ValueError("rope and pos go together")
    rd = None if rope is None else rope.desc(pos, t)
    _check("kv8_append", load().kv8_append(
        ctypes.addressof(desc), ctx_len.data_ptr(), q_start.data_ptr(), batch, t, max_new, k.data_ptr(), ks,
        v.data_ptr(), vs, _ptr(q), qh, qs, None if rd is None else ctypes.addressof(rd), _ptr(q_out), os_, _stream(k)))
    return q_out


def kv8_attention(q, cache: KVCache8, table, kv_len, q_start, max_new: int, max_kv: int, scale: Optional[float] = None,
                  causal: bool = True, window: int = 0, out=None, lse=None, workspace=None):
    """Attention of bf16 q [T, q_heads, head_dim], the last tokens of B sequences, over their
    kv_len[b] cached tokens (the new ones among them): bf16 [T, q_heads, head_dim].  scale
    defaults to head_dim ** -0.5; ``window`` > 0 keeps the last window tokens of each
    position.  ``lse`` float32 [T, q_heads] is written if given.  max_new and max_kv bound
    the new and the cached tokens of a sequence, and divide the work of the whole call: single
    tokens over long contexts are much faster in a call without prompts.  Rows of q that belong
    to no sequence, or lie past its max_new, are not written.  ``workspace``: a uint8 tensor of
    kv8_attention_workspace(...) bytes at least, allocated if None."""
    batch = kv_len.numel()
    desc = cache.desc(table, batch)
    _is(kv_len, (batch,), torch.int32, "kv_len")
    _is(q_start, (batch + 1,), torch.int32, "q_start")
    heads, d = cache.k.shape[1], cache.k.shape[3]
    qs = _heads(q, "q", None, d)
    t, qh, _ = q.shape
    if out is None:
        out = torch.empty(t, qh, d, dtype=torch.bfloat16, device=q.device)
    os_ = _heads(out, "out", qh, d, t)
    if lse is not None:
        _is(lse, (t, qh), torch.float32, "lse")
    lib = load()
    ws = lib.kv8_attention_workspace(batch, t, max_new, max_kv, qh, heads, d)
    workspace = _workspace(workspace, ws, q.device)
    _check("kv8_attention", lib.kv8_attention(
        q.data_ptr(), qh, qs, ctypes.addressof(desc), kv_len.data_ptr(), q_start.data_ptr(), batch, t, max_new, max_kv,
        1.0 / math.sqrt(d) if scale is None else scale, int(bool(causal)), window, out.data_ptr(), os_, _ptr(lse),
        _ptr(workspace), ws, _stream(q)))
    return out


def kv8_attention_workspace(batch: int, tokens: int, max_new: int, max_kv: int, q_heads: int, kv_heads: int,
                            head_dim: int) -> int:
    """Bytes of workspace of kv8_attention for these sizes (0: none)."""
    return int(load().kv8_attention_workspace(batch, tokens, max_new, max_kv, q_heads, kv_heads, head_dim))
