"""Rotary positions, the paged key/value cache, and the attention over it.

Argument marshalling for attn_rope, attn_paged_append and attn_fwd_paged
(include/attn.h holds their formulas and rules).  A decoding step or a chunk of
a prompt, for each layer:

    rotary = Rotary(inv_freq)                                       # once
    cache = PagedKV(k_cache, v_cache, page_table, seq_len, q_start)  # once per layer
    q = paged_append(cache, k, v, q=q, rotary=rotary)                # k, v into the cache; q rotated
    o, lse = fwd_paged(cache, q, causal=True)
"""
from __future__ import annotations

import contextlib
import ctypes
import math

import torch

from . import _abi
from ._abi import load

__all__ = ["Rotary", "PagedKV", "rope", "paged_append", "fwd_paged", "fwd_paged_workspace_size"]

_SAME = contextlib.nullcontext()
# The raw handle of a device's current stream, without the object around it (a call is a few microseconds).
_raw_stream = torch._C._cuda_getCurrentRawStream


def _like(t, dev):
    """An uninitialised dense tensor of t's shape and type."""
    return torch.empty_like(t) if t.is_contiguous() else torch.empty(t.shape, dtype=t.dtype, device=dev)


def _scope(stream, dev: torch.device):
    """The context of a call: its device current, and its stream (outputs and workspaces that the
    call allocates then belong to the stream its kernels run on).  Nothing to do in the usual case."""
    if stream is not None:
        if stream.device != dev:
            raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
        return torch.cuda.stream(stream)
    return _SAME if torch.cuda.current_device() == dev.index else torch.cuda.device(dev)


def _rows(name, t, dev, H=None, D=None):
    """Checks a bf16 [tokens, H, D] (or [B, S, H, D]) tensor whose heads are dense and
    whose tokens are evenly spaced; returns (tokens, H, D, elements between tokens)."""
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be torch.bfloat16, got {t.dtype}")
    if t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    shape, stride = t.shape, t.stride()
    if len(shape) == 4 and (shape[0] == 1 or shape[1] == 1 or stride[0] == shape[1] * stride[1]):
        tokens, step = shape[0] * shape[1], stride[1] if shape[1] > 1 else stride[0]
    elif len(shape) == 3:
        tokens, step = shape[0], stride[0]
    else:
        raise ValueError(f"{name} must be [tokens, H, D] or [B, S, H, D] with evenly spaced tokens, "
                         f"got shape {tuple(shape)}, strides {stride}")
    h, d = shape[-2], shape[-1]
    if (H is not None and h != H) or (D is not None and d != D):
        raise ValueError(f"{name} has {h} heads of {d}, expected {H} of {D}")
    if (d > 1 and stride[-1] != 1) or (h > 1 and stride[-2] != d):
        raise ValueError(f"{name} must have contiguous heads (D innermost), got strides {stride}")
    return tokens, h, d, step if tokens > 1 else h * d


class _Fixed:
    """Attributes are set once: the calls go by what the constructor checked."""

    def __setattr__(self, name, value):
        # (`cache.seq_len += 1` assigns the tensor it changed in place)
        if name in self.__dict__ and value is not self.__dict__[name]:
            raise AttributeError(f"{name} cannot be replaced: write into it, or make a new {type(self).__name__}")
        super().__setattr__(name, value)


class Rotary(_Fixed):
    """The frequencies of a rotation (attn_rotary_t).

    ``inv_freq``: fp32 CUDA tensor [n_freq]; the first 2 n_freq dims of a head turn.
    ``sections``: frequencies of each position axis, in order (default: one axis).
    ``interleaved``: pairs are dims (2i, 2i + 1) instead of (i, i + n_freq).
    The tensor is kept; its contents are read by each call.  Attributes cannot be replaced."""

    def __init__(self, inv_freq: torch.Tensor, sections=None, interleaved: bool = False):
        if inv_freq.dtype != torch.float32 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
            raise ValueError("inv_freq must be a contiguous float32 tensor [n_freq]")
        if not inv_freq.is_cuda:
            raise ValueError("inv_freq must be a CUDA tensor")
        n = inv_freq.numel()
        sections = (n,) if sections is None else tuple(int(x) for x in sections)
        if not 1 <= len(sections) <= 4 or min(sections) < 0 or sum(sections) != n:
            raise ValueError(f"sections {sections} must be 1 to 4 counts that sum to {n}")
        self.inv_freq, self.sections, self.interleaved = inv_freq, sections, bool(interleaved)
        self._section = (ctypes.c_int * 4)(*sections)

    @property
    def device(self):
        return self.inv_freq.device

    def _struct(self, positions, tokens, dev):
        if self.inv_freq.device != dev:
            raise ValueError(f"inv_freq is on {self.inv_freq.device}, expected {dev}")
        ptr = None
        if positions is not None:
            if positions.dtype != torch.int32 or positions.device != dev or not positions.is_contiguous():
                raise ValueError(f"positions must be a contiguous int32 tensor on {dev}")
            if positions.numel() != len(self.sections) * tokens or (
                    len(self.sections) > 1 and positions.shape[0] != len(self.sections)):
                raise ValueError(f"positions has shape {tuple(positions.shape)}, expected {len(self.sections)} axes "
                                 f"of {tokens} tokens")
            ptr = positions.data_ptr()
        elif len(self.sections) > 1:
            raise ValueError("several axes need positions")
        return _abi.RotaryStruct(self.inv_freq.data_ptr(), ptr, self.inv_freq.numel(), len(self.sections),
                                 self._section, int(self.interleaved))


def rope(q, k=None, *, rotary: Rotary, positions=None, inverse: bool = False, q_out=None, k_out=None, stream=None):
    """Rotates q (and k) in one launch (attn_rope).  q [B, S, H_q, D] or [tokens, H_q, D]
    bf16, k with the same tokens; ``positions`` int32 [B, S] (or [axes, B, S]), default
    0 .. S - 1 in each row.  ``inverse`` turns back: applied to dq, dk it is the backward
    pass.  ``q_out`` / ``k_out`` may be q / k (in place).  Returns q' or (q', k')."""
    dev = q.device
    if not q.is_cuda:
        raise ValueError("q must be a CUDA tensor")
    tokens, H_q, D, q_step = _rows("q", q, dev)
    period = q.shape[1] if q.dim() == 4 else tokens
    H_k = k_step = qo_step = ko_step = 0
    if q_out is not None and q_out.shape != q.shape:
        raise ValueError(f"q_out has shape {tuple(q_out.shape)}, expected {tuple(q.shape)}")
    if k is not None:
        if k.shape[:-2] != q.shape[:-2]:
            raise ValueError(f"k has tokens {tuple(k.shape[:-2])}, q {tuple(q.shape[:-2])}: rotate them in two calls")
        _, H_k, _, k_step = _rows("k", k, dev, D=D)
        if k_out is not None and k_out.shape != k.shape:
            raise ValueError(f"k_out has shape {tuple(k_out.shape)}, expected {tuple(k.shape)}")
    elif k_out is not None:
        raise ValueError("k_out is given without k")
    r = rotary._struct(positions, tokens, dev)
    with _scope(stream, dev):
        if q_out is None:
            q_out, qo_step = _like(q, dev), H_q * D
        else:
            qo_step = _rows("q_out", q_out, dev)[3]
        if k is not None:
            if k_out is None:
                k_out, ko_step = _like(k, dev), H_k * D
            else:
                ko_step = _rows("k_out", k_out, dev)[3]
        if tokens == 0:
            return q_out if k is None else (q_out, k_out)
        code = load().attn_rope(q.data_ptr(), None if k is None else k.data_ptr(), q_out.data_ptr(),
                                None if k is None else k_out.data_ptr(), tokens, H_q, H_k, D, q_step, k_step, qo_step,
                                ko_step, max(period, 1), ctypes.byref(r), int(bool(inverse)),
                                _raw_stream(dev.index))
    _abi.check(code, "attn_rope")
    return q_out if k is None else (q_out, k_out)


class PagedKV(_Fixed):
    """A paged key/value cache and the batch of sequences a call works on (attn_paged_kv_t).

    ``k``, ``v``: [n_pages, page_size, H_kv, D] bf16 or torch.float8_e4m3fn CUDA tensors of the
    same shape and strides (D innermost; the other dims in any order, so a
    transposed [n_pages, H_kv, page_size, D] or a slice of a larger pool will do).
    ``page_table`` int32 [n_seq, max_pages], ``seq_len`` int32 [n_seq] (keys of each sequence,
    new ones included), ``q_start`` int32 [n_seq + 1] (rows of each sequence's new tokens).
    ``k_scale``, ``v_scale``: an e4m3 cache holds k / k_scale and v / v_scale.

    The tensors are kept and their contents read on the device by each call, so a step updates them in
    place (inside a CUDA graph too); they may not be resized, and the attributes cannot be replaced."""

    def __init__(self, k, v, page_table, seq_len, q_start, k_scale: float = 1.0, v_scale: float = 1.0):
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride():
            raise ValueError("k and v must be [n_pages, page_size, H_kv, D] with the same shape and strides")
        if k.dtype != v.dtype or k.dtype not in (torch.bfloat16, torch.float8_e4m3fn):
            raise TypeError(f"k and v must both be bfloat16 or float8_e4m3fn, got {k.dtype} and {v.dtype}")
        dev = k.device
        for name, t in (("k", k), ("v", v), ("page_table", page_table), ("seq_len", seq_len), ("q_start", q_start)):
            if not t.is_cuda:
                raise ValueError(f"{name} must be a CUDA tensor")
            if t.device != dev:
                raise ValueError(f"tensors on different devices ({dev} and {t.device}): all must be on one device")
        for name, t in (("page_table", page_table), ("seq_len", seq_len), ("q_start", q_start)):
            if t.dtype != torch.int32:
                raise TypeError(f"{name} must be torch.int32, got {t.dtype}")
        n_seq = seq_len.numel()
        if page_table.dim() != 2 or page_table.shape[0] != n_seq or seq_len.dim() != 1 or tuple(q_start.shape) != (n_seq + 1,):
            raise ValueError(f"page_table {tuple(page_table.shape)}, seq_len {tuple(seq_len.shape)}, q_start "
                             f"{tuple(q_start.shape)}: expected [n, max_pages], [n], [n + 1]")
        if not (seq_len.is_contiguous() and q_start.is_contiguous()) or (
                page_table.shape[1] > 1 and page_table.stride(1) != 1):
            raise ValueError("seq_len and q_start must be contiguous, page_table's rows too")
        if k.shape[3] > 1 and k.stride(3) != 1:
            raise ValueError("the cache's head dim must be contiguous")
        self.k, self.v, self.page_table, self.seq_len, self.q_start = k, v, page_table, seq_len, q_start
        self.k_scale, self.v_scale = float(k_scale), float(v_scale)
        self.device, self.H_kv, self.D = dev, k.shape[2], k.shape[3]
        n_pages, page_size = k.shape[0], k.shape[1]
        self._s = _abi.PagedKVStruct(
            k.data_ptr(), v.data_ptr(), int(k.dtype == torch.float8_e4m3fn), n_pages, page_size, self.H_kv, self.D,
            k.stride(0), k.stride(1), k.stride(2), self.k_scale, self.v_scale, page_table.data_ptr(),
            page_table.stride(0) if n_seq > 1 else page_table.shape[1], page_table.shape[1], seq_len.data_ptr(),
            q_start.data_ptr(), n_seq)
        self._ref = ctypes.byref(self._s)


def paged_append(cache: PagedKV, k, v, q=None, rotary: Rotary | None = None, positions=None, q_out=None, stream=None):
    """Writes the new tokens' k (rotated) and v, [tokens, H_kv, D] bf16, into the cache and
    returns the rotated q [tokens, H_q, D] (None without q) (attn_paged_append).
    ``positions``: int32 [tokens] or [axes, tokens]; default: each token's key index in its sequence.
    ``q_out`` may be q (in place, contiguous)."""
    dev = cache.device
    tokens, _, _, k_step = _rows("k", k, dev, cache.H_kv, cache.D)
    v_tokens, _, _, v_step = _rows("v", v, dev, cache.H_kv, cache.D)
    if v_tokens != tokens:
        raise ValueError(f"k has {tokens} tokens, v {v_tokens}")
    H_q = q_step = 0
    if q is not None:
        if rotary is None:
            raise ValueError("q is only rotated: without rotary, leave it out")
        q_tokens, H_q, _, q_step = _rows("q", q, dev, D=cache.D)
        if q_tokens != tokens:
            raise ValueError(f"k has {tokens} tokens, q {q_tokens}")
        if q_out is not None and (
                q_out.shape != q.shape or q_out.dtype != q.dtype or q_out.device != dev or not q_out.is_contiguous()):
            raise ValueError(f"q_out must be a contiguous bfloat16 tensor of q's shape on {dev}")
    elif q_out is not None:
        raise ValueError("q_out is given without q")
    if rotary is None and positions is not None:
        raise ValueError("positions are given without rotary")
    r = None if rotary is None else ctypes.byref(rotary._struct(positions, tokens, dev))
    with _scope(stream, dev):
        if q is not None and q_out is None:
            q_out = _like(q, dev)
        if tokens == 0:
            return q_out
        code = load().attn_paged_append(cache._ref, None if q is None else q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                        None if q is None else q_out.data_ptr(), tokens, H_q, q_step, k_step, v_step,
                                        r, _raw_stream(dev.index))
    _abi.check(code, "attn_paged_append")
    return q_out


_workspace_sizes: dict = {}


def fwd_paged_workspace_size(H_q: int, H_kv: int, D: int) -> int:
    """Bytes of workspace fwd_paged needs (attn_fwd_paged_workspace_size)."""
    key = (H_q, H_kv, D)
    if key not in _workspace_sizes:
        _workspace_sizes[key] = int(load().attn_fwd_paged_workspace_size(H_q, H_kv, D))
    return _workspace_sizes[key]


def fwd_paged(cache: PagedKV, q, causal: bool = True, scale: float | None = None, max_new: int = 0, out=None, lse=None,
              workspace=None, stream=None):
    """Attention of each sequence's new tokens q [tokens, H_q, D] over its paged keys
    (attn_fwd_paged).  Returns (o bf16 [tokens, H_q, D], lse fp32 [H_q, tokens]); rows that
    belong to no sequence are left as ``out`` and ``lse`` had them.  ``max_new``: the most new
    tokens of any sequence (chooses the kernel only; 0 = unknown: the mean decides, which suits batches whose
    sequences bring about as many each)."""
    dev = cache.device
    if q.dim() != 3:
        raise ValueError(f"q must be [tokens, H_q, D], got shape {tuple(q.shape)}")
    tokens, H_q, D, q_step = _rows("q", q, dev, D=cache.D)
    if out is not None and (
            out.shape != q.shape or out.dtype != torch.bfloat16 or out.device != dev or not out.is_contiguous()):
        raise ValueError(f"out must be a contiguous bfloat16 tensor {tuple(q.shape)} on {dev}")
    if lse is not None and (
            tuple(lse.shape) != (H_q, tokens) or lse.dtype != torch.float32 or lse.device != dev or not lse.is_contiguous()):
        raise ValueError(f"lse must be a contiguous float32 tensor {(H_q, tokens)} on {dev}")
    need = fwd_paged_workspace_size(H_q, cache.H_kv, D)
    if workspace is not None and (workspace.device != dev or not workspace.is_contiguous()
                                  or workspace.numel() * workspace.element_size() < need):
        raise ValueError(f"workspace must be a contiguous buffer of at least {need} bytes on {dev}")
    with _scope(stream, dev):
        if out is None:
            out = _like(q, dev)
        if lse is None:
            lse = torch.empty_strided((H_q, tokens), (tokens, 1), dtype=torch.float32, device=dev)
        if workspace is None:
            workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dev)
        if tokens == 0:
            return out, lse
        code = load().attn_fwd_paged(cache._ref, q.data_ptr(), out.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
                                     tokens, H_q, q_step, int(max_new), int(bool(causal)),
                                     1.0 / math.sqrt(D) if scale is None else float(scale),
                                     _raw_stream(dev.index))
    _abi.check(code, "attn_fwd_paged")
    return out, lse
