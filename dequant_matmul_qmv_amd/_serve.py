"""ctypes binding of libmxq's serving operators (argument marshalling only):
rotary positions, the 8-bit paged key/value cache and what works on it, and
sampling.  As in ``_lib``: tensor metadata is checked, raw device pointers and
the current HIP stream are passed on, a non-OK status becomes an exception.

These calls are made once a layer for a single token, so their host time
counts: checks are plain attribute comparisons, and the device is only
switched when it is not the current one.
"""

from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import MXQ_BF16, MXQ_F16, MXQ_F32

_HALF = {torch.float16: MXQ_F16, torch.bfloat16: MXQ_BF16}
_LOGITS = {torch.float16: MXQ_F16, torch.bfloat16: MXQ_BF16, torch.float32: MXQ_F32}
_i32 = torch.int32
_f32 = torch.float32


class _CacheStruct(ctypes.Structure):
    """ctypes mirror of ``mxq_kv_cache`` (include/mxq.h)."""

    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("blocks", ctypes.c_int64), ("kv_heads", ctypes.c_int32),
                ("block", ctypes.c_int32), ("dim", ctypes.c_int32)]


class _SamplingStruct(ctypes.Structure):
    """ctypes mirror of ``mxq_sampling`` (include/mxq.h)."""

    _fields_ = [("temperature", ctypes.c_void_p), ("top_k", ctypes.c_void_p), ("top_p", ctypes.c_void_p),
                ("min_p", ctypes.c_void_p), ("temperature_all", ctypes.c_float), ("top_k_all", ctypes.c_int32),
                ("top_p_all", ctypes.c_float), ("min_p_all", ctypes.c_float)]


_fn = None


def _load():
    """The library with this module's signatures declared (once)."""
    global _fn
    if _fn is None:
        lib = _lib.load()
        i64, i32, vp = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
        lib.mxq_rope.argtypes = ([vp, i64, i64] * 4) + [vp, vp, i64, i32, i32, i32, i32, i32, i32, vp]
        cache = ctypes.POINTER(_CacheStruct)
        lib.mxq_kv_append.argtypes = [cache, vp, i64, i64, vp, i64, i64, vp, i64, i64, vp, vp, i64, i64, i32, vp]
        lib.mxq_attention.argtypes = [vp, i64, i64, cache, vp, i64, i64, vp, vp, i64, i64, i32, i64, ctypes.c_float, vp,
                                      vp, i32, vp]
        lib.mxq_sample.argtypes = [vp, i64, i64, i64, i32, vp, ctypes.POINTER(_SamplingStruct), vp, vp, vp]
        for f in (lib.mxq_rope, lib.mxq_kv_append, lib.mxq_attention, lib.mxq_sample):
            f.restype = i32
        _fn = lib
    return _fn


# The current stream's handle without the Stream object around it (1.7 us of a call).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = torch.cuda.current_device
_empty_like = torch.empty_like


def _call(f, dev, stream, *args):
    """f(*args, stream) with `dev` current; raises on a status other than OK."""
    index = dev.index
    handle = _raw_stream(index) if stream is None else stream.cuda_stream
    if _current_device() == index:
        st = f(*args, handle)
    else:
        with torch.cuda.device(dev):
            st = f(*args, handle)
    if st:
        _lib._check(_fn, st)


def _elsewhere(who, dev, **tensors):
    """Names the tensor that is not on `dev`."""
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{who}: {name} must be on {dev}, is on {t.device}")


def _rows(who, name, t, dtype):
    """Strides of a [tokens, heads, dim] tensor with a contiguous last dimension."""
    s = t.stride()
    if t.dtype != dtype or len(s) != 3:
        raise TypeError(f"{who}: {name} must be a 3-D {str(dtype).replace('torch.', '')} tensor [tokens, heads, dim]")
    if s[2] != 1 and t.shape[2] > 1:
        raise ValueError(f"{who}: {name}'s last dimension must be contiguous")
    return s


def _ints(who, name, t, shape):
    if t.dtype != _i32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{who}: {name} must be a contiguous int32 tensor of shape {list(shape)}")


def _device(who, name, t):
    if not t.is_cuda:
        raise ValueError(f"{who}: {name} must be a device tensor")
    return t.device


def mxq_rope(q, k, inv_freq, positions, q_out=None, k_out=None, *, interleaved: bool = False, stream=None):
    """q and k [tokens, heads, dim] (f16 or bf16) rotated by position; returns the rotated pair.

    The first ``2 * len(inv_freq)`` values of each head turn by
    ``positions[t] * inv_freq[i]``: neighbours as pairs if ``interleaved``, else
    the two halves; the rest is copied.  Token and head strides are free.
    ``q_out`` and ``k_out`` may be ``q`` and ``k``.  ``k`` may be None."""
    who = "mxq_rope"
    dtype, dev = q.dtype, q.device
    code = _HALF.get(dtype)
    if not q.is_cuda or code is None:
        _device(who, "q", q)
        raise TypeError(f"{who}: q must be float16 or bfloat16")
    qs = _rows(who, "q", q, dtype)
    n, heads, dim = q.shape
    if inv_freq.dtype != _f32 or inv_freq.dim() != 1 or not inv_freq.is_contiguous():
        raise ValueError(f"{who}: inv_freq must be a contiguous float32 vector")
    rot = 2 * inv_freq.shape[0]
    if rot > dim:
        raise ValueError(f"{who}: {rot // 2} frequencies rotate {rot} values, a head has {dim}")
    if positions.dtype != _i32 or positions.shape != (n,) or not positions.is_contiguous():
        _ints(who, "positions", positions, (n,))
    if inv_freq.device != dev or positions.device != dev:
        _elsewhere(who, dev, inv_freq=inv_freq, positions=positions)
    if q_out is None:
        q_out = _empty_like(q)   # q's type, shape, place and order of dimensions
        qo = q_out.stride()
    else:
        if q_out.shape != q.shape:
            raise ValueError(f"{who}: q_out must have q's shape")
        if q_out.device != dev:
            _elsewhere(who, dev, q_out=q_out)
        qo = _rows(who, "q_out", q_out, dtype)
    kv_heads, ks, ko, kp, kop = 0, (0, 0), (0, 0), None, None
    if k is not None:
        ks = _rows(who, "k", k, dtype)
        kn, kv_heads, kdim = k.shape
        if kn != n or kdim != dim:
            raise ValueError(f"{who}: k must be [{n}, kv_heads, {dim}]")
        if k.device != dev:
            _elsewhere(who, dev, k=k)
        if k_out is None:
            k_out = _empty_like(k)
            ko = k_out.stride()
        else:
            if k_out.shape != k.shape:
                raise ValueError(f"{who}: k_out must have k's shape")
            if k_out.device != dev:
                _elsewhere(who, dev, k_out=k_out)
            ko = _rows(who, "k_out", k_out, dtype)
        kp, kop = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None:
        raise ValueError(f"{who}: k_out without k")
    _call(_load().mxq_rope, dev, stream, q.data_ptr(), qs[0], qs[1], kp, ks[0], ks[1], q_out.data_ptr(), qo[0], qo[1],
          kop, ko[0], ko[1], inv_freq.data_ptr(), positions.data_ptr(), n, heads, kv_heads, dim, rot,
          1 if interleaved else 0, code)
    return q_out, k_out


class KvCache:
    """A paged key/value cache held in 8 bits; a code c stands for c * scale.

    ``k`` int8 [blocks, kv_heads, block, dim], ``v`` int8 [blocks, kv_heads, dim, block],
    ``k_scale`` and ``v_scale`` float32 [blocks, kv_heads], contiguous, on one device;
    block 16, 32, 64 or 128, dim 64 or 128.  A sequence's tokens ``j * block ..`` are in
    the page ``table[s, j]`` of the table that the calls take.  The tensors are read-only
    attributes: the calls work on the memory that the cache was made of."""

    __slots__ = ("_tensors", "_device", "_struct")

    def __init__(self, k, v, k_scale, v_scale):
        if k.dtype != torch.int8 or k.dim() != 4 or v.dtype != torch.int8 or v.dim() != 4:
            raise TypeError("KvCache: k and v must be 4-D int8 tensors")
        blocks, kv_heads, block, dim = k.shape
        if v.shape != (blocks, kv_heads, dim, block):
            raise ValueError(f"KvCache: v must be [blocks, kv_heads, dim, block] = {[blocks, kv_heads, dim, block]}")
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            if t.dtype != _f32 or t.shape != (blocks, kv_heads):
                raise ValueError(f"KvCache: {name} must be float32 {[blocks, kv_heads]}")
        dev = _device("KvCache", "k", k)
        for name, t in (("k", k), ("v", v), ("k_scale", k_scale), ("v_scale", v_scale)):
            if t.device != dev or not t.is_contiguous():
                raise ValueError(f"KvCache: {name} must be contiguous and on {dev}")
        if block not in (16, 32, 64, 128) or dim not in (64, 128):
            raise ValueError(f"KvCache: block must be 16, 32, 64 or 128 and dim 64 or 128, got {block} and {dim}")
        self._tensors, self._device = (k, v, k_scale, v_scale), dev
        self._struct = _CacheStruct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), blocks,
                                    kv_heads, block, dim)

    @classmethod
    def empty(cls, blocks: int, kv_heads: int, block: int, dim: int, device="cuda"):
        """A cache of zero codes and scales."""
        return cls(torch.zeros((blocks, kv_heads, block, dim), dtype=torch.int8, device=device),
                   torch.zeros((blocks, kv_heads, dim, block), dtype=torch.int8, device=device),
                   torch.zeros((blocks, kv_heads), dtype=_f32, device=device),
                   torch.zeros((blocks, kv_heads), dtype=_f32, device=device))

    @property
    def k(self):
        return self._tensors[0]

    @property
    def v(self):
        return self._tensors[1]

    @property
    def k_scale(self):
        return self._tensors[2]

    @property
    def v_scale(self):
        return self._tensors[3]

    @property
    def device(self):
        return self._device

    @property
    def blocks(self):
        return self._struct.blocks

    @property
    def kv_heads(self):
        return self._struct.kv_heads

    @property
    def block(self):
        return self._struct.block

    @property
    def dim(self):
        return self._struct.dim


def _paging(who, dev, table, lens, starts, tokens):
    """(seqs, table row stride, width, starts pointer) of checked paging tensors."""
    if table.dtype != _i32 or table.dim() != 2:
        raise TypeError(f"{who}: table must be a 2-D int32 tensor [sequences, pages]")
    seqs, width = table.shape
    row, one = table.stride()
    if (one != 1 and width > 1) or (row < width and seqs > 1):
        raise ValueError(f"{who}: table's rows must be contiguous")
    if lens.dtype != _i32 or lens.shape != (seqs,) or not lens.is_contiguous():
        _ints(who, "lens", lens, (seqs,))
    if starts is None:
        if tokens != seqs:
            raise ValueError(f"{who}: {tokens} tokens for {seqs} sequences need starts")
    else:
        _ints(who, "starts", starts, (seqs + 1,))
    if table.device != dev or lens.device != dev or (starts is not None and starts.device != dev):
        _elsewhere(who, dev, table=table, lens=lens, starts=starts)
    return seqs, row, width, None if starts is None else starts.data_ptr()


def mxq_kv_append(cache, k, v, table, lens, starts=None, *, stream=None):
    """New keys and values [tokens, kv_heads, dim] (f16 or bf16) quantized into ``cache``, in place; returns it.

    Sequence s has ``lens[s]`` tokens with its new ones, the rows
    ``starts[s]:starts[s + 1]`` of k and v, or row s alone without ``starts``.
    The scheme, and what becomes of tokens without a page, is in include/mxq.h."""
    who = "mxq_kv_append"
    dev = cache._device
    code = _HALF.get(k.dtype)
    if code is None:
        raise TypeError(f"{who}: k must be float16 or bfloat16")
    ks, vs = _rows(who, "k", k, k.dtype), _rows(who, "v", v, k.dtype)
    n, heads, dim = k.shape
    st = cache._struct
    if k.shape != v.shape or heads != st.kv_heads or dim != st.dim:
        raise ValueError(f"{who}: k and v must be [tokens, {st.kv_heads}, {st.dim}]")
    if k.device != dev or v.device != dev:
        _elsewhere(who, dev, k=k, v=v)
    seqs, row, width, sp = _paging(who, dev, table, lens, starts, n)
    _call(_load().mxq_kv_append, dev, stream, st, k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1],
          table.data_ptr(), row, width, lens.data_ptr(), sp, n, seqs, code)
    return cache


def mxq_attention(q, cache, table, lens, starts=None, out=None, *, window: int = 0, scale: float | None = None,
                  return_lse: bool = False, stream=None):
    """Causal attention of q [tokens, heads, dim] (f16 or bf16) over ``cache``, which holds the new tokens already.

    Sequences and their rows as in ``mxq_kv_append``.  ``window`` > 0: the last
    that many keys of each token; ``scale``: 1 / sqrt(dim) if None.  Returns out
    [tokens, heads, dim] in q's type, or (out, lse) with the log-sums float32
    [tokens, heads].  A row without keys gives 0 and -inf."""
    who = "mxq_attention"
    dev = cache._device
    code = _HALF.get(q.dtype)
    if code is None:
        raise TypeError(f"{who}: q must be float16 or bfloat16")
    qs = _rows(who, "q", q, q.dtype)
    n, heads, dim = q.shape
    st = cache._struct
    if dim != st.dim:
        raise ValueError(f"{who}: q's heads have {dim} values, the cache's {st.dim}")
    if q.device != dev:
        _elsewhere(who, dev, q=q)
    seqs, row, width, sp = _paging(who, dev, table, lens, starts, n)
    if out is None:
        out = _empty_like(q) if q.is_contiguous() else q.new_empty(q.shape)
    elif out.dtype != q.dtype or out.shape != q.shape or not out.is_contiguous() or out.device != dev:
        raise ValueError(f"{who}: out must be a contiguous tensor of q's shape and type on {dev}")
    lse = torch.empty((n, heads), dtype=_f32, device=dev) if return_lse else None
    _call(_load().mxq_attention, dev, stream, q.data_ptr(), qs[0], qs[1], st, table.data_ptr(), row, width, lens.data_ptr(), sp,
          n, seqs, heads, window, dim ** -0.5 if scale is None else scale, out.data_ptr(),
          None if lse is None else lse.data_ptr(), code)
    return (out, lse) if return_lse else out


def _setting(who, name, value, rows, dtype, dev):
    """(pointer, value for all) of a setting given as a tensor of one value a row, or as a number."""
    if isinstance(value, torch.Tensor):
        if value.dtype != dtype or value.shape != (rows,) or not value.is_contiguous() or value.device != dev:
            raise ValueError(f"{who}: {name} must be a number or a contiguous "
                             f"{str(dtype).replace('torch.', '')} tensor [{rows}] on {dev}")
        return value.data_ptr(), 0
    # (ctypes keeps an int's low 32 bits)
    return None, min(max(value, -1), 0x7FFFFFFF) if dtype == _i32 else value


def mxq_sample(logits, u, tokens=None, probs=None, *, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, stream=None):
    """One token for each row of ``logits`` [rows, vocab] (f16, bf16 or f32), drawn by the uniform numbers ``u`` [rows].

    ``temperature`` (<= 0: the largest logit), ``top_k`` (<= 0: off), ``top_p`` (>= 1: off) and ``min_p`` (<= 0: off)
    are numbers, or tensors of one value a row (float32; top_k int32).  Returns (tokens int32, probs float32), each
    token's probability being that among the kept ones.  The rule, ties included, is in include/mxq.h."""
    who = "mxq_sample"
    dev = _device(who, "logits", logits)
    code = _LOGITS.get(logits.dtype)
    if code is None or logits.dim() != 2:
        raise TypeError(f"{who}: logits must be a 2-D float16, bfloat16 or float32 tensor [rows, vocab]")
    rows, vocab = logits.shape
    row, one = logits.stride()
    if one != 1 and vocab > 1:
        raise ValueError(f"{who}: logits' rows must be contiguous")
    if u.dtype != _f32 or u.shape != (rows,) or not u.is_contiguous() or u.device != dev:
        raise ValueError(f"{who}: u must be a contiguous float32 tensor [{rows}] on {dev}")
    t, t_all = _setting(who, "temperature", temperature, rows, _f32, dev)
    k, k_all = _setting(who, "top_k", top_k, rows, _i32, dev)
    p, p_all = _setting(who, "top_p", top_p, rows, _f32, dev)
    m, m_all = _setting(who, "min_p", min_p, rows, _f32, dev)
    if tokens is None:
        tokens = _empty_like(u, dtype=_i32)
    else:
        _ints(who, "tokens", tokens, (rows,))
    if probs is None:
        probs = _empty_like(u)
    elif probs.dtype != _f32 or probs.shape != (rows,) or not probs.is_contiguous():
        raise ValueError(f"{who}: probs must be a contiguous float32 tensor [{rows}]")
    if tokens.device != dev or probs.device != dev:
        _elsewhere(who, dev, tokens=tokens, probs=probs)
    _call(_load().mxq_sample, dev, stream, logits.data_ptr(), row, rows, vocab, code, u.data_ptr(),
          _SamplingStruct(t, k, p, m, t_all, k_all, p_all, m_all), tokens.data_ptr(), probs.data_ptr())
    return tokens, probs
