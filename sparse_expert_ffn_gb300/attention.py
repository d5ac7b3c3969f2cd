"""Attention operators of a pre-norm decoder block (``include/colibri_attn.h``).

Argument marshalling only: the work is done by the CUDA library.  What a
program keeps between calls is described once, by :class:`PagedKVCache`,
:class:`Sequences` and :class:`Rope` over the program's own tensors; the
functions then take row tensors ``[rows, heads, head_dim]`` (any row stride)
and run on the tensors' device and its current stream (or ``stream``):

* :func:`append_qkv`, :func:`qk_norm_rope`: per-head norms, rotary positions
  and the write into the cache in one pass;
* :func:`attention_prompt`, :func:`attention_prompt_paged`: packed sequences of
  different lengths, grouped heads, causal or full;
* :func:`attention_decode`: one row per sequence, with a shared prefix;
* :func:`check`: whether a kernel's bounded wait has given up.

Results carry no gradient: the operators have no backward pass, and inputs that
require one are read like any others.
"""

from __future__ import annotations

import ctypes
import os
import threading
from typing import Optional

import torch

import sparse_expert_ffn_gb300 as _sef

_STYLE = {"half": 0, "interleaved": 1}
_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
_DTYPE = {torch.float32: _sef.DTYPE_FP32, torch.bfloat16: _sef.DTYPE_BF16}

KVPages, Seqs, RopeArgs = _sef.ColibriKVPages, _sef.ColibriSeqs, _sef.ColibriRope


def _int32(t, name, dim, device=None):
    if t.dtype != torch.int32 or t.dim() != dim or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA int32 tensor with {dim} dimension(s)")
    if device is not None and t.device != device:
        raise ValueError(f"{name} must be on {device}")


def rope_frequencies(rot_dim: int, theta: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     trained: int = 4096, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """(freq [rot_dim / 2] float64 CPU tensor, mscale) of ``colibri_rope_frequencies``:
    radians per position, for contexts ``factor`` times the trained one
    ("linear", "ntk", "yarn")."""
    if scaling not in _SCALING:
        raise ValueError(f"scaling must be one of {sorted(_SCALING)}")
    freq = torch.empty(max(int(rot_dim), 0) // 2, dtype=torch.float64)
    mscale = ctypes.c_float()
    _sef._check(_sef.library().colibri_rope_frequencies(
        int(rot_dim), float(theta), _SCALING[scaling], float(factor), int(trained), float(beta_fast),
        float(beta_slow), freq.data_ptr() or None, ctypes.byref(mscale)), "colibri_rope_frequencies")
    return freq, mscale.value


class Rope:
    """Rotary positions: ``freq`` [rot_dim / 2] float64 on the GPU (radians per
    position), pairing ``style`` "half" or "interleaved", ``mscale`` the factor
    of cos and sin."""

    def __init__(self, freq, style: str = "half", mscale: float = 1.0):
        if freq.dtype != torch.float64 or freq.dim() != 1 or not freq.is_cuda or not freq.is_contiguous():
            raise ValueError("freq must be a contiguous CUDA float64 vector")
        self.freq, self.device = freq, freq.device
        self._c = RopeArgs(freq.data_ptr(), 2 * freq.numel(), _STYLE[style], float(mscale))
        self._ref = ctypes.byref(self._c)


class PagedKVCache:
    """Keys and values in pages: ``k`` and ``v`` [pages, kv_heads, page_size,
    head_dim] with the same strides, the last dimension contiguous (a
    ``transpose(1, 2)`` of [pages, page_size, kv_heads, head_dim] storage
    serves as well).  The program owns the tensors and hands out the pages."""

    def __init__(self, k, v):
        if k.dim() != 4 or k.shape != v.shape or k.stride() != v.stride() or k.stride(3) != 1:
            raise ValueError("k and v must be [pages, kv_heads, page_size, head_dim] with equal strides "
                             "and a contiguous last dimension")
        if k.dtype not in _DTYPE or v.dtype != k.dtype or not k.is_cuda or v.device != k.device:
            raise ValueError("k and v must be float32 or bfloat16 tensors of one CUDA device")
        self.k, self.v, self.dtype, self.device = k, v, k.dtype, k.device
        self.num_pages, self.n_kv_heads, self.page_size, self.head_dim = k.shape
        self._c = KVPages(k.data_ptr(), v.data_ptr(), k.stride(0), k.stride(1), k.stride(2), k.shape[0],
                          k.shape[2], k.shape[1], k.shape[3], _DTYPE[k.dtype])
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, num_pages: int, page_size: int, n_kv_heads: int, head_dim: int,
              dtype=torch.bfloat16, device="cuda"):
        shape = (num_pages, n_kv_heads, page_size, head_dim)
        return cls(torch.empty(shape, dtype=dtype, device=device), torch.empty(shape, dtype=dtype, device=device))


class Sequences:
    """The sequences of a call (int32 CUDA tensors, read on the device at every
    call, so their contents may change between calls): ``seq_start`` [B + 1]
    first rows (None: row b is sequence b), ``kv_len`` [B] keys including the
    call's rows (None: the sequence's rows), ``page_table`` [B, width] page ids
    (None: no cache)."""

    def __init__(self, seq_start=None, kv_len=None, page_table=None):
        given = [t for t in (seq_start, kv_len, page_table) if t is not None]
        if not given or (seq_start is None and kv_len is None):
            raise ValueError("seq_start or kv_len must be given")
        self.device = given[0].device
        for t, name, dim in ((seq_start, "seq_start", 1), (kv_len, "kv_len", 1)):
            if t is not None:
                _int32(t, name, dim, self.device)
        if page_table is not None:
            _int32(page_table, "page_table", 2, self.device)
        n = kv_len.shape[0] if kv_len is not None else seq_start.shape[0] - 1
        if n < 0 or (seq_start is not None and seq_start.shape[0] != n + 1) or \
                (page_table is not None and page_table.shape[0] != n):
            raise ValueError("seq_start [B + 1], kv_len [B] and page_table [B, width] must agree on B")
        self.n_seqs = n
        self.seq_start, self.kv_len, self.page_table = seq_start, kv_len, page_table
        self._args = (_sef._ptr(seq_start), _sef._ptr(kv_len), _sef._ptr(page_table), n)
        self._last = (None, None)

    def _rows(self, t):
        """The C description for a call with t's rows (never changed once made:
        two threads may call with one object)."""
        rows = t.shape[0]
        last = self._last
        if last[0] != rows:
            if self.seq_start is None and rows != self.n_seqs:
                raise ValueError("without seq_start there is one row per sequence")
            width = 0 if self.page_table is None else self.page_table.shape[1]
            last = self._last = (rows, ctypes.byref(Seqs(*self._args, rows, width)))
        return last[1]


def _same(t, name, heads, head_dim, dtype, device, rows):
    """Checks a row tensor; returns its row stride."""
    if t.shape != (rows, heads, head_dim) or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name} must be [{rows}, {heads}, {head_dim}], {dtype}, on {device}")
    s0, s1, s2 = t.stride()
    if s2 != 1 or (heads > 1 and s1 != head_dim):
        raise ValueError(f"{name}'s heads must be contiguous")
    return s0 if rows > 1 else heads * head_dim


def _norm(w, name, head_dim, dtype, device):
    if w is None:
        return None
    if tuple(w.shape) != (head_dim,) or w.dtype != dtype or w.device != device or not w.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [{head_dim}] {dtype} vector on {device}")
    return w.data_ptr()


_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


_capturing = torch.cuda.is_current_stream_capturing


def _stream(stream, device):
    """The stream to run on: the device's current one by default."""
    if stream is None:
        return _raw_stream(device.index)
    if stream.device != device:
        raise ValueError(f"the stream must be on {device}")
    return stream.cuda_stream


def _empty(shape, dtype, device, stream):
    """A tensor for a call on `stream`, allocated there: its memory may have
    belonged to a tensor that work on another stream still uses."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _on(device, call, what, *args):
    """The C call with the tensors' device current."""
    prev = _current_device()
    if prev == device.index:
        status = call(*args)
    else:
        torch.cuda.set_device(device.index)
        try:
            status = call(*args)
        finally:
            torch.cuda.set_device(prev)
    if status:
        _sef._check(status, what)


def _rope_ref(rope, device):
    if rope is None:
        return None
    if rope.device != device:
        raise ValueError(f"rope.freq must be on {device}")
    return rope._ref


def _rows3(q):
    if q.dim() != 3 or q.dtype not in _DTYPE or not q.is_cuda:
        raise ValueError("q must be a [rows, heads, head_dim] float32 or bfloat16 CUDA tensor")


def append_qkv(cache: PagedKVCache, seqs: Sequences, q, k, v, *, rope: Optional[Rope] = None, q_norm=None,
               k_norm=None, eps: float = 1e-6, q_out=None, stream=None):
    """Normalise (q_norm / k_norm given) and rotate (rope given) the rows' query
    and key heads; keys and values go to their places in the cache, the queries
    to ``q_out`` (a new tensor by default, may be ``q``), which is returned."""
    _rows3(q)
    dev, dt, D, rows = cache.device, cache.dtype, cache.head_dim, q.shape[0]
    hq, hkv = q.shape[1], cache.n_kv_heads
    if seqs.device != dev:
        raise ValueError(f"seqs must be on {dev}")
    if q_out is None:
        q_out = _empty((rows, hq, D), dt, dev, stream)
    args = (_rope_ref(rope, dev), hq, q.data_ptr(), _same(q, "q", hq, D, dt, dev, rows),
            k.data_ptr(), _same(k, "k", hkv, D, dt, dev, rows), v.data_ptr(), _same(v, "v", hkv, D, dt, dev, rows),
            _norm(q_norm, "q_norm", D, dt, dev), _norm(k_norm, "k_norm", D, dt, dev), float(eps),
            q_out.data_ptr(), _same(q_out, "q_out", hq, D, dt, dev, rows))
    if rows == 0:
        return q_out
    _on(dev, _sef.library().colibri_append_qkv, "colibri_append_qkv", cache._ref, seqs._rows(q), *args,
        _stream(stream, dev))
    return q_out


def qk_norm_rope(seqs: Sequences, q, k, *, rope: Optional[Rope] = None, q_norm=None, k_norm=None,
                 eps: float = 1e-6, q_out=None, k_out=None, stream=None):
    """:func:`append_qkv` for rows that go to no cache; returns (q_out, k_out)."""
    _rows3(q)
    dev, dt, D, rows, hq, hkv = q.device, q.dtype, q.shape[2], q.shape[0], q.shape[1], k.shape[1]
    if seqs.device != dev:
        raise ValueError(f"seqs must be on {dev}")
    if q_out is None:
        q_out = _empty((rows, hq, D), dt, dev, stream)
    if k_out is None:
        k_out = _empty((rows, hkv, D), dt, dev, stream)
    args = (_rope_ref(rope, dev), hq, hkv, D, _DTYPE[dt], q.data_ptr(), _same(q, "q", hq, D, dt, dev, rows),
            k.data_ptr(), _same(k, "k", hkv, D, dt, dev, rows),
            _norm(q_norm, "q_norm", D, dt, dev), _norm(k_norm, "k_norm", D, dt, dev), float(eps),
            q_out.data_ptr(), _same(q_out, "q_out", hq, D, dt, dev, rows),
            k_out.data_ptr(), _same(k_out, "k_out", hkv, D, dt, dev, rows))
    if rows == 0:
        return q_out, k_out
    _on(dev, _sef.library().colibri_qk_norm_rope, "colibri_qk_norm_rope", seqs._rows(q), *args,
        _stream(stream, dev))
    return q_out, k_out


def _outputs(q, out, lse, stream):
    rows, hq, D = q.shape
    if out is None:
        out = _empty((rows, hq, D), q.dtype, q.device, stream)
    if lse is not None and (tuple(lse.shape) != (rows, hq) or lse.dtype != torch.float32 or
                            lse.device != q.device or not lse.is_contiguous()):
        raise ValueError(f"lse must be a contiguous [{rows}, {hq}] float32 tensor on {q.device}")
    return out, (None if lse is None else lse.data_ptr()), _same(out, "out", hq, D, q.dtype, q.device, rows)


# what os.environ holds, without the microsecond that a look-up through it takes
_env = getattr(os.environb, "_data", os.environb)
_waits = (None, None)


def _pass_on_waits():
    """Hands the two variables of failure detection to the library when they have
    changed: it reads the environment itself only once."""
    global _waits
    now = (_env.get(b"COLIBRI_WAIT_LIMIT_NS"), _env.get(b"COLIBRI_TEST_STALL_TMA"))
    if now != _waits:
        _sef._check(_sef.library().colibri_attention_waits(*(int(v or 0) for v in now)), "colibri_attention_waits")
        _waits = now


class _Kept(threading.local):
    place, tensor = None, None


_kept = _Kept()
_KEPT_BYTES = 1 << 24


def _workspace(nbytes, device, stream):
    """A call's workspace.  Calls on the current stream take a small one from the
    thread's last call there: the thread's calls follow each other on the stream,
    as their uses of a block that the caching allocator hands out again would, and a
    step of a few tokens takes 12 us of the host instead of 17.  Other threads,
    streams and devices, and graphs that are being captured, have their own.  It is
    kept, up to 16 MB, until the thread calls on another stream, needs a larger one, or
    ends; calls that need more (single rows of groups from 14 heads of 128 on) have
    theirs from the caching allocator every time."""
    if not nbytes:
        return None
    if stream is not None or nbytes > _KEPT_BYTES or _current_device() != device.index or _capturing():
        return _empty(nbytes, torch.uint8, device, stream)
    place = (device.index, _raw_stream(device.index))
    if _kept.place != place or _kept.tensor.numel() < nbytes:
        _kept.place, _kept.tensor = None, None
        _kept.tensor = torch.empty(nbytes, dtype=torch.uint8, device=device)
        _kept.place = place
    return _kept.tensor


def _prompt(kv, kv_ref, seqs, q, scale, causal, out, lse, stream):
    _rows3(q)
    dev, rows, hq, D = q.device, q.shape[0], q.shape[1], q.shape[2]
    if seqs.device != dev or kv.device != dev:
        raise ValueError(f"keys and seqs must be on {dev}")
    if q.dtype != kv.dtype or D != kv.head_dim:
        raise ValueError("q and the keys must share dtype and head_dim")
    stride = _same(q, "q", hq, D, q.dtype, dev, rows)
    out, lse_ptr, o_stride = _outputs(q, out, lse, stream)
    if rows == 0:
        return out
    ref, lib, need = seqs._rows(q), _sef.library(), ctypes.c_size_t()
    _sef._check(lib.colibri_attention_prompt_workspace(kv_ref, ref, hq, ctypes.byref(need)),
                "colibri_attention_prompt_workspace")
    ws = _workspace(need.value, dev, stream)
    _pass_on_waits()
    _on(dev, lib.colibri_attention_prompt, "colibri_attention_prompt", kv_ref, ref, hq, q.data_ptr(), stride,
        D ** -0.5 if scale is None else float(scale), int(causal), out.data_ptr(), o_stride, lse_ptr,
        None if ws is None else ws.data_ptr(), need.value, _stream(stream, dev))
    return out


class _Packed:
    """k and v rows [rows, kv_heads, head_dim] as one page."""

    def __init__(self, k, v):
        rows, hkv, D = k.shape
        sk = _same(k, "k", hkv, D, k.dtype, k.device, rows)
        if _same(v, "v", hkv, D, k.dtype, k.device, rows) != sk:
            raise ValueError("k and v must have the same row stride")
        self.dtype, self.device, self.head_dim = k.dtype, k.device, D
        self._c = KVPages(k.data_ptr(), v.data_ptr(), max(rows, 1) * sk, D, sk, 1, max(rows, 1), hkv, D,
                          _DTYPE.get(k.dtype, -1))


def attention_prompt(seqs: Sequences, q, k, v, *, scale: Optional[float] = None, causal: bool = True, out=None,
                     lse=None, stream=None):
    """Attention of packed sequences over their own rows: q [rows, heads,
    head_dim], k and v [rows, kv_heads, head_dim], sequence b at rows
    seq_start[b] .. seq_start[b + 1] - 1 (seqs without kv_len and page_table).
    scale defaults to head_dim ** -0.5; lse [rows, heads] float32 receives the
    logarithms of the softmax sums.  Rows of no sequence are left as they were."""
    if seqs.page_table is not None or seqs.kv_len is not None:
        raise ValueError("packed keys take Sequences(seq_start); use attention_prompt_paged with a cache")
    if k.dim() != 3 or v.dim() != 3 or k.shape[0] != q.shape[0]:
        raise ValueError("k and v must be [rows, kv_heads, head_dim] with q's rows")
    kv = _Packed(k, v)
    return _prompt(kv, ctypes.byref(kv._c), seqs, q, scale, causal, out, lse, stream)


def attention_prompt_paged(cache: PagedKVCache, seqs: Sequences, q, *, scale: Optional[float] = None,
                           causal: bool = True, out=None, lse=None, stream=None):
    """:func:`attention_prompt` over a cache's pages (seqs with kv_len and
    page_table): row i of n of sequence b stands at position kv_len[b] - n + i."""
    if seqs.page_table is None or seqs.kv_len is None:
        raise ValueError("seqs needs kv_len and page_table")
    return _prompt(cache, cache._ref, seqs, q, scale, causal, out, lse, stream)


def attention_decode(cache: PagedKVCache, seqs: Sequences, q, *, prefix_len: int = 0, prefix_table=None,
                     scale: Optional[float] = None, out=None, lse=None, stream=None):
    """Attention of one row per sequence (q [B, heads, head_dim]) over its
    kv_len[b] keys.  The first prefix_len keys (a multiple of the page size) of
    every sequence are those of prefix_table [prefix_len / page_size], read once
    for the batch."""
    _rows3(q)
    dev, rows, hq, D = q.device, q.shape[0], q.shape[1], q.shape[2]
    if seqs.page_table is None or seqs.kv_len is None or seqs.seq_start is not None:
        raise ValueError("seqs needs kv_len and page_table, and no seq_start")
    if seqs.device != dev or cache.device != dev:
        raise ValueError(f"the cache and seqs must be on {dev}")
    if q.dtype != cache.dtype or D != cache.head_dim:
        raise ValueError("q and the cache must share dtype and head_dim")
    table = None
    if prefix_table is not None:
        _int32(prefix_table, "prefix_table", 1, dev)
        if prefix_table.shape[0] * cache.page_size < prefix_len:
            raise ValueError("prefix_table is shorter than the prefix")
        table = prefix_table.data_ptr() if prefix_len else None
    stride = _same(q, "q", hq, D, q.dtype, dev, rows)
    out, lse_ptr, o_stride = _outputs(q, out, lse, stream)
    if rows == 0:
        return out
    ref, lib, need = seqs._rows(q), _sef.library(), ctypes.c_size_t()
    _sef._check(lib.colibri_attention_decode_workspace(cache._ref, ref, hq, int(prefix_len), ctypes.byref(need)),
                "colibri_attention_decode_workspace")
    ws = _workspace(need.value, dev, stream)
    _pass_on_waits()
    _on(dev, lib.colibri_attention_decode, "colibri_attention_decode", cache._ref, ref, hq, q.data_ptr(), stride,
        D ** -0.5 if scale is None else float(scale), int(prefix_len), table, out.data_ptr(), o_stride, lse_ptr,
        None if ws is None else ws.data_ptr(), need.value, _stream(stream, dev))
    return out


def check(stream=None, device=None) -> int:
    """Wait for the stream (the current one of ``device``, by default the current
    device); returns the library status: ``ERR_TIMEOUT`` when a wait of an attention
    kernel on the device gave up since the last check and left rows of NaN, 0 = OK."""
    if device is None:
        device = torch.device("cuda", torch.cuda.current_device()) if stream is None else stream.device
    device = torch.device(device)
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(device):
        return _sef.library().colibri_attention_check(_stream(stream, device))
