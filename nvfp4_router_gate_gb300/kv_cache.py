"""The paged NVFP4 key/value cache: Python binding of include/nvfp4_kv_cache.h.

* ``nvfp4_kv_append(q, k, v, positions, slots, cos, sin, cache, k_gsa, v_gsa, ...)`` -> q_out
* ``nvfp4_kv_attention(q, cache, page_table, kv_lens, k_gsa, v_gsa, ...)`` -> (out, lse)
* ``nvfp4_kv_gather(cache, slots, k_gsa, v_gsa, ...)`` -> (k, v)
* ``rope_table(n_pos, rot, ...)`` -> (cos, sin), plain, interpolated or scaled by parts

``Nvfp4KVCache`` keeps the pages, the global scales and the attention
workspace resident: its calls allocate nothing but outputs the caller does not
pass (CUDA-graph capturable).  What a call with ``stream=`` allocates belongs to
that stream.
"""

import contextlib
import math

import torch

from . import _dtype_code, _resident_workspace, new_workspace, nvr_read_device_status
from . import _native

_BF16, _F32, _I32, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.uint8
_empty = torch.empty


def _on(stream):
    if not isinstance(stream, torch.cuda.Stream):
        stream = torch.cuda.ExternalStream(stream.cuda_stream)
    return torch.cuda.stream(stream)


def _empty_on(stream, shape, **kw):
    with _on(stream):
        return _empty(shape, **kw)


def nvfp4_kv_page_bytes(page_size, D):
    """Bytes of one page of one KV head; 0 for an unsupported size."""
    return int(_native.lib().nvfp4_kv_page_bytes(page_size, D))


def nvfp4_kv_attention_workspace_size(T_max, B_max, n_heads, n_kv_heads, D):
    return int(_native.lib().nvfp4_kv_attention_workspace_size(T_max, B_max, n_heads, n_kv_heads, D))


def _raw_stream(stream):
    """The stream's handle; the current stream of the current device for None
    (its handle straight from torch: a Stream object costs as much as a launch)."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _refuse(t, dtype, n, name):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.numel() != n:
        raise ValueError("%s has %d elements, not %d" % (name, t.numel(), n))
    raise ValueError("%s must be contiguous" % name)


def _ptr(t, dtype, n, name):
    """Pointer of a contiguous CUDA tensor of n elements (None for None)."""
    if t is None:
        return None
    if t.dtype is not dtype or not t.is_cuda or t.numel() != n or not t.is_contiguous():
        _refuse(t, dtype, n, name)
    return t.data_ptr()


def _heads(t, T, H, D, name):
    """Pointer and token stride of t [T, H, D] with contiguous heads."""
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    s0, s1, s2 = t.stride()
    if s2 != 1 or (s1 != D and H > 1):
        raise ValueError("%s must have contiguous heads (a token stride is allowed)" % name)
    return t.data_ptr(), (s0 if T > 1 else H * D)


class _Pages:
    """A cache's geometry and pointers (and the tensors behind them): checked
    once, used by every call."""

    def __init__(self, cache, k_gsa, v_gsa, D):
        self.tensors = cache, k_gsa, v_gsa
        if cache.dtype != _U8 or cache.dim() != 3:
            raise TypeError("cache must be uint8 [n_pages, n_kv_heads, page_bytes]")
        self.n_pages, self.Hkv, nbytes = cache.shape
        self.D, self.S = D, nbytes * 8 // (9 * max(D, 1))
        if nbytes == 0 or nvfp4_kv_page_bytes(self.S, D) != nbytes:
            raise ValueError("no page_size has pages of %d bytes for heads of %d channels" % (nbytes, D))
        self.data = _ptr(cache, _U8, cache.numel(), "cache")
        self.lib = _native.lib()
        self.k_gsa, self.v_gsa = _ptr(k_gsa, _F32, self.Hkv, "k_gsa"), _ptr(v_gsa, _F32, self.Hkv, "v_gsa")


def _append(pages, q, k, v, positions, slots, cos, sin, q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
            q_out=None, stream=None):
    shape, dt = k.shape, k.dtype
    T, Hkv, D = shape
    if v.shape != shape or v.dtype is not dt:
        raise ValueError("k and v must have one shape and type")
    if Hkv != pages.Hkv or D != pages.D:
        raise ValueError("the cache holds %d KV heads of %d channels, k has %d of %d" % (pages.Hkv, pages.D, Hkv, D))
    kp, ks = _heads(k, T, Hkv, D, "k")
    vp, vs = _heads(v, T, Hkv, D, "v")
    Hq, qp, qs, op = 0, None, 0, None
    if q is not None:
        if q.dim() != 3 or q.dtype is not dt:
            raise ValueError("q must be [T, heads, D] of k's type")
        Tq, Hq, Dq = q.shape
        if Tq != T or Dq != D:
            raise ValueError("q must be [T, heads, D] of k's type")
        qp, qs = _heads(q, T, Hq, D, "q")
        if q_out is None:
            q_out = (_empty((T, Hq, D), dtype=_BF16, device=k.device) if stream is None else
                     _empty_on(stream, (T, Hq, D), dtype=_BF16, device=k.device))
            op = q_out.data_ptr()
        else:
            op = _ptr(q_out, _BF16, T * Hq * D, "q_out")
    rot = n_pos = 0
    if cos is not None:
        n_pos, half = cos.shape
        rot = 2 * half
        if sin is None or positions is None:
            raise ValueError("cos needs sin and positions")
    n = n_pos * rot // 2
    st = pages.lib.nvfp4_kv_append(
        qp, qs, kp, ks, vp, vs, _dtype_code(k), T, Hq, Hkv, D,
        _ptr(positions, _I32, T, "positions") if rot else None, _ptr(slots, _I32, T, "slots"),
        _ptr(cos, _F32, n, "cos") if rot else None, _ptr(sin, _F32, n, "sin") if rot else None, n_pos, rot, interleaved,
        None if q_weight is None else _ptr(q_weight, _F32, D, "q_weight"),
        None if k_weight is None else _ptr(k_weight, _F32, D, "k_weight"), eps, pages.k_gsa, pages.v_gsa,
        pages.data, pages.n_pages, pages.S, op, _raw_stream(stream))
    if st:
        _native.check("nvfp4_kv_append", st)
    return q_out


def nvfp4_kv_append(q, k, v, positions, slots, cos, sin, cache, k_gsa, v_gsa, **kw):
    """RMS norm of the heads of q [T, Hq, D] and k [T, Hkv, D] (where q_weight,
    k_weight [D] are given, with eps=1e-6), rotary positions, and k and v
    quantized into the cache's slots.  cos and sin are [n_pos, rot/2] (None: no
    rotation), paired by halves or interleaved=True; returns q_out [T, Hq, D] bf16
    (None for q None)."""
    return _append(_Pages(cache, k_gsa, v_gsa, k.shape[2]), q, k, v, positions, slots, cos, sin, **kw)


def _gather(pages, slots, out_dtype=_BF16, k_out=None, v_out=None, stream=None):
    n, Hkv, D = slots.numel(), pages.Hkv, pages.D
    sp = _ptr(slots, _I32, n, "slots")
    if k_out is None and v_out is None:
        if out_dtype is not _BF16 and out_dtype is not _F32:
            raise TypeError("out_dtype must be bfloat16 or float32, got %s" % out_dtype)
        shape, dev = (n, Hkv, D), slots.device
        if stream is None:
            k_out, v_out = _empty(shape, dtype=out_dtype, device=dev), _empty(shape, dtype=out_dtype, device=dev)
        else:
            k_out, v_out = (_empty_on(stream, shape, dtype=out_dtype, device=dev) for _ in range(2))
        kp, vp = k_out.data_ptr(), v_out.data_ptr()
    elif k_out is None or v_out is None:
        raise ValueError("pass both k_out and v_out, or neither")
    else:
        m, dt = n * Hkv * D, k_out.dtype
        kp, vp = _ptr(k_out, dt, m, "k_out"), _ptr(v_out, dt, m, "v_out")
    st = pages.lib.nvfp4_kv_gather(pages.data, pages.n_pages, pages.S, Hkv, D, sp, n, pages.k_gsa, pages.v_gsa, kp, vp,
                                   _dtype_code(k_out), _raw_stream(stream))
    if st:
        _native.check("nvfp4_kv_gather", st)
    return k_out, v_out


def nvfp4_kv_gather(cache, slots, k_gsa, v_gsa, D, **kw):
    """The values that the slots stand for: k and v [n, Hkv, D] of out_dtype
    (bfloat16 or float32) or into k_out and v_out; zeros for a slot outside the
    cache."""
    return _gather(_Pages(cache, k_gsa, v_gsa, D), slots, **kw)


def _attend(pages, q, page_table, kv_lens, cu_q=None, max_q=None, scale=None, causal=True, window=0, out=None,
            lse=None, workspace=None, ws=None, stream=None):
    T, Hq, D = q.shape
    if D != pages.D:
        raise ValueError("the cache holds heads of %d channels, q has %d" % (pages.D, D))
    B, max_pages = page_table.shape
    if cu_q is None:
        if T % B if B else T:
            raise ValueError("%d queries for %d sequences: pass cu_q" % (T, B))
        max_q = T // B if B else 0
    elif max_q is None:
        raise ValueError("cu_q needs max_q, the most queries of a sequence")
    qp, qs = _heads(q, T, Hq, D, "q")
    if out is None:
        out = (_empty((T, Hq, D), dtype=_BF16, device=q.device) if stream is None else
               _empty_on(stream, (T, Hq, D), dtype=_BF16, device=q.device))
    if ws is None:
        nbytes = workspace.numel()
        ws = _ptr(workspace, _U8, nbytes, "workspace"), nbytes
    st = pages.lib.nvfp4_kv_attention(
        qp, qs, T, Hq, pages.Hkv, D, pages.data, pages.n_pages, pages.S,
        _ptr(page_table, _I32, B * max_pages, "page_table"), B, max_pages, _ptr(kv_lens, _I32, B, "kv_lens"),
        None if cu_q is None else _ptr(cu_q, _I32, B + 1, "cu_q"), max_q, pages.k_gsa, pages.v_gsa, D ** -0.5 if scale is None else scale,
        causal, window, _ptr(out, _BF16, T * Hq * D, "out"), None if lse is None else _ptr(lse, _F32, T * Hq, "lse"), ws[0], ws[1],
        _raw_stream(stream))
    if st:
        _native.check("nvfp4_kv_attention", st)
    return out, lse


def nvfp4_kv_attention(q, cache, page_table, kv_lens, k_gsa, v_gsa, workspace=None, stream=None, **kw):
    """Attention of q [T, Hq, D] bf16 over the cached tokens of the sequences
    in page_table [B, max_pages] and kv_lens [B].  cu_q [B + 1] (with max_q, the
    most queries of a sequence) gives each sequence's rows of q; without it every
    sequence has T / B queries.  scale defaults to D ** -0.5, causal to True,
    window to 0 (none).  Returns (out [T, Hq, D] bf16, lse); lse [T, Hq] fp32 is
    written when it is given."""
    T, Hq, D = q.shape
    if q.dtype is not _BF16:
        raise TypeError("q must be bfloat16, got %s" % q.dtype)
    if workspace is None:
        # (zeroed on the stream that uses it)
        with _on(stream) if stream is not None else contextlib.nullcontext():
            workspace = new_workspace(nvfp4_kv_attention_workspace_size(T, page_table.shape[0], Hq, cache.shape[1], D),
                                      q.device)
    return _attend(_Pages(cache, k_gsa, v_gsa, D), q, page_table, kv_lens, workspace=workspace, stream=stream, **kw)


class Nvfp4KVCache:
    """Resident paged NVFP4 key/value cache of one layer.

    ``k_gsa`` and ``v_gsa`` are the global scales (a number or [n_kv_heads]
    fp32, max|x| / 2688 of calibration data per head); ``data`` an existing
    [n_pages, n_kv_heads, page_bytes] uint8 cache.  ``n_heads``,
    ``max_tokens`` and ``max_seqs`` are the query heads, queries and sequences
    that calls of ``attend`` are expected to have; larger calls work as well
    (the attention workspace's size goes by ``head_dim`` alone).  The workspace
    serves one stream at a time: calls of ``attend`` that may run at once each need
    another one (``workspace=``, zeroed once).  The attributes ``data``,
    ``k_gsa``, ``v_gsa`` and ``workspace`` may be set: later calls use the new
    buffers (a captured graph keeps the old ones' addresses).
    """

    def __init__(self, n_pages, n_kv_heads, head_dim, page_size=64, k_gsa=1.0, v_gsa=1.0, data=None, n_heads=None,
                 max_tokens=128, max_seqs=128, device=None):
        nbytes = nvfp4_kv_page_bytes(page_size, head_dim)
        if nbytes == 0:
            raise ValueError("page_size %d and head_dim %d are not supported" % (page_size, head_dim))
        self.head_dim, self.page_size, self.n_kv_heads = int(head_dim), int(page_size), int(n_kv_heads)
        dev = data.device if data is not None else torch.device(device or "cuda")
        shape = (int(n_pages), self.n_kv_heads, nbytes)
        if data is None:
            data = torch.zeros(shape, dtype=torch.uint8, device=dev)
        elif tuple(data.shape) != shape:
            raise ValueError("data is %s, not %s" % (tuple(data.shape), shape))
        self.max_tokens, self.max_seqs = int(max_tokens), int(max_seqs)
        self.n_heads = int(n_heads or n_kv_heads)
        ws_bytes = nvfp4_kv_attention_workspace_size(self.max_tokens, self.max_seqs, self.n_heads, self.n_kv_heads,
                                                     self.head_dim)
        if ws_bytes == 0:
            raise ValueError("%d query heads do not share %d KV heads" % (self.n_heads, self.n_kv_heads))
        self._bind(data, self._scale(k_gsa, dev), self._scale(v_gsa, dev))
        self.workspace = _resident_workspace(ws_bytes, dev)

    def _bind(self, data, k_gsa, v_gsa):
        # (checked here, not in every call)
        self._pages = _Pages(data, k_gsa, v_gsa, self.head_dim) if data.is_cuda else None
        self._data, self._k_gsa, self._v_gsa = data, k_gsa, v_gsa

    @property
    def data(self):
        return self._data

    @data.setter
    def data(self, data):
        if data.dim() != 3 or data.shape[1:] != self._data.shape[1:] or data.device != self._data.device:
            raise ValueError("data must be [n_pages, %d, %d] on %s" % (*self._data.shape[1:], self._data.device))
        self._bind(data, self._k_gsa, self._v_gsa)

    @property
    def k_gsa(self):
        return self._k_gsa

    @k_gsa.setter
    def k_gsa(self, g):
        self._bind(self._data, self._scale(g, self._data.device), self._v_gsa)

    @property
    def v_gsa(self):
        return self._v_gsa

    @v_gsa.setter
    def v_gsa(self, g):
        self._bind(self._data, self._k_gsa, self._scale(g, self._data.device))

    @property
    def workspace(self):
        return self._workspace

    @workspace.setter
    def workspace(self, workspace):
        n = workspace.numel()
        if workspace.dtype != _U8 or not workspace.is_contiguous() or workspace.device != self._data.device:
            raise ValueError("workspace must be contiguous uint8 on %s" % self._data.device)
        self._workspace, self._ws = workspace, (workspace.data_ptr(), n)

    def _scale(self, g, dev):
        if not isinstance(g, torch.Tensor):
            return torch.full((self.n_kv_heads,), float(g), dtype=torch.float32, device=dev)
        return g.to(device=dev, dtype=torch.float32).reshape(self.n_kv_heads).contiguous()

    def append(self, q, k, v, positions, slots, cos, sin, **kw):
        """nvfp4_kv_append into this cache."""
        if self._pages is None:
            raise ValueError("the cache must be on a GPU")
        return _append(self._pages, q, k, v, positions, slots, cos, sin, **kw)

    def gather(self, slots, **kw):
        """nvfp4_kv_gather from this cache."""
        if self._pages is None:
            raise ValueError("the cache must be on a GPU")
        return _gather(self._pages, slots, **kw)

    def attend(self, q, page_table, kv_lens, workspace=None, **kw):
        """nvfp4_kv_attention over this cache, with its own workspace unless one is given."""
        if q.dtype is not _BF16:
            raise TypeError("q must be bfloat16, got %s" % q.dtype)
        if self._pages is None:
            raise ValueError("the cache must be on a GPU")
        return _attend(self._pages, q, page_table, kv_lens, workspace=workspace,
                       ws=self._ws if workspace is None else None, **kw)

    def status(self, stream=None):
        """The workspace status word (0 ok, 6: a bounded wait timed out)."""
        return nvr_read_device_status(self.workspace, stream)


def rope_table(n_pos, rot, base=10000.0, factor=1.0, original=None, slow=1.0, fast=32.0, device=None):
    """cos and sin [n_pos, rot / 2] fp32 of the angles pos * base^(-2 i / rot).

    factor > 1 stretches the positions for contexts longer than the model's.
    Without ``original`` every angle is divided by the factor (position
    interpolation).  With ``original``, the context length of training, the
    channels are treated by parts: those that turn at least ``fast`` times over
    the original context keep their angle, those that turn at most ``slow``
    times take the interpolated one, between them the two are mixed linearly in
    the number of turns."""
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even and positive")
    i = torch.arange(0, rot, 2, dtype=torch.float64, device=device or "cuda")
    freq = base ** (-i / rot)
    if original is None:
        freq = freq / factor
    else:
        turns = original * freq / (2 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0.0, 1.0)
        freq = freq * keep + freq / factor * (1.0 - keep)
    angle = torch.arange(n_pos, dtype=torch.float64, device=freq.device)[:, None] * freq
    return angle.cos().float().contiguous(), angle.sin().float().contiguous()
