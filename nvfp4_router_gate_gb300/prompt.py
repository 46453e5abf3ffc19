"""A prompt's operators beside the NVFP4 key/value cache: Python binding of
include/nvfp4_prompt.h.

* ``prompt_rope(q, k, positions, cos, sin, axes, ...)`` -> (q_out, k_out): RMS norm of the heads
  and rotary positions with several axes
* ``rope_axes(sections, turns=False)`` -> the axis of each pair
* ``rope_axes_table(n_pos, sections, ...)`` -> (cos, sin) with frequencies of each axis's own
* ``prompt_attention(q, k, v, ...)`` -> (out, lse): attention of packed prompts over their own
  16-bit keys and values

``PromptAttention`` keeps the workspace resident: its calls allocate nothing but
outputs the caller does not pass (CUDA-graph capturable).  What a call with
``stream=`` allocates belongs to that stream.
"""

import contextlib

import torch

from . import _native, _resident_workspace, new_workspace, nvr_read_device_status
from .kv_cache import _empty, _empty_on, _on, _ptr

_BF16, _F16, _F32, _I32, _U8 = torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.uint8
_CODES = {_BF16: _native.NVR_BF16, _F32: _native.NVR_F32, _F16: _native.NVR_F16}
_MAX_AXES = 8
_current, _device = torch._C._cuda_getCurrentRawStream, torch._C._cuda_getDevice


def _here(t, name):
    """The tensor's device, which has to be the current one (launches go there), and its number."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    at = t.get_device()
    if at != _device():
        raise ValueError("%s is on %s, the current device is cuda:%d" % (name, t.device, _device()))
    return t.device, at


def _same(dev, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError("%s is on %s, not %s" % (name, t.device, dev))


def _steps(t, T, H, D, name):
    """Token stride of t [T, H, D] with contiguous heads."""
    s0, s1, s2 = t.stride()
    if (s2 != 1 and D > 1) or (s1 != D and H > 1):
        raise ValueError("%s must have contiguous heads (a token stride is allowed)" % name)
    return s0 if T > 1 else H * D


def _side(x, T, D, dt, at, name):
    """Pointer, token stride and heads of x [T, heads, D]."""
    shape = x.shape
    if len(shape) != 3 or shape[0] != T or shape[2] != D or x.dtype is not dt or x.get_device() != at:
        raise ValueError("%s must be [T, heads, D] of one type and device with the other" % name)
    H = shape[1]
    return x.data_ptr(), _steps(x, T, H, D, name), H


def _result(out, shape, dtype, dev, at, stream, name):
    """The tensor for a result, its pointer and token stride."""
    T, H, D = shape
    if out is None:
        out = _empty(shape, dtype=dtype, device=dev) if stream is None else _empty_on(stream, shape, dtype=dtype, device=dev)
        return out, out.data_ptr(), H * D
    if out.shape != shape or out.dtype is not dtype or out.get_device() != at:
        raise ValueError("%s must be %s of %s on %s" % (name, shape, dtype, dev))
    return out, out.data_ptr(), _steps(out, T, H, D, name)


def _floats(t, n, at, name):
    """Pointer of n contiguous fp32 on the device of that number."""
    if t.dtype is not _F32 or t.get_device() != at or t.numel() != n or not t.is_contiguous():
        _same(torch.device("cuda", at), **{name: t})
        _ptr(t, _F32, n, name)
    return t.data_ptr()


def rope_axes(sections, turns=False):
    """The axis of each pair of channels, where axis a has sections[a] pairs: the axes
    one after the other, or (turns) taking turns for as long as they have pairs left."""
    left = [int(n) for n in sections]
    if not left or len(left) > _MAX_AXES or min(left) < 0:
        raise ValueError("sections must be the pairs of 1 to %d axes" % _MAX_AXES)
    if not turns:
        return tuple(a for a, n in enumerate(left) for _ in range(n))
    return tuple(a for i in range(max(left)) for a, n in enumerate(left) if i < n)


def rope_axes_table(n_pos, sections, turns=False, base=10000.0, device=None):
    """cos and sin [n_pos, pairs] fp32 for rope_axes(sections, turns) where every axis has
    frequencies of its own: pair j of the n of an axis turns by pos * base^(-j / n).
    (Where the axes share one row of frequencies, rope_table gives the table.)"""
    axes, seen, freq = rope_axes(sections, turns), {}, []
    for a in axes:
        j = seen[a] = seen.get(a, -1) + 1
        freq.append(float(base) ** (-j / int(sections[a])))
    freq = torch.tensor(freq, dtype=torch.float64, device=device or "cuda")
    angle = torch.arange(n_pos, dtype=torch.float64, device=freq.device)[:, None] * freq
    return angle.cos().float().contiguous(), angle.sin().float().contiguous()


def prompt_rope(q, k, positions, cos, sin, axes=None, q_weight=None, k_weight=None, eps=1e-6, interleaved=False,
                q_out=None, k_out=None, out_dtype=None, stream=None):
    """RMS norm of the heads of q [T, Hq, D] and k [T, Hkv, D] (where q_weight, k_weight
    [D] are given) and rotary positions with several axes: pair i of a head turns by
    column i of row positions[axes[i]] of cos and sin [n_pos, pairs].  positions is
    [n_axes, T] int32 (or [T], one axis); axes a sequence of ints (``rope_axes``; None:
    the first axis for all pairs).  cos None: no rotation.  q or k may be None.  Types:
    bfloat16, float16 or float32; out_dtype (or q_out and k_out, which may be q and k
    themselves) the same, or a 16-bit one for float32 heads.  Returns (q_out, k_out)."""
    some = q if q is not None else k
    dev, at = _here(some, "q" if q is not None else "k")
    shape, dt = some.shape, some.dtype
    if len(shape) != 3:
        raise ValueError("heads must be [T, heads, D]")
    T, _, D = shape
    if dt not in _CODES:
        raise TypeError("heads must be bfloat16, float16 or float32, got %s" % dt)
    if out_dtype is None:
        out_dtype = dt if q_out is None and k_out is None else (k_out if q_out is None else q_out).dtype
    if out_dtype is not dt and (dt is not _F32 or out_dtype not in _CODES):
        raise TypeError("heads of %s do not become %s" % (dt, out_dtype))
    Hq = Hkv = qs = ks = qos = kos = 0
    qp = kp = qo = ko = None
    if q is not None:
        qp, qs, Hq = _side(q, T, D, dt, at, "q")
        q_out, qo, qos = _result(q_out, (T, Hq, D), out_dtype, dev, at, stream, "q_out")
    elif q_out is not None:
        raise ValueError("q_out without q")
    if k is not None:
        kp, ks, Hkv = _side(k, T, D, dt, at, "k")
        k_out, ko, kos = _result(k_out, (T, Hkv, D), out_dtype, dev, at, stream, "k_out")
    elif k_out is not None:
        raise ValueError("k_out without k")
    rot = n_pos = n_axes = step = 0
    code = where = cos_p = sin_p = None
    if cos is not None:
        if sin is None or positions is None or cos.dim() != 2:
            raise ValueError("cos [n_pos, pairs] needs sin and positions")
        n_pos, pairs = cos.shape
        if positions.dim() == 1:
            positions = positions[None]
        size, steps = positions.shape, positions.stride()
        if len(size) != 2 or size[1] != T or (T > 1 and steps[1] != 1) or positions.dtype is not _I32 or positions.get_device() != at:
            raise ValueError("positions must be int32 [n_axes, T] on %s, the tokens next to each other" % dev)
        axes = (0,) * pairs if axes is None else axes
        if len(axes) != pairs:
            raise ValueError("%d axes for %d pairs" % (len(axes), pairs))
        if pairs:
            rot, n_axes, step, code = 2 * pairs, size[0], steps[0], bytes(axes)       # (the library looks at the axes)
            where = positions.data_ptr()
            cos_p, sin_p = _floats(cos, n_pos * pairs, at, "cos"), _floats(sin, n_pos * pairs, at, "sin")
    qw = None if q_weight is None else _floats(q_weight, D, at, "q_weight")
    kw = None if k_weight is None else _floats(k_weight, D, at, "k_weight")
    st = _native.lib().prompt_rope(qp, qs, kp, ks, _CODES[dt], T, Hq, Hkv, D, where, step, n_axes, code, cos_p, sin_p, n_pos,
                                   rot, bool(interleaved), qw, kw, eps, qo, qos, ko, kos, _CODES[out_dtype],
                                   _current(at) if stream is None else stream.cuda_stream)
    if st:
        if code is not None and not (1 <= n_axes <= _MAX_AXES and max(code) < n_axes):
            raise ValueError("axes must be in [0, %d), positions of 1 to %d axes" % (n_axes, _MAX_AXES))
        _native.check("prompt_rope", st)
    return q_out, k_out


def prompt_attention_workspace_size(n_heads, n_kv_heads, D):
    return int(_native.lib().prompt_attention_workspace_size(n_heads, n_kv_heads, D))


def _offsets(cu, name):
    if cu.dim() != 1 or cu.shape[0] < 1:
        raise ValueError("%s must be [B + 1]" % name)
    return cu.shape[0] - 1


def _attend(q, k, v, ws, cu_q=None, max_q=None, cu_k=None, max_k=None, scale=None, causal=True, window=0, prefix=None,
            out=None, lse=None, stream=None):
    dev = q.device
    if k.dtype is not q.dtype or v.dtype is not q.dtype or q.dtype not in (_BF16, _F16):
        raise TypeError("q, k and v must be bfloat16 or float16, all three the same")
    if q.dim() != 3 or k.dim() != 3 or k.shape != v.shape:
        raise ValueError("q must be [T, heads, D], k and v [Tk, n_kv_heads, D]")
    T, Hq, D = q.shape
    Tk, Hkv, Dk = k.shape
    if Dk != D:
        raise ValueError("q has heads of %d channels, k of %d" % (D, Dk))
    if not (0 <= (max_q or 0) < 1 << 31 and 0 <= (max_k or 0) < 1 << 31 and 0 <= window < 1 << 31):
        raise ValueError("max_q, max_k and window must be in [0, 2^31)")      # (ctypes would cut them)
    if cu_q is not None:
        B = _offsets(cu_q, "cu_q")
        if max_q is None:
            raise ValueError("cu_q needs max_q, the most queries of a sequence")
    elif max_q is None:
        B, max_q = (1, T) if cu_k is None else (_offsets(cu_k, "cu_k"), None)
        if max_q is None:
            if T % B if B else T:
                raise ValueError("%d queries for %d sequences: pass cu_q" % (T, B))
            max_q = T // B if B else 0
    else:
        if max_q < 1 or T % max_q:
            raise ValueError("%d queries are not sequences of %d: pass cu_q" % (T, max_q))
        B = T // max_q
    if cu_k is not None:
        if _offsets(cu_k, "cu_k") != B:
            raise ValueError("cu_k is of %d sequences, not %d" % (cu_k.shape[0] - 1, B))
        if max_k is None:
            raise ValueError("cu_k needs max_k, the most keys of a sequence")
    elif Tk != T:
        raise ValueError("%d keys for %d queries: pass cu_k" % (Tk, T))
    q0, q1, q2 = q.stride()
    k0, k1, k2 = k.stride()
    v0, v1, v2 = v.stride()
    if not q2 == k2 == v2 == 1:
        raise ValueError("q, k and v must have contiguous channels")
    at = q.get_device()
    if k.get_device() != at or v.get_device() != at:
        _same(dev, k=k, v=v)
    po = pl = None
    if prefix is not None:
        po, pl = _ptr(prefix[0], q.dtype, T * Hq * D, "prefix out"), _ptr(prefix[1], _F32, T * Hq, "prefix lse")
        _same(dev, prefix=prefix[0], prefix_lse=prefix[1])
    if out is None:
        out = (_empty((T, Hq, D), dtype=q.dtype, device=dev) if stream is None else
               _empty_on(stream, (T, Hq, D), dtype=q.dtype, device=dev))
    for t in (cu_q, cu_k, out, lse):
        if t is not None and t.get_device() != at:
            _same(dev, cu_q=cu_q, cu_k=cu_k, out=out, lse=lse)
    st = _native.lib().prompt_attention(
        q.data_ptr(), q0, q1, k.data_ptr(), k0, k1, v.data_ptr(), v0, v1, _CODES[q.dtype], T, Tk,
        Hq, Hkv, D, _ptr(cu_q, _I32, B + 1, "cu_q"), _ptr(cu_k, _I32, B + 1, "cu_k"), B, max_q, max_k or 0,
        D ** -0.5 if scale is None else scale, causal, window, po, pl, _ptr(out, q.dtype, T * Hq * D, "out"),
        _ptr(lse, _F32, T * Hq, "lse"), ws[0], ws[1], _current(at) if stream is None else stream.cuda_stream)
    if st:
        _native.check("prompt_attention", st)
    return out, lse


def prompt_attention(q, k, v, workspace=None, stream=None, **kw):
    """Attention of q [T, Hq, D] over k and v [Tk, Hkv, D] (bfloat16 or float16; any token
    and head strides) of packed sequences: cu_q [B + 1] int32 (with max_q, the most queries
    of a sequence) gives each one's rows of q, cu_k (with max_k) those of k and v; without
    cu_k they are cu_q's.  Without cu_q all sequences have max_q queries (without max_q,
    either: one sequence).  scale defaults to D ** -0.5, causal to True (queries are a
    sequence's last positions), window to 0 (none).  prefix=(out, lse) of the same queries
    over other keys is joined with the result (the key/value cache's are bfloat16).  Returns
    (out [T, Hq, D], lse); lse [T, Hq] fp32 is written when it is given; out may be the
    prefix's, not q, k or v.  Scores, sums and results are accumulated in fp32; the weights
    are rounded to the values' type before they meet them (include/nvfp4_prompt.h)."""
    dev, _ = _here(q, "q")
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q must be [T, heads, D], k and v [Tk, n_kv_heads, D]")
    if workspace is None:
        n = prompt_attention_workspace_size(q.shape[1], k.shape[1], q.shape[2])
        # (zeroed on the stream that uses it)
        with _on(stream) if stream is not None else contextlib.nullcontext():
            workspace = new_workspace(n, dev)
    _same(dev, workspace=workspace)
    n = workspace.numel()
    return _attend(q, k, v, (_ptr(workspace, _U8, n, "workspace"), n), stream=stream, **kw)


class PromptAttention:
    """prompt_attention with its workspace resident, for n_heads query heads on
    n_kv_heads KV heads of head_dim channels.  The workspace serves one stream at a
    time, whichever it is: calls that may run at once each need another one (``workspace=``,
    zeroed once), graphs that may be replayed at once among them."""

    def __init__(self, n_heads, n_kv_heads, head_dim, device=None):
        n = prompt_attention_workspace_size(n_heads, n_kv_heads, head_dim)
        if n == 0:
            raise ValueError("%d query heads on %d KV heads of %d channels are not supported" % (
                n_heads, n_kv_heads, head_dim))
        self.n_heads, self.n_kv_heads, self.head_dim = int(n_heads), int(n_kv_heads), int(head_dim)
        self.workspace = _resident_workspace(n, torch.device(device or "cuda"))

    def __call__(self, q, k, v, workspace=None, **kw):
        dev, _ = _here(q, "q")
        if q.dim() != 3 or k.dim() != 3 or q.shape[1:] != (self.n_heads, self.head_dim) or k.shape[1] != self.n_kv_heads:
            raise ValueError("q must be [T, %d, %d] and k [Tk, %d, %d]" % (
                self.n_heads, self.head_dim, self.n_kv_heads, self.head_dim))
        ws = self.workspace if workspace is None else workspace
        _same(dev, workspace=ws)
        n = ws.numel()
        return _attend(q, k, v, (_ptr(ws, _U8, n, "workspace"), n), **kw)

    def status(self, stream=None):
        """The workspace status word (0 ok, 6: a bounded wait timed out)."""
        return nvr_read_device_status(self.workspace, stream)
