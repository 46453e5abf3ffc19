"""The paged NVFP4 key/value cache: Python binding of include/nvfp4_kv_cache.h.

* ``nvfp4_kv_append(q, k, v, positions, slots, cos, sin, cache, k_gsa, v_gsa, ...)`` -> q_out
* ``nvfp4_kv_attention(q, cache, page_table, kv_lens, k_gsa, v_gsa, ...)`` -> (out, lse)
* ``nvfp4_kv_gather(cache, slots, k_gsa, v_gsa, ...)`` -> (k, v)
* ``rope_table(n_pos, rot, ...)`` -> (cos, sin), plain, interpolated or scaled by parts

``Nvfp4KVCache`` keeps the pages, the global scales and the attention
workspace resident: its calls allocate nothing but outputs the caller does not
pass (CUDA-graph capturable).
"""

import math

import torch

from . import _dev, _dtype_code, _stream, new_workspace
from . import _native


def nvfp4_kv_page_bytes(page_size, D):
    """Bytes of one page of one KV head; 0 for an unsupported size."""
    return int(_native.lib().nvfp4_kv_page_bytes(page_size, D))


def nvfp4_kv_attention_workspace_size(T_max, B_max, n_heads, n_kv_heads, D):
    return int(_native.lib().nvfp4_kv_attention_workspace_size(T_max, B_max, n_heads, n_kv_heads, D))


def _page_size(cache, D):
    """The page size of a cache [n_pages, n_kv_heads, page_bytes] uint8."""
    if cache.dtype != torch.uint8 or cache.dim() != 3:
        raise TypeError("cache must be uint8 [n_pages, n_kv_heads, page_bytes]")
    return cache.shape[2] * 8 // (9 * D)


def _heads(t, name):
    """Pointer and token stride of [T, heads, D] with contiguous heads."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    T, H, D = t.shape
    s = t.stride()
    if (D > 1 and s[2] != 1) or (H > 1 and s[1] != D):
        raise ValueError("%s must have contiguous heads (a token stride is allowed)" % name)
    return t.data_ptr(), (s[0] if T > 1 else H * D)


def _typed(t, dtype, name):
    if t is None:
        return None
    if t.dtype != dtype:
        raise TypeError("%s must be %s" % (name, dtype))
    return _dev(t, name)


def _length(t, n, name):
    if t.numel() != n:
        raise ValueError("%s has %d elements, not %d" % (name, t.numel(), n))


def nvfp4_kv_append(q, k, v, positions, slots, cos, sin, cache, k_gsa, v_gsa, q_weight=None, k_weight=None,
                    eps=1e-6, interleaved=False, q_out=None, stream=None):
    """RMS norm of the heads of q [T, Hq, D] and k [T, Hkv, D] (where a weight
    is given), rotary positions, and k and v quantized into the cache's slots.
    cos and sin are [n_pos, rot/2] (None: no rotation); returns q_out [T, Hq, D]
    bf16 (None for q None)."""
    T, Hkv, D = k.shape
    if tuple(v.shape) != (T, Hkv, D) or v.dtype != k.dtype:
        raise ValueError("k and v must have one shape and type")
    kp, ks = _heads(k, "k")
    vp, vs = _heads(v, "v")
    Hq, qp, qs, op = 0, None, 0, None
    if q is not None:
        Hq = q.shape[1]
        if q.shape[0] != T or q.shape[2] != D or q.dtype != k.dtype:
            raise ValueError("q must be [T, heads, D] of k's type")
        qp, qs = _heads(q, "q")
        if q_out is None:
            q_out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=k.device)
        op = _typed(q_out, torch.bfloat16, "q_out")
        _length(q_out, T * Hq * D, "q_out")
    S = _page_size(cache, D)
    if cache.shape[1] != Hkv:
        raise ValueError("the cache has %d KV heads, k has %d" % (cache.shape[1], Hkv))
    _length(slots, T, "slots")
    _length(k_gsa, Hkv, "k_gsa")
    _length(v_gsa, Hkv, "v_gsa")
    rot, n_pos = 0, 0
    if cos is not None:
        n_pos, rot = cos.shape[0], 2 * cos.shape[1]
        if sin.shape != cos.shape:
            raise ValueError("cos and sin must have one shape")
        _length(positions, T, "positions")
    for w, name in ((q_weight, "q_weight"), (k_weight, "k_weight")):
        if w is not None:
            _length(w, D, name)
    f32, i32 = torch.float32, torch.int32
    st = _native.lib().nvfp4_kv_append(
        qp, qs, kp, ks, vp, vs, _dtype_code(k), T, Hq, Hkv, D, _typed(positions, i32, "positions"),
        _typed(slots, i32, "slots"), _typed(cos, f32, "cos"), _typed(sin, f32, "sin"), n_pos, rot, int(interleaved),
        _typed(q_weight, f32, "q_weight"), _typed(k_weight, f32, "k_weight"), float(eps),
        _typed(k_gsa, f32, "k_gsa"), _typed(v_gsa, f32, "v_gsa"), _dev(cache, "cache"), cache.shape[0], S, op,
        _stream(stream))
    _native.check("nvfp4_kv_append", st)
    return q_out


def nvfp4_kv_gather(cache, slots, k_gsa, v_gsa, D, out_dtype=torch.bfloat16, k_out=None, v_out=None, stream=None):
    """The values that the slots stand for: k and v [n, Hkv, D] (zeros for a
    slot outside the cache)."""
    n, Hkv = slots.numel(), cache.shape[1]
    if k_out is None:
        k_out = torch.empty((n, Hkv, D), dtype=out_dtype, device=cache.device)
    if v_out is None:
        v_out = torch.empty((n, Hkv, D), dtype=k_out.dtype, device=cache.device)
    if v_out.dtype != k_out.dtype:
        raise TypeError("k_out and v_out must have one type")
    for t, m, name in ((k_out, n * Hkv * D, "k_out"), (v_out, n * Hkv * D, "v_out"), (k_gsa, Hkv, "k_gsa"),
                       (v_gsa, Hkv, "v_gsa")):
        _length(t, m, name)
    st = _native.lib().nvfp4_kv_gather(
        _dev(cache, "cache"), cache.shape[0], _page_size(cache, D), Hkv, D, _typed(slots, torch.int32, "slots"), n,
        _typed(k_gsa, torch.float32, "k_gsa"), _typed(v_gsa, torch.float32, "v_gsa"), _dev(k_out, "k_out"),
        _dev(v_out, "v_out"), _dtype_code(k_out), _stream(stream))
    _native.check("nvfp4_kv_gather", st)
    return k_out, v_out


def nvfp4_kv_attention(q, cache, page_table, kv_lens, k_gsa, v_gsa, cu_q=None, max_q=None, scale=None, causal=True,
                       window=0, out=None, lse=None, workspace=None, stream=None):
    """Attention of q [T, Hq, D] bf16 over the cached tokens of the sequences
    in page_table [B, max_pages] and kv_lens [B].  cu_q [B + 1] (with max_q, the
    most queries of a sequence) gives each sequence's rows of q; without it every
    sequence has T / B queries.  Returns (out [T, Hq, D] bf16, lse); lse [T, Hq]
    fp32 is written when it is given."""
    T, Hq, D = q.shape
    if q.dtype != torch.bfloat16:
        raise TypeError("q must be bfloat16, got %s" % q.dtype)
    B, max_pages = page_table.shape
    Hkv = cache.shape[1]
    if cu_q is None:
        if B == 0 or T % B:
            raise ValueError("%d queries for %d sequences: pass cu_q" % (T, B))
        max_q = T // B
    else:
        _length(cu_q, B + 1, "cu_q")
        if max_q is None:
            raise ValueError("cu_q needs max_q, the most queries of a sequence")
    _length(kv_lens, B, "kv_lens")
    _length(k_gsa, Hkv, "k_gsa")
    _length(v_gsa, Hkv, "v_gsa")
    if out is None:
        out = torch.empty((T, Hq, D), dtype=torch.bfloat16, device=q.device)
    _length(out, T * Hq * D, "out")
    if lse is not None:
        _length(lse, T * Hq, "lse")
    if workspace is None:
        workspace = new_workspace(nvfp4_kv_attention_workspace_size(T, B, Hq, Hkv, D), q.device)
    qp, qs = _heads(q, "q")
    f32, i32 = torch.float32, torch.int32
    st = _native.lib().nvfp4_kv_attention(
        qp, qs, T, Hq, Hkv, D, _dev(cache, "cache"), cache.shape[0], _page_size(cache, D),
        _typed(page_table, i32, "page_table"), B, max_pages, _typed(kv_lens, i32, "kv_lens"),
        _typed(cu_q, i32, "cu_q"), int(max_q), _typed(k_gsa, f32, "k_gsa"), _typed(v_gsa, f32, "v_gsa"),
        float(D ** -0.5 if scale is None else scale), int(causal), int(window),
        _typed(out, torch.bfloat16, "out"), _typed(lse, f32, "lse"), _dev(workspace, "workspace"),
        workspace.numel(), _stream(stream))
    _native.check("nvfp4_kv_attention", st)
    return out, lse


class Nvfp4KVCache:
    """Resident paged NVFP4 key/value cache of one layer.

    ``k_gsa`` and ``v_gsa`` are the global scales (a number or [n_kv_heads]
    fp32, max|x| / 2688 of calibration data per head); ``data`` an existing
    [n_pages, n_kv_heads, page_bytes] uint8 cache.  ``n_heads``,
    ``max_tokens`` and ``max_seqs`` size the attention workspace.
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
        self.data = data
        self.k_gsa, self.v_gsa = (self._scale(g, dev) for g in (k_gsa, v_gsa))
        self.max_tokens, self.max_seqs = int(max_tokens), int(max_seqs)
        self.n_heads = int(n_heads or n_kv_heads)
        self.workspace = new_workspace(nvfp4_kv_attention_workspace_size(
            self.max_tokens, self.max_seqs, self.n_heads, self.n_kv_heads, self.head_dim), dev)

    def _scale(self, g, dev):
        if not isinstance(g, torch.Tensor):
            return torch.full((self.n_kv_heads,), float(g), dtype=torch.float32, device=dev)
        return g.to(device=dev, dtype=torch.float32).reshape(self.n_kv_heads).contiguous()

    def append(self, q, k, v, positions, slots, cos, sin, **kw):
        """nvfp4_kv_append into this cache."""
        return nvfp4_kv_append(q, k, v, positions, slots, cos, sin, self.data, self.k_gsa, self.v_gsa, **kw)

    def gather(self, slots, **kw):
        """nvfp4_kv_gather from this cache."""
        return nvfp4_kv_gather(self.data, slots, self.k_gsa, self.v_gsa, self.head_dim, **kw)

    def attend(self, q, page_table, kv_lens, **kw):
        """nvfp4_kv_attention over this cache."""
        if q.shape[0] > self.max_tokens or page_table.shape[0] > self.max_seqs or q.shape[1] != self.n_heads:
            raise ValueError("%d tokens of %d heads in %d sequences: the workspace is for %d, %d and %d" % (
                q.shape[0], q.shape[1], page_table.shape[0], self.max_tokens, self.n_heads, self.max_seqs))
        return nvfp4_kv_attention(q, self.data, page_table, kv_lens, self.k_gsa, self.v_gsa,
                                  workspace=self.workspace, **kw)

    def status(self, stream=None):
        """The workspace status word (0 ok, 6: a bounded wait timed out)."""
        from . import nvr_read_device_status
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
