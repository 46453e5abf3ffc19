"""The paged NVFP4 key/value cache: what append stores, and attention over it.

Test infrastructure only (see the package docstring).

The pages this project is built from stop at the router and the expert
products; the cache follows their number format ("nvfp4-megamoe-kernel commit
04cf8ca: dsv4/layers/router.py", runtime-gsa section: 16-element blocks, E4M3
scales, E2M1 codes, one fp32 global scale) for the keys and values of the
attention in front of the router.  Definitions:

* append, every step one float32 rounding: r = 1 / sqrt(sum x^2 / D + eps)
  with the sum taken by halving (element i + element i + D/2, and so on),
  x * r * weight; the rotation (a, b) -> (a c - b s, b c + a s) of channels
  (i, i + rot/2) or (2i, 2i+1); queries to bf16 (nearest even); keys and values
  quantized with the head's fixed global scale.
* attention, in float64: softmax of scale * q . k over the visible tokens.
"""

import numpy as np

from .formats import decode_e2m1, decode_e4m3
from .quantize import pack_fp4, quantize


def float32_to_bf16_bits(x):
    """Round to nearest even, as uint16 bit patterns (finite inputs)."""
    b = np.ascontiguousarray(x, dtype=np.float32).view(np.uint32).astype(np.uint64)
    return ((b + 0x7FFF + ((b >> 16) & 1)) >> 16).astype(np.uint16)


def head_norm(x, weight, eps):
    """RMS norm of the last axis in float32, one rounding a step."""
    x = np.asarray(x, np.float32)
    s = x * x
    while s.shape[-1] > 1:
        h = s.shape[-1] // 2
        s = s[..., :h] + s[..., h:]
    mean = s * np.float32(1.0 / x.shape[-1])
    r = np.float32(1.0) / np.sqrt(mean + np.float32(eps))
    return (x * r) * np.asarray(weight, np.float32)


def rotate(x, cos, sin, interleaved):
    """Rotary positions of x [T, H, D]; cos, sin [T, rot/2] float32."""
    y = np.array(x, np.float32)
    half = cos.shape[1]
    for i in range(half):
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        a, b, c, s = x[..., ia], x[..., ib], cos[:, i, None], sin[:, i, None]
        y[..., ia] = a * c - b * s
        y[..., ib] = b * c + a * s
    return y


def entry(x, gsa):
    """Codes [T, H, D/2] packed and scale bytes [T, H, D/16] of x [T, H, D]."""
    T, H, D = x.shape
    codes, scales = np.zeros((T, H, D // 2), np.uint8), np.zeros((T, H, D // 16), np.uint8)
    for h in range(H):
        c, s, _ = quantize(x[:, h], gsa=np.float32(gsa[h]))
        codes[:, h], scales[:, h] = pack_fp4(c), s
    return codes, scales


def region_offsets(S, D):
    """Byte offsets of key scales, value codes, value scales and the page's end."""
    return S * D // 2, S * D // 2 + S * D // 16, S * D + S * D // 16, S * D + S * D // 8


def store(cache, slots, kc, ks, vc, vs, S):
    """Write entries into cache [n_pages, H, page_bytes] at their slots."""
    D = kc.shape[2] * 2
    k_sc, v_co, v_sc, _ = region_offsets(S, D)
    for t, slot in enumerate(np.asarray(slots, np.int64)):
        if not 0 <= slot < cache.shape[0] * S:
            continue
        page, tok = divmod(int(slot), S)
        for h in range(cache.shape[1]):
            p = cache[page, h]
            p[tok * D // 2:(tok + 1) * D // 2] = kc[t, h]
            p[k_sc + tok * D // 16:k_sc + (tok + 1) * D // 16] = ks[t, h]
            for b in range(D // 16):
                at = v_co + (tok // 8) * 8 * (D // 2) + b * 64 + (tok % 8) * 8
                p[at:at + 8] = vc[t, h, 8 * b:8 * b + 8]
                p[v_sc + (tok // 8) * 8 * (D // 16) + b * 8 + tok % 8] = vs[t, h, b]
    return cache


def load(cache, slots, S, D, k_gsa, v_gsa):
    """float64 keys and values [n, H, D] of the slots (all inside the cache)."""
    k_sc, v_co, v_sc, _ = region_offsets(S, D)
    slots = np.asarray(slots, np.int64)
    page, tok = slots // S, slots % S
    p = cache[page]                                          # [n, H, bytes]
    n, H = p.shape[:2]
    row = np.arange(n)[:, None, None]
    head = np.arange(H)[None, :, None]
    blk = np.repeat(np.arange(D // 16), 8)
    byte = np.tile(np.arange(8), D // 16)
    g, i = (tok // 8)[:, None], (tok % 8)[:, None]
    kc = p[row, head, (tok[:, None] * (D // 2) + np.arange(D // 2))[:, None]]
    ks = p[row, head, (k_sc + tok[:, None] * (D // 16) + np.arange(D // 16))[:, None]]
    vc = p[row, head, (v_co + g * 8 * (D // 2) + blk * 64 + i * 8 + byte)[:, None]]
    vs = p[row, head, (v_sc + g * 8 * (D // 16) + np.arange(D // 16) * 8 + i)[:, None]]

    def value(c, s, gsa):
        x = np.stack([decode_e2m1(c & 15), decode_e2m1(c >> 4)], -1).reshape(n, H, D)
        return x * np.repeat(decode_e4m3(s), 16, axis=2) * np.asarray(gsa, np.float64)[None, :, None]

    return value(kc, ks, k_gsa), value(vc, vs, v_gsa)


def attention(q, k, v, scale, causal=True, window=0, seen=None):
    """One sequence, float64: q [m, Hq, D], k, v [n, H, D] -> out, lse and the
    bounds the tolerances use: sum p |v| / sum p [m, Hq, D] and the largest
    scale * sum |q k| of a seen token [m, Hq].  seen: bool [n], tokens that exist."""
    m, Hq, D = q.shape
    n, H = k.shape[:2]
    G = Hq // H
    out, mag = np.zeros((m, Hq, D)), np.zeros((m, Hq, D))
    lse, big = np.full((m, Hq), -np.inf), np.zeros((m, Hq))
    pos = n - m + np.arange(m)
    key = np.arange(n)
    ok = np.ones((m, n), bool)
    if causal:
        ok &= key[None] <= pos[:, None]
        if window:
            ok &= key[None] > pos[:, None] - window
    if seen is not None:
        ok &= seen[None]
    for h in range(Hq):
        kk, vv = k[:, h // G], v[:, h // G]
        for i in range(m):
            use = ok[i]
            if not use.any():
                continue
            s = scale * (kk[use] @ q[i, h])
            top = s.max()
            p = np.exp(s - top)
            out[i, h] = (p @ vv[use]) / p.sum()
            mag[i, h] = (p @ np.abs(vv[use])) / p.sum()
            lse[i, h] = top + np.log(p.sum())
            big[i, h] = abs(scale) * (np.abs(kk[use]) @ np.abs(q[i, h])).max()
    return out, lse, mag, big


def check_attention(out, lse, ref, n, v_max):
    """Outputs outside tolerance (out, lse), 0 and 0 when all pass.

    fp32 scores: the sum over D <= 128 products has relative error at most
    D 2^-23 = 2^-16 of sum |q k| (truncating accumulation), so every weight is
    within e = 2 * 2^-16 * scale * sum|qk| + 2^-20 (base-2 exponential and its
    argument's scaling) of its value, the normaliser too; the weights enter the
    second product as fp16 (2^-11, and 2^-25 absolute below the normal range,
    for weights relative to a maximum weight of at least 1), its fp32 sum over n
    tokens adds n 2^-23; one rounding to bf16 (2^-8)."""
    o, z, mag, big = ref
    e = 2.0 * 2.0 ** -16 * big + 2.0 ** -20
    tol = mag * (2 * e + 2.0 ** -11 + n * 2.0 ** -23)[..., None] + n * 2.0 ** -25 * v_max
    tol = tol + 2.0 ** -8 * (np.abs(o) + tol)
    bad = int(np.count_nonzero(~(np.abs(np.asarray(out, np.float64) - o) <= tol)))
    if lse is None:
        return bad, 0
    lse = np.asarray(lse, np.float64)
    empty = np.isneginf(z)
    zt = e + n * 2.0 ** -24 + np.abs(np.where(empty, 0.0, z)) * 2.0 ** -21
    with np.errstate(invalid="ignore"):
        off = ~(np.abs(lse - z) <= zt)
    off = np.where(empty, ~np.isneginf(lse), off)
    return bad, int(np.count_nonzero(off))
