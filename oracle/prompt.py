"""A prompt's operators: rotary positions with several axes, and attention of
packed sequences over their own keys and values.

Test infrastructure only (see the package docstring).  Both are written from
their formulas, in float64:

* rope: x / sqrt(mean x^2 + eps) * weight for every head; pair i of a head,
  channels (i, i + rot/2) or (2i, 2i + 1), turns by the angle whose cosine and
  sine stand in column i of row positions[axes[i]]:
  (a, b) -> (a c - b s, b c + a s);
* attention: softmax of scale * q . k over the keys a query sees; joined with a
  prefix's result (o', z') by out e^(z - z*) + o' e^(z' - z*), z* = log(e^z + e^z').
"""

import numpy as np

# half a step of each type, relative to the value, and half a step of its subnormals
HALF = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "f32": 2.0 ** -24}
TINY = {"bf16": 2.0 ** -134, "f16": 2.0 ** -25, "f32": 2.0 ** -150}


def rope(x, positions, axes, cos, sin, interleaved, weight=None, eps=0.0):
    """float64 x [T, H, D] -> the result and the magnitude its rounding errors go by
    (|a c| + |b s| of each channel); rows with a position outside the tables: zeros."""
    T, H, D = x.shape
    y = np.array(x, np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * weight
    out, mag = y.copy(), np.abs(y)
    ok = np.ones(T, bool)
    pairs = len(axes)
    for i, a in enumerate(axes):
        ia, ib = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        pos = positions[a].astype(np.int64)
        good = (pos >= 0) & (pos < cos.shape[0])
        ok &= good
        at = np.where(good, pos, 0)
        c, s = cos[at, i].astype(np.float64)[:, None], sin[at, i].astype(np.float64)[:, None]
        u, v = y[..., ia], y[..., ib]
        out[..., ia], out[..., ib] = u * c - v * s, v * c + u * s
        mag[..., ia], mag[..., ib] = np.abs(u * c) + np.abs(v * s), np.abs(v * c) + np.abs(u * s)
    out[~ok], mag[~ok] = 0.0, 0.0
    return out, mag


def check_rope(got, ref, D, dtype):
    """Elements outside tolerance.  fp32 arithmetic: the sum of D squares is off by at most
    D 2^-24 of itself, its root by half of that, and a channel passes at most eight more
    roundings (mean, eps, root, reciprocal, two products, the rotation's product and sum) of
    2^-24 each; then one rounding to the result's type."""
    out, mag = ref
    tol = mag * (D * 2.0 ** -25 + 8 * 2.0 ** -24)
    tol = tol + HALF[dtype] * (np.abs(out) + tol) + TINY[dtype]
    return int(np.count_nonzero(~(np.abs(np.asarray(got, np.float64) - out) <= tol)))


def attention(q, k, v, scale, causal=True, window=0):
    """One sequence, float64: q [m, Hq, D], k, v [n, H, D] -> out, lse and the
    bounds the tolerances use: sum p |v| / sum p [m, Hq, D] and the largest
    |scale| sum |q k| of a seen key [m, Hq].  Unseen keys do not count, whatever they hold."""
    m, Hq, D = q.shape
    n, H = k.shape[:2]
    out, mag = np.zeros((m, Hq, D)), np.zeros((m, Hq, D))
    lse, big = np.full((m, Hq), -np.inf), np.zeros((m, Hq))
    if n == 0 or m == 0:
        return out, lse, mag, big
    pos = n - m + np.arange(m)[:, None]
    key = np.arange(n)
    see = np.ones((m, n), bool)
    if causal:
        see = key <= pos
        if window:
            see &= key > pos - window
    some = see.any(-1)
    with np.errstate(invalid="ignore", over="ignore"):
        for h in range(Hq):
            kk, vv = k[:, h * H // Hq], v[:, h * H // Hq]
            s = np.where(see, scale * (q[:, h] @ kk.T), -np.inf)
            top = np.where(some, s.max(-1), 0.0)
            p = np.where(see, np.exp(s - top[:, None]), 0.0)
            total = np.where(some, p.sum(-1), 1.0)
            if np.isfinite(vv).all():
                out[:, h], mag[:, h] = p @ vv / total[:, None], p @ np.abs(vv) / total[:, None]
            else:                                            # (a key that is not seen adds nothing, not 0 * inf)
                for i in range(m):
                    out[i, h] = p[i, see[i]] @ vv[see[i]] / total[i]
                    mag[i, h] = p[i, see[i]] @ np.abs(vv[see[i]]) / total[i]
            lse[:, h] = np.where(some, top + np.log(total), -np.inf)
            big[:, h] = np.where(see, abs(scale) * (np.abs(q[:, h]) @ np.abs(kk).T), 0.0).max(-1)
    return out, lse, mag, big


def join(ref, o2, z2):
    """The result joined with a prefix's (o2 [m, Hq, D], z2 [m, Hq])."""
    o, z, mag, big = ref
    both = np.logaddexp(z, z2)
    with np.errstate(invalid="ignore"):
        a, b = (np.where(np.isneginf(x), 0.0, np.exp(x - both))[..., None] for x in (z, z2))
    o2 = np.where(b > 0, o2, 0.0)
    return o * a + o2 * b, both, mag * a + np.abs(o2) * b, big


def check_attention(out, lse, ref, n, v_max, dtype):
    """Outputs outside tolerance (out, lse), 0 and 0 when all pass.

    fp32 scores: the sum over D <= 128 products has relative error at most
    D 2^-23 = 2^-16 of sum |q k| (truncating accumulation), so every weight is
    within e = 2 * 2^-16 * scale * sum|qk| + 2^-20 (base-2 exponential and its
    argument's scaling) of its value, the normaliser too; the weights enter the
    second product rounded to the values' type (fp16: 2^-25 absolute below its normal
    range, relative to a largest weight of 2^7 at least), its fp32 sum over n
    tokens adds n 2^-23; the join with a prefix is two exponentials, a sum and a quotient
    (2^-20); one rounding to the result's type."""
    o, z, mag, big = ref
    e = 2.0 * 2.0 ** -16 * big + 2.0 ** -20
    tol = mag * (2 * e + HALF[dtype] + n * 2.0 ** -23 + 2.0 ** -20)[..., None]
    if dtype == "f16":
        tol = tol + n * 2.0 ** -32 * v_max
    tol = tol + HALF[dtype] * (np.abs(o) + tol) + TINY[dtype]
    bad = int(np.count_nonzero(~(np.abs(np.asarray(out, np.float64) - o) <= tol)))
    if lse is None:
        return bad, 0
    lse = np.asarray(lse, np.float64)
    empty = np.isneginf(z)
    zt = e + n * 2.0 ** -24 + 2.0 ** -20 + np.abs(np.where(empty, 0.0, z)) * 2.0 ** -21
    with np.errstate(invalid="ignore"):
        off = ~(np.abs(lse - z) <= zt)
    off = np.where(empty, ~np.isneginf(lse), off)
    return bad, int(np.count_nonzero(off))
