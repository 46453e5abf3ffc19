"""GPU parity of the NVFP4 key/value cache (append, gather, attention) against
the oracle (oracle/kv_cache.py): stored bytes bit for bit, attention within the
tolerances derived there, at the sizes, masks and layouts where such kernels go
wrong."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

import workloads as WL  # noqa: E402
from oracle import kv_cache as K  # noqa: E402
from gpu_util import to_device  # noqa: E402


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


# ----------------------------------------------------------------- append

def _rows(rng, T, H, D, dtype):
    x = rng.standard_normal((T, H, D)).astype(np.float32)
    x[..., rng.integers(0, D, 4)] *= 8.0
    if dtype == "bf16":
        b = WL.float32_to_bf16_bits(x)
        return b, WL.bf16_bits_to_float32(b)
    return x, x


APPEND = [  # T, Hq, Hkv, D, S, rot, interleaved, norm, dtype
    (1, 8, 1, 128, 64, 128, False, True, "bf16"),
    (1, 1, 1, 64, 16, 0, False, False, "f32"),
    (5, 3, 3, 64, 32, 64, True, True, "bf16"),
    (17, 6, 2, 128, 16, 64, False, True, "f32"),
    (33, 5, 5, 128, 128, 64, True, False, "bf16"),
    (70, 4, 2, 64, 16, 32, False, True, "bf16"),          # half pairs 16 apart
    (9, 2, 1, 128, 32, 34, False, True, "bf16"),          # and an odd distance
    (12, 9, 3, 64, 128, 6, True, True, "f32"),
    (700, 32, 8, 128, 64, 128, False, True, "bf16"),      # several groups of heads a warp
    (513, 20, 4, 64, 32, 64, False, True, "f32"),
]


@pytest.mark.parametrize("case", APPEND, ids=lambda c: "T%d_H%d_%d_D%d_S%d_r%d%s%s_%s" % (
    c[0], c[1], c[2], c[3], c[4], c[5], "i" if c[6] else "", "n" if c[7] else "", c[8]))
def test_append_stores_the_oracles_bits(case):
    import nvfp4_router_gate_gb300 as R
    T, Hq, Hkv, D, S, rot, inter, norm, dt = case
    rng = np.random.default_rng(T * 131 + D + rot)
    (qb, q), (kb, k), (vb, v) = (_rows(rng, T, h, D, dt) for h in (Hq, Hkv, Hkv))
    n_pages, n_pos = T // S + 3, 300
    ang = rng.uniform(-4, 4, (n_pos, max(rot // 2, 1)))
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    pos = rng.integers(0, n_pos, T).astype(np.int32)
    slots = rng.permutation(n_pages * S)[:T].astype(np.int32)
    if T > 4:
        slots[2], slots[3] = -1, n_pages * S                  # not stored
        if rot:
            pos[4] = n_pos                                    # no such row: zeros, not stored
    kg = (0.001 + 0.003 * rng.random(Hkv)).astype(np.float32)
    vg = (0.001 + 0.003 * rng.random(Hkv)).astype(np.float32)
    if Hkv > 1:
        kg[0] = 1e-4                                          # saturates
    qw, kw = (rng.standard_normal(D).astype(np.float32) for _ in range(2))
    junk = rng.integers(0, 256, (n_pages, Hkv, S * D * 9 // 8)).astype(np.uint8)
    cache = _dev(junk)
    # q, k, v as views of one fused tensor (token stride larger than the heads)
    fused = torch.cat([to_device(a, dt) for a in (qb, kb, vb)], dim=1).contiguous()
    qd, kd, vd = fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:]
    got = R.nvfp4_kv_append(qd, kd, vd, _dev(pos), _dev(slots), _dev(cos) if rot else None,
                            _dev(sin) if rot else None, cache, _dev(kg), _dev(vg),
                            q_weight=_dev(qw) if norm else None, k_weight=_dev(kw) if norm else None,
                            eps=1e-5, interleaved=inter)
    ok = np.ones(T, bool)
    if rot:
        ok = pos < n_pos
        p = np.where(ok, pos, 0)
    if norm:
        q, k = K.head_norm(q, qw, 1e-5), K.head_norm(k, kw, 1e-5)
    if rot:
        q, k = (K.rotate(x, cos[p], sin[p], inter) for x in (q, k))
    want_q = np.where(ok[:, None, None], K.float32_to_bf16_bits(q), 0)
    assert np.array_equal(got.view(torch.int16).cpu().numpy().view(np.uint16), want_q)
    kc, ks = K.entry(k, kg)
    vc, vs = K.entry(v, vg)
    want = K.store(junk.copy(), np.where(ok, slots, -1), kc, ks, vc, vs, S)
    assert np.array_equal(cache.cpu().numpy(), want)
    # and read back: the values the entries stand for
    ask = np.concatenate([slots, [-7]]).astype(np.int32)
    for odt in (torch.float32, torch.bfloat16):
        gk, gv = R.nvfp4_kv_gather(cache, _dev(ask), _dev(kg), _dev(vg), D, out_dtype=odt)
        inside = (ask >= 0) & (ask < n_pages * S) & np.concatenate([ok, [True]])
        rk, rv = K.load(want, np.where(inside, ask, 0), S, D, kg, vg)
        for g, r in ((gk, rk), (gv, rv)):
            g = g.float().cpu().numpy()
            r32 = r.astype(np.float32)                        # code * scale is exact: one rounding
            if odt == torch.bfloat16:
                r32 = WL.bf16_bits_to_float32(K.float32_to_bf16_bits(r32))
            assert np.array_equal(g[inside], r32[inside])
            out = ~inside & ((ask < 0) | (ask >= n_pages * S))
            assert not g[out].any()


def test_append_extreme_magnitudes_saturate():
    import nvfp4_router_gate_gb300 as R
    x = np.zeros((2, 1, 64), np.float32)
    x[0, 0, :5] = [3e38, -3e38, 1e-30, 0.0, -0.0]
    x[1, 0, :4] = [1e-6, -2e-6, 5e-7, 0.0]
    cache = torch.zeros(1, 1, 16 * 72, dtype=torch.uint8, device="cuda")
    g = np.array([1e-3], np.float32)
    d = to_device(x, "f32")
    R.nvfp4_kv_append(None, d, d, None, _dev(np.array([0, 1], np.int32)), None, None, cache, _dev(g), _dev(g))
    kc, ks = K.entry(x, g)
    want = K.store(np.zeros((1, 1, 16 * 72), np.uint8), [0, 1], kc, ks, kc, ks, 16)
    assert np.array_equal(cache.cpu().numpy(), want)


def test_append_under_a_scale_of_zero_stores_zeros():
    import nvfp4_router_gate_gb300 as R
    rng = np.random.default_rng(80)
    x = rng.standard_normal((3, 2, 128)).astype(np.float32)
    g = np.array([0.0, 2e-3], np.float32)
    cache = _dev(np.full((1, 2, 16 * 144), 255, np.uint8))
    d = to_device(x, "f32")
    slots = np.array([0, 5, 15], np.int32)
    R.nvfp4_kv_append(None, d, d, None, _dev(slots), None, None, cache, _dev(g), _dev(g))
    kc, ks = K.entry(x, g)
    assert not kc[:, 0].any() and not ks[:, 0].any()
    want = K.store(np.full((1, 2, 16 * 144), 255, np.uint8), slots, kc, ks, kc, ks, 16)
    assert np.array_equal(cache.cpu().numpy(), want)


def test_append_needs_no_queries_and_no_tokens():
    import nvfp4_router_gate_gb300 as R
    kv = R.Nvfp4KVCache(2, 2, 64, page_size=16)
    e = torch.zeros(0, 2, 64, device="cuda")
    i = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert kv.append(None, e, e, None, i, None, None) is None
    k, v = kv.gather(i)
    assert k.shape == (0, 2, 64) and v.shape == (0, 2, 64)
    with pytest.raises(TypeError):
        kv.append(None, e.half(), e.half(), None, i, None, None)
    with pytest.raises(ValueError):
        kv.append(None, torch.zeros(1, 3, 64, device="cuda"), torch.zeros(1, 3, 64, device="cuda"), None, i[:0], None,
                  None)
    with pytest.raises(R.RouterError):                        # token stride of 8 bytes off 16
        t = torch.zeros(2, 2 * 64 + 2, device="cuda")[:, :128].unflatten(1, (2, 64))
        kv.append(None, t, t, None, torch.zeros(2, dtype=torch.int32, device="cuda"), None, None)


# --------------------------------------------------------------- attention

class Cached:
    """A cache of random entries, the rest of its bytes random (NaN scales too)."""

    pad = 0                                                            # unused columns of the page table

    def __init__(self, rng, lens, H, D, S, spare=3, first_page=0, spread=1.0):
        self.lens, self.H, self.D, self.S = np.array(lens, np.int32), H, D, S
        used = [(int(n) + S - 1) // S for n in lens]
        n_pages = sum(used) + spare
        self.kg, self.vg = ((0.002 + 0.002 * rng.random(H)).astype(np.float32) for _ in range(2))
        cache = rng.integers(0, 256, (n_pages, H, S * D * 9 // 8)).astype(np.uint8)
        order = rng.permutation(n_pages)
        self.table = np.full((len(lens), max(max(used), 1) + 1 + self.pad), -1, np.int32)
        self.k, self.v = [], []
        at = 0
        for b, n in enumerate(lens):
            self.table[b, :used[b]] = order[at:at + used[b]]
            at += used[b]
            slots = self.table[b, np.arange(n) // S] * S + np.arange(n) % S
            ent = [K.entry((spread * f * rng.standard_normal((n, H, D))).astype(np.float32), g)
                   for f, g in ((1.0, self.kg), (0.5, self.vg))]
            K.store(cache, slots, ent[0][0], ent[0][1], ent[1][0], ent[1][1], S)
            k, v = K.load(cache, slots, S, D, self.kg, self.vg) if n else (np.zeros((0, H, D)),) * 2
            self.k.append(k)
            self.v.append(v)
        self.cache = _dev(cache)
        self.args = (_dev(self.table), _dev(self.lens))

    def run(self, q, **kw):
        import nvfp4_router_gate_gb300 as R
        lse = torch.full(q.shape[:2], 7.0, device="cuda")
        out, lse = R.nvfp4_kv_attention(q, self.cache, *self.args, _dev(self.kg), _dev(self.vg), lse=lse, **kw)
        torch.cuda.synchronize()
        return out.float().cpu().numpy(), lse.cpu().numpy()

    def check(self, q32, n_q, out, lse, scale=None, seen=None, rows=None, **kw):
        at = 0
        scale = self.D ** -0.5 if scale is None else scale
        for b, m in enumerate(n_q):
            if m == 0:
                continue
            pick = np.arange(m) if rows is None or m <= rows else np.unique(
                np.concatenate([np.arange(rows // 2), np.arange(m - rows // 2, m)]))
            if len(pick) < m:
                # rows m - i see the tokens of the last i queries: check a few of them alone
                ref = [K.attention(q32[at + i:at + i + 1].astype(np.float64), self.k[b][:len(self.k[b]) - m + 1 + i],
                                   self.v[b][:len(self.v[b]) - m + 1 + i], scale, **kw) for i in pick]
                ref = [np.concatenate(x) for x in zip(*ref)]
            else:
                ref = K.attention(q32[at:at + m].astype(np.float64), self.k[b], self.v[b], scale,
                                  seen=None if seen is None else seen[b], **kw)
            n = int(self.lens[b])
            vmax = np.abs(self.v[b]).max() if n else 0.0
            assert K.check_attention(out[at + pick], lse[at + pick], ref, n, vmax) == (0, 0), (b, m, n)
            at += m


def _queries(rng, T, Hq, D, loud=1.5):
    b = WL.float32_to_bf16_bits((loud * rng.standard_normal((T, Hq, D))).astype(np.float32))
    return to_device(b, "bf16"), WL.bf16_bits_to_float32(b)


DECODE = [  # lens, H, G, D, S
    ([1], 1, 1, 128, 64), ([1], 1, 1, 64, 16), ([77], 8, 4, 128, 64), ([16], 2, 3, 64, 16), ([17], 2, 5, 128, 16),
    ([63, 64, 65], 2, 8, 128, 64), ([63, 64, 65], 2, 8, 64, 32), ([0], 2, 2, 128, 64),
    ([0, 5, 0, 129, 0], 3, 7, 128, 128), ([127, 128, 129, 1, 2], 2, 16, 128, 128), ([300, 15], 2, 16, 64, 16),
    ([1000, 3, 500], 1, 12, 128, 32), ([250, 31], 2, 20, 128, 64), ([250, 31], 1, 32, 64, 64),
    ([90, 200], 1, 33, 128, 16), ([4097], 2, 8, 128, 64), ([9000], 1, 4, 64, 32),
    (list(range(1, 160, 7)), 4, 2, 128, 16), ([40] * 300, 2, 8, 128, 16), ([333] * 5 + [0] + [64] * 5, 8, 1, 64, 64),
]


@pytest.mark.parametrize("case", DECODE, ids=lambda c: "B%d_n%d_H%d_G%d_D%d_S%d" % (len(c[0]), max(c[0]), *c[1:]))
def test_one_query_per_sequence(case):
    lens, H, G, D, S = case
    rng = np.random.default_rng(sum(lens) + G)
    C = Cached(rng, lens, H, D, S)
    q, q32 = _queries(rng, len(lens), H * G, D)
    out, lse = C.run(q)
    C.check(q32, [1] * len(lens), out, lse)


MANY = [  # lens, n_q, H, G, D, S, window
    ([50, 9], [4, 4], 2, 2, 128, 64, 0), ([300], [5], 2, 3, 64, 16, 0), ([130, 70, 64], [4, 4, 4], 2, 8, 128, 64, 0),
    ([3, 0, 200], [5, 5, 5], 2, 2, 128, 32, 0),                       # more queries than tokens
    ([200], [200], 1, 4, 128, 64, 0), ([513, 40], [513, 40], 2, 1, 64, 16, 0),
    ([400, 100, 33, 7, 0, 260], [100, 1, 0, 7, 0, 33], 2, 4, 128, 64, 0),
    ([300, 300], [20, 20], 2, 5, 128, 16, 0), ([260, 90], [130, 90], 1, 8, 64, 128, 0),
    ([500, 40], [1, 1], 2, 8, 128, 64, 100), ([700], [64], 2, 4, 128, 32, 33), ([700], [9], 1, 16, 64, 64, 1),
    ([64, 640, 5], [5, 300, 5], 1, 2, 128, 16, 64), ([1200, 129], [257, 129], 2, 2, 128, 128, 300),
]


@pytest.mark.parametrize("case", MANY, ids=lambda c: "n%d_q%d_H%d_G%d_D%d_S%d_w%d" % (max(c[0]), max(c[1]), *c[2:]))
def test_several_queries_per_sequence(case):
    lens, n_q, H, G, D, S, window = case
    rng = np.random.default_rng(sum(lens) + sum(n_q))
    C = Cached(rng, lens, H, D, S)
    q, q32 = _queries(rng, sum(n_q), H * G, D)
    kw = {}
    if len(set(n_q)) > 1:
        kw = dict(cu_q=_dev(np.concatenate([[0], np.cumsum(n_q)]).astype(np.int32)), max_q=max(n_q))
    out, lse = C.run(q, window=window, **kw)
    C.check(q32, n_q, out, lse, window=window)


@pytest.mark.parametrize("m", [4, 70])
def test_window_without_end(m):
    """The largest window hides nothing, from queries in front of the first token either."""
    rng = np.random.default_rng(70 + m)
    C = Cached(rng, [3, 200], 1, 128, 16)
    q, q32 = _queries(rng, 2 * m, 8, 128)
    out, lse = C.run(q, window=2 ** 31 - 1)
    C.check(q32, [m] * 2, out, lse)


def test_long_chunk_spot_rows():
    rng = np.random.default_rng(11)
    C = Cached(rng, [3000, 700], 2, 128, 64)
    n_q = [2000, 700]
    q, q32 = _queries(rng, sum(n_q), 8, 128)
    out, lse = C.run(q, cu_q=_dev(np.array([0, 2000, 2700], np.int32)), max_q=2000)
    C.check(q32, n_q, out, lse, rows=24)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("m", [1, 6, 90])
def test_without_causal_mask(D, m):
    rng = np.random.default_rng(m + D)
    C = Cached(rng, [100, 37], 2, D, 32)
    q, q32 = _queries(rng, 2 * m, 4, D)
    out, lse = C.run(q, causal=False, scale=0.3)
    C.check(q32, [m, m], out, lse, scale=0.3, causal=False)


def test_one_long_sequence_over_the_whole_gpu():
    rng = np.random.default_rng(5)
    C = Cached(rng, [40000], 2, 128, 64)
    q, q32 = _queries(rng, 1, 16, 128, loud=4.0)                       # sharp softmax: the maximum moves
    out, lse = C.run(q)
    C.check(q32, [1], out, lse)
    again, lse2 = C.run(q)
    assert np.array_equal(out, again) and np.array_equal(lse, lse2)    # the join does not depend on timing


@pytest.mark.parametrize("m", [1, 40])
def test_large_scores_and_tiny_queries(m):
    rng = np.random.default_rng(6 + m)
    C = Cached(rng, [200, 90, 150], 1, 128, 64, spread=2.0)
    q, q32 = _queries(rng, 3 * m, 4, 128)
    f = np.ones((3 * m, 1, 1), np.float32)
    f[:m], f[m:2 * m], f[2 * m:] = 2.0 ** 8, 2.0 ** -30, 0.0           # exact in bf16
    q, q32 = q * _dev(f).to(torch.bfloat16), q32 * f
    out, lse = C.run(q)
    C.check(q32, [m] * 3, out, lse)


@pytest.mark.parametrize("m", [1, 40])
def test_pages_outside_the_cache_are_not_seen(m):
    rng = np.random.default_rng(7)
    C = Cached(rng, [150, 100], 2, 128, 16)
    bad = C.table.copy()
    bad[0, 2], bad[0, 5], bad[1, 0] = 10 ** 6, -1, -5
    seen = [np.repeat(~np.isin(np.arange(10), [2, 5]), 16)[:150], np.repeat(np.arange(7) > 0, 16)[:100]]
    C.args = (_dev(bad), C.args[1])
    q, q32 = _queries(rng, 2 * m, 4, 128)
    out, lse = C.run(q)
    C.check(q32, [m] * 2, out, lse, seen=seen)


def test_lengths_past_the_table_and_negative_are_cut():
    rng = np.random.default_rng(8)
    C = Cached(rng, [64, 20], 1, 64, 16)
    C.table = C.table[:, :4]
    C.lens = np.array([64, 0], np.int32)
    C.k[1], C.v[1] = C.k[1][:0], C.v[1][:0]
    C.args = (_dev(C.table), _dev(np.array([1000, -3], np.int32)))
    q, q32 = _queries(rng, 2, 2, 64)
    out, lse = C.run(q)
    C.check(q32, [1, 1], out, lse)


def test_strided_queries_other_stream_and_graph():
    import nvfp4_router_gate_gb300 as R
    rng = np.random.default_rng(9)
    C = Cached(rng, [300, 77, 5], 2, 128, 64)
    q, q32 = _queries(rng, 3, 12, 128)
    strided = q[:, :8]                                                 # heads of a wider projection
    kv = R.Nvfp4KVCache(C.cache.shape[0], 2, 128, page_size=64, k_gsa=_dev(C.kg), v_gsa=_dev(C.vg), data=C.cache,
                        n_heads=8)
    s = torch.cuda.Stream()
    out, lse = torch.empty(3, 8, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 8, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        kv.attend(strided, *C.args, out=out, lse=lse)
    s.synchronize()
    C.check(q32[:, :8], [1] * 3, out.float().cpu().numpy(), lse.cpu().numpy())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kv.attend(strided, *C.args, out=out, lse=lse)
    # the lengths are read at replay: one token less
    C.args[1].sub_(1)
    for _ in range(3):
        g.replay()
    torch.cuda.synchronize()
    C.lens = C.lens - 1
    C.k, C.v = [k[:-1] for k in C.k], [v[:-1] for v in C.v]
    C.check(q32[:, :8], [1] * 3, out.float().cpu().numpy(), lse.cpu().numpy())
    assert kv.status() == 0


def test_cache_past_four_gigabytes():
    """Pages at the far end of a cache of more than 2^32 bytes."""
    import nvfp4_router_gate_gb300 as R
    rng = np.random.default_rng(10)
    S, D, H = 128, 128, 8
    n_pages = (1 << 32) // (H * S * 144) + 40
    kv = R.Nvfp4KVCache(n_pages, H, D, page_size=S, k_gsa=0.002, v_gsa=0.002, n_heads=16)
    n = 300
    (kb, k), (vb, v) = (_rows(rng, n, H, D, "bf16") for _ in range(2))
    table = np.array([[n_pages - 1, n_pages - 30, n_pages - 7]], np.int32)
    slots = (table[0, np.arange(n) // S].astype(np.int64) * S + np.arange(n) % S).astype(np.int32)
    kv.append(None, to_device(kb, "bf16"), to_device(vb, "bf16"), None, _dev(slots), None, None)
    g = np.full(H, 0.002, np.float32)
    small = np.zeros((3, H, S * D * 9 // 8), np.uint8)
    kc, ks = K.entry(k, g)
    vc, vs = K.entry(v, g)
    K.store(small, np.arange(n), kc, ks, vc, vs, S)
    assert np.array_equal(kv.data[_dev(table[0]).long()].cpu().numpy(), small)
    q, q32 = _queries(rng, 1, 16, D)
    lse = torch.empty(1, 16, device="cuda")
    out, _ = kv.attend(q, _dev(table), _dev(np.array([n], np.int32)), lse=lse)
    ref = K.attention(q32.astype(np.float64), *K.load(small, np.arange(n), S, D, g, g), D ** -0.5)
    assert K.check_attention(out.float().cpu().numpy(), lse.cpu().numpy(), ref, n, np.abs(v).max()) == (0, 0)


COLUMNS = [  # lens, n_q, H, G, D, S, window: 17 to 256 (query, head) columns of a sequence
    ([400, 90], [3, 3], 2, 8, 128, 64, 0), ([400, 90], [4, 4], 2, 8, 64, 32, 0), ([700, 300], [33, 33], 2, 1, 128, 16, 0),
    ([600, 129], [6, 6], 1, 8, 128, 128, 0), ([600, 129], [8, 8], 1, 8, 64, 16, 0), ([500, 260, 7], [13, 13, 13], 2, 5, 128, 32, 0),
    ([900], [16], 1, 8, 128, 64, 200), ([640, 900], [9, 9], 2, 16, 64, 128, 130), ([900, 400], [12, 12], 1, 20, 128, 16, 0),
    ([300, 2000], [16, 16], 2, 16, 128, 64, 0), ([40, 41], [17, 17], 1, 4, 64, 64, 7),
]


@pytest.mark.parametrize("case", COLUMNS, ids=lambda c: "n%d_q%d_H%d_G%d_D%d_S%d_w%d" % (max(c[0]), max(c[1]), *c[2:]))
def test_columns_of_a_few_queries(case):
    test_several_queries_per_sequence(case)


@pytest.mark.parametrize("m", [1, 4, 8, 30])
def test_one_sequence_in_many_parts(m):
    """A single KV head: every block takes part of one key; a window cuts the others off."""
    rng = np.random.default_rng(20 + m)
    C = Cached(rng, [20000], 1, 128, 64)
    q, q32 = _queries(rng, m, 8, 128, loud=4.0)
    for window in (0, 6000):
        out, lse = C.run(q, window=window)
        C.check(q32, [m], out, lse, window=window)


@pytest.mark.parametrize("m", [1, 40])
@pytest.mark.parametrize("D", [64, 128])
def test_one_long_sequence_among_short_ones(m, D):
    """One key in many parts beside many that nothing cuts."""
    rng = np.random.default_rng(60 + m)
    lens = [30] * 30 + [12000] + [50] * 30
    C = Cached(rng, lens, 1, D, 128)
    n_q = [1] * 61
    n_q[30] = m
    q, q32 = _queries(rng, sum(n_q), 4, D, loud=3.0)
    cu = np.concatenate([[0], np.cumsum(n_q)]).astype(np.int32)
    out, lse = C.run(q, cu_q=_dev(cu), max_q=m)
    C.check(q32, n_q, out, lse)


@pytest.mark.parametrize("m", [1, 6, 50])
@pytest.mark.parametrize("rising", [False, True])
def test_maximum_moves_inside_a_tile(m, rising):
    """Scores that rise (or fall) by some powers of two every few tokens."""
    rng = np.random.default_rng(30 + m)
    C = Cached(rng, [500, 333], 1, 128, 32, spread=0.2)
    q, q32 = _queries(rng, 2 * m, 4, 128, loud=0.2)
    # every sequence's token t gets entry c in its first channel: 4-bit values on a coarse grid
    for b, n in enumerate(C.lens):
        k = C.k[b].copy()
        ramp = np.arange(n) if rising else np.arange(n)[::-1]
        k[:, 0, :16] = ((ramp // 5) * 0.01)[:, None]
        kc, ks = K.entry(k.astype(np.float32), C.kg)
        vc, vs = K.entry(C.v[b].astype(np.float32), C.vg)
        slots = C.table[b, np.arange(n) // 32] * 32 + np.arange(n) % 32
        host = C.cache.cpu().numpy()
        K.store(host, slots, kc, ks, vc, vs, 32)
        C.cache = _dev(host)
        C.k[b], C.v[b] = K.load(host, slots, 32, 128, C.kg, C.vg)
    q[..., :16], q32[..., :16] = 32.0, 32.0
    out, lse = C.run(q)
    C.check(q32, [m] * 2, out, lse)


@pytest.mark.parametrize("m", [1, 5, 40])
def test_pages_before_the_window_may_be_freed(m):
    rng = np.random.default_rng(40 + m)
    C = Cached(rng, [700, 90], 2, 64, 16)
    q, q32 = _queries(rng, 2 * m, 16, 64)
    table = C.table.copy()
    table[0, :(700 - m + 1 - 100) // 16] = -1                          # pages that no query sees
    C.args = (_dev(table), C.args[1])
    out, lse = C.run(q, window=100)
    C.check(q32, [m] * 2, out, lse, window=100)


def test_workspace_is_used_again_by_calls_of_other_shapes():
    import nvfp4_router_gate_gb300 as R
    rng = np.random.default_rng(50)
    C = Cached(rng, [3000, 200, 900], 2, 128, 64)
    ws = R.new_workspace(R.nvfp4_kv_attention_workspace_size(300, 3, 16, 2, 128))
    for m in (1, 40, 3, 1, 100, 1):
        q, q32 = _queries(rng, 3 * m, 16, 128)
        out, lse = C.run(q, workspace=ws)
        C.check(q32, [m] * 3, out, lse, rows=4)
    assert R.nvr_read_device_status(ws) == 0


# The same through the tensor-memory kernel, which takes the calls of many columns whose
# page tables are wide.

@pytest.fixture
def wide(monkeypatch):
    monkeypatch.setattr(Cached, "pad", 4096)


@pytest.mark.parametrize("case", MANY + COLUMNS, ids=lambda c: "n%d_q%d_H%d_G%d_D%d_S%d_w%d" % (max(c[0]), max(c[1]), *c[2:]))
def test_wide_tables(wide, case):
    test_several_queries_per_sequence(case)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("m", [40, 90])
def test_wide_tables_without_causal_mask(wide, D, m):
    test_without_causal_mask(D, m)


def test_wide_tables_extremes(wide):
    test_large_scores_and_tiny_queries(40)
    test_pages_outside_the_cache_are_not_seen(40)
    test_maximum_moves_inside_a_tile(50, True)
    test_maximum_moves_inside_a_tile(50, False)
    test_pages_before_the_window_may_be_freed(40)
    test_window_without_end(70)
    test_workspace_is_used_again_by_calls_of_other_shapes()
    test_one_long_sequence_among_short_ones(40, 128)


@pytest.mark.parametrize("D,S,window", [(128, 64, 1), (64, 16, 40), (128, 128, 130), (64, 32, 300), (128, 16, 77)])
def test_windows_of_many_columns(D, S, window):
    rng = np.random.default_rng(90 + window)
    n_q = [220, 150, 1, 64, 0, 200]
    lens = [220, 700, 500, 64, 33, 130]                                # the last has more queries than tokens
    C = Cached(rng, lens, 4, D, S)
    table = C.table.copy()
    table[1, :(700 - 150 + 1 - window) // S] = -1                      # pages in front of every window
    C.args = (_dev(table), C.args[1])
    q, q32 = _queries(rng, sum(n_q), 32, D)
    out, lse = C.run(q, cu_q=_dev(np.concatenate([[0], np.cumsum(n_q)]).astype(np.int32)), max_q=max(n_q), window=window)
    at = 0
    for b, m in enumerate(n_q):
        for i in sorted({0, 1, m // 2, m - 2, m - 1} & set(range(m))):
            n = lens[b] - m + 1 + i                                    # what a query at this place may see
            kk, vv = C.k[b][:max(n, 0)], C.v[b][:max(n, 0)]
            ref = K.attention(q32[at + i:at + i + 1].astype(np.float64), kk, vv, D ** -0.5, window=window)
            vmax = np.abs(C.v[b]).max()
            assert K.check_attention(out[at + i:at + i + 1], lse[at + i:at + i + 1], ref, max(n, 0), vmax) == (0, 0), (b, i)
        at += m
