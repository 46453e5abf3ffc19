"""What the key/value cache's calls promise beside their values: which bytes
may reach a result, rows that no sequence covers, streams, workspaces and the
buffers of an Nvfp4KVCache."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

from oracle import kv_cache as K  # noqa: E402
from test_gpu_kv_cache import Cached, _dev, _queries  # noqa: E402


class Wide(Cached):
    """Its page tables are wide: calls of more than 32 columns without a window take the tensor-memory kernel."""
    pad = 4096


def _takes_tensor_memory(B, H, cols, tokens):
    """The size rule of csrc/kv_attention.cu for calls of more than 32 columns: tokens is the tables' width, or the
    window and 15 more."""
    tiles = B * H * -(-cols // 16) * -(-tokens // 128)
    return cols > 32 and tiles > 6 * torch.cuda.get_device_properties(0).multi_processor_count


def _overwrite(C, b, tokens, byte, keys=True):
    """Bytes of tokens of sequence b (their codes and scales) in the cache."""
    host = C.cache.cpu().numpy()
    n, H, D = len(tokens), C.H, C.D
    slots = C.table[b, tokens // C.S] * C.S + tokens % C.S
    if not keys:
        kc, ks = _entry_bytes(host, slots, C.S, D)
    else:
        kc, ks = np.full((n, H, D // 2), byte, np.uint8), np.full((n, H, D // 16), byte, np.uint8)
    K.store(host, slots, kc, ks, np.full((n, H, D // 2), byte, np.uint8), np.full((n, H, D // 16), byte, np.uint8), C.S)
    C.cache = _dev(host)


def _entry_bytes(host, slots, S, D):
    """Key codes and scales as they lie in the cache."""
    at = K.region_offsets(S, D)[0]
    page = host[slots // S]
    t = (slots % S)[:, None, None]
    row, head = np.arange(len(slots))[:, None, None], np.arange(host.shape[1])[None, :, None]
    return (page[row, head, t * (D // 2) + np.arange(D // 2)], page[row, head, at + t * (D // 16) + np.arange(D // 16)])


# m queries a sequence, KV heads, heads of each: one query and a few through the
# streaming kernel, many columns through the tensor-memory kernel
FORMS = [(1, 2, 8), (5, 1, 3), (40, 8, 16)]


@pytest.mark.parametrize("byte", [0x7F, 0xFF])
@pytest.mark.parametrize("D,S", [(128, 16), (128, 32), (64, 16), (64, 64), (128, 128)])
@pytest.mark.parametrize("m,H,G", FORMS)
def test_bytes_before_the_window_do_not_reach_the_output(m, H, G, D, S, byte):
    """Every token in front of the first query's window holds NaN scales, its page's id still in the table."""
    rng = np.random.default_rng(100 + m + S + D)
    window = 100
    lens = [window + m - 1 + n for n in (5, 18, 300, 411)]             # the windows start at 5, 18, 300 and 411
    if m == 40:
        assert _takes_tensor_memory(len(lens), H, m * G, window + 15)
    C = Cached(rng, lens, H, D, S)
    for b, n in enumerate(lens):
        _overwrite(C, b, np.arange(n - m + 1 - window), byte)
    q, q32 = _queries(rng, m * len(lens), H * G, D)
    out, lse = C.run(q, window=window)
    C.check(q32, [m] * len(lens), out, lse, window=window, rows=4)


@pytest.mark.parametrize("D,S,window", [(128, 64, 0), (64, 16, 0), (128, 16, 33), (64, 128, 50)])
@pytest.mark.parametrize("m,H,G", FORMS[1:])
def test_a_nan_value_reaches_the_queries_that_see_it(m, H, G, D, S, window):
    """One value of a sequence has NaN scales: queries that see it get NaNs, the others what they get without it."""
    rng = np.random.default_rng(130 + m + S)
    lens = [m, 150, 290, 333]
    C = (Wide if window == 0 else Cached)(rng, lens, H, D, S)
    if m == 40:
        assert _takes_tensor_memory(len(lens), H, m * G, window + 15 if window else C.table.shape[1] * S)
    back = [m // 2, 2, m - 1, m // 3 + (window if window else 0)]     # tokens behind the newest
    for b, n in enumerate(lens):
        _overwrite(C, b, np.array([n - 1 - back[b]]), 0x7F, keys=False)
    q, q32 = _queries(rng, m * len(lens), H * G, D)
    out, lse = C.run(q, window=window)
    blind = 0
    for b, n in enumerate(lens):
        for i in range(m):
            pos, t, row = n - m + i, n - 1 - back[b], b * m + i
            sees = t <= pos and (not window or t > pos - window)
            blind += not sees
            assert np.isnan(out[row]).all() if sees else np.isfinite(out[row]).all(), (b, i)
            if 2 < i < m - 3 and i % 7:
                continue
            ref = K.attention(q32[row:row + 1].astype(np.float64), C.k[b][:pos + 1], C.v[b][:pos + 1], D ** -0.5,
                              window=window)
            got = ref[0] if sees else out[row:row + 1]                 # the lse is that of the scores
            assert K.check_attention(got, lse[row:row + 1], ref, pos + 1, np.abs(C.v[b]).max()) == (0, 0), (b, i)
    assert blind > 0


@pytest.mark.parametrize("form", [(Cached, [90, 40], 1), (Cached, [20000, 3], 1), (Wide, [600, 64], 40)],
                         ids=["one", "many_parts", "many_columns"])
def test_nan_queries_have_a_nan_lse(form):
    kind, lens, m = form
    rng = np.random.default_rng(150 + m)
    C = kind(rng, lens, 1, 128, 64)
    q, q32 = _queries(rng, 2 * m, 8, 128)
    bad = (m // 2, 3)                                                  # (query, head) of the first sequence
    q[bad[0], bad[1], 17] = float("nan")
    out, lse = C.run(q)
    assert np.isnan(out[bad]).all() and np.isnan(lse[bad])
    assert np.count_nonzero(np.isnan(lse)) == 1 and np.count_nonzero(np.isnan(out).any(axis=-1)) == 1
    ref = K.attention(q32[m:].astype(np.float64), C.k[1], C.v[1], 128 ** -0.5)
    assert K.check_attention(out[m:], lse[m:], ref, lens[1], np.abs(C.v[1]).max()) == (0, 0)


@pytest.mark.parametrize("kind,n,m", [(Cached, 20000, 1), (Cached, 900, 3), (Wide, 3000, 40)])
def test_tokens_beside_a_dominant_one(kind, n, m):
    """A first token of weight 1, whose value is 0, beside many of weight about 2^-27 each.

    Tolerance: the oracle's, but for the absolute rounding of the fp16 weights: 2^-25 a token below the normal
    range, relative to a largest weight of at least 2^7: n 2^-32 v_max."""
    rng = np.random.default_rng(160 + m)
    C = kind(rng, [n], 1, 128, 64)
    k, v = np.zeros((n, 1, 128), np.float32), np.full((n, 1, 128), 0.5, np.float32)
    k[0, :, 0], v[0] = 27 * np.log(2.0) / 8, 0.0
    (kc, ks), (vc, vs) = K.entry(k, C.kg), K.entry(v, C.vg)
    slots = C.table[0, np.arange(n) // 64] * 64 + np.arange(n) % 64
    host = K.store(C.cache.cpu().numpy(), slots, kc, ks, vc, vs, 64)
    C.cache = _dev(host)
    k, v = K.load(host, slots, 64, 128, C.kg, C.vg)
    q32 = np.zeros((m, 4, 128), np.float32)
    q32[..., 0] = 8.0
    out, lse = C.run(_dev(q32).to(torch.bfloat16), scale=1.0)
    o, z, mag, big = K.attention(q32.astype(np.float64), k, v, 1.0)
    assert 2.0 ** -29 * n < np.abs(o[-1]).max() < 2.0 ** -26 * n
    e = 2.0 * 2.0 ** -16 * big + 2.0 ** -20
    tol = mag * (2 * e + 2.0 ** -11 + n * 2.0 ** -23)[..., None] + n * 2.0 ** -32 * np.abs(v).max()
    tol = tol + 2.0 ** -8 * (np.abs(o) + tol)
    assert (np.abs(out - o) <= tol).all(), (out.ravel()[:4], o.ravel()[:4])
    assert (np.abs(lse - z) <= e + n * 2.0 ** -24 + np.abs(z) * 2.0 ** -21).all()


# ------------------------------------------------------- rows of sequences

@pytest.mark.parametrize("kind", [Cached, Wide])
def test_rows_that_no_sequence_covers_are_zero(kind):
    """In front of the first sequence, between the last one and T (a batch padded for a captured graph)."""
    rng = np.random.default_rng(170)
    lens = [50, 0, 333]
    C = kind(rng, lens, 2, 128, 32)
    cu = np.array([3, 10, 10, 15], np.int32)
    T = 700
    q, q32 = _queries(rng, T, 16, 128)
    out = torch.full((T, 16, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    out, lse = C.run(q, cu_q=_dev(cu), max_q=8, out=out)
    covered = np.zeros(T, bool)
    covered[3:15] = True
    assert not out[~covered].any() and np.isneginf(lse[~covered]).all()
    C.check(q32[3:15], [7, 0, 5], out[3:15], lse[3:15])


@pytest.mark.parametrize("kind", [Cached, Wide])
def test_sequences_of_more_than_max_q_rows_keep_their_positions(kind):
    rng = np.random.default_rng(171)
    n_q, most = [10, 5, 20, 6], 6
    lens = [40, 90, 20, 300]
    C = kind(rng, lens, 2, 64, 16)
    cu = np.concatenate([[0], np.cumsum(n_q)]).astype(np.int32)
    q, q32 = _queries(rng, cu[-1], 16, 64)
    out = torch.full((cu[-1], 16, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    out, lse = C.run(q, cu_q=_dev(cu), max_q=most, out=out)
    for b, (m, n) in enumerate(zip(n_q, lens)):
        at, keep = cu[b], min(m, most)
        ref = K.attention(q32[at:at + m].astype(np.float64), C.k[b], C.v[b], 64 ** -0.5)
        ref = [x[:keep] for x in ref]
        assert K.check_attention(out[at:at + keep], lse[at:at + keep], ref, n, np.abs(C.v[b]).max()) == (0, 0), b
        assert not out[at + keep:at + m].any() and np.isneginf(lse[at + keep:at + m]).all(), b


# ------------------------------------------------- windows of many columns

@pytest.mark.parametrize("D,S,window", [(128, 64, 100), (64, 16, 33), (128, 32, 1), (64, 128, 200), (128, 16, 300)])
def test_windows_through_the_tensor_memory_kernel(D, S, window):
    rng = np.random.default_rng(180 + window)
    n_q, lens, H, G = [64, 300, 0, 33, 1, 150], [64, 640, 7, 500, 400, 60], 8, 4
    assert _takes_tensor_memory(len(lens), H, max(n_q) * G, window + 15)
    C = Cached(rng, lens, H, D, S)
    table = C.table.copy()
    for b, (m, n) in enumerate(zip(n_q, lens)):
        if m:
            table[b, :max(n - m + 1 - window, 0) // S] = -1            # pages in front of every window
    C.args = (_dev(table), C.args[1])
    q, q32 = _queries(rng, sum(n_q), H * G, D)
    cu = np.concatenate([[0], np.cumsum(n_q)]).astype(np.int32)
    out, lse = C.run(q, cu_q=_dev(cu), max_q=max(n_q), window=window)
    for b, (m, n) in enumerate(zip(n_q, lens)):
        for i in sorted({0, m // 2, m - 1} & set(range(m))):
            row, see = cu[b] + i, max(n - m + 1 + i, 0)
            ref = K.attention(q32[row:row + 1].astype(np.float64), C.k[b][:see], C.v[b][:see], D ** -0.5, window=window)
            assert K.check_attention(out[row:row + 1], lse[row:row + 1], ref, see, np.abs(C.v[b]).max()) == (0, 0), (b, i)


# ------------------------------------------------------ the object's buffers

def _object(C, **kw):
    import nvfp4_router_gate_gb300 as R
    return R.Nvfp4KVCache(C.cache.shape[0], C.H, C.D, page_size=C.S, k_gsa=_dev(C.kg), v_gsa=_dev(C.vg), data=C.cache, **kw)


def _attend(kv, C, q, **kw):
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    out, lse = kv.attend(q, *C.args, lse=lse, **kw)
    torch.cuda.synchronize()
    return out.float().cpu().numpy(), lse.cpu().numpy()


def test_attend_takes_the_callers_workspace():
    rng = np.random.default_rng(190)
    C = Cached(rng, [9000], 1, 128, 64)                                # one key in many parts
    kv = _object(C, n_heads=8)
    q, q32 = _queries(rng, 1, 8, 128)
    mine = torch.zeros_like(kv.workspace)
    C.check(q32, [1], *_attend(kv, C, q, workspace=mine))
    assert bool(mine.any()) and not bool(kv.workspace.any())
    C.check(q32, [1], *_attend(kv, C, q))
    assert bool(kv.workspace.any())
    with pytest.raises(Exception, match="workspace"):
        kv.attend(q, *C.args, workspace=mine[:256])


def test_buffers_may_be_replaced():
    import nvfp4_router_gate_gb300 as R
    rng = np.random.default_rng(191)
    C, other = Cached(rng, [70, 5], 2, 128, 16), Cached(rng, [70, 5], 2, 128, 16)
    q, q32 = _queries(rng, 2, 4, 128)
    kv = _object(C, n_heads=4)
    kept = kv.data, kv.k_gsa, kv.v_gsa, kv.workspace                   # (alive: a stale pointer would still be readable)
    C.check(q32, [1, 1], *_attend(kv, C, q))
    kv.data, kv.k_gsa, kv.v_gsa = other.cache, _dev(other.kg), _dev(other.vg)
    other.check(q32, [1, 1], *_attend(kv, other, q))
    pos = np.arange(70)
    slots = (other.table[0, pos // 16] * 16 + pos % 16).astype(np.int32)
    k, v = kv.gather(_dev(slots), out_dtype=torch.float32)
    assert np.array_equal(k.cpu().numpy(), other.k[0].astype(np.float32))
    assert np.array_equal(v.cpu().numpy(), other.v[0].astype(np.float32))
    # a number of calibration stands for all heads; stored bytes go by it
    kv.k_gsa = 0.25
    assert kv.k_gsa.tolist() == [0.25, 0.25]
    x = (rng.standard_normal((1, 2, 128))).astype(np.float32)
    kv.append(None, _dev(x), _dev(x), None, _dev(slots[:1]), None, None)
    got = kv.gather(_dev(slots[:1]), out_dtype=torch.float32)
    for g, gsa in zip(got, (np.full(2, 0.25, np.float32), other.vg)):
        c, s = K.entry(x, gsa)
        page = K.store(np.zeros((1, 2, 16 * 144), np.uint8), [0], c, s, c, s, 16)
        assert np.array_equal(g.cpu().numpy(), K.load(page, [0], 16, 128, gsa, gsa)[0].astype(np.float32))
    kv.workspace = torch.zeros_like(kv.workspace)
    with pytest.raises(ValueError):
        kv.data = other.cache[:, :1]
    with pytest.raises((ValueError, RuntimeError)):
        kv.v_gsa = torch.ones(3)
    assert len(kept) == 4 and isinstance(kv, R.Nvfp4KVCache)


def test_calls_larger_than_expected_use_the_same_workspace():
    """Its size goes by the channels of a head alone."""
    rng = np.random.default_rng(192)
    C = Cached(rng, [300], 2, 128, 64)
    kv = _object(C)
    q, q32 = _queries(rng, 260, 8, 128)
    C.check(q32, [260], *_attend(kv, C, q), rows=8)
    assert kv.status() == 0


def test_empty_batches():
    rng = np.random.default_rng(193)
    C = Cached(rng, [5], 2, 64, 16)
    kv = _object(C)
    i32 = dict(dtype=torch.int32, device="cuda")
    q = torch.empty(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    for B in (0, 3):
        out, _ = kv.attend(q, torch.zeros(B, 2, **i32), torch.zeros(B, **i32))
        assert out.shape == (0, 4, 64)
    with pytest.raises(ValueError):
        kv.attend(torch.empty(2, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(0, 2, **i32), torch.zeros(0, **i32))


def test_what_a_call_allocates_belongs_to_its_stream():
    """Calls on another stream while the current one is busy: nothing of theirs waits for it or is written by it."""
    import nvfp4_router_gate_gb300 as R
    rng = np.random.default_rng(194)
    C = Cached(rng, [9000], 1, 128, 64)
    q, q32 = _queries(rng, 1, 8, 128)
    kg, vg, lse = _dev(C.kg), _dev(C.vg), torch.empty(1, 8, device="cuda")
    slots = _dev((C.table[0, :1] * 64).astype(np.int32))
    s = torch.cuda.Stream()

    def calls():
        return (R.nvfp4_kv_attention(q, C.cache, *C.args, kg, vg, lse=lse, stream=s)[0],
                *R.nvfp4_kv_gather(C.cache, slots, kg, vg, 128, out_dtype=torch.float32, stream=s))

    torch.cuda.synchronize()
    calls()                                                            # (the kernels are loaded)
    torch.cuda.synchronize()
    for stream in (torch.cuda.current_stream(), s):                    # free memory of either stream is not zero
        with torch.cuda.stream(stream):
            torch.full((128 << 20,), 255, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    torch.cuda._sleep(400_000_000)                                     # about a fifth of a second
    done = torch.cuda.Event()
    done.record()
    out, k, v = calls()
    s.synchronize()
    assert not done.query()
    with torch.cuda.stream(s):
        out, lse, k, v = (t.float().cpu().numpy() for t in (out, lse, k, v))
    assert not done.query()
    torch.cuda.synchronize()
    C.check(q32, [1], out, lse)
    assert np.array_equal(k, C.k[0][:1].astype(np.float32)) and np.array_equal(v, C.v[0][:1].astype(np.float32))
