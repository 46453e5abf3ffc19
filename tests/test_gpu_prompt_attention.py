"""GPU parity of prompt_attention against the float64 oracle (oracle/prompt.py):
lengths, heads, masks, types and layouts at the sizes where such a kernel can go
wrong; what may reach a result; prefixes; rows without a sequence."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

from oracle import prompt as P  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


def _cu(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


class Packed:
    """Sequences of nq[b] queries over nk[b] keys (nk None: their own), packed."""

    def __init__(self, seed, nq, H, G, D, dt="bf16", nk=None, spread=1.0, pad=0):
        self.nq, self.nk, self.own = list(nq), list(nq if nk is None else nk), nk is None
        self.H, self.Hq, self.D, self.dt = H, H * G, D, dt
        gen = torch.Generator(device="cuda").manual_seed(seed)

        def rows(T, heads, s):
            x = torch.randn(T, heads, D, generator=gen, device="cuda")
            x[..., torch.randint(0, D, (2,), generator=gen, device="cuda")] *= 3.0
            return (s * x).to(TYPES[dt])
        T, Tk = sum(self.nq) + pad, sum(self.nk) + (pad if nk is None else 0)
        if self.own:                                          # views of one fused projection
            qkv = rows(T, self.Hq + 2 * H, spread)
            self.q, self.k, self.v = qkv[:, :self.Hq], qkv[:, self.Hq:self.Hq + H], qkv[:, self.Hq + H:]
        else:
            self.q, self.k, self.v = rows(T, self.Hq, spread), rows(Tk, H, spread), rows(Tk, H, 1.0)
        self.kw = dict(cu_q=_cu(self.nq), max_q=max(max(self.nq), 1))
        if not self.own:
            self.kw.update(cu_k=_cu(self.nk), max_k=max(self.nk))

    def run(self, **kw):
        import nvfp4_router_gate_gb300 as R
        T = self.q.shape[0]
        att = R.PromptAttention(self.Hq, self.H, self.D)
        lse = torch.full((T, self.Hq), 7.0, device="cuda")
        out = torch.full((T, self.Hq, self.D), 7.0, dtype=TYPES[self.dt], device="cuda")
        att(self.q, self.k, self.v, out=out, lse=lse, **{**self.kw, **kw})
        torch.cuda.synchronize()
        assert att.status() == 0
        return out.double().cpu().numpy(), lse.double().cpu().numpy()

    def check(self, out, lse, prefix=None, rows=None, **kw):
        """Every sequence (its first, last and `rows` more queries when that is given)."""
        rng = np.random.default_rng(0)
        q0 = k0 = 0
        for m, n in zip(self.nq, self.nk):
            q, k, v = (t.double().cpu().numpy() for t in (self.q[q0:q0 + m], self.k[k0:k0 + n], self.v[k0:k0 + n]))
            at = np.arange(m)
            if rows is not None and m > rows + 2:
                at = np.unique(np.concatenate([[0, m - 1], rng.integers(0, m, rows)]))
            for i in ([at] if len(at) == m else at[:, None]):
                # (a query by itself: the last of the keys up to its position)
                last = n - m + int(i[-1]) + 1 if kw.get("causal", True) and len(i) < m else n
                ref = P.attention(q[i], k[:max(last, 0)], v[:max(last, 0)], kw.get("scale", self.D ** -0.5),
                                  kw.get("causal", True), kw.get("window", 0))
                if prefix is not None:
                    ref = P.join(ref, *(t[q0 + i].double().cpu().numpy() for t in prefix))
                bad = P.check_attention(out[q0 + i], lse[q0 + i], ref, n, np.abs(v).max() if n else 0.0, self.dt)
                assert bad == (0, 0), (m, n, i[:4], bad)
            q0, k0 = q0 + m, k0 + n


CASES = [  # queries of the sequences, KV heads, heads of each, D, type
    ([1], 1, 1, 64, "bf16"),
    ([1], 2, 8, 128, "bf16"),
    ([2, 1, 3], 1, 4, 64, "f16"),
    ([37], 8, 4, 128, "bf16"),
    ([127, 128, 129], 2, 1, 128, "bf16"),
    ([256, 255, 257], 1, 1, 64, "f16"),
    ([5, 0, 130, 1, 0, 64], 2, 3, 128, "f16"),
    ([300, 17, 1], 2, 7, 64, "bf16"),
    ([513], 4, 2, 128, "bf16"),
    ([90, 140], 1, 16, 128, "bf16"),
    ([33, 70], 1, 128, 64, "bf16"),                       # a query a row tile
    ([40], 1, 96, 128, "f16"),                            # heads of a KV head in several groups
    ([21, 50], 1, 67, 64, "bf16"),                        # one head at a time
    ([10], 2, 200, 64, "bf16"),
    ([0, 0, 9], 3, 5, 128, "bf16"),
    ([700, 650, 20, 333], 2, 4, 128, "bf16"),
    ([1500], 1, 8, 64, "f16"),
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "n%s_H%dx%d_D%d_%s" % ("+".join(map(str, c[0])), *c[1:]))
def test_causal_prompts(case):
    nq, H, G, D, dt = case
    C = Packed(sum(nq) + G + D, nq, H, G, D, dt)
    C.check(*C.run(), rows=40)


@pytest.mark.parametrize("D,dt", [(128, "bf16"), (64, "f16")])
@pytest.mark.parametrize("nq,H,G", [([1], 1, 2), ([129, 3, 128], 2, 4), ([700, 90], 1, 1), ([260], 3, 3)])
def test_prompts_that_see_all(nq, H, G, D, dt):
    C = Packed(1 + sum(nq), nq, H, G, D, dt)
    C.check(*C.run(causal=False), causal=False, rows=40)


@pytest.mark.parametrize("window", [1, 2, 33, 128, 200, 5000, 2 ** 31 - 1])
@pytest.mark.parametrize("nq,H,G,D,dt", [([300, 1, 129], 1, 2, 128, "bf16"), ([900], 2, 16, 64, "f16"), ([700], 1, 1, 128, "bf16")])
def test_windows(nq, H, G, D, dt, window):
    C = Packed(2 + sum(nq), nq, H, G, D, dt)
    C.check(*C.run(window=window), window=window, rows=40)


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 100), (False, 0)])
@pytest.mark.parametrize("nq,nk,H,G,D,dt", [
    ([1], [1000], 2, 8, 128, "bf16"),                     # one query over a long sequence
    ([3, 1, 2], [1, 0, 700], 1, 4, 64, "f16"),            # more queries than keys; no keys
    ([64, 300], [700, 200], 2, 2, 128, "bf16"),
    ([2, 0, 5], [0, 9, 0], 1, 1, 64, "bf16"),
    ([130], [2000], 4, 4, 64, "f16"),
    ([1, 1, 1], [5000, 17, 300], 1, 8, 128, "bf16"),
])
def test_other_numbers_of_keys(nq, nk, H, G, D, dt, causal, window):
    C = Packed(3 + sum(nk), nq, H, G, D, dt, nk=nk)
    C.check(*C.run(causal=causal, window=window), causal=causal, window=window, rows=40)


def test_no_keys_at_all():
    C = Packed(4, [3, 2], 1, 2, 64, nk=[0, 0])
    out, lse = C.run()
    assert (out == 0).all() and np.isneginf(lse).all()


@pytest.mark.parametrize("seed,nq,nk,H,G,D,dt", [
    (5, [1], [20000], 1, 8, 128, "bf16"),                 # one key over all blocks
    (6, [2000], None, 1, 1, 128, "bf16"),
    (7, [3000], None, 1, 4, 64, "f16"),
    (8, [900, 1200, 50], None, 2, 2, 128, "f16"),
])
def test_keys_cut_over_blocks(seed, nq, nk, H, G, D, dt):
    C = Packed(seed, nq, H, G, D, dt, nk=nk)
    C.check(*C.run(), rows=60)


@pytest.mark.parametrize("D,dt", [(128, "bf16"), (64, "f16")])
@pytest.mark.parametrize("nq,H,G", [([5, 300, 0, 64, 1], 2, 4), ([1100], 1, 1)])
def test_prefixes(nq, H, G, D, dt):
    """Rows with a prefix, without one (whatever its rows hold), and with nothing but one; also over its own inputs."""
    nk = [n if b != 3 else 0 for b, n in enumerate(nq)]
    C = Packed(9 + sum(nq), nq, H, G, D, dt, nk=nk)
    T = sum(nq)
    o = torch.randn(T, H * G, D, device="cuda").to(TYPES[dt])
    z = 4.0 + 3.0 * torch.randn(T, H * G, device="cuda")
    z[::3] = -float("inf")
    z[1::7] = 60.0
    C.check(*C.run(prefix=(o, z)), prefix=(o, z), rows=60)
    want = C.run(prefix=(o, z))
    o2 = torch.where(torch.isinf(z)[..., None], torch.full_like(o, float("nan")), o)
    import nvfp4_router_gate_gb300 as R
    att, z2 = R.PromptAttention(H * G, H, D), z.clone()
    att(C.q, C.k, C.v, prefix=(o2, z2), out=o2, lse=z2, **C.kw)
    assert np.array_equal(o2.double().cpu().numpy(), want[0]) and np.array_equal(z2.double().cpu().numpy(), want[1])


def test_a_prompt_in_two_parts_is_the_whole():
    """The second half over its own keys, joined with its result over the first half's."""
    C = Packed(10, [700], 2, 4, 128)
    import nvfp4_router_gate_gb300 as R
    att = R.PromptAttention(8, 2, 128)
    h = 300
    lse = torch.empty(400, 8, device="cuda")
    cu = lambda *n: torch.tensor(n, dtype=torch.int32, device="cuda")    # noqa: E731
    prefix = att(C.q[h:], C.k[:h], C.v[:h], cu_q=cu(0, 400), max_q=400, cu_k=cu(0, h), max_k=h, causal=False, lse=lse)
    out, lse = att(C.q[h:], C.k[h:], C.v[h:], prefix=prefix, lse=torch.empty_like(lse))
    whole = P.attention(*(t.double().cpu().numpy() for t in (C.q, C.k, C.v)), 128 ** -0.5)
    ref = tuple(x[h:] for x in whole)
    # (the prefix's result was rounded to bf16 as well)
    got = out.double().cpu().numpy()
    assert (np.abs(got - ref[0]) <= 2.0 ** -8 * ref[2] * 4 + 1e-6).all()
    assert np.abs(lse.double().cpu().numpy() - ref[1]).max() <= 1e-4


def test_a_chunk_on_a_cached_prefix():
    """Over the 4-bit pages for the prefix, over 16 bits for the chunk itself."""
    import nvfp4_router_gate_gb300 as R
    H, G, D, S = 2, 4, 128, 64
    n0, m = [200, 0, 77], [90, 300, 1]
    gen = torch.Generator(device="cuda").manual_seed(11)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)    # noqa: E731
    kv = R.Nvfp4KVCache(24, H, D, S, k_gsa=2e-3, v_gsa=2e-3, n_heads=H * G)
    table = torch.arange(24, dtype=torch.int32, device="cuda").view(3, 8)
    old = []
    for b, n in enumerate(n0):
        slots = (table[b].long()[torch.arange(n, device="cuda") // S] * S + torch.arange(n, device="cuda") % S).int()
        kv.append(None, rnd(n, H, D), rnd(n, H, D), None, slots, None, None)
        old.append([t.double().cpu().numpy() for t in kv.gather(slots, out_dtype=torch.float32)])
    T = sum(m)
    q, k, v = rnd(T, H * G, D), rnd(T, H, D), rnd(T, H, D)
    cu = _cu(m)
    lens = torch.tensor(n0, dtype=torch.int32, device="cuda")
    lse = torch.empty(T, H * G, device="cuda")
    prefix = kv.attend(q, table, lens, cu_q=cu, max_q=300, causal=False, lse=lse)
    out, lse = R.PromptAttention(H * G, H, D)(q, k, v, cu_q=cu, max_q=300, prefix=prefix, out=prefix[0], lse=prefix[1])
    at = 0
    for b, n in enumerate(m):
        x = [t[at:at + n].double().cpu().numpy() for t in (q, k, v)]
        ref = P.attention(x[0], np.concatenate([old[b][0], x[1]]), np.concatenate([old[b][1], x[2]]), D ** -0.5)
        got = out[at:at + n].double().cpu().numpy()
        # two results rounded to bf16, weights rounded to bf16 or fp16, scores as in check_attention
        e = 2 * (2.0 * 2.0 ** -16 * ref[3] + 2.0 ** -20)
        assert (np.abs(got - ref[0]) <= ref[2] * (e[..., None] + 3 * 2.0 ** -8) + 2.0 ** -8 * np.abs(ref[0])).all(), b
        assert (np.abs(lse[at:at + n].double().cpu().numpy() - ref[1]) <= e + 1e-5).all()
        at += n


@pytest.mark.parametrize("dt", ["bf16", "f16"])
def test_rows_that_no_sequence_covers_are_zero(dt):
    """In front of the first sequence, behind the last one, past max_q in one."""
    C = Packed(12, [40, 300, 9], 2, 4, 64, dt, pad=25)
    out, lse = C.run(cu_q=C.kw["cu_q"] + 11)
    for rows in (slice(0, 11), slice(360, None)):
        assert (out[rows] == 0).all() and np.isneginf(lse[rows]).all()
    whole, z = C.run()
    out, lse = C.run(max_q=100)
    assert (out[140:340] == 0).all() and np.isneginf(lse[140:340]).all()
    keep = np.r_[0:140, 340:349]
    assert np.array_equal(out[keep], whole[keep]) and np.array_equal(lse[keep], z[keep])


def test_offsets_out_of_range_stay_inside():
    C = Packed(13, [40, 60], 1, 2, 128)
    want = C.run()
    cu = C.kw["cu_q"].clone()
    cu[0], cu[2] = -5, 1 << 30
    got = C.run(cu_q=cu)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    cu[1] = -9                                                 # the first sequence is empty, the second has all rows
    out, lse = C.run(cu_q=cu, max_q=100)
    C.nq = C.nk = [100]
    C.check(out, lse)


@pytest.mark.parametrize("D,dt", [(128, "bf16"), (64, "bf16"), (128, "f16")])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_values_that_are_not_seen_do_not_count(D, dt, bad):
    """Infinities and NaNs among the keys and values of later tokens, of other sequences, in front of windows."""
    nq, t = [150, 131, 260], 100                              # token t of the middle one
    C = Packed(14, nq, 2, 4, D, dt)
    for window in (0, 20):
        want = C.run(window=window)
        keep = C.k[150 + t].clone(), C.v[150 + t].clone()
        C.k[150 + t], C.v[150 + t] = bad, bad
        out, lse = C.run(window=window)
        C.k[150 + t], C.v[150 + t] = keep
        sees = np.zeros(sum(nq), bool)
        sees[150 + t:150 + (min(131, t + window) if window else 131)] = True
        assert np.array_equal(out[~sees], want[0][~sees]) and np.array_equal(lse[~sees], want[1][~sees])
        assert not np.isfinite(out[sees]).any()


@pytest.mark.parametrize("D,dt", [(128, "bf16"), (64, "f16")])
def test_infinite_values_reach_those_that_see_them(D, dt):
    C = Packed(15, [200, 90], 1, 2, D, dt)
    C.v[130, 0, 3], C.v[20, 0, 7] = float("inf"), -float("inf")
    C.v[140, 0, 3], C.v[250, 0, 9] = -float("inf"), float("nan")
    C.v[199, 0, D - 1] = float("inf")
    out, lse = C.run()
    assert np.isfinite(lse).all()
    ref = [P.attention(*(t[a:b].double().cpu().numpy() for t in (C.q, C.k, C.v)), D ** -0.5)[0]
           for a, b in ((0, 200), (200, 290))]
    ref = np.concatenate(ref)
    odd = ~np.isfinite(ref)
    assert odd.sum() > 0 and np.array_equal(odd, ~np.isfinite(out))
    assert np.array_equal(out[130:140, :, 3], ref[130:140, :, 3]) and np.isnan(out[140:200, :, 3]).all()
    C.v[odd.nonzero()[0][0]:] = C.v[odd.nonzero()[0][0]:]
    fine = C.v.clone()
    C.v.copy_(torch.where(torch.isfinite(fine), fine, torch.zeros_like(fine)))
    plain, _ = C.run()
    assert np.array_equal(plain[~odd], out[~odd])


def test_nan_queries_and_keys():
    C = Packed(16, [150, 70], 1, 4, 128)
    want = C.run()
    C.q[60, 2, 17] = float("nan")
    out, lse = C.run()
    assert np.isnan(out[60, 2]).all() and np.isnan(lse[60, 2])
    hit = np.zeros(out.shape[:2], bool)
    hit[60, 2] = True
    assert np.array_equal(out[~hit], want[0][~hit]) and np.array_equal(lse[~hit], want[1][~hit])


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("seen_first", ["small", "large"])
def test_maxima_that_move(dt, seen_first):
    """Scores that grow by far more than the weights' range along the tokens, or fall."""
    n, D = 700, 64
    C = Packed(17, [n], 1, 2, D, dt)
    ramp = torch.linspace(0, 1, n, device="cuda")[:, None, None]
    ramp = ramp if seen_first == "small" else 1 - ramp
    C.q.copy_(torch.ones_like(C.q))
    C.k.copy_((40.0 * ramp * torch.ones(n, 1, D, device="cuda")).to(C.k.dtype))
    C.check(*C.run(), rows=80)
    for scale in (0.0, -0.2):
        C.check(*C.run(scale=scale), scale=scale, rows=30)


@pytest.mark.parametrize("lowest", [-65504.0, -float("inf")])
def test_keys_whose_scores_are_the_lowest(lowest):
    """Tokens in front that score the type's lowest value, or -inf: the others share the weight."""
    n, D = 300, 64
    C = Packed(18, [n], 1, 1, D, "f16")
    C.q.copy_(torch.zeros_like(C.q))
    C.q[:, :, 0] = 1.0
    C.k[:200] = 0.0
    C.k[:200, :, 0] = lowest
    out, lse = C.run(scale=1.0)
    k = C.k.double().cpu().numpy()
    k[:200, :, 0] = -65504.0
    ref = P.attention(C.q.double().cpu().numpy()[200:], k, C.v.double().cpu().numpy(), 1.0)
    assert P.check_attention(out[200:], lse[200:], ref, n, np.abs(C.v.double().cpu().numpy()).max(), "f16") == (0, 0)


@pytest.mark.parametrize("D", [64, 128])
def test_strides(D):
    """Heads outermost, padded rows, broadcast keys, one token of a large tensor."""
    import nvfp4_router_gate_gb300 as R
    m, H, G = 260, 2, 4
    C = Packed(19, [m], H, G, D)
    want = C.run()
    att = R.PromptAttention(H * G, H, D)

    def outer(t):
        return t.transpose(0, 1).contiguous().transpose(0, 1)

    def padded(t):
        big = torch.full((t.shape[0], t.shape[1] + 1, D + 8), float("nan"), dtype=t.dtype, device="cuda")
        big[:, :t.shape[1], :D] = t
        return big[:, :t.shape[1], :D]
    for f in (outer, padded, torch.clone):
        out, _ = att(f(C.q), f(C.k), f(C.v))
        assert np.array_equal(out.double().cpu().numpy(), want[0]), f
    out, _ = att(C.q[5:6], C.k[5:6], C.v[5:6])
    one = C.v[5].repeat_interleave(G, 0)
    assert torch.equal(out[0], one)


def test_sequences_of_one_length_need_no_offsets():
    C = Packed(20, [70, 70, 70], 2, 4, 128)
    want = C.run()
    got = C.run(cu_q=None, max_q=70)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


def test_many_sequences_and_workspaces_used_again():
    import nvfp4_router_gate_gb300 as R
    rng = np.random.default_rng(21)
    att = R.PromptAttention(8, 2, 128)
    for nq in (rng.integers(0, 30, 600).tolist(), [1900], rng.integers(0, 400, 20).tolist(), [3]):
        C = Packed(21 + len(nq), nq, 2, 4, 128)
        T = sum(nq)
        lse = torch.empty(T, 8, device="cuda")
        out, _ = att(C.q, C.k, C.v, lse=lse, **C.kw)
        C.check(out.double().cpu().numpy(), lse.double().cpu().numpy(), rows=4 if len(nq) > 100 else 30)
    assert att.status() == 0


def test_results_do_not_depend_on_the_run():
    C = Packed(22, [1500, 20, 800], 2, 2, 128)
    a = C.run()
    for _ in range(3):
        b = C.run()
        assert np.array_equal(a[0], b[0]) and np.array_equal(a[1], b[1])


def test_an_empty_call():
    import nvfp4_router_gate_gb300 as R
    att = R.PromptAttention(8, 2, 64)
    q, k = torch.empty(0, 8, 64, device="cuda", dtype=torch.bfloat16), torch.empty(0, 2, 64, device="cuda", dtype=torch.bfloat16)
    out, _ = att(q, k, k)
    assert out.shape == (0, 8, 64)
    out, _ = att(q, k, k, cu_q=torch.zeros(4, dtype=torch.int32, device="cuda"), max_q=0)
    assert out.shape == (0, 8, 64)


def test_a_captured_call_and_two_streams():
    import nvfp4_router_gate_gb300 as R
    C = Packed(23, [300, 90], 2, 4, 128)
    att = R.PromptAttention(8, 2, 128)
    want, _ = att(C.q, C.k, C.v, **C.kw)
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        att(C.q, C.k, C.v, out=out, **C.kw)
    # new lengths and values in the same buffers
    C.kw["cu_q"].copy_(_cu([10, 280]))
    C.q.copy_(C.q.flip(0))
    graph.replay()
    again, _ = att(C.q, C.k, C.v, **C.kw)
    assert torch.equal(out, again) and not torch.equal(out, want)
    assert bool((out[290:] == 0).all())
    # two streams at once, each with a workspace of its own
    streams = [torch.cuda.Stream() for _ in range(2)]
    ws = [torch.zeros_like(att.workspace) for _ in streams]
    torch.cuda.synchronize()
    got = [att(C.q, C.k, C.v, workspace=w, stream=s, **C.kw)[0] for _ in range(3) for w, s in zip(ws, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(g, again) for g in got)
