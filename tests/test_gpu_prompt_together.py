"""A prompt's operators as a model uses them: rotary positions, attention of a prompt
over itself and over a cached prefix, the append of its keys and values, steps after
it; captured and replayed.  And what the calls refuse, padded batches, prefixes and
values that are not finite where keys are cut over blocks."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

from oracle import kv_cache as K  # noqa: E402
from oracle import prompt as P  # noqa: E402
from test_gpu_prompt_attention import Packed, _cu  # noqa: E402

H, G, D, PAGE, PAGES = 2, 4, 128, 64, 12
I32 = dict(dtype=torch.int32, device="cuda")


class Block:
    """An attention block over text and pictures: three axes, head norms, 4-bit pages behind it."""

    def __init__(self, B, seed):
        import nvfp4_router_gate_gb300 as R
        self.R, self.B = R, B
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.kv = R.Nvfp4KVCache(B * PAGES, H, D, PAGE, k_gsa=3e-3, v_gsa=2e-3, n_heads=H * G)
        self.table = torch.arange(B * PAGES, **I32).view(B, PAGES)
        self.lens = torch.zeros(B, **I32)
        self.axes = R.rope_axes((16, 24, 24))
        self.cos, self.sin = R.rope_table(2048, D)
        self.norms = 1.0 + 0.2 * torch.randn(2, D, generator=self.gen, device="cuda")
        self.attention = R.PromptAttention(H * G, H, D)

    def tokens(self, T):
        """A fused projection, and positions: every other 40 tokens are a picture of 8 columns."""
        qkv = torch.randn(T, H * (G + 2), D, generator=self.gen, device="cuda").bfloat16()
        t = torch.arange(T, **I32)
        pos = t.repeat(3, 1)
        inside, picture = t % 40, t // 40 % 2 == 1
        pos[0] -= torch.where(picture, inside, 0)
        pos[1] -= torch.where(picture, inside - inside // 8, 0)
        pos[2] -= torch.where(picture, inside - inside % 8, 0)
        return qkv, pos

    def rotate(self, qkv, pos):
        return self.R.prompt_rope(qkv[:, :H * G], qkv[:, H * G:-H], pos, self.cos, self.sin, self.axes,
                                  q_weight=self.norms[0], k_weight=self.norms[1])

    def slots(self, cu, T):
        """The places of the rows in the cache (negative where no sequence has the row)."""
        row = torch.arange(T, **I32)
        b = (torch.searchsorted(cu, row, right=True) - 1).clamp(0, self.B - 1)
        pos = row - cu[b] + self.lens[b]
        at = self.table[b, (pos // PAGE).long().clamp(0, PAGES - 1)] * PAGE + pos % PAGE
        return torch.where(row < cu[-1], at, -1).int()

    def turn(self, qkv, pos, cu, max_q):
        """Tokens of every sequence on top of what the cache holds of it."""
        q, k = self.rotate(qkv, pos)
        v = qkv[:, -H:]
        lse = torch.empty(q.shape[:2], device="cuda")
        before = self.kv.attend(q, self.table, self.lens, cu_q=cu, max_q=max_q, causal=False, lse=lse)
        out, lse = self.attention(q, k, v, cu_q=cu, max_q=max_q, prefix=before, out=before[0], lse=before[1])
        self.kv.append(None, k, v, None, self.slots(cu, q.shape[0]), None, None)
        return q, k, v, out, lse

    def cached(self, b):
        n = int(self.lens[b])
        at = torch.arange(n, **I32)
        slots = (self.table[b, (at // PAGE).long()] * PAGE + at % PAGE).int()
        return [t.double().cpu().numpy() for t in self.kv.gather(slots, out_dtype=torch.float32)] if n else \
            [np.zeros((0, H, D)), np.zeros((0, H, D))]

    def check(self, got, old, n_q):
        q, k, v, out, lse = (t.double().cpu().numpy() for t in got)
        at = 0
        for (ok, ov), m in zip(old, n_q):
            s = slice(at, at + m)
            ref = P.attention(q[s], np.concatenate([ok, k[s]]), np.concatenate([ov, v[s]]), D ** -0.5)
            # the prefix's result was rounded to bf16 once more, its weights to fp16; scores as in check_attention
            e = 2 * (2.0 * 2.0 ** -16 * ref[3] + 2.0 ** -20)
            assert (np.abs(out[s] - ref[0]) <= ref[2] * (e[..., None] + 3 * 2.0 ** -8) + 2.0 ** -8 * np.abs(ref[0])).all()
            assert (np.abs(lse[s] - ref[1]) <= e + 1e-5).all()
            at += m


def test_turns_of_conversations():
    """First prompts, second turns of some (and a new one), then single tokens through the cache alone."""
    m = Block(4, 1)
    for n_q in ([200, 0, 90, 1], [30, 150, 0, 64], [1, 129, 7, 0]):
        T, cu = sum(n_q), _cu(n_q)
        qkv, pos = m.tokens(T)
        old = [m.cached(b) for b in range(4)]
        got = m.turn(qkv, pos, cu, max(n_q))
        # the rotation by itself
        for y, x, w in zip(got[:2], (qkv[:, :H * G], qkv[:, H * G:-H]), m.norms.cpu().numpy()):
            ref = P.rope(x.double().cpu().numpy(), pos.cpu().numpy(), m.axes, m.cos.cpu().numpy(), m.sin.cpu().numpy(), False,
                         w, 1e-6)
            assert P.check_rope(y.double().cpu().numpy(), ref, D, "bf16") == 0
        m.check(got, old, n_q)
        m.lens += torch.tensor(n_q, **I32)
    qkv, pos = m.tokens(4)
    q, k = m.rotate(qkv, pos)
    m.kv.append(None, k, qkv[:, -H:], None, m.slots(torch.arange(5, **I32), 4), None, None)
    m.lens += 1
    out, _ = m.kv.attend(q, m.table, m.lens)
    for b in range(4):
        keys, values = m.cached(b)
        ref = K.attention(q[b:b + 1].double().cpu().numpy(), keys, values, D ** -0.5)
        assert K.check_attention(out[b:b + 1].float().cpu().numpy(), None, ref, len(keys), np.abs(values).max()) == (0, 0)
    assert m.attention.status() == 0 and m.kv.status() == 0


def test_turns_from_a_graph():
    """One captured turn of padded batches, replayed with other lengths, equals the calls one by one."""
    T, most = 260, 140
    m, n = Block(3, 2), Block(3, 2)
    qkv, pos, cu = torch.zeros(T, H * (G + 2), D, dtype=torch.bfloat16, device="cuda"), torch.zeros(3, T, **I32), torch.zeros(4, **I32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):                          # (an empty batch: it stores nothing)
        n.turn(qkv, pos, cu, most)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = n.turn(qkv, pos, cu, most)
    for n_q in ([100, 140, 20], [0, 0, 1], [90, 17, 128]):
        rows, where = m.tokens(T)
        c = _cu(n_q)
        for a, b in ((qkv, rows), (pos, where), (cu, c)):
            a.copy_(b)
        graph.replay()
        want = m.turn(rows, where, c, most)
        t = sum(n_q)
        assert torch.equal(got[3], want[3]) and torch.equal(got[4], want[4])
        assert bool((got[3][t:] == 0).all()) and bool(torch.isneginf(got[4][t:]).all())
        assert torch.equal(m.kv.data, n.kv.data)
        for x in (m, n):
            x.lens += torch.tensor(n_q, **I32)


def test_a_batch_of_almost_nothing_but_padding():
    C = Packed(30, [5, 0, 130], 2, 4, 64, pad=20000)
    out, lse = C.run()
    assert (out[135:] == 0).all() and np.isneginf(lse[135:]).all()
    C.check(out, lse)


@pytest.mark.parametrize("D_,dt,window", [(128, "bf16", 0), (64, "f16", 0), (64, "bf16", 1700)])
def test_prefixes_of_rows_whose_keys_are_cut(D_, dt, window):
    """Written over, where parts of the rows are joined from several blocks."""
    import nvfp4_router_gate_gb300 as R
    C = Packed(31, [3500], 1, 1, D_, dt)
    o = torch.randn(3500, 1, D_, device="cuda").to(C.q.dtype)
    z = 6.0 + torch.randn(3500, 1, device="cuda")
    z[::5] = -float("inf")
    want = C.run(prefix=(o, z), window=window)
    C.check(*want, prefix=(o, z), rows=60, window=window)
    att = R.PromptAttention(1, 1, D_)
    att(C.q, C.k, C.v, prefix=(o, z), out=o, lse=z, window=window, **C.kw)
    assert np.array_equal(o.double().cpu().numpy(), want[0]) and np.array_equal(z.double().cpu().numpy(), want[1])


@pytest.mark.parametrize("D_,dt", [(128, "bf16"), (64, "f16")])
def test_unseen_values_of_keys_that_are_cut(D_, dt):
    C = Packed(32, [3300], 1, 1, D_, dt)
    want = C.run()
    t = 3172                                               # inside a tile of the last group of rows
    C.k[t], C.v[t] = float("nan"), float("inf")
    out, lse = C.run()
    assert np.array_equal(out[:t], want[0][:t]) and np.array_equal(lse[:t], want[1][:t])
    assert np.isnan(out[t:]).all() and np.isnan(lse[t:]).all()
    C.k[t] = 0.0
    out, lse = C.run()
    assert np.array_equal(out[:t], want[0][:t]) and np.isinf(out[t:]).all() and np.isfinite(lse).all()


def test_the_attention_refuses():
    import nvfp4_router_gate_gb300 as R
    att = R.PromptAttention(8, 2, 64)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    q, k = torch.zeros(6, 8, 64, **bf), torch.zeros(6, 2, 64, **bf)
    lse = torch.zeros(6, 8, device="cuda")
    cu = torch.tensor([0, 2, 6], **I32)
    ok = dict(cu_q=cu, max_q=4)
    att(q, k, k, **ok)
    for bad in (dict(cu_q=cu), dict(cu_q=cu.long(), max_q=4), dict(cu_q=cu.cpu(), max_q=4), dict(cu_q=cu[None], max_q=4),
                dict(max_q=4), dict(max_q=0), dict(max_q=1 << 32), dict(ok, cu_k=cu), dict(ok, cu_k=cu[:2], max_k=6),
                dict(ok, cu_k=cu, max_k=1 << 31), dict(ok, window=-1), dict(ok, window=(1 << 32) + 5), dict(ok, window=4, causal=False),
                dict(ok, scale=float("nan")), dict(ok, out=torch.zeros_like(q).float()), dict(ok, out=q), dict(ok, out=q[:5]),
                dict(ok, lse=lse.double()), dict(ok, lse=lse[:, :4]), dict(ok, prefix=(q.clone(), lse[:5])),
                dict(ok, prefix=(q.half(), lse)), dict(ok, workspace=att.workspace[:512]), dict(ok, workspace=att.workspace.cpu())):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            att(q, k, k, **bad)
    for args in ((q, k, k[:5]), (q, k[:5], k[:5]), (q, k.half(), k), (q.float(), k.float(), k.float()), (q[:, :7], k, k),
                 (q.cpu(), k, k), (q, k.cpu(), k), (q[0], k, k), (q, k[0], k[0]), (q.transpose(1, 2), k, k),
                 (q, k.expand(6, 2, 64)[:, :1].expand(6, 2, 64), k)):
        for f in (att, R.prompt_attention):
            with pytest.raises((ValueError, TypeError, RuntimeError, IndexError)):
                f(*args)
    with pytest.raises((ValueError, RuntimeError)):
        R.prompt_attention(torch.zeros(6, 8, 96, **bf), torch.zeros(6, 2, 96, **bf), torch.zeros(6, 2, 96, **bf))
    with pytest.raises((ValueError, RuntimeError)):
        R.prompt_attention(q[:, :7], k, k)
    # an address that is not of 16 bytes
    odd = torch.zeros(6 * 8 * 64 + 4, **bf)[4:].view(6, 8, 64)
    with pytest.raises((ValueError, RuntimeError)):
        att(odd, k, k, **ok)
    torch.cuda.synchronize()
    assert att.status() == 0


def test_the_rotation_refuses():
    import nvfp4_router_gate_gb300 as R
    bf = dict(dtype=torch.bfloat16, device="cuda")
    q, k = torch.zeros(6, 4, 64, **bf), torch.zeros(6, 2, 64, **bf)
    pos, (cos, sin) = torch.zeros(2, 6, **I32), R.rope_table(10, 64)
    axes = R.rope_axes((16, 16))
    w = torch.ones(64, device="cuda")
    R.prompt_rope(q, k, pos, cos, sin, axes, q_weight=w)
    good = dict(positions=pos, cos=cos, sin=sin, axes=axes)
    for bad in (dict(axes=axes[:-1]), dict(axes=(2,) * 32), dict(axes=(-1,) * 32), dict(axes=(300,) * 32), dict(positions=pos.long()),
                dict(positions=pos[:, :5]), dict(positions=pos.cpu()), dict(positions=pos.t().contiguous().t()), dict(positions=None),
                dict(positions=pos[None]), dict(positions=torch.zeros(9, 6, **I32)), dict(sin=None), dict(sin=sin[:5]),
                dict(cos=cos.double()), dict(cos=cos[0]), dict(cos=cos.cpu()), dict(q_weight=w[:32]), dict(k_weight=w.bfloat16()),
                dict(q_weight=w.cpu()), dict(eps=-1.0), dict(eps=float("nan")), dict(out_dtype=torch.float16), dict(out_dtype=torch.float32),
                dict(q_out=q[:5]), dict(q_out=q.float()), dict(k_out=torch.zeros(6, 2, 64, dtype=torch.float16, device="cuda"))):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            R.prompt_rope(q, k, **{**good, **bad})
    for args in ((q, k[:5]), (q, k[:, :, :32]), (q, k.half()), (q.cpu(), k), (q[0], k), (q.transpose(0, 1).contiguous().transpose(0, 1), k),
                 (q.double(), k.double()), (None, None)):
        with pytest.raises((ValueError, TypeError, RuntimeError)):
            R.prompt_rope(*args, **good)
    with pytest.raises((ValueError, RuntimeError)):                       # more pairs than channels
        R.prompt_rope(q[..., :32].contiguous(), None, **good)
    with pytest.raises((ValueError, RuntimeError)):                       # keys' result without keys
        R.prompt_rope(q, None, **good, k_out=k)
    torch.cuda.synchronize()


def test_long_keys_that_are_handed_out_whole():
    """So many that each block gets several: none is cut, in a call and in the next one with its workspace."""
    import nvfp4_router_gate_gb300 as R
    C = Packed(33, [6000, 10], 8, 8, 64)
    att = R.PromptAttention(64, 8, 64)
    lse = torch.empty(6010, 64, device="cuda")
    for _ in range(2):
        out, _ = att(C.q, C.k, C.v, lse=lse, **C.kw)
        C.check(out.double().cpu().numpy(), lse.double().cpu().numpy(), rows=2)
    assert att.status() == 0


@pytest.mark.parametrize("nq", [[5, 300, 0, 1, 77], [0, 0, 0, 2], [40] * 30])
def test_far_more_room_than_queries(nq):
    """max_q of a captured graph's largest batch: the groups behind a sequence's end are passed over."""
    C = Packed(34, nq, 2, 4, 128)
    want = C.run()
    got = C.run(max_q=20000)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


def test_two_graphs_with_one_workspace():
    """Replayed in turn: keys handed out whole in one, cut and joined in the other; counters are back at zero."""
    import nvfp4_router_gate_gb300 as R
    calls = [(Packed(35, [500, 3, 90], 2, 4, 128), {}), (Packed(36, [2, 1], 2, 4, 128, nk=[9000, 40]), {})]
    att = R.PromptAttention(8, 2, 128)
    graphs, outs = [], []
    for C, kw in calls:
        out = torch.empty(C.q.shape, dtype=C.q.dtype, device="cuda")
        att(C.q, C.k, C.v, out=out, **C.kw)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            att(C.q, C.k, C.v, out=out, **C.kw)
        graphs.append(graph)
        outs.append(out)
    want = [o.clone() for o in outs]
    for _ in range(20):
        for g, o, w in zip(graphs, outs, want):
            o.zero_()
            g.replay()
            assert torch.equal(o, w)
    for (C, _), o in zip(calls, outs):
        C.check(o.double().cpu().numpy(), C.run()[1], rows=20)
    assert att.status() == 0


def test_sequences_of_one_length_over_keys_of_others():
    C = Packed(37, [7, 7, 7], 2, 4, 64, nk=[300, 7, 40])
    want = C.run()
    got = C.run(cu_q=None, max_q=None)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    C.check(*want)


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("nq,nk,H,G,D_", [([40], [6000], 1, 4, 128), ([1, 2, 1], [3000, 5, 1300], 2, 8, 64), ([130], [4500], 1, 3, 128),
                                          ([1], [40000], 1, 1, 64)])
def test_few_queries_over_many_keys(nq, nk, H, G, D_, dt):
    """Keys cut into many parts, causal and not, with a window that hides some of the parts."""
    C = Packed(38, nq, H, G, D_, dt, nk=nk)
    C.check(*C.run(), rows=20)
    C.check(*C.run(causal=False), causal=False, rows=20)
    C.check(*C.run(window=1500), window=1500, rows=20)
