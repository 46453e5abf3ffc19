"""What a prompt's operators promise for calls at the edge of their range, on the GPU."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

from oracle import prompt as P  # noqa: E402
from test_gpu_prompt_attention import Packed, _cu  # noqa: E402


def _references(C, **kw):
    """out and lse of the formula, all sequences."""
    refs, q0, k0 = [], 0, 0
    for m, n in zip(C.nq, C.nk):
        q, k, v = (t.double().cpu().numpy() for t in (C.q[q0:q0 + m], C.k[k0:k0 + n], C.v[k0:k0 + n]))
        refs.append(P.attention(q, k, v, kw.get("scale", C.D ** -0.5), kw.get("causal", True), kw.get("window", 0))[:2])
        q0, k0 = q0 + m, k0 + n
    return [np.concatenate(x) for x in zip(*refs)]


@pytest.mark.parametrize("D,dt", [(128, "bf16"), (64, "bf16"), (128, "f16"), (64, "f16")])
@pytest.mark.parametrize("nq,G,kw", [([150, 290], 4, {}), ([150, 290], 4, dict(causal=False)), ([150, 290], 2, dict(window=70)),
                                     ([3300, 40], 1, {})],
                         ids=["causal", "all", "window", "cut"])
def test_a_scale_of_zero_keeps_what_is_not_finite(nq, G, kw, D, dt):
    """0 * NaN and 0 * inf are NaN: in the rows that see them, both results; in no other row."""
    C = Packed(40, nq, 1, G, D, dt)
    kw = dict(kw, scale=0.0)
    want = C.run(**kw)
    C.check(*want, rows=30, **kw)
    C.q[60, G - 1, 17] = float("nan")
    C.k[100, 0, 3] = float("nan")
    C.k[nq[0] + 20, 0, 5], C.k[nq[0] + 30, 0, D - 1] = float("inf"), -float("inf")
    out, lse = C.run(**kw)
    odd = np.isnan(_references(C, **kw)[1])
    # (without a mask every row of both sequences sees a key that is not finite)
    assert odd[60, G - 1] and odd[100].all() and odd[nq[0] + 20].all() and odd.all() == (not kw.get("causal", True))
    assert np.isnan(lse[odd]).all() and np.isnan(out[odd]).all()
    assert np.array_equal(lse[~odd], want[1][~odd]) and np.array_equal(out[~odd], want[0][~odd])


@pytest.mark.parametrize("nq,H,G,D", [([5, 300, 0, 1, 77, 117] + [0] * 122, 8, 8, 64), ([0] * 31 + [900], 2, 4, 128)])
def test_room_for_a_far_larger_batch(nq, H, G, D):
    """A captured graph's max_q and max_k, far above what the buffers hold."""
    C = Packed(41, nq, H, G, D, pad=20)
    want = C.run()
    C.check(*want, rows=20)
    for room in (8192, 131072, 2 ** 31 - 1):
        got = C.run(max_q=room)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    # (more room for keys changes where one is cut over blocks, so the sums' order: both are right)
    C = Packed(42, [3, 0, 40], H, G, D, nk=[2000, 9, 700])
    C.check(*C.run(), rows=20)
    C.check(*C.run(max_q=2 ** 31 - 1, max_k=2 ** 31 - 1), rows=20)


def test_offsets_that_decrease():
    """Rows that several sequences claim are unspecified, however often they are claimed; others, and later calls, are right."""
    import nvfp4_router_gate_gb300 as R
    T, H, D = 21000, 8, 64
    C = Packed(43, [T], H, 1, D)
    att = R.PromptAttention(H, H, D)
    want = att(C.q, C.k, C.v)[0].clone()
    cu = torch.zeros(20001, dtype=torch.int32, device="cuda")
    cu[1::2] = T                                              # 10000 times all rows: more places than fit 31 bits
    att(C.q, C.k, C.v, cu_q=cu, max_q=T, causal=False)
    torch.cuda.synchronize()
    assert att.status() == 0
    assert torch.equal(att(C.q, C.k, C.v)[0], want)
    cu = torch.tensor([0, 300, 200, 500, 700], dtype=torch.int32, device="cuda")    # rows 200 to 300 twice
    out = att(C.q, C.k, C.v, cu_q=cu, max_q=T)[0]
    assert torch.equal(out[:200], want[:200]) and bool((out[700:] == 0).all())
    C.q, C.k, C.v, C.nq, C.nk = C.q[500:700], C.k[500:700], C.v[500:700], [200], [200]
    C.kw = {}
    C.check(out[500:700].double().cpu().numpy(), C.run()[1])
    assert att.status() == 0


@pytest.mark.parametrize("make", ["PromptAttention", "Nvfp4KVCache", "Nvfp4Linear", "RouterGate"])
def test_workspaces_are_zero_before_other_streams_use_them(make):
    """Made behind work that is still running: nothing of the object is under way when it is handed out."""
    import nvfp4_router_gate_gb300 as R
    W = torch.randn(64, 512, device="cuda").bfloat16()
    new = {"PromptAttention": lambda: R.PromptAttention(8, 2, 64), "Nvfp4KVCache": lambda: R.Nvfp4KVCache(4, 2, 64),
           "Nvfp4Linear": lambda: R.Nvfp4Linear(W), "RouterGate": lambda: R.RouterGate(W)}[make]
    new()                                                     # (what the first one allocates and loads)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (torch.cuda.current_stream(), side):
        with torch.cuda.stream(stream):
            torch.cuda._sleep(100_000_000)                    # some 50 ms
            made = new()
            assert stream.query()
        assert not bool(made.workspace.any())
    # and in a capture, where nothing may be waited for
    graph = torch.cuda.CUDAGraph()
    if make in ("PromptAttention", "Nvfp4Linear"):
        with torch.cuda.graph(graph):
            made = new()
        graph.replay()
        torch.cuda.synchronize()
        assert not bool(made.workspace.any())


def test_a_first_call_on_another_stream():
    import nvfp4_router_gate_gb300 as R
    C = Packed(44, [3500, 20], 1, 1, 64)                      # (keys cut over blocks: parts are counted)
    want = C.run()[0]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(100_000_000)
    att = R.PromptAttention(1, 1, 64)
    out, _ = att(C.q, C.k, C.v, stream=side, **C.kw)
    side.synchronize()
    assert np.array_equal(out.double().cpu().numpy(), want) and att.status() == 0


@pytest.mark.parametrize("B,at", [(90, (3, 40, 89)), (3000, (0, 1500, 1501)), (70000, (2, 33000, 69999))])
@pytest.mark.parametrize("lens,H,G", [((3300, 40, 200), 1, 1), ((500, 300, 1), 2, 4)])
def test_sequences_among_many_empty_ones(B, at, lens, H, G):
    """Cut over blocks and handed out whole: groups without queries are passed over."""
    C = Packed(45, lens, H, G, 64)
    n = np.zeros(B, np.int64)
    n[list(at)] = lens
    C.kw["cu_q"] = _cu(n)
    C.check(*C.run(), rows=20)


@pytest.mark.parametrize("D,dt", [(128, "bf16"), (64, "bf16"), (128, "f16"), (64, "f16")])
@pytest.mark.parametrize("nq,G,kw", [([150, 290], 4, {}), ([150, 290], 4, dict(causal=False)), ([150, 290], 2, dict(window=70)),
                                     ([3300, 40], 1, {}), ([3300, 40], 1, dict(scale=-0.1))],
                         ids=["causal", "all", "window", "cut", "negative"])
def test_nan_and_infinite_keys(nq, G, kw, D, dt):
    """Beside finite values: a NaN reaches the rows that see its key, in tiles with masks and without; an infinity as
    its score says: nothing, or NaNs."""
    C = Packed(46, nq, 1, G, D, dt)
    C.q.copy_(C.q.abs() + 0.125)                              # (scores of infinities have the infinity's sign)
    want = C.run(**kw)
    C.k[100, 0, 3] = float("nan")
    C.k[nq[0] + 20, 0, 5], C.k[nq[0] + 30, 0, D - 1] = float("inf"), -float("inf")
    if nq[0] > 3000:
        C.k[3090, 0, 9] = float("inf")
    out, lse = C.run(**kw)
    ref = _references(C, **kw)
    odd = np.isnan(ref[1])
    low = np.zeros(odd.shape, bool)                           # rows that see a score of -inf beside finite ones
    for row, value in ((20, "inf"), (30, "-inf")):
        if (value == "-inf") == (kw.get("scale", 1.0) > 0):
            low[nq[0] + (0 if not kw.get("causal", True) else row):nq[0] + (row + kw["window"] if kw.get("window") else nq[1])] = True
    assert odd.any() and np.isnan(lse[odd]).all() and np.isnan(out[odd]).all()
    same = ~odd & ~low
    assert np.array_equal(lse[same], want[1][same]) and np.array_equal(out[same], want[0][same])
    low &= ~odd
    assert np.isfinite(out[low]).all() and np.isfinite(lse[low]).all()
    # scores by check_attention's bound, 2 * 2^-16 of a sum |q k| of some 10, 3300 keys' sum 2^-12, lse 2^-21 of itself
    assert not low.any() or (np.abs(lse[low] - ref[1][low]) <= 1e-3 * np.maximum(np.abs(ref[1][low]), 1.0)).all()


def test_heads_that_lie_past_31_bits():
    """Heads outermost, 2^30 elements apart: the third one's start behind 2^31 elements, its bytes behind 2^32."""
    import nvfp4_router_gate_gb300 as R
    m, H, G, D = 300, 3, 2, 64
    C = Packed(47, [m], H, G, D)
    want = C.run()
    far = (1 << 30) + 64
    big = torch.empty(2 * far + (2 * m + 8) * D * 3, dtype=torch.bfloat16, device="cuda")
    k, v = (big[i * m * D:].as_strided((m, H, D), (D, far, 1)) for i in (0, 1))
    q = big[2 * m * D:].as_strided((m, H * G, D), (D, far // 4, 1))     # (six heads, 2^28 apart)
    for view, t in ((q, C.q), (k, C.k), (v, C.v)):
        view.copy_(t)
    out, _ = R.PromptAttention(H * G, H, D)(q, k, v)
    assert np.array_equal(out.double().cpu().numpy(), want[0])


def test_queries_and_results_of_more_than_31_bits():
    """2^31 elements and some: the rotation over its inputs and the attention, at the end of the rows."""
    import nvfp4_router_gate_gb300 as R
    Hq, Hkv, D, n = 64, 2, 128, 110
    B = -(-(1 << 31) // (Hq * D * n)) + 3
    T = B * n
    assert T * Hq * D > 1 << 31
    gen = torch.Generator(device="cuda").manual_seed(48)
    q = torch.randn(T, Hq, D, generator=gen, device="cuda", dtype=torch.bfloat16)
    k, v = (torch.randn(T, Hkv, D, generator=gen, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    cos, sin = R.rope_table(n, D)
    pos = torch.arange(T, dtype=torch.int32, device="cuda") % n
    tail = slice(T - 2 * n, T)
    before = q[tail].double().cpu().numpy()
    R.prompt_rope(q, None, pos, cos, sin, q_out=q)
    host = lambda t: t.double().cpu().numpy()    # noqa: E731
    ref = P.rope(before, pos[None, tail].cpu().numpy(), (0,) * 64, cos.cpu().numpy(), sin.cpu().numpy(), False)
    assert P.check_rope(host(q[tail]), ref, D, "bf16") == 0
    lse = torch.empty(T, Hq, device="cuda")
    att = R.PromptAttention(Hq, Hkv, D)
    out, _ = att(q, k, v, max_q=n, lse=lse)
    for b in (0, B // 2, B - 2, B - 1):
        s = slice(b * n, (b + 1) * n)
        ref = P.attention(host(q[s]), host(k[s]), host(v[s]), D ** -0.5)
        assert P.check_attention(host(out[s]), host(lse[s]), ref, n, np.abs(host(v[s])).max(), "bf16") == (0, 0)
    assert att.status() == 0


@pytest.mark.parametrize("D,dt", [(128, "bf16"), (64, "f16")])
@pytest.mark.parametrize("nq,nk,H,G", [
    ([1] * 2000, ([3] + [0] * 9) * 200, 1, 1),            # several keys a block, most without tiles: whole
    ([40, 1, 1, 1, 1] * 60, [50, 0, 0, 0, 0] * 60, 4, 8),
    ([9, 3, 2, 5] * 100, [7000, 0, 0, 0] + [0] * 396, 2, 4),                    # and among those that are cut
    ([1500, 600, 1, 1] * 2, [100, 5, 0, 0] * 2, 8, 4),    # most queries in front of the first key
])
@pytest.mark.parametrize("causal", [True, False])
def test_several_in_a_row_that_see_nothing(nq, nk, H, G, causal, D, dt):
    """Sequences, and groups of queries, without a key to see: zeros, and nobody waits for their products."""
    C = Packed(49, nq, H, G, D, dt, nk=nk)
    out, lse = C.run(causal=causal)
    C.check(out, lse, causal=causal, rows=4)
    o = torch.randn(C.q.shape, device="cuda").to(C.q.dtype)
    z = torch.randn(C.q.shape[:2], device="cuda")
    z[::5] = -float("inf")
    C.check(*C.run(causal=causal, prefix=(o, z)), prefix=(o, z), causal=causal, rows=4)
