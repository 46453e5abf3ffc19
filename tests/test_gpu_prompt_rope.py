"""GPU parity of prompt_rope against the float64 oracle (oracle/prompt.py): head
sizes, pairings, axes, types and layouts; positions outside the tables; results
written over their inputs."""

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a GPU")]

from oracle import kv_cache as K  # noqa: E402
from oracle import prompt as P  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _inputs(rng, T, Hq, Hkv, D, pairs, axes, dt, n_pos=300):
    x = rng.standard_normal((T, Hq + 2 * Hkv, D)).astype(np.float32)
    x[..., rng.integers(0, D, 3)] *= 8.0
    fused = _dev(x).to(TYPES[dt])
    ang = rng.uniform(-4, 4, (n_pos, max(pairs, 1)))[:, :pairs]
    cos, sin = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    pos = rng.integers(0, n_pos, (axes, T)).astype(np.int32)
    w = rng.standard_normal((2, D)).astype(np.float32)
    return fused, cos, sin, pos, w


CASES = [  # T, Hq, Hkv, D, sections, turns, interleaved, norm, type in, type out
    (1, 64, 8, 128, (16, 24, 24), False, False, True, "bf16", None),
    (1, 1, 1, 64, (32,), False, False, False, "f32", None),
    (1, 3, 1, 64, (10, 11, 11), True, True, True, "f16", None),
    (5, 3, 3, 64, (8, 24), False, True, True, "bf16", None),
    (17, 6, 2, 128, (11, 11, 10), True, False, True, "f32", "bf16"),
    (33, 5, 5, 128, (16, 16), False, False, False, "f16", None),        # half of the head turns
    (33, 5, 2, 128, (20, 20, 20), True, True, True, "bf16", None),       # 120 channels do
    (29, 7, 1, 128, (28, 28), False, False, True, "bf16", None),         # 112 by halves
    (19, 4, 2, 64, (4, 2, 2), True, False, True, "f32", "f16"),
    (40, 9, 3, 256, (64, 32, 32), False, False, True, "bf16", None),
    (40, 2, 1, 256, (50, 50, 28), True, True, False, "f32", None),
    (9, 2, 1, 128, (9, 8), False, False, True, "bf16", None),            # halves at an odd distance
    (12, 9, 3, 64, (1, 1, 1), False, True, True, "f32", None),
    (21, 4, 4, 80, (16, 12, 12), False, False, True, "bf16", None),      # heads of other sizes
    (21, 4, 4, 96, (48,), False, True, False, "f16", None),
    (3, 8, 8, 2, (1,), False, False, True, "f32", None),
    (7, 4, 2, 102, (17, 17, 17), True, True, True, "f32", "bf16"),
    (700, 32, 8, 128, (16, 24, 24), False, False, True, "bf16", None),   # several groups of heads a warp
    (4100, 64, 8, 128, (22, 21, 21), True, False, True, "bf16", None),   # all of them
    (513, 20, 4, 64, (12, 10, 10), True, True, True, "f32", None),
    (6, 4, 1, 128, (), False, False, True, "bf16", None),                # the norm alone
    (11, 4, 1, 64, (4,) * 8, False, False, True, "bf16", None),          # as many axes as there may be
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: "T%d_H%d_%d_D%d_r%s%s%s%s_%s%s" % (
    c[0], c[1], c[2], c[3], "+".join(map(str, c[4])), "t" if c[5] else "", "i" if c[6] else "", "n" if c[7] else "", c[8],
    c[9] or ""))
def test_rope_matches_the_formula(case):
    import nvfp4_router_gate_gb300 as R
    T, Hq, Hkv, D, sections, turns, inter, norm, dt, out_dt = case
    rng = np.random.default_rng(T * 131 + D + sum(sections))
    axes = R.rope_axes(sections, turns) if sections else ()
    fused, cos, sin, pos, w = _inputs(rng, T, Hq, Hkv, D, len(axes), max(len(sections), 1), dt)
    if T > 4 and axes:
        pos[-1, 2], pos[0, 4] = -1, cos.shape[0]                         # no such rows: zeros
    q, k = fused[:, :Hq], fused[:, Hq:Hq + Hkv]
    keep = fused.clone()
    tables = (_dev(cos), _dev(sin)) if axes else (None, None)
    got = R.prompt_rope(q, k, _dev(pos), *tables, axes=axes, q_weight=_dev(w[0]) if norm else None,
                        k_weight=_dev(w[1]) if norm else None, eps=1e-5, interleaved=inter,
                        out_dtype=TYPES[out_dt] if out_dt else None)
    assert torch.equal(fused, keep)
    for x, y, weight in zip((q, k), got, w):
        assert y.dtype is TYPES[out_dt or dt] and y.is_contiguous()
        ref = P.rope(x.double().cpu().numpy(), pos, axes, cos, sin, inter, weight if norm else None, 1e-5)
        assert P.check_rope(y.double().cpu().numpy(), ref, D, out_dt or dt) == 0


@pytest.mark.parametrize("D,sections,inter", [(128, (16, 24, 24), False), (64, (10, 11, 11), True), (80, (16, 24), False),
                                              (128, (9, 8), False)])
def test_rope_over_its_inputs(D, sections, inter):
    """q_out and k_out are the views of the fused projection that went in; its values stay."""
    import nvfp4_router_gate_gb300 as R
    rng = np.random.default_rng(7 + D)
    axes = R.rope_axes(sections)
    fused, cos, sin, pos, w = _inputs(rng, 333, 12, 4, D, len(axes), len(sections), "bf16")
    args = (_dev(pos), _dev(cos), _dev(sin))
    kw = dict(axes=axes, q_weight=_dev(w[0]), interleaved=inter)
    values = fused[:, 16:].clone()
    q, k = R.prompt_rope(fused[:, :12], fused[:, 12:16], *args, **kw)
    at = fused[:, :12], fused[:, 12:16]
    got = R.prompt_rope(*at, *args, **kw, q_out=at[0], k_out=at[1])
    assert got[0] is at[0] and torch.equal(fused[:, :12], q) and torch.equal(fused[:, 12:16], k)
    assert torch.equal(fused[:, 16:], values)


@pytest.mark.parametrize("D,inter", [(128, False), (64, True)])
def test_rope_of_heads_that_are_not_aligned(D, inter):
    import nvfp4_router_gate_gb300 as R
    rng = np.random.default_rng(8 + D)
    axes = R.rope_axes((D // 4, D // 4))
    fused, cos, sin, pos, w = _inputs(rng, 23, 3, 1, D, len(axes), 2, "bf16")
    big = torch.zeros(23, 3 * D + 5, dtype=torch.bfloat16, device="cuda")
    q = big.as_strided((23, 3, D), (3 * D + 5, D, 1), 3)
    q.copy_(fused[:, :3])
    out = torch.empty(23 * 3 * D + 1, dtype=torch.bfloat16, device="cuda")[1:].view(23, 3, D)
    got = R.prompt_rope(q, None, _dev(pos), _dev(cos), _dev(sin), axes, q_weight=_dev(w[0]), interleaved=inter, q_out=out)[0]
    ref = P.rope(q.double().cpu().numpy(), pos, axes, cos, sin, inter, w[0], 1e-6)
    assert P.check_rope(got.double().cpu().numpy(), ref, D, "bf16") == 0


def test_rope_of_one_side():
    import nvfp4_router_gate_gb300 as R
    rng = np.random.default_rng(9)
    axes = R.rope_axes((20, 22, 22), turns=True)
    fused, cos, sin, pos, w = _inputs(rng, 21, 6, 2, 128, 64, 3, "bf16")
    args = (_dev(pos), _dev(cos), _dev(sin), axes)
    both = R.prompt_rope(fused[:, :6], fused[:, 6:8], *args, q_weight=_dev(w[0]))
    assert torch.equal(R.prompt_rope(fused[:, :6], None, *args, q_weight=_dev(w[0]))[0], both[0])
    only = R.prompt_rope(None, fused[:, 6:8], *args)
    assert only[0] is None and torch.equal(only[1], both[1])


def test_infinities_stay_in_their_pairs():
    """A channel that is not rotated, or another head, is not touched by an infinity beside it."""
    import nvfp4_router_gate_gb300 as R
    rng = np.random.default_rng(10)
    for D, pairs, inter in ((128, 32, False), (64, 20, True), (96, 17, False)):
        fused, cos, sin, pos, _ = _inputs(rng, 5, 2, 1, D, pairs, 1, "f32")
        args = (_dev(pos), _dev(cos), _dev(sin))
        q = fused[:, :2].contiguous()
        want = R.prompt_rope(q, None, *args, interleaved=inter)[0]
        q[2, 1, 2 * pairs + 3] = float("inf")                             # behind the rotated channels
        q[3, 0, 4] = float("nan")
        got = R.prompt_rope(q, None, *args, interleaved=inter)[0]
        other = 5 if inter else 4 + pairs
        hit = torch.zeros_like(got, dtype=torch.bool)
        hit[2, 1, 2 * pairs + 3] = hit[3, 0, 4] = hit[3, 0, other] = True
        assert torch.isinf(got[2, 1, 2 * pairs + 3]) and torch.isnan(got[3, 0, 4]) and torch.isnan(got[3, 0, other])
        assert torch.equal(got[~hit], want[~hit])


def test_text_positions_are_those_of_append():
    """Where all axes agree, the heads are what the cache's append makes of one axis."""
    import nvfp4_router_gate_gb300 as R
    rng = np.random.default_rng(11)
    T, Hq, Hkv, D = 70, 8, 2, 128
    fused, _, _, _, w = _inputs(rng, T, Hq, Hkv, D, 64, 1, "bf16")
    cos, sin = R.rope_table(400, D)
    pos = torch.arange(30, 30 + T, dtype=torch.int32, device="cuda")
    kv = R.Nvfp4KVCache(4, Hkv, D, k_gsa=3e-3, v_gsa=3e-3)
    want = kv.append(fused[:, :Hq], fused[:, Hq:Hq + Hkv], fused[:, Hq + Hkv:], pos, pos, cos, sin,
                     q_weight=_dev(w[0]), k_weight=_dev(w[1]))
    got = R.prompt_rope(fused[:, :Hq], fused[:, Hq:Hq + Hkv], pos.repeat(3, 1), cos, sin,
                        axes=R.rope_axes((16, 24, 24)), q_weight=_dev(w[0]), k_weight=_dev(w[1]))
    # both round an fp32 value that is off by a few 2^-24 once: a step of bf16 apart at most, mostly equal
    a, b = got[0].float(), want.float()
    assert bool(((a - b).abs() <= 2.0 ** -7 * b.abs() + 1e-6).all()) and float((a == b).float().mean()) > 0.99
    # the keys go into the cache as they are, without a second norm or rotation: the oracle's bytes of them
    # (a magnitude above 2688 k_gsa = 8.1 saturates; some of these are)
    kv.append(None, got[1], fused[:, Hq + Hkv:], None, pos, None, None)
    g = np.full(Hkv, 3e-3, np.float32)
    codes = [c for x in (got[1], fused[:, Hq + Hkv:]) for c in K.entry(x.float().cpu().numpy(), g)]
    host = K.store(np.zeros(tuple(kv.data.shape), np.uint8), pos.cpu().numpy(), *codes, kv.page_size)
    assert np.array_equal(kv.data.cpu().numpy(), host)


def test_tables_of_axes_with_their_own_frequencies():
    import nvfp4_router_gate_gb300 as R
    cos, sin = R.rope_axes_table(50, (3, 5), turns=True, base=100.0)
    axes = R.rope_axes((3, 5), turns=True)
    assert axes == (0, 1, 0, 1, 0, 1, 1, 1)
    j = np.array([0, 0, 1, 1, 2, 2, 3, 4])
    n = np.array([3, 5, 3, 5, 3, 5, 5, 5])
    ang = np.arange(50)[:, None] * 100.0 ** (-j / n)
    np.testing.assert_allclose(cos.cpu().numpy(), np.cos(ang), atol=2.0 ** -23)
    np.testing.assert_allclose(sin.cpu().numpy(), np.sin(ang), atol=2.0 ** -23)


def test_rope_in_a_graph_and_on_another_stream():
    import nvfp4_router_gate_gb300 as R
    rng = np.random.default_rng(12)
    axes = R.rope_axes((16, 24, 24))
    fused, cos, sin, pos, w = _inputs(rng, 50, 8, 2, 128, 64, 3, "bf16")
    args = (_dev(pos), _dev(cos), _dev(sin), axes)
    q, k = fused[:, :8], fused[:, 8:10]
    want = R.prompt_rope(q, k, *args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = R.prompt_rope(q, k, *args, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = [torch.empty_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        R.prompt_rope(q, k, *args, q_out=out[0], k_out=out[1])
    fused.copy_(fused.flip(0))
    graph.replay()
    again = R.prompt_rope(q, k, *args)
    assert all(torch.equal(a, b) for a, b in zip(out, again)) and not torch.equal(out[0], want[0])
