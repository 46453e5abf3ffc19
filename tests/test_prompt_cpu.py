"""A prompt's operators without a GPU: the oracle against the formulas, what the
entry points and the binding refuse, the axes of rotary positions."""

import ctypes
import math

import numpy as np
import pytest

from oracle import prompt as P
from test_abi_cpu import _lib


def test_oracle_rotation_is_a_rotation_of_pairs():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((5, 2, 12))
    ang = rng.uniform(-3, 3, (9, 4))
    pos = rng.integers(0, 9, (3, 5))
    axes = (0, 2, 1, 2)
    for inter in (False, True):
        y, mag = P.rope(x, pos, axes, np.cos(ang), np.sin(ang), inter)
        for i, a in enumerate(axes):
            ia, ib = (2 * i, 2 * i + 1) if inter else (i, i + 4)
            want = (x[..., ia] + 1j * x[..., ib]) * np.exp(1j * ang[pos[a], i])[:, None]
            assert np.allclose(y[..., ia], want.real) and np.allclose(y[..., ib], want.imag)
        assert np.array_equal(y[..., 8:], x[..., 8:]) and (mag >= np.abs(y) - 1e-12).all()
    w = rng.standard_normal(12)
    y, _ = P.rope(x, pos, (), np.zeros((1, 0)), np.zeros((1, 0)), False, w, 0.5)
    assert np.allclose(y, w * x / np.sqrt((x ** 2).mean(-1, keepdims=True) + 0.5))
    pos[1, 3] = 9
    y, _ = P.rope(x, pos, axes, np.cos(ang), np.sin(ang), True)
    assert (y[3] == 0).all() and (y[2] != 0).any()


@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 3)])
def test_oracle_attention_is_a_sum_over_seen_keys(causal, window):
    rng = np.random.default_rng(1)
    m, n = 5, 7
    q, k, v = rng.standard_normal((m, 4, 6)), rng.standard_normal((n, 2, 6)), rng.standard_normal((n, 2, 6))
    out, lse, mag, big = P.attention(q, k, v, 0.3, causal, window)
    for i in range(m):
        seen = [t for t in range(n) if not causal or (t <= n - m + i and (not window or t > n - m + i - window))]
        for h in range(4):
            p = [math.exp(0.3 * float(q[i, h] @ k[t, h // 2])) for t in seen]
            assert np.allclose(out[i, h], sum(x * v[t, h // 2] for x, t in zip(p, seen)) / sum(p))
            assert np.isclose(lse[i, h], math.log(sum(p)))
            assert np.allclose(mag[i, h], sum(x * abs(v[t, h // 2]) for x, t in zip(p, seen)) / sum(p))
            assert np.isclose(big[i, h], max(0.3 * float(abs(q[i, h]) @ abs(k[t, h // 2])) for t in seen))


def test_oracle_rows_that_see_nothing_and_the_join():
    rng = np.random.default_rng(2)
    q, k, v = rng.standard_normal((4, 2, 6)), rng.standard_normal((9, 1, 6)), rng.standard_normal((9, 1, 6))
    out, lse, _, _ = P.attention(q, k[:2], v[:2], 0.4)                    # two queries in front of the first key
    assert (out[:2] == 0).all() and np.isneginf(lse[:2]).all() and np.isfinite(lse[2:]).all()
    whole = P.attention(q, k, v, 0.4, False)
    a, b = P.attention(q, k[:4], v[:4], 0.4, False), P.attention(q, k[4:], v[4:], 0.4, False)
    o, z, _, _ = P.join(b, a[0], a[1])
    assert np.allclose(o, whole[0]) and np.allclose(z, whole[1])
    none = np.full(a[1].shape, -np.inf)
    o, z, _, _ = P.join(b, np.full(a[0].shape, np.nan), none)             # a prefix of nothing does not count
    assert np.allclose(o, b[0]) and np.allclose(z, b[1])


def test_oracle_checks_notice_mistakes():
    """A key too many, a key too few, a neighbour's head: each is outside the tolerance."""
    rng = np.random.default_rng(3)
    q, k, v = rng.standard_normal((40, 2, 64)), rng.standard_normal((40, 2, 64)), rng.standard_normal((40, 2, 64))
    ref = P.attention(q, k, v, 0.125)
    assert P.check_attention(ref[0], ref[1], ref, 40, np.abs(v).max(), "bf16") == (0, 0)
    for wrong in (P.attention(q, k, v, 0.125, True, 39), P.attention(q, k[:, ::-1], v[:, ::-1], 0.125),
                  P.attention(q, k, v, 0.125, False), P.attention(q, k, v, 0.126)):
        for dt in ("bf16", "f16"):
            assert P.check_attention(wrong[0], wrong[1], ref, 40, np.abs(v).max(), dt) != (0, 0)
    x = rng.standard_normal((6, 2, 16))
    ang, pos = rng.uniform(-3, 3, (9, 8)), rng.integers(0, 9, (2, 6))
    args = (pos, (0, 0, 0, 0, 1, 1, 1, 1), np.cos(ang), np.sin(ang))
    ref = P.rope(x, *args, False)
    assert P.check_rope(ref[0], ref, 16, "bf16") == 0
    assert P.check_rope(P.rope(x, *args, True)[0], ref, 16, "bf16") > 0
    assert P.check_rope(P.rope(x, pos[::-1], *args[1:], False)[0], ref, 16, "bf16") > 0


def test_rope_entry_point_refuses_bad_arguments():
    nat = _lib()
    L = nat.lib()
    fake, odd = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10001)
    INV, UNS, ALI = nat.NVR_ERR_INVALID_ARG, nat.NVR_ERR_UNSUPPORTED, nat.NVR_ERR_ALIGNMENT

    def call(**kw):
        a = dict(q=fake, qs=1024, k=fake, ks=256, dt=nat.NVR_BF16, T=4, Hq=8, Hkv=2, D=128, pos=fake, step=4, n_axes=3,
                 axes=bytes([0, 1, 2, 2] * 16), cos=fake, sin=fake, n_pos=100, rot=128, inter=0, qw=None, kw=None,
                 eps=1e-6, qo=fake, qos=1024, ko=fake, kos=256, out_dt=nat.NVR_BF16)
        a.update(kw)
        return L.prompt_rope(*a.values(), None)

    for bad in (dict(T=-1), dict(Hq=-1), dict(Hkv=-1), dict(Hq=0, Hkv=0), dict(Hq=65537), dict(dt=7), dict(out_dt=7),
                dict(out_dt=nat.NVR_F32), dict(out_dt=nat.NVR_F16), dict(D=0), dict(D=127), dict(rot=-2), dict(rot=130),
                dict(rot=5), dict(eps=-1.0), dict(eps=math.nan), dict(n_pos=0), dict(n_axes=0), dict(n_axes=9),
                dict(axes=None), dict(axes=bytes([0, 1, 2, 3] * 16)), dict(n_axes=2), dict(pos=None), dict(cos=None),
                dict(sin=None), dict(step=-1), dict(q=None), dict(k=None), dict(qo=None), dict(ko=None), dict(qs=1023),
                dict(ks=255), dict(qos=1023), dict(kos=255)):
        assert call(**bad) == INV, bad
    for bad in (dict(q=odd), dict(k=odd), dict(qo=odd), dict(ko=odd), dict(pos=odd), dict(cos=odd), dict(sin=odd),
                dict(qw=odd), dict(kw=odd), dict(dt=nat.NVR_F32, q=ctypes.c_void_p(0x10002)),
                dict(dt=nat.NVR_F32, out_dt=nat.NVR_F32, ko=ctypes.c_void_p(0x10002))):
        assert call(**bad) == ALI, bad
    assert call(D=258, rot=128, qs=1 << 20, ks=1 << 20, qos=1 << 20, kos=1 << 20) == UNS
    assert call(T=0) == nat.NVR_OK
    assert call(T=0, q=None, k=None, qo=None, ko=None, pos=None, cos=None, sin=None) == nat.NVR_OK


def test_attention_entry_point_refuses_bad_arguments():
    nat = _lib()
    L = nat.lib()
    fake, odd, other = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008), ctypes.c_void_p(0x20000)
    INV, UNS, ALI, WS = (nat.NVR_ERR_INVALID_ARG, nat.NVR_ERR_UNSUPPORTED, nat.NVR_ERR_ALIGNMENT,
                         nat.NVR_ERR_WORKSPACE)
    need = L.prompt_attention_workspace_size(8, 2, 128)
    assert need > 0 and L.prompt_attention_workspace_size(8, 2, 64) > 0
    for bad in ((7, 2, 128), (0, 2, 128), (8, 0, 128), (8, 2, 96), (8, -2, 64)):
        assert L.prompt_attention_workspace_size(*bad) == 0, bad

    def call(**kw):
        a = dict(q=fake, qs=1024, qhs=128, k=fake, ks=256, khs=128, v=fake, vs=256, vhs=128, dt=nat.NVR_BF16, T=4, Tk=4,
                 Hq=8, Hkv=2, D=128, cu_q=None, cu_k=None, B=2, max_q=2, max_k=2, scale=0.1, causal=1, window=0,
                 po=None, pl=None, out=other, lse=None, ws=fake, n=need)
        a.update(kw)
        return L.prompt_attention(*a.values(), None)

    for bad in (dict(T=-1), dict(Tk=-1), dict(B=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=7), dict(Hq=131072), dict(dt=7),
                dict(dt=nat.NVR_F32), dict(max_q=-1), dict(max_q=0), dict(max_k=-1), dict(window=-1),
                dict(window=3, causal=0), dict(scale=math.inf), dict(scale=-math.inf), dict(scale=math.nan), dict(ws=None),
                dict(po=fake), dict(pl=fake), dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(out=fake),
                dict(B=0, cu_q=fake), dict(B=3), dict(T=5), dict(Tk=5), dict(qs=120), dict(qs=1028), dict(qhs=120),
                dict(qhs=132), dict(ks=100), dict(khs=0), dict(vs=257), dict(vhs=129), dict(ks=1 << 38), dict(qhs=1 << 38)):
        assert call(**bad) == INV, bad
    for bad in (dict(D=96), dict(D=256), dict(T=1 << 31, B=1 << 30), dict(Tk=1 << 31, cu_k=fake),
                dict(B=(1 << 31) - 1, cu_q=fake)):
        assert call(**bad) == UNS, bad
    for bad in (dict(q=odd), dict(k=odd), dict(v=odd), dict(out=odd), dict(po=odd, pl=fake), dict(cu_q=ctypes.c_void_p(0x10002)),
                dict(cu_k=ctypes.c_void_p(0x10002)), dict(lse=ctypes.c_void_p(0x10002)),
                dict(po=fake, pl=ctypes.c_void_p(0x10002)), dict(ws=ctypes.c_void_p(0x10010))):
        assert call(**bad) == ALI, bad
    assert call(n=need - 1) == WS
    assert call(T=0, Tk=0, B=0, max_q=0, q=None, k=None, v=None, out=None) == nat.NVR_OK


def test_binding_refuses_before_the_library():
    torch = pytest.importorskip("torch")
    import nvfp4_router_gate_gb300 as R
    _lib()
    for heads in ((7, 2, 64), (8, 2, 96), (8, 0, 64)):
        with pytest.raises(ValueError, match="heads"):
            R.PromptAttention(*heads, device="cpu")
    att = R.PromptAttention(8, 2, 64, device="cpu")
    q, k = torch.zeros(3, 8, 64, dtype=torch.bfloat16), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    for f in (att, R.prompt_attention):
        with pytest.raises(ValueError, match="CUDA"):
            f(q, k, k)
    with pytest.raises(ValueError, match="CUDA"):
        R.prompt_rope(q, k, None, None, None)
    with pytest.raises(ValueError, match="CUDA"):
        R.prompt_rope(None, None, None, None, None)


def test_axes_of_pairs():
    import nvfp4_router_gate_gb300 as R
    assert R.rope_axes((2, 3, 1)) == (0, 0, 1, 1, 1, 2)
    assert R.rope_axes((2, 3, 1), turns=True) == (0, 1, 2, 0, 1, 1)
    assert R.rope_axes((0, 2)) == (1, 1) and R.rope_axes([4]) == (0,) * 4
    for bad in ((), (1,) * 9, (2, -1)):
        with pytest.raises(ValueError):
            R.rope_axes(bad)
    cos, sin = R.rope_axes_table(20, (2, 3), base=100.0, device="cpu")
    ang = np.arange(20)[:, None] * 100.0 ** -np.array([0, 1 / 2, 0, 1 / 3, 2 / 3])
    # an fp64 angle and its cosine rounded once to fp32
    assert np.abs(cos.numpy() - np.cos(ang)).max() <= 2.0 ** -24 and np.abs(sin.numpy() - np.sin(ang)).max() <= 2.0 ** -24
