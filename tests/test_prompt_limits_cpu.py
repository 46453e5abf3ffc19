"""Which calls the prompt's operators refuse for their size or for what their arguments
are to each other, without a GPU: every call here is refused for one reason or another, so
nothing is launched."""

import ctypes

import pytest

from test_abi_cpu import _lib

LIMIT = 2 ** 31 - 2 ** 24


def _attend(**kw):
    """prompt_attention into a workspace that is too small: NVR_ERR_WORKSPACE where nothing else is wrong."""
    nat = _lib()
    fake, other = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x20000)
    a = dict(T=4, Tk=None, Hq=64, Hkv=8, D=128, cu_q=None, cu_k=None, B=1, max_q=None, max_k=0, scale=0.1, causal=1,
             window=0)
    a.update(kw)
    T = a["T"]
    Tk = T if a["Tk"] is None else a["Tk"]
    max_q = T if a["max_q"] is None else a["max_q"]
    cu_q, cu_k = (fake if a[x] else None for x in ("cu_q", "cu_k"))
    return nat.lib().prompt_attention(
        fake, a["Hq"] * a["D"], a["D"], fake, a["Hkv"] * a["D"], a["D"], fake, a["Hkv"] * a["D"], a["D"], nat.NVR_BF16, T, Tk,
        a["Hq"], a["Hkv"], a["D"], cu_q, cu_k, a["B"], max_q, a["max_k"], a["scale"], a["causal"], a["window"], None, None,
        other, None, fake, 256, None)


@pytest.mark.parametrize("Hq,Hkv", [(64, 8), (64, 64), (64, 1), (8, 8)])
def test_the_largest_prompt(Hq, Hkv):
    """On each side of P (2 n + 5) = 2^31 - 2^24, P pairs of row tiles over n tiles of keys."""
    nat = _lib()
    s = 256 * Hkv // Hq
    groups = 1
    while Hkv * (groups + 1) * (2 * -(-s * (groups + 1) // 128) + 5) < LIMIT:
        groups += 1
    assert _attend(T=groups * s, Hq=Hq, Hkv=Hkv) == nat.NVR_ERR_WORKSPACE
    for n in (groups + 1, 4 * groups):
        assert _attend(T=n * s, Hq=Hq, Hkv=Hkv) == nat.NVR_ERR_UNSUPPORTED
        # a window leaves few tiles of them; few queries over as many keys are few pairs
        assert _attend(T=n * s, Hq=Hq, Hkv=Hkv, window=1024) == nat.NVR_ERR_WORKSPACE
        assert _attend(T=64, Tk=n * s, cu_k=True, max_k=n * s, Hq=Hq, Hkv=Hkv) == nat.NVR_ERR_WORKSPACE
    if (Hq, Hkv) == (64, 8):
        assert _attend(T=738304) == nat.NVR_ERR_WORKSPACE and _attend(T=738432) == nat.NVR_ERR_UNSUPPORTED


def test_room_above_the_batch_does_not_count():
    """One long prompt with short ones, and a captured graph's largest batch: the work of T queries counts."""
    nat = _lib()
    WS, UNS = nat.NVR_ERR_WORKSPACE, nat.NVR_ERR_UNSUPPORTED
    long_and_short = 131072 + 31 * 40
    assert _attend(T=long_and_short, cu_q=True, B=32, max_q=131072) == WS
    for T in (500, 32000, 65536):
        for max_q in (512, 8192, 131072, 2 ** 31 - 1):
            assert _attend(T=T, cu_q=True, B=128, max_q=max_q) == WS, (T, max_q)
            assert _attend(T=T, Tk=T + 7, cu_q=True, cu_k=True, B=128, max_q=max_q, max_k=2 ** 31 - 1) == WS
    # sequences of their own room each: as many pairs as queries and sequences make
    assert _attend(T=100 * 7, B=100, max_q=7) == WS
    assert _attend(T=1 << 20, cu_q=True, B=1 << 20, max_q=1 << 20) == UNS          # more items than are gone through
    assert _attend(T=1 << 20, cu_q=True, B=1 << 14, max_q=1 << 20) == UNS          # (2^20 / 32 + 2^14 groups of 8192 tiles)
    assert _attend(T=1 << 20, cu_q=True, B=1 << 14, max_q=1 << 12) == WS


def test_no_queries_need_nothing():
    nat = _lib()
    assert _attend(T=0, B=0, max_q=2 ** 31 - 1) == nat.NVR_ERR_WORKSPACE
    assert _attend(T=0, Tk=1 << 20, cu_q=True, cu_k=True, B=3, max_q=2 ** 31 - 1, max_k=2 ** 31 - 1) == nat.NVR_ERR_WORKSPACE


def test_the_most_sequences():
    nat = _lib()
    assert _attend(T=64, cu_q=True, B=1 << 24, max_q=1) == nat.NVR_ERR_WORKSPACE
    assert _attend(T=64, cu_q=True, B=(1 << 24) + 1, max_q=1) == nat.NVR_ERR_UNSUPPORTED


def test_the_longest_stretch_of_keys():
    """More than 2^18 tiles of keys only where 128 blocks share them out below that."""
    nat = _lib()
    WS, UNS = nat.NVR_ERR_WORKSPACE, nat.NVR_ERR_UNSUPPORTED
    few, many = dict(Hq=1, Hkv=1, T=1), dict(Hq=8, Hkv=8, T=19 * 256)              # 1 pair of row tiles, and 152
    for n in (1 << 18, (1 << 18) + 1, 1 << 20, 1 << 23):
        assert _attend(Tk=128 * n, cu_k=True, max_k=128 * n, **few) == WS
    for n, want in ((1 << 18, WS), ((1 << 18) + 1, UNS), (1 << 20, UNS)):
        assert _attend(Tk=128 * n, cu_k=True, max_k=128 * n, **many) == want
        assert _attend(Tk=128 * n, cu_k=True, max_k=128 * n, window=5000, **many) == WS
    # on each side of P (2 n + 5) = 2^26 + 2^8
    heads = 16
    n = (2 ** 26 + 2 ** 8 - 1) // heads // 2 - 2
    assert heads * (2 * n + 5) < 2 ** 26 + 2 ** 8 <= heads * (2 * n + 7) and n > 1 << 18
    for m, want in ((n, WS), (n + 1, UNS)):
        assert _attend(T=1, Tk=128 * m, Hq=heads, Hkv=heads, cu_k=True, max_k=128 * m) == want


def test_scales_that_overflow():
    """scale * log2(e) has to be finite: 3.4028e38 / 1.4427 = 2.3587e38."""
    nat = _lib()
    for scale, want in ((2.3586e38, nat.NVR_ERR_WORKSPACE), (-2.3586e38, nat.NVR_ERR_WORKSPACE), (2.3588e38, nat.NVR_ERR_INVALID_ARG),
                        (-3.4e38, nat.NVR_ERR_INVALID_ARG), (1e-45, nat.NVR_ERR_WORKSPACE), (0.0, nat.NVR_ERR_WORKSPACE)):
        assert _attend(scale=scale) == want, scale


def test_rotations_over_other_inputs():
    """A result over its own input has that one's type and stride; over the other side's, or the other result, it may not be."""
    nat = _lib()
    at = [ctypes.c_void_p(0x10000 * i) for i in (1, 2, 3, 4)]

    def call(**kw):
        a = dict(q=at[0], qs=1024, k=at[1], ks=256, dt=nat.NVR_BF16, T=4, Hq=8, Hkv=2, D=128, pos=None, step=0, n_axes=0,
                 axes=None, cos=None, sin=None, n_pos=0, rot=0, inter=0, qw=None, kw=None, eps=1e-6, qo=at[2], qos=1024,
                 ko=at[3], kos=256, out_dt=nat.NVR_BF16)
        a.update(kw)
        return nat.lib().prompt_rope(*a.values(), None)

    f32 = dict(dt=nat.NVR_F32, out_dt=nat.NVR_BF16)
    for bad in (dict(qo=at[0], qos=1280), dict(ko=at[1], kos=512), dict(qo=at[0], **f32), dict(ko=at[1], T=1, **f32), dict(qo=at[1]),
                dict(ko=at[0]), dict(ko=at[2]), dict(Hkv=0, k=None, ko=None, qo=at[0], qos=1280)):
        assert call(**bad) == nat.NVR_ERR_INVALID_ARG, bad
