"""The key/value cache oracle pinned on small cases, and the C entry points'
refusals on a machine without a GPU."""

import ctypes
import math

import numpy as np
import pytest

from oracle import kv_cache as K
from test_abi_cpu import _lib


def test_store_and_load_are_inverse_on_every_layout():
    rng = np.random.default_rng(1)
    for D in (64, 128):
        for S in (16, 32, 64, 128):
            H, pages = 2, 3
            cache = rng.integers(0, 256, (pages, H, S * D * 9 // 8)).astype(np.uint8)
            assert K.region_offsets(S, D)[3] == cache.shape[2]
            slots = rng.permutation(pages * S)
            kc, vc = (rng.integers(0, 256, (pages * S, H, D // 2)).astype(np.uint8) for _ in range(2))
            ks, vs = (rng.integers(0, 127, (pages * S, H, D // 16)).astype(np.uint8) for _ in range(2))
            K.store(cache, slots, kc, ks, vc, vs, S)
            k, v = K.load(cache, slots, S, D, [1.0, 0.5], [2.0, 1.0])
            from oracle.gemm import dequantize
            from oracle.quantize import unpack_fp4
            for h, (a, b) in enumerate(((1.0, 2.0), (0.5, 1.0))):
                assert np.array_equal(k[:, h], a * dequantize(unpack_fp4(kc[:, h]), ks[:, h]))
                assert np.array_equal(v[:, h], b * dequantize(unpack_fp4(vc[:, h]), vs[:, h]))


def test_norm_and_rotation_against_their_formulas():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 3, 64)).astype(np.float32)
    w = rng.standard_normal(64).astype(np.float32)
    want = x.astype(np.float64) / np.sqrt((x.astype(np.float64) ** 2).mean(-1, keepdims=True) + 1e-6) * w
    assert np.allclose(K.head_norm(x, w, 1e-6), want, rtol=1e-6)
    ang = rng.uniform(-3, 3, (5, 16))
    c, s = np.cos(ang).astype(np.float32), np.sin(ang).astype(np.float32)
    for inter in (False, True):
        y = K.rotate(x, c, s, inter)
        assert np.array_equal(y[..., 32:], x[..., 32:])
        z = x[..., 0:32:2] + 1j * x[..., 1:32:2] if inter else x[..., :16] + 1j * x[..., 16:32]
        z = z * np.exp(1j * ang)[:, None]
        got = y[..., 0:32:2] + 1j * y[..., 1:32:2] if inter else y[..., :16] + 1j * y[..., 16:32]
        assert np.allclose(got, z, atol=1e-5)


def test_bf16_rounding():
    x = np.array([1.0, 1.00390625, 1.01171875, -3.14159], np.float32)      # ties to even both ways
    b = K.float32_to_bf16_bits(x).astype(np.uint32) << 16
    assert np.array_equal(b.view(np.float32)[:3], np.array([1.0, 1.0, 1.015625], np.float32))


def test_attention_masks():
    rng = np.random.default_rng(3)
    q = rng.standard_normal((4, 2, 8))
    k, v = rng.standard_normal((2, 3, 1, 8))
    out, lse, _, _ = K.attention(q, k, v, 0.5)                 # 4 queries, 3 tokens: the first sees none
    assert np.all(out[0] == 0) and np.all(np.isneginf(lse[0]))
    assert np.allclose(out[1], v[0, 0]) and np.allclose(lse[1], 0.5 * (q[1] @ k[0, 0]))
    out, lse, _, _ = K.attention(q, k, v, 0.5, window=1)       # every query its own token
    assert np.allclose(out[2], v[1, 0]) and np.allclose(out[3], v[2, 0])
    full, _, _, _ = K.attention(q, k, v, 0.5, causal=False)
    p = np.exp(0.5 * q[0] @ k[:, 0].T)
    assert np.allclose(full[0], p @ v[:, 0] / p.sum(-1, keepdims=True))


def test_entry_points_refuse_bad_arguments():
    nat = _lib()
    L = nat.lib()
    fake, odd = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)
    INV, UNS, ALI, WS = (nat.NVR_ERR_INVALID_ARG, nat.NVR_ERR_UNSUPPORTED, nat.NVR_ERR_ALIGNMENT,
                         nat.NVR_ERR_WORKSPACE)
    assert L.nvfp4_kv_page_bytes(64, 128) == 9216 and L.nvfp4_kv_page_bytes(16, 64) == 1152
    assert L.nvfp4_kv_page_bytes(48, 128) == 0 and L.nvfp4_kv_page_bytes(64, 96) == 0

    def append(**kw):
        a = dict(q=fake, qs=1024, k=fake, ks=256, v=fake, vs=256, dt=nat.NVR_BF16, T=4, Hq=8, Hkv=2, D=128,
                 pos=fake, slots=fake, cos=fake, sin=fake, n_pos=100, rot=128, inter=0, qw=None, kw=None, eps=1e-6,
                 kg=fake, vg=fake, cache=fake, n_pages=10, S=64, out=fake)
        a.update(kw)
        return L.nvfp4_kv_append(*a.values(), None)

    for bad in (dict(T=-1), dict(Hkv=0), dict(Hq=-1), dict(dt=7), dict(k=None), dict(v=None), dict(q=None),
                dict(out=None), dict(slots=None), dict(pos=None), dict(cos=None), dict(rot=130), dict(rot=7),
                dict(rot=-2), dict(n_pos=0), dict(kg=None), dict(vg=None), dict(cache=None), dict(n_pages=0),
                dict(ks=255), dict(ks=128), dict(vs=260), dict(qs=1000), dict(eps=-1.0), dict(eps=math.nan)):
        assert append(**bad) == INV, bad
    for bad in (dict(D=96), dict(S=48), dict(n_pages=1 << 26)):
        assert append(**bad) == UNS, bad
    for bad in (dict(q=odd), dict(k=odd), dict(v=odd), dict(cache=odd), dict(out=odd), dict(cos=odd), dict(sin=odd),
                dict(qw=odd), dict(kw=odd), dict(slots=ctypes.c_void_p(0x10002))):
        assert append(**bad) == ALI, bad
    assert append(T=0) == nat.NVR_OK
    assert append(T=0, q=None, k=None, v=None, out=None, slots=None, pos=None) == nat.NVR_OK

    def gather(**kw):
        a = dict(cache=fake, n_pages=10, S=64, Hkv=2, D=128, slots=fake, n=4, kg=fake, vg=fake, k=fake, v=fake,
                 dt=nat.NVR_BF16)
        a.update(kw)
        return L.nvfp4_kv_gather(*a.values(), None)

    for bad in (dict(n=-1), dict(Hkv=0), dict(cache=None), dict(slots=None), dict(k=None), dict(v=None), dict(dt=3),
                dict(n_pages=0), dict(kg=None)):
        assert gather(**bad) == INV, bad
    assert gather(D=32) == UNS and gather(S=8) == UNS
    assert gather(k=odd) == ALI and gather(cache=odd) == ALI
    assert gather(n=0, slots=None, k=None, v=None) == nat.NVR_OK

    need = L.nvfp4_kv_attention_workspace_size(16, 4, 8, 2, 128)
    assert need > 0 and L.nvfp4_kv_attention_workspace_size(16, 4, 7, 2, 128) == 0

    def attend(**kw):
        a = dict(q=fake, qs=1024, T=4, Hq=8, Hkv=2, D=128, cache=fake, n_pages=10, S=64, table=fake, B=4,
                 max_pages=5, lens=fake, cu=None, max_q=1, kg=fake, vg=fake, scale=0.1, causal=1, window=0, out=fake,
                 lse=None, ws=fake, n=need)
        a.update(kw)
        return L.nvfp4_kv_attention(*a.values(), None)

    for bad in (dict(T=-1), dict(Hq=7), dict(Hkv=0), dict(Hq=0), dict(q=None), dict(out=None), dict(cache=None),
                dict(table=None), dict(lens=None), dict(B=0, T=0, max_q=-1), dict(T=5), dict(max_q=2), dict(window=-1),
                dict(window=8, causal=0), dict(scale=math.inf), dict(scale=math.nan), dict(ws=None), dict(qs=1020),
                dict(qs=512), dict(cu=fake, max_q=0), dict(n_pages=0), dict(max_pages=-1), dict(kg=None)):
        assert attend(**bad) == INV, bad
    for bad in (dict(D=96), dict(S=24), dict(max_pages=1 << 26)):
        assert attend(**bad) == UNS, bad
    for bad in (dict(q=odd), dict(cache=odd), dict(out=odd), dict(ws=odd), dict(lse=ctypes.c_void_p(0x10002))):
        assert attend(**bad) == ALI, bad
    assert attend(n=need - 1) == WS
    assert attend(T=0, B=0, q=None, out=None, table=None, lens=None) == nat.NVR_OK


def test_binding_refuses_before_the_library():
    torch = pytest.importorskip("torch")
    import nvfp4_router_gate_gb300 as R
    _lib()
    with pytest.raises(ValueError):
        R.Nvfp4KVCache(4, 2, 96, device="cpu")
    kv = R.Nvfp4KVCache(4, 2, 64, page_size=16, device="cpu")
    assert kv.data.shape == (4, 2, 1152) and kv.k_gsa.shape == (2,)
    with pytest.raises(ValueError):                                  # not on a GPU
        kv.attend(torch.zeros(1, 2, 64, dtype=torch.bfloat16), torch.zeros(1, 1, dtype=torch.int32),
                  torch.zeros(1, dtype=torch.int32))
    with pytest.raises(TypeError):
        kv.attend(torch.zeros(1, 2, 64), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):                                  # more heads than the workspace is for
        kv.attend(torch.zeros(1, 4, 64, dtype=torch.bfloat16), torch.zeros(1, 1, dtype=torch.int32),
                  torch.zeros(1, dtype=torch.int32))


def test_rope_table():
    import nvfp4_router_gate_gb300 as R
    cos, sin = R.rope_table(50, 64, device="cpu")
    i = np.arange(0, 64, 2) / 64
    ang = np.arange(50)[:, None] * 10000.0 ** -i
    assert np.abs(cos.numpy() - np.cos(ang)).max() < 1e-7 and np.abs(sin.numpy() - np.sin(ang)).max() < 1e-7
    c2, _ = R.rope_table(50, 64, factor=4.0, device="cpu")
    assert np.abs(c2.numpy() - np.cos(ang / 4)).max() < 1e-7
    c3, _ = R.rope_table(50, 64, factor=4.0, original=40, device="cpu")
    turns = 40 * 10000.0 ** -i / (2 * math.pi)
    fast, slow = turns >= 32, turns <= 1
    assert slow.any() and np.abs(c3.numpy() - np.cos(ang / 4))[:, slow].max() < 1e-7
    assert not fast.any() or np.abs(c3.numpy() - np.cos(ang))[:, fast].max() < 1e-7
    with pytest.raises(ValueError):
        R.rope_table(4, 7, device="cpu")
