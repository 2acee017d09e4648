"""The 4-bit cache without a GPU: its format pinned by hand-made rows, the eviction
rule by small cases, the argument checks of every entry point, and the
quantiser's divide-free rounding by arithmetic over every pair it can meet."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import kv4 as O

P = ctypes.c_void_p(16 * 1000)  # never dereferenced: validation rejects first


@pytest.fixture(scope="module")
def lib():
    from tiled_attention_24_b200 import build
    build.build()
    from tiled_attention_24_b200 import _binding
    return _binding.load()


# ------------------------------------------------------------------ format
def test_row_of_known_values():
    x = np.zeros((1, 64), dtype=np.float32)
    x[0, :8] = [7, -7, 3.5, 2.5, 0.5, 1.5, -0.5, 1]     # s = 1: ties to even
    x[0, 32:36] = [14, -2, 1, 0]                          # s = 2
    c, s = O.quantize(x)
    assert s.tolist() == [[1.0, 2.0]]
    assert c[0, :8].tolist() == [7, -7, 4, 2, 0, 2, 0, 1] and c[0, 32:36].tolist() == [7, -1, 0, 0]
    p = O.pack(c)
    # piece 0 (4 bytes): channels 0..3 of group 0, then 0..3 of group 1
    assert p[0, :4].tolist() == [0x97, 0x24, 0xF7, 0x00]
    assert p[0, 4:6].tolist() == [0x20, 0x10]
    assert np.array_equal(O.unpack(p), c)


@pytest.mark.parametrize("d", [64, 128])
def test_pack_is_a_permutation_of_nibbles(d):
    byte, nib = O.byte_of_channel(d)
    assert sorted(zip(byte.tolist(), nib.tolist())) == [(b, n) for b in range(d // 2) for n in (0, 1)]
    g = np.random.default_rng(0)
    c = g.integers(-7, 8, size=(5, 3, d))
    assert np.array_equal(O.unpack(O.pack(c)), c)


def test_zero_tiny_and_nonfinite_groups():
    x = np.zeros((4, 32), dtype=np.float32)
    x[1, 3] = 2.0 ** -133                                 # amax / 7 rounds to zero
    x[2, 5], x[2, 6] = np.inf, 1
    x[3, 5] = np.nan
    c, s = O.quantize(x)
    assert s[0, 0] == 0 and s[1, 0] == 0 and np.isnan(s[2, 0]) and np.isnan(s[3, 0])
    assert not c.any()


def test_divide_free_codes_equal_the_divide():
    """rne(x / s) as the kernel takes it, r = rn(1/s), y = x r rounded once to a multiple
    of 2^-11 (fp32 fma with 6144), then to the nearest even whole number: equal to
    rounding the exact quotient for every pair of 8-bit significands and every
    exponent difference that gives a code (fp64 holds x r exactly: 8 + 24 bits)."""
    m = np.arange(128, 256, dtype=np.float64)
    for e in range(-5, 4):
        x, s = (m * 2.0 ** e)[:, None], m[None, :]
        q = x / s
        r = (np.float32(1) / s.astype(np.float32)).astype(np.float64)
        y = np.rint(x * r * 2 ** 11) / 2 ** 11
        near = q <= 7.6
        exact = np.rint((2 * x - 0) / (2 * s))
        # fp64 division is exact enough: ties are exact quotients k + 1/2
        tie = (2 * x) % s == 0
        odd_half = tie & ((2 * x / s) % 2 == 1)
        k = np.floor(q)
        exact = np.where(odd_half, k + (k % 2), np.where(q - k > 0.5, k + 1, k))
        assert np.array_equal(np.rint(y)[near], exact[near]), e


# ------------------------------------------------------------------ eviction rule
def test_evict_rule():
    w = np.array([[[5, 1, 4, 1, 3, 9, 2, 0]]], dtype=np.float32)
    pos = np.arange(8)[None, None]
    k = O.evict(w, pos, [8], [8], 4, 0)
    assert k.tolist() == [[[0, 4, 2, 5]]]                 # 0, 2 stay; 4, 5 fill 1, 3
    k = O.evict(w, pos, [8], [8], 4, 2)                   # 6 and 7 are the newest
    assert k.tolist() == [[[0, 5, 6, 7]]]
    k = O.evict(w, pos, [3], [8], 4, 2)
    assert k.tolist() == [[[0, 1, 2, -1]]]
    same = np.ones((1, 1, 6), dtype=np.float32)
    assert O.evict(same, np.zeros((1, 1, 6), int), [6], [9], 3, 0).tolist() == [[[0, 1, 2]]]
    nan = np.array([[[np.nan, -np.inf, -0.0, 0.0]]], dtype=np.float32)
    assert O.evict(nan, np.zeros((1, 1, 4), int), [4], [9], 3, 0).tolist() == [[[0, 3, 2]]]


def test_oracle_decode_matches_softmax():
    g = torch.Generator().manual_seed(3)
    B, Hq, Hkv, cap, d = 2, 4, 2, 32, 64
    q = torch.randn(B, Hq, 1, d, generator=g).bfloat16()
    kc, ks = O.quantize(torch.randn(B, Hkv, cap, d, generator=g).bfloat16())
    vc, vs = O.quantize(torch.randn(B, Hkv, cap, d, generator=g).bfloat16())
    lens = [32, 9]
    o, lse, w = O.decode(q, O.pack(kc), ks, O.pack(vc), vs, lens, 0.125)[:3]
    for b, n in enumerate(lens):
        k = torch.from_numpy(kc[b, :, :n] * np.repeat(ks[b, :, :n], 32, axis=-1)).double().repeat_interleave(2, dim=0)
        v = torch.from_numpy(vc[b, :, :n] * np.repeat(vs[b, :, :n], 32, axis=-1)).double().repeat_interleave(2, dim=0)
        x = torch.einsum("hd,hnd->hn", q[b, :, 0].double(), k) * 0.125
        p = torch.softmax(x, dim=-1)
        assert np.allclose(o[b, :, 0], torch.einsum("hn,hnd->hd", p, v).numpy(), atol=1e-12)
        assert np.allclose(lse[b, :, 0], torch.logsumexp(x, dim=-1).numpy(), atol=1e-12)
        assert np.allclose(w[b, :, :n], p.reshape(2, 2, n).sum(dim=1).numpy(), atol=1e-12)


# ------------------------------------------------------------------ argument checks
ODD = ctypes.c_void_p(16 * 1000 + 2)


def test_append_and_read_validation(lib):
    def append(**kw):
        a = dict(k=P, v=P, kc=P, ks=P, vc=P, vs=P, starts=P, counts=None, w=None, pos=None, nxt=None, B=1, H=2, n=4,
                 cap=32, d=128)
        a.update(kw)
        return lib.attn_kv4_append(*a.values(), None)
    assert append(d=96) == -2 and append(cap=40) == -1 and append(cap=0) == -1 and append(B=-1) == -1
    assert append(n=-1) == -1 and append(n=0) == 0 and append(B=0) == 0 and append(starts=None) == -1
    assert append(k=None) == -1 and append(vs=None) == -1 and append(pos=P) == -1 and append(k=ODD) == -3
    assert append(w=ctypes.c_void_p(16 * 1000 + 1)) == -3 and append(counts=ODD) == -3
    assert append(B=1 << 16, H=1 << 10, cap=64) == -2

    def read(**kw):
        a = dict(c=P, s=P, o=P, starts=None, B=1, H=2, n=4, cap=32, d=64)
        a.update(kw)
        return lib.attn_kv4_read(*a.values(), None)
    assert read(d=32) == -2 and read(cap=17) == -1 and read(n=-2) == -1 and read(n=0) == 0 and read(o=None) == -1
    assert read(s=ODD) == -3 and read(starts=ODD) == -3


def test_decode_validation(lib):
    size = lib.attn_decode_kv4_workspace_bytes
    assert size(2, 8, 2, 64, 128, 4, 0) >= 2 * 8 * 130 * 4                 # a partial result per head at least
    assert size(2, 8, 2, 6400, 128, 4, 0) >= (2 * 2 * 4) * 4 * 130 * 4    # and per piece, of 4 heads each
    assert size(2, 8, 2, 64, 128, 4, 1) >= size(2, 8, 2, 64, 128, 4, 0) + 2 * 8 * 64 * 4
    assert size(2, 8, 2, 60, 128, 4, 0) == 0 and size(2, 8, 2, 64, 80, 4, 0) == 0 and size(0, 8, 2, 64, 128, 4, 0) == 0
    n = size(2, 8, 2, 64, 128, 4, 1)
    assert 1 <= lib.attn_decode_kv4_splits(1, 8, 2, 1 << 20, 128) <= 1024
    assert 1 <= lib.attn_decode_kv4_splits(64, 32, 8, 16, 64) <= 16 and lib.attn_decode_kv4_splits(512, 32, 8, 16, 64) == 1

    def call(**kw):
        a = dict(q=P, kc=P, ks=P, vc=P, vs=P, o=P, lse=P, w=P, lens=P, B=2, Hq=8, Hkv=2, cap=64, d=128, scale=0.1, S=4,
                 ws=P, nb=n)
        a.update(kw)
        return lib.attn_decode_kv4(*a.values(), None)
    assert call(d=96) == -2 and call(Hkv=3) == -1 and call(Hkv=0) == -1 and call(Hkv=16) == -1 and call(S=0) == -1
    assert call(S=1025) == -1 and call(scale=0.0) == -1 and call(scale=float("inf")) == -1 and call(nb=n - 1) == -1
    assert call(lens=None) == -1 and call(ws=None) == -1 and call(q=ODD) == -3 and call(lens=ODD) == -3
    assert call(B=0) == 0 and call(cap=24) == -1 and call(vc=None) == -1
    assert call(w=ctypes.c_void_p(16 * 1000 + 4)) == -3 and call(o=ctypes.c_void_p(16 * 1000 + 8)) == -3
    assert call(B=1 << 12, Hkv=1 << 10, Hq=1 << 10, cap=1 << 10) == -2          # more than 2^31 slots


def test_key_weights_validation(lib):
    def call(**kw):
        a = dict(q=P, k=P, lse=P, w=P, lens=None, B=1, Hq=4, Hkv=2, Nq=8, Nkv=8, d=128, causal=1, acc=0, scale=0.1, st=8,
                 ws=P, nb=1 << 20)
        a.update(kw)
        return lib.attn_key_weights(*a.values(), None)
    assert call(d=32) == -2 and call(Hkv=3) == -1 and call(Hkv=8) == -1 and call(st=7) == -1 and call(scale=-1.0) == -1
    assert call(Nq=-1) == -1 and call(q=None) == -1 and call(w=None) == -1 and call(k=ODD) == -3 and call(lens=ODD) == -3
    assert call(B=0) == 0 and call(Nkv=0) == 0


def test_evict_validation(lib):
    n = lib.attn_kv4_evict_workspace_bytes(2, 3, 64, 32)
    assert n > 0 and lib.attn_kv4_evict_workspace_bytes(2, 0, 64, 32) == 0

    def call(**kw):
        a = dict(kc=P, ks=P, vc=P, vs=P, w=P, pos=P, lens=P, nxt=P, wo=P, po=P, kept=P, B=2, H=3, cap=64, d=64, keep=32,
                 rec=4, ws=P, nb=n)
        a.update(kw)
        return lib.attn_kv4_evict(*a.values(), None)
    assert call(d=16) == -2 and call(cap=65) == -1 and call(keep=0) == -1 and call(keep=65) == -1 and call(rec=33) == -1
    assert call(rec=-1) == -1 and call(nb=n - 1) == -1 and call(kept=None) == -1 and call(ws=None) == -1
    assert call(w=None) == -1 and call(kc=ODD) == -3 and call(B=0) == 0


def test_binding_refuses_host_tensors():
    import tiled_attention_24_b200 as ta
    x = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        ta.attn_kv4_read(torch.zeros(1, 1, 16, 32, dtype=torch.uint8), torch.zeros(1, 1, 16, 2, dtype=torch.bfloat16), x)


def test_cache_refuses_bad_sizes_and_overflow():
    import tiled_attention_24_b200 as ta
    with pytest.raises(ValueError):
        ta.KV4Cache(1, 1, 16, 96, device="cpu")
    with pytest.raises(ValueError):
        ta.KV4Cache(1, 0, 16, 64, device="cpu")
    c = ta.KV4Cache(2, 1, 17, 64, device="cpu", track=False)
    assert c.capacity == 32 and c.kc.shape == (2, 1, 32, 32) and c.vs.shape == (2, 1, 32, 2)
    big = torch.zeros(2, 1, 33, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="may not fit"):
        c.append(big, big)
    with pytest.raises(ValueError, match="track"):
        c.evict(4)
