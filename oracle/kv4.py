"""The 4-bit key/value cache in numpy: format, decode, key weights, eviction.

Written from the definitions, with no tiling and no tricks:

* a row of d channels is cut into groups of 32; s = bf16(fp32(amax / 7)),
  c = clamp(rne(x / s), -7, 7), value c * s; s = 0 gives c = 0, a group with an
  infinity or a NaN gives s = NaN, c = 0;
* byte u*(d/16) + 2g + h of a row holds channels 32g + 4u + 2h (low nibble) and
  32g + 4u + 2h + 1 (high nibble), two's complement;
* attention, its log-sum-exp and the probabilities summed over the query heads
  of a cache head, in fp64.
"""
from __future__ import annotations

import numpy as np

from .attention import _f64

GROUP = 32


def bf16_round(x):
    """float32 -> the nearest bf16 value (ties to even), as float32; NaN stays NaN."""
    x = np.asarray(x, dtype=np.float32)
    b = x.view(np.uint32).astype(np.uint64)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32).view(np.float32)
    return np.where(np.isnan(x), np.float32(np.nan), r)


def quantize(x):
    """[..., d] -> (codes int8 [..., d], scales float32 [..., d/32], exact bf16 values)."""
    x = _f64(x).astype(np.float32)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    bad = ~np.isfinite(g).all(axis=-1)
    g = np.where(bad[..., None], np.float32(0), g)
    s = bf16_round(np.abs(g).max(axis=-1) / np.float32(7))
    div = np.where(s > 0, s, np.float32(1))[..., None]
    c = np.where(s[..., None] > 0, np.rint(np.clip(g / div, -7, 7)), 0).astype(np.int8)
    return c.reshape(x.shape), np.where(bad, np.float32(np.nan), s)


def byte_of_channel(d):
    """(byte index, nibble 0 or 1) of each channel of a row."""
    ch = np.arange(d)
    return (ch % 32) // 4 * (d // 16) + 2 * (ch // 32) + ch % 4 // 2, ch % 2


def pack(codes):
    codes = np.asarray(codes)
    d = codes.shape[-1]
    out = np.zeros(codes.shape[:-1] + (d // 2,), dtype=np.uint8)
    for ch, (byte, nib) in enumerate(zip(*byte_of_channel(d))):
        out[..., byte] |= ((codes[..., ch].astype(np.int64) & 15) << (4 * nib)).astype(np.uint8)
    return out


def unpack(packed):
    packed = np.asarray(packed)
    byte, nib = byte_of_channel(2 * packed.shape[-1])
    n = (packed[..., byte].astype(np.int64) >> (4 * nib)) & 15
    return np.where(n >= 8, n - 16, n)


def values(packed, scales):
    """fp64 values of packed rows and their scales."""
    return unpack(packed) * np.repeat(_f64(scales), GROUP, axis=-1)


def decode(q, kc, ks, vc, vs, seqlens, scale):
    """o [B,Hq,1,d], lse [B,Hq,1] and the probability mass per slot [B,Hkv,cap], with what
    error bounds are made of: sum_j p |v| and sum_j p s (s: the scale of v's group), both
    [B,Hq,1,d], and max_j sum |q k| scale."""
    q = _f64(q)
    B, Hq, _, d = q.shape
    Hkv, cap = kc.shape[1:3]
    G = Hq // Hkv
    o, lse = np.zeros((B, Hq, 1, d)), np.full((B, Hq, 1), -np.inf)
    w, sm = np.zeros((B, Hkv, cap)), np.zeros((B, Hq, 1))
    pv, ps = np.zeros((B, Hq, 1, d)), np.zeros((B, Hq, 1, d))
    for b in range(B):
        n = min(max(int(seqlens[b]), 0), cap)
        if n == 0:
            continue
        for h in range(Hkv):
            k, v = values(kc[b, h, :n], ks[b, h, :n]), values(vc[b, h, :n], vs[b, h, :n])
            for a in range(h * G, (h + 1) * G):
                x = k @ q[b, a, 0] * scale
                m = x.max()
                e = np.exp(x - m)
                p = e / e.sum()
                o[b, a, 0], lse[b, a, 0] = p @ v, m + np.log(e.sum())
                w[b, h, :n] += p
                pv[b, a, 0] = p @ np.abs(v)
                ps[b, a, 0] = p @ np.repeat(_f64(vs[b, h, :n]), GROUP, axis=-1)
                sm[b, a, 0] = (np.abs(k) @ np.abs(q[b, a, 0])).max() * scale
    return o, lse, w, pv, ps, sm


def key_weights(q, k, lse, causal, scale, seqlens=None):
    """[B,Hkv,Nkv]: column sums of exp(scale q k^T - lse) over the query heads of a
    key/value head; also the largest sum |q k| scale of any pair."""
    q, k, lse = _f64(q), _f64(k), _f64(lse)
    B, Hq, Nq, d = q.shape
    Hkv, Nkv = k.shape[1:3]
    w, sm = np.zeros((B, Hkv, Nkv)), 0.0
    i, j = np.arange(Nq)[:, None] + (Nkv - Nq), np.arange(Nkv)[None, :]
    for b in range(B):
        n = Nkv if seqlens is None else min(max(int(seqlens[b]), 0), Nkv)
        seen = (i < n) & (j < n) & ((j <= i) | (not causal))
        for h in range(Hq):
            g = h // (Hq // Hkv)
            x = np.where(seen, q[b, h] @ k[b, g].T * scale, -np.inf)
            z = np.where(np.isneginf(lse[b, h]), 0.0, lse[b, h])[:, None]
            w[b, g] += np.exp(np.where(seen, x - z, -np.inf)).sum(axis=0)
            sm = max(sm, float((np.abs(q[b, h]) @ np.abs(k[b, g]).T).max(initial=0)) * scale)
    return w, sm


def evict(weights, positions, seqlens, next_pos, n_keep, n_recent):
    """kept [B,Hkv,n_keep]: the old slot of each new slot, -1 where fewer are live."""
    weights, positions = np.asarray(weights), np.asarray(positions)
    B, Hkv, cap = weights.shape
    kept = np.full((B, Hkv, n_keep), -1, dtype=np.int64)
    for b in range(B):
        n = min(max(int(seqlens[b]), 0), cap)
        for h in range(Hkv):
            if n <= n_keep:
                kept[b, h, :n] = np.arange(n)
                continue
            w = [(-np.inf if np.isnan(x) else float(x)) for x in weights[b, h, :n]]
            older = [int(p) < int(next_pos[b]) - n_recent for p in positions[b, h, :n]]
            stay = set(sorted(range(n), key=lambda j: (older[j], -w[j] if older[j] else 0.0, j))[:n_keep])
            movers = iter(j for j in range(n_keep, n) if j in stay)
            kept[b, h] = [j if j in stay else next(movers) for j in range(n_keep)]
    return kept
