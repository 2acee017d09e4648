"""GPU parity of the 4-bit key/value cache (attn_kv4_append, attn_kv4_read,
attn_decode_kv4, attn_key_weights, attn_kv4_evict) against the fp64 oracle.

Codes, scales, moved rows, kept slots and positions are compared bit for bit.
Tolerances of the computed values, from the arithmetic:

* scores are fp32 sums of d exact products: |dx| <= ex = (d + 16) 2^-23 max_j
  sum_c |q_c k_c| scale (d roundings of partial sums, the scale factors and
  the base-2 constants), so a probability is off by a factor within ep = 2 ex +
  2^-18 (both numerator and denominator, the 2-ulp exponential, and sums of at
  most 2^5 serial steps per power of 2^-23);
* o: the kernel rounds p * (scale of v) once (to no less than bf16's 2^-8) and its
  result to bf16 (2^-8).  The codes enter the product as c + 8 and -8 comes off 16
  slots at a time: two matrix instructions, each a sum of 17 addends (16 products
  and the accumulator) aligned to the largest and cut at 2^-24 of it, products up
  to 15 p s (s: the scale).  What that adds is measured by the grid, not by the
  value: 2 * 17 * 15 * 2^-24 < 2^-15 of p s, summed over the slots (a slot with
  nearly all the probability and code 0 leaves 2^-15 s where another's tiny
  share is the result).  So |do| <= (2^-8 + ep) sum_j p |v| + 2^-15 sum_j p s + 2^-8 |o|;
* lse: |dl| <= ep + 2^-22 |lse|;
* weights, per slot: <= w (ep + 2^-20) (sums of up to 16 heads in fp32; a prompt's
  weights are sums of positive terms over its queries, each partial sum of n terms
  off by at most n 2^-24 of itself, n <= the query tile's 128 columns per head and
  tile, joined tile by tile: n 2^-24 with n the number of queries bounds it).
"""
import numpy as np
import pytest
import torch

from oracle import attention as A
from oracle import kv4 as O
from tests._guard import Guarded

pytestmark = pytest.mark.gpu


def bits(t):
    """A bf16 tensor's bit patterns on the host."""
    return t.detach().view(torch.int16).cpu().numpy()


def to_bf16(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(torch.bfloat16)


def same_values(a, b):
    """Equal, NaN where NaN."""
    a, b = a.float().cpu().numpy(), np.asarray(b, dtype=np.float32)
    return np.array_equal(a, b, equal_nan=True)


def make_cache(B, Hkv, cap, d, seed, gain=0.5):
    """Random packed rows (host arrays and device tensors) whose scales vary by channel group."""
    g = torch.Generator().manual_seed(seed)
    out = {}
    for n, gn in (("k", gain), ("v", 0.0)):
        x = torch.randn(B, Hkv, cap, d, generator=g) * torch.exp(gn * torch.randn(1, Hkv, 1, d, generator=g))
        c, s = O.quantize(x.bfloat16())
        out[n + "c"], out[n + "s"] = O.pack(c), s
    dev = {n: (torch.from_numpy(v) if v.dtype == np.uint8 else to_bf16(v)).cuda() for n, v in out.items()}
    return out, dev


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ append, read
@pytest.mark.parametrize("B,Hkv,n,cap,d,starts,counts", [
    (1, 1, 1, 16, 64, [0], None), (3, 2, 37, 64, 128, [0, 5, 27], None), (2, 3, 130, 160, 64, [30, 0], [130, 7]),
    (4, 1, 5, 32, 128, [0, 31, 29, 32], [5, 5, 0, 5]),          # rows past the capacity are dropped
    (2, 2, 3, 16, 64, [-2, 2 ** 31 - 1], None), (2, 1, 4, 16, 128, [0, 4], [-3, 9]),
])
def test_append(cuda_lib, B, Hkv, n, cap, d, starts, counts):
    ta = cuda_lib
    g = torch.Generator().manual_seed(n)
    k, v = (torch.randn(B, Hkv, n, d, generator=g).mul(2).bfloat16() for _ in range(2))
    bufs = [Guarded((B, Hkv, cap, d // 2), torch.uint8), Guarded((B, Hkv, cap, d // 32), torch.bfloat16),
            Guarded((B, Hkv, cap, d // 2), torch.uint8), Guarded((B, Hkv, cap, d // 32), torch.bfloat16),
            Guarded((B, Hkv, cap), torch.float32), Guarded((B, Hkv, cap), torch.int32)]
    kc, ks, vc, vs, w, pos = (b.t for b in bufs)
    before = [x.clone() for x in (kc, vc, ks.view(torch.int16), vs.view(torch.int16), w.view(torch.int32), pos)]
    nxt = [100 * (b + 1) for b in range(B)]
    ta.attn_kv4_append(k.cuda(), v.cuda(), kc, ks, vc, vs, ints(starts), None if counts is None else ints(counts), w,
                       pos, ints(nxt))
    torch.cuda.synchronize()
    for x in bufs:
        x.check("append")
    want = [x.cpu().numpy().copy() for x in before]
    qk, qv = O.quantize(k), O.quantize(v)
    for b in range(B):
        for i in range(n if counts is None else max(0, min(n, counts[b]))):
            at = starts[b] + i
            if 0 <= at < cap:
                want[0][b, :, at], want[1][b, :, at] = O.pack(qk[0])[b, :, i], O.pack(qv[0])[b, :, i]
                want[2][b, :, at], want[3][b, :, at] = bits(to_bf16(qk[1]))[b, :, i], bits(to_bf16(qv[1]))[b, :, i]
                want[4][b, :, at], want[5][b, :, at] = 0, nxt[b] + i
    got = (kc, vc, ks.view(torch.int16), vs.view(torch.int16), w.view(torch.int32), pos)
    for name, a, e in zip(("kc", "vc", "ks", "vs", "weights", "positions"), got, want):
        assert np.array_equal(a.cpu().numpy(), e), name


@pytest.mark.parametrize("d", [64, 128])
def test_append_rounding(cuda_lib, d):
    """Every significand against scales of several significands (exact ties among them),
    over the whole exponent range, subnormals, zeros, infinities and NaN."""
    ta = cuda_lib
    rows = []
    m = np.arange(128, 256, dtype=np.float64)
    for top in (128, 129, 131, 147, 189, 224, 255):
        for e in (0, -120, 100, -130):
            for k in range(0, 128, 31):
                for f in (-5, -3, -2, -1, 0):
                    row = np.zeros(32)
                    row[:31] = (m[k:k + 31] if k + 31 <= 128 else np.resize(m[k:], 31)) * 2.0 ** f
                    row = np.where(row > top, row / 2, row) * np.where(np.arange(32) % 2, 1, -1)
                    row[31] = top
                    rows.append(row * 2.0 ** e)
    rows += [np.zeros(32), np.full(32, 2.0 ** -133), np.full(32, 2.0 ** -128), np.arange(32) * 2.0 ** -133]
    special = np.zeros((3, 32))
    special[0, 7], special[1, 0], special[2, 31] = np.inf, -np.inf, np.nan
    special[:, 1] = 3
    rows = np.concatenate([np.stack(rows), special])
    per = d // 32
    rows = np.concatenate([rows, np.zeros((-len(rows) % per, 32))]).reshape(-1, d)
    x = torch.from_numpy(rows).to(torch.bfloat16)[None, None]
    n = x.shape[2]
    c = ta.KV4Cache(1, 1, n, d)
    c.append(x.cuda(), x.cuda())
    codes, scales = O.quantize(x)
    assert np.array_equal(c.kc[:, :, :n].cpu().numpy(), O.pack(codes)) and torch.equal(c.kc, c.vc)
    assert same_values(c.ks[:, :, :n], scales) and same_values(c.vs[:, :, :n], scales)
    k, v = c.read(n)
    val = codes * np.repeat(scales, 32, axis=-1)
    assert same_values(k, O.bf16_round(val.astype(np.float32))) and torch.equal(k.view(torch.int16), v.view(torch.int16))


@pytest.mark.parametrize("d", [64, 128])
def test_read_outside(cuda_lib, d):
    ta = cuda_lib
    host, dev = make_cache(2, 3, 48, d, 5)
    out = Guarded((2, 3, 21, d), torch.bfloat16)
    ta.attn_kv4_read(dev["kc"], dev["ks"], out.t, ints([40, -3]))
    torch.cuda.synchronize()
    out.check("read")
    val = O.values(host["kc"], host["ks"])
    want = np.zeros((2, 3, 21, d))
    want[0, :, :8], want[1, :, 3:] = val[0, :, 40:], val[1, :, :18]
    assert same_values(out.t, O.bf16_round(want.astype(np.float32)))


# ------------------------------------------------------------------ decode
def run_decode(ta, q, dev, lens, scale, splits, weights=None):
    B, Hq, _, d = q.shape
    Hkv, cap = dev["kc"].shape[1:3]
    splits = splits or ta.attn_decode_kv4_splits(B, Hq, Hkv, cap, d)
    ws = Guarded(None, torch.uint8, nbytes=ta.attn_decode_kv4_workspace_bytes(B, Hq, Hkv, cap, d, splits, weights is not None))
    o, lse = Guarded((B, Hq, 1, d), torch.bfloat16), Guarded((B, Hq, 1), torch.float32)
    w = None
    if weights is not None:
        w = Guarded(tuple(weights.shape), torch.float32)
        w.t.copy_(weights)
    ta.attn_decode_kv4(q, dev["kc"], dev["ks"], dev["vc"], dev["vs"], o.t, lse.t, lens, scale, splits, ws.t,
                       None if w is None else w.t)
    assert ta.attn_check_status() == 0
    for b in (ws, o, lse) + (() if w is None else (w,)):
        b.check("decode_kv4")
    return o.t, lse.t, None if w is None else w.t


def check_decode(got, ref, d, what, w0=None):
    o, lse, w = (None if t is None else t.double().cpu().numpy() for t in got)
    ro, rl, rw, pv, ps, sm = ref
    ep = 2 * (d + 16) * 2.0 ** -23 * sm + 2.0 ** -18
    err = np.abs(o - ro) - ((2.0 ** -8 + ep[..., None]) * pv + 2.0 ** -15 * ps + 2.0 ** -8 * np.abs(ro))
    assert (err <= 1e-30).all(), f"{what}: o off by {err.max():.3e} beyond its bound"
    empty = np.isneginf(rl)
    assert np.isneginf(lse[empty]).all(), what
    dl = np.abs(lse[~empty] - rl[~empty]) - (ep[~empty] + 2.0 ** -22 * np.abs(rl[~empty]))
    assert (dl <= 0).all(), f"{what}: lse off by {dl.max():.3e} beyond its bound"
    if w is not None:
        w0 = w0.double().cpu().numpy()
        dw = np.abs(w - (w0 + rw)) - (rw * (ep.max() + 2.0 ** -20) + 2.0 ** -23 * np.abs(w0 + rw))
        assert (dw <= 0).all(), f"{what}: weights off by {dw.max():.3e} beyond their bound"


# lengths 0, 1, tile edges, the capacity and beyond it (clamped); groups of 1 to 16
# heads; more splits than slots
@pytest.mark.parametrize("B,Hq,Hkv,cap,d,lens,splits", [
    (1, 1, 1, 16, 64, [1], 0), (1, 1, 1, 16, 128, [16], 1), (4, 4, 4, 48, 128, [0, 1, 17, 48], 3),
    (5, 8, 2, 144, 64, [15, 16, 33, 64, 129], 2), (3, 6, 2, 272, 128, [31, 32, 257], 1),
    (2, 10, 2, 528, 128, [513, 96], 4), (2, 7, 1, 320, 64, [320, 65], 0), (1, 16, 1, 1008, 128, [1000], 5),
    (1, 24, 2, 400, 64, [399], 1), (2, 12, 4, 16, 128, [400, -5], 2), (1, 32, 2, 640, 128, [611], 16),
    (1, 8, 8, 2048, 128, [2048], 7), (2, 3, 1, 4112, 64, [4097, 2000], 0), (1, 8, 1, 20000, 128, [19999], 0),
])
@pytest.mark.parametrize("track", [False, True])
def test_decode(cuda_lib, B, Hq, Hkv, cap, d, lens, splits, track):
    host, dev = make_cache(B, Hkv, cap, d, 11 + Hq)
    g = torch.Generator().manual_seed(cap)
    q = torch.randn(B, Hq, 1, d, generator=g).mul(1.5).bfloat16()
    # slots behind the live ones hold what must not be read: NaN scales, any codes
    for b, n in enumerate(lens):
        n = min(max(n, 0), cap)
        for s in ("ks", "vs"):
            dev[s][b, :, n:] = float("nan")
        for s in ("kc", "vc"):
            dev[s][b, :, n:] = 0x88
    w0 = torch.rand(B, Hkv, cap, generator=g).cuda() if track else None
    got = run_decode(cuda_lib, q.cuda(), dev, ints(lens), d ** -0.5, splits, w0)
    ref = O.decode(q, host["kc"], host["ks"], host["vc"], host["vs"], lens, d ** -0.5)
    check_decode(got, ref, d, f"decode {Hq}/{Hkv} {lens}", w0)
    if track:  # behind the live slots: left as they were
        for b, n in enumerate(lens):
            n = min(max(n, 0), cap)
            assert torch.equal(got[2][b, :, n:], w0[b, :, n:])


@pytest.mark.parametrize("d", [64, 128])
def test_decode_rising_and_peaked_scores(cuda_lib, d):
    """The running maximum moves at every tile, and one slot takes nearly all the mass."""
    host, dev = make_cache(1, 1, 1024, d, 3, gain=0.0)
    k = torch.zeros(1, 1, 1024, d)
    k[..., :] = torch.linspace(-6, 6, 1024)[None, None, :, None]
    c, s = O.quantize(k.bfloat16())
    host["kc"], host["ks"] = O.pack(c), s
    dev["kc"], dev["ks"] = torch.from_numpy(host["kc"]).cuda(), to_bf16(s).cuda()
    q = torch.ones(1, 4, 1, d).mul(torch.tensor([3.0, -3.0, 0.05, 40.0])[None, :, None, None]).bfloat16()
    w0 = torch.zeros(1, 1, 1024, device="cuda")
    for splits in (1, 5):
        got = run_decode(cuda_lib, q.cuda(), dev, ints([1024]), d ** -0.5, splits, w0)
        check_decode(got, O.decode(q, host["kc"], host["ks"], host["vc"], host["vs"], [1024], d ** -0.5), d, "rising", w0)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("mag", [2.0 ** -100, 2.0 ** -40, 2.0 ** 40, 2.0 ** 100])
def test_decode_scales_of_any_size(cuda_lib, d, mag):
    """Values far from 1 (queries scaled the other way keep the scores ordinary)."""
    host, dev = make_cache(1, 2, 96, d, 9)
    for n in ("ks", "vs"):
        host[n] = host[n] * np.float32(mag)
        dev[n] = to_bf16(host[n]).cuda()
    q = torch.randn(1, 8, 1, d, generator=torch.Generator().manual_seed(1)).bfloat16() * (1 / mag)
    got = run_decode(cuda_lib, q.cuda(), dev, ints([93]), d ** -0.5, 2)
    ref = O.decode(q, host["kc"], host["ks"], host["vc"], host["vs"], [93], d ** -0.5)
    check_decode(got, ref, d, f"mag {mag}")


# 8 partials a row and fewer, up to 64, more: each merged in its own way; 20 heads to a
# cache head are weighed in three turns, the last of four
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv,cap,lens,splits", [
    (40, 2, 1104, [1101, 0, 64], 8), (40, 2, 1104, [1, 1090, 700], 9), (8, 2, 4112, [4100, 0, 2077], 63),
    (20, 1, 4400, [4399, 1500, 3], 64), (6, 1, 9008, [9001, 5, 0], 140),
])
def test_decode_merges(cuda_lib, Hq, Hkv, cap, lens, splits, d):
    B = len(lens)
    host, dev = make_cache(B, Hkv, cap, d, 31 + splits)
    g = torch.Generator().manual_seed(splits)
    q = torch.randn(B, Hq, 1, d, generator=g).bfloat16()
    w0 = torch.rand(B, Hkv, cap, generator=g).cuda()
    got = run_decode(cuda_lib, q.cuda(), dev, ints(lens), d ** -0.5, splits, w0)
    check_decode(got, O.decode(q, host["kc"], host["ks"], host["vc"], host["vs"], lens, d ** -0.5), d, f"merge {splits}", w0)


def test_decode_many_sequences(cuda_lib):
    """More sequences than a warp has lanes, most of them empty or tiny, one long."""
    B, Hq, Hkv, cap, d = 77, 4, 2, 1008, 64
    lens = [(7 * b) % 5 if b % 3 else 0 for b in range(B)]
    lens[40], lens[76] = 1003, 65
    host, dev = make_cache(B, Hkv, cap, d, 17)
    q = torch.randn(B, Hq, 1, d, generator=torch.Generator().manual_seed(6)).bfloat16()
    for splits in (1, 0, 1024):
        w0 = torch.rand(B, Hkv, cap).cuda()
        got = run_decode(cuda_lib, q.cuda(), dev, ints(lens), 0.2, splits, w0)
        check_decode(got, O.decode(q, host["kc"], host["ks"], host["vc"], host["vs"], lens, 0.2), d, f"many {splits}", w0)


def test_offsets_beyond_32_bits(cuda_lib):
    """The last cache head of a cache of more than 2^32 bytes of codes: append, read, decode."""
    ta = cuda_lib
    B, Hkv, cap, d = 1, 36, 1 << 21, 128                      # 4.8 GB of codes each for K and V
    c = ta.KV4Cache(B, Hkv, cap, d, track=False)
    assert c.kc.numel() > 2 ** 32
    g = torch.Generator().manual_seed(12)
    k, v = (torch.randn(B, Hkv, 70, d, generator=g).bfloat16() for _ in range(2))
    c.append(k.cuda(), v.cuda())
    h = [0, Hkv - 1]
    (kc, ks), (vc, vs) = O.quantize(k[:, h]), O.quantize(v[:, h])
    assert np.array_equal(c.kc[:, h, :70].cpu().numpy(), O.pack(kc)) and np.array_equal(c.vc[:, h, :70].cpu().numpy(), O.pack(vc))
    kr, _ = c.read(70)
    assert same_values(kr[:, h], O.bf16_round((kc * np.repeat(ks, 32, axis=-1)).astype(np.float32)))
    q = torch.randn(B, 2 * Hkv, 1, d, generator=g).bfloat16()
    o, lse = ta.decode_kv4(q.cuda(), c, 0.1)
    assert ta.attn_check_status() == 0
    sel = [0, 1, 2 * Hkv - 2, 2 * Hkv - 1]
    ref = O.decode(q[:, sel], O.pack(kc), ks, O.pack(vc), vs, [70], 0.1)
    check_decode((o[:, sel], lse[:, sel], None), ref, d, "far offsets")


def test_decode_nan_row_poisons_its_heads_only(cuda_lib):
    host, dev = make_cache(2, 2, 64, 128, 21)
    for n in ("ks", "vs"):
        _, dev2 = make_cache(2, 2, 64, 128, 21)
        dev2[n][1, 0, 5, 2] = float("nan")
        q = torch.randn(2, 8, 1, 128, generator=torch.Generator().manual_seed(2)).bfloat16()
        o, lse, w = run_decode(cuda_lib, q.cuda(), dev2, ints([64, 40]), 0.1, 1, torch.zeros(2, 2, 64, device="cuda"))
        assert torch.isnan(o[1, :4]).any(dim=-1).all()
        o[1, :4], lse[1, :4], w[1, 0] = 0, 0, 0
        assert not torch.isnan(o).any() and not torch.isnan(lse).any() and not torch.isnan(w).any()


def test_decode_is_deterministic_and_stream_safe(cuda_lib):
    """Same bits on every call, on a side stream, and in a captured graph replayed on
    changed inputs."""
    ta = cuda_lib
    host, dev = make_cache(3, 2, 1024, 128, 4)
    q = torch.randn(3, 8, 1, 128, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    lens = ints([1024, 700, 3])
    first = run_decode(ta, q, dev, lens, 0.1, 0, torch.zeros(3, 2, 1024, device="cuda"))
    again = run_decode(ta, q, dev, lens, 0.1, 0, torch.zeros(3, 2, 1024, device="cuda"))
    assert all(torch.equal(a, b) for a, b in zip(first, again))
    S = ta.attn_decode_kv4_splits(3, 8, 2, 1024, 128)
    ws = torch.empty(ta.attn_decode_kv4_workspace_bytes(3, 8, 2, 1024, 128, S, True), dtype=torch.uint8, device="cuda")
    o, lse, w = torch.empty_like(first[0]), torch.empty_like(first[1]), torch.zeros(3, 2, 1024, device="cuda")
    qq = torch.zeros_like(q)

    def call():
        ta.attn_decode_kv4(qq, dev["kc"], dev["ks"], dev["vc"], dev["vs"], o, lse, lens, 0.1, S, ws, w)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    qq.copy_(q)
    w.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o, first[0]) and torch.equal(lse, first[1]) and torch.equal(w, first[2])


# ------------------------------------------------------------------ key weights
def weigh(ta, q, k, lse, causal, scale, stride=None, seqlens=None, accumulate=None):
    B, Hq, Nq, d = q.shape
    Hkv, Nkv = k.shape[1:3]
    stride = stride or Nkv
    w = Guarded((B, Hkv, stride), torch.float32)
    if accumulate is not None:
        w.t.copy_(accumulate)
    ws = Guarded(None, torch.uint8, nbytes=max(16, ta.attn_key_weights_workspace_bytes(B, Hq, Hkv, Nq, Nkv, d)))
    ta.attn_key_weights(q, k, lse, w.t, causal, scale, ws.t, seqlens, accumulate is not None)
    assert ta.attn_check_status() == 0
    w.check("key_weights")
    ws.check("key_weights workspace")
    return w.t


def check_weights(w, ref, sm, d, Nq, what):
    w = w.double().cpu().numpy()
    tol = ref * (2 * (d + 16) * 2.0 ** -23 * sm + 2.0 ** -18 + Nq * 2.0 ** -24) + 1e-35
    err = np.abs(w - ref) - tol
    assert (err <= 0).all(), f"{what}: off by {err.max():.3e} beyond the bound"


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("B,Hq,Hkv,Nq,Nkv,d", [
    (1, 1, 1, 1, 1, 64), (1, 2, 1, 1, 130, 128), (2, 4, 2, 128, 128, 128), (1, 6, 2, 129, 257, 64),
    (1, 3, 3, 300, 300, 128), (2, 8, 1, 17, 700, 64), (1, 5, 1, 640, 640, 128), (1, 2, 2, 200, 90, 64),
    (3, 4, 4, 33, 1000, 128), (1, 1, 1, 1500, 1500, 64), (1, 4, 2, 127, 129, 128),
])
def test_key_weights(cuda_lib, B, Hq, Hkv, Nq, Nkv, d, causal):
    g = torch.Generator().manual_seed(Nq + Nkv)
    q = torch.randn(B, Hq, Nq, d, generator=g).mul(1.5).bfloat16()
    k = torch.randn(B, Hkv, Nkv, d, generator=g).bfloat16()
    _, lse = A.attention_gqa(q, k, k, causal, d ** -0.5)
    lse = torch.from_numpy(lse).float()
    w = weigh(cuda_lib, q.cuda(), k.cuda(), lse.cuda(), causal, d ** -0.5)
    ref, sm = O.key_weights(q, k, lse, causal, d ** -0.5)
    check_weights(w, ref, sm, d, Nq, f"key weights {Nq}x{Nkv}")
    rows = min(Nq, Nkv) if causal else Nq       # every row that sees a key hands out one
    assert abs(float(w.double().sum()) - B * Hq * rows) < 1e-4 * B * Hq * rows


def test_key_weights_padded_strided_accumulated(cuda_lib):
    """A padded batch whose padding holds NaN, into the rows of a larger cache, adding."""
    g = torch.Generator().manual_seed(8)
    B, Hq, Hkv, N, d, cap = 4, 6, 2, 270, 128, 304
    lens = [270, 1, 0, 131]
    q, k = torch.randn(B, Hq, N, d, generator=g).bfloat16(), torch.randn(B, Hkv, N, d, generator=g).bfloat16()
    _, lse = A.attention_gqa(q, k, k, True, 0.1)
    lse = torch.from_numpy(lse).float()
    ref, sm = O.key_weights(q, k, lse, True, 0.1, lens)
    for b, n in enumerate(lens):
        q[b, :, n:], k[b, :, n:], lse[b, :, n:] = float("nan"), float("nan"), float("nan")
    w = weigh(cuda_lib, q.cuda(), k.cuda(), lse.cuda(), True, 0.1, seqlens=ints(lens))
    check_weights(w, ref, sm, d, N, "padded")
    assert all(not w[b, :, n:].any() for b, n in enumerate(lens))
    w0 = torch.rand(B, Hkv, cap, generator=g).cuda()
    w2 = weigh(cuda_lib, q.cuda(), k.cuda(), lse.cuda(), True, 0.1, stride=cap, seqlens=ints(lens), accumulate=w0)
    assert torch.equal(w2[..., N:], w0[..., N:])
    assert torch.equal(w2[..., :N], w0[..., :N] + w)


def test_key_weights_without_queries(cuda_lib):
    k = torch.randn(1, 2, 40, 64).bfloat16().cuda()
    q = torch.empty(1, 4, 0, 64, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(1, 4, 0, device="cuda")
    assert not weigh(cuda_lib, q, k, lse, True, 0.1).any()
    w0 = torch.rand(1, 2, 40, device="cuda")
    assert torch.equal(weigh(cuda_lib, q, k, lse, False, 0.1, accumulate=w0), w0)


def test_key_weights_from_the_forward(cuda_lib):
    """With the library's own lse; each query row hands out a weight of one."""
    ta = cuda_lib
    q = torch.randn(2, 8, 515, 128, generator=torch.Generator().manual_seed(4)).bfloat16().cuda()
    k = torch.randn(2, 2, 515, 128, generator=torch.Generator().manual_seed(5)).bfloat16().cuda()
    _, lse = ta.forward(q, k, k, True)
    w = ta.key_weights(q, k, lse, True)
    assert ta.attn_check_status() == 0
    ref, sm = O.key_weights(q, k, lse, True, 128 ** -0.5)
    check_weights(w, ref, sm, 128, 515, "from the forward")
    assert torch.equal(w, ta.key_weights(q, k, lse, True))


# ------------------------------------------------------------------ eviction
def run_evict(ta, dev, w, pos, lens, nxt, n_keep, n_recent, alias=False):
    B, Hkv, cap = w.shape
    dev = {n: t.clone() for n, t in dev.items()}
    wo, po = (w.clone(), pos.clone()) if alias else (torch.full_like(w, -7), torch.full_like(pos, -7))
    ws = Guarded(None, torch.uint8, nbytes=ta.attn_kv4_evict_workspace_bytes(B, Hkv, cap, n_keep))
    kept = Guarded((B, Hkv, n_keep), torch.int32)
    ta.attn_kv4_evict(dev["kc"], dev["ks"], dev["vc"], dev["vs"], wo if alias else w, po if alias else pos, lens, nxt,
                      wo, po, kept.t, n_recent, ws.t)
    torch.cuda.synchronize()
    ws.check("evict workspace")
    kept.check("evict kept")
    return dev, wo, po, kept.t


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("B,Hkv,cap,d,lens,n_keep,n_recent,kind", [
    (1, 1, 16, 64, [2], 1, 0, "random"), (2, 2, 64, 128, [64, 40], 40, 8, "random"), (3, 1, 48, 64, [0, 1, 48], 5, 5, "random"),
    (1, 3, 2064, 64, [2050], 1024, 100, "random"), (2, 1, 1040, 128, [1025, 1030], 1024, 0, "ties"),
    (1, 2, 3008, 64, [3000], 17, 3, "ties"), (1, 1, 4000, 64, [4000], 3999, 64, "random"),
    (2, 2, 96, 64, [200, -3], 96, 0, "random"), (1, 2, 528, 64, [520], 300, 10, "special"), (1, 1, 160, 128, [150], 30, 30, "special"),
    (1, 1, 40000, 64, [39990], 20000, 500, "random"), (1, 2, 20000, 64, [19999], 9000, 40, "ties"),
    (1, 1, 140000, 64, [139999], 70000, 1000, "random"), (1, 1, 135008, 128, [135001], 100, 7, "ties"),
    (20, 8, 2064, 64, [2060 - b for b in range(20)], 1500, 64, "special"),
])
def test_evict(cuda_lib, B, Hkv, cap, d, lens, n_keep, n_recent, kind, alias):
    g = torch.Generator().manual_seed(cap + n_keep)
    rows = [torch.randint(0, 256, (B, Hkv, cap, d // 2), generator=g, dtype=torch.uint8) for _ in range(2)]
    scales = [torch.randn(B, Hkv, cap, d // 32, generator=g).bfloat16() for _ in range(2)]
    dev = {n: t.cuda() for n, t in zip(("kc", "vc", "ks", "vs"), rows + scales)}
    w = torch.randn(B, Hkv, cap, generator=g).exp()
    if kind == "ties":
        w = torch.randint(0, 3, (B, Hkv, cap), generator=g).float()
    elif kind == "special":
        pool = torch.tensor([0.0, -0.0, 1.0, float("inf"), -float("inf"), float("nan"), 1e-45, -1.0, 3e38])
        w = pool[torch.randint(0, len(pool), (B, Hkv, cap), generator=g)]
    pos = torch.stack([torch.randperm(cap, generator=g) for _ in range(B * Hkv)]).reshape(B, Hkv, cap).int()
    nxt = [cap] * B
    out, wo, po, kept = run_evict(cuda_lib, dev, w.cuda(), pos.cuda(), ints(lens), ints(nxt), n_keep, n_recent, alias)
    want = O.evict(w.numpy(), pos.numpy(), lens, nxt, n_keep, n_recent)
    assert np.array_equal(kept.cpu().numpy(), want)
    src = torch.from_numpy(want)
    live = src >= 0
    j = torch.arange(n_keep).expand_as(src)
    at = torch.where(live, src, j)
    for n, t in dev.items():
        t = t.cpu().view(torch.uint8 if t.dtype == torch.uint8 else torch.int16)
        e = t.clone()
        e[:, :, :n_keep] = t.gather(2, at[..., None].expand(*at.shape, t.shape[-1]))
        assert torch.equal(out[n].cpu().view(t.dtype), e), n
    for got, given in ((wo, w), (po, pos)):
        got, given = got.cpu().view(torch.int32), given.view(torch.int32)
        assert torch.equal(got[..., :n_keep][live], given.gather(2, at)[live])
        if alias:
            assert torch.equal(got[..., n_keep:], given[..., n_keep:])


def test_weights_and_eviction_in_a_graph(cuda_lib):
    """Captured, replayed on other inputs: the same bits as the eager calls."""
    ta = cuda_lib
    g = torch.Generator().manual_seed(2)
    B, Hq, Hkv, N, d, n_keep = 2, 4, 2, 700, 64, 300
    q, k = (torch.randn(B, h, N, d, generator=g).bfloat16().cuda() for h in (Hq, Hkv))
    _, lse = ta.forward(q, k, k, True)
    c = ta.KV4Cache(B, Hkv, N, d)
    c.append(k, k)
    kept = torch.empty(B, Hkv, n_keep, dtype=torch.int32, device="cuda")
    w_out, p_out = torch.zeros_like(c.weights), torch.zeros_like(c.positions)
    ws = torch.empty(ta.attn_kv4_evict_workspace_bytes(B, Hkv, c.capacity, n_keep), dtype=torch.uint8, device="cuda")
    ws2 = torch.empty(max(16, ta.attn_key_weights_workspace_bytes(B, Hq, Hkv, N, N, d)), dtype=torch.uint8, device="cuda")
    qq = torch.zeros_like(q)

    def call():
        ta.attn_key_weights(qq, k, lse, c.weights, True, d ** -0.5, ws2)
        ta.attn_kv4_evict(c.kc, c.ks, c.vc, c.vs, c.weights, c.positions, c.seqlens, c.next_pos, w_out, p_out, kept, 20, ws)
    qq.copy_(q)
    call()
    first = [t.clone() for t in (c.weights, kept, w_out, p_out, c.kc, c.vs)]
    qq.zero_()
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        call()
    qq.copy_(q)
    for t in (w_out, p_out, kept):
        t.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert ta.attn_check_status() == 0
    assert all(torch.equal(a, b) for a, b in zip((c.weights, kept, w_out, p_out, c.kc, c.vs), first))


# ------------------------------------------------------------------ as they are used together
@pytest.mark.parametrize("d,Hq,Hkv", [(128, 8, 2), (64, 6, 3)])
def test_prompt_decode_evict_decode(cuda_lib, d, Hq, Hkv):
    """Prompt into the cache with its keys' weights, decode steps that append and
    accumulate, an eviction, further steps: against the oracle on the same history."""
    ta = cuda_lib
    B, N, steps, n_keep, n_recent = 2, 300, 5, 128, 16
    g = torch.Generator().manual_seed(d)
    rnd = lambda *s: torch.randn(*s, generator=g).bfloat16()  # noqa: E731
    q, k, v = rnd(B, Hq, N, d), rnd(B, Hkv, N, d), rnd(B, Hkv, N, d)
    cache = ta.KV4Cache(B, Hkv, N + steps, d)
    cache.append(k.cuda(), v.cuda())
    o, lse = ta.forward(q.cuda(), k.cuda(), v.cuda(), True)
    ta.key_weights(q.cuda(), k.cuda(), lse, True, out=cache.weights, accumulate=True)
    hk, hv = [k], [v]
    ref_w, _ = O.key_weights(q, k, lse, True, d ** -0.5)

    def step(w_ref, n):
        nk, nv, nq = rnd(B, Hkv, 1, d), rnd(B, Hkv, 1, d), rnd(B, Hq, 1, d)
        cache.append(nk.cuda(), nv.cuda())
        w0 = cache.weights.clone()
        got = ta.decode_kv4(nq.cuda(), cache)
        host = [cache.kc.cpu().numpy(), cache.ks.float().cpu().numpy(), cache.vc.cpu().numpy(), cache.vs.float().cpu().numpy()]
        ref = O.decode(nq, *host, [n + 1] * B, d ** -0.5)
        check_decode((got[0], got[1], cache.weights), ref, d, f"step at {n}", w0)
        return nk, nv

    n = N
    for _ in range(steps):
        nk, nv = step(ref_w, n)
        hk.append(nk), hv.append(nv)
        n += 1
    assert cache.seqlens.tolist() == [n, n] and cache.next_pos.tolist() == [n, n]
    allk, allv = torch.cat(hk, dim=2), torch.cat(hv, dim=2)
    ck, cs = O.quantize(allk)
    assert np.array_equal(cache.kc[:, :, :n].cpu().numpy(), O.pack(ck))
    w_before, kc_before = cache.weights.clone(), cache.kc.clone()
    want = O.evict(w_before.cpu().numpy(), cache.positions.cpu().numpy(), [n, n], [n, n], n_keep, n_recent)
    kept = cache.evict(n_keep, n_recent)
    assert np.array_equal(kept.cpu().numpy(), want) and cache.seqlens.tolist() == [n_keep] * 2
    assert cache.length_bound == n_keep
    assert torch.equal(cache.positions[..., :n_keep].cpu(), torch.from_numpy(want).int())  # slot s held token s
    idx = kept.long()
    assert torch.equal(cache.weights[..., :n_keep], w_before.gather(2, idx))
    assert torch.equal(cache.kc[:, :, :n_keep], kc_before.gather(2, idx[..., None].expand(-1, -1, -1, d // 2)))
    n = n_keep
    for _ in range(3):
        step(None, n)
        n += 1
    assert ta.attn_check_status() == 0
    k2, v2 = cache.read()
    assert k2.shape == (B, Hkv, n, d) and torch.isfinite(k2.float()).all() and torch.isfinite(v2.float()).all()


def test_conveniences_refuse(cuda_lib):
    ta = cuda_lib
    c = ta.KV4Cache(1, 2, 32, 64, track=False)
    q = torch.zeros(1, 4, 1, 64, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ValueError):
        ta.decode_kv4(q, c, track=True)
    with pytest.raises(ValueError):
        ta.decode_kv4(q[..., :32].contiguous(), c)                       # another head dimension
    with pytest.raises(ta.AttnError):
        ta.decode_kv4(q[:, :3].contiguous(), c)                          # 3 heads over 2
    with pytest.raises(ValueError):
        ta.attn_kv4_read(c.kc, c.ks, torch.zeros(1, 2, 4, 64, device="cuda"))   # fp32 out
    with pytest.raises(ValueError):
        ta.key_weights(q, q[:, :2].contiguous(), torch.zeros(1, 4, 1, device="cuda"), accumulate=True)
    with pytest.raises(ValueError):
        c.append(q[:, :2].transpose(2, 3), q[:, :2].transpose(2, 3))     # not contiguous
    o, lse = ta.decode_kv4(q, c)                                         # an empty cache
    assert not o.any() and torch.isneginf(lse).all()
