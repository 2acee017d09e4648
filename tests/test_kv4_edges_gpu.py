"""GPU parity of the 4-bit cache's decode where values, scales and queries
are of very different sizes, against an fp64 computation of the definition.

Tolerances, from the arithmetic (p: probability, s: scale of v's group, n: slots):

* scores: fp32 sums of d exact products and the factors of scale: off by at most
  ex = (d + 16) 2^-23 max_j sum_c |q_c k_c| scale; a probability by a factor within
  ep = 2 ex + 2^-21 + n 2^-24 (numerator and denominator; two exponentials of 2^-22;
  the sum, at most n / 8 serial additions of 2^-24 each in a lane, and one of a few
  partials);
* o: p s is rounded to fp16 once, 2^-11 (half of its eps).  Below fp16's normal numbers,
  2^-14, it is off by 2^-25 instead or lost whole: with s taken so that the largest scale
  s' is at most 2^15 and at least 2^14, and a sum of p no smaller than 2^-8, that is
  2^(-25 - 14 + 8) s' = 2^-31 s' for slots with p s < 2^(-14 - 14 + 8) s' = 2^-20 s', times a
  code of at most 8: min(8 p s, 2^-28 s') each;
* the offset of the codes: two matrix instructions a step of 16 slots, each a sum of 17
  addends cut at 2^-24 of the largest: 2 * 17 * 15 * 2^-24 < 2^-15 of p s, and 2^-24 of
  what has been summed up so far for 16 addends twice a step: n 2^-23 of sum p |v|;
* the result in bf16: 2^-8 of itself (half of its eps);
* lse: ep + 2^-22 |lse|; weights: w ep + 2^-23 of the sum they join, per head.
"""
import numpy as np
import pytest
import torch

from oracle import kv4 as O
from tests.test_kv4_gpu import ints, make_cache, run_decode, run_evict, to_bf16

pytestmark = pytest.mark.gpu


def reference(q, host, lens, scale):
    """o, lse, w and the two parts of o's bound, fp64, from the definition."""
    q = q.double().numpy()
    B, Hq, _, d = q.shape
    Hkv, cap = host["kc"].shape[1:3]
    G = Hq // Hkv
    o, lse, w = np.zeros((B, Hq, d)), np.full((B, Hq), -np.inf), np.zeros((B, Hkv, cap))
    grid, pv, ex = np.zeros((B, Hq, d)), np.zeros((B, Hq, d)), np.zeros((B, Hq))
    for b, n in enumerate(lens):
        for h in range(Hkv if n else 0):
            k, v = (O.values(host[c][b, h, :n], host[s][b, h, :n]) for c, s in (("kc", "ks"), ("vc", "vs")))
            s = np.repeat(host["vs"][b, h, :n].astype(np.float64), 32, axis=-1)
            top = s.max(axis=0)
            for a in range(h * G, (h + 1) * G):
                x = k @ q[b, a, 0] * scale
                z = x.max() + np.log(np.exp(x - x.max()).sum())
                p = np.exp(x - z)
                o[b, a], lse[b, a] = p @ v, z
                w[b, h, :n] += p
                ps = p[:, None] * s
                pv[b, a] = p @ np.abs(v)
                grid[b, a] = 2.0 ** -15 * ps.sum(axis=0) + np.where(ps < 2.0 ** -20 * top, np.minimum(8 * ps, 2.0 ** -28 * top), 0).sum(axis=0)
                ex[b, a] = (d + 16) * 2.0 ** -23 * (np.abs(k) @ np.abs(q[b, a, 0])).max() * scale
    return o, lse, w, pv, grid, ex


def check(got, ref, lens, what, w0=None):
    o, lse, w = (None if t is None else t.double().cpu().numpy() for t in got)
    ro, rl, rw, pv, grid, ex = ref
    n = np.array(lens, dtype=np.float64)[:, None]
    ep = 2 * ex + 2.0 ** -21 + n * 2.0 ** -24
    tol = (2.0 ** -11 + ep + n * 2.0 ** -23)[..., None] * pv + grid + 2.0 ** -8 * np.abs(ro) + 2.0 ** -133
    for name, err in (("lse", np.abs(lse[..., 0] - rl) - ep - 2.0 ** -22 * np.abs(rl)), ("o", np.abs(o[:, :, 0] - ro) - tol)):
        assert np.isfinite(err).all() and (err <= 0).all(), f"{what}: {name} off by {err.max()} beyond its bound"
    if w is not None:
        w0 = w0.double().cpu().numpy()
        G = ex.shape[1] // w0.shape[1]
        err = np.abs(w - w0 - rw) - (rw * ep.reshape(*w0.shape[:2], G).max(axis=2)[..., None] + G * 2.0 ** -23 * np.abs(w0 + rw))
        assert np.isfinite(err).all() and (err <= 0).all(), f"{what}: weights off by {err.max()} beyond their bound"


def upload(host):
    return {n: (torch.from_numpy(v) if v.dtype == np.uint8 else to_bf16(v)).cuda() for n, v in host.items()}


def case(Hkv, cap, d, seed):
    host, _ = make_cache(1, Hkv, cap, d, seed)
    return {n: v.astype(np.float32) if v.dtype != np.uint8 else v for n, v in host.items()}


def both(ta, q, host, lens, scale, what, splits=(1, 0)):
    dev, ref = upload(host), reference(q, host, lens, scale)
    w0 = torch.zeros(host["kc"].shape[:3], device="cuda")
    for s in splits:
        check(run_decode(ta, q.cuda(), dev, ints(lens), scale, s, w0), ref, lens, f"{what}, {s} splits", w0)


# ------------------------------------------------------------------ values of very different sizes
@pytest.mark.parametrize("Hq,d", [(3, 64), (4, 128), (6, 128), (8, 64)])
def test_zero_values_of_many_slots(cuda_lib, Hq, d):
    """V all zero: the sums of probabilities know nothing of V's size.  20000 slots whose
    scores lie just under 8 (log2 units) above the first tile's."""
    n = 20000
    host = case(1, n, d, 1)
    host["vs"][:], host["ks"][:] = 0, 0
    host["ks"][:, :, 64:] = 1
    k = np.zeros((1, 1, n, d))
    k[..., 64:, 5] = 7
    host["kc"] = O.pack(k.astype(np.int8))
    q = torch.zeros(1, Hq, 1, d)
    q[0, :, 0, 5] = 1.0 - torch.arange(Hq) / 16          # exact in bf16
    both(cuda_lib, q.bfloat16(), host, [n], 7.8 / 7 * np.log(2.0), "zero values")


@pytest.mark.parametrize("Hq,d", [(2, 128), (4, 64), (7, 64), (16, 128)])
@pytest.mark.parametrize("first,then", [(0.0, 2.0 ** 30), (2.0 ** 30, 0.0), (2.0 ** -110, 2.0 ** 60), (2.0 ** 100, 2.0 ** -60)])
@pytest.mark.parametrize("at", [64, 130, 300])
def test_values_grow_or_shrink_along_the_row(cuda_lib, Hq, d, first, then, at):
    """A slot's probability does not depend on what its or another's value is."""
    host = case(1, 400, d, 2)
    host["vs"][:, :, :at] *= np.float32(first)
    host["vs"][:, :, at:] *= np.float32(then)
    q = torch.randn(1, Hq, 1, d, generator=torch.Generator().manual_seed(at)).bfloat16()
    both(cuda_lib, q, host, [391], d ** -0.5, f"values {first} then {then}", splits=(1, 0, 3))


@pytest.mark.parametrize("Hq,d", [(1, 128), (4, 64), (4, 128), (5, 64), (8, 128)])
@pytest.mark.parametrize("spread", [2.0 ** 20, 2.0 ** 45])
def test_groups_of_very_different_size(cuda_lib, Hq, d, spread):
    """A channel group's values keep their accuracy beside much larger ones of another, which
    stand before it in one cache head and behind it in the other."""
    host = case(2, 400, d, 3)
    size = spread ** np.linspace(-1, 1, d // 32)
    host["vs"] *= np.stack([size, size[::-1]])[None, :, None, :].astype(np.float32)
    host["vs"] = O.bf16_round(host["vs"])
    q = torch.randn(1, 2 * Hq, 1, d, generator=torch.Generator().manual_seed(Hq)).bfloat16()
    both(cuda_lib, q, host, [391], d ** -0.5, f"groups {spread} apart", splits=(1, 0, 3))


# ------------------------------------------------------------------ queries and scales of any size
@pytest.mark.parametrize("Hq,d", [(4, 128), (8, 64)])
@pytest.mark.parametrize("q_size,k_size,scale", [
    (112, -112, 0.1), (119, -119, 0.1), (125, -124, 0.1), (-125, 120, 0.1), (-131, 120, 2.0 ** 7),
    (60, 60, 2.0 ** -123), (-60, -60, 2.0 ** 117), (0, 125, 2.0 ** -127), (100, -110, 100.0),
])
def test_queries_and_scale_of_any_size(cuda_lib, Hq, d, q_size, k_size, scale):
    """Powers of two that cancel in the scores: the same accuracy as without them."""
    host = case(1, 96, d, 4)
    host["ks"] = O.bf16_round(np.minimum(host["ks"], 0.5).astype(np.float64) * 2.0 ** k_size)
    q = torch.randn(1, Hq, 1, d, generator=torch.Generator().manual_seed(7)).clamp(-3, 3).double() * 2.0 ** q_size
    both(cuda_lib, q.bfloat16(), host, [93], scale, f"q 2^{q_size}, k 2^{k_size}")


@pytest.mark.parametrize("size", [0.0, 2.0 ** -133])
@pytest.mark.parametrize("scale", [1.0, 2.0 ** -40, 2.0 ** -126])
def test_queries_of_next_to_nothing(cuda_lib, size, scale):
    """Every live slot gets the same probability, dead ones of the tile none."""
    for d, Hq in ((128, 3), (64, 6)):
        host = case(1, 96, d, 5)
        q = torch.full((1, Hq, 1, d), size, dtype=torch.float64).bfloat16()
        both(cuda_lib, q, host, [75], scale, f"q {size}")


# ------------------------------------------------------------------ eviction
def keep_by_rule(weights, positions, n, next_pos, n_keep, n_recent):
    """Which of n slots stay, from the contract: the newest first, then the largest weights,
    a NaN with -infinity, the lower slot among equals."""
    newest = [j for j in range(n) if positions[j] >= next_pos - n_recent]
    rest = [j for j in range(n) if positions[j] < next_pos - n_recent]
    rest.sort(key=lambda j: (np.inf if np.isnan(weights[j]) else -weights[j], j))
    return set((newest + rest)[:n_keep])


def test_newest_slots_stay_before_infinite_weights(cuda_lib):
    """A weight of +infinity pins a slot behind the newest ones, not before them."""
    B, Hkv, cap, d = 2, 3, 2064, 64
    g = torch.Generator().manual_seed(9)
    pool = torch.tensor([float("inf")] * 6 + [1.0, 0.0, -float("inf"), float("nan")])
    w = pool[torch.randint(0, len(pool), (B, Hkv, cap), generator=g)]
    pos = torch.stack([torch.randperm(cap, generator=g) for _ in range(B * Hkv)]).reshape(B, Hkv, cap).int()
    _, dev = make_cache(B, Hkv, cap, d, 6)
    for lens, n_keep, n_recent in (([2060, 3], 2, 1), ([2060, 1500], 40, 40), ([2064, 2001], 700, 64), ([900, 1024], 800, 300)):
        kept = run_evict(cuda_lib, dev, w.cuda(), pos.cuda(), ints(lens), ints([cap] * B), n_keep, n_recent)[3].cpu().numpy()
        assert np.array_equal(kept, O.evict(w.numpy(), pos.numpy(), lens, [cap] * B, n_keep, n_recent))
        for b, n in enumerate(lens):
            for h in range(Hkv):
                want = keep_by_rule(w[b, h].numpy(), pos[b, h].numpy(), n, cap, n_keep, n_recent)
                assert set(kept[b, h].tolist()) - {-1} == want, (b, h, n_keep)


# ------------------------------------------------------------------ key weights
def test_key_weights_without_query_heads(cuda_lib):
    """The empty sum: zero, or what was there before."""
    k = torch.randn(2, 3, 40, 64).bfloat16().cuda()
    q = torch.empty(2, 0, 7, 64, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(2, 0, 7, device="cuda")
    w = torch.rand(2, 3, 48, device="cuda")
    before = w.clone()
    cuda_lib.attn_key_weights(q, k, lse, w, True, 0.1, accumulate=True)
    assert torch.equal(w, before)
    cuda_lib.attn_key_weights(q, k, lse, w, True, 0.1)
    assert not w[..., :40].any() and torch.equal(w[..., 40:], before[..., 40:])


# ------------------------------------------------------------------ the rounding of probabilities
@pytest.mark.parametrize("Hq,d", [(4, 64), (4, 128), (8, 64), (8, 128), (5, 128)])
def test_probabilities_keep_eleven_bits(cuda_lib, Hq, d):
    """Two slots with opposite values and about the same probability: the outputs are small
    beside what they are made of, so that the bound is that of p's own rounding (2^-11, and
    2^-15 of the codes' offset) and not that of the result's.  The same with p rounded to 8
    bits is outside of it."""
    B = 48
    host, _ = make_cache(B, 1, 16, d, 8)
    host = {n: v.astype(np.float32) if v.dtype != np.uint8 else v for n, v in host.items()}
    host["vs"][:, :, 1] = host["vs"][:, :, 0]
    byte = host["vc"][:, :, 0].astype(np.int64)               # 16 - nibble, both: the negative codes
    host["vc"][:, :, 1] = (((16 - (byte & 15)) & 15) | ((16 - (byte >> 4)) & 15) << 4).astype(np.uint8)
    q = torch.randn(B, Hq, 1, d, generator=torch.Generator().manual_seed(d + Hq)).mul(0.5).bfloat16()
    lens = [2] * B
    ref = reference(q, host, lens, 0.02)
    for s in (1, 0):
        check(run_decode(cuda_lib, q.cuda(), upload(host), ints(lens), 0.02, s), ref, lens, "two slots")
    o, _, _, pv, grid, ex = ref                              # the oracle's p in 8 bits: seen?
    far = 0.0
    for b in range(B):
        v = O.values(host["vc"][b, 0, :2], host["vs"][b, 0, :2])
        k = O.values(host["kc"][b, 0, :2], host["ks"][b, 0, :2])
        x = q[b, :, 0].double().numpy() @ k.T * 0.02
        p = np.exp(x - x.max(axis=1, keepdims=True))
        ps = p[:, :, None] * np.repeat(host["vs"][b, 0, :2].astype(np.float64), 32, axis=-1)
        bf = O.bf16_round(ps.astype(np.float32)) / ps * p[:, :, None]
        err = np.abs((bf * v).sum(axis=1) / p.sum(axis=1)[:, None] - o[b])
        tol = (2.0 ** -11 + 2 * ex[b][:, None] + 2.0 ** -20) * pv[b] + grid[b] + 2.0 ** -8 * np.abs(o[b])
        far = max(far, float(np.nan_to_num(err / np.maximum(tol, 1e-30)).max()))
    assert far > 1.0


# ------------------------------------------------------------------ NaN
@pytest.mark.parametrize("Hq,d", [(4, 64), (4, 128), (8, 64), (8, 128)])
def test_a_nan_group_reaches_what_reads_it(cuda_lib, Hq, d):
    """One group of one slot: in V its channels of the head's outputs, in K all that the
    head's queries give; the other cache head, and everything else, as without it."""
    n, slot, g = 150, 77, d // 32 - 1
    host = case(2, 160, d, 9)
    q = torch.randn(1, 2 * Hq, 1, d, generator=torch.Generator().manual_seed(3)).bfloat16()
    w0 = torch.zeros(1, 2, 160, device="cuda")
    for splits in (1, 0):
        want = run_decode(cuda_lib, q.cuda(), upload(host), ints([n]), 0.1, splits, w0)
        for side in ("ks", "vs"):
            bad = {x: y.copy() for x, y in host.items()}
            bad[side][0, 0, slot, g] = np.nan
            o, lse, w = run_decode(cuda_lib, q.cuda(), upload(bad), ints([n]), 0.1, splits, w0)
            first = 0 if side == "ks" else 32 * g
            assert torch.isnan(o[:, :Hq, :, first:]).all()
            assert torch.equal(o[:, :Hq, :, :first], want[0][:, :Hq, :, :first]) and torch.equal(o[:, Hq:], want[0][:, Hq:])
            assert torch.equal(lse[:, Hq:], want[1][:, Hq:]) and torch.equal(w[:, 1], want[2][:, 1])
            if side == "ks":
                assert torch.isnan(lse[:, :Hq]).all() and torch.isnan(w[:, 0, :n]).all() and not w[:, 0, n:].any()
            else:
                assert torch.equal(lse, want[1]) and torch.equal(w, want[2])
