"""GPU parity of the weights of a prompt's keys where a CTA has several items one after
another, and over padded batches of every form, against the definition in fp64.

The tolerance is tests/test_kv4_gpu.py's: fp32 scores, a 2-ulp exponential, fp32 sums."""
import math

import pytest
import torch

from tests.test_kv4_gpu import check_weights, ints, weigh

pytestmark = pytest.mark.gpu


def reference(q, k, causal, scale, lens):
    """lse [B,Hq,Nq] over the keys that count (-inf where a query sees none or does not
    count), weights [B,Hkv,Nkv] and the largest sum |q k| scale; fp64."""
    q, k = q.double(), k.double()
    B, Hq, Nq, _ = q.shape
    Hkv, Nkv = k.shape[1:3]
    off = Nkv - Nq
    lse, w, sm = torch.full((B, Hq, Nq), -math.inf, dtype=torch.float64), torch.zeros(B, Hkv, Nkv, dtype=torch.float64), 0.0
    for b, n in enumerate(lens):
        rows = min(Nq, max(0, n - off))
        if rows == 0 or n == 0:
            continue
        for h in range(Hq):
            g = h // (Hq // Hkv)
            x = q[b, h, :rows] @ k[b, g, :n].T * scale
            sm = max(sm, float((q[b, h, :rows].abs() @ k[b, g, :n].abs().T).max()) * scale)
            if causal:
                x.masked_fill_(torch.arange(n)[None] > torch.arange(rows)[:, None] + off, -math.inf)
            z = torch.logsumexp(x, dim=-1)
            lse[b, h, :rows] = z
            z = z.float().double()                           # as the kernel gets it
            w[b, g, :n] += torch.exp(x - torch.where(z.isneginf(), 0.0, z)[:, None]).sum(dim=0)
    return lse.float(), w, sm


MANY = [1000 if b in (3, 20, 36) else (37 * b) % 90 if b % 4 else 0 for b in range(40)]


# 324, 324, 512, 512, 1280 and 1184 items for 148 CTAs.  The last two leave an item up to 15
# query tiles (a ring has 12 tiles of d = 64, 6 of d = 128) and most items none
@pytest.mark.parametrize("B,Hq,Hkv,Nq,Nkv,d,causal,lens", [
    (3, 6, 2, 1500, 1500, 64, True, [1500, 0, 1]), (3, 6, 2, 1500, 1500, 128, False, [700, 1500, 129]),
    (4, 8, 8, 32, 4000, 128, True, None), (4, 8, 8, 32, 4000, 64, False, [4000, 3990, 0, 3970]),
    (40, 32, 8, 450, 1000, 64, True, MANY), (37, 32, 8, 450, 1000, 128, False, MANY[:37]),
    # windows over padded batches: sequences that end in the window, before it, and at its edge
    (5, 4, 2, 64, 700, 128, True, [700, 636, 637, 699, 20]), (4, 6, 2, 130, 257, 64, True, [257, 128, 127, 200]),
    (3, 4, 4, 5, 300, 128, False, [298, 300, 296]), (2, 3, 1, 300, 90, 64, True, [90, 17]), (2, 2, 2, 300, 90, 64, False, [90, 17]),
])
def test_key_weights_of_many_items_and_padded_windows(cuda_lib, B, Hq, Hkv, Nq, Nkv, d, causal, lens):
    g = torch.Generator().manual_seed(Nq + Nkv + d)
    q = torch.randn(B, Hq, Nq, d, generator=g).mul_(1.5).bfloat16()
    k = torch.randn(B, Hkv, Nkv, d, generator=g).bfloat16()
    seqlens = [Nkv] * B if lens is None else lens
    lse, ref, sm = reference(q, k, causal, d ** -0.5, seqlens)
    for b, n in enumerate(seqlens):                          # what the padding holds must not matter
        k[b, :, n:] = float("nan")
        rows = min(Nq, max(0, n - (Nkv - Nq)))
        q[b, :, rows:], lse[b, :, rows:] = float("nan"), float("nan")
    w = weigh(cuda_lib, q.cuda(), k.cuda(), lse.cuda(), causal, d ** -0.5, seqlens=None if lens is None else ints(lens))
    check_weights(w, ref.numpy(), sm, d, Nq * (Hq // Hkv), f"key weights {B}x{Nq}x{Nkv}")
    for b, n in enumerate(seqlens):
        assert not w[b, :, n:].any()
        rows = min(Nq, max(0, n - (Nkv - Nq)))
        if causal and Nq > Nkv:                              # the first queries see no key
            rows = n
        assert abs(float(w[b].double().sum()) - Hq * rows * (n > 0)) <= 1e-4 * Hq * max(rows, 1)
