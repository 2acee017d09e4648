"""KV4Cache on the GPU: what it keeps on the host beside the arrays (room, streams,
captured graphs).  Codes, scales, lengths and positions are compared bit for bit."""
import numpy as np
import pytest
import torch

from oracle import kv4 as O
from tests.test_kv4_gpu import bits, ints, to_bf16

pytestmark = pytest.mark.gpu


def rows(shape, seed):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16()


def same_rows(cache, b, at, k, v):
    """Slots [at, at + len) of sequence b hold k, v [Hkv, len, d]."""
    n = k.shape[1]
    for x, codes, scales in ((k, cache.kc, cache.ks), (v, cache.vc, cache.vs)):
        c, s = O.quantize(x)
        assert np.array_equal(codes[b, :, at:at + n].cpu().numpy(), O.pack(c))
        assert np.array_equal(bits(scales[b, :, at:at + n]), bits(to_bf16(s)))


def test_room_is_what_the_sequences_leave(cuda_lib):
    """Appends of up to 16 tokens of which each sequence takes some, until one is full;
    then a request ends and its place is used again."""
    B, Hkv, cap, d, n = 3, 2, 64, 64, 16
    c = cuda_lib.KV4Cache(B, Hkv, cap, d)
    lens = [0, 0, 0]
    for i in range(12):                                      # the bound alone would refuse the fifth
        counts = [16 if i % 3 == b else 1 for b in range(B)]
        if max(x + y for x, y in zip(lens, counts)) > cap:
            break
        k, v = rows((B, Hkv, n, d), i), rows((B, Hkv, n, d), 100 + i)
        c.append(k.cuda(), v.cuda(), ints(counts))
        for b in range(B):
            same_rows(c, b, lens[b], k[b, :, :counts[b]], v[b, :, :counts[b]])
            assert c.positions[b, 0, lens[b]:lens[b] + counts[b]].tolist() == list(range(lens[b], lens[b] + counts[b]))
            lens[b] += counts[b]
    assert i > 5 and c.seqlens.tolist() == lens and c.length_bound >= max(lens)
    k = rows((B, Hkv, n, d), 50)
    before = c.kc.clone()
    with pytest.raises(ValueError, match="may not fit"):
        c.append(k.cuda(), k.cuda())
    assert torch.equal(c.kc, before) and c.seqlens.tolist() == lens
    c.reset(torch.tensor([True, False, False], device="cuda"))
    c.append(k.cuda(), k.cuda(), ints([16, 0, 0]))
    same_rows(c, 0, 0, k[0], k[0])
    assert c.seqlens.tolist() == [16] + lens[1:] and c.positions[0, 0, :16].tolist() == list(range(16))
    assert torch.equal(c.kc[1:], before[1:])
    c.reset()
    big = rows((B, Hkv, cap, d), 51)
    c.append(big.cuda(), big.cuda())
    assert c.length_bound == cap and c.seqlens.tolist() == [cap] * B
