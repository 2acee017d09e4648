"""KV4Cache on the GPU: what it keeps on the host beside the arrays (room, streams,
captured graphs).  Codes, scales, lengths and positions are compared bit for bit."""
import numpy as np
import pytest
import torch

from oracle import kv4 as O
from tests.test_kv4_gpu import bits, check_weights, ints, to_bf16

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


def captured(call):
    """`call` in a graph, captured on a side stream as torch wants it, and not run yet."""
    graph = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.graph(graph, stream=side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    return graph


@pytest.mark.parametrize("ragged", [False, True])
def test_replayed_appends_keep_to_the_room(cuda_lib, ragged):
    """A decode step in a graph: its replays fill the cache, never run over its end, say
    which tokens found no room, and the host never goes by a bound that they outran."""
    ta = cuda_lib
    B, Hkv, Hq, cap, d = 3, 2, 4, 32, 64
    c = ta.KV4Cache(B, Hkv, cap, d)
    k = rows((B, Hkv, 20, d), 1)
    c.append(k.cuda(), k.cuda(), ints([20, 7, 0]))
    k1, v1, q1 = (rows((B, h, 1, d), 2 + h).cuda() for h in (Hkv, Hkv, Hq))
    counts = ints([1, 1, 0]) if ragged else None
    held = {}

    def step():
        c.append(k1, v1, counts)
        held["o"], _ = ta.decode_kv4(q1, c)
    graph = captured(step)
    assert c.seqlens.tolist() == [20, 7, 0]
    by = [1, 1, 0] if ragged else [1, 1, 1]
    for i in range(1, 15):
        graph.replay()
        want = [min(cap, x + i * y) for x, y in zip((20, 7, 0), by)]
        assert c.seqlens.tolist() == want
        assert c.dropped.tolist() == [max(0, 20 + i - cap), 0, 0]
        assert c.next_pos.tolist() == [x + i * y for x, y in zip((20, 7, 0), by)]
    assert torch.isfinite(held["o"][:2].float()).all()
    same_rows(c, 0, 31, k1[0].cpu(), v1[0].cpu())
    same_rows(c, 1, 20, k1[1].cpu(), v1[1].cpu())
    assert c.positions[0, 0].tolist() == list(range(32))
    assert c.read()[0].shape[2] == cap
    before = c.kc.clone()
    with pytest.raises(ValueError, match="no room"):
        c.append(k1, v1, ints([0, 1, 1]))
    c.reset(torch.tensor([True, False, False], device="cuda"))
    assert c.dropped.tolist() == [0, 0, 0]
    c.append(k1, v1, ints([1, 1, 0]))
    assert c.seqlens.tolist() == [1, 22, 14 * by[2]]
    same_rows(c, 0, 0, k1[0].cpu(), v1[0].cpu())
    assert torch.equal(c.kc[0, :, 1:], before[0, :, 1:])
    for _ in range(30):
        graph.replay()
    with pytest.raises(ValueError):                          # by the lengths, whatever the bound says
        c.append(k1, v1, ints([0, 1, 0]))


def test_a_graph_that_shrinks_the_cache(cuda_lib):
    ta = cuda_lib
    B, Hkv, cap, d = 2, 1, 48, 64
    c = ta.KV4Cache(B, Hkv, cap, d)
    k = rows((B, Hkv, 16, d), 5).cuda()
    graph = captured(lambda: c.evict(8, 2))
    assert c.length_bound == 0
    c.append(k, k)
    c.append(k, k)
    c.append(k, k)
    with pytest.raises(ValueError, match="may not fit"):
        c.append(k, k)
    graph.replay()
    assert c.seqlens.tolist() == [8, 8] and c.read()[0].shape[2] == 8
    c.append(k, k)
    assert c.seqlens.tolist() == [24, 24] and c.read()[0].shape[2] == 24

    def no_length():
        with pytest.raises(ValueError, match="n has to be given"):
            c.read()
        return c.read(16)
    captured(no_length)


# ------------------------------------------------------------------ streams
@pytest.mark.parametrize("raw", [False, True])
def test_calls_go_to_the_stream_they_are_given(cuda_lib, raw):
    """Inputs that arrive late on a side stream: a call that went to the current one would
    work on zeros, or on a cache that is not written yet."""
    ta = cuda_lib
    B, Hq, Hkv, N, d, cap, n_keep = 2, 4, 2, 200, 64, 208, 96
    data = [rows((B, h, n, d), 20 + i).cuda() for i, (h, n) in enumerate(((Hq, N), (Hkv, N), (Hkv, N), (Hq, 1), (Hkv, 8)))]
    counts, mask = ints([3, 8]), torch.tensor([True, False], device="cuda")

    def all_calls(c, q, k, v, q1, more, **on):
        c.append(k, v, **on)
        _, lse = ta.forward(q, k, v, True, **on)
        ta.key_weights(q, k, lse, True, out=c.weights, accumulate=True, **on)
        out = [ta.key_weights(q, k, lse, True, **on), *ta.decode_kv4(q1, c, **on), *c.read(N, **on), c.evict(n_keep, 8, **on)]
        c.append(more, more, counts, **on)
        c.reset(mask, **on)
        return [lse, *out, *ta.decode_kv4(q1, c, **on), c.kc, c.vc, c.ks, c.vs, c.weights, c.positions, c.seqlens, c.next_pos]

    want = all_calls(ta.KV4Cache(B, Hkv, cap, d), *data)
    late, cache = [torch.zeros_like(x) for x in data], ta.KV4Cache(B, Hkv, cap, d)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)                       # about 50 ms
        for x, y in zip(late, data):
            x.copy_(y)
    got = all_calls(cache, *late, stream=side.cuda_stream if raw else side)
    torch.cuda.synchronize()
    assert ta.attn_check_status() == 0
    for i, (x, y) in enumerate(zip(got, want)):
        x, y = (t.view(torch.int16) if t.dtype == torch.bfloat16 else t for t in (x, y))
        assert torch.equal(x, y), i


# ------------------------------------------------------------------ the prompt's weights in the cache
@pytest.mark.parametrize("d,Hq,Hkv", [(128, 8, 2), (64, 6, 3)])
def test_a_prompts_weights_carry_on(cuda_lib, d, Hq, Hkv):
    """The cache's weights after the prompt and after further steps, against the definition
    over the same history."""
    ta = cuda_lib
    B, N, steps = 2, 300, 4
    q, k, v = rows((B, Hq, N, d), 41), rows((B, Hkv, N, d), 42), rows((B, Hkv, N, d), 43)
    c = ta.KV4Cache(B, Hkv, N + steps, d)
    c.append(k.cuda(), v.cuda())
    _, lse = ta.forward(q.cuda(), k.cuda(), v.cuda(), True)
    ta.key_weights(q.cuda(), k.cuda(), lse, True, out=c.weights, accumulate=True)
    ref, sm = O.key_weights(q, k, lse, True, d ** -0.5)
    check_weights(c.weights[..., :N], ref, sm, d, N * (Hq // Hkv), "the prompt")
    total = np.zeros((B, Hkv, c.capacity))
    total[..., :N] = ref
    for i in range(steps):
        k1, v1, q1 = rows((B, Hkv, 1, d), 50 + i), rows((B, Hkv, 1, d), 60 + i), rows((B, Hq, 1, d), 70 + i)
        c.append(k1.cuda(), v1.cuda())
        ta.decode_kv4(q1.cuda(), c)
        host = [t.float().cpu().numpy() if t.dtype == torch.bfloat16 else t.cpu().numpy() for t in (c.kc, c.ks, c.vc, c.vs)]
        total += O.decode(q1, *host, [N + i + 1] * B, d ** -0.5)[2]
    got = c.weights.double().cpu().numpy()
    # the prompt's bound, the steps' (a factor within 2^-17 where scores stay below 2^4),
    # and an addition a head and step
    tol = total * (2 * (d + 16) * 2.0 ** -23 * sm + 2.0 ** -17 + (N * (Hq // Hkv) + steps * Hq) * 2.0 ** -24) + 1e-35
    assert (np.abs(got - total) <= tol).all() and not got[..., N + steps:].any()
