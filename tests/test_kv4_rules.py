"""The 4-bit cache's rules without a GPU, beyond tests/test_kv4.py."""
import numpy as np
import pytest
import torch

import tiled_attention_24_b200 as ta
from oracle import kv4 as O


def test_newest_slots_stay_before_infinite_weights():
    inf = np.inf
    w = np.array([[[inf, inf, 0.0]]], dtype=np.float32)
    assert O.evict(w, np.arange(3)[None, None], [3], [3], 2, 1).tolist() == [[[0, 2]]]
    w = np.array([[[inf, -inf, np.nan, inf, 1.0]]], dtype=np.float32)
    pos = np.array([[[4, 3, 0, 1, 2]]])                      # slots 0 and 1 hold the newest tokens
    assert O.evict(w, pos, [5], [5], 2, 2).tolist() == [[[0, 1]]]
    assert O.evict(w, pos, [5], [5], 3, 2).tolist() == [[[0, 1, 3]]]
    # more of them than are kept (a caller's positions): the lower slots
    assert O.evict(w, np.full((1, 1, 5), 9), [5], [5], 2, 2).tolist() == [[[0, 1]]]


def test_an_append_goes_by_the_lengths_where_the_bound_has_no_room():
    c = ta.KV4Cache(3, 1, 32, 64, device="cpu")
    x = torch.zeros(3, 1, 20, 64, dtype=torch.bfloat16)
    c.length_bound = 32
    c.seqlens[:] = torch.tensor([12, 3, 0])
    with pytest.raises(ValueError, match="CUDA tensors"):     # there is room: on to the kernel, which wants a GPU
        c.append(x, x)
    c.seqlens[1] = 13
    with pytest.raises(ValueError, match="may not fit"):
        c.append(x, x)
    with pytest.raises(ValueError, match="may not fit"):
        c.append(x, x, counts=torch.tensor([-5, 99, 0], dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA tensors"):
        c.append(x, x, counts=torch.tensor([20, 19, 20], dtype=torch.int32))
    assert c.seqlens.tolist() == [12, 13, 0] and c.length_bound == 32


def test_reset_empties_sequences():
    c = ta.KV4Cache(3, 1, 32, 64, device="cpu")
    c.length_bound = 30
    c.seqlens[:], c.next_pos[:] = torch.tensor([12, 30, 1]), torch.tensor([40, 50, 60])
    c.reset(torch.tensor([True, False, True]))
    assert c.seqlens.tolist() == [0, 30, 0] and c.next_pos.tolist() == [0, 50, 0] and c.length_bound == 30
    c.reset()
    assert c.seqlens.tolist() == [0, 0, 0] and c.next_pos.tolist() == [0, 0, 0] and c.length_bound == 0
