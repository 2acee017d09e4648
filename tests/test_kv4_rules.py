"""The 4-bit cache's rules without a GPU, beyond tests/test_kv4.py."""
import numpy as np

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
