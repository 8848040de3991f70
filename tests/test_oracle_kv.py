"""Pins of the key/value cache oracle (oracle/kv.py) on the CPU: hand-checked
layout and page assignment, the weights' quantizer on the same values, and
attention against a direct softmax."""

import numpy as np
import pytest

from oracle import kv, quantize_groups


def test_heads_quantize_as_weight_groups():
    x = np.random.default_rng(1).normal(0, 2, (5, 128)).astype(np.float16)
    for zp in (True, False):
        q, s, z = kv.quantize_heads(x.astype(np.float32), zp)
        rq, rs, rz = quantize_groups(x, 128, zero_point=zp)
        assert np.array_equal(q, rq) and np.array_equal(s, rs[:, 0])
        assert (z is None and rz is None) or np.array_equal(z, rz[:, 0])


def test_layout_by_hand():
    """Token 5 of page 1: key words together, value words four tokens apart."""
    D, page = 64, 16
    cache = kv.new_cache(2, 1, D, page)
    K = np.zeros((1, 1, D), np.float32)
    K[0, 0, 8 * 3 + 2] = 15.0               # word 3, channel 2: nibble 1 (ORDER[1] = 2)
    V = np.zeros((1, 1, D), np.float32)
    V[0, 0, 8 * 6 + 1] = -15.0              # word 6, channel 1: nibble 4 (ORDER[4] = 1)
    kv.append(cache, K, V, np.array([16 + 5]))
    codes, scales, zeros = cache
    assert codes[1, 0, 0, 5 * 8 + 3] == 0xF << 4
    assert scales[1, 0, 5].tolist() == [1.0, 1.0]
    assert zeros[1, 0, 5].tolist() == [0, 15]
    want = 0xFFFFFFFF
    for w in range(8):
        assert codes[1, 1, 0, (5 // 4) * 32 + w * 4 + 5 % 4] == (want & ~(0xF << 16) if w == 6 else want)
    assert codes[0].sum() == 0
    _, _, _, val = kv.read(cache, D, [21])
    assert np.array_equal(val[0, 0], K[0]) and np.array_equal(val[1, 0], V[0])


def test_assign_by_hand():
    table = np.array([[7, -1, -1], [-1, -1, -1], [3, 4, -1]], np.int32)
    t, lens, start, slots, used = kv.assign([15, 0, 32], [3, 0, 1], table, [9, 8], 16, 6)
    assert t.tolist() == [[7, 9, -1], [-1, -1, -1], [3, 4, 8]]
    assert lens.tolist() == [18, 0, 33] and start.tolist() == [0, 3, 3, 4] and used.tolist() == [2]
    assert slots.tolist() == [7 * 16 + 15, 9 * 16, 9 * 16 + 1, 8 * 16, -1, -1]


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 3), (False, 0)])
def test_attention_against_direct_softmax(causal, window):
    rng = np.random.default_rng(3)
    D, page, n, nq = 64, 16, 21, 4
    cache = kv.new_cache(3, 2, D, page)
    table = np.array([[2, 0]], np.int32)
    pos = np.arange(n)
    kv.append(cache, rng.normal(size=(n, 2, D)), rng.normal(size=(n, 2, D)), table[0, pos // page] * page + pos % page)
    Q = rng.normal(size=(nq, 4, D))
    O, lse, bound, _ = kv.attention64(Q, cache, table, [n], [0, nq], 0.125, causal, window)
    _, _, _, val = kv.read(cache, D, table[0, pos // page] * page + pos % page)
    for i in range(nq):
        last = n - nq + i if causal else n - 1
        lo = max(0, last - window + 1) if window else 0
        for j in range(4):
            e = np.exp(val[0, lo:last + 1, j // 2] @ Q[i, j] * 0.125)
            assert np.allclose(O[i, j], e @ val[1, lo:last + 1, j // 2] / e.sum(), atol=1e-12)
            assert np.isclose(lse[i, j], np.log(e.sum()))
    assert (bound > 0).all() and bound.max() < 0.02
