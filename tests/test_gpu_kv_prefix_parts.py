"""Requests behind a shared prefix whose own keys are split, too: the join over several parts of
the prefix and several of the rest.  Bounds are oracle/kv.py's, as in test_gpu_kv_some.py."""

import pytest

from test_gpu_kv_some import Behind

pytestmark = pytest.mark.gpu


def _parts(a):
    """Parts of the prefix and of the rest together, from the workspace that holds their results."""
    import bit_weight_only_quantize_amd as awq
    from test_gpu_kv import _to_cache
    T, Hq, D = a.Q.shape
    need = awq.awq_kv_attention_workspace_size(T, len(a.q_lens), Hq, _to_cache(a.cache), int(a.q_lens.max()),
                                               int(max(a.kv_lens)), prefix_len=a.prefix)
    each = T * Hq * (4 * D + 12)
    assert need % each == 0
    return need // each


@pytest.mark.parametrize("prefix,q_lens,kv_lens,Hq,Hkv,D,page,zp,dtype,parts", [
    (700, [1, 1], [2900, 2400], 8, 1, 64, 16, True, "float16", 11),                # 6 and 5
    (100, [1, 1, 1], [3000, 101, 1800], 4, 2, 128, 64, False, "bfloat16", 7),      # 1 and 6
    (1000, [3, 5], [3500, 2000], 6, 3, 128, 32, True, "float16", 13),              # 8 and 5
    (300, [40, 40], [1200, 900], 8, 1, 64, 16, True, "bfloat16", 7),               # a prompt's tiles: 3 and 4
    (300, [40, 1, 70], [1200, 301, 900], 4, 2, 128, 128, True, "float16", 7),
    (40, [129], [1500], 8, 8, 64, 64, False, "bfloat16", 7),                       # 1 and 6
])
def test_rest_in_parts(prefix, q_lens, kv_lens, Hq, Hkv, D, page, zp, dtype, parts):
    a = Behind(prefix, q_lens, kv_lens, Hq, Hkv, D, page, zp, dtype, seed=prefix)
    assert _parts(a) == parts
    a.check()


@pytest.mark.parametrize("kv_lens,D,zp,dtype,parts", [
    ([2601 + 3 * i for i in range(64)], 128, True, "float16", 12),                 # 11 and 1
    ([2601 + 37 * i for i in range(64)], 64, False, "bfloat16", 16),               # 11 and 5
])
def test_many_rows_of_many_parts(kv_lens, D, zp, dtype, parts):
    """2048 rows of more than eight parts: a wave joins a row, in two rounds or more."""
    a = Behind(2600, [1] * 64, kv_lens, 32, 2, D, 64, zp, dtype, seed=D)
    assert _parts(a) == parts
    a.check(whole=False)
