"""awq_kv_attention_ex without a GPU: every refusal before any HIP call, its workspaces, and
the oracle's sinks by hand."""

import ctypes

import numpy as np
import pytest

from oracle import kv
from test_kv_abi_cpu import CACHE_REFUSALS, INVALID, UNSUPPORTED, WORKSPACE, P, addr, binding, cache, cfg, i32, lib, tensors, torch

OK = binding.AWQ_OK


def opts(causal=1, window=0, sinks=0, prefix=0, table=addr(12), blocks=8):
    return ctypes.byref(binding.awq_kv_attention_options(causal, window, sinks, prefix, table, blocks))


def attend(o=None, c=None, conf=None, T=3, B=3, heads=4, qs=256, qt=0, Q=addr(7), table=addr(8), blocks=4,
           lens=addr(9), start=None, mq=1, mk=64, scale=0.1, O=addr(10), lse=None, ws=addr(13), wsb=1 << 20):
    return lib.awq_kv_attention_ex(Q, qt, T, qs, heads, cache() if c is None else c, conf or cfg(64), table, blocks, lens,
                                   start, B, mq, mk, scale, opts(prefix=20) if o is None else o, O, lse, ws, wsb, None)


@pytest.mark.parametrize("kw,status", CACHE_REFUSALS)
def test_cache_refusals(kw, status):
    assert attend(c=cache(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(o=ctypes.POINTER(binding.awq_kv_attention_options)()), INVALID),
    (dict(o=opts(window=-1)), INVALID), (dict(o=opts(sinks=-1, window=4)), INVALID), (dict(o=opts(sinks=2 ** 30 + 1, window=4)), INVALID),
    (dict(o=opts(causal=2)), INVALID), (dict(o=opts(causal=0, window=4, sinks=1)), INVALID),
    (dict(o=opts(prefix=-1)), INVALID), (dict(o=opts(prefix=20, blocks=-1)), INVALID), (dict(o=opts(prefix=20, blocks=1)), INVALID),
    (dict(o=opts(prefix=20, window=5)), UNSUPPORTED), (dict(o=opts(prefix=2 ** 30 + 1, blocks=2 ** 27)), UNSUPPORTED),
    (dict(o=opts(prefix=20, table=None), blocks=1), INVALID), (dict(o=opts(prefix=20, table=P(0x10002))), INVALID),
    (dict(T=2 ** 30, B=3, start=addr(11), mq=1, o=opts(prefix=20)), UNSUPPORTED),
    (dict(T=2 ** 24 + 1, B=3, start=addr(11), mq=1, o=opts(prefix=20)), UNSUPPORTED),
    (dict(qt=2), INVALID), (dict(T=-1), INVALID), (dict(heads=3), INVALID), (dict(qs=250), INVALID), (dict(mq=2), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(blocks=2 ** 28), INVALID), (dict(Q=None), INVALID), (dict(O=None), INVALID),
    (dict(lens=None), INVALID), (dict(table=None), INVALID), (dict(ws=None), WORKSPACE), (dict(wsb=64), WORKSPACE),
    (dict(ws=P(0x40000010)), INVALID), (dict(O=addr(12)), INVALID), (dict(ws=P(addr(12).value - 256)), INVALID),
    (dict(lse=P(addr(12).value + 28)), INVALID), (dict(O=addr(7)), INVALID),
])
def test_refusals(kw, status):
    assert attend(**kw) == status
    assert "awq_kv_attention_ex" in lib.awq_last_error().decode()


def test_workspaces():
    def size(T=3, B=3, heads=4, mq=1, mk=64, o=None):
        return lib.awq_kv_attention_ex_workspace_size(T, B, heads, cache(), cfg(64), mq, mk, o or opts())
    plain = lib.awq_kv_attention_workspace_size
    assert size(mk=60000) == plain(3, 3, 4, cache(), cfg(64), 1, 60000, 0) > 0
    assert size(mk=60000, o=opts(window=100, sinks=4)) == 0 < size(mk=60000, o=opts(window=100, sinks=50000))
    rows = 3 * 4 * (64 * 4 + 12)                            # a part's results: values, two floats, one
    assert size(o=opts(prefix=20)) == 2 * rows and size(T=0, B=0, o=opts(prefix=20)) == 0
    assert size(o=opts(prefix=20, table=None)) == 0         # (in one pass: too little to save)
    assert size(T=64, B=64, mk=9000, o=opts(prefix=8000, table=None)) == size(T=64, B=64, mk=9000, o=opts(prefix=8000, blocks=500)) > 0
    assert size(o=opts(prefix=200, blocks=8)) == 0 and size(o=opts(prefix=20, window=3)) == 0
    assert attend(T=0, B=0, Q=None, O=None, lens=None, table=None, ws=None) == OK
    assert attend(T=0, B=0, Q=None, O=None, lens=None, table=None, ws=None, o=opts(prefix=20, table=None)) == OK


def test_oracle_sinks_by_hand():
    """Row 9 of a window of 2 with 3 sinks: keys 0, 1, 2, 8, 9, weighed as a request of those."""
    rng = np.random.default_rng(0)
    c = kv.new_cache(2, 1, 64, 16)
    x = rng.normal(size=(2, 10, 1, 64))
    kv.append(c, x[0], x[1], np.arange(10))
    kv.append(c, x[0][[0, 1, 2, 8, 9]], x[1][[0, 1, 2, 8, 9]], np.arange(16, 21))
    q = rng.normal(size=(1, 2, 64))
    a = kv.attention64(q, c, np.array([[0]]), [10], [0, 1], 0.125, True, 2, sinks=3)
    b = kv.attention64(q, c, np.array([[1]]), [5], [0, 1], 0.125)
    assert np.allclose(a[0], b[0], rtol=1e-14) and np.allclose(a[1], b[1], rtol=1e-14)


def test_binding_refuses_wrong_prefixes():
    c = tensors()
    ok = dict(Q=torch.zeros((3, 4, 64), dtype=torch.float16), cache=c, block_table=i32(3, 4), seq_lens=i32(3), prefix_len=20)
    for kw, e in ((dict(prefix_table=i32(4).long()), TypeError), (dict(prefix_table=i32(1, 4)), ValueError),
                  (dict(prefix_table=i32(4), prefix_len=0), ValueError), (dict(workspace="x"), ValueError)):
        with pytest.raises(e):
            binding.awq_kv_attention(**{**ok, **kw})
    with pytest.raises(ValueError, match="GPU"):
        binding.awq_kv_attention(**ok)
    with pytest.raises(ValueError, match="GPU"):
        binding.awq_kv_attention(**{**ok, "prefix_len": 0, "window": 3, "sinks": 2})


@pytest.mark.parametrize("kw", [dict(prefix_table=i32(0)), dict(prefix_len=0, window=3, sinks=2, prefix_table=i32(4))])
def test_binding_refuses_tables_that_would_go_unread(kw):
    """An empty one (its address is NULL, which means none), and one beside sinks alone."""
    ok = dict(Q=torch.zeros((3, 4, 64), dtype=torch.float16), cache=tensors(), block_table=i32(3, 4), seq_lens=i32(3), prefix_len=20)
    with pytest.raises(ValueError, match="prefix_table"):
        binding.awq_kv_attention(**{**ok, **kw})
