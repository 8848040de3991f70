"""The page operations without a GPU: the oracle by hand, and every refusal before any
HIP call."""

import ctypes

import numpy as np
import pytest

from oracle import kv, kv_pages as pg
from test_kv_abi_cpu import CACHE_REFUSALS, INVALID, UNSUPPORTED, WORKSPACE, P, addr, binding, cache, cfg, i32, lib, tensors, torch

OK = binding.AWQ_OK


def test_oracle_by_hand():
    c = kv.new_cache(6, 1, 64, 16, True, np.random.default_rng(0))
    table = np.array([[4, 2, 5], [9, 9, 9]], np.int32)
    shared, free = np.zeros(6, np.int32), np.array([1, 0, 3], np.int32)
    assert pg.fork(c, table, [0], [1], [20], shared, free, 16, taken=1) == 2
    assert table.tolist() == [[4, 2, 5], [4, 0, 9]] and shared.tolist() == [0, 0, 0, 0, 1, 0]
    assert (c[0][0] == c[0][2]).all()
    free = pg.release(table, [48, 0], shared, free, 16, taken=2)
    assert free == [3, 2, 5] and table.tolist() == [[-1, -1, -1], [4, 0, 9]]
    free, n = pg.compact(c, table, [0, 20], shared, 16)
    assert n == 2 and table.tolist()[1] == [1, 0, 9] and free == [2, 3, 4, 5]


def test_oracle_releases_a_window():
    table, shared = np.array([[0, 1, 2, 3]], np.int32), np.zeros(4, np.int32)
    assert pg.release(table, [60], shared, [], 16, [4], [47]) == [1]        # page 2's last token is 47
    assert pg.release(table, [60], shared, [], 16, [4], [48]) == [2]
    assert pg.release(table, [60], shared, [], 16, [4], [60]) == [3]


def copy(c=None, conf=None, src=addr(4), dst=addr(5), n=3):
    return lib.awq_kv_copy_pages(cache() if c is None else c, conf or cfg(64), src, dst, n, None)


def fork(c=None, conf=None, n=2, B=3, blocks=4, free=5, p=None):
    a = [addr(i) for i in range(4, 12)]     # parents children lens table shared free taken used
    for i, v in (p or {}).items():
        a[i] = v
    return lib.awq_kv_fork(cache() if c is None else c, conf or cfg(64), a[0], a[1], a[2], n, a[3], B, blocks, a[4],
                           a[5], free, a[6], a[7], None)


def release(B=3, blocks=4, page=16, pages=8, free=5, out=8, ws=None, wsb=0, p=None):
    a = [addr(i) for i in range(4, 13)]     # table lens start end shared free taken free_out count
    for i, v in (p or {}).items():
        a[i] = v
    return lib.awq_kv_release(a[0], B, blocks, page, a[1], a[2], a[3], a[4], pages, a[5], free, a[6], a[7], out, a[8],
                              ws, wsb, None)


def compact(c=None, conf=None, B=3, blocks=4, ws=addr(12), wsb=1 << 16, p=None):
    a = [addr(i) for i in range(4, 9)]      # table lens shared free_out used
    for i, v in (p or {}).items():
        a[i] = v
    return lib.awq_kv_compact(cache() if c is None else c, conf or cfg(64), a[0], B, blocks, a[1], a[2], a[3], a[4], ws,
                              wsb, None)


@pytest.mark.parametrize("kw,status", CACHE_REFUSALS)
@pytest.mark.parametrize("call", [copy, fork, compact])
def test_cache_refusals(call, kw, status):
    assert call(c=cache(**kw)) == status


@pytest.mark.parametrize("call", [copy, fork, compact])
def test_config_refusals(call):
    assert call(conf=cfg(64, w_bit=8)) == UNSUPPORTED and call(conf=cfg(128)) == UNSUPPORTED
    assert call(c=ctypes.POINTER(binding.awq_kv_cache)()) == INVALID


ODD, CODES = P(0x10002), P(0x10000)


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), INVALID), (dict(n=2 ** 27 + 1), INVALID), (dict(src=None), INVALID), (dict(dst=None), INVALID),
    (dict(src=ODD), INVALID), (dict(src=CODES), INVALID), (dict(dst=P(0x300000)), INVALID),
])
def test_copy_refusals(kw, status):
    assert copy(**kw) == status and "awq_kv_copy_pages" in lib.awq_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(n=-1), INVALID), (dict(n=65536), UNSUPPORTED), (dict(B=-1), INVALID), (dict(B=2 ** 20 + 1), UNSUPPORTED),
    (dict(blocks=-1), INVALID), (dict(blocks=2 ** 27), UNSUPPORTED), (dict(free=-1), INVALID),
    *[(dict(p={i: None}), INVALID) for i in (0, 1, 2, 3, 4, 5, 7)],
    *[(dict(p={i: ODD}), INVALID) for i in range(8)],
    *[(dict(p={i: CODES}), INVALID) for i in range(8)],
    (dict(p={7: addr(10)}), INVALID), (dict(p={4: addr(7)}), INVALID), (dict(p={3: addr(4)}), INVALID),
    (dict(p={7: addr(7)}), INVALID),
])
def test_fork_refusals(kw, status):
    assert fork(**kw) == status and "awq_kv_fork" in lib.awq_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(page=24), UNSUPPORTED), (dict(B=-1), INVALID), (dict(B=2 ** 20 + 1), UNSUPPORTED), (dict(blocks=2 ** 27), UNSUPPORTED),
    (dict(pages=0), INVALID), (dict(pages=2 ** 27 + 1), INVALID), (dict(free=-1), INVALID), (dict(out=-1), INVALID),
    *[(dict(p={i: None}), INVALID) for i in (0, 1, 4, 5, 7, 8)],
    *[(dict(p={i: ODD}), INVALID) for i in range(9)],
    (dict(p={7: addr(9)}), INVALID), (dict(p={7: addr(8)}), INVALID), (dict(p={8: addr(10)}), INVALID), (dict(p={0: addr(5)}), INVALID),
    (dict(pages=40000), WORKSPACE), (dict(pages=40000, ws=P(0x40000010), wsb=1 << 20), INVALID),
    (dict(pages=40000, ws=addr(5), wsb=1 << 20), INVALID),
])
def test_release_refusals(kw, status):
    assert release(**kw) == status and "awq_kv_release" in lib.awq_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(B=-1), INVALID), (dict(B=2 ** 20 + 1), UNSUPPORTED), (dict(blocks=2 ** 27), UNSUPPORTED),
    *[(dict(p={i: None}), INVALID) for i in range(5)], *[(dict(p={i: ODD}), INVALID) for i in range(5)],
    *[(dict(p={i: CODES}), INVALID) for i in range(5)],
    (dict(ws=None), WORKSPACE), (dict(wsb=100), WORKSPACE), (dict(ws=P(0x40000010)), INVALID), (dict(ws=CODES), INVALID),
    (dict(ws=addr(5)), INVALID), (dict(p={3: addr(6)}), INVALID),
])
def test_compact_refusals(kw, status):
    assert compact(**kw) == status and "awq_kv_compact" in lib.awq_last_error().decode()


def test_workspaces():
    r, c = lib.awq_kv_release_workspace_size, lib.awq_kv_compact_workspace_size
    assert r(100, 100) == 0 and r(32768, 0) == 0 and 0 < r(32768, 1) <= 4096 and r(0, 5) == 0 and r(5, -1) == 0
    assert r(2 ** 27, 2 ** 31 - 1) > 0 and r(2 ** 27 + 1, 0) == 0
    assert c(100, 16) >= 1200 and c(100, 16) % 256 == 0 and c(0, 16) == 0 and c(100, 24) == 0
    assert c(2 ** 27, 16) > 3 * 2 ** 29 and c(2 ** 27, 32) == 0


def test_nothing_to_copy():
    assert copy(n=0, src=None, dst=None) == OK


def test_binding_refuses_wrong_tensors():
    c = tensors()
    ok = dict(cache=c, block_table=i32(3, 4), parents=i32(2), children=i32(2), lens=i32(2), shared=i32(4), free_pages=i32(5))
    for k, v, e in (("block_table", i32(12), ValueError), ("parents", i32(2).long(), TypeError), ("children", i32(3), ValueError),
                    ("lens", i32(1), ValueError), ("shared", i32(5), ValueError), ("free_pages", i32(1, 5), ValueError),
                    ("taken", i32(2), ValueError), ("out", i32(2), ValueError), ("parents", i32(1, 2), ValueError)):
        with pytest.raises(e):
            binding.awq_kv_fork(**{**ok, k: v})
    with pytest.raises(ValueError, match="GPU"):
        binding.awq_kv_fork(**ok)
    ok = dict(block_table=i32(3, 4), seq_lens=i32(3), shared=i32(4), free_pages=i32(5), page_size=16)
    for k, v, e in (("seq_lens", i32(4), ValueError), ("start", i32(2), ValueError), ("end", i32(3).long(), TypeError),
                    ("shared", i32(0), ValueError), ("pages_used", i32(), ValueError), ("out", (i32(4),), ValueError),
                    ("out", (i32(4), i32(2)), ValueError), ("workspace", "some", ValueError)):
        with pytest.raises(e):
            binding.awq_kv_release(**{**ok, k: v})
    with pytest.raises(ValueError, match="GPU"):
        binding.awq_kv_release(**ok)
    ok = dict(cache=c, block_table=i32(3, 4), seq_lens=i32(3), shared=i32(4))
    for k, v, e in (("seq_lens", i32(4), ValueError), ("shared", i32(3), ValueError), ("out", (i32(3), i32(1)), ValueError),
                    ("cache", c[:2], TypeError)):
        with pytest.raises(e):
            binding.awq_kv_compact(**{**ok, k: v})
    with pytest.raises(ValueError, match="GPU"):
        binding.awq_kv_compact(**ok)
    with pytest.raises(ValueError):
        binding.awq_kv_copy_pages(c, i32(3), i32(2))
    with pytest.raises(ValueError, match="GPU"):
        binding.awq_kv_copy_pages(c, i32(3), i32(3))
