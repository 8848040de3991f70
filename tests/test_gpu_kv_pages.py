"""GPU parity of the cache's page operations with oracle/kv_pages.py: tables, counts,
lists and every bit of the cache equal."""

import numpy as np
import pytest

from gpu_common import dev, out_to_f64, say, torch_mod
from oracle import kv
from oracle import kv_pages as pg
from test_gpu_kv import _i32, _rounded, _same_cache, _to_cache

pytestmark = pytest.mark.gpu


def _pool(rng, lens, page, spare, blocks=None, share=0.0):
    """(table, shared, free) of rows of these lengths, pages in random order; with `share`,
    some rows hold pages of an earlier one."""
    need = [-(-max(0, n) // page) for n in lens]
    blocks = blocks or max(max(need, default=0), 1) + 2
    pages = sum(need) + spare
    order = rng.permutation(pages).astype(np.int32)
    table = np.full((len(lens), blocks), -1, np.int32)
    shared = np.zeros(pages, np.int32)
    at = 0
    for b, n in enumerate(need):
        for j in range(min(n, blocks)):
            if b and rng.random() < share and table[b - 1, j] >= 0:
                table[b, j] = table[b - 1, j]
                shared[table[b, j]] += 1
            else:
                table[b, j] = order[at]
                at += 1
    return table, shared, order[at:].copy()


def _eq(got, want):
    assert np.array_equal(got.cpu().numpy().reshape(np.shape(want)), want)


@pytest.mark.parametrize("heads,D,page,zp,n", [(1, 64, 16, True, 1), (3, 128, 32, False, 7), (8, 128, 64, True, 40),
                                               (2, 64, 1024, True, 3), (5, 64, 16, False, 300)])
def test_copy_pages(heads, D, page, zp, n):
    import bit_weight_only_quantize_amd as awq
    say("copy", heads, D, page, zp, n)
    rng = np.random.default_rng(n)
    pages = 2 * n + 5
    cache = kv.new_cache(pages, heads, D, page, zp, rng)
    order = rng.permutation(pages).astype(np.int32)
    src, dst = order[:n].copy(), order[n:2 * n].copy()
    if n > 6:
        src[1], dst[2], src[3], dst[4] = -1, -5, pages, 2 ** 31 - 1
        dst[5] = src[5]
        src[6] = src[0]                             # one page to two places
    got = _to_cache(cache)
    assert awq.awq_kv_copy_pages(got, _i32(src), _i32(dst)) is got
    pg.copy_pages(cache, src, dst)
    _same_cache(got, cache)
    awq.awq_kv_copy_pages(got, _i32([]), _i32([]))
    _same_cache(got, cache)


def _fork_case(rng, n, page, blocks=9):
    rows = 2 * n + 3
    lens = [int(rng.integers(1, (blocks - 1) * page)) for _ in range(n + 3)] + [0] * n
    table, shared, free = _pool(rng, lens, page, n + 4, blocks, 0.2)
    table[n + 3:] = rng.integers(-9, 10 ** 6, (n, blocks))     # what lies in children's rows does not matter
    parents = rng.integers(0, n + 3, n)
    children = rng.permutation(np.arange(n + 3, rows))[:n]
    share = [int(rng.integers(0, lens[p] + 1)) for p in parents]
    return table, shared, free, parents, children, np.array(share)


@pytest.mark.parametrize("name,n,page,heads,D,zp,taken", [
    ("one", 1, 16, 1, 64, True, None), ("some", 9, 16, 2, 128, False, 2), ("large pages", 4, 1024, 1, 64, True, 0),
    ("many", 700, 16, 1, 64, True, 3), ("all heads", 5, 64, 32, 128, True, 1),
])
def test_fork(name, n, page, heads, D, zp, taken):
    import bit_weight_only_quantize_amd as awq
    say("fork", name)
    rng = np.random.default_rng(n)
    table, shared, free, parents, children, lens = _fork_case(rng, n, page, 4 if page == 1024 else 9)
    if n > 4:
        lens[0], lens[1], lens[2], lens[3] = 0, page, page - 1, 10 ** 9     # none, one full, a part, past the table
        parents[4] = -1
        table[parents[2], 0] = -1                   # a parent without the page that would be copied
    if name == "many":
        free = free[:n // 2]                        # the list runs out
        children[7], children[8] = len(table), -3   # rows outside the table
        parents[9] = children[9]
    cache = kv.new_cache(len(shared), heads, D, page, zp, rng)
    got, tab, sh = _to_cache(cache), _i32(table), _i32(shared)
    used = awq.awq_kv_fork(got, tab, _i32(parents), _i32(children), _i32(lens), sh, _i32(free),
                           taken=None if taken is None else _i32([taken]))
    want = pg.fork(cache, table, parents, children, lens, shared, free, page, taken or 0)
    _eq(tab, table), _eq(sh, shared), _eq(used, [want])
    _same_cache(got, cache)


def test_fork_of_nothing_reports_what_was_taken():
    import bit_weight_only_quantize_amd as awq
    cache = awq.empty_kv_cache(3, 1, 64, 16, dev())
    none = _i32([])
    args = (cache, _i32(np.zeros((2, 2))), none, none, none, _i32([0, 0, 0]), _i32([1]))
    assert awq.awq_kv_fork(*args, taken=_i32([5])).item() == 5 and awq.awq_kv_fork(*args).item() == 0
    assert awq.awq_kv_fork(*args, taken=_i32([-4])).item() == 0


@pytest.mark.parametrize("name,rows,most,page,spare,share", [
    ("one", 1, 30, 16, 0, 0.0), ("rows", 12, 300, 16, 9, 0.4), ("alone, full", 200, 3000, 16, 2000, 0.3),
    ("chunks", 300, 9000, 16, 3000, 0.3), ("large pages", 30, 9000, 1024, 100, 0.2),
])
@pytest.mark.parametrize("ranges", ["all", "behind", "window"])
def test_release(name, rows, most, page, spare, share, ranges):
    import bit_weight_only_quantize_amd as awq
    say("release", name, ranges)
    rng = np.random.default_rng(rows + most)
    lens = rng.integers(0, most + 1, rows)
    table, shared, free = _pool(rng, lens, page, spare, None, share)
    start = end = None
    if ranges == "behind":                          # some rows keep everything, some nothing
        start = np.where(rng.random(rows) < 0.3, lens, rng.integers(-5, most + 20, rows))
    elif ranges == "window":
        start, end = rng.integers(-3, 50, rows), rng.integers(-5, most + 40, rows)
    if rows > 5:
        table[2, 0] = -1                            # a hole, and an id outside the pool
        table[3, 0] = len(shared) + 3
        lens[4] = -7
        free = np.concatenate([free, [-1, len(shared), -1]]).astype(np.int32)
    taken = min(5, len(free)) if rows > 1 else 0
    tab, sh = _i32(table), _i32(shared)
    opt = lambda a: None if a is None else _i32(a)  # noqa: E731
    got, count = awq.awq_kv_release(tab, _i32(lens), sh, _i32(free), page, start=opt(start), end=opt(end),
                                    pages_used=_i32([taken]))
    want = pg.release(table, lens, shared, free, page, start, end, taken)
    _eq(tab, table), _eq(sh, shared), _eq(count, [len(want)]), _eq(got, pg.padded(want, len(shared)))
    # released once, there is nothing to release; a list shorter than what it should hold
    out = (_i32([7, 7]), _i32([0]))
    awq.awq_kv_release(tab, _i32(lens), sh, got, page, start=opt(start), end=opt(end), out=out)
    _eq(tab, table), _eq(sh, shared), _eq(out[0], pg.padded(want, 2)), _eq(out[1], [len(want)])


def test_release_keeps_pages_that_others_hold():
    import bit_weight_only_quantize_amd as awq
    table = np.array([[3, 1, -1], [3, 2, -1], [3, 0, -1]], np.int32)
    tab, sh = _i32(table), _i32([0, 0, 0, 2])
    none = _i32([])
    free, n = awq.awq_kv_release(tab, _i32([20, 0, 20]), sh, none, 16)
    _eq(free, [0, 1, -1, -1]), _eq(n, [2]), _eq(sh, [0, 0, 0, 0])
    free, n = awq.awq_kv_release(tab, _i32([0, 20, 0]), sh, free, 16)
    _eq(free, [0, 1, 2, 3]), _eq(n, [4]), _eq(tab, np.full((3, 3), -1))


@pytest.mark.parametrize("name,rows,most,page,spare,share,heads,D,zp", [
    ("one row", 1, 30, 16, 5, 0.0, 1, 64, True), ("rows", 12, 300, 16, 60, 0.4, 3, 128, False),
    ("full", 10, 200, 32, 0, 0.0, 2, 64, True), ("large pages", 6, 4000, 1024, 9, 0.2, 1, 128, True),
    ("sparse", 3, 100, 16, 3000, 0.0, 1, 64, True), ("chunks", 300, 1500, 16, 20000, 0.1, 1, 64, False),
])
def test_compact(name, rows, most, page, spare, share, heads, D, zp):
    import bit_weight_only_quantize_amd as awq
    say("compact", name)
    rng = np.random.default_rng(rows + most)
    lens = rng.integers(1, most + 1, rows)
    table, shared, _ = _pool(rng, lens, page, spare, None, share)
    if rows > 5:
        table[2, 0] = -1
        table[3, 0] = len(shared) + 3
        lens[4] = -7                                # its entries count for nothing, and are left alone
    shared[rng.integers(0, len(shared))] += 1       # a count of a page that may be in no use
    if name == "chunks":
        # more than one workgroup ranks: as many pages, but a cache of no size to speak of
        assert len(shared) > 32768
    cache = kv.new_cache(len(shared), heads, D, page, zp, rng)
    got, tab, sh = _to_cache(cache), _i32(table), _i32(shared)
    before = [None if a is None else a.copy() for a in cache]
    free, used = awq.awq_kv_compact(got, tab, _i32(lens), sh)
    want, n = pg.compact(cache, table, lens, shared, page)
    _eq(tab, table), _eq(sh, shared), _eq(used, [n]), _eq(free, pg.padded(want, len(shared)))
    _same_cache(got, cache)
    # what the rows hold is what they held, and there is nothing more to move
    free2, used2 = awq.awq_kv_compact(got, tab, _i32(lens), sh)
    _eq(tab, table), _eq(sh, shared), _eq(used2, [n]), _eq(free2, pg.padded(want, len(shared)))
    _same_cache(got, cache)
    assert before[0].shape == cache[0].shape


def test_compact_with_a_wide_table():
    """A small pool, and more table entries than one workgroup looks through."""
    import bit_weight_only_quantize_amd as awq
    rng = np.random.default_rng(5)
    lens = rng.integers(0, 200, 90)
    table, shared, _ = _pool(rng, lens, 16, 300, 800, 0.2)
    cache = kv.new_cache(len(shared), 1, 64, 16, True, rng)
    got, tab, sh = _to_cache(cache), _i32(table), _i32(shared)
    free, used = awq.awq_kv_compact(got, tab, _i32(lens), sh)
    want, n = pg.compact(cache, table, lens, shared, 16)
    _eq(tab, table), _eq(sh, shared), _eq(used, [n]), _eq(free, pg.padded(want, len(shared)))
    _same_cache(got, cache)


def test_compact_of_nothing():
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    cache = awq.empty_kv_cache(5, 1, 64, 16, dev())
    for table, lens in ((np.zeros((0, 3)), []), (np.full((2, 3), 4), [0, 0])):
        free, used = awq.awq_kv_compact(cache, _i32(table), _i32(lens), torch.zeros(5, dtype=torch.int32, device=dev()))
        _eq(free, [0, 1, 2, 3, 4]), _eq(used, [0])


def test_refusals_name_what_overlaps():
    import bit_weight_only_quantize_amd as awq
    cache = awq.empty_kv_cache(4, 1, 64, 16, dev())
    shared, table, lens = _i32([0, 0, 0, 0]), _i32(np.zeros((2, 2))), _i32([3, 3])
    with pytest.raises(awq.AwqError, match="overlap"):
        awq.awq_kv_release(table, lens, shared, _i32([1]), 16, out=(shared, _i32([0])))
    with pytest.raises(awq.AwqError, match="overlap"):
        awq.awq_kv_compact(cache, table, lens, shared, out=(shared, _i32([0])))
    with pytest.raises(awq.AwqError, match="workspace"):
        awq.awq_kv_compact(cache, table, lens, shared, workspace=None)
    with pytest.raises(awq.AwqError, match="overlap"):
        awq.awq_kv_fork(cache, table, lens, lens, lens, shared, _i32([1]), out=lens[:1])


def test_a_step_captured():
    """assign, append, fork, release and compact as one graph, replayed with other lengths: every
    replay leaves what the eager calls leave."""
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    rng = np.random.default_rng(2)
    B, blocks, page, pages, H, D = 6, 5, 16, 40, 2, 64
    lens0 = np.array([5, 40, 16, 0, 0, 63], np.int32)
    table0, shared0, free0 = _pool(rng, lens0, page, 0, blocks)
    extra = np.setdiff1d(np.arange(pages), table0[table0 >= 0])
    table0, free0 = table0, pg.padded(list(extra), pages)
    shared0 = np.zeros(pages, np.int32)
    cache0 = _to_cache(kv.new_cache(pages, H, D, page, True, np.random.default_rng(4)))
    new = lambda: [_i32(table0), _i32(shared0), _i32(free0), _i32(lens0), _i32([1, 3, 0, 0, 0, 2]),    # noqa: E731
                   _i32([1]), _i32([3]), _i32([37]), *[c.clone() for c in cache0]]
    K = torch.randn((9, H, D), device=dev()).half()
    bits = lambda t: t.view(torch.int16) if t.dtype is torch.float16 else t   # noqa: E731

    def step(table, shared, free, lens, more, parents, children, share, *cache):
        seq, start, slots, used = awq.awq_kv_assign(lens, more, table, free, page, 9)
        awq.awq_kv_append(K, K, cache, slots)
        used = awq.awq_kv_fork(cache, table, parents, children, share, shared, free, taken=used)
        zero = torch.zeros_like(lens)
        gone = torch.where(torch.arange(B, device=dev()) == 1, zero, seq)       # row 1 ends, its branch goes on
        free2, count = awq.awq_kv_release(table, seq, shared, free, page, start=gone, pages_used=used)
        live = gone.clone()
        live[3:4] = share
        free3, n = awq.awq_kv_compact(cache, table, live, shared)
        return table, shared, free2, count, free3, n, live, *cache

    state = new()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*new())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(*state)
    for i in range(4):
        for s, v in zip(state, new()):
            s.copy_(v)
        state[7].fill_(37 - 7 * i)
        graph.replay()
        torch.cuda.synchronize()
        fresh = new()
        fresh[7].fill_(37 - 7 * i)
        for a, b in zip(out, step(*fresh)):             # (bits: a step of the pool's may be NaN)
            assert torch.equal(bits(a), bits(b))
        # and the branch reads what its parent had
        k, _ = awq.awq_kv_gather(tuple(fresh[8:]), fresh[0][3, 0] * page + torch.arange(5, device=dev(), dtype=torch.int32))
        was, _ = awq.awq_kv_gather(cache0, _i32(table0[1, 0] * page + np.arange(5)))
        assert torch.equal(bits(k), bits(was))


def test_pages_past_32_bit_byte_offsets():
    """A cache of more than 4 GiB of codes: pages at its end are copied, forked from and drawn to the front."""
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    H, D, page = 8, 128, 64
    pages = 72 * 1024                                       # 4.5 GiB of codes
    cache = awq.empty_kv_cache(pages, H, D, page, dev())
    g = torch.Generator(device=dev()).manual_seed(3)
    last = [pages - 1, pages - 2]
    for c in cache:
        c[:4].zero_()
        for p in last:
            c[p] = torch.randint(0, 100, c[p].shape, generator=g, device=dev()).to(c.dtype)
    kept = [[c[p].clone() for c in cache] for p in last]
    same = lambda p, want: all(torch.equal(c[p], w) for c, w in zip(cache, want))     # noqa: E731
    awq.awq_kv_copy_pages(cache, _i32(last), _i32([1, pages - 3]))
    assert same(1, kept[0]) and same(pages - 3, kept[1]) and same(pages - 1, kept[0])
    table, shared = _i32([[pages - 1, pages - 2], [-1, -1]]), torch.zeros(pages, dtype=torch.int32, device=dev())
    used = awq.awq_kv_fork(cache, table, _i32([0]), _i32([1]), _i32([page + 5]), shared, _i32([pages - 4]))
    assert used.item() == 1 and table.tolist()[1] == [pages - 1, pages - 4] and same(pages - 4, kept[1])
    free, n = awq.awq_kv_compact(cache, table, _i32([2 * page, page + 5]), shared)
    assert n.item() == 3 and table.tolist() == [[0, 1], [0, 2]] and free[0].item() == 3
    assert same(0, kept[0]) and same(1, kept[1]) and same(2, kept[1])
    assert shared[0].item() == 1 and shared.sum().item() == 1


@pytest.mark.parametrize("blocks", [32, 33, 64, 65])
def test_release_of_small_and_large_tables(blocks):
    """64 rows of so many entries: up to 2048 one launch serves, beyond that two."""
    import bit_weight_only_quantize_amd as awq
    rng = np.random.default_rng(blocks)
    lens = rng.integers(1, blocks * 16 + 1, 64)
    lens[0] = blocks * 16
    table, shared, free = _pool(rng, lens, 16, 50, None, 0.3)
    assert table.shape[1] >= blocks
    table = np.ascontiguousarray(table[:, :blocks])
    start = np.where(rng.random(64) < 0.5, 0, rng.integers(0, blocks * 16, 64))
    tab, sh = _i32(table), _i32(shared)
    got, count = awq.awq_kv_release(tab, _i32(lens), sh, _i32(free), 16, start=_i32(start), pages_used=_i32([3]))
    want = pg.release(table, lens, shared, free, 16, start, None, 3)
    _eq(tab, table), _eq(sh, shared), _eq(count, [len(want)]), _eq(got, pg.padded(want, len(shared)))
