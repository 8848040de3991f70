"""Attention over a shared prefix without a table of its own: the pages come from a request that
holds them, wherever it stands in the batch, so a batch gives the same whether its prefix is read
once or by every request.  Where it is read once the result has the bits of the same call with a
table (which test_gpu_kv_some.py holds against the oracle), else those of the call without a prefix."""

import ctypes

import numpy as np
import pytest

from gpu_common import dev, say, torch_mod
from test_gpu_kv import _i32
from test_gpu_kv_some import Behind

pytestmark = pytest.mark.gpu


class Batch:
    """Requests of `q` tokens each (the first: `first`) behind a prefix, over a cache of random
    codes.  Rows share the prefix' full pages and have pages of their own behind them."""

    def __init__(self, n, q, first=None, prefix=3000, Hq=8, Hkv=8, D=128, page=64, seed=1):
        torch = torch_mod()
        g = torch.Generator(device=dev()).manual_seed(seed)
        full, own = prefix // page, 4
        self.prefix, self.page = prefix, page
        self.ids = np.random.default_rng(seed).permutation(full + n * own).astype(np.int32)
        self.whole = np.concatenate([np.tile(self.ids[:full], (n, 1)), self.ids[full:].reshape(n, own)], 1)
        self.table = self.whole.copy()
        pages = len(self.ids)
        self.cache = (torch.randint(-2 ** 31, 2 ** 31, (pages, 2, Hkv, page * D // 8), generator=g, device=dev(), dtype=torch.int32),
                      (torch.rand((pages, Hkv, page, 2), generator=g, device=dev()) * 0.2 + 0.01).half(),
                      torch.randint(0, 16, (pages, Hkv, page, 2), generator=g, device=dev(), dtype=torch.uint8))
        # the page that the prefix ends in: each row's own copy
        for c in self.cache:
            c[self.whole[1:, full].tolist()] = c[int(self.whole[0, full])].clone()
        self.q_lens = [q if first is None else first] + [q] * (n - 1)
        self.lens = np.array([prefix + q + 5 * b % (2 * page) for b in range(n)])
        self.start = np.concatenate([[0], np.cumsum(self.q_lens)])
        self.Q = torch.randn((int(self.start[-1]), Hq, D), generator=g, device=dev()).half()
        self.one = all(x == 1 for x in self.q_lens)

    def call(self, table, **kw):
        import bit_weight_only_quantize_amd as awq
        return awq.awq_kv_attention(self.Q, self.cache, _i32(table), _i32(self.lens), max_query_len=max(self.q_lens),
                                    query_start=None if self.one else _i32(self.start), max_seq_len=int(max(self.lens.max(), 0)),
                                    return_lse=True, **kw)

    def reads_once(self):
        """The workspace is then that of a call with a table."""
        from bit_weight_only_quantize_amd import binding
        T, Hq, D = self.Q.shape
        c = binding.awq_kv_cache(None, None, None, len(self.ids), self.page, self.cache[1].shape[1], D)
        need = lambda table: binding.lib.awq_kv_attention_ex_workspace_size(     # noqa: E731
            T, len(self.q_lens), Hq, c, binding.config(D), max(self.q_lens), int(max(self.lens.max(), 0)),
            ctypes.byref(binding.awq_kv_attention_options(1, 0, 0, self.prefix, table, -(-self.prefix // self.page))))
        return need(None) == need(256) > 0

    def check(self, once):
        torch = torch_mod()
        assert self.reads_once() == once
        kw = dict(prefix_len=self.prefix)
        want = self.call(self.whole, prefix_table=_i32(self.whole[0]), **kw) if once else self.call(self.whole)
        got = self.call(self.table, **kw)
        rows = [t for b in range(len(self.q_lens)) if self.lens[b] > 0 for t in range(self.start[b], self.start[b + 1])]
        say("prefix without a table", len(self.q_lens), self.q_lens[-1], once, len(rows), "rows that see keys")
        assert torch.isfinite(want[1][rows]).all()
        for w, g in zip(want, got):
            assert torch.equal(w, g)


# batches whose prefix is read once (in tiles of 16, 64 and 128 rows), and two whose requests each read it
BATCHES = [(32, 1, True), (40, 1, True), (100, 1, True), (20, 5, True), (3, 1, False), (2, 40, False)]


@pytest.mark.parametrize("n,q,once", BATCHES)
def test_a_padded_first_request(n, q, once):
    """seq_lens 0, no pages: its queries get zeros, the others lose nothing."""
    a = Batch(n, q)
    a.lens[0], a.table[0] = 0, -1
    a.check(once)
    assert (a.call(a.table, prefix_len=a.prefix)[0][:q] == 0).all()


@pytest.mark.parametrize("n,q,once", BATCHES)
def test_a_first_row_that_was_released(n, q, once):
    """No query tokens in the step; its seq_lens may still say what it held."""
    a = Batch(n, q, first=0)
    a.table[0] = -1
    a.check(once)


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 16, 16), (128, 16, 8)])
@pytest.mark.parametrize("n,q,once", BATCHES)
def test_first_requests_that_end_within_the_prefix(n, q, once, D, Hq, Hkv):
    """They hold the pages of their own tokens alone."""
    a = Batch(n, q, D=D, Hq=Hq, Hkv=Hkv, prefix=6000 if once else 200)
    for b, kept in ((0, 100), (1, 165))[:n - 1]:
        a.lens[b], a.table[b, -(-kept // 64):] = kept, -1
    a.check(once)


@pytest.mark.parametrize("n,q,once", BATCHES)
def test_no_request_that_reaches_the_end_of_the_prefix(n, q, once):
    """The longest holds what any row sees."""
    a = Batch(n, q)
    for b in range(n):
        a.lens[b] = 1500 + 10 * (b * 7 % n) + (b == n // 2) * 1400
        a.table[b, -(-a.lens[b] // 64):] = -1
    a.check(once)


@pytest.mark.parametrize("idle", [63, 64, 130])
def test_many_idle_rows_first(idle):
    """Rows without pages, of which the first still has a query token."""
    a = Batch(idle + 40, 1)
    a.q_lens = [1] + [0] * (idle - 1) + [1] * 40
    a.start, a.one = np.concatenate([[0], np.cumsum(a.q_lens)]), False
    a.Q = a.Q[:41]
    a.lens[:idle], a.table[:idle] = 0, -1
    a.check(True)


def test_no_request_with_a_key():
    a = Batch(40, 1)
    a.lens[:], a.table[:] = [0, -2] * 20, -1
    O, lse = a.call(a.table, prefix_len=a.prefix)
    assert (O == 0).all() and torch_mod().isneginf(lse).all()


def test_against_the_oracle():
    a = Behind(310, [1] * 34, [311 + i for i in range(34)], 64, 64, 64, 16, True, "bfloat16", seed=2)
    ids, a.kv_lens[0], a.table[0] = a.table[0].copy(), 0, -1
    a.check(prefix_table=ids)


def test_requests_that_end_between_replays():
    """The device's lengths choose the row: a captured call serves when the first requests leave."""
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    a = Batch(40, 1)
    table, lens = _i32(a.table), _i32(a.lens)
    call = lambda **kw: awq.awq_kv_attention(a.Q, a.cache, table, lens, max_query_len=1, max_seq_len=3200,   # noqa: E731
                                             prefix_len=3000, return_lse=True, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = call()
    for gone in range(4):
        if gone:
            a.lens[gone - 1], a.table[gone - 1] = 0, -1
            table.copy_(_i32(a.table)), lens.copy_(_i32(a.lens))
        graph.replay()
        torch.cuda.synchronize()
        want = call(prefix_table=_i32(a.whole[0]))
        assert all(torch.equal(x, y) for x, y in zip(out, want))
        assert all(torch.equal(x, y) for x, y in zip(call(), want))


@pytest.mark.parametrize("n,q,once", BATCHES)
def test_a_first_branch_that_found_no_page(n, q, once):
    """The page that the prefix ends in is -1 in its row, as awq_kv_fork leaves it when none is free: it
    misses those keys, and nobody else does."""
    torch = torch_mod()
    a = Batch(n, q)
    a.table[0, a.prefix // a.page] = -1
    assert a.reads_once() == once
    want = a.call(a.whole, prefix_table=_i32(a.whole[0]), prefix_len=a.prefix) if once else a.call(a.whole)
    got = a.call(a.table, prefix_len=a.prefix)
    assert all(torch.equal(w[q:], g[q:]) for w, g in zip(want, got))


def test_no_branch_found_a_page():
    """The longest that anybody sees is then what comes before it."""
    a = Batch(40, 1)
    a.lens[:] = a.prefix - np.arange(40)
    a.table[:, a.prefix // a.page] = -1
    torch = torch_mod()
    want = a.call(a.table, prefix_table=_i32(a.table[7]), prefix_len=a.prefix)
    assert a.reads_once()
    assert all(torch.equal(w, g) for w, g in zip(want, a.call(a.table, prefix_len=a.prefix)))
