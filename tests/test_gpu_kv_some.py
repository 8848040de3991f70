"""GPU parity of attention over some of the cached keys, a window with sinks and a prefix
that the batch shares, with oracle/kv.py: within the bound that attention64 derives
from the documented arithmetic, each row's keys being what they are by definition."""

import numpy as np
import pytest

from gpu_common import dev, out_to_f64, say, torch_mod
from oracle import kv
from test_gpu_kv import Attend, _i32, _to_cache

pytestmark = pytest.mark.gpu

EPS = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}


def _within(O, lse, want, wl, bound, lse_bound):
    err = np.abs(out_to_f64(O) - want)
    say("worst err / bound", float(np.max(err / np.maximum(bound, 1e-300), initial=0)))
    assert (err <= bound).all()
    got = lse.cpu().numpy().astype(np.float64)
    gone = np.isneginf(wl)
    assert np.array_equal(np.isneginf(got), gone) and (out_to_f64(O)[gone] == 0).all()
    assert (np.abs(got[~gone] - wl[~gone]) <= lse_bound[~gone]).all()


# ---- sinks ----------------------------------------------------------------------------

def _check_sinks(a, window, sinks, scale=None, **kw):
    O, lse = a.run(window=window, sinks=sinks, scale=scale, **kw)
    _within(O, lse, *kv.attention64(a.q64, a.cache, a.table, a.kv_lens, a.start, a.D ** -0.5 if scale is None else scale,
                                    True, window, EPS[a.dtype], sinks=sinks))
    return O


@pytest.mark.parametrize("kv_lens,window,sinks,Hq,Hkv,D,page,zp,dtype", [
    ([1, 5, 40, 0], 3, 1, 4, 4, 64, 16, True, "float16"),
    ([700, 33, 64, 65], 20, 4, 8, 2, 128, 16, True, "bfloat16"),        # a gap of many tiles
    ([300, 301], 32, 32, 8, 8, 64, 32, False, "bfloat16"),              # both end with a tile
    ([300, 301], 33, 33, 2, 1, 128, 64, True, "float16"),               # one past it
    ([100, 64, 95], 50, 64, 4, 1, 64, 16, True, "float16"),             # the window reaches into the sinks
    ([100, 3], 200, 7, 4, 2, 128, 128, False, "float16"),               # every key is in the window
    ([100, 3], 2, 500, 4, 2, 128, 16, True, "float16"),                 # every key is a sink
    ([2600], 1, 3, 6, 1, 64, 1024, True, "bfloat16"),
    ([2500, 1200], 1900, 100, 20, 1, 64, 16, True, "float16"),          # several parts
])
def test_decode_with_sinks(kv_lens, window, sinks, Hq, Hkv, D, page, zp, dtype):
    _check_sinks(Attend([1] * len(kv_lens), kv_lens, Hq, Hkv, D, page, zp, dtype, seed=sum(kv_lens)), window, sinks)


@pytest.mark.parametrize("q_lens,kv_lens,window,sinks,Hq,Hkv,D,page,zp,dtype", [
    ([3, 1, 2], [50, 1, 2], 5, 2, 4, 2, 128, 16, True, "float16"),
    ([4, 3], [4, 900], 7, 4, 8, 8, 64, 32, True, "bfloat16"),
    ([33], [33], 4, 1, 2, 1, 128, 16, True, "float16"),
    ([65, 1, 0, 20], [65, 40, 9, 850], 30, 65, 4, 2, 128, 64, False, "bfloat16"),
    ([70, 200], [700, 200], 50, 16, 4, 4, 64, 16, True, "float16"),
    ([300], [1600], 64, 64, 2, 1, 128, 128, True, "bfloat16"),
    ([300], [1000], 100, 300, 2, 1, 64, 16, False, "float16"),          # sinks over tiles that rows see in part
    ([40, 40], [39, 0], 5, 3, 2, 2, 64, 16, True, "float16"),           # rows before the first key
    ([600], [2200], 1000, 4, 8, 1, 64, 16, True, "float16"),            # parts
])
def test_several_query_tokens_with_sinks(q_lens, kv_lens, window, sinks, Hq, Hkv, D, page, zp, dtype):
    _check_sinks(Attend(q_lens, kv_lens, Hq, Hkv, D, page, zp, dtype, seed=sum(q_lens)), window, sinks)


@pytest.mark.parametrize("n", [1, 40])
def test_sinks_without_a_window_are_nothing(n):
    a = Attend([n, n], [200, 90], 4, 2, 64, 16, True, "float16", seed=5)
    assert torch_mod().equal(a.run(sinks=9)[0], a.run()[0])


@pytest.mark.parametrize("n", [1, 3, 40])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("zp", [True, False])
def test_pages_between_sinks_and_window_may_be_gone(n, D, zp):
    """Released entries, and infinite and NaN steps in the hidden slots of a page that is left.  (Not
    the same bits: a tile's running maximum follows its hidden steps too, within the bound.)"""
    a = Attend([n, n], [500 + n, 380], 4, 2, D, 16, zp, "bfloat16", seed=n)
    window, sinks = 60, 5
    _check_sinks(a, window, sinks)
    for b in range(2):
        lo, hi = -(-sinks // 16), (int(a.kv_lens[b]) - n - window + 1) // 16
        a.table[b, lo:hi] = -1
    _check_sinks(a, window, sinks)
    for b in range(2):                              # a page that the sinks end in: its hidden slots
        pos = np.arange(sinks, 16)
        a.cache[1][a.table[b, 0], :, pos] = np.array([np.nan, np.inf], np.float16)
    _check_sinks(a, window, sinks)


@pytest.mark.parametrize("n", [1, 40])
def test_a_missing_page_among_the_sinks(n):
    a = Attend([n], [400], 2, 1, 64, 16, True, "float16", seed=3)
    a.table[0, 1] = -1
    _check_sinks(a, 30, 50)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("scale", [-0.3, 0.0, 1e6, 1e30])
def test_sinks_and_scales(n, scale):
    _check_sinks(Attend([n, n], [350, 67], 4, 2, 64, 16, True, "bfloat16", seed=20), 40, 4, scale=scale)


# ---- a shared prefix -----------------------------------------------------------------------

class Behind(Attend):
    """A batch whose requests have the first `prefix` tokens in common: full pages shared, the
    page that it ends in a copy of each request's own."""

    def __init__(self, prefix, q_lens, kv_lens, Hq, Hkv, D, page, zp, dtype, seed=0, **kw):
        super().__init__(q_lens, kv_lens, Hq, Hkv, D, page, zp, dtype, seed, **kw)
        self.prefix = prefix
        codes, scales, zeros = self.cache
        src = self.table[0]
        same, rest = prefix // page, prefix % page
        for b in range(1, len(q_lens)):
            if self.kv_lens[b] <= 0:
                continue
            self.table[b, :same] = src[:same]
            if rest and self.kv_lens[b] > same * page:
                pos = np.arange(rest)
                words = np.arange(D // 8)
                for k in range(2):
                    for off in pos:
                        at = kv._word_index(k, int(off), words, D)
                        codes[self.table[b, same], k][:, at] = codes[src[same], k][:, at]
                scales[self.table[b, same]][:, pos] = scales[src[same]][:, pos]
                if zeros is not None:
                    zeros[self.table[b, same]][:, pos] = zeros[src[same]][:, pos]

    def check(self, causal=True, scale=None, table=None, prefix_table=None, whole=True):
        """Read once, from a table of its own, and (`whole`) as the rows' own entries have it."""
        want = kv.attention64(self.q64, self.cache, self.table if table is None else table, self.kv_lens, self.start,
                              self.D ** -0.5 if scale is None else scale, causal, 0, EPS[self.dtype])
        kw = dict(causal=causal, scale=scale, prefix_len=self.prefix)
        ids = self.table[0] if prefix_table is None else prefix_table
        _within(*self.run(prefix_table=_i32(ids), **kw), *want)
        if whole:
            _within(*self.run(**kw), *want)


@pytest.mark.parametrize("prefix,kv_lens,Hq,Hkv,D,page,zp,dtype", [
    (1, [2], 1, 1, 64, 16, True, "float16"),
    (16, [17, 40, 18], 4, 4, 128, 16, True, "bfloat16"),
    (33, [34, 64, 90, 0], 8, 2, 64, 32, False, "bfloat16"),             # a padded batch
    (100, [101, 350], 7, 1, 128, 64, True, "float16"),
    (130, [131] * 20, 4, 2, 64, 16, True, "float16"),                   # rows of many requests in a tile
    (64, [65 + 7 * i for i in range(40)], 2, 1, 128, 16, True, "bfloat16"),
    (1500, [1501, 1700, 0, 1600], 16, 2, 64, 128, False, "float16"),
    (700, [701 + i for i in range(9)], 40, 8, 64, 1024, True, "float16"),
    (2100, [2200] * 3, 36, 1, 64, 16, True, "bfloat16"),
])
def test_decode_behind_a_prefix(prefix, kv_lens, Hq, Hkv, D, page, zp, dtype):
    Behind(prefix, [1] * len(kv_lens), kv_lens, Hq, Hkv, D, page, zp, dtype, seed=prefix).check()


@pytest.mark.parametrize("prefix,q_lens,kv_lens,Hq,Hkv,D,page,zp,dtype,causal", [
    (40, [3, 1, 2], [50, 41, 42], 4, 2, 128, 16, True, "float16", True),
    (64, [4, 4, 1], [68, 90, 0], 8, 8, 64, 32, True, "bfloat16", True),
    (50, [33, 0, 5], [83, 60, 55], 2, 1, 128, 16, True, "float16", True),
    (200, [65, 1, 0, 20], [265, 240, 209, 350], 4, 2, 128, 64, False, "bfloat16", True),
    (90, [70, 30], [200, 120], 4, 4, 64, 16, True, "float16", False),
    (600, [129, 4], [800, 610], 3, 1, 64, 64, True, "bfloat16", True),
    (1100, [200], [1300], 2, 2, 128, 128, False, "float16", True),
])
def test_several_query_tokens_behind_a_prefix(prefix, q_lens, kv_lens, Hq, Hkv, D, page, zp, dtype, causal):
    Behind(prefix, q_lens, kv_lens, Hq, Hkv, D, page, zp, dtype, seed=sum(q_lens)).check(causal)


@pytest.mark.parametrize("n", [1, 5])
def test_requests_that_end_within_the_prefix(n):
    """Their rows see what their lengths say; those without any key get zeros, whatever the queries hold."""
    a = Behind(100, [n] * 5, [120 + n, 100, 60, n - 1, -3], 4, 2, 64, 16, True, "float16", seed=n)
    t = a.Q.clone()
    t[a.start[4]:] = float("nan")
    a.Q = t
    a.q64[a.start[4]:] = 0
    a.check()


@pytest.mark.parametrize("n", [1, 40])
def test_own_prefix_table(n):
    """The rows' own entries of the prefix' full pages do not matter."""
    a = Behind(80, [n, n], [130, 121], 4, 2, 128, 16, True, "bfloat16", seed=8)
    full = a.table.copy()
    a.table[:, :80 // 16] = [[-1], [2 ** 31 - 1]]
    ids = np.concatenate([full[0, :5], [-1, 7]])
    a.check(table=full, prefix_table=ids, whole=False)


@pytest.mark.parametrize("n", [1, 40])
def test_a_missing_page_of_the_prefix(n):
    a = Behind(96, [n, n], [150, 99 + n], 4, 2, 64, 16, True, "float16", seed=9)
    a.table[:, 2], a.table[0, 4], a.table[1, 4] = -1, -7, -7
    a.check()


def test_where_it_pays_the_first_row_is_read():
    """Enough requests behind a prefix long enough: the other rows' entries do not matter then."""
    a = Behind(3000, [1] * 40, [3001 + 3 * i for i in range(40)], 8, 8, 128, 64, True, "float16", seed=6)
    full = a.table.copy()
    a.check()
    a.table[1:, :3000 // 64] = -1
    a.check(table=full)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("spread,size,scale", [(20.0, 1.0, None), (1.0, 1.0, 2.0), (1.0, 1.0, -0.3), (1.0, 1.0, 0.0),
                                               (1.0, 1e-4, None), (1.0, 1e4, 1e6), (1.0, 1.0, 1e30)])
def test_prefix_with_steps_and_logits_of_many_sizes(n, spread, size, scale):
    Behind(150, [n, n], [220, 333], 4, 2, 64, 16, True, "bfloat16", seed=7, spread=spread, size=size).check(scale=scale)


def test_rows_of_no_request_are_left_alone():
    """Tokens before query_start[0], behind the last, and of a request beyond max_query_len."""
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    a = Behind(40, [2, 5], [60, 70], 4, 2, 64, 16, True, "float16", seed=3)
    Q = torch.randn((16, 4, 64), device=dev()).half()
    Q[3:10] = a.Q
    out = torch.full_like(Q, 7.0)
    cache = _to_cache(a.cache)
    row = _i32(a.table[0])
    awq.awq_kv_attention(Q, cache, _i32(a.table), _i32(a.kv_lens), query_start=_i32([3, 5, 10]), max_query_len=3,
                         out=out, prefix_len=40, prefix_table=row)
    full, _ = a.run(prefix_len=40, prefix_table=row)
    assert (out[:3] == 7).all() and (out[8:] == 7).all()
    # (split otherwise: equal up to rounding)
    assert (out[3:8].float() - full[:5].float()).abs().max().item() <= 2.0 ** -9 * float(full.abs().max())


def test_no_request_and_no_token():
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    cache = awq.empty_kv_cache(2, 1, 64, 16, dev())
    q = torch.empty((0, 2, 64), dtype=torch.float16, device=dev())
    assert awq.awq_kv_attention(q, cache, _i32(np.zeros((0, 3))), _i32([]), prefix_len=20).shape == q.shape
    assert awq.awq_kv_attention(q, cache, _i32(np.zeros((0, 3))), _i32([]), window=3, sinks=2).shape == q.shape


@pytest.mark.parametrize("kind", ["sinks", "prefix"])
@pytest.mark.parametrize("n", [1, 40])
def test_calls_repeat_and_do_not_depend_on_the_workspace(n, kind):
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    a = Behind(700, [n, n], [2400, 2300], 8, 1, 64, 16, True, "float16", seed=13)
    kw = dict(window=1900, sinks=70) if kind == "sinks" else dict(prefix_len=700)
    table = {} if kind == "sinks" else dict(prefix_table=_i32(a.table[0]))
    cache = _to_cache(a.cache)
    args = (a.Q, cache, _i32(a.table), _i32(a.kv_lens))
    more = dict(query_start=_i32(a.start), max_query_len=n, max_seq_len=2400, return_lse=True, **kw, **table)
    want = awq.awq_kv_attention(*args, **more)
    need = awq.awq_kv_attention_workspace_size(2 * n, 2, 8, cache, n, 2400, **kw)
    assert need > 0
    for fill in (0, 255):
        ws = torch.full((need,), fill, dtype=torch.uint8, device=dev())
        got = awq.awq_kv_attention(*args, workspace=ws, **more)
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    with pytest.raises(awq.AwqError, match="workspace"):
        awq.awq_kv_attention(*args, workspace=None, **more)


def test_branches_of_one_prompt_end_to_end_captured():
    """A prompt's tokens are rotated into the cache once, branches forked from it, and each step
    appends a token to every branch and attends behind the shared prompt, and through a window with sinks
    whose middle pages are given back: one graph per step, replayed, equal to the eager calls and
    to attention without the prefix."""
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    Hq, Hkv, D, page, n, L = 8, 2, 64, 16, 5, 75
    g = torch.Generator(device=dev()).manual_seed(1)
    rnd = lambda T, h: torch.randn((T, h, D), generator=g, device=dev()).half()  # noqa: E731
    inv, factor = awq.awq_rope_frequencies(D, scaling="yarn", factor=4.0, original_len=64, device=dev())
    cache = awq.empty_kv_cache(64, Hkv, D, page, dev())
    for c in cache:
        c.zero_()
    table = torch.full((n + 1, 10), -1, dtype=torch.int32, device=dev())
    shared, free = torch.zeros(64, dtype=torch.int32, device=dev()), torch.arange(64, dtype=torch.int32, device=dev())
    rows = lambda v: _i32([v] + [0] * n)           # noqa: E731
    _, _, slots, used = awq.awq_kv_assign(rows(0), rows(L), table, free, page, L)
    awq.awq_kv_append_rope(rnd(L, Hkv), rnd(L, Hkv), cache, slots, torch.arange(L, dtype=torch.int32, device=dev()), inv,
                           attention_factor=factor)
    used = awq.awq_kv_fork(cache, table, _i32([0] * n), _i32(range(1, n + 1)), _i32([L] * n), shared, free, taken=used)
    free, count = awq.awq_kv_release(table, rows(0), shared, free, page, pages_used=used)
    assert count.item() == 64 - 5 - n and shared.tolist().count(n) == L // page
    lens, ones = _i32([0] + [L] * n), _i32([0] + [1] * n)
    q, k, v = rnd(n, Hq), rnd(n, Hkv), rnd(n, Hkv)

    def step(q, k, v, lens, free):
        new, start, slots, used = awq.awq_kv_assign(lens, ones, table, free, page, n)
        qr = awq.awq_kv_append_rope(k, v, cache, slots, lens[1:], inv, Q=q, attention_factor=factor)
        args = dict(query_start=start, max_query_len=1, max_seq_len=160)
        a = awq.awq_kv_attention(qr, cache, table, new, prefix_len=L, prefix_table=table[1], **args)
        b = awq.awq_kv_attention(qr, cache, table, new, window=20, sinks=4, **args)
        left, _ = awq.awq_kv_release(table[:1], lens[:1], shared, free, page, pages_used=used)
        return new, a, b, left, qr

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(q, k, v, lens.clone(), free.clone())
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(q, k, v, lens, free)
    for i in range(20):
        q.copy_(rnd(n, Hq)), k.copy_(rnd(n, Hkv)), v.copy_(rnd(n, Hkv))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        args = dict(query_start=_i32([0, 0, 1, 2, 3, 4, 5]), max_query_len=1, max_seq_len=160)
        whole = awq.awq_kv_attention(got[4], cache, table, got[0], **args)
        behind = awq.awq_kv_attention(got[4], cache, table, got[0], prefix_len=L, prefix_table=table[1], **args)
        near = awq.awq_kv_attention(got[4], cache, table, got[0], window=20, sinks=4, **args)
        assert torch.equal(got[1], behind) and torch.equal(got[2], near)
        # two ways of splitting one softmax: two roundings to fp16 of weights and outputs each
        assert (behind.float() - whole.float()).abs().max().item() <= 2.0 ** -8 * float(whole.abs().max())
        lens.copy_(got[0]), free.copy_(got[3])
    assert lens.tolist() == [0] + [L + 20] * n
    # the middle of every branch is given back: what the window needs is still there
    first, last = _i32([0] + [4] * n), _i32([0] + [L + 20 - 20] * n)
    awq.awq_kv_release(table, lens, shared, free, page, start=first, end=last)
    assert (table[1:, 1:4] == -1).all() and (table[1:, 0] >= 0).all()
    assert torch.equal(awq.awq_kv_attention(got[4], cache, table, lens, window=20, sinks=4, **args), near)


@pytest.mark.parametrize("n", [1, 40])
def test_two_calls_at_once_on_two_streams(n):
    """Each with a workspace of its own, captured and replayed side by side."""
    torch = torch_mod()
    import bit_weight_only_quantize_amd as awq
    cases = [(Behind(300, [n] * 3, [900, 700, 0], 8, 2, 64, 16, True, "float16", seed=s),
              dict(prefix_len=300) if s else dict(window=200, sinks=40)) for s in (0, 1)]
    cases[1][1]["prefix_table"] = _i32(cases[1][0].table[0])
    calls, wants = [], []
    for a, kw in cases:
        args = (a.Q, _to_cache(a.cache), _i32(a.table), _i32(a.kv_lens))
        more = dict(query_start=_i32(a.start), max_query_len=n, max_seq_len=900, **kw)
        calls.append((args, more))
        wants.append(awq.awq_kv_attention(*args, **more).clone())
    torch.cuda.synchronize()
    streams, graphs, outs = [torch.cuda.Stream() for _ in calls], [], []
    for (args, more), st in zip(calls, streams):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=st):
            outs.append(awq.awq_kv_attention(*args, **more))
        graphs.append(gr)
    for _ in range(5):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for gr, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                gr.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, w) for o, w in zip(outs, wants))
