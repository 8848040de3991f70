"""GPU parity of the 4-bit key/value cache (awq_kv_*) with oracle/kv.py: pages
and slots and the cache's bits exactly, attention within the bound that
attention64 derives from the documented arithmetic."""

import numpy as np
import pytest

from gpu_common import dev, out_to_f64, say, to_dev, torch_mod
from oracle import kv

pytestmark = pytest.mark.gpu


def _to_cache(cache):
    torch = torch_mod()
    codes, scales, zeros = cache
    return (to_dev(codes), torch.from_numpy(scales.view(np.int16)).to(dev()).view(torch.float16),
            None if zeros is None else to_dev(zeros))


def _same_cache(got, want):
    torch = torch_mod()
    assert np.array_equal(got[0].cpu().numpy().view(np.uint32), want[0])
    assert np.array_equal(got[1].view(torch.int16).cpu().numpy(), want[1].view(np.int16))
    assert want[2] is None or np.array_equal(got[2].cpu().numpy(), want[2])


def _rounded(x, dtype):
    """x as a GPU tensor of dtype, and its values in fp32."""
    torch = torch_mod()
    t = torch.from_numpy(np.asarray(x, np.float32)).to(getattr(torch, dtype))
    return t.to(dev()), t.float().numpy()


def _i32(a):
    return torch_mod().tensor(np.asarray(a, np.int32), device=dev())


# ---- pages and slots -------------------------------------------------------------

def _assign_case(old, new, blocks, num_free, page, num_slots, seed=0):
    rng = np.random.default_rng(seed)
    B = len(old)
    have = [-(-max(0, o) // page) for o in old]
    ids = rng.permutation(sum(have) + num_free).astype(np.int32)
    table = np.full((B, blocks), -1, np.int32)
    at = 0
    for b, h in enumerate(have):
        n = min(h, blocks)
        table[b, :n] = ids[at:at + n]
        at += h
    return table, ids[at:at + num_free].copy()


@pytest.mark.parametrize("name,old,new,blocks,free,page,pad", [
    ("one", [0], [1], 1, 1, 16, 0),
    ("none", [], [], 3, 2, 16, 5),
    ("nothing new", [5, 16, 0], [0, 0, 0], 2, 4, 16, 2),
    ("page ends", [15, 16, 17, 31, 0], [1, 1, 1, 2, 16], 4, 9, 16, 3),
    ("negative", [-3, 4, 7], [5, -2, 1], 3, 4, 16, 1),
    ("free list runs out", [0, 10, 3], [40, 30, 64], 6, 4, 16, 0),
    ("table too narrow", [20, 0], [40, 70], 3, 20, 16, 4),
    ("large pages", [1000, 2047, 5], [1, 2, 3000], 9, 9, 1024, 0),
])
def test_assign(name, old, new, blocks, free, page, pad):
    import bit_weight_only_quantize_amd as awq
    say("assign", name)
    n = sum(max(0, x) for x in new) + pad
    table, pages = _assign_case(old, new, blocks, free, page, n)
    want = kv.assign(old, new, table, pages, page, n)
    tab = _i32(table)
    got = awq.awq_kv_assign(_i32(old), _i32(new), tab, _i32(pages), page, n)
    for g, w in zip((tab,) + got, want):
        assert np.array_equal(g.cpu().numpy().reshape(w.shape), w)


@pytest.mark.parametrize("B,most,page", [(37, 90, 16), (1024, 6, 32), (1025, 9, 16), (3001, 30, 16), (5000, 1, 64)])
def test_assign_many_requests(B, most, page):
    """More requests than a workgroup scans at once, more tokens than one serves."""
    import bit_weight_only_quantize_amd as awq
    rng = np.random.default_rng(B)
    old = rng.integers(0, 200, B)
    new = rng.integers(0, most + 1, B)
    new[rng.random(B) < 0.3] = 0
    n = int(new.sum()) + 17
    blocks = int(max(-(-(o + m) // page) for o, m in zip(old, new))) + 1
    table, pages = _assign_case(old, new, blocks, int(new.sum()) + 5, page, n, B)
    want = kv.assign(old, new, table, pages, page, n)
    for _ in range(2):                              # the same call again changes nothing
        tab = _i32(table)
        got = awq.awq_kv_assign(_i32(old), _i32(new), tab, _i32(pages), page, n)
        for g, w in zip((tab,) + got, want):
            assert np.array_equal(g.cpu().numpy().reshape(w.shape), w)


def test_assign_fewer_slots_than_tokens():
    import bit_weight_only_quantize_amd as awq
    old, new, page = [3, 0, 30], [20, 5, 40], 16
    table, pages = _assign_case(old, new, 6, 12, page, 30)
    want = kv.assign(old, new, table, pages, page, 30)
    tab = _i32(table)
    got = awq.awq_kv_assign(_i32(old), _i32(new), tab, _i32(pages), page, 30)
    for g, w in zip((tab,) + got, want):
        assert np.array_equal(g.cpu().numpy().reshape(w.shape), w)


# ---- append and gather --------------------------------------------------------------

@pytest.mark.parametrize("T,heads,D,page,zp,dtype", [
    (1, 1, 64, 16, True, "float16"), (5, 3, 128, 16, True, "bfloat16"),
    (67, 2, 64, 32, False, "bfloat16"), (130, 8, 128, 64, True, "float16"),
    (33, 5, 128, 128, False, "float16"), (250, 1, 64, 1024, True, "float16"),
])
def test_append_and_gather(T, heads, D, page, zp, dtype):
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    say("append", T, heads, D, page, zp, dtype)
    rng = np.random.default_rng(T)
    pages = -(-T // page) + 2
    cache = kv.new_cache(pages, heads, D, page, zp, rng)
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    slots[rng.random(T) < 0.1] = -1
    if T > 4:
        slots[2], slots[3] = pages * page, 2 ** 31 - 1     # past the cache: skipped
    x = rng.normal(0.2, 1.5, (2, T, heads, D)) * np.exp(rng.normal(0, 1, (2, T, heads, 1)))
    x[:, 0] = 0.0                                          # an empty range
    if T > 1:
        x[:, 1] = np.abs(x[:, 1])                          # zero point 0
    (K, k32), (V, v32) = _rounded(x[0], dtype), _rounded(x[1], dtype)
    got = _to_cache(cache)
    count = torch.zeros(1, dtype=torch.int32, device=dev())
    awq.awq_kv_append(K, V, got, _i32(slots), nonfinite_count=count)
    kv.append(cache, k32, v32, slots)
    _same_cache(got, cache)
    assert count.item() == 0
    inside = (slots >= 0) & (slots < pages * page)
    _, _, _, val = kv.read(cache, D, np.where(inside, slots, 0))
    val = np.where(inside[None, :, None, None], val, 0.0)
    for odt in (torch.float32, torch.float16, torch.bfloat16):
        gk, gv = awq.awq_kv_gather(got, _i32(slots), out_dtype=odt)
        for g, w in ((gk, val[0]), (gv, val[1])):
            w = torch.from_numpy(w.astype(np.float32)).to(odt)   # exact in fp32: 5 bits times 11
            assert torch.equal(g.cpu(), w)


def test_append_strided_tokens_and_nonfinite_count():
    """K and V as slices of one fused output; non-finite values are counted,
    skipped tokens are not, other tokens keep their codes."""
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    rng = np.random.default_rng(5)
    T, Hq, H, D, page = 9, 4, 2, 64, 16
    qkv, q32 = _rounded(rng.normal(size=(T, (Hq + 2 * H) * D)), "float16")
    qkv[4, Hq * D + 3] = float("nan")
    qkv[4, Hq * D + H * D + 70] = float("inf")
    qkv[6, Hq * D + 1] = float("inf")                       # this token is skipped
    K = qkv[:, Hq * D:(Hq + H) * D].unflatten(1, (H, D))
    V = qkv[:, (Hq + H) * D:].unflatten(1, (H, D))
    slots = np.arange(T, dtype=np.int32) * 2
    slots[6] = -1
    cache = kv.new_cache(2, H, D, page, True, rng)
    got = _to_cache(cache)
    count = torch.full((1,), 10, dtype=torch.int32, device=dev())
    awq.awq_kv_append(K, V, got, _i32(slots), nonfinite_count=count)
    assert count.item() == 12
    fine = [t for t in range(T) if t not in (4, 6)]
    kv.append(cache, q32[fine, Hq * D:(Hq + H) * D].reshape(-1, H, D),
              q32[fine, (Hq + H) * D:].reshape(-1, H, D), slots[fine])
    _, _, _, val = kv.read(cache, D, slots[fine])
    gk, gv = awq.awq_kv_gather(got, _i32(slots[fine]), out_dtype=torch.float32)
    assert np.array_equal(gk.cpu().numpy(), val[0].astype(np.float32))
    assert np.array_equal(gv.cpu().numpy(), val[1].astype(np.float32))


def test_slots_past_32_bit_byte_offsets():
    """A cache of more than 4 GiB of codes: the last slots land where they belong."""
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    H, D, page = 8, 128, 64
    pages = 72 * 1024                                       # 4.5 GiB of codes
    codes, scales, zeros = awq.empty_kv_cache(pages, H, D, page, dev())
    rng = np.random.default_rng(8)
    T = 40
    slots = np.concatenate([np.arange(pages * page - T + 4, pages * page), [0, 1, 2, 3]]).astype(np.int32)
    (K, k32), (V, v32) = _rounded(rng.normal(size=(T, H, D)), "float16"), _rounded(rng.normal(size=(T, H, D)), "float16")
    awq.awq_kv_append(K, V, (codes, scales, zeros), _i32(slots))
    small = kv.new_cache(1, H, D, page)
    kv.append(small, k32, v32, np.concatenate([np.arange(page - T + 4, page), [0, 1, 2, 3]]))
    _, _, _, val = kv.read(small, D, np.concatenate([np.arange(page - T + 4, page), [0, 1, 2, 3]]))
    gk, gv = awq.awq_kv_gather((codes, scales, zeros), _i32(slots), out_dtype=torch.float32)
    assert np.array_equal(gk.cpu().numpy(), val[0].astype(np.float32))
    assert np.array_equal(gv.cpu().numpy(), val[1].astype(np.float32))
    for nq in (1, 36):                                      # both attention kernels
        Q, q32 = _rounded(rng.normal(size=(nq, H, D)), "float16")
        table = np.array([[pages - 1]], np.int32)
        # the request's tokens are the last page's; those before slot 28 of it were never written
        ref = kv.new_cache(1, H, D, page)
        kv.append(ref, k32[:-4], v32[:-4], np.arange(page - T + 4, page))
        got = awq.awq_kv_attention(Q, (codes, scales, zeros), _i32(table), _i32([page]),
                                   query_start=_i32([0, nq]), max_query_len=nq, window=1)
        want, _, bound, _ = kv.attention64(q32.astype(np.float64), ref, np.array([[0]], np.int32), [page],
                                        [0, nq], D ** -0.5, True, 1)
        assert (np.abs(out_to_f64(got) - want) <= bound).all()


# ---- attention -----------------------------------------------------------------------

class Attend:
    """A batch of requests over a filled cache, on both sides."""

    def __init__(self, q_lens, kv_lens, Hq, Hkv, D, page, zp, dtype, seed=0, spread=1.0, size=1.0,
                 extra_blocks=1):
        rng = self.rng = np.random.default_rng(seed)
        self.D, self.page, self.dtype = D, page, dtype
        self.kv_lens, self.q_lens = np.asarray(kv_lens), np.asarray(q_lens)
        need = [-(-max(0, n) // page) for n in kv_lens]
        pages = sum(need) + 3
        self.cache = kv.new_cache(pages, Hkv, D, page, zp, rng)      # arbitrary bits, NaN and inf steps too
        ids = rng.permutation(pages).astype(np.int32)
        self.table = np.full((len(need), max(need + [1]) + extra_blocks), -1, np.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = ids[at:at + n]
            at += n
            if kv_lens[b] > 0:
                pos = np.arange(kv_lens[b])
                x = rng.normal(0, 1, (2, kv_lens[b], Hkv, D)) + rng.normal(0, 0.5, (2, 1, Hkv, D))
                x[1] *= size * spread ** rng.normal(0, 1, (kv_lens[b], Hkv, 1))
                kv.append(self.cache, x[0], x[1], self.table[b, pos // page] * page + pos % page)
        self.start = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        self.Q, q32 = _rounded(rng.normal(0, 1, (int(self.start[-1]), Hq, D)), dtype)
        self.q64 = q32.astype(np.float64)

    def run(self, **kw):
        import bit_weight_only_quantize_amd as awq
        one = (self.q_lens == 1).all()
        return awq.awq_kv_attention(self.Q, _to_cache(self.cache), _i32(self.table), _i32(self.kv_lens),
                                    query_start=None if one else _i32(self.start),
                                    max_query_len=int(self.q_lens.max()), max_seq_len=int(max(self.kv_lens)),
                                    return_lse=True, **kw)

    def check(self, causal=True, window=0, scale=None, **kw):
        O, lse = self.run(causal=causal, window=window, scale=scale, **kw)
        eps = 2.0 ** -11 if self.dtype == "float16" else 2.0 ** -8
        want, wl, bound, lse_bound = kv.attention64(self.q64, self.cache, self.table, self.kv_lens, self.start,
                                         self.D ** -0.5 if scale is None else scale, causal, window, eps)
        got = out_to_f64(O)
        # fp16 holds up to 65504: from 65520 on (half a step of 32 further) a value rounds to infinity
        over = (np.abs(want) + bound >= 65520) & np.isinf(got) & (got * want > 0) & (self.dtype == "float16")
        err = np.abs(np.where(over, want, got) - want)
        say("attention", self.q_lens.tolist()[:4], self.kv_lens.tolist()[:4], "worst err / bound",
            float(np.max(err / np.maximum(bound, 1e-300), initial=0)))
        assert (err <= bound).all()
        got = lse.cpu().numpy().astype(np.float64)
        gone = np.isneginf(wl)
        assert np.array_equal(np.isneginf(got), gone) and (out_to_f64(O)[gone] == 0).all()
        assert (np.abs(got[~gone] - wl[~gone]) <= lse_bound[~gone]).all()
        return O, lse


@pytest.mark.parametrize("kv_lens,Hq,Hkv,D,page,zp,dtype", [
    ([1], 1, 1, 64, 16, True, "float16"),
    ([1, 16, 17, 31, 33], 4, 4, 128, 16, True, "float16"),
    ([40, 0, 64, 65], 8, 2, 64, 32, False, "bfloat16"),
    ([127, 300], 8, 1, 128, 64, True, "bfloat16"),
    ([513, 5], 10, 2, 128, 128, False, "float16"),
    ([1500], 7, 1, 64, 16, True, "float16"),
    ([1100], 16, 2, 128, 16, True, "bfloat16"),
    ([200], 40, 2, 64, 1024, True, "float16"),            # 20 query heads share a key/value head
    ([70, 3], 36, 1, 128, 16, True, "float16"),           # 36: as many rows as a short prompt
])
def test_decode(kv_lens, Hq, Hkv, D, page, zp, dtype):
    Attend([1] * len(kv_lens), kv_lens, Hq, Hkv, D, page, zp, dtype, seed=len(kv_lens) + Hq).check()


@pytest.mark.parametrize("q_lens,kv_lens,Hq,Hkv,D,page,zp,dtype,causal,window", [
    ([3, 1, 2], [50, 1, 2], 4, 2, 128, 16, True, "float16", True, 0),
    ([4, 4], [4, 90], 8, 8, 64, 32, True, "bfloat16", True, 7),
    ([33], [33], 2, 1, 128, 16, True, "float16", True, 0),
    ([65, 1, 0, 20], [65, 40, 9, 150], 4, 2, 128, 64, False, "bfloat16", True, 0),
    ([70], [200], 4, 4, 64, 16, True, "float16", True, 50),
    ([129], [130], 3, 1, 64, 64, True, "bfloat16", True, 0),
    ([40, 50], [70, 64], 2, 2, 128, 32, True, "float16", False, 0),
    ([200], [260], 2, 1, 128, 128, False, "float16", True, 33),
    ([34], [700], 1, 1, 128, 16, True, "float16", True, 0),
])
def test_several_query_tokens(q_lens, kv_lens, Hq, Hkv, D, page, zp, dtype, causal, window):
    Attend(q_lens, kv_lens, Hq, Hkv, D, page, zp, dtype, seed=sum(q_lens)).check(causal, window)


@pytest.mark.parametrize("n", [2, 40])
def test_rows_that_see_no_key(n):
    """More query tokens than cached ones, cut lengths, requests without any:
    zero output and -inf, whatever the queries hold; negative lengths count as 0."""
    a = Attend([n, n, 1, n], [n - 1, 0, -5, n + 3], 4, 2, 64, 16, True, "float16", seed=2)
    t = a.Q.clone()
    t[a.start[1]:a.start[3]] = float("nan")
    a.Q = t
    a.check()


@pytest.mark.parametrize("n", [1, 48])
def test_entries_outside_the_cache_hold_no_tokens(n):
    a = Attend([n, n], [90, 75], 4, 2, 128, 16, True, "float16", seed=4)
    a.table[0, 1], a.table[0, 3], a.table[1, 0] = -1, 2 ** 31 - 1, len(a.cache[0])
    a.check()
    a.table[1, :] = -7
    a.check()


@pytest.mark.parametrize("n", [1, 3, 40])
def test_lengths_beyond_the_table_are_cut(n):
    a = Attend([n], [64], 2, 2, 64, 16, True, "float16", seed=6, extra_blocks=0)
    want, _ = a.run()
    a.kv_lens = np.array([1000])
    a.table = a.table[:, :4]
    got, _ = a.run()                                      # (its keys may be split differently)
    assert (got.float() - want.float()).abs().max().item() <= 2.0 ** -9 * float(want.abs().max())


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("spread,size,scale", [(20.0, 1.0, None), (1.0, 1.0, 2.0), (1.0, 1.0, -0.3),
                                               (1.0, 1.0, 0.0), (1.0, 1e-4, None), (1.0, 1e4, None)])
def test_steps_and_logits_of_many_sizes(n, spread, size, scale):
    """Value steps over orders of magnitude in one request, all tiny or all
    large; near one-hot and flat softmax, a negative scale."""
    Attend([n, n], [150, 333], 4, 2, 128, 16, True, "float16", seed=7, spread=spread,
           size=size).check(scale=scale)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("scale", [1e4, 1e6, 3e7, 2e8, 1e9, 1e12, 1e30])
def test_logits_past_the_fractions_of_fp32(n, dtype, scale):
    """Up to 1e33: one key takes all, or several whose logits fp32 cannot tell
    apart; nothing overflows."""
    for size in (1.0, 1e-4, 1e4):
        Attend([n, n], [150, 67], 4, 2, 64, 16, True, dtype, seed=20, size=size).check(scale=scale)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("gain", [1e-30, 1e5, 1e30])
def test_bfloat16_queries_outside_fp16(n, gain):
    a = Attend([n], [100], 4, 2, 64, 16, True, "bfloat16", seed=9)
    a.Q = (a.Q.float() * gain).to(a.Q.dtype)
    a.q64 = out_to_f64(a.Q)
    a.check(scale=0.125 / gain if gain > 1 else 0.125)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("gain,scale", [(2.0 ** 120, 2.0 ** -123), (2.0 ** 120, 2.0 ** -80), (2.0 ** -110, 2.0 ** 108),
                                        (2.0 ** -20, 2.0 ** 17), (1.0, 2.0 ** -126)])
def test_queries_and_scales_at_the_ends_of_their_range(n, gain, scale):
    a = Attend([n], [100], 4, 2, 64, 16, True, "bfloat16", seed=21)
    a.Q = (a.Q.float() * gain).to(a.Q.dtype)
    a.q64 = out_to_f64(a.Q)
    a.check(scale=scale)
    a.check(scale=-scale)


@pytest.mark.parametrize("n", [1, 40])
def test_nonfinite_keys_and_values_stay_with_those_who_see_them(n):
    """Tokens outside the window with infinite keys and values, and NaN queries
    of another request."""
    import bit_weight_only_quantize_amd as awq
    a = Attend([n, n], [96 + n, 96 + n], 4, 2, 64, 16, True, "float16", seed=11)
    W = 20
    want, _ = a.run(window=W)
    codes, scales, zeros = a.cache
    pos = np.arange(70)                                   # below every row's window
    for b in range(2):
        s = a.table[b, pos // 16]
        scales[s, :, pos % 16] = np.array([np.inf, np.inf], np.float16)
    got, _ = a.run(window=W)
    # the hidden steps no longer count for the running maximum's exponent: equal up to rounding
    eps = 2.0 ** -9 * float(want.abs().max())
    assert (got.float() - want.float()).abs().max().item() <= eps
    a.Q[:a.start[1]] = float("nan")
    got, _ = a.run(window=W)
    assert (got[a.start[1]:].float() - want[a.start[1]:].float()).abs().max().item() <= eps
    assert torch_mod().isnan(got[:a.start[1]]).all()


@pytest.mark.parametrize("n", [2, 40])
def test_infinite_values_of_keys_behind_a_row(n):
    """Causal rows before a token with an infinite step do not see it; the
    last row does."""
    torch = torch_mod()
    a = Attend([n], [60 + n], 2, 2, 64, 16, True, "float16", seed=12)
    want, _ = a.run()
    last = 60 + n - 1
    a.cache[1][a.table[0, last // 16], :, last % 16, 1] = np.float16(np.inf)
    got, _ = a.run()
    # another step in the tile may move the running maximum's exponent: equal up to rounding
    eps = 2.0 ** -9 * float(want.abs().max())
    assert (got[:-1].float() - want[:-1].float()).abs().max().item() <= eps
    assert not torch.isfinite(got[-1].float()).any()


@pytest.mark.parametrize("n", [3, 40])
def test_largest_window(n):
    """A window of 2^31 - 1 is none, also where the first rows see no key."""
    a = Attend([n, n], [n - 2, n + 9], 4, 2, 64, 16, True, "float16", seed=17)
    want, _ = a.check(window=0)
    got, _ = a.check(window=2 ** 31 - 1)
    assert torch_mod().equal(got, want)


@pytest.mark.parametrize("n", [3, 40])
@pytest.mark.parametrize("step", [60000.0, 0.25])
def test_large_steps_behind_a_row(n, step):
    """Values with steps near 1e-5, the last token's many orders larger: rows
    that do not see it keep their precision."""
    a = Attend([n, n], [60 + n, 64], 4, 2, 64, 16, True, "float16", seed=18, size=1e-4)
    for b in range(2):
        last = int(a.kv_lens[b]) - 1
        a.cache[1][a.table[b, last // 16], :, last % 16, 1] = np.float16(step)
    a.check()
    a.check(window=5)


@pytest.mark.parametrize("n", [3, 40])
@pytest.mark.parametrize("dtype,large,small", [("float16", 1e4, 1e-4), ("bfloat16", 1e20, 1e-10)])
def test_queries_of_many_sizes_in_one_request(n, dtype, large, small):
    """Rows whose queries differ by orders of magnitude keep their own precision."""
    torch = torch_mod()
    a = Attend([n], [60 + n], 4, 2, 64, 16, True, dtype, seed=19)
    gain = np.where(np.arange(n) % 2 == 0, large, small)
    a.Q = (a.Q.float() * torch.tensor(gain, dtype=torch.float32, device=dev())[:, None, None]).to(a.Q.dtype)
    a.q64 = out_to_f64(a.Q)
    a.check(scale=0.125 / small)


def test_rows_of_no_request_are_left_alone():
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    for n in (3, 40):
        a = Attend([n, n], [50, 80], 4, 2, 64, 16, True, "float16", seed=13)
        Q = torch.cat([a.Q[:5] * float("nan"), a.Q, a.Q[:7] * float("nan")])
        out = torch.full_like(Q, 7.0)
        awq.awq_kv_attention(Q, _to_cache(a.cache), _i32(a.table), _i32(a.kv_lens),
                             query_start=_i32(a.start + 5), max_query_len=n, out=out)
        assert (out[:5] == 7).all() and (out[5 + 2 * n:] == 7).all()
        want, _ = a.run()
        # (the expected longest request, which is not given here, may split the work differently)
        assert (out[5:5 + 2 * n].float() - want.float()).abs().max().item() <= 2.0 ** -9
        # a request longer than max_query_len: its first tokens are served, the rest left
        out = torch.full_like(a.Q, 7.0)
        awq.awq_kv_attention(a.Q, _to_cache(a.cache), _i32(a.table), _i32(a.kv_lens),
                             query_start=_i32(a.start), max_query_len=n - 1, out=out)
        for b in range(2):
            got = out[b * n:(b + 1) * n]
            assert (got[-1] == 7).all()
            assert (got[:-1].float() - want[b * n:(b + 1) * n - 1].float()).abs().max().item() <= 2.0 ** -9


@pytest.mark.parametrize("n", [1, 40])
def test_strided_queries_and_out(n):
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    a = Attend([n, n], [50, 80], 4, 2, 64, 16, True, "bfloat16", seed=14)
    want, _ = a.run()
    wide = torch.zeros((2 * n, 8, 64), dtype=a.Q.dtype, device=dev())
    wide[:, :4] = a.Q
    a.Q = wide[:, :4]
    out = torch.empty_like(want)
    got, _ = a.run(out=out)
    assert got is out and torch.equal(got, want)


@pytest.mark.parametrize("n", [1, 64])
def test_calls_repeat_and_do_not_depend_on_the_workspace(n):
    """Split keys (one request, a long context): the same bits from call to
    call, with a workspace full of NaN, on another stream, and whatever
    max_seq_len says within rounding."""
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    a = Attend([n], [3000], 4, 2, 64, 16, True, "float16", seed=15)
    cache, table, lens, start = _to_cache(a.cache), _i32(a.table), _i32(a.kv_lens), _i32(a.start)
    kw = dict(query_start=start, max_query_len=n)
    need = awq.awq_kv_attention_workspace_size(n, 1, 4, cache, n, 3000)
    assert need > 0
    want = awq.awq_kv_attention(a.Q, cache, table, lens, max_seq_len=3000, **kw)
    ws = torch.full((need,), 255, dtype=torch.uint8, device=dev())
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = awq.awq_kv_attention(a.Q, cache, table, lens, max_seq_len=3000, workspace=ws, **kw)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    for m in (0, 100, 100000):
        got = awq.awq_kv_attention(a.Q, cache, table, lens, max_seq_len=m, **kw)
        assert (got.float() - want.float()).abs().max().item() <= 2.0 ** -9 * want.float().abs().max().item()
    with pytest.raises(awq.AwqError, match="workspace"):
        awq.awq_kv_attention(a.Q, cache, table, lens, max_seq_len=3000, workspace=None, **kw)


def test_decode_steps_end_to_end_captured():
    """A run as a server makes it: assign, append, attend, then the same step
    captured once and replayed with other lengths and tokens, eager work between."""
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    rng = np.random.default_rng(16)
    B, Hq, H, D, page, blocks = 3, 4, 2, 64, 16, 12
    pages = B * blocks
    cache = awq.empty_kv_cache(pages, H, D, page, dev())
    ref = kv.new_cache(pages, H, D, page)
    table, free = _i32(np.full((B, blocks), -1)), rng.permutation(pages).astype(np.int32)
    old = np.zeros(B, np.int32)
    ref_table = np.full((B, blocks), -1, np.int32)

    def prompt(new):
        nonlocal old, free, ref_table
        T = int(sum(new))
        (Q, q), (K, k), (V, v) = (_rounded(rng.normal(size=(T, h, D)), "float16") for h in (Hq, H, H))
        lens, start, slots, used = awq.awq_kv_assign(_i32(old), _i32(new), table, _i32(free), page, T)
        awq.awq_kv_append(K, V, cache, slots)
        O = awq.awq_kv_attention(Q, cache, table, lens, query_start=start, max_query_len=max(new))
        ref_table, rl, rs, rslots, ru = kv.assign(old, new, ref_table, free, page, T)
        kv.append(ref, k, v, rslots)
        want, _, bound, _ = kv.attention64(q.astype(np.float64), ref, ref_table, rl, rs, D ** -0.5)
        assert (np.abs(out_to_f64(O) - want) <= bound).all()
        assert np.array_equal(table.cpu().numpy(), ref_table) and used.item() == ru[0]
        free, old = free[ru[0]:], rl

    prompt([40, 3, 17])
    prompt([5, 60, 1])

    # one decode step, captured: static inputs, the step's results as outputs
    s_old, s_new = _i32(old), _i32([1, 1, 1])
    s_free = _i32(np.concatenate([free, np.full(40 - len(free) % 40, -1, np.int32)]))
    Q = torch.zeros((B, Hq, D), dtype=torch.float16, device=dev())
    K, V = (torch.zeros((B, H, D), dtype=torch.float16, device=dev()) for _ in range(2))

    def step():
        lens, _, slots, used = awq.awq_kv_assign(s_old, s_new, table, s_free, page, B)
        awq.awq_kv_append(K, V, cache, slots)
        return awq.awq_kv_attention(Q, cache, table, lens), lens, used

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step()                                              # warm up: slots are written again below
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        O, lens, used = step()
    for _ in range(6):
        (q_t, q), (k_t, k), (v_t, v) = (_rounded(rng.normal(size=(B, h, D)), "float16") for h in (Hq, H, H))
        Q.copy_(q_t), K.copy_(k_t), V.copy_(v_t)
        graph.replay()
        torch.cuda.synchronize()
        ref_table, rl, rs, rslots, ru = kv.assign(old, [1] * B, ref_table, free, page, B)
        kv.append(ref, k, v, rslots)
        want, _, bound, _ = kv.attention64(q.astype(np.float64), ref, ref_table, rl, rs, D ** -0.5)
        assert (np.abs(out_to_f64(O) - want) <= bound).all()
        assert np.array_equal(lens.cpu().numpy(), rl) and used.item() == ru[0]
        eager = awq.awq_kv_attention(Q, cache, table, lens)
        assert torch.equal(eager, O)
        free, old = free[ru[0]:], rl
        s_old.copy_(lens)
        s_free[:len(free)] = _i32(free)


@pytest.mark.parametrize("D,kv_lens", [(64, [1, 63, 64, 65, 128, 129, 200, 700]), (128, [64, 130, 190, 260])])
@pytest.mark.parametrize("requests", [1, 40])
def test_prompts_of_few_and_many_workgroups(D, kv_lens, requests):
    """The same requests alone, where two groups of waves share the keys, and
    among so many that one does; one to a dozen tiles of keys, odd and even."""
    for n in kv_lens:
        q = min(n, 150)
        a = Attend([q] * requests, [n] * requests, 16, 16, D, 64, True, "float16", seed=n)
        O, _ = a.run()
        if requests == 1:
            a.check()
            a.check(window=70)
            continue
        one = Attend([q], [n], 16, 16, D, 64, True, "float16", seed=n)
        one.Q, one.cache, one.table = a.Q[:q], a.cache, a.table[:1]
        want, _ = one.run()
        # the same weights in another order of sums, and of M: a rounding of either output
        assert (O[:q].float() - want.float()).abs().max().item() <= 2.0 ** -9 * float(want.abs().max())


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 3, 40])
def test_any_bits_in_hidden_steps(n, D):
    """Slots behind a row, before its window, past the last token and in pages
    that no row names: infinities and NaN of either sign, negative and tiny
    steps, key and value, leave every row's result within its bound."""
    bits = np.array([0x7C00, 0xFC00, 0x7E00, 0xFE00, 0xBC00, 0x8000, 0x0001, 0x8001, 0x7BFF, 0xFBFF], np.uint16)
    a = Attend([n, n], [150 + n, 97 + n], 4, 2, D, 16, True, "float16", seed=22)
    W = 30
    for b in range(2):
        kv_len = int(a.kv_lens[b])
        first = kv_len - n - W + 1                       # of the first row's window
        for pos in list(range(first)) + list(range(kv_len, -(-kv_len // 16) * 16)):
            a.cache[1].view(np.uint16)[a.table[b, pos // 16], :, pos % 16] = \
                bits[[(pos * 3) % len(bits), (pos * 7 + b) % len(bits)]]
    a.check(window=W)


def test_two_graphs_and_two_streams_at_once():
    """Two captured attention calls over one cache, each with splits and its own
    scratch, replayed side by side on two streams and in turn: the eager results."""
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    a = Attend([1, 1], [5000, 3300], 4, 2, 64, 16, True, "float16", seed=23)
    b = Attend([64], [5000], 4, 2, 64, 16, True, "float16", seed=23)
    cache = _to_cache(a.cache)
    table, lens = _i32(a.table), _i32(a.kv_lens)
    start = _i32([0, 64])
    calls = (lambda: awq.awq_kv_attention(a.Q, cache, table, lens, max_seq_len=5000),
             lambda: awq.awq_kv_attention(b.Q, cache, table[:1], lens[:1], query_start=start, max_query_len=64,
                                          max_seq_len=5000))
    want = [f() for f in calls]
    graphs, outs, streams = [], [], [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for f in calls:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(f())
        graphs.append(g)
    for i in range(6):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        if i % 2:
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        else:
            for g in graphs:
                g.replay()
        eager = [f() for f in calls]
        torch.cuda.synchronize()
        for o, e, w in zip(outs, eager, want):
            assert torch.equal(o, w) and torch.equal(e, w)
