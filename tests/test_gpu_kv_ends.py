"""GPU parity of the 4-bit key/value cache at its ends: keys just outside what a
row sees, in every variant of the attention kernels; queries and logits near
fp32's limits; tied logits far past fp32's fractions; value steps many orders
apart, long tails of small weights, contexts of many parts and pages; keys and
values past fp16's range."""

import numpy as np
import pytest

from gpu_common import dev, out_to_f64, say, torch_mod
from oracle import kv
from test_gpu_kv import Attend, _i32, _rounded, _to_cache

pytestmark = pytest.mark.gpu

EPS = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}


class Request(Attend):
    """A batch whose keys, values and queries a test sets itself."""

    def put(self, b, pos, K, V):
        """K, V fp32 [n][heads][D] as the tokens at positions `pos` of request b."""
        pos = np.asarray(pos)
        kv.append(self.cache, np.asarray(K, np.float32), np.asarray(V, np.float32),
                  self.table[b, pos // self.page] * self.page + pos % self.page)

    def ask(self, Q):
        self.Q, q32 = _rounded(Q, self.dtype)
        self.q64 = q32.astype(np.float64)

    def tokens(self, b):
        """kv.read of all of request b's tokens."""
        pos = np.arange(int(self.kv_lens[b]))
        return kv.read(self.cache, self.D, self.table[b, pos // self.page] * self.page + pos % self.page)

    def answer(self, max_seq_len=None, max_query_len=None, **kw):
        """The output in fp64, for one query token per request or several."""
        import bit_weight_only_quantize_amd as awq
        one = (self.q_lens == 1).all()
        return awq.awq_kv_attention(self.Q, _to_cache(self.cache), _i32(self.table), _i32(self.kv_lens),
                                    query_start=None if one else _i32(self.start),
                                    max_query_len=max_query_len or int(self.q_lens.max()), return_lse=True,
                                    max_seq_len=int(max(self.kv_lens)) if max_seq_len is None else max_seq_len, **kw)


# ---- keys outside what a row sees --------------------------------------------------

@pytest.mark.parametrize("n,most", [(1, None), (1, 100000), (3, None), (3, 100000), (20, None)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("zp", [True, False])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_hidden_keys_of_every_variant(n, most, D, zp, dtype):
    """Every kernel variant (eight waves, four waves with parts, prompt), every
    place in a tile where a row's keys may end or begin: keys that a row does not
    see would take all of its weight."""
    for first in (33, 41):
        lens = [first + i * 17 for i in range(16)]
        a = Request([n] * 16, lens, 4, 2, D, 16, zp, dtype, seed=37)
        steps = a.cache[1].view(np.uint16)
        for b, L in enumerate(lens):                        # past the last token
            for pos in range(L, -(-L // 16) * 16):
                steps[a.table[b, pos // 16], :, pos % 16] = 0x7800      # 32768
        _check_hidden(a, most)
        for b, L in enumerate(lens):                        # before every row's window
            for pos in range(L - n - 9):
                steps[a.table[b, pos // 16], :, pos % 16] = 0x7800
        _check_hidden(a, most, 10)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("zp", [True, False])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_hidden_keys_in_the_prompt_kernel_of_one_group(D, zp, dtype):
    """Counted with the longest's tokens the requests here are 640 workgroups, which
    take one group of waves each."""
    n, B = 20, 32
    lens = [33 + i * 7 for i in range(B)]
    a = Request([n] * B, lens, 4, 2, D, 16, zp, dtype, seed=39)
    steps = a.cache[1].view(np.uint16)
    for b, L in enumerate(lens):
        for pos in list(range(L, -(-L // 16) * 16)) + list(range(L - n - 9)):
            steps[a.table[b, pos // 16], :, pos % 16] = 0x7800
    _check_hidden(a, None, 10, max_query_len=n * B)


def _check_hidden(a, most, window=0, **kw):
    O, lse = a.answer(max_seq_len=most, window=window, **kw)
    want, wl, bound, lse_bound = kv.attention64(a.q64, a.cache, a.table, a.kv_lens, a.start, a.D ** -0.5, True, window,
                                                EPS[a.dtype])
    assert (np.abs(out_to_f64(O) - want) <= bound).all()
    assert (np.abs(lse.cpu().numpy() - wl) <= lse_bound).all()


# ---- near fp32's limits ------------------------------------------------------------------

@pytest.mark.parametrize("n", [1, 3, 40])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("gain,scale", [(2.0 ** 120, 0.125), (2.0 ** 121, 0.125), (2.0 ** 123, 0.125),
                                        (2.0 ** 124, 2.0 ** -6), (2.0 ** 100, 2.0 ** 20)])
def test_largest_bfloat16_queries(n, D, gain, scale):
    """Finite logits up to 2^127 give finite results: those of the keys whose
    logits fp32 cannot tell from the largest."""
    a = Request([n], [100], 4, 2, D, 16, True, "bfloat16", seed=31)
    a.Q = (a.Q.float() * gain).to(a.Q.dtype)
    a.q64 = out_to_f64(a.Q)
    for s in (scale, -scale):
        _check_hull(a, s)


def _check_hull(a, scale):
    """O between the least and the largest value of the keys whose logits lie
    within fp32's error of the row's largest.  A logit's error is at most dl (D
    products, the zero term, the scaling: attention64), so a key more than 2 dl +
    40 below the largest has a weight below e^-40 of it.  Beside that the weights'
    rounding 2^-11 and the output's."""
    O, lse = a.answer(scale=scale)
    got = out_to_f64(O)
    assert np.isfinite(got).all() and torch_mod().isfinite(lse).all()
    heads, Hkv = a.Q.shape[1], a.cache[1].shape[1]
    for b in range(len(a.kv_lens)):
        c, z, s, val = a.tokens(b)
        for i in range(int(a.q_lens[b])):
            seen = int(a.kv_lens[b]) - int(a.q_lens[b]) + i + 1
            for j in range(heads):
                h, q = j * Hkv // heads, a.q64[a.start[b] + i, j]
                logit = (val[0, :seen, h] @ q) * scale
                mag = s[0, :seen, h] * ((c[0, :seen, h] + z[0, :seen, h][:, None] + 16) @ np.abs(q))
                dl = (a.D + 8) * 2.0 ** -24 * abs(scale) * mag.max()
                near = np.flatnonzero(logit >= logit.max() - 2 * dl - 40)
                v = val[1, near, h]
                tol = (EPS[a.dtype] + 2.0 ** -11) * np.abs(v).max(0) + 2.0 ** -11 * (
                    s[1, near, h][:, None] * np.abs(c[1, near, h])).max(0) + 2.0 ** -24
                o = got[a.start[b] + i, j]
                assert (o >= v.min(0) - tol).all() and (o <= v.max(0) + tol).all(), (b, i, j)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("scale", [1e4, 1e6, 3e7, 2e8, 1e9, 1e12, 1e30])
def test_logits_past_the_fractions_take_the_right_keys(n, dtype, scale):
    for size in (1.0, 1e-3, 1e3):
        _check_hull(Request([n, n], [150, 67], 4, 2, 64, 16, True, dtype, seed=20, size=size), scale)


@pytest.mark.parametrize("n", [1, 3, 40])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("scale", [1e4, 1e6, 3e7, 2e8, 1e9, 1e12, 1e30, -1e9])
def test_tied_logits_weigh_the_same(n, D, scale):
    """Two kinds of keys only, one far above the other; the values' steps differ
    by 2^17 from block to block.  The result is the mean of the winning kind's
    values, however the keys are dealt over waves and parts: few of one kind in
    some parts, many in others."""
    rng = np.random.default_rng(32)
    lens = [2100 + n, 700 + n]
    a = Request([n, n], lens, 4, 2, D, 16, True, "float16", seed=32)
    k0 = rng.normal(0, 1, (2, D))
    kinds = []
    for b, L in enumerate(lens):
        pos = np.arange(L)
        kind = np.where(pos < 600, pos % 97 != 5, pos % 3 == 0)
        size = np.where((pos // 130) % 2 == 0, 2.0 ** -9, 2.0 ** 8)
        a.put(b, pos, np.where(kind, -1.0, 1.0)[:, None, None] * k0,
              rng.normal(0.5, 1, (L, 2, D)) * size[:, None, None])
        kinds.append(kind)
    sign = np.where(rng.random((2 * n, 4)) < 0.5, -1.0, 1.0)
    a.ask(sign[..., None] * k0[[0, 0, 1, 1]] + rng.normal(0, 0.05, (2 * n, 4, D)))
    for most in (max(lens), 700, 100, 50000):
        O, _ = a.answer(max_seq_len=most, scale=scale)
        got = out_to_f64(O)
        for b, L in enumerate(lens):
            c, z, s, val = a.tokens(b)
            for i in range(n):
                for j in range(4):
                    h, r = j // 2, int(a.start[b]) + i
                    seen = np.arange(L) <= L - n + i
                    win = kinds[b] == (sign[r, j] * scale < 0)
                    at = np.flatnonzero(seen & win)
                    w = s[1, at, h]
                    want = val[1, at, h].mean(0)
                    cv = np.maximum(np.abs(c[1, at, h]), np.abs(c[1, at, h] - z[1, at, h][:, None]))
                    bound = (EPS["float16"] * np.abs(want) + 2.0 ** -11 * (w[:, None] * cv).mean(0)
                             + (len(at) + 64) * 2.0 ** -24 * (w[:, None] * (np.abs(c[1, at, h]) + 32)).mean(0) + 2.0 ** -25)
                    err = np.abs(got[r, j] - want)
                    assert (err <= bound).all(), (most, b, i, j, float((err / bound).max()))


@pytest.mark.parametrize("n", [1, 3, 40])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_rows_on_both_sides_of_the_fractions(n, sign, dtype):
    """Logits of one sign over a factor of 2^10, and rows 2^6 apart: from tile to
    tile and row to row on either side of where weights change their reference."""
    rng = np.random.default_rng(38)
    L = 1000
    a = Request([n], [L], 8, 2, 64, 16, True, dtype, seed=38)
    base = rng.normal(0, 1, (2, 64))
    a.put(0, np.arange(L), sign * base * 2.0 ** rng.uniform(-8, 2, (L, 1, 1)),
          rng.normal(0, 1, (L, 2, 64)) * 2.0 ** rng.integers(-4, 4, (L, 1, 1)))
    a.ask(base[[0] * 4 + [1] * 4] * 2.0 ** rng.integers(-3, 4, (n, 8, 1)))
    for e in range(10, 24, 2):
        _check_hull(a, 2.0 ** e)


# ---- value steps many orders apart, and long tails ---------------------------------------

@pytest.mark.parametrize("n", [1, 3, 40])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("ratio", [2.0 ** 14, 2.0 ** 20, 2.0 ** 24, 2.0 ** 28])
@pytest.mark.parametrize("at", [0, 150])
def test_large_steps_of_no_weight(n, D, ratio, at):
    """A token whose values are orders of magnitude larger, with a weight near
    2^-80: the others' weights keep their precision."""
    rng = np.random.default_rng(33)
    lens = [200 + n, 1700 + n]
    a = Request([n, n], lens, 4, 2, D, 16, True, "float16", seed=33)
    base = rng.normal(0, 1, (2, D))
    for b, L in enumerate(lens):
        V = rng.normal(0.3, 1, (L, 2, D)) * 2.0 ** -12
        K = rng.normal(0, 1, (L, 2, D))
        V[at] *= ratio
        K[at] = -56 * D ** -0.5 * base
        a.put(b, np.arange(L), K, V)
    a.ask(base[[0, 0, 1, 1]] + rng.normal(0, 0.1, (2 * n, 4, D)))
    _check_weighted(a)


@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("D", [64, 128])
def test_long_tails_of_small_weights(n, D):
    """One key with nearly all of the weight and a value of zeros in half of the
    channels, twenty thousand with 2^-25.5 of it each: the sum of the tail
    arrives."""
    rng = np.random.default_rng(34)
    L = 20000
    a = Request([n], [L], 2, 1, D, 64, True, "float16", seed=34)
    base = rng.normal(0, 1, D)
    K = rng.normal(0, 0.002, (L, 1, D))
    K[0, 0] = base * (25.5 * np.log(2) * D ** 0.5 / (base @ base))
    V = rng.uniform(0.5, 1, (L, 1, D))
    V[0, 0, :D // 2], V[0, 0, D // 2:] = 0.0, 1.0
    a.put(0, np.arange(L), K, V)
    a.ask(base + rng.normal(0, 0.01, (n, 2, D)))
    _check_weighted(a)
    _check_weighted(a, max_seq_len=1000)


def _check_weighted(a, relative=None, **kw):
    O, lse = a.answer(**kw)
    want, wl, bound, lse_bound = kv.attention64(a.q64, a.cache, a.table, a.kv_lens, a.start, a.D ** -0.5, True, 0,
                                                EPS[a.dtype], weighted=True)
    err = np.abs(out_to_f64(O) - want)
    say("worst err / bound", float(np.max(err / np.maximum(bound, 1e-300))))
    assert (err <= bound).all()
    assert (np.abs(lse.cpu().numpy() - wl) <= lse_bound).all()
    if relative is not None:
        assert np.linalg.norm(err) <= relative * np.linalg.norm(want)


# ---- contexts of many parts and pages ------------------------------------------------------

@pytest.mark.parametrize("n,L,Hq,D,page,zp,dtype,most", [
    (1, 20011, 2, 64, 16, True, "float16", 20011),          # 40 parts: the join's second turn
    (1, 20011, 2, 128, 64, False, "bfloat16", 20011),
    (1, 33000, 1, 64, 16, True, "float16", 60000),          # as many parts as there can be
    (1, 20000, 2, 64, 16, True, "float16", 100),            # one workgroup: waves of 157 pages
    (1, 9999, 2, 128, 16, True, "bfloat16", 1536),
    (2, 9000, 8, 128, 16, False, "float16", 3000),          # few parts of many pages
    (64, 5003, 1, 64, 16, True, "float16", 5003),           # the prompt kernel: 20 parts
    (64, 20001, 1, 128, 64, True, "bfloat16", 20001),       # ... as many as there can be
    (70, 9001, 1, 64, 32, False, "float16", 100),           # ... one part
])
def test_long_contexts(n, L, Hq, D, page, zp, dtype, most):
    """Against the oracle, and (random values: the rounding errors of the many
    weights cancel) within 1.25 times the output's rounding in the norm."""
    a = Request([n], [L], Hq, 1, D, page, zp, dtype, seed=35)
    _check_weighted(a, relative=1.25 * EPS[dtype], max_seq_len=most)


def test_prompt_chunk_and_long_decoding_requests():
    """One chunk of a prompt among requests of one token with long contexts."""
    lens = [260, 5000, 33, 4100, 1, 700, 2048, 3000]
    a = Request([200] + [1] * 7, lens, 4, 1, 64, 16, True, "float16", seed=36)
    _check_weighted(a)
    _check_weighted(a, max_seq_len=100)


# ---- append ----------------------------------------------------------------------------------

@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("zp", [True, False])
def test_steps_beyond_fp16_are_counted(D, zp):
    """bfloat16 keys and values can be so large that a group's step is not an fp16
    number: each such group counts once; the largest that fit do not."""
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    levels = 15 if zp else 7
    fits, not_ = (978944.0, 983040.0) if zp else (456704.0, 458752.0)      # bfloat16; steps 65263 (65243), 65536
    assert fits / levels < 65520 <= not_ / levels
    K, V = torch.ones((6, 3, D)), torch.ones((6, 3, D))
    K[0, 1, 7] = fits
    V[1, 2, D - 1] = not_
    K[2, 0, 0], K[2, 0, 1] = 3e38, -3e38                    # the range itself overflows
    V[3, 1, 5] = -not_
    K[4, 2, 9] = -fits
    K[5, 0, 3] = 3e38                                       # this token is skipped
    K, V = (x.to(torch.bfloat16).to(dev()) for x in (K, V))
    cache = awq.empty_kv_cache(1, 3, D, 16, dev(), zero_point=zp)
    count = torch.zeros(1, dtype=torch.int32, device=dev())
    awq.awq_kv_append(K, V, cache, _i32([0, 3, 4, 9, 15, -1]), nonfinite_count=count)
    assert count.item() == 3
    inf = torch.isinf(cache[1][0][:, [0, 3, 4, 9, 15]]).nonzero().cpu().tolist()      # [head][token][k, v]
    assert sorted(inf) == [[0, 2, 0], [1, 3, 1], [2, 1, 1]]
    K[0, 0, 0] = float("inf")                               # an infinite value counts as itself only
    awq.awq_kv_append(K[:1], V[:1], cache, _i32([0]), nonfinite_count=count)
    assert count.item() == 4
