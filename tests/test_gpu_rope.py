"""GPU parity of rotary positions with oracle/rope.py, and of the keys that go
rotated into the 4-bit cache, whose bits equal the oracle's.

Tolerance of a rotated element, y = own c + partner s with |own c| + |partner s| =
mag: c and s are rounded to fp32 (2^-24 of them), each product (2^-24) and the sum
(2^-24 of at most mag), so 4 * 2^-24 mag covers them to first order, and the
output's own rounding is half a step, eps/2 |y| or half a subnormal step."""

import numpy as np
import pytest

from gpu_common import dev, out_to_f64, say, torch_mod
from oracle import kv
from oracle.rope import frequencies, rotate32, rotate64
from test_gpu_kv import _i32, _rounded, _same_cache, _to_cache

pytestmark = pytest.mark.gpu

HALF_STEP = {"float16": (2.0 ** -11, 2.0 ** -25), "bfloat16": (2.0 ** -8, 2.0 ** -134)}


def _close(got, x32, pos, inv, dtype, factor=1.0, interleaved=False, inverse=False):
    y, mag = rotate64(x32, pos, inv, factor, interleaved, inverse)
    rel, sub = HALF_STEP[dtype]
    err = np.abs(out_to_f64(got) - y)
    over = err - (rel * np.abs(y) + sub + 4 * 2.0 ** -24 * mag * (1 + rel))
    assert (over <= 0).all(), over.max()


def _freq(inv):
    return torch_mod().from_numpy(inv).to(dev())


def _input(rng, shape, dtype):
    return _rounded(rng.normal(0, 1, shape) * np.exp(rng.normal(0, 2, shape[:-1] + (1,))), dtype)


@pytest.mark.parametrize("T,Hq,Hkv,D,R,interleaved,dtype", [
    (1, 1, 0, 64, 64, False, "float16"), (1, 32, 8, 128, 128, True, "bfloat16"),
    (5, 3, 1, 128, 32, False, "bfloat16"), (17, 4, 2, 64, 16, True, "float16"),
    (33, 5, 5, 80, 80, False, "float16"), (31, 2, 1, 96, 48, False, "bfloat16"),
    (9, 3, 2, 256, 256, True, "float16"), (13, 2, 1, 512, 512, False, "float16"),
    (7, 9, 4, 16, 16, False, "bfloat16"), (21, 2, 2, 272, 144, False, "bfloat16"),
    (2500, 2, 1, 128, 128, False, "float16"), (300, 70, 1, 64, 32, True, "bfloat16"),
])
def test_rope(T, Hq, Hkv, D, R, interleaved, dtype):
    import bit_weight_only_quantize_amd as awq
    say("rope", T, Hq, Hkv, D, R, interleaved, dtype)
    rng = np.random.default_rng(T * D + R)
    pos = rng.integers(-5000, 1 << 20, T)
    pos[:min(T, 4)] = [0, 1, 2 ** 31 - 1, -2 ** 31][:min(T, 4)]
    inv, factor = frequencies(R, 10000.0, "yarn", 8.0, 4096.0)
    q, q32 = _input(rng, (T, Hq, D), dtype)
    before = q.clone()
    k, k32 = _input(rng, (T, Hkv, D), dtype) if Hkv else (None, None)
    got = awq.awq_rope(q, _i32(pos), _freq(inv), K=k, attention_factor=factor, interleaved=interleaved)
    gq, gk = got if Hkv else (got, None)
    _close(gq, q32, pos, inv, dtype, factor, interleaved)
    assert (gq[..., R:] == q[..., R:]).all() and (q == before).all()
    if Hkv:
        _close(gk, k32, pos, inv, dtype, factor, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,R", [(128, 128), (80, 64), (64, 32)])
def test_slices_of_a_fused_projection_in_place(D, R, interleaved):
    import bit_weight_only_quantize_amd as awq
    rng = np.random.default_rng(D)
    T, Hq, Hkv = 41, 6, 2
    qkv, x32 = _input(rng, (T, Hq + 2 * Hkv, D), "bfloat16")
    pos = rng.integers(0, 9000, T)
    inv, _ = frequencies(R)
    want_q = awq.awq_rope(qkv[:, :Hq].contiguous(), _i32(pos), _freq(inv), interleaved=interleaved)
    v = qkv[:, Hq + Hkv:].clone()
    q, k = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv]
    got = awq.awq_rope(q, _i32(pos), _freq(inv), K=k, interleaved=interleaved, out=(q, k))
    assert got[0].data_ptr() == qkv.data_ptr()
    assert (qkv[:, :Hq] == want_q).all() and (qkv[:, Hq + Hkv:] == v).all()
    _close(k, x32[:, Hq:Hq + Hkv], pos, inv, "bfloat16", 1.0, interleaved)


@pytest.mark.parametrize("interleaved", [False, True])
def test_inverse_is_the_gradient(interleaved):
    """<rotate x, g> = <x, inverse g> for any x and g, and the inverse undoes the rotation."""
    import bit_weight_only_quantize_amd as awq
    rng = np.random.default_rng(3)
    T, H, D = 19, 3, 64
    inv, _ = frequencies(48)
    pos = rng.integers(0, 100000, T)
    (x, x32), (g, g32) = _input(rng, (T, H, D), "float16"), _input(rng, (T, H, D), "float16")
    kw = dict(interleaved=interleaved)
    y = awq.awq_rope(x, _i32(pos), _freq(inv), **kw)
    d = awq.awq_rope(g, _i32(pos), _freq(inv), inverse=True, **kw)
    _close(d, g32, pos, inv, "float16", 1.0, interleaved, True)
    # a difference in one channel changes the outputs by its column of the rotation
    lhs = (out_to_f64(y) * g32).sum((-1, -2))
    rhs = (out_to_f64(d) * x32).sum((-1, -2))
    _, my = rotate64(x32, pos, inv, 1.0, interleaved)
    _, mg = rotate64(g32, pos, inv, 1.0, interleaved, True)
    tol = (2.0 ** -11 + 2.0 ** -21) * ((my * np.abs(g32)).sum((-1, -2)) + (np.abs(x32) * mg).sum((-1, -2))) \
        + 2.0 ** -24 * (np.abs(g32) + np.abs(x32)).sum((-1, -2))
    # (mag is 0 behind the rotated channels, whose products are the same on both sides up to a rounding of nothing)
    tail = np.abs(x32[..., 48:] * g32[..., 48:]).sum((-1, -2)) * 2.0 ** -40
    assert (np.abs(lhs - rhs) <= tol + tail).all()
    back = out_to_f64(awq.awq_rope(y, _i32(pos), _freq(inv), inverse=True, **kw))
    _, mb = rotate64(out_to_f64(y), pos, inv, 1.0, interleaved, True)
    # y's rounding, turned back (|c| + |s| <= sqrt 2 of the larger), and its own
    lim = (2.0 ** -11 * 2 + 2.0 ** -20) * mb + 2.0 ** -24
    lim[..., :48] += 2.0 ** -11 * np.sqrt(2) * np.abs(out_to_f64(y)[..., :48]).max(-1, keepdims=True)
    assert (np.abs(back - x32) <= lim).all()


def test_infinities_and_nan_stay_in_their_pairs():
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    x = torch.ones((6, 2, 64), dtype=torch.bfloat16, device=dev())
    x[1, 0, 3] = float("inf")
    x[2, 1, 40] = float("nan")                     # behind the rotated channels
    x[3, 0, 17] = float("-inf")
    inv, _ = frequencies(32)
    got = awq.awq_rope(x, _i32(range(6)), _freq(inv)).float()
    bad = ~torch.isfinite(got)
    want = torch.zeros_like(bad)
    want[1, 0, [3, 19]] = True
    want[2, 1, 40] = True
    want[3, 0, [1, 17]] = True
    assert (bad == want).all()


def test_no_tokens_and_no_frequencies_of_another_size():
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    inv, f = awq.awq_rope_frequencies(64, device=dev())
    q = torch.empty((0, 4, 64), dtype=torch.float16, device=dev())
    assert awq.awq_rope(q, _i32([]), inv).shape == (0, 4, 64) and f == 1.0
    with pytest.raises(ValueError):
        awq.awq_rope(torch.empty((2, 4, 32), dtype=torch.float16, device=dev()), _i32([0, 1]), inv)
    with pytest.raises(awq.AwqError, match="overlaps"):
        x = torch.zeros((4, 4, 64), dtype=torch.float16, device=dev())
        awq.awq_rope(x[:3], _i32([0, 1, 2]), inv, out=x[1:])
    with pytest.raises(awq.AwqError, match="overlaps"):
        awq.awq_rope(x, _i32(range(4)), inv, K=x, out=(x, x))


@pytest.mark.parametrize("T,Hq,Hkv,D,R,page,zp,dtype,interleaved", [
    (1, 1, 1, 64, 64, 16, True, "float16", False), (3, 8, 2, 128, 128, 16, True, "bfloat16", False),
    (70, 0, 3, 64, 32, 32, False, "bfloat16", True), (130, 16, 8, 128, 64, 64, True, "float16", False),
    (45, 5, 5, 128, 16, 128, False, "float16", True), (300, 3, 1, 64, 48, 64, True, "bfloat16", False),
])
def test_append_rope(T, Hq, Hkv, D, R, page, zp, dtype, interleaved):
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    say("append_rope", T, Hq, Hkv, D, R, page, zp, dtype, interleaved)
    rng = np.random.default_rng(T + D)
    pages = -(-T // page) + 2
    cache = kv.new_cache(pages, Hkv, D, page, zp, rng)
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    slots[rng.random(T) < 0.1] = -1
    if T > 4:
        slots[2], slots[3] = pages * page, 2 ** 31 - 1
    pos = rng.integers(0, 1 << 20, T)
    inv, factor = frequencies(R, 500000.0, "bands", 8.0, 8192.0)
    (K, k32), (V, v32) = _input(rng, (T, Hkv, D), dtype), _input(rng, (T, Hkv, D), dtype)
    Q, q32 = _input(rng, (T, Hq, D), dtype) if Hq else (None, None)
    got = _to_cache(cache)
    count = torch.zeros(1, dtype=torch.int32, device=dev())
    out = awq.awq_kv_append_rope(K, V, got, _i32(slots), _i32(pos), _freq(inv), Q=Q, attention_factor=factor,
                                 interleaved=interleaved, nonfinite_count=count)
    kv.append(cache, rotate32(k32, pos, inv, factor, interleaved), v32, slots)
    _same_cache(got, cache)
    assert count.item() == 0
    if Hq:                                          # also of tokens without a slot, and as awq_rope has them
        _close(out, q32, pos, inv, dtype, factor, interleaved)
        again = awq.awq_rope(Q, _i32(pos), _freq(inv), attention_factor=factor, interleaved=interleaved)
        assert torch.equal(out, again)
    else:
        assert out is None


def test_append_rope_in_place_from_a_fused_projection():
    import bit_weight_only_quantize_amd as awq
    rng = np.random.default_rng(8)
    T, Hq, Hkv, D = 20, 4, 2, 128
    qkv, x32 = _input(rng, (T, Hq + 2 * Hkv, D), "float16")
    inv, _ = frequencies(128)
    pos, slots = rng.integers(0, 70000, T), rng.permutation(64)[:T].astype(np.int32)
    cache = kv.new_cache(4, Hkv, D, 16, True, rng)
    got, q = _to_cache(cache), qkv[:, :Hq]
    awq.awq_kv_append_rope(qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], got, _i32(slots), _i32(pos), _freq(inv), Q=q, out=q)
    kv.append(cache, rotate32(x32[:, Hq:Hq + Hkv], pos, inv), x32[:, Hq + Hkv:], slots)
    _same_cache(got, cache)
    _close(qkv[:, :Hq], x32[:, :Hq], pos, inv, "float16")
    assert (out_to_f64(qkv[:, Hq:]) == x32[:, Hq:]).all()


def test_append_rope_counts_what_is_not_finite():
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    K = torch.ones((3, 1, 64), dtype=torch.float16, device=dev())
    K[1, 0, 5] = float("inf")                      # its pair is not finite either
    V = torch.ones_like(K)
    V[2, 0, 1] = float("nan")
    count = torch.zeros(1, dtype=torch.int32, device=dev())
    cache = awq.empty_kv_cache(1, 1, 64, 16, dev())
    awq.awq_kv_append_rope(K, V, cache, _i32([0, 1, 2]), _i32([1, 2, 3]), _freq(frequencies(64)[0]),
                           nonfinite_count=count)
    assert count.item() == 3


def test_captured_and_on_another_stream():
    """Replays with other positions and inputs in the same buffers equal the eager calls."""
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    T, Hq, Hkv, D = 12, 4, 2, 64
    g = torch.Generator(device=dev()).manual_seed(5)
    new = lambda h: torch.randn((T, h, D), generator=g, device=dev()).half()   # noqa: E731
    inv, _ = awq.awq_rope_frequencies(64, device=dev())
    Q, K, V, pos, slots = new(Hq), new(Hkv), new(Hkv), _i32(range(T)), _i32(range(5, 5 + T))
    cache, out = awq.empty_kv_cache(2, Hkv, D, 16, dev()), torch.empty_like(Q)
    for c in cache:
        c.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        awq.awq_kv_append_rope(K, V, cache, slots, pos, inv, Q=Q, out=out)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        awq.awq_kv_append_rope(K, V, cache, slots, pos, inv, Q=Q, out=out)
    for i in range(4):
        Q.copy_(new(Hq)), K.copy_(new(Hkv)), V.copy_(new(Hkv)), pos.add_(777 * i)
        graph.replay()
        torch.cuda.synchronize()
        got = [out.clone(), *(c.clone() for c in cache)]
        want = awq.awq_kv_append_rope(K, V, cache, slots, pos, inv, Q=Q)
        for a, b in zip(got, (want, *cache)):
            assert torch.equal(a, b)


def test_strides_past_32_bits():
    """Tokens 2^27 elements apart: the last ones lie beyond 4 GiB."""
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    T, H, D, stride = 20, 2, 64, 1 << 27
    big = torch.empty((T - 1) * stride + H * D, dtype=torch.float16, device=dev())
    q = torch.as_strided(big, (T, H, D), (stride, D, 1))
    rng = np.random.default_rng(4)
    x, x32 = _input(rng, (T, H, D), "float16")
    q.copy_(x)
    pos, inv = rng.integers(0, 5000, T), frequencies(64)[0]
    got = awq.awq_rope(q, _i32(pos), _freq(inv), out=q)
    assert got.data_ptr() == big.data_ptr()
    _close(q, x32, pos, inv, "float16")
    q.copy_(x)
    cache = kv.new_cache(2, H, D, 16, True, rng)
    dc = _to_cache(cache)
    awq.awq_kv_append_rope(q, q, dc, _i32(range(T)), _i32(pos), _freq(inv))
    kv.append(cache, rotate32(x32, pos, inv), x32, np.arange(T))
    _same_cache(dc, cache)
