"""Rotary positions without a GPU: the frequencies, and every refusal before any HIP call."""

import ctypes

import numpy as np
import pytest

from oracle.rope import frequencies, rotate32, rotate64
from test_kv_abi_cpu import CACHE_REFUSALS, INVALID, UNSUPPORTED, P, addr, binding, cache, cfg, i32, lib, tensors, torch

OK = binding.AWQ_OK


@pytest.mark.parametrize("R,base,kw", [
    (128, 10000.0, {}), (16, 500000.0, {}), (64, 10000.0, dict(scaling="linear", factor=4.0)),
    (128, 10000.0, dict(scaling="ntk", factor=8.0)), (128, 10000.0, dict(scaling="yarn", factor=32.0, original_len=4096)),
    (64, 1000000.0, dict(scaling="yarn", factor=4.0, original_len=32768, low=2.0, high=20.0)),
    (48, 10000.0, dict(scaling="yarn", factor=0.5, original_len=100)),
    (128, 500000.0, dict(scaling="bands", factor=8.0, original_len=8192)),
    (96, 500000.0, dict(scaling="bands", factor=32.0, original_len=8192, low=0.5, high=7.0)),
])
def test_frequencies(R, base, kw):
    got, factor = binding.awq_rope_frequencies(R, base, device="cpu", **kw)
    names = {"scaling": "scaling", "factor": "s", "original_len": "L", "low": "low", "high": "high"}
    want, f = frequencies(R, base, **{names[k]: v for k, v in kw.items()})
    # a few roundings of pow, log and products, each 2^-53 (pow's to a few ulp)
    assert np.allclose(got.numpy(), want, rtol=2.0 ** -46, atol=0) and abs(factor - f) <= 2.0 ** -50 * f


def test_oracle_by_hand():
    """A quarter turn, and distances alone counting in products of queries and keys."""
    x = np.zeros((1, 1, 32))
    x[0, 0, 0] = 1.0
    inv = np.full(8, np.pi / 2)
    y, _ = rotate64(x, [1], inv)
    assert abs(y[0, 0, 8] - 1) < 1e-15 and abs(y[0, 0, 0]) < 1e-15
    y, _ = rotate64(x, [1], inv, interleaved=True)
    assert abs(y[0, 0, 1] - 1) < 1e-15
    rng = np.random.default_rng(0)
    q, k = rng.normal(size=(2, 1, 1, 64))
    inv, _ = frequencies(64)
    at = lambda x, p: rotate64(x, [p], inv)[0].ravel()      # noqa: E731
    assert abs(at(q, 70) @ at(k, 20) - at(q, 1050) @ at(k, 1000)) < 1e-12
    assert np.abs(rotate32(q, [70], inv) - at(q, 70)).max() < 1e-6


@pytest.mark.parametrize("R,base,scaling,status", [
    (0, 1e4, None, UNSUPPORTED), (24, 1e4, None, UNSUPPORTED), (-16, 1e4, None, UNSUPPORTED), (528, 1e4, None, UNSUPPORTED),
    (64, 1.0, None, INVALID), (64, float("nan"), None, INVALID), (64, float("inf"), None, INVALID),
    (64, 1e4, (5, 2.0, 0, 0, 0), INVALID), (64, 1e4, (1, 0.0, 0, 0, 0), INVALID), (64, 1e4, (1, float("nan"), 0, 0, 0), INVALID),
    (64, 1e4, (3, 2.0, 0.0, 0, 0), INVALID), (64, 1e4, (4, 2.0, 100.0, 4.0, 4.0), INVALID), (64, 1e4, (2, 1e-6, 0, 0, 0), INVALID),
    (64, 1e4, (4, 2.0, float("inf"), 0, 0), INVALID), (64, 1e4, (4, 2.0, 100.0, -1.0, 4.0), INVALID),
])
def test_frequency_refusals(R, base, scaling, status):
    inv, f = (ctypes.c_double * 256)(), ctypes.c_double()
    sc = None if scaling is None else ctypes.byref(binding.awq_rope_scaling(*scaling))
    assert lib.awq_rope_frequencies(R, base, sc, inv, ctypes.byref(f)) == status
    assert "awq_rope_frequencies" in lib.awq_last_error().decode()


def test_frequencies_need_places():
    f = ctypes.c_double()
    assert lib.awq_rope_frequencies(64, 1e4, None, None, ctypes.byref(f)) == INVALID
    assert lib.awq_rope_frequencies(64, 1e4, None, (ctypes.c_double * 32)(), None) == INVALID
    with pytest.raises(ValueError):
        binding.awq_rope_frequencies(64, scaling="other", device="cpu")
    with pytest.raises(binding.AwqError):
        binding.awq_rope_frequencies(20, device="cpu")


def args(pos=addr(12), inv=addr(13), factor=1.0, R=64, pairs=0, inverse=0):
    return ctypes.byref(binding.awq_rope_args(pos, inv, factor, R, pairs, inverse))


def rope(Q=addr(2), Qo=addr(3), heads=4, qs=256, qos=256, K=addr(4), Ko=addr(5), kv=2, ks=128, kos=128, xt=0, T=5,
         D=64, r=None):
    return lib.awq_rope(Q, Qo, heads, qs, qos, K, Ko, kv, ks, kos, xt, T, D, args() if r is None else r, None)


def append(Q=addr(2), Qo=addr(3), heads=4, qs=256, qos=256, K=addr(4), V=addr(5), xt=0, T=5, ks=128, vs=128, c=None,
           conf=None, slots=addr(6), r=None, nf=None):
    return lib.awq_kv_append_rope(Q, Qo, heads, qs, qos, K, V, xt, T, ks, vs, cache() if c is None else c,
                                  conf or cfg(64), slots, args() if r is None else r, nf, None)


ROPE_REFUSALS = [
    (dict(xt=2), INVALID), (dict(T=-1), INVALID), (dict(T=2 ** 25 + 1), INVALID), (dict(T=2 ** 27 + 1), INVALID), (dict(heads=-1), INVALID),
    (dict(heads=1025, qs=1 << 20, qos=1 << 20), INVALID), (dict(qs=248), INVALID), (dict(qos=260), INVALID),
    (dict(qs=1 << 58), INVALID), (dict(r=args(R=0)), UNSUPPORTED), (dict(r=args(R=24)), UNSUPPORTED),
    (dict(r=args(R=80)), UNSUPPORTED), (dict(r=args(pairs=2)), INVALID), (dict(r=args(inverse=-1)), INVALID),
    (dict(r=args(factor=float("nan"))), INVALID), (dict(r=args(pos=None)), INVALID), (dict(r=args(inv=None)), INVALID),
    (dict(r=args(pos=P(0x10002))), INVALID), (dict(r=args(inv=P(0x10004))), INVALID),
    (dict(r=ctypes.POINTER(binding.awq_rope_args)()), INVALID),
    (dict(Q=None), INVALID), (dict(Qo=None), INVALID), (dict(Qo=P(0x10008)), INVALID), (dict(K=None), INVALID),
    (dict(K=P(0x10008)), INVALID),
    (dict(Qo=P(addr(2).value + 16)), INVALID),                       # over Q, and not it
    (dict(Qo=addr(2), qos=512), INVALID),                            # in place with another stride
    (dict(Qo=addr(4)), INVALID), (dict(Qo=addr(12)), INVALID), (dict(Qo=P(addr(13).value + 240)), INVALID),
    (dict(qos=512, Qo=P(addr(4).value - 2 * 2 * 512)), INVALID),     # strided rows across K
]


@pytest.mark.parametrize("kw,status", ROPE_REFUSALS + [
    (dict(D=0), UNSUPPORTED), (dict(D=72), UNSUPPORTED), (dict(D=528, qs=1 << 20, qos=1 << 20), UNSUPPORTED),
    (dict(ks=120), INVALID), (dict(kos=130), INVALID), (dict(Ko=addr(3)), INVALID), (dict(Ko=addr(2)), INVALID),
    (dict(kv=-1), INVALID), (dict(Ko=None), INVALID),
])
def test_rope_refusals(kw, status):
    assert rope(**kw) == status
    assert "awq_rope" in lib.awq_last_error().decode()


@pytest.mark.parametrize("kw,status", ROPE_REFUSALS + [
    (dict(V=None), INVALID), (dict(slots=None), INVALID), (dict(vs=132), INVALID), (dict(nf=P(0x10001)), INVALID),
    (dict(Qo=P(0x10000)), INVALID), (dict(Qo=P(0x200000)), INVALID), (dict(Qo=P(0x300000)), INVALID),   # over the cache
    (dict(Qo=addr(5)), INVALID), (dict(Qo=addr(6)), INVALID), (dict(K=P(0x10000)), INVALID), (dict(Q=P(0x10000)), INVALID),
    (dict(r=args(pos=P(0x200000))), INVALID), (dict(nf=addr(12)), INVALID), (dict(nf=addr(3)), INVALID),
])
def test_append_rope_refusals(kw, status):
    assert append(**kw) == status
    assert "awq_kv_append_rope" in lib.awq_last_error().decode()


@pytest.mark.parametrize("kw,status", CACHE_REFUSALS)
def test_append_rope_cache_refusals(kw, status):
    assert append(c=cache(**kw)) == status


def test_nothing_to_do():
    none = dict(Q=None, Qo=None, K=None, T=0, r=args(pos=None, inv=None))
    assert rope(Ko=None, **none) == OK and append(V=None, slots=None, **none) == OK
    assert rope(heads=0, kv=0, Q=None, K=None) == OK


def test_binding_refuses_wrong_tensors():
    h = lambda *s: torch.zeros(s, dtype=torch.float16)   # noqa: E731
    inv = torch.zeros(32, dtype=torch.float64)
    ok = dict(Q=h(3, 4, 64), positions=i32(3), inv_freq=inv)
    for kw, e in ((dict(Q=h(3, 4, 64).float()), TypeError), (dict(Q=h(3, 256)), ValueError), (dict(Q=h(3, 4, 72)), ValueError),
                  (dict(positions=i32(4)), ValueError), (dict(positions=i32(3).long()), TypeError),
                  (dict(inv_freq=inv.float()), TypeError), (dict(inv_freq=inv[:12]), ValueError),
                  (dict(inv_freq=inv.view(2, 16)), ValueError), (dict(inv_freq=torch.zeros(40, dtype=torch.float64)), ValueError),
                  (dict(K=h(2, 2, 64)), ValueError), (dict(K=h(3, 2, 64).bfloat16()), TypeError), (dict(K=h(3, 2, 32)), ValueError),
                  (dict(out=h(3, 4, 32)), ValueError), (dict(out=h(3, 4, 64).float()), TypeError)):
        with pytest.raises(e):
            binding.awq_rope(**{**ok, **kw})
    with pytest.raises(ValueError, match="GPU"):
        binding.awq_rope(**ok)
    ok = dict(K=h(3, 2, 64), V=h(3, 2, 64), cache=tensors(), slots=i32(3), positions=i32(3), inv_freq=inv)
    for kw, e in ((dict(V=h(2, 2, 64)), ValueError), (dict(K=h(3, 1, 64)), ValueError), (dict(slots=i32(4)), ValueError),
                  (dict(Q=h(3, 4, 32)), ValueError), (dict(Q=h(2, 4, 64)), ValueError), (dict(out=h(3, 4, 64)), ValueError),
                  (dict(Q=h(3, 4, 64).bfloat16()), TypeError), (dict(nonfinite_count=i32(0)), ValueError)):
        with pytest.raises(e):
            binding.awq_kv_append_rope(**{**ok, **kw})
    with pytest.raises(ValueError, match="GPU"):
        binding.awq_kv_append_rope(**ok)
