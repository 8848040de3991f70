"""Rotary positions of many tokens, whose workgroups take many heads each: every lane then
walks several heads in several steps.  A sample of tokens is held against oracle/rope.py, and all
of them against the same tokens in small calls, whose workgroups take one step."""

import numpy as np
import pytest

from gpu_common import out_to_f64, say, torch_mod
from oracle import kv
from oracle.rope import frequencies, rotate32
from test_gpu_kv import _i32, _to_cache
from test_gpu_rope import _close, _freq, _input

pytestmark = pytest.mark.gpu

FEW = 97           # tokens of a small call: 25 workgroups along them, so parts of a step along the heads


@pytest.mark.parametrize("T,Hq,Hkv,D,R,interleaved,dtype", [
    (8200, 40, 9, 64, 64, False, "float16"), (8200, 20, 33, 80, 64, True, "bfloat16"),
    (8193, 9, 1, 512, 512, False, "bfloat16"), (8191, 17, 0, 128, 32, True, "float16"),
    (2100, 80, 40, 64, 48, False, "bfloat16"), (8200, 5, 5, 272, 144, False, "float16"),
])
def test_rope_of_many_heads(T, Hq, Hkv, D, R, interleaved, dtype):
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    say("rope of many heads", T, Hq, Hkv, D, R, interleaved, dtype)
    rng = np.random.default_rng(T + D)
    pos, inv = rng.integers(0, 1 << 20, T), frequencies(R)[0]
    (q, q32), (k, k32) = _input(rng, (T, Hq, D), dtype), _input(rng, (T, max(Hkv, 1), D), dtype)
    dp, df, kw = _i32(pos), _freq(inv), dict(interleaved=interleaved)
    gq, gk = awq.awq_rope(q, dp, df, K=k, **kw) if Hkv else (awq.awq_rope(q, dp, df, **kw), None)
    some = np.unique(np.concatenate([[0, 1, T - 2, T - 1], rng.integers(0, T, 60)]))
    _close(gq[some.tolist()], q32[some], pos[some], inv, dtype, 1.0, interleaved)
    if Hkv:
        _close(gk[some.tolist()], k32[some], pos[some], inv, dtype, 1.0, interleaved)
    for t in range(0, T, FEW):
        s = slice(t, min(t + FEW, T))
        assert torch.equal(awq.awq_rope(q[s], dp[s], df, **kw), gq[s])
        if Hkv:
            assert torch.equal(awq.awq_rope(k[s], dp[s], df, **kw), gk[s])
    got = awq.awq_rope(q, dp, df, K=k if Hkv else None, out=(q, k) if Hkv else q, **kw)    # in place
    assert torch.equal(q, gq) and (not Hkv or torch.equal(got[1], gk))


@pytest.mark.parametrize("T,Hq,Hkv,D,R,page,zp,dtype,interleaved", [
    (8200, 20, 9, 128, 128, 64, True, "float16", False), (8199, 0, 17, 64, 32, 16, False, "bfloat16", True),
    (8200, 3, 33, 64, 64, 128, True, "bfloat16", False), (2100, 8, 40, 128, 64, 1024, False, "float16", True),
])
def test_append_rope_of_many_heads(T, Hq, Hkv, D, R, page, zp, dtype, interleaved):
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    say("append_rope of many heads", T, Hq, Hkv, D, R, page, zp, dtype, interleaved)
    rng = np.random.default_rng(T + Hkv)
    pages = -(-T // page) + 2
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    slots[rng.random(T) < 0.1] = -1
    pos, (inv, factor) = rng.integers(0, 1 << 20, T), frequencies(R, 500000.0, "bands", 8.0, 8192.0)
    (K, k32), (V, v32) = _input(rng, (T, Hkv, D), dtype), _input(rng, (T, Hkv, D), dtype)
    Q = _input(rng, (T, Hq, D), dtype)[0] if Hq else None
    ds, dp, df = _i32(slots), _i32(pos), _freq(inv)
    kw = dict(attention_factor=factor, interleaved=interleaved)
    empty = kv.new_cache(pages, Hkv, D, page, zp)
    got, small = _to_cache(empty), _to_cache(empty)
    out = awq.awq_kv_append_rope(K, V, got, ds, dp, df, Q=Q, **kw)
    for t in range(0, T, FEW):
        s = slice(t, min(t + FEW, T))
        part = awq.awq_kv_append_rope(K[s], V[s], small, ds[s], dp[s], df, Q=Q[s] if Hq else None, **kw)
        assert part is None or torch.equal(part, out[s])
    assert all(a is b is None or torch.equal(a, b) for a, b in zip(got, small))
    if Hq:
        assert torch.equal(out, awq.awq_rope(Q, dp, df, **kw))
    some = np.unique(np.concatenate([[0, T - 1], rng.integers(0, T, 60)]))
    kv.append(empty, rotate32(k32[some], pos[some], inv, factor, interleaved), v32[some], slots[some])
    there = [int(s) for s in slots[some] if s >= 0]
    host = (got[0].cpu().numpy().view(np.uint32), got[1].cpu().numpy(), None if got[2] is None else got[2].cpu().numpy())
    for x, y in zip(kv.read(host, D, there), kv.read(empty, D, there)):
        assert np.array_equal(x, y)
    assert np.isfinite(out_to_f64(got[1])).all()
