"""Calls of the key/value cache whose outputs or workspace lie over what they read, or
over the cache, are refused before any HIP call: no GPU needed."""

import pytest

from test_kv_abi_cpu import INVALID, P, addr, append, attend, gather, lib

# cache(): codes of 16 KiB at 0x10000, scales of 1 KiB at 0x200000, zeros of 512 bytes at 0x300000
CACHE = {"codes, first byte": 0x10000, "codes, last bytes": 0x10000 + 16384 - 16, "scales": 0x200000 + 1024 - 16,
         "zeros": 0x300000 + 512 - 16}


def refused(status, who):
    return status == INVALID and "overlap" in lib.awq_last_error().decode() and who in lib.awq_last_error().decode()


@pytest.mark.parametrize("at", CACHE.values(), ids=CACHE.keys())
def test_attention_over_the_cache(at):
    assert refused(attend(O=P(at)), "awq_kv_attention")
    assert refused(attend(lse=P(at)), "awq_kv_attention")
    big = dict(T=1, B=1, mk=60000, wsb=1 << 40)
    assert refused(attend(ws=P(at & ~255), **big), "awq_kv_attention")


@pytest.mark.parametrize("what,at,size", [("Q", 7, 3 * 256 * 2), ("table", 8, 3 * 4 * 4), ("lens", 9, 3 * 4),
                                          ("start", 11, 4 * 4)])
def test_attention_over_what_it_reads(what, at, size):
    kw = dict(start=addr(11)) if what == "start" else {}
    last = (size - 4) & ~15
    for p in (P(addr(at).value), P(addr(at).value + last), P(addr(at).value - 16)):
        assert refused(attend(O=p, **kw), "awq_kv_attention"), p
    assert refused(attend(lse=P(addr(at).value + size - 4), **kw), "awq_kv_attention")
    kw = dict(T=1, B=1, mk=60000, wsb=1 << 40, **({"start": addr(11), "mq": 1} if what == "start" else {}))
    assert refused(attend(ws=addr(at), **kw), "awq_kv_attention")


def test_attention_over_the_gaps_between_strided_queries():
    """Q's extent is counted to its last element: a token's own heads may be a slice."""
    assert refused(attend(qs=1024, O=P(addr(7).value + 2 * 1024 * 2)), "awq_kv_attention")


@pytest.mark.parametrize("at", CACHE.values(), ids=CACHE.keys())
def test_append_of_the_cache_itself(at):
    assert refused(append(K=P(at)), "awq_kv_append")
    assert refused(append(V=P(at)), "awq_kv_append")
    assert refused(append(slots=P(at)), "awq_kv_append")
    assert refused(append(nf=P(at)), "awq_kv_append")


def test_append_counts_into_its_inputs():
    for p in (addr(4).value, addr(5).value + 3 * 128 * 2, addr(6).value + 12):
        assert refused(append(nf=P(p)), "awq_kv_append")


def test_cache_arrays_over_each_other():
    from test_kv_abi_cpu import cache
    for kw in (dict(scales=0x10000 + 16384 - 16), dict(zeros=0x10000), dict(zeros=0x200000 + 512)):
        assert refused(append(c=cache(**kw)), "awq_kv_append")


@pytest.mark.parametrize("at", CACHE.values(), ids=CACHE.keys())
def test_gather_into_the_cache(at):
    assert refused(gather(K=P(at)), "awq_kv_gather")
    assert refused(gather(V=P(at)), "awq_kv_gather")


def test_gather_into_its_slots():
    assert refused(gather(K=addr(6)), "awq_kv_gather")
    assert refused(gather(V=P(addr(6).value - 16)), "awq_kv_gather")
