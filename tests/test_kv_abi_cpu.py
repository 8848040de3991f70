"""Refusals of the key/value cache and epilogue entry points, before any HIP call:
no GPU needed.  Valid calls here are those with nothing to do."""

import ctypes

import pytest

binding = pytest.importorskip("bit_weight_only_quantize_amd.binding",
                              reason="libawq355.so not built")
lib = binding.lib
cfg = binding.config
P = ctypes.c_void_p
INVALID, UNSUPPORTED, WORKSPACE = (binding.AWQ_ERR_INVALID_ARG, binding.AWQ_ERR_UNSUPPORTED,
                                   binding.AWQ_ERR_WORKSPACE)


def addr(i):
    return P(0x10000 + (i << 20))           # aligned, apart, never dereferenced


def cache(**k):
    c = binding.awq_kv_cache(0x10000, 0x200000, 0x300000, 8, 16, 2, 64)
    for n, v in k.items():
        setattr(c, n, v)
    return ctypes.byref(c)


def assign(B=3, page=16, blocks=4, free=5, slots=7, p=None):
    a = [addr(i) for i in range(8)]         # old new table free seq start slots used
    for i, v in (p or {}).items():
        a[i] = v
    return lib.awq_kv_assign(a[0], a[1], B, page, a[2], blocks, a[3], free, a[4], a[5], a[6], slots,
                             a[7], None)


@pytest.mark.parametrize("kw,status", [
    (dict(page=8), UNSUPPORTED), (dict(page=48), UNSUPPORTED), (dict(page=2048), UNSUPPORTED),
    (dict(page=0), UNSUPPORTED), (dict(page=-16), UNSUPPORTED),
    (dict(B=-1), INVALID), (dict(blocks=-1), INVALID), (dict(free=-1), INVALID), (dict(slots=-1), INVALID),
    (dict(slots=2 ** 31), INVALID), (dict(blocks=2 ** 27), UNSUPPORTED),
    *[(dict(p={i: None}), INVALID) for i in range(8)],
    (dict(p={0: P(0x10002)}), INVALID),                      # misaligned
    (dict(p={4: addr(0)}), INVALID),                         # lengths updated in place
    (dict(p={6: P(0x10000 + (3 << 20) + 16)}), INVALID),     # slots over the free list
    (dict(p={7: addr(5)}), INVALID),                         # two outputs in one place
])
def test_assign_refusals(kw, status):
    assert assign(**kw) == status
    assert "awq_kv_assign" in lib.awq_last_error().decode()


CACHE_REFUSALS = [
    (dict(head_dim=80), UNSUPPORTED), (dict(head_dim=128), UNSUPPORTED),   # group_size stays 64
    (dict(page_size=24), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED),
    (dict(num_kv_heads=0), INVALID), (dict(num_kv_heads=2000), INVALID),
    (dict(num_pages=0), INVALID), (dict(num_pages=2 ** 28), UNSUPPORTED),
    (dict(codes=None), INVALID), (dict(scales=None), INVALID), (dict(zeros=None), INVALID),
    (dict(codes=0x10004), INVALID),
]


def append(c=None, T=4, ks=128, vs=128, xt=0, K=addr(4), V=addr(5), slots=addr(6), nf=None, conf=None):
    return lib.awq_kv_append(K, V, xt, T, ks, vs, cache() if c is None else c, conf or cfg(64), slots, nf, None)


def gather(c=None, T=4, ot=2, K=addr(4), V=addr(5), slots=addr(6), conf=None):
    return lib.awq_kv_gather(cache() if c is None else c, conf or cfg(64), slots, T, K, V, ot, None)


def attend(c=None, T=3, B=3, heads=4, qs=256, qt=0, conf=None, Q=addr(7), table=addr(8), blocks=4,
           lens=addr(9), start=None, mq=1, mk=64, scale=0.1, causal=1, window=0, O=addr(10), lse=None,
           ws=None, wsb=0):
    return lib.awq_kv_attention(Q, qt, T, qs, heads, cache() if c is None else c, conf or cfg(64), table, blocks, lens,
                                start, B, mq, mk, scale, causal, window, O, lse, ws, wsb, None)


@pytest.mark.parametrize("kw,status", CACHE_REFUSALS)
@pytest.mark.parametrize("call", [append, gather, attend])
def test_cache_refusals(call, kw, status):
    assert call(c=cache(**kw)) == status


@pytest.mark.parametrize("call", [append, gather, attend])
def test_config_refusals(call):
    assert call(conf=cfg(64, w_bit=8)) == UNSUPPORTED
    assert call(conf=cfg(128)) == UNSUPPORTED                # a token's head is one group
    assert call(conf=binding.awq_config(4, 64, 3)) == INVALID
    assert call(c=ctypes.POINTER(binding.awq_kv_cache)()) == INVALID


def test_append_refusals():
    assert append(xt=2) == INVALID
    assert append(T=-1) == INVALID and append(T=2 ** 31) == INVALID
    assert append(ks=120) == INVALID and append(vs=132) == INVALID      # too short; not of 16 bytes
    assert append(K=None) == INVALID and append(slots=None) == INVALID
    assert append(K=P(0x10008)) == INVALID and append(nf=P(0x10001)) == INVALID
    assert append(T=0, K=None, V=None, slots=None) == binding.AWQ_OK


def test_gather_refusals():
    assert gather(ot=3) == INVALID and gather(T=-1) == INVALID
    assert gather(K=None) == INVALID and gather(V=P(0x10008)) == INVALID
    assert gather(T=0, K=None, V=None, slots=None) == binding.AWQ_OK


@pytest.mark.parametrize("kw,status", [
    (dict(qt=2), INVALID), (dict(T=-1), INVALID), (dict(B=-1), INVALID), (dict(heads=3), INVALID),
    (dict(heads=0), INVALID), (dict(heads=4096, qs=1 << 20), INVALID), (dict(qs=250), INVALID),
    (dict(qs=260), INVALID), (dict(mq=-1), INVALID), (dict(mk=-1), INVALID),
    (dict(mq=2 ** 30, start=addr(11)), UNSUPPORTED), (dict(B=65536, T=65536), UNSUPPORTED),
    (dict(causal=2), INVALID), (dict(window=-1), INVALID), (dict(window=5, causal=0), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(blocks=-1), INVALID), (dict(blocks=2 ** 28), INVALID),
    (dict(T=4), INVALID), (dict(mq=2), INVALID),             # without query_start: one token each
    (dict(Q=None), INVALID), (dict(O=None), INVALID), (dict(lens=None), INVALID), (dict(table=None), INVALID),
    (dict(Q=P(0x10008)), INVALID), (dict(lse=P(0x10002)), INVALID), (dict(start=P(0x10001), T=5), INVALID),
    (dict(ws=P(0x10010), wsb=64), INVALID),                  # misaligned
    (dict(O=addr(7)), INVALID),                              # over Q
])
def test_attention_refusals(kw, status):
    assert attend(**kw) == status
    assert "awq_kv_attention" in lib.awq_last_error().decode()


@pytest.mark.parametrize("kw,status", [
    (dict(blocks=2 ** 26 + 1), INVALID),                     # 2^30 tokens and a page
    (dict(lse=P(addr(10).value + 1024)), INVALID),           # lse within O
    (dict(T=1, B=1, mk=60000, ws=P(addr(10).value - 4096), wsb=1 << 40), INVALID),
    (dict(T=1, B=1, mk=60000, ws=P(addr(9).value - 65536), wsb=1 << 40, lse=addr(9), lens=addr(12)), INVALID),
])
def test_attention_refuses_long_tables_and_overlaps(kw, status):
    assert attend(**kw) == status
    assert "awq_kv_attention" in lib.awq_last_error().decode()


def test_append_and_gather_refuse_what_a_grid_cannot_hold():
    assert append(T=2 ** 27 + 1) == INVALID and gather(T=2 ** 27 + 1) == INVALID
    assert gather(V=P(addr(4).value + 16)) == INVALID        # over K


def test_attention_workspace_of_no_more_query_tokens_than_there_are():
    size = lambda n, m: lib.awq_kv_attention_workspace_size(n, 1, 4, cache(), cfg(64), m, 60000, 0)  # noqa: E731
    for n in (1, 5, 40, 700):
        assert size(n, n) == size(n, 10 ** 8) > 0


def test_attention_workspace():
    size = lambda *a: lib.awq_kv_attention_workspace_size(a[0], a[1], 4, cache(), cfg(64), *a[2:])  # noqa: E731
    need = size(1, 1, 1, 60000, 0)
    assert need > 0 and need % 4 == 0
    assert size(1, 1, 1, 100, 0) == 0 and size(0, 0, 0, 60000, 0) == 0
    assert size(1, 1, 1, 60000, 100) == 0                   # a window bounds what a row sees
    assert size(1, 1, 1, 60000, -1) == 0 and size(-1, 1, 1, 60000, 0) == 0
    assert attend(T=1, B=1, mk=60000) == WORKSPACE
    assert attend(T=1, B=1, mk=60000, ws=P(0x100000000), wsb=need - 1) == WORKSPACE
    for kw in (dict(T=0, B=0), dict(mq=0, start=addr(11))):  # nothing to do
        assert attend(Q=None, O=None, lens=None, table=None, **kw) == binding.AWQ_OK


def test_epilogue_refusals():
    def call(epi, M=3, K=256, yt=0, kernel=0, Y=addr(5), ws=None, wsb=0):
        return lib.awq_linear_epilogue(addr(0), 0, addr(1), addr(2), addr(3), M, 64, K, cfg(128), epi, Y, yt,
                                       kernel, ws, wsb, None)
    E = binding.awq_epilogue
    assert call(None) == INVALID
    assert call(ctypes.byref(E(None, None, 5))) == INVALID and call(ctypes.byref(E(None, None, -1))) == INVALID
    assert call(ctypes.byref(E(0x10001, None, 0))) == INVALID           # bias misaligned
    assert call(ctypes.byref(E(None, 0x10002, 0)), yt=2) == INVALID     # residual of fp32
    fine = ctypes.byref(E(0x10000, 0x20000, 3))
    assert call(fine, K=200) == INVALID and call(fine, yt=9) == INVALID and call(fine, Y=None) == INVALID
    assert call(fine, M=17, kernel=1) == INVALID
    assert call(ctypes.byref(E(addr(5).value + 16, None, 0))) == INVALID     # bias within Y
    assert call(ctypes.byref(E(None, addr(5).value + 2, 0))) == INVALID      # residual across Y
    assert call(fine, M=0) == binding.AWQ_OK


# ---- the binding: wrong tensors raise, with or without a GPU ---------------------------

torch = pytest.importorskip("torch")


def tensors(page=16, D=64, H=2, pages=4, zp=True):
    return (torch.zeros((pages, 2, H, page * D // 8), dtype=torch.int32),
            torch.zeros((pages, H, page, 2), dtype=torch.float16),
            torch.zeros((pages, H, page, 2), dtype=torch.uint8) if zp else None)


def i32(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_binding_refuses_wrong_tensors():
    c = tensors()
    kvt = torch.zeros((3, 2, 64), dtype=torch.float16)
    for bad in ((c[0],), c[:2], "cache"):
        with pytest.raises(TypeError):
            binding.awq_kv_append(kvt, kvt, bad, i32(3))
    for bad in ((c[0].float(), c[1], c[2]), (c[0], c[1].float(), c[2]), (c[0], c[1], c[2].float())):
        with pytest.raises(TypeError):
            binding.awq_kv_gather(bad, i32(3))
    for bad in ((c[0][:, 0], c[1], c[2]), (c[0], c[1][:3], c[2]), (c[0], c[1], c[2][:, :1]),
                (c[0][..., :100], c[1], c[2]), tensors(page=24), tensors(D=32)):
        with pytest.raises(ValueError):
            binding.awq_kv_gather(bad, i32(3))
    with pytest.raises(ValueError):
        binding.awq_kv_append(kvt[:, :1], kvt, c, i32(3))
    with pytest.raises(TypeError):
        binding.awq_kv_append(kvt.float(), kvt, c, i32(3))
    with pytest.raises(ValueError, match="GPU"):
        binding.awq_kv_append(kvt, kvt, c, i32(3))
    for size in ((0, 2, 64, 16), (4, 2, 96, 16), (4, 2, 64, 20), (4, 0, 64, 16), (4, 2, 64, 2048)):
        with pytest.raises(ValueError):
            binding.empty_kv_cache(*size, device="cpu")


def test_binding_refuses_wrong_assignments():
    ok = dict(old_lens=i32(3), new_lens=i32(3), block_table=i32(3, 4), free_pages=i32(5), page_size=16, num_slots=9)
    for k, v, e in (("old_lens", i32(3).long(), TypeError), ("new_lens", i32(4), ValueError),
                    ("block_table", i32(12), ValueError), ("block_table", i32(2, 4), ValueError),
                    ("free_pages", [1, 2], TypeError), ("num_slots", -1, ValueError)):
        with pytest.raises(e):
            binding.awq_kv_assign(**{**ok, k: v})
    with pytest.raises(ValueError):
        binding.awq_kv_assign(**ok, out=(i32(3), i32(3), i32(9), i32(1)))
    with pytest.raises(ValueError, match="GPU"):
        binding.awq_kv_assign(**ok)


def test_binding_refuses_wrong_attention():
    c = tensors()
    Q = torch.zeros((3, 4, 64), dtype=torch.bfloat16)
    ok = dict(Q=Q, cache=c, block_table=i32(3, 4), seq_lens=i32(3))
    for k, v, e in (("Q", Q.float(), TypeError), ("Q", Q[..., :32], ValueError), ("Q", Q[:, :3], ValueError),
                    ("Q", Q[:2], ValueError), ("block_table", i32(12), ValueError),
                    ("seq_lens", i32(2), ValueError), ("query_start", i32(3), ValueError),
                    ("max_query_len", 2, ValueError), ("out", Q.half(), TypeError),
                    ("workspace", "some", ValueError)):
        with pytest.raises(e):
            binding.awq_kv_attention(**{**ok, k: v})
    with pytest.raises(ValueError, match="GPU"):
        binding.awq_kv_attention(**ok)


def test_binding_refuses_wrong_epilogues():
    X = torch.zeros((3, 128), dtype=torch.float16)
    w = (i32(16, 16), torch.zeros((16, 1), dtype=torch.float16), torch.zeros((16, 1), dtype=torch.uint8))
    h = lambda *s: torch.zeros(s, dtype=torch.float16)   # noqa: E731
    for kw, e in ((dict(activation="tanh"), ValueError), (dict(bias=h(17)), ValueError),
                  (dict(bias=h(16).float()), TypeError), (dict(bias=h(16, 1)), ValueError),
                  (dict(residual=h(3, 17)), ValueError), (dict(residual=h(3, 16).float()), TypeError),
                  (dict(residual=h(48)), ValueError), (dict(workspace="x"), ValueError),
                  (dict(out=h(3, 17)), ValueError), (dict(out_dtype=torch.int32), TypeError)):
        with pytest.raises(e):
            binding.awq_linear_epilogue(X, *w, **kw)
    with pytest.raises(ValueError, match="GPU"):
        binding.awq_linear_epilogue(X, *w, bias=h(16))
