"""Measured cases of rotary positions, the page operations of the 4-bit
key/value cache, and its attention with a window and sinks or with a prefix that
the batch shares.

``run`` computes each operator either in its plain form (elementary torch
operations in 32 bits, angles in 64, rounded once at the end) or, where ``own``
is true, with the library's entry points.  Both take the same inputs from
``prepare``.
"""

import math
import random

import numpy as np
import torch

own = False

#: Bit position of channel i of a packed word's 8 channels.
SHIFTS = tuple(4 * ((i >> 1) + 4 * (i & 1)) for i in range(8))
DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


# ---- the cases -----------------------------------------------------------------

def listed():
    return [
        # one decode step: queries and keys are rotated, keys and values go to the cache (70B-class heads)
        dict(name="rope_append_step_t32_64x8_d128", op="rope_append", T=32, Hq=64, Hkv=8, D=128, R=128, page=64,
             dtype="f16", zero_point=True, interleaved=False, scaling="none", far=4000),
        # the prompts of a step, 7B-class heads
        dict(name="rope_append_prompt_t8192_32x32_d128", op="rope_append", T=8192, Hq=32, Hkv=32, D=128, R=128,
             page=64, dtype="bf16", zero_point=True, interleaved=False, scaling="none", far=8192),
        # half of each head, neighbouring channels paired, a context stretched far beyond training
        dict(name="rope_t4097_32x8_d128_r64_pairs", op="rope", T=4097, Hq=32, Hkv=8, D=128, R=64, dtype="bf16",
             interleaved=True, scaling="yarn", far=131072),
        # four samples of each of two prompts branch off and end again
        dict(name="fork_release_n8_l1500", op="fork", B=24, n=8, most=1500, page=64, heads=8, D=128, zero_point=True,
             key=1),
        # many branches of long contexts, small pages
        dict(name="fork_release_n200_l20000", op="fork", B=500, n=200, most=20000, page=16, heads=2, D=128,
             zero_point=True, key=2),
        # pages of requests that are put aside, moved within the pool
        dict(name="copy_pages_n2000_h8_d128", op="copy", n=2000, page=64, heads=8, D=128, zero_point=True),
        # a pool that has come apart is drawn together, so that its tail can be given back
        dict(name="compact_b96_l6000_h8_d128", op="compact", B=96, most=6000, spare=0.6, page=64, heads=8, D=128,
             zero_point=False, key=3),
        # decoding of long conversations that keep their first tokens and the last few thousand
        dict(name="sinks_decode_b32_l20000_w4096", op="sinks", B=32, q_most=1, k_most=20000, window=4096, sinks=4,
             Hq=32, Hkv=8, D=128, page=64, dtype="f16", zero_point=True, key=4),
        # one long prompt, each token with its last 1024 and the first 64
        dict(name="sinks_prompt_q8192_w1024", op="sinks", B=1, q_most=8192, k_most=8192, window=1024, sinks=64,
             Hq=32, Hkv=8, D=128, page=64, dtype="bf16", zero_point=True, key=5),
        # a few requests behind one system prompt, drafts of up to 4 tokens
        dict(name="prefix_b8_p2000_s300_q4", op="prefix", B=8, q_most=4, prefix=2000, s_most=300, Hq=32, Hkv=8,
             D=128, page=16, dtype="f16", zero_point=True, pad=True, key=6),
        # a serving batch behind a long instruction, 7B-class heads without sharing
        dict(name="prefix_b64_p8192_s1000_32x32", op="prefix", B=64, q_most=1, prefix=8192, s_most=1000, Hq=32,
             Hkv=32, D=128, page=64, dtype="f16", zero_point=True, pad=False, key=7),
        # questions about one long document, 70B-class heads
        dict(name="prefix_b48_p32768_s2000_64x8", op="prefix", B=48, q_most=1, prefix=32768, s_most=2000, Hq=64,
             Hkv=8, D=128, page=128, dtype="bf16", zero_point=False, pad=False, key=8),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rope_append", "rope_append", "rope", "fork", "copy", "compact", "sinks", "sinks", "prefix",
                     "prefix"))
    key = rng.randrange(1 << 30)
    page = rng.choice((16, 32, 64, 128))
    dtype = rng.choice(("f16", "bf16"))
    zero_point = rng.random() < 0.7
    if op in ("rope_append", "rope"):
        Hkv = rng.choice((1, 2, 4, 8, 8, 16, 32))
        Hq = Hkv * rng.choice((1, 2, 4, 7)) if Hkv < 16 else Hkv
        D = rng.choice((64, 128, 128)) if op == "rope_append" else rng.choice((64, 80, 96, 128, 256))
        R = rng.choice((D, D, 16 * rng.randint(1, D // 16)))
        far = _log(rng, 100, 1000000)
        case = dict(op=op, T=_log(rng, 1, 8192 * 96 * 128 // max((Hq + 2 * Hkv) * D, 96 * 128)), Hq=Hq, Hkv=Hkv, D=D,
                    R=R, dtype=dtype, interleaved=rng.random() < 0.4,
                    scaling=rng.choice(("none", "none", "linear", "yarn")), far=far)
        return case | (dict(page=page, zero_point=zero_point) if op == "rope_append" else {})
    heads, D = rng.choice((1, 2, 4, 8)), rng.choice((64, 128))
    if op == "fork":
        B = _log(rng, 2, 600)
        return dict(op="fork", B=B, n=_log(rng, 1, max(1, B // 2)), most=_log(rng, 30, 20000), page=page,
                    heads=min(heads, 2), D=D, zero_point=zero_point, key=key)
    if op == "copy":
        return dict(op="copy", n=_log(rng, 1, 2000 * 64 * 8 * 128 // (page * heads * D) // 2), page=page, heads=heads,
                    D=D, zero_point=zero_point)
    if op == "compact":
        return dict(op="compact", B=_log(rng, 2, 96), most=_log(rng, 50, 6000), spare=rng.choice((0.1, 0.5, 0.9)),
                    page=page, heads=heads, D=D, zero_point=zero_point, key=key)
    Hkv = rng.choice((1, 2, 4, 8, 8, 16, 32))
    D = rng.choice((64, 128, 128))
    shared = rng.choice((1, 2, 4, 5, 7, 8))
    while Hkv * shared > 64:
        shared = max(1, shared // 2)
    if op == "sinks":
        if rng.random() < 0.5:
            B, q_most = _log(rng, 1, 48), rng.choice((1, 1, 1, 3, 4))
            k_most = _log(rng, 40, max(100, min(40000, 20000 * 32 * 8 // (B * Hkv))))
        else:
            B = _log(rng, 1, 8)
            q_most = _log(rng, 20, max(100, 4096 // B))
            k_most = _log(rng, q_most, max(q_most, min(16384, 32 * 8192 * 4096 // (Hkv * shared * q_most * B))))
        return dict(op="sinks", B=B, q_most=q_most, k_most=k_most, window=_log(rng, 1, max(1, k_most)),
                    sinks=rng.choice((1, 4, 4, 33, 128)), Hq=Hkv * shared, Hkv=Hkv, D=D, page=page, dtype=dtype,
                    zero_point=zero_point, key=key)
    B, q_most = _log(rng, 1, 64), rng.choice((1, 1, 1, 4, 30))
    rows = B * q_most * Hkv * shared
    prefix = _log(rng, 20, max(100, min(40000, 32768 * 48 * 64 // rows)))
    return dict(op="prefix", B=B, q_most=q_most, prefix=prefix, s_most=_log(rng, q_most + 1, max(40, 60000 // B)),
                Hq=Hkv * shared, Hkv=Hkv, D=D, page=page, dtype=dtype, zero_point=zero_point,
                pad=rng.random() < 0.3, key=key)


# ---- lengths of a case's requests (from the case alone) ----------------------------

def _lengths(case):
    """(query lengths, key lengths) of an attention case; the first request has the most of both.
    Keys of a prefix case are counted with the prefix; a padded batch ends in a request of none."""
    r = random.Random(case["key"])
    base = case["prefix"] if case["op"] == "prefix" else 0
    k_most = case["s_most"] if case["op"] == "prefix" else case["k_most"]
    q, k = [case["q_most"]], [base + k_most]
    for _ in range(case["B"] - 1):
        n = 1 if case["q_most"] == 1 else r.randint(1, case["q_most"])
        q.append(n)
        k.append(base + r.randint(min(n, k_most), k_most))
    if case.get("pad") and case["B"] > 1:
        k[-1] = 0
    return q, k


def _page_lengths(case):
    """Cached tokens of each request of a fork or compact case."""
    r = random.Random(case["key"])
    return [r.randint(1, case["most"]) for _ in range(case["B"])]


def _forks(case):
    """(parents, children, shared tokens): the children are the table's last rows."""
    r = random.Random(case["key"] + 1)
    lens, n = _page_lengths(case), case["n"]
    few = max(1, min(case["B"] - n, n // 4))
    parents = [r.randrange(few) for _ in range(n)]
    return parents, list(range(case["B"] - n, case["B"])), [r.randint(max(1, lens[p] // 2), lens[p]) for p in parents]


def _seen(q, k, case):
    """Query-key pairs of a request of q new tokens and k in all, and keys that any of them sees."""
    p = np.arange(max(k - q, 0) + 1, k + 1, dtype=np.int64)            # keys up to each query
    if case["op"] == "prefix":
        return int(p.sum()), max(0, k - case["prefix"])
    w, s = case["window"], case["sinks"]
    return int((np.minimum(p, w) + np.clip(p - w, 0, s)).sum()), min(k, q + w - 1 + s)


# ---- inputs -----------------------------------------------------------------------

def _normal(shape, gen, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda") * scale


def _cache_like(x, gen, spread):
    """Key- or value-like vectors [n][heads][D]: some channels shifted and larger, as keys have."""
    heads, D = x.shape[-2:]
    gain = torch.where(torch.rand((heads, D), generator=gen, device="cuda") < 0.03, spread, 1.0)
    shift = _normal((heads, D), gen, 0.3)
    return x * gain + shift


def _frequencies(case):
    """Radians per position of each pair (64 bits), and the factor on queries and keys."""
    R, base = case["R"], 10000.0
    f = base ** (-np.arange(0, R, 2, dtype=np.float64) / R)
    if case["scaling"] == "linear":
        return f / 4.0, 1.0
    if case["scaling"] == "yarn":                  # far pairs interpolated, near ones kept, a ramp between
        s, trained = 32.0, 4096.0
        turn = lambda n: R * math.log(trained / (n * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
        lo, hi = max(math.floor(turn(32.0)), 0), min(math.ceil(turn(1.0)), R - 1)
        ramp = np.clip((np.arange(R // 2) - lo) / max(hi - lo, 0.001), 0, 1)
        return f / s * ramp + f * (1 - ramp), 0.1 * math.log(s) + 1
    return f, 1.0


def _quantize(x, zero_point):
    """Group quantization of the last dimension: (codes, scale fp16, zero) of fp32 values."""
    if zero_point:
        lo = x.amin(-1, keepdim=True).clamp(max=0)
        hi = x.amax(-1, keepdim=True).clamp(min=0)
        scale = ((hi - lo) / 15).clamp(min=2.0 ** -14).half()
        zero = torch.round(-lo / scale.float()).clamp(0, 15)
        codes = (torch.round(x / scale.float()) + zero).clamp(0, 15)
        return codes.int(), scale[..., 0], zero[..., 0].to(torch.uint8)
    scale = (x.abs().amax(-1, keepdim=True) / 7).clamp(min=2.0 ** -14).half()
    codes = torch.round(x / scale.float()).clamp(-8, 7) + 8
    return codes.int(), scale[..., 0], None


def _pack(codes):
    """Codes [..., n] as words [..., n/8]."""
    shifts = torch.tensor(SHIFTS, dtype=torch.int32, device=codes.device)
    return (codes.unflatten(-1, (-1, 8)) << shifts).sum(-1, dtype=torch.int32)


def _unpack(words):
    shifts = torch.tensor(SHIFTS, dtype=torch.int32, device=words.device)
    return ((words.unsqueeze(-1) >> shifts) & 15).flatten(-2)


def _new_cache(pages, heads, D, page, zero_point, gen):
    """A cache whose unused slots hold what an earlier request left there."""
    codes = torch.randint(-2 ** 31, 2 ** 31 - 1, (pages, 2, heads, page * D // 8), generator=gen,
                          device="cuda", dtype=torch.int64).int()
    scales = (torch.rand((pages, heads, page, 2), generator=gen, device="cuda") + 0.1).half()
    zeros = (torch.randint(0, 16, (pages, heads, page, 2), generator=gen, device="cuda",
                           dtype=torch.uint8) if zero_point else None)
    return codes, scales, zeros


def _write(cache, D, slots, K, V):
    """K, V [n][heads][D] into the cache's slots."""
    codes, scales, zeros = cache
    page = scales.shape[2]
    slots = slots.long()
    at, off = slots // page, slots % page
    kc, ks, kz = _quantize(K.float(), zeros is not None)
    vc, vs, vz = _quantize(V.float(), zeros is not None)
    k_view = codes.view(codes.shape[0], 2, -1, page, D // 8)
    v_view = codes.view(codes.shape[0], 2, -1, page // 4, D // 8, 4)
    k_view[at, 0, :, off] = _pack(kc)
    v_view[at, 1, :, off // 4, :, off % 4] = _pack(vc)
    scales[at, :, off] = torch.stack((ks, vs), -1)
    if zeros is not None:
        zeros[at, :, off] = torch.stack((kz, vz), -1)


def _read(cache, D, slots):
    """The values that the cache's slots stand for, fp32 [n][heads][D] twice (0 for slots below 0)."""
    codes, scales, zeros = cache
    page = scales.shape[2]
    keep = (slots >= 0)[:, None, None]
    slots = slots.clamp(min=0).long()
    at, off = slots // page, slots % page
    k = _unpack(codes.view(codes.shape[0], 2, -1, page, D // 8)[at, 0, :, off])
    v = _unpack(codes.view(codes.shape[0], 2, -1, page // 4, D // 8, 4)[at, 1, :, off // 4, :, off % 4])
    s = scales[at, :, off].float()
    z = zeros[at, :, off].float() if zeros is not None else torch.full_like(s, 8.0)
    k = (k.float() - z[..., :1]) * s[..., :1]
    v = (v.float() - z[..., 1:]) * s[..., 1:]
    return torch.where(keep, k, 0.0), torch.where(keep, v, 0.0)


def _tables(lens, page, pages, order, blocks=0):
    """Block table of requests of these lengths with pages in the given order (int32 on the GPU, -1 behind)."""
    need = [-(-n // page) for n in lens]
    table = np.full((len(lens), max(max(need), blocks)), -1, np.int32)
    used = 0
    for b, n in enumerate(need):
        table[b, :n] = order[used:used + n]
        used += n
    return torch.from_numpy(table).cuda(), used


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state = dict(case)
    op = case["op"]
    if op in ("rope", "rope_append"):
        T, D, dt = case["T"], case["D"], DTYPES[case["dtype"]]
        freq, factor = _frequencies(case)
        first = torch.randint(0, max(1, case["far"] - T), (1,), generator=gen, device="cuda")
        pos = (torch.randint(0, case["far"], (T,), generator=gen, device="cuda") if T <= 256
               else first + torch.arange(T, device="cuda"))        # a decode step's tokens, or a chunk's
        state |= dict(pos=pos.int(), freq=torch.from_numpy(freq).cuda(), factor=factor,
                      Q=_normal((T, case["Hq"], D), gen).to(dt),
                      K=_cache_like(_normal((T, case["Hkv"], D), gen), gen, 4.0).to(dt))
        if op == "rope_append":
            page = case["page"]
            pages = -(-T // page) + 8
            slots = torch.randperm(pages, generator=gen, device="cuda").int()[:, None] * page + torch.arange(
                page, dtype=torch.int32, device="cuda")
            if T <= 256:
                slots = slots.flatten()[torch.randperm(pages * page, generator=gen, device="cuda")]
            state |= dict(cache=_new_cache(pages, case["Hkv"], D, page, case["zero_point"], gen),
                          slots=slots.flatten()[:T].contiguous(),
                          V=_cache_like(_normal((T, case["Hkv"], D), gen), gen, 1.0).to(dt))
        return state
    shape = (case.get("heads", case.get("Hkv")), case["D"], case["page"], case["zero_point"])
    if op == "copy":
        n = case["n"]
        order = torch.randperm(2 * n + 50, generator=gen, device="cuda").int()
        state |= dict(cache=_new_cache(2 * n + 50, *shape, gen), src=order[:n].clone(), dst=order[n:2 * n].clone())
        return state
    if op in ("fork", "compact"):
        lens = _page_lengths(case)
        if op == "fork":
            parents, children, share = _forks(case)
            lens = [0 if b in set(children) else n for b, n in enumerate(lens)]
        held = sum(-(-n // case["page"]) for n in lens)
        extra = case["n"] + 60 if op == "fork" else int(held * case["spare"]) + 3
        pages = held + extra
        order = torch.randperm(pages, generator=gen, device="cuda").int()
        table, used = _tables(lens, case["page"], pages, order.cpu().numpy(), -(-case["most"] // case["page"]) + 2)
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        state |= dict(cache=_new_cache(pages, *shape, gen), table=table, lens=i32(lens),
                      shared=torch.zeros(pages, dtype=torch.int32, device="cuda"))
        if op == "fork":
            ends = list(lens)
            for c, n in zip(children, share):
                ends[c] = n
            keep = [0 if b in set(children) else n for b, n in enumerate(lens)]
            state |= dict(free=order[used:].clone(), parents=i32(parents), children=i32(children), share=i32(share),
                          ends=i32(ends), keep=i32(keep))
        return state
    q, k = _lengths(case)
    B, Hkv, D, page, prefix = case["B"], case["Hkv"], case["D"], case["page"], case.get("prefix", 0)
    # pages of the prefix's full blocks are the same in every row; the block that it ends in is each request's own
    # but for its first tokens, which are equal
    same = prefix // page
    need = [max(0, -(-n // page) - same) for n in k]
    pages = sum(need) + same + 5
    cache = _new_cache(pages, Hkv, D, page, case["zero_point"], gen)
    order = torch.randperm(pages, generator=gen, device="cuda").int()
    table = torch.full((B, same + max(need)), -1, dtype=torch.int32, device="cuda")
    table[:, :same] = order[:same]
    offs = torch.arange(page, dtype=torch.int32, device="cuda")

    def fill(b, first, K, V):
        at = torch.arange(first, first + K.shape[0], device="cuda")
        _write(cache, D, table[b, at // page] * page + offs[at % page], K, V)

    def some(n):
        return (_cache_like(_normal((n, Hkv, D), gen), gen, 3.0), _cache_like(_normal((n, Hkv, D), gen), gen, 1.0))

    common = some(prefix) if prefix else None
    used = same
    for b, n in enumerate(need):
        table[b, same:same + n] = order[used:used + n]
        used += n
        if k[b] <= prefix:                         # (a padded batch's request of no tokens)
            table[b] = -1
            continue
        if prefix and b == 0:
            fill(b, 0, *common)
        elif prefix % page:
            fill(b, same * page, common[0][same * page:], common[1][same * page:])
        fill(b, prefix, *some(k[b] - prefix))
    start = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
    state |= dict(cache=cache, table=table, q_most=max(q), longest=max(k),
                  lens=torch.tensor(k, dtype=torch.int32, device="cuda"), start=torch.from_numpy(start).cuda(),
                  Q=_normal((int(start[-1]), case["Hq"], D), gen).to(DTYPES[case["dtype"]]))
    return state


# ---- one pass ----------------------------------------------------------------------

def run(state):
    return {"rope": _rope, "rope_append": _rope_append, "copy": _copy, "fork": _fork, "compact": _compact,
            "sinks": _sinks, "prefix": _prefix}[state["op"]](state)


def _rotate(x, s):
    """Rotated fp32 values of x [T][heads][D]."""
    angle = s["pos"].double()[:, None] * s["freq"]
    c = (torch.cos(angle) * s["factor"]).float()[:, None]
    n = (torch.sin(angle) * s["factor"]).float()[:, None]
    R = s["R"]
    x = x.float()
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if s["interleaved"] else (x[..., :R // 2], x[..., R // 2:R])
    ya, yb = a * c - b * n, b * c + a * n
    y = torch.stack((ya, yb), -1).flatten(-2) if s["interleaved"] else torch.cat((ya, yb), -1)
    return torch.cat((y, x[..., R:]), -1)


def _rope(s):
    if own:
        import bit_weight_only_quantize_amd as awq
        return awq.awq_rope(s["Q"], s["pos"], s["freq"], K=s["K"], attention_factor=s["factor"],
                            interleaved=s["interleaved"])
    return _rotate(s["Q"], s).to(s["Q"].dtype), _rotate(s["K"], s).to(s["K"].dtype)


def _rope_append(s):
    if own:
        import bit_weight_only_quantize_amd as awq
        q = awq.awq_kv_append_rope(s["K"], s["V"], s["cache"], s["slots"], s["pos"], s["freq"], Q=s["Q"],
                                   attention_factor=s["factor"], interleaved=s["interleaved"])
        return (q, *awq.awq_kv_gather(s["cache"], s["slots"], out_dtype=s["K"].dtype))
    _write(s["cache"], s["D"], s["slots"], _rotate(s["K"], s), s["V"])
    k, v = _read(s["cache"], s["D"], s["slots"])
    return _rotate(s["Q"], s).to(s["Q"].dtype), k.to(s["K"].dtype), v.to(s["V"].dtype)


def _copy(s):
    if own:
        import bit_weight_only_quantize_amd as awq
        return awq.awq_kv_copy_pages(s["cache"], s["src"], s["dst"])
    src, dst = s["src"].long(), s["dst"].long()
    for x in s["cache"]:
        if x is not None:
            x[dst] = x[src]
    return s["cache"]


def _fork(s):
    """Branches share their parents' full pages and get a copy of the page that they go on in; then they end.
    What they share is counted per page, as holders beyond the first."""
    page, table, shared = s["page"], s["table"], s["shared"]
    if own:
        import bit_weight_only_quantize_amd as awq
        used = awq.awq_kv_fork(s["cache"], table, s["parents"], s["children"], s["share"], shared, s["free"])
        forked, held = table.clone(), shared.clone()
        free, count = awq.awq_kv_release(table, s["ends"], shared, s["free"], page, start=s["keep"],
                                         pages_used=used)
        return {"forked": forked, "held": held, "used": used, "table": table, "shared": shared, "free": free,
                "count": count, "cache": s["cache"]}
    dev, pages = table.device, shared.shape[0]
    parents, children, n = s["parents"].long(), s["children"].long(), s["share"].long()
    block = torch.arange(table.shape[1], device=dev)
    full, part = n // page, (n % page != 0).long()
    rows = table[parents]
    at = torch.cumsum(part, 0) - part
    fresh = torch.where(at < s["free"].shape[0], s["free"][at.clamp(max=s["free"].shape[0] - 1)], -1)
    whole = block < full[:, None]
    opens = (block == full[:, None]) & (part[:, None] > 0)
    table[children] = torch.where(whole, rows, torch.where(opens, fresh[:, None], table[children]))
    shared += torch.bincount(rows[whole & (rows >= 0)], minlength=pages)
    last = rows.gather(1, full.clamp(max=table.shape[1] - 1)[:, None])[:, 0]
    found = (part > 0) & (fresh >= 0) & (last >= 0)
    for x in s["cache"]:
        if x is not None:
            x[fresh[found].long()] = x[last[found].long()]
    used = part.sum().int()[None]
    forked, held = table.clone(), shared.clone()
    ends, keep = s["ends"].long(), s["keep"].long()
    gone = (block >= ((keep + page - 1) // page)[:, None]) & (block < ((ends + page - 1) // page)[:, None])
    shared -= torch.bincount(table[gone & (table >= 0)], minlength=pages)
    table.masked_fill_(gone, -1)
    idle = shared < 0
    shared.masked_fill_(idle, 0)
    left = torch.arange(s["free"].shape[0], device=dev) >= used
    both = torch.cat((s["free"], torch.arange(pages, device=dev, dtype=torch.int32)))
    keep_it = torch.cat((left & (s["free"] >= 0), idle))
    place = torch.where(keep_it, torch.cumsum(keep_it, 0) - 1, pages)
    free = torch.full((pages + 1,), -1, dtype=torch.int32, device=dev)
    free.scatter_(0, place.clamp(max=pages), torch.where(keep_it, both, -1))
    return {"forked": forked, "held": held, "used": used, "table": table, "shared": shared, "free": free[:pages],
            "count": keep_it.sum().int()[None], "cache": s["cache"]}


def _compact(s):
    """Used pages behind the first n, n their number, move into the holes before it: the last into the first."""
    table, shared = s["table"].clone(), s["shared"].clone()
    if own:
        import bit_weight_only_quantize_amd as awq
        free, used = awq.awq_kv_compact(s["cache"], table, s["lens"], shared)
        return {"table": table, "shared": shared, "free": free, "used": used, "cache": s["cache"]}
    dev, pages, page = table.device, shared.shape[0], s["page"]
    block = torch.arange(table.shape[1], device=dev)
    live = (block < ((s["lens"].long() + page - 1) // page)[:, None]) & (table >= 0)
    mark = torch.bincount(table[live], minlength=pages) > 0
    n = mark.sum()
    ids = torch.arange(pages, device=dev)
    holes, movers = ids[~mark & (ids < n)], ids[mark & (ids >= n)].flip(0)
    for x in s["cache"]:
        if x is not None:
            x[holes] = x[movers]
    to = ids.clone()
    to[movers] = holes
    table = torch.where(live, to[table.clamp(min=0).long()].int(), table)
    shared[holes] = shared[movers]
    shared = torch.where(ids < n, shared, 0)
    return {"table": table, "shared": shared, "free": torch.where(ids + n < pages, ids + n, -1).int(),
            "used": n.int()[None], "cache": s["cache"]}


def _queries(s):
    """Query tokens by request: (token [B][n], position [B][n])."""
    lens, start, n = s["lens"].long(), s["start"].long(), s["q_most"]
    row = torch.arange(n, device=lens.device)
    ql = start[1:] - start[:-1]
    return (start[:-1, None] + row).clamp(max=s["Q"].shape[0] - 1), (lens - ql)[:, None] + row


def _by_head(s, at):
    """Queries as [B][Hkv][shared * n][D] fp32."""
    B, n = at.shape
    Hkv, D, Q = s["Hkv"], s["D"], s["Q"]
    shared = Q.shape[1] // Hkv
    return Q[at].float().view(B, n, Hkv, shared, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, shared * n, D)


def _by_token(s, o):
    """[B][Hkv][shared * n][D] as the tokens' rows."""
    B, Hkv, rows, D = o.shape
    n, start = s["q_most"], s["start"].long()
    o = o.view(B, Hkv, rows // n, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, Hkv * (rows // n), D)
    token = torch.arange(s["Q"].shape[0], device=o.device)
    b = torch.searchsorted(start[1:].contiguous(), token, right=True)
    return o[b, token - start[b]].to(s["Q"].dtype)


def _keys(s, pos, ok):
    """Keys [B][Hkv][D][n] and values [B][Hkv][n][D] at positions pos [B][n] of each request."""
    B, n = pos.shape
    Hkv, D, page = s["Hkv"], s["D"], s["page"]
    block = (pos // page).clamp(0, s["table"].shape[1] - 1)
    ids = s["table"].gather(1, block)
    slots = torch.where(ok & (ids >= 0), ids * page + (pos % page).int(), -1)
    k, v = _read(s["cache"], D, slots.flatten())
    return (k.view(B, n, Hkv, D).permute(0, 2, 3, 1).contiguous(),
            v.view(B, n, Hkv, D).transpose(1, 2).contiguous())


def _weights(logits):
    """Softmax of the last dimension, zeros for a row that sees nothing."""
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - torch.where(top.isinf(), 0.0, top))
    total = p.sum(-1, keepdim=True)
    return torch.where(total > 0, p / total, 0.0)


def _sinks(s):
    if own:
        import bit_weight_only_quantize_amd as awq
        return awq.awq_kv_attention(s["Q"], s["cache"], s["table"], s["lens"],
                                    query_start=s["start"] if s["q_most"] > 1 else None,
                                    max_query_len=s["q_most"], max_seq_len=s["longest"], window=s["window"],
                                    sinks=s["sinks"])
    w, first, lens = s["window"], s["sinks"], s["lens"].long()
    at, q_pos = _queries(s)
    B, n = at.shape
    ql = s["start"].long().diff()
    # the first tokens, then those from the earliest window's start on
    width = min(first + w + n - 1, max(s["longest"], first + 1))
    i = torch.arange(width, device=lens.device)
    base = (lens - ql - w + 1).clamp(min=first)
    pos = torch.where(i < first, i, base[:, None] + i - first)
    ok = pos < lens[:, None]
    k, v = _keys(s, pos, ok)
    logits = torch.matmul(_by_head(s, at), k).view(B, s["Hkv"], -1, n, width) / math.sqrt(s["D"])
    p_at = pos[:, None]
    seen = ok[:, None] & (p_at <= q_pos[..., None]) & ((p_at > q_pos[..., None] - w) | (p_at < first))
    p = _weights(torch.where(seen[:, None, None], logits, -math.inf))
    return _by_token(s, torch.matmul(p.view(B, s["Hkv"], -1, width), v))


def _prefix(s):
    if own:
        import bit_weight_only_quantize_amd as awq
        return awq.awq_kv_attention(s["Q"], s["cache"], s["table"], s["lens"],
                                    query_start=s["start"] if s["q_most"] > 1 else None,
                                    max_query_len=s["q_most"], max_seq_len=s["longest"], prefix_len=s["prefix"])
    L, Hkv, D, lens = s["prefix"], s["Hkv"], s["D"], s["lens"].long()
    at, q_pos = _queries(s)
    B, n = at.shape
    q = _by_head(s, at)
    rows = q.shape[2]
    pos = torch.arange(L, device=lens.device)
    slots = s["table"][0, pos // s["page"]] * s["page"] + (pos % s["page"]).int()
    kp, vp = _read(s["cache"], D, slots)
    every = q.transpose(0, 1).reshape(Hkv, B * rows, D)
    near = torch.matmul(every, kp.permute(1, 2, 0).contiguous()).view(Hkv, B, rows, L).transpose(0, 1)
    width = max(1, s["longest"] - L)
    own_pos = (L + torch.arange(width, device=lens.device)).expand(B, width)
    k, v = _keys(s, own_pos, own_pos < lens[:, None])
    logits = torch.cat((near, torch.matmul(q, k)), -1) / math.sqrt(D)
    key = torch.arange(L + width, device=lens.device)
    seen = ((key <= q_pos[..., None]) & (key < lens[:, None, None]))[:, None, None]
    p = _weights(torch.where(seen, logits.view(B, Hkv, -1, n, L + width), -math.inf)).view(B, Hkv, rows, L + width)
    o = torch.matmul(p[..., :L].transpose(0, 1).reshape(Hkv, B * rows, L), vp.transpose(0, 1).contiguous())
    return _by_token(s, o.view(Hkv, B, rows, D).transpose(0, 1) + torch.matmul(p[..., L:], v))


# ---- what a pass cannot do without ----------------------------------------------------

def work(case):
    op, D = case["op"], case["D"]
    meta = 6 if case.get("zero_point") else 4            # bytes of steps and zero points per token and head
    if op in ("rope", "rope_append"):
        T, Hq, Hkv, R = case["T"], case["Hq"], case["Hkv"], case["R"]
        table, flops = 4 * T + 4 * R, 3 * T * R * (Hq + Hkv)
        if op == "rope":
            return {"bytes": 2 * 2 * T * D * (Hq + Hkv) + table, "flops": flops}
        # Q in and out, K and V in, their packed form into the cache, the values that it stands for out
        return {"bytes": 4 * T * D * Hq + T * Hkv * (4 * D + D + meta + 4 * D) + table + 4 * T,
                "flops": flops + T * Hkv * 2 * D * 8}
    if op in ("copy", "fork", "compact"):
        each = case["page"] * case["heads"] * (D + meta)
        if op == "copy":
            return {"bytes": 2 * case["n"] * each + 8 * case["n"], "flops": 2 * case["n"]}
        lens, page = _page_lengths(case), case["page"]
        if op == "fork":
            parents, children, share = _forks(case)
            full, part = sum(n // page for n in share), [n % page for n in share]
            held = sum(-(-n // page) for b, n in enumerate(lens) if b not in set(children))
            pages = held + case["n"] + 60
            # the tokens of the copied pages, table entries read, written, read again and cleared, holders up and
            # down, the free list in and out
            return {"bytes": 2 * sum(part) * case["heads"] * (D + meta) + 4 * 4 * (full + len(share)) + 4 * 4 * pages
                    + 12 * case["n"], "flops": 4 * full}
        held = sum(-(-n // page) for n in lens)
        pages = held + int(held * case["spare"]) + 3
        moved = held * (pages - held) // pages               # (pages are spread evenly)
        return {"bytes": 2 * moved * each + 4 * (2 * held + 3 * pages), "flops": 4 * pages}
    q, k = _lengths(case)
    Hq, Hkv = case["Hq"], case["Hkv"]
    pairs, keys = map(sum, zip(*(_seen(a, b, case) for a, b in zip(q, k))))
    keys += case.get("prefix", 0)
    return {"bytes": 2 * 2 * sum(q) * Hq * D + keys * Hkv * (D + meta) + 4 * (keys // case["page"] + 2 * len(q)),
            "flops": 4 * D * Hq * pairs}


# ---- the definition in 64 bits -----------------------------------------------------------

def _nibbles(words):
    """Codes of packed words (last dimension), read byte by byte: fp64."""
    b = words.contiguous().view(torch.uint8)                 # little endian: byte j holds nibbles 2j, 2j+1
    n = torch.stack((b & 15, b >> 4), -1).flatten(-2).unflatten(-1, (-1, 8))
    return n[..., [0, 4, 1, 5, 2, 6, 3, 7]].flatten(-2).double()


def _round32(x):
    return x.float().double()


def _levels(x, zero_point):
    """x fp64 [..., D]: the values that its 4-bit codes stand for, step by step as the format says
    (quotients correctly rounded to 32 bits, as their double rounding through 64 bits is)."""
    if zero_point:
        lo, hi = x.amin(-1, keepdim=True).clamp(max=0), x.amax(-1, keepdim=True).clamp(min=0)
        s = _round32(_round32(hi - lo) / 15).clamp(min=2.0 ** -14).half().double()
        z = torch.round(_round32(-lo / s)).clamp(0, 15)
        return ((torch.round(_round32(x / s)) + z).clamp(0, 15) - z) * s
    s = _round32(x.abs().amax(-1, keepdim=True) / 7).clamp(min=2.0 ** -14).half().double()
    return torch.round(_round32(x / s)).clamp(-8, 7) * s


def _turned(x, s, rounded):
    """Rotation as a product of complex numbers; `rounded`: cosines, sines, products and sums taken to 32
    bits, as the values that a cache's codes are chosen by are."""
    r = _round32 if rounded else (lambda t: t)
    R, y = s["R"], x.double().clone()
    turn = s["factor"] * torch.polar(torch.ones((), dtype=torch.float64, device=x.device).expand(
        len(s["pos"]), R // 2), torch.outer(s["pos"].double(), s["freq"]))
    c, n = r(turn.real)[:, None], r(turn.imag)[:, None]
    a, b = (slice(0, R, 2), slice(1, R, 2)) if s["interleaved"] else (slice(0, R // 2), slice(R // 2, R))
    u, v = y[..., a].clone(), y[..., b].clone()
    y[..., a] = r(r(u * c) - r(v * n))
    y[..., b] = r(r(v * c) + r(u * n))
    return y


def _kv(s, row, lo, hi, h):
    """fp64 keys and values of head h, tokens lo .. hi of a table row."""
    codes, scales, zeros = s["cache"]
    D, page = s["D"], s["page"]
    ids = row[:-(-hi // page)].long()
    kw = codes[ids, 0, h].reshape(-1, D // 8)[lo:hi]
    vw = codes[ids, 1, h].reshape(-1, D // 8, 4).transpose(1, 2).reshape(-1, D // 8)[lo:hi]
    sc = scales[ids, h].reshape(-1, 2)[lo:hi].double()
    ze = torch.full_like(sc, 8.0) if zeros is None else zeros[ids, h].reshape(-1, 2)[lo:hi].double()
    return (_nibbles(kw) - ze[:, :1]) * sc[:, :1], (_nibbles(vw) - ze[:, 1:]) * sc[:, 1:]


def exact(case, seed):
    if case["op"] in ("copy", "fork", "compact"):
        return None
    s = prepare(case, seed)
    if case["op"] == "rope":
        return _turned(s["Q"], s, False), _turned(s["K"], s, False)
    if case["op"] == "rope_append":
        return (_turned(s["Q"], s, False), _levels(_turned(s["K"], s, True), case["zero_point"]),
                _levels(s["V"].double(), case["zero_point"]))
    q_len, k_len = _lengths(case)
    L, Hkv, D = case.get("prefix", 0), case["Hkv"], case["D"]
    group = case["Hq"] // Hkv
    Q = s["Q"].double().unflatten(1, (Hkv, group)) * D ** -0.5          # [T][Hkv][group][D]
    out = torch.zeros_like(Q)
    begin = np.concatenate([[0], np.cumsum(q_len)])
    for h in range(Hkv):
        if L:
            kp, vp = _kv(s, s["table"][0], 0, L, h)
            a_all = torch.matmul(Q[:, h].reshape(-1, D), kp.t().contiguous()).view(-1, group, L)
        for b in range(case["B"]):
            if k_len[b] <= L:
                continue
            rows = slice(int(begin[b]), int(begin[b + 1]))
            k, v = _kv(s, s["table"][b], L, k_len[b], h)
            place = torch.arange(k_len[b] - q_len[b], k_len[b], device="cuda")[:, None]
            key = torch.arange(L, k_len[b], device="cuda")
            hidden = key > place
            if not L:
                hidden = hidden | ((key <= place - case["window"]) & (key >= case["sinks"]))
            for j in range(group):
                a = (Q[rows, h, j] @ k.t().contiguous()).masked_fill(hidden, -math.inf)
                if L:
                    a = torch.cat((a_all[rows, j], a), -1)
                p = torch.softmax(a, -1)
                out[rows, h, j] = p[:, L:] @ v + (p[:, :L] @ vp if L else 0.0)
    return out.flatten(1, 2)
