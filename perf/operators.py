"""Measured cases of the 4-bit key/value cache, the attention over it and the
linear layer's epilogue.

``run`` computes each operator either in its plain form (elementary torch
operations in 32 bits, rounded once at the end) or, where ``own`` is true,
with the library's entry points.  Both take the same inputs from ``prepare``.
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
        # one step of continuous batching: every running request gets one token
        dict(name="assign_step_b24", op="assign", B=24, page=64, kind="step", most=2000, key=1),
        # a step that mixes decoding requests with new prompts and chunks of long ones
        dict(name="assign_mixed_b500", op="assign", B=500, page=16, kind="mixed", most=900, key=2),
        # the new tokens of one decode step, 8 key/value heads (70B-class layer)
        dict(name="append_step_t32_h8_d128", op="append", T=32, heads=8, D=128, page=64,
             dtype="f16", zero_point=True),
        # prompts of a 7B-class layer (32 heads of 128), bfloat16 activations
        dict(name="append_prompt_t8192_h32_d128", op="append", T=8192, heads=32, D=128, page=64,
             dtype="bf16", zero_point=True),
        # single-stream decode early in a conversation
        dict(name="decode_b1_l777_32x8_d128", op="attend", B=1, q_most=1, k_most=777, Hq=32, Hkv=8,
             D=128, page=64, dtype="f16", zero_point=True, window=0, key=3),
        # a serving batch of mid-length conversations, 7B-class heads without sharing
        dict(name="decode_b48_l4096_32x32_d128", op="attend", B=48, q_most=1, k_most=4096, Hq=32,
             Hkv=32, D=128, page=64, dtype="f16", zero_point=True, window=0, key=4),
        # few requests with long contexts, 70B-class heads
        dict(name="decode_b4_l65536_64x8_d128", op="attend", B=4, q_most=1, k_most=65536, Hq=64,
             Hkv=8, D=128, page=128, dtype="bf16", zero_point=False, window=0, key=5),
        # one long prompt
        dict(name="prompt_b1_l8192_32x8_d128", op="attend", B=1, q_most=8192, k_most=8192, Hq=32,
             Hkv=8, D=128, page=64, dtype="bf16", zero_point=True, window=0, key=6),
        # chunks of several prompts over what is cached already, a sliding window, heads of 64
        dict(name="chunk_b6_q515_l3000_16x4_d64", op="attend", B=6, q_most=515, k_most=3000, Hq=16,
             Hkv=4, D=64, page=16, dtype="f16", zero_point=True, window=1000, key=7),
        # output projection of a decode step: bias and the residual stream
        dict(name="epilogue_m1_4096x4096", op="linear", M=1, N=4096, K=4096, g=128, dtype="f16",
             zero_point=True, act="none", bias=True, residual=True),
        # first projection of an MLP for a decode batch
        dict(name="epilogue_m24_11008x4096_gelu", op="linear", M=24, N=11008, K=4096, g=128,
             dtype="bf16", zero_point=True, act="gelu_tanh", bias=True, residual=False),
        # prompt through the second projection of a 13B-class MLP
        dict(name="epilogue_m2048_5120x13824", op="linear", M=2048, N=5120, K=13824, g=128,
             dtype="f16", zero_point=True, act="none", bias=True, residual=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("assign", "append", "decode", "decode", "prompt", "prompt", "linear", "linear"))
    key = rng.randrange(1 << 30)
    page = rng.choice((16, 32, 64, 128))
    dtype = rng.choice(("f16", "bf16"))
    zero_point = rng.random() < 0.7
    if op == "assign":
        return dict(op="assign", B=_log(rng, 1, 1000), page=page, kind=rng.choice(("step", "mixed")),
                    most=_log(rng, 100, 4000), key=key)
    if op == "append":
        heads = rng.choice((1, 2, 4, 8, 16, 32, 40))
        return dict(op="append", T=_log(rng, 1, 8192 * 32 // max(heads, 32)), heads=heads,
                    D=rng.choice((64, 128)), page=page, dtype=dtype, zero_point=zero_point)
    if op in ("decode", "prompt"):
        Hkv = rng.choice((1, 2, 4, 8, 8, 16, 32))
        D = rng.choice((64, 128, 128))
        shared = rng.choice((1, 2, 4, 5, 7, 8))
        while Hkv * shared > 64:
            shared = max(1, shared // 2)
        B = _log(rng, 1, 48)
        if op == "decode":
            q_most = rng.choice((1, 1, 1, 1, 3, 4))
            k_most = _log(rng, max(q_most, 20), max(100, min(65536, 4096 * 24 * 32 // (B * Hkv))))
        else:
            B = _log(rng, 1, 12)
            q_most = _log(rng, 20, max(100, 4096 // B))
            most = min(8192, 32 * 8192 * 4096 // (Hkv * shared * q_most * B))
            k_most = q_most if rng.random() < 0.5 or most <= q_most else _log(rng, q_most, most)
        return dict(op="attend", B=B, q_most=q_most, k_most=k_most, Hq=Hkv * shared, Hkv=Hkv, D=D,
                    page=page, dtype=dtype, zero_point=zero_point,
                    window=rng.choice((0, 0, max(1, k_most // 3))), key=key)
    g = rng.choice((64, 128))
    return dict(op="linear", M=_log(rng, 1, 2048), N=_log(rng, 200, 11008),
                K=g * _log(rng, 4, 5120 // g), g=g, dtype=dtype, zero_point=zero_point,
                act=rng.choice(("none", "relu", "silu", "gelu", "gelu_tanh")),
                bias=rng.random() < 0.7, residual=rng.random() < 0.5)


# ---- lengths of a case's requests (from the case alone) ----------------------------

def _assign_lengths(case):
    r = random.Random(case["key"])
    if case["kind"] == "step":
        return [r.randint(1, case["most"]) for _ in range(case["B"])], [1] * case["B"]
    old, new = [], []
    for _ in range(case["B"]):
        if r.random() < 0.7:                       # decoding
            old.append(r.randint(1, case["most"]))
            new.append(1)
        else:                                      # a prompt, or a chunk of one
            old.append(r.choice((0, 0, r.randint(1, case["most"]))))
            new.append(r.randint(1, max(1, case["most"] // 4)))
    return old, new


def _attend_lengths(case):
    """(query lengths, key lengths); the first request has the most of both."""
    r = random.Random(case["key"])
    q, k = [case["q_most"]], [case["k_most"]]
    for _ in range(case["B"] - 1):
        n = 1 if case["q_most"] == 1 else r.randint(1, case["q_most"])
        q.append(n)
        k.append(r.randint(n, case["k_most"]))
    return q, k


def _pairs(q, k, window):
    """Query-key pairs that a causal request of q new tokens and k tokens in all has."""
    n = np.arange(k - q + 1, k + 1, dtype=np.int64)
    return int((np.minimum(n, window) if window else n).sum())


def _keys(q, k, window):
    return min(k, q + window - 1) if window else k


# ---- inputs -----------------------------------------------------------------------

def _normal(shape, gen, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda") * scale


def _cache_like(x, gen, spread):
    """Key- or value-like vectors [n][heads][D]: some channels shifted and larger, as keys have."""
    heads, D = x.shape[-2:]
    gain = torch.where(torch.rand((heads, D), generator=gen, device="cuda") < 0.03, spread, 1.0)
    shift = _normal((heads, D), gen, 0.3)
    return x * gain + shift


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


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state = dict(case)
    if case["op"] == "assign":
        old, new = _assign_lengths(case)
        page = case["page"]
        have = [-(-o // page) for o in old]
        want = [-(-(o + n) // page) for o, n in zip(old, new)]
        blocks = max(max(want), 1) + 4
        total = sum(want)
        pages = torch.randperm(total + 64, generator=gen, device="cuda").int()
        table = torch.full((case["B"], blocks), -1, dtype=torch.int32)
        used = 0
        host = pages.cpu()
        for b, h in enumerate(have):
            table[b, :h] = host[used:used + h]
            used += h
        state |= dict(old=torch.tensor(old, dtype=torch.int32, device="cuda"),
                      new=torch.tensor(new, dtype=torch.int32, device="cuda"),
                      table=table.cuda(), free=pages[used:].clone(), tokens=sum(new) + 7)
        return state
    if case["op"] == "append":
        T, heads, D, page = case["T"], case["heads"], case["D"], case["page"]
        pages = -(-T // page) + 8
        slots = torch.randperm(pages, generator=gen, device="cuda").int()[:, None] * page + torch.arange(
            page, dtype=torch.int32, device="cuda")
        if T <= 256:                               # a decode step: tokens anywhere in the cache
            slots = slots.flatten()[torch.randperm(pages * page, generator=gen, device="cuda")]
        dt = DTYPES[case["dtype"]]
        state |= dict(cache=_new_cache(pages, heads, D, page, case["zero_point"], gen),
                      slots=slots.flatten()[:T].contiguous(),
                      K=_cache_like(_normal((T, heads, D), gen), gen, 4.0).to(dt),
                      V=_cache_like(_normal((T, heads, D), gen), gen, 1.0).to(dt))
        return state
    if case["op"] == "attend":
        q, k = _attend_lengths(case)
        B, Hkv, D, page = case["B"], case["Hkv"], case["D"], case["page"]
        need = [-(-n // page) for n in k]
        pages = sum(need) + 5
        cache = _new_cache(pages, Hkv, D, page, case["zero_point"], gen)
        order = torch.randperm(pages, generator=gen, device="cuda").int()
        table = torch.full((B, max(need)), -1, dtype=torch.int32, device="cuda")
        offs = torch.arange(page, dtype=torch.int32, device="cuda")
        used = 0
        for b, n in enumerate(need):
            table[b, :n] = order[used:used + n]
            slots = (table[b, :n, None] * page + offs).flatten()[:k[b]]
            x = _cache_like(_normal((k[b], Hkv, D), gen), gen, 3.0)
            _write(cache, D, slots, x, _cache_like(_normal((k[b], Hkv, D), gen), gen, 1.0))
            used += n
        start = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
        state |= dict(cache=cache, table=table, q_most=max(q), k_most=max(k),
                      lens=torch.tensor(k, dtype=torch.int32, device="cuda"),
                      start=torch.from_numpy(start).cuda(),
                      Q=_normal((int(start[-1]), case["Hq"], D), gen).to(DTYPES[case["dtype"]]))
        return state
    M, N, K, g = case["M"], case["N"], case["K"], case["g"]
    dt = DTYPES[case["dtype"]]
    codes, scales, zeros = _quantize(_normal((N, K // g, g), gen, 0.02).half().float(),
                                     case["zero_point"])
    gain = torch.where(torch.rand(K, generator=gen, device="cuda") < 0.01, 20.0, 1.0)
    state |= dict(X=(_normal((M, K), gen) * gain).to(dt), qweight=_pack(codes.flatten(1)),
                  scales=scales.contiguous(), zeros=None if zeros is None else zeros.contiguous(),
                  b=_normal((N,), gen, 0.5).to(dt) if case["bias"] else None,
                  r=_normal((M, N), gen, 2.0).to(dt) if case["residual"] else None)
    return state


# ---- one pass ----------------------------------------------------------------------

def run(state):
    return {"assign": _assign, "append": _append, "attend": _attend, "linear": _linear}[state["op"]](state)


def _assign(s):
    if own:
        import bit_weight_only_quantize_amd as awq
        lens, start, slots, used = awq.awq_kv_assign(s["old"], s["new"], s["table"], s["free"],
                                                     s["page"], s["tokens"])
        return {"table": s["table"], "lens": lens, "start": start, "slots": slots, "used": used}
    old, new, page, T = s["old"].long(), s["new"].long(), s["page"], s["tokens"]
    B, blocks = s["table"].shape
    dev = old.device
    have, want = (old + page - 1) // page, (old + new + page - 1) // page
    first = torch.cumsum(want - have, 0) - (want - have)
    block = torch.arange(blocks, device=dev)
    fresh = (block >= have[:, None]) & (block < want[:, None])
    at = first[:, None] + block - have[:, None]
    ids = s["free"][at.clamp(0, len(s["free"]) - 1)]
    ids = torch.where(at < len(s["free"]), ids, -1)
    table = torch.where(fresh, ids, s["table"])
    start = torch.cat((torch.zeros(1, dtype=torch.int64, device=dev), torch.cumsum(new, 0)))
    t = torch.arange(T, device=dev)
    b = torch.searchsorted(start[1:].contiguous(), t, right=True)
    inside = b < B
    b = b.clamp(max=B - 1)
    pos = old[b] + t - start[b]
    p = table[b, (pos // page).clamp(0, blocks - 1)].long()
    slots = torch.where(inside & (p >= 0) & (pos // page < blocks), p * page + pos % page, -1)
    return {"table": table, "lens": (old + new).int(), "start": start.int(), "slots": slots.int(),
            "used": (want - have).sum().int()[None]}


def _append(s):
    if own:
        import bit_weight_only_quantize_amd as awq
        awq.awq_kv_append(s["K"], s["V"], s["cache"], s["slots"])
        return awq.awq_kv_gather(s["cache"], s["slots"], out_dtype=s["K"].dtype)
    _write(s["cache"], s["D"], s["slots"], s["K"], s["V"])
    k, v = _read(s["cache"], s["D"], s["slots"])
    return k.to(s["K"].dtype), v.to(s["V"].dtype)


def _attend(s):
    if own:
        import bit_weight_only_quantize_amd as awq
        return awq.awq_kv_attention(s["Q"], s["cache"], s["table"], s["lens"],
                                    query_start=s["start"] if s["q_most"] > 1 else None,
                                    max_query_len=s["q_most"], max_seq_len=s["k_most"],
                                    window=s["window"])
    Q, lens, start, page = s["Q"], s["lens"].long(), s["start"].long(), s["page"]
    B, Hkv, D, n, L = s["B"], s["Hkv"], s["D"], s["q_most"], s["k_most"]
    dev = Q.device
    shared = Q.shape[1] // Hkv
    pos = torch.arange(L, device=dev)
    slots = s["table"][:, pos // page] * page + (pos % page).int()
    slots = torch.where(pos < lens[:, None], slots, -1)
    k, v = _read(s["cache"], D, slots.flatten())
    k = k.view(B, L, Hkv, D).permute(0, 2, 3, 1).contiguous()       # [B][Hkv][D][L]
    v = v.view(B, L, Hkv, D).transpose(1, 2).contiguous()           # [B][Hkv][L][D]
    row = torch.arange(n, device=dev)
    ql = start[1:] - start[:-1]
    inside = row < ql[:, None]
    at = (start[:-1, None] + row).clamp(max=Q.shape[0] - 1)
    q = Q[at].float().view(B, n, Hkv, shared, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, shared * n, D)
    logits = torch.matmul(q, k).view(B, Hkv, shared, n, L) / math.sqrt(D)
    q_pos = (lens - ql)[:, None] + row
    seen = (pos <= q_pos[..., None]) & (pos < lens[:, None, None])
    if s["window"]:
        seen &= pos > q_pos[..., None] - s["window"]
    logits = torch.where(seen[:, None, None], logits, -math.inf)
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - torch.where(top.isinf(), 0.0, top))
    total = p.sum(-1)
    o = torch.matmul(p.view(B, Hkv, shared * n, L), v).view(B, Hkv, shared, n, D)
    o = torch.where(total[..., None] > 0, o / total[..., None], 0.0)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, Hkv * shared, D)
    token = torch.arange(Q.shape[0], device=dev)
    b = torch.searchsorted(start[1:].contiguous(), token, right=True)
    return o[b, token - start[b]].to(Q.dtype)


def _linear(s):
    if own:
        import bit_weight_only_quantize_amd as awq
        return awq.awq_linear_epilogue(s["X"], s["qweight"], s["scales"], s["zeros"], bias=s["b"],
                                       residual=s["r"], activation=s["act"], group_size=s["g"])
    N, K, g = s["N"], s["K"], s["g"]
    z = 8.0 if s["zeros"] is None else s["zeros"].float()[..., None]
    w = ((_unpack(s["qweight"]).view(N, K // g, g).float() - z) * s["scales"].float()[..., None]).view(N, K)
    y = torch.matmul(s["X"].float(), w.t())
    if s["b"] is not None:
        y = y + s["b"].float()
    if s["act"] == "relu":
        y = torch.where(y > 0, y, 0.0)
    elif s["act"] == "silu":
        y = y / (1 + torch.exp(-y))
    elif s["act"] == "gelu":
        y = 0.5 * y * (1 + torch.erf(y / math.sqrt(2)))
    elif s["act"] == "gelu_tanh":
        y = 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y * y * y)))
    if s["r"] is not None:
        y = y + s["r"].float()
    return y.to(s["X"].dtype)


# ---- what a pass cannot do without ----------------------------------------------------

def work(case):
    if case["op"] == "assign":
        old, new = _assign_lengths(case)
        page, B, T = case["page"], case["B"], sum(new) + 7
        fresh = sum(-(-(o + n) // page) - -(-o // page) for o, n in zip(old, new))
        blocks = max(max(-(-(o + n) // page) for o, n in zip(old, new)), 1) + 4
        # lengths in, table (its kept entries in, all of it out), free ids, lengths and starts, slots
        return {"bytes": 4 * (2 * B + 2 * B * blocks + fresh + 2 * B + 1 + T + 1), "flops": 8 * T + 8 * B}
    zeros = 2 if case.get("zero_point") else 0
    if case["op"] == "append":
        n = case["T"] * case["heads"]
        D = case["D"]
        # K and V in, their packed form into the cache, the values that it stands for out
        return {"bytes": n * (2 * 2 * D + D + 4 + zeros + 2 * 2 * D) + 4 * case["T"], "flops": n * 2 * D * 8}
    if case["op"] == "attend":
        q, k = _attend_lengths(case)
        D, Hq, Hkv, w = case["D"], case["Hq"], case["Hkv"], case["window"]
        tokens = sum(_keys(a, b, w) for a, b in zip(q, k))
        table = sum(-(-b // case["page"]) for b in k)
        return {"bytes": 2 * 2 * sum(q) * Hq * D + tokens * Hkv * (D + 4 + zeros) + 4 * (table + 2 * len(q)),
                "flops": 4 * D * Hq * sum(_pairs(a, b, w) for a, b in zip(q, k))}
    M, N, K, G = case["M"], case["N"], case["K"], case["K"] // case["g"]
    per_group = 3 if case["zero_point"] else 2
    return {"bytes": N * K // 2 + per_group * N * G + 2 * M * K + 2 * M * N * (2 if case["residual"] else 1)
            + (2 * N if case["bias"] else 0), "flops": 2 * M * N * K}


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


def exact(case, seed):
    if case["op"] == "assign":
        return None
    s = prepare(case, seed)
    if case["op"] == "append":
        return tuple(_levels(x.double(), case["zero_point"]) for x in (s["K"], s["V"]))
    if case["op"] == "attend":
        codes, scales, zeros = s["cache"]
        D, page, w = case["D"], case["page"], case["window"]
        q_len, k_len = _attend_lengths(case)
        out = torch.empty(s["Q"].shape, dtype=torch.float64, device="cuda")
        first = 0
        for b in range(case["B"]):
            ids = s["table"][b, :-(-k_len[b] // page)].long()
            place = torch.arange(k_len[b] - q_len[b], k_len[b], device="cuda")[:, None]
            key = torch.arange(k_len[b], device="cuda")
            hidden = (key > place) | ((key <= place - w) if w else False)
            for h in range(case["Hkv"]):
                kw = codes[ids, 0, h].reshape(-1, D // 8)[:k_len[b]]
                vw = codes[ids, 1, h].reshape(-1, D // 8, 4).transpose(1, 2).reshape(-1, D // 8)[:k_len[b]]
                sc = scales[ids, h].reshape(-1, 2)[:k_len[b]].double()
                ze = 8.0 if zeros is None else zeros[ids, h].reshape(-1, 2)[:k_len[b]].double()
                kv_zero = (8.0, 8.0) if zeros is None else (ze[:, :1], ze[:, 1:])
                k = (_nibbles(kw) - kv_zero[0]) * sc[:, :1]
                v = (_nibbles(vw) - kv_zero[1]) * sc[:, 1:]
                group = case["Hq"] // case["Hkv"]
                for j in range(h * group, (h + 1) * group):
                    q = s["Q"][first:first + q_len[b], j].double()
                    a = (q @ k.t().contiguous()) * D ** -0.5
                    p = torch.softmax(a.masked_fill(hidden, -math.inf), -1)
                    out[first:first + q_len[b], j] = p @ v
            first += q_len[b]
        return out
    N, G, g = case["N"], case["K"] // case["g"], case["g"]
    z = 8.0 if s["zeros"] is None else s["zeros"].double().repeat_interleave(g, 1)
    w = (_nibbles(s["qweight"]) - z) * s["scales"].double().repeat_interleave(g, 1)
    y = s["X"].double() @ w.t().contiguous()
    y = y if s["b"] is None else y + s["b"].double()
    act = {"none": lambda t: t, "relu": lambda t: t.clamp(min=0), "silu": lambda t: t * torch.sigmoid(t),
           "gelu": lambda t: t * 0.5 * torch.special.erfc(-t * 0.5 ** 0.5),
           "gelu_tanh": lambda t: t * torch.sigmoid(2 * (2 / math.pi) ** 0.5 * (t + 0.044715 * t ** 3))}
    y = act[case["act"]](y)
    return y if s["r"] is None else y + s["r"].double()
