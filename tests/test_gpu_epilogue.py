"""GPU parity of awq_linear_epilogue: act(X W^T + bias) + residual against fp64,
within a bound counted from the documented arithmetic, on every kernel of the
layer, and the layer's own results where the epilogue is empty."""

import numpy as np
import pytest
from scipy.special import erfc

import workloads as wl
from gpu_common import dev, out_to_f64, say, to_dev, torch_mod
from oracle import QuantConfig, bf16_bits_to_f32, dequantize, quantize_pack, unpack_codes

pytestmark = pytest.mark.gpu

ACTS = {
    "none": lambda x: x,
    "relu": lambda x: np.maximum(x, 0),
    "silu": lambda x: x / (1 + np.exp(-x)),
    "gelu": lambda x: 0.5 * x * erfc(-x / np.sqrt(2)),
    "gelu_tanh": lambda x: x / (1 + np.exp(-2 * np.sqrt(2 / np.pi) * (x + 0.044715 * x ** 3))),
}
EPS = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8, "float32": 2.0 ** -24}


def _case(M, N, K, g, xdt, odt, zp, seed):
    torch = torch_mod()
    rng = np.random.default_rng(seed)
    W = wl.gen_weight(N, K, seed)
    X = wl.gen_activation(M, K, seed + 1, seed + 2, "f16" if xdt == "float16" else "bf16")
    pk = quantize_pack(W, QuantConfig(group_size=g, zero_point=zp))
    Xd = to_dev(X, bf16=xdt == "bfloat16")
    x64 = (X if xdt == "float16" else bf16_bits_to_f32(X)).astype(np.float64)
    t = lambda a: torch.from_numpy(a.astype(np.float32)).to(getattr(torch, odt)).to(dev())   # noqa: E731
    bias, res = t(rng.normal(0, 0.5, N)), t(rng.normal(0, 2, (M, N)))
    return [None if a is None else to_dev(a) for a in pk], pk, Xd, x64, bias, res


def _reference(x64, pk, K, g, bias, res, act, odt, exact):
    """(y, bound).  Pre-activation error: fp32 sums of K products, K 2^-24 of
    sum |x w| (and 2^-11 of it where the kernel rounds the dequantized weight);
    the activations' slopes are at most 1.13; the activation itself and the
    three fp32 additions are good to 2^-19 of their operands; one rounding."""
    qw, sc, zr = pk
    w = dequantize(unpack_codes(qw, K), sc, zr, g).astype(np.float64)
    s, mag = x64 @ w.T, np.abs(x64) @ np.abs(w.T)
    err = mag * (K * 2.0 ** -24 + (0 if exact else 2.0 ** -11))
    if bias is not None:
        s = s + out_to_f64(bias)
    y = ACTS[act](s)
    err = 1.13 * err + 2.0 ** -19 * (np.abs(s) + np.abs(y))
    if res is not None:
        y = y + out_to_f64(res)
        err += 2.0 ** -22 * np.abs(out_to_f64(res))
    tiny = 2.0 ** -25 if odt == "float16" else 0.0           # half a step of fp16's subnormals
    return y, err * (1 + EPS[odt]) + EPS[odt] * np.abs(y) + tiny


# every kernel: GEMV with 16 and 8 waves, batched with and without splits, the
# GEMM's 32-, 64-, 128- and 256-row tiles, split and not; ragged and odd N
@pytest.mark.parametrize("M,N,K,g,xdt,odt,zp,kernel", [
    (1, 512, 512, 128, "float16", "float16", True, "gemv"),
    (3, 4099, 256, 64, "bfloat16", "float32", True, "gemv"),
    (16, 77, 1024, 128, "float16", "bfloat16", False, "gemv"),
    (4, 200, 12800, 64, "bfloat16", "bfloat16", True, "gemv"),
    (5, 300, 128, 128, "float16", "float16", True, "batched"),
    (24, 1000, 2048, 128, "bfloat16", "bfloat16", True, "batched"),
    (50, 513, 1024, 64, "float16", "float32", False, "batched"),
    (17, 4096, 4096, 128, "float16", "float16", True, "auto"),
    (20, 301, 512, 128, "float16", "float16", True, "gemm"),
    (33, 1001, 2048, 64, "bfloat16", "bfloat16", True, "gemm"),
    (100, 264, 320, 64, "float16", "float32", True, "gemm"),
    (130, 520, 1024, 128, "bfloat16", "float16", False, "gemm"),
    (300, 1023, 256, 128, "float16", "bfloat16", True, "gemm"),
    (1, 64, 64, 64, "float16", "float16", True, "auto"),
])
def test_epilogue(M, N, K, g, xdt, odt, zp, kernel):
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    say("epilogue", M, N, K, g, xdt, odt, zp, kernel)
    pd, pk, Xd, x64, bias, res = _case(M, N, K, g, xdt, odt, zp, M + N)
    kern = {"auto": awq.AWQ_KERNEL_AUTO, "gemv": awq.AWQ_KERNEL_GEMV, "batched": awq.AWQ_KERNEL_BATCHED,
            "gemm": awq.AWQ_KERNEL_GEMM}[kernel]
    kw = dict(group_size=g, kernel=kern, out_dtype=getattr(torch, odt))
    plain = awq.awq_linear_ex(Xd, *pd, **kw)
    assert torch.equal(awq.awq_linear_epilogue(Xd, *pd, **kw), plain)
    exact = M <= 32 or kernel in ("gemv", "batched")
    for act, b, r in (("none", bias, None), ("none", None, res), ("relu", bias, res), ("silu", None, res),
                      ("gelu", bias, None), ("gelu_tanh", bias, res)):
        y = awq.awq_linear_epilogue(Xd, *pd, bias=b, residual=r, activation=act, **kw)
        want, bound = _reference(x64, pk, K, g, b, r, act, odt, exact)
        err = np.abs(out_to_f64(y) - want)
        assert (err <= bound).all(), (act, float(np.max(err / np.maximum(bound, 1e-300))))


@pytest.mark.parametrize("M,splits", [(1, False), (24, True), (200, True), (40, True)])
def test_residual_in_place(M, splits):
    """residual is the output: the residual stream updated in place, the same
    bits as out of place, and again with a graph."""
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    N, K, g = 4096, 4096, 128
    pd, pk, Xd, x64, bias, res = _case(M, N, K, g, "float16", "float16", True, M)
    want = awq.awq_linear_epilogue(Xd, *pd, bias=bias, residual=res, activation="silu")
    assert (awq.awq_linear_workspace_size(M, N, K, g) > 0) == splits
    y = res.clone()
    got = awq.awq_linear_epilogue(Xd, *pd, bias=bias, residual=y, activation="silu", out=y)
    assert got is y and torch.equal(y, want)
    y.copy_(res)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        awq.awq_linear_epilogue(Xd, *pd, bias=bias, residual=y, activation="silu", out=y)
    for _ in range(3):
        y.copy_(res)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want)


def test_large_tile_with_unaligned_arrays():
    """The 256-row tile (every CU has one), odd N, bias and residual at odd
    element offsets."""
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    M, N, K, g = 4100, 4101, 256, 128
    pd, pk, Xd, x64, bias, res = _case(M, N, K, g, "bfloat16", "bfloat16", True, 9)
    big = torch.zeros(M * N + 3, dtype=torch.bfloat16, device=dev())
    big[3:] = res.flatten()
    r = big[3:].view(M, N)
    y = awq.awq_linear_epilogue(Xd, *pd, bias=bias, residual=r, activation="gelu_tanh")
    rows = np.array([0, 1, 255, 256, 2049, 4095, 4096, 4099])
    want, bound = _reference(x64[rows], pk, K, g, bias, r[torch.from_numpy(rows).to(dev())], "gelu_tanh",
                             "bfloat16", False)
    assert (np.abs(out_to_f64(y[torch.from_numpy(rows).to(dev())]) - want) <= bound).all()
    aligned = awq.awq_linear_epilogue(Xd, *pd, bias=bias, residual=res, activation="gelu_tanh")
    assert torch.equal(y, aligned)
    N = 4104                                                # whole 16-byte pieces
    pd, pk, Xd, x64, bias, res = _case(M, N, K, g, "float16", "float16", True, 10)
    y = awq.awq_linear_epilogue(Xd, *pd, bias=bias, residual=res, activation="gelu")
    want, bound = _reference(x64[rows], pk, K, g, bias, res[torch.from_numpy(rows).to(dev())], "gelu",
                             "float16", False)
    assert (np.abs(out_to_f64(y[torch.from_numpy(rows).to(dev())]) - want) <= bound).all()


def test_activations_at_the_ends():
    """One-channel layer whose sums are the inputs: large, tiny and infinite
    pre-activations, fp32 out."""
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    K = 64
    W = np.zeros((1, K), np.float16)
    W[0, 0] = 1.0
    pk = quantize_pack(W, QuantConfig(group_size=K))
    pd = [to_dev(a) for a in pk]
    w0 = float(dequantize(unpack_codes(pk[0], K), pk[1], pk[2], K)[0, 0])
    x = np.array([0.0, 1e-7, -1e-4, 0.5, -0.5, 3, -3, 5, -5, 8, -8, 12, -12, 60000, -60000], np.float16)
    X = np.zeros((len(x), K), np.float16)
    X[:, 0] = x
    s = x.astype(np.float64) * w0
    for act, f in ACTS.items():
        with np.errstate(over="ignore"):
            want = f(s)
        y = awq.awq_linear_epilogue(to_dev(X), *pd, activation=act, group_size=K, out_dtype=torch.float32,
                                    residual=torch.zeros((len(x), 1), device=dev()))
        # fp32 activations: 2^-19 relative (e^-z of |z| <= 100 carries 100 2^-24), flushed below 1e-30
        assert (np.abs(out_to_f64(y)[:, 0] - want) <= 2.0 ** -17 * np.abs(want) + 1e-30).all(), act


def test_infinite_pre_activation():
    """A bias of infinity passes every activation as their limit, and stays in
    its column."""
    import bit_weight_only_quantize_amd as awq
    torch = torch_mod()
    M, N, K, g = 40, 136, 128, 128
    pd, pk, Xd, x64, bias, _ = _case(M, N, K, g, "float16", "float16", True, 3)
    for m in (1, 20, 40):
        for act in ACTS:
            want = awq.awq_linear_epilogue(Xd[:m], *pd, bias=bias, activation=act)
            b = bias.clone()
            b[[0, 70]] = float("inf")
            y = awq.awq_linear_epilogue(Xd[:m], *pd, bias=b, activation=act)
            assert torch.isposinf(y[:, [0, 70]]).all(), (m, act)
            keep = [n for n in range(N) if n not in (0, 70)]
            assert torch.equal(y[:, keep], want[:, keep])
