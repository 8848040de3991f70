"""ctypes binding of libawq355.so (argument marshalling only).

Every function here validates its tensors (dtype, shape, device), allocates
outputs (and, where asked, a workspace) with torch when the caller does not
pass them, and calls the C entry point of the same name on the current HIP
stream.  All computation happens in the library's HIP
kernels; there is no fallback of any kind.  If the library is missing or
cannot be loaded, importing this module raises ImportError.
"""

from __future__ import annotations

import ctypes
import os

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libawq355.so")

AWQ_OK = 0
AWQ_ERR_INVALID_ARG = 1
AWQ_ERR_UNSUPPORTED = 2
AWQ_ERR_WORKSPACE = 3
AWQ_ERR_HIP = 4
AWQ_ERR_NONFINITE = 5

AWQ_F16, AWQ_BF16, AWQ_F32 = 0, 1, 2
AWQ_KERNEL_AUTO, AWQ_KERNEL_GEMV, AWQ_KERNEL_GEMM, AWQ_KERNEL_BATCHED = 0, 1, 2, 3
AWQ_EPILOGUE_NONE, AWQ_EPILOGUE_SILU_MUL = 0, 1
AWQ_ACT_NONE, AWQ_ACT_RELU, AWQ_ACT_SILU, AWQ_ACT_GELU, AWQ_ACT_GELU_TANH = 0, 1, 2, 3, 4
ACTIVATIONS = {"none": AWQ_ACT_NONE, "relu": AWQ_ACT_RELU, "silu": AWQ_ACT_SILU,
               "gelu": AWQ_ACT_GELU, "gelu_tanh": AWQ_ACT_GELU_TANH}
AWQ_MAX_PARTS = 4
AWQ_GEMV_MAX_M = 16
AWQ_BATCHED_MAX_M = 64
AWQ_KV_MIN_PAGE, AWQ_KV_MAX_PAGE, AWQ_KV_MAX_HEADS = 16, 1024, 1024
AWQ_ROPE_MAX_DIM = 512
ROPE_SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3, "bands": 4}

#: Every symbol include/awq355.h declares.
EXPORTS = (
    "awq_quantize_pack",
    "awq_dequantize",
    "awq_linear",
    "awq_linear_ex",
    "awq_linear_epilogue",
    "awq_linear_workspace_size",
    "awq_linear_ws",
    "awq_linear_noalloc",
    "awq_linear_fused_workspace_size",
    "awq_linear_fused",
    "awq_scale_search_workspace_size",
    "awq_scale_search",
    "awq_scale_search_workspace_size_ex",
    "awq_scale_search_ex",
    "awq_kv_assign",
    "awq_kv_append",
    "awq_kv_gather",
    "awq_kv_attention",
    "awq_kv_attention_workspace_size",
    "awq_kv_attention_ex",
    "awq_kv_attention_ex_workspace_size",
    "awq_kv_copy_pages",
    "awq_kv_fork",
    "awq_kv_release",
    "awq_kv_release_workspace_size",
    "awq_kv_compact",
    "awq_kv_compact_workspace_size",
    "awq_rope_frequencies",
    "awq_rope",
    "awq_kv_append_rope",
    "awq_status_string",
    "awq_last_error",
    "awq_version",
)


class awq_config(ctypes.Structure):
    _fields_ = [("w_bit", ctypes.c_int32), ("group_size", ctypes.c_int32),
                ("zero_point", ctypes.c_int32)]


class awq_linear_part(ctypes.Structure):
    _fields_ = [("qweight", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("zeros", ctypes.c_void_p), ("N", ctypes.c_int64), ("Y", ctypes.c_void_p)]


class awq_search_options(ctypes.Structure):
    _fields_ = [("duo_scaling", ctypes.c_int32), ("apply_clip", ctypes.c_int32)]


class awq_epilogue(ctypes.Structure):
    _fields_ = [("bias", ctypes.c_void_p), ("residual", ctypes.c_void_p),
                ("activation", ctypes.c_int32)]


class awq_kv_cache(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("zeros", ctypes.c_void_p), ("num_pages", ctypes.c_int64),
                ("page_size", ctypes.c_int32), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32)]


class awq_kv_attention_options(ctypes.Structure):
    _fields_ = [("causal", ctypes.c_int32), ("window", ctypes.c_int32), ("sinks", ctypes.c_int32),
                ("prefix_len", ctypes.c_int32), ("prefix_table", ctypes.c_void_p),
                ("prefix_blocks", ctypes.c_int32)]


class awq_rope_args(ctypes.Structure):
    _fields_ = [("positions", ctypes.c_void_p), ("inv_freq", ctypes.c_void_p),
                ("attention_factor", ctypes.c_double), ("rotary_dim", ctypes.c_int32),
                ("interleaved", ctypes.c_int32), ("inverse", ctypes.c_int32)]


class awq_rope_scaling(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("factor", ctypes.c_double), ("original_len", ctypes.c_double),
                ("low", ctypes.c_double), ("high", ctypes.c_double)]


class AwqError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{message} (status {status})")
        self.status = status


def _load():
    # torch bundles its own HIP runtime under the same soname
    # (libamdhip64.so.7).  Importing torch first maps that runtime, and the
    # dynamic loader then resolves this library's dependency to the same copy,
    # so torch's streams and allocations are valid here.  Loading this library
    # first would map /opt/rocm's runtime and torch would add a second one.
    import torch  # noqa: F401

    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m bit_weight_only_quantize_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
    lib.awq_quantize_pack.argtypes = [vp, i64, i64, awq_config, vp, vp, vp, vp, vp, vp]
    lib.awq_quantize_pack.restype = ctypes.c_int
    lib.awq_dequantize.argtypes = [vp, vp, vp, i64, i64, awq_config, vp, i32, vp]
    lib.awq_dequantize.restype = ctypes.c_int
    lib.awq_linear.argtypes = [vp, i32, vp, vp, vp, i64, i64, i64, awq_config, vp, i32, vp]
    lib.awq_linear.restype = ctypes.c_int
    lib.awq_linear_ex.argtypes = [vp, i32, vp, vp, vp, i64, i64, i64, awq_config, vp, i32, i32, vp,
                                  ctypes.c_size_t, vp]
    lib.awq_linear_ex.restype = ctypes.c_int
    lib.awq_linear_workspace_size.argtypes = [i64, i64, i64, awq_config, i32, i32]
    lib.awq_linear_workspace_size.restype = ctypes.c_size_t
    lib.awq_linear_ws.argtypes = [vp, i32, vp, vp, vp, i64, i64, i64, awq_config, vp, i32, vp,
                                  ctypes.c_size_t, vp]
    lib.awq_linear_ws.restype = ctypes.c_int
    pp = ctypes.POINTER(awq_linear_part)
    lib.awq_linear_fused_workspace_size.argtypes = [pp, i32, i64, i64, awq_config, i32, i32, i32]
    lib.awq_linear_fused_workspace_size.restype = ctypes.c_size_t
    lib.awq_linear_fused.argtypes = [vp, i32, pp, i32, i64, i64, awq_config, i32, vp, i32, i32,
                                     vp, ctypes.c_size_t, vp]
    lib.awq_linear_fused.restype = ctypes.c_int
    lib.awq_linear_noalloc.argtypes = [vp, i32, vp, vp, vp, i64, i64, i64, awq_config, vp, i32,
                                       vp]
    lib.awq_linear_noalloc.restype = ctypes.c_int
    lib.awq_scale_search_workspace_size.argtypes = [i64, i64, i64, awq_config, i32]
    lib.awq_scale_search_workspace_size.restype = ctypes.c_size_t
    lib.awq_scale_search.argtypes = [vp, vp, i64, i64, i64, awq_config,
                                     ctypes.POINTER(ctypes.c_double), i32, vp, ctypes.c_size_t,
                                     ctypes.POINTER(ctypes.c_int32),
                                     ctypes.POINTER(ctypes.c_double), vp, vp, vp, vp, vp]
    lib.awq_scale_search.restype = ctypes.c_int
    po = ctypes.POINTER(awq_search_options)
    lib.awq_scale_search_workspace_size_ex.argtypes = [i64, i64, i64, awq_config, i32, po]
    lib.awq_scale_search_workspace_size_ex.restype = ctypes.c_size_t
    lib.awq_scale_search_ex.argtypes = [vp, vp, i64, i64, i64, awq_config,
                                        ctypes.POINTER(ctypes.c_double), i32, po, vp,
                                        ctypes.c_size_t, ctypes.POINTER(ctypes.c_int32),
                                        ctypes.POINTER(ctypes.c_double), vp, vp, vp, vp, vp, vp]
    lib.awq_scale_search_ex.restype = ctypes.c_int
    lib.awq_linear_epilogue.argtypes = [vp, i32, vp, vp, vp, i64, i64, i64, awq_config,
                                        ctypes.POINTER(awq_epilogue), vp, i32, i32, vp,
                                        ctypes.c_size_t, vp]
    lib.awq_linear_epilogue.restype = ctypes.c_int
    pc = ctypes.POINTER(awq_kv_cache)
    lib.awq_kv_assign.argtypes = [vp, vp, i32, i32, vp, i32, vp, i32, vp, vp, vp, i64, vp, vp]
    lib.awq_kv_assign.restype = ctypes.c_int
    lib.awq_kv_append.argtypes = [vp, vp, i32, i64, i64, i64, pc, awq_config, vp, vp, vp]
    lib.awq_kv_append.restype = ctypes.c_int
    lib.awq_kv_gather.argtypes = [pc, awq_config, vp, i64, vp, vp, i32, vp]
    lib.awq_kv_gather.restype = ctypes.c_int
    lib.awq_kv_attention.argtypes = [vp, i32, i64, i64, i32, pc, awq_config, vp, i32, vp, vp, i32,
                                     i32, i64, ctypes.c_float, i32, i32, vp, vp, vp,
                                     ctypes.c_size_t, vp]
    lib.awq_kv_attention.restype = ctypes.c_int
    lib.awq_kv_attention_workspace_size.argtypes = [i64, i32, i32, pc, awq_config, i32, i64, i32]
    lib.awq_kv_attention_workspace_size.restype = ctypes.c_size_t
    pa = ctypes.POINTER(awq_kv_attention_options)
    lib.awq_kv_attention_ex.argtypes = [vp, i32, i64, i64, i32, pc, awq_config, vp, i32, vp, vp, i32,
                                        i32, i64, ctypes.c_float, pa, vp, vp, vp, ctypes.c_size_t, vp]
    lib.awq_kv_attention_ex.restype = ctypes.c_int
    lib.awq_kv_attention_ex_workspace_size.argtypes = [i64, i32, i32, pc, awq_config, i32, i64, pa]
    lib.awq_kv_attention_ex_workspace_size.restype = ctypes.c_size_t
    lib.awq_kv_copy_pages.argtypes = [pc, awq_config, vp, vp, i64, vp]
    lib.awq_kv_copy_pages.restype = ctypes.c_int
    lib.awq_kv_fork.argtypes = [pc, awq_config, vp, vp, vp, i32, vp, i32, i32, vp, vp, i32, vp, vp, vp]
    lib.awq_kv_fork.restype = ctypes.c_int
    lib.awq_kv_release.argtypes = [vp, i32, i32, i32, vp, vp, vp, vp, i64, vp, i32, vp, vp, i32, vp, vp,
                                   ctypes.c_size_t, vp]
    lib.awq_kv_release.restype = ctypes.c_int
    lib.awq_kv_release_workspace_size.argtypes = [i64, i32]
    lib.awq_kv_release_workspace_size.restype = ctypes.c_size_t
    lib.awq_kv_compact.argtypes = [pc, awq_config, vp, i32, i32, vp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    lib.awq_kv_compact.restype = ctypes.c_int
    lib.awq_kv_compact_workspace_size.argtypes = [i64, i32]
    lib.awq_kv_compact_workspace_size.restype = ctypes.c_size_t
    pr = ctypes.POINTER(awq_rope_args)
    lib.awq_rope_frequencies.argtypes = [i32, ctypes.c_double, ctypes.POINTER(awq_rope_scaling),
                                         ctypes.POINTER(ctypes.c_double), ctypes.POINTER(ctypes.c_double)]
    lib.awq_rope_frequencies.restype = ctypes.c_int
    lib.awq_rope.argtypes = [vp, vp, i32, i64, i64, vp, vp, i32, i64, i64, i32, i64, i32, pr, vp]
    lib.awq_rope.restype = ctypes.c_int
    lib.awq_kv_append_rope.argtypes = [vp, vp, i32, i64, i64, vp, vp, i32, i64, i64, i64, pc, awq_config, vp, pr, vp,
                                       vp]
    lib.awq_kv_append_rope.restype = ctypes.c_int
    lib.awq_status_string.argtypes = [ctypes.c_int]
    lib.awq_status_string.restype = ctypes.c_char_p
    lib.awq_last_error.argtypes = []
    lib.awq_last_error.restype = ctypes.c_char_p
    lib.awq_version.argtypes = []
    lib.awq_version.restype = ctypes.c_char_p
    return lib


lib = _load()
import torch as _TORCH  # noqa: E402  (after _load, which says why)


def config(group_size: int = 128, w_bit: int = 4, zero_point: bool = True) -> awq_config:
    return awq_config(int(w_bit), int(group_size), int(bool(zero_point)))


def check(status: int, what: str) -> None:
    if status != AWQ_OK:
        msg = lib.awq_last_error().decode() or lib.awq_status_string(status).decode()
        raise AwqError(status, f"{what}: {msg}")


# ---------------------------------------------------------------------------
# torch-facing wrappers
# ---------------------------------------------------------------------------
#
# Every wrapper checks, before any C call: that each argument is a tensor of
# the expected dtype and shape (so no kernel can read or write past an
# allocation), then that all tensors sit on one GPU, contiguously.  Shape and
# dtype errors raise TypeError / ValueError even on machines without a GPU.

def _torch():
    return _TORCH


def _tensor(t, name, dtype=None, shape=None):
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor, got {type(t).__name__}")
    if dtype is not None:
        ok = t.dtype in dtype if isinstance(dtype, tuple) else t.dtype == dtype
        if not ok:
            raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t


def _placed(*named):
    """All (tensor, name) pairs on one GPU and contiguous; returns the device."""
    dev = None
    for t, name in named:
        if t.device.type != "cuda":
            raise ValueError(f"{name} must be on a GPU device, got {t.device}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise ValueError(f"{name} is on {t.device}, expected {dev} like the other tensors")
    return dev


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr() if t.numel() else 0)


def _stream(device):
    torch = _torch()
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


# The calls below serve single tokens, where a few microseconds of Python are
# the kernel's own time: their checks take the cheap form first (identity of
# the dtype, comparison of the shape, device index) and come back to the
# functions above only to say what is wrong.

def _check(t, name, dtype, shape):
    """_tensor for one dtype and a shape tuple."""
    try:
        if t.dtype is dtype and t.shape == shape:
            return
    except AttributeError:
        pass
    _tensor(t, name, dtype, shape)


def _one_gpu(*named):
    """_placed, as a device index; None entries are skipped."""
    d = named[0][0].get_device()
    for pair in named:
        if pair is not None:
            t = pair[0]
            if d < 0 or t.get_device() != d or not t.is_contiguous():
                _placed(*[p for p in named if p is not None])
    return d


def _launch(fn, device, *args):
    """fn(*args, current stream) with `device` current, as the C calls want it; its status."""
    torch = _torch()                                # (a tensor on the device has initialised it)
    if torch._C._cuda_getDevice() == device:
        return fn(*args, torch._C._cuda_getCurrentRawStream(device))
    with torch.cuda.device(device):
        return fn(*args, torch._C._cuda_getCurrentRawStream(device))


def _address(t):
    """The pointer argument of a tensor or None (an empty tensor's is NULL too)."""
    return None if t is None else t.data_ptr() or None


def _scratch(workspace, need, like):
    """(tensor, bytes) of a workspace argument: 'auto', a tensor or None."""
    torch = _torch()
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be a tensor, None or 'auto'")
        if need == 0:
            return None, 0
        return like.new_empty(need, dtype=torch.uint8), need
    if workspace is None:
        return None, 0
    _tensor(workspace, "workspace")
    return workspace, workspace.numel() * workspace.element_size()


_CONFIGS = {(g, z): config(g, zero_point=z) for g in (64, 128) for z in (False, True)}


def _dtype_code(dt):
    torch = _torch()
    if dt == torch.float16:
        return AWQ_F16
    if dt == torch.bfloat16:
        return AWQ_BF16
    if dt == torch.float32:
        return AWQ_F32
    raise TypeError(f"unsupported dtype {dt}")


def empty_packed(N: int, K: int, group_size: int, device, zero_point: bool = True):
    """Allocate (qweight int32 [N][K/8], scales fp16 [N][K/g], zeros uint8 [N][K/g]);
    zeros is None for the symmetric grid (zero_point=False)."""
    torch = _torch()
    G = K // group_size
    return (torch.empty((N, K // 8), dtype=torch.int32, device=device),
            torch.empty((N, G), dtype=torch.float16, device=device),
            torch.empty((N, G), dtype=torch.uint8, device=device) if zero_point else None)


def _check_packed(qweight, scales, zeros, K, group_size):
    """Packed layer tensors for input width K (zeros None: the symmetric
    grid); returns N."""
    torch = _torch()
    if group_size <= 0 or K % group_size or K % 8:
        raise ValueError(f"K={K} must be a multiple of 8 and of group_size={group_size}")
    _tensor(qweight, "qweight", torch.int32)
    if qweight.dim() != 2:
        raise ValueError("qweight must be 2-D [N][K/8]")
    N = qweight.shape[0]
    _tensor(qweight, "qweight", shape=(N, K // 8))
    _tensor(scales, "scales", torch.float16, (N, K // group_size))
    if zeros is not None:
        _tensor(zeros, "zeros", torch.uint8, (N, K // group_size))
    return N


def _zp_ptr(zeros):
    return ctypes.c_void_p(0) if zeros is None else _ptr(zeros)


def awq_quantize_pack(W, group_size: int = 128, s=None, nonfinite_count=None, out=None,
                      zero_point: bool = True):
    """Quantize and pack W (fp16 [N][K], on the GPU).  Returns (qweight,
    scales, zeros); zeros is None for the symmetric grid (zero_point=False)."""
    torch = _torch()
    _tensor(W, "W", torch.float16)
    if W.dim() != 2:
        raise ValueError("W must be 2-D [N][K]")
    N, K = W.shape
    if group_size <= 0 or K % group_size or K % 8:
        raise ValueError(f"K={K} must be a multiple of 8 and of group_size={group_size}")
    if out is not None:
        qw, sc, zr = out
        if _check_packed(qw, sc, zr, K, group_size) != N:
            raise ValueError("out's packed tensors are not for N rows")
        if (zr is None) == bool(zero_point):
            raise ValueError("out's zeros must be a tensor exactly when zero_point is set")
    named = [(W, "W")]
    sp = ctypes.c_void_p(0)
    if s is not None:
        _tensor(s, "s", torch.float32, (K,))
        named.append((s, "s"))
        sp = _ptr(s)
    cp = ctypes.c_void_p(0)
    if nonfinite_count is not None:
        _tensor(nonfinite_count, "nonfinite_count", torch.int32)
        if nonfinite_count.numel() < 1:
            raise ValueError("nonfinite_count must hold one element")
        named.append((nonfinite_count, "nonfinite_count"))
        cp = _ptr(nonfinite_count)
    dev = _placed(*named)
    if out is None:
        qw, sc, zr = empty_packed(N, K, group_size, dev, zero_point)
    _placed((W, "W"), (qw, "qweight"), (sc, "scales"), *([] if zr is None else [(zr, "zeros")]))
    st = lib.awq_quantize_pack(_ptr(W), N, K, config(group_size, zero_point=zero_point), sp,
                               _ptr(qw), _ptr(sc), _zp_ptr(zr), cp, _stream(dev))
    check(st, "awq_quantize_pack")
    return qw, sc, zr


def awq_dequantize(qweight, scales, zeros, K: int, group_size: int = 128, out_dtype=None,
                   out=None):
    """(code - zero) * scale as a [N][K] tensor: float32 (exact, the default)
    or float16 (rounded once); zeros None for the symmetric grid."""
    torch = _torch()
    N = _check_packed(qweight, scales, zeros, K, group_size)
    odt = torch.float32 if out_dtype is None else out_dtype
    if out is not None:
        _tensor(out, "out", (torch.float16, torch.float32), (N, K))
        odt = out.dtype
    elif odt not in (torch.float16, torch.float32):
        raise TypeError(f"out_dtype {odt} is not float16 or float32")
    dev = _placed((qweight, "qweight"), (scales, "scales"),
                  *([] if zeros is None else [(zeros, "zeros")]))
    if out is None:
        out = torch.empty((N, K), dtype=odt, device=dev)
    _placed((qweight, "qweight"), (out, "out"))
    st = lib.awq_dequantize(_ptr(qweight), _ptr(scales), _zp_ptr(zeros), N, K,
                            config(group_size, zero_point=zeros is not None), _ptr(out),
                            _dtype_code(odt), _stream(dev))
    check(st, "awq_dequantize")
    return out


def _linear_args(X, qweight, scales, zeros, group_size, out_dtype, out):
    """Validate a linear call; returns (M, N, K, out, device)."""
    torch = _torch()
    _tensor(X, "X", (torch.float16, torch.bfloat16))
    if X.dim() != 2:
        raise ValueError("X must be 2-D [M][K]")
    M, K = X.shape
    N = _check_packed(qweight, scales, zeros, K, group_size)
    ydt = (torch.float16, torch.bfloat16, torch.float32)
    if out is not None:
        _tensor(out, "out", ydt, (M, N))
    elif out_dtype is not None and out_dtype not in ydt:
        raise TypeError(f"out_dtype {out_dtype} is not float16, bfloat16 or float32")
    dev = _placed((X, "X"), (qweight, "qweight"), (scales, "scales"),
                  *([] if zeros is None else [(zeros, "zeros")]))
    if out is None:
        out = torch.empty((M, N), dtype=X.dtype if out_dtype is None else out_dtype, device=dev)
    _placed((X, "X"), (out, "out"))
    return M, N, K, out, dev


def awq_linear_workspace_size(M: int, N: int, K: int, group_size: int = 128,
                              x_dtype=None, kernel: int = AWQ_KERNEL_AUTO) -> int:
    """Workspace bytes the GEMM path needs (awq_linear_workspace_size); x_dtype
    is a torch dtype (default float16)."""
    torch = _torch()
    xd = AWQ_F16 if x_dtype is None or x_dtype == torch.float16 else _dtype_code(x_dtype)
    return int(lib.awq_linear_workspace_size(M, N, K, config(group_size), xd, int(kernel)))


def _workspace_arg(workspace, need, dev):
    torch = _torch()
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError("workspace must be a tensor, None or 'auto'")
        if need == 0:
            return None
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if workspace is None:
        return None
    _tensor(workspace, "workspace")
    _placed((workspace, "workspace"))
    if workspace.device != dev:
        raise ValueError(f"workspace is on {workspace.device}, expected {dev}")
    return workspace


def awq_linear_ex(X, qweight, scales, zeros, kernel: int = AWQ_KERNEL_AUTO,
                  group_size: int = 128, out_dtype=None, out=None, workspace="auto"):
    """Y = X * deq(W)^T with an explicit kernel choice (AWQ_KERNEL_*).

    ``workspace``: 'auto' (a torch-allocated buffer of
    awq_linear_workspace_size bytes when the call needs one), a uint8 tensor
    of at least that size (any contents), or None (the scratch-free plan, as
    awq_linear)."""
    if isinstance(workspace, str) and workspace != "auto":
        raise ValueError("workspace must be a tensor, None or 'auto'")
    if workspace is not None and not isinstance(workspace, str):
        _tensor(workspace, "workspace")
    M, N, K, out, dev = _linear_args(X, qweight, scales, zeros, group_size, out_dtype, out)
    need = awq_linear_workspace_size(M, N, K, group_size, X.dtype, kernel)
    ws = _workspace_arg(workspace, need, dev)
    st = lib.awq_linear_ex(_ptr(X), _dtype_code(X.dtype), _ptr(qweight), _ptr(scales),
                           _zp_ptr(zeros), M, N, K,
                           config(group_size, zero_point=zeros is not None), _ptr(out),
                           _dtype_code(out.dtype), int(kernel),
                           ctypes.c_void_p(0) if ws is None else _ptr(ws),
                           0 if ws is None else ws.numel() * ws.element_size(), _stream(dev))
    check(st, "awq_linear_ex")
    return out


def awq_linear_epilogue(X, qweight, scales, zeros, bias=None, residual=None,
                        activation: str = "none", kernel: int = AWQ_KERNEL_AUTO,
                        group_size: int = 128, out_dtype=None, out=None, workspace="auto"):
    """activation(X * deq(W)^T + bias) + residual in one call; activation one of
    ACTIVATIONS.  bias [N] and residual [M][N] have the output's dtype (that of
    X unless out or out_dtype says otherwise); residual may be `out` itself.
    Kernel and workspace as in awq_linear_ex."""
    torch = _torch()
    act = ACTIVATIONS.get(activation)
    if act is None:
        raise ValueError(f"activation {activation!r} is not one of {sorted(ACTIVATIONS)}")
    _tensor(X, "X", (torch.float16, torch.bfloat16))
    if X.dim() != 2:
        raise ValueError("X must be 2-D [M][K]")
    M, K = X.shape
    if group_size <= 0 or K % group_size or K % 8:
        raise ValueError(f"K={K} must be a multiple of 8 and of group_size={group_size}")
    _tensor(qweight, "qweight", torch.int32)
    N = qweight.shape[0] if qweight.dim() else 0
    _check(qweight, "qweight", torch.int32, (N, K // 8))
    _check(scales, "scales", torch.float16, (N, K // group_size))
    if zeros is not None:
        _check(zeros, "zeros", torch.uint8, (N, K // group_size))
    odt = out.dtype if out is not None else X.dtype if out_dtype is None else out_dtype
    if odt not in (torch.float16, torch.bfloat16, torch.float32):
        raise TypeError(f"out_dtype {odt} is not float16, bfloat16 or float32")
    if out is not None:
        _check(out, "out", odt, (M, N))
    if bias is not None:
        _check(bias, "bias", odt, (N,))
    if residual is not None:
        _check(residual, "residual", odt, (M, N))
    xd = _dtype_code(X.dtype)
    od = xd if odt is X.dtype else _dtype_code(odt)
    cfg = _CONFIGS.get((group_size, zeros is not None)) or config(group_size, zero_point=zeros is not None)
    need = 0 if workspace is None else lib.awq_linear_workspace_size(M, N, K, cfg, xd, kernel)
    ws, ws_bytes = _scratch(workspace, need, X)
    dev = _one_gpu((X, "X"), (qweight, "qweight"), (scales, "scales"),
                   None if zeros is None else (zeros, "zeros"),
                   None if bias is None else (bias, "bias"),
                   None if residual is None else (residual, "residual"),
                   None if out is None else (out, "out"), None if ws is None else (ws, "workspace"))
    if out is None:
        out = X.new_empty((M, N), dtype=odt)
    st = _launch(lib.awq_linear_epilogue, dev, _address(X), xd, _address(qweight), _address(scales),
                 _address(zeros), M, N, K, cfg, awq_epilogue(_address(bias), _address(residual), act),
                 _address(out), od, kernel, _address(ws), ws_bytes)
    check(st, "awq_linear_epilogue")
    return out


def awq_linear(X, qweight, scales, zeros, group_size: int = 128, out_dtype=None, out=None):
    """Y = X * deq(W)^T with no scratch memory (the C awq_linear): small M
    runs the GEMV, larger M the GEMM without a K split; bf16 activations on
    the GEMM path raise AwqError (use awq_linear_ex or awq_linear_ws)."""
    M, N, K, out, dev = _linear_args(X, qweight, scales, zeros, group_size, out_dtype, out)
    st = lib.awq_linear(_ptr(X), _dtype_code(X.dtype), _ptr(qweight), _ptr(scales),
                        _zp_ptr(zeros), M, N, K, config(group_size, zero_point=zeros is not None),
                        _ptr(out), _dtype_code(out.dtype), _stream(dev))
    check(st, "awq_linear")
    return out


def awq_linear_ws(X, qweight, scales, zeros, workspace, group_size: int = 128, out_dtype=None,
                  out=None):
    """awq_linear with a caller workspace (uint8 tensor of at least
    awq_linear_workspace_size bytes, any contents); the call allocates nothing."""
    M, N, K, out, dev = _linear_args(X, qweight, scales, zeros, group_size, out_dtype, out)
    ws = _workspace_arg(workspace, 0, dev)
    st = lib.awq_linear_ws(_ptr(X), _dtype_code(X.dtype), _ptr(qweight), _ptr(scales),
                           _zp_ptr(zeros), M, N, K,
                           config(group_size, zero_point=zeros is not None), _ptr(out),
                           _dtype_code(out.dtype),
                           ctypes.c_void_p(0) if ws is None else _ptr(ws),
                           0 if ws is None else ws.numel() * ws.element_size(), _stream(dev))
    check(st, "awq_linear_ws")
    return out


def awq_linear_noalloc(X, qweight, scales, zeros, group_size: int = 128, out_dtype=None,
                       out=None):
    """awq_linear_ws with the library's static device scratch instead of a
    workspace: allocates nothing (pass `out` to allocate nothing here either).
    Calls that may overlap in time on one GPU must not be made."""
    M, N, K, out, dev = _linear_args(X, qweight, scales, zeros, group_size, out_dtype, out)
    st = lib.awq_linear_noalloc(_ptr(X), _dtype_code(X.dtype), _ptr(qweight), _ptr(scales),
                                _zp_ptr(zeros), M, N, K,
                                config(group_size, zero_point=zeros is not None), _ptr(out),
                                _dtype_code(out.dtype), _stream(dev))
    check(st, "awq_linear_noalloc")
    return out


def awq_linear_fused(X, parts, epilogue: str = "none", group_size: int = 128, out_dtype=None,
                     outs=None, kernel: int = AWQ_KERNEL_AUTO, workspace="auto"):
    """Several projections of one X (each part a (qweight, scales, zeros)
    tuple of the same K, group size and zero-point mode).  epilogue 'none'
    returns [X W_i^T for each part]; 'silu_mul' takes (gate, up) and returns
    silu(X Wg^T) * (X Wu^T).  `outs` optionally gives the output tensors (a
    list for 'none', one tensor for 'silu_mul')."""
    torch = _torch()
    if epilogue not in ("none", "silu_mul"):
        raise ValueError("epilogue must be 'none' or 'silu_mul'")
    if not 1 <= len(parts) <= AWQ_MAX_PARTS:
        raise ValueError(f"1 to {AWQ_MAX_PARTS} parts")
    pair = epilogue == "silu_mul"
    if pair and len(parts) != 2:
        raise ValueError("'silu_mul' takes exactly two parts (gate, up)")
    if isinstance(workspace, str) and workspace != "auto":
        raise ValueError("workspace must be a tensor, None or 'auto'")
    _tensor(X, "X", (torch.float16, torch.bfloat16))
    if X.dim() != 2:
        raise ValueError("X must be 2-D [M][K]")
    M, K = X.shape
    Ns = [_check_packed(qw, sc, zr, K, group_size) for (qw, sc, zr) in parts]
    zp = parts[0][2] is not None
    if any((zr is not None) != zp for (_, _, zr) in parts):
        raise ValueError("all parts must share the zero-point mode")
    if pair and Ns[0] != Ns[1]:
        raise ValueError("gate and up must have the same N")
    ydt = (torch.float16, torch.bfloat16, torch.float32)
    odt = X.dtype if out_dtype is None else out_dtype
    if odt not in ydt:
        raise TypeError(f"out_dtype {odt} is not float16, bfloat16 or float32")
    if outs is not None:
        outl = [outs] if pair else list(outs)
        if len(outl) != (1 if pair else len(parts)):
            raise ValueError("one output per part ('none') or one H ('silu_mul')")
        for o, n in zip(outl, Ns[:len(outl)]):
            _tensor(o, "out", ydt, (M, n))
        if len({o.dtype for o in outl}) != 1:
            raise TypeError("every output must have the same dtype")
        odt = outl[0].dtype
    named = [(X, "X")]
    for i, (qw, sc, zr) in enumerate(parts):
        named += [(qw, f"parts[{i}].qweight"), (sc, f"parts[{i}].scales")]
        if zr is not None:
            named.append((zr, f"parts[{i}].zeros"))
    dev = _placed(*named)
    if outs is None:
        outl = [torch.empty((M, n), dtype=odt, device=dev) for n in (Ns[:1] if pair else Ns)]
    _placed(*[(o, "out") for o in outl])
    arr = (awq_linear_part * len(parts))()
    for i, (qw, sc, zr) in enumerate(parts):
        arr[i] = awq_linear_part(qw.data_ptr() if qw.numel() else None,
                                 sc.data_ptr() if sc.numel() else None,
                                 None if zr is None or not zr.numel() else zr.data_ptr(), Ns[i],
                                 None if pair else (outl[i].data_ptr() if outl[i].numel() else None))
    cfg = config(group_size, zero_point=zp)
    epi = AWQ_EPILOGUE_SILU_MUL if pair else AWQ_EPILOGUE_NONE
    xd = _dtype_code(X.dtype)
    need = int(lib.awq_linear_fused_workspace_size(arr, len(parts), M, K, cfg, xd, epi,
                                                   int(kernel)))
    if workspace is not None and not isinstance(workspace, str):
        _tensor(workspace, "workspace")
    ws = _workspace_arg(workspace, need, dev)
    H = outl[0] if pair else None
    st = lib.awq_linear_fused(_ptr(X), xd, arr, len(parts), M, K, cfg, epi,
                              ctypes.c_void_p(0) if H is None else _ptr(H), _dtype_code(odt),
                              int(kernel), ctypes.c_void_p(0) if ws is None else _ptr(ws),
                              0 if ws is None else ws.numel() * ws.element_size(), _stream(dev))
    check(st, "awq_linear_fused")
    return H if pair else outl


def awq_scale_search_workspace_size(M: int, N: int, K: int, group_size: int = 128,
                                    n_alpha: int = 20, zero_point: bool = True,
                                    duo_scaling: bool = False, apply_clip: bool = False) -> int:
    cfg = config(group_size, zero_point=zero_point)
    opts = awq_search_options(int(bool(duo_scaling)), int(bool(apply_clip)))
    return int(lib.awq_scale_search_workspace_size_ex(M, N, K, cfg, n_alpha, ctypes.byref(opts)))


def awq_scale_search(X, W, group_size: int = 128, alphas=None, workspace=None, out=None,
                     zero_point: bool = True, duo_scaling: bool = False,
                     apply_clip: bool = False):
    """Alpha-grid scale search (awq_scale_search_ex).  Returns a dict with
    best_index, losses (numpy fp64), s (fp32 [K] tensor) and the packed
    weights for the chosen s (zeros None for the symmetric grid,
    zero_point=False); with apply_clip also clip_index (uint8 [N][K/g])."""
    torch = _torch()
    _tensor(X, "X", torch.float16)
    _tensor(W, "W", torch.float16)
    if X.dim() != 2 or W.dim() != 2:
        raise ValueError("X must be [M][K] and W [N][K]")
    M, K = X.shape
    N = W.shape[0]
    if W.shape[1] != K:
        raise ValueError(f"W has {W.shape[1]} input channels, X has {K}")
    n_alpha = 20 if alphas is None else len(alphas)
    need = awq_scale_search_workspace_size(M, N, K, group_size, n_alpha, zero_point, duo_scaling,
                                           apply_clip)
    if need == 0:
        check(AWQ_ERR_INVALID_ARG, "awq_scale_search_workspace_size")
    if out is not None:
        qw, sc, zr = out
        if _check_packed(qw, sc, zr, K, group_size) != N:
            raise ValueError("out's packed tensors are not for N rows")
        if (zr is None) == bool(zero_point):
            raise ValueError("out's zeros must be a tensor exactly when zero_point is set")
    if workspace is not None:
        _tensor(workspace, "workspace")
        if workspace.numel() * workspace.element_size() < need:
            raise ValueError(f"workspace holds {workspace.numel() * workspace.element_size()} "
                             f"bytes, {need} needed")
    dev = _placed((X, "X"), (W, "W"))
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    if out is None:
        qw, sc, zr = empty_packed(N, K, group_size, dev, zero_point)
    best_s = torch.empty(K, dtype=torch.float32, device=dev)
    _placed((X, "X"), (workspace, "workspace"), (qw, "qweight"), (sc, "scales"),
            *([] if zr is None else [(zr, "zeros")]))
    a_ptr = None
    if alphas is not None:
        a_arr = (ctypes.c_double * n_alpha)(*[float(a) for a in alphas])
        a_ptr = ctypes.cast(a_arr, ctypes.POINTER(ctypes.c_double))
    best = ctypes.c_int32(-1)
    losses = (ctypes.c_double * n_alpha)()
    opts = awq_search_options(int(bool(duo_scaling)), int(bool(apply_clip)))
    clip = (torch.empty((N, K // group_size), dtype=torch.uint8, device=dev)
            if apply_clip else None)
    st = lib.awq_scale_search_ex(_ptr(X), _ptr(W), M, N, K,
                                 config(group_size, zero_point=zero_point), a_ptr, n_alpha,
                                 ctypes.byref(opts), _ptr(workspace),
                                 workspace.numel() * workspace.element_size(),
                                 ctypes.byref(best), losses, _ptr(best_s), _ptr(qw), _ptr(sc),
                                 _zp_ptr(zr), ctypes.c_void_p(0) if clip is None else _ptr(clip),
                                 _stream(dev))
    check(st, "awq_scale_search_ex")
    res = {"best_index": int(best.value), "losses": np.array(losses[:], dtype=np.float64),
           "s": best_s, "qweight": qw, "scales": sc, "zeros": zr}
    if clip is not None:
        res["clip_index"] = clip
    return res


# ---- the 4-bit paged key/value cache --------------------------------------------

def empty_kv_cache(num_pages: int, num_kv_heads: int, head_dim: int, page_size: int = 64,
                   device="cuda", zero_point: bool = True):
    """Allocate a cache: (codes int32 [pages][2][heads][page_size * head_dim / 8],
    scales fp16 and zeros uint8 [pages][heads][page_size][2]); zeros is None for
    the symmetric grid (zero_point=False).  The contents are arbitrary."""
    torch = _torch()
    _check_cache_sizes(num_pages, num_kv_heads, head_dim, page_size)
    meta = (num_pages, num_kv_heads, page_size, 2)
    return (torch.empty((num_pages, 2, num_kv_heads, page_size * head_dim // 8), dtype=torch.int32,
                        device=device),
            torch.empty(meta, dtype=torch.float16, device=device),
            torch.empty(meta, dtype=torch.uint8, device=device) if zero_point else None)


def _check_cache_sizes(num_pages, num_kv_heads, head_dim, page_size):
    if head_dim not in (64, 128):
        raise ValueError(f"head_dim={head_dim}: supported values are 64 and 128")
    if page_size & (page_size - 1) or not AWQ_KV_MIN_PAGE <= page_size <= AWQ_KV_MAX_PAGE:
        raise ValueError(f"page_size={page_size} is not a power of two in "
                         f"[{AWQ_KV_MIN_PAGE}, {AWQ_KV_MAX_PAGE}]")
    if num_pages < 1 or not 1 <= num_kv_heads <= AWQ_KV_MAX_HEADS:
        raise ValueError(f"num_pages={num_pages} and num_kv_heads={num_kv_heads} must be positive "
                         f"(at most {AWQ_KV_MAX_HEADS} heads)")


def _cache_arg(cache):
    """(awq_kv_cache, awq_config) of a (codes, scales, zeros) cache; its device
    and layout are left to _one_gpu."""
    torch = _torch()
    if not isinstance(cache, (tuple, list)) or len(cache) != 3:
        raise TypeError("cache must be (codes, scales, zeros)")
    codes, scales, zeros = cache
    try:
        fine = codes.dtype is torch.int32 and scales.dtype is torch.float16
    except AttributeError:
        fine = False
    if not fine:
        _tensor(codes, "codes", torch.int32)
        _tensor(scales, "scales", torch.float16)
    shape, meta = codes.shape, scales.shape
    if len(shape) != 4 or shape[1] != 2:
        raise ValueError("codes must be [pages][2][heads][page_size * head_dim / 8]")
    if len(meta) != 4:
        raise ValueError("scales must be [pages][heads][page_size][2]")
    pages, _, heads, words = shape
    page = meta[2]
    if meta != (pages, heads, page, 2):
        _check(scales, "scales", torch.float16, (pages, heads, page, 2))
    if zeros is not None:
        _check(zeros, "zeros", torch.uint8, meta)
    if page < 1 or words * 8 % page:
        raise ValueError(f"codes hold {words} words per head and page, not a multiple of "
                         f"page_size={page} / 8")
    D = words * 8 // page
    _check_cache_sizes(pages, heads, D, page)
    return (awq_kv_cache(codes.data_ptr(), scales.data_ptr(),
                         None if zeros is None else zeros.data_ptr(), pages, page, heads, D),
            _CONFIGS[D, zeros is not None])


def _cache_tensors(cache):
    codes, scales, zeros = cache
    return (codes, "codes"), (scales, "scales"), None if zeros is None else (zeros, "zeros")


def _token_rows(t, name, heads, D):
    """Token stride of a GPU tensor [tokens][heads][D] whose heads are dense."""
    if t.dim() != 3 or t.shape[1:] != (heads, D):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected [tokens][{heads}][{D}]")
    T, width = t.shape[0], heads * D
    if T == 0:
        return width
    s0, s1, s2 = t.stride()
    if s2 != 1 or (heads > 1 and s1 != D):
        raise ValueError(f"{name}: a token's heads must be contiguous")
    if T == 1:
        return width
    if s0 < width or s0 % 8:
        raise ValueError(f"{name}: token stride {s0} must be a multiple of 8 of at least {width}")
    return s0


def _same_gpu(d, *named):
    for t, name in named:
        if t.get_device() != d:
            raise ValueError(f"{name} must be on a GPU device, cuda:{d} like the other tensors, "
                             f"got {t.device}")


def awq_kv_assign(old_lens, new_lens, block_table, free_pages, page_size: int, num_slots: int,
                  out=None):
    """Pages and slots for the new_lens tokens that each request gets on top of
    its old_lens (int32 [B]).  block_table (int32 [B][max_blocks]) is updated in
    place with pages from the front of free_pages (int32).  Returns (seq_lens
    int32 [B], query_start int32 [B + 1], slots int32 [num_slots], pages_used
    int32 [1]), or fills `out`, a tuple of those."""
    i32 = _torch().int32
    _tensor(old_lens, "old_lens", i32)
    _tensor(block_table, "block_table", i32)
    _tensor(free_pages, "free_pages", i32)
    if old_lens.dim() != 1 or free_pages.dim() != 1:
        raise ValueError("old_lens and free_pages must be 1-D")
    if block_table.dim() != 2:
        raise ValueError("block_table must be 2-D [B][max_blocks]")
    B, blocks = old_lens.shape[0], block_table.shape[1]
    _check(new_lens, "new_lens", i32, (B,))
    _check(block_table, "block_table", i32, (B, blocks))
    if num_slots < 0:
        raise ValueError(f"num_slots={num_slots} is negative")
    if out is not None:
        if len(out) != 4:
            raise ValueError("out must be (seq_lens, query_start, slots, pages_used)")
        for t, name, n in zip(out, ("seq_lens", "query_start", "slots", "pages_used"),
                              (B, B + 1, num_slots, 1)):
            _check(t, name, i32, (n,))
    dev = _one_gpu((old_lens, "old_lens"), (new_lens, "new_lens"), (block_table, "block_table"),
                   (free_pages, "free_pages"),
                   *(() if out is None else ((t, "out") for t in out)))
    if out is None:                                 # one allocation, in four parts
        out = old_lens.new_empty(2 * B + num_slots + 2).split_with_sizes((B, B + 1, num_slots, 1))
    seq_lens, query_start, slots, used = out
    st = _launch(lib.awq_kv_assign, dev, _address(old_lens), _address(new_lens), B, page_size,
                 _address(block_table), blocks, _address(free_pages), free_pages.shape[0],
                 _address(seq_lens), query_start.data_ptr(), _address(slots), num_slots,
                 used.data_ptr())
    check(st, "awq_kv_assign")
    return tuple(out)


def awq_kv_append(K, V, cache, slots, nonfinite_count=None):
    """Quantize K and V (fp16 or bf16 [tokens][heads][D]; tokens may be strided,
    as slices of a fused projection's output are) into the cache's slots (int32
    [tokens]; tokens with a negative slot are skipped).  ``nonfinite_count`` (int32)
    grows by the values that are not finite and by the groups of finite values
    (bfloat16 ones past fp16's range) whose step does not fit fp16.  Returns the
    cache."""
    torch = _torch()
    c, cfg = _cache_arg(cache)
    _tensor(K, "K", (torch.float16, torch.bfloat16))
    _tensor(V, "V", K.dtype)
    ks, vs = (_token_rows(K, "K", c.num_kv_heads, c.head_dim),
              _token_rows(V, "V", c.num_kv_heads, c.head_dim))
    T = K.shape[0]
    if V.shape[0] != T:
        raise ValueError("K and V must have the same number of tokens")
    _check(slots, "slots", torch.int32, (T,))
    if nonfinite_count is not None:
        _tensor(nonfinite_count, "nonfinite_count", torch.int32)
        if nonfinite_count.numel() < 1:
            raise ValueError("nonfinite_count must hold one element")
    dev = _one_gpu(*_cache_tensors(cache), (slots, "slots"),
                   None if nonfinite_count is None else (nonfinite_count, "nonfinite_count"))
    _same_gpu(dev, (K, "K"), (V, "V"))
    st = _launch(lib.awq_kv_append, dev, _address(K), _address(V), _dtype_code(K.dtype), T, ks, vs, c,
                 cfg, _address(slots), _address(nonfinite_count))
    check(st, "awq_kv_append")
    return cache


def awq_kv_gather(cache, slots, out_dtype=None, out=None):
    """The values that slots (int32 [tokens]) of the cache stand for: (K, V), each
    [tokens][heads][D] of out_dtype (float16 by default, bfloat16 or float32);
    zeros for negative slots."""
    torch = _torch()
    c, cfg = _cache_arg(cache)
    _tensor(slots, "slots", torch.int32)
    if slots.dim() != 1:
        raise ValueError("slots must be 1-D")
    T = slots.shape[0]
    shape = (T, c.num_kv_heads, c.head_dim)
    if out is not None and len(out) != 2:
        raise ValueError("out must be (K, V)")
    odt = out[0].dtype if out is not None else torch.float16 if out_dtype is None else out_dtype
    if odt not in (torch.float16, torch.bfloat16, torch.float32):
        raise TypeError(f"out_dtype {odt} is not float16, bfloat16 or float32")
    if out is not None:
        _check(out[0], "K", odt, shape)
        _check(out[1], "V", odt, shape)
    dev = _one_gpu(*_cache_tensors(cache), (slots, "slots"),
                   *(() if out is None else ((out[0], "K"), (out[1], "V"))))
    if out is None:
        out = slots.new_empty(shape, dtype=odt), slots.new_empty(shape, dtype=odt)
    st = _launch(lib.awq_kv_gather, dev, c, cfg, _address(slots), T, _address(out[0]),
                 _address(out[1]), _dtype_code(odt))
    check(st, "awq_kv_gather")
    return tuple(out)


def awq_kv_attention_workspace_size(num_tokens: int, num_seqs: int, num_heads: int, cache,
                                    max_query_len: int, max_seq_len: int, window: int = 0, sinks: int = 0,
                                    prefix_len: int = 0) -> int:
    """Workspace bytes of awq_kv_attention for these sizes; cache as passed to it."""
    c, cfg = _cache_arg(cache)
    if sinks != 0 or prefix_len != 0:
        need = lambda table: int(lib.awq_kv_attention_ex_workspace_size(      # noqa: E731
            num_tokens, num_seqs, num_heads, c, cfg, max_query_len, max_seq_len,
            awq_kv_attention_options(1, window, sinks, prefix_len, table, -(-prefix_len // c.page_size))))
        return max(need(None), need(256) if prefix_len > 0 else 0)    # (with a prefix_table or without)
    return int(lib.awq_kv_attention_workspace_size(num_tokens, num_seqs, num_heads, c, cfg,
                                                   max_query_len, max_seq_len, window))


def awq_kv_attention(Q, cache, block_table, seq_lens, query_start=None, max_query_len=None,
                     max_seq_len=None, scale=None, causal: bool = True, window: int = 0, out=None,
                     return_lse: bool = False, workspace="auto", sinks: int = 0, prefix_len: int = 0,
                     prefix_table=None):
    """Attention of Q (fp16 or bf16 [tokens][num_heads][D], tokens may be strided)
    over the cached keys and values of each request: block_table int32
    [B][max_blocks] and seq_lens int32 [B] as awq_kv_assign gives them.

    ``query_start`` (int32 [B + 1]) says which tokens are whose, the last ones of
    each request; without it every request has one.  ``max_query_len`` is the
    most tokens of a request (all tokens, if not given), ``max_seq_len`` the
    expected longest request (the table's width; it decides only how the work is
    split).  ``scale`` defaults to D ** -0.5.  ``window`` > 0 keeps the last
    `window` keys.  Returns O [tokens][num_heads][D], and with return_lse also
    the natural log of the softmax denominators, fp32 [tokens][num_heads]; rows
    of tokens of no request are not written (pass `out` to say what they hold).
    ``workspace``: as in awq_linear_ex.

    ``sinks``: beside a window's keys the first `sinks` stay visible.  ``prefix_len``:
    the first prefix_len tokens of every request are the same.  They are read once for all
    of them from prefix_table's pages (int32, at least ceil(prefix_len / page_size)), or
    without one, where that saves time, from those of the first request with query tokens
    that has the prefix up to its last page (or most of it, if none does); each request then
    holds them, as awq_kv_fork makes it, as far as its length goes, and idle or padded rows
    need not."""
    torch = _torch()
    c, cfg = _cache_arg(cache)
    D = c.head_dim
    _tensor(Q, "Q", (torch.float16, torch.bfloat16))
    if Q.dim() != 3 or Q.shape[2] != D:
        raise ValueError(f"Q has shape {tuple(Q.shape)}, expected [tokens][num_heads][{D}]")
    T, heads, _ = Q.shape
    if heads < 1 or heads % c.num_kv_heads:
        raise ValueError(f"{heads} query heads are not a multiple of {c.num_kv_heads} key/value heads")
    _tensor(block_table, "block_table", torch.int32)
    if block_table.dim() != 2:
        raise ValueError("block_table must be 2-D [B][max_blocks]")
    B, blocks = block_table.shape
    _check(seq_lens, "seq_lens", torch.int32, (B,))
    if query_start is not None:
        _check(query_start, "query_start", torch.int32, (B + 1,))
    elif T != B:
        raise ValueError(f"{T} query tokens for {B} requests need query_start")
    if max_query_len is None:
        max_query_len = T if query_start is not None else 1
    if query_start is None and max_query_len != 1:
        raise ValueError("without query_start, max_query_len is 1")
    if max_seq_len is None:
        max_seq_len = blocks * c.page_size
    if out is not None:
        _check(out, "out", Q.dtype, (T, heads, D))
    stride = _token_rows(Q, "Q", heads, D)
    if prefix_table is not None:
        if prefix_len == 0:
            raise ValueError("prefix_table needs prefix_len")
        _tensor(prefix_table, "prefix_table", torch.int32)
        if prefix_table.dim() != 1 or prefix_table.shape[0] < 1:     # (an empty tensor's address is NULL: no table)
            raise ValueError("prefix_table must be 1-D and hold a page")
    more = sinks != 0 or prefix_len != 0
    if more:
        opts = awq_kv_attention_options(int(causal), window, sinks, prefix_len, _address(prefix_table),
                                        0 if prefix_table is None else prefix_table.shape[0])
        need = 0 if workspace is None else lib.awq_kv_attention_ex_workspace_size(
            T, B, heads, c, cfg, max_query_len, max_seq_len, opts)
    else:
        need = 0 if workspace is None else lib.awq_kv_attention_workspace_size(
            T, B, heads, c, cfg, max_query_len, max_seq_len, window)
    ws, ws_bytes = _scratch(workspace, need, seq_lens)
    dev = _one_gpu(*_cache_tensors(cache), (block_table, "block_table"), (seq_lens, "seq_lens"),
                   None if query_start is None else (query_start, "query_start"),
                   None if out is None else (out, "out"), None if ws is None else (ws, "workspace"),
                   None if prefix_table is None else (prefix_table, "prefix_table"))
    _same_gpu(dev, (Q, "Q"))
    if out is None:
        out = Q.new_empty((T, heads, D))
    lse = Q.new_empty((T, heads), dtype=torch.float32) if return_lse else None
    if more:
        st = _launch(lib.awq_kv_attention_ex, dev, _address(Q), _dtype_code(Q.dtype), T, stride, heads, c, cfg,
                     _address(block_table), blocks, _address(seq_lens), _address(query_start), B, max_query_len,
                     max_seq_len, D ** -0.5 if scale is None else scale, opts, _address(out), _address(lse),
                     _address(ws), ws_bytes)
        check(st, "awq_kv_attention_ex")
        return (out, lse) if return_lse else out
    st = _launch(lib.awq_kv_attention, dev, _address(Q), _dtype_code(Q.dtype), T, stride, heads, c,
                 cfg, _address(block_table), blocks, _address(seq_lens), _address(query_start), B,
                 max_query_len, max_seq_len, D ** -0.5 if scale is None else scale, int(causal),
                 window, _address(out), _address(lse), _address(ws), ws_bytes)
    check(st, "awq_kv_attention")
    return (out, lse) if return_lse else out


# ---- pages of the cache -----------------------------------------------------------

def _table_arg(block_table, seq_lens=None):
    i32 = _torch().int32
    _tensor(block_table, "block_table", i32)
    if block_table.dim() != 2:
        raise ValueError("block_table must be 2-D [B][max_blocks]")
    if seq_lens is not None:
        _check(seq_lens, "seq_lens", i32, (block_table.shape[0],))
    return block_table.shape


def _free_arg(free_pages, taken, name="taken"):
    i32 = _torch().int32
    _tensor(free_pages, "free_pages", i32)
    if free_pages.dim() != 1:
        raise ValueError("free_pages must be 1-D")
    if taken is not None:
        _check(taken, name, i32, (1,))


def _maybe(t, name):
    return None if t is None else (t, name)


def awq_kv_copy_pages(cache, src, dst):
    """Copy page src[i] of the cache to page dst[i] (int32 [n] each; pairs with an id
    outside the cache are skipped).  Returns the cache."""
    i32 = _torch().int32
    c, cfg = _cache_arg(cache)
    _tensor(src, "src", i32)
    if src.dim() != 1:
        raise ValueError("src must be 1-D")
    _check(dst, "dst", i32, src.shape)
    dev = _one_gpu(*_cache_tensors(cache), (src, "src"), (dst, "dst"))
    check(_launch(lib.awq_kv_copy_pages, dev, c, cfg, _address(src), _address(dst), src.shape[0]), "awq_kv_copy_pages")
    return cache


def awq_kv_fork(cache, block_table, parents, children, lens, shared, free_pages, taken=None, out=None):
    """Row children[i] of block_table becomes a branch of the first lens[i] tokens of
    row parents[i] (int32 [n] each): full pages are shared, and counted in `shared`
    (int32 [pages]: holders beyond the first), a last page that is not full is copied to
    a page from the front of free_pages, behind the `taken` (int32 [1]) that awq_kv_assign
    has used of it.  Returns pages_used (int32 [1]), those and its own."""
    i32 = _torch().int32
    c, cfg = _cache_arg(cache)
    B, blocks = _table_arg(block_table)
    _tensor(parents, "parents", i32)
    if parents.dim() != 1:
        raise ValueError("parents must be 1-D")
    _check(children, "children", i32, parents.shape)
    _check(lens, "lens", i32, parents.shape)
    _check(shared, "shared", i32, (c.num_pages,))
    _free_arg(free_pages, taken)
    if out is not None:
        _check(out, "out", i32, (1,))
    dev = _one_gpu(*_cache_tensors(cache), (block_table, "block_table"), (parents, "parents"), (children, "children"),
                   (lens, "lens"), (shared, "shared"), (free_pages, "free_pages"), _maybe(taken, "taken"),
                   _maybe(out, "out"))
    if out is None:
        out = parents.new_empty(1)
    st = _launch(lib.awq_kv_fork, dev, c, cfg, _address(parents), _address(children), _address(lens),
                 parents.shape[0], _address(block_table), B, blocks, _address(shared), _address(free_pages),
                 free_pages.shape[0], _address(taken), out.data_ptr())
    check(st, "awq_kv_fork")
    return out


def awq_kv_release_workspace_size(num_pages: int, num_free: int) -> int:
    return int(lib.awq_kv_release_workspace_size(num_pages, num_free))


def awq_kv_release(block_table, seq_lens, shared, free_pages, page_size: int, start=None, end=None, pages_used=None,
                   out=None, workspace="auto"):
    """Give pages back: of each row, those whose tokens (below seq_lens) all lie between
    `start` (0 if not given) and `end` (seq_lens), int32 [B] each; their entries of
    block_table become -1.  Returns (free_pages, count): what is left of free_pages
    behind the pages_used (int32 [1]) of the step, then the pages that no row holds any
    more, then -1, as many entries as the pool has pages; and how many pages that is
    (int32 [1]).  ``out`` gives both tensors; ``workspace`` as in awq_linear_ex."""
    i32 = _torch().int32
    B, blocks = _table_arg(block_table, seq_lens)
    for t, name in ((start, "start"), (end, "end")):
        if t is not None:
            _check(t, name, i32, (B,))
    _tensor(shared, "shared", i32)
    if shared.dim() != 1 or shared.shape[0] < 1:
        raise ValueError("shared must be 1-D [pages]")
    pages = shared.shape[0]
    _free_arg(free_pages, pages_used, "pages_used")
    if out is not None:
        if len(out) != 2:
            raise ValueError("out must be (free_pages, count)")
        _tensor(out[0], "out", i32)
        if out[0].dim() != 1:
            raise ValueError("out's free_pages must be 1-D")
        _check(out[1], "count", i32, (1,))
    need = 0 if workspace is None else lib.awq_kv_release_workspace_size(pages, free_pages.shape[0])
    ws, ws_bytes = _scratch(workspace, need, shared)
    dev = _one_gpu((block_table, "block_table"), (seq_lens, "seq_lens"), _maybe(start, "start"), _maybe(end, "end"),
                   (shared, "shared"), (free_pages, "free_pages"), _maybe(pages_used, "pages_used"),
                   *(() if out is None else ((out[0], "out"), (out[1], "count"))), _maybe(ws, "workspace"))
    if out is None:                                 # one allocation, in two parts
        out = shared.new_empty(pages + 1).split_with_sizes((pages, 1))
    st = _launch(lib.awq_kv_release, dev, _address(block_table), B, blocks, page_size, _address(seq_lens),
                 _address(start), _address(end), _address(shared), pages, _address(free_pages), free_pages.shape[0],
                 _address(pages_used), _address(out[0]), out[0].shape[0], out[1].data_ptr(), _address(ws), ws_bytes)
    check(st, "awq_kv_release")
    return tuple(out)


def awq_kv_compact_workspace_size(num_pages: int, page_size: int) -> int:
    return int(lib.awq_kv_compact_workspace_size(num_pages, page_size))


def awq_kv_compact(cache, block_table, seq_lens, shared, out=None, workspace="auto"):
    """Move the n pages that the rows (of seq_lens tokens) use to the front of the pool;
    block_table and `shared` are updated in place.  Returns (free_pages, num_used): the
    pages from n on, then -1, int32 [pages]; n, int32 [1].  ``out`` gives both tensors;
    ``workspace`` as in awq_linear_ex."""
    i32 = _torch().int32
    c, cfg = _cache_arg(cache)
    B, blocks = _table_arg(block_table, seq_lens)
    _check(shared, "shared", i32, (c.num_pages,))
    if out is not None:
        if len(out) != 2:
            raise ValueError("out must be (free_pages, num_used)")
        _check(out[0], "free_pages", i32, (c.num_pages,))
        _check(out[1], "num_used", i32, (1,))
    need = 0 if workspace is None else lib.awq_kv_compact_workspace_size(c.num_pages, c.page_size)
    ws, ws_bytes = _scratch(workspace, need, shared)
    dev = _one_gpu(*_cache_tensors(cache), (block_table, "block_table"), (seq_lens, "seq_lens"), (shared, "shared"),
                   *(() if out is None else ((out[0], "free_pages"), (out[1], "num_used"))), _maybe(ws, "workspace"))
    if out is None:
        out = shared.new_empty(c.num_pages + 1).split_with_sizes((c.num_pages, 1))
    st = _launch(lib.awq_kv_compact, dev, c, cfg, _address(block_table), B, blocks, _address(seq_lens),
                 _address(shared), out[0].data_ptr(), out[1].data_ptr(), _address(ws), ws_bytes)
    check(st, "awq_kv_compact")
    return tuple(out)


# ---- rotary positions -------------------------------------------------------------

def awq_rope_frequencies(rotary_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                         original_len: float = 0.0, low: float = 0.0, high: float = 0.0, device="cuda"):
    """(inv_freq, attention_factor): radians per position of each pair, a float64
    tensor [rotary_dim / 2] on `device`, and the factor on cosines and sines.
    ``scaling`` stretches them for contexts beyond the trained ones: 'linear',
    'ntk', 'yarn' or 'bands', by `factor` from `original_len`; `low` and `high` are the
    numbers of turns between which 'yarn' (default 1 and 32) and 'bands' (1 and 4) blend."""
    torch = _torch()
    kind = ROPE_SCALINGS.get(scaling)
    if kind is None:
        raise ValueError(f"scaling {scaling!r} is not one of {sorted(ROPE_SCALINGS)}")
    inv = (ctypes.c_double * max(rotary_dim // 2, 1))()
    scale = ctypes.c_double()
    check(lib.awq_rope_frequencies(rotary_dim, base, awq_rope_scaling(kind, factor, original_len, low, high), inv,
                                   ctypes.byref(scale)), "awq_rope_frequencies")
    return torch.tensor(inv[:], dtype=torch.float64, device=device), scale.value


def _rope_arg(positions, inv_freq, tokens, D, attention_factor, interleaved, inverse):
    torch = _torch()
    _check(positions, "positions", torch.int32, (tokens,))
    _tensor(inv_freq, "inv_freq", torch.float64)
    if inv_freq.dim() != 1:
        raise ValueError("inv_freq must be 1-D [rotary_dim / 2]")
    R = 2 * inv_freq.shape[0]
    if R < 16 or R % 16 or R > D:
        raise ValueError(f"inv_freq stands for rotary_dim={R}, which must be a multiple of 16 in [16, {D}]")
    return awq_rope_args(_address(positions), inv_freq.data_ptr(), attention_factor, R, bool(interleaved),
                         bool(inverse))


def _rope_rows(x, name, tokens, D, out, dtype):
    """Token strides of queries or keys to rotate and of their output (dense if `out` is
    None)."""
    if x.dim() != 3 or x.shape[0] != tokens or x.shape[2] != D:
        raise ValueError(f"{name} has shape {tuple(x.shape)}, expected [{tokens}][heads][{D}]")
    heads = x.shape[1]
    stride = _token_rows(x, name, heads, D)
    if out is None:
        return stride, heads * D
    _tensor(out, f"{name}'s out", dtype, x.shape)
    return stride, _token_rows(out, f"{name}'s out", heads, D)


def awq_rope(Q, positions, inv_freq, K=None, attention_factor: float = 1.0, interleaved: bool = False,
             inverse: bool = False, out=None):
    """Q (fp16 or bf16 [tokens][heads][D], tokens may be strided) rotated by its
    tokens' positions (int32 [tokens]): the first 2 * len(inv_freq) channels of each
    head, halves paired, or neighbours with `interleaved`.  With K (the same for its own
    number of heads) returns (Q', K').  ``inv_freq`` and ``attention_factor`` as
    awq_rope_frequencies gives them.  ``inverse`` negates the angles: the gradient's
    rotation.  ``out``: where to write (a tensor, or a pair with K); Q and K themselves
    for a rotation in place."""
    torch = _torch()
    _tensor(Q, "Q", (torch.float16, torch.bfloat16))
    if Q.dim() != 3:
        raise ValueError("Q must be 3-D [tokens][heads][D]")
    T, heads, D = Q.shape
    if D % 16 or not 16 <= D <= AWQ_ROPE_MAX_DIM:
        raise ValueError(f"heads of {D} channels: a multiple of 16 of at most {AWQ_ROPE_MAX_DIM} is needed")
    q_out, k_out = (out, None) if K is None else (None, None) if out is None else out
    q_stride, qo_stride = _rope_rows(Q, "Q", T, D, q_out, Q.dtype)
    k_stride = ko_stride = kv_heads = 0
    if K is not None:
        _tensor(K, "K", Q.dtype)
        k_stride, ko_stride = _rope_rows(K, "K", T, D, k_out, Q.dtype)
        kv_heads = K.shape[1]
    rope = _rope_arg(positions, inv_freq, T, D, attention_factor, interleaved, inverse)
    dev = _one_gpu((inv_freq, "inv_freq"), (positions, "positions"))
    _same_gpu(dev, (Q, "Q"), *(() if K is None else ((K, "K"),)), *(() if q_out is None else ((q_out, "out"),)),
              *(() if k_out is None else ((k_out, "out"),)))
    if q_out is None:
        q_out = Q.new_empty((T, heads, D))
    if K is not None and k_out is None:
        k_out = K.new_empty((T, kv_heads, D))
    st = _launch(lib.awq_rope, dev, _address(Q), _address(q_out), heads, q_stride, qo_stride, _address(K),
                 _address(k_out), kv_heads, k_stride, ko_stride, _dtype_code(Q.dtype), T, D, rope)
    check(st, "awq_rope")
    return q_out if K is None else (q_out, k_out)


def awq_kv_append_rope(K, V, cache, slots, positions, inv_freq, Q=None, attention_factor: float = 1.0,
                       interleaved: bool = False, out=None, nonfinite_count=None):
    """awq_kv_append of K rotated as awq_rope rotates it (quantized from fp32), and
    of V as it is; with Q (the step's queries) also returns them rotated, in `out` if
    given (Q itself for a rotation in place)."""
    torch = _torch()
    c, cfg = _cache_arg(cache)
    D = c.head_dim
    _tensor(K, "K", (torch.float16, torch.bfloat16))
    _tensor(V, "V", K.dtype)
    ks, vs = _token_rows(K, "K", c.num_kv_heads, D), _token_rows(V, "V", c.num_kv_heads, D)
    T = K.shape[0]
    if V.shape[0] != T:
        raise ValueError("K and V must have the same number of tokens")
    _check(slots, "slots", torch.int32, (T,))
    if nonfinite_count is not None:
        _tensor(nonfinite_count, "nonfinite_count", torch.int32)
        if nonfinite_count.numel() < 1:
            raise ValueError("nonfinite_count must hold one element")
    q_stride = qo_stride = heads = 0
    if Q is not None:
        _tensor(Q, "Q", K.dtype)
        q_stride, qo_stride = _rope_rows(Q, "Q", T, D, out, K.dtype)
        heads = Q.shape[1]
    elif out is not None:
        raise ValueError("out is where Q goes: there is no Q")
    rope = _rope_arg(positions, inv_freq, T, D, attention_factor, interleaved, False)
    dev = _one_gpu(*_cache_tensors(cache), (slots, "slots"), (positions, "positions"), (inv_freq, "inv_freq"),
                   None if nonfinite_count is None else (nonfinite_count, "nonfinite_count"))
    _same_gpu(dev, (K, "K"), (V, "V"), *(() if Q is None else ((Q, "Q"),)),
              *(() if out is None else ((out, "out"),)))
    if Q is not None and out is None:
        out = Q.new_empty((T, heads, D))
    st = _launch(lib.awq_kv_append_rope, dev, _address(Q), _address(out), heads, q_stride, qo_stride, _address(K),
                 _address(V), _dtype_code(K.dtype), T, ks, vs, c, cfg, _address(slots), rope,
                 _address(nonfinite_count))
    check(st, "awq_kv_append_rope")
    return out
