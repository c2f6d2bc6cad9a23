"""Python binding of libgptq_w4a16.so (ctypes; argument marshalling only).

Every step of the layer runs in the library's CUDA kernels.  PyTorch supplies
device memory and the current stream; this module checks tensor dtypes,
devices and shapes, passes raw pointers, and turns status codes into
exceptions.  There is no CPU path: if the library is missing or the device is
not sm_100, calls raise.

No call takes part in autograd: outputs carry no history, whatever the inputs
require.  A training step calls the gradients (gemm_experts_dx, moe_combine and
moe_combine_backward) itself, from an autograd.Function of its own for instance.
"""
from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "_lib", "libgptq_w4a16.so")

KERNEL_AUTO, KERNEL_DECODE, KERNEL_PREFILL = 0, 1, 2
DECODE_MAX_M = 64
LORA_DECODE_MAX_M = 32
MAX_GROUPED = 8
MAX_LORA_RANK = 256
LORA_SCRATCH_BYTES = 8 << 20
GIDX_MAX_GROUPS = 640
MOE_MAX_EXPERTS = 1024
MOE_MAX_TOPK = 64
GROUP_SIZES = (-1, 16, 32, 64, 128, 256, 512, 1024)

STATUS = {0: "GPTQ_OK", 1: "GPTQ_ERR_NULL", 2: "GPTQ_ERR_SHAPE", 3: "GPTQ_ERR_GROUP",
          4: "GPTQ_ERR_ALIGN", 5: "GPTQ_ERR_DEVICE", 6: "GPTQ_ERR_CUDA",
          7: "GPTQ_ERR_TIMEOUT", 8: "GPTQ_ERR_ALIAS", 9: "GPTQ_ERR_KERNEL",
          10: "GPTQ_ERR_INDEX"}

# Every entry point declared in include/gptq_w4a16.h.
EXPORTS = ("gptq_w4a16_gemm", "gptq_w4a16_gemm_kernel", "gptq_w4a16_gemm_decode_splits",
           "gptq_w4a16_gemm_grouped", "gptq_w4a16_gemm_asym", "gptq_w4a16_gemm_gidx",
           "gptq_w4a16_gemm_lora", "gptq_w4a16_gemm_lora_noalloc",
           "gptq_moe_sort", "gptq_moe_combine", "gptq_moe_combine_backward",
           "gptq_w4a16_gemm_experts", "gptq_w4a16_gemm_experts_kernel",
           "gptq_w4a16_gemm_experts_dx", "gptq_dequant",
           "gptq_w4a16_select", "gptq_status_string", "gptq_device_error", "gptq_version")


class GptqError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


_lock = threading.Lock()
_lib = None

_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_i32 = ctypes.c_int32


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load the library once (raises if it has not been built)."""
    global _lib
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError(
                    f"CUDA library not built: {path} is missing "
                    "(run `python -m int4_weight_only_gptq_b200.build`)")
            lib = ctypes.CDLL(path)
            gemm_args = [_p, _p, _p, _i64, _i64, _i64, _i32, _p, _p]
            lib.gptq_w4a16_gemm.argtypes = gemm_args
            lib.gptq_w4a16_gemm_kernel.argtypes = gemm_args + [_i32]
            lib.gptq_w4a16_gemm_decode_splits.argtypes = gemm_args + [_i32]
            lib.gptq_w4a16_gemm_grouped.argtypes = [_p, _p, _p, _p, _i32, _i64, _i64, _i32,
                                                    _p, _p]
            lib.gptq_w4a16_gemm_lora.argtypes = [_p, _p, _p, _i64, _i64, _i64, _i32, _p, _p,
                                                 _i64, _p, _p, _p]
            lib.gptq_w4a16_gemm_asym.argtypes = [_p, _p, _p, _p, _i64, _i64, _i64, _i32, _p, _p]
            lib.gptq_w4a16_gemm_gidx.argtypes = [_p, _p, _p, _p, _i64, _i64, _i64, _i64, _p, _p]
            lib.gptq_w4a16_gemm_lora_noalloc.argtypes = [_p, _p, _p, _i64, _i64, _i64, _i32,
                                                         _p, _p, _i64, _p, _p]
            lib.gptq_moe_sort.argtypes = [_p, _p, _i32, _i64, _i64, _i64, _i64, _p, _p, _p, _p]
            lib.gptq_moe_combine.argtypes = [_p, _p, _p, _i64, _i64, _i64, _i64, _p, _p]
            lib.gptq_moe_combine_backward.argtypes = [_p, _p, _p, _p, _i64, _i64, _i64, _i64,
                                                      _p, _p, _p]
            experts_args = [_p, _p, _p, _p, _i64, _i64, _i64, _i64, _i32, _p, _p]
            lib.gptq_w4a16_gemm_experts.argtypes = experts_args
            lib.gptq_w4a16_gemm_experts_kernel.argtypes = experts_args + [_i32, _i32]
            lib.gptq_w4a16_gemm_experts_dx.argtypes = experts_args
            lib.gptq_dequant.argtypes = [_p, _p, _i64, _i64, _i32, _p, _p]
            lib.gptq_w4a16_select.argtypes = [_i64, _i64, _i64, _i32,
                                              ctypes.POINTER(_i32), ctypes.POINTER(_i32)]
            lib.gptq_status_string.restype = ctypes.c_char_p
            lib.gptq_status_string.argtypes = [ctypes.c_int]
            lib.gptq_device_error.argtypes = []
            lib.gptq_version.restype = ctypes.c_char_p
            for name in ("gptq_w4a16_gemm", "gptq_w4a16_gemm_kernel",
                         "gptq_w4a16_gemm_decode_splits", "gptq_w4a16_gemm_grouped",
                         "gptq_w4a16_gemm_asym", "gptq_w4a16_gemm_gidx", "gptq_w4a16_gemm_lora",
                         "gptq_w4a16_gemm_lora_noalloc",
                         "gptq_moe_sort", "gptq_moe_combine", "gptq_moe_combine_backward",
                         "gptq_w4a16_gemm_experts", "gptq_w4a16_gemm_experts_kernel",
                         "gptq_w4a16_gemm_experts_dx", "gptq_dequant",
                         "gptq_w4a16_select", "gptq_device_error"):
                getattr(lib, name).restype = ctypes.c_int
            _lib = lib
    return _lib


def status_string(status: int) -> str:
    return load().gptq_status_string(int(status)).decode()


def _check(status: int):
    if status != 0:
        raise GptqError(status, status_string(status))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _int32(value):
    """`value` as the library shall see it: ctypes keeps the low bits of a
    number that does not fit, which may be a valid one that was not checked
    here; the least number instead is none of its choices."""
    return value if -2 ** 31 <= value < 2 ** 31 else -2 ** 31


def _current(device):
    """The handle of torch.cuda.current_stream(device), without the object."""
    return ctypes.c_void_p(torch._C._cuda_getCurrentRawStream(device.index))


# stream=: a torch stream, or a raw handle, to run on instead of the current
# stream.  What a call allocates is that stream's memory, and no tensor of the
# call is reused before both streams are done with it; the caller orders the
# two streams' work itself.

def _torch_stream(stream, device):
    """A stream= argument as a torch stream: one already, or a raw handle."""
    if isinstance(stream, torch.cuda.Stream):
        if stream.device != device:
            raise ValueError(f"stream is on {stream.device}, expected {device}")
        return stream
    handle = stream.value or 0 if isinstance(stream, ctypes.c_void_p) else int(stream)
    # 0 and 1 (cudaStreamLegacy) both name the legacy default stream, which
    # torch would take for no handle at all
    if handle in (0, 1):
        return torch.cuda.default_stream(device)
    return torch.cuda.ExternalStream(handle, device=device)


def _tensors(args) -> list:
    """The tensors among args, those of its lists and tuples too."""
    found = []
    for a in args:
        if isinstance(a, torch.Tensor):
            found.append(a)
        elif isinstance(a, (list, tuple)):
            found += _tensors(a)
    return found


def _on_stream(fn, stream, *args):
    """fn(*args) with `stream` current, so that what it allocates is memory of
    that stream (a block of the caller's stream may still be in use there).
    Its results are kept from reuse until the caller's stream is done with them
    too, and the caller's tensors until `stream` is."""
    t = args[0]
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        return fn(*args)  # refuses it
    stream, index = _torch_stream(stream, t.device), t.get_device()
    if stream.cuda_stream == torch._C._cuda_getCurrentRawStream(index):
        return fn(*args)
    caller = torch.cuda.current_stream(index)
    with torch.cuda.device(index):  # set_stream makes the stream's device current
        torch.cuda.set_stream(stream)
        try:
            result = fn(*args)
        finally:
            torch.cuda.set_stream(caller)
    given = _tensors(args)
    for a in given:
        a.record_stream(stream)
    for r in _tensors((result,)):
        if not any(r is a for a in given):
            r.record_stream(caller)
    return result


def _as_bits16(t: torch.Tensor) -> torch.Tensor:
    if t.dtype == torch.float16:
        return t
    if t.dtype in (torch.int16, torch.uint16):
        return t
    raise TypeError(f"expected a float16 tensor, got {t.dtype}")


def _require(t: torch.Tensor, name: str, dtype_ok, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous (row-major)")
    if not dtype_ok(t.dtype):
        raise TypeError(f"{name} has dtype {t.dtype}")


def n_groups(K: int, group: int) -> int:
    """Scale rows of a layer: one for group -1 or a group of K or more, else
    ceil(K / group) (a ragged last group when group does not divide K)."""
    return 1 if group == -1 or group >= K else -(-K // group)


def layer_shapes(x, qweight, scales, group: int) -> tuple[int, int, int]:
    """(M, K, N) of a layer call, after checking that x [M, K], qweight
    [K/8, N] and scales [n_groups(K, group), N] agree.  The C ABI sees only
    pointers and the sizes it is given, and builds its tensor maps from them,
    so a tensor smaller than those sizes would be read past its end: the
    shapes are checked here, before the library is called.  An unsupported
    group is left to the library (GPTQ_ERR_GROUP)."""
    if x.dim() != 2 or qweight.dim() != 2 or scales.dim() != 2:
        raise ValueError("x, qweight and scales must be 2-D")
    M, K = (int(v) for v in x.shape)
    N = int(qweight.shape[1])
    if int(qweight.shape[0]) * 8 != K:
        raise ValueError(f"qweight rows {qweight.shape[0]} do not match K={K}")
    if group in GROUP_SIZES and K > 0:
        want = (n_groups(K, group), N)
        if tuple(scales.shape) != want:
            raise ValueError(f"scales has shape {tuple(scales.shape)}, expected {want} "
                             f"for K={K}, group={group}")
    return M, K, N


def adapter_shapes(lora_a, lora_b, K: int, N: int) -> int:
    """The adapter's rank, after checking lora_a [rank, K] and lora_b [N, rank]."""
    if lora_a.dim() != 2 or lora_b.dim() != 2:
        raise ValueError("lora_a and lora_b must be 2-D")
    rank = int(lora_a.shape[0])
    if int(lora_a.shape[1]) != K:
        raise ValueError(f"lora_a has shape {tuple(lora_a.shape)}, expected ({rank}, {K})")
    if tuple(lora_b.shape) != (N, rank):
        raise ValueError(f"lora_b has shape {tuple(lora_b.shape)}, expected {(N, rank)}")
    return rank


def _check_shape(t, name: str, shape: tuple):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def gemm(x: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor, group: int,
         out: torch.Tensor | None = None, stream=None, kernel: int = KERNEL_AUTO,
         decode_splits: int = 0) -> torch.Tensor:
    """Y[M, N] = x[M, K] . dequant(qweight[K/8, N], scales[n_groups, N]) (FP16)."""
    if stream is not None:
        return _on_stream(gemm, stream, x, qweight, scales, group, out, None, kernel,
                          decode_splits)
    lib = load()
    dev = qweight.device
    _require(qweight, "qweight", lambda d: d == torch.int32, None)
    _require(scales, "scales", lambda d: d == torch.float16, dev)
    _require(x, "x", lambda d: d == torch.float16, dev)
    M, K, N = layer_shapes(x, qweight, scales, group)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=dev)
    else:
        _require(out, "out", lambda d: d == torch.float16, dev)
        _check_shape(out, "out", (M, N))
    args = (_ptr(x), _ptr(qweight), _ptr(scales), M, K, N, _int32(group), _ptr(out),
            _current(dev))
    with torch.cuda.device(dev):  # the library works on the current device
        if decode_splits:
            _check(lib.gptq_w4a16_gemm_decode_splits(*args, _int32(decode_splits)))
        elif kernel == KERNEL_AUTO:
            _check(lib.gptq_w4a16_gemm(*args))
        else:
            _check(lib.gptq_w4a16_gemm_kernel(*args, _int32(kernel)))
    return out


def gemm_grouped(x: torch.Tensor, qweights, scales, group: int, outs=None,
                 stream=None) -> list:
    """Y_i = x . dequant(qweights[i], scales[i]) for linears sharing x (one
    decode launch for M <= DECODE_MAX_M)."""
    if stream is not None:
        return _on_stream(gemm_grouped, stream, x, qweights, scales, group, outs)
    lib = load()
    if not 1 <= len(qweights) <= MAX_GROUPED or len(scales) != len(qweights):
        raise ValueError(f"need 1..{MAX_GROUPED} linears with one scales tensor each")
    dev = qweights[0].device
    _require(x, "x", lambda d: d == torch.float16, dev)
    if x.dim() != 2:
        raise ValueError("x must be 2-D")
    M, K = x.shape
    Ns = []
    for i, (qw, sc) in enumerate(zip(qweights, scales)):
        _require(qw, f"qweights[{i}]", lambda d: d == torch.int32, dev)
        _require(sc, f"scales[{i}]", lambda d: d == torch.float16, dev)
        if qw.dim() != 2 or qw.shape[0] * 8 != K:
            raise ValueError(f"qweights[{i}] does not match K={K}")
        layer_shapes(x, qw, sc, group)
        Ns.append(int(qw.shape[1]))
    if outs is None:
        outs = [torch.empty((M, n), dtype=torch.float16, device=dev) for n in Ns]
    else:
        if len(outs) != len(Ns):
            raise ValueError("one output per linear")
        for i, (o, n) in enumerate(zip(outs, Ns)):
            _require(o, f"outs[{i}]", lambda d: d == torch.float16, dev)
            if tuple(o.shape) != (M, n):
                raise ValueError(f"outs[{i}] has shape {tuple(o.shape)}, expected {(M, n)}")
    count = len(Ns)
    qa = (ctypes.c_void_p * count)(*[_ptr(q) for q in qweights])
    sa = (ctypes.c_void_p * count)(*[_ptr(t) for t in scales])
    na = (ctypes.c_int64 * count)(*Ns)
    ya = (ctypes.c_void_p * count)(*[_ptr(o) for o in outs])
    with torch.cuda.device(dev):
        _check(lib.gptq_w4a16_gemm_grouped(_ptr(x), qa, sa, na, count, M, K, _int32(group), ya,
                                           _current(dev)))
    return outs


def gemm_asym(x: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor,
              qzeros: torch.Tensor, group: int, out: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """Y = x . W, W = fp16((q - z) * s) with zeros packed in qzeros
    [n_groups, N/8] int32 (eight per word along N); N % 32 == 0."""
    if stream is not None:
        return _on_stream(gemm_asym, stream, x, qweight, scales, qzeros, group, out)
    lib = load()
    dev = qweight.device
    _require(qweight, "qweight", lambda d: d == torch.int32, None)
    _require(scales, "scales", lambda d: d == torch.float16, dev)
    _require(qzeros, "qzeros", lambda d: d == torch.int32, dev)
    _require(x, "x", lambda d: d == torch.float16, dev)
    M, K, N = layer_shapes(x, qweight, scales, group)
    if qzeros.dim() != 2 or tuple(qzeros.shape) != (scales.shape[0], N // 8):
        raise ValueError(f"qzeros has shape {tuple(qzeros.shape)}, expected "
                         f"{(scales.shape[0], N // 8)}")
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=dev)
    else:
        _require(out, "out", lambda d: d == torch.float16, dev)
        _check_shape(out, "out", (M, N))
    with torch.cuda.device(dev):
        _check(lib.gptq_w4a16_gemm_asym(_ptr(x), _ptr(qweight), _ptr(scales), _ptr(qzeros), M,
                                        K, N, _int32(group), _ptr(out), _current(dev)))
    return out


def gidx_shapes(x, qweight, scales, g_idx) -> tuple[int, int, int, int]:
    """(M, K, N, n_groups) of an act-order call, after checking x [M, K],
    qweight [K/8, N], scales [n_groups, N] and g_idx [K]."""
    M, K, N = layer_shapes(x, qweight, scales, 0)  # 0: scales checked below
    if int(scales.shape[1]) != N:
        raise ValueError(f"scales has shape {tuple(scales.shape)}, expected (n_groups, {N})")
    if g_idx.dim() != 1 or int(g_idx.shape[0]) != K:
        raise ValueError(f"g_idx has shape {tuple(g_idx.shape)}, expected ({K},)")
    return M, K, N, int(scales.shape[0])


def gemm_gidx(x: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor,
              g_idx: torch.Tensor, out: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """Y = x . W, W[k, n] = fp16((q[k, n] - 8) * scales[g_idx[k], n]) (act
    order): g_idx [K] int32 with entries in 0 .. n_groups - 1, scales
    [n_groups, N], n_groups <= GIDX_MAX_GROUPS.  An out-of-range index is
    reported by device_error() as GPTQ_ERR_INDEX."""
    if stream is not None:
        return _on_stream(gemm_gidx, stream, x, qweight, scales, g_idx, out)
    lib = load()
    dev = qweight.device
    _require(qweight, "qweight", lambda d: d == torch.int32, None)
    _require(scales, "scales", lambda d: d == torch.float16, dev)
    _require(g_idx, "g_idx", lambda d: d == torch.int32, dev)
    _require(x, "x", lambda d: d == torch.float16, dev)
    M, K, N, ng = gidx_shapes(x, qweight, scales, g_idx)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=dev)
    else:
        _require(out, "out", lambda d: d == torch.float16, dev)
        _check_shape(out, "out", (M, N))
    with torch.cuda.device(dev):
        _check(lib.gptq_w4a16_gemm_gidx(_ptr(x), _ptr(qweight), _ptr(scales), _ptr(g_idx), M, K,
                                        N, ng, _ptr(out), _current(dev)))
    return out


def gemm_lora(x: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor, group: int,
              lora_a: torch.Tensor, lora_b: torch.Tensor, t_work: torch.Tensor | None = None,
              out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Y = x . dequant(qweight, scales) + fp16(x . lora_a^T) . lora_b^T (FP16),
    lora_a [rank, K], lora_b [N, rank] with the adapter's scaling applied;
    t_work [M, rank] receives fp16(x . lora_a^T)."""
    if stream is not None:
        return _on_stream(gemm_lora, stream, x, qweight, scales, group, lora_a, lora_b, t_work,
                          out)
    lib = load()
    dev = qweight.device
    _require(qweight, "qweight", lambda d: d == torch.int32, None)
    _require(scales, "scales", lambda d: d == torch.float16, dev)
    _require(x, "x", lambda d: d == torch.float16, dev)
    _require(lora_a, "lora_a", lambda d: d == torch.float16, dev)
    _require(lora_b, "lora_b", lambda d: d == torch.float16, dev)
    M, K, N = layer_shapes(x, qweight, scales, group)
    rank = adapter_shapes(lora_a, lora_b, K, N)
    if t_work is None:
        t_work = torch.empty((M, rank), dtype=torch.float16, device=dev)
    else:
        _require(t_work, "t_work", lambda d: d == torch.float16, dev)
        _check_shape(t_work, "t_work", (M, rank))
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=dev)
    else:
        _require(out, "out", lambda d: d == torch.float16, dev)
        _check_shape(out, "out", (M, N))
    with torch.cuda.device(dev):
        _check(lib.gptq_w4a16_gemm_lora(_ptr(x), _ptr(qweight), _ptr(scales), M, K, N,
                                        _int32(group), _ptr(lora_a), _ptr(lora_b), rank,
                                        _ptr(t_work), _ptr(out), _current(dev)))
    return out


def gemm_lora_noalloc(x: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor,
                      group: int, lora_a: torch.Tensor, lora_b: torch.Tensor,
                      out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """gemm_lora with T kept in the library's static device buffer (no work
    tensor; M * rank * 2 <= LORA_SCRATCH_BYTES; calls that may overlap in time
    share the buffer and race)."""
    if stream is not None:
        return _on_stream(gemm_lora_noalloc, stream, x, qweight, scales, group, lora_a, lora_b,
                          out)
    lib = load()
    dev = qweight.device
    _require(qweight, "qweight", lambda d: d == torch.int32, None)
    _require(scales, "scales", lambda d: d == torch.float16, dev)
    _require(x, "x", lambda d: d == torch.float16, dev)
    _require(lora_a, "lora_a", lambda d: d == torch.float16, dev)
    _require(lora_b, "lora_b", lambda d: d == torch.float16, dev)
    M, K, N = layer_shapes(x, qweight, scales, group)
    rank = adapter_shapes(lora_a, lora_b, K, N)
    if out is None:
        out = torch.empty((M, N), dtype=torch.float16, device=dev)
    else:
        _require(out, "out", lambda d: d == torch.float16, dev)
        _check_shape(out, "out", (M, N))
    with torch.cuda.device(dev):
        _check(lib.gptq_w4a16_gemm_lora_noalloc(_ptr(x), _ptr(qweight), _ptr(scales), M, K, N,
                                                _int32(group), _ptr(lora_a), _ptr(lora_b), rank,
                                                _ptr(out), _current(dev)))
    return out


# The calls of a decoding step's experts last a few microseconds on the device,
# about as long as a call takes on the host, so their checks are kept short:
# one expression per tensor, device indices instead of device objects, the
# stream's handle without the stream object.

def _bad(t, name: str, dtype, index: int, shape=None):
    """Raises for a tensor that _fits refused, in _require's words."""
    _require(t, name, lambda d: d == dtype, torch.device("cuda", index))
    raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _fits(t, dtype, index: int) -> bool:
    """A contiguous CUDA tensor of this type on this device."""
    return (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index
            and t.is_contiguous())


def _device_index(t, name: str) -> int:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    return t.get_device()


def _call(fn, index: int, *args):
    """fn(*args, handle of the current stream) with the tensors' device current."""
    # the handle of torch.cuda.current_stream(index), without the object
    stream = torch._C._cuda_getCurrentRawStream(index)
    if torch._C._cuda_getDevice() == index:
        status = fn(*args, stream)
    else:
        with torch.cuda.device(index):
            status = fn(*args, stream)
    if status != 0:
        _check(status)


def moe_sort(x: torch.Tensor, expert_ids: torch.Tensor, n_experts: int,
             out: torch.Tensor | None = None, stream=None):
    """The tokens' rows in the order of their experts.

    x [M, H] FP16; expert_ids [M, topk] int32 or int64, the experts chosen for
    each token (ids outside 0 .. n_experts - 1 drop the choice).  Returns
    (x_sorted [M * topk, H], offsets [n_experts + 1] int32, dest [M, topk]
    int32): expert e's rows are offsets[e] .. offsets[e + 1] - 1, choice j of
    token m is row dest[m, j] (-1 if dropped), in the order of (m, j) within an
    expert.  The rows from offsets[n_experts] on keep what `out` holds."""
    if stream is not None:
        return _on_stream(moe_sort, stream, x, expert_ids, n_experts, out)
    lib = _lib or load()
    dev = _device_index(x, "x")
    if not _fits(x, torch.float16, dev):
        _bad(x, "x", torch.float16, dev)
    wide = isinstance(expert_ids, torch.Tensor) and expert_ids.dtype is torch.int64
    id_dtype = torch.int64 if wide else torch.int32
    if not _fits(expert_ids, id_dtype, dev):
        _bad(expert_ids, "expert_ids", id_dtype, dev)
    if x.dim() != 2 or expert_ids.dim() != 2:
        raise ValueError("x and expert_ids must be 2-D")
    M, H = x.shape
    tokens, topk = expert_ids.shape
    if tokens != M:
        raise ValueError(f"expert_ids has {tokens} rows, expected one per token ({M})")
    if out is None:
        out = torch.empty((M * topk, H), dtype=torch.float16, device=x.device)
    elif not _fits(out, torch.float16, dev) or out.shape != (M * topk, H):
        _bad(out, "out", torch.float16, dev, (M * topk, H))
    # (the library refuses 0, and shall not see the low bits of a larger number)
    E = n_experts if 0 < n_experts <= MOE_MAX_EXPERTS else 0
    offsets = x.new_empty(E + 1, dtype=torch.int32)
    dest = (torch.empty_like(expert_ids, dtype=torch.int32) if wide
            else torch.empty_like(expert_ids))
    _call(lib.gptq_moe_sort, dev, x.data_ptr(), expert_ids.data_ptr(), 8 if wide else 4,
          M, H, topk, E, out.data_ptr(), offsets.data_ptr(), dest.data_ptr())
    return out, offsets, dest


def moe_combine(y_sorted: torch.Tensor, dest: torch.Tensor, weights: torch.Tensor | None = None,
                out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """out[m] = fp16(sum_j weights[m, j] * y_sorted[dest[m, j]]), FP32 sums in
    the order of j, dropped choices (dest -1) left out.  y_sorted [R, H] FP16,
    dest [M, topk] int32 from moe_sort, weights [M, topk] FP32 or None for
    ones (then it is moe_sort's gradient, applied to that of x_sorted)."""
    if stream is not None:
        return _on_stream(moe_combine, stream, y_sorted, dest, weights, out)
    lib = _lib or load()
    dev = _device_index(y_sorted, "y_sorted")
    if not _fits(y_sorted, torch.float16, dev):
        _bad(y_sorted, "y_sorted", torch.float16, dev)
    if not _fits(dest, torch.int32, dev):
        _bad(dest, "dest", torch.int32, dev)
    if y_sorted.dim() != 2 or dest.dim() != 2:
        raise ValueError("y_sorted and dest must be 2-D")
    M, topk = dest.shape
    R, H = y_sorted.shape
    if weights is not None and (not _fits(weights, torch.float32, dev)
                                or weights.shape != dest.shape):
        _bad(weights, "weights", torch.float32, dev, (M, topk))
    if out is None:
        out = torch.empty((M, H), dtype=torch.float16, device=y_sorted.device)
    elif not _fits(out, torch.float16, dev) or out.shape != (M, H):
        _bad(out, "out", torch.float16, dev, (M, H))
    _call(lib.gptq_moe_combine, dev, y_sorted.data_ptr(), dest.data_ptr(),
          None if weights is None else weights.data_ptr(), M, H, topk, R, out.data_ptr())
    return out


def moe_combine_backward(dout: torch.Tensor, y_sorted: torch.Tensor, dest: torch.Tensor,
                         weights: torch.Tensor, out: torch.Tensor | None = None, stream=None):
    """The gradients of moe_combine with weights: (dy_sorted [R, H] FP16,
    dweights [M, topk] FP32) from dout [M, H] FP16.  Rows that no entry of dest
    names keep what `out` (the buffer of dy_sorted) holds; dweights is 0 for
    dropped choices.  Entries of dest that are not dropped must differ from
    each other, as moe_sort's do: two that name one row both write it."""
    if stream is not None:
        return _on_stream(moe_combine_backward, stream, dout, y_sorted, dest, weights, out)
    lib = _lib or load()
    dev = _device_index(dout, "dout")
    if not _fits(dout, torch.float16, dev):
        _bad(dout, "dout", torch.float16, dev)
    if not _fits(y_sorted, torch.float16, dev):
        _bad(y_sorted, "y_sorted", torch.float16, dev)
    if not _fits(dest, torch.int32, dev):
        _bad(dest, "dest", torch.int32, dev)
    if dout.dim() != 2 or y_sorted.dim() != 2 or dest.dim() != 2:
        raise ValueError("dout, y_sorted and dest must be 2-D")
    M, topk = dest.shape
    R, H = y_sorted.shape
    if dout.shape != (M, H):
        raise ValueError(f"dout has shape {tuple(dout.shape)}, expected {(M, H)}")
    if not _fits(weights, torch.float32, dev) or weights.shape != dest.shape:
        _bad(weights, "weights", torch.float32, dev, (M, topk))
    if out is None:
        out = torch.empty_like(y_sorted)
    elif not _fits(out, torch.float16, dev) or out.shape != y_sorted.shape:
        _bad(out, "out", torch.float16, dev, (R, H))
    dweights = torch.empty_like(weights)
    _call(lib.gptq_moe_combine_backward, dev, dout.data_ptr(), y_sorted.data_ptr(),
          dest.data_ptr(), weights.data_ptr(), M, H, topk, R, out.data_ptr(),
          dweights.data_ptr())
    return out, dweights


def experts_shapes(rows, qweight, scales, offsets, group: int,
                   gradient: bool = False) -> tuple[int, int, int, int]:
    """(R, K, N, E) of an experts' product, after checking qweight [E, K/8, N],
    scales [E, n_groups(K, group), N], offsets [E + 1] and rows [R, K] (or
    [R, N], for the gradient).  As in layer_shapes, an unsupported group is
    left to the library."""
    if rows.dim() != 2 or qweight.dim() != 3 or scales.dim() != 3 or offsets.dim() != 1:
        raise ValueError("need 2-D rows, 3-D qweight and scales, 1-D offsets")
    E, packed, N = qweight.shape
    K = 8 * packed
    R, width = rows.shape
    if width != (N if gradient else K):
        raise ValueError(f"rows have {width} columns, expected {N if gradient else K}")
    if offsets.shape[0] != E + 1:
        raise ValueError(f"offsets has shape {tuple(offsets.shape)}, expected {(E + 1,)}")
    if group in GROUP_SIZES and K > 0 and scales.shape != (E, n_groups(K, group), N):
        raise ValueError(f"scales has shape {tuple(scales.shape)}, expected "
                         f"{(E, n_groups(K, group), N)} for K={K}, group={group}")
    return R, K, N, E


def _experts(fn, rows, qweight, scales, offsets, group, out, gradient, name):
    """Checks and output of an experts' product, and its library call; `fn`
    takes the entry's arguments without the kernel choice."""
    dev = _device_index(qweight, "qweight")
    if not _fits(qweight, torch.int32, dev):
        _bad(qweight, "qweight", torch.int32, dev)
    if not _fits(scales, torch.float16, dev):
        _bad(scales, "scales", torch.float16, dev)
    if not _fits(offsets, torch.int32, dev):
        _bad(offsets, "offsets", torch.int32, dev)
    if not _fits(rows, torch.float16, dev):
        _bad(rows, name, torch.float16, dev)
    R, K, N, E = experts_shapes(rows, qweight, scales, offsets, group, gradient)
    shape = (R, K if gradient else N)
    if out is None:
        out = torch.empty(shape, dtype=torch.float16, device=rows.device)
    elif not _fits(out, torch.float16, dev) or out.shape != shape:
        _bad(out, "out", torch.float16, dev, shape)
    _call(fn, dev, rows.data_ptr(), qweight.data_ptr(), scales.data_ptr(),
          offsets.data_ptr(), R, K, N, E, _int32(group), out.data_ptr())
    return out


def gemm_experts(x_sorted: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor,
                 offsets: torch.Tensor, group: int, out: torch.Tensor | None = None,
                 stream=None, kernel: int = KERNEL_AUTO, tile: int = 0) -> torch.Tensor:
    """Every expert's linear on its own rows: y_sorted[r] = x_sorted[r] .
    dequant(qweight[e], scales[e]) for offsets[e] <= r < offsets[e + 1].
    x_sorted [R, K] FP16 and offsets [E + 1] int32 as moe_sort returns them,
    qweight [E, K/8, N] int32, scales [E, n_groups, N] FP16.  Rows that belong
    to no expert keep what `out` holds.  kernel and tile force the kernel: tests
    and benchmarks (KERNEL_DECODE takes a tile of 16 or 32 rows)."""
    if stream is not None:
        return _on_stream(gemm_experts, stream, x_sorted, qweight, scales, offsets, group, out,
                          None, kernel, tile)
    lib = _lib or load()
    fn = lib.gptq_w4a16_gemm_experts
    if kernel != KERNEL_AUTO or tile != 0:
        fn = lambda *args: lib.gptq_w4a16_gemm_experts_kernel(*args, _int32(kernel),
                                                              _int32(tile))
    return _experts(fn, x_sorted, qweight, scales, offsets, group, out, False, "x_sorted")


def gemm_experts_dx(dy_sorted: torch.Tensor, qweight: torch.Tensor, scales: torch.Tensor,
                    offsets: torch.Tensor, group: int, out: torch.Tensor | None = None,
                    stream=None) -> torch.Tensor:
    """The gradient of gemm_experts with respect to x_sorted: dx_sorted[r] =
    dy_sorted[r] . dequant(qweight[e], scales[e])^T, [R, K] FP16 from dy_sorted
    [R, N] FP16 (the packed weights are frozen and have no gradient); N up to
    65536, the length of the sums."""
    if stream is not None:
        return _on_stream(gemm_experts_dx, stream, dy_sorted, qweight, scales, offsets, group,
                          out)
    return _experts((_lib or load()).gptq_w4a16_gemm_experts_dx, dy_sorted, qweight, scales,
                    offsets, group, out, True, "dy_sorted")


def dequant(qweight: torch.Tensor, scales: torch.Tensor, group: int,
            out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """W[K, N] = fp16((q - 8) * s): the debugging entry."""
    if stream is not None:
        return _on_stream(dequant, stream, qweight, scales, group, out)
    lib = load()
    dev = qweight.device
    _require(qweight, "qweight", lambda d: d == torch.int32, None)
    _require(scales, "scales", lambda d: d == torch.float16, dev)
    if qweight.dim() != 2 or scales.dim() != 2:
        raise ValueError("qweight and scales must be 2-D")
    K, N = int(qweight.shape[0]) * 8, int(qweight.shape[1])
    if group in GROUP_SIZES and tuple(scales.shape) != (n_groups(K, group), N):
        raise ValueError(f"scales has shape {tuple(scales.shape)}, expected "
                         f"{(n_groups(K, group), N)} for K={K}, group={group}")
    if out is None:
        out = torch.empty((K, N), dtype=torch.float16, device=dev)
    else:
        _require(out, "out", lambda d: d == torch.float16, dev)
        _check_shape(out, "out", (K, N))
    with torch.cuda.device(dev):
        _check(lib.gptq_dequant(_ptr(qweight), _ptr(scales), K, N, _int32(group), _ptr(out),
                                _current(dev)))
    return out


def select(M: int, K: int, N: int, group: int) -> tuple[int, int]:
    """(kernel_id, split_k) the dispatcher picks for this shape."""
    lib = load()
    k, s = _i32(-1), _i32(-1)
    _check(lib.gptq_w4a16_select(M, K, N, _int32(group), ctypes.byref(k), ctypes.byref(s)))
    return k.value, s.value


def device_error() -> int:
    """Read and clear the device error word (synchronises the device)."""
    return int(load().gptq_device_error())


def version() -> str:
    return load().gptq_version().decode()
