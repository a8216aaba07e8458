"""Python binding of libfp8blk (block-scaled FP8 linear algebra on GB300).

Argument marshalling only: every step of the computation runs in the CUDA
kernels of ``libfp8blk.so`` behind its C ABI (``include/fp8blk.h``). PyTorch
allocates device memory and supplies the current stream. There is no CPU or
PyTorch fallback: if the library is missing every call raises.

Names follow the DeepSeek-V3 inference kernels ("Administrator & Developer
Guide", 8.5 The Triton kernels): act_quant, weight_dequant, fp8_gemm, plus
the FP8 linear layer of 6.3 and the block weight quantisation of the README's
weight_scale_inv section.

Calls on a stream overlap. Those that end in a GEMM, mla_absorb, mla_append,
mla_attention and residual_norm let the next call start early, which then
reads its weight operands (w, w1, w3, w2, wkv_b and their block scales)
at once, any number of such calls in a row. So between the call that writes a
weight and the one that multiplies by it there has to be a synchronisation or
an ordering call (act_quant, weight_quant, weight_dequant, fp4_quant,
fp4_dequant, a moe_* call, or any kernel or copy of torch's) that is neither
of the two. Weights quantised when a model is loaded need nothing more;
``linear(x, *weight_quant(w))`` does: synchronise in between.
"""
from __future__ import annotations

import ctypes
import os
import re
import threading

import torch

__all__ = [
    "SCALE_FP32", "SCALE_UE8M0", "SCALE_PROMOTE", "BLOCK", "lib", "lib_path", "header_functions", "Fp8BlkError",
    "act_quant", "weight_quant", "weight_dequant", "fp8_gemm", "linear", "linear_host",
    "gemm_workspace_bytes", "linear_workspace_bytes", "linear_host_workspace_bytes", "linear_kernels",
    "last_device_error",
    "swiglu_gemm", "ffn", "moe_permute", "moe_workspace_bytes", "moe_grouped_gemm", "moe_gate", "moe_route",
    "mla_absorb", "mla_append", "mla_attention", "mla_attention_workspace_bytes",
    "moe_layer", "moe_layer_workspace_bytes", "SCORE_SOFTMAX", "SCORE_SIGMOID",
    "FP4_E4M3", "FP4_UE8M0", "fp4_quant", "fp4_dequant", "fp4_gemm", "fp4_linear", "fp4_linear_workspace_bytes",
    "fp4_scale_shape", "residual_norm",
]

SCALE_FP32 = 0
SCALE_UE8M0 = 1
SCALE_PROMOTE = 0x10   # | SCALE_UE8M0: GEMMs keep the per-block promotion
BLOCK = 128

_PKG = os.path.dirname(os.path.abspath(__file__))
_ROOT = os.path.dirname(_PKG)
HEADER = os.path.join(_ROOT, "include", "fp8blk.h")
_LIB_PATH = os.path.join(_PKG, "libfp8blk.so")
_lib = None
_lib_lock = threading.Lock()


class Fp8BlkError(RuntimeError):
    pass


def lib_path() -> str:
    return _LIB_PATH


def header_functions() -> list[str]:
    """Names of the functions the public header declares."""
    with open(HEADER) as f:
        text = f.read()
    return sorted(set(re.findall(r"FP8BLK_API\s+[\w\s\*]*?\b(fp8blk_\w+)\s*\(", text)))


def lib():
    """The loaded libfp8blk (ctypes). Raises if it has not been built."""
    global _lib
    with _lib_lock:
        if _lib is None:
            if not os.path.exists(_LIB_PATH):
                raise Fp8BlkError(f"{_LIB_PATH} is missing: build it with __graft_entry__.build() "
                                  "or python fp8_block_scaled_quant_gb300/_build.py")
            L = ctypes.CDLL(_LIB_PATH)
            vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
            L.fp8blk_status_string.argtypes = [i32]
            L.fp8blk_status_string.restype = ctypes.c_char_p
            L.fp8blk_version.argtypes = []
            L.fp8blk_version.restype = i32
            L.fp8blk_act_quant.argtypes = [vp, i64, i64, vp, vp, i32, vp]
            L.fp8blk_weight_quant.argtypes = [vp, i64, i64, vp, vp, i32, vp]
            L.fp8blk_weight_dequant.argtypes = [vp, vp, i64, i64, vp, vp]
            L.fp8blk_gemm_workspace_bytes.argtypes = [i64, i64, i64]
            L.fp8blk_gemm_workspace_bytes.restype = sz
            L.fp8blk_gemm.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, i32, vp, sz, vp]
            L.fp8blk_linear_workspace_bytes.argtypes = [i64, i64, i64]
            L.fp8blk_linear_workspace_bytes.restype = sz
            L.fp8blk_linear.argtypes = [vp, vp, vp, vp, i64, i64, i64, i32, vp, sz, vp]
            L.fp8blk_linear_host_workspace_bytes.argtypes = [i64, i64, i64]
            L.fp8blk_linear_host_workspace_bytes.restype = sz
            L.fp8blk_linear_host.argtypes = [vp, vp, vp, vp, i64, i64, i64, i32, vp, sz, vp]
            L.fp8blk_linear_kernels.argtypes = [i64, i64, i64, ctypes.POINTER(i32)]
            L.fp8blk_last_device_error.argtypes = [vp, ctypes.POINTER(ctypes.c_uint)]
            for name in header_functions():
                if getattr(L, name).restype is ctypes.c_int:
                    getattr(L, name).restype = i32
            _lib = L
    return _lib


def _check(status: int, what: str):
    if status != 0:
        msg = lib().fp8blk_status_string(status).decode()
        raise Fp8BlkError(f"{what}: {msg} (status {status})")


def _ptr(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need(t: torch.Tensor, dtype, name: str, ndim: int = 2):
    if t.is_cuda and t.dtype is dtype and t.dim() == ndim and t.is_contiguous():
        return
    if not t.is_cuda:
        raise Fp8BlkError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise Fp8BlkError(f"{name} must be {dtype}, got {t.dtype}")
    if t.dim() != ndim:
        raise Fp8BlkError(f"{name}: Input tensors must have {ndim} dimensions")
    if not t.is_contiguous():
        raise Fp8BlkError(f"{name}: Input tensor must be contiguous")


# ---- workspaces: zero-filled device buffers cached per (device, stream) ------
#
# A captured graph keeps the addresses of its calls' workspaces, so a buffer that
# a capture was given is never freed, also where a later call needs a larger one.
# A buffer made during a capture serves that capture alone: its fill is one of the
# graph's nodes, so no other graph and no eager call may rely on it. Replays of
# graphs captured on one stream share that stream's workspaces with its other calls:
# they must not run at the same time.

_ws_cache: dict = {}
_ws_captured: dict = {}   # by address: buffers of _ws_cache that a graph may hold
_ws_graph: dict = {}      # the last capture's own buffers: (its id, buffer)
_COUNTERS = 64 * 1024     # what any call needs as zeros lies in the first 64 KB of its workspace


def _capturing(on_gpu: bool) -> bool:
    return on_gpu and torch.cuda.is_current_stream_capturing()


def _capture_id(stream: int) -> int:
    n = ctypes.c_ulonglong(0)
    _check(_function("fp8blk_capture_id", "pp")(stream, ctypes.addressof(n)), "capture_id")
    return n.value


def _buffer(nbytes: int, device: torch.device, key: tuple, zeroed: int = _COUNTERS) -> torch.Tensor:
    """A uint8 buffer of (device, stream, name) with nbytes after its first 256-byte boundary, all zeros when it was
    made; `zeroed`: how many of them a call needs so, for a buffer that a graph fills in every replay."""
    buf = _ws_cache.get(key)
    fits = buf is not None and buf.numel() >= nbytes + 256
    if not _capturing(device.type == "cuda"):
        if not fits:
            buf = _ws_cache[key] = torch.zeros(max(nbytes, 256) + 256, dtype=torch.uint8, device=device)
    elif fits:
        _ws_captured[buf.data_ptr()] = buf
    else:
        capture = _capture_id(key[1])
        held, buf = _ws_graph.get(key, (None, None))
        if held != capture or buf.numel() < nbytes + 256:
            buf = torch.empty(max(nbytes, 256) + 256, dtype=torch.uint8, device=device)
            if zeroed:
                buf[:zeroed + 256].zero_()
            _ws_graph[key] = capture, buf
    return buf


def workspace(nbytes: int, device: torch.device, key: str = "gemm") -> torch.Tensor:
    """A zero-initialised uint8 device buffer of at least nbytes, reused by
    every call on the same device, stream and key. The GEMM leaves its
    counters at zero, so the buffer never needs clearing again. (First needed
    during a capture: the graph zeroes its first 64 KB, where the counters are.)"""
    stream = torch.cuda.current_stream(device).cuda_stream
    buf = _buffer(nbytes, device, (device.index, stream, key))
    off = (-buf.data_ptr()) % 256
    return buf[off:off + max(nbytes, 1)]


# The calls of a decode step are issued in less time than their kernels run
# only if the host side is short: these find the stream once per call, bind a
# function's types once, and pass addresses as plain integers.

_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_bound: dict = {}


def _stream_on(t: torch.Tensor) -> int:
    """The handle of the current stream of t's device."""
    if _raw_stream is not None:
        return _raw_stream(t.get_device())
    return torch.cuda.current_stream(t.device).cuda_stream


def _function(name: str, argtypes: str, restype=ctypes.c_int):
    """The library's function, its argument types bound at the first call: p pointer, i int64, e int, f float,
    z size_t."""
    f = _bound.get(name)
    if f is None:
        kinds = {"p": ctypes.c_void_p, "i": ctypes.c_int64, "e": ctypes.c_int, "f": ctypes.c_float,
                 "z": ctypes.c_size_t}
        f = _bound[name] = _set_types(name, [kinds[k] for k in argtypes], restype)
    return f


def _addr(t: torch.Tensor | None):
    return None if t is None else t.data_ptr()


def _scratch(ws: torch.Tensor | None, nbytes: int, t: torch.Tensor, stream: int, key: str, zeroed: int):
    """(address, bytes, tensor to hold until the launch) of the caller's workspace, or of the one kept for the device
    and stream; `zeroed`: its leading bytes that have to be zeros."""
    if ws is not None:
        if ws.get_device() != t.get_device() or not ws.is_contiguous():
            raise Fp8BlkError("ws must be a contiguous tensor on the device of the inputs")
        return ws.data_ptr(), ws.numel() * ws.element_size(), ws
    key = (t.get_device(), stream, key)
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < nbytes + 256 or _capturing(t.is_cuda):
        buf = _buffer(nbytes, t.device, key, zeroed)
    at = buf.data_ptr()
    return at + (-at) % 256, nbytes, buf


# ---- operations --------------------------------------------------------------

def act_quant(x: torch.Tensor, scale_fmt: int = SCALE_FP32, q: torch.Tensor | None = None,
              s: torch.Tensor | None = None):
    """x bf16 [M, K] -> (q float8_e4m3fn [M, K], s float32 [M, K/128])."""
    _need(x, torch.bfloat16, "x")
    M, K = x.shape
    if K % BLOCK:
        raise Fp8BlkError(f"Last dimension size must be divisible by block_size (block_size={BLOCK})")
    if q is None:
        q = torch.empty((M, K), dtype=torch.float8_e4m3fn, device=x.device)
    if s is None:
        s = torch.empty((M, K // BLOCK), dtype=torch.float32, device=x.device)
    _check(lib().fp8blk_act_quant(_ptr(x), M, K, _ptr(q), _ptr(s), scale_fmt, _stream(x.device)), "act_quant")
    return q, s


def weight_quant(w: torch.Tensor, scale_fmt: int = SCALE_FP32):
    """w float32 [N, K] -> (q float8_e4m3fn [N, K], s float32 [ceil(N/128), ceil(K/128)])."""
    _need(w, torch.float32, "w")
    N, K = w.shape
    q = torch.empty((N, K), dtype=torch.float8_e4m3fn, device=w.device)
    s = torch.empty(((N + BLOCK - 1) // BLOCK, (K + BLOCK - 1) // BLOCK), dtype=torch.float32, device=w.device)
    _check(lib().fp8blk_weight_quant(_ptr(w), N, K, _ptr(q), _ptr(s), scale_fmt, _stream(w.device)),
           "weight_quant")
    return q, s


def weight_dequant(q: torch.Tensor, s: torch.Tensor, out: torch.Tensor | None = None) -> torch.Tensor:
    """q float8_e4m3fn [N, K], s float32 [ceil(N/128), ceil(K/128)] -> bf16 [N, K]."""
    _need(q, torch.float8_e4m3fn, "q")
    _need(s, torch.float32, "s")
    N, K = q.shape
    if tuple(s.shape) != ((N + BLOCK - 1) // BLOCK, (K + BLOCK - 1) // BLOCK):
        raise Fp8BlkError("scale must have shape (ceil(N/128), ceil(K/128))")
    if out is None:
        out = torch.empty((N, K), dtype=torch.bfloat16, device=q.device)
    _check(lib().fp8blk_weight_dequant(_ptr(q), _ptr(s), N, K, _ptr(out), _stream(q.device)), "weight_dequant")
    return out


def gemm_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().fp8blk_gemm_workspace_bytes(M, N, K))


def linear_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().fp8blk_linear_workspace_bytes(M, N, K))


def linear_host_workspace_bytes(M: int, N: int, K: int) -> int:
    return int(lib().fp8blk_linear_host_workspace_bytes(M, N, K))


def linear_kernels(M: int, N: int, K: int) -> int:
    """Kernels one linear() call of this shape launches on the current device:
    1 when act_quant runs inside the GEMM kernel, 2 when it is a kernel of its
    own, 0 for an empty problem."""
    n = ctypes.c_int(0)
    _check(lib().fp8blk_linear_kernels(M, N, K, ctypes.byref(n)), "linear_kernels")
    return n.value


def fp8_gemm(a: torch.Tensor, a_s: torch.Tensor, w: torch.Tensor, w_s: torch.Tensor,
             scale_fmt: int = SCALE_FP32, out: torch.Tensor | None = None,
             ws: torch.Tensor | None = None) -> torch.Tensor:
    """a e4m3 [M, K], a_s fp32 [M, K/128], w e4m3 [N, K], w_s fp32 [ceil(N/128), K/128] -> bf16 [M, N]."""
    _need(a, torch.float8_e4m3fn, "a")
    _need(w, torch.float8_e4m3fn, "w")
    _need(a_s, torch.float32, "a_s")
    _need(w_s, torch.float32, "w_s")
    M, K = a.shape
    N = w.shape[0]
    if w.shape[1] != K:
        raise Fp8BlkError("a and w must share K")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=a.device)
    nbytes = gemm_workspace_bytes(M, N, K)
    if ws is None:
        ws = workspace(nbytes, a.device)
    _check(lib().fp8blk_gemm(_ptr(a), _ptr(a_s), _ptr(w), _ptr(w_s), _ptr(out), M, N, K, scale_fmt, _ptr(ws),
                             ws.numel(), _stream(a.device)), "fp8_gemm")
    return out


def linear(x: torch.Tensor, w: torch.Tensor, w_s: torch.Tensor, scale_fmt: int = SCALE_FP32,
           out: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """FP8 linear layer: fp8_gemm(act_quant(x), w). x bf16 [M, K] -> bf16 [M, N]."""
    _need(x, torch.bfloat16, "x")
    _need(w, torch.float8_e4m3fn, "w")
    _need(w_s, torch.float32, "w_s")
    M, K = x.shape
    N = w.shape[0]
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    if ws is None:
        ws = workspace(linear_workspace_bytes(M, N, K), x.device, "linear")
    _check(lib().fp8blk_linear(_ptr(x), _ptr(w), _ptr(w_s), _ptr(out), M, N, K, scale_fmt, _ptr(ws), ws.numel(),
                               _stream(x.device)), "linear")
    return out


def linear_host(x_host: torch.Tensor, w: torch.Tensor, w_s: torch.Tensor, y_host: torch.Tensor,
                scale_fmt: int = SCALE_FP32, ws: torch.Tensor | None = None) -> torch.Tensor:
    """The FP8 linear layer on host bf16 buffers, enqueued on the current stream of
    w's device: pinned buffers are read and written in place by the kernels,
    pageable ones are copied in and out. y_host is valid after that stream is
    synchronised."""
    if x_host.is_cuda or y_host.is_cuda:
        raise Fp8BlkError("x_host and y_host must be host tensors")
    if x_host.dtype != torch.bfloat16 or y_host.dtype != torch.bfloat16:
        raise Fp8BlkError("x_host and y_host must be bf16")
    if not (x_host.is_contiguous() and y_host.is_contiguous()):
        raise Fp8BlkError("Input tensor must be contiguous")
    _need(w, torch.float8_e4m3fn, "w")
    M, K = x_host.shape
    N = w.shape[0]
    if tuple(y_host.shape) != (M, N):
        raise Fp8BlkError("y_host must be [M, N]")
    if ws is None:
        ws = workspace(linear_host_workspace_bytes(M, N, K), w.device, "linear_host")
    _check(lib().fp8blk_linear_host(_ptr(x_host), _ptr(w), _ptr(w_s), _ptr(y_host), M, N, K, scale_fmt, _ptr(ws),
                                    ws.numel(), _stream(w.device)), "linear_host")
    return y_host


def last_device_error(device: torch.device | None = None) -> int:
    """Synchronises the current stream and returns (and clears) the device
    error bits: 0 when no kernel gave up waiting."""
    device = device or torch.device("cuda", torch.cuda.current_device())
    bits = ctypes.c_uint(0)
    st = lib().fp8blk_last_device_error(_stream(device), ctypes.byref(bits))
    if st not in (0, 6):
        _check(st, "last_device_error")
    return int(bits.value)


# ---- microscaled 4-bit floats ---------------------------------------------------

FP4_E4M3, FP4_UE8M0 = 0, 1   # 16 columns to an e4m3 scale and an fp32 scale per row; 32 to a power of two


def fp4_scale_shape(rows: int, K: int, fmt: int = FP4_E4M3):
    """Shape of the uint8 scale tensor of a [rows, K] matrix: the byte of (row, block) is at
    [row // 128, block // 4, row % 32, row % 128 // 32, block % 4]."""
    return ((rows + 127) // 128, K // (64 if fmt == FP4_E4M3 else 128), 32, 4, 4)


_bind = None


def _native():
    """The compiled part of this binding (csrc/bind.cpp): its calls check their tensors, allocate their outputs and call
    the library in a few microseconds less than Python needs for that."""
    global _bind
    if _bind is None:
        path = os.path.join(_PKG, "_bind.so")
        if not os.path.exists(path):
            raise Fp8BlkError(f"{path} is missing: build it with __graft_entry__.build() "
                              "or python fp8_block_scaled_quant_gb300/_build.py")
        import importlib.util
        from . import _build
        if os.path.exists(_build.BIND_FOR):
            with open(_build.BIND_FOR) as f:
                made = f.read()
            if made != _build.bind_for():
                raise Fp8BlkError(f"{path} was compiled for {made}: build it again for {_build.bind_for()}")
        spec = importlib.util.spec_from_file_location(__name__ + "._bind", path)
        m = importlib.util.module_from_spec(spec)
        spec.loader.exec_module(m)
        names = ["fp8blk_status_string"] + [n for n in header_functions() if "fp4" in n or "residual_norm" in n]
        m.setup({n: ctypes.cast(getattr(lib(), n), ctypes.c_void_p).value for n in names}, Fp8BlkError, _ws_cache, _buffer)
        _bind = m
    return _bind


def fp4_quant(x: torch.Tensor, fmt: int = FP4_E4M3):
    """x bf16 or float32 [M, K] (rows may be strided) -> (q uint8 [M, K/2], s uint8 scale tiles of fp4_scale_shape,
    g float32 [M]; g is None for FP4_UE8M0): e2m1 codes, low half first, with their block and row scales. The scale
    bytes of rows past M are not written. Before a product takes these as its weight (w, w_s, w_g), synchronise or issue
    another ordering call (the module's rule on overlap); as activations they may go straight into fp4_gemm."""
    return (_bind or _native()).fp4_quant(x, fmt)


def fp4_dequant(q: torch.Tensor, s: torch.Tensor, g: torch.Tensor | None, fmt: int = FP4_E4M3,
                out: torch.Tensor | None = None) -> torch.Tensor:
    """What fp4_quant gave -> bf16 [M, K]."""
    return (_bind or _native()).fp4_dequant(q, s, g, fmt, out)


def fp4_gemm(a: torch.Tensor, a_s: torch.Tensor, a_g: torch.Tensor | None, w: torch.Tensor, w_s: torch.Tensor,
             w_g: torch.Tensor | None, fmt: int = FP4_E4M3, out: torch.Tensor | None = None) -> torch.Tensor:
    """Two 4-bit matrices as fp4_quant gives them, a [M, K] and w [N, K] -> bf16 [M, N] = a w^T. w and w_s are read at
    once: they must not come from the call just before, nor from residual_norm without an ordering call since (the
    module's rule on overlap). a, a_s, a_g may come from any call."""
    return (_bind or _native()).fp4_gemm(a, a_s, a_g, w, w_s, w_g, fmt, out)


def fp4_linear_workspace_bytes(M: int, N: int, K: int, fmt: int = FP4_E4M3) -> int:
    return int(_function("fp8blk_fp4_linear_workspace_bytes", "iiie", ctypes.c_size_t)(M, N, K, fmt))


def fp4_linear(x: torch.Tensor, w: torch.Tensor, w_s: torch.Tensor, w_g: torch.Tensor | None, fmt: int = FP4_E4M3,
               out: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """FP4 linear layer: fp4_gemm(fp4_quant(x), w). x bf16 [M, K] (rows may be strided) -> bf16 [M, N]. ws: a workspace
    of fp4_linear_workspace_bytes, 256-byte aligned, any contents, used by one stream at a time. w and w_s are read at
    once, as in fp4_gemm: a weight that fp4_quant has just made needs a synchronisation in between."""
    return (_bind or _native()).fp4_linear(x, w, w_s, w_g, fmt, out, ws)


def residual_norm(y: torch.Tensor, x: torch.Tensor | None, norm_w: torch.Tensor, post_w: torch.Tensor | None = None,
                  gate: torch.Tensor | None = None, residual_scale: float = 1.0, eps: float = 1e-6,
                  quant: str | None = None, scale_fmt: int = 0, r: torch.Tensor | None = None):
    """The seam between two blocks, per token: z = post_w ? RMSNorm(y) * post_w : y; r = residual_scale * x + gate * z;
    h = RMSNorm(r) * norm_w. y, x bf16 [T, D] (rows may be strided; x None: r = gate * z), norm_w and post_w float32
    [D], gate float32 [D] or bf16 [T, D]. Returns (r bf16 [T, D], h): h is bf16 [T, D], or with quant="fp8"
    (q, s) of it as act_quant gives them (scale_fmt SCALE_*; from h in fp32, the codes by the scale's reciprocal), or with
    quant="fp4" (q, s, g) of it as fp4_quant gives them (scale_fmt FP4_*).
    r may be given; it may be x or y itself. fp32 until each output's one rounding. h is the next product's activation at
    once; to multiply by it as a weight needs an ordering call in between (the module's rule on overlap)."""
    return (_bind or _native()).residual_norm(y, x, norm_w, post_w, gate, residual_scale, eps, quant, scale_fmt, r)


# ---- SwiGLU FFN and routed experts -------------------------------------------

def _set_types(name, argtypes, restype=ctypes.c_int):
    f = getattr(lib(), name)
    f.argtypes = argtypes
    f.restype = restype
    return f


def swiglu_gemm(x: torch.Tensor, x_s: torch.Tensor, w1: torch.Tensor, w1_s: torch.Tensor, w3: torch.Tensor,
                w3_s: torch.Tensor, scale_fmt: int = SCALE_FP32, ws: torch.Tensor | None = None):
    """act_quant(bf16(silu(bf16(x w1^T))) * bf16(x w3^T)) -> (u float8_e4m3fn [M, inter], u_s float32 [M, inter/128])."""
    for t, n, dt in ((x, "x", torch.float8_e4m3fn), (w1, "w1", torch.float8_e4m3fn), (w3, "w3", torch.float8_e4m3fn),
                     (x_s, "x_s", torch.float32), (w1_s, "w1_s", torch.float32), (w3_s, "w3_s", torch.float32)):
        _need(t, dt, n)
    M, dim = x.shape
    inter = w1.shape[0]
    u = torch.empty((M, inter), dtype=torch.float8_e4m3fn, device=x.device)
    us = torch.empty((M, inter // BLOCK), dtype=torch.float32, device=x.device)
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    nb = _set_types("fp8blk_swiglu_workspace_bytes", [i64, i64, i64], sz)(M, inter, dim)
    if ws is None:
        ws = workspace(nb, x.device, "swiglu")
    f = _set_types("fp8blk_swiglu_gemm", [vp] * 8 + [i64, i64, i64, i32, vp, sz, vp])
    _check(f(_ptr(x), _ptr(x_s), _ptr(w1), _ptr(w1_s), _ptr(w3), _ptr(w3_s), _ptr(u), _ptr(us), M, inter, dim,
             scale_fmt, _ptr(ws), ws.numel(), _stream(x.device)), "swiglu_gemm")
    return u, us


def ffn_workspace_bytes(M: int, dim: int, inter: int) -> int:
    i64 = ctypes.c_int64
    return int(_set_types("fp8blk_ffn_workspace_bytes", [i64, i64, i64], ctypes.c_size_t)(M, dim, inter))


def ffn(x: torch.Tensor, w1, w1_s, w3, w3_s, w2, w2_s, scale_fmt: int = SCALE_FP32,
        out: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """Dense SwiGLU FFN with FP8 Linears: x bf16 [M, dim] -> bf16 [M, dim]."""
    _need(x, torch.bfloat16, "x")
    M, dim = x.shape
    inter = w1.shape[0]
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    nb = ffn_workspace_bytes(M, dim, inter)
    if ws is None:
        ws = workspace(nb, x.device, "ffn")
    if out is None:
        out = torch.empty((M, dim), dtype=torch.bfloat16, device=x.device)
    f = _set_types("fp8blk_ffn", [vp] * 8 + [i64, i64, i64, i32, vp, sz, vp])
    _check(f(_ptr(x), _ptr(w1), _ptr(w1_s), _ptr(w3), _ptr(w3_s), _ptr(w2), _ptr(w2_s), _ptr(out), M, dim, inter,
             scale_fmt, _ptr(ws), ws.numel(), _stream(x.device)), "ffn")
    return out


def moe_permute(topk_idx: torch.Tensor, E: int):
    """topk_idx int32 [T, topk] -> (counts int32 [E], offsets int32 [E+1], perm int32 [T*topk]);
    perm past offsets[E] is unspecified."""
    _need(topk_idx, torch.int32, "topk_idx")
    T, k = topk_idx.shape
    dev = topk_idx.device
    counts = torch.empty(E, dtype=torch.int32, device=dev)
    offsets = torch.empty(E + 1, dtype=torch.int32, device=dev)
    perm = torch.empty(max(T * k, 1), dtype=torch.int32, device=dev)
    vp, i64, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_size_t
    nbytes = int(_set_types("fp8blk_moe_permute_workspace_bytes", [i64] * 3, sz)(T, k, E))
    ws = workspace(nbytes, dev, "moe_permute")
    f = _set_types("fp8blk_moe_permute", [vp, i64, i64, i64, vp, vp, vp, vp, sz, vp])
    _check(f(_ptr(topk_idx), T, k, E, _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(ws), ws.numel(), _stream(dev)),
           "moe_permute")
    return counts, offsets, perm[: T * k]


def mla_absorb(inp: torch.Tensor, wkv_b: torch.Tensor, wkv_b_s: torch.Tensor, mode: str,
               out: torch.Tensor | None = None, dn: int = 128, dv: int = 128) -> torch.Tensor:
    """MLA absorb projections with the FP8 wkv_b (e4m3 [H*(dn+dv), C] + block scales).
    mode "qk": q_nope bf16 [T, H, dn] -> bf16 [T, H, C]; mode "v": x bf16 [T, H, C] -> bf16 [T, H, dv]."""
    _need(inp, torch.bfloat16, "inp", ndim=3)
    _need(wkv_b, torch.float8_e4m3fn, "wkv_b")
    _need(wkv_b_s, torch.float32, "wkv_b_s")
    T, H = inp.shape[0], inp.shape[1]
    C = wkv_b.shape[1]
    if out is None:
        out = torch.empty((T, H, C if mode == "qk" else dv), dtype=torch.bfloat16, device=inp.device)
    vp, i64 = ctypes.c_void_p, ctypes.c_int64
    name = "fp8blk_mla_absorb_qk" if mode == "qk" else "fp8blk_mla_absorb_v"
    f = _set_types(name, [vp] * 4 + [i64] * 5 + [vp])
    _check(f(_ptr(inp), _ptr(wkv_b), _ptr(wkv_b_s), _ptr(out), T, H, dn, dv, C, _stream(inp.device)), name)
    return out


MLA_LATENT, MLA_ROPE, MLA_NOPE = 512, 64, 128   # kv_lora_rank, qk_rope_head_dim, qk_nope_head_dim of every config


def mla_append(kv: torch.Tensor, norm_w: torch.Tensor, rope: torch.Tensor, positions: torch.Tensor,
               slots: torch.Tensor, cache: torch.Tensor, q: torch.Tensor | None = None, eps: float = 1e-6,
               q_nope: torch.Tensor | None = None, q_pe: torch.Tensor | None = None):
    """Writes each token's cache row: kv bf16 [T, 576] -> RMS-normed latent (norm_w fp32 [512]) and rotated key
    (rope fp32 [max_pos, 32, 2], positions int64 [T]) at row slots[t] (int64 [T], negative: not written) of
    cache bf16 [pages, page_size, 576]. With q bf16 [T, H, 192] returns (q_nope [T, H, 128], rotated q_pe
    [T, H, 64]), else None. kv and q may have strided rows (inner dimensions contiguous). A slot past the cache is not
    written; a position outside [0, max_pos) is taken as 0. Both set bit 0x100 of last_device_error()."""
    if not kv.is_cuda or kv.dtype != torch.bfloat16 or kv.dim() != 2 or kv.shape[1] != MLA_LATENT + MLA_ROPE:
        raise Fp8BlkError("kv must be a CUDA bfloat16 tensor [T, 576]")
    T = kv.shape[0]
    if kv.stride(1) != 1:
        raise Fp8BlkError("kv: the columns of a row must be contiguous")
    _need(norm_w, torch.float32, "norm_w", ndim=1)
    _need(rope, torch.float32, "rope", ndim=3)
    _need(positions, torch.int64, "positions", ndim=1)
    _need(slots, torch.int64, "slots", ndim=1)
    _need(cache, torch.bfloat16, "cache", ndim=3)
    if norm_w.shape[0] != MLA_LATENT or rope.shape[1:] != (MLA_ROPE // 2, 2) or cache.shape[2] != kv.shape[1]:
        raise Fp8BlkError("norm_w must be [512], rope [max_pos, 32, 2], cache [pages, page_size, 576]")
    if positions.shape[0] != T or slots.shape[0] != T:
        raise Fp8BlkError("positions and slots must be [T]")
    H, q_stride = 0, 0
    if q is not None:
        if not q.is_cuda or q.dtype != torch.bfloat16 or q.dim() != 3 or q.shape[0] != T or \
                q.shape[2] != MLA_NOPE + MLA_ROPE:
            raise Fp8BlkError("q must be a CUDA bfloat16 tensor [T, H, 192]")
        H = q.shape[1]
        if q.stride(2) != 1 or (H > 1 and q.stride(1) != MLA_NOPE + MLA_ROPE):
            raise Fp8BlkError("q: the heads of a token must be contiguous")
        q_stride = q.stride(0) if T > 1 else H * (MLA_NOPE + MLA_ROPE)
        if q_nope is None:
            q_nope = torch.empty((T, H, MLA_NOPE), dtype=torch.bfloat16, device=q.device)
        else:
            _need(q_nope, torch.bfloat16, "q_nope", ndim=3)
        if q_pe is None:
            q_pe = torch.empty((T, H, MLA_ROPE), dtype=torch.bfloat16, device=q.device)
        else:
            _need(q_pe, torch.bfloat16, "q_pe", ndim=3)
        if q_nope.shape != (T, H, MLA_NOPE) or q_pe.shape != (T, H, MLA_ROPE):
            raise Fp8BlkError("q_nope must be [T, H, 128] and q_pe [T, H, 64]")
    else:
        q_nope = q_pe = None
    f = _function("fp8blk_mla_append", "pipfpiipippipippp")
    _check(f(kv.data_ptr(), kv.stride(0) if T > 1 else MLA_LATENT + MLA_ROPE, norm_w.data_ptr(), float(eps), _addr(q),
             q_stride, H, rope.data_ptr(), rope.shape[0], positions.data_ptr(), slots.data_ptr(), T, cache.data_ptr(),
             cache.shape[0] * cache.shape[1], _addr(q_nope), _addr(q_pe), _stream_on(kv)), "mla_append")
    return None if q is None else (q_nope, q_pe)


def mla_attention_workspace_bytes(B: int, H: int, prefix_len: int = 0) -> int:
    return int(_function("fp8blk_mla_attention_workspace_bytes", "iii", ctypes.c_size_t)(B, H, prefix_len))


def mla_attention(q: torch.Tensor, q_pe: torch.Tensor, cache: torch.Tensor, block_table: torch.Tensor,
                  lens: torch.Tensor, scale: float, prefix_pages: torch.Tensor | None = None, prefix_len: int = 0,
                  out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                  ws: torch.Tensor | None = None) -> torch.Tensor:
    """Latent attention of one query token per request: q bf16 [B, H, 512] (mla_absorb "qk" output), q_pe bf16
    [B, H, 64], cache bf16 [pages, page_size, 576], block_table int32 [B, max_pages] and lens int32 [B] (a
    request's own keys), after prefix_len keys of prefix_pages (int32) that every request shares
    -> bf16 [B, H, 512]; lse fp32 [B, H] is written where given. ws: a workspace of mla_attention_workspace_bytes,
    256-byte aligned, any contents."""
    _need(q, torch.bfloat16, "q", ndim=3)
    _need(q_pe, torch.bfloat16, "q_pe", ndim=3)
    _need(cache, torch.bfloat16, "cache", ndim=3)
    _need(block_table, torch.int32, "block_table")
    _need(lens, torch.int32, "lens", ndim=1)
    B, H = q.shape[0], q.shape[1]
    if q.shape[2] != MLA_LATENT or q_pe.shape != (B, H, MLA_ROPE) or \
            cache.shape[2] != MLA_LATENT + MLA_ROPE:
        raise Fp8BlkError("q must be [B, H, 512], q_pe [B, H, 64], cache [pages, page_size, 576]")
    if block_table.shape[0] != B or lens.shape[0] != B:
        raise Fp8BlkError("block_table must be [B, max_pages] and lens [B]")
    pages, page_size = cache.shape[0], cache.shape[1]
    if prefix_len:
        if prefix_pages is None:
            raise Fp8BlkError("prefix_len needs prefix_pages")
        _need(prefix_pages, torch.int32, "prefix_pages", ndim=1)
        if prefix_len > prefix_pages.shape[0] * page_size:
            raise Fp8BlkError("prefix_pages has fewer than prefix_len keys")
    if out is None:
        out = torch.empty((B, H, MLA_LATENT), dtype=torch.bfloat16, device=q.device)
    else:
        _need(out, torch.bfloat16, "out", ndim=3)
        if out.shape != (B, H, MLA_LATENT):
            raise Fp8BlkError("out must be [B, H, 512]")
    if lse is not None:
        _need(lse, torch.float32, "lse")
        if tuple(lse.shape) != (B, H):
            raise Fp8BlkError("lse must be [B, H]")
    stream = _stream_on(q)
    at, room, held = _scratch(ws, 0 if ws is not None else mla_attention_workspace_bytes(B, H, prefix_len), q, stream,
                              "mla_attention", 0)
    f = _function("fp8blk_mla_attention", "ppiipiipipipfpppzp")
    _check(f(q.data_ptr(), q_pe.data_ptr(), B, H, cache.data_ptr(), pages, page_size,
             prefix_pages.data_ptr() if prefix_len else None, prefix_len, block_table.data_ptr(), block_table.shape[1],
             lens.data_ptr(), float(scale), out.data_ptr(), _addr(lse), at, room, stream), "mla_attention")
    return out


SCORE_SOFTMAX, SCORE_SIGMOID = 0, 1


def moe_gate(logits: torch.Tensor, bias: torch.Tensor | None = None, n_groups: int = 1, topk_groups: int = 1,
             topk: int = 8, score_func: int = SCORE_SIGMOID, route_scale: float = 1.0, normalize: bool = True,
             idx: torch.Tensor | None = None, w: torch.Tensor | None = None):
    """Gate logits fp32 [T, E] (+ bias fp32 [E]) -> (topk_idx int32 [T, topk],
    topk_w fp32 [T, topk]): scores, group-limited top-k, weights."""
    _need(logits, torch.float32, "logits")
    if bias is not None:
        _need(bias, torch.float32, "bias", ndim=1)
    T, E = logits.shape
    dev = logits.device
    if idx is None:
        idx = torch.empty((T, topk), dtype=torch.int32, device=dev)
    if w is None:
        w = torch.empty((T, topk), dtype=torch.float32, device=dev)
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int
    f = _set_types("fp8blk_moe_gate", [vp, vp, i64, i64, i64, i64, i64, i32, ctypes.c_float, i32, vp, vp, vp])
    _check(f(_ptr(logits), _ptr(bias), T, E, n_groups, topk_groups, topk, score_func, float(route_scale),
             int(bool(normalize)), _ptr(idx), _ptr(w), _stream(dev)), "moe_gate")
    return idx, w


def moe_route(logits: torch.Tensor, bias: torch.Tensor | None = None, n_groups: int = 1, topk_groups: int = 1,
              topk: int = 8, score_func: int = SCORE_SIGMOID, route_scale: float = 1.0, normalize: bool = True,
              out=None):
    """Gate and routing permutation in one call: logits fp32 [T, E] (+ bias)
    -> (topk_idx int32 [T, topk], topk_w fp32 [T, topk], counts int32 [E],
    offsets int32 [E+1], perm int32 [T*topk]). `out` may pass those five
    tensors to be written in place."""
    _need(logits, torch.float32, "logits")
    if bias is not None:
        _need(bias, torch.float32, "bias", ndim=1)
    T, E = logits.shape
    dev = logits.device
    if out is None:
        out = (torch.empty((T, topk), dtype=torch.int32, device=dev),
               torch.empty((T, topk), dtype=torch.float32, device=dev),
               torch.empty(E, dtype=torch.int32, device=dev), torch.empty(E + 1, dtype=torch.int32, device=dev),
               torch.empty(max(T * topk, 1), dtype=torch.int32, device=dev))
    idx, w, counts, offsets, perm = out
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    nbytes = int(_set_types("fp8blk_moe_route_workspace_bytes", [i64] * 3, sz)(T, topk, E))
    ws = workspace(nbytes, dev, "moe_route")
    f = _set_types("fp8blk_moe_route", [vp, vp, i64, i64, i64, i64, i64, i32, ctypes.c_float, i32] + [vp] * 6 +
                   [sz, vp])
    _check(f(_ptr(logits), _ptr(bias), T, E, n_groups, topk_groups, topk, score_func, float(route_scale),
             int(bool(normalize)), _ptr(idx), _ptr(w), _ptr(counts), _ptr(offsets), _ptr(perm), _ptr(ws), ws.numel(),
             _stream(dev)), "moe_route")
    return idx, w, counts, offsets, perm[: T * topk]


def moe_workspace_bytes(T: int, topk: int, E: int, dim: int, inter: int, n_shared: int = 0) -> int:
    i64 = ctypes.c_int64
    return int(_set_types("fp8blk_moe_workspace_bytes", [i64] * 6, ctypes.c_size_t)(T, topk, E, dim, inter, n_shared))


def moe_grouped_gemm(x: torch.Tensor, x_s: torch.Tensor, topk_idx: torch.Tensor, topk_w: torch.Tensor,
                     w1, w1_s, w3, w3_s, w2, w2_s, E: int, scale_fmt: int = SCALE_FP32,
                     out: torch.Tensor | None = None, ws: torch.Tensor | None = None,
                     n_shared: int = 0) -> torch.Tensor:
    """Routed-expert SwiGLU FFN over stacked block-FP8 experts.
    x e4m3 [T, dim] (+ x_s), topk_idx int32 / topk_w fp32 [T, topk] (ids < E),
    w1/w3 e4m3 [(E+n_shared)*inter, dim], w2 e4m3 [(E+n_shared)*dim, inter] (+ block scales)
    -> bf16 [T, dim]; the last n_shared experts are shared (every token, weight 1, added as y + z)."""
    _need(x, torch.float8_e4m3fn, "x")
    _need(topk_idx, torch.int32, "topk_idx")
    _need(topk_w, torch.float32, "topk_w")
    T, dim = x.shape
    k = topk_idx.shape[1]
    inter = w2.shape[1]
    if ws is None:
        ws = workspace(moe_workspace_bytes(T, k, E, dim, inter, n_shared), x.device, "moe")
    if out is None:
        out = torch.empty((T, dim), dtype=torch.bfloat16, device=x.device)
    vp, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    f = _set_types("fp8blk_moe_grouped_gemm", [vp] * 11 + [i64] * 6 + [i32, vp, sz, vp])
    _check(f(_ptr(x), _ptr(x_s), _ptr(topk_idx), _ptr(topk_w), _ptr(w1), _ptr(w1_s), _ptr(w3), _ptr(w3_s),
             _ptr(w2), _ptr(w2_s), _ptr(out), T, k, E, dim, inter, n_shared, scale_fmt, _ptr(ws), ws.numel(),
             _stream(x.device)), "moe_grouped_gemm")
    return out


MOE_LAYER_MAX_TOKENS = 32


def moe_layer_workspace_bytes(T: int, topk: int, E: int, dim: int, inter: int, n_shared: int = 0) -> int:
    return int(_function("fp8blk_moe_layer_workspace_bytes", "iiiiii", ctypes.c_size_t)(T, topk, E, dim, inter,
                                                                                        n_shared))


def moe_layer(x: torch.Tensor, gate_w: torch.Tensor, w1, w1_s, w3, w3_s, w2, w2_s, topk: int,
              gate_bias: torch.Tensor | None = None, n_groups: int = 1, topk_groups: int = 1,
              score_func: int = SCORE_SIGMOID, route_scale: float = 1.0, normalize: bool = True, n_shared: int = 0,
              scale_fmt: int = SCALE_FP32, out: torch.Tensor | None = None, idx: torch.Tensor | None = None,
              w: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """A whole MoE layer for up to 32 tokens in one kernel: gate product and gate (x bf16 [T, dim], gate_w bf16
    [E, dim], gate_bias fp32 [E]), routed and shared experts (stacked e4m3 weights and block scales as for
    moe_grouped_gemm) and their sum -> bf16 [T, dim]. idx int32 / w fp32 [T, topk] receive the routing where given.
    ws: a workspace of moe_layer_workspace_bytes, 256-byte aligned, whose first 256 bytes were ZERO-FILLED before its
    first use (every call leaves them at zero), used by one stream at a time."""
    _need(x, torch.bfloat16, "x")
    _need(gate_w, torch.bfloat16, "gate_w")
    for t, n, dt in ((w1, "w1", torch.float8_e4m3fn), (w3, "w3", torch.float8_e4m3fn), (w2, "w2", torch.float8_e4m3fn),
                     (w1_s, "w1_s", torch.float32), (w3_s, "w3_s", torch.float32), (w2_s, "w2_s", torch.float32)):
        _need(t, dt, n)
    T, dim = x.shape
    E, inter = gate_w.shape[0], w2.shape[1]
    K = E + n_shared
    if gate_w.shape[1] != dim or w1.shape != (K * inter, dim) or w3.shape != (K * inter, dim) or \
            w2.shape[0] != K * dim:
        raise Fp8BlkError("gate_w must be [E, dim], w1 and w3 [(E + n_shared) * inter, dim], "
                          "w2 [(E + n_shared) * dim, inter]")
    s13, s2 = (K * inter // BLOCK, dim // BLOCK), (K * dim // BLOCK, inter // BLOCK)
    if w1_s.shape != s13 or w3_s.shape != s13 or w2_s.shape != s2:
        raise Fp8BlkError("block scales must have one entry per 128x128 block")
    if gate_bias is not None:
        _need(gate_bias, torch.float32, "gate_bias", ndim=1)
        if gate_bias.shape[0] != E:
            raise Fp8BlkError("gate_bias must be [E]")
    if out is None:
        out = torch.empty((T, dim), dtype=torch.bfloat16, device=x.device)
    else:
        _need(out, torch.bfloat16, "out")
        if out.shape != (T, dim):
            raise Fp8BlkError("out must be [T, dim]")
    for t, n, dt in ((idx, "idx", torch.int32), (w, "w", torch.float32)):
        if t is not None:
            _need(t, dt, n)
            if tuple(t.shape) != (T, topk):
                raise Fp8BlkError(f"{n} must be [T, topk]")
    stream = _stream_on(x)
    at, room, held = _scratch(ws, 0 if ws is not None else moe_layer_workspace_bytes(T, topk, E, dim, inter, n_shared),
                              x, stream, "moe_layer", 256)
    f = _function("fp8blk_moe_layer", "p" * 10 + "i" * 8 + "efeepppzp")
    _check(f(x.data_ptr(), gate_w.data_ptr(), _addr(gate_bias), w1.data_ptr(), w1_s.data_ptr(), w3.data_ptr(),
             w3_s.data_ptr(), w2.data_ptr(), w2_s.data_ptr(), out.data_ptr(), T, topk, E, dim, inter, n_shared, n_groups,
             topk_groups, score_func, float(route_scale), 1 if normalize else 0, scale_fmt, _addr(idx), _addr(w), at, room,
             stream), "moe_layer")
    return out
