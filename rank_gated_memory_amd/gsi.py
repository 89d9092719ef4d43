"""Python binding of libgsi (include/gsi.h): argument marshalling only.

Every operation runs in the HIP kernels of libgsi.so; this module only turns
torch tensors into device pointers and status codes into exceptions.  If the
library is not built the first call raises, there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
from ctypes import POINTER, c_float, c_int32, c_int64, c_size_t, c_uint8, c_void_p

import torch

# GSI_LIBRARY names another build of the same library (the host-sanitizer
# build of build.build_sanitized, for the CPU-side argument tests).
LIB_PATH = os.environ.get("GSI_LIBRARY") or os.path.join(os.path.dirname(os.path.abspath(__file__)), "libgsi.so")

GSI_FP32, GSI_BF16 = 0, 1
GATED, FORCE_FAST, FORCE_SLOW = 0, 1, 2
PHASE_PROJECT, PHASE_APPLY = 1, 2
GSI_OK = 0

_DTYPES = {torch.float32: GSI_FP32, torch.bfloat16: GSI_BF16}


class GsiError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_str(status)} ({status})")


class GsiMapStruct(ctypes.Structure):
    _fields_ = [("d", c_int32), ("d_out", c_int32), ("k", c_int32), ("dtype", c_int32),
                ("W", c_void_p), ("V", c_void_p), ("M", c_void_p), ("G", c_void_p)]


class GsiCallStruct(ctypes.Structure):
    _fields_ = [("map", GsiMapStruct), ("x", c_void_p), ("y", c_void_p), ("eps", c_float),
                ("wave", c_int32), ("rho", c_void_p), ("slow", c_void_p)]


class GsiCalibStruct(ctypes.Structure):
    _fields_ = [("n", c_int32), ("d", c_int32), ("k", c_int32), ("dtype", c_int32),
                ("A", c_void_p), ("V0", c_void_p), ("V", c_void_p), ("iters", c_int32),
                ("reserved", c_int32)]


class GsiWeightsStruct(ctypes.Structure):
    _fields_ = [("d", c_int32), ("d_out", c_int32), ("n", c_int32), ("dtype", c_int32),
                ("bits", c_int32), ("group", c_int32), ("stride", c_int64),
                ("W", c_void_p), ("scales", c_void_p), ("zeros", c_void_p)]


class GsiCacheStruct(ctypes.Structure):
    _fields_ = [("pages", c_int32), ("page", c_int32), ("heads", c_int32), ("d", c_int32),
                ("dtype", c_int32), ("reserved", c_int32), ("page_stride", c_int64),
                ("head_stride", c_int64), ("slot_stride", c_int64), ("K", c_void_p), ("V", c_void_p),
                ("mass", c_void_p), ("age", c_void_p)]


class GsiTableStruct(ctypes.Structure):
    _fields_ = [("table", c_void_p), ("ld", c_int64), ("S", c_int32), ("most", c_int32)]


class GsiHeadsStruct(ctypes.Structure):
    _fields_ = [("p", c_void_p), ("row", c_int64), ("head", c_int64), ("n", c_int32), ("reserved", c_int32)]


class GsiRotationStruct(ctypes.Structure):
    _fields_ = [("d", c_int32), ("start", c_int32), ("layout", c_int32), ("amplitude", c_float),
                ("freq", c_void_p)]


_lib = None


def lib() -> ctypes.CDLL:
    """Load libgsi.so once; raise if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libgsi.so not built at {LIB_PATH}; run __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        L.gsi_abi_version.restype = c_int32
        L.gsi_status_str.restype = ctypes.c_char_p
        L.gsi_status_str.argtypes = [c_int32]
        L.gsi_image_bytes.restype = c_size_t
        L.gsi_image_bytes.argtypes = [c_int32, c_int32, c_int32]
        L.gsi_gram_bytes.restype = c_size_t
        L.gsi_gram_bytes.argtypes = [c_int32, c_int32]
        L.gsi_prepare.restype = c_int32
        L.gsi_prepare.argtypes = [POINTER(GsiMapStruct), c_void_p]
        L.gsi_linear_workspace.restype = c_size_t
        L.gsi_linear_workspace.argtypes = [POINTER(GsiMapStruct), c_int32]
        L.gsi_linear.restype = c_int32
        L.gsi_linear.argtypes = [POINTER(GsiMapStruct), c_void_p, c_void_p, c_int32, c_float,
                                 c_int32, c_void_p, c_void_p, c_void_p, c_size_t, c_void_p]
        L.gsi_stack_plan_bytes.restype = c_size_t
        L.gsi_stack_plan_bytes.argtypes = [POINTER(GsiCallStruct), c_int32]
        L.gsi_stack_plan.restype = c_int32
        L.gsi_stack_plan.argtypes = [POINTER(GsiCallStruct), c_int32, c_void_p, c_size_t]
        L.gsi_stack_workspace.restype = c_size_t
        L.gsi_stack_workspace.argtypes = [c_void_p]
        L.gsi_stack.restype = c_int32
        L.gsi_stack.argtypes = [c_void_p, c_void_p, c_int32, c_void_p, c_size_t, c_void_p]
        L.gsi_stack_status_offset.restype = c_size_t
        L.gsi_stack_status_offset.argtypes = [c_void_p]
        L.gsi_calibrate_workspace.restype = c_size_t
        L.gsi_calibrate_workspace.argtypes = [POINTER(GsiCalibStruct)]
        L.gsi_calibrate_status_offset.restype = c_size_t
        L.gsi_calibrate_status_offset.argtypes = []
        L.gsi_calibrate.restype = c_int32
        L.gsi_calibrate.argtypes = [POINTER(GsiCalibStruct), c_void_p, c_size_t, c_void_p]
        L.gsi_static_scratch_bytes.restype = c_size_t
        L.gsi_static_scratch_bytes.argtypes = []
        L.gsi_linear_static.restype = c_int32
        L.gsi_linear_static.argtypes = [POINTER(GsiMapStruct), c_void_p, c_void_p, c_int32, c_float,
                                        c_int32, c_void_p, c_void_p, c_void_p]
        L.gsi_stack_phase.restype = c_int32
        L.gsi_stack_phase.argtypes = [c_void_p, c_void_p, c_int32, c_int32, c_void_p, c_size_t,
                                      c_void_p]
        L.gsi_q4_linear.restype = c_int32
        L.gsi_q4_linear.argtypes = [POINTER(GsiWeightsStruct), c_void_p, c_int64, c_void_p, c_int64,
                                    c_int32, c_void_p]
        L.gsi_grouped_linear.restype = c_int32
        L.gsi_grouped_linear.argtypes = [POINTER(GsiWeightsStruct), c_void_p, c_int64, c_int32, c_void_p,
                                         c_void_p, c_void_p, c_int64, c_int32, c_void_p]
        L.gsi_group_rows.restype = c_int32
        L.gsi_group_rows.argtypes = [c_void_p, c_int32, c_int32, c_int32, c_int32, c_void_p, c_void_p,
                                     c_void_p, c_void_p]
        L.gsi_group_combine.restype = c_int32
        L.gsi_group_combine.argtypes = [c_void_p, c_int64, c_int32, c_void_p, c_void_p, c_void_p, c_int64,
                                        c_void_p, c_int64, c_int32, c_int32, c_int32, c_int32, c_void_p]
        rotation, heads = POINTER(GsiRotationStruct), POINTER(GsiHeadsStruct)
        cache, table = POINTER(GsiCacheStruct), POINTER(GsiTableStruct)
        L.gsi_rotary.restype = c_int32
        L.gsi_rotary.argtypes = [rotation, heads, heads, c_int32, c_int32, c_int32, c_void_p, c_int32, c_void_p]
        L.gsi_cache_append.restype = c_int32
        L.gsi_cache_append.argtypes = [cache, table, c_void_p, c_void_p, heads, heads, c_int32, rotation, c_void_p,
                                       c_int32, heads, heads, c_void_p]
        L.gsi_cache_attend_workspace.restype = c_size_t
        L.gsi_cache_attend_workspace.argtypes = [cache, table, c_int32, c_int32]
        L.gsi_cache_attend.restype = c_int32
        L.gsi_cache_attend.argtypes = [cache, table, c_void_p, heads, heads, c_float, c_int32, c_int32, c_void_p,
                                       c_void_p, c_size_t, c_void_p]
        L.gsi_cache_evict.restype = c_int32
        L.gsi_cache_evict.argtypes = [cache, table, c_void_p, c_int32, c_int32, table, c_void_p, c_void_p, c_void_p]
        _lib = L
    return _lib


def status_str(status: int) -> str:
    return lib().gsi_status_str(int(status)).decode()


def _check(status: int, where: str):
    if status != GSI_OK:
        raise GsiError(status, where)


def _ptr(t) -> int:
    return 0 if t is None else int(t.data_ptr())


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {t.dtype}")
    return _DTYPES[t.dtype]


def gsi_abi_version() -> int:
    return int(lib().gsi_abi_version())


def gsi_image_bytes(d_out: int, k: int, dtype: int) -> int:
    return int(lib().gsi_image_bytes(d_out, k, dtype))


class Map:
    """A linear map W [d_out][d] with basis V [d][k], its cached image M and,
    with exact_rho, the cached E = V^T V - I that makes its gates use the
    exact residual ratio of the stored basis."""

    def __init__(self, W: torch.Tensor, V: torch.Tensor, M: torch.Tensor | None = None,
                 exact_rho: bool = False):
        if W.dim() != 2 or V.dim() != 2 or W.shape[1] != V.shape[0]:
            raise ValueError(f"shapes W {tuple(W.shape)} and V {tuple(V.shape)} do not chain")
        if W.dtype != V.dtype:
            raise TypeError("W and V must share a dtype")
        if not (W.is_contiguous() and V.is_contiguous()):
            raise ValueError("W and V must be contiguous")
        self.W, self.V = W, V
        self.d_out, self.d = W.shape
        self.k = V.shape[1]
        self.dtype = _dtype_code(W)
        nbytes = gsi_image_bytes(self.d_out, self.k, self.dtype)
        if M is None:
            M = torch.empty(max(nbytes, 16), dtype=torch.uint8, device=W.device)
        self.M = M
        self.G = None
        if exact_rho:
            self.G = torch.empty(max(int(lib().gsi_gram_bytes(self.k, self.dtype)), 16), dtype=torch.uint8,
                                 device=W.device)
        self.struct = GsiMapStruct(self.d, self.d_out, self.k, self.dtype,
                                   _ptr(W), _ptr(V), _ptr(M), _ptr(self.G))

    def gram(self) -> torch.Tensor:
        """E = V^T V - I as built by gsi_prepare ([k][k], storage dtype)."""
        return self.G[: self.k * self.k * self.W.element_size()].view(self.W.dtype).view(self.k, self.k)

    def image_rows(self) -> torch.Tensor:
        """The image M as a [d_out][k] tensor (un-tiles the library layout)."""
        el = self.W.dtype
        vw = 16 // self.W.element_size()
        tiles = (self.d_out + 63) // 64
        m = self.M[: tiles * 64 * self.k * self.W.element_size()].view(el)
        m = m.view(tiles, self.k // vw, 64, vw).permute(0, 2, 1, 3).reshape(tiles * 64, self.k)
        return m[: self.d_out]


def gsi_prepare(m: Map, stream=None) -> Map:
    """Build M = W V_k into m.M."""
    _check(lib().gsi_prepare(ctypes.byref(m.struct), _stream(stream)), "gsi_prepare")
    return m


def gsi_linear_workspace(m: Map, T: int) -> int:
    return int(lib().gsi_linear_workspace(ctypes.byref(m.struct), int(T)))


def workspace(nbytes: int, device) -> torch.Tensor:
    """A zero-filled workspace buffer (zero before first use, as gsi.h requires),
    for calls of one layout: gsi_linear of one T and one size of map, or stacks of
    the same sizes and waves.  For calls of another layout take another one, or
    zero_() this one in between: where one layout counts, another keeps sums."""
    return torch.zeros(max(int(nbytes), 256), dtype=torch.uint8, device=device)


def gsi_linear(m: Map, x: torch.Tensor, eps: float, mode: int = GATED, y=None, rho=None,
               slow=None, ws=None, stream=None):
    """Gated map on x [T][d]; returns (y [T][d_out], rho [T], slow [T] uint8).
    ws: a workspace() of gsi_linear_workspace(m, T) bytes, used before only by
    calls of the same T and sizes of map, or zeroed since."""
    if x.dim() == 1:
        x = x[None]
    T = x.shape[0]
    if x.dtype != m.W.dtype or not x.is_contiguous() or x.shape[1] != m.d:
        raise ValueError("x must be a contiguous [T][d] tensor in the map's dtype")
    dev = x.device
    if y is None:
        y = torch.empty((T, m.d_out), dtype=x.dtype, device=dev)
    if rho is None:
        rho = torch.empty(T, dtype=torch.float32, device=dev)
    if slow is None:
        slow = torch.empty(T, dtype=torch.uint8, device=dev)
    need = gsi_linear_workspace(m, T)
    if ws is None:
        ws = workspace(need, dev)
    st = lib().gsi_linear(ctypes.byref(m.struct), _ptr(x), _ptr(y), int(T), float(eps), int(mode),
                          _ptr(rho), _ptr(slow), _ptr(ws), ws.numel() * ws.element_size(),
                          _stream(stream))
    _check(st, "gsi_linear")
    return y, rho, slow


def gsi_linear_static(m: Map, x: torch.Tensor, eps: float, mode: int = GATED, y=None, rho=None,
                      slow=None, stream=None):
    """gsi_linear with the library's own device scratch (no workspace, no
    allocation by the library); y, rho and slow are allocated here only if
    not given."""
    if x.dim() == 1:
        x = x[None]
    T = x.shape[0]
    if x.dtype != m.W.dtype or not x.is_contiguous() or x.shape[1] != m.d:
        raise ValueError("x must be a contiguous [T][d] tensor in the map's dtype")
    dev = x.device
    if y is None:
        y = torch.empty((T, m.d_out), dtype=x.dtype, device=dev)
    if rho is None:
        rho = torch.empty(T, dtype=torch.float32, device=dev)
    if slow is None:
        slow = torch.empty(T, dtype=torch.uint8, device=dev)
    st = lib().gsi_linear_static(ctypes.byref(m.struct), _ptr(x), _ptr(y), int(T), float(eps), int(mode),
                                 _ptr(rho), _ptr(slow), _stream(stream))
    _check(st, "gsi_linear_static")
    return y, rho, slow


def gsi_static_scratch_bytes() -> int:
    return int(lib().gsi_static_scratch_bytes())


class Stack:
    """A stack plan over batch-1 calls, with its device copy.

    calls: list of (Map, x [d], y [d_out], eps, rho (1 float) or None,
    slow (1 byte) or None[, wave]).  Calls of one wave are independent; a
    call may read the y of a call of an earlier wave.  Tensors must stay
    alive as long as the plan.
    """

    def __init__(self, calls, device=None):
        self._keep = calls
        n = len(calls)
        arr = (GsiCallStruct * max(n, 1))()
        for i, call in enumerate(calls):
            m, x, y, eps, rho, slow = call[:6]
            wave = int(call[6]) if len(call) > 6 else 0
            arr[i] = GsiCallStruct(m.struct, _ptr(x), _ptr(y), float(eps), wave, _ptr(rho), _ptr(slow))
        self._arr = arr
        nbytes = int(lib().gsi_stack_plan_bytes(arr, n))
        if n > 0 and nbytes == 0:
            # run the full check to get the failing status
            _check(lib().gsi_stack_plan(arr, n, None, 0), "gsi_stack_plan")
            raise GsiError(7, "gsi_stack_plan_bytes")
        self.host = torch.zeros(max(nbytes, 256), dtype=torch.uint8)
        _check(lib().gsi_stack_plan(arr, n, _ptr(self.host), self.host.numel()), "gsi_stack_plan")
        self.n = n
        self.ws_bytes = int(lib().gsi_stack_workspace(_ptr(self.host)))
        dev = device if device is not None else (calls[0][1].device if n else "cpu")
        self.dev = self.host.to(dev) if n else None
        self.status_offset = int(lib().gsi_stack_status_offset(_ptr(self.host)))

    def status(self, ws: torch.Tensor) -> int:
        """The device status word of this plan's runs in `ws` (0 = every run completed)."""
        o = self.status_offset
        return int(ws[o:o + 4].cpu().view(torch.int32)[0])

    def run(self, mode: int = GATED, ws=None, stream=None, check: bool = False):
        """Enqueue the plan's launch; with check=True wait for the stream and
        raise StackIncomplete if the launch left its status word set."""
        if ws is None:
            ws = workspace(self.ws_bytes, self.dev.device)
        gsi_stack(self, mode, ws, stream, check=check)
        return ws


class StackIncomplete(RuntimeError):
    """A stack launch ended with a device-side wait that ran out of its bound:
    the outputs of that run are incomplete (include/gsi.h, gsi_stack)."""

    def __init__(self, word: int):
        self.word = word
        super().__init__(f"gsi_stack: a device-side wait ran out (status word {word:#x}); outputs incomplete")


def gsi_stack(plan: Stack, mode: int, ws: torch.Tensor, stream=None, check: bool = False):
    """Run a plan (one launch).  ws: a workspace() of plan.ws_bytes, used before
    only by plans of the same sizes and waves, or zeroed since.  gsi_stack returns
    GSI_OK once the launch is
    enqueued; whether every device-side wait finished is only known from the
    workspace's status word after the stream has run, which check=True
    reads (synchronising the stream) and turns into StackIncomplete."""
    st = lib().gsi_stack(_ptr(plan.host), _ptr(plan.dev), int(mode), _ptr(ws),
                         ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "gsi_stack")
    if check:
        if stream is None:
            torch.cuda.current_stream().synchronize()
        elif hasattr(stream, "synchronize"):
            stream.synchronize()
        else:
            torch.cuda.synchronize()
        word = plan.status(ws)
        if word != 0:
            raise StackIncomplete(word)


def gsi_stack_phase(plan: Stack, mode: int, phase: int, ws: torch.Tensor, stream=None):
    st = lib().gsi_stack_phase(_ptr(plan.host), _ptr(plan.dev), int(mode), int(phase), _ptr(ws),
                               ws.numel() * ws.element_size(), _stream(stream))
    _check(st, "gsi_stack_phase")


def gsi_calibrate(A: torch.Tensor, V0: torch.Tensor, iters: int, V=None, ws=None, stream=None):
    """Basis of the dominant k-dim subspace of the samples A [n][d] after
    `iters` sweeps of subspace iteration from V0 [d][k] (random: a cold
    start; the previous layer's basis: the cascade).  Returns (V, status)
    where status is the device status word (0 = good) as a 1-element tensor."""
    if A.dim() != 2 or V0.dim() != 2 or A.shape[1] != V0.shape[0]:
        raise ValueError("A [n][d] and V0 [d][k] do not chain")
    if A.dtype != V0.dtype or not (A.is_contiguous() and V0.is_contiguous()):
        raise ValueError("A and V0 must be contiguous and share a dtype")
    n, d = A.shape
    k = V0.shape[1]
    if V is None:
        V = torch.empty_like(V0)
    c = GsiCalibStruct(n, d, k, _dtype_code(A), _ptr(A), _ptr(V0), _ptr(V), int(iters), 0)
    need = int(lib().gsi_calibrate_workspace(ctypes.byref(c)))
    if ws is None:
        ws = workspace(need, A.device)
    _check(lib().gsi_calibrate(ctypes.byref(c), _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)),
           "gsi_calibrate")
    o = int(lib().gsi_calibrate_status_offset())
    return V, ws[o:o + 4].view(torch.int32)


# ---- plain linear maps: weights in 4 bits, weights of many experts ----

# The raw handle of a device's current stream without building a Stream object
# (a microsecond and a half of a call's five), where this torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _call(where: str, fn, device: torch.device, stream, *args):
    """fn(*args, stream) on `device`: its own current stream unless one is given,
    whatever device is current."""
    if device.type != "cuda":
        raise ValueError(f"{where}: tensors must be on the GPU")
    index, current = device.index, _current_device()
    if stream is None:
        raw = _raw_stream(current if index is None else index)
    else:
        raw = int(stream.cuda_stream) if hasattr(stream, "cuda_stream") else int(stream)
    if index is None or index == current:
        status = fn(*args, raw)
    else:
        with torch.cuda.device(device):
            status = fn(*args, raw)
    if status != GSI_OK:
        raise GsiError(status, where)


def _empty(shape, dtype, device: torch.device, stream) -> torch.Tensor:
    """A new output, allocated on the stream that the call runs on: memory freed
    on the current one may still be written by what runs there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _sizes(where: str, *sizes: int):
    """The library's sizes are int32, and ctypes drops the bits above without a word."""
    if max(sizes) >= 1 << 31:
        raise ValueError(f"{where}: sizes must be below 2^31, are {sizes}")


def _rows2d(t: torch.Tensor, name: str, dtype, device, cols: int, n: int | None = None) -> int:
    """The row stride of a [n][cols] tensor whose rows are contiguous; fewer than
    two rows have none that counts."""
    shape = t.shape
    if len(shape) != 2 or shape[1] != cols or (n is not None and shape[0] != n):
        raise ValueError(f"{name} must be [{'n' if n is None else n}][{cols}], is {tuple(shape)}")
    if t.dtype is not dtype or t.device != device:
        raise ValueError(f"{name} must be {dtype} on {device}, is {t.dtype} on {t.device}")
    s0, s1 = t.stride()
    if s1 != 1 and cols > 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    return s0 if shape[0] > 1 else cols


def _ints(t: torch.Tensor, name: str, shape, device):
    if t.dtype is not torch.int32 or t.device != device or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous int32 {tuple(shape)} on {device}, "
                         f"is {t.dtype} {tuple(t.shape)} on {t.device}")


class Q4:
    """One map or the maps of n experts in 4 bits: w = scale (code - zero).

    codes  : uint8 [d_out][d / 2] or [n][d_out][d / 2], the even column of a
             pair in the low nibble
    scales : [..][ceil(d / group)] in the dtype of x and y (bf16 or fp32)
    zeros  : uint8 like scales, values 0..15, or None for 8 everywhere
    The tensors are used where they lie and must stay alive as long as this."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, zeros: torch.Tensor | None = None,
                 group: int = 128):
        if codes.dim() not in (2, 3) or codes.dtype != torch.uint8:
            raise ValueError("codes must be uint8 [d_out][d / 2] or [n][d_out][d / 2]")
        if group not in (32, 64, 128):
            raise ValueError(f"group must be 32, 64 or 128, is {group}")
        self.codes, self.scales, self.zeros, self.group = codes, scales, zeros, group
        self.n = codes.shape[0] if codes.dim() == 3 else 1
        self.d_out, self.d = codes.shape[-2], 2 * codes.shape[-1]
        _sizes("Q4", self.n, self.d_out, self.d)
        self.dtype, self.device = scales.dtype, codes.device
        want = (*codes.shape[:-1], (self.d + group - 1) // group)
        for t, name in ((scales, "scales"), (zeros, "zeros")):
            if t is not None and (tuple(t.shape) != want or t.device != codes.device):
                raise ValueError(f"{name} must be {want} on {codes.device}")
        if zeros is not None and zeros.dtype != torch.uint8:
            raise ValueError("zeros must be uint8")
        if not all(t is None or t.is_contiguous() for t in (codes, scales, zeros)):
            raise ValueError("codes, scales and zeros must be contiguous")
        self.struct = GsiWeightsStruct(self.d, self.d_out, self.n, _dtype_code(scales), 4, group, 0,
                                       _ptr(codes), _ptr(scales), _ptr(zeros))


def gsi_q4_linear(w: Q4, x: torch.Tensor, y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """y [T][d_out] = x [T][d] through one map in 4 bits; x [d] is one token
    and gives y [1][d_out]."""
    if x.dim() == 1:
        x = x[None]
    dtype, dev, d_out = w.dtype, w.device, w.d_out
    ldx = _rows2d(x, "x", dtype, dev, w.d)
    T = x.shape[0]
    _sizes("gsi_q4_linear", T)
    if y is None:
        y, ldy = _empty((T, d_out), dtype, dev, stream), d_out
    else:
        ldy = _rows2d(y, "y", dtype, dev, d_out, T)
    _call("gsi_q4_linear", lib().gsi_q4_linear, dev, stream, w.struct, x.data_ptr(), ldx, y.data_ptr(), ldy, T)
    return y


def gsi_grouped_linear(w, x: torch.Tensor, offsets: torch.Tensor, rows: torch.Tensor | None = None,
                       y: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """The rows of y ordered by expert: y[r] = W[e] x[rows[r]] for r in
    [offsets[e], offsets[e + 1]); without rows, y[r] = W[e] x[r].  w is a
    tensor [n][d_out][d] (each map contiguous, maps any stride apart) or a Q4
    of n maps.  Rows of y behind the last expert's are not written."""
    if isinstance(w, Q4):
        struct, d, d_out, n, dtype, dev = w.struct, w.d, w.d_out, w.n, w.dtype, w.device
    else:
        if w.dim() != 3:
            raise ValueError(f"W must be [n][d_out][d], is {tuple(w.shape)}")
        n, d_out, d = w.shape
        stride, s1, s2 = w.stride()
        if s2 != 1 or s1 != d:
            raise ValueError("every map of W must be contiguous")
        dtype, dev = w.dtype, w.device
        struct = GsiWeightsStruct(d, d_out, n, _dtype_code(w), 0, 0, stride, w.data_ptr(), None, None)
    ldx = _rows2d(x, "x", dtype, dev, d)
    R = x.shape[0] if rows is None else rows.shape[0]
    _sizes("gsi_grouped_linear", x.shape[0], R, n, d_out, d)
    _ints(offsets, "offsets", (n + 1,), dev)
    if rows is not None:
        _ints(rows, "rows", (R,), dev)
    if y is None:
        y, ldy = _empty((R, d_out), dtype, dev, stream), d_out
    else:
        ldy = _rows2d(y, "y", dtype, dev, d_out, R)
    _call("gsi_grouped_linear", lib().gsi_grouped_linear, dev, stream, struct, x.data_ptr(), ldx, x.shape[0],
          offsets.data_ptr(), _ptr(rows), y.data_ptr(), ldy, R)
    return y


def gsi_group_rows(ids: torch.Tensor, n: int, offsets: torch.Tensor | None = None,
                   rows: torch.Tensor | None = None, pos: torch.Tensor | None = None, stream=None):
    """Order the expert numbers ids [T][top] (int32 or int64; numbers outside
    [0, n) are dropped) by expert: (offsets [n + 1], rows [T * top], the token
    of each grouped row, pos [T][top], the grouped row of each choice or -1)."""
    if ids.dim() != 2 or ids.dtype not in (torch.int32, torch.int64) or not ids.is_contiguous():
        raise ValueError("ids must be contiguous [T][top], int32 or int64")
    T, top = ids.shape
    dev = ids.device
    _sizes("gsi_group_rows", T, top, n)
    if offsets is None and rows is None and pos is None:
        at = T * top
        rows, pos, offsets = _empty(2 * at + n + 1, torch.int32, dev, stream).split((at, at, n + 1))
        pos = pos.view(T, top)
    else:
        offsets = _empty(n + 1, torch.int32, dev, stream) if offsets is None else offsets
        rows = _empty(T * top, torch.int32, dev, stream) if rows is None else rows
        pos = _empty((T, top), torch.int32, dev, stream) if pos is None else pos
        _ints(offsets, "offsets", (n + 1,), dev)
        _ints(rows, "rows", (T * top,), dev)
        _ints(pos, "pos", (T, top), dev)
    _call("gsi_group_rows", lib().gsi_group_rows, dev, stream, ids.data_ptr(), ids.element_size(), T, top, n,
          offsets.data_ptr(), rows.data_ptr(), pos.data_ptr())
    return offsets, rows, pos


def gsi_group_combine(y: torch.Tensor, pos: torch.Tensor, weights: torch.Tensor | None = None,
                      base: torch.Tensor | None = None, out: torch.Tensor | None = None,
                      stream=None) -> torch.Tensor:
    """out[t] = base[t] + sum_j weights[t][j] y[pos[t][j]]; a pos outside y's
    rows adds nothing, weights None are 1, base None is 0; out may be base."""
    if y.dim() != 2 or pos.dim() != 2:
        raise ValueError("y must be [R][d] and pos [T][top]")
    T, top = pos.shape
    d, dtype, dev = y.shape[1], y.dtype, y.device
    _sizes("gsi_group_combine", T, top, y.shape[0], d)
    ldy = _rows2d(y, "y", dtype, dev, d)
    _ints(pos, "pos", (T, top), dev)
    if weights is not None and (weights.dtype != torch.float32 or weights.device != dev or not weights.is_contiguous()
                                or weights.shape != pos.shape):
        raise ValueError("weights must be contiguous fp32 like pos")
    ldb = 0 if base is None else _rows2d(base, "base", dtype, dev, d, T)
    if out is None:
        out, ldo = _empty((T, d), dtype, dev, stream), d
    else:
        ldo = _rows2d(out, "out", dtype, dev, d, T)
    _call("gsi_group_combine", lib().gsi_group_combine, dev, stream, y.data_ptr(), ldy, y.shape[0], pos.data_ptr(),
          _ptr(weights), _ptr(base), ldb, out.data_ptr(), ldo, T, top, d, _dtype_code(y))
    return out


# ---- a key-value cache in pages: rotary positions, appending, attention, eviction ----

_LAYOUTS = {"pairs": 0, "halves": 1}


def rotary_freqs(d: int, base: float = 10000.0, scaling: str | None = None, factor: float = 1.0,
                 original: int = 0, low: float = 1.0, high: float = 32.0) -> torch.Tensor:
    """Radians per position of the d / 2 pairs, f_i = base^(-2 i / d), in 64 bits;
    for contexts `factor` times as long as the weights were made for:

    scaling "linear" : f_i / factor, positions pressed together
            "base"   : the base times factor^(d / (d - 2)), so that the slowest
                       pair alone goes `factor` times slower (d > 2)
            "bands"  : pairs that turn at least `high` times within `original`
                       positions as they are, those that turn at most `low`
                       times `factor` times slower, in between in between
                       (usually with an amplitude of 0.1 ln(factor) + 1)"""
    if d < 2 or d % 2:
        raise ValueError(f"d must be even and at least 2, is {d}")
    if scaling not in (None, "linear", "base", "bands"):
        raise ValueError(f"scaling must be linear, base or bands, is {scaling!r}")
    if not factor > 0 or not base > 0:
        raise ValueError("base and factor must be positive")
    if scaling == "base":
        if d == 2:
            raise ValueError("scaling of the base needs d > 2")
        base = base * factor ** (d / (d - 2))
    f = float(base) ** (-torch.arange(0, d, 2, dtype=torch.float64) / d)
    if scaling == "linear":
        return f / factor
    if scaling == "bands":
        if original < 1 or not low < high:
            raise ValueError("scaling by bands needs original >= 1 and low < high")
        turns = original * f / (2.0 * torch.pi)
        keep = ((turns - low) / (high - low)).clamp(0.0, 1.0)
        return f * (keep + (1.0 - keep) / factor)
    return f


class Rotary:
    """Rotary positions: the frequencies of d / 2 pairs (radians per position, as
    rotary_freqs gives them), their layout in a head ("pairs": elements 2 i and
    2 i + 1; "halves": i and i + d / 2, from element `start` on) and the factor
    of the turned elements.  Elements outside stay as they are."""

    def __init__(self, freqs: torch.Tensor, layout: str = "halves", start: int = 0, amplitude: float = 1.0,
                 device=None):
        if layout not in _LAYOUTS:
            raise ValueError(f"layout must be pairs or halves, is {layout!r}")
        if freqs.dim() != 1 or freqs.numel() < 1:
            raise ValueError("freqs must hold a frequency for each pair")
        self.freqs = freqs.to(device=device, dtype=torch.float64).contiguous()
        self.d, self.layout, self.start, self.amplitude = 2 * freqs.numel(), layout, int(start), float(amplitude)
        self.device = self.freqs.device
        _sizes("Rotary", self.d, abs(self.start))
        self.struct = GsiRotationStruct(self.d, self.start, _LAYOUTS[layout], self.amplitude, _ptr(self.freqs))


class Cache:
    """A pool of pages of keys and values, K and V [pages][heads][page][d] with
    the elements of an entry contiguous and the same strides (a pool stored as
    [pages][page][heads][d] is passed as its transpose(1, 2)); mass fp32 and age
    int32 [pages][heads][page], contiguous, or None.  The tensors are used where
    they lie and must stay alive as long as this."""

    def __init__(self, K: torch.Tensor, V: torch.Tensor, mass: torch.Tensor | None = None,
                 age: torch.Tensor | None = None):
        if K.dim() != 4 or K.shape != V.shape:
            raise ValueError(f"K and V must be [pages][heads][page][d], are {tuple(K.shape)} and {tuple(V.shape)}")
        if K.dtype != V.dtype or K.device != V.device:
            raise ValueError("K and V must share a dtype and a device")
        self.K, self.V, self.mass, self.age = K, V, mass, age
        self.pages, self.heads, self.page, self.d = K.shape
        _sizes("Cache", *K.shape)
        self.dtype, self.device = K.dtype, K.device
        for t, name, dtype in ((mass, "mass", torch.float32), (age, "age", torch.int32)):
            if t is not None and (t.shape != K.shape[:3] or t.dtype != dtype or t.device != K.device
                                  or not t.is_contiguous()):
                raise ValueError(f"{name} must be contiguous {dtype} {tuple(K.shape[:3])} on {K.device}")
        strides = []  # those of a single page, head or slot do not count
        for n, k, v in zip(K.shape, K.stride(), V.stride()):
            if n > 1 and k != v:
                raise ValueError("K and V must have the same strides")
            strides.append(k if n > 1 else self.d)
        if K.stride(3) != 1 or V.stride(3) != 1:
            raise ValueError("the elements of an entry must be contiguous")
        self.struct = GsiCacheStruct(self.pages, self.page, self.heads, self.d, _dtype_code(K), 0, *strides[:3],
                                     _ptr(K), _ptr(V), _ptr(mass), _ptr(age))
        self.needs = {}  # bytes of workspace by the sizes of a gsi_cache_attend call


_INT = (1 << 31) - 1  # the library's sizes are int32, and ctypes drops the bits above without a word


def _heads(t: torch.Tensor, name: str, dtype, device, d: int, T: int | None = None, n: int | None = None):
    """A [T][n][d] tensor whose heads are contiguous."""
    shape = t.shape
    if len(shape) != 3 or shape[2] != d or (T is not None and shape[0] != T) or (n is not None and shape[1] != n):
        raise ValueError(f"{name} must be [{'T' if T is None else T}][{'heads' if n is None else n}][{d}], "
                         f"is {tuple(shape)}")
    if t.dtype is not dtype or t.device != device:
        raise ValueError(f"{name} must be {dtype} on {device}, is {t.dtype} on {t.device}")
    s0, s1, s2 = t.stride()
    if s2 != 1:
        raise ValueError(f"{name}: the elements of a head must be contiguous")
    heads = shape[1]
    if heads > _INT or shape[0] > _INT:
        raise ValueError(f"{name}: sizes must be below 2^31, are {tuple(shape)}")
    return GsiHeadsStruct(t.data_ptr(), s0, s1, heads)


def _new_heads(like: torch.Tensor, T: int, n: int, d: int, stream):
    """A new contiguous [T][n][d] tensor and its description."""
    if stream is not None:
        t = _empty((T, n, d), like.dtype, like.device, stream)
    elif like.is_contiguous():
        t = torch.empty_like(like)
    else:
        t = like.new_empty((T, n, d))
    return t, GsiHeadsStruct(t.data_ptr(), n * d, d, n)


def _table(t: torch.Tensor, name: str, device, S: int | None = None):
    """Page numbers [S][most], int32, rows contiguous."""
    shape = t.shape
    if len(shape) != 2 or t.dtype is not torch.int32 or t.device != device or (S is not None and shape[0] != S):
        raise ValueError(f"{name} must be int32 [{'S' if S is None else S}][most] on {device}, "
                         f"is {t.dtype} {tuple(shape)} on {t.device}")
    rows, most = shape
    s0, s1 = t.stride()
    if rows > _INT or most > _INT:
        raise ValueError(f"{name}: sizes must be below 2^31, are {tuple(shape)}")
    if s1 != 1 and most > 1:
        raise ValueError(f"{name}: the page numbers of a sequence must be contiguous")
    return GsiTableStruct(t.data_ptr(), s0 if rows > 1 else most, rows, most)


def _positions(t: torch.Tensor, T: int, device) -> int:
    """The bytes of a position."""
    dtype = t.dtype
    if (dtype is not torch.int64 and dtype is not torch.int32) or t.device != device or t.shape != (T,) \
            or not t.is_contiguous():
        raise ValueError(f"positions must be contiguous int32 or int64 ({T},) on {device}, "
                         f"is {t.dtype} {tuple(t.shape)} on {t.device}")
    return 8 if dtype is torch.int64 else 4


def gsi_rotary(r: Rotary, x: torch.Tensor, positions: torch.Tensor, y: torch.Tensor | None = None,
               stream=None) -> torch.Tensor:
    """y = x [T][heads][d] with every head turned by its token's position
    ([T], int32 or int64, may be negative); y may be x."""
    if x.dim() != 3:
        raise ValueError(f"x must be [T][heads][d], is {tuple(x.shape)}")
    T, n, d = x.shape
    dtype, dev = x.dtype, x.device
    hx = _heads(x, "x", dtype, dev, d)
    pos_bytes = _positions(positions, T, dev)
    if r.device != dev:
        raise ValueError(f"the frequencies must be on {dev}, are on {r.device}")
    code = _dtype_code(x)
    if y is None:
        y, hy = _new_heads(x, T, n, d, stream)
    else:
        hy = _heads(y, "y", dtype, dev, d, T, n)
    _call("gsi_rotary", lib().gsi_rotary, dev, stream, r.struct, hx, hy, T, d, code, positions.data_ptr(), pos_bytes)
    return y


def gsi_cache_append(c: Cache, table: torch.Tensor, slots: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                     seq: torch.Tensor | None = None, rotary: Rotary | None = None,
                     positions: torch.Tensor | None = None, q: torch.Tensor | None = None,
                     q_out: torch.Tensor | None = None, stream=None):
    """Write the keys k and values v [T][heads][d] into slot slots[t] of sequence
    seq[t] (None: t) of the table [S][most]; keys, and queries q [T][heads'][d],
    are turned by `rotary` at `positions`.  Rows whose slot has no page write
    nothing.  Returns the turned queries (q_out, which may be q), or None."""
    dtype, dev, d, heads = c.dtype, c.device, c.d, c.heads
    hk = _heads(k, "k", dtype, dev, d, None, heads)
    T = k.shape[0]
    hv = _heads(v, "v", dtype, dev, d, T, heads)
    pages = _table(table, "table", dev)
    _ints(slots, "slots", (T,), dev)
    if seq is not None:
        _ints(seq, "seq", (T,), dev)
    pos_bytes = 4 if positions is None else _positions(positions, T, dev)
    if rotary is not None and rotary.device != dev:
        raise ValueError(f"the frequencies must be on {dev}, are on {rotary.device}")
    hq = ho = None
    if q is not None:
        hq = _heads(q, "q", dtype, dev, d, T)
        if q_out is None:
            q_out, ho = _new_heads(q, T, hq.n, d, stream)
        else:
            ho = _heads(q_out, "q_out", dtype, dev, d, T, hq.n)
    elif q_out is not None:
        raise ValueError("q_out needs q")
    _call("gsi_cache_append", lib().gsi_cache_append, dev, stream, c.struct, pages, _ptr(seq), slots.data_ptr(), hk, hv,
          T, None if rotary is None else rotary.struct, _ptr(positions), pos_bytes, hq, ho)
    return q_out


def gsi_cache_attend_workspace(c: Cache, table: torch.Tensor, q_heads: int, accumulate: bool = False) -> int:
    return int(lib().gsi_cache_attend_workspace(c.struct, _table(table, "table", c.device), int(q_heads),
                                                int(accumulate)))


def gsi_cache_attend(c: Cache, table: torch.Tensor, lengths: torch.Tensor, q: torch.Tensor,
                     scale: float | None = None, window: int = 0, accumulate: bool = False,
                     out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
                     ws: torch.Tensor | None = None, stream=None):
    """Attention of one token q [S][q heads][d] of each sequence over the first
    lengths[s] slots of its pages, or the last `window` of them: (out like q,
    lse [S][q heads] fp32).  scale None is d^-0.5.  accumulate adds each slot's
    weights to the cache's mass.  ws: device memory of
    gsi_cache_attend_workspace() bytes with any contents; with accumulate it goes
    by the table's width: table[:, :m], of the pages that the longest sequence
    needs, asks for less."""
    dtype, dev, d = c.dtype, c.device, c.d
    hq = _heads(q, "q", dtype, dev, d)
    S, n = q.shape[0], hq.n
    if not 0 <= window <= _INT:
        raise ValueError(f"window must be in 0..2^31 - 1, is {window}")
    pages = _table(table, "table", dev, S)
    _ints(lengths, "lengths", (S,), dev)
    accumulate = bool(accumulate)
    if accumulate and c.mass is None:
        raise ValueError("accumulate needs a cache with mass")
    if out is None:
        out, ho = _new_heads(q, S, n, d, stream)
    else:
        ho = _heads(out, "out", dtype, dev, d, S, n)
    if lse is None:
        lse = q.new_empty((S, n), dtype=torch.float32) if stream is None else _empty((S, n), torch.float32, dev, stream)
    elif lse.dtype is not torch.float32 or lse.device != dev or lse.shape != (S, n) or not lse.is_contiguous():
        raise ValueError(f"lse must be contiguous fp32 ({S}, {n}) on {dev}")
    if ws is None:
        sizes = (S, pages.most, n, accumulate)
        need = c.needs.get(sizes)
        if need is None:
            if len(c.needs) >= 256:
                c.needs.clear()
            need = c.needs[sizes] = int(lib().gsi_cache_attend_workspace(c.struct, pages, n, accumulate))
        if need:
            ws = _empty(need, torch.uint8, dev, stream)
    else:
        if ws.device != dev or not ws.is_contiguous():
            raise ValueError(f"ws must be contiguous on {dev}")
        need = ws.numel() * ws.element_size()
    _call("gsi_cache_attend", lib().gsi_cache_attend, dev, stream, c.struct, pages, lengths.data_ptr(), hq, ho,
          d**-0.5 if scale is None else float(scale), int(window), accumulate, lse.data_ptr(), _ptr(ws), need)
    return out, lse


def gsi_cache_evict(c: Cache, table: torch.Tensor, lengths: torch.Tensor, budget: int, recent: int = 0,
                    to: torch.Tensor | None = None, lengths_out: torch.Tensor | None = None,
                    moved: torch.Tensor | None = None, stream=None):
    """Cut every sequence of more than `budget` entries to it: each key head keeps
    its `recent` newest entries and those of the largest mass, in place or, with
    `to` [S][most'], copied into other pages of the pool.  Returns (lengths_out
    [S], moved [S][heads][budget]: the slot each slot's entry came from, or -1).
    The call goes by the table's width: table[:, :m], of the pages that the longest
    sequence needs, is faster than a wide one."""
    dev = c.device
    pages = _table(table, "table", dev)
    S = pages.S
    _ints(lengths, "lengths", (S,), dev)
    if c.mass is None:
        raise ValueError("eviction needs a cache with mass")
    if not 1 <= budget <= _INT or not 0 <= recent <= budget:
        raise ValueError(f"budget must be in 1..2^31 - 1 and recent in 0..budget, are {budget} and {recent}")
    target = None if to is None else _table(to, "to", dev, S)
    if lengths_out is None:
        lengths_out = _empty(S, torch.int32, dev, stream)
    else:
        _ints(lengths_out, "lengths_out", (S,), dev)
    if moved is None:
        moved = _empty((S, c.heads, budget), torch.int32, dev, stream)
    else:
        _ints(moved, "moved", (S, c.heads, budget), dev)
    _call("gsi_cache_evict", lib().gsi_cache_evict, dev, stream, c.struct, pages, lengths.data_ptr(), int(budget),
          int(recent), target, lengths_out.data_ptr(), moved.data_ptr())
    return lengths_out, moved
