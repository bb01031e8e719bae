"""Python binding of liblowbit.so: weight-only low-bit GEMM for B200 (sm_100a).

Argument marshalling only: every step of the computation runs in the library's CUDA
kernels. PyTorch provides device memory and streams. The binding raises if the library
is missing; there is no fallback.

    Y = gemm(x, packed, scales, zeros, bits, group_size)   # Y[M][N] = X[M][K] W^T
    Y = adapter_gemm(x, packed, scales, zeros, bits, group_size, a, b, scaling, index)
    dX = gemm_dx(dy, packed_t, scales, zeros, bits, group_size)
    dX, dA, dB = adapter_backward(dy, x, p, packed_t, scales, zeros, bits, group_size, a, b, scaling, index)

Layouts (see include/lowbit.h): x bf16 [M][K]; packed int32 view of uint32 words
[N][K*bits/32]; scales / zeros fp16 [K/group_size][N]; y bf16 [M][N].
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
from typing import NamedTuple, Optional, Sequence, Union

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "liblowbit.so")
DEBUG_LIB_PATH = os.path.join(_HERE, "liblowbit_debug.so")

STATUS = {
    0: "LOWBIT_OK", 1: "LOWBIT_ERR_INVALID_ARG", 2: "LOWBIT_ERR_ALIGNMENT", 3: "LOWBIT_ERR_UNSUPPORTED",
    4: "LOWBIT_ERR_UNSUPPORTED_DEVICE", 5: "LOWBIT_ERR_BAD_CODE", 6: "LOWBIT_ERR_TIMEOUT", 7: "LOWBIT_ERR_CUDA",
    8: "LOWBIT_ERR_WORKSPACE", 9: "LOWBIT_ERR_DEVICE_CHECK",
}


class LowbitError(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {STATUS.get(status, status)}")


class GemmDesc(ctypes.Structure):
    _fields_ = [("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
                ("bits", ctypes.c_int), ("group_size", ctypes.c_int),
                ("X", ctypes.c_void_p), ("Wp", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("zeros", ctypes.c_void_p), ("Y", ctypes.c_void_p)]


class Adapters(ctypes.Structure):
    _fields_ = [("num", ctypes.c_int), ("rank", ctypes.c_int), ("A", ctypes.c_void_p), ("B", ctypes.c_void_p),
                ("scaling", ctypes.c_void_p), ("index", ctypes.c_void_p)]


_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load liblowbit.so (raises FileNotFoundError if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    _lib = open_library(path)
    return _lib


_debug_lib = None


def load_debug() -> ctypes.CDLL:
    """Load liblowbit_debug.so: the same library built with device-side index checks."""
    global _debug_lib
    if _debug_lib is None:
        _debug_lib = open_library(DEBUG_LIB_PATH)
    return _debug_lib


def open_library(path: str) -> ctypes.CDLL:
    """Open a build of the library at `path` and declare its C signatures."""
    if not os.path.exists(path):
        raise FileNotFoundError(f"{path} is missing: build it with `python -m bit_weight_only_w2_b200.build`")
    lib = ctypes.CDLL(path)
    i64, i32, p = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p
    lib.lowbit_status_string.argtypes = [i32]
    lib.lowbit_status_string.restype = ctypes.c_char_p
    lib.lowbit_version.restype = i32
    lib.lowbit_packed_words.argtypes = [i64, i64, i32]
    lib.lowbit_packed_words.restype = ctypes.c_size_t
    lib.lowbit_pack.argtypes = [p, i64, i64, i32, p, p]
    lib.lowbit_pack.restype = i32
    lib.lowbit_unpack.argtypes = [p, i64, i64, i32, p, p]
    lib.lowbit_unpack.restype = i32
    sz = ctypes.c_size_t
    lib.lowbit_gemm_workspace_size.argtypes = [i64, i64]
    lib.lowbit_gemm_workspace_size.restype = sz
    lib.lowbit_gemm.argtypes = [i64, i64, i64, i32, i32, p, p, p, p, p, p, sz, p]
    lib.lowbit_gemm.restype = i32
    lib.lowbit_gemm_ex.argtypes = [i64, i64, i64, i32, i32, p, p, p, p, p, p, sz, i32, i32, i32, p]
    lib.lowbit_gemm_ex.restype = i32
    lib.lowbit_gemm_batch.argtypes = [ctypes.POINTER(GemmDesc), i32, p, sz, p]
    lib.lowbit_gemm_batch.restype = i32
    lib.lowbit_device_status.argtypes = [i32]
    lib.lowbit_device_status.restype = i32
    lib.lowbit_selftest_bounded_wait.argtypes = [ctypes.c_longlong, p]
    lib.lowbit_selftest_bounded_wait.restype = i32
    lib.lowbit_last_device_status.argtypes = [p]
    lib.lowbit_last_device_status.restype = i32
    lib.lowbit_test_fail_next.argtypes = [i32]
    lib.lowbit_test_fail_next.restype = i32
    lib.lowbit_debug_checks_enabled.argtypes = []
    lib.lowbit_debug_checks_enabled.restype = i32
    lib.lowbit_selftest_index_check.argtypes = [p]
    lib.lowbit_selftest_index_check.restype = i32
    lib.lowbit_gemm_noalloc.argtypes = [i64, i64, i64, i32, i32, p, p, p, p, p, p]
    lib.lowbit_gemm_noalloc.restype = i32
    ad = ctypes.POINTER(Adapters)
    lib.lowbit_transposed_words.argtypes = [i64, i64, i32]
    lib.lowbit_transposed_words.restype = sz
    lib.lowbit_transpose.argtypes = [p, i64, i64, i32, p, p]
    lib.lowbit_transpose.restype = i32
    lib.lowbit_adapter_workspace_size.argtypes = [i64, i64, i64, i32, i32]
    lib.lowbit_adapter_workspace_size.restype = sz
    lib.lowbit_adapter_gemm.argtypes = [i64, i64, i64, i32, i32, p, p, p, p, ad, p, p, p, p, p, sz, p]
    lib.lowbit_adapter_gemm.restype = i32
    lib.lowbit_gemm_dx.argtypes = [i64, i64, i64, i32, i32, p, p, p, p, p, p, sz, p]
    lib.lowbit_gemm_dx.restype = i32
    lib.lowbit_adapter_backward.argtypes = [i64, i64, i64, i32, i32, p, p, p, p, ad, p, p, p, p, p, p, p, p, sz, p]
    lib.lowbit_adapter_backward.restype = i32
    lib.lowbit_checkpoint_store.argtypes = [p, i64, i64, p, p, p]
    lib.lowbit_checkpoint_store.restype = i32
    lib.lowbit_checkpoint_load.argtypes = [p, p, i64, i64, p, p]
    lib.lowbit_checkpoint_load.restype = i32
    return lib


def _check(st: int, what: str) -> None:
    if st != 0:
        raise LowbitError(st, what)


def _stream(t: Optional[torch.Tensor] = None) -> int:
    dev = t.device if t is not None else None
    return torch.cuda.current_stream(dev).cuda_stream


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _need(t: torch.Tensor, dtype, name: str, ndim: int = 2):
    if t.dtype != dtype or not t.is_contiguous() or t.dim() != ndim:
        raise ValueError(f"{name}: expected a contiguous {ndim}-D {dtype} tensor, got {t.dtype} "
                         f"{tuple(t.shape)} (contiguous={t.is_contiguous()})")


def _need_cuda(*named):
    for name, t in named:
        if t is not None and not t.is_cuda:
            raise ValueError(f"{name}: expected a CUDA tensor, got one on {t.device}")


def _check_gemm_args(x, packed, scales, zeros, out, bits: int, group_size: int):
    """Shapes, dtypes and devices of a GEMM's tensors against each other, before any library call:
    the tensor maps are built from M, N and K, so a buffer smaller than its shape implies would be
    read or written past its end on the GPU. Bits and group sizes the library rejects anyway are
    left to it (it returns LOWBIT_ERR_INVALID_ARG / _UNSUPPORTED)."""
    _need(x, torch.bfloat16, "x")
    _need(packed, torch.int32, "packed")
    _need(scales, torch.float16, "scales")
    if zeros is not None:
        _need(zeros, torch.float16, "zeros")
    if out is not None:
        _need(out, torch.bfloat16, "out")
    M, K = x.shape
    N = scales.shape[1]
    if group_size > 0 and K % group_size == 0 and scales.shape[0] != K // group_size:
        raise ValueError(f"scales: expected shape ({K // group_size}, N) (group-major [K/g][N]), "
                         f"got {tuple(scales.shape)}")
    if bits in (1, 2, 4) and K * bits % 32 == 0 and tuple(packed.shape) != (N, K * bits // 32):
        raise ValueError(f"packed: expected shape {(N, K * bits // 32)} for N={N}, K={K}, bits={bits}, "
                         f"got {tuple(packed.shape)}")
    if zeros is not None and tuple(zeros.shape) != tuple(scales.shape):
        raise ValueError(f"zeros: expected the scales' shape {tuple(scales.shape)}, got {tuple(zeros.shape)}")
    if out is not None and tuple(out.shape) != (M, N):
        raise ValueError(f"out: expected shape {(M, N)}, got {tuple(out.shape)}")
    for name, t in (("packed", packed), ("scales", scales), ("zeros", zeros), ("out", out)):
        if t is not None and t.device != x.device:
            raise ValueError(f"{name}: on {t.device}, but x is on {x.device}")
    _need_cuda(("x", x))
    return M, N, K


def version() -> int:
    return int(load().lowbit_version())


def packed_words(N: int, K: int, bits: int) -> int:
    return int(load().lowbit_packed_words(N, K, bits))


def pack(codes: torch.Tensor, bits: int) -> torch.Tensor:
    """int8 codes [N][K] (binary -1/+1, ternary -1/0/+1, uint4 0..15) -> packed words
    [N][K*bits/32] (int32 storage of uint32 words). Synchronous."""
    _need(codes, torch.int8, "codes")
    _need_cuda(("codes", codes))
    N, K = codes.shape
    out = torch.empty((N, K * bits // 32), dtype=torch.int32, device=codes.device)
    with torch.cuda.device(codes.device):
        _check(load().lowbit_pack(_ptr(codes), N, K, bits, _ptr(out), _stream(codes)), "lowbit_pack")
    return out


def unpack(packed: torch.Tensor, N: int, K: int, bits: int) -> torch.Tensor:
    """Inverse of pack: packed words [N][K*bits/32] -> int8 codes [N][K]. Synchronous."""
    _need(packed, torch.int32, "packed")
    if bits in (1, 2, 4) and N >= 0 and K >= 0 and K * bits % 32 == 0 and packed.numel() != N * K * bits // 32:
        raise ValueError(f"packed: {packed.numel()} words, but N={N}, K={K}, bits={bits} needs {N * K * bits // 32}")
    _need_cuda(("packed", packed))
    out = torch.empty((N, K), dtype=torch.int8, device=packed.device)
    with torch.cuda.device(packed.device):
        _check(load().lowbit_unpack(_ptr(packed), N, K, bits, _ptr(out), _stream(packed)), "lowbit_unpack")
    return out


def workspace_size(M: int, K: int) -> int:
    return int(load().lowbit_gemm_workspace_size(M, K))


def _workspace_size_fast(M: int, K: int) -> int:
    # the closed form lowbit_gemm_workspace_size returns (fp16 X copy + fp32 row factors, each
    # rounded up to 256 bytes); tests check the two agree
    return ((M * K * 2 + 255) // 256 + (M * 4 + 255) // 256) * 256


_workspaces = {}


def workspace(device: torch.device, nbytes: int) -> torch.Tensor:
    """A cached per-device workspace buffer of at least `nbytes` (grown on demand). Work that
    uses it is ordered on the current stream; callers running GEMMs on several streams at once
    should pass their own buffers."""
    dev = torch.device(device)
    key = dev.index if dev.index is not None else torch.cuda.current_device()
    buf = _workspaces.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.empty(max(nbytes, 1 << 20), dtype=torch.uint8, device=torch.device("cuda", key))
        _workspaces[key] = buf
    return buf


def gemm(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, zeros: Optional[torch.Tensor],
         bits: int, group_size: int, out: Optional[torch.Tensor] = None, tile_tokens: int = 0,
         ksplit: int = 0, ws: Optional[torch.Tensor] = None, tile_rows: int = 0) -> torch.Tensor:
    """Y[M][N] = X[M][K] * W^T with W decoded from `packed`, `scales` (and `zeros`)."""
    M, N, K = _check_gemm_args(x, packed, scales, zeros, out, bits, group_size)
    if ws is not None:
        _need(ws, torch.uint8, "ws", ndim=1)
        if ws.device != x.device:
            raise ValueError(f"ws: on {ws.device}, but x is on {x.device}")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    dev = x.get_device()
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            return _gemm_call(x, packed, scales, zeros, bits, group_size, out, tile_tokens, ksplit, ws, tile_rows,
                              M, N, K, dev)
    return _gemm_call(x, packed, scales, zeros, bits, group_size, out, tile_tokens, ksplit, ws, tile_rows, M, N, K,
                      dev)


def _gemm_call(x, packed, scales, zeros, bits, group_size, out, tile_tokens, ksplit, ws, tile_rows, M, N, K, dev):
    lib = _lib if _lib is not None else load()
    if ws is None:
        ws = workspace(x.device, _workspace_size_fast(M, K))
    stream = torch.cuda.current_stream().cuda_stream
    zp = None if zeros is None else zeros.data_ptr()
    if tile_tokens or ksplit or tile_rows:
        st = lib.lowbit_gemm_ex(M, N, K, bits, group_size, x.data_ptr(), packed.data_ptr(), scales.data_ptr(), zp,
                                out.data_ptr(), ws.data_ptr(), ws.numel(), tile_tokens, tile_rows, ksplit, stream)
    else:
        st = lib.lowbit_gemm(M, N, K, bits, group_size, x.data_ptr(), packed.data_ptr(), scales.data_ptr(), zp,
                             out.data_ptr(), ws.data_ptr(), ws.numel(), stream)
    if st != 0:
        raise LowbitError(st, "lowbit_gemm")
    return out


def make_desc(x, packed, scales, zeros, y, bits: int, group_size: int) -> GemmDesc:
    """One linear of a lowbit_gemm_batch call (the tensors must outlive the call)."""
    if y is None:
        raise ValueError("y: a batch descriptor needs its output tensor")
    M, N, K = _check_gemm_args(x, packed, scales, zeros, y, bits, group_size)
    return GemmDesc(M, N, K, bits, group_size, _ptr(x), _ptr(packed), _ptr(scales), _ptr(zeros), _ptr(y))


def gemm_batch(descs: Sequence[GemmDesc], device: Optional[torch.device] = None,
               ws: Optional[torch.Tensor] = None) -> None:
    """Run the descriptors in order on the current stream (see lowbit_gemm_batch)."""
    arr = (GemmDesc * len(descs))(*descs)
    dev = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
    with torch.cuda.device(dev):
        if ws is None:
            need = max((workspace_size(d.M, d.K) for d in descs), default=0)
            ws = workspace(dev, need)
        _check(load().lowbit_gemm_batch(arr, len(descs), _ptr(ws), ws.numel(), _stream()), "lowbit_gemm_batch")


# ---- adapters, gradients and 8-bit activation copies -----------------------------------------
class Checkpoint(NamedTuple):
    """8-bit copy of an activation [M][K]: `codes` float8_e4m3fn [M][K] and `exps` uint8 [M][K/32], a
    power-of-two exponent + 127 for each 32 values of a row (see lowbit_checkpoint_store)."""
    codes: torch.Tensor
    exps: torch.Tensor


def checkpoint_empty(M: int, K: int, device) -> Checkpoint:
    """Buffers for the 8-bit copy of an [M][K] activation (K a multiple of 32)."""
    if K % 32:
        raise ValueError(f"K: expected a multiple of 32, got {K}")
    return Checkpoint(torch.empty((M, K), dtype=torch.float8_e4m3fn, device=device),
                      torch.empty((M, K // 32), dtype=torch.uint8, device=device))


def _check_checkpoint(ck: Checkpoint, M: int, K: int, device, name: str = "checkpoint"):
    _need(ck.codes, torch.float8_e4m3fn, f"{name}.codes")
    _need(ck.exps, torch.uint8, f"{name}.exps")
    if tuple(ck.codes.shape) != (M, K) or tuple(ck.exps.shape) != (M, K // 32) or K % 32:
        raise ValueError(f"{name}: expected codes {(M, K)} and exps {(M, K // 32)} with K a multiple of 32, got "
                         f"{tuple(ck.codes.shape)} and {tuple(ck.exps.shape)}")
    for part, t in (("codes", ck.codes), ("exps", ck.exps)):
        if t.device != device:
            raise ValueError(f"{name}.{part}: on {t.device}, expected {device}")


# The entry points below run in a few microseconds on the GPU, so their arguments are checked in three
# forms that accept the same calls: compiled (_marshal.so: checks, allocations and the library call),
# one boolean expression over everything that a correct call satisfies (where _marshal.so was built
# for another PyTorch, or is not there), and, only when that does not hold, the checks that name what
# is wrong.
_BF16, _F16, _F32, _I32, _U8 = torch.bfloat16, torch.float16, torch.float32, torch.int32, torch.uint8
_F8 = torch.float8_e4m3fn


def _fits(t, dtype, shape, dev: int) -> bool:
    return t.dtype is dtype and t.shape == shape and t.get_device() == dev and t.is_contiguous()


class _Marshalled:
    """The compiled calls of the loaded library. Each returns None where it leaves the call to Python."""

    def __init__(self, lib):
        self.lib = lib
        try:
            from . import _marshal
        except ImportError:
            _marshal = None
        if _marshal is not None and _marshal.torch_version != torch.__version__.split("+")[0]:
            _marshal = None
        size = self._address("adapter_workspace_size")
        for name in ("adapter_gemm", "gemm_dx", "adapter_backward"):
            self._set(_marshal, name, size)
        for name in ("checkpoint_store", "checkpoint_load"):
            self._set(_marshal, name)

    def _address(self, name: str) -> int:
        return ctypes.cast(getattr(self.lib, "lowbit_" + name), ctypes.c_void_p).value

    def _set(self, module, name: str, *more) -> None:
        call = getattr(module, name, None)
        setattr(self, name, (lambda *args: None) if call is None else functools.partial(call, self._address(name), *more))


_marshalled: Optional[_Marshalled] = None


def _calls() -> _Marshalled:
    global _marshalled
    if _marshalled is None or _marshalled.lib is not _lib:
        _marshalled = _Marshalled(load())
    return _marshalled


def _raw_stream(dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev)


def _on_device(dev: int):
    """The context to launch on device `dev`: nothing to do on the current one."""
    return contextlib.nullcontext() if dev == torch._C._cuda_getDevice() else torch.cuda.device(dev)


def _check_like(t: torch.Tensor, name: str, shape, dtype, device):
    _need(t, dtype, name, ndim=len(shape))
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, expected {device}")


def _copy_fits(ck, M: int, K: int, dev: int) -> bool:
    return K % 32 == 0 and _fits(ck.codes, _F8, (M, K), dev) and _fits(ck.exps, _U8, (M, K // 32), dev)


def checkpoint_store(x: torch.Tensor, out: Optional[Checkpoint] = None) -> Checkpoint:
    """The 8-bit copy of x (bf16 [M][K], K a multiple of 32)."""
    r = _calls().checkpoint_store(x) if out is None else None
    if r is not None:
        if type(r) is int:
            raise LowbitError(r, "lowbit_checkpoint_store")
        return Checkpoint(*r)
    if not (x.dim() == 2 and x.dtype is _BF16 and x.is_contiguous() and x.is_cuda):
        _need(x, _BF16, "x")
        _need_cuda(("x", x))
    M, K = x.shape
    dev = x.get_device()
    if out is None:
        out = checkpoint_empty(M, K, x.device)
    elif not _copy_fits(out, M, K, dev):
        _check_checkpoint(out, M, K, x.device, "out")
    with _on_device(dev):
        _check(load().lowbit_checkpoint_store(x.data_ptr(), M, K, out.codes.data_ptr(), out.exps.data_ptr(),
                                              _raw_stream(dev)), "lowbit_checkpoint_store")
    return out


def checkpoint_load(ck: Checkpoint, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The bf16 values an 8-bit copy stands for."""
    codes = ck.codes
    r = _calls().checkpoint_load(codes, ck.exps, out)
    if r is not None:
        if type(r) is int:
            raise LowbitError(r, "lowbit_checkpoint_load")
        return r
    if not (codes.dim() == 2 and codes.is_cuda and _copy_fits(ck, *codes.shape, codes.get_device())):
        _need(codes, _F8, "checkpoint.codes")
        _need_cuda(("checkpoint.codes", codes))
        _check_checkpoint(ck, *codes.shape, codes.device)
    M, K = codes.shape
    dev = codes.get_device()
    if out is None:
        out = torch.empty((M, K), dtype=_BF16, device=codes.device)
    elif not _fits(out, _BF16, (M, K), dev):
        _check_like(out, "out", (M, K), _BF16, codes.device)
    with _on_device(dev):
        _check(load().lowbit_checkpoint_load(codes.data_ptr(), ck.exps.data_ptr(), M, K, out.data_ptr(),
                                             _raw_stream(dev)), "lowbit_checkpoint_load")
    return out


def transposed_words(N: int, K: int, bits: int) -> int:
    return int(load().lowbit_transposed_words(N, K, bits))


def transpose_packed(packed: torch.Tensor, K: int, bits: int) -> torch.Tensor:
    """W's packed words [N][K*bits/32] -> W^T's [K][ceil(N/128)*128*bits/32], which gemm_dx and
    adapter_backward read. Done once per weight."""
    _need(packed, torch.int32, "packed")
    _need_cuda(("packed", packed))
    N = packed.shape[0]
    if bits not in (1, 2, 4) or K * bits % 32 or packed.shape[1] != K * bits // 32:
        raise ValueError(f"packed: expected [N][{K * bits // 32 if bits in (1, 2, 4) else 'K*bits/32'}] words for K={K}, "
                         f"bits={bits}, got {tuple(packed.shape)}")
    out = torch.empty((K, (N + 127) // 128 * 128 * bits // 32), dtype=torch.int32, device=packed.device)
    with torch.cuda.device(packed.device):
        _check(load().lowbit_transpose(_ptr(packed), N, K, bits, _ptr(out), _stream()), "lowbit_transpose")
    return out


@functools.lru_cache(maxsize=4096)
def adapter_workspace_size(M: int, N: int, K: int, num: int, rank: int) -> int:
    """Bytes of workspace of adapter_gemm, adapter_backward and (num = rank = 0) gemm_dx."""
    return int(load().lowbit_adapter_workspace_size(M, N, K, num, rank))


def _own_workspace(ws: Optional[torch.Tensor], like: torch.Tensor, M, N, K, num, rank):
    # allocated per call by default: the caching allocator ties it to the current stream (and to the
    # pool of a graph under capture), so calls on several streams or in several graphs never share it
    if ws is None:
        need = adapter_workspace_size(M, N, K, num, rank)
        return like.new_empty(need // 2 + 1), need
    _need(ws, _U8, "ws", ndim=1)
    if ws.device != like.device:
        raise ValueError(f"ws: on {ws.device}, expected {like.device}")
    return ws, ws.numel()


def _adapters_fit(a, b, scaling, index, M: int, N: int, K: int, dev: int) -> bool:
    if a.dim() != 3:
        return False
    L, R, _ = a.shape
    return (_fits(a, _BF16, (L, R, K), dev) and _fits(b, _BF16, (L, N, R), dev) and _fits(scaling, _F32, (L,), dev) and
            (index is None or _fits(index, _I32, (M,), dev)))


def _check_adapters(a, b, scaling, index, M, N, K, device) -> None:
    _need(a, torch.bfloat16, "a", ndim=3)
    _need(b, torch.bfloat16, "b", ndim=3)
    L, R = a.shape[0], a.shape[1]
    if tuple(a.shape) != (L, R, K) or tuple(b.shape) != (L, N, R):
        raise ValueError(f"a, b: expected shapes (L, R, {K}) and (L, {N}, R), got {tuple(a.shape)} and {tuple(b.shape)}")
    _check_like(scaling, "scaling", (L,), torch.float32, device)
    if index is not None:
        _check_like(index, "index", (M,), torch.int32, device)
    for name, t in (("a", a), ("b", b)):
        if t.device != device:
            raise ValueError(f"{name}: on {t.device}, expected {device}")


def _linear_fits(x, words, scales, zeros, bits: int, group_size: int, transposed: bool) -> bool:
    """x [M][K] with W's words, or dy [M][N] with W^T's."""
    if not (x.dim() == 2 and scales.dim() == 2 and words.dim() == 2 and x.is_cuda and bits in (1, 2, 4) and group_size > 0):
        return False
    dev = x.get_device()
    M, red = x.shape
    N = scales.shape[1]
    K = words.shape[0] if transposed else red
    wide = (K, (N + 127) // 128 * 128 * bits // 32) if transposed else (N, K * bits // 32)
    groups = (K // group_size, N)
    return (K % group_size == 0 and x.dtype is _BF16 and x.is_contiguous() and _fits(words, _I32, wide, dev) and
            _fits(scales, _F16, groups, dev) and (zeros is None or _fits(zeros, _F16, groups, dev)) and
            (not transposed or red == N))


def adapter_gemm(x: torch.Tensor, packed: torch.Tensor, scales: torch.Tensor, zeros: Optional[torch.Tensor],
                 bits: int, group_size: int, a: torch.Tensor, b: torch.Tensor, scaling: torch.Tensor,
                 index: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                 p: Optional[torch.Tensor] = None, checkpoint: Optional[Checkpoint] = None,
                 ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Y = X W^T + p B^T, p = scaling * X A^T with each token's own adapter (see lowbit_adapter_gemm).

    a bf16 [L][R][K], b bf16 [L][N][R], scaling fp32 [L], index int32 [M] (values outside 0..L-1: no
    adapter; None: adapter 0 for every token). For training, pass buffers that the backward reads:
    `p` bf16 [M][R] and, to keep X in 8 bits, `checkpoint` (checkpoint_empty(M, K, device)). No autograd
    graph is recorded, whatever requires_grad says of the inputs: the caller calls adapter_backward (from a
    torch.autograd.Function, say). With an index and more than 16 tokens, an adapter whose b is not finite
    throughout gives its own tokens NaN in every column; else only the columns concerned change."""
    codes, exps = checkpoint if checkpoint is not None else (None, None)
    r = _calls().adapter_gemm(x, packed, scales, zeros, bits, group_size, a, b, scaling, index, out, p, codes, exps, ws)
    if r is not None:
        if type(r) is int:
            raise LowbitError(r, "lowbit_adapter_gemm")
        return r
    if not _linear_fits(x, packed, scales, zeros, bits, group_size, False):
        _check_gemm_args(x, packed, scales, zeros, out, bits, group_size)
    M, K = x.shape
    N = scales.shape[1]
    dev = x.get_device()
    if not _adapters_fit(a, b, scaling, index, M, N, K, dev):
        _check_adapters(a, b, scaling, index, M, N, K, x.device)
    L, R, _ = a.shape
    if out is None:
        out = x.new_empty((M, N))
    elif not _fits(out, _BF16, (M, N), dev):
        _check_like(out, "out", (M, N), _BF16, x.device)
    if p is not None and not _fits(p, _BF16, (M, R), dev):
        _check_like(p, "p", (M, R), _BF16, x.device)
    if checkpoint is not None and not _copy_fits(Checkpoint(codes, exps), M, K, dev):   # (any pair will do)
        _check_checkpoint(Checkpoint(codes, exps), M, K, x.device)
    ad = Adapters(L, R, a.data_ptr(), b.data_ptr(), scaling.data_ptr(), _ptr(index))
    with _on_device(dev):
        ws, ws_bytes = _own_workspace(ws, x, M, N, K, L, R)
        _check(load().lowbit_adapter_gemm(M, N, K, bits, group_size, x.data_ptr(), packed.data_ptr(), scales.data_ptr(),
                                          _ptr(zeros), ctypes.byref(ad), out.data_ptr(), _ptr(p), _ptr(codes), _ptr(exps),
                                          ws.data_ptr(), ws_bytes, _raw_stream(dev)), "lowbit_adapter_gemm")
    return out


def _check_grad_args(dy, packed_t, scales, zeros, bits: int, group_size: int):
    _need(dy, torch.bfloat16, "dy")
    _need(packed_t, torch.int32, "packed_t")
    _need(scales, torch.float16, "scales")
    M, N = dy.shape
    K = packed_t.shape[0]
    if bits in (1, 2, 4) and packed_t.shape[1] != (N + 127) // 128 * 128 * bits // 32:
        raise ValueError(f"packed_t: expected {(K, (N + 127) // 128 * 128 * bits // 32)} for N={N}, bits={bits}, "
                         f"got {tuple(packed_t.shape)}")
    if group_size > 0 and K % group_size == 0 and tuple(scales.shape) != (K // group_size, N):
        raise ValueError(f"scales: expected shape {(K // group_size, N)}, got {tuple(scales.shape)}")
    if zeros is not None:
        _need(zeros, torch.float16, "zeros")
        if tuple(zeros.shape) != tuple(scales.shape):
            raise ValueError(f"zeros: expected the scales' shape {tuple(scales.shape)}, got {tuple(zeros.shape)}")
    for name, t in (("packed_t", packed_t), ("scales", scales), ("zeros", zeros)):
        if t is not None and t.device != dy.device:
            raise ValueError(f"{name}: on {t.device}, but dy is on {dy.device}")
    _need_cuda(("dy", dy))
    return M, N, K


def gemm_dx(dy: torch.Tensor, packed_t: torch.Tensor, scales: torch.Tensor, zeros: Optional[torch.Tensor], bits: int,
            group_size: int, out: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None) -> torch.Tensor:
    """dX = dY W, the input gradient of gemm (dy bf16 [M][N], packed_t from transpose_packed). Like gemm
    it records no autograd graph."""
    r = _calls().gemm_dx(dy, packed_t, scales, zeros, bits, group_size, out, ws)
    if r is not None:
        if type(r) is int:
            raise LowbitError(r, "lowbit_gemm_dx")
        return r
    if not _linear_fits(dy, packed_t, scales, zeros, bits, group_size, True):
        _check_grad_args(dy, packed_t, scales, zeros, bits, group_size)
    M, N = dy.shape
    K = packed_t.shape[0]
    dev = dy.get_device()
    if out is None:
        out = dy.new_empty((M, K))
    elif not _fits(out, _BF16, (M, K), dev):
        _check_like(out, "out", (M, K), _BF16, dy.device)
    with _on_device(dev):
        ws, ws_bytes = _own_workspace(ws, dy, M, N, K, 0, 0)
        _check(load().lowbit_gemm_dx(M, N, K, bits, group_size, dy.data_ptr(), packed_t.data_ptr(), scales.data_ptr(),
                                     _ptr(zeros), out.data_ptr(), ws.data_ptr(), ws_bytes, _raw_stream(dev)),
               "lowbit_gemm_dx")
    return out


def adapter_backward(dy: torch.Tensor, x: Union[torch.Tensor, Checkpoint], p: torch.Tensor, packed_t: torch.Tensor,
                     scales: torch.Tensor, zeros: Optional[torch.Tensor], bits: int, group_size: int,
                     a: torch.Tensor, b: torch.Tensor, scaling: torch.Tensor, index: Optional[torch.Tensor] = None,
                     dx: Optional[torch.Tensor] = None, da: Optional[torch.Tensor] = None,
                     db: Optional[torch.Tensor] = None, need_dx: bool = True, ws: Optional[torch.Tensor] = None):
    """Gradients of adapter_gemm: (dx [M][K], da [L][R][K], db [L][N][R]), all bf16.

    x is the forward's input, or the Checkpoint it filled; p what it wrote. need_dx=False skips
    dx (a first layer) and returns None in its place. Called by the user: adapter_gemm records no
    autograd graph, and this call has no gradients of its own."""
    xs = (None, x.codes, x.exps) if isinstance(x, Checkpoint) else (x, None, None)
    r = _calls().adapter_backward(dy, packed_t, scales, zeros, bits, group_size, a, b, scaling, index, *xs, p, dx, da, db,
                                  need_dx, ws)
    if r is not None:
        if type(r) is int:
            raise LowbitError(r, "lowbit_adapter_backward")
        return r
    if not _linear_fits(dy, packed_t, scales, zeros, bits, group_size, True):
        _check_grad_args(dy, packed_t, scales, zeros, bits, group_size)
    M, N = dy.shape
    K = packed_t.shape[0]
    dev = dy.get_device()
    if not _adapters_fit(a, b, scaling, index, M, N, K, dev):
        _check_adapters(a, b, scaling, index, M, N, K, dy.device)
    L, R, _ = a.shape
    if not _fits(p, _BF16, (M, R), dev):
        _check_like(p, "p", (M, R), _BF16, dy.device)
    if isinstance(x, Checkpoint):
        if not _copy_fits(x, M, K, dev):
            _check_checkpoint(x, M, K, dy.device, "x")
        xs = (None, x.codes.data_ptr(), x.exps.data_ptr())
    else:
        if not _fits(x, _BF16, (M, K), dev):
            _check_like(x, "x", (M, K), _BF16, dy.device)
        xs = (x.data_ptr(), None, None)
    for name, t, shape in (("dx", dx, (M, K)), ("da", da, (L, R, K)), ("db", db, (L, N, R))):
        if t is not None and not _fits(t, _BF16, shape, dev):
            _check_like(t, name, shape, _BF16, dy.device)
    if dx is not None and not need_dx:
        raise ValueError("dx: a buffer was passed, but need_dx is False")
    if need_dx and dx is None:
        dx = dy.new_empty((M, K))
    if da is None:
        da = dy.new_empty((L, R, K))
    if db is None:
        db = dy.new_empty((L, N, R))
    ad = Adapters(L, R, a.data_ptr(), b.data_ptr(), scaling.data_ptr(), _ptr(index))
    with _on_device(dev):
        ws, ws_bytes = _own_workspace(ws, dy, M, N, K, L, R)
        _check(load().lowbit_adapter_backward(M, N, K, bits, group_size, dy.data_ptr(), packed_t.data_ptr(),
                                              scales.data_ptr(), _ptr(zeros), ctypes.byref(ad), *xs, p.data_ptr(),
                                              _ptr(dx), da.data_ptr(), db.data_ptr(), ws.data_ptr(), ws_bytes,
                                              _raw_stream(dev)), "lowbit_adapter_backward")
    return dx, da, db


def device_status(clear: bool = True) -> int:
    """The device status word (0 = OK, LOWBIT_ERR_TIMEOUT if a kernel wait gave up)."""
    return int(load().lowbit_device_status(1 if clear else 0))


def last_device_status(stream: Optional[torch.cuda.Stream] = None) -> int:
    """The device status word read (and cleared) in the order of `stream` (default: the current
    stream), waiting for that stream only (see lowbit_last_device_status)."""
    st = stream if stream is not None else torch.cuda.current_stream()
    return int(load().lowbit_last_device_status(st.cuda_stream))


def selftest_bounded_wait(limit_cycles: int = 50_000_000) -> None:
    """Launch the bounded-wait self-test kernel (see lowbit_selftest_bounded_wait)."""
    _check(load().lowbit_selftest_bounded_wait(limit_cycles, _stream()), "lowbit_selftest_bounded_wait")
