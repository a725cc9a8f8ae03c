"""Python binding of libgemm355 (gfx950 HIP kernels behind a C ABI).

Argument marshalling only (through ctypes, the layer calls through
csrc/marshal.c): every step of the product runs in the HIP kernels of
``libgemm355.so``. There is no CPU path and no fallback -- if the library
cannot be loaded, every call raises.

The functions mirror the C entry points declared in ``include/gemm355.h``:

    gemm_bf16_nt(M, N, K, A, B, C, stream=None)
    gemm_bf16_nt_bias_act(M, N, K, A, B, bias, activation, C, stream=None)
    gemm_bf16_nt_ws(M, N, K, A, B, C, workspace, workspace_bytes=None, stream=None)
    gemm_bf16_nt_bias_act_ws(M, N, K, A, B, bias, activation, C, workspace, workspace_bytes=None, stream=None)
    workspace_size(M, N, K)           # bytes the *_ws calls need on the current device
    gemm_bf16_nt_noalloc(M, N, K, A, B, C, stream=None)   # *_ws plan, library's fixed scratch
    gemm_nvfp4_nt(M, N, K, Aq, SFA, Bq, SFB, C, stream=None)
    gemm_nvfp4_nt_bias_act(M, N, K, Aq, SFA, Bq, SFB, bias, activation, C, stream=None)
    gemm_nvfp4_nt_ws(M, N, K, Aq, SFA, Bq, SFB, C, workspace, workspace_bytes=None, stream=None)
    gemm_nvfp4_nt_bias_act_ws(M, N, K, Aq, SFA, Bq, SFB, bias, activation, C, workspace,
                              workspace_bytes=None, stream=None)
    nvfp4_workspace_size(M, N, K)     # bytes the NVFP4 *_ws calls need on the current device
    nvfp4_plan(M, N, K, compute_units)  # (decode_first, workspace_bytes) of those calls
    force_fp4_path(path)              # their path for the process (diagnostic)
    gemm_mxfp4_nt(M, N, K, Aq, SA, Bq, SB, C, stream=None)
    gemm_mxfp4_nt_bias_act(M, N, K, Aq, SA, Bq, SB, bias, activation, C, stream=None)
    gemm_bf16_nt_bias_act_res(M, N, K, A, B, bias, activation, R, Z, C, workspace=None, workspace_bytes=None,
                              stream=None)
    gemm_bf16_nt_bias_act_bwd(M, N, K, A, B, Z, activation, dC, dA, dB, dbias, workspace=None,
                              workspace_bytes=None, stream=None)
    gemm_bf16_nt_gated(M, N, K, A, B, bias, activation, Z, C, workspace=None, workspace_bytes=None, stream=None)
    gemm_bf16_nt_gated_bwd(M, N, K, A, B, Z, activation, dC, dA, dB, dbias, workspace=None,
                           workspace_bytes=None, stream=None)
    newton_schulz(batch, rows, cols, G, O, steps, coefficients, eps, workspace, workspace_bytes=None, stream=None)
    bias_act_res_workspace_size(M, N, K)               # bytes of workspace of the five calls above
    bias_act_bwd_workspace_size(M, N, K, activation)   # on the current device
    gated_workspace_size(M, N, K)
    gated_bwd_workspace_size(M, N, K)
    newton_schulz_workspace_size(batch, rows, cols)
    embedding(tokens, vocab, cols, ids, E, Y, scale=1.0, stream=None)
    embedding_bwd(tokens, vocab, cols, ids, dY, R, dE, scale=1.0, workspace=None, workspace_bytes=None, stream=None)
    embedding_bwd_workspace_size(tokens, vocab, cols)
    layer_norm(rows, cols, X, gamma, beta, Y, mean, rstd, eps=1e-5, stream=None)
    layer_norm_bwd(rows, cols, X, gamma, mean, rstd, dY, R, dX, dgamma, dbeta, workspace=None, workspace_bytes=None,
                   stream=None)
    layer_norm_bwd_workspace_size(rows, cols)
    gemm_bf16_nt_cross_entropy(M, V, K, A, B, targets, loss, lse, workspace, workspace_bytes=None, stream=None)
    gemm_bf16_nt_cross_entropy_bwd(M, V, K, A, B, targets, lse, dloss, dA, dB, workspace, workspace_bytes=None,
                                   stream=None)
    cross_entropy_workspace_size(M, V, K)
    cross_entropy_bwd_workspace_size(M, V, K)
    force_layer_kernel(kernel)        # kernel of these calls' products (diagnostic)
    force_instance(instance)          # BF16 instance override (diagnostic)
    force_supergroup(width)           # band width of the tile order (diagnostic)
    supergroup(tiles_n, K, kernel)    # the default band width of a kernel's visiting order
    force_schedule(mode)              # static or dynamic tile order of the NVFP4 kernel (diagnostic)
    bf16_plan(M, N, K, compute_units, with_workspace=False)  # (instance, splits) a BF16 call would run
    bf16_plan_workspace_bytes(M, N, K, compute_units)  # workspace bytes of the *_ws plan

Operands may be torch tensors on a ROCm device (their storage is checked
against the sizes before the call, since the C side cannot see it) or raw
device addresses as ints (unchecked). The layer calls (gemm_bf16_nt_bias_act_res
and those after it) also refuse tensors of another floating type than they
compute with; integer tensors are taken as the values' bits. ``stream`` is a ``torch.cuda.Stream``,
a raw hipStream_t as int, or None for torch's current stream.
"""
from __future__ import annotations

import ctypes
import os
import re

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB_PATH = os.path.join(HERE, "libgemm355.so")
HEADER = os.path.join(ROOT, "include", "gemm355.h")

OK = 0
ERR_INVALID_ARG = 1
ERR_UNSUPPORTED = 2
ERR_NO_DEVICE = 3
ERR_LAUNCH = 4

ACT_NONE = 0         # fused epilogue activations (gemm_bf16_nt_bias_act)
ACT_RELU = 1
ACT_GELU_TANH = 2
ACT_SILU = 3         # the layer calls only (gemm_bf16_nt_bias_act_res and those after it)

BF16 = 0             # types of newton_schulz's input and of the row calls' arrays
FP32 = 1
INT32 = 0            # types of ids and targets
INT64 = 1

INSTANCE_AUTO = 0    # gemm_bf16_nt picks the instance by shape
INSTANCE_LARGE = 1   # 256 x 256 output tiles
INSTANCE_SMALL = 2   # 64 x 64 output tiles
KERNEL_BF16 = 0     # kernels of the supergroup rule (gemm355_supergroup)
KERNEL_NVFP4 = 1
KERNEL_MXFP4 = 2
KERNEL_BF16_SMALL = 3
FP4_PATH_AUTO = 0    # gemm_nvfp4_nt_ws: decode first by shape (gemm355_force_fp4_path)
FP4_PATH_STAGING = 1  # always the kernel that decodes while staging
FP4_PATH_DECODE_FIRST = 2  # always decode into the workspace, then the BF16 product
LAYER_AUTO = 0       # the layer calls' products: by size (gemm355_force_layer_kernel)
LAYER_LARGE = 1      # 256 x 256 output tiles
LAYER_SPLIT = 2      # the same, K of the last round's tiles split
LAYER_TILE = 3       # 128 x 128 output tiles
LAYER_SMALL = 4      # 64 x 64 output tiles
LAYER_NARROW = 5     # 32 x 32 and, for few tokens, narrower ones
SCHEDULE_STATIC = 0  # the NVFP4 kernel's tile order (gemm355_force_schedule)
SCHEDULE_DYNAMIC = 1
INSTANCE_SPLITK = 3  # 128 x 128 output tiles; with a workspace (the *_ws calls) K split over workgroups

_lib = None


class Gemm355Error(RuntimeError):
    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__("%s: %s (status %d)" % (what, status_string(status), status))


def load() -> ctypes.CDLL:
    """Load libgemm355.so, building it first if (and only if) none is built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        from . import build as _build
        _build.build()
    try:
        lib = ctypes.CDLL(LIB_PATH)
    except OSError as e:  # no silent fallback: the HIP library is the product
        raise RuntimeError("libgemm355.so could not be loaded from %s: %s" % (LIB_PATH, e)) from e
    p, i = ctypes.c_void_p, ctypes.c_int
    lib.gemm_bf16_nt.argtypes = [i, i, i, p, p, p, p]
    lib.gemm_bf16_nt.restype = i
    lib.gemm_bf16_nt_bias_act.argtypes = [i, i, i, p, p, p, i, p, p]
    lib.gemm_bf16_nt_bias_act.restype = i
    sz = ctypes.c_size_t
    lib.gemm_bf16_nt_ws.argtypes = [i, i, i, p, p, p, p, sz, p]
    lib.gemm_bf16_nt_ws.restype = i
    lib.gemm_bf16_nt_bias_act_ws.argtypes = [i, i, i, p, p, p, i, p, p, sz, p]
    lib.gemm_bf16_nt_bias_act_ws.restype = i
    lib.gemm_bf16_nt_noalloc.argtypes = [i, i, i, p, p, p, p]
    lib.gemm_bf16_nt_noalloc.restype = i
    lib.gemm_bf16_nt_workspace_size.argtypes = [i, i, i, ctypes.POINTER(sz)]
    lib.gemm_bf16_nt_workspace_size.restype = i
    lib.gemm_nvfp4_nt.argtypes = [i, i, i, p, p, p, p, p, p]
    lib.gemm_nvfp4_nt.restype = i
    lib.gemm_nvfp4_nt_bias_act.argtypes = [i, i, i, p, p, p, p, p, i, p, p]
    lib.gemm_nvfp4_nt_bias_act.restype = i
    lib.gemm_nvfp4_nt_ws.argtypes = [i, i, i, p, p, p, p, p, p, sz, p]
    lib.gemm_nvfp4_nt_ws.restype = i
    lib.gemm_nvfp4_nt_bias_act_ws.argtypes = [i, i, i, p, p, p, p, p, i, p, p, sz, p]
    lib.gemm_nvfp4_nt_bias_act_ws.restype = i
    lib.gemm_nvfp4_nt_workspace_size.argtypes = [i, i, i, ctypes.POINTER(sz)]
    lib.gemm_nvfp4_nt_workspace_size.restype = i
    lib.gemm355_nvfp4_plan.argtypes = [i, i, i, i, p, p]
    lib.gemm355_nvfp4_plan.restype = i
    lib.gemm355_force_fp4_path.argtypes = [i]
    lib.gemm355_force_fp4_path.restype = i
    lib.gemm_mxfp4_nt.argtypes = [i, i, i, p, p, p, p, p, p]
    lib.gemm_mxfp4_nt.restype = i
    lib.gemm_mxfp4_nt_bias_act.argtypes = [i, i, i, p, p, p, p, p, i, p, p]
    lib.gemm_mxfp4_nt_bias_act.restype = i
    f, psz = ctypes.c_float, ctypes.POINTER(sz)
    lib.gemm_bf16_nt_bias_act_res.argtypes = [i, i, i, p, p, p, i, p, p, p, p, sz, p]
    lib.gemm_bf16_nt_bias_act_res.restype = i
    lib.gemm_bf16_nt_bias_act_res_workspace_size.argtypes = [i, i, i, psz]
    lib.gemm_bf16_nt_bias_act_res_workspace_size.restype = i
    lib.gemm_bf16_nt_bias_act_bwd.argtypes = [i, i, i, p, p, p, i, p, p, p, p, p, sz, p]
    lib.gemm_bf16_nt_bias_act_bwd.restype = i
    lib.gemm_bf16_nt_bias_act_bwd_workspace_size.argtypes = [i, i, i, i, psz]
    lib.gemm_bf16_nt_bias_act_bwd_workspace_size.restype = i
    lib.gemm_bf16_nt_gated.argtypes = [i, i, i, p, p, p, i, p, p, p, sz, p]
    lib.gemm_bf16_nt_gated.restype = i
    lib.gemm_bf16_nt_gated_workspace_size.argtypes = [i, i, i, psz]
    lib.gemm_bf16_nt_gated_workspace_size.restype = i
    lib.gemm_bf16_nt_gated_bwd.argtypes = [i, i, i, p, p, p, i, p, p, p, p, p, sz, p]
    lib.gemm_bf16_nt_gated_bwd.restype = i
    lib.gemm_bf16_nt_gated_bwd_workspace_size.argtypes = [i, i, i, psz]
    lib.gemm_bf16_nt_gated_bwd_workspace_size.restype = i
    lib.gemm355_newton_schulz.argtypes = [i, i, i, i, p, i, f, f, f, f, p, p, sz, p]
    lib.gemm355_newton_schulz.restype = i
    lib.gemm355_newton_schulz_workspace_size.argtypes = [i, i, i, psz]
    lib.gemm355_newton_schulz_workspace_size.restype = i
    lib.gemm355_embedding.argtypes = [i, i, i, i, p, i, p, f, i, p, p]
    lib.gemm355_embedding.restype = i
    lib.gemm355_embedding_bwd.argtypes = [i, i, i, i, p, i, p, f, i, p, p, p, sz, p]
    lib.gemm355_embedding_bwd.restype = i
    lib.gemm355_embedding_bwd_workspace_size.argtypes = [i, i, i, psz]
    lib.gemm355_embedding_bwd_workspace_size.restype = i
    lib.gemm355_layer_norm.argtypes = [i, i, i, p, i, p, p, f, p, p, p, p]
    lib.gemm355_layer_norm.restype = i
    lib.gemm355_layer_norm_bwd.argtypes = [i, i, i, p, i, p, p, p, p, p, p, p, p, p, sz, p]
    lib.gemm355_layer_norm_bwd.restype = i
    lib.gemm355_layer_norm_bwd_workspace_size.argtypes = [i, i, psz]
    lib.gemm355_layer_norm_bwd_workspace_size.restype = i
    lib.gemm_bf16_nt_cross_entropy.argtypes = [i, i, i, p, p, i, p, p, p, p, sz, p]
    lib.gemm_bf16_nt_cross_entropy.restype = i
    lib.gemm_bf16_nt_cross_entropy_workspace_size.argtypes = [i, i, i, psz]
    lib.gemm_bf16_nt_cross_entropy_workspace_size.restype = i
    lib.gemm_bf16_nt_cross_entropy_bwd.argtypes = [i, i, i, p, p, i, p, p, p, p, p, p, sz, p]
    lib.gemm_bf16_nt_cross_entropy_bwd.restype = i
    lib.gemm_bf16_nt_cross_entropy_bwd_workspace_size.argtypes = [i, i, i, psz]
    lib.gemm_bf16_nt_cross_entropy_bwd_workspace_size.restype = i
    lib.gemm355_force_layer_kernel.argtypes = [i]
    lib.gemm355_force_layer_kernel.restype = i
    lib.gemm355_status_string.argtypes = [i]
    lib.gemm355_status_string.restype = ctypes.c_char_p
    lib.gemm355_tile_order.argtypes = [i, i, i, p, p]
    lib.gemm355_tile_order.restype = i
    lib.gemm355_schedule.argtypes = [i, i, p, i]
    lib.gemm355_schedule.restype = i
    lib.gemm355_force_instance.argtypes = [i]
    lib.gemm355_force_instance.restype = i
    lib.gemm355_force_schedule.argtypes = [i]
    lib.gemm355_force_schedule.restype = i
    lib.gemm355_supergroup.argtypes = [i, i, i]
    lib.gemm355_supergroup.restype = i
    lib.gemm355_force_supergroup.argtypes = [i]
    lib.gemm355_force_supergroup.restype = i
    lib.gemm355_bf16_plan.argtypes = [i, i, i, i, i, p, p, p]
    lib.gemm355_bf16_plan.restype = i
    _lib = lib
    return lib


def declared_functions() -> list:
    """Names of the functions declared in include/gemm355.h."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return re.findall(r"^\s*(?:const\s+)?\w+\s*\*?\s*(\w+)\s*\(", text, flags=re.M)


def status_string(status: int) -> str:
    return load().gemm355_status_string(int(status)).decode()


# ---- marshalling -----------------------------------------------------------

_torch = None   # imported with the first tensor or stream
_tensor = _raw_stream = _current_device = None


def _import_torch():
    global _torch, _tensor, _raw_stream, _current_device
    import torch
    # the address of a device's current stream without building a Stream object
    # (3 us a call, as long as the rest of a small product's call)
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
        (lambda device: torch.cuda.current_stream(device).cuda_stream)
    _current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    _torch, _tensor = torch, torch.Tensor
    return torch


def _addr(x, need_bytes: int, what: str, device=None):
    """Device address of a tensor (checked) or a raw int address (unchecked).
    With `device`, the tensor has to be on that one."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    torch = _torch or _import_torch()
    if not isinstance(x, torch.Tensor):
        raise TypeError("%s: expected a torch tensor or an int address, got %r" % (what, type(x)))
    if not x.is_cuda:
        raise ValueError("%s must be on the GPU, got device %s" % (what, x.device))
    if device is not None and x.get_device() != device:
        raise ValueError("%s is on device %d, the current device is %d" % (what, x.get_device(), device))
    if not x.is_contiguous():
        raise ValueError("%s must be contiguous" % what)
    if x.nbytes < need_bytes:
        raise ValueError("%s holds %d bytes, the sizes need %d" % (what, x.nbytes, need_bytes))
    return x.data_ptr()


def _typed_addr(x, need_bytes: int, what: str, device=None, dtype=None):
    """_addr of an array of BF16 (or `dtype`) values: a tensor of another
    floating type is refused, one of integers holds the values' bits."""
    if x is not None and not isinstance(x, int):
        torch = _torch or _import_torch()
        dtype = dtype or torch.bfloat16
        if isinstance(x, torch.Tensor) and x.dtype != dtype and (x.dtype.is_floating_point or x.dtype.is_complex):
            raise TypeError("%s: expected %s values, got %s" % (what, dtype, x.dtype))
    return _addr(x, need_bytes, what, device)


def _stream(stream, device=None):
    if stream is None:
        torch = _torch or _import_torch()
        return _raw_stream(torch.cuda.current_device() if device is None else device)
    if isinstance(stream, int):
        return stream
    if device is not None and stream.device_index != device:
        raise ValueError("the stream is on device %d, the current device is %d" % (stream.device_index, device))
    return stream.cuda_stream


def _device() -> int:
    """The current device, which runs the layer calls."""
    if _torch is None:
        _import_torch()
    return _current_device()


def _check(status: int, what: str):
    if status != OK:
        raise Gemm355Error(status, what)


# ---- entry points ------------------------------------------------------------

def gemm_bf16_nt(M: int, N: int, K: int, A, B, C, stream=None) -> None:
    """C (M x N, BF16) = A (M x K, BF16) @ B (N x K, BF16)^T, FP32 sums."""
    lib = load()
    M, N, K = int(M), int(N), int(K)
    nz = M > 0 and N > 0
    a = _addr(A, M * K * 2 if nz else 0, "A")
    b = _addr(B, N * K * 2 if nz else 0, "B")
    c = _addr(C, M * N * 2 if nz else 0, "C")
    _check(lib.gemm_bf16_nt(M, N, K, a, b, c, _stream(stream)), "gemm_bf16_nt")


def gemm_bf16_nt_bias_act(M: int, N: int, K: int, A, B, bias, activation: int, C, stream=None) -> None:
    """C = act(A @ B^T + bias), bias (N BF16 values, or None) and activation
    (ACT_NONE, ACT_RELU, ACT_GELU_TANH) applied in the kernels' epilogue."""
    lib = load()
    M, N, K = int(M), int(N), int(K)
    nz = M > 0 and N > 0
    a = _addr(A, M * K * 2 if nz else 0, "A")
    b = _addr(B, N * K * 2 if nz else 0, "B")
    bb = _addr(bias, N * 2 if nz else 0, "bias")
    c = _addr(C, M * N * 2 if nz else 0, "C")
    _check(lib.gemm_bf16_nt_bias_act(M, N, K, a, b, bb, int(activation), c, _stream(stream)),
           "gemm_bf16_nt_bias_act")


def _unsigned(nbytes) -> int:
    """A workspace's size for a C size_t (ctypes would make -1 the largest)."""
    if int(nbytes) < 0:
        raise ValueError("workspace_bytes is negative: %d" % int(nbytes))
    return int(nbytes)


def _workspace(ws, nbytes, device=None):
    """(address, bytes) of a workspace tensor, int address or None."""
    if ws is None:
        return None, 0 if nbytes is None else int(nbytes)
    if isinstance(ws, int):
        if nbytes is None:
            raise ValueError("workspace_bytes is needed with a raw workspace address")
        return ws, _unsigned(nbytes)
    have = ws.nbytes
    nb = have if nbytes is None else _unsigned(nbytes)
    if nb > have:
        raise ValueError("workspace holds %d bytes, workspace_bytes says %d" % (have, nb))
    return _addr(ws, nb, "workspace", device), nb


def gemm_bf16_nt_ws(M: int, N: int, K: int, A, B, C, workspace, workspace_bytes=None, stream=None) -> None:
    """gemm_bf16_nt with a caller-owned workspace (a device tensor of at least
    workspace_size(M, N, K) bytes, or None when that is 0), which lets the
    128 x 128 instance split K."""
    lib = load()
    M, N, K = int(M), int(N), int(K)
    nz = M > 0 and N > 0
    a = _addr(A, M * K * 2 if nz else 0, "A")
    b = _addr(B, N * K * 2 if nz else 0, "B")
    c = _addr(C, M * N * 2 if nz else 0, "C")
    w, nb = _workspace(workspace, workspace_bytes)
    _check(lib.gemm_bf16_nt_ws(M, N, K, a, b, c, w, nb, _stream(stream)), "gemm_bf16_nt_ws")


def gemm_bf16_nt_bias_act_ws(M: int, N: int, K: int, A, B, bias, activation: int, C, workspace,
                             workspace_bytes=None, stream=None) -> None:
    """gemm_bf16_nt_bias_act with a caller-owned workspace (see gemm_bf16_nt_ws)."""
    lib = load()
    M, N, K = int(M), int(N), int(K)
    nz = M > 0 and N > 0
    a = _addr(A, M * K * 2 if nz else 0, "A")
    b = _addr(B, N * K * 2 if nz else 0, "B")
    bb = _addr(bias, N * 2 if nz else 0, "bias")
    c = _addr(C, M * N * 2 if nz else 0, "C")
    w, nb = _workspace(workspace, workspace_bytes)
    _check(lib.gemm_bf16_nt_bias_act_ws(M, N, K, a, b, bb, int(activation), c, w, nb, _stream(stream)),
           "gemm_bf16_nt_bias_act_ws")


def gemm_bf16_nt_noalloc(M: int, N: int, K: int, A, B, C, stream=None) -> None:
    """gemm_bf16_nt_ws's product with the library's fixed scratch array as
    the workspace: allocates nothing (for graph capture and the like); calls
    overlapping on one GPU race on the scratch."""
    lib = load()
    M, N, K = int(M), int(N), int(K)
    nz = M > 0 and N > 0
    a = _addr(A, M * K * 2 if nz else 0, "A")
    b = _addr(B, N * K * 2 if nz else 0, "B")
    c = _addr(C, M * N * 2 if nz else 0, "C")
    _check(lib.gemm_bf16_nt_noalloc(M, N, K, a, b, c, _stream(stream)), "gemm_bf16_nt_noalloc")


def workspace_size(M: int, N: int, K: int) -> int:
    """Bytes of workspace gemm_bf16_nt_ws / gemm_bf16_nt_bias_act_ws need for
    this shape on the current device (0: no split, no workspace)."""
    out = ctypes.c_size_t(0)
    _check(load().gemm_bf16_nt_workspace_size(int(M), int(N), int(K), ctypes.byref(out)),
           "gemm_bf16_nt_workspace_size")
    return out.value


def gemm_nvfp4_nt(M: int, N: int, K: int, Aq, SFA, Bq, SFB, C, stream=None) -> None:
    """C (M x N, BF16) = dec(Aq, SFA) @ dec(Bq, SFB)^T for E2M1 codes + E4M3 scales."""
    lib = load()
    M, N, K = int(M), int(N), int(K)
    nz = M > 0 and N > 0
    aq = _addr(Aq, M * K // 2 if nz else 0, "Aq")
    sfa = _addr(SFA, M * K // 16 if nz else 0, "SFA")
    bq = _addr(Bq, N * K // 2 if nz else 0, "Bq")
    sfb = _addr(SFB, N * K // 16 if nz else 0, "SFB")
    c = _addr(C, M * N * 2 if nz else 0, "C")
    _check(lib.gemm_nvfp4_nt(M, N, K, aq, sfa, bq, sfb, c, _stream(stream)), "gemm_nvfp4_nt")


def gemm_nvfp4_nt_ws(M: int, N: int, K: int, Aq, SFA, Bq, SFB, C, workspace, workspace_bytes=None,
                     stream=None) -> None:
    """gemm_nvfp4_nt with a caller-owned workspace (a device tensor of at least
    nvfp4_workspace_size(M, N, K) bytes, or None when that is 0): large
    products decode each operand once into BF16 there and run the BF16 core."""
    lib = load()
    M, N, K = int(M), int(N), int(K)
    nz = M > 0 and N > 0
    aq = _addr(Aq, M * K // 2 if nz else 0, "Aq")
    sfa = _addr(SFA, M * K // 16 if nz else 0, "SFA")
    bq = _addr(Bq, N * K // 2 if nz else 0, "Bq")
    sfb = _addr(SFB, N * K // 16 if nz else 0, "SFB")
    c = _addr(C, M * N * 2 if nz else 0, "C")
    w, nb = _workspace(workspace, workspace_bytes)
    _check(lib.gemm_nvfp4_nt_ws(M, N, K, aq, sfa, bq, sfb, c, w, nb, _stream(stream)), "gemm_nvfp4_nt_ws")


def nvfp4_workspace_size(M: int, N: int, K: int) -> int:
    """Workspace bytes gemm_nvfp4_nt_ws uses for this shape on the current device."""
    out = ctypes.c_size_t(0)
    _check(load().gemm_nvfp4_nt_workspace_size(int(M), int(N), int(K), ctypes.byref(out)),
           "gemm_nvfp4_nt_workspace_size")
    return out.value


def nvfp4_plan(M: int, N: int, K: int, compute_units: int):
    """(decode_first, workspace_bytes) of gemm_nvfp4_nt_ws on a device with
    `compute_units` compute units; host only."""
    d = ctypes.c_int(0)
    nb = ctypes.c_size_t(0)
    _check(load().gemm355_nvfp4_plan(int(M), int(N), int(K), int(compute_units), ctypes.byref(d), ctypes.byref(nb)),
           "gemm355_nvfp4_plan")
    return bool(d.value), nb.value


def force_fp4_path(path: int) -> None:
    """gemm_nvfp4_nt_ws's path for the whole process: FP4_PATH_AUTO (default),
    FP4_PATH_STAGING or FP4_PATH_DECODE_FIRST (a diagnostic)."""
    _check(load().gemm355_force_fp4_path(int(path)), "gemm355_force_fp4_path")


def gemm_nvfp4_nt_bias_act(M: int, N: int, K: int, Aq, SFA, Bq, SFB, bias, activation: int, C,
                           stream=None) -> None:
    """C = act(dec(Aq, SFA) @ dec(Bq, SFB)^T + bias) with the fused epilogue."""
    lib = load()
    M, N, K = int(M), int(N), int(K)
    nz = M > 0 and N > 0
    aq = _addr(Aq, M * K // 2 if nz else 0, "Aq")
    sfa = _addr(SFA, M * K // 16 if nz else 0, "SFA")
    bq = _addr(Bq, N * K // 2 if nz else 0, "Bq")
    sfb = _addr(SFB, N * K // 16 if nz else 0, "SFB")
    bb = _addr(bias, N * 2 if nz else 0, "bias")
    c = _addr(C, M * N * 2 if nz else 0, "C")
    _check(lib.gemm_nvfp4_nt_bias_act(M, N, K, aq, sfa, bq, sfb, bb, int(activation), c, _stream(stream)),
           "gemm_nvfp4_nt_bias_act")


def gemm_nvfp4_nt_bias_act_ws(M: int, N: int, K: int, Aq, SFA, Bq, SFB, bias, activation: int, C, workspace,
                              workspace_bytes=None, stream=None) -> None:
    """gemm_nvfp4_nt_bias_act with a caller-owned workspace, sized and used as
    for gemm_nvfp4_nt_ws."""
    lib = load()
    M, N, K = int(M), int(N), int(K)
    nz = M > 0 and N > 0
    aq = _addr(Aq, M * K // 2 if nz else 0, "Aq")
    sfa = _addr(SFA, M * K // 16 if nz else 0, "SFA")
    bq = _addr(Bq, N * K // 2 if nz else 0, "Bq")
    sfb = _addr(SFB, N * K // 16 if nz else 0, "SFB")
    bb = _addr(bias, N * 2 if nz else 0, "bias")
    c = _addr(C, M * N * 2 if nz else 0, "C")
    w, nb = _workspace(workspace, workspace_bytes)
    _check(lib.gemm_nvfp4_nt_bias_act_ws(M, N, K, aq, sfa, bq, sfb, bb, int(activation), c, w, nb, _stream(stream)),
           "gemm_nvfp4_nt_bias_act_ws")


def gemm_mxfp4_nt(M: int, N: int, K: int, Aq, SA, Bq, SB, C, stream=None) -> None:
    """C (M x N, BF16) = dec(Aq, SA) @ dec(Bq, SB)^T for E2M1 codes with one
    E8M0 scale per 32 elements (microscaled FP4)."""
    lib = load()
    M, N, K = int(M), int(N), int(K)
    nz = M > 0 and N > 0
    aq = _addr(Aq, M * K // 2 if nz else 0, "Aq")
    sa = _addr(SA, M * K // 32 if nz else 0, "SA")
    bq = _addr(Bq, N * K // 2 if nz else 0, "Bq")
    sb = _addr(SB, N * K // 32 if nz else 0, "SB")
    c = _addr(C, M * N * 2 if nz else 0, "C")
    _check(lib.gemm_mxfp4_nt(M, N, K, aq, sa, bq, sb, c, _stream(stream)), "gemm_mxfp4_nt")


def gemm_mxfp4_nt_bias_act(M: int, N: int, K: int, Aq, SA, Bq, SB, bias, activation: int, C, stream=None) -> None:
    """C = act(dec(Aq, SA) @ dec(Bq, SB)^T + bias), microscaled FP4 with the
    fused epilogue."""
    lib = load()
    M, N, K = int(M), int(N), int(K)
    nz = M > 0 and N > 0
    aq = _addr(Aq, M * K // 2 if nz else 0, "Aq")
    sa = _addr(SA, M * K // 32 if nz else 0, "SA")
    bq = _addr(Bq, N * K // 2 if nz else 0, "Bq")
    sb = _addr(SB, N * K // 32 if nz else 0, "SB")
    bb = _addr(bias, N * 2 if nz else 0, "bias")
    c = _addr(C, M * N * 2 if nz else 0, "C")
    _check(lib.gemm_mxfp4_nt_bias_act(M, N, K, aq, sa, bq, sb, bb, int(activation), c, _stream(stream)),
           "gemm_mxfp4_nt_bias_act")


# ---- layers ------------------------------------------------------------------

_bound = None   # csrc/marshal.c: checks the arguments and makes the call


def _layers():
    """The compiled marshalling of the layer calls, bound to the library."""
    global _bound
    if _bound is None:
        lib = load()
        if _torch is None:
            _import_torch()
        from . import build as _build
        if not os.path.exists(_build.MARSHAL_PATH):
            _build.build_marshal()
        from . import _marshal as m
        m.bind(_tensor, _current_device, _raw_stream, _typed_addr, _workspace, _stream, _torch.bfloat16, _torch.int16,
               *[ctypes.cast(getattr(lib, fn), ctypes.c_void_p).value for fn in (
                   "gemm_bf16_nt_bias_act_res", "gemm_bf16_nt_gated", "gemm_bf16_nt_bias_act_bwd",
                   "gemm_bf16_nt_gated_bwd")])
        m.bind_ends(_torch.nn.Parameter, _torch.float32, _torch.int32, _torch.int64,
                    *[ctypes.cast(getattr(lib, fn), ctypes.c_void_p).value for fn in (
                        "gemm355_embedding", "gemm355_embedding_bwd", "gemm355_layer_norm", "gemm355_layer_norm_bwd",
                        "gemm_bf16_nt_cross_entropy", "gemm_bf16_nt_cross_entropy_bwd")])
        _bound = m
    return _bound


def _int32(v) -> int:
    """A number for a C int (ctypes would cut it to its low 32 bits)."""
    v = int(v)
    if not -(1 << 31) <= v < 1 << 31:
        raise OverflowError("size beyond 32 bits")
    return v


def _size_of(fn, *args) -> int:
    out = ctypes.c_size_t(0)
    _check(getattr(load(), fn)(*map(_int32, args), ctypes.byref(out)), fn)
    return out.value


def gemm_bf16_nt_bias_act_res(M: int, N: int, K: int, A, B, bias, activation: int, R, Z, C, workspace=None,
                              workspace_bytes=None, stream=None) -> None:
    """C = act(A @ B^T + bias) + R, and Z = A @ B^T + bias where Z is given.

    bias (N), R (M x N, may be C itself) and Z (M x N, an output) may be None;
    activation: ACT_NONE, ACT_RELU, ACT_GELU_TANH or ACT_SILU. The workspace
    holds bias_act_res_workspace_size(M, N, K) bytes (None when that is 0)."""
    status = (_bound or _layers()).forward(0, M, N, K, A, B, bias, activation, R, Z, C, workspace, workspace_bytes,
                                             stream)
    if status:
        raise Gemm355Error(status, "gemm_bf16_nt_bias_act_res")


def bias_act_res_workspace_size(M: int, N: int, K: int) -> int:
    """Workspace bytes of gemm_bf16_nt_bias_act_res on the current device."""
    return _size_of("gemm_bf16_nt_bias_act_res_workspace_size", M, N, K)


def gemm_bf16_nt_bias_act_bwd(M: int, N: int, K: int, A, B, Z, activation: int, dC, dA, dB, dbias, workspace=None,
                              workspace_bytes=None, stream=None) -> None:
    """Gradients of act(A @ B^T + bias): dA (M x K), dB (N x K), dbias (N) from
    dC (M x N) and the forward call's Z (None with ACT_NONE). Each output may
    be None if it is not wanted (the residual's gradient is dC itself). The
    workspace holds bias_act_bwd_workspace_size(M, N, K, activation) bytes."""
    status = (_bound or _layers()).backward(0, M, N, K, A, B, Z, activation, dC, dA, dB, dbias, workspace,
                                              workspace_bytes, stream)
    if status:
        raise Gemm355Error(status, "gemm_bf16_nt_bias_act_bwd")


def bias_act_bwd_workspace_size(M: int, N: int, K: int, activation: int) -> int:
    """Workspace bytes of gemm_bf16_nt_bias_act_bwd on the current device."""
    return _size_of("gemm_bf16_nt_bias_act_bwd_workspace_size", M, N, K, activation)


def gemm_bf16_nt_gated(M: int, N: int, K: int, A, B, bias, activation: int, Z, C, workspace=None,
                       workspace_bytes=None, stream=None) -> None:
    """C = act(Z[:, :N]) * Z[:, N:] with Z = A @ B^T + bias, M x 2N: B (2N x K)
    holds the gate rows, then the up rows. bias (2N) and Z (an output) may be
    None; activations and workspace (gated_workspace_size(M, N, K) bytes) as
    for gemm_bf16_nt_bias_act_res."""
    status = (_bound or _layers()).forward(1, M, N, K, A, B, bias, activation, None, Z, C, workspace,
                                             workspace_bytes, stream)
    if status:
        raise Gemm355Error(status, "gemm_bf16_nt_gated")


def gated_workspace_size(M: int, N: int, K: int) -> int:
    """Workspace bytes of gemm_bf16_nt_gated on the current device."""
    return _size_of("gemm_bf16_nt_gated_workspace_size", M, N, K)


def gemm_bf16_nt_gated_bwd(M: int, N: int, K: int, A, B, Z, activation: int, dC, dA, dB, dbias, workspace=None,
                           workspace_bytes=None, stream=None) -> None:
    """Gradients of the gated layer: dA (M x K), dB (2N x K), dbias (2N) from
    dC (M x N) and the forward call's Z (M x 2N); otherwise as for
    gemm_bf16_nt_bias_act_bwd (gated_bwd_workspace_size(M, N, K) bytes)."""
    status = (_bound or _layers()).backward(1, M, N, K, A, B, Z, activation, dC, dA, dB, dbias, workspace,
                                              workspace_bytes, stream)
    if status:
        raise Gemm355Error(status, "gemm_bf16_nt_gated_bwd")


def gated_bwd_workspace_size(M: int, N: int, K: int) -> int:
    """Workspace bytes of gemm_bf16_nt_gated_bwd on the current device."""
    return _size_of("gemm_bf16_nt_gated_bwd_workspace_size", M, N, K)


def newton_schulz(batch: int, rows: int, cols: int, G, O, steps: int = 5, coefficients=(3.4445, -4.7750, 2.0315),
                  eps: float = 1e-7, workspace=None, workspace_bytes=None, stream=None, g_type=None) -> None:
    """O (BF16) = the batch's matrices G (rows x cols, BF16 or FP32) after
    division by their Frobenius norm + eps and `steps` Newton-Schulz steps
    X <- a X + (b X X^T + c (X X^T)^2) X with coefficients (a, b, c). G's type
    is its tensor's (g_type, BF16 or FP32, names it for a raw address). The
    workspace holds newton_schulz_workspace_size(batch, rows, cols) bytes."""
    batch, rows, cols, steps = _int32(batch), _int32(rows), _int32(cols), _int32(steps)
    if g_type is None:
        import torch
        types = {torch.bfloat16: BF16, torch.int16: BF16, torch.uint16: BF16, torch.float32: FP32}
        if not isinstance(G, torch.Tensor) or G.dtype not in types:
            raise TypeError("G: expected a BF16 or FP32 tensor, or an address with g_type")
        g_type = types[G.dtype]
    g_type = _int32(g_type)
    dev = _device()
    n = batch * rows * cols if min(batch, rows, cols) > 0 else 0
    fp32 = g_type == FP32
    gg = _typed_addr(G, n * (4 if fp32 else 2), "G", dev, _torch.float32 if fp32 else None)
    o = _typed_addr(O, n * 2, "O", dev)
    w, nb = _workspace(workspace, workspace_bytes, dev)
    a, b, c = coefficients
    _check(load().gemm355_newton_schulz(batch, rows, cols, g_type, gg, steps, a, b, c, eps, o, w, nb,
                                        _stream(stream, dev)), "gemm355_newton_schulz")


def newton_schulz_workspace_size(batch: int, rows: int, cols: int) -> int:
    """Workspace bytes of newton_schulz on the current device."""
    return _size_of("gemm355_newton_schulz_workspace_size", batch, rows, cols)


# ---- the ends of a network ---------------------------------------------------

def _is_tensor(x) -> bool:
    return x is not None and not isinstance(x, int) and isinstance(x, (_torch or _import_torch()).Tensor)


def _type_of(given, what: str, *arrays) -> int:
    """BF16 or FP32: `given`, or the type of the first tensor among `arrays`
    (integers of 16 bits hold BF16 values' bits); BF16 if there is none to tell."""
    if given is not None:
        given = _int32(given)
        if given not in (BF16, FP32):
            raise ValueError("%s: expected BF16 or FP32, got %d" % (what, given))
        return given
    for x in arrays:
        if _is_tensor(x):
            t = _torch
            kind = {t.float32: FP32, t.bfloat16: BF16, t.int16: BF16, t.uint16: BF16}.get(x.dtype)
            if kind is None:
                raise TypeError("%s: expected bfloat16 or float32 values, got %s" % (what, x.dtype))
            return kind
    if any(x is not None for x in arrays):
        raise ValueError("%s: its type has to be given with a raw address" % what)
    return BF16


def _values(x, kind: int, count: int, what: str, device):
    """Address of `count` values of a type that _type_of has given."""
    t = _torch or _import_torch()
    if kind == FP32:
        return _floats(x, count, what, device)
    if _is_tensor(x) and x.dtype not in (t.bfloat16, t.int16, t.uint16):
        raise TypeError("%s: expected torch.bfloat16 values, got %s" % (what, x.dtype))
    return _addr(x, 2 * count, what, device)


def _floats(x, count: int, what: str, device):
    """Address of `count` FP32 values."""
    if _is_tensor(x) and x.dtype != _torch.float32:
        raise TypeError("%s: expected torch.float32 values, got %s" % (what, x.dtype))
    return _addr(x, 4 * count, what, device)


def _ids(x, given, count: int, what: str, device):
    """(address, type) of `count` ids."""
    if _is_tensor(x):
        kind = {_torch.int32: INT32, _torch.int64: INT64}.get(x.dtype)
        if kind is None:
            raise TypeError("%s: expected int32 or int64 values, got %s" % (what, x.dtype))
    elif given is None and x is not None:
        raise ValueError("%s: its type has to be given with a raw address" % what)
    else:
        kind = _int32(given or 0)
    return _addr(x, count * (8 if kind == INT64 else 4), what, device), kind


def _count(*sizes) -> int:
    """Elements of an array of these sizes (none where the call refuses them)."""
    n = 1
    for s in sizes:
        n *= max(0, s)
    return n


def embedding(tokens: int, vocab: int, cols: int, ids, E, Y, scale: float = 1.0, stream=None, id_type=None,
              e_type=None, y_type=None) -> None:
    """Y[t] = scale * E[ids[t]] (tokens x cols), zeros where ids[t] lies outside
    0 .. vocab - 1.

    E (vocab x cols) and Y are BF16 or FP32 each, ids (tokens) int32 or int64;
    id_type (INT32, INT64), e_type and y_type (BF16, FP32) name the types of raw
    addresses."""
    if id_type is None and e_type is None and y_type is None:
        status = (_bound or _layers()).embedding(tokens, vocab, cols, ids, E, Y, scale, stream)
        if status is not None:      # (None: something that the long way knows about)
            if status:
                raise Gemm355Error(status, "gemm355_embedding")
            return
    tokens, vocab, cols = _int32(tokens), _int32(vocab), _int32(cols)
    dev = _device()
    i, it = _ids(ids, id_type, _count(tokens), "ids", dev)
    et, yt = _type_of(e_type, "E", E), _type_of(y_type, "Y", Y)
    e = _values(E, et, _count(vocab, cols), "E", dev)
    y = _values(Y, yt, _count(tokens, cols), "Y", dev)
    _check(load().gemm355_embedding(tokens, vocab, cols, it, i, et, e, scale, yt, y, _stream(stream, dev)),
           "gemm355_embedding")


def embedding_bwd(tokens: int, vocab: int, cols: int, ids, dY, R, dE, scale: float = 1.0, workspace=None,
                  workspace_bytes=None, stream=None, id_type=None, y_type=None, e_type=None) -> None:
    """dE[v] = R[v] + scale * the sum of dY[t] over the tokens with ids[t] = v.

    dY (tokens x cols) and dE (vocab x cols) are BF16 or FP32 each; R, of dE's
    type, may be None for zeros, or dE itself: only rows that occur are then read
    and written. The workspace holds embedding_bwd_workspace_size(tokens, vocab,
    cols) bytes."""
    if id_type is None and y_type is None and e_type is None:
        status = (_bound or _layers()).embedding_bwd(tokens, vocab, cols, ids, dY, R, dE, scale, workspace, workspace_bytes,
                                                     stream)
        if status is not None:      # (None: something that the long way knows about)
            if status:
                raise Gemm355Error(status, "gemm355_embedding_bwd")
            return
    tokens, vocab, cols = _int32(tokens), _int32(vocab), _int32(cols)
    dev = _device()
    i, it = _ids(ids, id_type, _count(tokens), "ids", dev)
    yt, et = _type_of(y_type, "dY", dY), _type_of(e_type, "dE", dE)
    y = _values(dY, yt, _count(tokens, cols), "dY", dev)
    r = _values(R, et, _count(vocab, cols), "R", dev)
    e = _values(dE, et, _count(vocab, cols), "dE", dev)
    w, nb = _workspace(workspace, workspace_bytes, dev)
    _check(load().gemm355_embedding_bwd(tokens, vocab, cols, it, i, yt, y, scale, et, r, e, w, nb, _stream(stream, dev)),
           "gemm355_embedding_bwd")


def embedding_bwd_workspace_size(tokens: int, vocab: int, cols: int) -> int:
    """Workspace bytes of embedding_bwd on the current device."""
    return _size_of("gemm355_embedding_bwd_workspace_size", tokens, vocab, cols)


def layer_norm(rows: int, cols: int, X, gamma, beta, Y, mean, rstd, eps: float = 1e-5, stream=None, x_type=None,
               w_type=None) -> None:
    """Y (BF16) = (X - mean) * rstd * gamma + beta with each row's mean and
    rstd = 1 / sqrt(variance + eps).

    X (rows x cols) is BF16 or FP32, gamma and beta (cols, or None) likewise;
    mean and rstd (rows, FP32) are outputs for layer_norm_bwd, or None."""
    if x_type is None and w_type is None:
        status = (_bound or _layers()).layer_norm(rows, cols, X, gamma, beta, Y, mean, rstd, eps, stream)
        if status is not None:      # (None: something that the long way knows about)
            if status:
                raise Gemm355Error(status, "gemm355_layer_norm")
            return
    rows, cols = _int32(rows), _int32(cols)
    dev = _device()
    xt, wt = _type_of(x_type, "X", X), _type_of(w_type, "gamma", gamma, beta)
    x = _values(X, xt, _count(rows, cols), "X", dev)
    ga = _values(gamma, wt, _count(cols), "gamma", dev)
    be = _values(beta, wt, _count(cols), "beta", dev)
    y = _values(Y, BF16, _count(rows, cols), "Y", dev)
    m, s = _floats(mean, _count(rows), "mean", dev), _floats(rstd, _count(rows), "rstd", dev)
    _check(load().gemm355_layer_norm(rows, cols, xt, x, wt, ga, be, eps, y, m, s, _stream(stream, dev)),
           "gemm355_layer_norm")


def layer_norm_bwd(rows: int, cols: int, X, gamma, mean, rstd, dY, R, dX, dgamma, dbeta, workspace=None,
                   workspace_bytes=None, stream=None, x_type=None, w_type=None) -> None:
    """Gradients of layer_norm: dX (of X's type) from dY (rows x cols, BF16) and
    the forward call's mean and rstd, plus R (of X's type, None for zeros; may be
    dX itself), and dgamma and dbeta (of gamma's type). Each output may be None if
    it is not wanted. The workspace holds layer_norm_bwd_workspace_size(rows, cols)
    bytes (None where that is 0)."""
    if x_type is None and w_type is None:
        status = (_bound or _layers()).layer_norm_bwd(rows, cols, X, gamma, mean, rstd, dY, R, dX, dgamma, dbeta, workspace,
                                                      workspace_bytes, stream)
        if status is not None:      # (None: something that the long way knows about)
            if status:
                raise Gemm355Error(status, "gemm355_layer_norm_bwd")
            return
    rows, cols = _int32(rows), _int32(cols)
    dev = _device()
    xt, wt = _type_of(x_type, "X", X, dX), _type_of(w_type, "gamma", gamma, dgamma, dbeta)
    n, c = _count(rows, cols), _count(cols)
    x = _values(X, xt, n, "X", dev)
    ga = _values(gamma, wt, c, "gamma", dev)
    m, s = _floats(mean, _count(rows), "mean", dev), _floats(rstd, _count(rows), "rstd", dev)
    dy = _values(dY, BF16, n, "dY", dev)
    r, dx = _values(R, xt, n, "R", dev), _values(dX, xt, n, "dX", dev)
    dg, db = _values(dgamma, wt, c, "dgamma", dev), _values(dbeta, wt, c, "dbeta", dev)
    w, nb = _workspace(workspace, workspace_bytes, dev)
    _check(load().gemm355_layer_norm_bwd(rows, cols, xt, x, wt, ga, m, s, dy, r, dx, dg, db, w, nb, _stream(stream, dev)),
           "gemm355_layer_norm_bwd")


def layer_norm_bwd_workspace_size(rows: int, cols: int) -> int:
    """Workspace bytes of layer_norm_bwd on the current device."""
    return _size_of("gemm355_layer_norm_bwd_workspace_size", rows, cols)


def gemm_bf16_nt_cross_entropy(M: int, V: int, K: int, A, B, targets, loss, lse, workspace=None, workspace_bytes=None,
                               stream=None, target_type=None) -> None:
    """loss[m] = lse[m] - z[m][targets[m]] and lse[m] = log sum exp z[m] of the
    logits z = A @ B^T, which are not kept.

    A (M x K) and B (V x K) are BF16, targets (M) int32 or int64 (target_type,
    INT32 or INT64, names the type of a raw address), loss and lse (M) FP32
    outputs. A row whose target lies outside 0 .. V - 1 is left out: zeros. The
    workspace holds cross_entropy_workspace_size(M, V, K) bytes."""
    if target_type is None:
        status = (_bound or _layers()).entropy(M, V, K, A, B, targets, loss, lse, workspace, workspace_bytes, stream)
        if status is not None:      # (None: something that the long way knows about)
            if status:
                raise Gemm355Error(status, "gemm_bf16_nt_cross_entropy")
            return
    M, V, K = _int32(M), _int32(V), _int32(K)
    dev = _device()
    a, b = _values(A, BF16, _count(M, K), "A", dev), _values(B, BF16, _count(V, K), "B", dev)
    t, tt = _ids(targets, target_type, _count(M), "targets", dev)
    lo, ls = _floats(loss, _count(M), "loss", dev), _floats(lse, _count(M), "lse", dev)
    w, nb = _workspace(workspace, workspace_bytes, dev)
    _check(load().gemm_bf16_nt_cross_entropy(M, V, K, a, b, tt, t, lo, ls, w, nb, _stream(stream, dev)),
           "gemm_bf16_nt_cross_entropy")


def cross_entropy_workspace_size(M: int, V: int, K: int) -> int:
    """Workspace bytes of gemm_bf16_nt_cross_entropy on the current device."""
    return _size_of("gemm_bf16_nt_cross_entropy_workspace_size", M, V, K)


def gemm_bf16_nt_cross_entropy_bwd(M: int, V: int, K: int, A, B, targets, lse, dloss, dA, dB, workspace=None,
                                   workspace_bytes=None, stream=None, target_type=None) -> None:
    """Gradients of gemm_bf16_nt_cross_entropy: dA (M x K) and dB (V x K), BF16,
    each None if it is not wanted, from the forward call's lse and dloss (M, FP32;
    None for ones), the gradient of each row's loss. Rows that are left out get
    zeros in dA and add nothing to dB. The workspace holds
    cross_entropy_bwd_workspace_size(M, V, K) bytes."""
    if target_type is None:
        status = (_bound or _layers()).entropy_bwd(M, V, K, A, B, targets, lse, dloss, dA, dB, workspace, workspace_bytes,
                                                   stream)
        if status is not None:      # (None: something that the long way knows about)
            if status:
                raise Gemm355Error(status, "gemm_bf16_nt_cross_entropy_bwd")
            return
    M, V, K = _int32(M), _int32(V), _int32(K)
    dev = _device()
    a, b = _values(A, BF16, _count(M, K), "A", dev), _values(B, BF16, _count(V, K), "B", dev)
    t, tt = _ids(targets, target_type, _count(M), "targets", dev)
    ls, dl = _floats(lse, _count(M), "lse", dev), _floats(dloss, _count(M), "dloss", dev)
    da, db = _values(dA, BF16, _count(M, K), "dA", dev), _values(dB, BF16, _count(V, K), "dB", dev)
    w, nb = _workspace(workspace, workspace_bytes, dev)
    _check(load().gemm_bf16_nt_cross_entropy_bwd(M, V, K, a, b, tt, t, ls, dl, da, db, w, nb, _stream(stream, dev)),
           "gemm_bf16_nt_cross_entropy_bwd")


def cross_entropy_bwd_workspace_size(M: int, V: int, K: int) -> int:
    """Workspace bytes of gemm_bf16_nt_cross_entropy_bwd on the current device."""
    return _size_of("gemm_bf16_nt_cross_entropy_bwd_workspace_size", M, V, K)


def force_layer_kernel(kernel: int) -> None:
    """Kernel of the layer calls' products for the whole process: LAYER_AUTO
    (default), LAYER_LARGE, LAYER_SPLIT, LAYER_TILE, LAYER_SMALL or
    LAYER_NARROW (a diagnostic)."""
    _check(load().gemm355_force_layer_kernel(_int32(kernel)), "gemm355_force_layer_kernel")


def force_instance(instance: int) -> None:
    """Force gemm_bf16_nt's kernel instance for the whole process
    (INSTANCE_AUTO, INSTANCE_LARGE, INSTANCE_SMALL or INSTANCE_SPLITK)."""
    _check(load().gemm355_force_instance(instance), "gemm355_force_instance")


def force_supergroup(width: int) -> None:
    """Force the band width of the persistent kernels' supergroup tile order
    for the whole process (0 = the default)."""
    _check(load().gemm355_force_supergroup(width), "gemm355_force_supergroup")


def _plan(M, N, K, compute_units, with_workspace):
    inst = ctypes.c_int(0)
    splits = ctypes.c_int(0)
    nbytes = ctypes.c_size_t(0)
    _check(load().gemm355_bf16_plan(M, N, K, compute_units, int(bool(with_workspace)), ctypes.byref(inst),
                                    ctypes.byref(splits), ctypes.byref(nbytes)), "gemm355_bf16_plan")
    return inst.value, splits.value, nbytes.value


def force_schedule(mode: int) -> None:
    """Tile order of the NVFP4 kernel for the whole process: SCHEDULE_STATIC
    (default) or SCHEDULE_DYNAMIC (a measurement option)."""
    _check(load().gemm355_force_schedule(mode), "gemm355_force_schedule")


def supergroup(tiles_n: int, K: int, kernel: int = 0) -> int:
    """Default band width of the visiting order (kernel: KERNEL_BF16,
    KERNEL_NVFP4, KERNEL_MXFP4 or KERNEL_BF16_SMALL); host only."""
    r = load().gemm355_supergroup(int(kernel), int(tiles_n), int(K))
    if r < 0:
        raise Gemm355Error(-r, "gemm355_supergroup")
    return r


def bf16_plan(M: int, N: int, K: int, compute_units: int, with_workspace: bool = False):
    """(instance, splits) that gemm_bf16_nt (or, with_workspace, gemm_bf16_nt_ws)
    runs for this shape on a device with `compute_units` compute units; host only."""
    return _plan(M, N, K, compute_units, with_workspace)[:2]


def bf16_plan_workspace_bytes(M: int, N: int, K: int, compute_units: int) -> int:
    """Workspace bytes of gemm_bf16_nt_ws's plan on such a device; host only."""
    return _plan(M, N, K, compute_units, True)[2]


def tile_order(tiles_m: int, tiles_n: int, supergroup: int):
    """Visiting order of output tiles as two lists (tm, tn); host only."""
    lib = load()
    n = tiles_m * tiles_n
    tm = (ctypes.c_int * max(n, 1))()
    tn = (ctypes.c_int * max(n, 1))()
    _check(lib.gemm355_tile_order(tiles_m, tiles_n, supergroup, tm, tn), "gemm355_tile_order")
    return list(tm[:n]), list(tn[:n])


def schedule(tiles: int, grid: int):
    """slot[w][r] = visiting-order position of workgroup w in round r (-1: none)."""
    lib = load()
    rounds = -(-tiles // grid) if tiles > 0 and grid > 0 else 1
    buf = (ctypes.c_int * max(rounds * max(grid, 1), 1))()
    r = lib.gemm355_schedule(tiles, grid, buf, len(buf))
    if r < 0:
        raise Gemm355Error(-r, "gemm355_schedule")
    return [list(buf[w * r:(w + 1) * r]) for w in range(grid)]
