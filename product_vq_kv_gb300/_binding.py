"""ctypes binding of ``libvqenc.so``: argument marshalling only.

Every function here has the name of the C entry point it calls (declared in
``include/vq_encode.h``) and does nothing but check and convert its arguments,
allocate the output tensor when asked to (on the stream of the call), and pass the
current CUDA stream or the given one.
All computation happens in the library's CUDA kernels; there is no other code
path.  If the library has not been built the first call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading

import torch

from .build import LIB_PATH

VQ_OK, VQ_ERR_INVALID_ARG, VQ_ERR_UNSUPPORTED, VQ_ERR_CUDA, VQ_ERR_INTERNAL = range(5)
VQ_F16, VQ_BF16, VQ_F32 = 0, 1, 2

_TORCH_DTYPES = {torch.float16: VQ_F16, torch.bfloat16: VQ_BF16, torch.float32: VQ_F32}

_lock = threading.Lock()
_lib = None


class VQError(RuntimeError):
    """A non-OK status returned by the library."""

    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {vq_status_string(status)}")


class VqSlice(ctypes.Structure):
    """``vq_slice``: rows [row, row + n_rows) of groups [group, group + n_groups)."""
    _fields_ = [("group", ctypes.c_int64), ("n_groups", ctypes.c_int64),
                ("row", ctypes.c_int64), ("n_rows", ctypes.c_int64)]


class VqPagePool(ctypes.Structure):
    """``vq_page_pool``: pages of one pool, possibly of several layers."""
    _fields_ = [("base", ctypes.c_void_p), ("page_stride", ctypes.c_int64), ("page_bytes", ctypes.c_int64),
                ("layer_stride", ctypes.c_int64), ("layers", ctypes.c_int32)]


# Pools of one vq_paged_copy (VQ_PAGED_MAX_POOLS).
PAGED_MAX_POOLS = 8


def _configure(lib: ctypes.CDLL) -> ctypes.CDLL:
    """Declare the argument and result types of every entry point on ``lib``
    (the library, or its bounds-checked build, which has the same ABI)."""
    i64, i32, vp = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p
    lib.vq_encode.restype = i32
    lib.vq_encode.argtypes = [vp, vp, i64, i32, i32, i32, vp, vp]
    lib.vq_encode_grouped.restype = i32
    lib.vq_encode_grouped.argtypes = [vp, vp, i64, i64, i32, i32, i32, vp, vp]
    lib.vq_encode_grouped_host.restype = i32
    lib.vq_encode_grouped_host.argtypes = [vp, vp, i64, i64, i32, i32, i32, vp, vp, vp,
                                           vp, vp]
    lib.vq_encode_grouped_u8.restype = i32
    lib.vq_encode_grouped_u8.argtypes = [vp, vp, i64, i64, i32, i32, i32, vp, vp]
    lib.vq_dequantize_grouped.restype = i32
    lib.vq_dequantize_grouped.argtypes = [vp, i32, vp, i64, i64, i32, i32, i32, vp, vp]
    lib.vq_attention_decode.restype = i32
    lib.vq_attention_decode.argtypes = [vp, vp, vp, vp, vp, i64, i32, i32, i64, i32, i32, i32,
                                        i64, ctypes.c_float, i32, vp, vp, ctypes.c_size_t, vp]
    lib.vq_attention_decode_static.restype = i32
    lib.vq_attention_decode_static.argtypes = [vp, vp, vp, vp, vp, i64, i32, i32, i64, i32,
                                               i32, i32, i64, ctypes.c_float, i32, vp, vp]
    lib.vq_encode_grouped_smooth.restype = i32
    lib.vq_encode_grouped_smooth.argtypes = [vp, vp, vp, i64, i64, i32, i32, i32, i32, vp,
                                             i32, vp]
    lib.vq_scalar_quantize_workspace_bytes.restype = ctypes.c_size_t
    lib.vq_scalar_quantize_workspace_bytes.argtypes = [i32]
    lib.vq_scalar_quantize.restype = i32
    lib.vq_scalar_quantize.argtypes = [vp, i32, i64, vp, i32, vp, vp, ctypes.c_size_t, vp]
    lib.vq_scalar_dequantize.restype = i32
    lib.vq_scalar_dequantize.argtypes = [vp, i64, vp, i32, i32, vp, vp]
    lib.vq_hadamard_rotate.restype = i32
    lib.vq_hadamard_rotate.argtypes = [vp, i32, vp, i64, i32, vp, vp]
    lib.vq_hadamard_quantize.restype = i32
    lib.vq_hadamard_quantize.argtypes = [vp, i32, vp, i64, i32, vp, i32, vp, vp]
    lib.vq_attention_workspace_bytes.restype = ctypes.c_size_t
    lib.vq_attention_workspace_bytes.argtypes = [i64, i32, i32, i64, i32, i32, i32, i64]
    lib.vq_paged_reserve.restype = i32
    lib.vq_paged_reserve.argtypes = [vp, vp, i64, vp, vp, i64, vp, i64, i32, i64, vp, vp, vp, vp,
                                     vp]
    lib.vq_paged_trim.restype = i32
    lib.vq_paged_trim.argtypes = [vp, vp, i64, vp, i64, i32, vp, vp, i64, vp, vp, vp]
    lib.vq_paged_append.restype = i32
    lib.vq_paged_append.argtypes = [vp, vp, i64, i64, vp, i64, i32, i32, i32, i32, vp, vp, vp, vp,
                                    vp, i64, i32, i64, i32, vp]
    lib.vq_paged_attention.restype = i32
    lib.vq_paged_attention.argtypes = [vp, i64, vp, vp, i64, i64, i64, vp, i64, vp, vp, i64, i32,
                                       i64, vp, vp, i32, i32, i32, i32, i32, i64, ctypes.c_float,
                                       i32, vp, vp, vp, ctypes.c_size_t, vp]
    lib.vq_paged_attention_slots.restype = i32
    lib.vq_paged_attention_slots.argtypes = lib.vq_paged_attention.argtypes[:4] + [vp] + lib.vq_paged_attention.argtypes[4:]
    lib.vq_paged_attention_workspace_bytes.restype = ctypes.c_size_t
    lib.vq_paged_attention_workspace_bytes.argtypes = [i64, i64, i64, i32, i32, i32, i32, i32, i32]
    lib.vq_paged_scalar_append.restype = i32
    lib.vq_paged_scalar_append.argtypes = [vp, vp, i64, i64, vp, i64, i32, i32, i32, vp, vp, vp, vp, vp,
                                           vp, vp, i64, i32, i64, i64, i32, vp]
    lib.vq_paged_scalar_attention.restype = i32
    lib.vq_paged_scalar_attention.argtypes = [vp, i64, vp, vp, vp, i64, i64, i64, vp, i64, vp, vp, vp, vp,
                                              i64, i32, i64, i64, vp, vp, i32, i32, i32, i32, i64,
                                              ctypes.c_float, i32, vp, vp, vp, ctypes.c_size_t, vp]
    lib.vq_paged_scalar_attention_workspace_bytes.restype = ctypes.c_size_t
    lib.vq_paged_scalar_attention_workspace_bytes.argtypes = [i64, i64, i64, i32, i32, i32, i32]
    lib.vq_paged_fork_workspace_bytes.restype = ctypes.c_size_t
    lib.vq_paged_fork_workspace_bytes.argtypes = [i64]
    lib.vq_paged_fork.restype = i32
    lib.vq_paged_fork.argtypes = [vp, vp, vp, i64, vp, i64, i32, vp, vp, i64, vp, vp, vp, vp, vp,
                                  ctypes.c_size_t, vp]
    lib.vq_paged_compact.restype = i32
    lib.vq_paged_compact.argtypes = [vp, i64, vp, i64, i32, vp, vp, i64, vp, vp, vp, vp, vp, vp,
                                     ctypes.c_size_t, vp]
    lib.vq_paged_compact_workspace_bytes.restype = ctypes.c_size_t
    lib.vq_paged_compact_workspace_bytes.argtypes = [i64]
    lib.vq_paged_copy.restype = i32
    lib.vq_paged_copy.argtypes = [vp, i64, vp, i32, i64, vp]
    lib.vq_status_string.restype = ctypes.c_char_p
    lib.vq_status_string.argtypes = [i32]
    lib.vq_describe_launch.restype = i32
    lib.vq_describe_launch.argtypes = [i64, i64, i32, i32, i32, vp, ctypes.c_char_p, i32]
    lib.vq_abi_version.restype = i32
    lib.vq_abi_version.argtypes = []
    lib.vq_kernel_status.restype = i32
    lib.vq_kernel_status.argtypes = [ctypes.POINTER(ctypes.c_uint32), i32]
    lib.vq_partition.restype = i32
    lib.vq_partition.argtypes = [i64, i64, i32, i32, ctypes.POINTER(VqSlice),
                                 ctypes.POINTER(ctypes.c_int32)]
    return lib


def load_library() -> ctypes.CDLL:
    """Load ``libvqenc.so`` (once).  Raises if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing; build it with `python -m product_vq_kv_gb300.build` "
                "(there is no fallback implementation)")
        _lib = _configure(ctypes.CDLL(LIB_PATH))
        return _lib


def vq_status_string(status: int) -> str:
    return load_library().vq_status_string(int(status)).decode()


def vq_abi_version() -> int:
    return int(load_library().vq_abi_version())


# Bits of the device status word (vq_kernel_status).
VQ_KSTATUS_WAIT_GAVE_UP = 0x1
VQ_KSTATUS_OUT_OF_BOUNDS = 0x2


def vq_kernel_status(clear: bool = True, device=None) -> int:
    """The status bits the library's kernels set on ``device`` (default: the
    current device) since the last clear, after waiting for that device to
    finish; 0 means every kernel finished normally.  Clears them if
    ``clear``."""
    bits = ctypes.c_uint32(0)
    with torch.cuda.device(device if device is not None else torch.cuda.current_device()):
        st = load_library().vq_kernel_status(ctypes.byref(bits), 1 if clear else 0)
    _check(st, "vq_kernel_status")
    return int(bits.value)


def _dtype_code(t: torch.Tensor) -> int:
    try:
        return _TORCH_DTYPES[t.dtype]
    except KeyError:
        raise TypeError(f"unsupported dtype {t.dtype}; expected float16, bfloat16 or float32")


def _stream_handle(stream, device) -> int:
    if stream is None:
        stream = torch.cuda.current_stream(device)
    return int(stream.cuda_stream)


# The current stream's handle by device index: what torch.cuda.current_stream
# wraps, without building the wrapper (2 us of a call of 10).
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _launch(fn, where: str, device, stream, *args) -> None:
    """``fn(*args, stream handle)`` with ``device`` current."""
    if stream is not None:
        handle = int(stream.cuda_stream)
    elif _raw_stream is not None:
        handle = _raw_stream(device.index)
    else:
        handle = int(torch.cuda.current_stream(device).cuda_stream)
    if torch.cuda.current_device() == device.index:
        status = fn(*args, handle)
    else:
        with torch.cuda.device(device):
            status = fn(*args, handle)
    if status != VQ_OK:
        raise VQError(status, where)


def _check(status: int, where: str) -> None:
    if status != VQ_OK:
        raise VQError(status, where)


def _device_tensor(t: torch.Tensor, name: str) -> None:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _empty(shape, dtype, device, stream) -> torch.Tensor:
    """A new tensor for work on ``stream`` (None: the current stream).

    torch hands the memory of a freed tensor out again in the order of the stream
    that the tensor was made on.  One made on the current stream for work on another
    could lie where the current stream still reads, and be handed out again while
    the other still writes: so it is made on ``stream`` itself."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def vq_encode(x: torch.Tensor, codebook: torch.Tensor, out: torch.Tensor | None = None,
              stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Indices of the nearest centroid for each row of ``x``.

    ``x`` ``[N, sub_dim]`` and ``codebook`` ``[n_centroids, sub_dim]`` are
    contiguous CUDA tensors of one dtype (float16, bfloat16 or float32).
    Returns (or fills ``out``) a ``[N]`` uint32 tensor.  Asynchronous on
    ``stream`` (default: the current stream).
    """
    _device_tensor(x, "x")
    _device_tensor(codebook, "codebook")
    if x.dim() != 2 or codebook.dim() != 2 or x.shape[1] != codebook.shape[1]:
        raise ValueError(f"expected x [N, sub_dim] and codebook [n_centroids, sub_dim], got "
                         f"{tuple(x.shape)} and {tuple(codebook.shape)}")
    if x.dtype != codebook.dtype:
        raise TypeError("x and codebook must share a dtype")
    if out is None:
        out = _empty(x.shape[0], torch.uint32, x.device, stream)
    elif out.dtype != torch.uint32 or out.shape != (x.shape[0],) or not out.is_contiguous():
        raise ValueError("out must be a contiguous uint32 tensor of shape [N]")
    st = load_library().vq_encode(x.data_ptr(), codebook.data_ptr(), x.shape[0],
                                  codebook.shape[0], x.shape[1], _dtype_code(x),
                                  out.data_ptr(), _stream_handle(stream, x.device))
    _check(st, "vq_encode")
    return out


def vq_encode_grouped(x: torch.Tensor, codebooks: torch.Tensor,
                      out: torch.Tensor | None = None,
                      stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Grouped encode: ``x`` ``[G, M, sub_dim]`` against ``codebooks``
    ``[G, n_centroids, sub_dim]`` (row block g uses codebook g).  Returns (or
    fills ``out``) a ``[G, M]`` uint32 tensor.  Asynchronous on ``stream``."""
    _device_tensor(x, "x")
    _device_tensor(codebooks, "codebooks")
    if (x.dim() != 3 or codebooks.dim() != 3 or x.shape[0] != codebooks.shape[0]
            or x.shape[2] != codebooks.shape[2]):
        raise ValueError(f"expected x [G, M, sub_dim] and codebooks [G, n_centroids, sub_dim], "
                         f"got {tuple(x.shape)} and {tuple(codebooks.shape)}")
    if x.dtype != codebooks.dtype:
        raise TypeError("x and codebooks must share a dtype")
    g, m, sub = x.shape
    if out is None:
        out = _empty((g, m), torch.uint32, x.device, stream)
    elif out.dtype != torch.uint32 or out.shape != (g, m) or not out.is_contiguous():
        raise ValueError("out must be a contiguous uint32 tensor of shape [G, M]")
    st = load_library().vq_encode_grouped(x.data_ptr(), codebooks.data_ptr(), g, m,
                                          codebooks.shape[1], sub, _dtype_code(x),
                                          out.data_ptr(), _stream_handle(stream, x.device))
    _check(st, "vq_encode_grouped")
    return out


def vq_encode_grouped_u8(x: torch.Tensor, codebooks: torch.Tensor,
                         out: torch.Tensor | None = None,
                         stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Grouped encode to 8-bit codes (at most 256 centroids): the indices of
    :func:`vq_encode_grouped` as a ``[G, M]`` uint8 tensor."""
    _device_tensor(x, "x")
    _device_tensor(codebooks, "codebooks")
    if (x.dim() != 3 or codebooks.dim() != 3 or x.shape[0] != codebooks.shape[0]
            or x.shape[2] != codebooks.shape[2]):
        raise ValueError(f"expected x [G, M, sub_dim] and codebooks [G, n_centroids, sub_dim], "
                         f"got {tuple(x.shape)} and {tuple(codebooks.shape)}")
    if x.dtype != codebooks.dtype:
        raise TypeError("x and codebooks must share a dtype")
    g, m, sub = x.shape
    if out is None:
        out = _empty((g, m), torch.uint8, x.device, stream)
    elif out.dtype != torch.uint8 or out.shape != (g, m) or not out.is_contiguous():
        raise ValueError("out must be a contiguous uint8 tensor of shape [G, M]")
    st = load_library().vq_encode_grouped_u8(x.data_ptr(), codebooks.data_ptr(), g, m,
                                             codebooks.shape[1], sub, _dtype_code(x),
                                             out.data_ptr(), _stream_handle(stream, x.device))
    _check(st, "vq_encode_grouped_u8")
    return out


def vq_encode_grouped_smooth(x: torch.Tensor, smooth: torch.Tensor, codebooks: torch.Tensor,
                             head_dim: int, index_bytes: int = 1, out: torch.Tensor | None = None,
                             stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Grouped encode of smoothed keys: every element of ``x`` ``[G, M,
    sub_dim]`` divided by its channel's factor in ``smooth`` ``[G, head_dim]``
    (float32; row ``m`` holds channels ``(m % (head_dim // sub_dim)) * sub_dim
    + i``) before the encode.  Returns ``[G, M]`` uint8 codes
    (``index_bytes=1``) or uint32 indices (``index_bytes=4``)."""
    _device_tensor(x, "x")
    _device_tensor(smooth, "smooth")
    _device_tensor(codebooks, "codebooks")
    if (x.dim() != 3 or codebooks.dim() != 3 or x.shape[0] != codebooks.shape[0]
            or x.shape[2] != codebooks.shape[2]):
        raise ValueError(f"expected x [G, M, sub_dim] and codebooks [G, n_centroids, sub_dim], "
                         f"got {tuple(x.shape)} and {tuple(codebooks.shape)}")
    if x.dtype != codebooks.dtype:
        raise TypeError("x and codebooks must share a dtype")
    if smooth.dtype != torch.float32 or tuple(smooth.shape) != (x.shape[0], head_dim):
        raise ValueError("smooth must be float32 of shape [G, head_dim]")
    if index_bytes not in (1, 4):
        raise ValueError("index_bytes must be 1 or 4")
    g, m, sub = x.shape
    odt = torch.uint8 if index_bytes == 1 else torch.uint32
    if out is None:
        out = _empty((g, m), odt, x.device, stream)
    elif out.dtype != odt or out.shape != (g, m) or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous {odt} tensor of shape [G, M]")
    st = load_library().vq_encode_grouped_smooth(
        x.data_ptr(), smooth.data_ptr(), codebooks.data_ptr(), g, m, codebooks.shape[1], sub,
        head_dim, _dtype_code(x), out.data_ptr(), index_bytes, _stream_handle(stream, x.device))
    _check(st, "vq_encode_grouped_smooth")
    return out


def _f32_vector(t: torch.Tensor, name: str) -> None:
    _device_tensor(t, name)
    if t.dtype != torch.float32 or t.dim() != 1:
        raise ValueError(f"{name} must be a 1-D float32 device tensor")


def vq_scalar_quantize(x: torch.Tensor, centroids: torch.Tensor, out: torch.Tensor | None = None,
                       workspace: torch.Tensor | None = None, use_table: bool = True,
                       stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Scalar (sub_dim = 1) quantize of every element of ``x`` against the
    float32 ``centroids``: uint8 indices of ``x``'s shape.  fp16 input with
    2, 4, 8 or 16 centroids takes the bucket table the kernel builds itself
    (the workspace goes unused); other fp16 / bf16 input takes the table pass
    when a 64 KiB ``workspace`` is given (allocated here when omitted and
    ``use_table``)."""
    _device_tensor(x, "x")
    _f32_vector(centroids, "centroids")
    if out is None:
        out = _empty(x.shape, torch.uint8, x.device, stream)
    elif out.dtype != torch.uint8 or out.shape != x.shape or not out.is_contiguous():
        raise ValueError("out must be a contiguous uint8 tensor of x's shape")
    code = _dtype_code(x)
    lib = load_library()
    need = int(lib.vq_scalar_quantize_workspace_bytes(code))
    if workspace is None and use_table and need:
        workspace = _empty(need, torch.uint8, x.device, stream)
    ws_ptr = workspace.data_ptr() if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib.vq_scalar_quantize(x.data_ptr(), code, x.numel(), centroids.data_ptr(),
                                centroids.numel(), out.data_ptr(), ws_ptr, ws_bytes,
                                _stream_handle(stream, x.device))
    _check(st, "vq_scalar_quantize")
    return out


def vq_scalar_dequantize(idx: torch.Tensor, centroids: torch.Tensor,
                         dtype: torch.dtype = torch.float16, out: torch.Tensor | None = None,
                         stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """``centroids[idx]`` in ``dtype`` (round to nearest); out-of-range
    indices give 0."""
    _device_tensor(idx, "idx")
    _f32_vector(centroids, "centroids")
    if idx.dtype != torch.uint8:
        raise TypeError("idx must be uint8")
    if out is None:
        out = _empty(idx.shape, dtype, idx.device, stream)
    st = load_library().vq_scalar_dequantize(idx.data_ptr(), idx.numel(), centroids.data_ptr(),
                                             centroids.numel(), _dtype_code(out), out.data_ptr(),
                                             _stream_handle(stream, idx.device))
    _check(st, "vq_scalar_dequantize")
    return out


def vq_hadamard_rotate(x: torch.Tensor, diag: torch.Tensor, out: torch.Tensor | None = None,
                       stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Randomised Hadamard rotation of the rows of ``x`` ``[..., D]``:
    float32 of the same shape."""
    _device_tensor(x, "x")
    _f32_vector(diag, "diag")
    dim = x.shape[-1]
    if diag.numel() != dim:
        raise ValueError("diag must have one entry per column")
    if out is None:
        out = _empty(x.shape, torch.float32, x.device, stream)
    st = load_library().vq_hadamard_rotate(x.data_ptr(), _dtype_code(x), diag.data_ptr(),
                                           x.numel() // dim, dim, out.data_ptr(),
                                           _stream_handle(stream, x.device))
    _check(st, "vq_hadamard_rotate")
    return out


def vq_hadamard_quantize(x: torch.Tensor, diag: torch.Tensor, centroids: torch.Tensor,
                         out: torch.Tensor | None = None,
                         stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Rotation fused with the scalar quantize: uint8 indices of ``x``'s
    shape."""
    _device_tensor(x, "x")
    _f32_vector(diag, "diag")
    _f32_vector(centroids, "centroids")
    dim = x.shape[-1]
    if diag.numel() != dim:
        raise ValueError("diag must have one entry per column")
    if out is None:
        out = _empty(x.shape, torch.uint8, x.device, stream)
    st = load_library().vq_hadamard_quantize(x.data_ptr(), _dtype_code(x), diag.data_ptr(),
                                             x.numel() // dim, dim, centroids.data_ptr(),
                                             centroids.numel(), out.data_ptr(),
                                             _stream_handle(stream, x.device))
    _check(st, "vq_hadamard_quantize")
    return out


def vq_dequantize_grouped(idx: torch.Tensor, codebooks: torch.Tensor,
                          out: torch.Tensor | None = None,
                          stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Decode ``idx`` ``[G, M]`` (uint32 or uint8) against ``codebooks``
    ``[G, n_centroids, sub_dim]``: returns (or fills ``out``) the ``[G, M,
    sub_dim]`` tensor of codebook rows, in the codebooks' dtype; out-of-range
    indices give zero rows.  Asynchronous on ``stream``."""
    _device_tensor(idx, "idx")
    _device_tensor(codebooks, "codebooks")
    if idx.dtype not in (torch.uint32, torch.uint8):
        raise TypeError("idx must be uint32 or uint8")
    if idx.dim() != 2 or codebooks.dim() != 3 or idx.shape[0] != codebooks.shape[0]:
        raise ValueError(f"expected idx [G, M] and codebooks [G, n_centroids, sub_dim], got "
                         f"{tuple(idx.shape)} and {tuple(codebooks.shape)}")
    g, m = idx.shape
    n_c, sub = codebooks.shape[1], codebooks.shape[2]
    if out is None:
        out = _empty((g, m, sub), codebooks.dtype, idx.device, stream)
    elif out.dtype != codebooks.dtype or out.shape != (g, m, sub) or not out.is_contiguous():
        raise ValueError("out must be a contiguous tensor of shape [G, M, sub_dim] in the "
                         "codebooks' dtype")
    st = load_library().vq_dequantize_grouped(
        idx.data_ptr(), 4 if idx.dtype == torch.uint32 else 1, codebooks.data_ptr(), g, m, n_c,
        sub, _dtype_code(codebooks), out.data_ptr(), _stream_handle(stream, idx.device))
    _check(st, "vq_dequantize_grouped")
    return out


def vq_attention_workspace_bytes(batch: int, heads_q: int, heads_kv: int, tokens: int,
                                 head_dim: int, sub_dim: int, n_centroids: int,
                                 window: int = 0) -> int:
    return int(load_library().vq_attention_workspace_bytes(batch, heads_q, heads_kv, tokens,
                                                           head_dim, sub_dim, n_centroids,
                                                           window))


def _check_attention_args(q, k_codes, k_codebooks, v_codes, v_codebooks):
    """Validate the tensors of an attention call before any pointer is taken.

    Shapes and dtypes are checked first (so every mismatch is reported the
    same way whatever the device), then that every tensor is a contiguous CUDA
    tensor on q's device.  Returns ``(B, Hq, Hkv, T, D, sub_dim, n_c)``.
    """
    named = (("q", q), ("k_codes", k_codes), ("k_codebooks", k_codebooks),
             ("v_codes", v_codes), ("v_codebooks", v_codebooks))
    for name, t in named:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    if q.dim() != 3 or k_codes.dim() != 4 or k_codebooks.dim() != 3:
        raise ValueError(f"expected q [B, Hq, D], k_codes [B, Hkv, T, D/sub_dim] and "
                         f"k_codebooks [Hkv, n_c, sub_dim], got {tuple(q.shape)}, "
                         f"{tuple(k_codes.shape)} and {tuple(k_codebooks.shape)}")
    _dtype_code(q)
    if k_codes.dtype != torch.uint8 or v_codes.dtype != torch.uint8:
        raise TypeError("codes must be uint8")
    if k_codebooks.dtype != q.dtype or v_codebooks.dtype != q.dtype:
        raise TypeError("codebooks must share q's dtype")
    b, hq, d = q.shape
    _, hkv, tokens, ns = k_codes.shape
    n_c, sub = k_codebooks.shape[1], k_codebooks.shape[2]
    if (tuple(v_codes.shape) != tuple(k_codes.shape) or k_codes.shape[0] != b or ns * sub != d
            or tuple(k_codebooks.shape) != (hkv, n_c, sub)
            or tuple(v_codebooks.shape) != (hkv, n_c, sub)):
        raise ValueError("inconsistent shapes: q [B, Hq, D], codes [B, Hkv, T, D/sub_dim] (keys "
                         "and values alike), codebooks [Hkv, n_c, sub_dim] (keys and values alike)")
    for name, t in named:
        _device_tensor(t, name)
        if t.device != q.device:
            raise ValueError(f"{name} is on {t.device}, q on {q.device}")
    return b, hq, hkv, tokens, d, sub, n_c


def _check_attention_out(out, q, stream):
    if out is None:
        return _empty(q.shape, q.dtype, q.device, stream)
    if (not isinstance(out, torch.Tensor) or out.dtype != q.dtype or out.shape != q.shape
            or out.device != q.device or not out.is_contiguous()):
        raise ValueError("out must be a contiguous tensor of q's shape, dtype and device")
    return out


def vq_attention_decode(q: torch.Tensor, k_codes: torch.Tensor, k_codebooks: torch.Tensor,
                        v_codes: torch.Tensor, v_codebooks: torch.Tensor, window: int = 0,
                        scale: float = 0.0, out: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None,
                        stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Decode attention over 8-bit product-VQ codes.

    ``q`` ``[B, Hq, D]``; ``k_codes`` / ``v_codes`` ``[B, Hkv, T, D/sub_dim]``
    uint8; ``k_codebooks`` / ``v_codebooks`` ``[Hkv, n_c, sub_dim]`` in q's
    dtype.  Returns (or fills ``out``) ``[B, Hq, D]``.  ``workspace`` is a
    device byte tensor for the per-slice partials; if omitted one of
    :func:`vq_attention_workspace_bytes` bytes is allocated here (by torch).
    """
    b, hq, hkv, tokens, d, sub, n_c = _check_attention_args(q, k_codes, k_codebooks, v_codes,
                                                            v_codebooks)
    out = _check_attention_out(out, q, stream)
    if workspace is None:
        nbytes = vq_attention_workspace_bytes(b, hq, hkv, tokens, d, sub, n_c, window)
        workspace = _empty(max(nbytes, 16), torch.uint8, q.device, stream)
    else:
        _device_tensor(workspace, "workspace")
        if workspace.device != q.device:
            raise ValueError(f"workspace is on {workspace.device}, q on {q.device}")
    with torch.cuda.device(q.device):
        st = load_library().vq_attention_decode(
            q.data_ptr(), k_codes.data_ptr(), k_codebooks.data_ptr(), v_codes.data_ptr(),
            v_codebooks.data_ptr(), b, hq, hkv, tokens, d, sub, n_c, window, scale,
            _dtype_code(q), out.data_ptr(), workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), _stream_handle(stream, q.device))
    _check(st, "vq_attention_decode")
    return out


def _i32_tensor(t, name: str, shape: tuple, device) -> None:
    """A contiguous int32 device tensor of ``shape`` (None: any extent) on ``device``."""
    if (isinstance(t, torch.Tensor) and t.dtype is torch.int32 and t.is_cuda and t.is_contiguous()
            and (device is None or t.device == device) and t.shape == shape):
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != torch.int32:
        raise TypeError(f"{name} must be int32")
    if t.dim() != len(shape) or any(want is not None and have != want
                                    for have, want in zip(t.shape, shape)):
        want = "[" + ", ".join("any" if n is None else str(n) for n in shape) + "]"
        raise ValueError(f"{name} must have shape {want}, got {tuple(t.shape)}")
    _device_tensor(t, name)
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")


def _table_tensor(t, requests: int, device) -> int:
    """Check a block table ``[requests, max_blocks]``; returns max_blocks."""
    blocks = t.shape[1] if isinstance(t, torch.Tensor) and t.dim() == 2 else None
    _i32_tensor(t, "block_table", (requests, blocks), device)
    return blocks


def _extent(t) -> int | None:
    """The extent of a 1-D tensor; None if it is none."""
    return t.shape[0] if isinstance(t, torch.Tensor) and t.dim() == 1 else None


def _out_like(out, name, shape, dtype, device, stream):
    if out is None:
        return _empty(shape, dtype, device, stream)
    if (not isinstance(out, torch.Tensor) or out.dtype != dtype or tuple(out.shape) != tuple(shape)
            or out.device != device or not out.is_contiguous()):
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}")
    return out


def vq_paged_reserve(lens: torch.Tensor, new_lens: torch.Tensor, free_pages: torch.Tensor,
                     free_count: torch.Tensor, block_table: torch.Tensor, page_size: int,
                     total_new: int, lens_out: torch.Tensor | None = None,
                     free_count_out: torch.Tensor | None = None,
                     cu_new: torch.Tensor | None = None, slots: torch.Tensor | None = None,
                     stream: torch.cuda.Stream | None = None) -> tuple:
    """Pages and slots for ``new_lens[r]`` more tokens of each request.

    ``lens`` / ``new_lens`` ``[R]``, ``free_pages`` ``[num_pages]`` (a stack of
    ``free_count`` ``[1]`` pages) and ``block_table`` ``[R, max_blocks]`` are
    int32; ``total_new`` is the number of rows of the packed new tokens.  The
    table's entries of new pages are written in place.  Returns ``(lens_out,
    free_count_out, cu_new, slots)``; pass ``lens_out=lens`` and
    ``free_count_out=free_count`` to update those in place.  Refused requests
    (see ``include/vq_encode.h``) keep their length and get slots of -1.  New outputs
    are allocated on ``stream``."""
    r = _extent(lens)
    _i32_tensor(lens, "lens", (r,), None)
    dev, pages = lens.device, _extent(free_pages)
    _i32_tensor(new_lens, "new_lens", (r,), dev)
    _i32_tensor(free_pages, "free_pages", (pages,), dev)
    _i32_tensor(free_count, "free_count", (1,), dev)
    blocks = _table_tensor(block_table, r, dev)
    if total_new < 0:
        raise ValueError("total_new must not be negative")
    lens_out = _out_like(lens_out, "lens_out", (r,), torch.int32, dev, stream)
    free_count_out = _out_like(free_count_out, "free_count_out", (1,), torch.int32, dev, stream)
    cu_new = _out_like(cu_new, "cu_new", (r + 1,), torch.int32, dev, stream)
    slots = _out_like(slots, "slots", (total_new,), torch.int64, dev, stream)
    _launch(load_library().vq_paged_reserve, "vq_paged_reserve", dev, stream, lens.data_ptr(),
            new_lens.data_ptr(), r, free_pages.data_ptr(), free_count.data_ptr(), pages,
            block_table.data_ptr(), blocks, page_size, total_new, lens_out.data_ptr(),
            free_count_out.data_ptr(), cu_new.data_ptr(), slots.data_ptr())
    return lens_out, free_count_out, cu_new, slots


def vq_paged_trim(lens: torch.Tensor, keep_lens: torch.Tensor, block_table: torch.Tensor,
                  page_size: int, free_pages: torch.Tensor, free_count: torch.Tensor,
                  lens_out: torch.Tensor | None = None,
                  free_count_out: torch.Tensor | None = None,
                  stream: torch.cuda.Stream | None = None) -> tuple:
    """Cut each request to ``keep_lens[r]`` tokens and push the pages it no
    longer needs on ``free_pages`` (in place).  Returns ``(lens_out,
    free_count_out)``, which may be ``lens`` and ``free_count`` themselves; new ones are
    allocated on ``stream``."""
    r = _extent(lens)
    _i32_tensor(lens, "lens", (r,), None)
    dev, pages = lens.device, _extent(free_pages)
    _i32_tensor(keep_lens, "keep_lens", (r,), dev)
    blocks = _table_tensor(block_table, r, dev)
    _i32_tensor(free_pages, "free_pages", (pages,), dev)
    _i32_tensor(free_count, "free_count", (1,), dev)
    lens_out = _out_like(lens_out, "lens_out", (r,), torch.int32, dev, stream)
    free_count_out = _out_like(free_count_out, "free_count_out", (1,), torch.int32, dev, stream)
    _launch(load_library().vq_paged_trim, "vq_paged_trim", dev, stream, lens.data_ptr(),
            keep_lens.data_ptr(), r, block_table.data_ptr(), blocks, page_size, free_pages.data_ptr(),
            free_count.data_ptr(), pages, lens_out.data_ptr(), free_count_out.data_ptr())
    return lens_out, free_count_out


def _token_rows(t, name: str, device) -> None:
    """A CUDA tensor [T, H, D] whose tokens may be strided, each contiguous."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 3:
        raise ValueError(f"{name} must have shape [tokens, heads, head_dim], got {tuple(t.shape)}")
    _dtype_code(t)
    (n, h, d), (sn, sh, sd) = t.shape, t.stride()
    if n * h * d and (sd != 1 and d > 1 or sh != d and h > 1 or sn < h * d and n > 1):
        raise ValueError(f"{name} must be contiguous within a token and its tokens must not overlap")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")


def _token_stride(t) -> int:
    n, h, d = t.shape
    return t.stride(0) if n > 1 else h * d


def _page_tensors(k_codes, v_codes, k_codebooks, v_codebooks, dtype, device):
    """Check the pages and codebooks; returns (num_pages, heads, page_size, ns,
    page stride in bytes, n_centroids, sub_dim)."""
    if (isinstance(k_codes, torch.Tensor) and isinstance(v_codes, torch.Tensor)
            and isinstance(k_codebooks, torch.Tensor) and isinstance(v_codebooks, torch.Tensor)
            and k_codes.dim() == 4 and k_codebooks.dim() == 3):
        # the usual case in one test; anything else is told apart below
        shape, strides, books = k_codes.shape, k_codes.stride(), k_codebooks.shape
        pages, heads, page_size, ns = shape
        if (pages > 1 and k_codes.dtype is torch.uint8 and v_codes.dtype is torch.uint8
                and k_codebooks.dtype is dtype and v_codebooks.dtype is dtype and v_codes.shape == shape
                and v_codes.stride() == strides and v_codebooks.shape == books and books[0] == heads
                and strides[1:] == (page_size * ns, ns, 1) and strides[0] >= heads * page_size * ns
                and k_codebooks.is_contiguous() and v_codebooks.is_contiguous()
                and k_codes.device == device and v_codes.device == device
                and k_codebooks.device == device and v_codebooks.device == device):
            return pages, heads, page_size, ns, strides[0], books[1], books[2]
    for name, t in (("k_codes", k_codes), ("v_codes", v_codes), ("k_codebooks", k_codebooks),
                    ("v_codebooks", v_codebooks)):
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    if k_codes.dim() != 4 or k_codebooks.dim() != 3:
        raise ValueError(f"expected codes [pages, heads, page_size, ns] and codebooks [heads, "
                         f"n_centroids, sub_dim], got {tuple(k_codes.shape)} and {tuple(k_codebooks.shape)}")
    if k_codes.dtype != torch.uint8 or v_codes.dtype != torch.uint8:
        raise TypeError("codes must be uint8")
    if k_codebooks.dtype != dtype or v_codebooks.dtype != dtype:
        raise TypeError(f"codebooks must be {dtype}, as the rows are")
    pages, heads, page_size, ns = k_codes.shape
    if tuple(v_codes.shape) != tuple(k_codes.shape):
        raise ValueError("k_codes and v_codes must have one shape")
    if tuple(v_codebooks.shape) != tuple(k_codebooks.shape) or k_codebooks.shape[0] != heads:
        raise ValueError("k_codebooks and v_codebooks must have one shape, [heads, n_centroids, sub_dim]")
    inner = heads * page_size * ns
    strides = []
    for name, t in (("k_codes", k_codes), ("v_codes", v_codes)):
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.numel() and not t[0].is_contiguous():
            raise ValueError(f"each page of {name} must be contiguous")
        strides.append(t.stride(0) if pages > 1 else inner)
    if strides[0] != strides[1] or strides[0] < inner:
        raise ValueError("the pages of k_codes and v_codes must not overlap and must have one stride")
    for name, t in (("k_codebooks", k_codebooks), ("v_codebooks", v_codebooks)):
        _device_tensor(t, name)
    for name, t in (("k_codes", k_codes), ("v_codes", v_codes), ("k_codebooks", k_codebooks),
                    ("v_codebooks", v_codebooks)):
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, not on {device}")
    return pages, heads, page_size, ns, strides[0], k_codebooks.shape[1], k_codebooks.shape[2]


def vq_paged_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor,
                    k_codebooks: torch.Tensor, v_codebooks: torch.Tensor, k_codes: torch.Tensor,
                    v_codes: torch.Tensor, k_smooth: torch.Tensor | None = None,
                    stream: torch.cuda.Stream | None = None) -> None:
    """Encode the keys and values of new tokens into their slots of the pages.

    ``k`` / ``v`` ``[T, H, D]`` (tokens may be strided), ``slots`` ``[T]`` int64
    (-1: skipped), codebooks ``[H, n_centroids, sub_dim]`` in k's dtype,
    ``k_codes`` / ``v_codes`` ``[num_pages, H, page_size, D/sub_dim]`` uint8,
    written in place; ``k_smooth`` ``[H, D]`` float32 divides the keys first."""
    _token_rows(k, "k", None)
    dev = k.device
    _token_rows(v, "v", dev)
    if v.dtype != k.dtype or v.shape != k.shape:
        raise ValueError("k and v must share shape and dtype")
    pages, heads, page_size, ns, stride, n_c, sub = _page_tensors(k_codes, v_codes, k_codebooks,
                                                                  v_codebooks, k.dtype, dev)
    tokens, h, d = k.shape
    if h != heads or ns * sub != d:
        raise ValueError(f"k {tuple(k.shape)} does not match codes {tuple(k_codes.shape)} and "
                         f"codebooks {tuple(k_codebooks.shape)}")
    if not isinstance(slots, torch.Tensor) or slots.dtype != torch.int64 or tuple(slots.shape) != (tokens,):
        raise ValueError("slots must be an int64 tensor of shape [T]")
    _device_tensor(slots, "slots")
    if slots.device != dev:
        raise ValueError(f"slots is on {slots.device}, not on {dev}")
    if k_smooth is not None:
        if not isinstance(k_smooth, torch.Tensor):
            raise TypeError("k_smooth must be a torch.Tensor")
        if k_smooth.dtype != torch.float32 or tuple(k_smooth.shape) != (heads, d):
            raise ValueError("k_smooth must be float32 of shape [H, D]")
        _device_tensor(k_smooth, "k_smooth")
        if k_smooth.device != dev:
            raise ValueError(f"k_smooth is on {k_smooth.device}, not on {dev}")
    _launch(load_library().vq_paged_append, "vq_paged_append", dev, stream, k.data_ptr(), v.data_ptr(),
            _token_stride(k), _token_stride(v), slots.data_ptr(), tokens, heads, d, sub, n_c,
            k_codebooks.data_ptr(), v_codebooks.data_ptr(),
            k_smooth.data_ptr() if k_smooth is not None else None, k_codes.data_ptr(),
            v_codes.data_ptr(), pages, page_size, stride, _dtype_code(k))


def vq_paged_attention_workspace_bytes(requests: int, tokens: int, max_new: int, heads_q: int,
                                       heads_kv: int, head_dim: int, sub_dim: int,
                                       n_centroids: int, page_size: int) -> int:
    return int(load_library().vq_paged_attention_workspace_bytes(
        requests, tokens, max_new, heads_q, heads_kv, head_dim, sub_dim, n_centroids, page_size))


@functools.lru_cache(maxsize=1024)
def _paged_workspace(device_index: int, *sizes) -> int:
    """The workspace of a device for these sizes, as often as a step asks for it."""
    with torch.cuda.device(device_index):
        return max(vq_paged_attention_workspace_bytes(*sizes), 16)


def vq_paged_attention(q: torch.Tensor, cu_new: torch.Tensor, lens: torch.Tensor,
                       block_table: torch.Tensor, k_codes: torch.Tensor, v_codes: torch.Tensor,
                       k_codebooks: torch.Tensor, v_codebooks: torch.Tensor, max_new: int = 0,
                       window: int = 0, scale: float = 0.0, out: torch.Tensor | None = None,
                       lse: torch.Tensor | None = None, return_lse: bool = False,
                       workspace: torch.Tensor | None = None,
                       stream: torch.cuda.Stream | None = None,
                       slots: torch.Tensor | None = None):
    """Causal attention of the new tokens of every request over its pages.

    ``q`` ``[T, Hq, D]`` (tokens may be strided); ``cu_new`` ``[R + 1]``,
    ``lens`` ``[R]`` (with the new tokens) and ``block_table`` ``[R,
    max_blocks]`` int32; pages and codebooks as in :func:`vq_paged_append`,
    codebooks in q's dtype.  ``max_new`` is the most new tokens of a request
    where the host knows it.  Returns ``out`` ``[T, Hq, D]``, or ``(out, lse)``
    with ``lse`` ``[T, Hq]`` float32 where ``return_lse`` is set or ``lse`` is
    given.  ``slots`` (at least ``[T]`` int64, of :func:`vq_paged_reserve`) makes the
    rows of refused requests zeros with an lse of -inf; without it they are taken for
    the last tokens their request has in the cache.  A workspace of :func:`vq_paged_attention_workspace_bytes` bytes is
    allocated here (by torch) if none is given; it and new outputs are allocated on
    ``stream``."""
    _token_rows(q, "q", None)
    dev = q.device
    tokens, hq, d = q.shape
    pages, hkv, page_size, ns, stride, n_c, sub = _page_tensors(k_codes, v_codes, k_codebooks,
                                                                v_codebooks, q.dtype, dev)
    if ns * sub != d or hkv < 1 or hq % hkv:
        raise ValueError(f"q {tuple(q.shape)} does not match codes {tuple(k_codes.shape)} and "
                         f"codebooks {tuple(k_codebooks.shape)}")
    r = _extent(lens)
    _i32_tensor(lens, "lens", (r,), dev)
    _i32_tensor(cu_new, "cu_new", (r + 1,), dev)
    blocks = _table_tensor(block_table, r, dev)
    if max_new < 0:
        raise ValueError("max_new must not be negative")
    if slots is not None:
        if not isinstance(slots, torch.Tensor) or slots.dtype != torch.int64 or slots.dim() != 1 or slots.shape[0] < tokens:
            raise ValueError("slots must be an int64 tensor of at least [T]")
        _device_tensor(slots, "slots")
        if slots.device != dev:
            raise ValueError(f"slots is on {slots.device}, not on {dev}")
    out = _out_like(out, "out", (tokens, hq, d), q.dtype, dev, stream)
    if return_lse or lse is not None:
        lse = _out_like(lse, "lse", (tokens, hq), torch.float32, dev, stream)
    if workspace is None:
        nbytes = _paged_workspace(dev.index, r, tokens, max_new, hq, hkv, d, sub, n_c, page_size)
        workspace = _empty(nbytes, torch.uint8, dev, stream)
    else:
        _device_tensor(workspace, "workspace")
        if workspace.device != dev:
            raise ValueError(f"workspace is on {workspace.device}, not on {dev}")
        nbytes = workspace.numel() * workspace.element_size()
    _launch(load_library().vq_paged_attention_slots, "vq_paged_attention", dev, stream, q.data_ptr(),
            _token_stride(q), cu_new.data_ptr(), lens.data_ptr(),
            slots.data_ptr() if slots is not None else None, r, tokens, max_new,
            block_table.data_ptr(), blocks, k_codes.data_ptr(), v_codes.data_ptr(), pages, page_size,
            stride, k_codebooks.data_ptr(), v_codebooks.data_ptr(), hq, hkv, d, sub, n_c, window, scale,
            _dtype_code(q), out.data_ptr(), lse.data_ptr() if lse is not None else None,
            workspace.data_ptr(), nbytes)
    return (out, lse) if lse is not None else out


def _scalar_page_tensors(k_codes, v_codes, k_scales, v_scales, k_centroids, v_centroids, dtype, device):
    """Check the pages and centroids of the cache in 4 bits; returns (num_pages, heads,
    page_size, dim, page stride in bytes, scale stride in elements, n_centroids)."""
    if (isinstance(k_codes, torch.Tensor) and isinstance(v_codes, torch.Tensor) and isinstance(k_scales, torch.Tensor)
            and isinstance(v_scales, torch.Tensor) and isinstance(k_centroids, torch.Tensor)
            and isinstance(v_centroids, torch.Tensor) and k_codes.dim() == 4 and k_scales.dim() == 3
            and k_centroids.dim() == 1):
        # the usual case in one test; anything else is told apart below
        shape, strides, scale_strides = k_codes.shape, k_codes.stride(), k_scales.stride()
        pages, heads, page_size, ns = shape
        if (pages > 1 and k_codes.dtype is torch.uint8 and v_codes.dtype is torch.uint8 and k_scales.dtype is dtype
                and v_scales.dtype is dtype and k_centroids.dtype is torch.float32 and v_centroids.dtype is torch.float32
                and v_codes.shape == shape and v_codes.stride() == strides and k_scales.shape == shape[:3]
                and v_scales.shape == shape[:3] and v_scales.stride() == scale_strides
                and v_centroids.shape == k_centroids.shape and strides[1:] == (page_size * ns, ns, 1)
                and strides[0] >= heads * page_size * ns and scale_strides[1:] == (page_size, 1)
                and scale_strides[0] >= heads * page_size and k_centroids.is_contiguous() and v_centroids.is_contiguous()
                and k_codes.device == device and v_codes.device == device and k_scales.device == device
                and v_scales.device == device and k_centroids.device == device and v_centroids.device == device):
            return pages, heads, page_size, 2 * ns, strides[0], scale_strides[0], k_centroids.shape[0]
    named = (("k_codes", k_codes), ("v_codes", v_codes), ("k_scales", k_scales), ("v_scales", v_scales),
             ("k_centroids", k_centroids), ("v_centroids", v_centroids))
    for name, t in named:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
    if k_codes.dim() != 4 or k_scales.dim() != 3 or k_centroids.dim() != 1:
        raise ValueError(f"expected codes [pages, heads, page_size, dim / 2], scales [pages, heads, page_size] and "
                         f"centroids [n_centroids], got {tuple(k_codes.shape)}, {tuple(k_scales.shape)} and "
                         f"{tuple(k_centroids.shape)}")
    if k_codes.dtype is not torch.uint8 or v_codes.dtype is not torch.uint8:
        raise TypeError("codes must be uint8")
    if k_scales.dtype is not dtype or v_scales.dtype is not dtype:
        raise TypeError(f"scales must be {dtype}, as the rows are")
    if k_centroids.dtype is not torch.float32 or v_centroids.dtype is not torch.float32:
        raise TypeError("centroids must be float32")
    if v_codes.shape != k_codes.shape:
        raise ValueError("k_codes and v_codes must have one shape")
    if v_scales.shape != k_scales.shape or k_scales.shape != k_codes.shape[:3]:
        raise ValueError("k_scales and v_scales must have the shape of the codes but for the last axis")
    if v_centroids.shape != k_centroids.shape:
        raise ValueError("k_centroids and v_centroids must have one shape")
    pages, heads, page_size, ns = k_codes.shape
    for name, t in named:
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, not on {device}")
    strides = []
    for (name, a), (_, b), inner in ((named[0], named[1], (page_size * ns, ns, 1)), (named[2], named[3], (page_size, 1))):
        least = heads * inner[0]
        for t in (a, b):
            if t.numel() and t.stride()[1:] != inner and not t[0].is_contiguous():
                raise ValueError(f"each page of {name[2:]} must be contiguous")
        mine = [t.stride(0) if pages > 1 else least for t in (a, b)]
        if mine[0] != mine[1] or mine[0] < least:
            raise ValueError(f"the pages of k_{name[2:]} and v_{name[2:]} must not overlap and must have one stride")
        strides.append(mine[0])
    for name, t in named[4:]:
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
    return pages, heads, page_size, 2 * ns, strides[0], strides[1], k_centroids.shape[0]


def _slots_tensor(slots, tokens: int, device, exact: bool) -> None:
    """A contiguous int64 device tensor of ``tokens`` slots (at least, unless ``exact``)."""
    if not isinstance(slots, torch.Tensor) or slots.dtype != torch.int64 or slots.dim() != 1 or \
            slots.shape[0] < tokens or exact and slots.shape[0] != tokens:
        raise ValueError(f"slots must be an int64 tensor of {'shape' if exact else 'at least'} [T]")
    _device_tensor(slots, "slots")
    if slots.device != device:
        raise ValueError(f"slots is on {slots.device}, not on {device}")


def vq_paged_scalar_append(k: torch.Tensor, v: torch.Tensor, slots: torch.Tensor, k_centroids: torch.Tensor,
                           v_centroids: torch.Tensor, k_codes: torch.Tensor, v_codes: torch.Tensor,
                           k_scales: torch.Tensor, v_scales: torch.Tensor, k_signs: torch.Tensor | None = None,
                           stream: torch.cuda.Stream | None = None) -> None:
    """The keys and values of new tokens as 4-bit scalar codes and a scale a row, into
    their slots of the pages.

    ``k`` / ``v`` ``[T, H, D]`` (tokens may be strided, ``D`` even), ``slots`` ``[T]`` int64
    (-1: skipped), ``k_centroids`` / ``v_centroids`` ``[n]`` float32 (up to 16, for rows of
    root mean square one), ``k_codes`` / ``v_codes`` ``[num_pages, H, page_size, D/2]`` uint8
    (the even element's code in the low half) and ``k_scales`` / ``v_scales`` ``[num_pages, H,
    page_size]`` in k's dtype, written in place.  ``k_signs`` ``[D]`` float32 rotates the keys
    first, as :func:`vq_hadamard_rotate` does; the queries are then to be rotated alike."""
    _token_rows(k, "k", None)
    dev = k.device
    _token_rows(v, "v", dev)
    if v.dtype != k.dtype or v.shape != k.shape:
        raise ValueError("k and v must share shape and dtype")
    pages, heads, page_size, dim, stride, scale_stride, n_c = _scalar_page_tensors(
        k_codes, v_codes, k_scales, v_scales, k_centroids, v_centroids, k.dtype, dev)
    tokens, h, d = k.shape
    if h != heads or d != dim:
        raise ValueError(f"k {tuple(k.shape)} does not match codes {tuple(k_codes.shape)}")
    _slots_tensor(slots, tokens, dev, True)
    if k_signs is not None:
        if not isinstance(k_signs, torch.Tensor):
            raise TypeError("k_signs must be a torch.Tensor")
        if k_signs.dtype != torch.float32 or tuple(k_signs.shape) != (d,):
            raise ValueError("k_signs must be float32 of shape [D]")
        _device_tensor(k_signs, "k_signs")
        if k_signs.device != dev:
            raise ValueError(f"k_signs is on {k_signs.device}, not on {dev}")
    _launch(load_library().vq_paged_scalar_append, "vq_paged_scalar_append", dev, stream, k.data_ptr(), v.data_ptr(),
            _token_stride(k), _token_stride(v), slots.data_ptr(), tokens, heads, d, n_c, k_centroids.data_ptr(),
            v_centroids.data_ptr(), k_signs.data_ptr() if k_signs is not None else None, k_codes.data_ptr(),
            v_codes.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(), pages, page_size, stride, scale_stride,
            _dtype_code(k))


def vq_paged_scalar_attention_workspace_bytes(requests: int, tokens: int, max_new: int, heads_q: int, heads_kv: int,
                                              head_dim: int, page_size: int) -> int:
    return int(load_library().vq_paged_scalar_attention_workspace_bytes(requests, tokens, max_new, heads_q, heads_kv,
                                                                        head_dim, page_size))


@functools.lru_cache(maxsize=1024)
def _paged_scalar_workspace(device_index: int, *sizes) -> int:
    """The workspace of a device for these sizes, as often as a step asks for it."""
    with torch.cuda.device(device_index):
        return max(vq_paged_scalar_attention_workspace_bytes(*sizes), 16)


def vq_paged_scalar_attention(q: torch.Tensor, cu_new: torch.Tensor, lens: torch.Tensor, block_table: torch.Tensor,
                              k_codes: torch.Tensor, v_codes: torch.Tensor, k_scales: torch.Tensor,
                              v_scales: torch.Tensor, k_centroids: torch.Tensor, v_centroids: torch.Tensor,
                              max_new: int = 0, window: int = 0, scale: float = 0.0, out: torch.Tensor | None = None,
                              lse: torch.Tensor | None = None, return_lse: bool = False,
                              workspace: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None,
                              slots: torch.Tensor | None = None):
    """Causal attention of the new tokens of every request over pages of 4-bit scalar codes.

    :func:`vq_paged_attention` with pages and centroids as in :func:`vq_paged_scalar_append`,
    the scales in q's dtype.  Returns ``out`` ``[T, Hq, D]``, or ``(out, lse)`` where
    ``return_lse`` is set or ``lse`` is given.  A workspace of
    :func:`vq_paged_scalar_attention_workspace_bytes` bytes is allocated here (by torch) if
    none is given; it and new outputs are allocated on ``stream``."""
    _token_rows(q, "q", None)
    dev = q.device
    tokens, hq, d = q.shape
    pages, hkv, page_size, dim, stride, scale_stride, n_c = _scalar_page_tensors(
        k_codes, v_codes, k_scales, v_scales, k_centroids, v_centroids, q.dtype, dev)
    if dim != d or hkv < 1 or hq % hkv:
        raise ValueError(f"q {tuple(q.shape)} does not match codes {tuple(k_codes.shape)}")
    r = _extent(lens)
    _i32_tensor(lens, "lens", (r,), dev)
    _i32_tensor(cu_new, "cu_new", (r + 1,), dev)
    blocks = _table_tensor(block_table, r, dev)
    if max_new < 0:
        raise ValueError("max_new must not be negative")
    if slots is not None:
        _slots_tensor(slots, tokens, dev, False)
    out = _out_like(out, "out", (tokens, hq, d), q.dtype, dev, stream)
    if return_lse or lse is not None:
        lse = _out_like(lse, "lse", (tokens, hq), torch.float32, dev, stream)
    need = _paged_scalar_workspace(dev.index, r, tokens, max_new, hq, hkv, d, page_size) if workspace is None else 0
    workspace, nbytes = _workspace_of(workspace, need, dev, stream)
    _launch(load_library().vq_paged_scalar_attention, "vq_paged_scalar_attention", dev, stream, q.data_ptr(),
            _token_stride(q), cu_new.data_ptr(), lens.data_ptr(), slots.data_ptr() if slots is not None else None, r,
            tokens, max_new, block_table.data_ptr(), blocks, k_codes.data_ptr(), v_codes.data_ptr(),
            k_scales.data_ptr(), v_scales.data_ptr(), pages, page_size, stride, scale_stride, k_centroids.data_ptr(),
            v_centroids.data_ptr(), hq, hkv, d, n_c, window, scale, _dtype_code(q), out.data_ptr(),
            lse.data_ptr() if lse is not None else None, workspace.data_ptr(), nbytes)
    return (out, lse) if lse is not None else out


def vq_paged_fork_workspace_bytes(num_pages: int) -> int:
    return int(load_library().vq_paged_fork_workspace_bytes(num_pages))


def vq_paged_compact_workspace_bytes(num_pages: int) -> int:
    return int(load_library().vq_paged_compact_workspace_bytes(num_pages))


def _workspace_of(workspace, need: int, device, stream) -> tuple:
    """A workspace of at least ``need`` bytes: the given one, checked, or a new one; and
    its size."""
    if workspace is None:
        workspace = _empty(max(need, 16), torch.uint8, device, stream)
    else:
        if not isinstance(workspace, torch.Tensor):
            raise TypeError("workspace must be a torch.Tensor")
        _device_tensor(workspace, "workspace")
        if workspace.device != device:
            raise ValueError(f"workspace is on {workspace.device}, not on {device}")
    return workspace, workspace.numel() * workspace.element_size()


def vq_paged_fork(lens: torch.Tensor, parents: torch.Tensor, block_table: torch.Tensor, page_size: int,
                  free_pages: torch.Tensor, free_count: torch.Tensor, keep_lens: torch.Tensor | None = None,
                  lens_out: torch.Tensor | None = None, table_out: torch.Tensor | None = None,
                  free_count_out: torch.Tensor | None = None, copies: torch.Tensor | None = None,
                  workspace: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None) -> tuple:
    """Seat ``d`` goes on with the first ``keep_lens[d]`` tokens (None: all) of seat
    ``parents[d]``; a parent outside ``[0, S)`` empties it.

    ``lens`` / ``parents`` / ``keep_lens`` ``[S]``, ``block_table`` ``[S, max_blocks]``,
    ``free_pages`` ``[num_pages]`` (pushed to and popped from in place) and ``free_count``
    ``[1]`` are int32.  Whole pages are shared; a page that several seats end inside is left
    to one of them and the others get pages of their own, whose contents :func:`vq_paged_copy`
    brings over (see ``include/vq_encode.h``).  Returns ``(lens_out, table_out, free_count_out,
    copies)``: ``lens_out`` may be ``lens`` and ``free_count_out`` ``free_count``; ``table_out``
    must not overlap ``block_table``; ``copies`` ``[S, 2]`` holds (from, to) or -1, -1.  A
    workspace of :func:`vq_paged_fork_workspace_bytes` bytes is allocated here (by torch) if
    none is given; it and new outputs are allocated on ``stream``."""
    n = _extent(lens)
    _i32_tensor(lens, "lens", (n,), None)
    dev, pages = lens.device, _extent(free_pages)
    _i32_tensor(parents, "parents", (n,), dev)
    blocks = _table_tensor(block_table, n, dev)
    _i32_tensor(free_pages, "free_pages", (pages,), dev)
    _i32_tensor(free_count, "free_count", (1,), dev)
    if keep_lens is not None:
        _i32_tensor(keep_lens, "keep_lens", (n,), dev)
    lens_out = _out_like(lens_out, "lens_out", (n,), torch.int32, dev, stream)
    table_out = _out_like(table_out, "table_out", (n, blocks), torch.int32, dev, stream)
    free_count_out = _out_like(free_count_out, "free_count_out", (1,), torch.int32, dev, stream)
    copies = _out_like(copies, "copies", (n, 2), torch.int32, dev, stream)
    lib = load_library()
    workspace, nbytes = _workspace_of(workspace, lib.vq_paged_fork_workspace_bytes(pages), dev, stream)
    _launch(lib.vq_paged_fork, "vq_paged_fork", dev, stream, lens.data_ptr(), parents.data_ptr(),
            keep_lens.data_ptr() if keep_lens is not None else None, n, block_table.data_ptr(), blocks, page_size,
            free_pages.data_ptr(), free_count.data_ptr(), pages, lens_out.data_ptr(), table_out.data_ptr(),
            free_count_out.data_ptr(), copies.data_ptr(), workspace.data_ptr(), nbytes)
    return lens_out, table_out, free_count_out, copies


def vq_paged_compact(lens: torch.Tensor, block_table: torch.Tensor, page_size: int, free_pages: torch.Tensor,
                     free_count: torch.Tensor, table_out: torch.Tensor | None = None,
                     free_pages_out: torch.Tensor | None = None, free_count_out: torch.Tensor | None = None,
                     moves: torch.Tensor | None = None, page_map: torch.Tensor | None = None,
                     workspace: torch.Tensor | None = None, stream: torch.cuda.Stream | None = None) -> tuple:
    """Number the held pages ``0 .. used - 1``, those not on the free list.

    Arguments as in :func:`vq_paged_fork`.  Returns ``(table_out, free_pages_out,
    free_count_out, moves, page_map)``; the first three may be ``block_table``,
    ``free_pages`` and ``free_count`` themselves.  ``moves`` ``[num_pages // 2, 2]`` names
    the pages (from, to) whose contents :func:`vq_paged_copy` brings over, then -1, -1;
    ``page_map`` ``[num_pages]`` is the new number of every page, -1 of a free one.  A
    workspace of :func:`vq_paged_compact_workspace_bytes` bytes is allocated here (by torch) if
    none is given; it and new outputs are allocated on ``stream``."""
    n = _extent(lens)
    _i32_tensor(lens, "lens", (n,), None)
    dev, pages = lens.device, _extent(free_pages)
    blocks = _table_tensor(block_table, n, dev)
    _i32_tensor(free_pages, "free_pages", (pages,), dev)
    _i32_tensor(free_count, "free_count", (1,), dev)
    table_out = _out_like(table_out, "table_out", (n, blocks), torch.int32, dev, stream)
    free_pages_out = _out_like(free_pages_out, "free_pages_out", (pages,), torch.int32, dev, stream)
    free_count_out = _out_like(free_count_out, "free_count_out", (1,), torch.int32, dev, stream)
    moves = _out_like(moves, "moves", (pages // 2, 2), torch.int32, dev, stream)
    page_map = _out_like(page_map, "page_map", (pages,), torch.int32, dev, stream)
    lib = load_library()
    workspace, nbytes = _workspace_of(workspace, lib.vq_paged_compact_workspace_bytes(pages), dev, stream)
    _launch(lib.vq_paged_compact, "vq_paged_compact", dev, stream, lens.data_ptr(), n,
            block_table.data_ptr(), blocks, page_size, free_pages.data_ptr(), free_count.data_ptr(), pages,
            table_out.data_ptr(), free_pages_out.data_ptr(), free_count_out.data_ptr(), moves.data_ptr(),
            page_map.data_ptr(), workspace.data_ptr(), nbytes)
    return table_out, free_pages_out, free_count_out, moves, page_map


def vq_paged_copy(pairs: torch.Tensor, pools, layered: bool = False,
                  stream: torch.cuda.Stream | None = None) -> None:
    """Copy page ``pairs[i, 0]`` to page ``pairs[i, 1]`` in every pool.

    ``pairs`` ``[N, 2]`` int32 on the device (pairs of -1 are skipped), as
    :func:`vq_paged_fork` and :func:`vq_paged_compact` return them.  ``pools`` are up to 8
    tensors ``[num_pages, ...]`` (``layered``: ``[layers, num_pages, ...]``) of any dtype, each
    page contiguous; the pages may be strided.  Pages are written in place."""
    rows = pairs.shape[0] if isinstance(pairs, torch.Tensor) and pairs.dim() == 2 else None
    _i32_tensor(pairs, "pairs", (rows, 2), None)
    pools = None if isinstance(pools, torch.Tensor) else list(pools)  # (a generator can be read once)
    if pools is None or not all(isinstance(t, torch.Tensor) for t in pools):
        raise TypeError("pools must be a list of torch.Tensor")
    if not 1 <= len(pools) <= PAGED_MAX_POOLS:
        raise ValueError(f"expected 1 to {PAGED_MAX_POOLS} pools, got {len(pools)}")
    at = 1 if layered else 0  # the axis of pages
    array = (VqPagePool * len(pools))()
    pages = None
    for i, t in enumerate(pools):
        name = f"pools[{i}]"
        if t.dim() <= at:
            raise ValueError(f"{name} must have shape [{'layers, ' if layered else ''}num_pages, ...]")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.device != pairs.device:
            raise ValueError(f"{name} is on {t.device}, not on {pairs.device}")
        if pages is None:
            pages = t.shape[at]
        elif t.shape[at] != pages:
            raise ValueError("the pools must have one number of pages")
        page = t[(0,) * (at + 1)] if t.numel() else None
        if page is not None and not page.is_contiguous():
            raise ValueError(f"each page of {name} must be contiguous")
        size = t.element_size()
        array[i] = VqPagePool(t.data_ptr(), t.stride(at) * size if pages > 1 else 0,
                              page.numel() * size if page is not None else 0,
                              t.stride(0) * size if layered and t.shape[0] > 1 else 0, t.shape[0] if layered else 1)
    _launch(load_library().vq_paged_copy, "vq_paged_copy", pairs.device, stream, pairs.data_ptr(), rows,
            ctypes.addressof(array), len(pools), pages)


# Bytes of the library's built-in scratch array (VQ_ATTN_STATIC_SCRATCH_BYTES).
ATTN_STATIC_SCRATCH_BYTES = 8 << 20


def vq_attention_decode_static(q: torch.Tensor, k_codes: torch.Tensor, k_codebooks: torch.Tensor,
                               v_codes: torch.Tensor, v_codebooks: torch.Tensor, window: int = 0,
                               scale: float = 0.0, out: torch.Tensor | None = None,
                               stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """:func:`vq_attention_decode` with its partials in the library's one
    built-in device array instead of a workspace, for callers that cannot
    allocate device memory per call (a decode loop whose HBM is planned up
    front, host code without a caching allocator).  The library allocates
    nothing; pass ``out`` to allocate nothing here either.  Calls that overlap
    on the GPU share that array and race: keep them in one stream order.  The
    call runs with q's device current, whose copy of the array it uses."""
    b, hq, hkv, tokens, d, sub, n_c = _check_attention_args(q, k_codes, k_codebooks, v_codes,
                                                            v_codebooks)
    if b * hq * (d + 2) * 4 > ATTN_STATIC_SCRATCH_BYTES:
        raise VQError(VQ_ERR_INVALID_ARG,
                      f"vq_attention_decode_static (one token slice needs {b * hq * (d + 2) * 4} "
                      f"bytes of scratch; the built-in array holds {ATTN_STATIC_SCRATCH_BYTES})")
    out = _check_attention_out(out, q, stream)
    with torch.cuda.device(q.device):
        st = load_library().vq_attention_decode_static(
            q.data_ptr(), k_codes.data_ptr(), k_codebooks.data_ptr(), v_codes.data_ptr(),
            v_codebooks.data_ptr(), b, hq, hkv, tokens, d, sub, n_c, window, scale,
            _dtype_code(q), out.data_ptr(), _stream_handle(stream, q.device))
    _check(st, "vq_attention_decode_static")
    return out


def vq_encode_grouped_host(x_host: torch.Tensor, codebooks_host: torch.Tensor,
                           out_host: torch.Tensor, x_dev: torch.Tensor,
                           codebooks_dev: torch.Tensor, out_dev: torch.Tensor,
                           stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Grouped encode of HOST tensors through the caller's device buffers.

    ``x_host`` ``[G, M, sub_dim]``, ``codebooks_host`` ``[G, n_c, sub_dim]`` and
    ``out_host`` ``[G, M]`` uint32 live in host memory (pin them for
    asynchronous copies); ``x_dev``, ``codebooks_dev`` and ``out_dev`` are
    device buffers of at least the same sizes.  Returns ``out_host`` once it
    holds the indices.
    """
    for t, name in ((x_host, "x_host"), (codebooks_host, "codebooks_host"),
                    (out_host, "out_host")):
        if t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous host tensor")
    for t, name in ((x_dev, "x_dev"), (codebooks_dev, "codebooks_dev"), (out_dev, "out_dev")):
        _device_tensor(t, name)
    if x_host.dim() != 3 or codebooks_host.dim() != 3:
        raise ValueError("expected x_host [G, M, sub_dim] and codebooks_host [G, n_c, sub_dim]")
    g, m, sub = x_host.shape
    n_c = codebooks_host.shape[1]
    if (x_dev.dtype != x_host.dtype or codebooks_dev.dtype != x_host.dtype
            or codebooks_host.dtype != x_host.dtype):
        raise TypeError("all x and codebook tensors must share a dtype")
    if out_host.dtype != torch.uint32 or out_dev.dtype != torch.uint32:
        raise TypeError("out_host and out_dev must be uint32")
    if (x_dev.numel() < x_host.numel() or codebooks_dev.numel() < codebooks_host.numel()
            or out_dev.numel() < g * m or out_host.numel() < g * m):
        raise ValueError("device or output buffers are too small")
    st = load_library().vq_encode_grouped_host(
        x_host.data_ptr(), codebooks_host.data_ptr(), g, m, n_c, sub, _dtype_code(x_host),
        out_host.data_ptr(), x_dev.data_ptr(), codebooks_dev.data_ptr(), out_dev.data_ptr(),
        _stream_handle(stream, x_dev.device))
    _check(st, "vq_encode_grouped_host")
    return out_host


def vq_partition(n_groups: int, n_per_group: int, world: int, rank: int) -> list:
    """The rows of a ``[n_groups, n_per_group]`` encode job that ``rank`` of
    ``world`` owns, as ``(group, n_groups, row, n_rows)`` slices in row order
    (see ``vq_partition`` in ``include/vq_encode.h``)."""
    buf = (VqSlice * 3)()
    count = ctypes.c_int32(0)
    st = load_library().vq_partition(n_groups, n_per_group, world, rank, buf, ctypes.byref(count))
    _check(st, "vq_partition")
    return [(s.group, s.n_groups, s.row, s.n_rows) for s in buf[:count.value]]


def vq_encode_partition(x: torch.Tensor, codebooks: torch.Tensor, world: int, rank: int,
                        out: torch.Tensor | None = None,
                        stream: torch.cuda.Stream | None = None) -> torch.Tensor:
    """Rank ``rank``'s share of the grouped encode of ``x`` ``[G, M, sub_dim]``
    against the replicated ``codebooks`` ``[G, n_c, sub_dim]``: the indices of
    the rows :func:`vq_partition` gives it, as a 1-D uint32 tensor in row
    order (one grouped encode per slice; no collective).  Concatenated over
    the ranks in rank order they are ``vq_encode_grouped(x, codebooks)``
    flattened."""
    _device_tensor(x, "x")
    _device_tensor(codebooks, "codebooks")
    if (x.dim() != 3 or codebooks.dim() != 3 or x.shape[0] != codebooks.shape[0]
            or x.shape[2] != codebooks.shape[2]):
        raise ValueError(f"expected x [G, M, sub_dim] and codebooks [G, n_centroids, sub_dim], "
                         f"got {tuple(x.shape)} and {tuple(codebooks.shape)}")
    if x.dtype != codebooks.dtype:
        raise TypeError("x and codebooks must share a dtype")
    g, m, sub = x.shape
    slices = vq_partition(g, m, world, rank)
    n = sum(ng * nr for _, ng, _, nr in slices)
    if out is None:
        out = _empty(n, torch.uint32, x.device, stream)
    elif out.dtype != torch.uint32 or out.shape != (n,) or not out.is_contiguous():
        raise ValueError(f"out must be a contiguous uint32 tensor of shape [{n}]")
    lib = load_library()
    handle = _stream_handle(stream, x.device)
    off = 0
    for g0, ng, r0, nr in slices:
        xs = x[g0:g0 + ng, r0:r0 + nr]  # contiguous: one group, or whole groups
        st = lib.vq_encode_grouped(xs.data_ptr(), codebooks[g0:g0 + ng].data_ptr(), ng, nr,
                                   codebooks.shape[1], sub, _dtype_code(x),
                                   out.data_ptr() + off * 4, handle)
        _check(st, "vq_encode_partition")
        off += ng * nr
    return out


def vq_describe_launch(n_groups: int, n_per_group: int, n_centroids: int, sub_dim: int,
                       dtype: torch.dtype, x_ptr: int = 0) -> str:
    """The kernel and launch shape the library would use (no launch)."""
    buf = ctypes.create_string_buffer(512)
    st = load_library().vq_describe_launch(n_groups, n_per_group, n_centroids, sub_dim,
                                           _TORCH_DTYPES[dtype], x_ptr, buf, len(buf))
    _check(st, "vq_describe_launch")
    return buf.value.decode()
