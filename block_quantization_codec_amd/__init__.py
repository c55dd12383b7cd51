"""ZeRO++ block-quantization codec on AMD Instinct MI355X (gfx950).

Thin Python binding of ``libzpp.so``, whose C ABI is ``include/zpp.h``. The
functions named like the C entry points take the same arguments in the same
order; a pointer argument may be a torch tensor (its ``data_ptr()`` is used)
or a plain integer address, and ``stream`` may be ``None`` (torch's current
stream), a ``torch.cuda.Stream`` or an integer ``hipStream_t``. They only
marshal arguments: every step runs in the library's HIP kernels, and a
non-OK status raises :class:`ZppError`.

The short helpers (:func:`quantize`, :func:`dequantize`, :func:`reorder`,
:func:`dequant_reduce_requant`, :func:`dequant_reduce_average`,
:func:`quantize_reordered`, :func:`linear`, :func:`linear_grad`,
:func:`layer_norm`, :func:`layer_norm_grad`) allocate their outputs with torch on the
input's device and call the same entry points. With ``stream`` they do so as
under ``torch.cuda.stream(stream)``: what they allocate is that stream's, so it
is not handed out again while the stream still uses it. When the inputs are
ready for that stream, and its results for others, is the caller's to order.

Importing the package fails with ``ImportError`` when ``libzpp.so`` has not
been built (``python block_quantization_codec_amd/_build.py``); there is no
fallback path.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libzpp.so")

ZPP_OK = 0
ZPP_ERR_NULL = 1
ZPP_ERR_ARG = 2
ZPP_ERR_ALIGN = 3
ZPP_ERR_UNSUPPORTED = 4
ZPP_ERR_LAUNCH = 5
ZPP_ERR_OVERLAP = 6
ZPP_ERR_POINTER = 7

ZPP_BF16 = 1
ZPP_FP32 = 2

ZPP_MIN_BLOCK = 32
ZPP_MAX_BLOCK = 4096
ZPP_MAX_INPUTS = 4096
ZPP_MAX_DIVISOR = 1 << 24
ZPP_MAX_NUMEL = 1 << 40
ZPP_MAX_FEATURES = 1 << 22
ZPP_MAX_ROWS = 1 << 30

EXPORTED = ("zpp_quantize_blocks", "zpp_quantize_reordered", "zpp_dequantize_blocks", "zpp_reorder_slices",
            "zpp_dequant_reduce_requant", "zpp_dequant_reduce_requant_split", "zpp_dequant_reduce_average",
            "zpp_linear_blocks", "zpp_linear_blocks_grad", "zpp_linear_blocks_workspace", "zpp_layer_norm",
            "zpp_layer_norm_grad", "zpp_layer_norm_grad_workspace",
            "zpp_set_pointer_checks", "zpp_status_string", "zpp_abi_version")


class ZppError(RuntimeError):
    def __init__(self, status: int, func: str):
        self.status = status
        super().__init__(f"{func}: {_lib.zpp_status_string(status).decode()}")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: the codec runs only in its HIP library; build it with "
            "`python block_quantization_codec_amd/_build.py` (or __graft_entry__.build())")
    lib = ctypes.CDLL(LIB_PATH)
    P, I64, I32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    sig = {
        "zpp_quantize_blocks": [P, I32, I64, I32, I32, P, P, P],
        "zpp_quantize_reordered": [P, I32, I64, I32, I32, I32, I32, I32, I32, P, P, P],
        "zpp_dequantize_blocks": [P, P, I32, I64, I32, P, I32, P],
        "zpp_reorder_slices": [P, P, I64, I32, I32, P],
        "zpp_dequant_reduce_requant": [P, I64, P, I64, I32, I32, I64, I32, P, P, I32, P, P],
        "zpp_dequant_reduce_requant_split": [P, I64, P, I64, I32, I32, I64, I32, I64, I64, P, P, P, P, I32, P],
        "zpp_dequant_reduce_average": [P, I64, P, I64, I32, I32, I64, I32, I32, P, P],
        "zpp_linear_blocks": [P, I32, I64, I64, P, P, I32, I64, I64, I32, P, I32, I64, P, I64, P],
        "zpp_linear_blocks_grad": [P, I32, I64, I64, P, P, I32, I64, I64, I32, P, I32, I64, P, I64, P],
        "zpp_layer_norm": [P, I32, I64, I64, I64, P, P, I32, ctypes.c_float, P, I64, P, P, P],
        "zpp_layer_norm_grad": [P, I64, P, I32, I64, I64, I64, P, I32, P, P, P, I64, P, P, P, I64, P],
    }
    for name, args in sig.items():
        f = getattr(lib, name)
        f.argtypes = args
        f.restype = ctypes.c_int
    lib.zpp_linear_blocks_workspace.argtypes = [I32, I32, I64, I32, I64, I64, I64]
    lib.zpp_linear_blocks_workspace.restype = I64
    lib.zpp_layer_norm_grad_workspace.argtypes = [I64, I64]
    lib.zpp_layer_norm_grad_workspace.restype = I64
    lib.zpp_set_pointer_checks.argtypes = [ctypes.c_int32]
    lib.zpp_set_pointer_checks.restype = ctypes.c_int32
    lib.zpp_status_string.argtypes = [ctypes.c_int]
    lib.zpp_status_string.restype = ctypes.c_char_p
    lib.zpp_abi_version.argtypes = []
    lib.zpp_abi_version.restype = ctypes.c_int32
    return lib


_lib = _load()


def library() -> ctypes.CDLL:
    """The loaded ``libzpp.so``."""
    return _lib


def _ptr(a):
    if a is None:
        return None
    if isinstance(a, int):
        return a
    return a.data_ptr()


def _stream(stream):
    if stream is None:
        import torch

        # the current stream's handle, without the Stream object around it
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _under(stream, helper, *args):
    """``helper(*args)`` with ``stream`` as torch's current one, so that what it
    allocates, temporaries too, belongs to the stream that uses it. Its arguments
    stay valid for the work on that stream, and its results for the caller's
    current one, whichever of them is freed first."""
    import torch

    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream(stream)
        stream = torch.cuda.ExternalStream(handle) if handle else torch.cuda.default_stream()
    caller = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        out = helper(*args)
    for t in args:
        if isinstance(t, torch.Tensor) and t.is_cuda:
            t.record_stream(stream)
    for t in out if isinstance(out, tuple) else (out,):
        if t is not None and t.is_cuda:
            t.record_stream(caller)
    return out


def _call(name: str, *args) -> None:
    status = getattr(_lib, name)(*args)
    if status != ZPP_OK:
        raise ZppError(status, name)


# ---- the C entry points, same names and argument order ----------------------

def zpp_quantize_blocks(x, x_dtype, numel, block, bits, codes, scales, stream=None) -> None:
    _call("zpp_quantize_blocks", _ptr(x), x_dtype, numel, block, bits, _ptr(codes), _ptr(scales),
          _stream(stream))


def zpp_quantize_reordered(x, x_dtype, slice_elems, n_nodes, gpus_per_node, first_slice, n_slices, block, bits,
                           codes, scales, stream=None) -> None:
    _call("zpp_quantize_reordered", _ptr(x), x_dtype, slice_elems, n_nodes, gpus_per_node, first_slice, n_slices,
          block, bits, _ptr(codes), _ptr(scales), _stream(stream))


def zpp_dequantize_blocks(codes, scales, bits, numel, block, y, y_dtype, stream=None) -> None:
    _call("zpp_dequantize_blocks", _ptr(codes), _ptr(scales), bits, numel, block, _ptr(y), y_dtype,
          _stream(stream))


def zpp_reorder_slices(inp, out, slice_bytes, n_nodes, gpus_per_node, stream=None) -> None:
    _call("zpp_reorder_slices", _ptr(inp), _ptr(out), slice_bytes, n_nodes, gpus_per_node, _stream(stream))


def zpp_dequant_reduce_requant(codes_in, codes_stride_bytes, scales_in, scales_stride, n_inputs, bits_in,
                               numel, block, codes_out, scales_out, bits_out, sum_out, stream=None) -> None:
    _call("zpp_dequant_reduce_requant", _ptr(codes_in), codes_stride_bytes, _ptr(scales_in), scales_stride,
          n_inputs, bits_in, numel, block, _ptr(codes_out), _ptr(scales_out), bits_out, _ptr(sum_out),
          _stream(stream))


def zpp_dequant_reduce_requant_split(codes_in, codes_stride_bytes, scales_in, scales_stride, n_inputs, bits_in,
                                     numel, block, keep_begin, keep_elems, codes_send, scales_send, codes_keep,
                                     scales_keep, bits_out, stream=None) -> None:
    _call("zpp_dequant_reduce_requant_split", _ptr(codes_in), codes_stride_bytes, _ptr(scales_in), scales_stride,
          n_inputs, bits_in, numel, block, keep_begin, keep_elems, _ptr(codes_send), _ptr(scales_send),
          _ptr(codes_keep), _ptr(scales_keep), bits_out, _stream(stream))


def zpp_dequant_reduce_average(codes_in, codes_stride_bytes, scales_in, scales_stride, n_inputs, bits_in, numel,
                               block, divisor, avg_out, stream=None) -> None:
    _call("zpp_dequant_reduce_average", _ptr(codes_in), codes_stride_bytes, _ptr(scales_in), scales_stride,
          n_inputs, bits_in, numel, block, divisor, _ptr(avg_out), _stream(stream))


def zpp_linear_blocks(x, x_dtype, x_stride, rows, codes, scales, bits, out_features, in_features, block, y, y_dtype,
                      y_stride, workspace, workspace_bytes, stream=None) -> None:
    _call("zpp_linear_blocks", _ptr(x), x_dtype, x_stride, rows, _ptr(codes), _ptr(scales), bits, out_features,
          in_features, block, _ptr(y), y_dtype, y_stride, _ptr(workspace), workspace_bytes, _stream(stream))


def zpp_linear_blocks_grad(dy, dy_dtype, dy_stride, rows, codes, scales, bits, out_features, in_features, block, dx,
                           dx_dtype, dx_stride, workspace, workspace_bytes, stream=None) -> None:
    _call("zpp_linear_blocks_grad", _ptr(dy), dy_dtype, dy_stride, rows, _ptr(codes), _ptr(scales), bits,
          out_features, in_features, block, _ptr(dx), dx_dtype, dx_stride, _ptr(workspace), workspace_bytes,
          _stream(stream))


def zpp_linear_blocks_workspace(grad, in_dtype, in_stride, out_dtype, rows, out_features, in_features) -> int:
    return int(_lib.zpp_linear_blocks_workspace(grad, in_dtype, in_stride, out_dtype, rows, out_features,
                                                in_features))


def zpp_layer_norm(x, x_dtype, x_stride, rows, width, weight, bias, w_dtype, eps, y, y_stride, mean, rstd,
                   stream=None) -> None:
    _call("zpp_layer_norm", _ptr(x), x_dtype, x_stride, rows, width, _ptr(weight), _ptr(bias), w_dtype, eps, _ptr(y),
          y_stride, _ptr(mean), _ptr(rstd), _stream(stream))


def zpp_layer_norm_grad(dy, dy_stride, x, x_dtype, x_stride, rows, width, weight, w_dtype, mean, rstd, dx, dx_stride,
                        dweight, dbias, workspace, workspace_bytes, stream=None) -> None:
    _call("zpp_layer_norm_grad", _ptr(dy), dy_stride, _ptr(x), x_dtype, x_stride, rows, width, _ptr(weight), w_dtype,
          _ptr(mean), _ptr(rstd), _ptr(dx), dx_stride, _ptr(dweight), _ptr(dbias), _ptr(workspace), workspace_bytes,
          _stream(stream))


def zpp_layer_norm_grad_workspace(rows, width) -> int:
    return int(_lib.zpp_layer_norm_grad_workspace(rows, width))


def zpp_set_pointer_checks(enabled: bool) -> bool:
    """Switch the library's HIP-runtime pointer and range checks on or off for
    the process (see include/zpp.h); returns the previous setting."""
    return bool(_lib.zpp_set_pointer_checks(1 if enabled else 0))


def zpp_status_string(status: int) -> str:
    return _lib.zpp_status_string(status).decode()


def zpp_abi_version() -> int:
    return int(_lib.zpp_abi_version())


# ---- allocating helpers ------------------------------------------------------

def _dtype_code(t) -> int:
    import torch

    if t.dtype == torch.bfloat16:
        return ZPP_BF16
    if t.dtype == torch.float32:
        return ZPP_FP32
    raise TypeError(f"unsupported dtype {t.dtype}: bf16 or fp32 expected")


def _need_contiguous(**tensors) -> None:
    """The kernels read flat buffers from data_ptr(): a strided view would be misread."""
    for name, t in tensors.items():
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")


def quantize(x, block: int, bits: int, stream=None):
    """Block-quantize a contiguous bf16/fp32 device tensor. Returns (codes uint8, scales fp32)."""
    if stream is not None:
        return _under(stream, quantize, x, block, bits)
    import torch

    _need_contiguous(x=x)
    n = x.numel()
    codes = torch.empty(n * bits // 8, dtype=torch.uint8, device=x.device)
    scales = torch.empty(n // block, dtype=torch.float32, device=x.device)
    zpp_quantize_blocks(x, _dtype_code(x), n, block, bits, codes, scales, stream)
    return codes, scales


def quantize_reordered(x, n_nodes: int, gpus_per_node: int, block: int, bits: int, first_slice: int = 0,
                       n_slices: int | None = None, stream=None):
    """Quantize the tensor-slice reordered view of contiguous x (N equal slices)
    without writing the reordered tensor. Returns (codes, scales) of output slices
    [first_slice, first_slice + n_slices)."""
    if stream is not None:
        return _under(stream, quantize_reordered, x, n_nodes, gpus_per_node, block, bits, first_slice, n_slices)
    import torch

    _need_contiguous(x=x)
    n = n_nodes * gpus_per_node
    if x.numel() % n:
        raise ValueError("tensor does not split into equal slices")
    slice_elems = x.numel() // n
    n_slices = n - first_slice if n_slices is None else n_slices
    out = slice_elems * n_slices
    codes = torch.empty(out * bits // 8, dtype=torch.uint8, device=x.device)
    scales = torch.empty(out // block, dtype=torch.float32, device=x.device)
    zpp_quantize_reordered(x, _dtype_code(x), slice_elems, n_nodes, gpus_per_node, first_slice, n_slices, block,
                           bits, codes, scales, stream)
    return codes, scales


def dequantize(codes, scales, bits: int, numel: int, block: int, dtype=None, stream=None):
    """Rebuild ``numel`` values (bf16 by default, or fp32) from codes and scales."""
    if stream is not None:
        return _under(stream, dequantize, codes, scales, bits, numel, block, dtype)
    import torch

    _need_contiguous(codes=codes, scales=scales)
    dtype = dtype or torch.bfloat16
    y = torch.empty(numel, dtype=dtype, device=codes.device)
    zpp_dequantize_blocks(codes, scales, bits, numel, block, y, _dtype_code(y), stream)
    return y


def reorder(t, n_nodes: int, gpus_per_node: int, stream=None):
    """Reorder the n_nodes*gpus_per_node equal slices of a contiguous device tensor."""
    if stream is not None:
        return _under(stream, reorder, t, n_nodes, gpus_per_node)
    import torch

    _need_contiguous(t=t)
    n = n_nodes * gpus_per_node
    nbytes = t.numel() * t.element_size()
    if nbytes % n:
        raise ValueError("tensor does not split into equal slices")
    out = torch.empty_like(t)
    zpp_reorder_slices(t, out, nbytes // n, n_nodes, gpus_per_node, stream)
    return out


def dequant_reduce_requant(codes_in, scales_in, n_inputs: int, bits_in: int, numel: int, block: int,
                           bits_out: int = 0, want_sum: bool = True, codes_stride_bytes: int | None = None,
                           scales_stride: int | None = None, stream=None):
    """Sum ``n_inputs`` quantized pieces laid side by side (strides default to one
    piece) and optionally requantize. Returns (codes_out, scales_out, sum_out),
    with None for outputs not requested."""
    if stream is not None:
        return _under(stream, dequant_reduce_requant, codes_in, scales_in, n_inputs, bits_in, numel, block,
                      bits_out, want_sum, codes_stride_bytes, scales_stride)
    import torch

    _need_contiguous(codes_in=codes_in, scales_in=scales_in)
    dev = codes_in.device
    cs = codes_stride_bytes if codes_stride_bytes is not None else numel * bits_in // 8
    ss = scales_stride if scales_stride is not None else numel // block
    co = so = su = None
    if bits_out:
        co = torch.empty(numel * bits_out // 8, dtype=torch.uint8, device=dev)
        so = torch.empty(numel // block, dtype=torch.float32, device=dev)
    if want_sum:
        su = torch.empty(numel, dtype=torch.float32, device=dev)
    zpp_dequant_reduce_requant(codes_in, cs, scales_in, ss, n_inputs, bits_in, numel, block, co, so,
                               bits_out, su, stream)
    return co, so, su


def dequant_reduce_requant_split(codes_in, scales_in, n_inputs: int, bits_in: int, numel: int, block: int,
                                 keep_begin: int, keep_elems: int, bits_out: int,
                                 codes_stride_bytes: int | None = None, scales_stride: int | None = None,
                                 stream=None):
    """The requantized sum of ``n_inputs`` pieces split in one pass: elements
    [keep_begin, keep_begin + keep_elems) (whole blocks) to the kept pair, all
    others, in order, to the send pair. Returns (send_codes, send_scales,
    keep_codes, keep_scales), with None for an empty pair."""
    if stream is not None:
        return _under(stream, dequant_reduce_requant_split, codes_in, scales_in, n_inputs, bits_in, numel, block,
                      keep_begin, keep_elems, bits_out, codes_stride_bytes, scales_stride)
    import torch

    _need_contiguous(codes_in=codes_in, scales_in=scales_in)
    dev = codes_in.device
    cs = codes_stride_bytes if codes_stride_bytes is not None else numel * bits_in // 8
    ss = scales_stride if scales_stride is not None else numel // block
    send = numel - keep_elems
    sc = torch.empty(send * bits_out // 8, dtype=torch.uint8, device=dev) if send > 0 else None
    sS = torch.empty(send // block, dtype=torch.float32, device=dev) if send > 0 else None
    kc = torch.empty(keep_elems * bits_out // 8, dtype=torch.uint8, device=dev) if keep_elems > 0 else None
    kS = torch.empty(keep_elems // block, dtype=torch.float32, device=dev) if keep_elems > 0 else None
    zpp_dequant_reduce_requant_split(codes_in, cs, scales_in, ss, n_inputs, bits_in, numel, block, keep_begin,
                                     keep_elems, sc, sS, kc, kS, bits_out, stream)
    return sc, sS, kc, kS


def dequant_reduce_average(codes_in, scales_in, n_inputs: int, bits_in: int, numel: int, block: int, divisor: int,
                           codes_stride_bytes: int | None = None, scales_stride: int | None = None, stream=None):
    """Sum ``n_inputs`` quantized pieces laid side by side and divide by ``divisor``
    (the number of contributing GPUs). Returns the fp32 average."""
    if stream is not None:
        return _under(stream, dequant_reduce_average, codes_in, scales_in, n_inputs, bits_in, numel, block, divisor,
                      codes_stride_bytes, scales_stride)
    import torch

    _need_contiguous(codes_in=codes_in, scales_in=scales_in)
    cs = codes_stride_bytes if codes_stride_bytes is not None else numel * bits_in // 8
    ss = scales_stride if scales_stride is not None else numel // block
    avg = torch.empty(numel, dtype=torch.float32, device=codes_in.device)
    zpp_dequant_reduce_average(codes_in, cs, scales_in, ss, n_inputs, bits_in, numel, block, divisor, avg, stream)
    return avg


_CODES: dict = {}  # torch dtype -> zpp_dtype, filled at the first use


def _code(dtype) -> int:
    c = _CODES.get(dtype)
    if c is None:
        import torch

        _CODES.update({torch.bfloat16: ZPP_BF16, torch.float32: ZPP_FP32})
        c = _CODES.get(dtype)
        if c is None:
            raise TypeError(f"unsupported dtype {dtype}: bf16 or fp32 expected")
    return c


def _rows(t, name: str):
    """(rows, width, row stride in elements) of a tensor whose leading dimensions
    follow one stride and whose last one is contiguous."""
    shape = t.shape
    if not shape:
        raise ValueError(f"{name} must have at least one dimension")
    width = shape[-1]
    rows = t.numel() // width if width else 0
    if t.is_contiguous():
        return rows, width, width
    if rows <= 1:
        if width > 1 and t.stride(-1) != 1:
            raise ValueError(f"{name}'s last dimension must be contiguous")
        return rows, width, width
    lead = [(n, s) for n, s in zip(shape[:-1], t.stride()[:-1]) if n > 1]
    if (width > 1 and t.stride(-1) != 1) or any(a[1] != b[0] * b[1] for a, b in zip(lead, lead[1:])):
        raise ValueError(f"{name} must be rows of contiguous elements with one stride between them")
    return rows, width, lead[-1][1]


def _check_weight(codes, scales, bits: int, block: int, numel: int) -> None:
    import torch

    if not (codes.is_contiguous() and scales.is_contiguous()):
        raise ValueError("codes and scales must be contiguous")
    if codes.element_size() != 1 or scales.dtype != torch.float32:
        raise TypeError("codes must be bytes and scales float32")
    if codes.numel() * 8 != numel * bits or scales.numel() * block != numel:
        raise ValueError(f"codes and scales do not hold {numel} weights in {bits}-bit blocks of {block}")


def _workspace(workspace, need: int, like):
    """(address, bytes, the tensor to keep) of a call's workspace, on ``like``'s device."""
    if workspace is None:
        if not need:
            return None, 0, None
        import torch

        workspace = like.new_empty(need, dtype=torch.uint8)
    elif not workspace.is_contiguous():  # it would be taken for as many bytes from its first one on
        raise ValueError("workspace must be contiguous")
    return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace


def _linear(name: str, grad: int, a, codes, scales, bits, block, out_len, dtype, out, workspace, stream):
    rows, width, stride = _rows(a, "dy" if grad else "x")
    n_out, n_in = (width, out_len) if grad else (out_len, width)
    _check_weight(codes, scales, bits, block, n_out * n_in)
    adt, ostride = _code(a.dtype), out_len
    if out is None:
        dtype = dtype or a.dtype
        odt = _code(dtype)
        out = a.new_empty((*a.shape[:-1], out_len), dtype=dtype)
    else:
        if tuple(out.shape) != (*a.shape[:-1], out_len) or (dtype or out.dtype) != out.dtype:
            raise ValueError(f"out must be of shape {(*a.shape[:-1], out_len)} and of the dtype asked for")
        odt, ostride = _code(out.dtype), _rows(out, "out")[2]
    need = _lib.zpp_linear_blocks_workspace(grad, adt, stride, odt, rows, n_out, n_in)
    ws, ws_bytes, keep = _workspace(workspace, need, a)
    _call(name, a.data_ptr(), adt, stride, rows, codes.data_ptr(), scales.data_ptr(), bits, n_out, n_in, block,
          out.data_ptr(), odt, ostride, ws, ws_bytes, _stream(stream))
    return out


def linear(x, codes, scales, bits: int, block: int, out_features: int, dtype=None, out=None, workspace=None,
           stream=None):
    """x @ W.T for x [..., in_features] and the [out_features, in_features] weight
    that ``quantize`` turned into codes and scales. The result is of ``dtype``
    (x's by default), or written into ``out``. From bf16 to bf16, weights may be
    rounded to bf16 (past 64 rows, and in the gradient); with a float32 result
    they are not. Autograd does not see the call: the result never requires a
    gradient, :func:`linear_grad` gives it. ``workspace``, if given, is a
    device tensor of at least ``zpp_linear_blocks_workspace`` bytes."""
    if stream is not None:
        return _under(stream, linear, x, codes, scales, bits, block, out_features, dtype, out, workspace)
    return _linear("zpp_linear_blocks", 0, x, codes, scales, bits, block, out_features, dtype, out, workspace, stream)


def linear_grad(dy, codes, scales, bits: int, block: int, in_features: int, dtype=None, out=None, workspace=None,
                stream=None):
    """dy @ W: the gradient of :func:`linear` with respect to x, for dy
    [..., out_features]. Arguments as there."""
    if stream is not None:
        return _under(stream, linear_grad, dy, codes, scales, bits, block, in_features, dtype, out, workspace)
    return _linear("zpp_linear_blocks_grad", 1, dy, codes, scales, bits, block, in_features, dtype, out, workspace,
                   stream)


def _vector(v, width: int, name: str):
    """(address, dtype code) of a weight-like vector, (None, None) of None."""
    if v is None:
        return None, None
    if not v.is_contiguous() or v.numel() != width:
        raise ValueError(f"{name} must be contiguous, of {width} elements")
    return v.data_ptr(), _code(v.dtype)


def _buffer(t, shape, dtype, name: str, x):
    """``t``, for a result of that shape and dtype, or a new tensor on x's device."""
    if t is None:
        return x.new_empty(shape, dtype=dtype)
    if tuple(t.shape) != tuple(shape) or t.dtype != dtype or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, of shape {tuple(shape)} and {dtype}")
    return t


def _like(out, x):
    """``out`` (or a new tensor) of x's shape and dtype, and its row stride."""
    if out is None:
        import torch

        return torch.empty_like(x, memory_format=torch.contiguous_format), x.shape[-1]
    if out.shape != x.shape or out.dtype != x.dtype:
        raise ValueError("out must be of x's shape and dtype")
    return out, _rows(out, "out")[2]


def layer_norm(x, weight=None, bias=None, eps: float = 1e-5, out=None, stream=None, mean=None, rstd=None):
    """Layer norm over x's last dimension. Returns (y, mean, rstd): y of x's
    shape and dtype (or ``out``), mean and rstd float32, one each per row, as
    :func:`layer_norm_grad` takes them (new tensors, or those passed in).
    Autograd does not see the call, as with :func:`linear`."""
    if stream is not None:
        return _under(stream, layer_norm, x, weight, bias, eps, out, None, mean, rstd)
    import torch

    rows, width, stride = _rows(x, "x")
    xdt = _code(x.dtype)
    w, wdt = _vector(weight, width, "weight")
    b, bdt = _vector(bias, width, "bias")
    if wdt and bdt and wdt != bdt:
        raise TypeError("weight and bias must be of one dtype")
    out, ostride = _like(out, x)
    mean = _buffer(mean, x.shape[:-1], torch.float32, "mean", x)
    rstd = torch.empty_like(mean) if rstd is None else _buffer(rstd, x.shape[:-1], torch.float32, "rstd", x)
    _call("zpp_layer_norm", x.data_ptr(), xdt, stride, rows, width, w, b, wdt or bdt or xdt, eps, out.data_ptr(),
          ostride, mean.data_ptr(), rstd.data_ptr(), _stream(stream))
    return out, mean, rstd


def layer_norm_grad(dy, x, weight, mean, rstd, out=None, workspace=None, w_dtype=None, stream=None, dweight=None,
                    dbias=None):
    """Backward pass of :func:`layer_norm`. Returns (dx, dweight, dbias); the
    last two in weight's dtype (``w_dtype``, or x's, when weight is None), in
    new tensors or in those passed in.
    ``workspace``, if given, is a device tensor of at least
    ``zpp_layer_norm_grad_workspace(rows, width)`` bytes."""
    if stream is not None:
        return _under(stream, layer_norm_grad, dy, x, weight, mean, rstd, out, workspace, w_dtype, None, dweight, dbias)
    import torch

    rows, width, stride = _rows(x, "x")
    if dy.shape != x.shape or dy.dtype != x.dtype:
        raise ValueError("dy must be of x's shape and dtype")
    f32 = torch.float32
    if not (mean.is_contiguous() and rstd.is_contiguous() and mean.numel() == rstd.numel() == rows
            and mean.dtype == rstd.dtype == f32):
        raise ValueError("mean and rstd must be contiguous float32, one element per row")
    w, _ = _vector(weight, width, "weight")
    wt = weight.dtype if weight is not None else (w_dtype or x.dtype)
    xdt, wdt, dy_stride = _code(x.dtype), _code(wt), _rows(dy, "dy")[2]
    out, ostride = _like(out, x)
    dw = _buffer(dweight, (width,), wt, "dweight", x)
    db = torch.empty_like(dw) if dbias is None else _buffer(dbias, (width,), wt, "dbias", x)
    need = _lib.zpp_layer_norm_grad_workspace(rows, width) if workspace is None else 0
    ws, ws_bytes, keep = _workspace(workspace, need, x)
    _call("zpp_layer_norm_grad", dy.data_ptr(), dy_stride, x.data_ptr(), xdt, stride, rows, width, w, wdt,
          mean.data_ptr(), rstd.data_ptr(), out.data_ptr(), ostride, dw.data_ptr(), db.data_ptr(), ws, ws_bytes,
          _stream(stream))
    return out, dw, db
