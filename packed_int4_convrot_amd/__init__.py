"""Python binding of libck, the MI355X ConvRot packed-INT4 linear.

Argument marshalling only: tensors are checked for dtype, device and layout,
their pointers and strides are handed to the C ABI (include/ck.h) together with
torch's current HIP stream, and a status other than CK_OK becomes an exception
(ValueError for invalid arguments, RuntimeError otherwise).  Every step of the
computation runs in the HIP kernels of libck.so; there is no other code path.
Importing this package fails if libck.so has not been built
(``python -m packed_int4_convrot_amd.build``).
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libck.so")

CK_OK, CK_ERR_INVALID_ARG, CK_ERR_UNSUPPORTED, CK_ERR_WORKSPACE, CK_ERR_HIP = range(5)
CK_WS_PER_CHANNEL, CK_WS_PER_GROUP = 0, 1
CK_LOGITS_F32, CK_LOGITS_BF16 = 0, 1

_p = ctypes.c_void_p
_i64 = ctypes.c_int64
_i32 = ctypes.c_int32
_f32 = ctypes.c_float
_sz = ctypes.c_size_t

SIGNATURES = {
    "ck_status_str": ([_i32], ctypes.c_char_p),
    "ck_last_error_msg": ([], ctypes.c_char_p),
    "ck_version": ([], ctypes.c_char_p),
    "ck_rotate_quant": ([_p, _i64, _i64, _i64, _i32, _i32, _p, _i64, _p, _p], ctypes.c_int),
    "ck_w4_gemm_q": ([_p, _i64, _p, _i64, _i64, _p, _i64, _p, _i32, _i32, _i64, _p, _p, _i64, _p],
                     ctypes.c_int),
    "ck_w4_gemv": ([_p, _i64, _p, _i64, _i64, _p, _i64, _p, _i32, _i32, _i64, _p, _p, _i64, _p],
                   ctypes.c_int),
    "ck_linear_workspace_bytes": ([_i64, _i64, _i64], _sz),
    "ck_w4a8_linear": ([_p, _i64, _i64, _i64, _i32, _p, _i64, _p, _i32, _i32, _i64, _p, _f32, _p,
                        _i64, _p, _sz, _p], ctypes.c_int),
    "ck_w4a4_linear": ([_p, _i64, _i64, _i64, _i32, _p, _i64, _p, _i32, _i32, _i64, _p, _f32, _p,
                        _i64, _p, _sz, _p], ctypes.c_int),
    "ck_w4a4_linear_noalloc": ([_p, _i64, _i64, _i64, _i32, _p, _i64, _p, _i32, _i32, _i64, _p, _f32, _p,
                                _i64, _p], ctypes.c_int),
    "ck_w4a16_gemv": ([_p, _i64, _i64, _i64, _p, _i64, _p, _p, _i32, _i64, _p, _p, _i64, _p],
                      ctypes.c_int),
    "ck_w4a16_gemm": ([_p, _i64, _i64, _i64, _p, _i64, _p, _p, _i32, _i64, _p, _p, _i64, _p],
                      ctypes.c_int),
    "ck_quantize_weights": ([_p, _i64, _i64, _i64, _i32, _i32, _p, _i64, _p, _p], ctypes.c_int),
    "ck_test_rotate_f32": ([_p, _i64, _i64, _i64, _i32, _p, _i64, _p], ctypes.c_int),
    "ck_test_gemm_i32": ([_p, _i64, _i64, _i64, _p, _i64, _i64, _p, _i64, _p], ctypes.c_int),
    "ck_rotate_quant_packed4": ([_p, _i64, _i64, _i64, _i32, _p, _i64, _p, _p], ctypes.c_int),
    "ck_w4a4_gemm_packed": ([_p, _i64, _p, _i64, _i64, _p, _i64, _p, _i32, _i32, _i64, _p, _p, _i64, _p],
                            ctypes.c_int),
    "ck_test_gemm_i32_a4": ([_p, _i64, _i64, _i64, _p, _i64, _i64, _p, _i64, _p], ctypes.c_int),
    "ck_test_linear_mfma_one_launch": ([_i32, _p, _i64, _i64, _i64, _i32, _p, _i64, _p, _i32, _i32, _i64, _p,
                                        _f32, _p, _i64, _p], ctypes.c_int),
    "ck_moe_route": ([_p, _i32, _i64, _i64, _i64, _i32, _i32, _p, _p, _p], ctypes.c_int),
    "ck_moe_workspace_bytes": ([_i64, _i64, _i64, _i32], _sz),
    "ck_moe_w4a16": ([_p, _i64, _i64, _i64, _p, _i32, _i64, _i32, _i32, _i64, _i64, _i32, _p, _p, _p, _p, _p, _p,
                      _p, _i64, _p, _p, _p, _sz, _p], ctypes.c_int),
    "ck_moe_experts_w4a16": ([_p, _i64, _i64, _i64, _p, _p, _i32, _i64, _i64, _i32, _p, _p, _p, _p, _p, _p, _p, _i64,
                              _p, _sz, _p], ctypes.c_int),
    "ck_fp8_quant": ([_p, _i64, _i64, _i64, _p, _i64, _p, _i64, _p], ctypes.c_int),
    "ck_fp8_quantize_weights": ([_p, _i64, _i64, _i64, _p, _i64, _p, _p], ctypes.c_int),
    "ck_fp8_transpose_weights": ([_p, _i64, _p, _i64, _i64, _p, _i64, _p, _p], ctypes.c_int),
    "ck_fp8_gemm": ([_p, _i64, _p, _i64, _i64, _i64, _p, _i64, _p, _i64, _p, _p, _i64, _p], ctypes.c_int),
    "ck_fp8_linear_workspace_bytes": ([_i64, _i64, _i64], _sz),
    "ck_fp8_linear": ([_p, _i64, _i64, _i64, _p, _i64, _p, _i64, _p, _p, _i64, _p, _sz, _p], ctypes.c_int),
    "ck_fp8_ffn_workspace_bytes": ([_i64, _i64, _i64], _sz),
    "ck_fp8_ffn_backward_workspace_bytes": ([_i64, _i64, _i64], _sz),
    "ck_fp8_ffn": ([_p, _i64, _i64, _i64, _i64, _p, _p, _p, _p, _p, _i64, _p, _i64, _p, _sz, _p], ctypes.c_int),
    "ck_fp8_ffn_backward": ([_p, _i64, _i64, _i64, _p, _i64, _i64, _p, _p, _p, _p, _p, _i64, _p, _sz, _p],
                            ctypes.c_int),
    "ck_lora_workspace_bytes": ([_i64, _i64, _i64, _i64], _sz),
    "ck_lora_add": ([_p, _i64, _i64, _i64, _p, _i64, _i64, _p, _p, _p, _p, _i64, _p, _i64, _p, _i64, _p, _sz, _p],
                    ctypes.c_int),
}


def _load_library():
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            "libck.so is not built (expected at %s); run `python -m packed_int4_convrot_amd.build`"
            % LIB_PATH)
    lib = ctypes.CDLL(LIB_PATH)
    for name, (args, res) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    return lib


lib = _load_library()


class CKError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__("%s: %s" % (lib.ck_status_str(status).decode(), msg))
        self.status = status


class CKInvalidArgument(CKError, ValueError):
    pass


def last_error() -> str:
    return lib.ck_last_error_msg().decode()


def version() -> str:
    return lib.ck_version().decode()


def _check(status: int):
    if status == CK_OK:
        return
    if status == CK_ERR_INVALID_ARG:
        raise CKInvalidArgument(status, last_error())
    raise CKError(status, last_error())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# The handle alone: a torch.cuda.Stream object costs 2 us of host time, as much as a launch.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(t):
    """Handle of the current stream of t's device."""
    if _raw_stream is not None and t.is_cuda:
        return _raw_stream(t.get_device())
    return torch.cuda.current_stream(t.device).cuda_stream


def _matrix(t, name, dtypes):
    """A 2-D GPU tensor of one of `dtypes` whose rows are disjoint runs of unit-stride
    elements (the layout the C ABI describes with one row stride)."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        raise ValueError("%s must be a 2-D tensor" % name)
    if t.dtype not in dtypes:
        raise ValueError("%s has dtype %s, expected one of %s" % (name, t.dtype, dtypes))
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("%s must have unit column stride" % name)
    if t.shape[0] > 1 and t.stride(0) < t.shape[1]:
        # expanded (stride 0) or overlapping rows: the C ABI would take them as
        # disjoint rows of stride >= K and touch memory past the tensor's storage
        raise ValueError("%s has row stride %d below its row length %d (expanded or overlapping rows)"
                         % (name, t.stride(0), t.shape[1]))
    if not t.is_cuda:
        raise ValueError("%s must be a GPU tensor" % name)
    return t


def _ld(t):
    """Row stride in elements.  A single row may report any stride, so it counts as its
    own length; for more rows _matrix has checked that the stride covers a row."""
    if t.shape[0] <= 1:
        return max(t.stride(0), t.shape[1])
    if t.stride(0) < t.shape[1]:
        raise ValueError("row stride %d below the row length %d" % (t.stride(0), t.shape[1]))
    return t.stride(0)


def _same_device(ref, *named):
    for name, t in named:
        if t is not None and t.device != ref.device:
            raise ValueError("%s is on %s, expected %s" % (name, t.device, ref.device))


def _dense(t, name, dtype, shape):
    """A contiguous tensor of exactly this shape and dtype on the GPU (the kernels index
    it as a packed array)."""
    if not isinstance(t, torch.Tensor) or t.dtype != dtype or tuple(t.shape) != tuple(shape):
        raise ValueError("%s must be a %s tensor of shape %s" % (name, dtype, tuple(shape)))
    if not t.is_cuda or not t.is_contiguous():
        raise ValueError("%s must be a contiguous GPU tensor" % name)
    return t


def _out(t, name, dtype, M, N):
    """An output matrix of M rows of N elements (row stride may exceed N)."""
    _matrix(t, name, (dtype,))
    if tuple(t.shape) != (M, N):
        raise ValueError("%s has shape %s, expected (%d, %d)" % (name, tuple(t.shape), M, N))
    return t


def _weights(packed, w_scales, per_group, K):
    _matrix(packed, "packed", (torch.uint8, torch.int8))
    if packed.shape[1] != K // 2:
        raise ValueError("packed has %d bytes per row, expected K/2 = %d" % (packed.shape[1], K // 2))
    N = packed.shape[0]
    if w_scales is not None:
        _dense(w_scales, "weight scales", torch.bfloat16, (K // 64, N) if per_group else (N,))
    return N


def workspace_bytes(M: int, K: int, N: int) -> int:
    """Workspace bytes of the whole-linear entry points for M rows, K columns, N outputs."""
    return int(lib.ck_linear_workspace_bytes(M, K, N))


def rotate_quant(x, G: int, bits: int, codes=None, row_scales=None):
    """codes int8 [M, K] and fp32 row scales [M] of a bf16 [M, K] (possibly strided) input."""
    _matrix(x, "x", (torch.bfloat16,))
    M, K = x.shape
    if codes is None:
        codes = torch.empty((M, K), dtype=torch.int8, device=x.device)
    if row_scales is None:
        row_scales = torch.empty((M,), dtype=torch.float32, device=x.device)
    _out(codes, "codes", torch.int8, M, K)
    _dense(row_scales, "row_scales", torch.float32, (M,))
    _same_device(x, ("codes", codes), ("row_scales", row_scales))
    _check(lib.ck_rotate_quant(_ptr(x), M, K, _ld(x), G, bits, _ptr(codes), _ld(codes),
                               _ptr(row_scales), _stream(x)))
    return codes, row_scales


def quantize_weights(w, G: int, per_group: bool, packed=None, scales=None):
    """Packed uint4 weights uint8 [N, K/2] and bf16 scales ([N] or [K/64, N]) of a
    bf16 weight [N, K] rotated by H_G: the producer of the matmuls' weight format."""
    _matrix(w, "w", (torch.bfloat16,))
    N, K = w.shape
    if packed is None:
        packed = torch.empty((N, K // 2), dtype=torch.uint8, device=w.device)
    if scales is None:
        shape = (K // 64, N) if per_group else (N,)
        scales = torch.empty(shape, dtype=torch.bfloat16, device=w.device)
    _out(packed, "packed", torch.uint8, N, K // 2)
    _dense(scales, "scales", torch.bfloat16, (K // 64, N) if per_group else (N,))
    _same_device(w, ("packed", packed), ("scales", scales))
    _check(lib.ck_quantize_weights(_ptr(w), N, K, _ld(w), G, 1 if per_group else 0, _ptr(packed),
                                   _ld(packed), _ptr(scales), _stream(w)))
    return packed, scales


def rotated_f32(x, G: int):
    """Rotated rows as the rotate-quant kernel holds them (divided by sqrt(G)), fp32 [M, K]."""
    _matrix(x, "x", (torch.bfloat16,))
    M, K = x.shape
    xr = torch.empty((M, K), dtype=torch.float32, device=x.device)
    _check(lib.ck_test_rotate_f32(_ptr(x), M, K, _ld(x), G, _ptr(xr), _ld(xr), _stream(x)))
    return xr


def gemm_q(codes, row_scales, packed, w_scales, per_group: bool, bias=None, out=None,
           gemv: bool = False):
    """bf16 [M, N] matmul + scale epilogue on already quantised activations."""
    _matrix(codes, "codes", (torch.int8,))
    M, K = codes.shape
    N = _weights(packed, w_scales, per_group, K)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=codes.device)
    _dense(row_scales, "row_scales", torch.float32, (M,))
    if bias is not None:
        _dense(bias, "bias", torch.bfloat16, (N,))
    _out(out, "out", torch.bfloat16, M, N)
    _same_device(codes, ("row_scales", row_scales), ("packed", packed), ("w_scales", w_scales),
                 ("bias", bias), ("out", out))
    fn = lib.ck_w4_gemv if gemv else lib.ck_w4_gemm_q
    _check(fn(_ptr(codes), _ld(codes), _ptr(row_scales), M, K, _ptr(packed), _ld(packed),
              _ptr(w_scales), CK_WS_PER_GROUP if per_group else CK_WS_PER_CHANNEL, 64, N,
              _ptr(bias), _ptr(out), _ld(out), _stream(codes)))
    return out


def gemv(codes, row_scales, packed, w_scales, per_group: bool, bias=None, out=None):
    """Decode form of gemm_q (1 <= M <= 8)."""
    return gemm_q(codes, row_scales, packed, w_scales, per_group, bias, out, gemv=True)


def linear(x, G: int, bits: int, packed, w_scales, per_group: bool, bias=None,
           x_scale: float = 1.0, out=None, workspace=None):
    """Whole ConvRot linear: bf16 [M, N] = rotate-quant(x) @ W4^T with the scale epilogue."""
    _matrix(x, "x", (torch.bfloat16,))
    M, K = x.shape
    N = _weights(packed, w_scales, per_group, K)
    if bits not in (8, 4):
        raise ValueError("bits must be 8 or 4")
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    need = workspace_bytes(M, K, N)
    if workspace is None:
        workspace = torch.empty((max(need, 1),), dtype=torch.uint8, device=x.device)
    if bias is not None:
        _dense(bias, "bias", torch.bfloat16, (N,))
    _out(out, "out", torch.bfloat16, M, N)
    if workspace.dtype != torch.uint8 or workspace.dim() != 1 or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous 1-D uint8 tensor")
    _same_device(x, ("packed", packed), ("w_scales", w_scales), ("bias", bias), ("out", out),
                 ("workspace", workspace))
    fn = lib.ck_w4a8_linear if bits == 8 else lib.ck_w4a4_linear
    _check(fn(_ptr(x), M, K, _ld(x), G, _ptr(packed), _ld(packed), _ptr(w_scales),
              CK_WS_PER_GROUP if per_group else CK_WS_PER_CHANNEL, 64, N, _ptr(bias), x_scale,
              _ptr(out), _ld(out), _ptr(workspace), workspace.numel() * workspace.element_size(),
              _stream(x)))
    return out


def linear_mfma_one_launch(x, G: int, bits: int, packed, w_scales, per_group: bool, bias=None,
                                x_scale: float = 1.0, out=None):
    """ck_test_linear_mfma_one_launch: the whole linear forced onto its one-launch
    MFMA kernel (1 <= M <= 8, K <= 4096, any N), for testing its launch shapes."""
    _matrix(x, "x", (torch.bfloat16,))
    M, K = x.shape
    N = _weights(packed, w_scales, per_group, K)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    if bias is not None:
        _dense(bias, "bias", torch.bfloat16, (N,))
    _out(out, "out", torch.bfloat16, M, N)
    _same_device(x, ("packed", packed), ("w_scales", w_scales), ("bias", bias), ("out", out))
    _check(lib.ck_test_linear_mfma_one_launch(bits, _ptr(x), M, K, _ld(x), G, _ptr(packed), _ld(packed),
                                              _ptr(w_scales), CK_WS_PER_GROUP if per_group else CK_WS_PER_CHANNEL,
                                              64, N, _ptr(bias), x_scale, _ptr(out), _ld(out), _stream(x)))
    return out


NOALLOC_SCRATCH_BYTES = (64 << 20) + (64 << 10)   # the library's static scratch per GPU (include/ck.h)


def w4a4_linear_noalloc(x, G: int, packed, w_scales, per_group: bool, bias=None,
                        x_scale: float = 1.0, out=None):
    """ck_w4a4_linear without a workspace: the codes live in the library's static
    scratch (one per GPU, shared by every call on it; calls must not overlap)."""
    _matrix(x, "x", (torch.bfloat16,))
    M, K = x.shape
    N = _weights(packed, w_scales, per_group, K)
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    if bias is not None:
        _dense(bias, "bias", torch.bfloat16, (N,))
    _out(out, "out", torch.bfloat16, M, N)
    _same_device(x, ("packed", packed), ("w_scales", w_scales), ("bias", bias), ("out", out))
    _check(lib.ck_w4a4_linear_noalloc(_ptr(x), M, K, _ld(x), G, _ptr(packed), _ld(packed), _ptr(w_scales),
                                      CK_WS_PER_GROUP if per_group else CK_WS_PER_CHANNEL, 64, N, _ptr(bias),
                                      x_scale, _ptr(out), _ld(out), _stream(x)))
    return out


def w4a8_linear(x, G, packed, w_scales, per_group, **kw):
    return linear(x, G, 8, packed, w_scales, per_group, **kw)


def w4a4_linear(x, G, packed, w_scales, per_group, **kw):
    return linear(x, G, 4, packed, w_scales, per_group, **kw)


def w4a16_gemm(x, packed, scales, zeros, bias=None, out=None):
    """AWQ W4A16 product for any M on the dequantise path (W rebuilt in bf16), bf16 [M, N]."""
    _matrix(x, "x", (torch.bfloat16,))
    M, K = x.shape
    N = _weights(packed, scales, True, K)
    _dense(zeros, "zeros", torch.bfloat16, (K // 64, N))
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    if bias is not None:
        _dense(bias, "bias", torch.bfloat16, (N,))
    _out(out, "out", torch.bfloat16, M, N)
    _same_device(x, ("packed", packed), ("scales", scales), ("zeros", zeros), ("bias", bias),
                 ("out", out))
    _check(lib.ck_w4a16_gemm(_ptr(x), M, K, _ld(x), _ptr(packed), _ld(packed), _ptr(scales),
                             _ptr(zeros), 64, N, _ptr(bias), _ptr(out), _ld(out), _stream(x)))
    return out


def w4a16_gemv(x, packed, scales, zeros, bias=None, out=None):
    """AWQ W4A16 product, bf16 [M, N] (1 <= M <= 8)."""
    _matrix(x, "x", (torch.bfloat16,))
    M, K = x.shape
    N = _weights(packed, scales, True, K)
    _dense(zeros, "zeros", torch.bfloat16, (K // 64, N))
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    if bias is not None:
        _dense(bias, "bias", torch.bfloat16, (N,))
    _out(out, "out", torch.bfloat16, M, N)
    _same_device(x, ("packed", packed), ("scales", scales), ("zeros", zeros), ("bias", bias),
                 ("out", out))
    _check(lib.ck_w4a16_gemv(_ptr(x), M, K, _ld(x), _ptr(packed), _ld(packed), _ptr(scales),
                             _ptr(zeros), 64, N, _ptr(bias), _ptr(out), _ld(out), _stream(x)))
    return out


def rotate_quant_packed4(x, G: int, codes4=None, row_scales=None):
    """W4A4 codes packed two per byte, uint8 [M, K/2] (column 2j in the low
    nibble, 4-bit two's complement), and fp32 row scales [M]."""
    _matrix(x, "x", (torch.bfloat16,))
    M, K = x.shape
    if codes4 is None:
        codes4 = torch.empty((M, K // 2), dtype=torch.uint8, device=x.device)
    if row_scales is None:
        row_scales = torch.empty((M,), dtype=torch.float32, device=x.device)
    _out(codes4, "codes4", torch.uint8, M, K // 2)
    _dense(row_scales, "row_scales", torch.float32, (M,))
    _same_device(x, ("codes4", codes4), ("row_scales", row_scales))
    _check(lib.ck_rotate_quant_packed4(_ptr(x), M, K, _ld(x), G, _ptr(codes4), _ld(codes4),
                                       _ptr(row_scales), _stream(x)))
    return codes4, row_scales


def gemm_packed4(codes4, row_scales, packed, w_scales, per_group: bool, bias=None, out=None):
    """bf16 [M, N] linear output from packed W4A4 codes (rotate_quant_packed4) on the tiled GEMM."""
    _matrix(codes4, "codes4", (torch.uint8,))
    M = codes4.shape[0]
    K = 2 * codes4.shape[1]
    N = _weights(packed, w_scales, per_group, K)
    _dense(row_scales, "row_scales", torch.float32, (M,))
    if bias is not None:
        _dense(bias, "bias", torch.bfloat16, (N,))
    if out is None:
        out = torch.empty((M, N), dtype=torch.bfloat16, device=codes4.device)
    _out(out, "out", torch.bfloat16, M, N)
    _same_device(codes4, ("row_scales", row_scales), ("packed", packed), ("w_scales", w_scales),
                 ("bias", bias), ("out", out))
    _check(lib.ck_w4a4_gemm_packed(_ptr(codes4), _ld(codes4), _ptr(row_scales), M, K, _ptr(packed),
                                   _ld(packed), _ptr(w_scales), 1 if per_group else 0, 64, N, _ptr(bias),
                                   _ptr(out), _ld(out), _stream(codes4)))
    return out


def accumulators_i32_a4(codes4, K: int, packed):
    """int32 [M, N] accumulators of the tiled GEMM on packed W4A4 codes uint8 [M, K/2]."""
    _matrix(codes4, "codes4", (torch.uint8,))
    M = codes4.shape[0]
    if codes4.shape[1] != K // 2:
        raise ValueError("codes4 must have K/2 = %d columns (got %d)" % (K // 2, codes4.shape[1]))
    N = _weights(packed, None, False, K)
    acc = torch.empty((M, N), dtype=torch.int32, device=codes4.device)
    _same_device(codes4, ("packed", packed))
    _check(lib.ck_test_gemm_i32_a4(_ptr(codes4), _ld(codes4), M, K, _ptr(packed), _ld(packed), N,
                                   _ptr(acc), _ld(acc), _stream(codes4)))
    return acc


def accumulators_i32(codes, packed):
    """int32 [M, N] accumulators sum_k codes[m,k] * (q[n,k] - 8) from the matmul kernels."""
    _matrix(codes, "codes", (torch.int8,))
    M, K = codes.shape
    N = _weights(packed, None, False, K)
    acc = torch.empty((M, N), dtype=torch.int32, device=codes.device)
    _check(lib.ck_test_gemm_i32(_ptr(codes), _ld(codes), M, K, _ptr(packed), _ld(packed), N,
                                _ptr(acc), _ld(acc), _stream(codes)))
    return acc


# ----------------------------------------------- weights chosen row by row
# These run many times a decode step, where the call itself costs as much as the
# kernels: the weights are checked once, when their handle is made.

_LOGIT_KIND = {torch.float32: CK_LOGITS_F32, torch.bfloat16: CK_LOGITS_BF16}


# What is not a tensor shows by the attributes it lacks: isinstance() for each argument would
# cost every call.

def _row_count(t, name):
    """Rows of a 2-D tensor."""
    try:
        rows, _ = t.shape
    except (AttributeError, TypeError, ValueError):
        raise ValueError("%s must be a 2-D tensor" % name) from None
    return rows


def _rows(t, name, dtype, device, shape):
    """Row stride of a matrix of exactly this shape, dtype and device with unit column stride."""
    try:
        fits = t.dtype is dtype and t.device == device and t.shape == shape
        if not fits:
            raise ValueError("%s must be a %s tensor of shape %s on %s (got %s %s on %s)"
                             % (name, dtype, shape, device, t.dtype, tuple(t.shape), t.device))
    except AttributeError:
        raise ValueError("%s must be a tensor" % name) from None
    ld, col = t.stride()
    if col != 1 and shape[1] > 1:
        raise ValueError("%s must have unit column stride" % name)
    if shape[0] <= 1:
        return max(ld, shape[1])
    if ld < shape[1]:
        raise ValueError("%s has row stride %d below its row length %d (expanded or overlapping rows)"
                         % (name, ld, shape[1]))
    return ld


def _flat(t, name, dtype, device, shape):
    """Pointer of a contiguous tensor of exactly this shape, dtype and device."""
    try:
        if t.dtype is dtype and t.device == device and t.shape == shape and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    raise ValueError("%s must be a contiguous %s tensor of shape %s on %s" % (name, dtype, shape, device))


def _logits(logits):
    """(kind, row stride) of a [T, E] GPU matrix of router logits."""
    _row_count(logits, "logits")
    kind = _LOGIT_KIND.get(getattr(logits, "dtype", None))
    if kind is None or not logits.is_cuda:
        raise ValueError("logits must be a 2-D fp32 or bf16 GPU tensor")
    return kind, _rows(logits, "logits", logits.dtype, logits.device, logits.shape)


def _space(workspace, need, device):
    """A workspace tensor of at least `need` bytes."""
    if workspace is None:
        return torch.empty((max(need, 1),), dtype=torch.uint8, device=device)
    try:
        if workspace.dtype is torch.uint8 and workspace.dim() == 1 and workspace.is_contiguous() \
                and workspace.device == device:
            return workspace
    except AttributeError:
        pass
    raise ValueError("workspace must be a contiguous 1-D uint8 tensor on %s" % device)


def _slots(ids, weights, T, k, device):
    if not 1 <= k < 2 ** 31:
        raise ValueError("k must be positive (got %s)" % k)
    ids = torch.empty((T, k), dtype=torch.int32, device=device) if ids is None else ids
    weights = torch.empty((T, k), dtype=torch.float32, device=device) if weights is None else weights
    return ids, weights


def moe_route(logits, k: int, renormalize: bool = True, ids=None, weights=None):
    """Top-k routing of fp32 or bf16 logits [T, E]: int32 ids and fp32 softmax weights [T, k],
    descending, ties to the lowest expert; -inf (and NaN) logits are never chosen (id -1,
    weight 0).  renormalize: weights over the chosen experts sum to 1."""
    kind, ldl = _logits(logits)
    T, E = logits.shape
    dev = logits.device
    ids, weights = _slots(ids, weights, T, k, dev)
    _check(lib.ck_moe_route(logits.data_ptr(), kind, T, E, ldl, k, 1 if renormalize else 0,
                            _flat(ids, "ids", torch.int32, dev, (T, k)),
                            _flat(weights, "weights", torch.float32, dev, (T, k)), _stream(logits)))
    return ids, weights


def moe_workspace_bytes(T: int, I: int, E: int, k: int) -> int:
    """Workspace bytes of moe and moe_experts for T tokens, inner width I, E experts, k slots."""
    return int(lib.ck_moe_workspace_bytes(T, I, E, k))


def _absent():
    """The address of a tensor that was not given."""
    return None


def _held(tensors):
    """The tensors' storages, and a function of each that tells its address (read for each
    call: an address of last time may be freed memory)."""
    held = tuple(None if t is None else t.detach() for t in tensors)
    return held, tuple(_absent if t is None else t.data_ptr for t in held)


class MoeExperts:
    """The packed uint4 weights of a mixture-of-experts layer (AWQ W4A16, group 64):
    w1 uint8 [E, 2I, H/2] (I gate rows, then I up rows), s1 and z1 bf16 [E, H/64, 2I],
    w2 uint8 [E, H, I/2], s2 and z2 bf16 [E, I/64, H]; the zero points may be None.
    The tensors' storages are kept, not copied: values written into the tensors later count, a
    storage that is put in a tensor's place (t.data = ...) does not."""

    def __init__(self, w1, s1, z1, w2, s2, z2):
        if not isinstance(w1, torch.Tensor) or w1.dim() != 3 or not isinstance(w2, torch.Tensor) or w2.dim() != 3:
            raise ValueError("w1 and w2 must be 3-D tensors")
        E, H, I = w1.shape[0], 2 * w1.shape[2], w1.shape[1] // 2
        if w1.shape[1] % 2 or H <= 0 or I <= 0 or H % 64 or I % 64:
            raise ValueError("w1 has shape %s: expected [E, 2I, H/2] with H and I multiples of 64" % (tuple(w1.shape),))
        for name, t, shape in (("w1", w1, (E, 2 * I, H // 2)), ("w2", w2, (E, H, I // 2))):
            if t.dtype not in (torch.uint8, torch.int8):
                raise ValueError("%s must be uint8 or int8" % name)
            _dense(t, name, t.dtype, shape)
        for name, t, shape in (("s1", s1, (E, H // 64, 2 * I)), ("z1", z1, (E, H // 64, 2 * I)),
                               ("s2", s2, (E, I // 64, H)), ("z2", z2, (E, I // 64, H))):
            if t is None and name[0] == "z":
                continue
            _dense(t, name, torch.bfloat16, shape)
        _same_device(w1, ("s1", s1), ("z1", z1), ("w2", w2), ("s2", s2), ("z2", z2))
        self.tensors, self._at = _held((w1, s1, z1, w2, s2, z2))
        self.E, self.H, self.I, self.device = E, H, I, w1.device

    def _args(self):
        w1, s1, z1, w2, s2, z2 = self._at
        at = (self.E, self.I, 64, w1(), s1(), z1(), w2(), s2(), z2())
        if 0 in at:
            raise ValueError("experts: none, or a tensor has no storage any more")
        return at


def _moe_buffers(x, experts, k, out, workspace):
    T = _row_count(x, "x")
    ldx = _rows(x, "x", torch.bfloat16, experts.device, (T, experts.H))
    out = torch.empty((T, experts.H), dtype=torch.bfloat16, device=experts.device) if out is None else out
    ldo = _rows(out, "out", torch.bfloat16, experts.device, (T, experts.H))
    workspace = _space(workspace, lib.ck_moe_workspace_bytes(T, experts.I, experts.E, k) if workspace is None else 0,
                       experts.device)
    return T, ldx, out, ldo, workspace


def moe(x, logits, experts: MoeExperts, k: int, renormalize: bool = True, out=None, ids=None, weights=None,
        workspace=None):
    """Whole mixture-of-experts layer on packed experts, for few tokens: routes bf16 x [T, H]
    by logits [T, E] as moe_route and returns (out bf16 [T, H], ids, weights) with
    out[t] = sum_j weights[t, j] W2[e] (silu(W1[e][:I] x) * (W1[e][I:] x)), e = ids[t, j]."""
    kind, ldl = _logits(logits)
    T, ldx, out, ldo, workspace = _moe_buffers(x, experts, k, out, workspace)
    dev = experts.device
    if logits.shape != (T, experts.E) or logits.device != dev:
        raise ValueError("logits must have shape (%d, %d) on %s" % (T, experts.E, dev))
    ids, weights = _slots(ids, weights, T, k, dev)
    _check(lib.ck_moe_w4a16(x.data_ptr(), T, experts.H, ldx, logits.data_ptr(), kind, ldl, k, 1 if renormalize else 0,
                            *experts._args(), out.data_ptr(), ldo, _flat(ids, "ids", torch.int32, dev, (T, k)),
                            _flat(weights, "weights", torch.float32, dev, (T, k)), workspace.data_ptr(),
                            workspace.numel(), _stream(x)))
    return out, ids, weights


def moe_experts(x, ids, weights, experts: MoeExperts, out=None, workspace=None):
    """The experts' part of moe from given int32 ids and fp32 weights [T, k] (an id outside
    [0, E) is an empty slot): out bf16 [T, H]."""
    _row_count(ids, "ids")
    k = ids.shape[1]
    T, ldx, out, ldo, workspace = _moe_buffers(x, experts, k, out, workspace)
    dev = experts.device
    _check(lib.ck_moe_experts_w4a16(x.data_ptr(), T, experts.H, ldx, _flat(ids, "ids", torch.int32, dev, (T, k)),
                                    _flat(weights, "weights", torch.float32, dev, (T, k)), k, *experts._args(),
                                    out.data_ptr(), ldo, workspace.data_ptr(), workspace.numel(), _stream(x)))
    return out


class LoraAdapters:
    """L slots of low-rank adapters of up to R ranks: a bf16 [L, R, K], b bf16 [L, N, R],
    scaling fp32 [L] or None (1), ranks int32 [L] or None (R); what a slot holds beyond its
    rank is not used.  The tensors' storages are kept, not copied, as in MoeExperts."""

    def __init__(self, a, b, scaling=None, ranks=None):
        if not isinstance(a, torch.Tensor) or a.dim() != 3 or not isinstance(b, torch.Tensor) or b.dim() != 3:
            raise ValueError("a and b must be 3-D tensors")
        (L, R, K), N = a.shape, b.shape[1]
        _dense(a, "a", torch.bfloat16, (L, R, K))
        _dense(b, "b", torch.bfloat16, (L, N, R))
        if scaling is not None:
            _dense(scaling, "scaling", torch.float32, (L,))
        if ranks is not None:
            _dense(ranks, "ranks", torch.int32, (L,))
        _same_device(a, ("b", b), ("scaling", scaling), ("ranks", ranks))
        self.tensors, self._at = _held((a, b, scaling, ranks))
        self.L, self.R, self.K, self.N, self.device = L, R, K, N, a.device

    def _args(self):
        a, b, scaling, ranks = self._at
        at = (self.L, self.R, a(), b(), scaling(), ranks(), self.N)
        if 0 in at:
            raise ValueError("adapters: no slots, or a tensor has no storage any more")
        return at


def lora_workspace_bytes(M: int, K: int, R: int, L: int) -> int:
    """Workspace bytes of lora_add for M rows of K columns and L adapters of up to R ranks."""
    return int(lib.ck_lora_workspace_bytes(M, K, R, L))


def lora_add(x, adapters: LoraAdapters, index, base=None, out=None, workspace=None):
    """bf16 [M, N]: base[m] + scaling[l] B_l (A_l x[m]) with l = index[m] (int32 [M]), and base[m]
    where l is outside [0, L).  base None: zeros; out may be base (in place)."""
    M, dev = _row_count(x, "x"), adapters.device
    ldx = _rows(x, "x", torch.bfloat16, dev, (M, adapters.K))
    shape = (M, adapters.N)
    out = torch.empty(shape, dtype=torch.bfloat16, device=dev) if out is None else out
    ldo = _rows(out, "out", torch.bfloat16, dev, shape)
    ldb = ldo if base is None else _rows(base, "base", torch.bfloat16, dev, shape)
    workspace = _space(workspace, lib.ck_lora_workspace_bytes(M, adapters.K, adapters.R, adapters.L)
                       if workspace is None else 0, dev)
    _check(lib.ck_lora_add(x.data_ptr(), M, adapters.K, ldx, _flat(index, "index", torch.int32, dev, (M,)),
                           *adapters._args(), None if base is None else base.data_ptr(), ldb, out.data_ptr(), ldo,
                           workspace.data_ptr(), workspace.numel(), _stream(x)))
    return out


# ------------------------------------------------------ 8-bit float products
# e4m3 codes with power-of-two (e8m0) scales for each block of 128.  As above, the weights
# are checked once, when their handle is made.

E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def fp8_blocks(n: int) -> int:
    """Blocks of 128 in n columns or rows."""
    return -(-n // 128)


def fp8_empty(M: int, K: int, device):
    """Room for quantised activations: codes e4m3 [M, K] and scales e8m0 [M, ceil(K / 128)], whose
    rows lie a multiple of four bytes apart, as the products read them."""
    blocks = fp8_blocks(K)
    return (torch.empty((M, K), dtype=E4M3, device=device),
            torch.empty((M, -(-blocks // 4) * 4), dtype=E8M0, device=device)[:, :blocks])


def _fp8_scales(t, M, K, device):
    """Row stride of an activation's scales."""
    lds = _rows(t, "scales", E8M0, device, (M, fp8_blocks(K)))
    if M <= 1:
        lds = -(-lds // 4) * 4
    return lds


def fp8_quant(x, codes=None, scales=None):
    """(codes, scales) of bf16 x [M, K]: e4m3 [M, K] and, for each row and 128 columns, the smallest
    power of two s with |x| <= 448 s, e8m0 [M, ceil(K / 128)] (1 for zeros)."""
    M = _row_count(x, "x")
    K, dev = x.shape[1], x.device
    ldx = _rows(x, "x", torch.bfloat16, dev, (M, K))
    if not x.is_cuda:
        raise ValueError("x must be a GPU tensor")
    if codes is None or scales is None:
        room = fp8_empty(M, K, dev)
        codes, scales = room[0] if codes is None else codes, room[1] if scales is None else scales
    ldq = _rows(codes, "codes", E4M3, dev, (M, K))
    _check(lib.ck_fp8_quant(x.data_ptr(), M, K, ldx, codes.data_ptr(), ldq, scales.data_ptr(),
                            _fp8_scales(scales, M, K, dev), _stream(x)))
    return codes, scales


def fp8_quantize_weights(w, codes=None, scales=None):
    """(codes, scales) of a bf16 weight [N, K]: e4m3 [N, K] and e8m0 [ceil(N / 128), ceil(K / 128)],
    one scale for each 128 x 128 block."""
    N = _row_count(w, "w")
    K, dev = w.shape[1], w.device
    ldw = _rows(w, "w", torch.bfloat16, dev, (N, K))
    if not w.is_cuda:
        raise ValueError("w must be a GPU tensor")
    shape = (fp8_blocks(N), fp8_blocks(K))
    codes = torch.empty((N, K), dtype=E4M3, device=dev) if codes is None else codes
    scales = torch.empty(shape, dtype=E8M0, device=dev) if scales is None else scales
    ldc = _rows(codes, "codes", E4M3, dev, (N, K))
    _check(lib.ck_fp8_quantize_weights(w.data_ptr(), N, K, ldw, codes.data_ptr(), ldc,
                                       _flat(scales, "scales", E8M0, dev, shape), _stream(w)))
    return codes, scales


def _fp8_transpose(codes, scales):
    N, K = codes.shape
    codes_t = torch.empty((K, N), dtype=E4M3, device=codes.device)
    scales_t = torch.empty((fp8_blocks(K), fp8_blocks(N)), dtype=E8M0, device=codes.device)
    _check(lib.ck_fp8_transpose_weights(codes.data_ptr(), _ld(codes), scales.data_ptr(), N, K, codes_t.data_ptr(),
                                        _ld(codes_t), scales_t.data_ptr(), _stream(codes)))
    return codes_t, scales_t


class Fp8Weights:
    """An 8-bit float weight: codes e4m3 [N, K] (rows may be strided), scales e8m0 [ceil(N / 128),
    ceil(K / 128)].  The tensors' storages are kept, not copied, as in MoeExperts."""

    def __init__(self, codes, scales):
        _matrix(codes, "codes", (E4M3,))
        self.N, self.K = codes.shape
        if not self.N or not self.K or self.N % 16 or self.K % 16:
            raise ValueError("codes has shape %s: expected multiples of 16" % (tuple(codes.shape),))
        _dense(scales, "scales", E8M0, (fp8_blocks(self.N), fp8_blocks(self.K)))
        _same_device(codes, ("scales", scales))
        self.tensors, self._at = _held((codes, scales))
        self.device, self._ldw = codes.device, _ld(codes)

    def transposed(self):
        """The transposed weight, laid out anew: the linear's backward pass to its input is the
        linear of it."""
        return Fp8Weights(*_fp8_transpose(*self.tensors))

    def _args(self):
        codes, scales = self._at
        at = (codes(), self._ldw, scales(), self.N)
        if 0 in at:
            raise ValueError("weights: none, or a tensor has no storage any more")
        return at


def _fp8_result(out, name, M, N, device):
    out = torch.empty((M, N), dtype=torch.bfloat16, device=device) if out is None else out
    return out, _rows(out, name, torch.bfloat16, device, (M, N))


def fp8_gemm(codes, scales, weights: Fp8Weights, bias=None, out=None):
    """bf16 [M, N] of quantised activations and a weight, plus bias bf16 [N].  Rows of scales lie a
    multiple of four bytes apart, as fp8_quant and fp8_empty lay them out (.contiguous() undoes it).
    K is not split over workgroups, as fp8_linear does where rows are some hundred and K is long."""
    M, dev = _row_count(codes, "codes"), weights.device
    ldq = _rows(codes, "codes", E4M3, dev, (M, weights.K))
    lds = _fp8_scales(scales, M, weights.K, dev)
    # The last row's bytes up to the next multiple of four are read.
    end = scales.storage_offset() + max(M - 1, 0) * lds + -(-fp8_blocks(weights.K) // 4) * 4
    if M and end > scales.untyped_storage().nbytes():
        raise ValueError("scales: a row of %d blocks needs room up to a multiple of four (fp8_empty)"
                         % fp8_blocks(weights.K))
    out, ldo = _fp8_result(out, "out", M, weights.N, dev)
    _check(lib.ck_fp8_gemm(codes.data_ptr(), ldq, scales.data_ptr(), lds, M, weights.K, *weights._args(),
                           None if bias is None else _flat(bias, "bias", torch.bfloat16, dev, (weights.N,)),
                           out.data_ptr(), ldo, _stream(codes)))
    return out


def fp8_linear_workspace_bytes(M: int, K: int, N: int) -> int:
    """Workspace bytes of fp8_linear for M rows, K columns and N outputs."""
    return int(lib.ck_fp8_linear_workspace_bytes(M, K, N))


def fp8_linear(x, weights: Fp8Weights, bias=None, out=None, workspace=None):
    """Whole linear, bf16 [M, N]: quantises bf16 x [M, K] as fp8_quant and multiplies as fp8_gemm."""
    M, dev = _row_count(x, "x"), weights.device
    ldx = _rows(x, "x", torch.bfloat16, dev, (M, weights.K))
    out, ldo = _fp8_result(out, "out", M, weights.N, dev)
    workspace = _space(workspace, lib.ck_fp8_linear_workspace_bytes(M, weights.K, weights.N)
                       if workspace is None else 0, dev)
    _check(lib.ck_fp8_linear(x.data_ptr(), M, weights.K, ldx, *weights._args(),
                             None if bias is None else _flat(bias, "bias", torch.bfloat16, dev, (weights.N,)),
                             out.data_ptr(), ldo, workspace.data_ptr(), workspace.numel(), _stream(x)))
    return out


class _Fp8Pair:
    """Two dense weights of a feed-forward block, whose shapes are checked."""

    def _keep(self, w1, s1, w2, s2, shape1, shape2):
        for name, w, s, (rows, columns) in (("1", w1, s1, shape1), ("2", w2, s2, shape2)):
            _dense(w, "w" + name, E4M3, (rows, columns))
            _dense(s, "s" + name, E8M0, (fp8_blocks(rows), fp8_blocks(columns)))
        _same_device(w1, ("s1", s1), ("w2", w2), ("s2", s2))
        self.tensors, self._at = _held((w1, s1, w2, s2))
        self.device = w1.device

    def _args(self):
        at = tuple(address() for address in self._at)
        if 0 in at:
            raise ValueError("feed-forward weights: a tensor has no storage any more")
        return at


def _fp8_matrix(t, name):
    if not isinstance(t, torch.Tensor) or t.dim() != 2 or not t.shape[0] or not t.shape[1]:
        raise ValueError("%s must be a 2-D tensor" % name)
    return t.shape


class Fp8Ffn(_Fp8Pair):
    """The weights of a gated feed-forward block: w1 e4m3 [2I, H] (I gate rows, then I up rows),
    w2 e4m3 [H, I], their e8m0 scales of 128 x 128 blocks; I a multiple of 128.  The tensors'
    storages are kept, not copied, as in MoeExperts."""

    def __init__(self, w1, s1, w2, s2):
        rows, self.H = _fp8_matrix(w1, "w1")
        self.I = rows // 2
        if rows % 256 or self.H % 16:
            raise ValueError("w1 has shape (%d, %d): expected 2I, I a multiple of 128, by H, a multiple of 16"
                             % (rows, self.H))
        self._keep(w1, s1, w2, s2, (rows, self.H), (self.H, self.I))

    def transposed(self):
        """The transposed weights, laid out anew, which fp8_ffn_backward takes."""
        w1, s1, w2, s2 = self.tensors
        return Fp8FfnTransposed(*_fp8_transpose(w1, s1), *_fp8_transpose(w2, s2))


class Fp8FfnTransposed(_Fp8Pair):
    """The transposed weights of an Fp8Ffn: w1t e4m3 [H, 2I], w2t e4m3 [I, H] and their scales."""

    def __init__(self, w1t, s1t, w2t, s2t):
        self.I, self.H = _fp8_matrix(w2t, "w2t")
        if self.I % 128 or self.H % 16:
            raise ValueError("w2t has shape (%d, %d): expected multiples of 128 and of 16" % (self.I, self.H))
        self._keep(w1t, s1t, w2t, s2t, (self.H, 2 * self.I), (self.I, self.H))


def fp8_ffn_workspace_bytes(M: int, H: int, I: int) -> int:
    """Workspace bytes of fp8_ffn for M rows, H columns and inner width I."""
    return int(lib.ck_fp8_ffn_workspace_bytes(M, H, I))


def fp8_ffn_backward_workspace_bytes(M: int, H: int, I: int) -> int:
    """Workspace bytes of fp8_ffn_backward."""
    return int(lib.ck_fp8_ffn_backward_workspace_bytes(M, H, I))


def fp8_ffn(x, ffn: Fp8Ffn, out=None, gate_up=None, workspace=None):
    """Gated feed-forward block, bf16 [M, H]: W2 Q(silu(g) u) with [g; u] = W1 Q(x), Q the quantiser
    of fp8_quant.  gate_up bf16 [M, 2I], if given, receives g and u for fp8_ffn_backward."""
    M, dev = _row_count(x, "x"), ffn.device
    ldx = _rows(x, "x", torch.bfloat16, dev, (M, ffn.H))
    out, ldo = _fp8_result(out, "out", M, ffn.H, dev)
    ldg = 0 if gate_up is None else _rows(gate_up, "gate_up", torch.bfloat16, dev, (M, 2 * ffn.I))
    workspace = _space(workspace, lib.ck_fp8_ffn_workspace_bytes(M, ffn.H, ffn.I) if workspace is None else 0, dev)
    _check(lib.ck_fp8_ffn(x.data_ptr(), M, ffn.H, ldx, ffn.I, *ffn._args(), out.data_ptr(), ldo,
                          None if gate_up is None else gate_up.data_ptr(), ldg, workspace.data_ptr(),
                          workspace.numel(), _stream(x)))
    return out


def fp8_ffn_backward(dy, gate_up, ffn: Fp8FfnTransposed, dx=None, workspace=None):
    """The gradient bf16 [M, H] of fp8_ffn's input from its output's, dy bf16 [M, H], the gate_up
    that it kept and the transposed weights (the weights are frozen)."""
    M, dev = _row_count(dy, "dy"), ffn.device
    ldy = _rows(dy, "dy", torch.bfloat16, dev, (M, ffn.H))
    ldg = _rows(gate_up, "gate_up", torch.bfloat16, dev, (M, 2 * ffn.I))
    dx, lddx = _fp8_result(dx, "dx", M, ffn.H, dev)
    workspace = _space(workspace, lib.ck_fp8_ffn_backward_workspace_bytes(M, ffn.H, ffn.I)
                       if workspace is None else 0, dev)
    _check(lib.ck_fp8_ffn_backward(dy.data_ptr(), M, ffn.H, ldy, gate_up.data_ptr(), ldg, ffn.I, *ffn._args(),
                                   dx.data_ptr(), lddx, workspace.data_ptr(), workspace.numel(), _stream(dy)))
    return dx
