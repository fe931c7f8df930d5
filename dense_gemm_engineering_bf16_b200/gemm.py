"""ctypes binding of the C ABI in ``include/b200gemm.h``.

Argument marshalling only: tensors become device pointers, streams become
``cudaStream_t`` handles, and a non-OK status becomes ``GemmError``.  Every
step of the computation runs in the library's kernels.  Importing this module
without the built library raises -- there is no fallback.
"""
from __future__ import annotations

import ctypes
import os
import struct

PKG = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(PKG, "libb200gemm.so")

if not os.path.exists(library_path):
    raise ImportError(
        f"{library_path} is missing: build it with "
        "`python -m dense_gemm_engineering_bf16_b200.build` (nvcc, sm_100a)")

lib = ctypes.CDLL(library_path)

OUT_F32 = 0
OUT_BF16 = 1
KMAJOR = 0      # A as M x K, B as N x K
MNMAJOR = 1     # A as K x M, B as K x N (row-major K x N)
FP4_MX = 0      # blocks of 32, E8M0 scales
FP4_NV = 1      # blocks of 16, E4M3 scales, one fp32 scale of the matrix
ACT_NONE = 0
ACT_RELU = 1
ACT_GELU = 2
ACT_GELU_TANH = 3

CONFIGS = {
    "auto": 0,
    "1cta_128x256": 1,
    "1cta_128x128": 2,
    "2cta_256x256": 3,
    "skinny": 4,
    "2cta_256x256_clc": 5,
    "1cta_128x256_clc": 6,
    "mxfp8_1cta_128x256": 7,
    "mxfp8_2cta_256x256": 8,
    "2cta_512x256_clc": 9,
    "2cta_256x256_sk": 10,
    "2cta_256x224": 11,
    "1cta_128x128_splitk": 12,
    "1cta_128x256_splitk": 13,
    "small": 14,
}

STATUS_NAMES = {
    0: "GEMM_OK", 1: "GEMM_ERR_INVALID_VALUE", 2: "GEMM_ERR_MISALIGNED", 3: "GEMM_ERR_ALIAS",
    4: "GEMM_ERR_UNSUPPORTED_DEVICE", 5: "GEMM_ERR_LAUNCH", 6: "GEMM_ERR_TIMEOUT",
    7: "GEMM_ERR_TOO_LARGE", 8: "GEMM_ERR_CAPTURE",
}

_i64 = ctypes.c_int64
_vp = ctypes.c_void_p
_int = ctypes.c_int

lib.gemm_bf16.argtypes = [_vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _i64, _int, _vp]
lib.gemm_bf16.restype = _int
lib.gemm_bf16_noalloc.argtypes = [_vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _i64, _int, _vp]
lib.gemm_bf16_noalloc.restype = _int
lib.gemm_bf16_ex.argtypes = [_vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _i64, _int, _int, _int,
                             ctypes.c_float, ctypes.c_float, _vp]
lib.gemm_bf16_ex.restype = _int
lib.gemm_bf16_fused.argtypes = [_vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _i64, _int, _int, _int,
                                ctypes.c_float, ctypes.c_float, _vp, _int, _vp]
lib.gemm_bf16_fused.restype = _int
lib.gemm_bf16_allgather.argtypes = [_vp, _vp, ctypes.POINTER(_vp), _int, _i64, _i64, _i64, _i64, _i64, _i64,
                                    _i64, _int, _vp]
lib.gemm_bf16_allgather.restype = _int
lib.gemm_mxfp8.argtypes = [_vp, _vp, _vp, _vp, _vp, _i64, _i64, _i64, _i64, _i64, _i64, _vp]
lib.gemm_mxfp8.restype = _int
lib.gemm_rmsnorm.argtypes = [_vp] * 8 + [_i64] * 7 + [_int, _int, ctypes.c_float, _vp]
lib.gemm_rmsnorm.restype = _int
lib.gemm_rmsnorm_backward.argtypes = [_vp] * 8 + [_i64] * 7 + [_int, _int, _int, _vp]
lib.gemm_rmsnorm_backward.restype = _int
lib.gemm_rmsnorm_backward_workspace.argtypes = [_i64, _i64]
lib.gemm_rmsnorm_backward_workspace.restype = _i64
lib.gemm_mxfp8_quantize.argtypes = [_vp, _vp, _vp, _i64, _i64, _i64, _i64, _int, _int, _vp]
lib.gemm_mxfp8_quantize.restype = _int
lib.gemm_bf16_w4.argtypes = [_vp] * 5 + [_i64] * 8 + [_int, _vp]
lib.gemm_bf16_w4.restype = _int
lib.gemm_bf16_grouped.argtypes = [_vp] * 4 + [_i64] * 8 + [_int, _int, _vp]
lib.gemm_bf16_grouped.restype = _int
lib.gemm_bf16_grouped_wgrad.argtypes = [_vp] * 4 + [_i64] * 8 + [_int, _int, ctypes.c_float, _vp]
lib.gemm_bf16_grouped_wgrad.restype = _int
lib.gemm_call.argtypes = [_int, ctypes.c_char_p]
lib.gemm_call.restype = _int
lib.gemm_fp4_scale_bytes.argtypes = [_i64, _i64, _int]
lib.gemm_fp4_scale_bytes.restype = _i64
lib.gemm_fp4_quantize.argtypes = [_vp] * 4 + [_i64] * 4 + [_int, _int, _int, _vp]
lib.gemm_fp4_quantize.restype = _int
lib.gemm_fp4.argtypes = [_vp] * 7 + [_i64] * 6 + [_int, _int, _vp]
lib.gemm_fp4.restype = _int
lib.gemm_check_device_status.argtypes = [_vp]
lib.gemm_check_device_status.restype = _int
lib.gemm_last_timeout_detail.argtypes = [ctypes.POINTER(ctypes.c_int32), ctypes.POINTER(ctypes.c_int32)]
lib.gemm_last_timeout_detail.restype = None
lib.gemm_status_string.argtypes = [_int]
lib.gemm_status_string.restype = ctypes.c_char_p
lib.gemm_last_cuda_error.argtypes = []
lib.gemm_last_cuda_error.restype = _int
lib.gemm_force_config.argtypes = [_int]
lib.gemm_force_config.restype = _int
lib.gemm_select_config.argtypes = [_i64, _i64, _i64]
lib.gemm_select_config.restype = _int
lib.gemm_launches_per_call.argtypes = [_i64, _i64, _i64, _int]
lib.gemm_launches_per_call.restype = _int


class GemmError(RuntimeError):
    def __init__(self, status: int, where: str = ""):
        self.status = int(status)
        msg = gemm_status_string(self.status)
        if self.status == 5:
            msg += f" (CUDA error {lib.gemm_last_cuda_error()})"
        super().__init__(f"{where}: {msg}" if where else msg)


def gemm_status_string(status: int) -> str:
    return lib.gemm_status_string(int(status)).decode()


def _ptr(x) -> int:
    if x is None:
        return 0
    if isinstance(x, int):
        return x
    return int(x.data_ptr())


def _stream(s) -> int:
    if s is None:
        import torch
        return int(torch.cuda.current_stream().cuda_stream)
    if isinstance(s, int):
        return s
    return int(s.cuda_stream)


def _check(status: int, where: str, check: bool) -> int:
    if check and status != 0:
        raise GemmError(status, where)
    return status


def gemm_bf16(A, B, C, M: int, N: int, K: int, lda: int, ldb: int, ldc: int,
              c_type: int = OUT_F32, stream=None, check: bool = True) -> int:
    """C = A.B (bf16 A row-major M x K, bf16 B stored N x K, C M x N of c_type).

    A, B, C: torch tensors (device) or raw device pointers; stream: a
    torch.cuda.Stream, a raw handle, or None for torch's current stream.
    """
    st = lib.gemm_bf16(_ptr(A), _ptr(B), _ptr(C), M, N, K, lda, ldb, ldc, int(c_type), _stream(stream))
    return _check(st, "gemm_bf16", check)


def gemm_bf16_ex(A, B, C, M: int, N: int, K: int, lda: int, ldb: int, ldc: int,
                 c_type: int = OUT_F32, a_layout: int = KMAJOR, b_layout: int = KMAJOR,
                 alpha: float = 1.0, beta: float = 0.0, stream=None, check: bool = True) -> int:
    """C = alpha * A.B + beta * C with K-major or MN-major operands
    (see include/b200gemm.h, gemm_bf16_ex)."""
    st = lib.gemm_bf16_ex(_ptr(A), _ptr(B), _ptr(C), M, N, K, lda, ldb, ldc, int(c_type), int(a_layout),
                          int(b_layout), float(alpha), float(beta), _stream(stream))
    return _check(st, "gemm_bf16_ex", check)


def gemm_bf16_fused(A, B, C, M: int, N: int, K: int, lda: int, ldb: int, ldc: int,
                    c_type: int = OUT_F32, a_layout: int = KMAJOR, b_layout: int = KMAJOR,
                    alpha: float = 1.0, beta: float = 0.0, bias=None, act: int = ACT_NONE,
                    stream=None, check: bool = True) -> int:
    """C = act(alpha * A.B + beta * C + bias) with bias one fp32 value per
    column of C, fused into the GEMM's write-back (see include/b200gemm.h,
    gemm_bf16_fused)."""
    st = lib.gemm_bf16_fused(_ptr(A), _ptr(B), _ptr(C), M, N, K, lda, ldb, ldc, int(c_type), int(a_layout),
                             int(b_layout), float(alpha), float(beta), _ptr(bias) if bias is not None else None,
                             int(act), _stream(stream))
    return _check(st, "gemm_bf16_fused", check)


def gemm_bf16_allgather(A, B, C_dst, M: int, N: int, K: int, lda: int, ldb: int, ldc: int, row0: int,
                        c_type: int = OUT_F32, stream=None, check: bool = True) -> int:
    """This GPU's slab C[row0:row0+M] = A.B written into every C of C_dst
    (this GPU's own C first, then other GPUs' mapped C buffers): a row-
    sharded GEMM with its all-gather in the write-back (see
    include/b200gemm.h, gemm_bf16_allgather)."""
    ptrs = (_vp * len(C_dst))(*[_ptr(c) for c in C_dst])
    st = lib.gemm_bf16_allgather(_ptr(A), _ptr(B), ptrs, len(C_dst), M, N, K, lda, ldb, ldc, row0, int(c_type),
                                 _stream(stream))
    return _check(st, "gemm_bf16_allgather", check)


def gemm_mxfp8(A, sfa, B, sfb, C, M: int, N: int, K: int, lda: int, ldb: int, ldc: int,
               stream=None, check: bool = True) -> int:
    """Block-scaled C = (sa.A).(sb.B): E4M3 A (M x lda bytes), E4M3 B stored
    N x ldb, E8M0 scales sfa (M x K/32) and sfb (N x K/32), bf16 C (M x ldc)."""
    st = lib.gemm_mxfp8(_ptr(A), _ptr(sfa), _ptr(B), _ptr(sfb), _ptr(C), M, N, K, lda, ldb, ldc,
                        _stream(stream))
    return _check(st, "gemm_mxfp8", check)


def gemm_bf16_noalloc(A, B, C, M: int, N: int, K: int, lda: int, ldb: int, ldc: int,
                      c_type: int = OUT_F32, stream=None, check: bool = True) -> int:
    """gemm_bf16 without any device allocation: the kernels' scratch is a
    static array inside the library (see include/b200gemm.h)."""
    st = lib.gemm_bf16_noalloc(_ptr(A), _ptr(B), _ptr(C), M, N, K, lda, ldb, ldc, int(c_type),
                               _stream(stream))
    return _check(st, "gemm_bf16_noalloc", check)


# The dtypes that an operand's tensor may have, by gemm_out_t (and for the byte
# formats); filled on first use, so that importing this module does not import
# torch.
_DTYPES: dict = {}


def _here(stream):
    """The current device (None: not asked for yet) and the call's stream
    handle.  Without a stream it is the device's current one, asked for
    without building a Stream object, which would cost more than the launch;
    where torch lacks those two functions its public ones answer."""
    if not _DTYPES:
        import torch
        device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        queue = getattr(torch._C, "_cuda_getCurrentRawStream",
                        lambda dev: torch.cuda.current_stream(dev).cuda_stream)
        _DTYPES.update({OUT_F32: (torch.float32,), OUT_BF16: (torch.bfloat16,), "bytes": (torch.uint8,),
                        "ints": (torch.int32,),
                        "fp4": (torch.uint8,) + ((torch.float4_e2m1fn_x2,) if hasattr(torch, "float4_e2m1fn_x2") else ()),
                        FP4_MX + 2: (torch.float8_e8m0fnu, torch.uint8),
                        FP4_NV + 2: (torch.float8_e4m3fn, torch.uint8),
                        "codes": (torch.float8_e4m3fn, torch.uint8), "scales": (torch.float8_e8m0fnu, torch.uint8),
                        "device": device, "stream": queue})
    if stream is not None:
        return None, _stream(stream)
    dev = _device()
    return dev, _DTYPES["stream"](dev)


def _device() -> int:
    """The current device; without CUDA, in the driver or in this torch, the
    library's own status for that."""
    try:
        return _DTYPES["device"]()
    except (AssertionError, RuntimeError) as e:
        raise GemmError(4, str(e).split(".")[0]) from e


def _operand(x, kind, dev, what: str, packed: bool = False):
    """Device pointer of an operand: None, a raw pointer, or a tensor, which
    has to be on the current device (whose stream the call runs on) and to
    hold the type that the call reads there.  packed: the call has no pitch for
    it (vectors, scales, a workspace), so the tensor must be contiguous."""
    if x is None or type(x) is int:
        return x
    if dev is None:
        dev = _device()
    if x.get_device() != dev:
        raise GemmError(1, f"{what} is on {x.device}, the call runs on cuda:{dev}")
    if kind is not None and x.dtype not in _DTYPES.get(kind, ()):
        raise GemmError(1, f"{what} is {x.dtype}")
    if packed and not x.is_contiguous():
        raise GemmError(1, f"{what} is not contiguous")
    return x.data_ptr()


def _refused(e: GemmError, check: bool) -> int:
    """An operand that `_operand` refused: raised, or with check=False returned
    as its status, like the library's own refusals."""
    if check:
        raise e
    return e.status


def gemm_rmsnorm(X, R, H, weight, Y, Q, sf, rstd, M: int, K: int, ldx: int, ldr: int, ldh: int, ldy: int, ldq: int,
                 x_type: int = OUT_BF16, h_type: int = OUT_BF16, eps: float = 1e-5, stream=None,
                 check: bool = True) -> int:
    """h = X + R (stored to H), y = h / rms(h) * weight, written as bf16 to Y
    and / or as MXFP8 codes and scales to Q and sf; 1 / rms to rstd.  R, H, Y,
    Q with sf, and rstd may be None (see include/b200gemm.h, gemm_rmsnorm)."""
    try:
        dev, queue = _here(stream)
        st = lib.gemm_rmsnorm(_operand(X, x_type, dev, "gemm_rmsnorm: X"), _operand(R, h_type, dev, "gemm_rmsnorm: R"),
                              _operand(H, h_type, dev, "gemm_rmsnorm: H"),
                              _operand(weight, OUT_F32, dev, "gemm_rmsnorm: weight", True),
                              _operand(Y, OUT_BF16, dev, "gemm_rmsnorm: Y"),
                              _operand(Q, "codes", dev, "gemm_rmsnorm: Q"),
                              _operand(sf, "scales", dev, "gemm_rmsnorm: sf", True),
                              _operand(rstd, OUT_F32, dev, "gemm_rmsnorm: rstd", True), M, K, ldx, ldr, ldh, ldy, ldq,
                              int(x_type), int(h_type), eps, queue)
    except GemmError as e:
        return _refused(e, check)
    return _check(st, "gemm_rmsnorm", check)


def gemm_rmsnorm_backward_workspace(M: int, K: int) -> int:
    """Bytes of workspace that gemm_rmsnorm_backward needs for a dW."""
    return int(lib.gemm_rmsnorm_backward_workspace(M, K))


def gemm_rmsnorm_backward(dY, H, weight, rstd, dR, dH, dW, workspace, M: int, K: int, lddy: int, ldh: int, lddr: int,
                          lddh: int, dy_type: int = OUT_BF16, h_type: int = OUT_BF16, dh_type: int = OUT_BF16,
                          workspace_bytes: int | None = None, stream=None, check: bool = True) -> int:
    """Gradients of gemm_rmsnorm: dH (of X and of R alike, dR added) and dW.
    dR may be None; dW with workspace may be None (see include/b200gemm.h,
    gemm_rmsnorm_backward).  workspace_bytes: needed where workspace is a raw
    pointer; a tensor's own size otherwise."""
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None or isinstance(workspace, int) else \
            workspace.numel() * workspace.element_size()
    try:
        dev, queue = _here(stream)
        st = lib.gemm_rmsnorm_backward(
            _operand(dY, dy_type, dev, "gemm_rmsnorm_backward: dY"),
            _operand(H, h_type, dev, "gemm_rmsnorm_backward: H"),
            _operand(weight, OUT_F32, dev, "gemm_rmsnorm_backward: weight", True),
            _operand(rstd, OUT_F32, dev, "gemm_rmsnorm_backward: rstd", True),
            _operand(dR, dh_type, dev, "gemm_rmsnorm_backward: dR"),
            _operand(dH, dh_type, dev, "gemm_rmsnorm_backward: dH"),
            _operand(dW, OUT_F32, dev, "gemm_rmsnorm_backward: dW", True),
            _operand(workspace, None, dev, "gemm_rmsnorm_backward: workspace", True), workspace_bytes, M, K, lddy, ldh,
            lddr, lddh, int(dy_type), int(h_type), int(dh_type), queue)
    except GemmError as e:
        return _refused(e, check)
    return _check(st, "gemm_rmsnorm_backward", check)


def gemm_mxfp8_quantize(X, Q, sf, M: int, K: int, ldx: int, ldq: int, x_type: int = OUT_BF16, layout: int = KMAJOR,
                        stream=None, check: bool = True) -> int:
    """E4M3 codes Q (M x ldq) and E8M0 scales sf (M x K/32) of X, stored M x K
    (KMAJOR) or K x M (MNMAJOR): an operand of gemm_mxfp8."""
    try:
        dev, queue = _here(stream)
        st = lib.gemm_mxfp8_quantize(_operand(X, x_type, dev, "gemm_mxfp8_quantize: X"),
                                     _operand(Q, "codes", dev, "gemm_mxfp8_quantize: Q"),
                                     _operand(sf, "scales", dev, "gemm_mxfp8_quantize: sf", True), M, K, ldx, ldq,
                                     int(x_type), int(layout), queue)
    except GemmError as e:
        return _refused(e, check)
    return _check(st, "gemm_mxfp8_quantize", check)


def gemm_bf16_w4(A, B, scales, zeros, C, M: int, N: int, K: int, lda: int, ldb: int, lds: int, ldc: int, group: int,
                 c_type: int = OUT_F32, stream=None, check: bool = True) -> int:
    """C = A.W^T with W[j][k] = scales[j][k/group] (q[j][k] - zeros[j][k/group]):
    bf16 A (M x K), 4-bit codes B (N x ldb bytes, two each, even k in the low
    half), bf16 scales and byte zeros (N x lds; zeros None: 8), C M x N."""
    try:
        dev, queue = _here(stream)
        st = lib.gemm_bf16_w4(_operand(A, OUT_BF16, dev, "gemm_bf16_w4: A"),
                              _operand(B, "bytes", dev, "gemm_bf16_w4: B"),
                              _operand(scales, OUT_BF16, dev, "gemm_bf16_w4: scales"),
                              _operand(zeros, "bytes", dev, "gemm_bf16_w4: zeros"),
                              _operand(C, c_type, dev, "gemm_bf16_w4: C"), M, N, K, lda, ldb, lds, ldc, group,
                              int(c_type), queue)
    except GemmError as e:
        return _refused(e, check)
    return _check(st, "gemm_bf16_w4", check)


# The arguments of the entry points below as gemm_call's words: ctypes takes 0.1
# us an argument, these blocks of 12 to 16 a third of a microsecond.
_GROUPED, _WGRAD, _QUANTIZE, _FP4 = (struct.Struct(f).pack for f in ("<15q", "<14qf4xq", "<12q", "<16q"))


def _call(entry: int, pack, *words) -> int:
    try:
        return lib.gemm_call(entry, pack(*words))
    except (struct.error, OverflowError, TypeError) as e:       # no number, or none that a word or an fp32 holds
        raise GemmError(1, str(e)) from e


def gemm_bf16_grouped(A, B, ends, C, groups: int, M: int, N: int, K: int, lda: int, ldb: int, strideb: int, ldc: int,
                      c_type: int = OUT_F32, b_layout: int = KMAJOR, stream=None, check: bool = True) -> int:
    """C[r] = A[r].B_e for the rows r of every expert e: bf16 A (M x K, rows
    sorted by expert), `groups` bf16 matrices B (N x K each, or K x N with
    MNMAJOR) strideb elements apart, int32 ends[e] where expert e's rows end
    (on the device), C M x N; rows of no expert are left as they are (see
    include/b200gemm.h, gemm_bf16_grouped)."""
    try:
        dev, queue = _here(stream)
        st = _call(0, _GROUPED, _operand(A, OUT_BF16, dev, "gemm_bf16_grouped: A") or 0,
                   _operand(B, OUT_BF16, dev, "gemm_bf16_grouped: B") or 0,
                   _operand(ends, "ints", dev, "gemm_bf16_grouped: ends", True) or 0,
                   _operand(C, c_type, dev, "gemm_bf16_grouped: C") or 0, groups, M, N, K, lda, ldb, strideb, ldc, c_type,
                   b_layout, queue)
    except GemmError as e:
        return _refused(e, check)
    return _check(st, "gemm_bf16_grouped", check)


def gemm_bf16_grouped_wgrad(dC, A, ends, dB, groups: int, M: int, N: int, K: int, lddc: int, lda: int, lddb: int,
                            stridedb: int, db_type: int = OUT_F32, db_layout: int = KMAJOR, beta: float = 0.0,
                            stream=None, check: bool = True) -> int:
    """dB_e = beta dB_e + dC_e^T.A_e, the gradient of gemm_bf16_grouped's B_e:
    bf16 dC (M x N) and A (M x K), `groups` matrices dB (N x K each, or K x N
    with MNMAJOR) stridedb elements apart (see include/b200gemm.h,
    gemm_bf16_grouped_wgrad)."""
    try:
        dev, queue = _here(stream)
        st = _call(1, _WGRAD, _operand(dC, OUT_BF16, dev, "gemm_bf16_grouped_wgrad: dC") or 0,
                   _operand(A, OUT_BF16, dev, "gemm_bf16_grouped_wgrad: A") or 0,
                   _operand(ends, "ints", dev, "gemm_bf16_grouped_wgrad: ends", True) or 0,
                   _operand(dB, db_type, dev, "gemm_bf16_grouped_wgrad: dB") or 0, groups, M, N, K, lddc, lda, lddb,
                   stridedb, db_type, db_layout, beta, queue)
    except GemmError as e:
        return _refused(e, check)
    return _check(st, "gemm_bf16_grouped_wgrad", check)


def gemm_fp4_scale_bytes(rows: int, K: int, format: int) -> int:
    """Bytes of the tiled scales of a rows x K matrix in 4 bits."""
    return int(lib.gemm_fp4_scale_bytes(rows, K, int(format)))


def gemm_fp4_quantize(X, scale, Q, sf, M: int, K: int, ldx: int, ldq: int, format: int = FP4_NV, x_type: int = OUT_BF16,
                      layout: int = KMAJOR, stream=None, check: bool = True) -> int:
    """E2M1 codes Q (M x ldq bytes, two each, even k in the low half) and tiled
    scales sf (gemm_fp4_scale_bytes) of X, stored M x K (KMAJOR) or K x M
    (MNMAJOR): an operand of gemm_fp4.  scale: FP4_NV's scale of the matrix, one
    float on the device, or None (see include/b200gemm.h, gemm_fp4_quantize)."""
    try:
        dev, queue = _here(stream)
        st = _call(2, _QUANTIZE, _operand(X, x_type, dev, "gemm_fp4_quantize: X") or 0,
                   _operand(scale, OUT_F32, dev, "gemm_fp4_quantize: scale", True) or 0,
                   _operand(Q, "fp4", dev, "gemm_fp4_quantize: Q") or 0,
                   _operand(sf, format + 2, dev, "gemm_fp4_quantize: sf", True) or 0, M, K, ldx, ldq, format, x_type,
                   layout, queue)
    except GemmError as e:
        return _refused(e, check)
    return _check(st, "gemm_fp4_quantize", check)


def gemm_fp4(A, sfa, scale_a, B, sfb, scale_b, C, M: int, N: int, K: int, lda: int, ldb: int, ldc: int,
             format: int = FP4_NV, c_type: int = OUT_F32, stream=None, check: bool = True) -> int:
    """C = ga gb (sa.A).(sb.B)^T: E2M1 codes A (M x lda bytes) and B (N x ldb),
    tiled scales sfa and sfb, FP4_NV's scales of the matrices scale_a and
    scale_b (one float each on the device, or None), C M x N (see
    include/b200gemm.h, gemm_fp4)."""
    try:
        dev, queue = _here(stream)
        sf = format + 2
        st = _call(3, _FP4, _operand(A, "fp4", dev, "gemm_fp4: A") or 0, _operand(sfa, sf, dev, "gemm_fp4: sfa", True) or 0,
                   _operand(scale_a, OUT_F32, dev, "gemm_fp4: scale_a", True) or 0,
                   _operand(B, "fp4", dev, "gemm_fp4: B") or 0, _operand(sfb, sf, dev, "gemm_fp4: sfb", True) or 0,
                   _operand(scale_b, OUT_F32, dev, "gemm_fp4: scale_b", True) or 0,
                   _operand(C, c_type, dev, "gemm_fp4: C") or 0, M, N, K, lda, ldb, ldc, format, c_type, queue)
    except GemmError as e:
        return _refused(e, check)
    return _check(st, "gemm_fp4", check)


def gemm_check_device_status(stream=None, check: bool = True) -> int:
    st = lib.gemm_check_device_status(_stream(stream))
    return _check(st, "gemm_check_device_status", check)


def gemm_last_timeout_detail():
    w = ctypes.c_int32()
    b = ctypes.c_int32()
    lib.gemm_last_timeout_detail(ctypes.byref(w), ctypes.byref(b))
    return int(w.value), int(b.value)


def gemm_force_config(config) -> None:
    cid = CONFIGS[config] if isinstance(config, str) else int(config)
    _check(lib.gemm_force_config(cid), "gemm_force_config", True)


def gemm_select_config(M: int, N: int, K: int) -> int:
    return int(lib.gemm_select_config(M, N, K))


def gemm_launches_per_call(M: int, N: int, K: int, block_scaled: bool = False) -> int:
    return int(lib.gemm_launches_per_call(M, N, K, int(bool(block_scaled))))
