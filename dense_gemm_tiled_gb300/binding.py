"""Thin Python binding over libgemm_gb300.so (include/gemm.h).

Argument marshalling only: every step of the GEMM runs in the library's
kernels.  PyTorch supplies device memory and the current CUDA stream.  If the
library has not been built this module raises ImportError; there is no
fallback implementation.
"""
import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgemm_gb300.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(
        f"{LIB_PATH} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`"
        " or `python -m dense_gemm_tiled_gb300.build`")

_lib = ctypes.CDLL(LIB_PATH)

_i64, _int, _flt, _vp = ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_void_p
_GEMM_ARGS = [_int, _int, _i64, _i64, _i64, _int, _flt, _flt, _vp, _i64, _vp, _i64, _vp, _i64,
              _vp]
_lib.gemm.argtypes = _GEMM_ARGS
_lib.gemm.restype = _int
_lib.gemm_ex.argtypes = _GEMM_ARGS[:-1] + [_vp, _int, _vp]
_lib.gemm_ex.restype = _int
_lib.gemm_host.argtypes = _GEMM_ARGS
_lib.gemm_host.restype = _int
_lib.gemm_strided_batched.argtypes = [_int, _int, _i64, _i64, _i64, _int, _flt, _flt, _vp, _i64,
                                      _i64, _vp, _i64, _i64, _vp, _i64, _i64, _i64, _vp]
_lib.gemm_strided_batched.restype = _int
_lib.gemm_fused.argtypes = [_int, _int, _i64, _i64, _i64, _int, _flt, _vp, _i64, _vp, _i64, _vp,
                            _int, _flt, _vp, _i64, _vp, _i64, _vp, _i64, _vp]
_lib.gemm_fused.restype = _int
_lib.gemm_fused_backward.argtypes = [_int, _int, _i64, _i64, _i64, _int, _flt, _vp, _i64, _vp,
                                     _i64, _int, _vp, _i64, _vp, _i64, _vp, _vp]
_lib.gemm_fused_backward.restype = _int
_lib.gemm_grouped.argtypes = [_int, _i64, _i64, _i64, _i64, _vp, _int, _flt, _vp, _i64, _vp, _i64,
                              _i64, _vp, _int, _flt, _vp, _i64, _vp, _i64, _vp, _i64, _vp]
_lib.gemm_grouped.restype = _int
_lib.gemm_grouped_backward.argtypes = [_int, _i64, _i64, _i64, _i64, _vp, _int, _flt, _vp, _i64,
                                       _vp, _i64, _i64, _int, _vp, _i64, _vp, _i64, _vp, _vp]
_lib.gemm_grouped_backward.restype = _int
_lib.gemm_grouped_wgrad.argtypes = [_i64, _i64, _i64, _i64, _vp, _int, _flt, _flt, _vp, _i64, _vp,
                                    _i64, _vp, _i64, _i64, _vp]
_lib.gemm_grouped_wgrad.restype = _int
_lib.gemm_mx_row_bytes.argtypes = [_int, _i64]
_lib.gemm_mx_row_bytes.restype = _i64
_lib.gemm_mx_scale_bytes.argtypes = [_int, _i64, _i64]
_lib.gemm_mx_scale_bytes.restype = _i64
_lib.gemm_mx_quantize.argtypes = [_int, _int, _i64, _i64, _int, _flt, _vp, _i64, _int, _vp, _i64,
                                  _vp, _i64, _vp, _vp]
_lib.gemm_mx_quantize.restype = _int
_lib.gemm_mx_dequantize.argtypes = [_int, _i64, _i64, _vp, _i64, _vp, _int, _vp, _i64, _vp]
_lib.gemm_mx_dequantize.restype = _int
_lib.gemm_mx_act_backward.argtypes = [_i64, _i64, _int, _int, _vp, _i64, _vp, _i64, _vp, _vp,
                                      _i64, _vp, _vp]
_lib.gemm_mx_act_backward.restype = _int
_lib.gemm_mx4.argtypes = [_int, _i64, _i64, _i64, _int, _flt, _flt, _vp, _i64, _vp, _vp, _i64,
                          _vp, _vp, _i64, _vp, _int, _vp]
_lib.gemm_mx4.restype = _int
_lib.gemm_mx.argtypes = [_int, _int, _int, _i64, _i64, _i64, _int, _flt, _flt, _vp, _i64, _vp,
                         _i64, _vp, _vp, _i64, _vp, _int, _vp]
_lib.gemm_mx.restype = _int
_lib.gemm_check_device_status.argtypes = [_vp]
_lib.gemm_check_device_status.restype = _int
_lib.gemm_status_string.argtypes = [_int]
_lib.gemm_status_string.restype = ctypes.c_char_p
_lib.gemm_version.restype = _int
_lib.gemm_last_path.restype = _int
_lib.gemm_last_launches.restype = _int
_lib.gemm_last_grid.restype = _int
_lib.gemm_total_launches.restype = _i64
_lib.gemm_set_wait_timeout_ns.argtypes = [_i64]
_lib.gemm_set_wait_timeout_ns.restype = None
_lib.gemm_set_fault_injection.argtypes = [_int]
_lib.gemm_set_fault_injection.restype = None
_lib.gemm_set_kernel_events.argtypes = [_vp, _vp]
_lib.gemm_set_kernel_events.restype = None
_lib.gemm_scratch_high_water.argtypes = [_int]
_lib.gemm_scratch_high_water.restype = _i64

F32 = 0
F16_F32ACC = 1
BF16_F32ACC = 2
F32_TF32 = 3
F32_3XTF32 = 4
OK, ERR_INVALID_ARG, ERR_UNSUPPORTED, ERR_ALIAS, ERR_CUDA, ERR_NO_MEMORY, ERR_TIMEOUT = range(7)
PATHS = {0: "none", 1: "scale", 2: "ffma", 3: "ffma_splitk", 4: "tc", 5: "tc_splitk",
         6: "ffma_batched", 7: "tc_batched", 8: "per_entry", 9: "mx", 10: "mx_tc",
         11: "mx_stream", 12: "mx_convert", 13: "fused_tc", 14: "fused_ffma",
         15: "fused_stream"}


class GemmError(RuntimeError):
    def __init__(self, code: int):
        self.code = code
        super().__init__(status_string(code))


def status_string(code: int) -> str:
    return _lib.gemm_status_string(int(code)).decode()


def version() -> int:
    return _lib.gemm_version()


def last_path() -> str:
    return PATHS.get(_lib.gemm_last_path(), "unknown")


def last_launches() -> int:
    return _lib.gemm_last_launches()


def last_grid() -> int:
    return _lib.gemm_last_grid()


def total_launches() -> int:
    return _lib.gemm_total_launches()


def set_wait_timeout_ns(ns: int) -> None:
    _lib.gemm_set_wait_timeout_ns(int(ns))


def set_fault_injection(mode: int) -> None:
    _lib.gemm_set_fault_injection(int(mode))


def scratch_high_water(reset: bool = False) -> int:
    """Most bytes in use at once from the library's scratch pool on the
    current device since the last reset (0: none taken); reset=True then
    clears the mark."""
    return _lib.gemm_scratch_high_water(1 if reset else 0)


def set_kernel_events(start=None, end=None) -> None:
    """Brackets the main GEMM kernel of later calls on this thread with two
    torch.cuda.Event objects (each recorded once beforehand, so that its CUDA
    event exists); no arguments turns it off."""
    if start is None or end is None:
        _lib.gemm_set_kernel_events(None, None)
        return
    s, e = int(start.cuda_event), int(end.cuda_event)
    if not s or not e:
        raise ValueError("record each event once before passing it")
    _lib.gemm_set_kernel_events(s, e)


def gemm_raw(transA, transB, M, N, K, dtype, alpha, beta, A, lda, B, ldb, C, ldc,
             stream=0) -> int:
    """The C entry point with plain integers (device addresses, stream handle)."""
    return _lib.gemm(int(transA), int(transB), int(M), int(N), int(K), int(dtype), float(alpha),
                     float(beta), A or None, int(lda), B or None, int(ldb), C or None, int(ldc),
                     stream or None)


def gemm_ex_raw(transA, transB, M, N, K, dtype, alpha, beta, A, lda, B, ldb, C, ldc, bias, act,
                stream=0) -> int:
    """gemm_ex with plain integers (device addresses, act code)."""
    return _lib.gemm_ex(int(transA), int(transB), int(M), int(N), int(K), int(dtype),
                        float(alpha), float(beta), A or None, int(lda), B or None, int(ldb),
                        C or None, int(ldc), bias or None, int(act), stream or None)


def gemm_host_raw(transA, transB, M, N, K, dtype, alpha, beta, A, lda, B, ldb, C, ldc,
                  stream=0) -> int:
    """gemm_host with plain integers (host addresses)."""
    return _lib.gemm_host(int(transA), int(transB), int(M), int(N), int(K), int(dtype),
                          float(alpha), float(beta), A or None, int(lda), B or None, int(ldb),
                          C or None, int(ldc), stream or None)


def gemm_strided_batched_raw(transA, transB, M, N, K, dtype, alpha, beta, A, lda, strideA, B,
                             ldb, strideB, C, ldc, strideC, batch, stream=0) -> int:
    """gemm_strided_batched with plain integers (device addresses, element
    pitches, stream handle)."""
    return _lib.gemm_strided_batched(int(transA), int(transB), int(M), int(N), int(K), int(dtype),
                                     float(alpha), float(beta), A or None, int(lda), int(strideA),
                                     B or None, int(ldb), int(strideB), C or None, int(ldc),
                                     int(strideC), int(batch), stream or None)


def _ld3(t) -> int:
    """Row pitch of a [batch, rows, cols] tensor (the _ld rule per matrix)."""
    if t.shape[2] > 1 and t.stride(2) != 1:
        raise ValueError("rows must be contiguous (stride(2) == 1)")
    if t.shape[1] <= 1:
        return max(int(t.stride(1)), int(t.shape[2]), 1)
    return int(t.stride(1))


def gemm_strided_batched(A, B, C, transA=False, transB=False, alpha=1.0, beta=0.0, stream=None):
    """C[b] = alpha * op(A[b]) @ op(B[b]) + beta * C[b] for every b, in place.

    A, B, C are 3-D CUDA tensors [batch, rows, cols] with contiguous rows; the
    batch pitch is each tensor's stride(0) (0, via expand(), shares one A or
    B across the batch).  Shapes per entry as gemm().  Returns C.
    """
    import torch
    if A.dim() != 3 or B.dim() != 3 or C.dim() != 3:
        raise ValueError("batched operands are 3-D [batch, rows, cols]")
    batch = int(C.shape[0])
    if A.shape[0] != batch or B.shape[0] != batch:
        raise ValueError("A, B and C must have the same batch size")
    if A.dtype != B.dtype or A.dtype != C.dtype:
        raise TypeError("A, B and C must share a dtype")
    dtype = _DTYPES.get(A.dtype)
    if dtype is None:
        raise TypeError(f"unsupported dtype {A.dtype}")
    M, K = (A.shape[2], A.shape[1]) if transA else (A.shape[1], A.shape[2])
    Kb, N = (B.shape[2], B.shape[1]) if transB else (B.shape[1], B.shape[2])
    if K != Kb:
        raise ValueError(f"inner dimensions differ: {K} vs {Kb}")
    if C.shape[1] != M or C.shape[2] != N:
        raise ValueError(f"C is {tuple(C.shape)}, expected {(batch, M, N)}")
    if not (A.is_cuda and B.is_cuda and C.is_cuda):
        raise ValueError("gemm_strided_batched() takes CUDA tensors")
    s = stream if stream is not None else torch.cuda.current_stream(C.device)
    pitch = (lambda t: int(t.stride(0)) if batch > 1 else 0)
    rc = _lib.gemm_strided_batched(
        int(transA), int(transB), int(M), int(N), int(K), dtype, float(alpha), float(beta),
        A.data_ptr() or None, _ld3(A), pitch(A), B.data_ptr() or None, _ld3(B), pitch(B),
        C.data_ptr() or None, _ld3(C), pitch(C), batch, s.cuda_stream or None)
    if rc != OK:
        raise GemmError(rc)
    return C


def _ld(t) -> int:
    if t.dim() != 2:
        raise ValueError("matrices are 2-D")
    if t.shape[1] > 1 and t.stride(1) != 1:
        raise ValueError("rows must be contiguous (stride(1) == 1)")
    if t.shape[0] <= 1:  # a single row: any ld >= its length is valid
        return max(int(t.stride(0)), int(t.shape[1]), 1)
    return int(t.stride(0))


_DTYPES = {}
_get_raw_stream = None  # device index -> raw handle of its current stream, where torch has it


def _torch_tables():
    global _get_raw_stream
    import torch
    _get_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    _DTYPES.update({torch.float32: F32, torch.float16: F16_F32ACC, torch.bfloat16: BF16_F32ACC})


def _dims(A, B, C, transA, transB):
    if A.dtype != B.dtype or A.dtype != C.dtype:
        raise TypeError("A, B and C must share a dtype")
    dtype = _DTYPES.get(A.dtype)
    if dtype is None:
        raise TypeError(f"unsupported dtype {A.dtype}")
    M, K = (A.shape[1], A.shape[0]) if transA else (A.shape[0], A.shape[1])
    Kb, N = (B.shape[1], B.shape[0]) if transB else (B.shape[0], B.shape[1])
    if K != Kb:
        raise ValueError(f"inner dimensions differ: {K} vs {Kb}")
    if tuple(C.shape) != (M, N):
        raise ValueError(f"C is {tuple(C.shape)}, expected {(M, N)}")
    return dtype, int(M), int(N), int(K)


ACTS = {"none": 0, "relu": 1, "gelu": 2}


def _current_stream(device_index: int) -> int:
    """Raw handle of the current CUDA stream of a device."""
    if _get_raw_stream is not None:
        return _get_raw_stream(device_index)
    import torch
    return torch.cuda.current_stream(device_index).cuda_stream


def _ld_of(shape, stride) -> int:
    """_ld from a 2-D shape and stride already fetched."""
    rows, cols = shape
    ld, step = stride
    if step != 1 and cols > 1:
        raise ValueError("rows must be contiguous (stride(1) == 1)")
    if rows <= 1:
        return max(ld, cols, 1)
    return ld


def gemm(A, B, C, transA=False, transB=False, alpha=1.0, beta=0.0, stream=None, bias=None,
         act="none", tf32=False, tf32x3=False):
    """C = act(alpha * op(A) @ op(B) + beta * C + bias) in place, on torch CUDA
    tensors.

    A is [M,K] (or [K,M] with transA), B is [K,N] (or [N,K] with transB),
    C is [M,N]; all float32, all float16 or all bfloat16 (fp32 accumulation), rows
    contiguous, any leading dimension.  bias: None or a contiguous CUDA tensor
    of N elements of C's dtype (per output column); act: 'none', 'relu' or
    'gelu'.  tf32=True (float32 tensors only) opts into the reduced-precision
    TF32 tensor-core path; tf32x3=True into the 3xTF32 tensor-core path (about
    fp32 accuracy, finite inputs).  Runs on `stream` (a torch.cuda.Stream) or
    the current stream.  Returns C.
    """
    dt = A.dtype
    dtype = _DTYPES.get(dt)
    if dtype is None or B.dtype != dt or C.dtype != dt:
        if B.dtype != dt or C.dtype != dt:
            raise TypeError("A, B and C must share a dtype")
        raise TypeError(f"unsupported dtype {dt}")
    sa, sb, sc = A.shape, B.shape, C.shape
    if len(sa) != 2 or len(sb) != 2 or len(sc) != 2:
        raise ValueError("matrices are 2-D")
    M, K = (sa[1], sa[0]) if transA else (sa[0], sa[1])
    Kb, N = (sb[1], sb[0]) if transB else (sb[0], sb[1])
    if K != Kb:
        raise ValueError(f"inner dimensions differ: {K} vs {Kb}")
    if sc[0] != M or sc[1] != N:
        raise ValueError(f"C is {tuple(sc)}, expected {(M, N)}")
    if tf32 or tf32x3:
        if dtype != F32 or (tf32 and tf32x3):
            raise TypeError("tf32=True or tf32x3=True (one of them) takes float32 tensors")
        dtype = F32_TF32 if tf32 else F32_3XTF32
    if not (A.is_cuda and B.is_cuda and C.is_cuda):
        raise ValueError("gemm() takes CUDA tensors; use gemm_host() for host memory")
    s = stream.cuda_stream if stream is not None else _current_stream(C.get_device())
    lda, ldb, ldc = _ld_of(sa, A.stride()), _ld_of(sb, B.stride()), _ld_of(sc, C.stride())
    if bias is not None or act != "none":
        if bias is not None:
            if not bias.is_cuda or bias.dtype != C.dtype or bias.numel() != N or \
                    not bias.is_contiguous():
                raise ValueError("bias: a contiguous CUDA tensor of N elements of C's dtype")
        rc = _lib.gemm_ex(int(transA), int(transB), M, N, K, dtype, float(alpha), float(beta),
                          A.data_ptr() or None, lda, B.data_ptr() or None, ldb,
                          C.data_ptr() or None, ldc,
                          (bias.data_ptr() or None) if bias is not None else None, ACTS[act],
                          s or None)
        if rc != OK:
            raise GemmError(rc)
        return C
    rc = _gemm_fn(int(transA), int(transB), M, N, K, dtype, float(alpha), float(beta),
                  A.data_ptr() or None, lda, B.data_ptr() or None, ldb, C.data_ptr() or None,
                  ldc, s or None)
    if rc != OK:
        raise GemmError(rc)
    return C


_gemm_fn = _lib.gemm

# ---------------------------------------------------------------------------
# Microscaled operands (include/gemm.h, gemm_mx_format_t)
# ---------------------------------------------------------------------------
MX_FORMATS = {"fp4": 0, "fp4_e4m3": 1, "int8": 2}


def mx_row_bytes(fmt, cols) -> int:
    """Bytes of a row of codes (whole 16-byte units)."""
    return _lib.gemm_mx_row_bytes(MX_FORMATS[fmt], int(cols))


def mx_scale_bytes(fmt, rows, cols) -> int:
    """Bytes of the scale tiles."""
    return _lib.gemm_mx_scale_bytes(MX_FORMATS[fmt], int(rows), int(cols))


class Mx:
    """A matrix [rows, cols] in microscaled storage: `codes`, a 2-D uint8 CUDA
    tensor of `rows` rows (row pitch a multiple of 16 bytes, at least
    mx_row_bytes), and `scales`, a contiguous uint8 CUDA tensor of at least
    mx_scale_bytes elements.  fmt: 'fp4', 'fp4_e4m3' or 'int8'.

    The tensors' addresses are read on each call, as gemm() reads its operands':
    storage that was replaced (`.data`, `set_()`, a new tensor in `codes`) is used
    from then on, and refused if it does not hold the matrix."""
    __slots__ = ("codes", "scales", "fmt", "format", "rows", "cols", "device", "_seen",
                 "_operand")

    def __init__(self, codes, scales, fmt, rows, cols):
        code = MX_FORMATS.get(fmt)
        if code is None:
            raise ValueError(f"unknown format {fmt!r}")
        if type(rows) is not int or type(cols) is not int:
            rows, cols = int(rows), int(cols)
        device = codes.get_device()
        if device < 0 or scales.get_device() != device:
            raise ValueError("codes and scales are CUDA tensors of one device")
        if codes.itemsize != 1 or scales.itemsize != 1:
            raise TypeError("codes and scales are bytes")
        # (mx_row_bytes and mx_scale_bytes, without a call into the library)
        need = ((cols if code == 2 else (cols + 1) >> 1) + 15) & -16
        blocks = (cols + 15) >> 4 if code == 1 else (cols + 31) >> 5
        shape, stride = codes.shape, codes.stride()
        if len(shape) != 2 or shape[0] != rows or shape[1] < need or \
                (shape[1] > 1 and stride[1] != 1):
            raise ValueError(f"codes: {rows} rows of at least {need} bytes, contiguous within a row")
        held = scales.nbytes
        if held < ((rows + 127) >> 7) * ((blocks + 3) >> 2) * 512 or not scales.is_contiguous():
            raise ValueError("scales: a contiguous tensor of mx_scale_bytes(fmt, rows, cols) bytes")
        self.codes, self.scales, self.fmt, self.format = codes, scales, fmt, code
        self.rows, self.cols, self.device = rows, cols, device
        at, scales_at = codes.data_ptr(), scales.data_ptr()
        self._seen = (at, scales_at, rows * shape[1], held)
        # (a single row's pitch is not used: any valid one)
        self._operand = (at or None, stride[0] if rows > 1 else max(need, 16), scales_at or None)

    def operand(self):
        """(address of the codes, their row pitch, address of the scales), of the
        tensors as they are now; checked again whenever one of them lies elsewhere
        or has another size."""
        codes, scales = self.codes, self.scales
        at, scales_at, held, scales_held = self._seen
        if at != codes.data_ptr() or scales_at != scales.data_ptr() or held != codes.nbytes or \
                scales_held != scales.nbytes:
            self.__init__(codes, scales, self.fmt, self.rows, self.cols)
        return self._operand


def _not_stored(Q, name):
    return TypeError(f"{name} is a stored operand (an Mx), not a {type(Q).__name__}")


def mx_empty(rows, cols, fmt, device="cuda") -> Mx:
    """Room for a stored matrix."""
    import torch
    if fmt not in MX_FORMATS:
        raise ValueError(f"unknown format {fmt!r}")
    return Mx(torch.empty((rows, mx_row_bytes(fmt, cols)), dtype=torch.uint8, device=device),
              torch.empty(mx_scale_bytes(fmt, rows, cols), dtype=torch.uint8, device=device),
              fmt, rows, cols)


def mx_quantize(X, Q, transX=False, mult=1.0, act="none", Y=None, stream=None):
    """Stores mult * op(X) in Q (an Mx) and, with Y, writes Y = act(op(X)) in the
    same pass: the forward pass of an activation whose input is checkpointed.
    X is [rows, cols] (or [cols, rows] with transX) float32, float16 or bfloat16;
    Y has X's dtype and shape and may be X.  Returns Q.

    mult is not kept with Q, whose values are those of mult * X: give 1 / mult to a
    product as alpha, or multiply what mx_dequantize() returns by it."""
    dt, sx = X.dtype, X.shape
    dtype = _DTYPES.get(dt)
    if dtype is None:
        raise TypeError(f"unsupported dtype {dt}")
    if not isinstance(Q, Mx):
        raise _not_stored(Q, "Q")
    want = (Q.cols, Q.rows) if transX else (Q.rows, Q.cols)
    if sx != want:
        raise ValueError(f"X is {tuple(sx)}, expected {want}")
    dev = X.get_device()
    q, pitch, scales = Q.operand()
    if dev < 0 or Q.device != dev:
        raise ValueError("mx_quantize() takes CUDA tensors of one device")
    yp, ldy = None, 0
    if Y is not None:
        if Y.dtype != dt or Y.shape != sx or Y.get_device() != dev:
            raise ValueError("Y has X's dtype, shape and device")
        yp, ldy = Y.data_ptr() or None, _ld_of(sx, Y.stride())
    elif act != "none":
        raise ValueError("act needs Y")
    s = (stream.cuda_stream if stream is not None else _current_stream(dev)) or None
    rc = _lib.gemm_mx_quantize(Q.format, 1 if transX else 0, Q.rows, Q.cols, dtype, float(mult),
                               X.data_ptr() or None, _ld_of(sx, X.stride()), ACTS[act], yp, ldy,
                               q, pitch, scales, s)
    if rc != OK:
        raise GemmError(rc)
    return Q


def mx_dequantize(Q, Y, stream=None):
    """Y = the values of Q, in Y's dtype.  Returns Y."""
    dtype = _DTYPES.get(Y.dtype)
    if dtype is None:
        raise TypeError(f"unsupported dtype {Y.dtype}")
    if not isinstance(Q, Mx):
        raise _not_stored(Q, "Q")
    sy = Y.shape
    if sy != (Q.rows, Q.cols):
        raise ValueError(f"Y is {tuple(sy)}, expected {(Q.rows, Q.cols)}")
    dev = Y.get_device()
    q, pitch, scales = Q.operand()
    if dev < 0 or Q.device != dev:
        raise ValueError("mx_dequantize() takes CUDA tensors of one device")
    s = (stream.cuda_stream if stream is not None else _current_stream(dev)) or None
    rc = _lib.gemm_mx_dequantize(Q.format, Q.rows, Q.cols, q, pitch, scales, dtype,
                                 Y.data_ptr() or None, _ld_of(sy, Y.stride()), s)
    if rc != OK:
        raise GemmError(rc)
    return Y


def mx_act_backward(dY, Q, dX, act="gelu", dbias=None, stream=None):
    """dX = dY * act'(x) with x read from its 8-bit checkpoint Q ('int8'), and
    dbias[j] = sum_i dX[i, j] (a contiguous float32 tensor of cols elements, or
    None).  dX may be dY.  Returns dX."""
    dt, sy = dY.dtype, dY.shape
    dtype = _DTYPES.get(dt)
    if dtype is None:
        raise TypeError(f"unsupported dtype {dt}")
    if not isinstance(Q, Mx):
        raise _not_stored(Q, "Q")
    if Q.fmt != "int8":
        raise TypeError("the checkpoint is an 'int8' Mx")
    if dX.dtype != dt or sy != (Q.rows, Q.cols) or dX.shape != sy:
        raise ValueError(f"dY and dX: {(Q.rows, Q.cols)} CUDA tensors of one dtype")
    dev = dY.get_device()
    q, pitch, scales = Q.operand()
    if dev < 0 or Q.device != dev or dX.get_device() != dev:
        raise ValueError("mx_act_backward() takes CUDA tensors of one device")
    bp = None
    if dbias is not None:
        if dbias.get_device() != dev or dbias.numel() != Q.cols or \
                _DTYPES.get(dbias.dtype) != F32 or not dbias.is_contiguous():
            raise ValueError("dbias: a contiguous float32 CUDA tensor of cols elements")
        bp = dbias.data_ptr() or None
    s = (stream.cuda_stream if stream is not None else _current_stream(dev)) or None
    rc = _lib.gemm_mx_act_backward(Q.rows, Q.cols, dtype, ACTS[act], dY.data_ptr() or None,
                                   _ld_of(sy, dY.stride()), q, pitch, scales,
                                   dX.data_ptr() or None, _ld_of(sy, dX.stride()), bp, s)
    if rc != OK:
        raise GemmError(rc)
    return dX


def gemm_mx(A, B, C, transA=False, transB=False, alpha=1.0, beta=0.0, stream=None, bias=None,
            act="none"):
    """The product with stored operands, in place on C; alpha, beta, bias and
    act as gemm().

    A a tensor, B an Mx: C = act(alpha * op(A) @ op(B) + beta * C + bias), B
    stored [K, N], or [N, K] with transB; A and C share a dtype.
    A and B Mx of the same 4-bit format, both stored along K (A [M, K], B
    [N, K]): C = act(alpha * A @ B.T + beta * C + bias); transA and transB stay
    False.  Returns C.

    With a float16 tensor A the values of B are rounded to float16 first: exact but
    beyond its range (below 2^-14, above 65504).  Up to 32 rows of A with transB a
    power-of-two scale of 4-bit codes stays in fp32 there instead, so such an
    operand gives other results from 33 rows on."""
    dt = C.dtype
    dtype = _DTYPES.get(dt)
    if dtype is None:
        raise TypeError(f"unsupported dtype {dt}")
    dev = C.get_device()
    if dev < 0:
        raise ValueError("gemm_mx() takes CUDA tensors")
    sc = C.shape
    if len(sc) != 2:
        raise ValueError("matrices are 2-D")
    M, N = sc
    bp = None
    if bias is not None:
        if bias.get_device() != dev or bias.dtype != dt or bias.numel() != N or \
                not bias.is_contiguous():
            raise ValueError("bias: a contiguous CUDA tensor of N elements of C's dtype")
        bp = bias.data_ptr() or None
    s = (stream.cuda_stream if stream is not None else _current_stream(dev)) or None
    if not isinstance(B, Mx):
        raise _not_stored(B, "B")
    codes, pitch, scales = B.operand()
    if isinstance(A, Mx):
        if transA or transB:
            raise ValueError("two stored operands are both stored along K")
        if A.format != B.format:
            raise TypeError("both operands have the same format")
        K = A.cols
        if K != B.cols:
            raise ValueError(f"inner dimensions differ: {K} vs {B.cols}")
        if A.rows != M or B.rows != N:
            raise ValueError(f"C is {(M, N)}, expected {(A.rows, B.rows)}")
        a, lda, a_scales = A.operand()
        if A.device != dev or B.device != dev:
            raise ValueError("A, B and C are on one device")
        rc = _lib.gemm_mx4(A.format, M, N, K, dtype, float(alpha), float(beta), a, lda, a_scales,
                           codes, pitch, scales, C.data_ptr() or None, _ld_of(sc, C.stride()), bp,
                           ACTS[act], s)
    else:
        if A.dtype != dt:
            raise TypeError("A and C must share a dtype")
        sa = A.shape
        if len(sa) != 2:
            raise ValueError("matrices are 2-D")
        if A.get_device() != dev or B.device != dev:
            raise ValueError("A, B and C are CUDA tensors of one device")
        Ma, K = (sa[1], sa[0]) if transA else sa
        Kb, Nb = (B.cols, B.rows) if transB else (B.rows, B.cols)
        if K != Kb:
            raise ValueError(f"inner dimensions differ: {K} vs {Kb}")
        if Ma != M or Nb != N:
            raise ValueError(f"C is {(M, N)}, expected {(Ma, Nb)}")
        rc = _lib.gemm_mx(B.format, 1 if transA else 0, 1 if transB else 0, M, N, K, dtype,
                          float(alpha), float(beta), A.data_ptr() or None,
                          _ld_of(sa, A.stride()), codes, pitch, scales, C.data_ptr() or None,
                          _ld_of(sc, C.stride()), bp, ACTS[act], s)
    if rc != OK:
        raise GemmError(rc)
    return C


# ---------------------------------------------------------------------------
# Products with a full epilogue, and products grouped by expert
# ---------------------------------------------------------------------------
def _like(t, name, dt, dev, shape):
    """(address, row pitch) of a further matrix of a call, or (None, 0) for None."""
    if t is None:
        return None, 0
    if t.dtype != dt or t.get_device() != dev or t.shape != shape:
        raise ValueError(f"{name}: a {tuple(shape)} CUDA tensor of the operands' dtype and device")
    return t.data_ptr() or None, _ld_of(shape, t.stride())


def _flat(t, name, dt, dev, shape):
    """Address of a contiguous tensor of a call, or None for None."""
    if t is None:
        return None
    if t.dtype != dt or t.get_device() != dev or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous {tuple(shape)} CUDA tensor of dtype {dt} on the "
                         "operands' device")
    return t.data_ptr() or None


def _common(A, B, Y, name):
    """dtype code, torch dtype and device of a call's matrices."""
    dt = Y.dtype
    dtype = _DTYPES.get(dt)
    if A.dtype != dt or B.dtype != dt:
        raise TypeError("the operands and the result share a dtype")
    if dtype is None:
        raise TypeError(f"unsupported dtype {dt}")
    dev = Y.get_device()
    if dev < 0 or A.get_device() != dev or B.get_device() != dev:
        raise ValueError(f"{name}() takes CUDA tensors of one device")
    return dtype, dt, dev


def _product(A, B, Y, transA, transB):
    sa, sb, sy = A.shape, B.shape, Y.shape
    if len(sa) != 2 or len(sb) != 2 or len(sy) != 2:
        raise ValueError("matrices are 2-D")
    M, K = (sa[1], sa[0]) if transA else sa
    Kb, N = (sb[1], sb[0]) if transB else sb
    if K != Kb:
        raise ValueError(f"inner dimensions differ: {K} vs {Kb}")
    if sy[0] != M or sy[1] != N:
        raise ValueError(f"the result is {tuple(sy)}, expected {(M, N)}")
    return M, N, K, _ld_of(sa, A.stride()), _ld_of(sb, B.stride()), _ld_of(sy, Y.stride())


def _act_code(act):
    code = ACTS.get(act)
    if code is None:
        raise ValueError(f"unknown activation {act!r}")
    return code


def gemm_fused(A, B, Y, transA=False, transB=False, alpha=1.0, bias=None, act="none",
               residual=None, beta=1.0, preact=None, stream=None):
    """U = alpha * op(A) @ op(B) + bias and Y = act(U) + beta * residual, in one pass.

    A, B as in gemm(); Y [M, N].  bias: N contiguous elements; residual: [M, N], which
    may be Y; preact: [M, N], receives U (rounded to its dtype) for the backward pass;
    each may be None.  All share a dtype (float32, float16 or bfloat16) and a device.
    Returns Y."""
    dtype, dt, dev = _common(A, B, Y, "gemm_fused")
    M, N, K, lda, ldb, ldy = _product(A, B, Y, transA, transB)
    code = _act_code(act)
    bp = _flat(bias, "bias", dt, dev, (N,))
    rp, ldr = _like(residual, "residual", dt, dev, Y.shape)
    up, ldu = _like(preact, "preact", dt, dev, Y.shape)
    s = (stream.cuda_stream if stream is not None else _current_stream(dev)) or None
    rc = _lib.gemm_fused(1 if transA else 0, 1 if transB else 0, M, N, K, dtype, float(alpha),
                         A.data_ptr() or None, lda, B.data_ptr() or None, ldb, bp, code,
                         float(beta), rp, ldr, up, ldu, Y.data_ptr() or None, ldy, s)
    if rc != OK:
        raise GemmError(rc)
    return Y


def gemm_fused_backward(A, B, dX, preact, transA=False, transB=False, alpha=1.0, act="gelu",
                        dbias=None, stream=None):
    """dX = (alpha * op(A) @ op(B)) * act'(preact), and dbias[j] = sum_i dX[i, j] (a
    contiguous float32 tensor of N elements, or None): with A the gradient of a layer's
    output and B its weight, the gradient of what went into the activation before it.
    preact [M, N] as gemm_fused() stored it (None with act 'none'); dX may be preact.
    Returns dX."""
    import torch
    dtype, dt, dev = _common(A, B, dX, "gemm_fused_backward")
    M, N, K, lda, ldb, ldx = _product(A, B, dX, transA, transB)
    code = _act_code(act)
    up, ldu = _like(preact, "preact", dt, dev, dX.shape)
    if code and preact is None:
        raise ValueError("preact: the activation's input")
    dp = _flat(dbias, "dbias", torch.float32, dev, (N,))
    s = (stream.cuda_stream if stream is not None else _current_stream(dev)) or None
    rc = _lib.gemm_fused_backward(1 if transA else 0, 1 if transB else 0, M, N, K, dtype,
                                  float(alpha), A.data_ptr() or None, lda, B.data_ptr() or None,
                                  ldb, code, up, ldu, dX.data_ptr() or None, ldx, dp, s)
    if rc != OK:
        raise GemmError(rc)
    return dX


def _groups(offsets, dev):
    """Number of groups and address of the offsets."""
    import torch
    if offsets.dtype != torch.int32:
        raise TypeError("offsets are int32")
    if offsets.dim() != 1 or offsets.numel() < 1 or offsets.get_device() != dev or \
            not offsets.is_contiguous():
        raise ValueError("offsets: groups + 1 contiguous int32 values on the operands' device")
    return offsets.numel() - 1, offsets.data_ptr()


def _grouped_product(A, B, Y, offsets, dev, transB):
    sa, sb, sy = A.shape, B.shape, Y.shape
    if len(sa) != 2 or len(sb) != 3 or len(sy) != 2:
        raise ValueError("A and the result are 2-D, B is [groups, rows, cols]")
    groups, op = _groups(offsets, dev)
    if sb[0] != groups:
        raise ValueError(f"B holds {sb[0]} matrices, offsets {groups} groups")
    rows, K = sa
    Kb, N = (sb[2], sb[1]) if transB else (sb[1], sb[2])
    if K != Kb:
        raise ValueError(f"inner dimensions differ: {K} vs {Kb}")
    if sy[0] != rows or sy[1] != N:
        raise ValueError(f"the result is {tuple(sy)}, expected {(rows, N)}")
    return (rows, N, K, groups, op, _ld_of(sa, A.stride()), _ld3(B),
            int(B.stride(0)) if groups > 1 else 0, _ld_of(sy, Y.stride()))


def gemm_grouped(A, B, Y, offsets, transB=False, alpha=1.0, bias=None, act="none",
                 residual=None, beta=1.0, preact=None, stream=None):
    """gemm_fused() by groups of rows, as a router sends tokens to experts: on rows
    offsets[g] .. offsets[g + 1] of A, residual, preact and Y,
        U = alpha * A @ op(B[g]) + bias[g],  Y = act(U) + beta * residual.

    A [rows, K]; B [groups, K, N], or [groups, N, K] with transB; Y [rows, N]; offsets:
    groups + 1 ascending int32 on the GPU (nothing waits for them); bias [groups, N].
    Rows outside every group are left as they are.  Returns Y."""
    dtype, dt, dev = _common(A, B, Y, "gemm_grouped")
    rows, N, K, groups, op, lda, ldb, strideb, ldy = _grouped_product(A, B, Y, offsets, dev, transB)
    code = _act_code(act)
    bp = _flat(bias, "bias", dt, dev, (groups, N))
    rp, ldr = _like(residual, "residual", dt, dev, Y.shape)
    up, ldu = _like(preact, "preact", dt, dev, Y.shape)
    s = (stream.cuda_stream if stream is not None else _current_stream(dev)) or None
    rc = _lib.gemm_grouped(1 if transB else 0, rows, N, K, groups, op, dtype, float(alpha),
                           A.data_ptr() or None, lda, B.data_ptr() or None, ldb, strideb, bp, code,
                           float(beta), rp, ldr, up, ldu, Y.data_ptr() or None, ldy, s)
    if rc != OK:
        raise GemmError(rc)
    return Y


def gemm_grouped_backward(A, B, dX, offsets, preact, transB=False, alpha=1.0, act="gelu",
                          dbias=None, stream=None):
    """gemm_fused_backward() by groups of rows (see gemm_grouped()): dX = (alpha * A @
    op(B[g])) * act'(preact) on each group's rows, dbias [groups, N] float32 its column
    sums by group (zero for an empty one), or None.  Returns dX."""
    import torch
    dtype, dt, dev = _common(A, B, dX, "gemm_grouped_backward")
    rows, N, K, groups, op, lda, ldb, strideb, ldx = _grouped_product(A, B, dX, offsets, dev, transB)
    code = _act_code(act)
    up, ldu = _like(preact, "preact", dt, dev, dX.shape)
    if code and preact is None:
        raise ValueError("preact: the activation's input")
    dp = _flat(dbias, "dbias", torch.float32, dev, (groups, N))
    s = (stream.cuda_stream if stream is not None else _current_stream(dev)) or None
    rc = _lib.gemm_grouped_backward(1 if transB else 0, rows, N, K, groups, op, dtype, float(alpha),
                                    A.data_ptr() or None, lda, B.data_ptr() or None, ldb, strideb,
                                    code, up, ldu, dX.data_ptr() or None, ldx, dp, s)
    if rc != OK:
        raise GemmError(rc)
    return dX


def gemm_grouped_wgrad(A, B, C, offsets, alpha=1.0, beta=0.0, stream=None):
    """C[g] = alpha * A[rows of g].T @ B[rows of g] + beta * C[g]: the gradient of each
    group's matrix.  A [rows, M], B [rows, N], C [groups, M, N]; offsets as in
    gemm_grouped().  An empty group's C[g] becomes beta * C[g].  Returns C."""
    dtype, dt, dev = _common(A, B, C, "gemm_grouped_wgrad")
    sa, sb, sc = A.shape, B.shape, C.shape
    if len(sa) != 2 or len(sb) != 2 or len(sc) != 3:
        raise ValueError("A and B are 2-D, C is [groups, M, N]")
    groups, op = _groups(offsets, dev)
    if sa[0] != sb[0]:
        raise ValueError(f"A has {sa[0]} rows, B {sb[0]}")
    if sc[0] != groups or sc[1] != sa[1] or sc[2] != sb[1]:
        raise ValueError(f"C is {tuple(sc)}, expected {(groups, sa[1], sb[1])}")
    s = (stream.cuda_stream if stream is not None else _current_stream(dev)) or None
    rc = _lib.gemm_grouped_wgrad(sa[0], sa[1], sb[1], groups, op, dtype, float(alpha), float(beta),
                                 A.data_ptr() or None, _ld_of(sa, A.stride()),
                                 B.data_ptr() or None, _ld_of(sb, B.stride()),
                                 C.data_ptr() or None, _ld3(C),
                                 int(C.stride(0)) if groups > 1 else 0, s)
    if rc != OK:
        raise GemmError(rc)
    return C


def gemm_host(A, B, C, transA=False, transB=False, alpha=1.0, beta=0.0, stream=None):
    """The same product on host (CPU) tensors, pinned or not; the library
    copies them to the GPU, computes, copies C back and synchronises."""
    import torch
    dtype, M, N, K = _dims(A, B, C, transA, transB)
    for t in (A, B, C):
        if t.is_cuda:
            raise ValueError("gemm_host() takes host tensors")
    s = stream if stream is not None else torch.cuda.current_stream()
    rc = _lib.gemm_host(int(transA), int(transB), M, N, K, dtype, float(alpha), float(beta),
                        A.data_ptr() or None, _ld(A), B.data_ptr() or None, _ld(B),
                        C.data_ptr() or None, _ld(C), s.cuda_stream or None)
    if rc != OK:
        raise GemmError(rc)
    return C


def check_device_status(stream=None) -> int:
    """Synchronises the stream and returns (and clears) the device status:
    OK, ERR_TIMEOUT (a kernel's bounded wait ran out) or ERR_CUDA."""
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return _lib.gemm_check_device_status(s.cuda_stream or None)


try:
    _torch_tables()
except ImportError:  # pragma: no cover - torch is needed only by the tensor wrappers
    pass
