"""Python binding of libtplinear (include/tplinear.h), the tensor-parallel
Linear Y = X W on one MI355X with all P shards resident.

Argument marshalling only: every function passes device pointers, sizes and
leading dimensions taken from torch tensors to the C entry point of the same
name and turns a non-zero status into an exception (ValueError for argument
errors, RuntimeError for TP_ERR_HIP).  All arithmetic runs in the HIP
kernels of the library; there is no fallback.  The first call raises
ImportError if libtplinear.so has not been built
(python -m tensor_linear_amd.build).

Tensors: 2-D row-major views with unit column stride; the row stride is the
leading dimension.  X is [M, K], W is stored [N, K] ([out, in]), Y is [M, N].
"""
import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtplinear.so")

_lib = None


def _get_lib():
    """Load libtplinear.so once; fail loudly if it has not been built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with `python -m tensor_linear_amd.build` "
            "(hipcc, gfx950)")
    _lib = _declare(ctypes.CDLL(LIB_PATH))
    return _lib


def __getattr__(name):
    if name == "lib":
        return _get_lib()
    raise AttributeError(name)


# ---- constants (mirror include/tplinear.h) --------------------------------
TP_OK, TP_ERR_NULL, TP_ERR_SHAPE, TP_ERR_INDIVISIBLE, TP_ERR_PLACEMENT, \
    TP_ERR_DTYPE, TP_ERR_MODE, TP_ERR_WORKSPACE, TP_ERR_HIP = range(9)
TP_F32, TP_BF16 = 0, 1
TP_REPLICATE, TP_SHARD, TP_PARTIAL = 0, 1, 2
TP_Y_CONCAT, TP_Y_SHARDS = 0, 1
TP_ROW_PARTIAL, TP_ROW_SUM, TP_ROW_FUSED, TP_ROW_SCATTER = 0, 1, 2, 3
TP_ACT_NONE, TP_ACT_SWIGLU = 0, 1
TP_ROPE_HALVES, TP_ROPE_PAIRS = 0, 1
TP_MAX_SHARDS = 64

EXPORTS = ("tp_shard_layout", "tp_linear_column", "tp_linear_row", "tp_shard_reduce",
           "tp_linear_column_ex", "tp_linear_row_ex", "tp_shard_reduce_ex", "tp_embedding",
           "tp_row_workspace_bytes", "tp_workspace_zero", "tp_status_str", "tp_version",
           "tp_linear_row_noalloc", "tp_quantize_rows", "tp_linear_column_quant",
           "tp_linear_row_quant", "tp_qk_norm_rope", "tp_qk_norm_rope_backward",
           "tp_qk_norm_rope_workspace_bytes", "tp_kv_append")
TP_NOALLOC_SCRATCH_BYTES = 32 << 20


class tp_placement(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("dim", ctypes.c_int32)]


class tp_view(ctypes.Structure):
    _fields_ = [("elem_offset", ctypes.c_int64), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64), ("ld", ctypes.c_int64),
                ("row0", ctypes.c_int64), ("col0", ctypes.c_int64)]


_i32, _i64, _ptr, _sz = ctypes.c_int32, ctypes.c_int64, ctypes.c_void_p, ctypes.c_size_t
_f32 = ctypes.c_float


def _declare(lib):
    lib.tp_shard_layout.argtypes = [_i64, _i64, _i64, tp_placement, _i32, ctypes.POINTER(tp_view)]
    lib.tp_shard_layout.restype = _i32
    lib.tp_linear_column.argtypes = [_ptr, _i64, _ptr, _i64, _ptr, _i64, _i32, _i64, _i64, _i64,
                                     _i32, _i32, _ptr]
    lib.tp_linear_column.restype = _i32
    lib.tp_linear_row.argtypes = [_ptr, _i64, _ptr, _i64, _ptr, _i64, _i64, _i32, _ptr, _sz,
                                  _i64, _i64, _i64, _i32, _i32, _ptr]
    lib.tp_linear_row.restype = _i32
    lib.tp_shard_reduce.argtypes = [_ptr, _i64, _i64, _ptr, _i64, _i64, _i32, _i64, _i64, _i32,
                                    _i32, _ptr]
    lib.tp_shard_reduce.restype = _i32
    lib.tp_linear_column_ex.argtypes = [_ptr, _ptr, _i64, _ptr, _i64, _ptr, _ptr, _i64, _i32,
                                        _i32, _i64, _i64, _i64, _i32, _i32, _ptr]
    lib.tp_linear_column_ex.restype = _i32
    lib.tp_linear_row_ex.argtypes = [_ptr, _i64, _ptr, _i64, _ptr, _ptr, _ptr, _i64, _i64, _i32,
                                     _ptr, _sz, _i64, _i64, _i64, _i32, _i32, _ptr]
    lib.tp_linear_row_ex.restype = _i32
    lib.tp_shard_reduce_ex.argtypes = [_ptr, _i64, _i64, _ptr, _ptr, _ptr, _i64, _i64, _i32,
                                       _i64, _i64, _i32, _i32, _ptr]
    lib.tp_shard_reduce_ex.restype = _i32
    lib.tp_embedding.argtypes = [_ptr, _i64, _ptr, _ptr, _i64, _i64, _i64, _ptr, _i64, _i32,
                                 _i32, _i32, _ptr, _ptr]
    lib.tp_embedding.restype = _i32
    lib.tp_linear_row_noalloc.argtypes = [_ptr, _i64, _ptr, _i64, _ptr, _i64, _i64, _i32,
                                          _i64, _i64, _i64, _i32, _i32, _ptr]
    lib.tp_linear_row_noalloc.restype = _i32
    lib.tp_quantize_rows.argtypes = [_ptr, _i64, _ptr, _i64, _ptr, _i64, _i64, _i64, _i32, _i32,
                                     _ptr]
    lib.tp_quantize_rows.restype = _i32
    lib.tp_linear_column_quant.argtypes = [_ptr, _i64, _ptr, _i64, _ptr, _i64, _ptr, _ptr, _ptr,
                                           _i64, _i32, _i32, _i64, _i64, _i64, _i32, _i32, _ptr]
    lib.tp_linear_column_quant.restype = _i32
    lib.tp_linear_row_quant.argtypes = [_ptr, _i64, _ptr, _i64, _i32, _ptr, _i64, _ptr, _ptr, _ptr,
                                        _ptr, _i64, _i64, _i32, _ptr, _sz, _i64, _i64, _i64, _i32,
                                        _i32, _ptr]
    lib.tp_linear_row_quant.restype = _i32
    # the QKV matrix, the rotation and the norms, then the tokens and heads
    rot = [_ptr, _ptr, _i64, _i64, _i32, _ptr, _ptr, _f32]
    heads = [_i64, _i64, _i64, _i64, _i32, _i32, _ptr, _ptr]
    lib.tp_qk_norm_rope.argtypes = ([_ptr, _i64, _i32, _ptr] + rot + [_ptr, _i64, _ptr, _i64] +
                                    heads)
    lib.tp_qk_norm_rope.restype = _i32
    lib.tp_qk_norm_rope_backward.argtypes = ([_ptr, _i64, _i32, _ptr] + rot + [_ptr, _i64] * 4 +
                                             [_ptr, _ptr, _ptr, _sz] + heads)
    lib.tp_qk_norm_rope_backward.restype = _i32
    lib.tp_qk_norm_rope_workspace_bytes.argtypes = [_i64, _i64]
    lib.tp_qk_norm_rope_workspace_bytes.restype = _sz
    lib.tp_kv_append.argtypes = ([_ptr, _i64, _i32] + rot + [_ptr, _ptr, _i64, _ptr, _i64, _i64,
                                 _ptr, _ptr, _i64, _i64, _i64, _i64, _i64, _ptr, _i64] + heads)
    lib.tp_kv_append.restype = _i32
    lib.tp_row_workspace_bytes.argtypes = [_i32, _i64, _i64, _i32]
    lib.tp_row_workspace_bytes.restype = _sz
    lib.tp_workspace_zero.argtypes = [_ptr, _sz, _ptr]
    lib.tp_workspace_zero.restype = _i32
    lib.tp_status_str.argtypes = [_i32]
    lib.tp_status_str.restype = ctypes.c_char_p
    lib.tp_version.argtypes = []
    lib.tp_version.restype = _i32
    return lib


class TPError(ValueError):
    def __init__(self, status: int):
        self.status = status
        super().__init__(_get_lib().tp_status_str(status).decode())


class TPHipError(RuntimeError):
    def __init__(self, status: int):
        self.status = status
        super().__init__(_get_lib().tp_status_str(status).decode())


def check(status: int) -> None:
    if status == TP_OK:
        return
    if status == TP_ERR_HIP:
        raise TPHipError(status)
    raise TPError(status)


def tp_status_str(status: int) -> str:
    return _get_lib().tp_status_str(status).decode()


def tp_version() -> int:
    return int(_get_lib().tp_version())


# ---- marshalling helpers --------------------------------------------------

# torch is imported at the first call that is given a tensor (the C library and
# this module's constants need none).  A call's checks cost the host more than a
# small kernel runs, so they read each tensor's shape, strides and device once.

def _torch():
    global _torch_module, _DTYPES
    if _torch_module is None:
        import torch
        # the table first: another thread that finds the module set uses it
        _DTYPES = {torch.bfloat16: TP_BF16, torch.float32: TP_F32}
        _torch_module = torch
    return _torch_module


_torch_module = None
_DTYPES = {}


def _dtype_code(t) -> int:
    c = _DTYPES.get(t.dtype)
    if c is None:
        _torch()
        c = _DTYPES.get(t.dtype)
        if c is None:
            raise TypeError(f"unsupported dtype {t.dtype}: bfloat16 or float32")
    return c


def _mat(t, name):
    """(data pointer, rows, cols, leading dim) of a 2-D unit-column-stride view."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be 2-D, got shape {tuple(shape)}")
    rows, cols = shape
    ld, unit = t.stride()
    if cols > 1 and unit != 1:
        raise ValueError(f"{name} must have unit column stride")
    if rows > 1 and ld < cols:   # an expanded row: no leading dimension says that
        raise ValueError(f"{name} must have a row stride of at least its {cols} columns")
    # A one-row view keeps the row stride of the buffer it was cut from when
    # that stride is a valid leading dim (it places the blocks of a [P, 1, N]
    # output); otherwise its leading dim is its width.
    if ld < cols:
        ld = cols
    return t.data_ptr(), rows, cols, ld or 1


def _same_gpu(*items):
    """Every tensor given (lists of tensors included, None skipped) must live
    on one GPU: the kernels dereference the data pointers on that device, so
    a host tensor or a second device is rejected here, before any launch."""
    dev = first = None
    for it in items:
        if it is None:
            continue
        for t in (it if isinstance(it, (list, tuple)) else (it,)):
            if t is None:
                continue
            d = t.get_device()
            if d == dev:
                continue
            if not t.is_cuda:
                raise ValueError("every tensor must be a GPU tensor (got one on "
                                 f"{t.device})")
            if dev is None:
                dev, first = d, t
            else:
                raise ValueError(f"tensors on {first.device} and {t.device}: all must share one GPU")


def _ptr_array(ts, name):
    """Host array of the data pointers of a list of tensors (or None)."""
    if ts is None:
        return None
    return (ctypes.c_void_p * len(ts))(*[t.data_ptr() for t in ts])


def _check_p(P):
    if not 1 <= P <= TP_MAX_SHARDS:
        check(TP_ERR_SHAPE)


def _expect_shape(t, shape, name):
    """The library writes exactly `shape`; a smaller or differently shaped
    output would be written out of bounds, so it is refused here."""
    if t.shape != shape and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _expect_room(t, elems, name):
    """t's storage must hold `elems` elements from t's first element."""
    have = t.untyped_storage().nbytes() // t.element_size() - t.storage_offset()
    if elems > have:
        raise ValueError(f"{name}: the output needs {elems} elements from its first one, "
                         f"its storage holds {have}")


def _scatter_out(Y, M, N, P, scatter, y_slice_stride, name="Y"):
    """Row stride of a fold / reduce-scatter output Y: [M, N], or for a
    reduce-scatter with a nonzero slice stride the [M/P, N] view of slice 0
    inside a buffer that holds all P slices."""
    if scatter and M % P:
        check(TP_ERR_INDIVISIBLE)
    yp, _, _, ldy = _mat(Y, name)
    if scatter and y_slice_stride:
        s = M // P
        _expect_shape(Y, (s, N), name)
        if s and N:
            _expect_room(Y, (P - 1) * y_slice_stride + (s - 1) * ldy + N, name)
    else:
        _expect_shape(Y, (M, N), name)
    return yp, ldy


def _block_out(Y, P, rows, cols, name="Y"):
    """Pointer and row stride of a [P, rows, cols] output whose blocks are
    rows*ldy elements apart."""
    _expect_shape(Y, (P, rows, cols), name)
    block, ldy, unit = Y.stride()
    if cols > 1 and unit != 1:
        raise ValueError(f"{name}[0] must have unit column stride")
    if rows > 1 and ldy < cols:
        raise ValueError(f"{name}[0] must have a row stride of at least its {cols} columns")
    ldy = max(ldy, cols, 1)
    if P > 1 and block != rows * ldy:
        raise ValueError(f"{name} blocks must be rows*ldy elements apart")
    return Y.data_ptr(), ldy


def _bias_ptr(bias, dt):
    if bias is None:
        return None
    if bias.dim() != 1 or (bias.numel() > 1 and bias.stride(0) != 1):
        raise ValueError("bias must be a contiguous 1-D tensor")
    if _dtype_code(bias) != dt:
        raise TypeError("bias must have the output dtype")
    return bias.data_ptr()


def _stream(t, stream):
    """The stream handle of a call: the one given, or the current one of t's
    device."""
    if stream is not None:
        return int(stream)
    if t.is_cuda:
        return _torch()._C._cuda_getCurrentRawStream(t.get_device())
    return 0


def _here(stream, t, *others):
    """The stream handle of a call on tensors (None skipped) that must all be
    on the current device: a stream of another device would run there or here
    by the runtime's choice, and the kernels' grids are sized for the current
    one."""
    dev = t.get_device()
    for o in others:
        if o is not None and o.get_device() != dev:
            _same_gpu(t, *others)
    c = _torch()._C
    if dev < 0:
        _same_gpu(t)
    if dev != c._cuda_getDevice():
        raise ValueError(f"the tensors are on {t.device}, which is not the current device")
    return c._cuda_getCurrentRawStream(dev) if stream is None else int(stream)


# ---- entry points ---------------------------------------------------------

def tp_shard_layout(rows: int, cols: int, ld: int, kind: int, dim: int, P: int) -> list:
    """Views of the P shards as (elem_offset, rows, cols, ld, row0, col0)."""
    if not 1 <= P <= TP_MAX_SHARDS:
        check(TP_ERR_SHAPE)
    views = (tp_view * P)()
    check(_get_lib().tp_shard_layout(rows, cols, ld, tp_placement(kind, dim), P, views))
    return [(v.elem_offset, v.rows, v.cols, v.ld, v.row0, v.col0) for v in views]


def tp_linear_column(X, W, Y, P: int, y_mode: int = TP_Y_CONCAT, stream=None) -> None:
    """Column-parallel Linear.  X [M, K], W [N, K]; Y [M, N] for TP_Y_CONCAT
    or [P, M, N/P] (block stride M*ldy) for TP_Y_SHARDS."""
    xp, M, K, ldx = _mat(X, "X")
    wp, N, Kw, ldw = _mat(W, "W")
    if Kw != K:
        raise ValueError(f"X has K={K} but W has K={Kw}")
    dt = _dtype_code(X)
    if _dtype_code(W) != dt or _dtype_code(Y) != dt:
        raise TypeError("X, W and Y must share one dtype")
    _check_p(P)
    if N % P:
        check(TP_ERR_INDIVISIBLE)
    if y_mode == TP_Y_SHARDS:
        yp, ldy = _block_out(Y, P, M, N // P)
    else:
        yp, _, _, ldy = _mat(Y, "Y")
        _expect_shape(Y, (M, N), "Y")
    _same_gpu(X, W, Y)
    check(_get_lib().tp_linear_column(xp, ldx, wp, ldw, yp, ldy, y_mode, M, N, K, P, dt,
                               _stream(X, stream)))


def tp_row_workspace_bytes(mode: int, M: int, N: int, P: int) -> int:
    return int(_get_lib().tp_row_workspace_bytes(mode, M, N, P))


def tp_workspace_zero(buf, stream=None) -> None:
    _same_gpu(buf)
    check(_get_lib().tp_workspace_zero(buf.data_ptr(), buf.numel() * buf.element_size(),
                                _stream(buf, stream)))


def tp_linear_row(X, W, Y, P: int, mode: int = TP_ROW_SUM, workspace=None,
                  y_slice_stride: int = 0, stream=None) -> None:
    """Row-parallel Linear.  X [M, K], W [N, K].  Y: TP_ROW_PARTIAL ->
    float32 [P, M, N]; TP_ROW_SUM / TP_ROW_FUSED -> [M, N]; TP_ROW_SCATTER ->
    [M, N] whose row blocks are the slices (y_slice_stride = 0), or a buffer
    with slice j at element offset j*y_slice_stride and rows [:M/P] of its
    2-D view Y."""
    xp, M, K, ldx = _mat(X, "X")
    wp, N, Kw, ldw = _mat(W, "W")
    if Kw != K:
        raise ValueError(f"X has K={K} but W has K={Kw}")
    dt = _dtype_code(X)
    if _dtype_code(W) != dt:
        raise TypeError("X and W must share one dtype")
    _check_p(P)
    if mode == TP_ROW_PARTIAL:
        import torch
        if Y.dtype != torch.float32:
            raise ValueError("Y must be float32 [P, M, N] for TP_ROW_PARTIAL")
        yp, ldy = _block_out(Y, P, M, N)
    else:
        if _dtype_code(Y) != dt:
            raise TypeError("Y must have the dtype of X")
        yp, ldy = _scatter_out(Y, M, N, P, mode == TP_ROW_SCATTER, y_slice_stride)
    if workspace is not None:
        wsp, wsb = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    else:
        wsp, wsb = None, 0
    _same_gpu(X, W, Y, workspace)
    check(_get_lib().tp_linear_row(xp, ldx, wp, ldw, yp, ldy, y_slice_stride, mode, wsp, wsb,
                            M, N, K, P, dt, _stream(X, stream)))


def tp_linear_row_noalloc(X, W, Y, P: int, mode: int = TP_ROW_SUM, y_slice_stride: int = 0,
                          stream=None) -> None:
    """tp_linear_row without a workspace argument: the library's fixed
    per-GPU array of TP_NOALLOC_SCRATCH_BYTES serves as the workspace, so
    nothing is allocated (calls that may overlap on one GPU race on it).
    Shapes whose workspace would exceed it raise TPError(TP_ERR_WORKSPACE)."""
    xp, M, K, ldx = _mat(X, "X")
    wp, N, Kw, ldw = _mat(W, "W")
    if Kw != K:
        raise ValueError(f"X has K={K} but W has K={Kw}")
    dt = _dtype_code(X)
    if _dtype_code(W) != dt:
        raise TypeError("X and W must share one dtype")
    _check_p(P)
    if mode == TP_ROW_PARTIAL:
        import torch
        if Y.dtype != torch.float32:
            raise ValueError("Y must be float32 [P, M, N] for TP_ROW_PARTIAL")
        yp, ldy = _block_out(Y, P, M, N)
    else:
        if _dtype_code(Y) != dt:
            raise TypeError("Y must have the dtype of X")
        yp, ldy = _scatter_out(Y, M, N, P, mode == TP_ROW_SCATTER, y_slice_stride)
    _same_gpu(X, W, Y)
    check(_get_lib().tp_linear_row_noalloc(xp, ldx, wp, ldw, yp, ldy, y_slice_stride, mode,
                                           M, N, K, P, dt, _stream(X, stream)))


def tp_shard_reduce(partials, Y, P: int, scatter: int = 0, y_slice_stride: int = 0,
                    stream=None) -> None:
    """Fold float32 partials [P, M, N] (or any [P, M, ldp] view) into Y [M, N]
    (scatter=0) or into P token slices (scatter=1)."""
    import torch
    _check_p(P)
    if partials.dtype != torch.float32 or partials.dim() != 3 or partials.shape[0] != P:
        raise ValueError("partials must be float32 [P, M, N]")
    _, M, N, ldp = _mat(partials[0], "partials[0]")
    ss = partials.stride(0) if P > 1 else M * ldp
    yp, ldy = _scatter_out(Y, M, N, P, scatter, y_slice_stride)
    _same_gpu(partials, Y)
    check(_get_lib().tp_shard_reduce(partials.data_ptr(), ss, ldp, yp, ldy, y_slice_stride, scatter,
                              M, N, P, _dtype_code(Y), _stream(partials, stream)))


def tp_linear_column_ex(X, W, Y, P: int, y_mode: int = TP_Y_CONCAT, bias=None,
                        act: int = TP_ACT_NONE, x_slices=None, stream=None) -> None:
    """Column-parallel Linear with a bias, the gated unit and token-slice
    input.  Exactly one of X ([M, K]) and x_slices (P tensors [M/P, K] with
    one row stride) is given.  W [N, K]; bias [N] or None.  Output columns per
    shard On = N/P, or N/(2P) with TP_ACT_SWIGLU; Y [M, P*On] for TP_Y_CONCAT
    or [P, M, On] for TP_Y_SHARDS."""
    _check_p(P)
    if (X is None) == (x_slices is None):
        raise ValueError("give exactly one of X and x_slices")
    if X is not None:
        xp, M, K, ldx = _mat(X, "X")
        ref = X
        sl = None
    else:
        if len(x_slices) != P:
            raise ValueError(f"x_slices must hold P={P} tensors")
        _, ms, K, ldx = _mat(x_slices[0], "x_slices[0]")
        for j, t in enumerate(x_slices):
            _, mj, kj, lj = _mat(t, f"x_slices[{j}]")
            if (mj, kj) != (ms, K) or (mj > 1 and lj != ldx):
                raise ValueError("token slices must share shape and row stride")
            if _dtype_code(t) != _dtype_code(x_slices[0]):
                raise TypeError("token slices must share one dtype")
        M, xp, ref = ms * P, None, x_slices[0]
        sl = _ptr_array(x_slices, "x_slices")
    wp, N, Kw, ldw = _mat(W, "W")
    if Kw != K:
        raise ValueError(f"X has K={K} but W has K={Kw}")
    dt = _dtype_code(ref)
    if _dtype_code(W) != dt or _dtype_code(Y) != dt:
        raise TypeError("X, W and Y must share one dtype")
    if N % P or (act == TP_ACT_SWIGLU and (N // P) % 2):
        check(TP_ERR_INDIVISIBLE)
    On = N // P // 2 if act == TP_ACT_SWIGLU else N // P
    if bias is not None:
        _expect_shape(bias, (N,), "bias")
    if y_mode == TP_Y_SHARDS:
        yp, ldy = _block_out(Y, P, M, On)
    else:
        yp, _, _, ldy = _mat(Y, "Y")
        _expect_shape(Y, (M, P * On), "Y")
    _same_gpu(X, W, Y, bias, x_slices)
    check(_get_lib().tp_linear_column_ex(xp, sl, ldx, wp, ldw, _bias_ptr(bias, dt), yp, ldy,
                                         y_mode, act, M, N, K, P, dt, _stream(ref, stream)))


def tp_linear_row_ex(X, W, Y, P: int, mode: int = TP_ROW_SUM, workspace=None, bias=None,
                     y_slices=None, y_slice_stride: int = 0, stream=None) -> None:
    """Row-parallel Linear with the row bias (added once after the fold) and,
    for TP_ROW_SCATTER, token slices in separate tensors (y_slices: P tensors
    [M/P, N] with one row stride; Y is then None).  Otherwise as
    tp_linear_row."""
    _check_p(P)
    xp, M, K, ldx = _mat(X, "X")
    wp, N, Kw, ldw = _mat(W, "W")
    if Kw != K:
        raise ValueError(f"X has K={K} but W has K={Kw}")
    dt = _dtype_code(X)
    if _dtype_code(W) != dt:
        raise TypeError("X and W must share one dtype")
    if bias is not None:
        _expect_shape(bias, (N,), "bias")
    ys = None
    if y_slices is not None:
        if Y is not None:
            raise ValueError("give Y or y_slices, not both")
        if len(y_slices) != P:
            raise ValueError(f"y_slices must hold P={P} tensors")
        if M % P:
            check(TP_ERR_INDIVISIBLE)
        _, _, _, ldy = _mat(y_slices[0], "y_slices[0]")
        for j, t in enumerate(y_slices):
            _, mj, nj, lj = _mat(t, f"y_slices[{j}]")
            if (mj, nj) != (M // P, N) or (mj > 1 and lj != ldy) or _dtype_code(t) != dt:
                raise ValueError("y_slices must be [M/P, N] of the input dtype, one row stride")
        yp, ys = None, _ptr_array(y_slices, "y_slices")
    elif mode == TP_ROW_PARTIAL:
        import torch
        if Y.dtype != torch.float32:
            raise ValueError("Y must be float32 [P, M, N] for TP_ROW_PARTIAL")
        yp, ldy = _block_out(Y, P, M, N)
    else:
        if _dtype_code(Y) != dt:
            raise TypeError("Y must have the dtype of X")
        yp, ldy = _scatter_out(Y, M, N, P, mode == TP_ROW_SCATTER, y_slice_stride)
    if workspace is not None:
        wsp, wsb = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    else:
        wsp, wsb = None, 0
    _same_gpu(X, W, Y, workspace, bias, y_slices)
    check(_get_lib().tp_linear_row_ex(xp, ldx, wp, ldw, _bias_ptr(bias, dt), yp, ys, ldy,
                                      y_slice_stride, mode, wsp, wsb, M, N, K, P, dt,
                                      _stream(X, stream)))


def tp_shard_reduce_ex(partials, Y, P: int, scatter: int = 0, bias=None, y_slices=None,
                       y_slice_stride: int = 0, stream=None) -> None:
    """tp_shard_reduce with the row bias and, for scatter=1, token slices in
    separate tensors (y_slices: P tensors [M/P, N], one row stride; Y None)."""
    import torch
    _check_p(P)
    if partials.dtype != torch.float32 or partials.dim() != 3 or partials.shape[0] != P:
        raise ValueError("partials must be float32 [P, M, N]")
    _, M, N, ldp = _mat(partials[0], "partials[0]")
    ss = partials.stride(0) if P > 1 else M * ldp
    if bias is not None:
        _expect_shape(bias, (N,), "bias")
    if y_slices is not None:
        if Y is not None:
            raise ValueError("give Y or y_slices, not both")
        if len(y_slices) != P:
            raise ValueError(f"y_slices must hold P={P} tensors")
        if M % P:
            check(TP_ERR_INDIVISIBLE)
        _, _, _, ldy = _mat(y_slices[0], "y_slices[0]")
        odt = _dtype_code(y_slices[0])
        for j, t in enumerate(y_slices):
            _, mj, nj, lj = _mat(t, f"y_slices[{j}]")
            if (mj, nj) != (M // P, N) or (mj > 1 and lj != ldy) or _dtype_code(t) != odt:
                raise ValueError("y_slices must be [M/P, N] of one dtype and row stride")
        yp, ys = None, _ptr_array(y_slices, "y_slices")
    else:
        yp, ldy = _scatter_out(Y, M, N, P, scatter, y_slice_stride)
        odt, ys = _dtype_code(Y), None
    _same_gpu(partials, Y, bias, y_slices)
    check(_get_lib().tp_shard_reduce_ex(partials.data_ptr(), ss, ldp, _bias_ptr(bias, odt), yp,
                                        ys, ldy, y_slice_stride, scatter, M, N, P, odt,
                                        _stream(partials, stream)))


def tp_embedding(ids, Y, P: int, E=None, e_shards=None, y_mode: int = TP_Y_CONCAT, bad=None,
                 stream=None) -> None:
    """Feature-sharded embedding lookup (EmbeddingWithReplicateOutput).
    ids: int64 [T].  Exactly one of E ([V, D]) and e_shards (P tensors
    [V, D/P], one row stride).  Y: [T, D] (TP_Y_CONCAT) or [P, T, D/P]
    (TP_Y_SHARDS).  bad: None or an int32 tensor set to 1 when an id is
    outside [0, V) (its output row is zero)."""
    import torch
    _check_p(P)
    if ids.dtype != torch.int64 or ids.dim() != 1 or (ids.numel() > 1 and ids.stride(0) != 1):
        raise ValueError("ids must be a contiguous int64 [T] tensor")
    T = ids.shape[0]
    if (E is None) == (e_shards is None):
        raise ValueError("give exactly one of E and e_shards")
    if E is not None:
        ep, V, D, lde = _mat(E, "E")
        dt, es = _dtype_code(E), None
    else:
        if len(e_shards) != P:
            raise ValueError(f"e_shards must hold P={P} tensors")
        _, V, Ds, lde = _mat(e_shards[0], "e_shards[0]")
        dt = _dtype_code(e_shards[0])
        for i, t in enumerate(e_shards):
            _, vi, di, li = _mat(t, f"e_shards[{i}]")
            if (vi, di) != (V, Ds) or (vi > 1 and li != lde) or _dtype_code(t) != dt:
                raise ValueError("e_shards must share shape, dtype and row stride")
        ep, D, es = None, Ds * P, _ptr_array(e_shards, "e_shards")
    if _dtype_code(Y) != dt:
        raise TypeError("Y must have the table's dtype")
    if D % P:
        check(TP_ERR_INDIVISIBLE)
    if y_mode == TP_Y_SHARDS:
        yp, ldy = _block_out(Y, P, T, D // P)
    else:
        yp, _, _, ldy = _mat(Y, "Y")
        _expect_shape(Y, (T, D), "Y")
    if bad is not None and (bad.dtype != torch.int32 or bad.numel() < 1):
        raise ValueError("bad must be an int32 tensor")
    _same_gpu(ids, Y, E, e_shards, bad)
    check(_get_lib().tp_embedding(ids.data_ptr(), T, ep, es, lde, V, D, yp, ldy, y_mode, P, dt,
                                  None if bad is None else bad.data_ptr(), _stream(ids, stream)))


def _workspace(t):
    """Pointer and bytes of a workspace, or of none."""
    if t is None:
        return None, 0
    if not t.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return t.data_ptr(), t.numel() * t.element_size()


# ---- 8-bit integers -------------------------------------------------------

def _int8_mat(t, name):
    torch = _torch()
    if t.dtype != torch.int8:
        raise TypeError(f"{name} must be int8, got {t.dtype}")
    return _mat(t, name)


def _token_scales(t, M, groups, name):
    """(pointer, row stride, scales a token) of fp32 scales [M] or [M, G], G
    one of `groups`."""
    torch = _torch()
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    shape, strides = t.shape, t.stride()
    G = shape[1] if len(shape) == 2 else 1
    if len(shape) not in (1, 2) or shape[0] != M or G not in groups:
        raise ValueError(f"{name} must have shape [{M}] or [{M}, G] with G in {groups}, "
                         f"got {tuple(shape)}")
    if G > 1 and strides[1] != 1:
        raise ValueError(f"{name} must have unit column stride")
    ld = strides[0] if M > 1 else G
    if ld < G:
        raise ValueError(f"{name} must have a row stride of at least {G}")
    return t.data_ptr(), ld, G


def _channel_scales(t, N, name):
    torch = _torch()
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    _expect_shape(t, (N,), name)
    if N > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be a contiguous 1-D tensor")
    return t.data_ptr()


def tp_quantize_rows(X, Q, scale, stream=None) -> None:
    """Rows to int8.  X [M, K] bfloat16 or float32; Q int8 [M, K]; scale
    float32 [M] or [M, G]: one scale for each row and each of G equal column
    groups (G = P for a row layer's input)."""
    xp, M, K, ldx = _mat(X, "X")
    qp, _, _, ldq = _int8_mat(Q, "Q")
    _expect_shape(Q, (M, K), "Q")
    G = scale.shape[1] if scale.dim() == 2 else 1
    _check_p(G)
    sp, lds, _ = _token_scales(scale, M, (G,), "scale")
    check(_get_lib().tp_quantize_rows(xp, ldx, qp, ldq, sp, lds, M, K, G, _dtype_code(X),
                                      _here(stream, X, Q, scale)))


def tp_linear_column_quant(X, x_scale, W, w_scale, Y, P: int, y_mode: int = TP_Y_CONCAT,
                           bias=None, act: int = TP_ACT_NONE, stream=None) -> None:
    """Column-parallel Linear on int8 operands.  X int8 [M, K] with x_scale
    float32 [M] or [M, 1]; W int8 [N, K] with w_scale float32 [N]; Y and bias
    [N] as in tp_linear_column_ex, bfloat16 or float32."""
    _check_p(P)
    xp, M, K, ldx = _int8_mat(X, "X")
    wp, N, Kw, ldw = _int8_mat(W, "W")
    if Kw != K:
        raise ValueError(f"X has K={K} but W has K={Kw}")
    dt = _dtype_code(Y)
    if N % P or (act == TP_ACT_SWIGLU and (N // P) % 2):
        check(TP_ERR_INDIVISIBLE)
    On = N // P // 2 if act == TP_ACT_SWIGLU else N // P
    sp, lds, _ = _token_scales(x_scale, M, (1,), "x_scale")
    wsp = _channel_scales(w_scale, N, "w_scale")
    if bias is not None:
        _expect_shape(bias, (N,), "bias")
    if y_mode == TP_Y_SHARDS:
        yp, ldy = _block_out(Y, P, M, On)
    else:
        yp, _, _, ldy = _mat(Y, "Y")
        _expect_shape(Y, (M, P * On), "Y")
    check(_get_lib().tp_linear_column_quant(xp, ldx, sp, lds, wp, ldw, wsp, _bias_ptr(bias, dt),
                                            yp, ldy, y_mode, act, M, N, K, P, dt,
                                            _here(stream, X, x_scale, W, w_scale, Y, bias)))


def tp_linear_row_quant(X, x_scale, W, w_scale, Y, P: int, mode: int = TP_ROW_SUM,
                        workspace=None, bias=None, y_slices=None, y_slice_stride: int = 0,
                        stream=None) -> None:
    """Row-parallel Linear on int8 operands.  X int8 [M, K] with x_scale
    float32 [M], [M, 1] or [M, P] (a scale for each token and shard); W int8
    [N, K] with w_scale float32 [N]; the rest as in tp_linear_row_ex (Y or
    y_slices bfloat16 or float32; float32 [P, M, N] for TP_ROW_PARTIAL)."""
    _check_p(P)
    xp, M, K, ldx = _int8_mat(X, "X")
    wp, N, Kw, ldw = _int8_mat(W, "W")
    if Kw != K:
        raise ValueError(f"X has K={K} but W has K={Kw}")
    sp, lds, G = _token_scales(x_scale, M, (1, P), "x_scale")
    wsp = _channel_scales(w_scale, N, "w_scale")
    if bias is not None:
        _expect_shape(bias, (N,), "bias")
    ys = None
    if y_slices is not None:
        if Y is not None:
            raise ValueError("give Y or y_slices, not both")
        if len(y_slices) != P:
            raise ValueError(f"y_slices must hold P={P} tensors")
        if M % P:
            check(TP_ERR_INDIVISIBLE)
        _, _, _, ldy = _mat(y_slices[0], "y_slices[0]")
        dt = _dtype_code(y_slices[0])
        for j, t in enumerate(y_slices):
            _, mj, nj, lj = _mat(t, f"y_slices[{j}]")
            if (mj, nj) != (M // P, N) or (mj > 1 and lj != ldy) or _dtype_code(t) != dt:
                raise ValueError("y_slices must be [M/P, N] of one dtype and row stride")
        yp, ys = None, _ptr_array(y_slices, "y_slices")
    elif mode == TP_ROW_PARTIAL:
        torch = _torch()
        if Y.dtype != torch.float32:
            raise ValueError("Y must be float32 [P, M, N] for TP_ROW_PARTIAL")
        dt = TP_F32
        yp, ldy = _block_out(Y, P, M, N)
    else:
        dt = _dtype_code(Y)
        yp, ldy = _scatter_out(Y, M, N, P, mode == TP_ROW_SCATTER, y_slice_stride)
    wkp, wkb = _workspace(workspace)
    on = _here(stream, X, x_scale, W, w_scale, Y, workspace, bias, *(y_slices or ()))
    check(_get_lib().tp_linear_row_quant(xp, ldx, sp, lds, G, wp, ldw, wsp, _bias_ptr(bias, dt),
                                         yp, ys, ldy, y_slice_stride, mode, wkp, wkb, M, N, K, P,
                                         dt, on))


# ---- heads of a fused QKV layer -------------------------------------------

def _qkv(X, P, Hq, Hkv, x_mode, name):
    """(pointer, row stride, T, D) of a fused QKV layer's output: [T, N] or
    [P, T, N/P], N = (Hq + 2 Hkv) D."""
    _check_p(P)
    if Hq < 0 or Hkv < 0 or Hq + Hkv < 1:
        raise ValueError(f"Hq={Hq} and Hkv={Hkv} heads: at least one head is needed")
    if Hq % P or Hkv % P:
        check(TP_ERR_INDIVISIBLE)
    shards = x_mode == TP_Y_SHARDS
    shape = X.shape
    if len(shape) != (3 if shards else 2) or (shards and shape[0] != P):
        raise ValueError(f"{name} must be [T, N], or [P, T, N/P] with TP_Y_SHARDS, got "
                         f"{tuple(shape)}")
    T, cols = shape[-2], shape[-1]
    heads = (Hq + 2 * Hkv) // (P if shards else 1)
    if cols == 0 or cols % heads:
        raise ValueError(f"{name} has {cols} columns: not a multiple of its {heads} heads")
    if shards:
        xp, ld = _block_out(X, P, T, cols, name)
    else:
        xp, _, _, ld = _mat(X, name)
    return xp, ld, T, cols // heads


def _rows(t, T, cols, dt, name):
    """(pointer, row stride) of a [T, cols] tensor of dtype code dt, or of
    none."""
    if t is None:
        return None, 0
    p, rows, n, ld = _mat(t, name)
    if rows != T or n != cols:
        _expect_shape(t, (T, cols), name)
    if _DTYPES.get(t.dtype) != dt:
        raise TypeError(f"{name} must have the dtype of the QKV matrix")
    return p, ld


def _rotation(cos, sin, q_weight, k_weight, D, dt, eps, style):
    """The rotation's and norms' arguments in the order of the C calls."""
    n_pos = R = 0
    cp = sp = wq = wk = None
    if cos is not None and sin is not None:
        shape, f32 = cos.shape, _torch().float32
        if cos.dtype != f32 or sin.dtype != f32 or len(shape) != 2 or not (
                cos.is_contiguous() and sin.is_contiguous()):
            raise ValueError("cos and sin must be contiguous float32 [n_pos, R/2] tensors")
        if sin.shape != shape:
            _expect_shape(sin, shape, "sin")
        n_pos, R = shape[0], 2 * shape[1]
        cp, sp = cos.data_ptr(), sin.data_ptr()
    elif cos is not sin:
        raise ValueError("give both cos and sin, or neither")
    if q_weight is not None:
        wq = _weight(q_weight, D, dt, "q_weight")
    if k_weight is not None:
        wk = _weight(k_weight, D, dt, "k_weight")
    return cp, sp, n_pos, R, style, wq, wk, eps


def _weight(t, D, dt, name):
    if t.shape != (D,):
        _expect_shape(t, (D,), name)
    if D > 1 and t.stride(0) != 1:
        raise ValueError(f"{name} must be a contiguous 1-D tensor")
    if _DTYPES.get(t.dtype) != dt:
        raise TypeError(f"{name} must have the dtype of the QKV matrix")
    return t.data_ptr()


def _positions(pos, T, R):
    if pos is None:
        if R:
            raise ValueError("pos is needed where heads are rotated")
        return None
    if pos.shape != (T,):
        _expect_shape(pos, (T,), "pos")
    if pos.dtype != _torch().int64 or (T > 1 and pos.stride(0) != 1):
        raise ValueError("pos must be a contiguous int64 [T] tensor")
    return pos.data_ptr()


def _flag(bad):
    if bad is None:
        return None
    if bad.dtype != _torch().int32 or bad.numel() < 1:
        raise ValueError("bad must be an int32 tensor")
    return bad.data_ptr()


def tp_qk_norm_rope(X, pos, cos, sin, Q, K, P: int, Hq: int, Hkv: int, q_weight=None,
                    k_weight=None, eps: float = 1e-6, style: int = TP_ROPE_HALVES,
                    x_mode: int = TP_Y_CONCAT, bad=None, stream=None) -> None:
    """Norm and rotation of the query and key heads of a fused QKV layer's
    output X ([T, N], or [P, T, N/P] with x_mode TP_Y_SHARDS).  pos int64 [T];
    cos, sin float32 [n_pos, R/2] (None: no rotation); q_weight, k_weight [D]
    (None: no norm); Q [T, Hq*D] and K [T, Hkv*D], either may be None.  A
    position outside the table gives zero rows and sets bad (int32)."""
    xp, ldx, T, D = _qkv(X, P, Hq, Hkv, x_mode, "X")
    dt = _dtype_code(X)
    rot = _rotation(cos, sin, q_weight, k_weight, D, dt, eps, style)
    pp = _positions(pos, T, rot[3])
    qp, ldq = _rows(Q, T, Hq * D, dt, "Q")
    kp, ldk = _rows(K, T, Hkv * D, dt, "K")
    on = _here(stream, X, pos, cos, sin, Q, K, q_weight, k_weight, bad)
    check(_get_lib().tp_qk_norm_rope(xp, ldx, x_mode, pp, *rot, qp, ldq, kp, ldk, T, Hq, Hkv, D, P,
                                     dt, _flag(bad), on))


def tp_qk_norm_rope_workspace_bytes(T: int, D: int) -> int:
    return int(_get_lib().tp_qk_norm_rope_workspace_bytes(T, D))


def tp_qk_norm_rope_backward(X, pos, cos, sin, dQ, dK, dX, P: int, Hq: int, Hkv: int, dV=None,
                             q_weight=None, k_weight=None, dq_weight=None, dk_weight=None,
                             workspace=None, eps: float = 1e-6, style: int = TP_ROPE_HALVES,
                             x_mode: int = TP_Y_CONCAT, bad=None, stream=None) -> None:
    """Gradients of tp_qk_norm_rope: dX (the layout of X) from dQ [T, Hq*D], dK
    and dV [T, Hkv*D] (dV is copied into the value features; a part whose
    gradient is None is left as it is), and the weights' gradients dq_weight,
    dk_weight (float32 [D], or None), which need a workspace of
    tp_qk_norm_rope_workspace_bytes(T, D).  X may be None without a norm."""
    torch = _torch()
    dxp, lddx, T, D = _qkv(dX, P, Hq, Hkv, x_mode, "dX")
    dt = _dtype_code(dX)
    xp, ldx = None, lddx
    if X is not None:
        xp, ldx, _, _ = _qkv(X, P, Hq, Hkv, x_mode, "X")
        _expect_shape(X, dX.shape, "X")
        if _dtype_code(X) != dt:
            raise TypeError("X and dX must share one dtype")
    rot = _rotation(cos, sin, q_weight, k_weight, D, dt, eps, style)
    pp = _positions(pos, T, rot[3])
    qp, ldq = _rows(dQ, T, Hq * D, dt, "dQ")
    kp, ldk = _rows(dK, T, Hkv * D, dt, "dK")
    vp, ldv = _rows(dV, T, Hkv * D, dt, "dV")
    for t, name in ((dq_weight, "dq_weight"), (dk_weight, "dk_weight")):
        if t is not None:
            _expect_shape(t, (D,), name)
            if t.dtype != torch.float32 or (D > 1 and t.stride(0) != 1):
                raise ValueError(f"{name} must be a contiguous float32 [D] tensor")
    wkp, wkb = _workspace(workspace)
    on = _here(stream, dX, X, pos, cos, sin, dQ, dK, dV, q_weight, k_weight, dq_weight, dk_weight,
               workspace, bad)
    check(_get_lib().tp_qk_norm_rope_backward(
        xp, ldx, x_mode, pp, *rot, qp, ldq, kp, ldk, vp, ldv, dxp, lddx,
        None if dq_weight is None else dq_weight.data_ptr(),
        None if dk_weight is None else dk_weight.data_ptr(), wkp, wkb, T, Hq, Hkv, D, P, dt,
        _flag(bad), on))


def tp_kv_append(X, cos, sin, past, cu, table, k_cache, v_cache, P: int, Hq: int, Hkv: int,
                 Q=None, q_weight=None, k_weight=None, eps: float = 1e-6,
                 style: int = TP_ROPE_HALVES, x_mode: int = TP_Y_CONCAT, bad=None,
                 stream=None) -> None:
    """Append the keys (normed, rotated) and values of a fused QKV layer's
    output X to a paged cache, and with Q ([T, Hq*D]) write the queries.
    past int32 [B], cu int32 [B + 1], table int32 [B, max_pages]; k_cache and
    v_cache [n_pages, page_size, Hkv, D] views of one set of strides with
    contiguous features (a permuted view gives another order in memory)."""
    torch = _torch()
    xp, ldx, T, D = _qkv(X, P, Hq, Hkv, x_mode, "X")
    dt = _dtype_code(X)
    rot = _rotation(cos, sin, q_weight, k_weight, D, dt, eps, style)
    i32 = torch.int32
    if past.dtype != i32 or cu.dtype != i32 or past.dim() != 1 or cu.dim() != 1 or not (
            past.is_contiguous() and cu.is_contiguous()):
        raise ValueError("past [B] and cu [B + 1] must be int32 with unit stride")
    B = past.shape[0]
    if cu.shape[0] != B + 1:
        _expect_shape(cu, (B + 1,), "cu")
    tp, rows, max_pages, ldt = _mat(table, "table")
    if table.dtype != i32 or rows != B:
        raise ValueError(f"table must be int32 [{B}, max_pages]")
    shape, strides = k_cache.shape, k_cache.stride()
    if len(shape) != 4 or shape[2] != Hkv or shape[3] != D:
        raise ValueError(f"k_cache must be [n_pages, page_size, {Hkv}, {D}]")
    _expect_shape(v_cache, shape, "v_cache")
    if D > 1 and strides[3] != 1:
        raise ValueError("k_cache and v_cache must have contiguous features")
    if strides != v_cache.stride():
        raise ValueError("k_cache and v_cache must have the same strides")
    if _dtype_code(k_cache) != dt or _dtype_code(v_cache) != dt:
        raise TypeError("k_cache and v_cache must have the dtype of the QKV matrix")
    qp, ldq = _rows(Q, T, Hq * D, dt, "Q")
    on = _here(stream, X, cos, sin, past, cu, table, k_cache, v_cache, Q, q_weight, k_weight, bad)
    check(_get_lib().tp_kv_append(
        xp, ldx, x_mode, *rot, cu.data_ptr(), past.data_ptr(), B, tp, ldt, max_pages,
        k_cache.data_ptr(), v_cache.data_ptr(), shape[0], shape[1], strides[0], strides[1],
        strides[2], qp, ldq, T, Hq, Hkv, D, P, dt, _flag(bad), on))
