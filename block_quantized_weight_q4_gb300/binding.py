"""ctypes binding over libqmv.so (C ABI declared in include/qmv.h).

Argument marshalling only: tensors are passed as raw device pointers with the current
torch CUDA stream; every step of the computation runs in the library's kernels.  If the
library has not been built, every call raises: there is no CPU fallback.

Format (Krafla ".mlb model format v1", "Body"): a matrix image is the q array, zero
padding to 64 bytes, then the d array; W below is a uint8 CUDA tensor holding it.
"""
from __future__ import annotations

import ctypes
import os

Q8_0 = 1
Q4_0 = 2
SCALE_F32 = 0
SCALE_F16 = 1
X_F32 = 0
X_BF16 = 1

OK = 0
E_FORMAT = 2
E_SHAPE = 3
E_ARG = 4
E_ALIGN = 5
E_CUDA = 6
E_TIMEOUT = 7

_HERE = os.path.dirname(os.path.abspath(__file__))
_lib = None


class QmvError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: status {status} ({strerror(status)})")


def library_path() -> str:
    return os.path.join(_HERE, "libqmv.so")


def load_library():
    """Load libqmv.so (raises OSError if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    path = library_path()
    if not os.path.exists(path):
        raise OSError(f"libqmv.so not built ({path}); run block_quantized_weight_q4_gb300.build")
    lib = ctypes.CDLL(path)
    i64, i32, vp, sz = ctypes.c_int64, ctypes.c_int, ctypes.c_void_p, ctypes.c_size_t
    lib.qmv_weight_bytes.restype = sz
    lib.qmv_weight_bytes.argtypes = [i32, i32, i64, i64]
    lib.qmv_scale_offset.restype = i64
    lib.qmv_scale_offset.argtypes = [i32, i32, i64, i64]
    lib.qmv_matrix_wtype.restype = i32
    lib.qmv_matrix_wtype.argtypes = [i32, ctypes.c_uint32, i32, i32]
    lib.qmv_matvec.restype = i32
    lib.qmv_matvec.argtypes = [i32, i32, i64, i64, vp, vp, i32, vp, i32, vp]
    lib.qmv_matvec_grouped.restype = i32
    lib.qmv_matvec_grouped.argtypes = [i32, i32, i32, i32, vp, i32, ctypes.c_uint, vp]
    lib.qmv_matvec_grouped_noalloc.argtypes = [i32, i32, i32, i32, vp, i32, ctypes.c_uint, vp]
    lib.qmv_matvec_glu.restype = i32
    lib.qmv_matvec_glu.argtypes = [i32, i32, i64, i64, vp, vp, vp, i32, i32, vp, ctypes.c_uint, vp]
    lib.qmv_dequant.restype = i32
    lib.qmv_dequant.argtypes = [i32, i32, i64, i64, vp, vp, vp]
    lib.qmv_validate.restype = i32
    lib.qmv_validate.argtypes = [i32, i32, i64, i64, vp, vp, vp]
    lib.qmv_quantize.restype = i32
    lib.qmv_quantize.argtypes = [i32, i32, i64, i64, vp, vp, vp, vp]
    lib.qmv_step_create.restype = i32
    lib.qmv_step_create.argtypes = [vp, i32, vp, i32, vp, i32, ctypes.POINTER(vp)]
    lib.qmv_step_run.restype = i32
    lib.qmv_step_run.argtypes = [vp, vp]
    lib.qmv_step_run_wait.restype = i32
    lib.qmv_step_run_wait.argtypes = [vp, vp]
    lib.qmv_step_destroy.restype = i32
    lib.qmv_step_destroy.argtypes = [vp]
    lib.qmv_step_create_gated.restype = i32
    lib.qmv_step_create_gated.argtypes = [vp, i32, vp, i32, vp, i32, ctypes.POINTER(vp)]
    lib.qmv_step_open.restype = i32
    lib.qmv_step_open.argtypes = [vp]
    lib.qmv_step_wait.restype = i32
    lib.qmv_step_wait.argtypes = [vp, ctypes.c_longlong]
    lib.qmv_step_open_wait.restype = i32
    lib.qmv_step_open_wait.argtypes = [vp, vp, vp, ctypes.c_longlong]
    lib.qmv_gguf_bytes.restype = ctypes.c_size_t
    lib.qmv_gguf_bytes.argtypes = [i32, i64, i64]
    lib.qmv_gguf_to_mlb.restype = i32
    lib.qmv_gguf_to_mlb.argtypes = [i32, i64, i64, vp, vp, vp]
    lib.qmv_quantize_q4_fit.restype = i32
    lib.qmv_quantize_q4_fit.argtypes = [i32, i64, i64, vp, vp, vp, vp]
    lib.qmv_quantize_x.restype = i32
    lib.qmv_quantize_x.argtypes = [i32, i64, i64, vp, vp, vp]
    lib.qmv_matvec_qx_grouped.restype = i32
    lib.qmv_matvec_qx_grouped.argtypes = [i32, i32, i32, i32, vp, i32, ctypes.c_uint, vp]
    lib.qmv_matvec_qx.restype = i32
    lib.qmv_matvec_qx.argtypes = [i32, i32, i64, i64, vp, vp, vp, i32, vp]
    f32 = ctypes.c_float
    lib.qmv_rmsnorm.restype = i32
    lib.qmv_rmsnorm.argtypes = [i32, i64, i64, vp, vp, vp, vp, f32, i32, vp, vp]
    lib.qmv_kv_write.restype = i32
    lib.qmv_kv_write.argtypes = [vp, vp, i32, vp, i64, vp, i64, vp]
    lib.qmv_kv_read.restype = i32
    lib.qmv_kv_read.argtypes = [vp, vp, i32, vp, vp, vp]
    lib.qmv_attend.restype = i32
    lib.qmv_attend.argtypes = [vp, vp, i32, i32, vp, i64, f32, i32, i32, vp, i64, vp]
    lib.qmv_logprobs.restype = i32
    lib.qmv_logprobs.argtypes = [i64, i64, vp, i64, vp, i32, vp, vp, i32, vp, vp, vp]
    lib.qmv_sample.restype = i32
    lib.qmv_sample.argtypes = [i64, i64, vp, i64, vp, i64, vp, vp, vp, vp, vp, vp]
    lib.qmv_embed.restype = i32
    lib.qmv_embed.argtypes = [i32, i32, i64, i64, vp, vp, i64, f32, i32, vp, vp]
    lib.qmv_qk_rope.restype = i32
    lib.qmv_qk_rope.argtypes = [i32, i64, i32, i32, i32, vp, i64, vp, i64, vp, vp, f32, vp, vp, i32, i32, f32, i32, vp, i64, vp, i64, vp]
    lib.qmv_moe_scratch_bytes.restype = sz
    lib.qmv_moe_scratch_bytes.argtypes = [i64, i32, i64, i32]
    lib.qmv_moe.restype = i32
    lib.qmv_moe.argtypes = [vp, i64, vp, i64, i32, i32, f32, i32, i32, vp, i32, vp, vp, vp, vp, vp]
    lib.qmv_check_device.restype = i32
    lib.qmv_check_device.argtypes = []
    lib.qmv_strerror.restype = ctypes.c_char_p
    lib.qmv_strerror.argtypes = [i32]
    _lib = lib
    return lib


def strerror(status: int) -> str:
    try:
        return load_library().qmv_strerror(status).decode()
    except OSError:
        return "libqmv not loaded"


def _check(status: int, where: str):
    if status != OK:
        raise QmvError(status, where)


def _stream(stream):
    """The stream's handle as an integer; the current device's current stream by default (asked for as a
    handle: making torch's stream object takes about 3 us of the host's time a call)."""
    if stream is not None:
        return stream.cuda_stream
    import torch
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())


def _x_dtype(x) -> int:
    import torch
    if x.dtype == torch.float32:
        return X_F32
    if x.dtype == torch.bfloat16:
        return X_BF16
    raise TypeError("x must be float32 or bfloat16")


def weight_bytes(wtype: int, scale_dtype: int, rows: int, cols: int) -> int:
    return int(load_library().qmv_weight_bytes(wtype, scale_dtype, rows, cols))


def scale_offset(wtype: int, scale_dtype: int, rows: int, cols: int) -> int:
    return int(load_library().qmv_scale_offset(wtype, scale_dtype, rows, cols))


def matrix_wtype(file_wtype: int, q8_mask: int, class_bit: int, shared_classifier: bool = False) -> int:
    return int(load_library().qmv_matrix_wtype(file_wtype, q8_mask, class_bit, int(bool(shared_classifier))))


def matvec(wtype: int, scale_dtype: int, rows: int, cols: int, W, x, y=None, stream=None):
    """y = W x.  W: uint8 CUDA tensor (matrix image); x: (batch, cols) float32/bfloat16
    CUDA tensor; y: optional (batch, rows) float32 CUDA tensor.  Returns y."""
    import torch
    if x.dim() == 1:
        x = x.unsqueeze(0)
    batch = x.shape[0]
    if x.shape[1] != cols or not x.is_contiguous():
        raise ValueError("x must be a contiguous (batch, cols) tensor")
    if y is None:
        y = torch.empty((batch, rows), dtype=torch.float32, device=x.device)
    if y.dtype != torch.float32 or tuple(y.shape) != (batch, rows) or not y.is_contiguous():
        raise ValueError("y must be a contiguous float32 (batch, rows) tensor")
    st = load_library().qmv_matvec(wtype, scale_dtype, rows, cols, W.data_ptr(), x.data_ptr(), _x_dtype(x),
                                   y.data_ptr(), batch, _stream(stream))
    _check(st, "qmv_matvec")
    return y


class Problem(ctypes.Structure):
    """qmv_problem of include/qmv.h."""
    _fields_ = [("rows", ctypes.c_int64), ("cols", ctypes.c_int64), ("W", ctypes.c_void_p),
                ("x", ctypes.c_void_p), ("y", ctypes.c_void_p)]


FLAG_OVERLAP = 1
FLAG_BF16_WEIGHTS = 2
MAX_GROUP = 8
X_SILU_GLU_F32 = 2
X_GELU_GLU_F32 = 3
X_BF16_PAIR = 4
ACTS = {"silu": X_SILU_GLU_F32, "gelu": X_GELU_GLU_F32}
ACT_SILU = 0
ACT_GELU_TANH = 1
ACT_CODES = {"silu": ACT_SILU, "gelu": ACT_GELU_TANH}
NOALLOC_MAX_BATCH = 8


def _problem_array(problems, act=None, pair=False):
    """act: None, or "silu" / "gelu" for gated activations (x of each problem: float32
    (2, batch, cols), gate then up).  pair: one vector given as bfloat16 (2, cols), hi parts
    then lo parts (the layout matvec_glu writes)."""
    n = len(problems)
    if not 1 <= n <= MAX_GROUP:
        raise ValueError("1..8 problems per group")
    arr = (Problem * n)()
    if pair:
        import torch
        for i, (rows, cols, W, x, y) in enumerate(problems):
            if x.dtype != torch.bfloat16 or tuple(x.shape) != (2, cols) or not x.is_contiguous():
                raise ValueError("a pair x is a contiguous bfloat16 (2, cols) tensor: hi, lo")
            if tuple(y.shape) != (1, rows) or not y.is_contiguous():
                raise ValueError("y must be a contiguous (1, rows) tensor")
            arr[i] = Problem(rows, cols, W.data_ptr(), x.data_ptr(), y.data_ptr())
        return arr, n, 1, X_BF16_PAIR
    if act is not None:
        import torch
        if act not in ACTS:
            raise ValueError("act must be 'silu' or 'gelu'")
        batch = problems[0][3].shape[1]
        for (rows, cols, W, x, y) in problems:
            if x.dtype != torch.float32 or tuple(x.shape) != (2, batch, cols):
                raise ValueError("gated activations need float32 x of shape (2, batch, cols)")
        xdt = ACTS[act]
    else:
        batch = problems[0][3].shape[0]
        xdt = _x_dtype(problems[0][3])
    for i, (rows, cols, W, x, y) in enumerate(problems):
        xshape = (2, batch, cols) if act is not None else (batch, cols)
        xdt_i = xdt if act is not None else _x_dtype(x)
        if tuple(x.shape) != xshape or tuple(y.shape) != (batch, rows) or xdt_i != xdt:
            raise ValueError("every problem needs x (batch, cols) of one dtype and y (batch, rows)")
        if not (x.is_contiguous() and y.is_contiguous()):
            raise ValueError("x and y must be contiguous")
        arr[i] = Problem(rows, cols, W.data_ptr(), x.data_ptr(), y.data_ptr())
    return arr, n, batch, xdt


def _flags(overlap: bool, bf16_weights: bool = False) -> int:
    return (FLAG_OVERLAP if overlap else 0) | (FLAG_BF16_WEIGHTS if bf16_weights else 0)


def matvec_grouped(wtype: int, scale_dtype: int, problems, overlap: bool = False, stream=None, act=None,
                   bf16_weights: bool = False, pair: bool = False):
    """Several products in one launch.  problems: list of (rows, cols, W, x, y) with W a
    uint8 CUDA tensor, x (batch, cols) and y (batch, rows) CUDA tensors; all share wtype,
    scale_dtype, the x dtype and batch.  overlap: QMV_FLAG_OVERLAP (the weights must not be
    written by the preceding kernel on the stream).  act: "silu" / "gelu" for gated
    activations, x then float32 (2, batch, cols): gate, up; the product takes act(gate) * up.
    bf16_weights: QMV_FLAG_BF16_WEIGHTS (prefill passes round each weight once to bfloat16).
    pair: each x is one vector as a bfloat16 (2, cols) pair (QMV_X_BF16_PAIR), y (1, rows)."""
    arr, n, batch, xdt = _problem_array(problems, act, pair)
    st = load_library().qmv_matvec_grouped(wtype, scale_dtype, xdt, batch, ctypes.addressof(arr), n,
                                           _flags(overlap, bf16_weights), _stream(stream))
    _check(st, "qmv_matvec_grouped")


def matvec_glu(wtype: int, scale_dtype: int, rows: int, cols: int, W1, W3, x, act: str = "silu", h=None,
               overlap: bool = False, stream=None):
    """The FFN's gate and up projections with the gated activation as their epilogue
    (qmv_matvec_glu): x a bfloat16 (cols,) or (1, cols) CUDA tensor; returns h, a bfloat16 (2, rows)
    CUDA tensor holding act(W1 x) * (W3 x) as hi and lo parts (the pair layout matvec_grouped
    takes with pair=True)."""
    import torch
    if act not in ACT_CODES:
        raise ValueError("act must be 'silu' or 'gelu'")
    if x.dtype != torch.bfloat16 or x.numel() != cols or not x.is_contiguous():
        raise ValueError("x must be one contiguous bfloat16 vector of cols values")
    if h is None:
        h = torch.empty((2, rows), dtype=torch.bfloat16, device=x.device)
    if h.dtype != torch.bfloat16 or tuple(h.shape) != (2, rows) or not h.is_contiguous():
        raise ValueError("h must be a contiguous bfloat16 (2, rows) tensor")
    st = load_library().qmv_matvec_glu(wtype, scale_dtype, rows, cols, W1.data_ptr(), W3.data_ptr(), x.data_ptr(),
                                       X_BF16, ACT_CODES[act], h.data_ptr(), FLAG_OVERLAP if overlap else 0,
                                       _stream(stream))
    _check(st, "qmv_matvec_glu")
    return h


def matvec_grouped_noalloc(wtype: int, scale_dtype: int, problems, overlap: bool = False, stream=None):
    """matvec_grouped that allocates no device memory (qmv_matvec_grouped_noalloc): bfloat16
    x, at most NOALLOC_MAX_BATCH vectors, cols % 256 == 0; its scratch is one fixed array
    in the library, so calls that may overlap in time must be ordered on one stream."""
    arr, n, batch, xdt = _problem_array(problems)
    st = load_library().qmv_matvec_grouped_noalloc(wtype, scale_dtype, xdt, batch, ctypes.addressof(arr), n,
                                                   FLAG_OVERLAP if overlap else 0, _stream(stream))
    _check(st, "qmv_matvec_grouped_noalloc")


class Copy(ctypes.Structure):
    """qmv_copy of include/qmv.h."""
    _fields_ = [("dst", ctypes.c_void_p), ("src", ctypes.c_void_p), ("bytes", ctypes.c_size_t)]


class Group(ctypes.Structure):
    """qmv_group of include/qmv.h."""
    _fields_ = [("wtype", ctypes.c_int), ("scale_dtype", ctypes.c_int), ("x_dtype", ctypes.c_int),
                ("batch", ctypes.c_int), ("problems", ctypes.c_void_p), ("n", ctypes.c_int),
                ("flags", ctypes.c_uint)]


def _copies(pairs):
    arr = (Copy * max(len(pairs), 1))()
    for i, (dst, src) in enumerate(pairs):
        nbytes = src.numel() * src.element_size()
        if dst.numel() * dst.element_size() != nbytes or not (dst.is_contiguous() and src.is_contiguous()):
            raise ValueError("a copy needs contiguous tensors of equal size")
        arr[i] = Copy(dst.data_ptr(), src.data_ptr(), nbytes)
    return arr


class Step:
    """A compiled step (qmv_step_create): `before` copies, product groups, `after` copies,
    recorded once as a CUDA graph; run() enqueues it with one library call.

    before / after: lists of (dst, src) tensors (device or pinned host); groups: list of
    (wtype, scale_dtype, problems, overlap[, act[, bf16_weights]]) with problems as for
    matvec_grouped.  Creating the
    step runs it once.  The tensors are kept alive with the step; a run reads and writes the
    same buffers.  Runs of one step must not overlap in time.  close() (or leaving a `with`
    block) waits for the device and frees the step.

    gated=True (qmv_step_create_gated): each run waits on the device until open() (its `before`
    copies: pinned host to device memory), and wait() spins on the host until the opened runs
    are done; a decode loop enqueues the next run before it needs it and only opens it then."""

    def __init__(self, groups, before=(), after=(), gated=False):
        keep = [list(before), list(after)]
        garr = (Group * max(len(groups), 1))()
        for i, grp in enumerate(groups):
            wtype, scale_dtype, problems, overlap = grp[:4]
            parr, n, batch, xdt = _problem_array(problems, grp[4] if len(grp) > 4 else None)
            keep.append((parr, problems))
            garr[i] = Group(wtype, scale_dtype, xdt, batch, ctypes.addressof(parr), n,
                            _flags(overlap, len(grp) > 5 and bool(grp[5])))
        b, a = _copies(list(before)), _copies(list(after))
        handle = ctypes.c_void_p()
        create = load_library().qmv_step_create_gated if gated else load_library().qmv_step_create
        st = create(ctypes.addressof(b), len(before), ctypes.addressof(garr), len(groups),
                    ctypes.addressof(a), len(after), ctypes.byref(handle))
        _check(st, "qmv_step_create_gated" if gated else "qmv_step_create")
        self._handle = handle
        self._keep = keep

    def run(self, stream=None, wait=False):
        """Enqueue one run on `stream` (the current stream by default); wait=True also waits for
        the stream in the same library call (qmv_step_run_wait)."""
        if self._handle is None:
            raise ValueError("step destroyed")
        if wait:
            _check(load_library().qmv_step_run_wait(self._handle, _stream(stream)), "qmv_step_run_wait")
        else:
            _check(load_library().qmv_step_run(self._handle, _stream(stream)), "qmv_step_run")

    def open(self):
        """Open the oldest enqueued run of a gated step (qmv_step_open)."""
        if self._handle is None:
            raise ValueError("step destroyed")
        _check(load_library().qmv_step_open(self._handle), "qmv_step_open")

    def wait(self, timeout_us=0):
        """Wait on the host until the opened runs of a gated step are done (qmv_step_wait)."""
        if self._handle is None:
            raise ValueError("step destroyed")
        _check(load_library().qmv_step_wait(self._handle, int(timeout_us)), "qmv_step_wait")

    def open_wait(self, next_step=None, stream=None, timeout_us=0):
        """open(), then next_step.run(stream) when given, then wait(): one library call
        (qmv_step_open_wait), a decode loop's step with the next run enqueued behind it."""
        if self._handle is None or (next_step is not None and next_step._handle is None):
            raise ValueError("step destroyed")
        _check(load_library().qmv_step_open_wait(self._handle, None if next_step is None else next_step._handle,
                                                 _stream(stream), int(timeout_us)), "qmv_step_open_wait")

    def close(self):
        if self._handle is not None:
            st = load_library().qmv_step_destroy(self._handle)
            self._handle = None
            self._keep = None
            _check(st, "qmv_step_destroy")

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        self.close()
        return False


def dequant(wtype: int, scale_dtype: int, rows: int, cols: int, W, out=None, stream=None):
    """float32 (rows, cols) = level * d.  Returns out."""
    import torch
    if out is None:
        out = torch.empty((rows, cols), dtype=torch.float32, device=W.device)
    st = load_library().qmv_dequant(wtype, scale_dtype, rows, cols, W.data_ptr(), out.data_ptr(), _stream(stream))
    _check(st, "qmv_dequant")
    return out


def validate(wtype: int, scale_dtype: int, rows: int, cols: int, W, stream=None) -> int:
    """Index of the first Q8_0 quant byte equal to -128, or -1 (waits for the stream)."""
    import torch
    first = torch.empty(1, dtype=torch.int64, device=W.device)
    st = load_library().qmv_validate(wtype, scale_dtype, rows, cols, W.data_ptr(), first.data_ptr(),
                                     _stream(stream))
    _check(st, "qmv_validate")
    return int(first.item())


def quantize(wtype: int, scale_dtype: int, src, W=None, stream=None):
    """Matrix bytes (uint8 CUDA tensor of weight_bytes()) from float32 (rows, cols) by the
    writer rules.  Returns (W, first refused block index or -1); waits for the stream."""
    import torch
    rows, cols = src.shape
    if src.dtype != torch.float32 or not src.is_contiguous():
        raise ValueError("src must be a contiguous float32 (rows, cols) tensor")
    if W is None:
        W = torch.empty(weight_bytes(wtype, scale_dtype, rows, cols), dtype=torch.uint8, device=src.device)
    first = torch.empty(1, dtype=torch.int64, device=src.device)
    st = load_library().qmv_quantize(wtype, scale_dtype, rows, cols, src.data_ptr(), W.data_ptr(), first.data_ptr(),
                                     _stream(stream))
    _check(st, "qmv_quantize")
    return W, int(first.item())


def gguf_bytes(wtype: int, rows: int, cols: int) -> int:
    """Bytes of a rows x cols tensor in GGUF interleaved blocks (0 when invalid)."""
    return int(load_library().qmv_gguf_bytes(wtype, rows, cols))


def gguf_to_mlb(wtype: int, rows: int, cols: int, src, W=None, stream=None):
    """A tensor in GGUF interleaved blocks (uint8 CUDA tensor) into the two-array layout with
    f16 scales (uint8 CUDA tensor of weight_bytes(wtype, SCALE_F16, rows, cols)).  Returns W."""
    import torch
    if W is None:
        W = torch.empty(max(weight_bytes(wtype, SCALE_F16, rows, cols), 0), dtype=torch.uint8, device=src.device)
    st = load_library().qmv_gguf_to_mlb(wtype, rows, cols, src.data_ptr(), W.data_ptr(), _stream(stream))
    _check(st, "qmv_gguf_to_mlb")
    return W


def quantize_x(x, xq=None, stream=None):
    """The runtime's activation quantizer: x (batch, cols) float32/bfloat16 CUDA tensor into
    xq, the Q8_0 / f32-scale image of the batch x cols matrix (uint8 CUDA tensor of
    weight_bytes(Q8_0, SCALE_F32, batch, cols)).  Returns xq."""
    import torch
    if x.dim() == 1:
        x = x.unsqueeze(0)
    batch, cols = x.shape
    if not x.is_contiguous():
        raise ValueError("x must be a contiguous (batch, cols) tensor")
    if xq is None:
        xq = torch.empty(max(weight_bytes(Q8_0, SCALE_F32, batch, cols), 0), dtype=torch.uint8, device=x.device)
    st = load_library().qmv_quantize_x(_x_dtype(x), batch, cols, x.data_ptr(), xq.data_ptr(), _stream(stream))
    _check(st, "qmv_quantize_x")
    return xq


def matvec_qx(wtype: int, scale_dtype: int, rows: int, cols: int, W, xq, batch: int, y=None, stream=None):
    """Activation-quantized product: y[v][r] = sum_b d_w d_x (exact integer block dot) for the
    quantized activations xq (as quantize_x returns them, batch vectors).  Returns y."""
    import torch
    if y is None:
        y = torch.empty((batch, rows), dtype=torch.float32, device=xq.device)
    if y.dtype != torch.float32 or tuple(y.shape) != (batch, rows) or not y.is_contiguous():
        raise ValueError("y must be a contiguous float32 (batch, rows) tensor")
    st = load_library().qmv_matvec_qx(wtype, scale_dtype, rows, cols, W.data_ptr(), xq.data_ptr(), y.data_ptr(),
                                      batch, _stream(stream))
    _check(st, "qmv_matvec_qx")
    return y


def matvec_qx_grouped(wtype: int, scale_dtype: int, problems, overlap: bool = False, stream=None):
    """The activation-quantized product with the activation quantizer inside the launch
    (qmv_matvec_qx_grouped): problems as for matvec_grouped, x float32 or bfloat16 (batch, cols);
    each y receives matvec_qx(W, quantize_x(x))."""
    arr, n, batch, xdt = _problem_array(problems)
    st = load_library().qmv_matvec_qx_grouped(wtype, scale_dtype, xdt, batch, ctypes.addressof(arr), n,
                                              FLAG_OVERLAP if overlap else 0, _stream(stream))
    _check(st, "qmv_matvec_qx_grouped")


def quantize_q4_fit(scale_dtype: int, src, W=None, stream=None):
    """Q4_0 matrix bytes from float32 (rows, cols) by the best-fit rule (qmv_quantize_q4_fit).
    Returns (W, first refused block index or -1); waits for the stream."""
    import torch
    rows, cols = src.shape
    if src.dtype != torch.float32 or not src.is_contiguous():
        raise ValueError("src must be a contiguous float32 (rows, cols) tensor")
    if W is None:
        W = torch.empty(weight_bytes(Q4_0, scale_dtype, rows, cols), dtype=torch.uint8, device=src.device)
    first = torch.empty(1, dtype=torch.int64, device=src.device)
    st = load_library().qmv_quantize_q4_fit(scale_dtype, rows, cols, src.data_ptr(), W.data_ptr(), first.data_ptr(),
                                            _stream(stream))
    _check(st, "qmv_quantize_q4_fit")
    return W, int(first.item())


OUT_Q8 = 16
NORM_MAX_COLS = 32768
MAX_TOP = 32
MAX_GIVEN = 64


def _raw_stream(stream, device_index, *others):
    """The stream's handle as an integer; the device's current stream by default.  device_index and others: the
    devices of the call's tensors (get_device(), -1 on the host), which must be one, the current one: the kernels
    follow the pointers as they are."""
    if device_index < 0:
        raise ValueError("CUDA tensors are needed")
    for other in others:
        if other != device_index:
            raise ValueError("all tensors of a call must be on one CUDA device")
    import torch
    if torch._C._cuda_getDevice() != device_index:
        raise ValueError("the tensors' device must be the current one (torch.cuda.device)")
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(device_index)


def _device_of(tensors, what):
    """The one device (get_device()) of tensors, None among them left out."""
    index = {t.get_device() for t in tensors if t is not None}
    if len(index) != 1:
        raise ValueError(f"{what} must be on one device")
    return index.pop()


def rmsnorm(x, weight, eps: float = 1e-5, residual=None, residual_out=None, out="q8", y=None, stream=None):
    """Root-mean-square norm with the residual's addition (qmv_rmsnorm): with s = x + residual,
    y = s * weight / sqrt(mean(s^2) + eps).  x: (rows, cols) or (cols,) float32/bfloat16 CUDA tensor;
    residual: float32 of x's shape or None; residual_out: where s is stored (residual itself for an
    update in place), or None.  out: "q8" (the uint8 Q8_0 / f32-scale image that matvec_qx reads),
    "bf16" or "f32".  Returns y."""
    import torch
    shape = x.shape
    if len(shape) == 2:
        rows, cols = shape
    elif len(shape) == 1:
        rows, cols = 1, shape[0]
    else:
        raise ValueError("x must be a contiguous (rows, cols) tensor")
    if not x.is_contiguous():
        raise ValueError("x must be a contiguous (rows, cols) tensor")
    f32 = torch.float32
    if weight.dtype is not f32 or weight.numel() != cols or not weight.is_contiguous():
        raise ValueError("weight must be a contiguous float32 (cols,) tensor")
    for t in (residual, residual_out):
        if t is not None and (t.dtype is not f32 or t.shape != shape or not t.is_contiguous()):
            raise ValueError("residual and residual_out must be contiguous float32 tensors of x's shape")
    if out == "q8":
        code = OUT_Q8
        # the image's bytes: quants, their padding to 64, a float32 scale for each 32
        need = (rows * cols + 63) // 64 * 64 + rows * cols // 8
        if y is None:
            y = torch.empty(need, dtype=torch.uint8, device=x.device)
        elif y.dtype is not torch.uint8 or y.numel() < need or not y.is_contiguous():
            raise ValueError("y must be a contiguous uint8 tensor of the image's bytes")
    elif out == "bf16" or out == "f32":
        code, dtype = (X_BF16, torch.bfloat16) if out == "bf16" else (X_F32, f32)
        if y is None:
            y = torch.empty(shape, dtype=dtype, device=x.device)
        elif y.dtype is not dtype or y.shape != shape or not y.is_contiguous():
            raise ValueError("y must be a contiguous tensor of x's shape and the output's type")
    else:
        raise ValueError("out must be 'q8', 'bf16' or 'f32'")
    st = load_library().qmv_rmsnorm(_x_dtype(x), rows, cols, x.data_ptr(),
                                    None if residual is None else residual.data_ptr(),
                                    None if residual_out is None else residual_out.data_ptr(), weight.data_ptr(), eps,
                                    code, y.data_ptr(),
                                    _raw_stream(stream, x.get_device(), weight.get_device(), y.get_device(),
                                                *[t.get_device() for t in (residual, residual_out) if t is not None]))
    _check(st, "qmv_rmsnorm")
    return y


class _KvCacheC(ctypes.Structure):
    """qmv_kv_cache of include/qmv.h."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("n_pages", ctypes.c_int64), ("kv_heads", ctypes.c_int),
                ("head_dim", ctypes.c_int), ("page_tokens", ctypes.c_int)]


class _KvBatchC(ctypes.Structure):
    """qmv_kv_batch of include/qmv.h."""
    _fields_ = [("page_table", ctypes.c_void_p), ("table_stride", ctypes.c_int64), ("table_pages", ctypes.c_int), ("kv_len", ctypes.c_void_p),
                ("starts", ctypes.c_void_p), ("n_seq", ctypes.c_int), ("rows", ctypes.c_int64),
                ("max_rows", ctypes.c_int), ("max_len", ctypes.c_int)]


class KvCache:
    """One layer's paged cache of keys and values in 8 bits (qmv_kv_cache): k and v are int8 CUDA
    tensors (pages, kv_heads, page_tokens, head_dim), k_scale and v_scale float32 (pages, kv_heads).
    KvCache.empty() makes them."""

    def __init__(self, k, v, k_scale, v_scale):
        import torch
        if k.dim() != 4 or v.shape != k.shape or k.dtype != torch.int8 or v.dtype != torch.int8:
            raise ValueError("k and v must be int8 (pages, kv_heads, page_tokens, head_dim) tensors")
        for t in (k_scale, v_scale):
            if t.dtype != torch.float32 or t.shape != k.shape[:2] or not t.is_contiguous():
                raise ValueError("k_scale and v_scale must be contiguous float32 (pages, kv_heads) tensors")
        if not (k.is_contiguous() and v.is_contiguous()):
            raise ValueError("k and v must be contiguous")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.kv_heads, self.page_tokens, self.head_dim = k.shape
        self._c = _KvCacheC(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), self.n_pages,
                            self.kv_heads, self.head_dim, self.page_tokens)
        self._p = ctypes.addressof(self._c)
        self.device = k.device
        self._index = _device_of((k, v, k_scale, v_scale), "a cache's tensors")

    @classmethod
    def empty(cls, n_pages: int, kv_heads: int, head_dim: int, page_tokens: int = 64, device="cuda"):
        """A cache of zero levels and scales."""
        import torch
        shape = (n_pages, kv_heads, page_tokens, head_dim)
        return cls(torch.zeros(shape, dtype=torch.int8, device=device), torch.zeros(shape, dtype=torch.int8, device=device),
                   torch.zeros(shape[:2], device=device), torch.zeros(shape[:2], device=device))


class KvBatch:
    """The rows of calls over a cache (qmv_kv_batch): page_table (sequences, pages) int32, kv_len
    (sequences,) int32, starts (sequences + 1,) int32 or None for one row a sequence: CUDA tensors whose
    contents are read when a call runs on the device, so a decode loop updates them in place.  rows: the
    call's rows in all; max_rows, max_len: upper bounds of a sequence's rows and of kv_len (by
    default rows, and what the table would hold in pages of 128).
    A close max_len lets the calls choose better."""

    def __init__(self, page_table, kv_len, starts=None, rows=None, max_rows=None, max_len=None):
        import torch
        if page_table.dim() != 2 or page_table.dtype != torch.int32 or (page_table.shape[1] > 0 and page_table.stride(1) != 1):
            raise ValueError("page_table must be an int32 (sequences, pages) tensor with contiguous rows")
        n = page_table.shape[0]
        if kv_len.dtype != torch.int32 or tuple(kv_len.shape) != (n,) or not kv_len.is_contiguous():
            raise ValueError("kv_len must be a contiguous int32 (sequences,) tensor")
        if starts is None:
            rows, max_rows = n, 1
        else:
            if starts.dtype != torch.int32 or tuple(starts.shape) != (n + 1,) or not starts.is_contiguous():
                raise ValueError("starts must be a contiguous int32 (sequences + 1,) tensor")
            if rows is None:
                raise ValueError("rows is needed with starts")
            max_rows = rows if max_rows is None else max_rows
        self.page_table, self.kv_len, self.starts = page_table, kv_len, starts
        self.n_seq, self.rows, self.max_rows = n, rows, max_rows
        self.max_len = 128 * page_table.shape[1] if max_len is None else max_len
        stride = page_table.stride(0) if n > 1 else page_table.shape[1]
        self._c = _KvBatchC(page_table.data_ptr(), stride, page_table.shape[1], kv_len.data_ptr(), None if starts is None else starts.data_ptr(),
                            n, rows, max_rows, self.max_len)
        self._p = ctypes.addressof(self._c)
        self._index = _device_of((page_table, kv_len, starts), "page_table, kv_len and starts")


def _head_rows(t, heads, dim, rows, what):
    """The row stride of a (rows, heads, dim) tensor whose rows are contiguous."""
    if tuple(t.shape) == (rows, heads, dim):
        row, head, value = t.stride()
        if rows == 0 or (value == 1 and (head == dim or heads == 1)):
            return row if rows > 1 else heads * dim
    raise ValueError(f"{what} must be a ({rows}, {heads}, {dim}) tensor with contiguous rows")


def kv_write(cache: KvCache, batch: KvBatch, k, v, stream=None):
    """Writes the call's rows into the cache (qmv_kv_write): k and v (rows, kv_heads, head_dim) CUDA
    tensors of one type, float32 or bfloat16; rows may be strided (a slice of a wider row)."""
    if k.dtype != v.dtype:
        raise ValueError("k and v must have one type")
    ks = _head_rows(k, cache.kv_heads, cache.head_dim, batch.rows, "k")
    vs = _head_rows(v, cache.kv_heads, cache.head_dim, batch.rows, "v")
    st = load_library().qmv_kv_write(cache._p, batch._p, _x_dtype(k), k.data_ptr(), ks, v.data_ptr(), vs,
                                     _raw_stream(stream, k.get_device(), v.get_device(), cache._index, batch._index))
    _check(st, "qmv_kv_write")


def kv_read(cache: KvCache, batch: KvBatch, dtype=None, k=None, v=None, stream=None):
    """Reads the call's rows back (qmv_kv_read) as (rows, kv_heads, head_dim) tensors of dtype
    (torch.bfloat16 by default, or torch.float32).  Returns k, v."""
    import torch
    if dtype is None:
        dtype = torch.bfloat16 if k is None else k.dtype
    shape = (batch.rows, cache.kv_heads, cache.head_dim)
    for t in (k, v):
        if t is not None and (t.dtype != dtype or tuple(t.shape) != shape or not t.is_contiguous()):
            raise ValueError("k and v must be contiguous (rows, kv_heads, head_dim) tensors of the asked type")
    if k is None:
        k = torch.empty(shape, dtype=dtype, device=cache.device)
    if v is None:
        v = torch.empty(shape, dtype=dtype, device=cache.device)
    st = load_library().qmv_kv_read(cache._p, batch._p, _x_dtype(k), k.data_ptr(), v.data_ptr(),
                                    _raw_stream(stream, k.get_device(), v.get_device(), cache._index, batch._index))
    _check(st, "qmv_kv_read")
    return k, v


def attend(cache: KvCache, batch: KvBatch, q, out=None, scale=None, causal: bool = True, window: int = 0, stream=None):
    """Softmax attention of the call's rows over the cache (qmv_attend): q (rows, heads, head_dim)
    float32/bfloat16 CUDA tensor, rows may be strided; scale defaults to 1 / sqrt(head_dim).  Returns
    out, (rows, heads, head_dim) of q's type."""
    import torch
    if q.dim() != 3:
        raise ValueError("q must be a (rows, heads, head_dim) tensor")
    heads = q.shape[1]
    qs = _head_rows(q, heads, cache.head_dim, batch.rows, "q")
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        os_ = heads * cache.head_dim
    else:
        if out.dtype != q.dtype:
            raise ValueError("out must have q's type")
        os_ = _head_rows(out, heads, cache.head_dim, batch.rows, "out")
    st = load_library().qmv_attend(cache._p, batch._p, heads, _x_dtype(q), q.data_ptr(), qs,
                                   cache.head_dim ** -0.5 if scale is None else scale, 1 if causal else 0, window,
                                   out.data_ptr(), os_,
                                   _raw_stream(stream, q.get_device(), out.get_device(), cache._index, batch._index))
    _check(st, "qmv_attend")
    return out


def logprobs(logits, given=None, top: int = 0, entropy: bool = True, stream=None):
    """Log probabilities from logits (rows, vocab), float32, rows may be strided (qmv_logprobs): of
    the given ids (rows, n) int64, the entropy, and the `top` largest with their ids.  Returns
    (given_logprob, entropy, top_ids, top_logprob); what was not asked for is None."""
    import torch
    if logits.dim() != 2 or logits.dtype != torch.float32 or (logits.shape[1] > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be a float32 (rows, vocab) tensor with contiguous rows")
    rows, vocab = logits.shape
    dev = logits.device
    n = 0
    glp = ent = ids = tlp = None
    if given is not None:
        if given.dtype != torch.int64 or given.dim() != 2 or given.shape[0] != rows or not given.is_contiguous():
            raise ValueError("given must be a contiguous int64 (rows, n) tensor")
        n = given.shape[1]
        glp = torch.empty((rows, n), dtype=torch.float32, device=dev)
    if entropy:
        ent = torch.empty((rows,), dtype=torch.float32, device=dev)
    if top > 0:
        ids = torch.empty((rows, top), dtype=torch.int32, device=dev)
        tlp = torch.empty((rows, top), dtype=torch.float32, device=dev)
    st = load_library().qmv_logprobs(rows, vocab, logits.data_ptr(), logits.stride(0) if rows > 1 else vocab,
                                     None if n == 0 else given.data_ptr(), n, None if n == 0 else glp.data_ptr(),
                                     None if ent is None else ent.data_ptr(), top, None if ids is None else ids.data_ptr(),
                                     None if tlp is None else tlp.data_ptr(),
                                     _raw_stream(stream, logits.get_device(), *(() if given is None else (given.get_device(),))))
    _check(st, "qmv_logprobs")
    return glp, ent, ids, tlp


def sample(logits, noise, temperature=None, top_k=None, top_p=None, min_p=None, ids=None, stream=None):
    """The next id of each row of logits (qmv_sample): logits and noise (rows, vocab) float32, rows may be strided or one (expand);
    noise: exponential random numbers (torch.empty_like(logits).exponential_()).  temperature, top_p, min_p: float32
    (rows,), top_k int32 (rows,) CUDA tensors, whose contents are read when the call runs on the device, or None.
    Returns ids, int64 (rows,): what embed() and logprobs() take."""
    import torch
    f32 = torch.float32
    shape = logits.shape
    if len(shape) != 2 or logits.dtype is not f32 or noise.dtype is not f32:
        raise ValueError("logits and noise must be float32 (rows, vocab) tensors with contiguous rows")
    rows, vocab = shape
    if noise.shape != shape:
        raise ValueError("noise must have the logits' shape")
    ls, ns = logits.stride(), noise.stride()
    if vocab > 1 and (ls[1] != 1 or ns[1] != 1):
        raise ValueError("logits and noise must be float32 (rows, vocab) tensors with contiguous rows")
    if ids is None:
        ids = torch.empty((rows,), dtype=torch.int64, device=logits.device)
    elif ids.dtype is not torch.int64 or ids.shape != (rows,) or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous int64 (rows,) tensor")
    on, at = [noise.get_device(), ids.get_device()], []
    for t, dtype in ((temperature, f32), (top_k, torch.int32), (top_p, f32), (min_p, f32)):
        if t is None:
            at.append(None)
            continue
        if t.dtype is not dtype or t.shape != (rows,) or not t.is_contiguous():
            raise ValueError("temperature, top_p and min_p must be contiguous float32 (rows,) tensors, top_k int32")
        at.append(t.data_ptr())
        on.append(t.get_device())
    st = load_library().qmv_sample(rows, vocab, logits.data_ptr(), ls[0] if rows > 1 else vocab, noise.data_ptr(),
                                   ns[0] if rows > 1 else vocab, *at, ids.data_ptr(), _raw_stream(stream, logits.get_device(), *on))
    _check(st, "qmv_sample")
    return ids


_OUT_TYPES = None


def _out_type(out):
    """The code and torch type of "f32" or "bf16"."""
    global _OUT_TYPES
    if _OUT_TYPES is None:
        import torch
        _OUT_TYPES = {"f32": (X_F32, torch.float32), "bf16": (X_BF16, torch.bfloat16)}
    found = _OUT_TYPES.get(out)
    if found is None:
        raise ValueError("out must be 'bf16' or 'f32'")
    return found


def embed(wtype: int, scale_dtype: int, vocab: int, cols: int, W, ids, scale: float = 1.0, out="f32", y=None, stream=None):
    """Rows of a block-quantized token table (qmv_embed): W the uint8 image of the (vocab, cols) matrix, ids an int64 CUDA
    tensor of any shape.  Returns y, ids.shape + (cols,) of the type `out` ("f32" or "bf16"): the rows times scale, zeros
    for ids outside the table."""
    import torch
    code, dtype = _out_type(out)
    if ids.dtype is not torch.int64 or not ids.is_contiguous():
        raise ValueError("ids must be a contiguous int64 tensor")
    n = vocab * cols
    need = ((n if wtype == Q8_0 else n // 2) + 63) // 64 * 64 + n // 32 * (2 if scale_dtype == SCALE_F16 else 4)  # the image's bytes
    if W.dtype is not torch.uint8 or W.numel() < need or not W.is_contiguous():
        raise ValueError("W must be a contiguous uint8 tensor of the matrix image's bytes")
    shape = ids.shape + (cols,)
    if y is None:
        y = torch.empty(shape, dtype=dtype, device=ids.device)
    elif y.dtype is not dtype or y.shape != shape or not y.is_contiguous():
        raise ValueError("y must be a contiguous tensor of ids' shape and cols, of the output's type")
    st = load_library().qmv_embed(wtype, scale_dtype, vocab, cols, W.data_ptr(), ids.data_ptr(), ids.numel(), scale, code,
                                  y.data_ptr(), _raw_stream(stream, W.get_device(), ids.get_device(), y.get_device()))
    _check(st, "qmv_embed")
    return y


ROPE_PAIRS = {"neighbours": 0, "halves": 1}


def _new_like(t, dtype):
    """A contiguous tensor of t's shape (empty_like() takes the least of the host's time, new_empty() twice that of empty())."""
    import torch
    return torch.empty_like(t) if t.dtype is dtype and t.is_contiguous() else torch.empty(t.shape, dtype=dtype, device=t.device)


def _stride_of_rows(t, shape, what):
    """The row stride of a tensor of that shape, (rows, heads, dim), whose rows are contiguous."""
    if t.shape == shape:
        rows, heads, dim = shape
        if t.is_contiguous():
            return heads * dim
        row, head, value = t.stride()
        if (value == 1 and (head == dim or heads == 1)) or rows == 0:
            return row if rows > 1 else heads * dim
    raise ValueError(f"{what} must be a {tuple(shape)} tensor with contiguous rows")


def qk_rope(q, k, pos, freq, q_weight=None, k_weight=None, eps: float = 1e-6, pairs="halves", factor: float = 1.0, out=None,
            q_out=None, k_out=None, stream=None):
    """Norms of queries and keys for each head and the position rotation, in one pass (qmv_qk_rope).  q (rows, heads, head_dim)
    and k (rows, kv_heads, head_dim) or None: float32 or bfloat16 CUDA tensors, rows may be strided (slices of a
    fused projection).  pos: int32 (rows,); freq: float32 (rot_dim / 2,) in radians a position; both None for norms alone.
    q_weight, k_weight: float32 (head_dim,), or None for no norm.  pairs: "halves" (i and i + rot_dim / 2) or "neighbours"
    (2i and 2i + 1).  out: "f32" or "bf16" (q's own type by default).  q_out, k_out: where to write (q and k themselves
    for an update in place).  Returns q_out, k_out."""
    import torch
    shape, xt, f32 = q.shape, q.dtype, torch.float32
    if len(shape) != 3:
        raise ValueError("q must be a (rows, heads, head_dim) tensor")
    rows, heads, dim = shape
    x = _x_dtype(q)
    if pairs not in ROPE_PAIRS:
        raise ValueError("pairs must be 'halves' or 'neighbours'")
    code, dtype = (x, xt) if out is None else _out_type(out)
    qs = _stride_of_rows(q, shape, "q")
    if q_out is None:
        q_out, qos = _new_like(q, dtype), heads * dim
    else:
        qos = _stride_of_rows(q_out, shape, "q_out")
    on = [q_out.get_device()]
    if k is None:
        if k_out is not None or k_weight is not None:
            raise ValueError("k_out and k_weight need k")
        kvh = ks = kos = 0
        kp = kop = None
    else:
        kshape = k.shape
        if len(kshape) != 3 or k.dtype is not xt:
            raise ValueError("k must be a (rows, kv_heads, head_dim) tensor of q's type")
        kvh = kshape[1]
        ks = _stride_of_rows(k, (rows, kvh, dim), "k")
        if k_out is None:
            k_out, kos = _new_like(k, dtype), kvh * dim
        else:
            kos = _stride_of_rows(k_out, (rows, kvh, dim), "k_out")
            if k_out.dtype is not dtype:
                raise ValueError("q_out and k_out must be of the output's type")
        kp, kop = k.data_ptr(), k_out.data_ptr()
        on += (k.get_device(), k_out.get_device())
    if q_out.dtype is not dtype:
        raise ValueError("q_out and k_out must be of the output's type")
    if freq is None or pos is None:
        if freq is not pos:
            raise ValueError("pos and freq go together")
        rot, pp, fp = 0, None, None
    else:
        if freq.dtype is not f32 or freq.dim() != 1 or not freq.is_contiguous():
            raise ValueError("freq must be a contiguous float32 (rot_dim / 2,) tensor")
        if pos.dtype is not torch.int32 or pos.shape != (rows,) or not pos.is_contiguous():
            raise ValueError("pos must be a contiguous int32 (rows,) tensor")
        rot, pp, fp = 2 * freq.numel(), pos.data_ptr(), freq.data_ptr()
        on += (pos.get_device(), freq.get_device())
    wp = [None, None]
    for i, w in enumerate((q_weight, k_weight)):
        if w is not None:
            if w.dtype is not f32 or w.shape != (dim,) or not w.is_contiguous():
                raise ValueError("q_weight and k_weight must be contiguous float32 (head_dim,) tensors")
            wp[i] = w.data_ptr()
            on.append(w.get_device())
    st = load_library().qmv_qk_rope(x, rows, heads, kvh, dim, q.data_ptr(), qs, kp, ks, wp[0], wp[1], eps, pp, fp, rot, ROPE_PAIRS[pairs],
                                    factor, code, q_out.data_ptr(), qos, kop, kos, _raw_stream(stream, q.get_device(), *on))
    _check(st, "qmv_qk_rope")
    return q_out, k_out


class _MoeC(ctypes.Structure):
    """qmv_moe_layer of include/qmv.h."""
    _fields_ = [("wtype13", ctypes.c_int), ("wtype2", ctypes.c_int), ("scale_dtype", ctypes.c_int), ("experts", ctypes.c_int),
                ("dim", ctypes.c_int64), ("hidden", ctypes.c_int64), ("W1", ctypes.c_void_p), ("W3", ctypes.c_void_p),
                ("W2", ctypes.c_void_p)]


class Moe:
    """A layer of experts (qmv_moe_layer): W1 and W3 the uint8 images of (experts * hidden, dim) matrices of type wtype13, W2
    that of (experts * dim, hidden) of type wtype2; CUDA tensors, kept with the layer."""

    def __init__(self, wtype13: int, wtype2: int, scale_dtype: int, experts: int, dim: int, hidden: int, W1, W3, W2):
        import torch
        for W, wt, rows, cols in ((W1, wtype13, experts * hidden, dim), (W3, wtype13, experts * hidden, dim), (W2, wtype2, experts * dim, hidden)):
            need = weight_bytes(wt, scale_dtype, rows, cols)
            if W.dtype is not torch.uint8 or not W.is_contiguous() or need == 0 or W.numel() < need:
                raise ValueError("W1, W3 and W2 must be contiguous uint8 tensors of the matrix images' bytes")
        self.experts, self.dim, self.hidden = experts, dim, hidden
        self._scratch = (None, 0)  # the last call's numbers, and its bytes of scratch memory
        self.W1, self.W3, self.W2 = W1, W3, W2
        self._c = _MoeC(wtype13, wtype2, scale_dtype, experts, dim, hidden, W1.data_ptr(), W3.data_ptr(), W2.data_ptr())
        self._p = ctypes.addressof(self._c)
        self._index = _device_of((W1, W3, W2), "a layer's matrices")


def moe(layer: Moe, x, logits, top: int, renorm: bool = True, scale: float = 1.0, act: str = "silu", out="f32", y=None,
        routing: bool = False, scratch=None, stream=None):
    """The layer of experts for a few tokens (qmv_moe): x (tokens, dim) float32/bfloat16, logits (tokens, experts) float32
    (rows may be strided).  Returns y, (tokens, dim) of the type `out` ("f32" or "bf16"); with routing also the experts
    (tokens, top) int32 and their shares float32.  scratch: a uint8 CUDA tensor of moe_scratch_bytes(), by default one from
    torch's allocator for this call (with a stream other than the current one, give it, and keep it until that stream is done)."""
    import torch
    code, dtype = _out_type(out)
    act_code = ACT_CODES.get(act)
    if act_code is None:
        raise ValueError("act must be 'silu' or 'gelu'")
    shape = x.shape
    if len(shape) != 2 or shape[1] != layer.dim or not x.is_contiguous():
        raise ValueError("x must be a contiguous (tokens, dim) tensor")
    n, experts = shape[0], layer.experts
    if logits.dtype is not torch.float32 or logits.shape != (n, experts) or (experts > 1 and logits.stride(1) != 1):
        raise ValueError("logits must be a float32 (tokens, experts) tensor with contiguous rows")
    if y is None:
        y = _new_like(x, dtype)
    elif y.dtype is not dtype or y.shape != shape or not y.is_contiguous():
        raise ValueError("y must be a contiguous (tokens, dim) tensor of the output's type")
    numbers, need = layer._scratch
    if numbers != (n, top, code):
        need = moe_scratch_bytes(n, top, layer.hidden, out)
        layer._scratch = (n, top, code), need
    if scratch is None:
        scratch = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
        if stream is not None:
            scratch.record_stream(stream)
    elif scratch.dtype is not torch.uint8 or scratch.numel() < need or not scratch.is_contiguous():
        raise ValueError("scratch must be a contiguous uint8 tensor of moe_scratch_bytes()")
    ids = shares = ip = sp = None
    if routing:
        ids = torch.empty((n, max(top, 0)), dtype=torch.int32, device=x.device)
        shares = torch.empty((n, max(top, 0)), dtype=torch.float32, device=x.device)
        ip, sp = ids.data_ptr(), shares.data_ptr()
    st = load_library().qmv_moe(layer._p, n, logits.data_ptr(), logits.stride(0) if n > 1 else experts, top, 1 if renorm else 0, scale,
                                act_code, _x_dtype(x), x.data_ptr(), code, y.data_ptr(), ip, sp, scratch.data_ptr(),
                                _raw_stream(stream, x.get_device(), logits.get_device(), y.get_device(), scratch.get_device(), layer._index))
    _check(st, "qmv_moe")
    return (y, ids, shares) if routing else y


def moe_scratch_bytes(tokens: int, top: int, hidden: int, out="f32") -> int:
    """Bytes of scratch memory that moe() needs for `tokens` tokens of `top` experts (0 for numbers that it refuses)."""
    return int(load_library().qmv_moe_scratch_bytes(tokens, top, hidden, _out_type(out)[0]))


def last_error() -> int:
    """Synchronize the device; return and clear the kernels' status word."""
    return int(load_library().qmv_check_device())
