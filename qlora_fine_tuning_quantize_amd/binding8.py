"""Python binding of the 8-bit operators (the C ABI in include/qlora_8bit.h):
matrices in 8-bit floating point with a scale for each block of 128, their
product, and an AdamW step over many tensors with moments in 32 or 8 bits.

As in binding.py: argument marshalling only, the C entry points' names, work
on the current stream of the tensors' device, no CPU fallback.
"""
from __future__ import annotations

import ctypes

import torch

from .binding import QL_BF16, QL_F16, QL_F32, _check, lib

QL_E4M3, QL_E5M2 = 3, 4
FP8_BLOCK, STATE_BLOCK = 128, 256

# every extern "C" symbol declared in include/qlora_8bit.h
EXPORTED8 = ("ql_fp8_sizes", "fp8_quantize", "ql_fp8_workspace_bytes", "fp8_matmul",
             "ql_adamw_step_many", "ql_8bit_version")

_FORMATS = {torch.float8_e4m3fn: QL_E4M3, torch.float8_e5m2: QL_E5M2}


class QlFp8(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("format", ctypes.c_int32), ("reserved", ctypes.c_int32)]


class QlAdamwTensor(ctypes.Structure):
    _fields_ = [("param", ctypes.c_void_p), ("grad", ctypes.c_void_p),
                ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p),
                ("exp_avg_scale", ctypes.c_void_p), ("exp_avg_sq_scale", ctypes.c_void_p),
                ("copy", ctypes.c_void_p), ("n", ctypes.c_int64)]


_lib8 = None


def lib8() -> ctypes.CDLL:
    """libqlora.so with the argument types of include/qlora_8bit.h set."""
    global _lib8
    if _lib8 is not None:
        return _lib8
    L = lib()
    p, i32, i64, f64, sz = (ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_double,
                            ctypes.c_size_t)
    L.ql_fp8_sizes.argtypes = [i64, i64, ctypes.POINTER(sz * 2)]
    L.ql_fp8_sizes.restype = ctypes.c_int
    L.fp8_quantize.argtypes = [p, i32, i32, p, p, p]
    L.fp8_quantize.restype = ctypes.c_int
    L.ql_fp8_workspace_bytes.argtypes = [i64, i64, i64]
    L.ql_fp8_workspace_bytes.restype = sz
    L.fp8_matmul.argtypes = [p, p, p, i32, i32, p, sz, p]
    L.fp8_matmul.restype = ctypes.c_int
    L.ql_adamw_step_many.argtypes = [i32, p, p, i32, i32, i32, p, f64, f64, f64, f64, f64, i64,
                                     ctypes.c_uint64, p]
    L.ql_adamw_step_many.restype = ctypes.c_int
    L.ql_8bit_version.restype = ctypes.c_int
    _lib8 = L
    return L


# The current device, and a device's current stream as a number.  The public
# ways check that CUDA is set up, which a tensor on the GPU has done, and make a
# Stream object: 0.2 and 2 us a call.
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)
_DTYPES = {torch.float32: QL_F32, torch.bfloat16: QL_BF16, torch.float16: QL_F16}


def _code(dtype: torch.dtype) -> int:
    code = _DTYPES.get(dtype)
    if code is None:
        raise ValueError(f"unsupported dtype {dtype}")
    return code


def _call(fn, what: str, index: int, *args):
    """fn(*args, stream) on the current stream of GPU `index`, with that GPU current."""
    if index == _device():
        status = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status:
        _check(status, what)


def _need(ok: bool, message: str):
    if not ok:
        raise ValueError(message)


def fp8_sizes(rows: int, cols: int) -> list[int]:
    """Bytes of the codes and of the scales of a rows x cols matrix."""
    out = (ctypes.c_size_t * 2)()
    _check(lib8().ql_fp8_sizes(rows, cols, ctypes.byref(out)), "ql_fp8_sizes")
    return list(out)


class FP8Matrix:
    """A matrix [rows, cols] in 8-bit floating point on the GPU.

    codes   float8_e4m3fn or float8_e5m2 [rows, cols rounded up to 128], zero beyond cols
    scales  float8_e8m0fnu [that / 128, rows rounded up to 16]: scales[b, i]
            belongs to columns 128 b .. 128 b + 127 of row i

    Its buffers are those it was made with, for good; what they hold may change.
    """
    __slots__ = ("_codes", "_scales", "_rows", "_cols", "_index", "_struct", "_ref")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, rows: int, cols: int):
        _need(codes.dtype in _FORMATS, f"codes are {codes.dtype}: float8_e4m3fn or float8_e5m2")
        _need(scales.dtype == torch.float8_e8m0fnu, f"scales are {scales.dtype}: float8_e8m0fnu")
        _need(codes.is_cuda and codes.device == scales.device, "codes and scales on one GPU")
        _need(codes.is_contiguous() and scales.is_contiguous(), "codes and scales are contiguous")
        n_codes, n_scales = fp8_sizes(rows, cols)
        ld = n_codes // rows
        _need(tuple(codes.shape) == (rows, ld), f"codes are {tuple(codes.shape)}: {(rows, ld)}")
        want = (ld // FP8_BLOCK, n_scales * FP8_BLOCK // ld)
        _need(tuple(scales.shape) == want, f"scales are {tuple(scales.shape)}: {want}")
        # tensors of their own, which keep the memory where another's would be exchanged
        self._codes, self._scales = codes.detach(), scales.detach()
        self._rows, self._cols = rows, cols
        self._index = codes.get_device()
        self._struct = QlFp8(codes.data_ptr(), scales.data_ptr(), rows, cols,
                             _FORMATS[codes.dtype], 0)
        self._ref = ctypes.addressof(self._struct)

    codes = property(lambda self: self._codes.detach())
    scales = property(lambda self: self._scales.detach())
    rows = property(lambda self: self._rows)
    cols = property(lambda self: self._cols)
    format = property(lambda self: self._codes.dtype)
    device = property(lambda self: self._codes.device)

    @staticmethod
    def empty(rows: int, cols: int, device, format: torch.dtype = torch.float8_e4m3fn) -> "FP8Matrix":
        n_codes, n_scales = fp8_sizes(rows, cols)
        ld = n_codes // rows
        blocks = ld // FP8_BLOCK
        return FP8Matrix(torch.empty((rows, ld), dtype=format, device=device),
                         torch.empty((blocks, n_scales // blocks), dtype=torch.uint8,
                                     device=device).view(torch.float8_e8m0fnu), rows, cols)

    def storage_bytes(self) -> int:
        return sum(fp8_sizes(self._rows, self._cols))


def fp8_quantize(x: torch.Tensor, block_rows: int = 1, format: torch.dtype = torch.float8_e4m3fn,
                 transposed: bool = False, out: FP8Matrix | None = None,
                 out_t: FP8Matrix | None = None):
    """Quantise x [R, C] (bf16, fp16 or fp32) with a scale for each 128 values
    of a row (block_rows 1) or each 128 x 128 tile (128).

    Without out and out_t: returns an FP8Matrix of `format`, or with
    transposed=True that and the transpose.  With out (x) or out_t (x
    transposed) or both: fills what is given, each in its own format (`format`
    is not looked at), and returns (out, out_t)."""
    index = x.get_device()
    if not (x.dim() == 2 and x.is_contiguous() and index >= 0):
        raise ValueError("x is 2-D, contiguous and on the GPU")
    R, C = x.shape
    made = out is None and out_t is None
    if made:
        out = FP8Matrix.empty(R, C, x.device, format)
        out_t = FP8Matrix.empty(C, R, x.device, format) if transposed else None
    elif transposed and out_t is None:
        raise ValueError("transposed with an out given needs an out_t")
    to = to_t = None
    if out is not None:
        to = out._ref
        if out._rows != R or out._cols != C or out._index != index:
            raise ValueError(f"out is {out._rows} x {out._cols} on {out.device}: "
                             f"{R} x {C} on {x.device}")
    if out_t is not None:
        to_t = out_t._ref
        if out_t._rows != C or out_t._cols != R or out_t._index != index:
            raise ValueError(f"out_t is {out_t._rows} x {out_t._cols} on {out_t.device}: "
                             f"{C} x {R} on {x.device}")
    _call(lib8().fp8_quantize, "fp8_quantize", index, x.data_ptr(), _code(x.dtype), block_rows, to,
          to_t)
    return out if made and not transposed else (out, out_t)


def fp8_matmul_workspace(M: int, N: int, K: int, device) -> torch.Tensor:
    """Workspace of fp8_matmul for a [M, K] and b [N, K].  Products that can
    run at the same time need one each."""
    nbytes = max(int(lib8().ql_fp8_workspace_bytes(M, N, K)), 256)
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def fp8_matmul(a: FP8Matrix, b: FP8Matrix, out: torch.Tensor | None = None,
               dtype: torch.dtype = torch.bfloat16, accumulate: bool = False,
               ws: torch.Tensor | None = None) -> torch.Tensor:
    """out [M, N] = a b^T for a [M, K] of either format and b [N, K] in
    float8_e4m3fn, in out's type (or a new tensor of `dtype`); accumulate:
    out += a b^T, fp32 only."""
    M, N, index = a._rows, b._rows, a._index
    if a._cols != b._cols or b._index != index:
        raise ValueError(f"a has {a._cols} columns on {a.device}, b {b._cols} on {b.device}")
    if out is None:
        _need(not accumulate, "accumulate needs the out to add into")
        out = torch.empty((M, N), dtype=dtype, device=a.device)
    elif not (out.shape == (M, N) and out.is_contiguous() and out.get_device() == index):
        raise ValueError(f"out is a contiguous {(M, N)} tensor on a's device")
    if ws is None:
        ws = fp8_matmul_workspace(M, N, a._cols, a.device)
    elif not (ws.get_device() == index and ws.is_contiguous()):
        raise ValueError("ws is contiguous and on a's device")
    _call(lib8().fp8_matmul, "fp8_matmul", index, a._ref, b._ref, out.data_ptr(), _code(out.dtype),
          1 if accumulate else 0, ws.data_ptr(), ws.numel() * ws.element_size())
    return out


class AdamWTensors:
    """The tensors of an AdamW step, checked and laid out once for
    adamw_step_many: lists of equal length of fp32 parameters, their gradients
    (all fp32, bf16 or fp16), and their moments: fp32 (no scales), or
    float8_e4m3fn exp_avgs and float8_e5m2 exp_avg_sqs with fp32 scales of one
    value for 256.  copies: bf16 or fp16 tensors that receive the rounded
    parameters, or None (the list, or single ones).

    Every tensor is contiguous, on one GPU, and shares no memory with another
    that is written; the object keeps them alive.  Gradients are read from the
    tensors given here: write new ones into them.  Their addresses are uploaded
    once, here, and their memory is kept: a tensor that is given other memory
    (p.data = ...) needs a new object.  Memory made here (the addresses, and the
    moments of zeros()) may go with the object while a step on another stream
    still runs; of tensors given, that is their owner's care.  A graph that
    captures a step needs the object as long as it lives."""

    def __init__(self, params, grads, exp_avgs, exp_avg_sqs, exp_avg_scales=None,
                 exp_avg_sq_scales=None, copies=None):
        n = len(params)
        none = [None] * n
        eight = exp_avg_scales is not None
        _need(eight == (exp_avg_sq_scales is not None), "scales for both moments or neither")
        lists = [list(params), list(grads), list(exp_avgs), list(exp_avg_sqs),
                 list(exp_avg_scales) if eight else none,
                 list(exp_avg_sq_scales) if eight else none,
                 list(copies) if copies is not None else none]
        _need(all(len(x) == n for x in lists), "the lists are of one length")
        tensors = lambda given: (t for t in given if isinstance(t, torch.Tensor))
        grad_type = next((g.dtype for g in tensors(lists[1])), torch.float32)
        copy_type = next((c.dtype for c in tensors(lists[6])), torch.bfloat16)
        _need(copy_type in (torch.bfloat16, torch.float16), f"copies are {copy_type}: bf16 or fp16")
        types = (torch.float32, grad_type, torch.float8_e4m3fn if eight else torch.float32,
                 torch.float8_e5m2 if eight else torch.float32, torch.float32, torch.float32,
                 copy_type)
        names = ("param", "grad", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale",
                 "copy")
        self._tensors = lists
        first = next(tensors(lists[0]), None)
        dev, index = (None, None) if first is None else (first.device, first.get_device())
        sizes = [p.numel() if isinstance(p, torch.Tensor) else 0 for p in lists[0]]
        blocks = [-(-m // STATE_BLOCK) for m in sizes]
        spans, columns = [], []
        for k, (name, dtype, given) in enumerate(zip(names, types, lists)):
            if k in (4, 5) and not eight:
                columns.append([0] * n)
                continue
            wanted = blocks if k in (4, 5) else sizes
            for i, (t, m) in enumerate(zip(given, wanted)):
                if t is None and k == 6:
                    continue
                if not (isinstance(t, torch.Tensor) and t.dtype == dtype and t.numel() == m
                        and t.is_contiguous() and t.get_device() == index >= 0):
                    raise ValueError(f"{name} {i}: a contiguous {dtype} tensor of {m} values on "
                                     f"{dev}, the parameters' GPU")
            at = [0 if t is None else t.data_ptr() for t in given]
            columns.append(at)
            spans += [(x, x + m * dtype.itemsize, k == 1, name, i)
                      for i, (x, m) in enumerate(zip(at, wanted)) if x and m]
        self._no_overlap(spans)
        self._memory = [t.untyped_storage() for given in lists for t in given if t is not None]
        # the C ABI's structs: seven pointers and n
        self._structs = torch.tensor(columns + [sizes], dtype=torch.int64).t().contiguous()
        self._table = self._structs.to(dev) if n else None
        self.count, self._state_bits = n, 8 if eight else 32
        self._grad_code, self._copy_code = _code(grad_type), _code(copy_type)
        self._refs = (self._structs.data_ptr(), self._table.data_ptr()) if n else (None, None)
        self._index = index
        # memory made here, and the streams that it is known to be used on
        self._own = [self._table] if n else []
        self._streams = {_raw_stream(index)} if n else set()

    @staticmethod
    def _no_overlap(spans):
        """No written memory twice (gradients are only read: two may be the same)."""
        end, last, read_end, read_last = 0, None, 0, None
        for lo, hi, read, name, i in sorted(spans):
            if lo < end or (not read and lo < read_end):
                raise ValueError("%s %d shares memory with %s %d"
                                 % (name, i, *(last if lo < end else read_last)))
            if read and hi > read_end:
                read_end, read_last = hi, (name, i)
            elif not read:
                end, last = hi, (name, i)

    @staticmethod
    def zeros(params, grads, bits: int = 8, copies=None) -> "AdamWTensors":
        """With moments of zeros, in 8 or 32 bits, made here (exp_avgs,
        exp_avg_sqs and their scales are attributes)."""
        _need(bits in (8, 32), f"bits is {bits}: 8 or 32")
        _need(all(isinstance(p, torch.Tensor) for p in params), "params are tensors")
        mk = lambda p, dt: torch.zeros(p.numel(), dtype=torch.uint8 if bits == 8 else torch.float32,
                                       device=p.device).view(dt)
        sc = lambda p: torch.zeros(-(-p.numel() // STATE_BLOCK), device=p.device)
        if bits == 32:
            made = [[mk(p, torch.float32) for p in params] for _ in range(2)]
        else:
            made = [[mk(p, torch.float8_e4m3fn) for p in params],
                    [mk(p, torch.float8_e5m2) for p in params],
                    [sc(p) for p in params], [sc(p) for p in params]]
        plan = AdamWTensors(params, grads, *made, copies=copies)
        plan._own += [t.detach() for given in made for t in given]
        return plan

    params = property(lambda self: self._tensors[0])
    grads = property(lambda self: self._tensors[1])
    exp_avgs = property(lambda self: self._tensors[2])
    exp_avg_sqs = property(lambda self: self._tensors[3])
    exp_avg_scales = property(lambda self: self._tensors[4])
    exp_avg_sq_scales = property(lambda self: self._tensors[5])
    copies = property(lambda self: self._tensors[6])


def adamw_step_many(tensors: AdamWTensors, lr: float, step: int, beta1: float = 0.9,
                    beta2: float = 0.999, eps: float = 1e-8, weight_decay: float = 0.01,
                    grad_scale: torch.Tensor | None = None, seed: int = 0) -> None:
    """One AdamW step in place over all the tensors.  grad_scale: a one-value
    fp32 tensor on the GPU that every gradient is multiplied by first; seed
    draws the rounding of 8-bit moments.  (8-bit second moments below 2^-100 are
    not kept: under an eps below 1e-10, gradients below 3e-14 want 32 bits.)"""
    if tensors.count == 0:
        return
    index = tensors._index
    if grad_scale is not None and not (grad_scale.dtype == torch.float32
                                       and grad_scale.numel() == 1
                                       and grad_scale.get_device() == index):
        raise ValueError("grad_scale is one fp32 value on the parameters' GPU")
    if _raw_stream(index) not in tensors._streams:
        # memory made for the object is not to be given away before this stream is done with it
        stream = torch.cuda.current_stream(index)
        for t in tensors._own:
            t.record_stream(stream)
        tensors._streams.add(stream.cuda_stream)
    _call(lib8().ql_adamw_step_many, "ql_adamw_step_many", index, tensors.count, *tensors._refs,
          tensors._grad_code, tensors._state_bits, tensors._copy_code,
          None if grad_scale is None else grad_scale.data_ptr(), lr, beta1, beta2, eps,
          weight_decay, step, seed & (2**64 - 1))
