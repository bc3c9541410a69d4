"""ctypes binding of libharp (include/harp.h): argument marshalling only.

Every step of the transform runs in the library's CUDA kernels; this module
passes device pointers and the current CUDA stream through.  Loading fails
loudly when libharp.so has not been built — there is no CPU fallback.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional, Sequence

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("HARP_LIB", os.path.join(_HERE, "libharp.so"))

HARP_OK = 0
HARP_ERR_INVALID_ARG = 1
HARP_ERR_SCHEDULE = 2
HARP_ERR_UNSUPPORTED = 3
HARP_ERR_NOT_MATERIALIZED = 4
HARP_ERR_ALLOC = 5
HARP_ERR_CUDA = 6
HARP_ERR_TIMEOUT = 7
HARP_ERR_WRONG_DEVICE = 8

HARP_THETA_F32 = 0
HARP_THETA_I8 = 1
HARP_F32 = 0
HARP_BF16 = 1
HARP_CODE_I8 = 0
HARP_CODE_E4M3 = 1
HARP_FORWARD = 0
HARP_INVERSE = 1

MAX_STAGES = 16

_c_i64 = ctypes.c_int64
_c_i32 = ctypes.c_int32
_c_u64 = ctypes.c_uint64
_vp = ctypes.c_void_p


class HarpError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        super().__init__(f"{where}: {detail or status}")
        self.status = status


_lib = None


def lib():
    """The loaded libharp handle (raises if the library is missing)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libharp.so not found at {LIB_PATH}; build it with "
                          f"`python -m structured_rotations_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    sig = {
        "harp_plan_create": (_c_i32, [ctypes.POINTER(_vp), _c_i64, ctypes.POINTER(_c_i32), _c_i32,
                                      _c_i32, _vp, ctypes.POINTER(ctypes.c_float), _c_u64, _c_u64]),
        "harp_materialize_blocks": (_c_i32, [_vp, _vp]),
        "harp_apply": (_c_i32, [_vp, _vp, _vp, _c_i64, _c_i64, _c_i64, _c_i32, _c_i32, _vp]),
        "harp_apply_ex": (_c_i32, [_vp, _vp, _vp, _c_i64, _c_i64, _c_i64, _c_i32, _c_i32, _c_i32, _vp]),
        "harp_apply_columns": (_c_i32, [_vp, _vp, _c_i64, _c_i64, _vp, _c_i64, _c_i32, _c_i32, _vp]),
        "harp_apply_host": (_c_i32, [_vp, _vp, _vp, _c_i64, _c_i64, _c_i64, _c_i32, _c_i32]),
        "harp_two_sided_workspace_bytes": (ctypes.c_size_t, [_c_i64, _c_i64]),
        "harp_apply_two_sided": (_c_i32, [_vp, _vp, _vp, _vp, _c_i64, _c_i64, _c_i64, _c_i32, _vp,
                                          ctypes.c_size_t, _vp]),
        "harp_apply_two_sided_noalloc": (_c_i32, [_vp, _vp, _vp, _vp, _c_i64, _c_i64, _c_i64, _c_i32,
                                                  _vp]),
        "harp_noalloc_scratch_bytes": (ctypes.c_size_t, []),
        "harp_plan_device_status": (_c_i32, [_vp]),
        "harp_device_status": (_c_i32, []),
        "harp_grad_workspace_bytes": (ctypes.c_size_t, [_vp]),
        "harp_plan_compose": (_c_i32, [ctypes.POINTER(_vp), ctypes.POINTER(_vp), _c_i32, _vp]),
        "harp_apply_quant": (_c_i32, [_vp, _vp, _c_i64, _c_i64, _c_i32, _vp, _c_i64, _vp, _c_i64, _c_i32, _c_i32,
                                      _vp]),
        "harp_apply_quant_ex": (_c_i32, [_vp, _vp, _c_i64, _c_i64, _c_i32, _c_i32, _vp, _c_i64, _vp, _c_i64, _c_i32,
                                         _c_i32, _vp]),
        "harp_quantize": (_c_i32, [_vp, _c_i64, _c_i64, _c_i64, _c_i32, _c_i32, _c_i32, _c_i32, _vp, _c_i64, _vp,
                                   _c_i64, _vp]),
        "harp_dequantize": (_c_i32, [_vp, _c_i64, _vp, _c_i64, _c_i32, _c_i32, _c_i32, _c_i64, _c_i64, _vp, _c_i64,
                                     _c_i32, _vp]),
        "harp_rms_norm_quant": (_c_i32, [_vp, _c_i64, _vp, _c_i64, _vp, _c_i64, _c_i64, _c_i32, ctypes.c_double, _vp,
                                         _c_i64, _vp, _c_i64, _c_i32, _c_i32, _vp, _c_i64, _vp, _c_i64, _vp]),
        "harp_matmul_quant": (_c_i32, [_vp, _c_i64, _vp, _c_i64, _vp, _c_i64, _vp, _c_i64, _c_i64, _c_i64, _c_i64,
                                       _vp, _c_i64, _c_i32, _vp]),
        "harp_grad_theta_quant": (_c_i32, [_vp, _vp, _c_i64, _c_i32, _vp, _c_i64, _c_i32, _vp, _c_i64, _c_i32, _c_i64,
                                           _vp, _vp, ctypes.c_size_t, _vp]),
        "harp_grad_theta": (_c_i32, [_vp, _vp, _vp, _c_i64, _c_i64, _c_i64, _c_i32, _vp, _vp, ctypes.c_size_t,
                                     _vp]),
        "harp_off_block_energy": (_c_i32, [_vp, _c_i64, _c_i64, _c_i32, _c_i32, _vp, _vp]),
        "harp_l_diag": (_c_i32, [_vp, _c_i64, _c_i64, _c_i64, _c_i32, _vp, _c_i64, _c_i32, _vp, _vp]),
        "harp_test_inject_wait_timeout": (_c_i32, [_c_i64, ctypes.c_uint32]),
        "harp_moment_check": (_c_i32, [_vp, _c_i64, _c_i64, _c_i64, _c_i32, ctypes.c_double, ctypes.c_double, _vp,
                                       _vp, _vp]),
        "harp_plan_destroy": (_c_i32, [_vp]),
        "harp_status_string": (ctypes.c_char_p, [_c_i32]),
        "harp_last_error": (ctypes.c_char_p, []),
        "harp_last_kernel": (ctypes.c_char_p, []),
        "harp_theta_count": (_c_i64, [ctypes.POINTER(_c_i32), _c_i32]),
        "harp_splitmix64": (_c_i32, [_c_u64, _c_i64, ctypes.POINTER(_c_u64)]),
        "harp_plan_base_mixer": (_c_i32, [_vp, _c_i32, ctypes.POINTER(ctypes.c_double)]),
        "harp_plan_signs": (_c_i32, [_vp, ctypes.POINTER(ctypes.c_int8)]),
        "harp_plan_shape": (_c_i32, [_vp, ctypes.POINTER(_c_i64), ctypes.POINTER(_c_i32),
                                     ctypes.POINTER(_c_i32)]),
    }
    for name, (res, args) in sig.items():
        fn = getattr(L, name)
        fn.restype = res
        fn.argtypes = args
    _lib = L
    return L


def _check(status: int, where: str):
    if status != HARP_OK:
        L = lib()
        detail = (L.harp_last_error() or b"").decode()
        name = L.harp_status_string(status).decode()
        raise HarpError(status, where, detail or name)


def _radices(schedule: Sequence[int]):
    arr = (_c_i32 * len(schedule))(*[int(b) for b in schedule])
    return arr


def theta_count(schedule: Sequence[int]) -> int:
    return int(lib().harp_theta_count(_radices(schedule), len(schedule)))


def splitmix64(seed: int, n: int) -> np.ndarray:
    out = np.empty(n, dtype=np.uint64)
    _check(lib().harp_splitmix64(_c_u64(seed), n, out.ctypes.data_as(ctypes.POINTER(_c_u64))),
           "harp_splitmix64")
    return out


def _stream_handle(stream) -> Optional[int]:
    if stream is None:
        import torch
        C = torch._C
        if hasattr(C, "_cuda_getCurrentRawStream"):   # the handle without a Stream object
            return C._cuda_getCurrentRawStream(C._cuda_getDevice())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _on(stream):
    """The context of a call on `stream` (a torch stream or a handle): what the call allocates belongs to
    that stream, so its memory neither comes from work that another stream has still under way nor
    goes to another stream before the call's kernels are done."""
    import torch
    if isinstance(stream, int):
        stream = torch.cuda.ExternalStream(stream) if stream else torch.cuda.default_stream()
    return torch.cuda.stream(stream)


_DTYPE = {"float32": HARP_F32, "bfloat16": HARP_BF16}


_DTYPE_OF = {}   # torch dtype -> code, filled on first use


def _dtype_code(t) -> int:
    code = _DTYPE_OF.get(t.dtype)
    if code is None:
        name = str(t.dtype).replace("torch.", "")
        if name not in _DTYPE:
            raise TypeError(f"unsupported dtype {t.dtype}; use float32 or bfloat16")
        code = _DTYPE_OF[t.dtype] = _DTYPE[name]
    return code


def _ld(t) -> int:
    if t.dim() != 2:
        raise ValueError("expected a 2-D tensor of rows")
    if t.stride(1) != 1:
        raise ValueError("rows must be contiguous (stride(1) == 1)")
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


_CODE_DTYPE = {}   # code -> torch dtype, filled on first use
_CODE = {"int8": HARP_CODE_I8, "e4m3": HARP_CODE_E4M3}


def _code(name: str) -> int:
    if name not in _CODE:
        raise ValueError(f"code must be 'int8' or 'e4m3', not {name!r}")
    return _CODE[name]


def _code_dtype(code: int):
    """The tensor type that holds codes of this format."""
    if not _CODE_DTYPE:
        import torch
        _CODE_DTYPE.update({HARP_CODE_I8: torch.int8, HARP_CODE_E4M3: torch.float8_e4m3fn})
    return _CODE_DTYPE[code]


def _code_of(q) -> int:
    """The code format of a tensor of codes, by its type."""
    for code in _CODE.values():
        if q.dtype is _code_dtype(code):
            return code
    raise TypeError(f"codes are int8 or float8_e4m3fn tensors, not {q.dtype}")


def _expect(t, shape, dtype, dev: int, what: str):
    """(address, leading dimension) of a 2-D tensor (address alone of a 1-D one), which must be on the CUDA
    device dev with this shape and type and contiguous rows.  One pass over the tensor's attributes:
    calls of a few microseconds spend most of their time here."""
    if t.shape != shape:
        raise ValueError(f"{what} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise TypeError(f"{what} must be {dtype}, not {t.dtype}")
    if t.get_device() != dev:
        raise ValueError(f"{what} must be on the current CUDA device, not {t.device}")
    if t.is_contiguous():   # also a single row of any stride, whose leading dimension no entry looks at
        return (t.data_ptr(), shape[1]) if len(shape) == 2 else t.data_ptr()
    st = t.stride()
    if len(st) == 1:
        raise ValueError(f"{what} must be contiguous")
    if st[1] != 1 and shape[1] > 1:
        raise ValueError(f"the rows of {what} must be contiguous (stride(1) == 1)")
    return t.data_ptr(), (st[0] if shape[0] > 1 else max(st[0], shape[1]))


_TORCH = None   # (float8_e4m3fn, float32, current device, its current raw stream), filled on first use


def _torch():
    global _TORCH
    if _TORCH is None:
        import torch
        C = torch._C
        raw = getattr(C, "_cuda_getCurrentRawStream", None) or (lambda dev: torch.cuda.current_stream(dev).cuda_stream)
        _TORCH = (torch.float8_e4m3fn, torch.float32, C._cuda_getDevice, raw)
    return _TORCH


def _device(t, what: str, current) -> int:
    """The current CUDA device (current()), which must be t's."""
    dev = t.get_device()
    if dev < 0 or dev != current():
        raise ValueError(f"{what} must be on the current CUDA device, not {t.device}")
    return dev


def _rows_of(t, what: str):
    s = t.shape
    if len(s) != 2:
        raise ValueError(f"{what} must be a 2-D tensor")
    return s


def _cdiv(a: int, b: int) -> int:
    return -(-a // b)


class Plan:
    """One HARP rotation: schedule, parameters, signs, mixers and device blocks."""

    def __init__(self, d: int, schedule: Sequence[int], theta=None, sign_seed: int = 0,
                 qr_seed: int = 0, codes=None, scales=None):
        L = lib()
        self.d = int(d)
        self.schedule = tuple(int(b) for b in schedule)
        handle = _vp()
        if codes is not None:
            codes = np.ascontiguousarray(codes, dtype=np.int8)
            scales = np.ascontiguousarray(scales, dtype=np.float32)
            kind, ptr = HARP_THETA_I8, codes.ctypes.data
            sptr = scales.ctypes.data_as(ctypes.POINTER(ctypes.c_float))
            self._keep = (codes, scales)
        else:
            kind = HARP_THETA_F32
            if theta is not None:
                theta = np.ascontiguousarray(theta, dtype=np.float32)
                ptr = theta.ctypes.data
            else:
                ptr = None
            sptr = None
            self._keep = (theta,)
        st = L.harp_plan_create(ctypes.byref(handle), self.d, _radices(self.schedule),
                                len(self.schedule), kind, ptr, sptr, _c_u64(sign_seed), _c_u64(qr_seed))
        _check(st, "harp_plan_create")
        self._h = handle

    @property
    def handle(self):
        return self._h

    @classmethod
    def compose(cls, plans: Sequence["Plan"], stream=None) -> "Plan":
        """One plan for T_{k-1} ... T_0 of materialized plans of one dimension (plans[0]
        acts first), applied in a single pass (harp_plan_compose)."""
        if not plans:
            raise ValueError("need at least one plan")
        arr = (_vp * len(plans))(*[p.handle for p in plans])
        handle = _vp()
        _check(lib().harp_plan_compose(ctypes.byref(handle), arr, len(plans), _stream_handle(stream)),
               "harp_plan_compose")
        c = cls.__new__(cls)
        c.d = plans[0].d
        c.schedule = tuple(b for p in plans for b in p.schedule)
        c._keep = ()
        c._h = handle
        c.composite = True
        return c

    def materialize(self, stream=None) -> "Plan":
        _check(lib().harp_materialize_blocks(self._h, _stream_handle(stream)), "harp_materialize_blocks")
        return self

    def apply(self, x, y=None, direction: str = "forward", stream=None, rows: Optional[int] = None):
        """y = T x (forward) or T^T x (inverse) row by row; y defaults to a new tensor."""
        import torch
        if y is None:
            y = torch.empty_like(x)
        if x.dtype != y.dtype:
            raise TypeError("x and y must share a dtype")
        if x.shape[-1] != self.d or y.shape[-1] != self.d:
            raise ValueError(f"last dimension must be d={self.d}")
        n = x.shape[0] if rows is None else rows
        d = HARP_FORWARD if direction == "forward" else HARP_INVERSE
        _check(lib().harp_apply(self._h, x.data_ptr(), y.data_ptr(), n, _ld(x), _ld(y),
                                _dtype_code(x), d, _stream_handle(stream)), "harp_apply")
        return y

    def apply_quant(self, x, qblock: int = 128, direction: str = "forward", q=None, scales=None, stream=None,
                    code: str = "int8"):
        """T x (or T^T x) with the fused blockwise quantizer (harp_apply_quant_ex): bf16 rows in,
        codes [rows, d] (int8, or float8_e4m3fn for code="e4m3") and float32 scales
        [rows, d / qblock] out, y ~= q * scale per aligned block of qblock coordinates.
        Returns (q, scales); e4m3 codes in blocks of 128 are matmul_quant's row operand.  Forward batches of
        32 rows or more of a d = 4096 (8,8,8,8) plan are multiplied in TF32 hi and lo parts, all others in
        fp32 (see harp_apply_quant_ex for how far the codes differ)."""
        import torch
        if stream is not None:
            with _on(stream):
                return self.apply_quant(x, qblock, direction, q, scales, None, code)
        if x.shape[-1] != self.d:
            raise ValueError(f"last dimension must be d={self.d}")
        fmt = _code(code)
        rows = x.shape[0]
        if q is None:
            q = torch.empty(rows, self.d, dtype=_code_dtype(fmt), device=x.device)
        if scales is None:
            scales = torch.empty(rows, max(1, self.d // qblock), dtype=torch.float32, device=x.device)
        if fmt == HARP_CODE_E4M3:
            dev = _device(x, "x", (_TORCH or _torch())[2])
            xp, ldx = _expect(x, (rows, self.d), x.dtype, dev, "x")
            qp, ldq = _expect(q, (rows, self.d), torch.float8_e4m3fn, dev, "q")
            sp, lds = _expect(scales, (rows, max(1, self.d // qblock)), torch.float32, dev, "scales")
        else:
            if q.dtype is torch.float8_e4m3fn:
                raise TypeError("q holds e4m3 codes: give code='e4m3'")
            xp, ldx, qp, ldq, sp, lds = x.data_ptr(), _ld(x), q.data_ptr(), _ld(q), scales.data_ptr(), _ld(scales)
        d = HARP_FORWARD if direction == "forward" else HARP_INVERSE
        _check(lib().harp_apply_quant_ex(self._h, xp, rows, ldx, _dtype_code(x), fmt, qp, ldq, sp, lds, qblock, d,
                                         _stream_handle(None)), "harp_apply_quant")
        return q, scales

    def grad_workspace(self, device=None):
        """A workspace for grad_theta and grad_theta_quant (uint8, harp_grad_workspace_bytes), to keep
        between calls; calls that may run at once need one each."""
        import torch
        return torch.empty(int(lib().harp_grad_workspace_bytes(self._h)), dtype=torch.uint8,
                           device="cuda" if device is None else device)

    def grad_theta_quant(self, q, scales, g, dtheta=None, workspace=None, stream=None, qblock: Optional[int] = None):
        """dL/dtheta for L = sum_r g_r . (T x_r) with the rows x kept as 8-bit checkpoints
        (harp_grad_theta_quant): codes q [rows, d] (int8 or float8_e4m3fn) and float32 scales
        [rows, ceil(d / qblock)] of H.quantize(x, (1, qblock), ...), upstream gradients g [rows, d]
        (bf16 or fp32).  qblock defaults to the one that the scales' shape gives when it divides d.
        Returns a float32 tensor of theta_count entries."""
        import torch
        if stream is not None:
            with _on(stream):
                return self.grad_theta_quant(q, scales, g, dtheta, workspace, None, qblock)
        rows = q.shape[0]
        if qblock is None:
            nb = scales.shape[1] if scales.dim() == 2 else 0
            if nb < 1 or self.d % nb or self.d // nb not in (32, 64, 128, 256):
                raise ValueError("give qblock: the scales' shape does not tell it")
            qblock = self.d // nb
        if qblock not in (32, 64, 128, 256):
            raise ValueError("qblock must be 32, 64, 128 or 256")
        code, dev = _code_of(q), _device(q, "q", (_TORCH or _torch())[2])
        qp, ldq = _expect(q, (rows, self.d), q.dtype, dev, "q")
        sp, lds = _expect(scales, (rows, _cdiv(self.d, qblock)), torch.float32, dev, "scales")
        gt = _dtype_code(g)
        gp, ldg = _expect(g, (rows, self.d), g.dtype, dev, "g")
        n = theta_count(self.schedule) if not getattr(self, "composite", False) else 1
        if dtheta is None:
            dtheta = torch.empty(n, dtype=torch.float32, device=q.device)
        tp = _expect(dtheta, (n,), torch.float32, dev, "dtheta")
        if workspace is None:
            workspace = self.grad_workspace(q.device)
        elif not workspace.is_contiguous() or workspace.get_device() != dev:
            raise ValueError("workspace must be contiguous, on the current CUDA device")
        _check(lib().harp_grad_theta_quant(self._h, qp, ldq, code, sp, lds, qblock, gp, ldg, gt, rows, tp,
                                           workspace.data_ptr(), workspace.numel() * workspace.element_size(),
                                           _stream_handle(None)),
               "harp_grad_theta_quant")
        return dtheta

    def grad_theta(self, x, g, dtheta=None, workspace=None, stream=None):
        """dL/dtheta for L = sum_r g_r . (T x_r) (harp_grad_theta): the calibration backward
        through the forward transform, for rows x and upstream gradients g = dL/dy of one
        dtype on the GPU.  Returns a float32 tensor of theta_count entries (dtheta, if
        given, is filled).  dL/dx is self.apply(g, direction="inverse")."""
        import torch
        if stream is not None:
            with _on(stream):
                return self.grad_theta(x, g, dtheta, workspace)
        if x.dtype != g.dtype or x.shape != g.shape or x.shape[-1] != self.d:
            raise ValueError(f"x and g must be rows of d={self.d} of one dtype")
        # a composite's schedule is its plans' schedules in a row (no theta count of its
        # own): the library declines it, so any buffer does
        n = theta_count(self.schedule) if not getattr(self, "composite", False) else 1
        if dtheta is None:
            dtheta = torch.empty(n, dtype=torch.float32, device=x.device)
        if dtheta.dtype != torch.float32 or dtheta.numel() != n or not dtheta.is_contiguous():
            raise ValueError(f"dtheta must be a contiguous float32 tensor of {n} entries")
        if workspace is None:
            workspace = self.grad_workspace(x.device)
        _check(lib().harp_grad_theta(self._h, x.data_ptr(), g.data_ptr(), x.shape[0], _ld(x), _ld(g),
                                     _dtype_code(x), dtheta.data_ptr(), workspace.data_ptr(),
                                     workspace.numel() * workspace.element_size(), _stream_handle(None)),
               "harp_grad_theta")
        return dtheta

    def apply_host(self, x, y=None, direction: str = "forward"):
        """Rows of a host (CPU) tensor through the GPU and back (harp_apply_host): copies,
        kernels and copies overlap in chunks; pin x and y (tensor.pin_memory()) for the
        overlap.  Returns y (a new host tensor by default)."""
        import torch
        if x.device.type != "cpu":
            raise ValueError("apply_host takes host tensors; use apply for device tensors")
        if y is None:
            y = torch.empty_like(x, pin_memory=x.is_pinned())
        if x.dtype != y.dtype or x.shape != y.shape or x.shape[-1] != self.d:
            raise ValueError(f"x and y must be rows of d={self.d} of one dtype")
        d = HARP_FORWARD if direction == "forward" else HARP_INVERSE
        _check(lib().harp_apply_host(self._h, x.data_ptr(), y.data_ptr(), x.shape[0], _ld(x), _ld(y),
                                     _dtype_code(x), d), "harp_apply_host")
        return y

    def apply_ex(self, x, y, direction: str = "forward", stream=None):
        """Rows of x (float32 or bfloat16) into y of its own type (harp_apply_ex), e.g. bf16
        rows into an fp32 intermediate."""
        if x.shape[-1] != self.d or y.shape[-1] != self.d or x.shape[0] != y.shape[0]:
            raise ValueError(f"x and y must both be rows of d={self.d}")
        d = HARP_FORWARD if direction == "forward" else HARP_INVERSE
        _check(lib().harp_apply_ex(self._h, x.data_ptr(), y.data_ptr(), x.shape[0], _ld(x), _ld(y),
                                   _dtype_code(x), _dtype_code(y), d, _stream_handle(stream)), "harp_apply_ex")
        return y

    def apply_columns(self, x, y=None, direction: str = "forward", stream=None):
        """Every column of the fp32 matrix x (d rows) takes T or T^T (harp_apply_columns);
        y defaults to x itself (in place); a bfloat16 y receives the rounded result.  x is
        overwritten either way."""
        import torch
        if x.dtype != torch.float32 or x.shape[0] != self.d:
            raise ValueError(f"x must be float32 with d={self.d} rows")
        if y is None:
            y = x
        if y.shape != x.shape:
            raise ValueError("y must have the shape of x")
        d = HARP_FORWARD if direction == "forward" else HARP_INVERSE
        _check(lib().harp_apply_columns(self._h, x.data_ptr(), _ld(x), x.shape[1], y.data_ptr(), _ld(y),
                                        _dtype_code(y), d, _stream_handle(stream)), "harp_apply_columns")
        return y

    def device_status(self) -> None:
        """Synchronize and raise HarpError(HARP_ERR_TIMEOUT) if a bounded device
        wait of a kernel launched with this plan gave up."""
        _check(lib().harp_plan_device_status(self._h), "harp_plan_device_status")

    def base_mixer(self, radix: int) -> np.ndarray:
        out = np.empty((radix, radix), dtype=np.float64)
        _check(lib().harp_plan_base_mixer(self._h, radix, out.ctypes.data_as(ctypes.POINTER(ctypes.c_double))),
               "harp_plan_base_mixer")
        return out

    def signs(self) -> np.ndarray:
        out = np.empty(self.d, dtype=np.int8)
        _check(lib().harp_plan_signs(self._h, out.ctypes.data_as(ctypes.POINTER(ctypes.c_int8))),
               "harp_plan_signs")
        return out

    def shape(self):
        d = _c_i64()
        m = _c_i32()
        r = (_c_i32 * MAX_STAGES)()
        _check(lib().harp_plan_shape(self._h, ctypes.byref(d), ctypes.byref(m), r), "harp_plan_shape")
        return d.value, tuple(r[: m.value])

    def close(self):
        if getattr(self, "_h", None):
            lib().harp_plan_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def last_kernel() -> str:
    """Name of the last kernel launched by this thread through the library."""
    return (lib().harp_last_kernel() or b"").decode()


def workspace_bytes(n_out: int, n_in: int) -> int:
    return int(lib().harp_two_sided_workspace_bytes(n_out, n_in))


def apply_two_sided(plan_u: Plan, plan_v: Plan, w, w_out=None, workspace=None, stream=None):
    """W_out = T_U^T W T_V (U on the output side, V on the input side)."""
    import torch
    n_out, n_in = w.shape
    if w_out is None:
        w_out = torch.empty_like(w)
    need = workspace_bytes(n_out, n_in)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=w.device)
    ld = _ld(w)
    if _ld(w_out) != ld:
        raise ValueError("W and W_out must share a leading dimension")
    _check(lib().harp_apply_two_sided(plan_u.handle, plan_v.handle, w.data_ptr(), w_out.data_ptr(),
                                      n_out, n_in, ld, _dtype_code(w), workspace.data_ptr(),
                                      workspace.numel() * workspace.element_size(),
                                      _stream_handle(stream)), "harp_apply_two_sided")
    return w_out


def off_block_energy(h, q: int, out=None, stream=None):
    """(energy of the square matrix h outside its q x q diagonal blocks, total energy) as a
    device float64 tensor of 2 (harp_off_block_energy); R_bd = out[0] / out[1]."""
    import torch
    n = h.shape[0]
    if h.dim() != 2 or h.shape[1] != n:
        raise ValueError("h must be square")
    if out is None:
        out = torch.empty(2, dtype=torch.float64, device=h.device)
    _check(lib().harp_off_block_energy(h.data_ptr(), n, _ld(h), _dtype_code(h), q, out.data_ptr(),
                                       _stream_handle(stream)), "harp_off_block_energy")
    return out


def l_diag(w, h, qblock: int, out=None, stream=None):
    """sum_j h_jj sum_r (w_rj - Q(w)_rj)^2 with Q the blockwise int8 quantizer along the rows
    (harp_l_diag), as a device float64 tensor of 1; h is float32 (only its diagonal is read)."""
    import torch
    rows, cols = w.shape
    if h.dtype != torch.float32 or h.shape[0] < cols or h.shape[1] < cols:
        raise ValueError("h must be a float32 matrix of at least cols x cols")
    if out is None:
        out = torch.empty(1, dtype=torch.float64, device=w.device)
    _check(lib().harp_l_diag(w.data_ptr(), rows, cols, _ld(w), _dtype_code(w), h.data_ptr(), _ld(h), qblock,
                             out.data_ptr(), _stream_handle(stream)), "harp_l_diag")
    return out


def inject_wait_timeout(poll_limit: int = 0, extra_bytes: int = 0) -> None:
    """Test hook (harp_test_inject_wait_timeout): make the staging waits of this thread's
    next tiled-kernel launches run out after poll_limit polls, and the waits of its matmul_quant
    launches on the tensor cores after poll_limit clocks; (0, 0) clears it."""
    _check(lib().harp_test_inject_wait_timeout(poll_limit, extra_bytes), "harp_test_inject_wait_timeout")


def moment_check(x, tau1: float = 0.0, tau2: float = 0.0, moments=None, passes=None, stream=None):
    """Per row of the device rows x (harp_moment_check): (sum x^2, sum |x|^3, sum x^4) as a float64
    tensor [rows, 3], and the number of composed passes (1 if m4 / m2^2 <= tau1, 2 if <= tau2, else
    3) as an int32 tensor [rows].  Returns (moments, passes)."""
    import torch
    rows, d = x.shape
    if moments is None:
        moments = torch.empty(rows, 3, dtype=torch.float64, device=x.device)
    if passes is None:
        passes = torch.empty(rows, dtype=torch.int32, device=x.device)
    _check(lib().harp_moment_check(x.data_ptr(), rows, d, _ld(x), _dtype_code(x), float(tau1), float(tau2),
                                   moments.data_ptr(), passes.data_ptr(), _stream_handle(stream)),
           "harp_moment_check")
    return moments, passes


def quantize(x, block=(1, 128), code: str = "e4m3", q=None, scales=None, stream=None):
    """8-bit codes of the device matrix x with one float32 scale per block (harp_quantize):
    x ~= q * scale, q int8 or float8_e4m3fn [rows, cols], scales [ceil(rows / b0), ceil(cols / b1)]
    for block = (b0, b1): (1, 32 | 64 | 128 | 256) for rows (checkpoints for Plan.grad_theta_quant;
    e4m3 with 128: matmul_quant's row operand), (128, 128) for a weight (matmul_quant's).
    Returns (q, scales).  A new q has rows a multiple of 16 bytes apart."""
    if stream is not None:
        with _on(stream):
            return quantize(x, block, code, q, scales)
    _, f32, current, raw = _TORCH or _torch()
    fmt, dev = _code(code), _device(x, "x", current)
    rows, cols = shape = _rows_of(x, "x")
    dt, qt = _dtype_code(x), _code_dtype(fmt)
    xp, ldx = _expect(x, shape, x.dtype, dev, "x")
    br, bc = block
    if br < 1 or bc < 1:
        raise ValueError("blocks are (1, 32 | 64 | 128 | 256) or (128, 128)")
    sshape = (-(-rows // br), -(-cols // bc))
    if q is None:
        q = x.new_empty((rows, _cdiv(cols, 16) * 16), dtype=qt)[:, :cols]
    if scales is None:
        scales = x.new_empty(sshape, dtype=f32)
    qp, ldq = _expect(q, shape, qt, dev, "q")
    sp, lds = _expect(scales, sshape, f32, dev, "scales")
    _check(lib().harp_quantize(xp, rows, cols, ldx, dt, fmt, br, bc, qp, ldq, sp, lds,
                               raw(dev)), "harp_quantize")
    return q, scales


def dequantize(q, scales, block=(1, 128), out=None, dtype=None, stream=None):
    """The values q * scale of quantize's codes (harp_dequantize), rounded to out's type (a new tensor
    of `dtype`, bfloat16 by default).  Returns out."""
    if stream is not None:
        with _on(stream):
            return dequantize(q, scales, block, out, dtype)
    _, f32, current, raw = _TORCH or _torch()
    code, dev = _code_of(q), _device(q, "q", current)
    rows, cols = shape = _rows_of(q, "q")
    qp, ldq = _expect(q, shape, q.dtype, dev, "q")
    br, bc = block
    if br < 1 or bc < 1:
        raise ValueError("blocks are (1, 32 | 64 | 128 | 256) or (128, 128)")
    if out is None:
        import torch
        out = torch.empty(rows, cols, dtype=dtype or torch.bfloat16, device=q.device)
    elif dtype is not None and out.dtype != dtype:
        raise TypeError("out has another dtype")
    sp, lds = _expect(scales, (-(-rows // br), -(-cols // bc)), f32, dev, "scales")
    dt = _dtype_code(out)
    yp, ldy = _expect(out, shape, out.dtype, dev, "out")
    _check(lib().harp_dequantize(qp, ldq, sp, lds, code, br, bc, rows, cols, yp, ldy, dt,
                                 raw(dev)), "harp_dequantize")
    return out


def rms_norm_quant(x, weight=None, residual=None, eps: float = 1e-6, qblock: int = 128, code: str = "e4m3", h=None,
                   y=None, q=None, scales=None, stream=None):
    """h = x + residual, u = h / sqrt(mean(h^2) + eps) * weight and u's 8-bit codes in one pass
    (harp_rms_norm_quant).  x and residual: rows [rows, d] (bf16 or fp32), weight [d] of their type or
    None.  h receives the sum (it may be x or residual; a new tensor where there is a residual),
    y, if given, u rounded to x's type.  Returns (q, scales, h): codes [rows, d] (int8 or
    float8_e4m3fn), float32 scales [rows, ceil(d / qblock)], and the sum (x itself without a
    residual, unless h is given)."""
    if stream is not None:
        with _on(stream):
            return rms_norm_quant(x, weight, residual, eps, qblock, code, h, y, q, scales)
    _, f32, current, raw = _TORCH or _torch()
    fmt, dev = _code(code), _device(x, "x", current)
    rows, d = shape = _rows_of(x, "x")
    dt, t = _dtype_code(x), x.dtype
    if qblock not in (32, 64, 128, 256):
        raise ValueError("qblock must be 32, 64, 128 or 256")
    xp, ldx = _expect(x, shape, t, dev, "x")
    rp = wp = hp = yp = None
    ldr = ldh = ldy = 0
    if residual is not None:
        rp, ldr = _expect(residual, shape, t, dev, "residual")
        if h is None:
            h = x.new_empty(shape)
    if weight is not None:
        wp = _expect(weight, (d,), t, dev, "weight")
    if h is not None:
        hp, ldh = _expect(h, shape, t, dev, "h")
    if y is not None:
        yp, ldy = _expect(y, shape, t, dev, "y")
    qt, nb = _code_dtype(fmt), _cdiv(d, qblock)
    if q is None:
        q = x.new_empty((rows, _cdiv(d, 16) * 16), dtype=qt)[:, :d]
    if scales is None:
        scales = x.new_empty((rows, nb), dtype=f32)
    qp, ldq = _expect(q, shape, qt, dev, "q")
    sp, lds = _expect(scales, (rows, nb), f32, dev, "scales")
    _check(lib().harp_rms_norm_quant(xp, ldx, rp, ldr, wp, rows, d, dt, eps, hp, ldh, yp, ldy, fmt, qblock, qp, ldq,
                                     sp, lds, raw(dev)),
           "harp_rms_norm_quant")
    return q, scales, x if h is None else h


def matmul_quant(xq, xs, wq, ws, out=None, dtype=None, stream=None):
    """out = (xq * xs) (wq * ws)^T (harp_matmul_quant): e4m3 codes xq [rows, k] with float32 scales
    xs [rows, ceil(k / 128)], e4m3 codes wq [n, k] with scales ws [ceil(n / 128), ceil(k / 128)];
    out [rows, n] in bfloat16 (the default) or float32.  Operands 16-byte aligned with leading
    dimensions that are multiples of 16, as quantize and apply_quant make them, run on the tensor
    cores.  Returns out."""
    if stream is not None:
        with _on(stream):
            return matmul_quant(xq, xs, wq, ws, out, dtype)
    f8, f32, current, raw = _TORCH or _torch()
    dev = _device(xq, "xq", current)
    rows, k = xshape = _rows_of(xq, "xq")
    n, kw = wshape = _rows_of(wq, "wq")
    kb = -(-k // 128)
    if kw != k:
        raise ValueError(f"wq must have {k} columns as xq, not {kw}")
    xp, ldx = _expect(xq, xshape, f8, dev, "xq")
    wp, ldw = _expect(wq, wshape, f8, dev, "wq")
    sp, lds = _expect(xs, (rows, kb), f32, dev, "xs")
    vp, ldv = _expect(ws, (-(-n // 128), kb), f32, dev, "ws")
    if out is None:
        import torch
        out = torch.empty(rows, n, dtype=dtype or torch.bfloat16, device=xq.device)
    elif dtype is not None and out.dtype != dtype:
        raise TypeError("out has another dtype")
    dt = _dtype_code(out)
    yp, ldy = _expect(out, (rows, n), out.dtype, dev, "out")
    _check(lib().harp_matmul_quant(xp, ldx, sp, lds, wp, ldw, vp, ldv, rows, n, k, yp, ldy, dt,
                                   raw(dev)), "harp_matmul_quant")
    return out


def device_status() -> None:
    """Synchronize the current device and raise HarpError(HARP_ERR_TIMEOUT) if a bounded device wait of
    matmul_quant gave up since the last call (harp_device_status).  The device has one status word for all
    threads and streams: the call that raises clears it, whoever launched the kernel."""
    _check(lib().harp_device_status(), "harp_device_status")
