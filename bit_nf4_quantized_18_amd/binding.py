"""Thin ctypes binding over libqlora_nf4.so (the C ABI in include/qlora_nf4.h).

Argument marshalling only: every step of the layer runs in the HIP kernels.
Tensors are torch tensors on the current HIP device; work is enqueued on
torch's current stream. There is no fallback: if the library is missing the
functions raise.
"""
from __future__ import annotations

import array
import ctypes
import dataclasses
import operator
import os

PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(PKG, "libqlora_nf4.so")

QLORA_BF16, QLORA_F32, QLORA_F16 = 0, 1, 2
MAX_RANK = 128
BLOCK, DQ_GROUP = 64, 256
INT8_MAX_COLS, INT8_MAX_K = 1 << 22, 131008  # QLORA_INT8_MAX_COLS, QLORA_INT8_MAX_K

STATUS = {0: "QLORA_OK", -1: "QLORA_ERR_NULL", -2: "QLORA_ERR_SHAPE", -3: "QLORA_ERR_ALIGN",
          -4: "QLORA_ERR_UNSUPPORTED", -5: "QLORA_ERR_WORKSPACE", -6: "QLORA_ERR_HIP"}

# Every symbol include/qlora_nf4.h declares.
EXPORTS = ("qlora_nf4_quantize", "qlora_nf4_dequantize", "qlora_linear_fwd", "qlora_linear_bwd",
           "qlora_linear_workspace_bytes", "qlora_linear_fwd_grouped", "qlora_linear_bwd_grouped",
           "qlora_linear_grouped_workspace_bytes", "qlora_status_string", "qlora_nf4_levels",
           "qlora_quantize_codebook", "qlora_codebook_levels", "qlora_merge", "qlora_unmerge",
           "qlora_requantize", "qlora_linear_dropout_workspace_bytes", "qlora_linear_fwd_dropout",
           "qlora_linear_bwd_dropout", "qlora_dropout_mask", "qlora_linear_fwd_f16", "qlora_linear_bwd_f16",
           "qlora_linear_fwd_grouped_f16", "qlora_linear_bwd_grouped_f16", "qlora_linear_fwd_dropout_f16",
           "qlora_linear_bwd_dropout_f16", "qlora_linear_fwd_noalloc", "qlora_int8_quantize",
           "qlora_int8_dequantize", "qlora_rmsnorm_int8", "qlora_int8_linear_fwd",
           "qlora_grad_norm", "qlora_grad_clip", "qlora_grad_workspace_bytes", "qlora_linear_fwd_gated",
           "qlora_linear_fwd_gated_f16", "qlora_linear_gated_workspace_bytes", "qlora_gated_fwd", "qlora_gated_fwd_x8",
           "qlora_gated_bwd", "qlora_gated_bwd_x8", "qlora_int8_linear_fwd_gated", "qlora_linear_bwd_x8",
           "qlora_linear_bwd_x8_f16", "qlora_linear_bwd_grouped_x8", "qlora_linear_bwd_grouped_x8_f16",
           "qlora_linear_x8_workspace_bytes", "qlora_linear_gated_least_workspace_bytes",
           "qlora_linear_x8_least_workspace_bytes")
NOALLOC_SCRATCH_BYTES = 16 << 20  # QLORA_NOALLOC_SCRATCH_BYTES

CODEBOOK_NF4 = 0   # normal-quantile levels
CODEBOOK_INT4 = 1  # 16 evenly spaced levels on [-1, 1]

ACT_SILU = 0  # g / (1 + e^-g)
ACT_GELU = 1  # the tanh form: g / 2 (1 + tanh(sqrt(2 / pi) (g + 0.044715 g^3)))


class QloraError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {STATUS.get(status, status)} ({status_string(status)})")


class NF4WeightC(ctypes.Structure):
    _fields_ = [("n", ctypes.c_int64), ("k", ctypes.c_int64), ("codes", ctypes.c_void_p),
                ("scale_codes", ctypes.c_void_p), ("group_scale", ctypes.c_void_p), ("absmax", ctypes.c_void_p),
                ("double_quant", ctypes.c_int32), ("codebook", ctypes.c_int32)]


_LIB = None


def load():
    """Load the library (once). Raises if it has not been built."""
    global _LIB
    if _LIB is not None:
        return _LIB
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with `python -m bit_nf4_quantized_18_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    vp, i64, i32, f32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
    wp = ctypes.POINTER(NF4WeightC)
    lib.qlora_nf4_quantize.argtypes = [vp, i64, i32, vp, vp, vp, vp, vp]
    lib.qlora_nf4_quantize.restype = i32
    lib.qlora_nf4_dequantize.argtypes = [wp, i32, vp, vp]
    lib.qlora_nf4_dequantize.restype = i32
    lib.qlora_linear_fwd.argtypes = [wp, vp, i64, vp, vp, i32, f32, vp, vp, vp, sz, vp]
    lib.qlora_linear_fwd.restype = i32
    lib.qlora_linear_bwd.argtypes = [wp, vp, vp, i64, vp, vp, i32, f32, vp, vp, vp, vp, vp, sz, vp]
    lib.qlora_linear_bwd.restype = i32
    lib.qlora_linear_fwd_f16.argtypes = lib.qlora_linear_fwd.argtypes
    lib.qlora_linear_fwd_f16.restype = i32
    lib.qlora_linear_bwd_f16.argtypes = lib.qlora_linear_bwd.argtypes
    lib.qlora_linear_bwd_f16.restype = i32
    lib.qlora_linear_fwd_noalloc.argtypes = [wp, vp, i64, vp, vp, i32, f32, vp, vp, vp]
    lib.qlora_linear_fwd_noalloc.restype = i32
    lib.qlora_linear_workspace_bytes.argtypes = [i64, i64, i64, i32]
    lib.qlora_linear_workspace_bytes.restype = sz
    p64 = ctypes.POINTER(ctypes.c_int64)
    lib.qlora_linear_fwd_grouped.argtypes = [wp, i32, p64, vp, i64, vp, vp, i32, f32, vp, vp, vp, sz, vp]
    lib.qlora_linear_fwd_grouped.restype = i32
    lib.qlora_linear_bwd_grouped.argtypes = [wp, i32, p64, vp, vp, i64, vp, vp, i32, f32, vp, vp, vp, vp, vp, sz, vp]
    lib.qlora_linear_bwd_grouped.restype = i32
    lib.qlora_linear_grouped_workspace_bytes.argtypes = [i64, i64, i64, i32, i32]
    lib.qlora_linear_grouped_workspace_bytes.restype = sz
    lib.qlora_status_string.argtypes = [i32]
    lib.qlora_status_string.restype = ctypes.c_char_p
    lib.qlora_nf4_levels.argtypes = [ctypes.POINTER(ctypes.c_float)]
    lib.qlora_nf4_levels.restype = i32
    lib.qlora_quantize_codebook.argtypes = [vp, i64, i32, i32, vp, vp, vp, vp, vp]
    lib.qlora_quantize_codebook.restype = i32
    lib.qlora_codebook_levels.argtypes = [i32, ctypes.POINTER(ctypes.c_float)]
    lib.qlora_codebook_levels.restype = i32
    lib.qlora_merge.argtypes = [wp, vp, vp, i32, f32, i32, vp, vp]
    lib.qlora_merge.restype = i32
    lib.qlora_unmerge.argtypes = [vp, i32, i64, i64, vp, vp, i32, f32, vp, vp]
    lib.qlora_unmerge.restype = i32
    lib.qlora_requantize.argtypes = [wp, vp, vp, i32, f32, i32, i32, vp, vp, vp, vp, vp, vp]
    lib.qlora_requantize.restype = i32
    lib.qlora_linear_dropout_workspace_bytes.argtypes = [i64, i64, i64, i32]
    lib.qlora_linear_dropout_workspace_bytes.restype = sz
    lib.qlora_linear_fwd_dropout.argtypes = [wp, vp, i64, vp, vp, i32, f32, vp, f32, vp, vp, vp, sz, vp]
    lib.qlora_linear_fwd_dropout.restype = i32
    lib.qlora_linear_bwd_dropout.argtypes = [wp, vp, vp, i64, vp, vp, i32, f32, vp, f32, vp, vp, vp, vp, vp, sz, vp]
    lib.qlora_linear_bwd_dropout.restype = i32
    lib.qlora_dropout_mask.argtypes = [ctypes.c_uint64, ctypes.c_uint64, i64, f32, vp, vp]
    lib.qlora_dropout_mask.restype = i32
    lib.qlora_int8_quantize.argtypes = [vp, i32, i64, i64, vp, i64, vp, vp]
    lib.qlora_int8_quantize.restype = i32
    lib.qlora_int8_dequantize.argtypes = [vp, i64, vp, i64, i64, i32, vp, vp]
    lib.qlora_int8_dequantize.restype = i32
    lib.qlora_rmsnorm_int8.argtypes = [vp, vp, vp, i32, i32, i64, i64, f32, vp, vp, i64, vp, vp]
    lib.qlora_rmsnorm_int8.restype = i32
    lib.qlora_int8_linear_fwd.argtypes = [vp, vp, i64, i64, vp, vp, i64, i32, vp, vp]
    lib.qlora_int8_linear_fwd.restype = i32
    lib.qlora_linear_fwd_gated.argtypes = [wp, vp, i64, vp, vp, i32, f32, i32, vp, vp, vp, vp, sz, vp]
    lib.qlora_linear_gated_workspace_bytes.argtypes = [i64, i64, i64, i32]
    lib.qlora_gated_fwd.argtypes = [vp, i32, i64, i64, i32, vp, vp]
    lib.qlora_gated_fwd_x8.argtypes = [vp, i64, vp, i32, i64, i64, i32, vp, vp]
    lib.qlora_gated_bwd.argtypes = [vp, vp, i32, i64, i64, i32, vp, vp]
    lib.qlora_gated_bwd_x8.argtypes = [vp, i64, vp, vp, i32, i64, i64, i32, vp, vp]
    lib.qlora_int8_linear_fwd_gated.argtypes = [vp, vp, i64, i64, vp, vp, i64, i32, i32, vp, vp]
    lib.qlora_linear_bwd_x8.argtypes = [wp, vp, i64, vp, vp, i64, vp, vp, i32, f32, vp, vp, vp, vp, vp, sz, vp]
    lib.qlora_linear_bwd_grouped_x8.argtypes = [wp, i32, p64, vp, i64, vp, vp, i64, vp, vp, i32, f32, vp, vp, vp, vp,
                                                vp, sz, vp]
    lib.qlora_linear_x8_workspace_bytes.argtypes = [i64, i64, i64, i32, i32]
    for name in ("gated", "x8"):
        full, least = (getattr(lib, f"qlora_linear_{name}_{s}workspace_bytes") for s in ("", "least_"))
        least.argtypes = full.argtypes
        full.restype = least.restype = sz
    for name in ("linear_fwd_gated", "linear_bwd_x8", "linear_bwd_grouped_x8"):
        fn, f16 = getattr(lib, f"qlora_{name}"), getattr(lib, f"qlora_{name}_f16")
        f16.argtypes = fn.argtypes
        fn.restype = f16.restype = i32
    for name in ("gated_fwd", "gated_fwd_x8", "gated_bwd", "gated_bwd_x8", "int8_linear_fwd_gated"):
        getattr(lib, f"qlora_{name}").restype = i32
    lib.qlora_grad_workspace_bytes.argtypes = [vp, i32]
    lib.qlora_grad_workspace_bytes.restype = sz
    lib.qlora_grad_norm.argtypes = [vp, vp, i32, i32, vp, vp, sz, vp]
    lib.qlora_grad_norm.restype = i32
    lib.qlora_grad_clip.argtypes = [vp, vp, i32, i32, f32, vp, vp, vp, sz, vp]
    lib.qlora_grad_clip.restype = i32
    # the fp16 compute calls share their bf16 counterparts' signatures
    for name in ("grouped", "dropout"):
        for d in ("fwd", "bwd"):
            f16 = getattr(lib, f"qlora_linear_{d}_{name}_f16")
            f16.argtypes = getattr(lib, f"qlora_linear_{d}_{name}").argtypes
            f16.restype = i32
    _LIB = lib
    return lib


def status_string(status: int) -> str:
    return load().qlora_status_string(status).decode()


def levels(codebook: int = CODEBOOK_NF4):
    """The 16 float32 levels the kernels use for `codebook` (host call)."""
    buf = (ctypes.c_float * 16)()
    if codebook == CODEBOOK_NF4:
        n = load().qlora_nf4_levels(buf)
    else:
        n = load().qlora_codebook_levels(int(codebook), buf)
    if n != 16:
        raise QloraError(n, "qlora_codebook_levels")
    return list(buf)


def workspace_bytes(m: int, n: int, k: int, r: int) -> int:
    return int(load().qlora_linear_workspace_bytes(m, n, k, r))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    import torch

    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _check(status: int, where: str):
    if status != 0:
        raise QloraError(status, where)


def _need(t, name, shape, dtypes, device, optional=False):
    """Raise unless ``t`` is a contiguous tensor of one of ``dtypes`` on
    ``device`` with exactly ``shape`` (None allowed only when ``optional``).
    The library takes raw pointers and sizes, so a tensor that does not match
    what the call assumes is refused here rather than read out of bounds."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, the weight on {device}")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {' or '.join(str(d) for d in dtypes)}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _need_packed(q):
    """The packed weight's buffers: uint8 codes / scale codes, float32 group
    scales / absmax, contiguous, on one device, at least as long as n x k needs."""
    import torch

    dev = q.codes.device
    numel = q.n * q.k
    nb = -(-numel // BLOCK)
    ng = -(-nb // DQ_GROUP)
    for name, t, dt, need in (("codes", q.codes, torch.uint8, (numel + 1) // 2),
                              ("scale_codes", q.scale_codes, torch.uint8, nb if q.double_quant else 0),
                              ("group_scale", q.group_scale, torch.float32, ng if q.double_quant else 0),
                              ("absmax", q.absmax, torch.float32, 0 if q.double_quant else nb)):
        if t is None:
            if need:
                raise ValueError(f"packed weight: {name} is required")
            continue
        if t.device != dev or t.dtype != dt or not t.is_contiguous() or t.numel() < need:
            raise ValueError(f"packed weight: {name} must be a contiguous {dt} tensor on {dev} "
                             f"with at least {need} elements")
    return dev


def _half_types(t, name):
    import torch

    if t.dtype not in (torch.bfloat16, torch.float16):
        raise TypeError(f"{name} must be bfloat16 or float16, got {t.dtype}")
    return (t.dtype,)


def _need_ws(ws, device):
    import torch

    if ws is not None and (ws.device != device or ws.dtype != torch.uint8 or not ws.is_contiguous()):
        raise ValueError("ws must be a contiguous uint8 tensor on the weight's device")


def _need_adapter(a, b, r, k, n, types, device, rb=None):
    if (a is None) != (b is None):
        raise ValueError("a and b are given together or not at all")
    if a is None:
        return
    _need(a, "a", (r, k), types, device)
    _need(b, "b", (n, r if rb is None else rb), types, device)


@dataclasses.dataclass
class PackedNF4:
    """A packed NF4 weight on the device (n x k row-major)."""
    n: int
    k: int
    codes: "object"                 # uint8 [ceil(n*k/2)]
    double_quant: bool
    scale_codes: "object" = None    # uint8 [nblocks]        (double quant)
    group_scale: "object" = None    # float32 [ngroups]      (double quant)
    absmax: "object" = None         # float32 [nblocks]      (exact a_b; required without double quant)
    codebook: int = CODEBOOK_NF4    # level table the codes index

    def c_struct(self) -> NF4WeightC:
        return NF4WeightC(self.n, self.k, self.codes.data_ptr(),
                          None if self.scale_codes is None else self.scale_codes.data_ptr(),
                          None if self.group_scale is None else self.group_scale.data_ptr(),
                          None if self.absmax is None else self.absmax.data_ptr(), int(self.double_quant),
                          int(self.codebook))


def _empty(n, dtype, device):
    import torch

    # 16 extra bytes so even empty-ish buffers get a real, aligned allocation
    return torch.empty(max(n, 1), dtype=dtype, device=device)


def quantize(w, double_quant: bool = True, keep_absmax: bool = False, codebook: int = CODEBOOK_NF4) -> PackedNF4:
    """Quantize a float32 CUDA tensor (any shape; flattened row-major).
    A 2-D tensor gives n, k = its shape; other shapes give n = 1.
    codebook: CODEBOOK_NF4 (qlora_nf4_quantize) or CODEBOOK_INT4."""
    import torch

    if w.dtype != torch.float32 or not w.is_cuda:
        raise TypeError("quantize expects a float32 tensor on the GPU")
    w = w.contiguous()
    numel = w.numel()
    n, k = (w.shape[0], w.shape[1]) if w.dim() == 2 else (1, numel)
    nb = -(-numel // BLOCK)
    ng = -(-nb // DQ_GROUP)
    dev = w.device
    codes = _empty((numel + 1) // 2, torch.uint8, dev)
    sc = _empty(nb, torch.uint8, dev) if double_quant else None
    gs = _empty(ng, torch.float32, dev) if double_quant else None
    am = _empty(nb, torch.float32, dev) if (keep_absmax or not double_quant) else None
    if codebook == CODEBOOK_NF4:
        st = load().qlora_nf4_quantize(_ptr(w), numel, int(double_quant), _ptr(codes), _ptr(sc), _ptr(gs),
                                       _ptr(am), _stream())
        _check(st, "qlora_nf4_quantize")
    else:
        st = load().qlora_quantize_codebook(_ptr(w), numel, int(double_quant), int(codebook), _ptr(codes),
                                            _ptr(sc), _ptr(gs), _ptr(am), _stream())
        _check(st, "qlora_quantize_codebook")
    return PackedNF4(n, k, codes[: (numel + 1) // 2], double_quant, None if sc is None else sc[:nb],
                     None if gs is None else gs[:ng], None if am is None else am[:nb], int(codebook))


def dequantize(q: PackedNF4, dtype=None):
    import torch

    dtype = torch.bfloat16 if dtype is None else dtype
    code = {torch.bfloat16: QLORA_BF16, torch.float32: QLORA_F32, torch.float16: QLORA_F16}[dtype]
    dev = _need_packed(q)
    out = torch.empty((q.n, q.k), dtype=dtype, device=dev)
    ws = q.c_struct()
    _check(load().qlora_nf4_dequantize(ctypes.byref(ws), code, _ptr(out), _stream()), "qlora_nf4_dequantize")
    return out


def _adapter(a, b, n, k, device):
    """(r, a pointer, b pointer) of a bf16 adapter a (r, k), b (n, r), or none."""
    import torch

    r = 0 if a is None else a.shape[0]
    _need_adapter(a, b, r, k, n, (torch.bfloat16,), device)
    return r, _ptr(a), _ptr(b)


def merge(q: PackedNF4, a, b, alpha: float, dtype=None, out=None):
    """W16 + fl32(alpha/r) B A with the float32 order of qlora_merge.
    a: bf16 (r, k), b: bf16 (n, r), or both None. Returns (n, k) of dtype."""
    import torch

    dtype = torch.bfloat16 if dtype is None else dtype
    code = {torch.bfloat16: QLORA_BF16, torch.float32: QLORA_F32}[dtype]
    dev = _need_packed(q)
    out = torch.empty((q.n, q.k), dtype=dtype, device=dev) if out is None else out
    _need(out, "out", (q.n, q.k), (dtype,), dev)
    r, ap, bp = _adapter(a, b, q.n, q.k, dev)
    ws = q.c_struct()
    _check(load().qlora_merge(ctypes.byref(ws), ap, bp, r, float(alpha), code, _ptr(out), _stream()), "qlora_merge")
    return out


def unmerge(merged, a, b, alpha: float, out=None):
    """merged - fl32(alpha/r) B A (qlora_unmerge); merged: bf16 or float32
    (n, k). ``out`` may be ``merged`` (in place)."""
    import torch

    code = {torch.bfloat16: QLORA_BF16, torch.float32: QLORA_F32}[merged.dtype]
    if merged.dim() != 2:
        raise ValueError("merged must be 2-D (n, k)")
    dev = merged.device
    _need(merged, "merged", tuple(merged.shape), (merged.dtype,), dev)
    out = torch.empty_like(merged) if out is None else out
    _need(out, "out", tuple(merged.shape), (merged.dtype,), dev)
    r, ap, bp = _adapter(a, b, merged.shape[0], merged.shape[1], dev)
    _check(load().qlora_unmerge(_ptr(merged), code, merged.shape[0], merged.shape[1], ap, bp, r, float(alpha),
                                _ptr(out), _stream()), "qlora_unmerge")
    return out


def requantize(q: PackedNF4, a, b, alpha: float, double_quant: bool = True, codebook: int = CODEBOOK_NF4,
               keep_absmax: bool = False):
    """The merged weight quantized again (qlora_requantize). Returns
    (PackedNF4 of the merged weight, merged float32 (n, k))."""
    import torch

    dev = _need_packed(q)
    numel = q.n * q.k
    nb = -(-numel // BLOCK)
    ng = -(-nb // DQ_GROUP)
    merged = torch.empty((q.n, q.k), dtype=torch.float32, device=dev)
    codes = _empty((numel + 1) // 2, torch.uint8, dev)
    sc = _empty(nb, torch.uint8, dev) if double_quant else None
    gs = _empty(ng, torch.float32, dev) if double_quant else None
    am = _empty(nb, torch.float32, dev) if (keep_absmax or not double_quant) else None
    r, ap, bp = _adapter(a, b, q.n, q.k, dev)
    ws = q.c_struct()
    _check(load().qlora_requantize(ctypes.byref(ws), ap, bp, r, float(alpha), int(double_quant), int(codebook),
                                   _ptr(merged), _ptr(codes), _ptr(sc), _ptr(gs), _ptr(am), _stream()),
           "qlora_requantize")
    packed = PackedNF4(q.n, q.k, codes[: (numel + 1) // 2], double_quant, None if sc is None else sc[:nb],
                       None if gs is None else gs[:ng], None if am is None else am[:nb], int(codebook))
    return packed, merged


def _workspace(m, n, k, r, device):
    import torch

    nbytes = workspace_bytes(m, n, k, r)
    return (torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None), nbytes


def linear_fwd(q: PackedNF4, x, a=None, b=None, alpha: float = 0.0, want_h: bool = True, out=None, h_out=None,
               ws=None):
    """Y = X W16^T + (alpha/r) (X A^T) B^T. x: bf16 (m, k), or fp16 for the
    fp16 compute entry point (A, B and Y then fp16 too). Returns (y, h).
    ``out``, ``h_out`` and ``ws`` (uint8 workspace) may be preallocated."""
    import torch

    dev = _need_packed(q)
    m = x.shape[0]
    r = 0 if a is None else a.shape[0]
    t16 = _half_types(x, "x")
    f16 = x.dtype == torch.float16  # fp16 compute: the _f16 entry point
    _need(x, "x", (m, q.k), t16, dev)
    _need_adapter(a, b, r, q.k, q.n, t16, dev)
    y = out if out is not None else torch.empty((m, q.n), dtype=x.dtype, device=dev)
    h = h_out if h_out is not None else (
        torch.empty((m, r), dtype=torch.float32, device=dev) if (want_h and r > 0) else None)
    _need(y, "out", (m, q.n), t16, dev)
    _need(h, "h_out", (m, r), (torch.float32,), dev, optional=True)
    _need_ws(ws, dev)
    if ws is None:
        ws, nbytes = _workspace(m, q.n, q.k, r, dev)
    else:
        nbytes = ws.numel()
    wc = q.c_struct()
    fn = load().qlora_linear_fwd_f16 if f16 else load().qlora_linear_fwd
    st = fn(ctypes.byref(wc), _ptr(x), m, _ptr(a), _ptr(b), r, float(alpha), _ptr(y), _ptr(h), _ptr(ws), nbytes,
            _stream())
    _check(st, "qlora_linear_fwd_f16" if f16 else "qlora_linear_fwd")
    return y, h


def linear_fwd_noalloc(q: PackedNF4, x, a=None, b=None, alpha: float = 0.0, out=None, h_out=None):
    """qlora_linear_fwd_noalloc: the bf16 forward on the library's own scratch
    array (no workspace). ``out`` (bf16 (m, n)) and ``h_out`` (float32
    (m, r)) may be preallocated; h is returned only when ``h_out`` is given."""
    import torch

    dev = _need_packed(q)
    m = x.shape[0]
    r = 0 if a is None else a.shape[0]
    _need(x, "x", (m, q.k), (torch.bfloat16,), dev)
    _need_adapter(a, b, r, q.k, q.n, (torch.bfloat16,), dev)
    y = out if out is not None else torch.empty((m, q.n), dtype=x.dtype, device=dev)
    _need(y, "out", (m, q.n), (torch.bfloat16,), dev)
    _need(h_out, "h_out", (m, r), (torch.float32,), dev, optional=True)
    wc = q.c_struct()
    st = load().qlora_linear_fwd_noalloc(ctypes.byref(wc), _ptr(x), m, _ptr(a), _ptr(b), r, float(alpha), _ptr(y),
                                         _ptr(h_out), _stream())
    _check(st, "qlora_linear_fwd_noalloc")
    return y, h_out


def linear_bwd(q: PackedNF4, x, dy, a=None, b=None, alpha: float = 0.0, h=None, need_dx: bool = True,
               dx=None, da=None, db=None, ws=None):
    """Returns (dx (m,k) of dy's 16-bit type or None, dA float32 (r,k), dB
    float32 (n,r)). fp16 inputs take the fp16 entry point. Outputs and the
    workspace may be preallocated. ``x`` may be a PackedInt8 of m rows of k
    values, an input kept in 8 bits (qlora_linear_bwd_x8); ``h`` is then
    required with an adapter."""
    import torch

    if isinstance(x, PackedInt8):
        return _linear_bwd_x8(q, None, x, dy, a, b, alpha, h, need_dx, dx, da, db, ws)
    dev = _need_packed(q)
    m = dy.shape[0]
    r = 0 if a is None else a.shape[0]
    t16 = _half_types(dy, "dy")
    f16 = dy.dtype == torch.float16
    _need(dy, "dy", (m, q.n), t16, dev)
    _need(x, "x", (m, q.k), t16, dev, optional=r == 0)
    _need_adapter(a, b, r, q.k, q.n, t16, dev)
    _need(h, "h", (m, r), (torch.float32,), dev, optional=True)
    if dx is None and need_dx:
        dx = torch.empty((m, q.k), dtype=dy.dtype, device=dev)
    if r and da is None:
        da = torch.empty((r, q.k), dtype=torch.float32, device=dev)
    if r and db is None:
        db = torch.empty((q.n, r), dtype=torch.float32, device=dev)
    _need(dx, "dx", (m, q.k), t16, dev, optional=True)
    _need(da, "da", (r, q.k), (torch.float32,), dev, optional=r == 0)
    _need(db, "db", (q.n, r), (torch.float32,), dev, optional=r == 0)
    _need_ws(ws, dev)
    if ws is None:
        ws, nbytes = _workspace(m, q.n, q.k, r, dev)
    else:
        nbytes = ws.numel()
    wc = q.c_struct()
    fn = load().qlora_linear_bwd_f16 if f16 else load().qlora_linear_bwd
    st = fn(ctypes.byref(wc), _ptr(x), _ptr(dy), m, _ptr(a), _ptr(b), r, float(alpha), _ptr(h), _ptr(dx), _ptr(da),
            _ptr(db), _ptr(ws), nbytes, _stream())
    _check(st, "qlora_linear_bwd_f16" if f16 else "qlora_linear_bwd")
    return dx, da, db


def dropout_workspace_bytes(m: int, n: int, k: int, r: int) -> int:
    return int(load().qlora_linear_dropout_workspace_bytes(m, n, k, r))


def _drop_ws(ws, m, n, k, r, dev):
    import torch

    if ws is not None:
        return ws, ws.numel()
    nbytes = dropout_workspace_bytes(m, n, k, r)
    return (torch.empty(nbytes, dtype=torch.uint8, device=dev) if nbytes else None), nbytes


def dropout_mask(seed: int, offset: int, shape, p: float, out=None):
    """Keep mask (uint8, 1 = kept) drawn on the GPU by qlora_dropout_mask:
    elements offset .. offset + numel - 1 of the stream of `seed`."""
    import torch

    out = torch.empty(shape, dtype=torch.uint8, device="cuda") if out is None else out
    _check(load().qlora_dropout_mask(int(seed), int(offset), out.numel(), float(p), _ptr(out), _stream()),
           "qlora_dropout_mask")
    return out


def linear_fwd_dropout(q: PackedNF4, x, a, b, alpha: float, keep, p: float, want_h: bool = True, out=None,
                       h_out=None, ws=None):
    """qlora_linear_fwd_dropout. keep: uint8 (m, k) on the GPU, non-zero =
    kept; p: drop probability. Returns (y, h) with h from the dropped input."""
    import torch

    dev = _need_packed(q)
    m, r = x.shape[0], a.shape[0]
    t16 = _half_types(x, "x")
    _need(x, "x", (m, q.k), t16, dev)
    _need_adapter(a, b, r, q.k, q.n, t16, dev)
    _need(keep, "keep", (m, q.k), (torch.uint8,), dev)
    y = out if out is not None else torch.empty((m, q.n), dtype=x.dtype, device=dev)
    h = h_out if h_out is not None else (torch.empty((m, r), dtype=torch.float32, device=dev) if want_h else None)
    _need(y, "out", (m, q.n), t16, dev)
    _need(h, "h_out", (m, r), (torch.float32,), dev, optional=True)
    _need_ws(ws, dev)
    ws, nbytes = _drop_ws(ws, m, q.n, q.k, r, dev)
    wc = q.c_struct()
    fn = load().qlora_linear_fwd_dropout_f16 if x.dtype == torch.float16 else load().qlora_linear_fwd_dropout
    st = fn(ctypes.byref(wc), _ptr(x), m, _ptr(a), _ptr(b), r, float(alpha),
            _ptr(keep), float(p), _ptr(y), _ptr(h), _ptr(ws), nbytes, _stream())
    _check(st, "qlora_linear_fwd_dropout")
    return y, h


def linear_bwd_dropout(q: PackedNF4, x, dy, a, b, alpha: float, keep, p: float, h=None, need_dx: bool = True,
                       dx=None, da=None, db=None, ws=None):
    """qlora_linear_bwd_dropout with the forward's mask. Returns (dx, dA, dB)."""
    import torch

    dev = _need_packed(q)
    m, r = dy.shape[0], a.shape[0]
    t16 = _half_types(dy, "dy")
    _need(dy, "dy", (m, q.n), t16, dev)
    _need(x, "x", (m, q.k), t16, dev)
    _need_adapter(a, b, r, q.k, q.n, t16, dev)
    _need(keep, "keep", (m, q.k), (torch.uint8,), dev)
    _need(h, "h", (m, r), (torch.float32,), dev, optional=True)
    if dx is None and need_dx:
        dx = torch.empty((m, q.k), dtype=dy.dtype, device=dev)
    da = torch.empty((r, q.k), dtype=torch.float32, device=dev) if da is None else da
    db = torch.empty((q.n, r), dtype=torch.float32, device=dev) if db is None else db
    _need(dx, "dx", (m, q.k), t16, dev, optional=True)
    _need(da, "da", (r, q.k), (torch.float32,), dev)
    _need(db, "db", (q.n, r), (torch.float32,), dev)
    _need_ws(ws, dev)
    ws, nbytes = _drop_ws(ws, m, q.n, q.k, r, dev)
    wc = q.c_struct()
    fn = load().qlora_linear_bwd_dropout_f16 if dy.dtype == torch.float16 else load().qlora_linear_bwd_dropout
    st = fn(ctypes.byref(wc), _ptr(x), _ptr(dy), m, _ptr(a), _ptr(b), r, float(alpha),
            _ptr(keep), float(p), _ptr(h), _ptr(dx), _ptr(da), _ptr(db), _ptr(ws),
            nbytes, _stream())
    _check(st, "qlora_linear_bwd_dropout")
    return dx, da, db


def grouped_workspace_bytes(m: int, n: int, k: int, g: int, r: int) -> int:
    return int(load().qlora_linear_grouped_workspace_bytes(m, n, k, g, r))


def _parts(parts):
    arr = (ctypes.c_int64 * len(parts))(*[int(p) for p in parts])
    return arr


def linear_fwd_grouped(q: PackedNF4, parts, x, a, b, alpha: float, want_h: bool = True, out=None, h_out=None,
                       ws=None):
    """Grouped forward over a stacked weight (row counts ``parts``): y (m, n)
    with part l's columns = X W_l^T + (alpha/r) (X A_l^T) B_l^T; a is the
    stacked (g r, k) A, b the stacked (n, r) B. Returns (y, h (m, g r))."""
    import torch

    dev = _need_packed(q)
    m, g, r = x.shape[0], len(parts), b.shape[1]
    t16 = _half_types(x, "x")
    _need(x, "x", (m, q.k), t16, dev)
    _need_adapter(a, b, g * r, q.k, q.n, t16, dev, rb=r)
    y = out if out is not None else torch.empty((m, q.n), dtype=x.dtype, device=dev)
    h = h_out if h_out is not None else (torch.empty((m, g * r), dtype=torch.float32, device=dev) if want_h else None)
    _need(y, "out", (m, q.n), t16, dev)
    _need(h, "h_out", (m, g * r), (torch.float32,), dev, optional=True)
    _need_ws(ws, dev)
    if ws is None:
        nbytes = grouped_workspace_bytes(m, q.n, q.k, g, r)
        ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    nbytes = ws.numel()
    wc = q.c_struct()
    pa = _parts(parts)
    fn = load().qlora_linear_fwd_grouped_f16 if x.dtype == torch.float16 else load().qlora_linear_fwd_grouped
    st = fn(ctypes.byref(wc), g, pa, _ptr(x), m, _ptr(a), _ptr(b), r, float(alpha),
            _ptr(y), _ptr(h), _ptr(ws), nbytes, _stream())
    _check(st, "qlora_linear_fwd_grouped")
    return y, h


def linear_bwd_grouped(q: PackedNF4, parts, x, dy, a, b, alpha: float, h=None, need_dx: bool = True, dx=None,
                       da=None, db=None, ws=None):
    """Grouped backward: (dx (m, k) = sum over parts, dA stacked (g r, k),
    dB stacked (n, r)). ``x`` may be a PackedInt8, as in linear_bwd."""
    import torch

    if isinstance(x, PackedInt8):
        return _linear_bwd_x8(q, parts, x, dy, a, b, alpha, h, need_dx, dx, da, db, ws)
    dev = _need_packed(q)
    m, g, r = dy.shape[0], len(parts), b.shape[1]
    t16 = _half_types(dy, "dy")
    _need(dy, "dy", (m, q.n), t16, dev)
    _need(x, "x", (m, q.k), t16, dev)
    _need_adapter(a, b, g * r, q.k, q.n, t16, dev, rb=r)
    _need(h, "h", (m, g * r), (torch.float32,), dev, optional=True)
    if dx is None and need_dx:
        dx = torch.empty((m, q.k), dtype=dy.dtype, device=dev)
    if da is None:
        da = torch.empty((g * r, q.k), dtype=torch.float32, device=dev)
    if db is None:
        db = torch.empty((q.n, r), dtype=torch.float32, device=dev)
    _need(dx, "dx", (m, q.k), t16, dev, optional=True)
    _need(da, "da", (g * r, q.k), (torch.float32,), dev)
    _need(db, "db", (q.n, r), (torch.float32,), dev)
    _need_ws(ws, dev)
    if ws is None:
        nbytes = grouped_workspace_bytes(m, q.n, q.k, g, r)
        ws = torch.empty(max(nbytes, 1), dtype=torch.uint8, device=dev)
    nbytes = ws.numel()
    wc = q.c_struct()
    pa = _parts(parts)
    fn = load().qlora_linear_bwd_grouped_f16 if dy.dtype == torch.float16 else load().qlora_linear_bwd_grouped
    st = fn(ctypes.byref(wc), g, pa, _ptr(x), _ptr(dy), m, _ptr(a), _ptr(b), r,
            float(alpha), _ptr(h), _ptr(dx), _ptr(da), _ptr(db), _ptr(ws), nbytes,
            _stream())
    _check(st, "qlora_linear_bwd_grouped")
    return dx, da, db


# ---------------------------------------------------------------- 8-bit rows
# A merged weight quantized by output channel, activations by token, and their
# product in 8-bit integers. At decode these calls take less time on the GPU
# than their issue on the host, so they look torch and the library up once and
# read each attribute of a tensor once.
_torch = None      # the torch module, after _init()
_DTYPE = None      # torch dtype -> element code of the 16- and 32-bit types
_raw_stream = None  # device index -> the current stream's handle
_device_now = None  # the current device's index
_dtype_of = operator.attrgetter("dtype")


def _init():
    global _torch, _DTYPE, _raw_stream, _device_now
    import torch

    _DTYPE = {torch.bfloat16: QLORA_BF16, torch.float32: QLORA_F32, torch.float16: QLORA_F16}
    # torch's own accessors behind torch.cuda.current_stream() and
    # current_device(), without the stream object these make
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: torch.cuda.current_stream(index).cuda_stream)
    _device_now = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
    load()
    _torch = torch  # last: it tells other threads that all of this is there


def _launch(fn, index, *args):
    """The library's function ``fn`` with args and the current stream of GPU
    ``index``, that GPU being current; raises on a status."""
    if index < 0:
        raise ValueError("expected tensors on the GPU")
    if index == _device_now():
        status = fn(*args, _raw_stream(index))
    else:
        with _torch.cuda.device(index):
            status = fn(*args, _raw_stream(index))
    if status:
        raise QloraError(status, fn.__name__)


@dataclasses.dataclass
class PackedInt8:
    """8-bit rows on the device: n rows of k values, value = code * scale of
    its row. Rows of codes are padded with zeros to a multiple of 64. As every
    buffer of the library both start at a multiple of 16 bytes: a view of some
    rows is taken where its first row's number is a multiple of 4, and needs
    ``scale[i:].clone()`` elsewhere (QLORA_ERR_ALIGN)."""
    n: int
    k: int
    codes: "object"  # int8 [n, ld], ld % 64 == 0, ld >= k, zeros behind the k codes
    scale: "object"  # float32 [n]


def _need_rows(x, name):
    """(dtype code, rows, cols, GPU index) of a contiguous 2-D tensor of a 16-
    or 32-bit type with one column at least (-1: not on a GPU)."""
    if _torch is None:
        _init()
    code = _DTYPE.get(x.dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16, float16 or float32, got {x.dtype}")
    shape = x.shape
    if len(shape) != 2 or shape[1] < 1:
        raise ValueError(f"{name} must be 2-D (rows, cols >= 1), got shape {tuple(shape)}")
    if not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return code, shape[0], shape[1], x.get_device()


def _need_int8(q, name, index):
    """ld of the 8-bit rows ``q``, whose buffers are checked against n and k."""
    if _torch is None:
        _init()
    codes, scale = q.codes, q.scale
    if codes.dtype is not _torch.int8 or scale.dtype is not _torch.float32:
        raise TypeError(f"{name}: codes must be int8 and scale float32")
    shape = codes.shape
    if len(shape) != 2 or shape[0] != q.n or shape[1] % 64 or not 1 <= q.k <= shape[1]:
        raise ValueError(f"{name}: codes must be ({q.n}, ld) with ld a multiple of 64 and at least k = {q.k}, "
                         f"got {tuple(shape)}")
    if scale.shape != (q.n,):
        raise ValueError(f"{name}: scale must have shape ({q.n},), got {tuple(scale.shape)}")
    if codes.get_device() != index or scale.get_device() != index:
        raise ValueError(f"{name}: codes and scale must be on one GPU, the call's")
    if not codes.is_contiguous() or not scale.is_contiguous():
        raise ValueError(f"{name}: codes and scale must be contiguous")
    return shape[1]


def _int8_out(out, n, k, like, index):
    """(PackedInt8 of n rows of k values on ``like``'s device, its ld): new, or ``out`` checked."""
    if out is not None:
        if out.n != n or out.k != k:
            raise ValueError(f"out holds {out.n} rows of {out.k} values, expected {n} of {k}")
        return out, _need_int8(out, "out", index)
    ld = -(-k // 64) * 64
    if ld > INT8_MAX_COLS:
        raise ValueError(f"rows of {k} values are longer than {INT8_MAX_COLS}")
    # sizes as arguments: 0.2 us less than as a tuple
    return PackedInt8(n, k, like.new_empty(n, ld, dtype=_torch.int8), like.new_empty(n, dtype=_torch.float32)), ld


def _out_dtype(dtype):
    """(torch dtype, its code); None is bfloat16."""
    if _torch is None:
        _init()
    if dtype is None:
        dtype = _torch.bfloat16
    code = _DTYPE.get(dtype)
    if code is None:
        raise TypeError(f"dtype must be bfloat16, float16 or float32, got {dtype}")
    return dtype, code


def quantize_int8(x, out=None) -> PackedInt8:
    """8-bit rows of x (rows, cols; bf16, fp16 or float32): a weight by output
    channel or activations by token (qlora_int8_quantize). ``out`` may be a
    PackedInt8 of the same sizes."""
    code, n, k, index = _need_rows(x, "x")
    q, ld = _int8_out(out, n, k, x, index)
    _launch(_LIB.qlora_int8_quantize, index, x.data_ptr(), code, n, k, q.codes.data_ptr(), ld, q.scale.data_ptr())
    return q


def dequantize_int8(q: PackedInt8, dtype=None, out=None):
    """The values of 8-bit rows as (n, k) of ``dtype`` (bf16 by default)."""
    dtype, code = _out_dtype(dtype)
    codes = q.codes
    index = codes.get_device()
    ld = _need_int8(q, "q", index)
    if out is None:
        out = codes.new_empty(q.n, q.k, dtype=dtype)
    else:
        _need(out, "out", (q.n, q.k), (dtype,), codes.device)
    _launch(_LIB.qlora_int8_dequantize, index, codes.data_ptr(), ld, q.scale.data_ptr(), q.n, q.k, code, out.data_ptr())
    return out


def rmsnorm_int8(x, gain, eps: float = 1e-6, residual=None, residual_out=None, out=None):
    """Root-mean-square norm of h = x + residual into 8-bit rows
    (qlora_rmsnorm_int8). x: (rows, cols) bf16, fp16 or float32; residual: the
    same, or None; gain: (cols,) of x's type or float32. Returns (PackedInt8,
    h in x's type, or None without a residual). ``residual_out`` may be
    preallocated, or be ``residual`` or ``x`` itself (in place); ``out`` may be
    a PackedInt8 of x's sizes. Outputs that overlap the inputs or each other in
    any other way are refused."""
    code, n, k, index = _need_rows(x, "x")
    dtype = x.dtype
    gain_code = code if gain.dtype is dtype else QLORA_F32
    if gain_code != code and gain.dtype is not _torch.float32:
        raise TypeError(f"gain has dtype {gain.dtype}, expected {dtype} or torch.float32")
    if gain.shape != (k,) or gain.get_device() != index or not gain.is_contiguous():
        raise ValueError(f"gain must be a contiguous ({k},) tensor on x's device")
    rp = op = None
    if residual is None:
        if residual_out is not None:
            raise ValueError("residual_out is given without a residual")
    else:
        _need_like(residual, "residual", x, index)
        if residual_out is None:
            residual_out = _torch.empty_like(x)
        else:
            _need_like(residual_out, "residual_out", x, index)
        rp, op = residual.data_ptr(), residual_out.data_ptr()
    q, ld = _int8_out(out, n, k, x, index)
    _launch(_LIB.qlora_rmsnorm_int8, index, x.data_ptr(), rp, gain.data_ptr(), code, gain_code, n, k, float(eps), op,
            q.codes.data_ptr(), ld, q.scale.data_ptr())
    return q, residual_out


def _need_like(t, name, x, index):
    if t.dtype is not x.dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {x.dtype}")
    if t.shape != x.shape or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous, of shape {tuple(x.shape)} on x's device")


def _overlap(s, t):
    """Two contiguous tensors share memory."""
    a, b = s.data_ptr(), t.data_ptr()
    return max(a, b) < min(a + s.nbytes, b + t.nbytes)


def int8_linear_fwd(q: PackedInt8, x: PackedInt8, dtype=None, out=None):
    """Y = X W^T of 8-bit rows: q the weight by channel (n, k), x the input by
    token (m, k). Returns (m, n) of ``dtype`` (bf16, fp16 or float32; bf16 by
    default). ``out`` may be preallocated; over the operands it is refused."""
    dtype, code = _out_dtype(dtype)
    codes = q.codes
    index = codes.get_device()
    ld = _need_int8(q, "q", index)
    if x.k != q.k:
        raise ValueError(f"x holds rows of {x.k} values, the weight rows of {q.k}")
    if _need_int8(x, "x", index) != ld:
        raise ValueError("the rows of x and of the weight must be padded to the same length")
    m, n = x.n, q.n
    if out is None:
        out = codes.new_empty(m, n, dtype=dtype)
    else:
        _need(out, "out", (m, n), (dtype,), codes.device)
        for name, t in (("the weight's codes", codes), ("the weight's scale", q.scale), ("x's codes", x.codes),
                        ("x's scale", x.scale)):
            if _overlap(out, t):
                raise ValueError(f"out overlaps {name}")
    _launch(_LIB.qlora_int8_linear_fwd, index, codes.data_ptr(), q.scale.data_ptr(), n, ld, x.codes.data_ptr(),
            x.scale.data_ptr(), m, code, out.data_ptr())
    return out


def x8_workspace_bytes(m: int, n: int, k: int, g: int, r: int, restored: bool = True) -> int:
    """For linear_bwd (g = 1) and linear_bwd_grouped from 8-bit rows. ``restored``: with the
    weight restored to 16 bits where the call uses it, 2 n k bytes; without it a call takes
    longer, but for one that needs no dX."""
    lib = load()
    fn = lib.qlora_linear_x8_workspace_bytes if restored else lib.qlora_linear_x8_least_workspace_bytes
    return int(fn(m, n, k, g, r))


def _linear_bwd_x8(q, parts, x, dy, a, b, alpha, h, need_dx, dx, da, db, ws):
    """linear_bwd (``parts`` None) and linear_bwd_grouped with x as 8-bit rows."""
    if _torch is None:
        _init()
    dev = _need_packed(q)
    index = q.codes.get_device()
    m, n, k = dy.shape[0], q.n, q.k
    g = 1 if parts is None else len(parts)
    r = 0 if b is None else b.shape[-1]
    t16 = _half_types(dy, "dy")
    _need(dy, "dy", (m, n), t16, dev)
    ld = _need_int8(x, "x", index)
    if x.n != m or x.k != k:
        raise ValueError(f"x holds {x.n} rows of {x.k} values, expected {m} of {k}")
    _need_adapter(a, b, g * r, k, n, t16, dev, rb=r)
    if r:
        f32 = (_torch.float32,)
        _need(h, "h", (m, g * r), f32, dev)
        if da is None:
            da = dy.new_empty(g * r, k, dtype=_torch.float32)
        else:
            _need(da, "da", (g * r, k), f32, dev)
        if db is None:
            db = dy.new_empty(n, r, dtype=_torch.float32)
        else:
            _need(db, "db", (n, r), f32, dev)
    else:
        h = da = db = None
    if dx is not None:
        _need(dx, "dx", (m, k), t16, dev)
    elif need_dx:
        dx = dy.new_empty(m, k)
    if ws is None:
        nbytes = x8_workspace_bytes(m, n, k, g, r, restored=dx is not None)
        ws = dy.new_empty(nbytes, dtype=_torch.uint8) if nbytes else None
    else:
        _need_ws(ws, dev)
        nbytes = ws.numel()
    f16 = dy.dtype is _torch.float16
    if parts is None:
        fn, lead = _LIB.qlora_linear_bwd_x8_f16 if f16 else _LIB.qlora_linear_bwd_x8, ()
    else:
        fn, lead = _LIB.qlora_linear_bwd_grouped_x8_f16 if f16 else _LIB.qlora_linear_bwd_grouped_x8, (g, _parts(parts))
    at = [None if t is None else t.data_ptr() for t in (a, b, h, dx, da, db, ws)]
    wc = q.c_struct()
    _launch(fn, index, ctypes.byref(wc), *lead, x.codes.data_ptr(), ld, x.scale.data_ptr(), dy.data_ptr(), m, at[0], at[1],
            r, float(alpha), *at[2:], nbytes)
    return dx, da, db


# ---------------------------------------------------------------- gated block
def gated_workspace_bytes(m: int, n: int, k: int, r: int, restored: bool = True) -> int:
    """For linear_fwd_gated over a stacked weight of n rows (gate's and up's). ``restored``:
    with the weight restored to 16 bits where the call uses it, 2 n k bytes; without it the
    call takes longer."""
    lib = load()
    fn = lib.qlora_linear_gated_workspace_bytes if restored else lib.qlora_linear_gated_least_workspace_bytes
    return int(fn(m, n, k, r))


def linear_fwd_gated(q: PackedNF4, x, a=None, b=None, alpha: float = 0.0, act: int = ACT_SILU, want_y: bool = True,
                     want_h: bool = True, out=None, y_out=None, h_out=None, ws=None):
    """The gated feed-forward block (qlora_linear_fwd_gated): P = act(G) U with
    [G | U] = X W16^T + (alpha/r) (X A_l^T) B_l^T over a weight that holds gate's
    rows above up's (q.n a multiple of 512). x: bf16 or fp16 (m, k); a: the stacked
    (2 r, k) A, b: the stacked (q.n, r) B, or both None. Returns (p (m, q.n / 2),
    y (m, q.n) = [G | U] in x's type or None, h (m, 2 r) float32 or None).
    gated_bwd and linear_bwd_grouped are its backward."""
    if _torch is None:
        _init()
    dev = _need_packed(q)
    index = q.codes.get_device()
    m = x.shape[0]
    r = 0 if b is None else b.shape[-1]
    t16 = _half_types(x, "x")
    _need(x, "x", (m, q.k), t16, dev)
    _need_adapter(a, b, 2 * r, q.k, q.n, t16, dev, rb=r)
    p = out if out is not None else x.new_empty(m, q.n // 2)
    y = y_out if y_out is not None else (x.new_empty(m, q.n) if want_y else None)
    h = h_out if h_out is not None else (x.new_empty(m, 2 * r, dtype=_torch.float32) if want_h and r else None)
    _need(p, "out", (m, q.n // 2), t16, dev)
    _need(y, "y_out", (m, q.n), t16, dev, optional=True)
    _need(h, "h_out", (m, 2 * r), (_torch.float32,), dev, optional=True)
    _need_ws(ws, dev)
    if ws is None:
        nbytes = gated_workspace_bytes(m, q.n, q.k, r)
        ws = x.new_empty(nbytes, dtype=_torch.uint8) if nbytes else None
    else:
        nbytes = ws.numel()
    wc = q.c_struct()
    fn = _LIB.qlora_linear_fwd_gated_f16 if x.dtype is _torch.float16 else _LIB.qlora_linear_fwd_gated
    _launch(fn, index, ctypes.byref(wc), x.data_ptr(), m, _ptr(a), _ptr(b), r, float(alpha), int(act), _ptr(y),
            p.data_ptr(), _ptr(h), _ptr(ws), nbytes)
    return p, y, h


def _gated_input(y):
    """(type code or None, tokens, n, GPU index, leading arguments) of gate and up's
    pre-activations: (m, 2 n), or a PackedInt8 of 2 m rows of n values."""
    if isinstance(y, PackedInt8):
        index = y.codes.get_device()
        ld = _need_int8(y, "y", index)
        if y.n % 2:
            raise ValueError(f"y holds {y.n} rows, expected two a token: gate's and up's")
        return None, y.n // 2, y.k, index, (y.codes.data_ptr(), ld, y.scale.data_ptr())
    code, m, two_n, index = _need_rows(y, "y")
    if two_n % 2:
        raise ValueError(f"y has {two_n} columns, expected gate's and as many of up's")
    return code, m, two_n // 2, index, (y.data_ptr(),)


def gated_fwd(y, act: int = ACT_SILU, dtype=None, out=None):
    """P = act(G) U (m, n) of the pre-activations [G | U] (qlora_gated_fwd). y: (m,
    2 n) bf16, fp16 or float32, or a PackedInt8 of 2 m rows of n values, which
    ``quantize_int8(y.view(2 * m, n))`` gives. ``dtype``: y's type, and for a
    PackedInt8 the result's (bf16 by default). ``out`` may be preallocated."""
    code, m, n, index, args = _gated_input(y)
    rows = code is None
    if rows:
        dtype, code = _out_dtype(dtype)
    elif dtype is not None and dtype is not y.dtype:
        raise TypeError(f"dtype is {dtype}, y's {y.dtype}: they must agree")
    like = y.codes if rows else y
    dtype = dtype if rows else y.dtype
    if out is None:
        out = like.new_empty(m, n, dtype=dtype)
    else:
        _need(out, "out", (m, n), (dtype,), like.device)
    _launch(_LIB.qlora_gated_fwd_x8 if rows else _LIB.qlora_gated_fwd, index, *args, code, m, n, int(act), out.data_ptr())
    return out


def gated_bwd(y, dp, act: int = ACT_SILU, out=None):
    """d[G | U] (m, 2 n) of P = act(G) U for dP = dp (m, n) (qlora_gated_bwd). y: (m,
    2 n) of dp's type or a PackedInt8 of 2 m rows of n values, as in gated_fwd.
    ``out`` may be preallocated, or be y itself (in place)."""
    code, m, n, index, args = _gated_input(y)
    dcode = _need_rows(dp, "dp")[0]
    if dp.shape != (m, n) or dp.get_device() != index:
        raise ValueError(f"dp must have shape {(m, n)} on y's device, got {tuple(dp.shape)} on {dp.device}")
    if code is not None and code != dcode:
        raise TypeError(f"dp has dtype {dp.dtype}, expected {y.dtype}")
    if out is None:
        out = dp.new_empty(m, 2 * n)
    else:
        _need(out, "out", (m, 2 * n), (dp.dtype,), dp.device)
    _launch(_LIB.qlora_gated_bwd_x8 if code is None else _LIB.qlora_gated_bwd, index, *args, dp.data_ptr(), dcode, m, n,
            int(act), out.data_ptr())
    return out


def int8_linear_fwd_gated(q: PackedInt8, x: PackedInt8, act: int = ACT_SILU, dtype=None, out=None):
    """The gated feed-forward block in 8 bits (qlora_int8_linear_fwd_gated): P =
    act(G) U with [G | U] = X W^T, q holding gate's rows above up's (2 n, k), x the
    input by token (m, k). Returns (m, n) of ``dtype`` (bf16, fp16 or float32; bf16
    by default). ``out`` may be preallocated; over the operands it is refused."""
    dtype, code = _out_dtype(dtype)
    codes = q.codes
    index = codes.get_device()
    ld = _need_int8(q, "q", index)
    if q.n % 2:
        raise ValueError(f"q holds {q.n} rows, expected gate's and as many of up's")
    if x.k != q.k:
        raise ValueError(f"x holds rows of {x.k} values, the weight rows of {q.k}")
    if _need_int8(x, "x", index) != ld:
        raise ValueError("the rows of x and of the weight must be padded to the same length")
    m, n = x.n, q.n // 2
    if out is None:
        out = codes.new_empty(m, n, dtype=dtype)
    else:
        _need(out, "out", (m, n), (dtype,), codes.device)
    _launch(_LIB.qlora_int8_linear_fwd_gated, index, codes.data_ptr(), q.scale.data_ptr(), n, ld, x.codes.data_ptr(),
            x.scale.data_ptr(), m, int(act), code, out.data_ptr())
    return out


# ---------------------------------------------------------------- gradients
class GradList:
    """Gradients (contiguous tensors of one type on one GPU) for grad_norm and
    grad_clip calls of every step on the same buffers. Each call reads the
    tensors' addresses again and refuses those whose type, device, length or
    contiguity is no longer the list's."""

    def __init__(self, grads):
        if _torch is None:
            _init()
        grads = tuple(grads)
        self.dtype = grads[0].dtype if grads else None
        self.code = _DTYPE.get(self.dtype) if grads else QLORA_F32
        self.index = grads[0].get_device() if grads else None
        if self.code is None:
            raise TypeError(f"gradients must be bfloat16, float16 or float32, got {self.dtype}")
        self.grads = grads
        self._check()
        self.sizes = list(map(_torch.Tensor.numel, grads))
        self.total = sum(self.sizes)
        self._numel = (ctypes.c_int64 * max(len(grads), 1))(*self.sizes)
        self.ws_bytes = int(_LIB.qlora_grad_workspace_bytes(self._numel, len(grads)))
        if self.total and not self.ws_bytes:
            raise ValueError("too many gradients or elements for one call")

    def _check(self):
        """Raise unless every tensor is as the kernels will read it: a tensor's
        ``data`` may have been replaced since the last call."""
        tensor, grads = _torch.Tensor, self.grads
        if (set(map(_dtype_of, grads)) <= {self.dtype} and set(map(tensor.get_device, grads)) <= {self.index}
                and all(map(tensor.is_contiguous, grads))):
            return
        for i, g in enumerate(grads):
            if g.dtype is not self.dtype:
                raise TypeError(f"gradient {i} has dtype {g.dtype}, the list {self.dtype}")
            if g.get_device() != self.index:
                raise ValueError(f"gradient {i} is on {g.device}, the list on GPU {self.index}")
            if not g.is_contiguous():
                raise ValueError(f"gradient {i} must be contiguous")

    def _pointers(self):
        """The addresses as they are now, in an array of 64-bit numbers."""
        return array.array("Q", map(_torch.Tensor.data_ptr, self.grads))


def _grad_list(grads):
    """The GradList of a call, as its tensors are now."""
    if not isinstance(grads, GradList):
        return GradList(grads)
    grads._check()
    if list(map(_torch.Tensor.numel, grads.grads)) != grads.sizes:
        raise ValueError("a gradient changed its length since the list was made")
    return grads


def _grad_buffers(g, index, norm, ws):
    if norm is None:
        norm = _torch.empty((), dtype=_torch.float32, device=f"cuda:{index}") if not g.grads else \
            g.grads[0].new_empty((), dtype=_torch.float32)
    elif norm.dtype is not _torch.float32 or norm.numel() != 1 or norm.get_device() != index:
        raise ValueError("norm must be one float32 on the gradients' device")
    if ws is None:
        ws = norm.new_empty(g.ws_bytes, dtype=_torch.uint8)
    else:
        _need_ws(ws, norm.device)
    return norm, ws


def grad_norm(grads, norm=None, ws=None):
    """The norm of all elements of ``grads`` (a list of tensors, or a GradList)
    as one float32 on the GPU (qlora_grad_norm). ``norm`` and ``ws`` (uint8,
    GradList.ws_bytes) may be preallocated."""
    g = _grad_list(grads)
    index = g.index if g.grads else _device_now()
    norm, ws = _grad_buffers(g, index, norm, ws)
    at = g._pointers()
    _launch(_LIB.qlora_grad_norm, index, at.buffer_info()[0], g._numel, len(at), g.code, norm.data_ptr(),
            ws.data_ptr(), ws.numel())
    return norm


def grad_clip(grads, max_norm: float, out=None, norm=None, ws=None):
    """Scale ``grads`` (a list of tensors, or a GradList) by min(1, max_norm /
    (norm + 1e-6)), in place, or packed one behind the other into ``out`` (1-D,
    their type and total length). An infinite max_norm scales nothing, NaN and
    infinite norms included. Returns the norm before clipping as one float32 on
    the GPU (qlora_grad_clip)."""
    g = _grad_list(grads)
    index = g.index if g.grads else _device_now()
    op = None
    if out is not None and g.grads:
        _need(out, "out", (g.total,), (g.dtype,), g.grads[0].device)
        op = out.data_ptr() if g.total else None
    norm, ws = _grad_buffers(g, index, norm, ws)
    at = g._pointers()
    _launch(_LIB.qlora_grad_clip, index, at.buffer_info()[0], g._numel, len(at), g.code, float(max_norm), op,
            norm.data_ptr(), ws.data_ptr(), ws.numel())
    return norm


# ---------------------------------------------------------------- storage
# A packed weight on disk: one .npz of plain arrays (no pickled objects), the
# buffers byte for byte as the kernels read them plus n, k, the scale-code kind
# and the codebook id.
def save_packed(path, q: PackedNF4):
    """Write ``q``'s buffers (copied to the host) and sizes to ``path`` (.npz)."""
    import numpy as np

    _need_packed(q)
    arrays = {"n": np.int64(q.n), "k": np.int64(q.k), "double_quant": np.int32(int(q.double_quant)),
              "codebook": np.int32(int(q.codebook)), "codes": q.codes.cpu().numpy()}
    for name in ("scale_codes", "group_scale", "absmax"):
        t = getattr(q, name)
        if t is not None:
            arrays[name] = t.cpu().numpy()
    np.savez(path, **arrays)


def load_packed(path, device="cuda") -> PackedNF4:
    """Read a packed weight written by ``save_packed`` onto ``device``; the
    buffer lengths are checked against n and k."""
    import numpy as np
    import torch

    with np.load(path, allow_pickle=False) as f:
        n, k = int(f["n"]), int(f["k"])
        dq, cb = int(f["double_quant"]), int(f["codebook"])
        get = (lambda name, dt: torch.from_numpy(np.ascontiguousarray(f[name], dtype=dt)).to(device)
               if name in f.files else None)
        q = PackedNF4(n, k, get("codes", np.uint8), dq, get("scale_codes", np.uint8),
                      get("group_scale", np.float32), get("absmax", np.float32), cb)
    _need_packed(q)
    return q
