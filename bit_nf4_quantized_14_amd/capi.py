"""Thin Python binding of the C ABI in ``include/qlora_nf4.h``.

Functions carry the same names as the C entry points and only marshal
arguments: torch supplies device memory and the current HIP stream, every
step of the computation runs in the library's HIP kernels.  There is no CPU
or PyTorch fallback: if ``libqlora_nf4.so`` is missing or a call fails, an
exception is raised.
"""

from __future__ import annotations

import ctypes
import os
from dataclasses import dataclass

import numpy as np

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libqlora_nf4.so")
# the same library built with QN_PROFILE_HOOK (qn_profile_kernel active)
PROF_LIB_PATH = os.path.join(_PKG, "libqlora_nf4_prof.so")
_use_prof = False

QN_OK, QN_EINVAL, QN_EWORKSPACE, QN_EHIP, QN_ENONFINITE = 0, -1, -2, -3, -4
QN_ESYNC = -5
QN_F32, QN_BF16 = 0, 1
QN_FWD, QN_BWD, QN_FWD_DROPOUT = 0, 1, 2
QN_BLOCK, QN_GROUP, QN_MAX_RANK = 64, 256, 256

# Every symbol the header declares (tests check the library exports them).
EXPORTS = ("nf4_codebook", "nf4_quantize", "nf4_dequantize",
           "nf4_dequantize_batch", "nf4_merge",
           "qn_codebook", "qn_quantize", "qn_dequantize",
           "qn_adamw8_step", "qn_adamw8_staging_bytes", "qn_adamw8_paged_step",
           "qlora_linear_fwd_dropout", "qlora_linear_bwd_dropout",
           "qlora_workspace_bytes", "qlora_linear_fwd", "qlora_linear_bwd",
           "qn_strerror", "qn_profile_kernel", "qlora_linear_fwd_noalloc",
           "qlora_fwd_batch_workspace_bytes", "qlora_linear_fwd_batch",
           "qn_act8_encode", "qn_act8_decode", "qlora_linear_bwd_act8",
           "qlora_bwd_act8_workspace_bytes",
           "qn_seq_workspace_bytes", "qn_seq_logprob", "qn_seq_logprob_bwd",
           "qn_pref_loss_fwd", "qn_pref_loss_bwd")
QN_FWD_BATCH_MAX = 8
QN_DEQUANT_BATCH_MAX = 16
QN_CODE_NF4, QN_CODE_FP4, QN_CODE_INT4 = 0, 1, 2
QN_CONST_DQ8, QN_CONST_FP32, QN_CONST_CENTERED = 0, 1, 2
QN_ADAMW_BLOCK = 256
QN_NOALLOC_SCRATCH_BYTES = 32 << 20


class _NF4Struct(ctypes.Structure):
    _fields_ = [("packed", ctypes.c_void_p), ("qabs", ctypes.c_void_p),
                ("gscale", ctypes.c_void_p), ("rows", ctypes.c_int64),
                ("cols", ctypes.c_int64)]


class _QStruct(ctypes.Structure):
    _fields_ = [("packed", ctypes.c_void_p), ("consts", ctypes.c_void_p),
                ("gscale", ctypes.c_void_p), ("gmean", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("code", ctypes.c_int32), ("consts_mode", ctypes.c_int32)]


class _AdamHP(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double),
                ("beta2", ctypes.c_double), ("eps", ctypes.c_double),
                ("weight_decay", ctypes.c_double),
                ("grad_scale", ctypes.c_double)]


class _Adam8State(ctypes.Structure):
    _fields_ = [("m_codes", ctypes.c_void_p), ("m_scale", ctypes.c_void_p),
                ("r_codes", ctypes.c_void_p), ("r_scale", ctypes.c_void_p)]


class _FwdJob(ctypes.Structure):
    _fields_ = [("x", ctypes.c_void_p), ("M", ctypes.c_int64),
                ("w", ctypes.POINTER(_NF4Struct)), ("A", ctypes.c_void_p),
                ("B", ctypes.c_void_p), ("r", ctypes.c_int32),
                ("alpha", ctypes.c_float), ("y", ctypes.c_void_p),
                ("y_dtype", ctypes.c_int32), ("t_save", ctypes.c_void_p)]


class _Dropout(ctypes.Structure):
    _fields_ = [("p", ctypes.c_double), ("seed", ctypes.c_uint64)]


class _Act8Struct(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scale", ctypes.c_void_p),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


class _SeqBatch(ctypes.Structure):
    _fields_ = [("logits", ctypes.c_void_p), ("dtype", ctypes.c_int32),
                ("rows", ctypes.c_int64), ("vocab", ctypes.c_int64),
                ("ld", ctypes.c_int64), ("labels", ctypes.c_void_p),
                ("offsets", ctypes.c_void_p), ("nseq", ctypes.c_int64),
                ("lse_lo", ctypes.c_void_p)]


class _PrefHP(ctypes.Structure):
    _fields_ = [("beta", ctypes.c_double), ("label_smoothing", ctypes.c_double)]


_lib = None


def use_profiling_build() -> None:
    """Load the profiling variant (libqlora_nf4_prof.so, whose
    qn_profile_kernel records per-launch HIP events) instead of the default
    library.  Must be called before the first call into the library."""
    global _use_prof
    if _lib is not None and not _use_prof:
        raise RuntimeError("the default library is already loaded")
    _use_prof = True


def lib_path() -> str:
    return PROF_LIB_PATH if _use_prof else LIB_PATH


def lib() -> ctypes.CDLL:
    """Load the HIP library once; raise if it has not been built.

    torch is imported first: PyTorch ships its own HIP runtime, and the
    library's dependency on the HIP runtime must resolve to that one (which
    owns the streams and memory the calls receive).  Loaded before torch,
    the library would bind the system runtime, and its launches on torch's
    streams would fail."""
    global _lib
    if _lib is not None:
        return _lib
    path = lib_path()
    if not os.path.exists(path):
        raise RuntimeError(
            f"{path} is not built; run `python -m "
            "bit_nf4_quantized_14_amd.build` (hipcc, gfx950)")
    import torch  # noqa: F401  (binds torch's HIP runtime first)
    L = ctypes.CDLL(path)
    vp, i64, i32, f32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float
    sp = ctypes.POINTER(_NF4Struct)
    L.nf4_codebook.argtypes = [vp, vp]
    L.nf4_codebook.restype = ctypes.c_int
    L.nf4_quantize.argtypes = [vp, sp, vp, vp]
    L.nf4_quantize.restype = ctypes.c_int
    L.nf4_dequantize.argtypes = [sp, vp, vp]
    L.nf4_dequantize.restype = ctypes.c_int
    L.nf4_dequantize_batch.argtypes = [sp, ctypes.POINTER(vp), i32, vp]
    L.nf4_dequantize_batch.restype = ctypes.c_int
    L.nf4_merge.argtypes = [sp, vp, vp, i32, f32, vp, vp]
    L.nf4_merge.restype = ctypes.c_int
    qp = ctypes.POINTER(_QStruct)
    L.qn_codebook.argtypes = [i32, vp, vp]
    L.qn_codebook.restype = ctypes.c_int
    L.qn_quantize.argtypes = [vp, qp, vp, vp]
    L.qn_quantize.restype = ctypes.c_int
    L.qn_dequantize.argtypes = [qp, vp, vp]
    L.qn_dequantize.restype = ctypes.c_int
    hpp, stp = ctypes.POINTER(_AdamHP), ctypes.POINTER(_Adam8State)
    L.qn_adamw8_step.argtypes = [vp, vp, i64, stp, hpp, i64, vp]
    L.qn_adamw8_step.restype = ctypes.c_int
    L.qn_adamw8_staging_bytes.argtypes = [i64]
    L.qn_adamw8_staging_bytes.restype = ctypes.c_size_t
    L.qn_adamw8_paged_step.argtypes = [vp, vp, i64, stp, vp, ctypes.c_size_t,
                                       i64, hpp, i64, vp, vp, vp]
    L.qn_adamw8_paged_step.restype = ctypes.c_int
    L.qlora_workspace_bytes.argtypes = [i64, i64, i64, i32, i32]
    L.qlora_workspace_bytes.restype = ctypes.c_size_t
    L.qlora_linear_fwd.argtypes = [vp, i64, sp, vp, vp, i32, f32, vp, i32, vp,
                                   vp, ctypes.c_size_t, vp]
    L.qlora_linear_fwd.restype = ctypes.c_int
    L.qlora_linear_bwd.argtypes = [vp, vp, i64, sp, vp, vp, i32, f32, vp, vp,
                                   i32, vp, vp, vp, ctypes.c_size_t, vp]
    L.qlora_linear_bwd.restype = ctypes.c_int
    dp = ctypes.POINTER(_Dropout)
    L.qlora_linear_fwd_dropout.argtypes = [vp, i64, sp, vp, vp, i32, f32, vp,
                                           i32, vp, dp, vp, ctypes.c_size_t, vp]
    L.qlora_linear_fwd_dropout.restype = ctypes.c_int
    L.qlora_linear_bwd_dropout.argtypes = [vp, vp, i64, sp, vp, vp, i32, f32,
                                           vp, vp, i32, vp, vp, dp, vp,
                                           ctypes.c_size_t, vp]
    L.qlora_linear_bwd_dropout.restype = ctypes.c_int
    jp = ctypes.POINTER(_FwdJob)
    L.qlora_fwd_batch_workspace_bytes.argtypes = [jp, i32]
    L.qlora_fwd_batch_workspace_bytes.restype = ctypes.c_size_t
    L.qlora_linear_fwd_batch.argtypes = [jp, i32, vp, ctypes.c_size_t, vp]
    L.qlora_linear_fwd_batch.restype = ctypes.c_int
    L.qlora_linear_fwd_noalloc.argtypes = [vp, i64, sp, vp, vp, i32, f32, vp,
                                           i32, vp, vp]
    L.qlora_linear_fwd_noalloc.restype = ctypes.c_int
    ap = ctypes.POINTER(_Act8Struct)
    L.qn_act8_encode.argtypes = [vp, i32, ap, vp]
    L.qn_act8_encode.restype = ctypes.c_int
    L.qn_act8_decode.argtypes = [ap, vp, i32, vp]
    L.qn_act8_decode.restype = ctypes.c_int
    L.qlora_bwd_act8_workspace_bytes.argtypes = [i64, i64, i64, i32]
    L.qlora_bwd_act8_workspace_bytes.restype = ctypes.c_size_t
    L.qlora_linear_bwd_act8.argtypes = [vp, ap, i64, sp, vp, vp, i32, f32, vp,
                                        vp, i32, vp, vp, dp, vp,
                                        ctypes.c_size_t, vp]
    L.qlora_linear_bwd_act8.restype = ctypes.c_int
    bp, pp = ctypes.POINTER(_SeqBatch), ctypes.POINTER(_PrefHP)
    L.qn_seq_workspace_bytes.argtypes = [i64, i64, i64]
    L.qn_seq_workspace_bytes.restype = ctypes.c_size_t
    L.qn_seq_logprob.argtypes = [bp, vp, vp, vp, vp, ctypes.c_size_t, vp]
    L.qn_seq_logprob.restype = ctypes.c_int
    L.qn_seq_logprob_bwd.argtypes = [bp, vp, vp, vp, i32, i64, i64, vp]
    L.qn_seq_logprob_bwd.restype = ctypes.c_int
    L.qn_pref_loss_fwd.argtypes = [bp, vp, pp, vp, vp, vp, vp, vp, vp,
                                   ctypes.c_size_t, vp]
    L.qn_pref_loss_fwd.restype = ctypes.c_int
    L.qn_pref_loss_bwd.argtypes = [bp, vp, vp, vp, vp, i32, i64, i64, vp]
    L.qn_pref_loss_bwd.restype = ctypes.c_int
    L.qn_profile_kernel.argtypes = [ctypes.c_char_p, vp, vp, i32]
    L.qn_profile_kernel.restype = ctypes.c_int
    L.qn_strerror.argtypes = [ctypes.c_int]
    L.qn_strerror.restype = ctypes.c_char_p
    _lib = L
    return L


def qn_strerror(code: int) -> str:
    return lib().qn_strerror(int(code)).decode()


class QNError(RuntimeError):
    def __init__(self, fn: str, code: int, detail: str = ""):
        super().__init__(f"{fn}: {qn_strerror(code)} ({code})" +
                         (f": {detail}" if detail else ""))
        self.code = code


def _check(fn: str, code: int) -> None:
    if code != QN_OK:
        raise QNError(fn, code)


def _ptr(t) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(stream) -> int | None:
    import torch
    if stream is None:
        return torch.cuda.current_stream().cuda_stream
    return getattr(stream, "cuda_stream", stream)


@dataclass
class NF4Tensor:
    """Device buffers of an NF4 + double-quantized weight (see nf4_tensor in
    the header): packed codes, 8-bit block codes, fp32 group scales."""
    packed: "object"
    qabs: "object"
    gscale: "object"
    rows: int
    cols: int

    @property
    def numel(self) -> int:
        return self.rows * self.cols

    @staticmethod
    def sizes(rows: int, cols: int):
        numel = rows * cols
        nb = -(-numel // QN_BLOCK)
        return (numel + 1) // 2, nb, -(-nb // QN_GROUP)

    @classmethod
    def empty(cls, rows: int, cols: int, device="cuda"):
        import torch
        npk, nb, ng = cls.sizes(rows, cols)
        return cls(torch.empty(npk, dtype=torch.uint8, device=device),
                   torch.empty(nb, dtype=torch.uint8, device=device),
                   torch.empty(ng, dtype=torch.float32, device=device),
                   rows, cols)

    def as_struct(self) -> _NF4Struct:
        return _NF4Struct(self.packed.data_ptr(), self.qabs.data_ptr(),
                          self.gscale.data_ptr(), self.rows, self.cols)


def nf4_codebook():
    """(levels float32[16], thresholds float32[15]) from the library."""
    lv = np.zeros(16, dtype=np.float32)
    th = np.zeros(15, dtype=np.float32)
    _check("nf4_codebook", lib().nf4_codebook(lv.ctypes.data, th.ctypes.data))
    return lv, th


def nf4_quantize(w, out: NF4Tensor | None = None, status=None, stream=None):
    """Quantize a device fp32 weight [rows, cols]; returns the NF4Tensor."""
    rows, cols = (w.shape[0], w.shape[1]) if w.dim() == 2 else (1, w.numel())
    if out is None:
        out = NF4Tensor.empty(rows, cols, device=w.device)
    st = out.as_struct()
    _check("nf4_quantize", lib().nf4_quantize(_ptr(w), ctypes.byref(st),
                                              _ptr(status), _stream(stream)))
    return out


def nf4_dequantize(w: NF4Tensor, out=None, stream=None):
    """Dequantize to a bf16 device tensor [rows, cols]."""
    import torch
    if out is None:
        out = torch.empty((w.rows, w.cols), dtype=torch.bfloat16,
                          device=w.packed.device)
    st = w.as_struct()
    _check("nf4_dequantize", lib().nf4_dequantize(ctypes.byref(st), _ptr(out),
                                                  _stream(stream)))
    return out


def nf4_dequantize_batch(ws, outs=None, stream=None):
    """Dequantize several NF4 tensors in one launch; returns the bf16
    outputs (allocated when `outs` is None)."""
    import torch
    ws = list(ws)
    if outs is None:
        outs = [torch.empty((w.rows, w.cols), dtype=torch.bfloat16,
                            device=w.packed.device) for w in ws]
    structs = (_NF4Struct * len(ws))(*[w.as_struct() for w in ws])
    ptrs = (ctypes.c_void_p * len(ws))(*[_ptr(o) for o in outs])
    _check("nf4_dequantize_batch", lib().nf4_dequantize_batch(
        structs, ptrs, len(ws), _stream(stream)))
    return outs


def nf4_merge(w: NF4Tensor, A, B, r: int, alpha: float, out=None,
              stream=None):
    """Dense bf16 [rows, cols] = bf16(W' + (alpha / r) B A)."""
    import torch
    if out is None:
        out = torch.empty((w.rows, w.cols), dtype=torch.bfloat16,
                          device=w.packed.device)
    st = w.as_struct()
    _check("nf4_merge", lib().nf4_merge(ctypes.byref(st), _ptr(A), _ptr(B),
                                        int(r), float(alpha), _ptr(out),
                                        _stream(stream)))
    return out


@dataclass
class QTensor:
    """Device buffers of a codec-variant weight (see qn_qtensor in the
    header): packed codes, per-block constants (uint8, float32 or int8 by
    consts_mode), per-group scale and mean (empty where unused)."""
    packed: "object"
    consts: "object"
    gscale: "object"
    gmean: "object"
    rows: int
    cols: int
    code: int
    consts_mode: int

    @property
    def numel(self) -> int:
        return self.rows * self.cols

    @classmethod
    def empty(cls, rows: int, cols: int, code: int, consts_mode: int,
              device="cuda"):
        import torch
        npk, nb, ng = NF4Tensor.sizes(rows, cols)
        cdt = {QN_CONST_DQ8: torch.uint8, QN_CONST_FP32: torch.float32,
               QN_CONST_CENTERED: torch.int8}[consts_mode]
        has_scale = consts_mode != QN_CONST_FP32
        has_mean = consts_mode == QN_CONST_CENTERED
        return cls(torch.empty(npk, dtype=torch.uint8, device=device),
                   torch.empty(nb, dtype=cdt, device=device),
                   torch.empty(ng if has_scale else 0, dtype=torch.float32, device=device),
                   torch.empty(ng if has_mean else 0, dtype=torch.float32, device=device),
                   rows, cols, code, consts_mode)

    def as_struct(self) -> _QStruct:
        def p(t):
            return t.data_ptr() if t is not None and t.numel() > 0 else None
        return _QStruct(self.packed.data_ptr(), p(self.consts), p(self.gscale),
                        p(self.gmean), self.rows, self.cols, self.code,
                        self.consts_mode)


def qn_codebook(code: int):
    """(levels float32[16], thresholds float32[15]) of a QN_CODE_* table."""
    lv = np.zeros(16, dtype=np.float32)
    th = np.zeros(15, dtype=np.float32)
    _check("qn_codebook", lib().qn_codebook(int(code), lv.ctypes.data,
                                            th.ctypes.data))
    return lv, th


def qn_quantize(w, code: int, consts_mode: int, out: QTensor | None = None,
                status=None, stream=None):
    """Quantize a device fp32 weight into a variant format; returns it."""
    rows, cols = (w.shape[0], w.shape[1]) if w.dim() == 2 else (1, w.numel())
    if out is None:
        out = QTensor.empty(rows, cols, code, consts_mode, device=w.device)
    st = out.as_struct()
    _check("qn_quantize", lib().qn_quantize(_ptr(w), ctypes.byref(st),
                                            _ptr(status), _stream(stream)))
    return out


def qn_dequantize(w: QTensor, out=None, stream=None):
    """bf16 device tensor [rows, cols] of a variant-format weight."""
    import torch
    if out is None:
        out = torch.empty((w.rows, w.cols), dtype=torch.bfloat16,
                          device=w.packed.device)
    st = w.as_struct()
    _check("qn_dequantize", lib().qn_dequantize(ctypes.byref(st), _ptr(out),
                                                _stream(stream)))
    return out


@dataclass
class AdamW8State:
    """8-bit AdamW state of n parameters (see qn_adamw8_state in the header):
    E4M3 codes of m and sqrt(v), one fp32 scale each per 256 elements.
    Device tensors, or pinned host tensors for the paged step."""
    m_codes: "object"
    m_scale: "object"
    r_codes: "object"
    r_scale: "object"

    @classmethod
    def zeros(cls, n: int, device="cuda", pin_memory=False):
        import torch
        nb = -(-n // QN_ADAMW_BLOCK)
        kw = dict(device=device) if not pin_memory else dict(pin_memory=True)
        return cls(torch.zeros(n, dtype=torch.uint8, **kw),
                   torch.zeros(nb, dtype=torch.float32, **kw),
                   torch.zeros(n, dtype=torch.uint8, **kw),
                   torch.zeros(nb, dtype=torch.float32, **kw))

    def as_struct(self) -> _Adam8State:
        return _Adam8State(self.m_codes.data_ptr(), self.m_scale.data_ptr(),
                           self.r_codes.data_ptr(), self.r_scale.data_ptr())


def _hparams(lr, beta1, beta2, eps, weight_decay, grad_scale) -> _AdamHP:
    return _AdamHP(float(lr), float(beta1), float(beta2), float(eps),
                   float(weight_decay), float(grad_scale))


def qn_adamw8_step(p, g, state: AdamW8State, step: int, lr=2e-4, beta1=0.9,
                   beta2=0.999, eps=1e-8, weight_decay=0.0, grad_scale=1.0,
                   stream=None):
    """One 8-bit AdamW step on bf16 parameters p (in place) with fp32
    gradients g and a device-resident state."""
    hp = _hparams(lr, beta1, beta2, eps, weight_decay, grad_scale)
    st = state.as_struct()
    _check("qn_adamw8_step", lib().qn_adamw8_step(
        _ptr(p), _ptr(g), p.numel(), ctypes.byref(st), ctypes.byref(hp),
        int(step), _stream(stream)))


def qn_adamw8_staging_bytes(chunk: int) -> int:
    return int(lib().qn_adamw8_staging_bytes(int(chunk)))


def qn_adamw8_paged_step(p, g, host_state: AdamW8State, staging, chunk: int,
                         step: int, lr=2e-4, beta1=0.9, beta2=0.999,
                         eps=1e-8, weight_decay=0.0, grad_scale=1.0,
                         stream=None, h2d_stream=None, d2h_stream=None):
    """The same step with the state in pinned host memory, paged through
    the device `staging` buffer in pages of `chunk` elements."""
    hp = _hparams(lr, beta1, beta2, eps, weight_decay, grad_scale)
    st = host_state.as_struct()
    cs = _stream(stream)
    hs = None if h2d_stream is None else getattr(h2d_stream, "cuda_stream", h2d_stream)
    ds = None if d2h_stream is None else getattr(d2h_stream, "cuda_stream", d2h_stream)
    _check("qn_adamw8_paged_step", lib().qn_adamw8_paged_step(
        _ptr(p), _ptr(g), p.numel(), ctypes.byref(st), _ptr(staging),
        staging.numel() * staging.element_size(), int(chunk),
        ctypes.byref(hp), int(step), cs, hs, ds))


def qlora_workspace_bytes(M: int, N: int, K: int, r: int, which: int) -> int:
    return int(lib().qlora_workspace_bytes(M, N, K, r, which))


def qlora_linear_fwd(x, w: NF4Tensor, A, B, r: int, alpha: float, y=None,
                     y_dtype: int = QN_F32, t_save=None, ws=None,
                     stream=None):
    """Fused forward; returns (y, t_save)."""
    import torch
    M = x.shape[0]
    dev = x.device
    if y is None:
        y = torch.empty((M, w.rows), device=dev,
                        dtype=torch.float32 if y_dtype == QN_F32 else torch.bfloat16)
    if t_save is None:
        t_save = torch.empty((M, r), device=dev, dtype=torch.float32)
    need = qlora_workspace_bytes(M, w.rows, w.cols, r, QN_FWD)
    if ws is None and need:
        ws = torch.empty(need, dtype=torch.uint8, device=dev)
    st = w.as_struct()
    _check("qlora_linear_fwd", lib().qlora_linear_fwd(
        _ptr(x), M, ctypes.byref(st), _ptr(A), _ptr(B), r, float(alpha),
        _ptr(y), y_dtype, _ptr(t_save), _ptr(ws),
        0 if ws is None else ws.numel() * ws.element_size(), _stream(stream)))
    return y, t_save


class FwdBatch:
    """Descriptors of a qlora_linear_fwd_batch call, kept alive with the
    tensors they point to.  jobs: sequence of (x, w, A, B, r, alpha, y,
    y_dtype, t_save) with y / t_save None to allocate them."""

    def __init__(self, jobs):
        import torch
        self.keep, self.outs = [], []
        arr = (_FwdJob * len(jobs))()
        for i, (x, w, A, B, r, alpha, y, y_dtype, t_save) in enumerate(jobs):
            M = x.shape[0]
            if y is None:
                y = torch.empty((M, w.rows), device=x.device,
                                dtype=torch.float32 if y_dtype == QN_F32
                                else torch.bfloat16)
            if t_save is None:
                t_save = torch.empty((M, r), device=x.device, dtype=torch.float32)
            st = w.as_struct()
            self.keep += [x, A, B, y, t_save, st]
            self.outs.append((y, t_save))
            arr[i] = _FwdJob(_ptr(x), M, ctypes.pointer(st), _ptr(A), _ptr(B), r,
                             float(alpha), _ptr(y), y_dtype, _ptr(t_save))
        self.arr, self.count = arr, len(jobs)
        self.ws_bytes = lib().qlora_fwd_batch_workspace_bytes(arr, self.count)
        self.ws = torch.empty(max(self.ws_bytes, 1), dtype=torch.uint8,
                              device=jobs[0][0].device)


def qlora_fwd_batch_workspace_bytes(batch: FwdBatch) -> int:
    return int(lib().qlora_fwd_batch_workspace_bytes(batch.arr, batch.count))


def qlora_linear_fwd_batch(batch: FwdBatch, stream=None):
    """Batched skinny forward (every job M <= 16); returns [(y, t_save)]."""
    _check("qlora_linear_fwd_batch", lib().qlora_linear_fwd_batch(
        batch.arr, batch.count, _ptr(batch.ws),
        batch.ws.numel() * batch.ws.element_size(), _stream(stream)))
    return batch.outs


def qlora_linear_fwd_noalloc(x, w: NF4Tensor, A, B, r: int, alpha: float,
                             y=None, y_dtype: int = QN_F32, t_save=None,
                             stream=None):
    """Fused forward with the library's own per-GPU scratch array as its
    workspace (no workspace argument); returns (y, t_save).  Calls on one
    GPU share the array: do not overlap them."""
    import torch
    M = x.shape[0]
    dev = x.device
    if y is None:
        y = torch.empty((M, w.rows), device=dev,
                        dtype=torch.float32 if y_dtype == QN_F32 else torch.bfloat16)
    if t_save is None:
        t_save = torch.empty((M, r), device=dev, dtype=torch.float32)
    st = w.as_struct()
    _check("qlora_linear_fwd_noalloc", lib().qlora_linear_fwd_noalloc(
        _ptr(x), M, ctypes.byref(st), _ptr(A), _ptr(B), r, float(alpha),
        _ptr(y), y_dtype, _ptr(t_save), _stream(stream)))
    return y, t_save


def qlora_linear_bwd(dy, x, w: NF4Tensor, A, B, r: int, alpha: float,
                     t_saved, dx=None, dx_dtype: int = QN_F32, dA=None,
                     dB=None, ws=None, stream=None):
    """Fused backward; returns (dx, dA, dB)."""
    import torch
    M = x.shape[0]
    dev = x.device
    if dx is None:
        dx = torch.empty((M, w.cols), device=dev,
                         dtype=torch.float32 if dx_dtype == QN_F32 else torch.bfloat16)
    if dA is None:
        dA = torch.empty((r, w.cols), device=dev, dtype=torch.float32)
    if dB is None:
        dB = torch.empty((w.rows, r), device=dev, dtype=torch.float32)
    if ws is None:
        ws = torch.empty(max(1, qlora_workspace_bytes(M, w.rows, w.cols, r, QN_BWD)),
                         dtype=torch.uint8, device=dev)
    st = w.as_struct()
    _check("qlora_linear_bwd", lib().qlora_linear_bwd(
        _ptr(dy), _ptr(x), M, ctypes.byref(st), _ptr(A), _ptr(B), r,
        float(alpha), _ptr(t_saved), _ptr(dx), dx_dtype, _ptr(dA), _ptr(dB),
        _ptr(ws), ws.numel() * ws.element_size(), _stream(stream)))
    return dx, dA, dB


def qlora_linear_fwd_dropout(x, w: NF4Tensor, A, B, r: int, alpha: float,
                             p: float, seed: int, y=None,
                             y_dtype: int = QN_F32, t_save=None, ws=None,
                             stream=None):
    """Fused forward with LoRA dropout (probability p, 64-bit seed) on the
    adapter input; returns (y, t_save)."""
    import torch
    M = x.shape[0]
    dev = x.device
    if y is None:
        y = torch.empty((M, w.rows), device=dev,
                        dtype=torch.float32 if y_dtype == QN_F32 else torch.bfloat16)
    if t_save is None:
        t_save = torch.empty((M, r), device=dev, dtype=torch.float32)
    if ws is None:
        ws = torch.empty(max(1, qlora_workspace_bytes(M, w.rows, w.cols, r,
                                                      QN_FWD_DROPOUT)),
                         dtype=torch.uint8, device=dev)
    st = w.as_struct()
    d = _Dropout(float(p), int(seed) & 0xFFFFFFFFFFFFFFFF)
    _check("qlora_linear_fwd_dropout", lib().qlora_linear_fwd_dropout(
        _ptr(x), M, ctypes.byref(st), _ptr(A), _ptr(B), r, float(alpha),
        _ptr(y), y_dtype, _ptr(t_save), ctypes.byref(d), _ptr(ws),
        ws.numel() * ws.element_size(), _stream(stream)))
    return y, t_save


def qlora_linear_bwd_dropout(dy, x, w: NF4Tensor, A, B, r: int, alpha: float,
                             t_saved, p: float, seed: int, dx=None,
                             dx_dtype: int = QN_F32, dA=None, dB=None,
                             ws=None, stream=None):
    """Fused backward with the forward's dropout mask; returns (dx, dA, dB)."""
    import torch
    M = x.shape[0]
    dev = x.device
    if dx is None:
        dx = torch.empty((M, w.cols), device=dev,
                         dtype=torch.float32 if dx_dtype == QN_F32 else torch.bfloat16)
    if dA is None:
        dA = torch.empty((r, w.cols), device=dev, dtype=torch.float32)
    if dB is None:
        dB = torch.empty((w.rows, r), device=dev, dtype=torch.float32)
    if ws is None:
        ws = torch.empty(max(1, qlora_workspace_bytes(M, w.rows, w.cols, r, QN_BWD)),
                         dtype=torch.uint8, device=dev)
    st = w.as_struct()
    d = _Dropout(float(p), int(seed) & 0xFFFFFFFFFFFFFFFF)
    _check("qlora_linear_bwd_dropout", lib().qlora_linear_bwd_dropout(
        _ptr(dy), _ptr(x), M, ctypes.byref(st), _ptr(A), _ptr(B), r,
        float(alpha), _ptr(t_saved), _ptr(dx), dx_dtype, _ptr(dA), _ptr(dB),
        ctypes.byref(d), _ptr(ws), ws.numel() * ws.element_size(),
        _stream(stream)))
    return dx, dA, dB


# ---------------------------------------------------------------------------
# 8-bit activation checkpoints and the preference loss.  Tensors are checked
# here (device, type, shape, layout) before their addresses are passed on;
# calls run on the device of their tensors, and what they allocate belongs to
# the stream they run on.  Small calls take a few microseconds on the GPU, so
# the checks build no text unless they fail and the plain case (the current
# device's current stream) enters no context.
# ---------------------------------------------------------------------------

def _bad(fn: str, what: str):
    return QNError(fn, QN_EINVAL, what)


_raw = None


def _raw_stream(index: int) -> int:
    """Handle of device `index`'s current stream."""
    global _raw
    if _raw is None:
        import torch
        _raw = getattr(torch._C, "_cuda_getCurrentRawStream",
                       lambda i: torch.cuda.current_stream(i).cuda_stream)
    return _raw(index)


def _run_on(index: int, stream, body):
    """body(handle) on the stream given, or on device `index`'s current one;
    that stream and device are current inside."""
    import torch
    if stream is None:
        if index == torch.cuda.current_device():
            return body(_raw_stream(index))
        with torch.cuda.device(index):
            return body(_raw_stream(index))
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream), device=index)
    if stream.device_index != index:
        raise _bad("stream", f"the stream is on device {stream.device_index}, the tensors "
                   f"on {index}")
    with torch.cuda.stream(stream):
        return body(stream.cuda_stream)


def _gpu(fn: str, name: str, t) -> int:
    if not t.is_cuda:
        raise _bad(fn, f"{name} must be on a GPU")
    return t.get_device()


def _dtype_code(fn: str, name: str, t) -> int:
    import torch
    dt = t.dtype
    if dt is torch.bfloat16:
        return QN_BF16
    if dt is torch.float32:
        return QN_F32
    raise _bad(fn, f"{name} must be float32 or bfloat16, not {dt}")


def _torch_dtype(fn: str, code: int):
    import torch
    if code not in (QN_F32, QN_BF16):
        raise _bad(fn, f"unknown dtype {code}")
    return torch.float32 if code == QN_F32 else torch.bfloat16


def _tensor(fn: str, name: str, t, shape: tuple, dtype, index: int) -> int:
    """The address of `t`, a dense tensor of that shape and type (None: any)
    on device `index`."""
    if (t.shape == shape and (dtype is None or t.dtype is dtype) and t.is_contiguous()
            and t.is_cuda and t.get_device() == index):
        return t.data_ptr()
    if not t.is_cuda or t.get_device() != index:
        raise _bad(fn, f"{name} is on {t.device}, not on GPU {index}")
    if dtype is not None and t.dtype is not dtype:
        raise _bad(fn, f"{name} must be {dtype}, not {t.dtype}")
    if t.shape != shape:
        raise _bad(fn, f"{name} must have shape {tuple(shape)}, not {tuple(t.shape)}")
    raise _bad(fn, f"{name} must be contiguous")


def _workspace(fn: str, ws, index: int) -> tuple[int, int]:
    """(address, bytes) of a caller's workspace."""
    if not ws.is_cuda or ws.get_device() != index or not ws.is_contiguous():
        raise _bad(fn, f"ws must be contiguous and on GPU {index}")
    return ws.data_ptr(), ws.numel() * ws.element_size()


def _weight(fn: str, w: NF4Tensor, index: int) -> _NF4Struct:
    """The struct of a weight whose buffers are on device `index`, of the
    codec's types and hold its size."""
    import torch
    a, b, c = w.packed, w.qabs, w.gscale
    n = w.rows * w.cols
    nb = -(-n // QN_BLOCK)
    u8 = torch.uint8
    if (a.get_device() == index == b.get_device() and c.get_device() == index
            and a.dtype is u8 and b.dtype is u8 and c.dtype is torch.float32
            and 2 * a.numel() >= n and b.numel() >= nb and c.numel() * QN_GROUP >= nb
            and a.is_contiguous() and b.is_contiguous() and c.is_contiguous()):
        return _NF4Struct(a.data_ptr(), b.data_ptr(), c.data_ptr(), w.rows, w.cols)
    raise _bad(fn, f"w must be contiguous, on GPU {index}, uint8, uint8 and float32, and of "
               f"{w.sizes(w.rows, w.cols)} elements")


@dataclass
class Act8Tensor:
    """Device buffers of an 8-bit activation checkpoint (see qn_act8 in the
    header): int8 codes [rows, cols], fp32 scales [rows, ceil(cols / 64)]."""
    codes: "object"
    scale: "object"
    rows: int
    cols: int

    @classmethod
    def empty(cls, rows: int, cols: int, device="cuda"):
        import torch
        return cls(torch.empty((rows, cols), dtype=torch.int8, device=device),
                   torch.empty((rows, -(-cols // QN_BLOCK)), dtype=torch.float32,
                               device=device), rows, cols)

    def as_struct(self) -> _Act8Struct:
        return _Act8Struct(self.codes.data_ptr(), self.scale.data_ptr(),
                           self.rows, self.cols)

    def checked_struct(self, fn: str, index: int) -> _Act8Struct:
        import torch
        rows, cols = self.rows, self.cols
        if cols < 1:
            raise _bad(fn, "a checkpoint has at least one column")
        return _Act8Struct(
            _tensor(fn, "codes", self.codes, (rows, cols), torch.int8, index),
            _tensor(fn, "scale", self.scale, (rows, -(-cols // QN_BLOCK)), torch.float32, index),
            rows, cols)


def qn_act8_encode(x, out: Act8Tensor | None = None, stream=None):
    """8-bit checkpoint of a device activation [rows, cols] (fp32 or bf16,
    contiguous); returns the Act8Tensor."""
    fn = "qn_act8_encode"
    index = _gpu(fn, "x", x)
    code = _dtype_code(fn, "x", x)
    shape = x.shape
    if len(shape) != 2 or shape[1] < 1:
        raise _bad(fn, "x must be [rows, cols]")
    px = _tensor(fn, "x", x, shape, None, index)
    if out is not None and (out.rows, out.cols) != shape:
        raise _bad(fn, "out has another shape than x")

    def body(st):
        t = out
        if t is None:
            t = Act8Tensor.empty(shape[0], shape[1], device=x.device)
            s = t.as_struct()
        else:
            s = t.checked_struct(fn, index)
        _check(fn, lib().qn_act8_encode(px, code, s, st))
        return t
    return _run_on(index, stream, body)


def qn_act8_decode(x8: Act8Tensor, out=None, dtype: int = QN_BF16, stream=None):
    """The restored activation [rows, cols] in bf16 or fp32 (`out`'s type
    when it is given)."""
    fn = "qn_act8_decode"
    index = _gpu(fn, "codes", x8.codes)
    s = x8.checked_struct(fn, index)
    shape = (x8.rows, x8.cols)

    def body(st):
        y, code = out, dtype
        if y is None:
            y = x8.codes.new_empty(shape, dtype=_torch_dtype(fn, dtype))
            py = y.data_ptr()
        else:
            py, code = _tensor(fn, "out", y, shape, None, index), _dtype_code(fn, "out", y)
        _check(fn, lib().qn_act8_decode(s, py, code, st))
        return y
    return _run_on(index, stream, body)


def qlora_bwd_act8_workspace_bytes(M: int, N: int, K: int, r: int) -> int:
    return int(lib().qlora_bwd_act8_workspace_bytes(M, N, K, r))


def qlora_linear_bwd_act8(dy, x8: Act8Tensor, w: NF4Tensor, A, B, r: int,
                          alpha: float, t_saved, p: float = 0.0, seed: int = 0,
                          dx=None, dx_dtype: int = QN_F32, need_dx: bool = True,
                          dA=None, dB=None, ws=None, stream=None):
    """Fused backward from an 8-bit checkpoint of the layer's input, with LoRA
    dropout (probability p, 64-bit seed) if p > 0; returns (dx, dA, dB), dx
    None where need_dx is False."""
    import torch
    fn = "qlora_linear_bwd_act8"
    index = _gpu(fn, "dy", dy)
    M, N, K = x8.rows, w.rows, w.cols
    bf, f32 = torch.bfloat16, torch.float32
    xt = x8.checked_struct(fn, index)
    if x8.cols != K:
        raise _bad(fn, f"the checkpoint has {x8.cols} columns, the weight {K}")
    if M < 1 or not 1 <= r <= QN_MAX_RANK:
        raise _bad(fn, "M or r out of range")
    if dx is not None and not need_dx:
        raise _bad(fn, "dx given with need_dx=False")
    pdy = _tensor(fn, "dy", dy, (M, N), bf, index)
    pA = _tensor(fn, "A", A, (r, K), bf, index)
    pB = _tensor(fn, "B", B, (N, r), bf, index)
    pt = _tensor(fn, "t_saved", t_saved, (M, r), f32, index)
    wt = _weight(fn, w, index)

    def body(st):
        gx, gA, gB = dx, dA, dB
        pdx, code = None, dx_dtype
        if gx is not None:
            pdx, code = _tensor(fn, "dx", gx, (M, K), None, index), _dtype_code(fn, "dx", gx)
        elif need_dx:
            gx = dy.new_empty((M, K), dtype=_torch_dtype(fn, dx_dtype))
            pdx = gx.data_ptr()
        if gA is None:
            gA = dy.new_empty((r, K), dtype=f32)
        else:
            _tensor(fn, "dA", gA, (r, K), f32, index)
        if gB is None:
            gB = dy.new_empty((N, r), dtype=f32)
        else:
            _tensor(fn, "dB", gB, (N, r), f32, index)
        if ws is None:
            nw = qlora_bwd_act8_workspace_bytes(M, N, K, r)
            wk = dy.new_empty(nw, dtype=torch.uint8)
            pw = wk.data_ptr()
        else:
            pw, nw = _workspace(fn, ws, index)
        _check(fn, lib().qlora_linear_bwd_act8(
            pdy, xt, M, wt, pA, pB, int(r), float(alpha), pt, pdx, code,
            gA.data_ptr(), gB.data_ptr(),
            _Dropout(float(p), int(seed) & 0xFFFFFFFFFFFFFFFF), pw, nw, st))
        return gx, gA, gB
    return _run_on(index, stream, body)


def qn_seq_workspace_bytes(rows: int, vocab: int, nseq: int) -> int:
    return int(lib().qn_seq_workspace_bytes(rows, vocab, nseq))


def _seq_batch(fn: str, logits, labels, offsets):
    """(device index, qn_seq_batch) of logits [rows, vocab] whose rows may be
    apart (stride(0) >= vocab), labels [rows] and offsets [nseq + 1]."""
    import torch
    index = _gpu(fn, "logits", logits)
    code = _dtype_code(fn, "logits", logits)
    shape = logits.shape
    if len(shape) != 2 or shape[1] < 1:
        raise _bad(fn, "logits must be [rows, vocab]")
    rows, vocab = shape
    ld, step = logits.stride()
    if step != 1 and vocab > 1:
        raise _bad(fn, "a row of logits must be contiguous")
    if rows <= 1:
        ld = vocab
    if ld < vocab:
        raise _bad(fn, "rows of logits overlap")
    n = offsets.shape
    if len(n) != 1 or n[0] < 2:
        raise _bad(fn, "offsets must be [nseq + 1]")
    return index, _SeqBatch(
        logits.data_ptr(), code, rows, vocab, ld,
        _tensor(fn, "labels", labels, (rows,), torch.int64, index),
        _tensor(fn, "offsets", offsets, n, torch.int64, index), n[0] - 1)


def _seq_output(fn, name, t, like, n, index):
    """(tensor, address) of an fp32 output of n elements: the one given, or a
    new one with memory of its own."""
    import torch
    if t is not None:
        return t, _tensor(fn, name, t, (n,), torch.float32, index)
    t = like.new_empty(n, dtype=torch.float32)
    return t, t.data_ptr()


def _seq_workspace(fn, b, like, ws, index):
    """(address, bytes, what keeps it alive) of a forward's workspace."""
    import torch
    if ws is not None:
        return *_workspace(fn, ws, index), ws
    nw = qn_seq_workspace_bytes(b.rows, b.vocab, b.nseq)
    ws = like.new_empty(nw, dtype=torch.uint8)
    return ws.data_ptr(), nw, ws


def _status_ptr(fn, status, index):
    import torch
    return None if status is None else _tensor(fn, "status", status, (1,), torch.int32, index)


def _set_lse_lo(fn, b, lse_lo, index):
    import torch
    if lse_lo is not None:
        b.lse_lo = _tensor(fn, "lse_lo", lse_lo, (b.rows,), torch.float32, index)


def qn_seq_logprob(logits, labels, offsets, lse=None, logp=None, status=None,
                   ws=None, stream=None, lse_lo=None):
    """Log-probability of each packed sequence and log-sum-exp of each row;
    returns (logp [nseq], lse [rows]).  lse_lo (fp32 [rows]), if given, is set
    to what lse loses by its rounding, for qn_seq_logprob_bwd."""
    fn = "qn_seq_logprob"
    index, b = _seq_batch(fn, logits, labels, offsets)
    _set_lse_lo(fn, b, lse_lo, index)

    def body(st):
        lp, plp = _seq_output(fn, "logp", logp, logits, b.nseq, index)
        ls, pls = _seq_output(fn, "lse", lse, logits, b.rows, index)
        pw, nw, _keep = _seq_workspace(fn, b, logits, ws, index)
        _check(fn, lib().qn_seq_logprob(b, pls, plp, _status_ptr(fn, status, index), pw, nw, st))
        return lp, ls
    return _run_on(index, stream, body)


@dataclass
class PrefLoss:
    """Outputs of qn_pref_loss_fwd: loss [P], logp [2P], dlogp [2P] (the
    derivative of a pair's loss by its sequences' logp), lse [rows] and lse_lo
    [rows] (what lse loses by its rounding).  Those of a call without `out`
    share one allocation."""
    loss: "object"
    logp: "object"
    dlogp: "object"
    lse: "object"
    lse_lo: "object" = None


def qn_pref_loss_fwd(logits, labels, offsets, ref_logp, beta: float,
                     label_smoothing: float = 0.0, out: PrefLoss | None = None,
                     status=None, ws=None, stream=None):
    """Paired log-ratio loss of sequences p (chosen) and P + p (rejected);
    ref_logp [2P] or None for zeros; returns a PrefLoss (`out` when it is
    given; its fields that are None are allocated and set)."""
    import torch
    fn = "qn_pref_loss_fwd"
    index, b = _seq_batch(fn, logits, labels, offsets)
    f32, rows, nseq = torch.float32, b.rows, b.nseq
    pairs = nseq // 2
    if nseq != 2 * pairs:
        raise _bad(fn, "sequences must come in pairs")
    pr = None if ref_logp is None else _tensor(fn, "ref_logp", ref_logp, (nseq,), f32, index)

    def body(st):
        sizes = (pairs, nseq, nseq, rows, rows)
        if out is None:              # the fields of one result: one allocation
            buf = logits.new_empty(pairs + 2 * (nseq + rows), dtype=f32)
            o, p = buf.split_with_sizes(sizes), [buf.data_ptr()]
            for n in sizes[:-1]:
                p.append(p[-1] + 4 * n)
        else:
            o, p = zip(*(_seq_output(fn, k, getattr(out, k), logits, n, index) for k, n in
                         zip(("loss", "logp", "dlogp", "lse", "lse_lo"), sizes)))
        pw, nw, _keep = _seq_workspace(fn, b, logits, ws, index)
        b.lse_lo = p[4]
        _check(fn, lib().qn_pref_loss_fwd(
            b, pr, _PrefHP(float(beta), float(label_smoothing)), p[3], p[1], p[0], p[2],
            _status_ptr(fn, status, index), pw, nw, st))
        if out is None:
            return PrefLoss(*o)
        out.loss, out.logp, out.dlogp, out.lse, out.lse_lo = o
        return out
    return _run_on(index, stream, body)


def _seq_bwd(fn, logits, labels, offsets, lse, lse_lo, dlogp, dloss, dlogits, dl_dtype, stream):
    import torch
    index, b = _seq_batch(fn, logits, labels, offsets)
    _set_lse_lo(fn, b, lse_lo, index)
    f32, rows, vocab, nseq = torch.float32, b.rows, b.vocab, b.nseq
    args = [b, _tensor(fn, "lse", lse, (rows,), f32, index),
            _tensor(fn, "dlogp", dlogp, (nseq,), f32, index)]
    if fn == "qn_pref_loss_bwd":
        if nseq % 2:
            raise _bad(fn, "sequences must come in pairs")
        args.append(None if dloss is None
                    else _tensor(fn, "dloss", dloss, (nseq // 2,), f32, index))
    call = getattr(lib(), fn)

    def body(st):
        dl = dlogits
        if dl is None:
            dl = logits.new_empty((rows, vocab), dtype=logits.dtype if dl_dtype is None
                                  else _torch_dtype(fn, dl_dtype))
        code = _dtype_code(fn, "dlogits", dl)
        shape = dl.shape
        if not dl.is_cuda or dl.get_device() != index:
            raise _bad(fn, f"dlogits is on {dl.device}, not on GPU {index}")
        if len(shape) != 2 or shape[0] != rows or shape[1] < vocab:
            raise _bad(fn, "dlogits must be [rows, cols], cols >= vocab")
        cols = shape[1]
        ld, step = dl.stride()
        if step != 1 and cols > 1:
            raise _bad(fn, "a row of dlogits must be contiguous")
        if rows <= 1:
            ld = max(cols, b.ld)
        _check(fn, call(*args, dl.data_ptr(), code, cols, ld, st))
        return dl
    return _run_on(index, stream, body)


def qn_seq_logprob_bwd(logits, labels, offsets, lse, dlogp, dlogits=None,
                       dl_dtype: int | None = None, stream=None, lse_lo=None):
    """Gradient of sum(dlogp * logp) by the logits.  dlogits may have more
    columns than the logits (written as zeros) and may be the logits
    themselves; it is allocated in dl_dtype (the logits' type) when None.
    lse_lo as set by the forward; without it the probabilities of a row are
    off by the rounding of its lse."""
    return _seq_bwd("qn_seq_logprob_bwd", logits, labels, offsets, lse, lse_lo, dlogp, None,
                    dlogits, dl_dtype, stream)


def qn_pref_loss_bwd(logits, labels, offsets, fwd: PrefLoss, dloss=None,
                     dlogits=None, dl_dtype: int | None = None, stream=None):
    """Gradient of sum(dloss * loss) by the logits (dloss None: the mean
    loss), from what qn_pref_loss_fwd returned; dlogits as in
    qn_seq_logprob_bwd."""
    return _seq_bwd("qn_pref_loss_bwd", logits, labels, offsets, fwd.lse, fwd.lse_lo, fwd.dlogp,
                    dloss, dlogits, dl_dtype, stream)


def qn_profile_kernel(name: str | None, starts=None, stops=None) -> int:
    """Arm (or with name=None disarm) per-launch event timing of one internal
    kernel.  ``starts``/``stops`` are lists of torch.cuda.Event created with
    enable_timing=True; returns the number of launches recorded before this
    call re-armed or disarmed."""
    if name is None:
        return int(lib().qn_profile_kernel(None, None, None, 0))
    import torch
    n = len(starts)
    assert len(stops) == n
    for e in list(starts) + list(stops):
        if not e.cuda_event:           # torch creates the event on first record
            e.record()
    torch.cuda.synchronize()
    if not all(e.cuda_event for e in list(starts) + list(stops)):
        raise RuntimeError("qn_profile_kernel: event handles are not created")
    arr_t = ctypes.c_void_p * max(n, 1)
    a = arr_t(*[e.cuda_event for e in starts])
    b = arr_t(*[e.cuda_event for e in stops])
    _profile_keepalive[:] = [a, b, starts, stops]
    rc = int(lib().qn_profile_kernel(name.encode(), a, b, n))
    if rc < 0:
        raise QNError("qn_profile_kernel", rc)
    return rc


_profile_keepalive: list = []
