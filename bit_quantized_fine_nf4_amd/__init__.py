"""Python binding of libqlora_nf4.so — the MI355X (gfx950) NF4 + LoRA linear layer.

Argument marshalling only: every step runs in the library's HIP kernels.
PyTorch provides device memory and the current stream.  The functions carry
the C ABI's names (include/qlora_nf4.h).  Importing this module loads the
library; if it has not been built, the import raises (there is no fallback).
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
from typing import Optional, Tuple

import torch  # noqa: F401  (loads the HIP runtime the library then shares)

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libqlora_nf4.so")

QLORA_OK, QLORA_ERR_INVALID_VALUE, QLORA_ERR_UNSUPPORTED, QLORA_ERR_LAUNCH, QLORA_ERR_INTERNAL = range(5)
QLORA_F32, QLORA_BF16 = 0, 1
QLORA_CB_NF4, QLORA_CB_INT4, QLORA_CB_FP4 = 0, 1, 2
CODEBOOKS = {"nf4": QLORA_CB_NF4, "int4": QLORA_CB_INT4, "fp4": QLORA_CB_FP4}
QLORA_OP_DOUBLE_QUANT, QLORA_OP_LINEAR_FWD, QLORA_OP_LINEAR_BWD = 0, 1, 2
QLORA_OP_NORM_BWD, QLORA_OP_LOSS_FWD, QLORA_OP_LOSS_BWD, QLORA_OP_LINEAR_DROPOUT = 3, 4, 5, 6
BLOCK, CHUNK, MAX_RANK = 64, 256, 128

EXPORTED = ("qlora_quantize", "qlora_double_quant", "qlora_dequantize", "qlora_linear_fwd",
            "qlora_linear_bwd", "qlora_merge_adapter", "qlora_merge_requantize", "qlora_adamw_step",
            "qlora_quantize_cb", "qlora_dequantize_cb", "qlora_dequantize_nodq", "qlora_codebook_levels",
            "qlora_linear_fwd_cb", "qlora_linear_bwd_cb", "qlora_merge_adapter_cb", "qlora_merge_requantize_cb",
            "qlora_silu_gate_fwd", "qlora_silu_gate_bwd", "qlora_grad_sum", "qlora_double_quant_noalloc",
            "qlora_norm_fwd", "qlora_norm_bwd", "qlora_loss_fwd", "qlora_loss_bwd",
            "qlora_dropout", "qlora_linear_fwd_dropout", "qlora_linear_bwd_dropout",
            "qlora_workspace_size", "qlora_stream_probe",
            "qlora_status_string", "qlora_nf4_levels", "qlora_set_timing_events")


class QloraError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {lib.qlora_status_string(status).decode()} (status {status})")
        self.status = status


class NF4WeightT(ctypes.Structure):
    """qlora_nf4_weight_t: four device pointers, then h and o."""
    _fields_ = [("codes", ctypes.c_void_p), ("qabsmax", ctypes.c_void_p), ("scale2", ctypes.c_void_p),
                ("mean", ctypes.c_void_p), ("h", ctypes.c_int64), ("o", ctypes.c_int64)]


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is missing: build it with `python bit_quantized_fine_nf4_amd/build.py`")
    L = ctypes.CDLL(LIB_PATH)
    vp, i64, i32, f32, st = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_int
    sz = ctypes.c_size_t
    L.qlora_quantize.argtypes = [vp, st, i64, vp, vp, vp]
    L.qlora_double_quant.argtypes = [vp, i64, vp, vp, vp, vp, sz, vp]
    L.qlora_double_quant_noalloc.argtypes = [vp, i64, vp, vp, vp, vp]
    L.qlora_dequantize.argtypes = [vp, vp, vp, vp, i64, vp, st, vp]
    L.qlora_quantize_cb.argtypes = [vp, st, i64, st, vp, vp, vp]
    L.qlora_dequantize_cb.argtypes = [vp, vp, vp, vp, i64, st, vp, st, vp]
    L.qlora_dequantize_nodq.argtypes = [vp, vp, i64, st, vp, st, vp]
    L.qlora_codebook_levels.argtypes = [st, ctypes.POINTER(ctypes.c_float)]
    L.qlora_linear_fwd.argtypes = [ctypes.POINTER(NF4WeightT), vp, i64, vp, vp, i32, f32, vp, vp, vp, sz, vp]
    L.qlora_linear_bwd.argtypes = [ctypes.POINTER(NF4WeightT), vp, vp, vp, i64, vp, vp, i32, f32, vp, vp, vp,
                                   vp, sz, vp]
    L.qlora_merge_adapter.argtypes = [ctypes.POINTER(NF4WeightT), vp, vp, i32, f32, vp, st, vp]
    L.qlora_merge_requantize.argtypes = [ctypes.POINTER(NF4WeightT), vp, vp, i32, f32, vp, vp, vp]
    W = ctypes.POINTER(NF4WeightT)
    L.qlora_linear_fwd_cb.argtypes = [W, st] + L.qlora_linear_fwd.argtypes[1:]
    L.qlora_linear_bwd_cb.argtypes = [W, st] + L.qlora_linear_bwd.argtypes[1:]
    L.qlora_merge_adapter_cb.argtypes = [W, st] + L.qlora_merge_adapter.argtypes[1:]
    L.qlora_merge_requantize_cb.argtypes = [W, st] + L.qlora_merge_requantize.argtypes[1:]
    L.qlora_silu_gate_fwd.argtypes = [vp, vp, i64, vp, vp]
    L.qlora_silu_gate_bwd.argtypes = [vp, vp, vp, i64, vp, vp, vp]
    L.qlora_grad_sum.argtypes = [ctypes.POINTER(vp), i32, i64, vp, vp]
    L.qlora_norm_fwd.argtypes = [vp, st, vp, vp, vp, f32, vp, f32, i64, i64, vp, vp, vp, vp, vp]
    L.qlora_norm_bwd.argtypes = [vp, vp, st, vp, vp, vp, vp, vp, vp, f32, vp, i64, i64, vp, vp, vp, vp, vp, vp, sz, vp]
    L.qlora_loss_fwd.argtypes = [vp, vp, vp, i64, i64, i64, vp, vp, vp, sz, vp]
    L.qlora_loss_bwd.argtypes = [vp, vp, vp, vp, vp, i64, i64, i64, vp, vp, vp, sz, vp]
    f64 = ctypes.c_double
    L.qlora_dropout.argtypes = [vp, st, i64, f64, vp, vp, vp]
    L.qlora_linear_fwd_dropout.argtypes = [W, st, vp, i64, vp, vp, i32, f32, f64, vp, vp, vp, vp, sz, vp]
    L.qlora_linear_bwd_dropout.argtypes = [W, st, vp, vp, vp, i64, vp, vp, i32, f32, f64, vp, vp, vp, vp, vp, sz, vp]
    L.qlora_stream_probe.argtypes = [i32, i32, i32, i32, vp, vp, i64, vp]
    L.qlora_adamw_step.argtypes = [vp, vp, vp, vp, i64, i64, f32, f32, f32, f32, f32, vp, vp]
    L.qlora_workspace_size.argtypes = [st, i64, i64, i64, i32, ctypes.POINTER(sz)]
    L.qlora_status_string.argtypes = [st]
    L.qlora_status_string.restype = ctypes.c_char_p
    L.qlora_nf4_levels.argtypes = [ctypes.POINTER(ctypes.c_float)]
    L.qlora_set_timing_events.argtypes = [i32, vp, vp]
    for name in EXPORTED:
        if name != "qlora_status_string":
            getattr(L, name).restype = ctypes.c_int
    return L


lib = _load()


def _check(status: int, where: str):
    if status != QLORA_OK:
        raise QloraError(status, where)


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _dev_check(*ts):
    for t in ts:
        if t is not None and (not t.is_cuda or not t.is_contiguous()):
            raise ValueError("tensors must be contiguous and on the GPU")


def _want(name: str, t: Optional[torch.Tensor], dtype, shape: tuple, device):
    """Refuses a tensor that the C call would misread: its type, shape, layout or device."""
    if t is not None and (t.dtype is not dtype or t.shape != shape or not t.is_contiguous()
                          or t.get_device() != device.index):  # (a CPU tensor: -1 and None)
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {tuple(shape)} on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def _at(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _call(device, name: str, *args):
    """Entry point `name` on `device`'s current stream, with that device current."""
    stream = torch._C._cuda_getCurrentRawStream(device.index)
    if torch._C._cuda_getDevice() == device.index:
        status = getattr(lib, name)(*args, stream)
    else:
        with torch.cuda.device(device):
            status = getattr(lib, name)(*args, stream)
    _check(status, name)


def nf4_levels() -> list:
    buf = (ctypes.c_float * 16)()
    _check(lib.qlora_nf4_levels(buf), "qlora_nf4_levels")
    return list(buf)


TIMED_GEMM_FWD, TIMED_GEMM_DX, TIMED_GEMV = 0, 1, 2


def _event_handle(ev):
    if ev is None:
        return None
    if hasattr(ev, "cuda_event"):          # torch.cuda.Event (recorded by the library, so read it
        return ctypes.c_void_p(ev.cuda_event)  # back with hipEventElapsedTime, not torch)
    return ctypes.c_void_p(ev.value if isinstance(ev, ctypes.c_void_p) else int(ev))


def qlora_set_timing_events(kernel: int, start=None, stop=None):
    """Record the hipEvent_t pair (start, stop) around later launches of `kernel`
    by this thread (None, None switches the hook off)."""
    _check(lib.qlora_set_timing_events(kernel, _event_handle(start), _event_handle(stop)),
           "qlora_set_timing_events")


def workspace_size(op: int, a: int, b: int = 0, c: int = 0, r: int = 0) -> int:
    out = ctypes.c_size_t(0)
    _check(lib.qlora_workspace_size(op, a, b, c, r, ctypes.byref(out)), "qlora_workspace_size")
    return out.value


@dataclasses.dataclass
class NF4Weight:
    """A frozen NF4 weight with double-quantized scales, logical shape h x o,
    stored in [o][h] order (PyTorch Linear.weight)."""
    codes: torch.Tensor    # uint8 [o*h/2]
    qabsmax: torch.Tensor  # int8 [o*h/64]
    scale2: torch.Tensor   # float32 [ceil(o*h/64/256)]
    mean: torch.Tensor     # float32 [1]
    h: int
    o: int
    codebook: int = QLORA_CB_NF4

    def as_ctypes(self) -> NF4WeightT:
        return NF4WeightT(self.codes.data_ptr(), self.qabsmax.data_ptr(), self.scale2.data_ptr(),
                          self.mean.data_ptr(), self.h, self.o)

    def check(self, device):
        """Refuses parts that the C call would misread, which does not know their sizes: of
        another type, too short, not contiguous or not on `device`."""
        n = self.h * self.o
        at = device.index
        for name, t, dtype, least in (("codes", self.codes, torch.uint8, n // 2),
                                      ("qabsmax", self.qabsmax, torch.int8, n // BLOCK),
                                      ("scale2", self.scale2, torch.float32, -(-n // (BLOCK * CHUNK))),
                                      ("mean", self.mean, torch.float32, 1)):
            if t.dtype is not dtype or t.numel() < least or not t.is_contiguous() or t.get_device() != at:
                raise ValueError(f"the weight's {name} must be a contiguous {dtype} tensor of {least} values on "
                                 f"{device}, got {t.dtype} {tuple(t.shape)} on {t.device}")

    def call(self, name: str, *args):
        """Call entry point `name` on this weight: the NF4 entry point, or its `_cb` variant
        with the codebook for other codebooks."""
        self.check(self.codes.device)  # (host codes: None, which no tensor's index is)
        wt = self.as_ctypes()
        if self.codebook == QLORA_CB_NF4:
            return getattr(lib, name)(ctypes.byref(wt), *args)
        return getattr(lib, name + "_cb")(ctypes.byref(wt), self.codebook, *args)


# ---------------------------------------------------------------------------
# The entry points
# ---------------------------------------------------------------------------

def codebook_levels(codebook: int = QLORA_CB_NF4) -> list:
    buf = (ctypes.c_float * 16)()
    _check(lib.qlora_codebook_levels(codebook, buf), "qlora_codebook_levels")
    return list(buf)


def qlora_quantize(w: torch.Tensor, codes: Optional[torch.Tensor] = None,
                   absmax: Optional[torch.Tensor] = None, codebook: int = QLORA_CB_NF4) -> Tuple[torch.Tensor, torch.Tensor]:
    """Blockwise 4-bit quantization (NF4 unless `codebook` says otherwise) of any float32/bf16
    GPU tensor (flattened)."""
    _dev_check(w)
    n = w.numel()
    dtype = {torch.float32: QLORA_F32, torch.bfloat16: QLORA_BF16}[w.dtype]
    if codes is None:
        codes = torch.empty((n + 1) // 2, dtype=torch.uint8, device=w.device)
    if absmax is None:
        absmax = torch.empty((n + BLOCK - 1) // BLOCK, dtype=torch.float32, device=w.device)
    if codebook == QLORA_CB_NF4:
        _check(lib.qlora_quantize(_ptr(w), dtype, n, _ptr(codes), _ptr(absmax), _stream(w.device)), "qlora_quantize")
    else:
        _check(lib.qlora_quantize_cb(_ptr(w), dtype, n, codebook, _ptr(codes), _ptr(absmax), _stream(w.device)),
               "qlora_quantize_cb")
    return codes, absmax


def qlora_double_quant(absmax: torch.Tensor, qabsmax: Optional[torch.Tensor] = None,
                       scale2: Optional[torch.Tensor] = None, mean: Optional[torch.Tensor] = None,
                       workspace: Optional[torch.Tensor] = None):
    """Double quantization of the float32 block scales -> (qabsmax int8, scale2 f32, mean f32[1])."""
    _dev_check(absmax)
    nb = absmax.numel()
    dev = absmax.device
    if qabsmax is None:
        qabsmax = torch.empty(nb, dtype=torch.int8, device=dev)
    if scale2 is None:
        scale2 = torch.empty((nb + CHUNK - 1) // CHUNK, dtype=torch.float32, device=dev)
    if mean is None:
        mean = torch.empty(1, dtype=torch.float32, device=dev)
    ws_bytes = workspace_size(QLORA_OP_DOUBLE_QUANT, nb)
    if workspace is None:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    _check(lib.qlora_double_quant(_ptr(absmax), nb, _ptr(qabsmax), _ptr(scale2), _ptr(mean), _ptr(workspace),
                                  workspace.numel(), _stream(dev)), "qlora_double_quant")
    return qabsmax, scale2, mean


def qlora_dequantize(codes: torch.Tensor, qabsmax: torch.Tensor, scale2: torch.Tensor, mean: torch.Tensor,
                     n: int, out_dtype: torch.dtype = torch.bfloat16,
                     out: Optional[torch.Tensor] = None, codebook: int = QLORA_CB_NF4) -> torch.Tensor:
    """Rebuild n weights as float32 or bf16."""
    _dev_check(codes, qabsmax, scale2, mean)
    dt = {torch.float32: QLORA_F32, torch.bfloat16: QLORA_BF16}[out_dtype]
    if out is None:
        out = torch.empty(n, dtype=out_dtype, device=codes.device)
    if codebook == QLORA_CB_NF4:
        _check(lib.qlora_dequantize(_ptr(codes), _ptr(qabsmax), _ptr(scale2), _ptr(mean), n, _ptr(out), dt,
                                    _stream(codes.device)), "qlora_dequantize")
    else:
        _check(lib.qlora_dequantize_cb(_ptr(codes), _ptr(qabsmax), _ptr(scale2), _ptr(mean), n, codebook,
                                       _ptr(out), dt, _stream(codes.device)), "qlora_dequantize_cb")
    return out


def qlora_dequantize_nodq(codes: torch.Tensor, absmax: torch.Tensor, n: int, out_dtype: torch.dtype = torch.bfloat16,
                          out: Optional[torch.Tensor] = None, codebook: int = QLORA_CB_NF4) -> torch.Tensor:
    """Rebuild n weights from the float32 block scales (no double quantization)."""
    _dev_check(codes, absmax)
    dt = {torch.float32: QLORA_F32, torch.bfloat16: QLORA_BF16}[out_dtype]
    if out is None:
        out = torch.empty(n, dtype=out_dtype, device=codes.device)
    _check(lib.qlora_dequantize_nodq(_ptr(codes), _ptr(absmax), n, codebook, _ptr(out), dt, _stream(codes.device)),
           "qlora_dequantize_nodq")
    return out


def quantize_weight(w_oh: torch.Tensor, codebook: int = QLORA_CB_NF4) -> NF4Weight:
    """quantize + double_quant of a [o][h] float32/bf16 weight."""
    o, h = w_oh.shape
    codes, absmax = qlora_quantize(w_oh, codebook=codebook)
    qa, s2, mean = qlora_double_quant(absmax)
    return NF4Weight(codes, qa, s2, mean, h, o, codebook)


def qlora_linear_fwd(W: NF4Weight, X: torch.Tensor, L1: Optional[torch.Tensor], L2: Optional[torch.Tensor],
                     s: float, Y: Optional[torch.Tensor] = None, T: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None):
    """Y = X·W_hat + s·(X·L1)·L2 -> (Y bf16 [M][o], T bf16 [M][r] or None)."""
    _dev_check(X, L1, L2)
    M = X.shape[0]
    r = 0 if L1 is None else L1.shape[1]
    dev = X.device
    if Y is None:
        Y = torch.empty(M, W.o, dtype=torch.bfloat16, device=dev)
    if T is None and r:
        T = torch.empty(M, r, dtype=torch.bfloat16, device=dev)
    ws_bytes = workspace_size(QLORA_OP_LINEAR_FWD, M, W.h, W.o, r)
    if workspace is None and ws_bytes:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    _check(W.call("qlora_linear_fwd", _ptr(X), M, _ptr(L1), _ptr(L2), r, float(s), _ptr(Y), _ptr(T),
                  _ptr(workspace), 0 if workspace is None else workspace.numel(), _stream(dev)),
           "qlora_linear_fwd")
    return Y, T


def qlora_merge_adapter(W: NF4Weight, L1: Optional[torch.Tensor], L2: Optional[torch.Tensor], s: float,
                        out_dtype: torch.dtype = torch.float32, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Dense merged weight W' = W_hat + s·L1·L2 in [o][h] storage (float32 or bf16)."""
    _dev_check(L1, L2)
    r = 0 if L1 is None else L1.shape[1]
    dt = {torch.float32: QLORA_F32, torch.bfloat16: QLORA_BF16}[out_dtype]
    if out is None:
        out = torch.empty(W.o, W.h, dtype=out_dtype, device=W.codes.device)
    _check(W.call("qlora_merge_adapter", _ptr(L1), _ptr(L2), r, float(s), _ptr(out), dt, _stream(W.codes.device)),
           "qlora_merge_adapter")
    return out


def qlora_merge_requantize(W: NF4Weight, L1: Optional[torch.Tensor], L2: Optional[torch.Tensor], s: float,
                           codes: Optional[torch.Tensor] = None, absmax: Optional[torch.Tensor] = None):
    """NF4 codes and float32 block absmax of the merged weight -> (codes, absmax)."""
    _dev_check(L1, L2)
    r = 0 if L1 is None else L1.shape[1]
    dev = W.codes.device
    n = W.h * W.o
    if codes is None:
        codes = torch.empty(n // 2, dtype=torch.uint8, device=dev)
    if absmax is None:
        absmax = torch.empty(n // BLOCK, dtype=torch.float32, device=dev)
    _check(W.call("qlora_merge_requantize", _ptr(L1), _ptr(L2), r, float(s), _ptr(codes), _ptr(absmax),
                  _stream(dev)), "qlora_merge_requantize")
    return codes, absmax


def qlora_adamw_step(param: torch.Tensor, grad: torch.Tensor, exp_avg: torch.Tensor, exp_avg_sq: torch.Tensor,
                     step: int, lr: float, beta1: float = 0.9, beta2: float = 0.999, eps: float = 1e-8,
                     weight_decay: float = 0.0, param_bf16: Optional[torch.Tensor] = None,
                     device=None) -> None:
    """AdamW step on float32 `param` (in place, with its moments).  Each tensor is a
    contiguous float32 GPU tensor or a pinned host tensor (optimizer state kept in CPU RAM);
    `device` names the GPU whose current stream runs the step (default: param's, else cuda:0)."""
    ts = (param, grad, exp_avg, exp_avg_sq)
    for t in ts + (param_bf16,):
        if t is None:
            continue
        if not t.is_contiguous() or not (t.is_cuda or t.is_pinned()):
            raise ValueError("tensors must be contiguous, on the GPU or in pinned host memory")
    if any(t.dtype != torch.float32 for t in ts) or (param_bf16 is not None and param_bf16.dtype != torch.bfloat16):
        raise ValueError("param, grad and moments are float32; param_bf16 is bf16")
    n = param.numel()
    if any(t.numel() != n for t in ts[1:]) or (param_bf16 is not None and param_bf16.numel() != n):
        raise ValueError("all arrays must have param's size")
    if device is None:
        device = param.device if param.is_cuda else torch.device("cuda:0")
    _check(lib.qlora_adamw_step(_ptr(param), _ptr(grad), _ptr(exp_avg), _ptr(exp_avg_sq), n, int(step), float(lr),
                                float(beta1), float(beta2), float(eps), float(weight_decay), _ptr(param_bf16),
                                _stream(device)), "qlora_adamw_step")


def qlora_linear_bwd(W: NF4Weight, X: Optional[torch.Tensor], T: Optional[torch.Tensor], dY: torch.Tensor,
                     L1: Optional[torch.Tensor], L2: Optional[torch.Tensor], s: float,
                     dX: Optional[torch.Tensor] = None, dL1: Optional[torch.Tensor] = None,
                     dL2: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Backward through the frozen NF4 weight -> (dX bf16 [M][h], dL1 f32 [h][r], dL2 f32 [r][o])."""
    _dev_check(X, T, dY, L1, L2)
    M = dY.shape[0]
    r = 0 if L1 is None else L1.shape[1]
    dev = dY.device
    if dX is None:
        dX = torch.empty(M, W.h, dtype=torch.bfloat16, device=dev)
    if r and dL1 is None:
        dL1 = torch.empty(W.h, r, dtype=torch.float32, device=dev)
    if r and dL2 is None:
        dL2 = torch.empty(r, W.o, dtype=torch.float32, device=dev)
    ws_bytes = workspace_size(QLORA_OP_LINEAR_BWD, M, W.h, W.o, r)
    if workspace is None and ws_bytes:
        workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=dev)
    _check(W.call("qlora_linear_bwd", _ptr(X), _ptr(T), _ptr(dY), M, _ptr(L1), _ptr(L2), r, float(s),
                  _ptr(dX), _ptr(dL1), _ptr(dL2), _ptr(workspace),
                  0 if workspace is None else workspace.numel(), _stream(dev)),
           "qlora_linear_bwd")
    return dX, dL1, dL2


# ---------------------------------------------------------------------------
# Block glue between the linears
# ---------------------------------------------------------------------------

def _same(*ts):
    n = ts[0].numel()
    for t in ts:
        if t.dtype != torch.bfloat16 or t.numel() != n:
            raise ValueError("glue tensors are bf16 of one size")
    return n


def qlora_silu_gate_fwd(G: torch.Tensor, U: torch.Tensor, H: Optional[torch.Tensor] = None) -> torch.Tensor:
    """H = SiLU(G) * U (bf16, elementwise)."""
    _dev_check(G, U, H)
    if H is None:
        H = torch.empty_like(G)
    n = _same(G, U, H)
    _check(lib.qlora_silu_gate_fwd(_ptr(G), _ptr(U), n, _ptr(H), _stream(G.device)), "qlora_silu_gate_fwd")
    return H


def qlora_silu_gate_bwd(G: torch.Tensor, U: torch.Tensor, dH: torch.Tensor, dG: Optional[torch.Tensor] = None,
                        dU: Optional[torch.Tensor] = None):
    """(dG, dU) of H = SiLU(G) * U for the upstream gradient dH."""
    _dev_check(G, U, dH, dG, dU)
    dG = torch.empty_like(G) if dG is None else dG
    dU = torch.empty_like(U) if dU is None else dU
    n = _same(G, U, dH, dG, dU)
    _check(lib.qlora_silu_gate_bwd(_ptr(G), _ptr(U), _ptr(dH), n, _ptr(dG), _ptr(dU), _stream(G.device)),
           "qlora_silu_gate_bwd")
    return dG, dU


def qlora_stream_probe(rd: int, wr: int, src: torch.Tensor, dst: torch.Tensor, n_tiles: int,
                       depth: int = 2, blocks: int = 0) -> None:
    """Measurement helper: stream n_tiles tiles of rd KB read and wr KB written, depth tiles per
    wave and pass, `blocks` workgroups (0: the library's default) (see the C header)."""
    _dev_check(src, dst)
    if src.numel() * src.element_size() < n_tiles * 1024 * rd or dst.numel() * dst.element_size() < max(16, n_tiles * 1024 * wr):
        raise ValueError("qlora_stream_probe: buffers too small for n_tiles")
    _check(lib.qlora_stream_probe(rd, wr, depth, blocks, _ptr(src), _ptr(dst), n_tiles, _stream(src.device)),
           "qlora_stream_probe")


def qlora_grad_sum(parts, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """out = parts[0] + ... + parts[k-1] (bf16, float32 sum in order, one rounding)."""
    parts = list(parts)
    _dev_check(*parts, out)
    if out is None:
        out = torch.empty_like(parts[0])
    n = _same(*parts, out)
    arr = (ctypes.c_void_p * len(parts))(*[p.data_ptr() for p in parts])
    _check(lib.qlora_grad_sum(arr, len(parts), n, _ptr(out), _stream(out.device)), "qlora_grad_sum")
    return out


# ---------------------------------------------------------------------------
# Norms before and after a block, with its gate and residual scale
# ---------------------------------------------------------------------------

_STREAM_TYPES = {torch.float32: QLORA_F32, torch.bfloat16: QLORA_BF16}


def _stream_type(t: torch.Tensor) -> int:
    if t.dim() != 2 or t.dtype not in _STREAM_TYPES:
        raise ValueError("the residual stream is a [rows][width] float32 or bf16 tensor")
    return _STREAM_TYPES[t.dtype]


def qlora_norm_fwd(R: torch.Tensor, Y: Optional[torch.Tensor] = None, w_pre: Optional[torch.Tensor] = None,
                   w_post: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, alpha: float = 1.0,
                   eps: float = 1e-6, R_out: Optional[torch.Tensor] = None, N: Optional[torch.Tensor] = None,
                   rstd_pre: Optional[torch.Tensor] = None, rstd_post: Optional[torch.Tensor] = None):
    """R_out = R + alpha * gate * u with u = Y or RMS norm(Y) * w_post, and
    N = RMS norm(R_out) * w_pre -> (R_out, N, rstd_pre, rstd_post).  Without Y (the norm
    before the first block) R_out is R; without w_pre N and rstd_pre are None."""
    dt = _stream_type(R)
    M, h = R.shape
    dev = R.device
    if Y is None:
        R_out = R if R_out is None else R_out
    elif R_out is None:
        R_out = torch.empty_like(R)
    if w_pre is not None:
        N = torch.empty(M, h, dtype=torch.bfloat16, device=dev) if N is None else N
        rstd_pre = torch.empty(M, dtype=torch.float32, device=dev) if rstd_pre is None else rstd_pre
    if w_post is not None and rstd_post is None:
        rstd_post = torch.empty(M, dtype=torch.float32, device=dev)
    rows, cols, one, bf, f32 = (M, h), (h,), (M,), torch.bfloat16, torch.float32
    _want("R", R, R.dtype, rows, dev)
    _want("R_out", R_out, R.dtype, rows, dev)
    _want("Y", Y, bf, rows, dev)
    _want("N", N, bf, rows, dev)
    _want("w_pre", w_pre, f32, cols, dev)
    _want("w_post", w_post, f32, cols, dev)
    _want("gate", gate, f32, cols, dev)
    _want("rstd_pre", rstd_pre, f32, one, dev)
    _want("rstd_post", rstd_post, f32, one, dev)
    _call(dev, "qlora_norm_fwd", _at(R), dt, _at(Y), _at(w_post), _at(gate), float(alpha), _at(w_pre),
          float(eps), M, h, _at(R_out), _at(N), _at(rstd_post), _at(rstd_pre))
    return R_out, N, rstd_pre, rstd_post


def qlora_norm_bwd(dN: Optional[torch.Tensor], dR_out: Optional[torch.Tensor], R_out: Optional[torch.Tensor],
                   Y: Optional[torch.Tensor] = None, rstd_pre: Optional[torch.Tensor] = None,
                   rstd_post: Optional[torch.Tensor] = None, w_pre: Optional[torch.Tensor] = None,
                   w_post: Optional[torch.Tensor] = None, gate: Optional[torch.Tensor] = None, alpha: float = 1.0,
                   weight_grads: bool = False, block: bool = True, dR: Optional[torch.Tensor] = None,
                   dY: Optional[torch.Tensor] = None, dw_pre: Optional[torch.Tensor] = None,
                   dw_post: Optional[torch.Tensor] = None, dgate: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None):
    """Backward of qlora_norm_fwd for the gradients dN of N and dR_out of R_out ->
    (dR, dY, dw_pre, dw_post, dgate).  `block` False: the forward had no Y (dY is None).
    `weight_grads`: allocate the gradient of every weight given (or pass the wanted
    buffers); the others are None."""
    like = R_out if R_out is not None else dR_out
    if like is None:
        raise ValueError("qlora_norm_bwd needs R_out or dR_out")
    dt = _stream_type(like)
    M, h = like.shape
    dev = like.device
    dR = torch.empty_like(like) if dR is None else dR
    if block and dY is None:
        dY = torch.empty(M, h, dtype=torch.bfloat16, device=dev)
    if weight_grads:
        new = lambda w, d: torch.empty(h, dtype=torch.float32, device=dev) if w is not None and d is None else d
        dw_pre, dw_post, dgate = new(w_pre, dw_pre), new(w_post, dw_post), new(gate, dgate)
    sums = dw_pre is not None or dw_post is not None or dgate is not None
    if sums and workspace is None:
        workspace = torch.empty(workspace_size(QLORA_OP_NORM_BWD, M, h), dtype=torch.uint8, device=dev)
    for name, t, dtype, shape in (("dN", dN, torch.bfloat16, (M, h)), ("dR_out", dR_out, like.dtype, (M, h)),
                                  ("R_out", R_out, like.dtype, (M, h)), ("Y", Y, torch.bfloat16, (M, h)),
                                  ("rstd_pre", rstd_pre, torch.float32, (M,)),
                                  ("rstd_post", rstd_post, torch.float32, (M,)),
                                  ("w_pre", w_pre, torch.float32, (h,)), ("w_post", w_post, torch.float32, (h,)),
                                  ("gate", gate, torch.float32, (h,)), ("dR", dR, like.dtype, (M, h)),
                                  ("dY", dY, torch.bfloat16, (M, h)), ("dw_pre", dw_pre, torch.float32, (h,)),
                                  ("dw_post", dw_post, torch.float32, (h,)), ("dgate", dgate, torch.float32, (h,)),
                                  ("workspace", workspace, torch.uint8,
                                   () if workspace is None else (workspace.numel(),))):
        _want(name, t, dtype, shape, dev)
    _call(dev, "qlora_norm_bwd", _at(dN), _at(dR_out), dt, _at(R_out), _at(Y if block else None),
          _at(rstd_post), _at(rstd_pre), _at(w_post), _at(gate), float(alpha), _at(w_pre), M, h, _at(dR),
          _at(dY), _at(dw_pre), _at(dw_post), _at(dgate), _at(workspace),
          0 if workspace is None else workspace.numel())
    return dR, dY, dw_pre, dw_post, dgate


# ---------------------------------------------------------------------------
# Cross entropy of an output head, without kept logits
# ---------------------------------------------------------------------------

def _workspace(op: int, given: Optional[torch.Tensor], device, *sizes) -> torch.Tensor:
    if given is None:
        return torch.empty(workspace_size(op, *sizes), dtype=torch.uint8, device=device)
    _want("workspace", given, torch.uint8, (given.numel(),), device)
    return given


def _head_shapes(H: torch.Tensor, W: torch.Tensor):
    if H.dim() != 2 or W.dim() != 2 or H.shape[1] != W.shape[1]:
        raise ValueError("hidden states [tokens][h] and a head [vocabulary][h] are wanted")
    return H.shape[0], H.shape[1], W.shape[0]


def qlora_loss_fwd(H: torch.Tensor, W: torch.Tensor, labels: torch.Tensor, loss: Optional[torch.Tensor] = None,
                   lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """Cross entropy of softmax(H·W^T) with `labels` per token -> (loss f32 [M], lse f32 [M]).
    Tokens whose label is outside [0, V) carry none (both 0)."""
    M, h, V = _head_shapes(H, W)
    dev = H.device
    loss = torch.empty(M, dtype=torch.float32, device=dev) if loss is None else loss
    lse = torch.empty(M, dtype=torch.float32, device=dev) if lse is None else lse
    for name, t, dtype, shape in (("H", H, torch.bfloat16, (M, h)), ("W", W, torch.bfloat16, (V, h)),
                                  ("labels", labels, torch.int64, (M,)), ("loss", loss, torch.float32, (M,)),
                                  ("lse", lse, torch.float32, (M,))):
        _want(name, t, dtype, shape, dev)
    ws = _workspace(QLORA_OP_LOSS_FWD, workspace, dev, M, h, V)
    _call(dev, "qlora_loss_fwd", _at(H), _at(W), _at(labels), M, h, V, _at(loss), _at(lse), _at(ws), ws.numel())
    return loss, lse


def qlora_loss_bwd(H: torch.Tensor, W: torch.Tensor, labels: torch.Tensor, lse: torch.Tensor, dloss: torch.Tensor,
                   train_head: bool = False, dH: Optional[torch.Tensor] = None, dW: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None):
    """Gradients of qlora_loss_fwd for the gradient `dloss` of each token's loss ->
    (dH bf16 [M][h], dW bf16 [V][h], or None for a frozen head)."""
    M, h, V = _head_shapes(H, W)
    dev = H.device
    dH = torch.empty(M, h, dtype=torch.bfloat16, device=dev) if dH is None else dH
    if train_head and dW is None:
        dW = torch.empty(V, h, dtype=torch.bfloat16, device=dev)
    for name, t, dtype, shape in (("H", H, torch.bfloat16, (M, h)), ("W", W, torch.bfloat16, (V, h)),
                                  ("labels", labels, torch.int64, (M,)), ("lse", lse, torch.float32, (M,)),
                                  ("dloss", dloss, torch.float32, (M,)), ("dH", dH, torch.bfloat16, (M, h)),
                                  ("dW", dW, torch.bfloat16, (V, h))):
        _want(name, t, dtype, shape, dev)
    ws = _workspace(QLORA_OP_LOSS_BWD, workspace, dev, M, h, V)
    _call(dev, "qlora_loss_bwd", _at(H), _at(W), _at(labels), _at(lse), _at(dloss), M, h, V, _at(dH), _at(dW),
          _at(ws), ws.numel())
    return dH, dW


# ---------------------------------------------------------------------------
# Dropout from a counter-based generator
# ---------------------------------------------------------------------------

def _rng_state(rng: torch.Tensor, device):
    _want("rng", rng, torch.int64, (2,), device)
    return rng.data_ptr()


def qlora_dropout(x: torch.Tensor, p: float, rng: torch.Tensor, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Inverted dropout of a float32 or bf16 tensor with probability p.  `rng` is an int64
    GPU tensor {seed, offset}; the same state makes the same decisions (the backward is the
    same call on the gradient), and the next use takes an offset ceil(x.numel() / 8) further."""
    if x.dtype not in _STREAM_TYPES:
        raise ValueError("x is float32 or bf16")
    out = torch.empty_like(x) if out is None else out
    _want("x", x, x.dtype, x.shape, x.device)
    _want("out", out, x.dtype, x.shape, x.device)
    _call(x.device, "qlora_dropout", _at(x), _STREAM_TYPES[x.dtype], x.numel(), float(p), _rng_state(rng, x.device),
          _at(out))
    return out


def _drop_check(W: NF4Weight, X, T, dY, L1, L2, outs):
    """Shapes of a linear with dropout; returns (M, r, device)."""
    dev = X.device
    if X.dim() != 2 or L1 is not None and (L2 is None or L1.dim() != 2):
        raise ValueError("X [tokens][h] and factors L1 [h][r], L2 [r][o] are wanted")
    M, r = X.shape[0], 0 if L1 is None else L1.shape[1]
    bf = torch.bfloat16
    for name, t, dtype, shape in (("X", X, bf, (M, W.h)), ("T", T, bf, (M, r)), ("dY", dY, bf, (M, W.o)),
                                  ("L1", L1, bf, (W.h, r)), ("L2", L2, bf, (r, W.o)),
                                  ("codes", W.codes, torch.uint8, (W.h * W.o // 2,))) + outs(M, r):
        _want(name, t, dtype, shape, dev)
    W.check(dev)
    return M, r, dev


def _drop_workspace(given, dev, M, W, r):
    """The workspace, which the caller holds until its call is enqueued, or None where none is needed."""
    if given is None:
        size = workspace_size(QLORA_OP_LINEAR_DROPOUT, M, W.h, W.o, r)
        return torch.empty(size, dtype=torch.uint8, device=dev) if size else None
    _want("workspace", given, torch.uint8, (given.numel(),), dev)
    return given


def qlora_linear_fwd_dropout(W: NF4Weight, X: torch.Tensor, L1: Optional[torch.Tensor], L2: Optional[torch.Tensor],
                             s: float, p: float, rng: torch.Tensor, Y: Optional[torch.Tensor] = None,
                             T: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None):
    """The linear with dropout on its adapter's input: T = (keep * X)·L1,
    Y = X·W_hat + s / (1 - p)·T·L2 -> (Y bf16 [M][o], T bf16 [M][r] or None)."""
    M, r, dev = _drop_check(W, X, T, None, L1, L2, lambda M, r: (("Y", Y, torch.bfloat16, (M, W.o)),))
    Y = torch.empty(M, W.o, dtype=torch.bfloat16, device=dev) if Y is None else Y
    T = torch.empty(M, r, dtype=torch.bfloat16, device=dev) if T is None and r else T
    ws = _drop_workspace(workspace, dev, M, W, r)
    _call(dev, "qlora_linear_fwd_dropout", ctypes.byref(W.as_ctypes()), W.codebook, _at(X), M, _at(L1), _at(L2), r,
          float(s), float(p), _rng_state(rng, dev), _at(Y), _at(T), _at(ws), 0 if ws is None else ws.numel())
    return Y, T


def qlora_linear_bwd_dropout(W: NF4Weight, X: torch.Tensor, T: Optional[torch.Tensor], dY: torch.Tensor,
                             L1: Optional[torch.Tensor], L2: Optional[torch.Tensor], s: float, p: float,
                             rng: torch.Tensor, dX: Optional[torch.Tensor] = None,
                             dL1: Optional[torch.Tensor] = None, dL2: Optional[torch.Tensor] = None,
                             workspace: Optional[torch.Tensor] = None):
    """Backward of qlora_linear_fwd_dropout at the same generator state ->
    (dX bf16 [M][h], dL1 f32 [h][r], dL2 f32 [r][o])."""
    M, r, dev = _drop_check(W, X, T, dY, L1, L2, lambda M, r: (
        ("dX", dX, torch.bfloat16, (M, W.h)), ("dL1", dL1, torch.float32, (W.h, r)),
        ("dL2", dL2, torch.float32, (r, W.o))))
    dX = torch.empty(M, W.h, dtype=torch.bfloat16, device=dev) if dX is None else dX
    if r:
        dL1 = torch.empty(W.h, r, dtype=torch.float32, device=dev) if dL1 is None else dL1
        dL2 = torch.empty(r, W.o, dtype=torch.float32, device=dev) if dL2 is None else dL2
    ws = _drop_workspace(workspace, dev, M, W, r)
    _call(dev, "qlora_linear_bwd_dropout", ctypes.byref(W.as_ctypes()), W.codebook, _at(X), _at(T), _at(dY), M,
          _at(L1), _at(L2), r, float(s), float(p), _rng_state(rng, dev), _at(dX), _at(dL1), _at(dL2),
          _at(ws), 0 if ws is None else ws.numel())
    return dX, dL1, dL2
