"""MI355X (gfx950) QLoRA frozen-base linear layer: blockwise NF4 quantization
with double quantization, and the LoRA forward / backward on the 4-bit base.

The functions below carry the names of the C ABI (include/qlora_nf4.h) and do
argument marshalling only: every step runs in the HIP library
libqlora_nf4.so. torch supplies device memory and the current stream.
Importing this package fails if the library has not been built.
"""

import ctypes
import functools
from dataclasses import dataclass

import torch
from torch.autograd.graph import increment_version

from . import _lib

lib = _lib.load()

__all__ = [
    "NF4Weight",
    "QLoraError",
    "nf4_quantize",
    "nf4_double_quant",
    "nf4_dequantize",
    "qlora_merge",
    "q4_quant_error",
    "qlora_linear_fwd",
    "qlora_linear_fwd_group",
    "qlora_linear_bwd",
    "qlora_linear_bwd_group",
    "quantize_weight",
    "Act8",
    "act8_quantize",
    "act8_dequantize",
    "swiglu_fwd",
    "swiglu_bwd",
    "qlora_linear_bwd_act8",
    "qlora_linear_bwd_group_act8",
    "Q4GWeight",
    "q4g_quantize",
    "q4g_dequantize",
    "q4g_linear_fwd",
    "QLoRALinearFunction",
    "QLoRAGroupFunction",
    "QLoRAGroupAct8Function",
    "SwiGLUFunction",
    "KernelTimer",
    "lib",
]

BLOCKSIZE = 64
DQ_BLOCKSIZE = 256


class QLoraError(RuntimeError):
    def __init__(self, status, message):
        super().__init__("%s (%d): %s" % (lib.qlora_status_string(status).decode(), status, message))
        self.status = status


def _check(status):
    if status != _lib.QL_OK:
        raise QLoraError(status, lib.qlora_last_error().decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream():
    return ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)


def _bits(t):
    """bf16 tensor -> its storage (the library takes bf16 as raw 16-bit)."""
    if t is None:
        return None
    assert t.dtype == torch.bfloat16 and t.is_contiguous(), "expected a contiguous bf16 tensor"
    return t


def _workspace(nbytes, device):
    if nbytes == 0:
        return None, 0
    return torch.empty(nbytes, dtype=torch.uint8, device=device), nbytes


@dataclass
class NF4Weight:
    """A frozen weight in NF4 (+ double-quantized constants) on the device."""

    rows: int
    cols: int
    packed: torch.Tensor
    absmax: torch.Tensor = None  # fp32 [nblocks]; kept when double_quant=False
    c8: torch.Tensor = None  # uint8 [nblocks]
    dq_scale: torch.Tensor = None  # fp32 [ngroups]
    dq_mean: torch.Tensor = None  # fp32 [1]

    @property
    def double_quant(self):
        return self.c8 is not None

    @property
    def shape(self):
        return (self.rows, self.cols)

    def nbytes(self):
        n = self.packed.numel()
        if self.double_quant:
            n += self.c8.numel() + 4 * self.dq_scale.numel() + 4
        else:
            n += 4 * self.absmax.numel()
        return n

    def descriptor(self):
        d = _lib.QlNf4Weight()
        d.rows = self.rows
        d.cols = self.cols
        d.blocksize = BLOCKSIZE
        d.dq_blocksize = DQ_BLOCKSIZE if self.double_quant else 0
        d.packed = self.packed.data_ptr()
        d.absmax = self.absmax.data_ptr() if self.absmax is not None else None
        d.c8 = self.c8.data_ptr() if self.double_quant else None
        d.dq_scale = self.dq_scale.data_ptr() if self.double_quant else None
        d.dq_mean = self.dq_mean.data_ptr() if self.double_quant else None
        return d


def nf4_quantize(W, packed=None, absmax=None):
    """First-level NF4 quantization of a 2-D fp32/bf16 device tensor.
    Returns (packed uint8 [ceil(n/2)], absmax fp32 [ceil(n/64)])."""
    assert W.is_cuda and W.dim() == 2 and W.is_contiguous()
    rows, cols = W.shape
    dtype = {torch.float32: _lib.QL_F32, torch.bfloat16: _lib.QL_BF16}[W.dtype]
    if packed is None:
        packed = torch.empty(lib.nf4_packed_bytes(rows, cols), dtype=torch.uint8, device=W.device)
    if absmax is None:
        absmax = torch.empty(lib.nf4_num_blocks(rows, cols, BLOCKSIZE), dtype=torch.float32, device=W.device)
    _check(lib.nf4_quantize(_ptr(W), dtype, rows, cols, BLOCKSIZE, _ptr(packed), _ptr(absmax), _stream()))
    return packed, absmax


def nf4_double_quant(absmax):
    """Second-level quantization of the fp32 absmax constants.
    Returns (c8 uint8 [n1], scale fp32 [ceil(n1/256)], mean fp32 [1])."""
    n1 = absmax.numel()
    dev = absmax.device
    c8 = torch.empty(n1, dtype=torch.uint8, device=dev)
    scale = torch.empty(lib.nf4_dq_num_groups(n1, DQ_BLOCKSIZE), dtype=torch.float32, device=dev)
    mean = torch.empty(1, dtype=torch.float32, device=dev)
    ws, wsb = _workspace(lib.nf4_double_quant_workspace(n1), dev)
    _check(
        lib.nf4_double_quant(_ptr(absmax), n1, DQ_BLOCKSIZE, _ptr(c8), _ptr(scale), _ptr(mean), _ptr(ws), wsb, _stream())
    )
    return c8, scale, mean


def nf4_quantize_dq(W):
    """nf4_quantize and nf4_double_quant in one call (two launches where the
    size allows). Returns (packed, absmax, c8, scale, mean)."""
    assert W.is_cuda and W.dim() == 2 and W.is_contiguous()
    rows, cols = W.shape
    dtype = {torch.float32: _lib.QL_F32, torch.bfloat16: _lib.QL_BF16}[W.dtype]
    dev = W.device
    n1 = lib.nf4_num_blocks(rows, cols, BLOCKSIZE)
    packed = torch.empty(lib.nf4_packed_bytes(rows, cols), dtype=torch.uint8, device=dev)
    absmax = torch.empty(n1, dtype=torch.float32, device=dev)
    c8 = torch.empty(n1, dtype=torch.uint8, device=dev)
    scale = torch.empty(lib.nf4_dq_num_groups(n1, DQ_BLOCKSIZE), dtype=torch.float32, device=dev)
    mean = torch.empty(1, dtype=torch.float32, device=dev)
    ws, wsb = _workspace(lib.nf4_quantize_dq_workspace(rows, cols, dtype), dev)
    _check(lib.nf4_quantize_dq(_ptr(W), dtype, rows, cols, BLOCKSIZE, _ptr(packed), _ptr(absmax), DQ_BLOCKSIZE,
                               _ptr(c8), _ptr(scale), _ptr(mean), _ptr(ws), wsb, _stream()))
    return packed, absmax, c8, scale, mean


def quantize_weight(W, double_quant=True, keep_absmax=False):
    """nf4_quantize_dq (or nf4_quantize alone) into an NF4Weight."""
    if not double_quant:
        packed, absmax = nf4_quantize(W)
        return NF4Weight(W.shape[0], W.shape[1], packed, absmax=absmax)
    packed, absmax, c8, scale, mean = nf4_quantize_dq(W)
    return NF4Weight(W.shape[0], W.shape[1], packed, absmax=absmax if keep_absmax else None, c8=c8, dq_scale=scale,
                     dq_mean=mean)


def nf4_dequantize(w, dtype=torch.bfloat16, out=None):
    """Expand an NF4Weight to a [rows, cols] bf16 (or fp32) device tensor."""
    od = {torch.float32: _lib.QL_F32, torch.bfloat16: _lib.QL_BF16}[dtype]
    if out is None:
        out = torch.empty(w.rows, w.cols, dtype=dtype, device=w.packed.device)
    d = w.descriptor()
    _check(lib.nf4_dequantize(ctypes.byref(d), _ptr(out), od, _stream()))
    return out


def qlora_merge(w, A=None, B=None, scale=1.0, out=None):
    """bf16 [rows, cols] = dequant(W) + scale * B @ A (one rounding to bf16)."""
    r = 0 if A is None else A.shape[0]
    if out is None:
        out = torch.empty(w.rows, w.cols, dtype=torch.bfloat16, device=w.packed.device)
    d = w.descriptor()
    _check(lib.qlora_merge(ctypes.byref(d), _ptr(_bits(A)), _ptr(_bits(B)), r, float(scale), _ptr(out), _stream()))
    return out


def q4_quant_error(W, grid="nf4", stats=None):
    """Blockwise-absmax 4-bit quantization error of W (fp32 or bf16, 2-D) on
    the NF4 or the uniform grid: fp64 device tensor [sum (w-w')^2, sum w^2,
    max |w-w'|]."""
    dt = {torch.float32: _lib.QL_F32, torch.bfloat16: _lib.QL_BF16}[W.dtype]
    g = {"nf4": _lib.QL_GRID_NF4, "uniform": _lib.QL_GRID_UNIFORM}[grid]
    assert W.is_contiguous()
    rows, cols = (W.shape[0], W.numel() // W.shape[0]) if W.dim() >= 1 and W.shape[0] > 0 else (0, 0)
    if stats is None:
        stats = torch.empty(3, dtype=torch.float64, device=W.device)
    ws, wsb = _workspace(lib.q4_quant_error_workspace(rows, cols, dt), W.device)
    _check(lib.q4_quant_error(_ptr(W), dt, rows, cols, BLOCKSIZE, g, _ptr(stats), _ptr(ws), wsb, _stream()))
    return stats


def _keep(keep, T, K):
    assert keep.dtype == torch.uint8 and keep.is_contiguous() and keep.numel() == T * (K // 8), \
        "keep: bit-packed uint8 [T, K/8]"
    return keep


def qlora_linear_fwd(w, X, A=None, B=None, scale=1.0, save_u=True, out=None, keep=None, p=0.0):
    """Y = X W'^T + scale (X A^T) B^T. Returns (Y bf16 [T, N], U fp32 [T, r] or None).
    With ``keep`` (bit-packed uint8 [T, K/8]) and ``p``: dropout on the
    adapter input, U = (X * keep) A^T / (1 - p)."""
    T = X.shape[0]
    r = 0 if A is None else A.shape[0]
    dev = X.device
    Y = out if out is not None else torch.empty(T, w.rows, dtype=torch.bfloat16, device=dev)
    U = torch.empty(T, r, dtype=torch.float32, device=dev) if (save_u and r > 0) else None
    d = w.descriptor()
    if keep is None:
        ws, wsb = _workspace(lib.qlora_linear_fwd_workspace(w.rows, w.cols, max(T, 1), r), dev)
        _check(
            lib.qlora_linear_fwd(ctypes.byref(d), _ptr(_bits(X)), T, _ptr(_bits(A)), _ptr(_bits(B)), r, float(scale),
                                 _ptr(Y), _ptr(U), _ptr(ws), wsb, _stream())
        )
    else:
        ws, wsb = _workspace(lib.qlora_linear_fwd_dropout_workspace(w.rows, w.cols, max(T, 1), r), dev)
        _check(
            lib.qlora_linear_fwd_dropout(ctypes.byref(d), _ptr(_bits(X)), T, _ptr(_bits(A)), _ptr(_bits(B)), r,
                                         float(scale), _ptr(_keep(keep, T, w.cols)), float(p), _ptr(Y), _ptr(U),
                                         _ptr(ws), wsb, _stream())
        )
    return Y, U


def qlora_linear_fwd_noalloc(w, X, A=None, B=None, scale=1.0, save_u=True, out=None, U_out=None):
    """qlora_linear_fwd through the entry point that allocates nothing (its
    scratch is a device array of the library, shared by every call on a GPU).
    Pass ``out`` (and ``U_out``) to keep this function from allocating the
    outputs as well. Returns (Y, U or None)."""
    T = X.shape[0]
    r = 0 if A is None else A.shape[0]
    dev = X.device
    Y = out if out is not None else torch.empty(T, w.rows, dtype=torch.bfloat16, device=dev)
    U = U_out
    if U is None and save_u and r > 0:
        U = torch.empty(T, r, dtype=torch.float32, device=dev)
    d = w.descriptor()
    _check(lib.qlora_linear_fwd_noalloc(ctypes.byref(d), _ptr(_bits(X)), T, _ptr(_bits(A)), _ptr(_bits(B)), r,
                                        float(scale), _ptr(Y), _ptr(U), _stream()))
    return Y, U


def qlora_linear_fwd_group(ws, X, As=None, Bs=None, scale=1.0, save_u=True):
    """qlora_linear_fwd for up to four layers that read the same X (q/k/v,
    gate/up): one launch when T <= 16. ``ws`` NF4Weights sharing ``cols``;
    ``As``/``Bs`` lists of adapters (None for r = 0). Returns a list of
    (Y, U) pairs, as qlora_linear_fwd."""
    nw = len(ws)
    T = X.shape[0]
    r = 0 if As is None else As[0].shape[0]
    dev = X.device
    Ys = [torch.empty(T, w.rows, dtype=torch.bfloat16, device=dev) for w in ws]
    Us = [torch.empty(T, r, dtype=torch.float32, device=dev) if (save_u and r > 0) else None for _ in ws]
    descs = [w.descriptor() for w in ws]
    arr = lambda ts: (ctypes.c_void_p * max(nw, 1))(*[_ptr(t) for t in ts])
    wp = (ctypes.c_void_p * max(nw, 1))(*[ctypes.addressof(d) for d in descs])
    rows = (ctypes.c_int64 * max(nw, 1))(*[w.rows for w in ws])
    cols = ws[0].cols if nw else 0
    ws_, wsb = _workspace(lib.qlora_linear_fwd_group_workspace(rows, nw, cols, max(T, 1), r), dev)
    As_ = arr([_bits(a) for a in As]) if As is not None else None
    Bs_ = arr([_bits(b) for b in Bs]) if Bs is not None else None
    _check(
        lib.qlora_linear_fwd_group(wp, nw, _ptr(_bits(X)), T, As_, Bs_, r, float(scale), arr(Ys), arr(Us), _ptr(ws_),
                                   wsb, _stream())
    )
    return list(zip(Ys, Us))


def qlora_linear_bwd(w, X, dY, A=None, B=None, scale=1.0, U=None, need_dx=True, need_da=True, need_db=True, dA=None,
                     dB=None, accumulate=False, keep=None, p=0.0):
    """Returns (dX bf16 [T, K] or None, dA fp32 [r, K] or None, dB fp32 [N, r] or None).
    ``keep`` / ``p``: the forward's dropout mask and probability."""
    T = dY.shape[0]
    r = 0 if A is None else A.shape[0]
    dev = dY.device
    dX = torch.empty(T, w.cols, dtype=torch.bfloat16, device=dev) if need_dx else None
    if r > 0 and need_da and dA is None:
        dA = (torch.zeros if accumulate else torch.empty)(r, w.cols, dtype=torch.float32, device=dev)
    if r > 0 and need_db and dB is None:
        dB = (torch.zeros if accumulate else torch.empty)(w.rows, r, dtype=torch.float32, device=dev)
    if not need_da:
        dA = None
    if not need_db:
        dB = None
    d = w.descriptor()
    if keep is None:
        ws, wsb = _workspace(lib.qlora_linear_bwd_workspace(w.rows, w.cols, max(T, 1), r), dev)
        _check(
            lib.qlora_linear_bwd(ctypes.byref(d), _ptr(_bits(X)), _ptr(_bits(dY)), T, _ptr(_bits(A)), _ptr(_bits(B)),
                                 r, float(scale), _ptr(U), _ptr(dX), _ptr(dA), _ptr(dB), 1 if accumulate else 0,
                                 _ptr(ws), wsb, _stream())
        )
    else:
        ws, wsb = _workspace(lib.qlora_linear_bwd_dropout_workspace(w.rows, w.cols, max(T, 1), r), dev)
        _check(
            lib.qlora_linear_bwd_dropout(ctypes.byref(d), _ptr(_bits(X)), _ptr(_bits(dY)), T, _ptr(_bits(A)),
                                         _ptr(_bits(B)), r, float(scale), _ptr(_keep(keep, T, w.cols)), float(p),
                                         _ptr(U), _ptr(dX), _ptr(dA), _ptr(dB), 1 if accumulate else 0, _ptr(ws), wsb,
                                         _stream())
        )
    return dX, dA, dB


def qlora_linear_bwd_group(ws, X, dYs, As=None, Bs=None, scale=1.0, Us=None, need_dx=True, need_da=True,
                           need_db=True, dAs=None, dBs=None, accumulate=False):
    """qlora_linear_bwd for up to four layers that read the same X (q/k/v,
    gate/up). Returns (dX bf16 [T, K] = the sum of the layers' input
    gradients, or None; list of dA or None; list of dB or None). ``ws``
    NF4Weights sharing ``cols``; ``dYs`` their upstream gradients; ``As``,
    ``Bs``, ``Us`` lists per layer (None for r = 0 / no saved U)."""
    nw = len(ws)
    T = dYs[0].shape[0]
    r = 0 if As is None else As[0].shape[0]
    dev = dYs[0].device
    cols = ws[0].cols if nw else 0
    dX = torch.empty(T, cols, dtype=torch.bfloat16, device=dev) if need_dx else None
    new = torch.zeros if accumulate else torch.empty
    if r > 0 and need_da and dAs is None:
        dAs = [new(r, cols, dtype=torch.float32, device=dev) for _ in ws]
    if r > 0 and need_db and dBs is None:
        dBs = [new(w.rows, r, dtype=torch.float32, device=dev) for w in ws]
    if not need_da:
        dAs = None
    if not need_db:
        dBs = None
    descs = [w.descriptor() for w in ws]
    arr = lambda ts: (ctypes.c_void_p * max(nw, 1))(*[_ptr(t) for t in ts]) if ts is not None else None
    wp = (ctypes.c_void_p * max(nw, 1))(*[ctypes.addressof(d) for d in descs])
    rows = (ctypes.c_int64 * max(nw, 1))(*[w.rows for w in ws])
    ws_, wsb = _workspace(lib.qlora_linear_bwd_group_workspace(rows, nw, cols, max(T, 1), r), dev)
    _check(
        lib.qlora_linear_bwd_group(wp, nw, _ptr(_bits(X)), arr([_bits(d) for d in dYs]), T,
                                   arr([_bits(a) for a in As]) if As is not None else None,
                                   arr([_bits(b) for b in Bs]) if Bs is not None else None, r, float(scale), arr(Us),
                                   _ptr(dX), arr(dAs), arr(dBs), 1 if accumulate else 0, _ptr(ws_), wsb, _stream())
    )
    return dX, dAs, dBs


# ---- 8-bit activation checkpoints ----------------------------------------
def _refuse(status, message):
    raise QLoraError(status, message)


def _tensor(t, name, dtype, shape, device=None):
    """t, checked: a contiguous device tensor of this dtype and shape (on
    ``device`` where given)."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.shape == shape and t.is_contiguous()
            and (t.is_cuda if device is None else t.device == device)):
        return t
    if not isinstance(t, torch.Tensor):
        _refuse(_lib.QL_ERR_NULL, "%s is no tensor" % name)
    if t.dtype != dtype:
        _refuse(_lib.QL_ERR_UNSUPPORTED, "%s is %s, expected %s" % (name, t.dtype, dtype))
    if t.shape != shape:
        _refuse(_lib.QL_ERR_SHAPE, "%s is %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if not t.is_contiguous():
        _refuse(_lib.QL_ERR_UNSUPPORTED, "%s is not contiguous" % name)
    _refuse(_lib.QL_ERR_UNSUPPORTED, "%s is on %s, expected %s" % (name, t.device, device or "a GPU"))


def _matrix(t, name, dtype=torch.bfloat16):
    """t, checked: a contiguous 2-D device tensor."""
    if not isinstance(t, torch.Tensor) or t.dim() != 2:
        _refuse(_lib.QL_ERR_SHAPE, "%s is not 2-D" % name)
    return _tensor(t, name, dtype, t.shape)


# The handle of a device's current stream. torch's own accessor makes a Stream
# object first: 2.8 us a call against 0.1 us, a third of a small call's time.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)


def _addr(t):
    return None if t is None else t.data_ptr()


def _launch(device, call, *args):
    """call(*args, stream) on ``device`` and its current stream."""
    if device.index == torch.cuda.current_device():
        _check(call(*args, _raw_stream(device.index)))
    else:
        with torch.cuda.device(device):
            _check(call(*args, _raw_stream(device.index)))


@dataclass
class Act8:
    """An activation in 8 bits: E4M3 codes uint8 [rows, cols] with one scale
    2^(scale - 127) per 32 values of a row, uint8 [rows, cols / 32]."""

    rows: int
    cols: int
    codes: torch.Tensor
    scale: torch.Tensor

    def nbytes(self):
        return self.codes.numel() + self.scale.numel()

    def descriptor(self):
        _tensor(self.codes, "codes", torch.uint8, (self.rows, self.cols))
        _tensor(self.scale, "scale", torch.uint8, (self.rows, self.cols // _lib.QL_ACT8_BLOCK), self.codes.device)
        return self._struct()

    def _struct(self):
        return _lib.QlAct8(self.rows, self.cols, self.codes.data_ptr(), self.scale.data_ptr())


def _act8_empty(rows, cols, device):
    if cols % _lib.QL_ACT8_BLOCK:
        _refuse(_lib.QL_ERR_SHAPE, "%d columns, not a multiple of %d" % (cols, _lib.QL_ACT8_BLOCK))
    return Act8(rows, cols, torch.empty(rows, cols, dtype=torch.uint8, device=device),
                torch.empty(rows, cols // _lib.QL_ACT8_BLOCK, dtype=torch.uint8, device=device))


def act8_quantize(X, out=None):
    """8-bit checkpoint (an Act8) of a bf16 activation [rows, cols], cols a
    multiple of 32: nearest E4M3 value under one power-of-two scale per 32
    values; NaN and infinities become NaN. ``out``: an Act8 to write into."""
    rows, cols = _matrix(X, "X").shape
    if out is None:
        a = _act8_empty(rows, cols, X.device)
        d = a._struct()
    else:
        a, d = out, out.descriptor()
        if (a.rows, a.cols) != (rows, cols) or a.codes.device != X.device:
            _refuse(_lib.QL_ERR_SHAPE, "out is %d x %d on %s, X %d x %d on %s"
                    % (a.rows, a.cols, a.codes.device, rows, cols, X.device))
    _launch(X.device, lib.act8_quantize, X.data_ptr(), d)
    if out is not None:  # a backward that kept these tensors must not take the new values for the old
        increment_version((a.codes, a.scale))
    return a


def act8_dequantize(a, dtype=torch.bfloat16, out=None):
    """The stored values of an Act8 as a bf16 or fp32 tensor (exact)."""
    if dtype not in (torch.bfloat16, torch.float32):
        _refuse(_lib.QL_ERR_UNSUPPORTED, "output dtype %s" % dtype)
    d = a.descriptor()
    dev = a.codes.device
    new = out is None
    if new:
        out = torch.empty(a.rows, a.cols, dtype=dtype, device=dev)
    else:
        _tensor(out, "out", dtype, (a.rows, a.cols), dev)
    _launch(dev, lib.act8_dequantize, d, out.data_ptr(), _lib.QL_BF16 if dtype == torch.bfloat16 else _lib.QL_F32)
    if not new:
        increment_version(out)
    return out


def swiglu_fwd(gate, up, checkpoint=True, h8=False):
    """H = gate sigmoid(gate) up (bf16 [rows, cols], cols a multiple of 32).
    Returns (H, gate8, up8, h8): the Act8 checkpoints of gate and up that
    swiglu_bwd takes (None without ``checkpoint``) and, with ``h8``, that of H
    for the down projection's backward."""
    rows, cols = _matrix(gate, "gate").shape
    dev = gate.device
    _tensor(up, "up", torch.bfloat16, (rows, cols), dev)
    H = torch.empty_like(gate)
    acts = [_act8_empty(rows, cols, dev) if want else None for want in (checkpoint, checkpoint, h8)]
    _launch(dev, lib.qlora_swiglu_fwd, gate.data_ptr(), up.data_ptr(), rows, cols, H.data_ptr(),
            *[a._struct() if a is not None else None for a in acts])
    return (H, *acts)


def swiglu_bwd(gate8, up8, dH):
    """(dgate, dup) bf16 of swiglu_fwd from its checkpoints and dH bf16."""
    dg, du = gate8.descriptor(), up8.descriptor()
    dev, shape = gate8.codes.device, (gate8.rows, gate8.cols)
    _tensor(dH, "dH", torch.bfloat16, shape, dev)
    if (up8.rows, up8.cols) != shape or up8.codes.device != dev:
        _refuse(_lib.QL_ERR_SHAPE, "up8 is %d x %d on %s, gate8 %d x %d on %s"
                % (up8.rows, up8.cols, up8.codes.device, *shape, dev))
    dgate, dup = torch.empty_like(dH), torch.empty_like(dH)
    _launch(dev, lib.qlora_swiglu_bwd, dg, du, dH.data_ptr(), dgate.data_ptr(), dup.data_ptr())
    return dgate, dup


def _adapters(A, B, rows, cols, device):
    """The rank of an adapter pair (0 when A is None), shapes checked."""
    if A is None:
        return 0
    r = A.shape[0] if isinstance(A, torch.Tensor) and A.dim() == 2 else _refuse(_lib.QL_ERR_SHAPE, "A is not 2-D")
    _tensor(A, "A", torch.bfloat16, (r, cols), device)
    _tensor(B, "B", torch.bfloat16, (rows, r), device)
    return r


def _grads(want, given, shape, name, accumulate, device):
    """The fp32 gradient to write: the caller's, a new one, or None."""
    if not want:
        return None
    if given is not None:
        _tensor(given, name, torch.float32, shape, device)
        increment_version(given)  # written through its address
        return given
    return (torch.zeros if accumulate else torch.empty)(*shape, dtype=torch.float32, device=device)


def _outputs(dX, dA, dB):
    """The QL_OUT_* of the gradients that there are."""
    return (dX is not None) * _lib.QL_OUT_DX | (dA is not None) * _lib.QL_OUT_DA | (dB is not None) * _lib.QL_OUT_DB


def qlora_linear_bwd_act8(w, X8, dY, A=None, B=None, scale=1.0, U=None, need_dx=True, need_da=True, need_db=True,
                          dA=None, dB=None, accumulate=False, keep=None, p=0.0):
    """qlora_linear_bwd with the layer's input kept as an Act8 ``X8``. ``U``
    (fp32 [T, r], from the forward) is required for dB; X8 may be None without
    dA. dA and dB use U and G = s dY B in fp32."""
    if not isinstance(dY, torch.Tensor) or dY.dim() != 2:
        _refuse(_lib.QL_ERR_SHAPE, "dY is not 2-D")
    T, dev = dY.shape[0], dY.device
    _tensor(dY, "dY", torch.bfloat16, (T, w.rows), w.packed.device)
    r = _adapters(A, B, w.rows, w.cols, dev)
    dX = torch.empty(T, w.cols, dtype=torch.bfloat16, device=dev) if need_dx else None
    dA = _grads(r > 0 and need_da, dA, (r, w.cols), "dA", accumulate, dev)
    dB = _grads(r > 0 and need_db, dB, (w.rows, r), "dB", accumulate, dev)
    if dB is not None:
        _tensor(U, "U", torch.float32, (T, r), dev)
    x8 = None
    if dA is not None:
        x8 = X8.descriptor() if X8 is not None else _refuse(_lib.QL_ERR_NULL, "X8 is None (dA needs it)")
        if (X8.rows, X8.cols) != (T, w.cols) or X8.codes.device != dev:
            _refuse(_lib.QL_ERR_SHAPE, "X8 is %d x %d on %s, expected %d x %d on %s"
                    % (X8.rows, X8.cols, X8.codes.device, T, w.cols, dev))
    if keep is not None:
        if not isinstance(keep, torch.Tensor) or keep.numel() != T * (w.cols // 8):
            _refuse(_lib.QL_ERR_SHAPE, "keep is no tensor of %d x %d bytes" % (T, w.cols // 8))
        _tensor(keep, "keep", torch.uint8, keep.shape, dev)
    ws, wsb = _workspace(lib.qlora_linear_bwd_act8_workspace_for(w.rows, w.cols, max(T, 1), r, keep is not None,
                                                                 _outputs(dX, dA, dB)), dev)
    if T == 0:  # no token: the sums are empty
        for g in (dA, dB):
            if g is not None and not accumulate:
                g.zero_()
        return dX, dA, dB
    _launch(dev, lib.qlora_linear_bwd_act8, w.descriptor(), x8, dY.data_ptr(), T, _addr(A), _addr(B), r, float(scale),
            _addr(keep), float(p), _addr(U) if dB is not None else None, _addr(dX), _addr(dA), _addr(dB),
            1 if accumulate else 0, _addr(ws), wsb)
    return dX, dA, dB


def qlora_linear_bwd_group_act8(ws, X8, dYs, As=None, Bs=None, scale=1.0, Us=None, need_dx=True, need_da=True,
                                need_db=True, dAs=None, dBs=None, accumulate=False):
    """qlora_linear_bwd_group with the shared input kept as an Act8 ``X8``.
    ``need_da`` and ``need_db`` may be lists, a layer each. Returns (dX, list
    of dA or None, list of dB or None), None in a list for a layer's that is
    not wanted."""
    nw = len(ws)
    if nw < 1 or len(dYs) != nw:
        _refuse(_lib.QL_ERR_SHAPE, "%d weights and %d dY" % (nw, len(dYs)))
    need_da, need_db = (list(n) if isinstance(n, (list, tuple)) else [n] * nw for n in (need_da, need_db))
    for name, ts in (("As", As), ("Bs", Bs), ("Us", Us), ("dAs", dAs), ("dBs", dBs), ("need_da", need_da),
                     ("need_db", need_db)):
        if ts is not None and len(ts) != nw:
            _refuse(_lib.QL_ERR_SHAPE, "%d weights and %d %s" % (nw, len(ts), name))
    T = _matrix(dYs[0], "dY").shape[0]
    dev = dYs[0].device
    cols = ws[0].cols
    r = 0
    pick = lambda ts, i: ts[i] if ts is not None else None
    for i, w in enumerate(ws):
        _tensor(dYs[i], "dY", torch.bfloat16, (T, w.rows), dev)
        if w.packed.device != dev:
            _refuse(_lib.QL_ERR_UNSUPPORTED, "weight %d is on %s, dY on %s" % (i, w.packed.device, dev))
        ri = _adapters(pick(As, i), pick(Bs, i), w.rows, cols, dev)
        if i > 0 and ri != r:
            _refuse(_lib.QL_ERR_SHAPE, "layer %d has rank %d, layer 0 rank %d" % (i, ri, r))
        r = ri
    dX = torch.empty(T, cols, dtype=torch.bfloat16, device=dev) if need_dx else None
    any_da, any_db = any(need_da) and r > 0, any(need_db) and r > 0
    dAs = [_grads(need_da[i], pick(dAs, i), (r, cols), "dA", accumulate, dev) for i in range(nw)] if any_da else None
    dBs = [_grads(need_db[i], pick(dBs, i), (w.rows, r), "dB", accumulate, dev) for i, w in enumerate(ws)] if any_db else None
    for i in range(nw):
        if any_db and need_db[i]:
            _tensor(pick(Us, i), "U", torch.float32, (T, r), dev)
    x8 = None
    if any_da:
        x8 = X8.descriptor() if X8 is not None else _refuse(_lib.QL_ERR_NULL, "X8 is None (dA needs it)")
        _tensor(X8.codes, "X8", torch.uint8, (T, cols), dev)
    if T == 0:
        for g in (dAs or []) + (dBs or []):
            if g is not None and not accumulate:
                g.zero_()
        return dX, dAs, dBs
    arr = lambda ts: (ctypes.c_void_p * nw)(*[_addr(t) for t in ts]) if ts is not None else None
    descs = [w.descriptor() for w in ws]
    wp = (ctypes.c_void_p * nw)(*[ctypes.addressof(d) for d in descs])
    rows = (ctypes.c_int64 * nw)(*[w.rows for w in ws])
    ws_, wsb = _workspace(lib.qlora_linear_bwd_group_act8_workspace_for(rows, nw, cols, T, r, _outputs(dX, dAs, dBs)),
                          dev)
    _launch(dev, lib.qlora_linear_bwd_group_act8, wp, nw, x8, arr(dYs), T, arr(As) if r > 0 else None,
            arr(Bs) if r > 0 else None, r, float(scale), arr(Us) if any_db else None, _ptr(dX), arr(dAs), arr(dBs),
            1 if accumulate else 0, _ptr(ws_), wsb)
    return dX, dAs, dBs


# ---- 4-bit weights with group scales ---------------------------------------
@dataclass
class Q4GWeight:
    """A weight in 4 bits with group scales: w' = scale (q - zero)."""

    rows: int
    cols: int
    group: int  # 32, 64 or 128 values along a row
    packed: torch.Tensor  # uint8 [rows, 16 ceil(cols / 32)]
    scale: torch.Tensor  # bf16 or fp32 [rows, ceil(cols / group)]
    zero: torch.Tensor = None  # uint8 like scale, or None: 8 throughout

    @property
    def shape(self):
        return (self.rows, self.cols)

    def nbytes(self):
        n = self.packed.numel() + self.scale.numel() * self.scale.element_size()
        return n + (self.zero.numel() if self.zero is not None else 0)

    def descriptor(self):
        rows, cols, group, packed, scale, zero = self.rows, self.cols, self.group, self.packed, self.scale, self.zero
        if group not in (32, 64, 128):
            _refuse(_lib.QL_ERR_UNSUPPORTED, "group %s (32, 64 or 128)" % (group,))
        groups = (rows, -(-cols // group))
        _tensor(packed, "packed", torch.uint8, (rows, 16 * -(-cols // 32)))
        dev = packed.device
        code = _DTYPES.get(scale.dtype) if isinstance(scale, torch.Tensor) else None
        if code is None:
            _refuse(_lib.QL_ERR_UNSUPPORTED, "scale is no bf16 or fp32 tensor")
        _tensor(scale, "scale", scale.dtype, groups, dev)
        if zero is not None:
            _tensor(zero, "zero", torch.uint8, groups, dev)
        return _lib.QlQ4GWeight(rows, cols, group, code, packed.data_ptr(), scale.data_ptr(), _addr(zero))


_DTYPES = {torch.float32: _lib.QL_F32, torch.bfloat16: _lib.QL_BF16}


def q4g_quantize(W, group=128, symmetric=False, scale_dtype=torch.bfloat16):
    """Round a 2-D fp32 or bf16 weight to 4 bits with one scale (and, unless
    ``symmetric``, one zero point) per ``group`` values of a row."""
    if not isinstance(W, torch.Tensor) or W.dtype not in _DTYPES or scale_dtype not in _DTYPES:
        _refuse(_lib.QL_ERR_UNSUPPORTED, "W and its scales are bf16 or fp32")
    rows, cols = _matrix(W, "W", W.dtype).shape
    if group not in (32, 64, 128):
        _refuse(_lib.QL_ERR_UNSUPPORTED, "group %s (32, 64 or 128)" % (group,))
    dev = W.device
    groups = (rows, -(-cols // group))
    packed = torch.empty(rows, 16 * -(-cols // 32), dtype=torch.uint8, device=dev)
    scale = torch.empty(groups, dtype=scale_dtype, device=dev)
    zero = None if symmetric else torch.empty(groups, dtype=torch.uint8, device=dev)
    _launch(dev, lib.q4g_quantize, W.data_ptr(), _DTYPES[W.dtype], rows, cols, group, packed.data_ptr(),
            scale.data_ptr(), _DTYPES[scale_dtype], zero.data_ptr() if zero is not None else None)
    return Q4GWeight(rows, cols, group, packed, scale, zero)


def q4g_dequantize(w, dtype=torch.bfloat16, out=None):
    """Expand a Q4GWeight to a [rows, cols] bf16 (or fp32) tensor."""
    if dtype not in _DTYPES:
        _refuse(_lib.QL_ERR_UNSUPPORTED, "output dtype %s" % dtype)
    d = w.descriptor()
    dev = w.packed.device
    new = out is None
    if new:
        out = torch.empty(w.rows, w.cols, dtype=dtype, device=dev)
    else:
        _tensor(out, "out", dtype, (w.rows, w.cols), dev)
    _launch(dev, lib.q4g_dequantize, d, out.data_ptr(), _DTYPES[dtype])
    if not new:
        increment_version(out)
    return out


def q4g_linear_fwd(w, X, out=None):
    """Y = X W'^T (bf16 [T, rows]) on a Q4GWeight, X bf16 [T, cols]; made for
    decoding (up to 64 tokens read the weight once)."""
    if not isinstance(X, torch.Tensor) or X.dim() != 2:
        _refuse(_lib.QL_ERR_SHAPE, "X is not 2-D")
    d = w.descriptor()
    T, dev = X.shape[0], w.packed.device
    _tensor(X, "X", torch.bfloat16, (T, w.cols), dev)
    new = out is None
    if new:
        out = torch.empty(T, w.rows, dtype=torch.bfloat16, device=dev)
    else:
        _tensor(out, "out", torch.bfloat16, (T, w.rows), dev)
    _launch(dev, lib.q4g_linear_fwd, d, X.data_ptr(), T, out.data_ptr())
    if not new:
        increment_version(out)
    return out


def paged_adamw_step(param, grad, exp_avg, exp_avg_sq, step, lr=2e-4, betas=(0.9, 0.999), eps=1e-8,
                     weight_decay=0.0, param_bf16=None, copy_stream=None):
    """One AdamW step (fp32 state) of a flat fp32 parameter tensor in place.
    ``exp_avg`` / ``exp_avg_sq``: fp32 tensors of the same size, both on the
    GPU or both in pinned host memory (``pin_memory=True``): paged-out state
    is read and written in place over the host link (pinned memory is mapped
    into the device's address space); with QLORA_NF4_ADAMW_PAGING=staged it
    streams through a device staging buffer instead, its copies on
    ``copy_stream`` (a torch.cuda.Stream; None runs them on the current
    stream).
    ``param_bf16``: optional bf16 tensor that receives the updated values."""
    n = param.numel()
    for t in (param, grad, exp_avg, exp_avg_sq):
        assert t.dtype == torch.float32 and t.is_contiguous() and t.numel() == n
    if param_bf16 is not None:
        assert param_bf16.dtype == torch.bfloat16 and param_bf16.is_contiguous() and param_bf16.numel() == n
    ws, wsb = (None, 0)
    if not exp_avg.is_cuda:
        ws, wsb = _workspace(lib.qlora_paged_adamw_workspace(n), param.device)
    cs = ctypes.c_void_p(copy_stream.cuda_stream) if copy_stream is not None else None
    _check(lib.qlora_paged_adamw(_ptr(param), _ptr(param_bf16), _ptr(grad), _ptr(exp_avg), _ptr(exp_avg_sq), n,
                                 int(step), float(lr), float(betas[0]), float(betas[1]), float(eps),
                                 float(weight_decay), _ptr(ws), wsb, _stream(), cs))
    return param


class _FirstOrderOnly(torch.autograd.Function):
    """Hands gradients on; differentiating them raises. The first ``n`` inputs
    are what the gradients depend on: autograd comes here on its way to them."""

    @staticmethod
    def forward(ctx, n, *ts):
        return tuple(t.view_as(t) for t in ts[n:])

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("the gradients from 8-bit checkpoints cannot be differentiated again")


@functools.lru_cache(None)
def _no_rows(device):
    with torch.inference_mode(False):
        return torch.empty(0, dtype=torch.int64, device=device)


def _tie(*inputs):
    """Tensors without elements (and without the inputs' memory) that depend on
    the inputs, for those that a backward does not keep."""
    with torch.enable_grad():  # 2 us each; a slice and its copy take 5
        return [t.index_select(0, _no_rows(t.device)) for t in inputs if t.requires_grad]


def _first_order_only(backward):
    """A backward whose gradients raise when they are differentiated. They come
    from a library call, constants to autograd: under create_graph a loss of
    them would lose their part without a word, also where dY is a constant."""

    @functools.wraps(backward)
    def run(ctx, *dYs):
        if not torch.is_grad_enabled():
            return backward(ctx, *dYs)
        with torch.no_grad():
            grads = backward(ctx, *dYs)
        of = [t for t in (*ctx.tie, *ctx.saved_tensors, *dYs) if t is not None and t.requires_grad]
        at = [i for i, g in enumerate(grads) if g is not None]
        grads = list(grads)
        for i, g in zip(at, _FirstOrderOnly.apply(len(of), *of, *[grads[i] for i in at])):
            grads[i] = g
        return tuple(grads)

    return run


class QLoRALinearFunction(torch.autograd.Function):
    """autograd wrapper: forward / backward run in the HIP library; W is frozen
    (no gradient), A and B receive fp32 gradients cast to their dtype.
    ``act8``: True keeps X as an 8-bit checkpoint instead of itself, an Act8
    of X (shared with other layers, or swiglu_fwd's h8) is kept as it is; dA
    then comes from the checkpoint. First order only: with ``act8`` the
    gradients raise when differentiated again, without they are constants."""

    @staticmethod
    def forward(ctx, X, A, B, w, scale, keep=None, p=0.0, act8=None):
        Y, U = qlora_linear_fwd(w, X.contiguous(), A.contiguous(), B.contiguous(), scale, save_u=True, keep=keep, p=p)
        ctx.act8 = act8 is not None and act8 is not False
        if ctx.act8:
            ctx.tie = _tie(X)
            need_a, need_b = ctx.needs_input_grad[1:3]
            if act8 is not True and (act8.rows, act8.cols) != tuple(X.shape):
                _refuse(_lib.QL_ERR_SHAPE, "act8 is %d x %d, X %s" % (act8.rows, act8.cols, tuple(X.shape)))
            X8 = None  # only dA reads it
            if need_a:
                X8 = act8_quantize(X.contiguous()) if act8 is True else act8
            ctx.save_for_backward(X8.codes if need_a else None, X8.scale if need_a else None, A, B,
                                  U if need_b else None, keep)
        else:
            ctx.save_for_backward(X, A, B, U)
        ctx.w = w
        ctx.scale = scale
        ctx.keep = keep
        ctx.p = p
        return Y

    @staticmethod
    def backward(ctx, dY):
        if ctx.act8:
            return QLoRALinearFunction._backward_act8(ctx, dY)
        X, A, B, U = ctx.saved_tensors
        dX, dA, dB = qlora_linear_bwd(ctx.w, X, dY.contiguous().to(torch.bfloat16), A, B, ctx.scale, U=U,
                                      need_dx=ctx.needs_input_grad[0], keep=ctx.keep, p=ctx.p)
        return dX, dA.to(A.dtype), dB.to(B.dtype), None, None, None, None, None

    @staticmethod
    @_first_order_only
    def _backward_act8(ctx, dY):
        codes, xs, A, B, U, keep = ctx.saved_tensors
        need = ctx.needs_input_grad
        X8 = Act8(*codes.shape, codes, xs) if need[1] else None
        dX, dA, dB = qlora_linear_bwd_act8(ctx.w, X8, dY.contiguous().to(torch.bfloat16), A.contiguous(),
                                           B.contiguous(), ctx.scale, U=U, need_dx=need[0], need_da=need[1],
                                           need_db=need[2], keep=keep, p=ctx.p)
        return (dX, dA.to(A.dtype) if need[1] else None, dB.to(B.dtype) if need[2] else None,
                None, None, None, None, None)


class QLoRAGroupFunction(torch.autograd.Function):
    """autograd wrapper for up to four layers that read the same X (q/k/v,
    gate/up): apply(X, scale, ws, A_0, B_0, A_1, B_1, ...) returns the
    layers' Y; the forward is one qlora_linear_fwd_group call, the backward
    one qlora_linear_bwd_group call (X receives the summed input gradient;
    the weights in ``ws`` are frozen)."""

    @staticmethod
    def forward(ctx, X, scale, ws, *adapters):
        As, Bs = [a.contiguous() for a in adapters[0::2]], [b.contiguous() for b in adapters[1::2]]
        outs = qlora_linear_fwd_group(ws, X.contiguous(), As, Bs, scale)
        ctx.save_for_backward(X, *As, *Bs, *[U for _, U in outs])
        ctx.ws = ws
        ctx.scale = scale
        return tuple(Y for Y, _ in outs)

    @staticmethod
    def backward(ctx, *dYs):
        n = len(ctx.ws)
        saved = ctx.saved_tensors
        X, As, Bs, Us = saved[0], list(saved[1:1 + n]), list(saved[1 + n:1 + 2 * n]), list(saved[1 + 2 * n:])
        dYs = [(d if d is not None else torch.zeros(X.shape[0], w.rows, device=X.device)).contiguous()
               .to(torch.bfloat16) for d, w in zip(dYs, ctx.ws)]
        dX, dAs, dBs = qlora_linear_bwd_group(ctx.ws, X, dYs, As, Bs, ctx.scale, Us=Us,
                                              need_dx=ctx.needs_input_grad[0])
        grads = []
        for i in range(n):
            grads += [dAs[i].to(As[i].dtype), dBs[i].to(Bs[i].dtype)]
        return (dX, None, None, *grads)


class QLoRAGroupAct8Function(torch.autograd.Function):
    """QLoRAGroupFunction with the shared X kept as one 8-bit checkpoint:
    apply(X, act8, scale, ws, A_0, B_0, A_1, B_1, ...), ``act8`` an Act8 of X
    or None to make one here. First order only."""

    @staticmethod
    def forward(ctx, X, act8, scale, ws, *adapters):
        As, Bs = [a.contiguous() for a in adapters[0::2]], [b.contiguous() for b in adapters[1::2]]
        outs = qlora_linear_fwd_group(ws, X.contiguous(), As, Bs, scale)
        if act8 is not None and (act8.rows, act8.cols) != tuple(X.shape):
            _refuse(_lib.QL_ERR_SHAPE, "act8 is %d x %d, X %s" % (act8.rows, act8.cols, tuple(X.shape)))
        need_a, need_b = ctx.needs_input_grad[4::2], ctx.needs_input_grad[5::2]
        X8 = None  # only the dA read it
        if any(need_a):
            X8 = act8 if act8 is not None else act8_quantize(X.contiguous())
        ctx.save_for_backward(X8.codes if X8 is not None else None, X8.scale if X8 is not None else None, *As, *Bs,
                              *[U if n else None for (_, U), n in zip(outs, need_b)])
        ctx.tie = _tie(X, *[a for a in adapters if not a.is_contiguous()])  # the others are kept themselves
        ctx.ws = ws
        ctx.scale = scale
        return tuple(Y for Y, _ in outs)

    @staticmethod
    @_first_order_only
    def backward(ctx, *dYs):
        n = len(ctx.ws)
        codes, xs, *rest = ctx.saved_tensors
        As, Bs, Us = rest[:n], rest[n:2 * n], rest[2 * n:]
        dYs = [d.contiguous().to(torch.bfloat16) for d in dYs]
        need = ctx.needs_input_grad
        X8 = Act8(*codes.shape, codes, xs) if codes is not None else None
        dX, dAs, dBs = qlora_linear_bwd_group_act8(ctx.ws, X8, dYs, As, Bs, ctx.scale, Us=Us, need_dx=need[0],
                                                   need_da=need[4::2], need_db=need[5::2])
        grads = []
        for i in range(n):
            grads += [dAs[i].to(As[i].dtype) if need[4 + 2 * i] else None,
                      dBs[i].to(Bs[i].dtype) if need[5 + 2 * i] else None]
        return (dX, None, None, None, *grads)


class SwiGLUFunction(torch.autograd.Function):
    """autograd wrapper of the gated activation: apply(gate, up) returns H
    and keeps gate and up as 8-bit checkpoints for the backward, where one of
    them needs a gradient. apply(gate, up, True) returns (H, h8) with H's own
    checkpoint, an Act8 for QLoRALinearFunction's ``act8`` in the down
    projection. First order only."""

    @staticmethod
    def forward(ctx, gate, up, h8=False):
        keep = any(ctx.needs_input_grad[:2])
        H, g8, u8, a8 = swiglu_fwd(gate.contiguous(), up.contiguous(), checkpoint=keep, h8=h8)
        if keep:
            ctx.save_for_backward(g8.codes, g8.scale, u8.codes, u8.scale)
            ctx.tie = _tie(gate, up)
        return (H, a8) if h8 else H

    @staticmethod
    @_first_order_only
    def backward(ctx, dH, _h8=None):
        gc, gs, uc, us = ctx.saved_tensors
        rows, cols = gc.shape
        dg, du = swiglu_bwd(Act8(rows, cols, gc, gs), Act8(rows, cols, uc, us), dH.contiguous().to(torch.bfloat16))
        need = ctx.needs_input_grad
        return dg if need[0] else None, du if need[1] else None, None


class KernelTimer:
    """HIP-event timer of one library kernel (QL_KERNEL_* id): arm(), run the
    work, read() -> (launches, total milliseconds)."""

    def __init__(self, kernel_id):
        self.kid = kernel_id

    def arm(self):
        _check(lib.qlora_timer_arm(self.kid))

    def read(self):
        n = ctypes.c_int64(0)
        ms = ctypes.c_double(0.0)
        _check(lib.qlora_timer_read(self.kid, ctypes.byref(n), ctypes.byref(ms)))
        return n.value, ms.value

    def disarm(self):
        _check(lib.qlora_timer_disarm(self.kid))
