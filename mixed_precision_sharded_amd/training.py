"""ctypes binding of the operators before the optimizer step (C ABI in
include/mps_train.h, in the same library): activations kept in 8 bits for the
backward pass, the weight gradients made from them, and the clipped policy
loss with its gradient.

Argument marshalling only, as in `binding`: the caller owns every buffer, and
each call enqueues its kernels on `stream` (default: the current stream of
the tensors' device) and returns its output.

A matrix is a 2-D CUDA tensor, float32 or bfloat16, whose rows are contiguous
(any row stride and offset).  An 8-bit activation is a pair of uint8 tensors,
codes [rows, act8_row(cols)] and scales [rows, act8_row(cols) / 32], both
contiguous (see act8_empty).  A workspace is a uint8 tensor of at least the
bytes that the operator's *_workspace_bytes states; it holds nothing between
calls.
"""
import ctypes
from typing import Optional

import torch

from . import binding
from .binding import MPS_DTYPE_BF16, MPS_DTYPE_F32, MPS_Q8_BLOCK

_P, _I64, _INT, _SIZE, _F64 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t,
                               ctypes.c_double)
_SIGNATURES = {
    "act8_save": (_P, _INT, _I64, _I64, _I64, _P, _P, _P),
    "act8_load": (_P, _P, _I64, _I64, _P, _INT, _I64, _P),
    "act8_rmsnorm": (_P, _INT, _I64, _I64, _I64, _P, _F64, _P, _I64, _P, _P, _P, _P),
    "act8_rmsnorm_backward": (_P, _INT, _I64, _P, _P, _P, _I64, _I64, _P, _P, _I64, _P, _I64, _P,
                              _INT, _P, _P, _P, _SIZE, _P),
    "act8_swiglu": (_P, _I64, _P, _I64, _INT, _I64, _I64, _P, _I64, _P, _P, _P, _P, _P),
    "act8_swiglu_backward": (_P, _INT, _I64, _P, _P, _P, _P, _I64, _I64, _P, _I64, _P, _I64, _P, _P,
                             _P),
    "act8_weight_grad": (_P, _INT, _I64, _P, _P, _I64, _I64, _I64, _P, _INT, _INT, _P, _SIZE, _P),
    "policy_loss": (_P, _INT, _I64, _I64, _I64, _P, _P, _P, _P, _P, _F64, _F64, _F64, _P, _P, _I64,
                    _P, _P, _P, _SIZE, _P),
    "token_logprobs": (_P, _INT, _I64, _I64, _I64, _P, _P, _P, _SIZE, _P),
}
_SIZES = {
    "act8_rmsnorm_backward_workspace_bytes": (_I64, _I64),
    "act8_weight_grad_workspace_bytes": (_I64, _I64, _I64),
    "policy_loss_workspace_bytes": (_I64, _I64),
}
# (library, its entry points by name), replaced as a whole: threads that come
# here for the first time at once each see one that is complete.
_bound = (object(), {})


def _function(name: str):
    """The library's entry point, with its C types."""
    global _bound
    lib = binding.lib()
    bound = _bound
    if bound[0] is not lib:
        functions = {}
        for names, restype in ((_SIGNATURES, ctypes.c_int), (_SIZES, ctypes.c_size_t)):
            for n, argtypes in names.items():
                f = getattr(lib, n)
                f.argtypes, f.restype = argtypes, restype
                functions[n] = f
        _bound = bound = (lib, functions)
    return bound[1][name]


# A call's checks cost the host about as much as its launch, so they are kept
# short: a device is its index, and the current device and stream come without
# building Python objects where torch offers that.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _enqueue(name: str, device: int, stream: Optional[torch.cuda.Stream], *args) -> None:
    """Call an entry point on `stream` with the tensors' device current."""
    if stream is None:
        handle = _raw_stream(device)
    else:
        if stream.device.index != device:
            raise ValueError(f"stream: of {stream.device}, with tensors on cuda:{device}")
        handle = stream.cuda_stream
    bound = _bound
    f = bound[1][name] if bound[0] is binding._lib else _function(name)
    if _current_device() == device:
        rc = f(*args, handle)
    else:
        with torch.cuda.device(device):
            rc = f(*args, handle)
    if rc:
        binding._check(rc, name)


def _matrix(t: torch.Tensor, name: str):
    """(C dtype, rows, cols, row stride, device) of the matrix that fixes a call's
    type, shape and device."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name}: a matrix, got {len(shape)} dimensions")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be on a CUDA device, got {t.device}")
    dtype = t.dtype
    if dtype is torch.bfloat16:
        kind = MPS_DTYPE_BF16
    elif dtype is torch.float32:
        kind = MPS_DTYPE_F32
    else:
        raise TypeError(f"{name}: expected float32 or bfloat16, got {dtype}")
    rows, cols = shape
    return kind, rows, cols, _row_stride(t, rows, cols, name), t.get_device()


def _row_stride(t: torch.Tensor, rows: int, cols: int, name: str) -> int:
    down, across = t.stride()
    if across != 1 and cols > 1 and rows:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    return down if rows > 1 else cols  # one row: its stride says nothing


def _rows(t: torch.Tensor, like: torch.Tensor, shape, name: str) -> int:
    """The row stride of a matrix of `like`'s type and device."""
    if t.dtype is not like.dtype:
        raise TypeError(f"{name}: expected {like.dtype}, got {t.dtype}")
    if t.device != like.device:
        raise ValueError(f"{name}: must be on {like.device}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected {tuple(shape)}, got {tuple(t.shape)}")
    return _row_stride(t, shape[0], shape[1], name)


def _flat(t: torch.Tensor, dtype, shape, device: int, name: str) -> int:
    """The address of a contiguous tensor of this type and shape."""
    if t.dtype is dtype and t.shape == shape and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    if t.dtype is not dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.get_device() != device:
        raise ValueError(f"{name}: must be on cuda:{device}, got {t.device}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name}: must be contiguous")


def _kept(codes: torch.Tensor, scales: torch.Tensor, rows: int, cols: int, device: int, name: str = ""):
    runs = (cols + MPS_Q8_BLOCK - 1) // MPS_Q8_BLOCK
    return (_flat(codes, torch.uint8, (rows, runs * MPS_Q8_BLOCK), device, name + "codes"),
            _flat(scales, torch.uint8, (rows, runs), device, name + "scales"))


def _workspace(t: Optional[torch.Tensor], device: int):
    if t is None:
        return None, 0
    if t.dtype is not torch.uint8 or t.get_device() != device or not t.is_contiguous():
        raise ValueError(f"workspace: contiguous uint8 tensor on cuda:{device}")
    return t.data_ptr(), t.numel()


# ------------------------------------------------------- 8-bit activations ---

def act8_row(cols: int) -> int:
    """Codes in a row of an 8-bit activation: cols rounded up to whole runs."""
    return (cols + MPS_Q8_BLOCK - 1) // MPS_Q8_BLOCK * MPS_Q8_BLOCK


def act8_empty(rows: int, cols: int, device) -> tuple:
    """(codes, scales) for an activation [rows, cols]; the contents are not set."""
    row = act8_row(cols)
    return (torch.empty(rows, row, dtype=torch.uint8, device=device),
            torch.empty(rows, row // MPS_Q8_BLOCK, dtype=torch.uint8, device=device))


def act8_save(x: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
              stream: Optional[torch.cuda.Stream] = None) -> tuple:
    """Keep the matrix x in 8 bits; returns (codes, scales)."""
    kind, rows, cols, stride, dev = _matrix(x, "x")
    _enqueue("act8_save", dev, stream, x.data_ptr(), kind, stride, rows, cols,
             *_kept(codes, scales, rows, cols, dev))
    return codes, scales


def act8_load(codes: torch.Tensor, scales: torch.Tensor, out: torch.Tensor,
              stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """The values that codes and scales stand for, in out's type."""
    kind, rows, cols, stride, dev = _matrix(out, "out")
    _enqueue("act8_load", dev, stream, *_kept(codes, scales, rows, cols, dev), rows, cols,
             out.data_ptr(), kind, stride)
    return out


def act8_rmsnorm(x: torch.Tensor, weight: torch.Tensor, eps: float, out: torch.Tensor,
                 rstd: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                 stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """out = x * rstd * weight per row, rstd = 1 / sqrt(mean(x^2) + eps) (float32,
    one per row); x is kept in codes and scales.  weight: float32."""
    kind, rows, cols, stride, dev = _matrix(x, "x")
    _enqueue("act8_rmsnorm", dev, stream, x.data_ptr(), kind, stride, rows, cols,
             _flat(weight, torch.float32, (cols,), dev, "weight"), float(eps), out.data_ptr(),
             _rows(out, x, x.shape, "out"), _flat(rstd, torch.float32, (rows,), dev, "rstd"),
             *_kept(codes, scales, rows, cols, dev))
    return out


def act8_rmsnorm_backward_workspace_bytes(rows: int, cols: int) -> int:
    return _size("act8_rmsnorm_backward_workspace_bytes", rows, cols)


def act8_rmsnorm_backward(dy: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor,
                          rstd: torch.Tensor, weight: torch.Tensor, dx: torch.Tensor,
                          dweight: torch.Tensor, workspace: Optional[torch.Tensor],
                          residual_grad: Optional[torch.Tensor] = None, accumulate: bool = False,
                          out_codes: Optional[torch.Tensor] = None,
                          out_scales: Optional[torch.Tensor] = None,
                          stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """dx and dweight (float32; added to with accumulate) of act8_rmsnorm from dy
    and the kept x and rstd; dx gets residual_grad added, and out_codes and
    out_scales, if given, the norm's output again in 8 bits."""
    kind, rows, cols, stride, dev = _matrix(dy, "dy")
    if (out_codes is None) != (out_scales is None):
        raise ValueError("out_codes and out_scales: both or neither")
    res = (None, 0) if residual_grad is None else (residual_grad.data_ptr(),
                                                   _rows(residual_grad, dy, dy.shape, "residual_grad"))
    again = (None, None) if out_codes is None else _kept(out_codes, out_scales, rows, cols, dev, "out_")
    _enqueue("act8_rmsnorm_backward", dev, stream, dy.data_ptr(), kind, stride,
             *_kept(codes, scales, rows, cols, dev), _flat(rstd, torch.float32, (rows,), dev, "rstd"),
             rows, cols, _flat(weight, torch.float32, (cols,), dev, "weight"), *res, dx.data_ptr(),
             _rows(dx, dy, dy.shape, "dx"), _flat(dweight, torch.float32, (cols,), dev, "dweight"),
             1 if accumulate else 0, *again, *_workspace(workspace, dev))
    return dx


def act8_swiglu(gate: torch.Tensor, up: torch.Tensor, out: torch.Tensor, gate_codes: torch.Tensor,
                gate_scales: torch.Tensor, up_codes: torch.Tensor, up_scales: torch.Tensor,
                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """out = gate * sigmoid(gate) * up; gate and up are kept in 8 bits."""
    kind, rows, cols, stride, dev = _matrix(gate, "gate")
    _enqueue("act8_swiglu", dev, stream, gate.data_ptr(), stride,
             up.data_ptr(), _rows(up, gate, gate.shape, "up"), kind, rows, cols, out.data_ptr(),
             _rows(out, gate, gate.shape, "out"), *_kept(gate_codes, gate_scales, rows, cols, dev, "gate_"),
             *_kept(up_codes, up_scales, rows, cols, dev, "up_"))
    return out


def act8_swiglu_backward(dout: torch.Tensor, gate_codes: torch.Tensor, gate_scales: torch.Tensor,
                         up_codes: torch.Tensor, up_scales: torch.Tensor, dgate: torch.Tensor,
                         dup: torch.Tensor, out_codes: Optional[torch.Tensor] = None,
                         out_scales: Optional[torch.Tensor] = None,
                         stream: Optional[torch.cuda.Stream] = None) -> tuple:
    """(dgate, dup) of act8_swiglu from dout and the kept gate and up; out_codes
    and out_scales, if given, get the forward output again in 8 bits."""
    kind, rows, cols, stride, dev = _matrix(dout, "dout")
    if (out_codes is None) != (out_scales is None):
        raise ValueError("out_codes and out_scales: both or neither")
    again = (None, None) if out_codes is None else _kept(out_codes, out_scales, rows, cols, dev, "out_")
    _enqueue("act8_swiglu_backward", dev, stream, dout.data_ptr(), kind,
             stride, *_kept(gate_codes, gate_scales, rows, cols, dev, "gate_"),
             *_kept(up_codes, up_scales, rows, cols, dev, "up_"), rows, cols, dgate.data_ptr(),
             _rows(dgate, dout, dout.shape, "dgate"), dup.data_ptr(), _rows(dup, dout, dout.shape, "dup"),
             *again)
    return dgate, dup


def act8_weight_grad_workspace_bytes(tokens: int, out_features: int, in_features: int) -> int:
    return _size("act8_weight_grad_workspace_bytes", tokens, out_features, in_features)


def act8_weight_grad(dy: torch.Tensor, codes: torch.Tensor, scales: torch.Tensor, dw: torch.Tensor,
                     workspace: Optional[torch.Tensor], accumulate: bool = False,
                     stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """dw[out_features, in_features] (float32 or bfloat16, contiguous; added to with
    accumulate) = dy^T x, x the kept activation [tokens, in_features]."""
    kind, tokens, n, stride, dev = _matrix(dy, "dy")
    dw_kind, _, k, _, _ = _matrix(dw, "dw")
    _enqueue("act8_weight_grad", dev, stream, dy.data_ptr(), kind, stride,
             *_kept(codes, scales, tokens, k, dev), tokens, n, k, _flat(dw, dw.dtype, (n, k), dev, "dw"),
             dw_kind, 1 if accumulate else 0, *_workspace(workspace, dev))
    return dw


# ------------------------------------------------------------- policy loss ---

def policy_loss_workspace_bytes(rows: int, vocab: int) -> int:
    return _size("policy_loss_workspace_bytes", rows, vocab)


def policy_loss(logits: torch.Tensor, labels: torch.Tensor, old_logp: torch.Tensor,
                advantage: torch.Tensor, weight: torch.Tensor, loss: torch.Tensor,
                workspace: Optional[torch.Tensor], clip_low: float = 0.2, clip_high: float = 0.2,
                ref_logp: Optional[torch.Tensor] = None, kl_coef: float = 0.0,
                dlogits: Optional[torch.Tensor] = None, token_logp: Optional[torch.Tensor] = None,
                token_kl: Optional[torch.Tensor] = None,
                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """loss[0] (float32) = the clipped policy loss over the rows of logits with its
    KL term, and with dlogits (logits' type; may be logits itself) the gradient.
    labels: int64; the other vectors float32, one value per row.  Rows with a
    label outside the vocabulary or a weight of 0 are left out."""
    kind, rows, vocab, stride, dev = _matrix(logits, "logits")

    def vector(t, name):
        return None if t is None else _flat(t, torch.float32, (rows,), dev, name)

    d = (None, 0) if dlogits is None else (dlogits.data_ptr(), _rows(dlogits, logits, logits.shape, "dlogits"))
    _enqueue("policy_loss", dev, stream, logits.data_ptr(), kind, stride,
             rows, vocab, _flat(labels, torch.int64, (rows,), dev, "labels"), vector(old_logp, "old_logp"),
             vector(ref_logp, "ref_logp"), vector(advantage, "advantage"), vector(weight, "weight"),
             float(clip_low), float(clip_high), float(kl_coef), _flat(loss, torch.float32, (1,), dev, "loss"),
             *d, vector(token_logp, "token_logp"), vector(token_kl, "token_kl"), *_workspace(workspace, dev))
    return loss


def token_logprobs(logits: torch.Tensor, labels: torch.Tensor, out: torch.Tensor,
                   workspace: Optional[torch.Tensor],
                   stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """out (float32, one per row) = logits[label] - logsumexp(logits)."""
    kind, rows, vocab, stride, dev = _matrix(logits, "logits")
    _enqueue("token_logprobs", dev, stream, logits.data_ptr(), kind,
             stride, rows, vocab,
             _flat(labels, torch.int64, (rows,), dev, "labels"), _flat(out, torch.float32, (rows,), dev, "out"),
             *_workspace(workspace, dev))
    return out


def _size(name: str, *sizes: int) -> int:
    for s in sizes:
        if not -(1 << 63) <= s < (1 << 63):
            raise ValueError(f"{name}: {sizes}")
    n = _function(name)(*sizes)
    if n == 0 and binding.last_error():
        raise binding.MpsError(-22, name, binding.last_error())
    return n
