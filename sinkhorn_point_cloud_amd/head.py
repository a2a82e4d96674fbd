"""The output end of a model on the library's HIP kernels: norm, 8-bit product, token scores.

The binding of ``include/sinkhorn_head.h``; the calls are reached through the package
itself (``sinkhorn_point_cloud_amd.token_scores`` and so on).  Their outputs are what the
losses over logits take of a frozen model: old and reference log-probabilities, a teacher's
top tokens.

Common to all: matrices [T, values] float32 or bfloat16 on the GPU (int8 for the product's
inputs); rows may lie further apart than their length (a view of padded columns), other
layouts are copied.  The work runs on the current stream of the tensors' device.  ``out``
reuses buffers; one may be an input itself where the call says so, any other overlap is
refused.  ``workspace`` is a uint8 tensor of at least ``head_workspace_bytes``; calls that
overlap, and graphs that are replayed, need one each.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import _check_out, load_library
from .losses import _TYPES, _at, _check_gradient, _new_gradient, _row_array, _rows, _run

SK_OP_RMS_NORM_BACKWARD, SK_OP_INT8_LINEAR, SK_OP_TOKEN_SCORES, \
    SK_OP_TOKEN_SCORES_BACKWARD = range(4)

HEAD_EXPORTS = ("sinkhorn_head_workspace_bytes", "sinkhorn_rms_norm", "sinkhorn_rms_norm_int8",
                "sinkhorn_quantize_int8", "sinkhorn_rms_norm_backward", "sinkhorn_int8_linear",
                "sinkhorn_token_scores", "sinkhorn_token_scores_backward")


def declare(lib):
    """Argument types of the entry points of sinkhorn_head.h."""
    P, I, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    D, L = ctypes.c_double, ctypes.c_int64
    types = dict(
        sinkhorn_head_workspace_bytes=[I, I, I, I, I],
        sinkhorn_rms_norm=[P, I, L, P, L, P, I, I, D, P, L, P, L, P],
        sinkhorn_rms_norm_int8=[P, I, L, P, L, P, I, I, D, P, L, P, P, L, P],
        sinkhorn_quantize_int8=[P, I, L, I, I, P, L, P, P],
        sinkhorn_rms_norm_backward=[P, I, L, P, L, P, P, L, I, I, D, P, L, P, P, Z, P],
        sinkhorn_int8_linear=[P, L, P, P, L, P, P, I, I, I, I, P, L, P, Z, P],
        sinkhorn_token_scores=[P, I, L, P, I, I, D, I, P, P, P, P, P, P, Z, P],
        sinkhorn_token_scores_backward=[P, I, L, P, P, P, I, I, D, P, L, P, Z, P])
    for name in HEAD_EXPORTS:
        getattr(lib, name).argtypes = types[name]
        getattr(lib, name).restype = I
    lib.sinkhorn_head_workspace_bytes.restype = Z


def head_workspace_bytes(op: int, T: int, V: int, k: int, dtype: int) -> int:
    return int(load_library().sinkhorn_head_workspace_bytes(op, T, V, k, dtype))


# a pure function of its arguments: programs ask for the same sizes again and again
_space_bytes = functools.lru_cache(maxsize=4096)(head_workspace_bytes)


def _space(op, T, V, k, dt, device, workspace):
    need = _space_bytes(op, T, V, k, dt)
    if workspace is None:
        return torch.empty(need or 1, dtype=torch.uint8, device=device)
    if not isinstance(workspace, torch.Tensor) or workspace.device != device \
            or workspace.dtype != torch.uint8 or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")
    if workspace.numel() < need:
        raise ValueError(f"workspace of {need} bytes needed, {workspace.numel()} given")
    return workspace


def _matrix(x, what):
    """(x, dtype code, rows, columns, row distance); copies a layout the kernels do not take."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2:
        raise ValueError(f"{what} must be a [T, values] tensor")
    dt = _TYPES.get(x.dtype)
    if dt is None:
        raise TypeError(f"{what} must be float32 or bfloat16")
    if not x.is_cuda:
        raise ValueError(f"{what} must be a GPU tensor")
    T, d = x.shape
    if d < 1:
        raise ValueError(f"{what} has rows of no values")
    if x.is_contiguous():
        return x, dt, T, d, d
    if (d > 1 and x.stride(1) != 1) or (T > 1 and x.stride(0) < d):
        return x.contiguous(), dt, T, d, d
    return x, dt, T, d, max(x.stride(0), d) if T > 1 else d


def _beside(x, like, what):
    """A further matrix of the call: the type, shape and device of `like`; None stays."""
    if x is None:
        return None, 0
    if not isinstance(x, torch.Tensor) or x.dtype != like.dtype or x.shape != like.shape \
            or x.device != like.device:
        raise ValueError(f"{what} must be {like.dtype} {tuple(like.shape)} on {like.device}")
    if x.is_contiguous():
        return x, like.shape[1]
    x, _, _, _, ld = _matrix(x, what)
    return x, ld


def _new_like(x):
    """An output of the shape and type of x, its rows side by side (for a contiguous x the call that
    takes least time)."""
    return torch.empty_like(x, memory_format=torch.contiguous_format)


def _out_matrix(x, shape, dtype, device, what):
    """Row distance of a caller's output matrix."""
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"out: {what} must be a tensor")
    T, d = shape
    if x.dtype != dtype or x.shape != (T, d) or x.device != device \
            or (d > 1 and T > 0 and x.stride(1) != 1) or (T > 1 and x.stride(0) < d):
        raise ValueError(f"out: {what} must be {dtype} {(T, d)} on {device} with its values side "
                         "by side in each row")
    return max(x.stride(0), d) if T > 1 else d


def _weight(weight, x):
    return _row_array(weight, (x.shape[1],), x.dtype, x.device, "weight", optional=True)


def _sixteen(n):
    return (n + 15) // 16 * 16


def _new_eight(T, d, device):
    """int8 [T, d], each row at a multiple of 16 bytes, as the product takes it; longer ones at
    multiples of 128, the lines it reads (333 x 1500 to 50001: 47 us, from rows of 1504 bytes 51)."""
    wide = _sixteen(d) if d < 1024 else (d + 127) // 128 * 128
    q = torch.empty((T, wide), dtype=torch.int8, device=device)
    return q if wide == d else q[:, :d]


def rms_norm(x, weight=None, residual=None, eps: float = 1e-6, out=None):
    """(y [T, d], h [T, d]): h = x + residual and its root-mean-square norm times ``weight`` [d].

    h is rounded to the type and y is the norm of that; without a residual h is x.
    ``out`` = (y, h), either of which may be x or the residual; h may be None (not kept)."""
    lib = load_library()
    x, dt, T, d, ldx = _matrix(x, "x")
    dev = x.device
    residual, ldr = _beside(residual, x, "residual")
    weight = _weight(weight, x)
    if out is not None:
        y, h = out
        ldy = _out_matrix(y, (T, d), x.dtype, dev, "y")
        ldh = 0 if h is None else _out_matrix(h, (T, d), x.dtype, dev, "h")
        kept = h
    else:
        y, ldy = _new_like(x), d
        h = x if residual is None else _new_like(x)
        kept, ldh = (None, 0) if residual is None else (h, d)
    _run(lib.sinkhorn_rms_norm, dev, _at(x), dt, ldx, _at(residual), ldr, _at(weight), T, d, eps,
         _at(y), ldy, _at(kept), ldh)
    return y, h


def rms_norm_int8(x, weight=None, residual=None, eps: float = 1e-6, out=None):
    """(q [T, d] int8, scale [T], h [T, d]): rms_norm's y in 8 bits, y ~ scale q.

    A row's largest value is 127 scale.  q's rows start at multiples of 16 bytes, as
    int8_linear takes them.  ``out`` = (q, scale, h); h may be x or the residual, or None."""
    lib = load_library()
    x, dt, T, d, ldx = _matrix(x, "x")
    dev = x.device
    residual, ldr = _beside(residual, x, "residual")
    weight = _weight(weight, x)
    if out is not None:
        q, scale, h = out
        ldq = _out_matrix(q, (T, d), torch.int8, dev, "q")
        _check_eight_scale(scale, T, dev)
        ldh = 0 if h is None else _out_matrix(h, (T, d), x.dtype, dev, "h")
        kept = h
    else:
        q = _new_eight(T, d, dev)
        ldq = q.stride(0)
        scale = torch.empty(T, dtype=torch.float32, device=dev)
        h = x if residual is None else _new_like(x)
        kept, ldh = (None, 0) if residual is None else (h, d)
    _run(lib.sinkhorn_rms_norm_int8, dev, _at(x), dt, ldx, _at(residual), ldr, _at(weight), T, d,
         eps, _at(q), ldq, _at(scale), _at(kept), ldh)
    return q, scale, h


def _check_eight_scale(scale, T, device):
    if scale is None:
        raise ValueError("out needs a scale tensor")
    _check_out(((scale, (T,)),), torch.float32, device, "out")


def quantize_int8(x, out=None):
    """(q [T, d] int8, scale [T]): rows in 8 bits, x ~ scale q, the largest value 127 scale.

    For the product's weights (a row is an output channel) and for activations without a
    norm.  q's rows start at multiples of 16 bytes.  ``out`` = (q, scale)."""
    lib = load_library()
    x, dt, T, d, ldx = _matrix(x, "x")
    dev = x.device
    if out is not None:
        q, scale = out
        ldq = _out_matrix(q, (T, d), torch.int8, dev, "q")
        _check_eight_scale(scale, T, dev)
    else:
        q = _new_eight(T, d, dev)
        ldq = q.stride(0)
        scale = torch.empty(T, dtype=torch.float32, device=dev)
    _run(lib.sinkhorn_quantize_int8, dev, _at(x), dt, ldx, T, d, _at(q), ldq, _at(scale))
    return q, scale


def rms_norm_backward(dy, h, weight=None, dh=None, eps: float = 1e-6, out=None, workspace=None):
    """(dx [T, d], dweight [d] float32): gradient of rms_norm from dy, with the h that it returned.

    ``dh``: the gradient that reaches h along the residual stream.  dx is the gradient of
    x and of the residual alike.  Without a weight dweight is None.  ``out`` = (dx,
    dweight); dx may be dy, dh or h, and dweight None (not computed)."""
    lib = load_library()
    h, dt, T, d, ldh = _matrix(h, "h")
    dev = h.device
    if dy is None:
        raise ValueError("dy must be a tensor")
    dy, lddy = _beside(dy, h, "dy")
    dh, lddh = _beside(dh, h, "dh")
    weight = _weight(weight, h)
    if out is not None:
        dx, dw = out
        lddx = _out_matrix(dx, (T, d), h.dtype, dev, "dx")
        _check_out(((dw, (d,)),), torch.float32, dev, "out")
    else:
        dx, lddx = _new_like(h), d
        dw = None if weight is None else torch.empty(d, dtype=torch.float32, device=dev)
    ws = _space(SK_OP_RMS_NORM_BACKWARD, T, d, 0, dt, dev, workspace)
    _run(lib.sinkhorn_rms_norm_backward, dev, _at(dy), dt, lddy, _at(h), ldh, _at(weight), _at(dh),
         lddh, T, d, eps, _at(dx), lddx, _at(dw), _at(ws), ws.numel())
    return dx, dw


def _eight(x, what, device=None):
    """(x, rows, columns, row distance) of an int8 matrix; rows that do not start at multiples of
    16 bytes are copied."""
    if not isinstance(x, torch.Tensor) or x.dim() != 2 or x.dtype != torch.int8:
        raise TypeError(f"{what} must be an int8 [rows, K] tensor")
    if not x.is_cuda or (device is not None and x.device != device):
        raise ValueError(f"{what} must be on {device or 'the GPU'}, got {x.device}")
    rows, K = x.shape
    if K < 1:
        raise ValueError(f"{what} has rows of no values")
    if (K > 1 and x.stride(1) != 1) or x.data_ptr() % 16 \
            or (rows > 1 and (x.stride(0) % 16 or x.stride(0) < K)):
        own = _new_eight(rows, K, x.device)
        own.copy_(x)
        return own, rows, K, own.stride(0)
    return x, rows, K, x.stride(0) if rows > 1 else _sixteen(K)


def int8_linear(x, xscale, w, wscale, bias=None, dtype=torch.bfloat16, out=None, workspace=None):
    """out [T, N] = xscale[:, None] * wscale * (x @ w.T) + bias, in ``dtype`` (or ``out``'s).

    ``x`` [T, K] int8 with a scale for each token (rms_norm_int8, quantize_int8), ``w``
    [N, K] int8 with one for each channel (quantize_int8 of the weights), ``bias`` [N]
    float32.  The sum of the products is exact.  Rows that do not start at multiples of 16
    bytes are copied on every call: keep weights as quantize_int8 returns them."""
    lib = load_library()
    x, T, K, ldx = _eight(x, "x")
    dev = x.device
    w, N, Kw, ldw = _eight(w, "w", dev)
    if Kw != K:
        raise ValueError(f"x has rows of {K} values, w of {Kw}")
    xscale = _row_array(xscale, (T,), torch.float32, dev, "xscale")
    wscale = _row_array(wscale, (N,), torch.float32, dev, "wscale")
    bias = _row_array(bias, (N,), torch.float32, dev, "bias", optional=True)
    if out is not None:
        dtype = out.dtype if isinstance(out, torch.Tensor) else None
    dt = _TYPES.get(dtype)
    if dt is None:
        raise TypeError("the result must be float32 or bfloat16")
    if out is not None:
        ldo = _out_matrix(out, (T, N), dtype, dev, "the result")
    else:
        out, ldo = torch.empty((T, N), dtype=dtype, device=dev), N
    ws = _space(SK_OP_INT8_LINEAR, T, N, K, dt, dev, workspace)
    _run(lib.sinkhorn_int8_linear, dev, _at(x), ldx, _at(xscale), _at(w), ldw, _at(wscale),
         _at(bias), T, K, N, dt, _at(out), ldo, _at(ws), ws.numel())
    return out


def token_scores(logits, labels=None, top: int = 0, scale: float = 1.0, out=None, workspace=None):
    """(logp [T], lse [T], entropy [T], index [T, top], best [T, top]) of softmax(scale * logits).

    logp: log-probability of ``labels`` (None without labels); a negative label marks a
    row that is not scored.  index (int32), best: the ``top`` most likely tokens (at most
    128) and their log-probabilities in falling order, the lower index first among equal
    ones; None with top = 0.  Places that stay empty hold -1 and -inf, no entry to
    distill_loss.  ``out`` = the five buffers, the last two None with top = 0, of the first
    three any but not all may be None."""
    lib = load_library()
    logits, dt, T, V, ld = _rows(logits)
    dev = logits.device
    labels = _row_array(labels, (T,), torch.int32, dev, "labels", optional=True)
    if out is not None:
        logp, lse, entropy, index, best = out
        _check_out(((logp, (T,)), (lse, (T,)), (entropy, (T,)), (best, (T, top))), torch.float32,
                   dev, "out")
        _check_out(((index, (T, top)),), torch.int32, dev, "out")
    else:
        lse = torch.empty(T, dtype=torch.float32, device=dev)
        entropy = torch.empty_like(lse)
        logp = None if labels is None else torch.empty_like(lse)
        index = torch.empty((T, top), dtype=torch.int32, device=dev) if top else None
        best = torch.empty((T, top), dtype=torch.float32, device=dev) if top else None
    ws = _space(SK_OP_TOKEN_SCORES, T, V, top, dt, dev, workspace)
    _run(lib.sinkhorn_token_scores, dev, _at(logits), dt, ld, _at(labels), T, V, scale, top,
         _at(logp), _at(lse), _at(entropy), _at(index), _at(best), _at(ws), ws.numel())
    return logp, lse, entropy, index, best


def token_scores_backward(logits, labels=None, grad=None, grad_entropy=None, scale: float = 1.0,
                          out=None, workspace=None):
    """dlogits [T, V] from grad [T] = dL/dlogp and grad_entropy [T] = dL/dentropy of token_scores.

    Either may be None (0); a row where both are 0, or that is not scored, is not read.
    ``out`` may be the logits themselves."""
    lib = load_library()
    logits, dt, T, V, ld = _rows(logits)
    dev = logits.device
    labels = _row_array(labels, (T,), torch.int32, dev, "labels", optional=True)
    grad = _row_array(grad, (T,), torch.float32, dev, "grad", optional=True)
    grad_entropy = _row_array(grad_entropy, (T,), torch.float32, dev, "grad_entropy", optional=True)
    if out is None:
        d, dld = _new_gradient(logits, ld)
    else:
        d, dld = out, _check_gradient(out, logits)
    ws = _space(SK_OP_TOKEN_SCORES_BACKWARD, T, V, 0, dt, dev, workspace)
    _run(lib.sinkhorn_token_scores_backward, dev, _at(logits), dt, ld, _at(labels), _at(grad),
         _at(grad_entropy), T, V, scale, _at(d), dld, _at(ws), ws.numel())
    return d
