"""Losses over rows of logits, with their gradients, on the library's HIP kernels.

The binding of ``include/sinkhorn_losses.h``; the calls are reached through the
package itself (``sinkhorn_point_cloud_amd.policy_loss`` and so on).

Common to all: ``logits`` [T, V] float32 or bfloat16 on the GPU; rows may lie
further apart than V (a view of padded columns), other layouts are copied.
Labels and indices are int32, offsets int64, everything else float32.  The work
runs on the current stream of the tensors' device.  A returned gradient has the
logits' dtype and, where their rows are padded, their row distance; it is the
gradient of the sum of the returned losses.  ``out`` reuses buffers, and its
gradient may be the logits themselves; ``grad=False`` skips the gradient (None), also
where ``out`` holds a buffer for it.  Rows outside every sequence get zeros in
outputs that the call allocates and are left alone in the caller's.  Buffers that share
memory with other arguments (but for that gradient) are refused.
``workspace`` is a uint8 tensor of at least ``losses_workspace_bytes``; calls
that overlap, and graphs that are replayed, need one each.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import SK_BF16, SK_F32, _check, _check_out, load_library

SK_OP_TOKEN_LOGPROBS, SK_OP_POLICY_LOSS, SK_OP_PREFERENCE_LOSS, SK_OP_DISTILL_LOSS, \
    SK_OP_BALANCE_LOSS = range(5)
SK_LOSS_MEAN, SK_LOSS_FILL, SK_LOSS_ROW_ADVANTAGE = 1, 2, 4
_TYPES = {torch.float32: SK_F32, torch.bfloat16: SK_BF16}
PREFERENCE_KINDS = {"sigmoid": 0, "square": 1}

LOSS_EXPORTS = ("sinkhorn_losses_workspace_bytes", "sinkhorn_token_logprobs",
                "sinkhorn_token_logprobs_backward", "sinkhorn_policy_loss",
                "sinkhorn_preference_loss", "sinkhorn_distill_loss", "sinkhorn_balance_loss")


def declare(lib):
    """Argument types of the entry points of sinkhorn_losses.h."""
    P, I, U, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_uint, ctypes.c_size_t
    D, L = ctypes.c_double, ctypes.c_int64
    types = dict(
        sinkhorn_losses_workspace_bytes=[I, I, I, I, I],
        sinkhorn_token_logprobs=[P, I, L, P, I, I, D, P, P, P, Z, P],
        sinkhorn_token_logprobs_backward=[P, I, L, P, P, I, I, D, P, L, P, Z, P],
        sinkhorn_policy_loss=[P, I, L, P, I, I, P, I, P, P, P, P, D, D, D, D, U, P, P, P, P, L,
                              P, Z, P],
        sinkhorn_preference_loss=[P, I, L, P, I, I, P, I, P, P, D, I, D, D, U, P, P, P, P, L,
                                  P, Z, P],
        sinkhorn_distill_loss=[P, I, L, I, I, P, P, I, P, P, D, P, P, L, P, Z, P],
        sinkhorn_balance_loss=[P, I, L, I, I, P, I, P, I, D, D, U, P, P, P, P, L, P, Z, P])
    for name in LOSS_EXPORTS:
        getattr(lib, name).argtypes = types[name]
        getattr(lib, name).restype = I
    lib.sinkhorn_losses_workspace_bytes.restype = Z


def losses_workspace_bytes(op: int, T: int, V: int, k: int, dtype: int) -> int:
    return int(load_library().sinkhorn_losses_workspace_bytes(op, T, V, k, dtype))


# a pure function of its arguments: training loops ask for the same sizes again and again
_space_bytes = functools.lru_cache(maxsize=4096)(losses_workspace_bytes)


def _rows(logits):
    """(logits, dtype code, rows, columns, row distance); copies a layout the kernels do not take."""
    if not isinstance(logits, torch.Tensor) or logits.dim() != 2:
        raise ValueError("logits must be a [T, V] tensor")
    dt = _TYPES.get(logits.dtype)
    if dt is None:
        raise TypeError("logits must be float32 or bfloat16")
    if not logits.is_cuda:
        raise ValueError("logits must be a GPU tensor")
    T, V = logits.shape
    if logits.is_contiguous():
        return logits, dt, T, V, V
    if (V > 1 and logits.stride(1) != 1) or (T > 1 and logits.stride(0) < V):
        return logits.contiguous(), dt, T, V, V
    return logits, dt, T, V, logits.stride(0) if T > 1 else V


def _row_array(x, shape, dtype, device, what, optional=False):
    """An input array checked for type, shape and device, made contiguous."""
    if x is None and optional:
        return None
    if not isinstance(x, torch.Tensor):
        raise TypeError(f"{what} must be a tensor")
    if x.dtype != dtype:
        raise TypeError(f"{what} must be {dtype}, got {x.dtype}")
    if x.shape != shape or x.device != device:
        raise ValueError(f"{what} must be {tuple(shape)} on {device}, got {tuple(x.shape)} "
                         f"on {x.device}")
    return x if x.is_contiguous() else x.contiguous()


def _offsets(offsets, device):
    if not isinstance(offsets, torch.Tensor) or offsets.dim() != 1 or offsets.numel() < 2:
        raise ValueError("offsets must be a tensor of at least two row numbers")
    return _row_array(offsets, offsets.shape, torch.int64, device, "offsets")


def _at(x):
    """Address of a tensor for the C ABI (None: NULL)."""
    return None if x is None else x.data_ptr()


def _new_gradient(logits, ld):
    T, V = logits.shape
    if V < ld <= 2 * V:   # padded rows: the same distance keeps both at the same alignment
        return torch.empty((T, ld), dtype=logits.dtype, device=logits.device)[:, :V], ld
    return torch.empty((T, V), dtype=logits.dtype, device=logits.device), V


def _check_gradient(d, logits):
    """Row distance of a caller's gradient buffer."""
    if d is None:
        return 0
    if not isinstance(d, torch.Tensor):
        raise TypeError("out: the gradient must be a tensor")
    T, V = logits.shape
    if d.dtype != logits.dtype or d.shape != logits.shape or d.device != logits.device \
            or (V > 1 and T > 0 and d.stride(1) != 1) or (T > 1 and d.stride(0) < V):
        raise ValueError(f"out: the gradient must be {logits.dtype} {tuple(logits.shape)} on "
                         f"{logits.device} with its values side by side in each row")
    return max(d.stride(0) if T > 1 else V, V)


def _space(op, T, V, k, dt, device, workspace):
    need = _space_bytes(op, T, V, k, dt)
    if workspace is None:
        return torch.empty(need or 1, dtype=torch.uint8, device=device)
    if workspace.device != device or workspace.dtype != torch.uint8 \
            or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on {device}")
    if workspace.numel() < need:
        raise ValueError(f"workspace of {need} bytes needed, {workspace.numel()} given")
    return workspace


def _run(entry, device, *args):
    """Calls an entry point on the current stream of the tensors' device."""
    index = device.index
    if index == torch.cuda.current_device():
        # the raw handle: building a Stream object for it takes 2 us
        _check(entry(*args, torch._C._cuda_getCurrentRawStream(index)))
    else:
        with torch.cuda.device(index):
            _check(entry(*args, torch._C._cuda_getCurrentRawStream(index)))


def token_logprobs(logits, labels, scale: float = 1.0, out=None, workspace=None):
    """(logp [T], lse [T]): log softmax(scale * logits) at ``labels`` and the row's log-sum-exp.

    A negative label marks a row that is not scored: both are 0 there."""
    lib = load_library()
    logits, dt, T, V, ld = _rows(logits)
    dev = logits.device
    labels = _row_array(labels, (T,), torch.int32, dev, "labels")
    if out is not None:
        logp, lse = out
        _check_out(((logp, (T,)), (lse, (T,))), torch.float32, dev, "out")
    else:
        logp = torch.empty(T, dtype=torch.float32, device=dev)
        lse = torch.empty(T, dtype=torch.float32, device=dev)
    ws = _space(SK_OP_TOKEN_LOGPROBS, T, V, 0, dt, dev, workspace)
    _run(lib.sinkhorn_token_logprobs, dev, _at(logits), dt, ld, _at(labels), T, V, scale,
         _at(logp), _at(lse), _at(ws), ws.numel())
    return logp, lse


def token_logprobs_backward(logits, labels, grad, scale: float = 1.0, out=None, workspace=None):
    """dlogits [T, V] from grad [T] = dL/dlogp of token_logprobs; a row of grad 0 is not read."""
    lib = load_library()
    logits, dt, T, V, ld = _rows(logits)
    dev = logits.device
    labels = _row_array(labels, (T,), torch.int32, dev, "labels")
    grad = _row_array(grad, (T,), torch.float32, dev, "grad")
    if out is None:
        d, dld = _new_gradient(logits, ld)
    else:
        d, dld = out, _check_gradient(out, logits)
    ws = _space(SK_OP_TOKEN_LOGPROBS, T, V, 0, dt, dev, workspace)
    _run(lib.sinkhorn_token_logprobs_backward, dev, _at(logits), dt, ld, _at(labels), _at(grad), T,
         V, scale, _at(d), dld, _at(ws), ws.numel())
    return d


def policy_loss(logits, labels, offsets, old, adv, ref=None, clip=(0.2, 0.2), kl: float = 0.0,
                scale: float = 1.0, weights=None, mean: bool = True, grad: bool = True, out=None,
                workspace=None):
    """(loss [n], kl [n], logp [T], dlogits): clipped policy loss per packed sequence.

    ``old`` [T]: the behaviour policy's log-probabilities; ``adv``: advantages, one per
    sequence [n] or one per row [T] (where n == T, per row); ``ref`` [T]: a reference
    model's log-probabilities, for the KL term of coefficient ``kl``; ``weights`` [n]:
    one per sequence.  ``mean`` divides a sequence's sum by its number of labels.
    ``out`` = (loss, kl, logp, dlogits), the last two may be None."""
    lib = load_library()
    logits, dt, T, V, ld = _rows(logits)
    dev = logits.device
    labels = _row_array(labels, (T,), torch.int32, dev, "labels")
    offsets = _offsets(offsets, dev)
    n = offsets.numel() - 1
    per_row = isinstance(adv, torch.Tensor) and adv.shape == (T,)
    old = _row_array(old, (T,), torch.float32, dev, "old")
    adv = _row_array(adv, (T,) if per_row else (n,), torch.float32, dev, "adv")
    ref = _row_array(ref, (T,), torch.float32, dev, "ref", optional=True)
    weights = _row_array(weights, (n,), torch.float32, dev, "weights", optional=True)
    flags = (SK_LOSS_MEAN if mean else 0) | (SK_LOSS_ROW_ADVANTAGE if per_row else 0)
    if out is not None:
        loss, kls, logp, d = out
        d = d if grad else None
        dld = _check_gradient(d, logits)
        if loss is None or kls is None:
            raise ValueError("out needs loss and kl tensors")
        _check_out(((loss, (n,)), (kls, (n,)), (logp, (T,))), torch.float32, dev, "out")
    else:
        flags |= SK_LOSS_FILL
        loss = torch.empty(n, dtype=torch.float32, device=dev)
        kls = torch.empty(n, dtype=torch.float32, device=dev)
        logp = torch.empty(T, dtype=torch.float32, device=dev)
        d, dld = _new_gradient(logits, ld) if grad else (None, 0)
    ws = _space(SK_OP_POLICY_LOSS, T, V, 0, dt, dev, workspace)
    _run(lib.sinkhorn_policy_loss, dev, _at(logits), dt, ld, _at(labels), T, V, _at(offsets), n,
         _at(old), _at(adv), _at(ref), _at(weights), scale, clip[0], clip[1], kl, flags, _at(loss),
         _at(kls), _at(logp), _at(d), dld, _at(ws), ws.numel())
    return loss, kls, logp, d


def preference_loss(logits, labels, offsets, ref=None, beta: float = 0.1, smoothing: float = 0.0,
                    kind: str = "sigmoid", scale: float = 1.0, weights=None, mean: bool = False,
                    grad: bool = True, out=None, workspace=None):
    """(loss [pairs], reward [2 pairs], logp [T], dlogits): preference loss of paired sequences.

    Sequence 2i of ``offsets`` is the preferred one of pair i and 2i + 1 the other.
    ``ref`` [T]: a reference model's log-probabilities; ``kind`` "sigmoid" (with label
    ``smoothing``) or "square"; ``weights`` [pairs].  ``mean`` takes the mean over a
    sequence's labels instead of the sum.  ``out`` = (loss, reward, logp, dlogits), the
    last may be None."""
    lib = load_library()
    logits, dt, T, V, ld = _rows(logits)
    dev = logits.device
    labels = _row_array(labels, (T,), torch.int32, dev, "labels")
    offsets = _offsets(offsets, dev)
    n = offsets.numel() - 1
    if n % 2:
        raise ValueError(f"pairs need an even number of sequences, offsets hold {n}")
    if kind not in PREFERENCE_KINDS:
        raise ValueError(f"kind must be one of {sorted(PREFERENCE_KINDS)}, got {kind!r}")
    ref = _row_array(ref, (T,), torch.float32, dev, "ref", optional=True)
    weights = _row_array(weights, (n // 2,), torch.float32, dev, "weights", optional=True)
    flags = SK_LOSS_MEAN if mean else 0
    if out is not None:
        loss, reward, logp, d = out
        d = d if grad else None
        dld = _check_gradient(d, logits)
        if loss is None or reward is None or logp is None:
            raise ValueError("out needs loss, reward and logp tensors")
        _check_out(((loss, (n // 2,)), (reward, (n,)), (logp, (T,))), torch.float32, dev, "out")
    else:
        flags |= SK_LOSS_FILL
        loss = torch.empty(n // 2, dtype=torch.float32, device=dev)
        reward = torch.empty(n, dtype=torch.float32, device=dev)
        logp = torch.empty(T, dtype=torch.float32, device=dev)
        d, dld = _new_gradient(logits, ld) if grad else (None, 0)
    ws = _space(SK_OP_PREFERENCE_LOSS, T, V, 0, dt, dev, workspace)
    _run(lib.sinkhorn_preference_loss, dev, _at(logits), dt, ld, _at(labels), T, V, _at(offsets), n
         // 2, _at(ref), _at(weights), scale, PREFERENCE_KINDS[kind], beta, smoothing, flags,
         _at(loss), _at(reward), _at(logp), _at(d), dld, _at(ws), ws.numel())
    return loss, reward, logp, d


def distill_loss(logits, index, teacher, teacher_lse=None, temperature: float = 1.0, weights=None,
                 grad: bool = True, out=None, workspace=None):
    """(loss [T], dlogits): divergence from a teacher's top logits, per row.

    ``teacher`` [T, K]: its logits at tokens ``index`` [T, K] (negative: no entry).  They
    are normalised among themselves, or with ``teacher_lse`` [T], the teacher's
    log-sum-exp of logits / temperature over its whole vocabulary.  ``weights`` [T]: a row
    of weight 0 is not read.  ``out`` = (loss, dlogits), the last may be None."""
    lib = load_library()
    logits, dt, T, V, ld = _rows(logits)
    dev = logits.device
    if not isinstance(index, torch.Tensor) or index.dim() != 2:
        raise ValueError("index must be a [T, K] tensor")
    K = index.shape[1]
    index = _row_array(index, (T, K), torch.int32, dev, "index")
    teacher = _row_array(teacher, (T, K), torch.float32, dev, "teacher")
    teacher_lse = _row_array(teacher_lse, (T,), torch.float32, dev, "teacher_lse", optional=True)
    weights = _row_array(weights, (T,), torch.float32, dev, "weights", optional=True)
    if not temperature > 0:
        raise ValueError(f"temperature must be positive, got {temperature}")
    if out is not None:
        loss, d = out
        d = d if grad else None
        dld = _check_gradient(d, logits)
        if loss is None:
            raise ValueError("out needs a loss tensor")
        _check_out(((loss, (T,)),), torch.float32, dev, "out")
    else:
        loss = torch.empty(T, dtype=torch.float32, device=dev)
        d, dld = _new_gradient(logits, ld) if grad else (None, 0)
    ws = _space(SK_OP_DISTILL_LOSS, T, V, K, dt, dev, workspace)
    _run(lib.sinkhorn_distill_loss, dev, _at(logits), dt, ld, T, V, _at(index), _at(teacher), K,
         _at(teacher_lse), _at(weights), temperature, _at(loss), _at(d), dld, _at(ws), ws.numel())
    return loss, d


def balance_loss(logits, index, offsets=None, balance: float = 1.0, z: float = 0.0,
                 grad: bool = True, out=None, workspace=None):
    """(loss [G], zloss [G], counts [G, E], dlogits): an expert router's balance loss.

    ``logits`` [T, E]; ``index`` [T, K]: the experts each row was sent to (negative:
    none).  With ``offsets`` [G + 1] the loss is taken within each packed sequence,
    without them over all rows (G = 1).  loss and zloss are without their coefficients;
    the gradient is that of balance * loss + z * zloss, summed over the groups, the
    counts held fixed.  ``out`` = (loss, zloss, counts, dlogits), the last may be None."""
    lib = load_library()
    logits, dt, T, E, ld = _rows(logits)
    dev = logits.device
    if not isinstance(index, torch.Tensor) or index.dim() != 2:
        raise ValueError("index must be a [T, K] tensor")
    K = index.shape[1]
    index = _row_array(index, (T, K), torch.int32, dev, "index")
    if offsets is not None:
        offsets = _offsets(offsets, dev)
    G = 1 if offsets is None else offsets.numel() - 1
    flags = 0
    if out is not None:
        loss, zloss, counts, d = out
        d = d if grad else None
        dld = _check_gradient(d, logits)
        if loss is None or zloss is None or counts is None:
            raise ValueError("out needs loss, zloss and counts tensors")
        _check_out(((loss, (G,)), (zloss, (G,))), torch.float32, dev, "out")
        _check_out(((counts, (G, E)),), torch.int32, dev, "out")
    else:
        flags |= SK_LOSS_FILL
        loss = torch.empty(G, dtype=torch.float32, device=dev)
        zloss = torch.empty(G, dtype=torch.float32, device=dev)
        counts = torch.empty(G, E, dtype=torch.int32, device=dev)
        d, dld = _new_gradient(logits, ld) if grad else (None, 0)
    ws = _space(SK_OP_BALANCE_LOSS, T, E, G, dt, dev, workspace)
    _run(lib.sinkhorn_balance_loss, dev, _at(logits), dt, ld, T, E, _at(index), K, _at(offsets), G,
         balance, z, flags, _at(loss), _at(zloss), _at(counts), _at(d), dld, _at(ws), ws.numel())
    return loss, zloss, counts, d
