"""Post-training losses of the output layer (``include/flce.h``): the clipped
policy loss with a KL term and distillation from a teacher's top logits, each on
given logits and through the LM head.

The family is the one the pages name ("Liger-Kernel: Triton kernels that replace
Hugging Face training ops", section "Installation and the one-line patch": losses
called with the LM-head weight, the hidden states and the targets).  Like the rest
of the binding this module only marshals arguments; every function returns
device tensors without waiting, the device status word (0, or a
``flce_status_t``) among them.

``stream``: the CUDA stream to run on (default: the current one).  The call does
not make ``stream`` wait for the streams that produced its inputs.  Calls through
the head run one at a time on a device: order those on several streams by events.
"""
from __future__ import annotations

import torch
# the handles without the objects around them: a few us less per call
from torch._C import _cuda_getCurrentRawStream as _current_stream_handle
from torch._C import _cuda_getDevice as _current_device

from .flce import REDUCTIONS, _check, _check_tensors, load_library

DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
MAX_TEACHER_ENTRIES = 1024
CLIPPED_POLICY_NO_WORKSPACE = 2048


def _p(t):
    return None if t is None else t.data_ptr()


def _vec(t, dtype, N, dev, name, optional=False):
    """A per-row vector of the call: contiguous, ``dtype``, [N], on ``dev``."""
    if t is None:
        if optional:
            return
        raise ValueError(f"{name} is required")
    if t.dtype != dtype or t.dim() != 1 or t.shape[0] != N or not t.is_contiguous() or t.device != dev:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape [{N}] on {dev}, "
                         f"got {t.dtype} {tuple(t.shape)} on {t.device}")


def _scale(t, reduction, N, dev, name):
    if reduction not in REDUCTIONS:
        raise ValueError(f"reduction must be one of {sorted(REDUCTIONS)}, got {reduction!r}")
    _vec(t, torch.float32, N, dev, name, optional=True)
    if t is not None and reduction != "none":
        raise ValueError(f"{name} goes with reduction='none'")
    return REDUCTIONS[reduction]


def _logits(logits, y, grad):
    """Checks logits [N, V] (rows at any stride >= V) and targets [N]; returns the row stride."""
    if logits.dtype not in DTYPES or logits.dim() != 2:
        raise ValueError("expected bf16, fp16 or fp32 logits [N, V]")
    N, V = logits.shape
    if N < 1 or V < 1:
        raise ValueError("logits must have at least one row and one column")
    ld = logits.stride(0) if N > 1 else max(logits.stride(0), V)
    if (V > 1 and logits.stride(1) != 1) or ld < V:
        raise ValueError("a row's logits must be adjacent and the rows must not overlap")
    if not logits.is_cuda:
        raise ValueError("logits must be a CUDA tensor")
    _vec(y, torch.int32, N, logits.device, "y")
    if grad not in ("new", "inplace", "none"):
        raise ValueError("grad must be 'new', 'inplace' or 'none'")
    return ld


def _grad_like(logits, ld, grad):
    """The gradient tensor and its row stride.  A new one takes the logits' row
    stride, so that both have their rows at the same alignment, unless the
    logits are a narrow slice of a much wider buffer."""
    N, V = logits.shape
    if grad == "none":
        return None, ld
    if grad == "inplace":
        return logits, ld
    ldg = ld if ld <= V + V // 8 + 64 else V
    return torch.empty_strided((N, V), (ldg, 1), dtype=logits.dtype, device=logits.device), ldg


def _teacher(ids, logits, lse, N, dev):
    if ids.dtype != torch.int32 or ids.dim() != 2 or ids.shape[0] != N or not ids.is_contiguous() or ids.device != dev:
        raise ValueError(f"teacher_ids must be a contiguous int32 tensor [{N}, K] on {dev}")
    K = ids.shape[1]
    if not 1 <= K <= MAX_TEACHER_ENTRIES:
        raise ValueError(f"teacher_ids must have 1 to {MAX_TEACHER_ENTRIES} columns, got {K}")
    if logits.dtype not in DTYPES or logits.shape != ids.shape or not logits.is_contiguous() or logits.device != dev:
        raise ValueError("teacher_logits must be a contiguous bf16, fp16 or fp32 tensor of teacher_ids' shape and device")
    _vec(lse, torch.float32, N, dev, "teacher_lse", optional=True)
    return K


def _elsewhere(fn, dev, stream, args, kw):
    """``fn(*args, **kw)`` on ``dev`` and, if given, ``stream``, neither of which
    is current.  Outputs and scratch are allocated for that stream, and the
    allocator is told who else uses the outputs and the inputs."""
    if stream is not None and stream.device != dev:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {dev}")
    with torch.cuda.device(dev):
        current = torch.cuda.current_stream()
        if stream is None or stream == current:
            return fn(*args, **kw)
        with torch.cuda.stream(stream):
            out = fn(*args, **kw)
    for t in out:
        if t is not None:
            t.record_stream(current)
    for t in (*args, *kw.values()):
        if isinstance(t, torch.Tensor):
            t.record_stream(stream)
    return out


def _workspace(ws, nbytes, like):
    """The caller's workspace, checked, or a new one on ``like``'s device."""
    if ws is None:
        return like.new_empty(nbytes, dtype=torch.uint8)
    if (ws.dtype != torch.uint8 or ws.dim() != 1 or not ws.is_contiguous() or ws.device != like.device
            or ws.numel() < nbytes):
        raise ValueError(f"workspace must be a contiguous 1-D uint8 tensor of at least {nbytes} bytes on {like.device}")
    return ws


def clipped_policy(row_loss, y, old_logp, advantages, *, ref_logp=None, clip_low: float = 0.2, clip_high: float = 0.2,
                   kl_coef: float = 0.0, reduction: str = "mean", row_scale=None, ignore_index: int = -100,
                   workspace=None, stream=None):
    """flce_clipped_policy on the head's row losses (row_loss fp32 [N], y int32
    [N]; old_logp fp32 [N] or None for ratio 1; advantages fp32 [N]; ref_logp
    fp32 [N] or None).  Returns (loss fp64[1], policy_loss fp32[N], kl fp32[N],
    row_weight fp32[N], status int32[1]); row_weight is the upstream gradient
    of each row loss, to pass as grad_row_scale with reduction 'none'."""
    lib = load_library()
    dev = row_loss.device
    N = row_loss.shape[0] if row_loss.dim() == 1 else -1
    if not row_loss.is_cuda or N < 1:
        raise ValueError("row_loss must be a CUDA tensor [N] with N >= 1")
    _vec(row_loss, torch.float32, N, dev, "row_loss")
    _vec(y, torch.int32, N, dev, "y")
    _vec(old_logp, torch.float32, N, dev, "old_logp", optional=True)
    _vec(advantages, torch.float32, N, dev, "advantages")
    _vec(ref_logp, torch.float32, N, dev, "ref_logp", optional=True)
    red = _scale(row_scale, reduction, N, dev, "row_scale")
    if stream is not None or dev.index != _current_device():
        return _elsewhere(clipped_policy, dev, stream, (row_loss, y, old_logp, advantages),
                          dict(ref_logp=ref_logp, clip_low=clip_low, clip_high=clip_high, kl_coef=kl_coef,
                               reduction=reduction, row_scale=row_scale, ignore_index=ignore_index,
                               workspace=workspace))
    nbytes = lib.flce_ce_workspace_size(N, 1) if N > CLIPPED_POLICY_NO_WORKSPACE else 0
    ws = _workspace(workspace, nbytes, row_loss) if nbytes else None
    loss = row_loss.new_empty(1, dtype=torch.float64)
    rows, kl, weight = row_loss.new_empty(N), row_loss.new_empty(N), row_loss.new_empty(N)
    status = y.new_empty(1)
    _check(lib.flce_clipped_policy(_p(row_loss), _p(y), N, ignore_index, _p(old_logp), _p(advantages), _p(ref_logp),
                                   clip_low, clip_high, kl_coef, red, _p(row_scale), _p(loss), _p(rows), _p(kl),
                                   _p(weight), _p(status), _p(ws), nbytes, _current_stream_handle(dev.index)),
           "flce_clipped_policy")
    return loss, rows, kl, weight, status


def policy_loss(logits, y, old_logp, advantages, *, ref_logp=None, clip_low: float = 0.2, clip_high: float = 0.2,
                kl_coef: float = 0.0, entropy_coef: float = 0.0, temperature: float = 1.0, reduction: str = "mean",
                grad_row_scale=None, ignore_index: int = -100, grad: str = "new", workspace=None, stream=None):
    """flce_policy_loss on given logits [N, V] (bf16, fp16 or fp32; rows may be
    strided).  Returns (loss fp32[1], status int32[1], logp fp32[N], entropy
    fp32[N], kl fp32[N], dlogits or None).  grad: 'new' (a new tensor), 'inplace'
    (overwrite ``logits``) or 'none'."""
    lib = load_library()
    ld = _logits(logits, y, grad)
    N, V = logits.shape
    dev = logits.device
    _vec(old_logp, torch.float32, N, dev, "old_logp", optional=True)
    _vec(advantages, torch.float32, N, dev, "advantages")
    _vec(ref_logp, torch.float32, N, dev, "ref_logp", optional=True)
    red = _scale(grad_row_scale, reduction, N, dev, "grad_row_scale")
    if stream is not None or dev.index != _current_device():
        return _elsewhere(policy_loss, dev, stream, (logits, y, old_logp, advantages),
                          dict(ref_logp=ref_logp, clip_low=clip_low, clip_high=clip_high, kl_coef=kl_coef,
                               entropy_coef=entropy_coef, temperature=temperature, reduction=reduction,
                               grad_row_scale=grad_row_scale, ignore_index=ignore_index, grad=grad,
                               workspace=workspace))
    ws = _workspace(workspace, lib.flce_ce_workspace_size(N, V), y)
    g, ldg = _grad_like(logits, ld, grad)
    loss, logp, entropy, kl = (advantages.new_empty(1), advantages.new_empty(N), advantages.new_empty(N),
                               advantages.new_empty(N))
    status = y.new_empty(1)
    _check(lib.flce_policy_loss(_p(logits), DTYPES[logits.dtype], ld, _p(y), N, V, ignore_index, temperature,
                                _p(old_logp), _p(advantages), _p(ref_logp), clip_low, clip_high, kl_coef,
                                entropy_coef, red, _p(grad_row_scale), _p(loss), _p(logp), _p(entropy), _p(kl),
                                _p(status), _p(g), ldg, _p(ws), ws.numel(), _current_stream_handle(dev.index)),
           "flce_policy_loss")
    return loss, status, logp, entropy, kl, g


def distill_topk(logits, y, teacher_ids, teacher_logits, *, teacher_lse=None, temperature: float = 1.0,
                 kd_weight: float = 1.0, ce_weight: float = 0.0, reduction: str = "mean", grad_row_scale=None,
                 ignore_index: int = -100, row_loss: bool = False, grad: str = "new", workspace=None, stream=None):
    """flce_distill_topk on given student logits [N, V] (as :func:`policy_loss`):
    teacher_ids int32 [N, K] (negative: empty slot), teacher_logits [N, K] bf16,
    fp16 or fp32, teacher_lse fp32 [N] or None.  Returns (loss fp32[1], status
    int32[1], row_loss fp32[N] or None, dlogits or None)."""
    lib = load_library()
    ld = _logits(logits, y, grad)
    N, V = logits.shape
    dev = logits.device
    K = _teacher(teacher_ids, teacher_logits, teacher_lse, N, dev)
    red = _scale(grad_row_scale, reduction, N, dev, "grad_row_scale")
    if stream is not None or dev.index != _current_device():
        return _elsewhere(distill_topk, dev, stream, (logits, y, teacher_ids, teacher_logits),
                          dict(teacher_lse=teacher_lse, temperature=temperature, kd_weight=kd_weight,
                               ce_weight=ce_weight, reduction=reduction, grad_row_scale=grad_row_scale,
                               ignore_index=ignore_index, row_loss=row_loss, grad=grad, workspace=workspace))
    ws = _workspace(workspace, lib.flce_ce_workspace_size(N, V), y)
    g, ldg = _grad_like(logits, ld, grad)
    loss = y.new_empty(1, dtype=torch.float32)
    rows = y.new_empty(N, dtype=torch.float32) if row_loss else None
    status = y.new_empty(1)
    _check(lib.flce_distill_topk(_p(logits), DTYPES[logits.dtype], ld, _p(y), N, V, ignore_index, _p(teacher_ids),
                                 _p(teacher_logits), DTYPES[teacher_logits.dtype], K, _p(teacher_lse), temperature,
                                 kd_weight, ce_weight, red, _p(grad_row_scale), _p(loss), _p(rows), _p(status),
                                 _p(g), ldg, _p(ws), ws.numel(), _current_stream_handle(dev.index)),
           "flce_distill_topk")
    return loss, status, rows, g


def _head_outputs(X, W, grads):
    return (torch.empty_like(X), torch.empty_like(W)) if grads else (None, None)


def policy_workspace_size(N: int, H: int, V: int, reorder: bool = False) -> int:
    """flce_policy_workspace_size: bytes one :func:`policy_forward_backward` takes,
    or with ``reorder`` those that let it skip scattered ignored rows.  It also
    runs on flce_workspace_size bytes, small batches more slowly."""
    return int(load_library().flce_policy_workspace_size(N, H, V, 1 if reorder else 0))


def policy_forward_backward(X, W, y, old_logp, advantages, *, ref_logp=None, clip_low: float = 0.2,
                            clip_high: float = 0.2, kl_coef: float = 0.0, reduction: str = "mean",
                            grad_row_scale=None, mean_count=None, ignore_index: int = -100, grads: bool = True,
                            workspace=None, stream=None):
    """flce_policy_forward_backward: the clipped policy loss of hidden states X
    [N, H] and LM-head weight W [V, H] (bf16) without the logits.  Returns (loss
    fp32[1], status int32[1], logp fp32[N], dX or None, dW or None)."""
    lib = load_library()
    _check_tensors(X, W, y, workspace=workspace)
    N, H = X.shape
    V = W.shape[0]
    dev = X.device
    _vec(old_logp, torch.float32, N, dev, "old_logp", optional=True)
    _vec(advantages, torch.float32, N, dev, "advantages")
    _vec(ref_logp, torch.float32, N, dev, "ref_logp", optional=True)
    _vec(mean_count, torch.int32, 1, dev, "mean_count", optional=True)
    red = _scale(grad_row_scale, reduction, N, dev, "grad_row_scale")

    if stream is not None or dev.index != _current_device():
        return _elsewhere(policy_forward_backward, dev, stream, (X, W, y, old_logp, advantages),
                          dict(ref_logp=ref_logp, clip_low=clip_low, clip_high=clip_high, kl_coef=kl_coef,
                               reduction=reduction, grad_row_scale=grad_row_scale, mean_count=mean_count,
                               ignore_index=ignore_index, grads=grads, workspace=workspace))
    ws = y.new_empty(policy_workspace_size(N, H, V), dtype=torch.uint8) if workspace is None else workspace
    loss, logp = advantages.new_empty(1), advantages.new_empty(N)
    status = y.new_empty(1)
    dX, dW = _head_outputs(X, W, grads)
    _check(lib.flce_policy_forward_backward(_p(X), _p(W), _p(y), N, H, V, ignore_index, _p(old_logp), _p(advantages),
                                            _p(ref_logp), clip_low, clip_high, kl_coef, red, _p(grad_row_scale),
                                            _p(mean_count), _p(loss), _p(logp), _p(status), _p(dX), _p(dW), _p(ws),
                                            ws.numel(), _current_stream_handle(dev.index)),
           "flce_policy_forward_backward")
    return loss, status, logp, dX, dW


def distill_workspace_size(N: int, H: int, V: int, K: int, reorder: bool = False) -> int:
    """flce_distill_workspace_size: as :func:`policy_workspace_size`, for
    :func:`distill_forward_backward` with K teacher entries per row."""
    return int(load_library().flce_distill_workspace_size(N, H, V, K, 1 if reorder else 0))


def distill_forward_backward(X, W, y, teacher_ids, teacher_logits, *, teacher_lse=None, temperature: float = 1.0,
                             kd_weight: float = 1.0, ce_weight: float = 0.0, reduction: str = "mean",
                             grad_row_scale=None, mean_count=None, ignore_index: int = -100, row_loss: bool = False,
                             grads: bool = True, workspace=None, stream=None):
    """flce_distill_forward_backward: distillation through the head, X [N, H] and
    W [V, H] bf16, teacher arguments as :func:`distill_topk` (ce_weight needs
    temperature 1).  Returns (loss fp32[1], status int32[1], row_loss fp32[N] or
    None, dX or None, dW or None)."""
    lib = load_library()
    _check_tensors(X, W, y, workspace=workspace)
    N, H = X.shape
    V = W.shape[0]
    dev = X.device
    K = _teacher(teacher_ids, teacher_logits, teacher_lse, N, dev)
    _vec(mean_count, torch.int32, 1, dev, "mean_count", optional=True)
    red = _scale(grad_row_scale, reduction, N, dev, "grad_row_scale")

    if stream is not None or dev.index != _current_device():
        return _elsewhere(distill_forward_backward, dev, stream, (X, W, y, teacher_ids, teacher_logits),
                          dict(teacher_lse=teacher_lse, temperature=temperature, kd_weight=kd_weight,
                               ce_weight=ce_weight, reduction=reduction, grad_row_scale=grad_row_scale,
                               mean_count=mean_count, ignore_index=ignore_index, row_loss=row_loss, grads=grads,
                               workspace=workspace))
    ws = y.new_empty(distill_workspace_size(N, H, V, K), dtype=torch.uint8) if workspace is None else workspace
    loss = y.new_empty(1, dtype=torch.float32)
    rows = y.new_empty(N, dtype=torch.float32) if row_loss else None
    status = y.new_empty(1)
    dX, dW = _head_outputs(X, W, grads)
    _check(lib.flce_distill_forward_backward(_p(X), _p(W), _p(y), N, H, V, ignore_index, _p(teacher_ids),
                                             _p(teacher_logits), DTYPES[teacher_logits.dtype], K, _p(teacher_lse),
                                             temperature, kd_weight, ce_weight, red, _p(grad_row_scale),
                                             _p(mean_count), _p(loss), _p(rows), _p(status), _p(dX), _p(dW), _p(ws),
                                             ws.numel(), _current_stream_handle(dev.index)),
           "flce_distill_forward_backward")
    return loss, status, rows, dX, dW
