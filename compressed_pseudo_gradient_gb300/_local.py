"""ctypes binding of the local step's operators (include/spl_local.h): argument marshalling only,
by the rules of ``_binding``.  Outputs that the caller does not pass are allocated with torch on
the input's device; so is a workspace that is not passed."""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import torch

from ._binding import _BF16, _F32, _check, _flags_ptr, _stream, library

MAX_TOP = 32
NEWTON_SCHULZ = (3.4445, -4.7750, 2.0315)   # the usual coefficients for 5 steps
_DENSE = (torch.float32, torch.bfloat16)
_IDS = (torch.int64, torch.int32)


class TokenLogprobs(NamedTuple):
    """Results of token_logprobs; logp is None without targets, the last two without top."""
    logp: Optional[torch.Tensor]
    lse: torch.Tensor
    entropy: torch.Tensor
    top_ids: Optional[torch.Tensor]
    top_logp: Optional[torch.Tensor]


def _cuda(t, name, dtypes, dev=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} has dtype {t.dtype}; expected one of {dtypes}")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} must be on {dev}")
    return t


def _rows(t, name):
    """Row stride of a 2-D tensor whose rows are contiguous and do not overlap."""
    if t.dim() != 2:
        raise ValueError(f"{name} must be 2-D")
    rows, cols = t.shape
    if cols > 1 and t.stride(1) != 1:
        raise ValueError(f"the rows of {name} must be contiguous")
    if rows > 1 and t.stride(0) < cols:
        raise ValueError(f"the rows of {name} must not overlap")
    return t.stride(0) if rows > 1 else cols


def _vector(t, name, n, dtypes, dev):
    _cuda(t, name, dtypes, dev)
    if not t.is_contiguous() or t.numel() != n:
        raise ValueError(f"{name} must hold {n} contiguous values")
    return t


def _ids(t, name, n, dev):
    t = _vector(t, name, n, _IDS, dev)
    return t.data_ptr(), 64 if t.dtype == torch.int64 else 32


def _dt(t):
    return _BF16 if t.dtype == torch.bfloat16 else _F32


def _workspace(workspace, need, dev):
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=dev)
    _cuda(workspace, "workspace", (torch.uint8,), dev)
    if not workspace.is_contiguous() or workspace.numel() < need:
        raise ValueError(f"the workspace must hold {need} contiguous bytes")
    return workspace


def token_logprobs(logits, targets=None, *, scale: float = 1.0, top: int = 0,
                   flags=None) -> TokenLogprobs:
    """Log-probabilities of ``targets`` under softmax(scale * logits), with log-sum-exp, entropy
    and the ``top`` most probable tokens per row (spl_token_logprobs).

    logits: fp32 or bf16 [rows, vocab], rows contiguous, any row stride; targets: int64 or int32
    [rows], negative = outside the loss (logp 0), or None.  Ties in the top list go to the lower
    id.  All results are fp32 (top_ids int64 [rows, top])."""
    lib = library()
    _cuda(logits, "logits", _DENSE)
    stride = _rows(logits, "logits")
    rows, vocab = logits.shape
    dev, top = logits.device, int(top)
    ids, bits = (None, 64) if targets is None else _ids(targets, "targets", rows, dev)
    stats = torch.empty((3, rows), dtype=torch.float32, device=dev)
    top_ids = top_logp = None
    if top > 0:
        top_ids = torch.empty((rows, top), dtype=torch.int64, device=dev)
        top_logp = torch.empty((rows, top), dtype=torch.float32, device=dev)
    base, step = stats.data_ptr(), 4 * rows
    with torch.cuda.device(dev):
        st = lib.spl_token_logprobs(logits.data_ptr(), _dt(logits), rows, vocab, stride, ids, bits,
                                    float(scale), top, None if ids is None else base, base + step,
                                    base + 2 * step, None if top_ids is None else top_ids.data_ptr(),
                                    None if top_logp is None else top_logp.data_ptr(),
                                    _flags_ptr(flags, dev), _stream(dev))
    _check("spl_token_logprobs", st)
    return TokenLogprobs(None if ids is None else stats[0], stats[1], stats[2], top_ids, top_logp)


def token_logprobs_grad(logits, targets, lse, d_logp, *, entropy=None, d_entropy=None,
                        scale: float = 1.0, out=None, flags=None):
    """Gradient with respect to the logits of sum(d_logp * logp + d_entropy * entropy), from
    token_logprobs' lse and entropy (spl_token_logprobs_grad).  targets and d_logp may both be
    None (entropy term only), d_entropy too (then entropy is not read).  ``out`` may be the
    logits themselves.  Returns out, of the logits' dtype."""
    lib = library()
    _cuda(logits, "logits", _DENSE)
    stride = _rows(logits, "logits")
    rows, vocab = logits.shape
    dev, f32 = logits.device, (torch.float32,)
    ids, bits = (None, 64) if targets is None else _ids(targets, "targets", rows, dev)
    _vector(lse, "lse", rows, f32, dev)
    if (targets is None) != (d_logp is None):
        raise ValueError("targets and d_logp go together")
    if d_logp is not None:
        _vector(d_logp, "d_logp", rows, f32, dev)
    if d_entropy is not None:
        _vector(d_entropy, "d_entropy", rows, f32, dev)
        if entropy is None:
            raise ValueError("d_entropy needs the forward call's entropy")
        _vector(entropy, "entropy", rows, f32, dev)
    if out is None:   # rows as far apart as the logits': both then move in whole vectors
        out = torch.empty((rows, stride), dtype=logits.dtype, device=dev)[:, :vocab] \
            if rows and vocab <= stride <= vocab + 64 else torch.empty_like(logits)
    _cuda(out, "out", (logits.dtype,), dev)
    if out.shape != logits.shape:
        raise ValueError("out must have the logits' shape")
    ptr = lambda t: None if t is None else t.data_ptr()  # noqa: E731
    with torch.cuda.device(dev):
        st = lib.spl_token_logprobs_grad(logits.data_ptr(), _dt(logits), rows, vocab, stride, ids,
                                         bits, float(scale), lse.data_ptr(), ptr(d_logp),
                                         ptr(entropy), ptr(d_entropy), out.data_ptr(),
                                         _rows(out, "out"), _flags_ptr(flags, dev), _stream(dev))
    _check("spl_token_logprobs_grad", st)
    return out


def embedding(ids, table, *, scale: float = 1.0, out=None, flags=None):
    """scale * table[ids] (spl_embedding): ids int64 or int32 of any shape, table fp32 or bf16
    [vocab, width], rows contiguous.  Ids outside the table give zeros and set
    FLAG_BAD_TOKEN.  Returns [*ids.shape, width] of the table's dtype."""
    lib = library()
    _cuda(table, "table", _DENSE)
    stride = _rows(table, "table")
    vocab, width = table.shape
    dev = table.device
    _cuda(ids, "ids", _IDS, dev)
    n = ids.numel()
    id_ptr, bits = _ids(ids, "ids", n, dev)
    if out is None:
        out = torch.empty((*ids.shape, width), dtype=table.dtype, device=dev)
    _cuda(out, "out", (table.dtype,), dev)
    if out.shape != (*ids.shape, width) or (out.dim() != 2 and not out.is_contiguous()):
        raise ValueError("out must be [*ids.shape, width] (contiguous unless 2-D)")
    out_stride = _rows(out, "out") if out.dim() == 2 else width
    with torch.cuda.device(dev):
        st = lib.spl_embedding(id_ptr, bits, n, table.data_ptr(), _dt(table), vocab, width, stride,
                               float(scale), out.data_ptr(), out_stride, _flags_ptr(flags, dev),
                               _stream(dev))
    _check("spl_embedding", st)
    return out


def embedding_grad(ids, d_out, vocab: int, *, scale: float = 1.0, padding_id: int = -1, out=None,
                   accumulate: bool = False, workspace=None, flags=None):
    """Gradient of embedding with respect to its table (spl_embedding_grad): fp32 [vocab, width],
    scale times the sum of d_out over each id's tokens, the same bits every time.

    d_out: fp32 or bf16 [*ids.shape, width], rows contiguous.  With ``accumulate`` the sums are
    added to ``out`` (which must then be given); otherwise every row is written.  Tokens equal to
    padding_id take no part."""
    lib = library()
    _cuda(d_out, "d_out", _DENSE)
    dev = d_out.device
    _cuda(ids, "ids", _IDS, dev)
    n, width = ids.numel(), d_out.shape[-1]
    if d_out.shape != (*ids.shape, width):
        raise ValueError("d_out must be [*ids.shape, width]")
    if d_out.dim() != 2:
        if not d_out.is_contiguous():
            raise ValueError("d_out must be contiguous unless 2-D")
        d_out = d_out.reshape(n, width)
    id_ptr, bits = _ids(ids, "ids", n, dev)
    if out is None:
        if accumulate:
            raise ValueError("accumulate needs out")
        out = torch.empty((vocab, width), dtype=torch.float32, device=dev)
    _cuda(out, "out", (torch.float32,), dev)
    if out.shape != (vocab, width):
        raise ValueError("out must be [vocab, width]")
    need = lib.spl_embedding_grad_workspace(n, int(vocab), width)
    workspace = _workspace(workspace, need, dev)
    with torch.cuda.device(dev):
        st = lib.spl_embedding_grad(id_ptr, bits, n, d_out.data_ptr(), _dt(d_out), width,
                                    _rows(d_out, "d_out"), int(vocab), float(scale),
                                    int(padding_id), int(bool(accumulate)), out.data_ptr(),
                                    _rows(out, "out"), workspace.data_ptr(), workspace.numel(),
                                    _flags_ptr(flags, dev), _stream(dev))
    _check("spl_embedding_grad", st)
    return out


def orthogonalize_workspace(shape) -> int:
    """Bytes of workspace orthogonalize needs for an update of the given shape."""
    batch, rows, cols = shape if len(shape) == 3 else (1, *shape)
    return int(library().spl_orthogonalize_workspace(batch, rows, cols))


def orthogonalize(update, *, momentum=None, mu: float = 0.95, nesterov: bool = True,
                  steps: int = 5, coefficients=NEWTON_SCHULZ, eps: float = 1e-7, out=None,
                  workspace=None, flags=None):
    """Orthogonalised update of a matrix, or of a stack of matrices, by Newton-Schulz products
    (spl_orthogonalize).

    update: fp32 or bf16 [rows, cols] or [batch, rows, cols], rows contiguous; momentum: fp32,
    contiguous, same shape, updated in place (mu * momentum + update) and, with nesterov, looked
    ahead, or None.  ``workspace`` (uint8, orthogonalize_workspace(update.shape) bytes) may be
    kept between calls on one stream.  Returns out: bf16, contiguous, the update's shape."""
    lib = library()
    _cuda(update, "update", _DENSE)
    if update.dim() not in (2, 3) or update.numel() == 0:
        raise ValueError("update must be a non-empty matrix or stack of matrices")
    dev = update.device
    u = update if update.dim() == 3 else update.unsqueeze(0)
    batch, rows, cols = u.shape
    if cols > 1 and u.stride(2) != 1:
        raise ValueError("the rows of update must be contiguous")
    row_stride = u.stride(1) if rows > 1 else cols
    batch_stride = u.stride(0) if batch > 1 else rows * row_stride
    if row_stride < cols or (batch > 1 and batch_stride < (rows - 1) * row_stride + cols):
        raise ValueError("the rows and matrices of update must not overlap")
    if momentum is not None:
        _cuda(momentum, "momentum", (torch.float32,), dev)
        if momentum.shape != update.shape or not momentum.is_contiguous():
            raise ValueError("momentum must be contiguous, of the update's shape")
    if out is None:
        out = torch.empty(update.shape, dtype=torch.bfloat16, device=dev)
    _cuda(out, "out", (torch.bfloat16,), dev)
    if out.shape != update.shape or not out.is_contiguous():
        raise ValueError("out must be contiguous, of the update's shape")
    workspace = _workspace(workspace, lib.spl_orthogonalize_workspace(batch, rows, cols), dev)
    coef = (ctypes.c_float * 3)(*[float(c) for c in coefficients])
    with torch.cuda.device(dev):
        st = lib.spl_orthogonalize(update.data_ptr(), _dt(update), batch, rows, cols, row_stride,
                                   batch_stride, None if momentum is None else momentum.data_ptr(),
                                   float(mu), int(bool(nesterov)), int(steps), coef, float(eps),
                                   out.data_ptr(), workspace.data_ptr(), workspace.numel(),
                                   _flags_ptr(flags, dev), _stream(dev))
    _check("spl_orthogonalize", st)
    return out
