"""Losses on the steps of a sequence model, on the gfx950 library (libsdtw.so).

Beside an alignment loss on its outputs, a sequence model trains a head over
the entries of a vocabulary, or over the bins of a quantised series, step by
step.  Here are that head's log-probabilities with entropy and top
alternatives (``token_logprobs``), and the distillation from a teacher's top
entries (``distillation_loss``, ``DistillationLoss``,
``distillation_value_and_grad``), as differentiable functions of the logits.
The two fit together: a teacher's ``token_logprobs(z, top_k=K,
temperature=T)`` gives what a student's ``distillation_loss(..., top_tokens,
top_logprobs, temperature=T, tail=True)`` takes.

Logits are float32, bfloat16 or float16 of shape (..., V) on a GPU (there is
no CPU path), V contiguous; the leading dimensions may be strided, as in the
view ``logits[:, :-1]``, and are copied only where three or more of them
cannot be walked with two strides.  Values are float32, gradients have the
logits' type.  PyTorch provides memory, streams and autograd; every step runs
in the library's HIP kernels.  Derivatives are reverse-mode and of first order;
tensors with a forward-mode tangent are refused.
"""
from __future__ import annotations

import math
from typing import NamedTuple, Optional

import torch
import torch.autograd.forward_ad as fwad
from torch.autograd.function import once_differentiable

from . import _lib as L

_DTYPES = {torch.float32: L.SDTW_DTYPE_F32, torch.bfloat16: L.SDTW_DTYPE_BF16,
           torch.float16: L.SDTW_DTYPE_F16}
_ID_BYTES = {torch.int32: 4, torch.int64: 8}
TOP_K_MAX = 128
LIST_MAX = 256


class TokenLogProbs(NamedTuple):
    """Results of ``token_logprobs``; fields that were not asked for are None."""
    logprobs: Optional[torch.Tensor]
    entropy: torch.Tensor
    top_logprobs: Optional[torch.Tensor]
    top_tokens: Optional[torch.Tensor]


class _Here:
    """Stands for torch.cuda.device(d) where d is the current device already
    (entering that context costs as much as two allocations)."""

    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


_here = _Here()


def _on(device):
    return _here if torch.cuda.current_device() == device.index else torch.cuda.device(device)


def _stream(device) -> int:
    # The handle alone: building torch.cuda.current_stream's object takes 2 us,
    # a tenth of a small call.
    return torch._C._cuda_getCurrentRawStream(device.index)


def _check_tangent(name, t):
    # The kernels have no forward-mode derivative: a tangent would be lost
    # without a word.  (The level alone where there is none: 0.1 us of 0.4.)
    if fwad._current_level >= 0 and fwad.unpack_dual(t).tangent is not None:
        raise ValueError(f"forward-mode derivatives are not supported, and {name} carry a tangent")


def _check_logits(logits, temperature) -> float:
    if not isinstance(logits, torch.Tensor):
        raise ValueError("logits must be a tensor")
    _check_tangent("logits", logits)
    t = float(temperature)
    if not (math.isfinite(t) and 1e-6 <= t <= 1e6):
        raise ValueError(f"temperature must be within [1e-6, 1e6], got {temperature}")
    if logits.dim() < 1 or logits.shape[-1] < 1:
        raise ValueError(f"logits must be (..., V) with V >= 1, got {tuple(logits.shape)}")
    if logits.dtype not in _DTYPES:
        raise ValueError(f"logits must be float32, bfloat16 or float16, got {logits.dtype}")
    return t


def _check_ignore(ignore_index) -> int:
    try:
        i = int(ignore_index)
        ok = i == ignore_index and -(1 << 63) <= i < 1 << 63
    except (TypeError, ValueError, OverflowError):
        ok = False
    if not ok:
        raise ValueError(f"ignore_index must be an integer of 64 bits, got {ignore_index}")
    return i


def _check_device(logits):
    # Last of the checks, so that the others can be met without a GPU.
    if logits.device.type != "cuda":
        raise ValueError("logits must be on a GPU (there is no CPU path)")


def _check_beside(name, t, logits, shape, dtypes):
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a tensor")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {tuple(shape)} beside logits {tuple(logits.shape)}, "
                         f"got {tuple(t.shape)}")
    if t.dtype not in dtypes:
        names = " or ".join(str(d).replace("torch.", "") for d in dtypes)
        raise ValueError(f"{name} must be {names}, got {t.dtype}")
    if t.device != logits.device:
        raise ValueError(f"{name} and logits are on different devices: {t.device} vs {logits.device}")


def _walk(t: torch.Tensor, lead: int):
    """(t, stride of the outer leading dimensions as one, stride of the last
    leading dimension): t itself where two strides reach every row and the
    rest is contiguous, else a contiguous copy of it."""
    if t.numel() == 0:
        return t, 0, 0      # (contiguous by any strides: a copy would be the same)
    shape, stride = t.shape, t.stride()
    ok = t.dim() == lead or shape[-1] == 1 or stride[-1] == 1
    outer = 0
    have = 1            # rows the outer dimensions have so far
    for i in range(lead - 2, -1, -1):
        if shape[i] == 1:
            continue
        if have == 1:
            outer = stride[i]
        elif stride[i] != outer * have:
            ok = False
        have *= shape[i]
    if not ok:
        t = t.contiguous()
        return _walk(t, lead)
    return t, outer, (stride[lead - 1] if lead else 0)


def _size(logits):
    shape = logits.shape
    lead = len(shape) - 1
    N = shape[-2] if lead else 1
    B = 1
    for i in range(lead - 1):
        B *= shape[i]
    return lead, B, N, shape[-1]


def _row_grad(g):
    """(g, step) of an upstream gradient with one value a row: step 0 where
    one value is broadcast to all rows, 1 for contiguous ones."""
    if g is None:
        return None, 0
    if g.dtype != torch.float32:
        g = g.float()
    if all(st == 0 or n == 1 for n, st in zip(g.shape, g.stride())):
        return g, 0
    return g.contiguous(), 1


def _ptr(t):
    return None if t is None else t.data_ptr()


def _workspace(nbytes, device):
    """(pointer, size, owner) of a workspace; none where nothing is kept in it."""
    if nbytes == 0:
        raise ValueError("sizes the library does not take (rows and V below 2^31)")
    if nbytes == L.SDTW_ROWS_WORKSPACE_MIN:
        return None, nbytes, None
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    return ws.data_ptr(), nbytes, ws


class _Rows(NamedTuple):
    """How the kernels walk a call's tensors: logits, and the tensors with one
    or K entries a row beside them, each as (tensor, outer and inner stride)."""
    B: int
    N: int
    V: int
    logits: tuple
    first: tuple          # tokens, or the teacher's ids; None without
    second: tuple         # the teacher's values; None without


def _rows(logits, first=None, second=None):
    lead, B, N, V = _size(logits)
    return _Rows(B, N, V, _walk(logits, lead), None if first is None else _walk(first, lead),
                 None if second is None else _walk(second, lead))


def _logit_args(r):
    z, ld_b, ld_n = r.logits
    return z.data_ptr(), _DTYPES[z.dtype], r.B, r.N, r.V, ld_b, ld_n


def _token_args(r):
    if r.first is None:
        return None, 0, 0, 0
    tok, tok_b, tok_n = r.first
    return tok.data_ptr(), _ID_BYTES[tok.dtype], tok_b, tok_n


def _token_forward(logits, tokens, temperature, top_k, ignore_index, keep):
    """(logprobs, entropy, top_logprobs, top_tokens, stats, rows); stats only if keep."""
    dev = logits.device
    shape = logits.shape[:-1]
    with _on(dev):
        r = _rows(logits, tokens)
        entropy = torch.empty(shape, dtype=torch.float32, device=dev)
        logprobs = None if tokens is None else torch.empty(shape, dtype=torch.float32, device=dev)
        top_lp = top_tok = stats = None
        if top_k:
            top_lp = torch.empty((*shape, top_k), dtype=torch.float32, device=dev)
            top_tok = torch.empty((*shape, top_k), dtype=torch.int64, device=dev)
        if keep:
            stats = torch.empty((r.B * r.N, 4), dtype=torch.float32, device=dev)
        if r.B * r.N:
            ws, nbytes, _owner = _workspace(
                L.sdtw_token_workspace_bytes(r.B, r.N, r.V, top_k), dev)
            L.check(L.sdtw_token_logprobs(
                *_logit_args(r), *_token_args(r), ignore_index, temperature, top_k, ws, nbytes,
                _ptr(logprobs), entropy.data_ptr(), _ptr(stats), _ptr(top_lp), _ptr(top_tok),
                _stream(dev)), "sdtw_token_logprobs")
    return logprobs, entropy, top_lp, top_tok, stats, r


class _TokenLogProbsFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, temperature, top_k, ignore_index):
        ctx.set_materialize_grads(False)
        logprobs, entropy, top_lp, top_tok, stats, r = _token_forward(
            logits, tokens, temperature, top_k, ignore_index, True)
        if top_tok is not None:
            ctx.mark_non_differentiable(top_tok)
        # (A copy that the kernels walk is kept in place of what it copies.)
        z = r.logits[0]
        tok = None if tokens is None else r.first[0]
        ctx.save_for_backward(z, tok, top_tok, stats)
        ctx.rows = r._replace(logits=r.logits[1:], first=None if tok is None else r.first[1:])
        ctx.args = (temperature, top_k, ignore_index)
        ctx.shape = logits.shape
        return logprobs, entropy, top_lp, top_tok

    @staticmethod
    @once_differentiable
    def backward(ctx, g_lp, g_ent, g_top, _):
        if g_lp is None and g_ent is None and g_top is None:
            return None, None, None, None, None
        z, tok, top_tok, stats = ctx.saved_tensors
        temperature, top_k, ignore_index = ctx.args
        r = ctx.rows
        r = r._replace(logits=(z, *r.logits), first=None if tok is None else (tok, *r.first))
        dev = z.device
        with _on(dev):
            grad = torch.empty(ctx.shape, dtype=z.dtype, device=dev)
            if r.B * r.N:
                g_lp, lp_step = _row_grad(g_lp)
                g_ent, ent_step = _row_grad(g_ent)
                if g_top is not None:
                    g_top = g_top.float().contiguous()
                L.check(L.sdtw_token_backward(
                    *_logit_args(r), *_token_args(r), ignore_index, temperature, top_k,
                    stats.data_ptr(), _ptr(top_tok), _ptr(g_lp), lp_step, _ptr(g_ent), ent_step,
                    _ptr(g_top), grad.data_ptr(), _stream(dev)), "sdtw_token_backward")
        return grad, None, None, None, None


def token_logprobs(logits: torch.Tensor, tokens: Optional[torch.Tensor] = None,
                   temperature: float = 1.0, top_k: int = 0,
                   ignore_index: int = -100) -> TokenLogProbs:
    """Log-probabilities of given tokens under softmax(logits / temperature),
    with each row's entropy and its most likely entries.

    ``logits`` (..., V); ``tokens`` (...) int32 or int64, or None.  Returns
    ``TokenLogProbs``: ``logprobs`` (...), at most 0 (None without tokens; 0 where the
    token is ``ignore_index``, NaN where it is any other id outside the
    vocabulary), ``entropy`` (...) in nats, and with ``top_k`` (at most 128)
    ``top_logprobs`` and ``top_tokens`` (..., top_k), falling, ties to the
    lower id.  Differentiable in logprobs, entropy and top_logprobs.

    Entries of -inf have probability zero.  A row of nothing else has
    log-probabilities -inf, entropy 0 and gradient 0; a row with a NaN or
    +inf has NaN.  A row whose upstream gradients are all zero gets a zero
    gradient."""
    t = _check_logits(logits, temperature)
    k = int(top_k)
    V = logits.shape[-1]
    if k != top_k or not 0 <= k <= min(TOP_K_MAX, V):
        raise ValueError(f"top_k must be an integer from 0 to min({TOP_K_MAX}, V = {V}), got {top_k}")
    ignore = _check_ignore(ignore_index)
    if tokens is not None:
        _check_beside("tokens", tokens, logits, logits.shape[:-1], _ID_BYTES)
    _check_device(logits)
    if torch.is_grad_enabled() and logits.requires_grad:
        out = _TokenLogProbsFunction.apply(logits, tokens, t, k, ignore)
        return TokenLogProbs(*out)
    return TokenLogProbs(*_token_forward(logits, tokens, t, k, ignore, False)[:4])


def _check_distill(logits, ids, values, temperature, ignore_index, weights=None):
    t = _check_logits(logits, temperature)
    ignore = _check_ignore(ignore_index)
    if not isinstance(ids, torch.Tensor) or ids.dim() < 1:
        raise ValueError("teacher_tokens must be a tensor (..., K)")
    K = ids.shape[-1]
    if not 1 <= K <= LIST_MAX:
        raise ValueError(f"a teacher's list has 1 to {LIST_MAX} entries, got {K}")
    shape = (*logits.shape[:-1], K)
    _check_beside("teacher_tokens", ids, logits, shape, _ID_BYTES)
    _check_beside("teacher_logits", values, logits, shape, _DTYPES)
    _check_tangent("teacher_logits", values)
    if torch.is_grad_enabled() and values.requires_grad:
        raise ValueError("teacher_logits are constants of the loss: detach them")
    if weights is not None:
        _check_beside("weights", weights, logits, logits.shape[:-1], (torch.float32,))
        _check_tangent("weights", weights)
    _check_device(logits)
    return t, ignore


def _distill(r, t, tail, ignore_index, loss, stats, gl, grad):
    """One sdtw_distill call: loss and stats, the gradient, or all of them."""
    if r.B * r.N == 0:
        return
    ids, id_b, id_n = r.first
    values, val_b, val_n = r.second
    dev = ids.device
    K = ids.shape[-1]
    gl, gl_step = _row_grad(gl)
    ws, nbytes, _owner = None, 0, None
    if loss is not None:
        ws, nbytes, _owner = _workspace(L.sdtw_distill_workspace_bytes(r.B, r.N, r.V, K), dev)
    L.check(L.sdtw_distill(
        *_logit_args(r), ids.data_ptr(), _ID_BYTES[ids.dtype], id_b, id_n, values.data_ptr(),
        _DTYPES[values.dtype], val_b, val_n, K, ignore_index, t, tail, ws, nbytes, _ptr(loss),
        _ptr(stats), _ptr(gl), gl_step, _ptr(grad), _stream(dev)), "sdtw_distill")


class _DistillationFunction(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, ids, values, t, tail, ignore_index):
        dev = logits.device
        with _on(dev):
            r = _rows(logits, ids, values)
            loss = torch.empty(logits.shape[:-1], dtype=torch.float32, device=dev)
            stats = torch.empty((r.B * r.N, 8), dtype=torch.float32, device=dev)
            _distill(r, t, tail, ignore_index, loss, stats, None, None)
        # (A copy that the kernels walk is kept in place of what it copies.)
        ctx.save_for_backward(r.logits[0], r.first[0], r.second[0], stats)
        ctx.rows = r._replace(logits=r.logits[1:], first=r.first[1:], second=r.second[1:])
        ctx.args = (t, tail, ignore_index)
        ctx.shape = logits.shape
        return loss

    @staticmethod
    @once_differentiable
    def backward(ctx, grad_loss):
        z, ids, values, stats = ctx.saved_tensors
        r = ctx.rows
        r = r._replace(logits=(z, *r.logits), first=(ids, *r.first), second=(values, *r.second))
        with _on(z.device):
            grad = torch.empty(ctx.shape, dtype=z.dtype, device=z.device)
            _distill(r, *ctx.args, None, stats, grad_loss, grad)
        return grad, None, None, None, None, None


def distillation_loss(logits: torch.Tensor, teacher_tokens: torch.Tensor,
                      teacher_logits: torch.Tensor, temperature: float = 1.0,
                      tail: bool = False, ignore_index: int = -100) -> torch.Tensor:
    """Per-row divergence (...) of softmax(logits / temperature) from a
    teacher that is known by its K (at most 256) top entries: ids
    ``teacher_tokens`` (..., K) int32 or int64, padded with ``ignore_index``
    where a row has fewer, and ``teacher_logits`` (..., K) of any of the
    logits' types.

    ``tail=False``: the teacher's probabilities q are the softmax of its
    listed values / temperature (logits or log-probabilities alike), and the
    loss is sum q (log q - log p).  ``tail=True``: the values are the
    teacher's log-probabilities at this temperature over its whole vocabulary,
    and what they leave is one more class: the loss adds q_r (log q_r -
    log p_r) with q_r = 1 - sum q and p_r the student's probability off the
    list.  Where that is nothing (below 2^-126: a list of every entry, or the
    others masked), a q_r no larger than the roundings behind the values counts
    as zero; a larger one is a loss of +inf if there is no other entry at all.
    The factor temperature^2 that some recipes apply is the caller's.

    Differentiable in the logits; the teacher is constant.  An id listed twice
    adds in q and counts once in p; an id outside the vocabulary makes its row
    NaN.  A row without entries has loss 0 and gradient 0, whatever its logits
    hold."""
    t, ignore = _check_distill(logits, teacher_tokens, teacher_logits, temperature, ignore_index)
    if torch.is_grad_enabled() and logits.requires_grad:
        return _DistillationFunction.apply(logits, teacher_tokens, teacher_logits, t,
                                           int(bool(tail)), ignore)
    with _on(logits.device):
        loss = torch.empty(logits.shape[:-1], dtype=torch.float32, device=logits.device)
        _distill(_rows(logits, teacher_tokens, teacher_logits), t, int(bool(tail)), ignore,
                 loss, None, None, None)
    return loss


def distillation_value_and_grad(logits: torch.Tensor, teacher_tokens: torch.Tensor,
                                teacher_logits: torch.Tensor,
                                weights: Optional[torch.Tensor] = None,
                                temperature: float = 1.0, tail: bool = False,
                                ignore_index: int = -100):
    """(loss, grad): ``distillation_loss`` per row (unweighted) and the
    gradient of sum(weights * loss) with respect to the logits, in one call.
    Up to 131072 entries a row that is one launch: what a block holds of its row
    in registers (32768 entries of 16 bits, 16384 of 32, with 256 threads) is read
    once, the rest twice, the second time from the last-level cache where it
    still is there.  Longer rows take three launches and are read twice.  For
    training steps that know each row's weight beforehand
    (1 / rows for a mean); ``logits.backward(grad)`` then continues below the
    head.  ``weights`` (...) float32, or None for ones; no graph is recorded."""
    t, ignore = _check_distill(logits, teacher_tokens, teacher_logits, temperature, ignore_index,
                               weights)
    dev = logits.device
    with _on(dev), torch.no_grad():
        r = _rows(logits, teacher_tokens, teacher_logits)
        loss = torch.empty(logits.shape[:-1], dtype=torch.float32, device=dev)
        grad = torch.empty(logits.shape, dtype=logits.dtype, device=dev)
        stats = None
        if r.V > L.SDTW_ROWS_WHOLE:       # split rows pass their statistics on
            stats = torch.empty((r.B * r.N, 8), dtype=torch.float32, device=dev)
        _distill(r, t, int(bool(tail)), ignore, loss, stats, weights, grad)
    return loss, grad


class DistillationLoss(torch.nn.Module):
    """``DistillationLoss(temperature=1.0, tail=False, ignore_index=-100)``:
    ``distillation_loss`` as a module, called as ``loss_fn(logits,
    teacher_tokens, teacher_logits)`` -> (...)."""

    def __init__(self, temperature: float = 1.0, tail: bool = False, ignore_index: int = -100):
        super().__init__()
        t = float(temperature)
        if not (math.isfinite(t) and 1e-6 <= t <= 1e6):
            raise ValueError(f"temperature must be within [1e-6, 1e6], got {temperature}")
        self.temperature = t
        self.tail = bool(tail)
        self.ignore_index = _check_ignore(ignore_index)

    def forward(self, logits, teacher_tokens, teacher_logits):
        return distillation_loss(logits, teacher_tokens, teacher_logits, self.temperature,
                                 self.tail, self.ignore_index)

    def extra_repr(self) -> str:
        return (f"temperature={self.temperature}, tail={self.tail}, "
                f"ignore_index={self.ignore_index}")
