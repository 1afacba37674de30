"""The learner's and the actor's operators beside the replay buffer, over torch tensors.

  distill_forward / distill_backward / distill_step   loss of a student's logits against a
      teacher's top logits, its gradient, both in one pass; the row losses are the next priorities
  verify_draft                                         drafted tokens against the target's
      probabilities, from given random numbers
  scan_forward / scan_backward / scan_step             a gated linear recurrence with episode
      resets, its gradient, its single step
  distill_loss, gated_scan                             the same for torch.autograd

Nothing here computes: arguments are checked and marshalled, outputs allocated, and each call
enqueues one kernel of libgbper on the given (or current) stream without a synchronisation.
include/gbper.h defines every operator; the innermost axis of every tensor must be contiguous, the
outer ones may have any stride.  `out` takes a dict of preallocated outputs under the names that the
call returns.
"""
from __future__ import annotations

import ctypes
import struct

import torch

from . import capi
from .capi import PerError

GATE_DECAY = 0        # a is the state's weight itself
GATE_SIGMOID = capi.PER_SCAN_SIGMOID

_TYPES = {torch.float32: capi.PER_TYPE_F32, torch.float16: capi.PER_TYPE_F16,
          torch.bfloat16: capi.PER_TYPE_BF16}
# the C structures per_distill_shape, per_verify_shape and per_scan_shape, packed
_DISTILL = struct.Struct("@Q4I4qfI")
_VERIFY = struct.Struct("@4I6q2I")
_SCAN = struct.Struct("@Q4I14qQ2I")
assert _DISTILL.size == ctypes.sizeof(capi.per_distill_shape)
assert _VERIFY.size == ctypes.sizeof(capi.per_verify_shape)
assert _SCAN.size == ctypes.sizeof(capi.per_scan_shape)


def _bad(what, want, t):
    if not isinstance(t, torch.Tensor):
        return TypeError(f"{what} must be a tensor {want}")
    return (TypeError if "dtype" in want else ValueError)(
        f"{what} must be {want}, got {tuple(t.shape)} {t.dtype} on {t.device}, strides {t.stride()}")


def _arg(t, what, shape, dtype, dev):
    """Checks a tensor's place, type and shape; its innermost axis must be contiguous."""
    if not isinstance(t, torch.Tensor) or t.get_device() != dev:
        raise _bad(what, f"on cuda:{dev}", t)
    if t.dtype is not dtype:
        raise _bad(what, f"of dtype {dtype}", t)
    if t.shape != shape:
        raise _bad(what, f"of shape {tuple(shape)}", t)
    if not t.is_contiguous() and shape[-1] > 1 and t.stride(-1) != 1:
        raise _bad(what, "contiguous in its last axis", t)
    return t.data_ptr()


def _whole(t, what, shape, dtype, dev):
    """As _arg, for a tensor that must be contiguous; None gives a null pointer."""
    if t is None:
        return None
    p = _arg(t, what, shape, dtype, dev)
    if not t.is_contiguous():
        raise _bad(what, "contiguous", t)
    return p


def _lead(t, what, dims):
    """The type code and device of the argument that the others follow."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise _bad(what, "on a CUDA device", t)
    code = _TYPES.get(t.dtype)
    if code is None:
        raise _bad(what, "of dtype float32, float16 or bfloat16", t)
    if t.dim() != dims:
        raise _bad(what, f"of {dims} axes", t)
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise _bad(what, "contiguous in its last axis", t)
    return code, t.get_device()


def _given(out, name, shape, dtype, dev, like):
    """The output `name`: the caller's, checked, or a new one."""
    t = out.get(name) if out is not None else None
    if t is None:
        return torch.empty(shape, dtype=dtype, device=like.device)   # (new_empty takes twice as long)
    _arg(t, name, torch.Size(shape), dtype, dev)
    return t


class _On:
    """Runs a call on `stream` where that is not the current stream (or device): new outputs are
    allocated for it, and the memory of the inputs, the caller's outputs and the status is held until
    the stream has passed the call."""

    def __init__(self, stream, dev, inputs, out, status):
        self.stream = stream if stream is not None else torch.cuda.current_stream(dev)
        if self.stream.device_index != dev:
            raise ValueError(f"stream must be of cuda:{dev}, the tensors' device, got {self.stream}")
        self.tensors = [*inputs, *(out or {}).values(), status]
        self.guard = None

    def __enter__(self):
        self.guard = torch.cuda.stream(self.stream)
        self.guard.__enter__()
        for t in self.tensors:
            if isinstance(t, torch.Tensor) and t.is_cuda:
                t.record_stream(self.stream)
        return self

    def __exit__(self, *exc):
        return self.guard.__exit__(*exc)


def _elsewhere(stream, dev):
    return stream is not None or dev != torch._C._cuda_getDevice()


def _raw_stream(dev):
    return torch._C._cuda_getCurrentRawStream(dev)


_lib = None


def _library():
    global _lib
    if _lib is None:
        _lib = capi.load()
    return _lib


def _check(status, name):
    if status != capi.PER_OK:
        raise PerError(status, capi.per_last_op_error() or name)


def _status_ptr(status, dev):
    if status is None:
        return None
    return _whole(status, "status", torch.Size((1,)), torch.int32, dev)


class _FirstOnly(torch.autograd.Function):
    """A gradient tied to what it was computed from, whose own derivative is refused.  (torch's
    once_differentiable lets it pass as a constant where the incoming gradient needs none itself.)"""

    @staticmethod
    def forward(ctx, grad, *of):
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, *grads):
        raise RuntimeError("second derivatives of the operators in rl_infra_gb300.ops are not available")


def _first_only(grad, *of):
    """`grad`, where a graph of the backward pass is being made (create_graph=True) not as a constant."""
    if grad is None or not torch.is_grad_enabled():
        return grad
    return _FirstOnly.apply(grad, *of)


# -- distillation from a teacher's top logits --------------------------------------------------

def _distill_args(logits, top_logits, top_idx, teacher_lse):
    code, dev = _lead(logits, "logits", 2)
    n, v = logits.shape
    tcode, tdev = _lead(top_logits, "top_logits", 2)
    k = top_logits.shape[1]
    if top_logits.shape[0] != n or tdev != dev:
        raise _bad("top_logits", f"of shape ({n}, K) on cuda:{dev}", top_logits)
    if not isinstance(top_idx, torch.Tensor) or top_idx.dtype not in (torch.int32, torch.int64):
        raise _bad("top_idx", "of dtype int32 or int64", top_idx)
    ip = _arg(top_idx, "top_idx", top_logits.shape, top_idx.dtype, dev)
    lp = _whole(teacher_lse, "teacher_lse", torch.Size((n,)), torch.float32, dev)
    return code, dev, n, v, tcode, k, top_logits.data_ptr(), ip, lp


def _distill_shape(n, v, k, code, tcode, logits, top_logits, top_idx, sg, tau):
    return _DISTILL.pack(n, v, k, code, tcode, logits.stride(0), top_logits.stride(0), top_idx.stride(0), sg,
                         tau, capi.PER_DISTILL_IDX64 if top_idx.dtype == torch.int64 else 0)


def distill_forward(logits, top_logits, top_idx, temperature=1.0, teacher_lse=None, out=None, status=None,
                    stream=None):
    """{"loss", "lse"} (float [N]) of logits [N, V] against the teacher's top_logits [N, K] at top_idx
    [N, K] (negative: left out); see per_distill_forward."""
    code, dev, n, v, tcode, k, tp, ip, lp = _distill_args(logits, top_logits, top_idx, teacher_lse)
    if _elsewhere(stream, dev):
        with _On(stream, dev, (logits, top_logits, top_idx, teacher_lse), out, status):
            return distill_forward(logits, top_logits, top_idx, temperature, teacher_lse, out, status)
    loss = _given(out, "loss", (n,), torch.float32, dev, logits)
    lse = _given(out, "lse", (n,), torch.float32, dev, logits)
    _check(_library().per_distill_forward(
        _distill_shape(n, v, k, code, tcode, logits, top_logits, top_idx, v, temperature), logits.data_ptr(), tp,
        ip, lp, loss.data_ptr(), lse.data_ptr(), _status_ptr(status, dev), _raw_stream(dev)), "distill_forward")
    return {"loss": loss, "lse": lse}


def distill_backward(logits, top_logits, top_idx, lse, row_scale=None, temperature=1.0, teacher_lse=None,
                     out=None, status=None, stream=None):
    """{"grad"} [N, V] from distill_forward's lse, each row times row_scale (None: 1); see
    per_distill_backward.  out={"grad": logits} writes it in the logits' place."""
    code, dev, n, v, tcode, k, tp, ip, lp = _distill_args(logits, top_logits, top_idx, teacher_lse)
    if lse is None:
        raise TypeError("lse is required")
    ep = _whole(lse, "lse", torch.Size((n,)), torch.float32, dev)
    sp = _whole(row_scale, "row_scale", torch.Size((n,)), torch.float32, dev)
    if _elsewhere(stream, dev):
        with _On(stream, dev, (logits, top_logits, top_idx, lse, row_scale, teacher_lse), out, status):
            return distill_backward(logits, top_logits, top_idx, lse, row_scale, temperature, teacher_lse, out,
                                    status)
    grad = _given(out, "grad", (n, v), logits.dtype, dev, logits)
    _check(_library().per_distill_backward(
        _distill_shape(n, v, k, code, tcode, logits, top_logits, top_idx, grad.stride(0), temperature),
        logits.data_ptr(), tp, ip, lp, ep, sp, grad.data_ptr(), _status_ptr(status, dev), _raw_stream(dev)),
        "distill_backward")
    return {"grad": grad}


def distill_step(logits, top_logits, top_idx, row_scale=None, temperature=1.0, teacher_lse=None, out=None,
                 status=None, stream=None):
    """{"loss", "lse", "grad"} in one pass over the logits; the gradient's rows are times row_scale (an
    importance weight over the batch's size, say).  out={"grad": logits} writes it in the logits'
    place.  See per_distill_step."""
    code, dev, n, v, tcode, k, tp, ip, lp = _distill_args(logits, top_logits, top_idx, teacher_lse)
    sp = _whole(row_scale, "row_scale", torch.Size((n,)), torch.float32, dev)
    if _elsewhere(stream, dev):
        with _On(stream, dev, (logits, top_logits, top_idx, row_scale, teacher_lse), out, status):
            return distill_step(logits, top_logits, top_idx, row_scale, temperature, teacher_lse, out, status)
    loss = _given(out, "loss", (n,), torch.float32, dev, logits)
    lse = _given(out, "lse", (n,), torch.float32, dev, logits)
    grad = _given(out, "grad", (n, v), logits.dtype, dev, logits)
    _check(_library().per_distill_step(
        _distill_shape(n, v, k, code, tcode, logits, top_logits, top_idx, grad.stride(0), temperature),
        logits.data_ptr(), tp, ip, lp, sp, loss.data_ptr(), lse.data_ptr(), grad.data_ptr(),
        _status_ptr(status, dev), _raw_stream(dev)), "distill_step")
    return {"loss": loss, "lse": lse, "grad": grad}


class _DistillLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, top_logits, top_idx, temperature, teacher_lse):
        got = distill_forward(logits, top_logits, top_idx, temperature, teacher_lse)
        ctx.save_for_backward(logits, top_logits, top_idx, got["lse"], teacher_lse)
        ctx.temperature = temperature
        return got["loss"]

    @staticmethod
    def backward(ctx, grad_loss):
        logits, top_logits, top_idx, lse, teacher_lse = ctx.saved_tensors
        got = distill_backward(logits, top_logits, top_idx, lse, grad_loss.contiguous(), ctx.temperature,
                               teacher_lse)
        return _first_only(got["grad"], logits, grad_loss), None, None, None, None


def distill_loss(logits, top_logits, top_idx, temperature=1.0, teacher_lse=None):
    """The row losses [N] (float) as a function that torch.autograd can differentiate by the logits, once (a
    second derivative is refused)."""
    return _DistillLoss.apply(logits, top_logits, top_idx, temperature, teacher_lse)


# -- verification of drafted tokens ------------------------------------------------------------

def verify_draft(target_probs, draft_probs, draft_tokens, accept_u, sample_u, draft_lens=None, out=None,
                 status=None, stream=None):
    """{"accepted" int32 [B], "tokens" int32 [B, D + 1], "accept_p" float [B, D]} for target_probs [B, D + 1, V],
    draft_probs [B, D, V] (None: the draft was certain of its tokens), draft_tokens [B, D] and the
    uniform numbers accept_u [B, D] and sample_u [B]; see per_verify_draft."""
    code, dev = _lead(target_probs, "target_probs", 3)
    b, d1, v = target_probs.shape
    d = d1 - 1
    if d < 0:
        raise _bad("target_probs", "of shape (B, D + 1, V)", target_probs)
    if not isinstance(draft_tokens, torch.Tensor) or draft_tokens.dtype not in (torch.int32, torch.int64):
        raise _bad("draft_tokens", "of dtype int32 or int64", draft_tokens)
    shape = torch.Size((b, d))
    tp = _arg(draft_tokens, "draft_tokens", shape, draft_tokens.dtype, dev)
    up = _arg(accept_u, "accept_u", shape, torch.float32, dev)
    sp = _whole(sample_u, "sample_u", torch.Size((b,)), torch.float32, dev)
    if sp is None:
        raise TypeError("sample_u is required")
    lp = _whole(draft_lens, "draft_lens", torch.Size((b,)), torch.int32, dev)
    q0 = q1 = 0
    qp = None
    if draft_probs is not None:
        qp = _arg(draft_probs, "draft_probs", torch.Size((b, d, v)), target_probs.dtype, dev)
        q0, q1 = draft_probs.stride(0), draft_probs.stride(1)
    if _elsewhere(stream, dev):
        with _On(stream, dev, (target_probs, draft_probs, draft_tokens, accept_u, sample_u, draft_lens), out, status):
            return verify_draft(target_probs, draft_probs, draft_tokens, accept_u, sample_u, draft_lens, out, status)
    got = {"accepted": _given(out, "accepted", (b,), torch.int32, dev, target_probs),
           "tokens": _given(out, "tokens", (b, d1), torch.int32, dev, target_probs),
           "accept_p": _given(out, "accept_p", (b, d), torch.float32, dev, target_probs)}
    if out is not None:
        for name, t in got.items():
            if not t.is_contiguous():
                raise _bad(name, "contiguous", t)
    _check(_library().per_verify_draft(
        _VERIFY.pack(b, d, v, code, target_probs.stride(0), target_probs.stride(1), q0, q1, draft_tokens.stride(0),
                     accept_u.stride(0), capi.PER_VERIFY_TOKENS64 if draft_tokens.dtype == torch.int64 else 0, 0),
        target_probs.data_ptr(), qp, tp, lp, up, sp, got["accepted"].data_ptr(), got["tokens"].data_ptr(),
        got["accept_p"].data_ptr(), _status_ptr(status, dev), _raw_stream(dev)), "verify_draft")
    return got


# -- the gated linear recurrence ---------------------------------------------------------------

_NO_STRIDE = (0, 0)


def _gate_flags(gate, reverse):
    if gate not in (GATE_DECAY, GATE_SIGMOID):
        raise ValueError("gate must be GATE_DECAY or GATE_SIGMOID")
    return gate | capi.PER_SCAN_REVERSE if reverse else gate


def _resets_ptr(resets, shape, dev):
    if resets is None:
        return None
    if not isinstance(resets, torch.Tensor) or resets.get_device() != dev:
        raise _bad("resets", f"on cuda:{dev}", resets)
    if resets.dtype not in (torch.uint8, torch.bool):
        raise _bad("resets", "of dtype uint8 or bool", resets)
    if resets.shape != shape:
        raise _bad("resets", f"of shape {tuple(shape)}", resets)
    return resets.data_ptr()


def scan_forward(a, x, h0=None, resets=None, gate=GATE_DECAY, reverse=False, out=None, stream=None,
                 status=None):
    """{"h" [B, T, C], "last" float [B, C]} of h_t = a_t h_{t-1} + x_t (or with a sigmoid gate); h0 float
    [B, C], resets uint8 or bool [B, T]: a step that drops the state coming into it, an episode's first
    in the direction of the pass (a buffer's dones mark last steps: one step earlier, or as they are with
    reverse).  reverse: from the last step to the first.  status int32 [1] takes PER_DEVFLAG_* bits.
    See per_scan_forward."""
    code, dev = _lead(a, "a", 3)
    b, t, c = a.shape
    xp = _arg(x, "x", a.shape, a.dtype, dev)
    edge = torch.Size((b, c))
    hp = _whole(h0, "h0", edge, torch.float32, dev)
    rp = _resets_ptr(resets, (b, t), dev)
    flags = _gate_flags(gate, reverse)
    if _elsewhere(stream, dev):
        with _On(stream, dev, (a, x, h0, resets), out, status):
            return scan_forward(a, x, h0, resets, gate, reverse, out, None, status)
    h = _given(out, "h", a.shape, a.dtype, dev, a)
    last = _given(out, "last", edge, torch.float32, dev, a)
    if out is not None:
        _whole(last, "last", edge, torch.float32, dev)
    sa, sx, sh = a.stride(), x.stride(), h.stride()
    sr = resets.stride() if rp is not None else _NO_STRIDE
    _check(_library().per_scan_forward(
        _SCAN.pack(t, b, c, code, flags, sa[0], sa[1], sx[0], sx[1], sh[0], sh[1], 0, 0, 0, 0, 0, 0, sr[0], sr[1],
                   _status_ptr(status, dev) or 0, 0, 0),
        a.data_ptr(), xp, hp, rp, h.data_ptr(), last.data_ptr(), _raw_stream(dev)), "scan_forward")
    return {"h": h, "last": last}


def scan_step(a, x, state, resets=None, gate=GATE_DECAY, out=None, stream=None):
    """One step for a batch that is being served: {"h" [B, C], "state" float [B, C]} from a, x [B, C] and the
    state; out={"state": state} updates it in place.  resets [B]."""
    code, dev = _lead(a, "a", 2)
    b, c = a.shape
    xp = _arg(x, "x", a.shape, a.dtype, dev)
    hp = _whole(state, "state", a.shape, torch.float32, dev)
    if hp is None:
        raise TypeError("state is required")
    rp = _resets_ptr(resets, (b,), dev)
    flags = _gate_flags(gate, False)
    if _elsewhere(stream, dev):
        with _On(stream, dev, (a, x, state, resets), out, None):
            return scan_step(a, x, state, resets, gate, out)
    h = _given(out, "h", a.shape, a.dtype, dev, a)
    new = _given(out, "state", a.shape, torch.float32, dev, a)
    if out is not None:
        _whole(new, "state", a.shape, torch.float32, dev)
    _check(_library().per_scan_forward(
        _SCAN.pack(1, b, c, code, flags, a.stride(0), 0, x.stride(0), 0, h.stride(0), 0, 0, 0, 0, 0, 0, 0,
                   resets.stride(0) if rp is not None else 0, 0, 0, 0, 0),
        a.data_ptr(), xp, hp, rp, h.data_ptr(), new.data_ptr(), _raw_stream(dev)), "scan_step")
    return {"h": h, "state": new}


def scan_backward(a, x, h, grad_h, h0=None, resets=None, grad_last=None, gate=GATE_DECAY, reverse=False, out=None,
                  stream=None, status=None, skip=()):
    """{"grad_a", "grad_x" [B, T, C], "grad_h0" float [B, C]} of scan_forward (same arguments) from the h
    that it returned and the gradients of h and of last (None: 0); without those named in `skip`, which
    are not computed.  x may be None where decays are given.  See per_scan_backward."""
    code, dev = _lead(a, "a", 3)
    b, t, c = a.shape
    shape, dt = a.shape, a.dtype
    xp, sx = None, _NO_STRIDE
    if x is not None:
        xp, sx = _arg(x, "x", shape, dt, dev), x.stride()
    yp = _arg(h, "h", shape, dt, dev)
    if grad_h is None:
        grad_h = torch.zeros(c, dtype=dt, device=a.device).expand(shape)   # one row for all steps
    gp = _arg(grad_h, "grad_h", shape, dt, dev)
    edge = torch.Size((b, c))
    hp = _whole(h0, "h0", edge, torch.float32, dev)
    lp = _whole(grad_last, "grad_last", edge, torch.float32, dev)
    rp = _resets_ptr(resets, (b, t), dev)
    flags = _gate_flags(gate, reverse)
    if _elsewhere(stream, dev):
        with _On(stream, dev, (a, x, h, grad_h, h0, resets, grad_last), out, status):
            return scan_backward(a, x, h, grad_h, h0, resets, grad_last, gate, reverse, out, None, status, skip)
    ga = _given(out, "grad_a", shape, dt, dev, a) if "grad_a" not in skip else None
    gx = _given(out, "grad_x", shape, dt, dev, a) if "grad_x" not in skip else None
    g0 = _given(out, "grad_h0", edge, torch.float32, dev, a) if "grad_h0" not in skip else None
    if out is not None:
        _whole(g0, "grad_h0", edge, torch.float32, dev)
    sa, sh, sg = a.stride(), h.stride(), grad_h.stride()
    pa, sga = (ga.data_ptr(), ga.stride()) if ga is not None else (None, _NO_STRIDE)
    px, sgx = (gx.data_ptr(), gx.stride()) if gx is not None else (None, _NO_STRIDE)
    sr = resets.stride() if rp is not None else _NO_STRIDE
    _check(_library().per_scan_backward(
        _SCAN.pack(t, b, c, code, flags, sa[0], sa[1], sx[0], sx[1], sh[0], sh[1], sg[0], sg[1], sga[0], sga[1],
                   sgx[0], sgx[1], sr[0], sr[1], _status_ptr(status, dev) or 0, 0, 0),
        a.data_ptr(), xp, yp, hp, rp, gp, lp, pa, px, None if g0 is None else g0.data_ptr(), _raw_stream(dev)),
        "scan_backward")
    got = {"grad_a": ga, "grad_x": gx, "grad_h0": g0}
    return {k: z for k, z in got.items() if z is not None} if skip else got


class _GatedScan(torch.autograd.Function):
    @staticmethod
    def forward(ctx, a, x, h0, resets, gate, reverse):
        got = scan_forward(a, x, h0, resets, gate, reverse)
        # with given decays the gradient does not depend on x
        ctx.save_for_backward(a, x if gate == GATE_SIGMOID else None, got["h"], h0, resets)
        ctx.set_materialize_grads(False)
        ctx.gate, ctx.reverse = gate, reverse
        return got["h"], got["last"]

    @staticmethod
    def backward(ctx, grad_h, grad_last):
        a, x, h, h0, resets = ctx.saved_tensors
        wanted = dict(zip(("grad_a", "grad_x", "grad_h0"), ctx.needs_input_grad))
        if (grad_h is None and grad_last is None) or not any(wanted.values()):
            return None, None, None, None, None, None
        if grad_h is not None and a.shape[-1] > 1 and grad_h.stride(-1) != 1:
            grad_h = grad_h.contiguous()
        if grad_last is not None:
            grad_last = grad_last.contiguous()
        got = scan_backward(a, x, h, grad_h, h0, resets, grad_last, ctx.gate, ctx.reverse,
                            skip=[name for name, want in wanted.items() if not want])
        of = [t for t in (a, x, h0, grad_h, grad_last) if t is not None]
        return (*(_first_only(got.get(name), *of) for name in wanted), None, None, None)


def gated_scan(a, x, h0=None, resets=None, gate=GATE_DECAY, reverse=False):
    """(h, last) as a function that torch.autograd can differentiate by a, x and h0, once (a second
    derivative is refused).  Arguments as scan_forward's: resets mark first steps."""
    return _GatedScan.apply(a, x, h0, resets, gate, reverse)
