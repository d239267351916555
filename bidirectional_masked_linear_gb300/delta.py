"""Python binding of the delta rule's operators: the norms of queries and keys
for each head with the position rotation, the gated delta rule over chunks,
both with their gradients, and the delta rule's one-token step
(``include/lion.h``).

Argument marshalling only, with the conventions of :mod:`.ssm`: activations
are token-major ``[B, L, H, d]`` (bfloat16 or float32), each may be a slice of
a wider tensor whose tokens are evenly spaced, weights and states are float32,
``stream``, ``out`` and ``workspace`` as there.  Head sizes are multiples of 8.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple, Optional

import torch

from . import lion
from .lion import _check
from .ssm import _code, _first_only, _handle, _i, _layout, _ll, _new, _ptr, _query, _sz, _tight, _token, _vp, _workspace

QKNORM_L2, QKNORM_RMS = 0, 1
NORMS = {"l2": QKNORM_L2, "rms": QKNORM_RMS}
QKNORM_MAX_D = 256
DELTA_MAX_D = 128

_f = ctypes.c_float


class _QKNormArgs(ctypes.Structure):
    _fields_ = [("q", _vp), ("k", _vp), ("q_weight", _vp), ("k_weight", _vp), ("freqs", _vp), ("positions", _vp),
                ("q_out", _vp), ("k_out", _vp), ("q_token", _ll), ("k_token", _ll), ("B", _i), ("L", _i), ("Hq", _i),
                ("Hk", _i), ("d", _i), ("rot", _i), ("norm", _i), ("interleaved", _i), ("eps", _f), ("dtype", _i),
                ("stream", _vp)]


class _QKNormBwdArgs(ctypes.Structure):
    _fields_ = [("dq_out", _vp), ("dk_out", _vp), ("q", _vp), ("k", _vp), ("q_weight", _vp), ("k_weight", _vp),
                ("freqs", _vp), ("positions", _vp), ("dq", _vp), ("dk", _vp), ("dq_weight", _vp), ("dk_weight", _vp),
                ("q_token", _ll), ("k_token", _ll), ("B", _i), ("L", _i), ("Hq", _i), ("Hk", _i), ("d", _i),
                ("rot", _i), ("norm", _i), ("interleaved", _i), ("eps", _f), ("dtype", _i), ("workspace", _vp),
                ("workspace_bytes", _sz), ("stream", _vp)]


class _DeltaStepArgs(ctypes.Structure):
    _fields_ = [("h", _vp), ("q", _vp), ("k", _vp), ("v", _vp), ("g", _vp), ("beta", _vp), ("out", _vp), ("B", _i),
                ("Hk", _i), ("Hv", _i), ("dk", _i), ("dv", _i), ("scale", _f), ("dtype", _i), ("stream", _vp)]


class _DeltaArgs(ctypes.Structure):
    _fields_ = [("q", _vp), ("k", _vp), ("v", _vp), ("g", _vp), ("beta", _vp), ("h0", _vp), ("lengths", _vp),
                ("out", _vp), ("h_out", _vp), ("saved", _vp), ("q_token", _ll), ("k_token", _ll), ("v_token", _ll),
                ("g_token", _ll), ("beta_token", _ll), ("B", _i), ("L", _i), ("Hk", _i), ("Hv", _i), ("dk", _i),
                ("dv", _i), ("scale", _f), ("reverse", _i), ("dtype", _i), ("workspace", _vp),
                ("workspace_bytes", _sz), ("stream", _vp)]


class _DeltaBwdArgs(ctypes.Structure):
    _fields_ = [("dout", _vp), ("q", _vp), ("k", _vp), ("v", _vp), ("g", _vp), ("beta", _vp), ("h0", _vp),
                ("lengths", _vp), ("saved", _vp), ("dq", _vp), ("dk_out", _vp), ("dv_out", _vp), ("dg", _vp),
                ("dbeta", _vp), ("dh0", _vp), ("q_token", _ll), ("k_token", _ll), ("v_token", _ll), ("g_token", _ll),
                ("beta_token", _ll), ("B", _i), ("L", _i), ("Hk", _i), ("Hv", _i), ("dk", _i), ("dv", _i),
                ("scale", _f), ("reverse", _i), ("dtype", _i), ("workspace", _vp), ("workspace_bytes", _sz),
                ("stream", _vp)]


EXPORTS = ("lion_qknorm_fwd", "lion_qknorm_bwd", "lion_qknorm_bwd_workspace_bytes", "lion_delta_fwd",
           "lion_delta_saved_bytes", "lion_delta_workspace_bytes", "lion_delta_bwd", "lion_delta_bwd_workspace_bytes",
           "lion_delta_step")

_QKNorm_pack, _QKNormBwd_pack, _Delta_pack, _DeltaBwd_pack, _DeltaStep_pack = (
    _layout(c) for c in (_QKNormArgs, _QKNormBwdArgs, _DeltaArgs, _DeltaBwdArgs, _DeltaStepArgs))

_lib = None


def load():
    """liblion.so with this module's entry points declared."""
    global _lib
    if _lib is None:
        lib = lion.load()
        for name in ("qknorm_fwd", "qknorm_bwd", "delta_fwd", "delta_bwd", "delta_step"):
            f = getattr(lib, "lion_" + name)
            f.argtypes, f.restype = [ctypes.c_char_p], _i
        for name, n in (("qknorm_bwd_workspace", 6), ("delta_saved", 7), ("delta_workspace", 8),
                        ("delta_bwd_workspace", 8)):
            f = getattr(lib, f"lion_{name}_bytes")
            f.argtypes, f.restype = [_i] * n, _sz
        _lib = lib
    return _lib


def _like(stream, x):
    """An uninitialised contiguous tensor of x's shape and type that belongs to `stream`."""
    if stream is None:
        return torch.empty_like(x, memory_format=torch.contiguous_format)
    return _new(stream, x.shape, x.dtype, x)


def _result(name, out, stream, x):
    """The caller's tensor for a result like x, or a new one, and its address."""
    if out is None:
        out = _like(stream, x)
        return out, out.data_ptr()
    return out, _tight(name, out, x.dtype, x.shape)


# ------------------------------------------------------- norms of q and k

class QKNormGrads(NamedTuple):
    dq: torch.Tensor
    dk: torch.Tensor
    dq_weight: Optional[torch.Tensor]
    dk_weight: Optional[torch.Tensor]


def _norm_kind(norm):
    kind = NORMS.get(norm)
    if kind is None:
        raise ValueError(f"norm must be 'l2' or 'rms', got {norm!r}")
    return kind


def _qknorm_args(q, k, q_weight, k_weight, freqs, positions):
    """Sizes, distances between tokens, addresses in the structures' order."""
    B, L, Hq, d = q.shape
    Hk, T, f32 = k.shape[2], q.dtype, torch.float32
    qp, ql = _token("q", q, T, (B, L, Hq, d))
    kp, kl = _token("k", k, T, (B, L, Hk, d))
    rot = 0
    if freqs is not None:
        if freqs.dim() != 1:
            raise ValueError(f"freqs must have one dimension, got {tuple(freqs.shape)}")
        rot = 2 * freqs.shape[0]
    elif positions is not None:
        raise ValueError("positions are given without freqs")
    return ((B, L, Hq, Hk, d, rot), (ql, kl),
            (qp, kp, 0 if q_weight is None else _tight("q_weight", q_weight, f32, (d,)),
             0 if k_weight is None else _tight("k_weight", k_weight, f32, (d,)),
             0 if freqs is None else _tight("freqs", freqs, f32, (rot // 2,)),
             0 if positions is None else _tight("positions", positions, torch.int32, (B, L))))


def qknorm_bwd_workspace_bytes(B, L, Hq, Hk, d, weights=True) -> int:
    load()
    return _query("qknorm_bwd", B, L, Hq, Hk, d, int(weights))


def qknorm_fwd(q, k, q_weight=None, k_weight=None, norm="l2", eps=1e-6, freqs=None, positions=None,
               interleaved=False, q_out=None, k_out=None, stream=None):
    """``(q_out, k_out)``: every head of ``q`` [B, L, Hq, d] and ``k``
    [B, L, Hk, d] divided by its length (``norm="l2"``) or the root of its
    mean square (``"rms"``), times its weight [d] if one is given, and with
    ``freqs`` (float32 [rot/2], rot a multiple of 8) its first rot values
    turned by position times frequency.  ``positions``: int32 [B, L], by
    default a token's index.  The pairs that turn are the two halves' values
    of the same place or, with ``interleaved``, adjacent ones."""
    lib, code = load(), _code(q)
    sizes, tokens, ptrs = _qknorm_args(q, k, q_weight, k_weight, freqs, positions)
    qo, qp = _result("q_out", q_out, stream, q)
    ko, kp = _result("k_out", k_out, stream, k)
    a = _QKNorm_pack(*ptrs, qp, kp, *tokens, *sizes, _norm_kind(norm), int(interleaved), eps, code, _handle(stream, q))
    _check(lib.lion_qknorm_fwd(a))
    return qo, ko


def qknorm_bwd(dq_out, dk_out, q, k, q_weight=None, k_weight=None, norm="l2", eps=1e-6, freqs=None, positions=None,
               interleaved=False, workspace=None, stream=None):
    """Gradients through :func:`qknorm_fwd`: :class:`QKNormGrads` (a weight's
    is None where there is no weight)."""
    lib, code = load(), _code(q)
    sizes, tokens, ptrs = _qknorm_args(q, k, q_weight, k_weight, freqs, positions)
    T = q.dtype
    dqp, dkp = _tight("dq_out", dq_out, T, q.shape), _tight("dk_out", dk_out, T, k.shape)
    dq, dk = _like(stream, q), _like(stream, k)
    dwq = None if q_weight is None else _like(stream, q_weight)
    dwk = None if k_weight is None else _like(stream, k_weight)
    weights = int(dwq is not None or dwk is not None)
    ws, nb, _keep = _workspace(workspace, q, stream, "qknorm_bwd", *sizes[:5], weights)
    a = _QKNormBwd_pack(dqp, dkp, *ptrs, dq.data_ptr(), dk.data_ptr(), _ptr(dwq), _ptr(dwk), *tokens, *sizes,
                        _norm_kind(norm), int(interleaved), eps, code, ws, nb, _handle(stream, q))
    _check(lib.lion_qknorm_bwd(a))
    return QKNormGrads(dq, dk, dwq, dwk)


def _no_gradient(ctx, **of):
    """Raises if a gradient is wanted for one of these inputs (by their index), which have none here."""
    for name, i in of.items():
        if any(ctx.needs_input_grad[i:i + 1]):   # as many as the call had arguments
            raise RuntimeError(f"{name} has no gradient here: pass it detached")


class QKNorm(torch.autograd.Function):
    """The norms and rotation as a differentiable op: ``apply(q, k, q_weight,
    k_weight, norm, eps, freqs, positions, interleaved)`` gives ``(q_out,
    k_out)``.  ``freqs`` has no gradient: backward raises if it wants one."""

    @staticmethod
    def forward(ctx, q, k, q_weight=None, k_weight=None, norm="l2", eps=1e-6, freqs=None, positions=None,
                interleaved=False):
        ctx.save_for_backward(q, k, q_weight, k_weight, freqs, positions)
        ctx.how = norm, eps, interleaved
        return qknorm_fwd(q, k, q_weight, k_weight, norm, eps, freqs, positions, interleaved)

    @staticmethod
    @_first_only
    def backward(ctx, dq_out, dk_out):
        _no_gradient(ctx, eps=5, freqs=6)
        q, k, q_weight, k_weight, freqs, positions = ctx.saved_tensors
        norm, eps, interleaved = ctx.how
        g = qknorm_bwd(dq_out.contiguous(), dk_out.contiguous(), q, k, q_weight, k_weight, norm, eps, freqs, positions,
                       interleaved)
        return g.dq, g.dk, g.dq_weight, g.dk_weight, None, None, None, None, None


# ------------------------------------------------------------ the delta rule

class DeltaOut(NamedTuple):
    out: torch.Tensor
    h: Optional[torch.Tensor]
    saved: Optional[torch.Tensor]


class DeltaGrads(NamedTuple):
    dq: torch.Tensor
    dk: torch.Tensor
    dv: torch.Tensor
    dg: torch.Tensor
    dbeta: torch.Tensor
    dh0: Optional[torch.Tensor]


def _delta_args(q, k, v, g, beta, h0, lengths):
    """Sizes, distances between tokens, addresses in the structures' order."""
    B, L, Hk, dk = q.shape
    Hv, dv = v.shape[2:]
    T = q.dtype
    qp, ql = _token("q", q, T, (B, L, Hk, dk))
    kp, kl = _token("k", k, T, (B, L, Hk, dk))
    vp, vl = _token("v", v, T, (B, L, Hv, dv))
    gp, gl = _token("g", g, T, (B, L, Hv))
    bp, bl = _token("beta", beta, T, (B, L, Hv))
    return ((B, L, Hk, Hv, dk, dv), (ql, kl, vl, gl, bl),
            (qp, kp, vp, gp, bp, 0 if h0 is None else _tight("h0", h0, torch.float32, (B, Hv, dk, dv)),
             0 if lengths is None else _tight("lengths", lengths, torch.int32, (B,))))


@functools.lru_cache(maxsize=256)
def delta_saved_bytes(B, L, Hk, Hv, dk, dv, dtype=lion.DTYPE_BF16) -> int:
    return int(load().lion_delta_saved_bytes(B, L, Hk, Hv, dk, dv, dtype))


def delta_workspace_bytes(B, L, Hk, Hv, dk, dv, dtype=lion.DTYPE_BF16, save=False) -> int:
    load()
    return _query("delta", B, L, Hk, Hv, dk, dv, dtype, int(save))


def delta_bwd_workspace_bytes(B, L, Hk, Hv, dk, dv, dtype=lion.DTYPE_BF16, have_saved=True) -> int:
    load()
    return _query("delta_bwd", B, L, Hk, Hv, dk, dv, dtype, int(have_saved))


def delta_fwd(q, k, v, g, beta, scale=None, h0=None, lengths=None, reverse=False, return_state=False, save=False,
              out=None, workspace=None, stream=None):
    """The gated delta rule over ``q``, ``k`` [B, L, Hk, dk], ``v``
    [B, L, Hv, dv], ``g`` (the decays' logarithms) and ``beta`` [B, L, Hv]:
    with a state S [dk, dv] for each value head, which uses query and key head
    h // (Hv // Hk),  S = exp(g) S,  S += beta k (v - S^T k)^T,  out = scale
    S^T q.  Returns :class:`DeltaOut`: ``out`` [B, L, Hv, dv], with
    ``return_state`` the state ``h`` [B, Hv, dk, dv] after the last token,
    with ``save`` what spares :func:`delta_bwd` the recomputation.  ``scale``:
    dk ** -0.5 by default; ``h0``: the state before the first token;
    ``lengths``: int32 [B], the tokens each sequence has; ``reverse``: walk
    from the last token.  Keys longer than sqrt(2 / beta) make the state grow
    (:func:`qknorm_fwd`)."""
    lib, code = load(), _code(q)
    sizes, tokens, ptrs = _delta_args(q, k, v, g, beta, h0, lengths)
    B, L, Hk, Hv, dk, dv = sizes
    y, yp = _result("out", out, stream, v)
    h = _new(stream, (B, Hv, dk, dv), torch.float32, q) if return_state else None
    saved = _new(stream, (delta_saved_bytes(*sizes, code),), torch.uint8, q) if save else None
    ws, nb, _keep = _workspace(workspace, q, stream, "delta", *sizes, code, int(save))
    a = _Delta_pack(*ptrs, yp, _ptr(h), _ptr(saved), *tokens, *sizes,
                    dk ** -0.5 if scale is None else scale, int(reverse), code, ws, nb, _handle(stream, q))
    _check(lib.lion_delta_fwd(a))
    return DeltaOut(y, h, saved)


def delta_bwd(dout, q, k, v, g, beta, scale=None, h0=None, lengths=None, reverse=False, saved=None, workspace=None,
              stream=None):
    """Gradients through :func:`delta_fwd`'s ``out`` given ``dout``
    [B, L, Hv, dv]: :class:`DeltaGrads` (``dh0`` None where there is no
    ``h0``).  ``saved``: the forward's (recomputed if None)."""
    lib, code = load(), _code(q)
    sizes, tokens, ptrs = _delta_args(q, k, v, g, beta, h0, lengths)
    T = q.dtype
    dop = _tight("dout", dout, T, v.shape)
    sp = 0 if saved is None else _tight("saved", saved, torch.uint8, (delta_saved_bytes(*sizes, code),))
    dq, dk, dv, dg, db = (_like(stream, t) for t in (q, k, v, g, beta))
    dh0 = None if h0 is None else _like(stream, h0)
    ws, nb, _keep = _workspace(workspace, q, stream, "delta_bwd", *sizes, code, int(saved is not None))
    a = _DeltaBwd_pack(dop, *ptrs, sp, dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), dg.data_ptr(), db.data_ptr(),
                       _ptr(dh0), *tokens, *sizes, sizes[4] ** -0.5 if scale is None else scale, int(reverse), code, ws,
                       nb, _handle(stream, q))
    _check(lib.lion_delta_bwd(a))
    return DeltaGrads(dq, dk, dv, dg, db, dh0)


def delta_step(h, q, k, v, g, beta, scale=None, out=None, stream=None):
    """One token of the gated delta rule: ``q``, ``k`` [B, Hk, dk], ``v``
    [B, Hv, dv], ``g`` (the decay's logarithm) and ``beta`` [B, Hv]; returns
    its output [B, Hv, dv], with the state ``h`` [B, Hv, dk, dv] updated in
    place.  ``scale``: of the output, dk ** -0.5 by default."""
    lib, code = load(), _code(q)
    T, f32 = q.dtype, torch.float32
    B, Hk, dk = q.shape
    Hv, dv = v.shape[1:]
    y, yp = _result("out", out, stream, v)
    a = _DeltaStep_pack(_tight("h", h, f32, (B, Hv, dk, dv)), _tight("q", q, T, (B, Hk, dk)),
                        _tight("k", k, T, (B, Hk, dk)), _tight("v", v, T, (B, Hv, dv)), _tight("g", g, T, (B, Hv)),
                        _tight("beta", beta, T, (B, Hv)), yp, B, Hk, Hv, dk, dv, dk ** -0.5 if scale is None else scale,
                        code, _handle(stream, q))
    _check(lib.lion_delta_step(a))
    return y


class GatedDelta(torch.autograd.Function):
    """The gated delta rule as a differentiable op: ``apply(q, k, v, g, beta,
    scale, h0, lengths, reverse)`` gives ``out``.  ``scale`` has no gradient:
    backward raises if it wants one."""

    @staticmethod
    def forward(ctx, q, k, v, g, beta, scale=None, h0=None, lengths=None, reverse=False):
        f = delta_fwd(q, k, v, g, beta, scale, h0, lengths, reverse, save=any(ctx.needs_input_grad))
        ctx.save_for_backward(q, k, v, g, beta, h0, lengths, f.saved)
        ctx.how = scale, reverse
        return f.out

    @staticmethod
    @_first_only
    def backward(ctx, dout):
        _no_gradient(ctx, scale=5)
        q, k, v, g, beta, h0, lengths, saved = ctx.saved_tensors
        scale, reverse = ctx.how
        r = delta_bwd(dout.contiguous(), q, k, v, g, beta, scale, h0, lengths, reverse, saved)
        return r.dq, r.dk, r.dv, r.dg, r.dbeta, None, r.dh0, None, None
