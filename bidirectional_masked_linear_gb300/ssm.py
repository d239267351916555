"""Python binding of the state space block's operators: layer norm, the short
causal depthwise convolution and the selective scan, with their gradients, and
the one-token steps that serving uses (``include/lion.h``).

Argument marshalling only, as in :mod:`.lion`: tensors are PyTorch CUDA
tensors, every step runs in ``liblion.so``, and the calls raise if it is not
built.  Activations are ``[B, L, D]`` (bfloat16 or float32), parameters and
the scan's states float32.  An activation may be a slice of a wider tensor
(one half of a projection's output): its channels have to be adjacent and its
sequences evenly laid out.

``stream``: the stream to run on (the current one by default).  Outputs and
workspaces belong to it; inputs made on another stream have to be ready on it.
"""
from __future__ import annotations

import contextlib
import ctypes
from typing import NamedTuple, Optional

import torch

from . import lion
from .lion import _check, _dtype_code, _ptr

ACT_NONE, ACT_SILU = 0, 1
ACTIVATIONS = {"none": ACT_NONE, None: ACT_NONE, "silu": ACT_SILU}
LAYERNORM_MAX_COLS = 16384
STATE_SIZES = (8, 16, 32, 64)
STATE_EVERY = 16

_vp, _i, _ll, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_size_t


class _NormArgs(ctypes.Structure):
    _fields_ = [("x", _vp), ("weight", _vp), ("bias", _vp), ("y", _vp), ("mean", _vp), ("rstd", _vp),
                ("x_row", _ll), ("rows", _i), ("cols", _i), ("eps", ctypes.c_float), ("dtype", _i), ("stream", _vp)]


class _NormBwdArgs(ctypes.Structure):
    _fields_ = [("dy", _vp), ("x", _vp), ("weight", _vp), ("mean", _vp), ("rstd", _vp), ("dx", _vp),
                ("dweight", _vp), ("dbias", _vp), ("x_row", _ll), ("rows", _i), ("cols", _i), ("dtype", _i),
                ("workspace", _vp), ("workspace_bytes", _sz), ("stream", _vp)]


class _ConvArgs(ctypes.Structure):
    _fields_ = [("x", _vp), ("weight", _vp), ("bias", _vp), ("state", _vp), ("lengths", _vp), ("y", _vp),
                ("state_out", _vp), ("x_token", _ll), ("B", _i), ("L", _i), ("D", _i), ("K", _i), ("act", _i),
                ("reverse", _i), ("dtype", _i), ("stream", _vp)]


class _ConvBwdArgs(ctypes.Structure):
    _fields_ = [("dy", _vp), ("x", _vp), ("weight", _vp), ("bias", _vp), ("state", _vp), ("lengths", _vp),
                ("dx", _vp), ("dweight", _vp), ("dbias", _vp), ("dstate", _vp), ("x_token", _ll), ("B", _i),
                ("L", _i), ("D", _i), ("K", _i), ("act", _i), ("reverse", _i), ("dtype", _i), ("workspace", _vp),
                ("workspace_bytes", _sz), ("stream", _vp)]


class _ScanArgs(ctypes.Structure):
    _fields_ = [("u", _vp), ("dt", _vp), ("A", _vp), ("Bm", _vp), ("Cm", _vp), ("Dskip", _vp), ("z", _vp),
                ("dt_bias", _vp), ("h0", _vp), ("lengths", _vp), ("out", _vp), ("h_out", _vp), ("states", _vp),
                ("u_token", _ll), ("dt_token", _ll), ("z_token", _ll), ("b_token", _ll), ("c_token", _ll),
                ("B", _i), ("L", _i), ("D", _i), ("N", _i), ("G", _i), ("dt_softplus", _i), ("reverse", _i),
                ("dtype", _i), ("workspace", _vp), ("workspace_bytes", _sz), ("stream", _vp)]


class _ScanBwdArgs(ctypes.Structure):
    _fields_ = [("dout", _vp), ("u", _vp), ("dt", _vp), ("A", _vp), ("Bm", _vp), ("Cm", _vp), ("Dskip", _vp),
                ("z", _vp), ("dt_bias", _vp), ("h0", _vp), ("lengths", _vp), ("states", _vp), ("du", _vp),
                ("ddt", _vp), ("dA", _vp), ("dB", _vp), ("dC", _vp), ("dDskip", _vp), ("dz", _vp),
                ("ddt_bias", _vp), ("dh0", _vp),
                ("u_token", _ll), ("dt_token", _ll), ("z_token", _ll), ("b_token", _ll), ("c_token", _ll),
                ("B", _i), ("L", _i), ("D", _i), ("N", _i), ("G", _i), ("dt_softplus", _i), ("reverse", _i),
                ("dtype", _i), ("workspace", _vp), ("workspace_bytes", _sz), ("stream", _vp)]


class _ScanStepArgs(ctypes.Structure):
    _fields_ = [("h", _vp), ("u", _vp), ("dt", _vp), ("A", _vp), ("Bm", _vp), ("Cm", _vp), ("Dskip", _vp),
                ("z", _vp), ("dt_bias", _vp), ("out", _vp), ("B", _i), ("D", _i), ("N", _i), ("G", _i),
                ("dt_softplus", _i), ("dtype", _i), ("stream", _vp)]


EXPORTS = ("lion_layernorm_fwd", "lion_layernorm_bwd", "lion_layernorm_bwd_workspace_bytes", "lion_conv_fwd",
           "lion_conv_bwd", "lion_conv_bwd_workspace_bytes", "lion_conv_step", "lion_scan_fwd",
           "lion_scan_workspace_bytes", "lion_scan_bwd", "lion_scan_bwd_workspace_bytes", "lion_scan_step")

_lib = None


def load():
    """liblion.so with this module's entry points declared."""
    global _lib
    if _lib is None:
        lib = lion.load()
        for name, args in (("layernorm_fwd", _NormArgs), ("layernorm_bwd", _NormBwdArgs), ("conv_fwd", _ConvArgs),
                           ("conv_bwd", _ConvBwdArgs), ("scan_fwd", _ScanArgs), ("scan_bwd", _ScanBwdArgs),
                           ("scan_step", _ScanStepArgs)):
            f = getattr(lib, "lion_" + name)
            f.argtypes, f.restype = [ctypes.POINTER(args)], _i
        lib.lion_conv_step.argtypes, lib.lion_conv_step.restype = [_vp] * 5 + [_i] * 5 + [_vp], _i
        for name, n in (("layernorm_bwd", 2), ("conv_bwd", 4), ("scan", 5), ("scan_bwd", 6)):
            f = getattr(lib, f"lion_{name}_workspace_bytes")
            f.argtypes, f.restype = [_i] * n, _sz
        _lib = lib
    return _lib


# ------------------------------------------------------------ argument checks

def _on(stream):
    """The context that makes outputs and workspaces belong to `stream`."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _handle(stream):
    return (torch.cuda.current_stream() if stream is None else stream).cuda_stream


def _act(activation):
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of 'silu', 'none', None, got {activation!r}")
    return ACTIVATIONS[activation]


def _f32(name, t, shape):
    if t is None:
        return
    if t.dtype != torch.float32:
        raise TypeError(f"{name} must be float32, got {t.dtype}")
    _tight(name, t, shape)


def _tight(name, t, shape):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _same(name, t, dtype):
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} as the other activations, got {t.dtype}")


def _lengths(lengths, B):
    if lengths is None:
        return
    if lengths.dtype != torch.int32:
        raise TypeError(f"lengths must be int32, got {lengths.dtype}")
    _tight("lengths", lengths, (B,))


def _token(name, t, B, L, width):
    """The distance between tokens of a [B, L, ...] activation whose last
    dimensions, `width` values in all, are adjacent."""
    if t.is_contiguous():
        return width
    s, run = t.stride(), 1
    for k in range(t.dim() - 1, 1, -1):
        if t.shape[k] != 1 and s[k] != run:
            raise ValueError(f"{name}: the values of a token must be adjacent")
        run *= t.shape[k]
    if L == 1:
        ld = s[0] if B > 1 else width
    else:
        ld = s[1]
        if B > 1 and s[0] != L * ld:
            raise ValueError(f"{name}: sequences must lie L tokens apart")
    if ld < width:
        raise ValueError(f"{name}: tokens must not overlap")
    return ld


def _cuda(*tensors):
    for t in tensors:
        if t is not None and not t.is_cuda:
            raise ValueError("tensors must be on the GPU")


def _workspace(workspace, nbytes, like):
    """(pointer, bytes) of the caller's workspace, or of one from PyTorch's
    allocator (kept alive by the third value)."""
    if workspace is not None:
        return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace
    if nbytes == 0:
        return None, 0, None
    ws = torch.empty(nbytes, dtype=torch.uint8, device=like.device)
    return ws.data_ptr(), nbytes, ws


# ------------------------------------------------------------------ layer norm

def _rows(x):
    """(rows, cols, distance between rows) of x's last dimension."""
    cols = x.shape[-1]
    if x.is_contiguous():
        return x.numel() // max(1, cols), cols, cols
    if x.dim() == 2 and x.stride(1) == 1 and x.stride(0) >= cols:
        return x.shape[0], cols, x.stride(0)
    raise ValueError("x must be contiguous, or two-dimensional with adjacent columns")


def layernorm_bwd_workspace_bytes(rows, cols) -> int:
    return int(load().lion_layernorm_bwd_workspace_bytes(rows, cols))


def layernorm_fwd(x, weight, bias=None, eps=1e-5, save_stats=False, out=None, stream=None):
    """Layer norm over the last dimension: ``y``, or ``(y, mean, rstd)`` with
    ``save_stats`` (float32, one per row, for :func:`layernorm_bwd`)."""
    lib = load()
    rows, cols, ld = _rows(x)
    code = _dtype_code(x)
    _f32("weight", weight, (cols,))
    _f32("bias", bias, (cols,))
    _cuda(x, weight, bias, out)
    with _on(stream):
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device) if out is None else out
        mean = torch.empty(x.shape[:-1], dtype=torch.float32, device=x.device) if save_stats else None
        rstd = torch.empty_like(mean) if save_stats else None
    _same("out", y, x.dtype)
    _tight("out", y, x.shape)
    a = _NormArgs(_ptr(x), _ptr(weight), _ptr(bias), _ptr(y), _ptr(mean), _ptr(rstd), ld, rows, cols, eps, code,
                  _handle(stream))
    _check(lib.lion_layernorm_fwd(ctypes.byref(a)))
    return (y, mean, rstd) if save_stats else y


def layernorm_bwd(dy, x, weight, mean, rstd, bias=True, workspace=None, stream=None):
    """``(dx, dweight, dbias)`` given ``dy`` and the forward's ``mean`` and
    ``rstd``; ``dbias`` is None with ``bias=False``."""
    lib = load()
    rows, cols, ld = _rows(x)
    code = _dtype_code(x)
    _same("dy", dy, x.dtype)
    _tight("dy", dy, x.shape)
    _f32("weight", weight, (cols,))
    _f32("mean", mean, x.shape[:-1])
    _f32("rstd", rstd, x.shape[:-1])
    _cuda(dy, x, weight, mean, rstd)
    with _on(stream):
        dx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        dw = torch.empty(cols, dtype=torch.float32, device=x.device)
        db = torch.empty_like(dw) if bias else None
        ws, nb, keep = _workspace(workspace, 0 if workspace is not None
                                  else lib.lion_layernorm_bwd_workspace_bytes(rows, cols), x)
    a = _NormBwdArgs(_ptr(dy), _ptr(x), _ptr(weight), _ptr(mean), _ptr(rstd), _ptr(dx), _ptr(dw), _ptr(db), ld,
                     rows, cols, code, ws, nb, _handle(stream))
    _check(lib.lion_layernorm_bwd(ctypes.byref(a)))
    return dx, dw, db


class LayerNorm(torch.autograd.Function):
    """Layer norm as a differentiable op: ``apply(x, weight, bias, eps)``."""

    @staticmethod
    def forward(ctx, x, weight, bias, eps=1e-5):
        x = x.contiguous()
        y, mean, rstd = layernorm_fwd(x, weight, bias, eps, save_stats=True)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.bias = bias is not None
        return y

    @staticmethod
    def backward(ctx, dy):
        x, weight, mean, rstd = ctx.saved_tensors
        dx, dw, db = layernorm_bwd(dy.contiguous(), x, weight, mean, rstd, ctx.bias)
        return dx, dw, db, None


# ----------------------------------------------------------------- convolution

class ConvGrads(NamedTuple):
    dx: torch.Tensor
    dweight: torch.Tensor
    dbias: Optional[torch.Tensor]
    dstate: Optional[torch.Tensor]


def _conv_args(x, weight, bias, state, lengths):
    B, L, D = x.shape
    if weight.dim() != 2:
        raise ValueError("weight must have shape [D, K]")
    K = weight.shape[1]
    _f32("weight", weight, (D, K))
    _f32("bias", bias, (D,))
    if state is not None:
        _same("state", state, x.dtype)
        _tight("state", state, (B, K - 1, D))
    _lengths(lengths, B)
    _cuda(x, weight, bias, state, lengths)
    return B, L, D, K, _token("x", x, B, L, D)


def conv_bwd_workspace_bytes(B, L, D, K) -> int:
    return int(load().lion_conv_bwd_workspace_bytes(B, L, D, K))


def conv_fwd(x, weight, bias=None, activation="silu", state=None, lengths=None, reverse=False, return_state=False,
             out=None, stream=None):
    """Causal depthwise convolution of ``x`` [B, L, D] with ``weight`` [D, K]
    (K 2 to 4): ``y``, or ``(y, state)`` with ``return_state`` (the last K-1
    inputs, [B, K-1, D], for the next call or :func:`conv_step`).  ``state``:
    the inputs before the first token.  ``lengths``: int32 [B], the tokens
    each sequence has.  ``reverse``: walk from the last token."""
    lib = load()
    code = _dtype_code(x)
    B, L, D, K, ld = _conv_args(x, weight, bias, state, lengths)
    with _on(stream):
        y = torch.empty((B, L, D), dtype=x.dtype, device=x.device) if out is None else out
        new = torch.empty((B, K - 1, D), dtype=x.dtype, device=x.device) if return_state else None
    _same("out", y, x.dtype)
    _tight("out", y, (B, L, D))
    _cuda(y)
    a = _ConvArgs(_ptr(x), _ptr(weight), _ptr(bias), _ptr(state), _ptr(lengths), _ptr(y), _ptr(new), ld, B, L, D, K,
                  _act(activation), int(reverse), code, _handle(stream))
    _check(lib.lion_conv_fwd(ctypes.byref(a)))
    return (y, new) if return_state else y


def conv_bwd(dy, x, weight, bias=None, activation="silu", state=None, lengths=None, reverse=False, workspace=None,
             stream=None):
    """Gradients through :func:`conv_fwd`'s ``y``: :class:`ConvGrads`
    (``dbias`` and ``dstate`` None where there is no bias or state)."""
    lib = load()
    code = _dtype_code(x)
    B, L, D, K, ld = _conv_args(x, weight, bias, state, lengths)
    _same("dy", dy, x.dtype)
    _tight("dy", dy, (B, L, D))
    _cuda(dy)
    with _on(stream):
        dx = torch.empty((B, L, D), dtype=x.dtype, device=x.device)
        dw = torch.empty((D, K), dtype=torch.float32, device=x.device)
        db = None if bias is None else torch.empty(D, dtype=torch.float32, device=x.device)
        ds = None if state is None else torch.empty_like(state)
        ws, nb, keep = _workspace(workspace, 0 if workspace is not None
                                  else lib.lion_conv_bwd_workspace_bytes(B, L, D, K), x)
    a = _ConvBwdArgs(_ptr(dy), _ptr(x), _ptr(weight), _ptr(bias), _ptr(state), _ptr(lengths), _ptr(dx), _ptr(dw),
                     _ptr(db), _ptr(ds), ld, B, L, D, K, _act(activation), int(reverse), code, ws, nb,
                     _handle(stream))
    _check(lib.lion_conv_bwd(ctypes.byref(a)))
    return ConvGrads(dx, dw, db, ds)


def conv_step(x, state, weight, bias=None, activation="silu", out=None, stream=None):
    """One token ``x`` [B, D]: its output, with the window in ``state``
    [B, K-1, D] moved on in place."""
    lib = load()
    code = _dtype_code(x)
    B, D = x.shape
    if weight.dim() != 2:
        raise ValueError("weight must have shape [D, K]")
    K = weight.shape[1]
    _f32("weight", weight, (D, K))
    _f32("bias", bias, (D,))
    _tight("x", x, (B, D))
    _same("state", state, x.dtype)
    _tight("state", state, (B, K - 1, D))
    with _on(stream):
        y = torch.empty((B, D), dtype=x.dtype, device=x.device) if out is None else out
    _same("out", y, x.dtype)
    _tight("out", y, (B, D))
    _cuda(x, weight, bias, state, y)
    _check(lib.lion_conv_step(_ptr(x), _ptr(state), _ptr(weight), _ptr(bias), _ptr(y), B, D, K, _act(activation),
                              code, _handle(stream)))
    return y


class CausalConv(torch.autograd.Function):
    """The convolution as a differentiable op (the state, if any, gets its
    gradient): ``apply(x, weight, bias, activation, state, lengths, reverse)``."""

    @staticmethod
    def forward(ctx, x, weight, bias, activation="silu", state=None, lengths=None, reverse=False):
        ctx.save_for_backward(x, weight, bias, state, lengths)
        ctx.how = activation, reverse
        return conv_fwd(x, weight, bias, activation, state, lengths, reverse)

    @staticmethod
    def backward(ctx, dy):
        x, weight, bias, state, lengths = ctx.saved_tensors
        activation, reverse = ctx.how
        g = conv_bwd(dy.contiguous(), x, weight, bias, activation, state, lengths, reverse)
        return g.dx, g.dweight, g.dbias, None, g.dstate, None, None


# -------------------------------------------------------------- selective scan

class ScanOut(NamedTuple):
    out: torch.Tensor
    h: Optional[torch.Tensor]
    states: Optional[torch.Tensor]


class ScanGrads(NamedTuple):
    du: torch.Tensor
    ddt: torch.Tensor
    dA: torch.Tensor
    dB: torch.Tensor
    dC: torch.Tensor
    dDskip: Optional[torch.Tensor]
    dz: Optional[torch.Tensor]
    ddt_bias: Optional[torch.Tensor]
    dh0: Optional[torch.Tensor]


def _scan_args(u, dt, A, Bm, Cm, Dskip, z, dt_bias, h0, lengths):
    B, L, D = u.shape
    if A.dim() != 2 or A.shape[0] != D:
        raise ValueError("A must have shape [D, N]")
    N = A.shape[1]
    if Bm.dim() == 3:   # one group
        Bm, Cm = Bm.unsqueeze(2), Cm.unsqueeze(2)
    G = Bm.shape[2]
    for name, t, shape in (("dt", dt, (B, L, D)), ("Bm", Bm, (B, L, G, N)), ("Cm", Cm, (B, L, G, N)),
                           ("z", z, (B, L, D))):
        if t is not None:
            _same(name, t, u.dtype)
            if tuple(t.shape) != shape:
                raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    _f32("A", A, (D, N))
    _f32("Dskip", Dskip, (D,))
    _f32("dt_bias", dt_bias, (D,))
    _f32("h0", h0, (B, D, N))
    _lengths(lengths, B)
    _cuda(u, dt, A, Bm, Cm, Dskip, z, dt_bias, h0, lengths)
    tokens = (_token("u", u, B, L, D), _token("dt", dt, B, L, D), 0 if z is None else _token("z", z, B, L, D),
              _token("Bm", Bm, B, L, G * N), _token("Cm", Cm, B, L, G * N))
    return B, L, D, N, G, tokens


def scan_workspace_bytes(B, L, D, N, G=1) -> int:
    return int(load().lion_scan_workspace_bytes(B, L, D, N, G))


def scan_bwd_workspace_bytes(B, L, D, N, G=1, have_states=True) -> int:
    return int(load().lion_scan_bwd_workspace_bytes(B, L, D, N, G, int(have_states)))


def scan_fwd(u, dt, A, Bm, Cm, Dskip=None, z=None, dt_bias=None, dt_softplus=True, h0=None, lengths=None,
             reverse=False, return_state=False, save_states=False, out=None, workspace=None, stream=None):
    """The selective scan of ``u`` [B, L, D] with step sizes ``dt`` [B, L, D],
    ``A`` [D, N] (N 8, 16, 32 or 64) and ``Bm``, ``Cm`` [B, L, G, N] or
    [B, L, N]:  h = exp(delta A) h + delta u B,  out = (C h + Dskip u) silu(z)
    with delta = softplus(dt + dt_bias).  Returns :class:`ScanOut`: ``out``,
    with ``return_state`` the state ``h`` [B, D, N] after the last token, with
    ``save_states`` the ``states`` that spare :func:`scan_bwd` the
    recomputation.  ``h0``: the state before the first token; ``lengths``,
    ``reverse``: as :func:`conv_fwd`."""
    lib = load()
    code = _dtype_code(u)
    B, L, D, N, G, tokens = _scan_args(u, dt, A, Bm, Cm, Dskip, z, dt_bias, h0, lengths)
    with _on(stream):
        y = torch.empty((B, L, D), dtype=u.dtype, device=u.device) if out is None else out
        h = torch.empty((B, D, N), dtype=torch.float32, device=u.device) if return_state else None
        states = (torch.empty((B, -(-L // STATE_EVERY), D, N), dtype=torch.float32, device=u.device) if save_states
                  else None)
        ws, nb, keep = _workspace(workspace, 0 if workspace is not None
                                  else lib.lion_scan_workspace_bytes(B, L, D, N, G), u)
    _same("out", y, u.dtype)
    _tight("out", y, (B, L, D))
    _cuda(y)
    a = _ScanArgs(_ptr(u), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(Dskip), _ptr(z), _ptr(dt_bias), _ptr(h0),
                  _ptr(lengths), _ptr(y), _ptr(h), _ptr(states), *tokens, B, L, D, N, G, int(dt_softplus),
                  int(reverse), code, ws, nb, _handle(stream))
    _check(lib.lion_scan_fwd(ctypes.byref(a)))
    return ScanOut(y, h, states)


def scan_bwd(dout, u, dt, A, Bm, Cm, Dskip=None, z=None, dt_bias=None, dt_softplus=True, h0=None, lengths=None,
             reverse=False, states=None, workspace=None, stream=None):
    """Gradients through :func:`scan_fwd`'s ``out`` given ``dout`` [B, L, D]:
    :class:`ScanGrads`, with None for what was not given.  ``states``: the
    forward's (recomputed if None)."""
    lib = load()
    code = _dtype_code(u)
    B, L, D, N, G, tokens = _scan_args(u, dt, A, Bm, Cm, Dskip, z, dt_bias, h0, lengths)
    _same("dout", dout, u.dtype)
    _tight("dout", dout, (B, L, D))
    _f32("states", states, (B, -(-L // STATE_EVERY), D, N))
    _cuda(dout, states)
    with _on(stream):
        du = torch.empty((B, L, D), dtype=u.dtype, device=u.device)
        ddt = torch.empty_like(du)
        dz = None if z is None else torch.empty_like(du)
        dB = torch.empty(Bm.shape, dtype=u.dtype, device=u.device)
        dC = torch.empty_like(dB)
        dA = torch.empty((D, N), dtype=torch.float32, device=u.device)
        dD = None if Dskip is None else torch.empty(D, dtype=torch.float32, device=u.device)
        dbias = None if dt_bias is None else torch.empty(D, dtype=torch.float32, device=u.device)
        dh0 = None if h0 is None else torch.empty((B, D, N), dtype=torch.float32, device=u.device)
        ws, nb, keep = _workspace(workspace, 0 if workspace is not None else
                                  lib.lion_scan_bwd_workspace_bytes(B, L, D, N, G, int(states is not None)), u)
    a = _ScanBwdArgs(_ptr(dout), _ptr(u), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(Dskip), _ptr(z),
                     _ptr(dt_bias), _ptr(h0), _ptr(lengths), _ptr(states), _ptr(du), _ptr(ddt), _ptr(dA), _ptr(dB),
                     _ptr(dC), _ptr(dD), _ptr(dz), _ptr(dbias), _ptr(dh0), *tokens, B, L, D, N, G,
                     int(dt_softplus), int(reverse), code, ws, nb, _handle(stream))
    _check(lib.lion_scan_bwd(ctypes.byref(a)))
    return ScanGrads(du, ddt, dA, dB, dC, dD, dz, dbias, dh0)


def scan_step(h, u, dt, A, Bm, Cm, Dskip=None, z=None, dt_bias=None, dt_softplus=True, out=None, stream=None):
    """One token: ``u``, ``dt``, ``z`` [B, D], ``Bm``, ``Cm`` [B, G, N] or
    [B, N]; returns its output [B, D], with the state ``h`` [B, D, N]
    updated in place."""
    lib = load()
    code = _dtype_code(u)
    B, D = u.shape
    if A.dim() != 2 or A.shape[0] != D:
        raise ValueError("A must have shape [D, N]")
    N = A.shape[1]
    G = Bm.shape[1] if Bm.dim() == 3 else 1
    for name, t in (("u", u), ("dt", dt), ("z", z)):
        if t is not None:
            _same(name, t, u.dtype)
            _tight(name, t, (B, D))
    for name, t in (("Bm", Bm), ("Cm", Cm)):
        _same(name, t, u.dtype)
        _tight(name, t, (B, G, N) if Bm.dim() == 3 else (B, N))
    _f32("h", h, (B, D, N))
    _f32("A", A, (D, N))
    _f32("Dskip", Dskip, (D,))
    _f32("dt_bias", dt_bias, (D,))
    with _on(stream):
        y = torch.empty((B, D), dtype=u.dtype, device=u.device) if out is None else out
    _same("out", y, u.dtype)
    _tight("out", y, (B, D))
    _cuda(h, u, dt, A, Bm, Cm, Dskip, z, dt_bias, y)
    a = _ScanStepArgs(_ptr(h), _ptr(u), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(Dskip), _ptr(z), _ptr(dt_bias),
                      _ptr(y), B, D, N, G, int(dt_softplus), code, _handle(stream))
    _check(lib.lion_scan_step(ctypes.byref(a)))
    return y


class SelectiveScan(torch.autograd.Function):
    """The scan as a differentiable op: ``apply(u, dt, A, Bm, Cm, Dskip, z,
    dt_bias, dt_softplus, h0, lengths, reverse)`` gives ``out``."""

    @staticmethod
    def forward(ctx, u, dt, A, Bm, Cm, Dskip=None, z=None, dt_bias=None, dt_softplus=True, h0=None, lengths=None,
                reverse=False):
        f = scan_fwd(u, dt, A, Bm, Cm, Dskip, z, dt_bias, dt_softplus, h0, lengths, reverse, save_states=True)
        ctx.save_for_backward(u, dt, A, Bm, Cm, Dskip, z, dt_bias, h0, lengths, f.states)
        ctx.how = dt_softplus, reverse
        return f.out

    @staticmethod
    def backward(ctx, dout):
        u, dt, A, Bm, Cm, Dskip, z, dt_bias, h0, lengths, states = ctx.saved_tensors
        softplus, reverse = ctx.how
        g = scan_bwd(dout.contiguous(), u, dt, A, Bm, Cm, Dskip, z, dt_bias, softplus, h0, lengths, reverse, states)
        return (g.du, g.ddt, g.dA, g.dB, g.dC, g.dDskip, g.dz, g.ddt_bias, None, g.dh0, None, None)
