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
Tensors and stream belong to the current device (``torch.cuda.device``), on
which the library launches; any other is refused.  ``out``: the tensor to
write to, which must not overlap an input.
"""
from __future__ import annotations

import ctypes
import functools
import struct
from typing import NamedTuple, Optional

import torch

from . import lion
from .lion import _check

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


def _layout(args):
    """A structure's fields in struct's notation: packing bytes takes a third
    of the time of a ctypes structure, a microsecond of a one-token call."""
    codes = {_vp: "P", _i: "i", _ll: "q", _sz: "N", ctypes.c_float: "f"}
    packed = struct.Struct("@" + "".join(codes[t] for _, t in args._fields_))
    assert packed.size <= ctypes.sizeof(args)   # but for the padding behind the last field
    return packed.pack


EXPORTS = ("lion_layernorm_fwd", "lion_layernorm_bwd", "lion_layernorm_bwd_workspace_bytes", "lion_conv_fwd",
           "lion_conv_bwd", "lion_conv_bwd_workspace_bytes", "lion_conv_step", "lion_scan_fwd",
           "lion_scan_workspace_bytes", "lion_scan_bwd", "lion_scan_bwd_workspace_bytes", "lion_scan_step")

_Norm_pack, _NormBwd_pack, _Conv_pack, _ConvBwd_pack, _Scan_pack, _ScanBwd_pack, _ScanStep_pack = (
    _layout(c) for c in (_NormArgs, _NormBwdArgs, _ConvArgs, _ConvBwdArgs, _ScanArgs, _ScanBwdArgs, _ScanStepArgs))

_lib = None


def load():
    """liblion.so with this module's entry points declared."""
    global _lib
    if _lib is None:
        lib = lion.load()
        for name in ("layernorm_fwd", "layernorm_bwd", "conv_fwd", "conv_bwd", "scan_fwd", "scan_bwd", "scan_step"):
            f = getattr(lib, "lion_" + name)
            f.argtypes, f.restype = [ctypes.c_char_p], _i
        lib.lion_conv_step.argtypes, lib.lion_conv_step.restype = [_vp] * 5 + [_i] * 5 + [_vp], _i
        for name, n in (("layernorm_bwd", 2), ("conv_bwd", 4), ("scan", 5), ("scan_bwd", 6)):
            f = getattr(lib, f"lion_{name}_workspace_bytes")
            f.argtypes, f.restype = [_i] * n, _sz
        _lib = lib
    return _lib


# ------------------------------------------------------------ argument checks
#
# A one-token call takes some ten microseconds, most of them here: the checks
# test for the right argument first and look for what is wrong only after.

_CODES = {torch.bfloat16: lion.DTYPE_BF16, torch.float32: lion.DTYPE_FP32}
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _handle(stream, x):
    if stream is not None:
        if stream.device != x.device:
            raise ValueError(f"stream is on {stream.device}, the tensors are on {x.device}")
        return stream.cuda_stream
    if _raw_stream is None:
        return torch.cuda.current_stream(x.device).cuda_stream
    return _raw_stream(x.get_device())


def _new(stream, shape, dtype, like):
    """An uninitialised tensor that belongs to `stream`."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _code(x):
    code = _CODES.get(x.dtype)
    if code is None:
        raise TypeError(f"activations must be bfloat16 or float32, got {x.dtype}")
    if not x.is_cuda:
        raise ValueError("tensors must be on the GPU")
    if x.get_device() != _current_device():
        raise ValueError(f"tensors are on {x.device}, the current device is cuda:{_current_device()}")
    return code


def _act(activation):
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of 'silu', 'none', None, got {activation!r}")
    return ACTIVATIONS[activation]


def _ptr(t):
    return 0 if t is None else t.data_ptr()


def _tight(name, t, dtype, shape):
    """The address of a contiguous tensor of this type and shape (the library
    refuses one that is not the GPU's)."""
    if t.dtype is dtype and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} must be contiguous")


def _token(name, t, dtype, shape):
    """(address, distance between tokens) of a [B, L, ...] activation whose
    last dimensions are adjacent."""
    width = shape[2] if len(shape) == 3 else shape[2] * shape[3]
    if t.dtype is dtype and t.shape == shape:
        if t.is_contiguous():
            return t.data_ptr(), width
    elif t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype} as the other activations, got {t.dtype}")
    else:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    B, L = shape[:2]
    s, run = t.stride(), 1
    if s[-1] != 1 or len(s) == 4 and s[2] != shape[3]:   # not so of dimensions of one element, whose strides do not matter
        for k in range(t.dim() - 1, 1, -1):
            if shape[k] != 1 and s[k] != run:
                raise ValueError(f"{name}: the values of a token must be adjacent")
            run *= shape[k]
    if L == 1:
        ld = s[0] if B > 1 else width
    else:
        ld = s[1]
        if B > 1 and s[0] != L * ld:
            raise ValueError(f"{name}: sequences must lie L tokens apart")
    if ld < width:
        raise ValueError(f"{name}: tokens must not overlap")
    return t.data_ptr(), ld


@functools.lru_cache(maxsize=256)
def _query(name, *sizes):
    return int(getattr(load(), f"lion_{name}_workspace_bytes")(*sizes))


def _workspace(workspace, like, stream, name, *sizes):
    """(address, bytes, owner) of the caller's workspace, or of one from
    PyTorch's allocator (which reuses it once the stream has passed the call)."""
    if workspace is not None:
        if not workspace.is_contiguous():   # its elements would not be the bytes that it has
            raise ValueError("workspace must be contiguous")
        return workspace.data_ptr(), workspace.numel() * workspace.element_size(), workspace
    n = _query(name, *sizes)
    if n == 0:
        return 0, 0, None
    ws = _new(stream, n, torch.uint8, like)
    return ws.data_ptr(), n, ws


# ------------------------------------------------------------ first derivatives

class _Refuse(torch.autograd.Function):
    @staticmethod
    def forward(ctx, needs, grad):
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, _):
        raise RuntimeError("these operators' gradients cannot be differentiated again")


def _first_only(backward):
    """Gradients that raise if they are differentiated, as the kernels' are
    not: without this a second derivative would lack their terms.  (PyTorch's
    own ``once_differentiable`` looks at the incoming gradient alone, which may
    be a constant.)"""
    @functools.wraps(backward)
    def first(ctx, *dy):
        with torch.no_grad():
            grads = backward(ctx, *dy)
        if not torch.is_grad_enabled():
            return grads
        needs = next((t for t in (*dy, *ctx.saved_tensors) if t is not None and t.requires_grad), None)
        return tuple(g if g is None or needs is None else _Refuse.apply(needs, g) for g in grads)
    return first


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
    return _query("layernorm_bwd", rows, cols)


def layernorm_fwd(x, weight, bias=None, eps=1e-5, save_stats=False, out=None, stream=None):
    """Layer norm over the last dimension: ``y``, or ``(y, mean, rstd)`` with
    ``save_stats`` (float32, one per row, for :func:`layernorm_bwd`)."""
    lib, code = load(), _code(x)
    rows, cols, ld = _rows(x)
    w = _tight("weight", weight, torch.float32, (cols,))
    b = 0 if bias is None else _tight("bias", bias, torch.float32, (cols,))
    if out is None:
        y = _new(stream, x.shape, x.dtype, x)
        yp = y.data_ptr()
    else:
        y, yp = out, _tight("out", out, x.dtype, x.shape)
    mean = rstd = None
    if save_stats:
        mean, rstd = (_new(stream, x.shape[:-1], torch.float32, x) for _ in range(2))
    a = _Norm_pack(x.data_ptr(), w, b, yp, _ptr(mean), _ptr(rstd), ld, rows, cols, eps, code, _handle(stream, x))
    _check(lib.lion_layernorm_fwd(a))
    return (y, mean, rstd) if save_stats else y


def layernorm_bwd(dy, x, weight, mean, rstd, bias=True, workspace=None, stream=None):
    """``(dx, dweight, dbias)`` given ``dy`` and the forward's ``mean`` and
    ``rstd``; ``dbias`` is None with ``bias=False``."""
    lib, code = load(), _code(x)
    rows, cols, ld = _rows(x)
    f32, per = torch.float32, x.shape[:-1]
    ptrs = (_tight("dy", dy, x.dtype, x.shape), x.data_ptr(), _tight("weight", weight, f32, (cols,)),
            _tight("mean", mean, f32, per), _tight("rstd", rstd, f32, per))
    dx = _new(stream, x.shape, x.dtype, x)
    dw = _new(stream, (cols,), f32, x)
    db = _new(stream, (cols,), f32, x) if bias else None
    ws, nb, _keep = _workspace(workspace, x, stream, "layernorm_bwd", rows, cols)
    a = _NormBwd_pack(*ptrs, dx.data_ptr(), dw.data_ptr(), _ptr(db), ld, rows, cols, code, ws, nb, _handle(stream, x))
    _check(lib.lion_layernorm_bwd(a))
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
    @_first_only
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
    shape = B, L, D = x.shape
    K = weight.shape[-1]
    w = _tight("weight", weight, torch.float32, (D, K))
    xp, ld = _token("x", x, x.dtype, shape)
    return (B, L, D, K), ld, (xp, w, 0 if bias is None else _tight("bias", bias, torch.float32, (D,)),
                              0 if state is None else _tight("state", state, x.dtype, (B, K - 1, D)),
                              0 if lengths is None else _tight("lengths", lengths, torch.int32, (B,)))


def conv_bwd_workspace_bytes(B, L, D, K) -> int:
    return _query("conv_bwd", B, L, D, K)


def conv_fwd(x, weight, bias=None, activation="silu", state=None, lengths=None, reverse=False, return_state=False,
             out=None, stream=None):
    """Causal depthwise convolution of ``x`` [B, L, D] with ``weight`` [D, K]
    (K 2 to 4): ``y``, or ``(y, state)`` with ``return_state`` (the last K-1
    inputs, [B, K-1, D], for the next call or :func:`conv_step`).  ``state``:
    the inputs before the first token.  ``lengths``: int32 [B], the tokens
    each sequence has.  ``reverse``: walk from the last token."""
    lib, code = load(), _code(x)
    (B, L, D, K), ld, ptrs = _conv_args(x, weight, bias, state, lengths)
    y = _new(stream, x.shape, x.dtype, x) if out is None else out
    new = _new(stream, (B, K - 1, D), x.dtype, x) if return_state else None
    a = _Conv_pack(*ptrs, _tight("out", y, x.dtype, x.shape), _ptr(new), ld, B, L, D, K, _act(activation),
                  int(reverse), code, _handle(stream, x))
    _check(lib.lion_conv_fwd(a))
    return (y, new) if return_state else y


def conv_bwd(dy, x, weight, bias=None, activation="silu", state=None, lengths=None, reverse=False, workspace=None,
             stream=None):
    """Gradients through :func:`conv_fwd`'s ``y``: :class:`ConvGrads`
    (``dbias`` and ``dstate`` None where there is no bias or state)."""
    lib, code = load(), _code(x)
    (B, L, D, K), ld, ptrs = _conv_args(x, weight, bias, state, lengths)
    dyp = _tight("dy", dy, x.dtype, x.shape)
    f32 = torch.float32
    dx, dw = _new(stream, x.shape, x.dtype, x), _new(stream, (D, K), f32, x)
    db = None if bias is None else _new(stream, (D,), f32, x)
    ds = None if state is None else _new(stream, state.shape, x.dtype, x)
    ws, nb, _keep = _workspace(workspace, x, stream, "conv_bwd", B, L, D, K)
    a = _ConvBwd_pack(dyp, *ptrs, dx.data_ptr(), dw.data_ptr(), _ptr(db), _ptr(ds), ld, B, L, D, K, _act(activation),
                     int(reverse), code, ws, nb, _handle(stream, x))
    _check(lib.lion_conv_bwd(a))
    return ConvGrads(dx, dw, db, ds)


def conv_step(x, state, weight, bias=None, activation="silu", out=None, stream=None):
    """One token ``x`` [B, D]: its output, with the window in ``state``
    [B, K-1, D] moved on in place."""
    lib, code = load(), _code(x)
    B, D = x.shape
    K = weight.shape[-1]
    w = _tight("weight", weight, torch.float32, (D, K))
    if out is None:
        y = _new(stream, (B, D), x.dtype, x)
        yp = y.data_ptr()
    else:
        y, yp = out, _tight("out", out, x.dtype, (B, D))
    _check(lib.lion_conv_step(_tight("x", x, x.dtype, (B, D)), _tight("state", state, x.dtype, (B, K - 1, D)), w,
                              0 if bias is None else _tight("bias", bias, torch.float32, (D,)), yp, B, D, K,
                              _act(activation), code, _handle(stream, x)))
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
    @_first_only
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
    """Sizes, addresses in the structures' order, distances between tokens."""
    shape = B, L, D = u.shape
    N, T, f32 = A.shape[-1], u.dtype, torch.float32
    if Bm.dim() == 3:   # one group
        Bm, Cm = Bm.unsqueeze(2), Cm.unsqueeze(2)
    G = Bm.shape[2]
    up, ul = _token("u", u, T, shape)
    dp, dl = _token("dt", dt, T, shape)
    bp, bl = _token("Bm", Bm, T, (B, L, G, N))
    cp, cl = _token("Cm", Cm, T, (B, L, G, N))
    zp, zl = (0, 0) if z is None else _token("z", z, T, shape)
    return ((B, L, D, N, G),
            (up, dp, _tight("A", A, f32, (D, N)), bp, cp,
             0 if Dskip is None else _tight("Dskip", Dskip, f32, (D,)), zp,
             0 if dt_bias is None else _tight("dt_bias", dt_bias, f32, (D,)),
             0 if h0 is None else _tight("h0", h0, f32, (B, D, N)),
             0 if lengths is None else _tight("lengths", lengths, torch.int32, (B,))),
            (ul, dl, zl, bl, cl))


def scan_workspace_bytes(B, L, D, N, G=1) -> int:
    return _query("scan", B, L, D, N, G)


def scan_bwd_workspace_bytes(B, L, D, N, G=1, have_states=True) -> int:
    return _query("scan_bwd", B, L, D, N, G, int(have_states))


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
    lib, code = load(), _code(u)
    sizes, ptrs, tokens = _scan_args(u, dt, A, Bm, Cm, Dskip, z, dt_bias, h0, lengths)
    B, L, D, N, G = sizes
    y = _new(stream, u.shape, u.dtype, u) if out is None else out
    h = _new(stream, (B, D, N), torch.float32, u) if return_state else None
    states = _new(stream, (B, -(-L // STATE_EVERY), D, N), torch.float32, u) if save_states else None
    ws, nb, _keep = _workspace(workspace, u, stream, "scan", *sizes)
    a = _Scan_pack(*ptrs, _tight("out", y, u.dtype, u.shape), _ptr(h), _ptr(states), *tokens, *sizes,
                  int(dt_softplus), int(reverse), code, ws, nb, _handle(stream, u))
    _check(lib.lion_scan_fwd(a))
    return ScanOut(y, h, states)


def scan_bwd(dout, u, dt, A, Bm, Cm, Dskip=None, z=None, dt_bias=None, dt_softplus=True, h0=None, lengths=None,
             reverse=False, states=None, workspace=None, stream=None):
    """Gradients through :func:`scan_fwd`'s ``out`` given ``dout`` [B, L, D]:
    :class:`ScanGrads`, with None for what was not given.  ``states``: the
    forward's (recomputed if None)."""
    lib, code = load(), _code(u)
    sizes, ptrs, tokens = _scan_args(u, dt, A, Bm, Cm, Dskip, z, dt_bias, h0, lengths)
    B, L, D, N, G = sizes
    f32 = torch.float32
    dop = _tight("dout", dout, u.dtype, u.shape)
    sp = 0 if states is None else _tight("states", states, f32, (B, -(-L // STATE_EVERY), D, N))
    du, ddt = (_new(stream, u.shape, u.dtype, u) for _ in range(2))
    dB, dC = (_new(stream, Bm.shape, u.dtype, u) for _ in range(2))
    dz = None if z is None else _new(stream, u.shape, u.dtype, u)
    dA = _new(stream, (D, N), f32, u)
    dD = None if Dskip is None else _new(stream, (D,), f32, u)
    dbias = None if dt_bias is None else _new(stream, (D,), f32, u)
    dh0 = None if h0 is None else _new(stream, (B, D, N), f32, u)
    ws, nb, _keep = _workspace(workspace, u, stream, "scan_bwd", *sizes, int(states is not None))
    a = _ScanBwd_pack(dop, *ptrs, sp, du.data_ptr(), ddt.data_ptr(), dA.data_ptr(), dB.data_ptr(), dC.data_ptr(),
                     _ptr(dD), _ptr(dz), _ptr(dbias), _ptr(dh0), *tokens, *sizes, int(dt_softplus), int(reverse),
                     code, ws, nb, _handle(stream, u))
    _check(lib.lion_scan_bwd(a))
    return ScanGrads(du, ddt, dA, dB, dC, dD, dz, dbias, dh0)


def scan_step(h, u, dt, A, Bm, Cm, Dskip=None, z=None, dt_bias=None, dt_softplus=True, out=None, stream=None):
    """One token: ``u``, ``dt``, ``z`` [B, D], ``Bm``, ``Cm`` [B, G, N] or
    [B, N]; returns its output [B, D], with the state ``h`` [B, D, N]
    updated in place."""
    lib, code = load(), _code(u)
    shape = B, D = u.shape
    N, T, f32 = A.shape[-1], u.dtype, torch.float32
    G = Bm.shape[1] if Bm.dim() == 3 else 1
    bc = (B, G, N) if Bm.dim() == 3 else (B, N)
    if out is None:
        y = _new(stream, shape, T, u)
        yp = y.data_ptr()
    else:
        y, yp = out, _tight("out", out, T, shape)
    a = _ScanStep_pack(_tight("h", h, f32, (B, D, N)), _tight("u", u, T, shape), _tight("dt", dt, T, shape),
                      _tight("A", A, f32, (D, N)), _tight("Bm", Bm, T, bc), _tight("Cm", Cm, T, bc),
                      0 if Dskip is None else _tight("Dskip", Dskip, f32, (D,)),
                      0 if z is None else _tight("z", z, T, shape),
                      0 if dt_bias is None else _tight("dt_bias", dt_bias, f32, (D,)), yp, B, D, N, G,
                      int(dt_softplus), code, _handle(stream, u))
    _check(lib.lion_scan_step(a))
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
    @_first_only
    def backward(ctx, dout):
        u, dt, A, Bm, Cm, Dskip, z, dt_bias, h0, lengths, states = ctx.saved_tensors
        softplus, reverse = ctx.how
        g = scan_bwd(dout.contiguous(), u, dt, A, Bm, Cm, Dskip, z, dt_bias, softplus, h0, lengths, reverse, states)
        return (g.du, g.ddt, g.dA, g.dB, g.dC, g.dDskip, g.dz, g.ddt_bias, None, g.dh0, None, None)
