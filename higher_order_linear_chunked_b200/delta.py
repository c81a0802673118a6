"""The gated delta rule and the group norm around it: binding over ``include/hla_delta.h``.

* :func:`gated_delta` - a whole sequence (training, prefill), from and to a carried state;
* :func:`gated_delta_step` - one token of every sequence (decode), the state in place;
* :func:`gated_delta_backward` - the gradients of a forward;
* :func:`group_norm`, :func:`group_norm_backward` - each group of channels of every row
  normalised, with an activation or a gate.

As in the package's other calls the library's kernels do all the work, on the tensors' device and
the current torch stream; arguments are checked here and again at the C boundary.  A call on another
stream (``stream=``) takes what it allocates from that stream's memory; ordering that stream behind the
inputs, and the use of the results behind it, is the caller's.
"""
from __future__ import annotations

import ctypes
import functools
from typing import Optional

import torch

from . import HLAError, HLA_BF16, HLA_F32, HLA_OK, _check_workspace, _empty, load_library as _load

LAYOUTS = {"bhtd": 0, "bthd": 1}
ACTIVATIONS = ("none", "silu")
NORM_CENTER, NORM_SILU = 1, 2
WIDTHS = (32, 64, 128)
_CODES = {torch.float32: HLA_F32, torch.bfloat16: HLA_BF16}

# Every symbol include/hla_delta.h declares.
EXPORTS = ("hla_delta_abi_version", "hla_delta_workspace_bytes", "hla_delta_kernel_launches", "hla_delta_forward",
           "hla_delta_step", "hla_delta_backward_workspace_bytes", "hla_delta_backward_kernel_launches",
           "hla_delta_backward", "hla_group_norm_forward", "hla_group_norm_backward_workspace_bytes",
           "hla_group_norm_backward")

_bound = None


def _library():
    global _bound
    if _bound is None:
        lib = _load()
        vp, i, f, sz, ll = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t, ctypes.c_longlong
        sizes = [i] * 7
        for name, args, res in (
                ("hla_delta_abi_version", [], i),
                ("hla_delta_workspace_bytes", sizes, sz),
                ("hla_delta_kernel_launches", sizes, i),
                ("hla_delta_forward", [vp] * 9 + [i] * 8 + [f, vp, sz, vp], i),
                ("hla_delta_backward_workspace_bytes", sizes, sz),
                ("hla_delta_backward_kernel_launches", sizes, i),
                ("hla_delta_backward", [vp] * 15 + [i] * 8 + [f, vp, sz, vp], i),
                ("hla_delta_step", [vp] * 7 + [i] * 6 + [f, vp], i),
                ("hla_group_norm_forward", [vp] * 5 + [ll, i, i, i, f, i, vp], i),
                ("hla_group_norm_backward_workspace_bytes", [i, ll, i, i], sz),
                ("hla_group_norm_backward", [vp] * 9 + [ll, i, i, i, f, i, vp, sz, vp], i)):
            fn = getattr(lib, name)
            fn.argtypes, fn.restype = args, res
        _bound = lib
    return _bound


@functools.lru_cache(maxsize=1024)
def _bytes(query, *sizes) -> int:
    """A workspace query's answer: sizes alone decide it."""
    return int(getattr(_library(), query)(*sizes))


def _ptr(t):
    return t.data_ptr() if t is not None else None


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)     # both None in a torch without CUDA
_current_device = getattr(torch._C, "_cuda_getDevice", None)


def _stream_of(device: int, stream) -> int:
    return _raw_stream(device) if stream is None else stream.cuda_stream


def _likes(on: int, stream, *tensors):
    """Results shaped like the given tensors (None for None), allocated as by :func:`_empty`."""
    if stream is None:
        return [torch.empty_like(t) if t is not None else None for t in tensors]
    current = torch.cuda.current_stream(on)
    with torch.cuda.stream(stream):
        made = [torch.empty_like(t) if t is not None else None for t in tensors]
    if stream != current:
        for t in made:
            if t is not None:
                t.record_stream(current)
    return made


def _given(workspace, device, stream):
    """A caller's workspace, checked, and kept for the stream that uses it."""
    _check_workspace(workspace, device)
    if stream is not None:
        workspace.record_stream(stream)


def _call(device: int, fn, what, *args) -> None:
    """One library call with the tensors' device current."""
    if _current_device() == device:
        rc = fn(*args)
    else:
        with torch.cuda.device(device):
            rc = fn(*args)
    if rc != HLA_OK:
        raise HLAError(rc, what)


def _expect(name, t, shape, dtype, device):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (this library has no CPU path)")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, q on {device}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def _first(name, t, dims):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor (this library has no CPU path)")
    if t.dtype not in _CODES:
        raise TypeError(f"{name} must be float32 or bfloat16, got {t.dtype}")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} axes, got {list(t.shape)}")


def _leaves(q, k, v, g, beta, layout, step=False):
    """Checked sizes (B, Hk, H, T, d, dv) of one call's inputs."""
    _first("q", q, 3 if step else 4)
    if v.dim() != q.dim():
        raise ValueError(f"v must have {q.dim()} axes, got {list(v.shape)}")
    dt, dev = q.dtype, q.device
    if step:
        (B, Hk, d), (H, dv), T = q.shape, v.shape[1:], 1
        lead = (B, H)
    elif layout == "bhtd":
        (B, Hk, T, d), H, dv = q.shape, v.shape[1], v.shape[3]
        lead = (B, H, T)
    elif layout == "bthd":
        (B, T, Hk, d), H, dv = q.shape, v.shape[2], v.shape[3]
        lead = (B, T, H)
    else:
        raise ValueError(f"layout must be one of {sorted(LAYOUTS)}, got {layout!r}")
    on = q.get_device()
    if not (k.shape == q.shape and v.shape == (*lead, dv) and g.shape == lead and beta.shape == lead and
            k.dtype is dt and v.dtype is dt and g.dtype is torch.float32 and beta.dtype is torch.float32 and
            k.get_device() == on and v.get_device() == on and g.get_device() == on and beta.get_device() == on and
            q.is_contiguous() and k.is_contiguous() and v.is_contiguous() and g.is_contiguous() and beta.is_contiguous()):
        _expect("q", q, tuple(q.shape), dt, dev)
        _expect("k", k, tuple(q.shape), dt, dev)
        _expect("v", v, (*lead, dv), dt, dev)
        _expect("g", g, lead, torch.float32, dev)
        _expect("beta", beta, lead, torch.float32, dev)
    if min(B, Hk, H, T, d, dv) < 1:
        raise HLAError(2, f"an empty axis: B={B} Hk={Hk} H={H} T={T} d={d} dv={dv}")
    if H % Hk:
        raise ValueError(f"{H} value heads cannot share {Hk} key heads: a multiple is wanted")
    return B, Hk, H, T, d, dv


def _lengths(lengths, B, device):
    if lengths is not None:
        _expect("lengths", lengths, (B,), torch.int32, device)


def gated_delta_workspace_bytes(dtype, B: int, Hk: int, H: int, T: int, d: int, dv: int) -> int:
    """Bytes of workspace :func:`gated_delta` needs (0: no such call); ``dtype`` is torch's."""
    return _bytes("hla_delta_workspace_bytes", _CODES.get(dtype, -1), B, Hk, H, T, d, dv)


def gated_delta(q, k, v, g, beta, scale: Optional[float] = None, initial_state=None, lengths=None,
                layout: str = "bhtd", return_state: bool = False, out=None, state_out=None, workspace=None,
                stream=None):
    """Gated delta rule over a sequence.  Each value head's state S [d, dv] takes, token by token,
    ``S *= exp(g); S += beta k (v - S^T k)^T`` and answers ``o = scale S^T q``.

    q, k [B, Hk, T, d], v [B, H, T, dv] (fp32 or bf16), g, beta [B, H, T] fp32, with layout "bthd"
    the head and time axes the other way round.  H is a multiple of Hk (value head h uses key head
    h // (H // Hk)); d and dv are 32, 64 or 128.  ``scale`` defaults to d**-0.5.  ``initial_state``
    [B, H, d, dv] fp32 (default: zeros).  ``lengths`` int32 [B]: tokens of each sequence of a padded
    batch; rows behind them are not used and their output is zero.  Returns o (shaped and typed like
    v), with ``return_state`` also the state after the last token.  ``state_out`` may be
    ``initial_state``."""
    B, Hk, H, T, d, dv = _leaves(q, k, v, g, beta, layout)
    dev = q.device
    _lengths(lengths, B, dev)
    if initial_state is not None:
        _expect("initial_state", initial_state, (B, H, d, dv), torch.float32, dev)
    on = q.get_device()
    lib = _library()
    if out is None:
        out, = _likes(on, stream, v)
    else:
        _expect("out", out, tuple(v.shape), v.dtype, dev)
    if state_out is not None:
        _expect("state_out", state_out, (B, H, d, dv), torch.float32, dev)
    elif return_state:
        state_out = _empty(stream, (B, H, d, dv), torch.float32, dev, result=True)
    code = _CODES[q.dtype]
    if workspace is None:
        n = _bytes("hla_delta_workspace_bytes", code, B, Hk, H, T, d, dv)
        if n == 0:
            raise HLAError(5, f"no gated delta kernel for B={B} Hk={Hk} H={H} T={T} d={d} dv={dv}")
        workspace = _empty(stream, n, torch.uint8, dev)
    else:
        _given(workspace, dev, stream)
    _call(on, lib.hla_delta_forward, "hla_delta_forward rejected the call", q.data_ptr(), k.data_ptr(), v.data_ptr(),
            g.data_ptr(), beta.data_ptr(), _ptr(initial_state), _ptr(lengths), out.data_ptr(), _ptr(state_out), B, Hk,
            H, T, d, dv, code, LAYOUTS[layout], d ** -0.5 if scale is None else scale, workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), _stream_of(on, stream))
    return (out, state_out) if return_state else out


def gated_delta_step(state, q, k, v, g, beta, scale: Optional[float] = None, out=None, stream=None):
    """One token of every sequence: q, k [B, Hk, d], v [B, H, dv], g, beta [B, H]; advances
    ``state`` [B, H, d, dv] fp32 in place and returns o [B, H, dv] in v's type."""
    B, Hk, H, _, d, dv = _leaves(q, k, v, g, beta, None, step=True)
    on = q.get_device()
    if not (state.shape == (B, H, d, dv) and state.dtype is torch.float32 and state.get_device() == on and
            state.is_contiguous()):
        _expect("state", state, (B, H, d, dv), torch.float32, q.device)
    if out is None:
        out, = _likes(on, stream, v)
    else:
        _expect("out", out, tuple(v.shape), v.dtype, q.device)
    _call(on, _library().hla_delta_step, "hla_delta_step rejected the call", state.data_ptr(), q.data_ptr(),
          k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), out.data_ptr(), B, Hk, H, d, dv, _CODES[q.dtype],
          d ** -0.5 if scale is None else scale, _stream_of(on, stream))
    return out


def gated_delta_backward_workspace_bytes(dtype, B: int, Hk: int, H: int, T: int, d: int, dv: int) -> int:
    """Bytes of workspace :func:`gated_delta_backward` needs (0: no such call); ``dtype`` is torch's."""
    return _bytes("hla_delta_backward_workspace_bytes", _CODES.get(dtype, -1), B, Hk, H, T, d, dv)


def gated_delta_backward(q, k, v, g, beta, dout, scale: Optional[float] = None, initial_state=None, dstate=None,
                         lengths=None, layout: str = "bhtd", workspace=None, stream=None):
    """Gradients (dq, dk, dv, dg, dbeta, dstate0) of ``sum(o * dout) + sum(state * dstate)`` for
    ``o, state = gated_delta(q, k, v, g, beta, scale, initial_state, lengths, layout,
    return_state=True)``.  dout is shaped and typed like v; ``dstate`` [B, H, d, dv] fp32 (default:
    zeros).  dq, dk, dv come in the inputs' type, the others in fp32; dstate0 is None without an
    initial state.  Nothing of the forward call is needed."""
    B, Hk, H, T, d, dv = _leaves(q, k, v, g, beta, layout)
    dev = q.device
    _lengths(lengths, B, dev)
    _expect("dout", dout, tuple(v.shape), v.dtype, dev)
    for name, t in (("initial_state", initial_state), ("dstate", dstate)):
        if t is not None:
            _expect(name, t, (B, H, d, dv), torch.float32, dev)
    on = q.get_device()
    lib = _library()
    code = _CODES[q.dtype]
    if workspace is None:
        n = _bytes("hla_delta_backward_workspace_bytes", code, B, Hk, H, T, d, dv)
        if n == 0:
            raise HLAError(5, f"no gated delta kernel for B={B} Hk={Hk} H={H} T={T} d={d} dv={dv}")
        workspace = _empty(stream, n, torch.uint8, dev)
    else:
        _given(workspace, dev, stream)
    dq, dk, dvv, dg, dbeta, dstate0 = _likes(on, stream, q, k, v, g, beta, initial_state)
    _call(on, lib.hla_delta_backward, "hla_delta_backward rejected the call", q.data_ptr(), k.data_ptr(), v.data_ptr(),
            g.data_ptr(), beta.data_ptr(), _ptr(initial_state), _ptr(lengths), dout.data_ptr(), _ptr(dstate),
            dq.data_ptr(), dk.data_ptr(), dvv.data_ptr(), dg.data_ptr(), dbeta.data_ptr(), _ptr(dstate0), B, Hk, H, T, d,
            dv, code, LAYOUTS[layout], d ** -0.5 if scale is None else scale, workspace.data_ptr(),
            workspace.numel() * workspace.element_size(), _stream_of(on, stream))
    return dq, dk, dvv, dg, dbeta, dstate0


# ---------------------------------------------------------------------------
# group norm
# ---------------------------------------------------------------------------

def _norm_args(x, groups, weight, bias, gate, activation, center):
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor (this library has no CPU path)")
    if x.dtype not in _CODES:
        raise TypeError(f"x must be float32 or bfloat16, got {x.dtype}")
    if x.dim() < 1 or not x.is_contiguous():
        raise ValueError("x must be contiguous, channels last")
    if activation not in ACTIVATIONS:
        raise ValueError(f"activation must be one of {ACTIVATIONS}, got {activation!r}")
    C = x.shape[-1]
    if groups < 1 or C % groups:
        raise ValueError(f"{C} channels do not divide into {groups} groups")
    on = x.get_device()
    if gate is not None and not (gate.shape == x.shape and gate.dtype is x.dtype and gate.get_device() == on and
                                 gate.is_contiguous()):
        _expect("gate", gate, tuple(x.shape), x.dtype, x.device)
    for name, t in (("weight", weight), ("bias", bias)):
        if t is not None and not (t.shape == (C,) and t.dtype is torch.float32 and t.get_device() == on and
                                  t.is_contiguous()):
            _expect(name, t, (C,), torch.float32, x.device)
    if x.numel() == 0:
        raise HLAError(2, f"x has no elements: {list(x.shape)}")
    return C, x.numel() // C, (NORM_CENTER if center else 0) | (NORM_SILU if activation == "silu" else 0)


def group_norm(x, groups: int, weight=None, bias=None, gate=None, eps: float = 1e-5, activation: str = "none",
               center: bool = True, out=None, stream=None):
    """Each group of C // groups neighbouring channels of every row of ``x`` [..., C] normalised by
    itself: ``n = (x - mean) / sqrt(var + eps)`` (without ``center``: ``x / sqrt(mean(x^2) + eps)``),
    ``z = n * weight + bias`` (fp32 [C], either may be None), then ``act(z)``, or ``z * act(gate)``
    with a gate shaped like x.  activation: "none" or "silu".  Returns y in x's type; ``out`` may be
    x or gate.  A row here is one position: nothing is shared between positions."""
    C, rows, flags = _norm_args(x, groups, weight, bias, gate, activation, center)
    on = x.get_device()
    if out is None:
        out, = _likes(on, stream, x)
    else:
        _expect("out", out, tuple(x.shape), x.dtype, x.device)
    _call(on, _library().hla_group_norm_forward, "hla_group_norm_forward rejected the call", x.data_ptr(), _ptr(gate),
            _ptr(weight), _ptr(bias), out.data_ptr(), rows, C, groups, _CODES[x.dtype], eps, flags,
          _stream_of(on, stream))
    return out


def group_norm_backward(x, dy, groups: int, weight=None, bias=None, gate=None, eps: float = 1e-5,
                        activation: str = "none", center: bool = True, workspace=None, stream=None):
    """Gradients (dx, dgate, dweight, dbias) of ``sum(group_norm(x, ...) * dy)``: dx and dgate in
    x's type, dweight and dbias fp32, each None where its input is None."""
    C, rows, flags = _norm_args(x, groups, weight, bias, gate, activation, center)
    _expect("dy", dy, tuple(x.shape), x.dtype, x.device)
    on = x.get_device()
    lib = _library()
    dx, dgate, dweight, dbias = _likes(on, stream, x, gate, weight, bias)
    nbytes = 0
    if workspace is not None:
        _given(workspace, x.device, stream)
    if weight is not None or bias is not None:
        if workspace is None:
            n = _bytes("hla_group_norm_backward_workspace_bytes", _CODES[x.dtype], rows, C, groups)
            if n == 0:
                raise HLAError(5, f"no group norm kernel for {rows} rows of {C} channels in {groups} groups")
            workspace = _empty(stream, n, torch.uint8, x.device)
        nbytes = workspace.numel() * workspace.element_size()
    _call(on, lib.hla_group_norm_backward, "hla_group_norm_backward rejected the call", x.data_ptr(), _ptr(gate),
            _ptr(weight), _ptr(bias), dy.data_ptr(), dx.data_ptr(), _ptr(dgate), _ptr(dweight), _ptr(dbias), rows, C,
            groups, _CODES[x.dtype], eps, flags, _ptr(workspace), nbytes, _stream_of(on, stream))
    return dx, dgate, dweight, dbias
