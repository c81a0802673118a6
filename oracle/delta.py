"""64-bit values of the gated delta rule and the group norm, token by token and group by group.

Plain torch in float64 on the CPU, written from the definitions: one loop over the tokens, its
adjoint run backwards over stored states, and the group norm's formulas.  Nothing here is shared
with the kernels (no chunks, no triangular systems).

Tensors are [B, Hk, T, d] (q, k), [B, H, T, dv] (v, dout), [B, H, T] (g, beta), [B, H, d, dv]
(states); H is a multiple of Hk.
"""
from __future__ import annotations

import torch


def _wide(x, H):
    return x.double().repeat_interleave(H // x.shape[1], 1)


def _live(lengths, B, T):
    if lengths is None:
        return torch.ones(B, 1, T, dtype=torch.bool)
    return (torch.arange(T)[None, None, :] < lengths.clamp(0, T)[:, None, None].long())


def _inputs(q, k, v, g, beta, lengths):
    H = v.shape[1]
    live = _live(lengths, v.shape[0], v.shape[2])
    keep = lambda x: torch.where(live[..., None] if x.dim() == 4 else live, x, torch.zeros_like(x))  # noqa: E731
    q, k, v = keep(_wide(q, H)), keep(_wide(k, H)), keep(v.double())
    a = torch.where(live, g.double().exp(), torch.ones(1, dtype=torch.float64))
    return q, k, v, a, keep(beta.double()), live


def forward(q, k, v, g, beta, scale, state=None, lengths=None, every=False):
    """(o, state after the last token); with ``every`` also the state before each token and each
    token's error v - S^T k."""
    q, k, v, a, beta, _ = _inputs(q, k, v, g, beta, lengths)
    B, H, T, d = q.shape
    S = torch.zeros(B, H, d, v.shape[-1], dtype=torch.float64) if state is None else state.double()
    o, before, errs = [], [], []
    for t in range(T):
        before.append(S)
        S = a[:, :, t, None, None] * S
        e = v[:, :, t] - (S * k[:, :, t, :, None]).sum(-2)
        S = S + beta[:, :, t, None, None] * k[:, :, t, :, None] * e[:, :, None, :]
        o.append(scale * (S * q[:, :, t, :, None]).sum(-2))
        errs.append(e)
    o = torch.stack(o, 2)
    return (o, S, before + [S], errs) if every else (o, S)


def backward(q, k, v, g, beta, scale, dout, state=None, dstate=None, lengths=None):
    """Gradients of sum(o * dout) + sum(last state * dstate):
    {"dq", "dk", "dv", "dg", "dbeta", "dstate"}."""
    Hk = q.shape[1]
    _, _, states, errs = forward(q, k, v, g, beta, scale, state, lengths, every=True)
    q, k, v, a, beta, live = _inputs(q, k, v, g, beta, lengths)
    dout = torch.where(live[..., None], dout.double(), torch.zeros(1, dtype=torch.float64))
    B, H, T, d = q.shape
    dS = torch.zeros_like(states[0]) if dstate is None else dstate.double()
    dq, dk, dv, dg, db = (torch.zeros_like(x) for x in (q, k, v, beta, beta))
    for t in reversed(range(T)):
        kt, at, bt, e = k[:, :, t], a[:, :, t, None, None], beta[:, :, t], errs[t]
        dq[:, :, t] = scale * (states[t + 1] * dout[:, :, t, None, :]).sum(-1)
        dS = dS + scale * q[:, :, t, :, None] * dout[:, :, t, None, :]
        w = (dS * kt[..., None]).sum(-2)                        # dS^T k
        db[:, :, t] = (w * e).sum(-1)
        de = bt[..., None] * w
        dv[:, :, t] = de
        faded = at * states[t]
        dk[:, :, t] = bt[..., None] * (dS * e[..., None, :]).sum(-1) - (faded * de[..., None, :]).sum(-1)
        dS = dS - kt[..., None] * de[..., None, :]
        dg[:, :, t] = (dS * faded).sum((-1, -2))
        dS = at * dS
    zero = lambda x: torch.where(live[..., None] if x.dim() == 4 else live, x, torch.zeros_like(x))  # noqa: E731
    shared = lambda x: zero(x).unflatten(1, (Hk, H // Hk)).sum(2)  # noqa: E731
    return {"dq": shared(dq), "dk": shared(dk), "dv": zero(dv), "dg": zero(dg), "dbeta": zero(db), "dstate": dS}


def _act(a, activation):
    return a / (1 + torch.exp(-a)) if activation == "silu" else a


def group_norm(x, groups, weight=None, bias=None, gate=None, eps=1e-5, activation="none", center=True):
    C = x.shape[-1]
    xg = x.double().reshape(-1, groups, C // groups)
    if center:
        xg = xg - xg.mean(-1, keepdim=True)
    z = (xg / torch.sqrt((xg * xg).mean(-1, keepdim=True) + eps)).reshape(x.shape)
    if weight is not None:
        z = z * weight.double()
    if bias is not None:
        z = z + bias.double()
    return _act(z, activation) if gate is None else z * _act(gate.double(), activation)


def group_norm_backward(x, dy, groups, weight=None, bias=None, gate=None, eps=1e-5, activation="none", center=True):
    """(dx, dgate, dweight, dbias), None where the input is None, by the chain rule on the formulas."""
    C = x.shape[-1]
    shape = (-1, groups, C // groups)
    xg = x.double().reshape(shape)
    xc = xg - xg.mean(-1, keepdim=True) if center else xg
    r = 1 / torch.sqrt((xc * xc).mean(-1, keepdim=True) + eps)
    n = (xc * r).reshape(-1, C)
    w = weight.double() if weight is not None else torch.ones(C, dtype=torch.float64)
    z = n * w + (bias.double() if bias is not None else 0)
    hot = z if gate is None else gate.double().reshape(-1, C)
    s = 1 / (1 + torch.exp(-hot))
    slope = s + hot * s * (1 - s) if activation == "silu" else torch.ones_like(hot)
    dy = dy.double().reshape(-1, C)
    dz = dy * slope if gate is None else dy * _act(hot, activation)
    dgate = None if gate is None else (dy * z * slope).reshape(x.shape)
    e, n3 = (dz * w).reshape(shape), n.reshape(shape)
    dx = e - n3 * (e * n3).mean(-1, keepdim=True)
    if center:
        dx = dx - e.mean(-1, keepdim=True)
    return ((dx * r).reshape(x.shape), dgate, (dz * n).sum(0) if weight is not None else None,
            dz.sum(0) if bias is not None else None)
