"""The 64-bit gated delta rule and group norm of oracle/delta.py against literal sums, closed forms
and differences (CPU)."""
import math

import pytest
import torch

from oracle import delta as od


def leaves(B, Hk, H, T, d, dv, seed, state=True):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    q, k, v = r(B, Hk, T, d) / math.sqrt(d), r(B, Hk, T, d) / math.sqrt(d), r(B, H, T, dv)
    g, beta = -torch.rand(B, H, T, generator=gen, dtype=torch.float64), torch.rand(B, H, T, generator=gen, dtype=torch.float64)
    return q, k, v, g, beta, (r(B, H, d, dv) * 0.3 if state else None)


def test_products_of_transitions():
    """S_T = sum_t (prod_{s>t} a_s (I - b_s k_s k_s^T)) b_t k_t v_t^T + (all of them) S_0, literally."""
    q, k, v, g, beta, S0 = leaves(1, 1, 1, 7, 4, 3, 0)
    a = g.exp()
    step = [a[0, 0, t] * (torch.eye(4, dtype=torch.float64) - beta[0, 0, t] * torch.outer(k[0, 0, t], k[0, 0, t]))
            for t in range(7)]
    want = torch.zeros(4, 3, dtype=torch.float64)
    for t in range(-1, 7):
        term = S0[0, 0] if t < 0 else beta[0, 0, t] * torch.outer(k[0, 0, t], v[0, 0, t])
        for s in range(t + 1, 7):
            term = step[s] @ term
        want = want + term
    o, S = od.forward(q, k, v, g, beta, 0.5, S0)
    assert torch.allclose(S[0, 0], want, rtol=0, atol=1e-13)
    assert torch.allclose(o[0, 0, -1], 0.5 * want.T @ q[0, 0, -1], rtol=0, atol=1e-13)


def test_orthonormal_keys_store_and_recall():
    """With orthonormal keys, no decay and beta = 1 the state answers each key with its last value."""
    d = 8
    k = torch.eye(d, dtype=torch.float64)[torch.tensor([0, 1, 2, 1, 0])][None, None]
    v = torch.arange(10, dtype=torch.float64).reshape(1, 1, 5, 2)
    zero, one = torch.zeros(1, 1, 5, dtype=torch.float64), torch.ones(1, 1, 5, dtype=torch.float64)
    _, S = od.forward(k, k, v, zero, one, 1.0)
    assert torch.equal(S[0, 0, :3], torch.stack([v[0, 0, 4], v[0, 0, 3], v[0, 0, 2]]))


def test_infinite_decay_starts_anew():
    q, k, v, g, beta, S0 = leaves(1, 1, 2, 9, 4, 4, 3)
    g[:, :, 4] = -math.inf
    o, S = od.forward(q, k, v, g, beta, 1.0, S0)
    o2, S2 = od.forward(q[:, :, 4:], k[:, :, 4:], v[:, :, 4:], g[:, :, 4:], beta[:, :, 4:], 1.0)
    assert torch.equal(o[:, :, 4:], o2) and torch.equal(S, S2)


def test_gradients_against_automatic_differentiation():
    q, k, v, g, beta, S0 = leaves(2, 2, 4, 6, 5, 3, 1)
    lens = torch.tensor([6, 4])
    gen = torch.Generator().manual_seed(9)
    dout = torch.randn(v.shape, generator=gen, dtype=torch.float64)
    dS = torch.randn(S0.shape, generator=gen, dtype=torch.float64)
    xs = [x.clone().requires_grad_() for x in (q, k, v, g, beta, S0)]
    o, S = od.forward(*xs[:5], 0.7, xs[5], lens)
    want = torch.autograd.grad((o * dout).sum() + (S * dS).sum(), xs)
    got = od.backward(q, k, v, g, beta, 0.7, dout, S0, dS, lens)
    for name, w in zip(("dq", "dk", "dv", "dg", "dbeta", "dstate"), want):
        assert torch.allclose(got[name], w, rtol=1e-11, atol=1e-12), name


def test_gradients_against_differences():
    q, k, v, g, beta, S0 = leaves(1, 1, 2, 5, 4, 3, 5)
    gen = torch.Generator().manual_seed(2)
    dout = torch.randn(v.shape, generator=gen, dtype=torch.float64)
    dS = torch.randn(S0.shape, generator=gen, dtype=torch.float64)
    xs = [q, k, v, g, beta, S0]

    def loss(*y):
        o, S = od.forward(*y[:5], 0.7, y[5])
        return float((o * dout).sum() + (S * dS).sum())

    got = od.backward(q, k, v, g, beta, 0.7, dout, S0, dS)
    h = 1e-5
    for i, name in enumerate(("dq", "dk", "dv", "dg", "dbeta", "dstate")):
        way = torch.randn(xs[i].shape, generator=gen, dtype=torch.float64)
        up, down = ([x + s * h * way if j == i else x for j, x in enumerate(xs)] for s in (1, -1))
        slope = (loss(*up) - loss(*down)) / (2 * h)
        # the second-order error of a central difference is about h^2 = 1e-10 of the loss's scale
        assert abs(slope - float((got[name] * way).sum())) < 1e-7 * max(1.0, abs(slope)), name


@pytest.mark.parametrize("center", [True, False])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("activation", ["none", "silu"])
def test_group_norm_gradients(center, gated, activation):
    gen = torch.Generator().manual_seed(4)
    r = lambda *s: torch.randn(s, generator=gen, dtype=torch.float64)  # noqa: E731
    x, w, b, gate, dy = r(3, 2, 12), r(12), r(12), r(3, 2, 12) if gated else None, r(3, 2, 12)
    xs = [t.clone().requires_grad_() for t in (x, w, b)] + ([gate.clone().requires_grad_()] if gated else [])
    y = od.group_norm(xs[0], 3, xs[1], xs[2], xs[3] if gated else None, 1e-3, activation, center)
    want = torch.autograd.grad((y * dy).sum(), xs)
    dx, dgate, dw, db = od.group_norm_backward(x, dy, 3, w, b, gate, 1e-3, activation, center)
    for got, ref in zip((dx, dw, db, dgate), want):
        assert torch.allclose(got, ref, rtol=1e-11, atol=1e-12)


def test_group_norm_agrees_with_torch():
    x = torch.randn(5, 24, dtype=torch.float64, generator=torch.Generator().manual_seed(8))
    want = torch.nn.functional.group_norm(x, 4, eps=1e-5)
    assert torch.allclose(od.group_norm(x, 4), want, rtol=1e-12, atol=1e-12)
