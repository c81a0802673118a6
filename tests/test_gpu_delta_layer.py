"""The group norm and the gated delta rule together, as a linear-attention layer has them: keys and
queries normalised per head, the rule over the prompt, the outputs normalised per head and gated, then
decode steps from the carried state; and the gradients of the whole run.

Tolerances: each bf16 tensor on the way is rounded once (2^-8 of its value), and the 64-bit run here
takes the same rounded tensors at each place where the GPU run does, so that what is compared is one
operator's own rounding at a time plus the fp32 part, 2e-5 of the largest value.
"""
import pytest

torch = pytest.importorskip("torch")
import higher_order_linear_chunked_b200 as hla  # noqa: E402
from oracle import delta as od  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def close(got, want, room=2e-5):
    got = got.detach().cpu()
    rounding = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    off = (got.double() - want).abs()
    assert bool((off <= rounding * want.abs() + room * float(want.abs().max())).all()), float(off.max())


def first(x):          # [B, T, H, d] to the oracle's [B, H, T, d]
    return x.cpu().transpose(1, 2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_layer_prefill_and_decode(dtype):
    B, T, H, d, more = 2, 150, 4, 64, 3
    gen = torch.Generator().manual_seed(0)
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    n = T + more
    raw_q, raw_k, v, gate = (r(B, n, H * d).to(dtype).to(DEV) for _ in range(4))
    g, beta = -torch.rand(B, n, H, generator=gen).to(DEV), torch.sigmoid(r(B, n, H)).to(DEV)
    unit = torch.full((H * d,), d ** -0.5)      # x / |x| = (x / rms) / sqrt(d)
    w = (1 + 0.2 * r(H * d)).to(DEV)
    q = hla.group_norm(raw_q, H, weight=unit.to(DEV), eps=1e-6, center=False)
    k = hla.group_norm(raw_k, H, weight=unit.to(DEV), eps=1e-6, center=False)
    close(k, od.group_norm(raw_k.cpu(), H, unit, eps=1e-6, center=False))
    heads = lambda x: x.unflatten(-1, (H, d))  # noqa: E731
    cut = lambda x, a, b: x[:, a:b].contiguous()  # noqa: E731
    o, S = hla.gated_delta(*(cut(heads(x), 0, T) for x in (q, k, v)), cut(g, 0, T), cut(beta, 0, T), layout="bthd",
                           return_state=True)
    outs = [o]
    for t in range(T, n):
        outs.append(hla.gated_delta_step(S, *(heads(x)[:, t].contiguous() for x in (q, k, v)), g[:, t].contiguous(),
                                         beta[:, t].contiguous())[:, None])
    o = torch.cat(outs, 1)
    want, last = od.forward(*(first(heads(x)) for x in (q, k, v)), first(g), first(beta), d ** -0.5)
    close(first(o), want)
    close(S, last)
    y = hla.group_norm(o.flatten(2), H, weight=w, gate=gate, activation="silu", center=False)
    close(y, od.group_norm(o.flatten(2).cpu(), H, w.cpu(), None, gate.cpu(), activation="silu", center=False))


def test_layer_gradients_against_the_64_bit_chain():
    """fp32 run of norm, rule and gated norm, backwards by hand; the 64-bit chain by automatic
    differentiation of the oracle's forward.  Four operators' fp32 parts in a row: 1e-4 of the largest."""
    B, T, H, d = 1, 70, 2, 32
    gen = torch.Generator().manual_seed(5)
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    raw_q, raw_k, v, gate, dy = (r(B, T, H * d) for _ in range(5))
    g, beta = -torch.rand(B, T, H, generator=gen), torch.sigmoid(r(B, T, H))
    unit, w = torch.full((H * d,), d ** -0.5), 1 + 0.2 * r(H * d)
    heads = lambda x: x.unflatten(-1, (H, d))  # noqa: E731
    dev = lambda x: x.to(DEV)  # noqa: E731
    norm_qk = dict(weight=dev(unit), eps=1e-6, center=False)
    q, k = hla.group_norm(dev(raw_q), H, **norm_qk), hla.group_norm(dev(raw_k), H, **norm_qk)
    o = hla.gated_delta(heads(q), heads(k), heads(dev(v)), dev(g), dev(beta), layout="bthd")
    how = dict(weight=dev(w), gate=dev(gate), activation="silu", center=False)
    do, dgate, dw, _ = hla.group_norm_backward(o.flatten(2), dev(dy), H, **how)
    dq, dk, dv, dg, db, _ = hla.gated_delta_backward(heads(q), heads(k), heads(dev(v)), dev(g), dev(beta), heads(do).contiguous(),
                                                     layout="bthd")
    draw_q = hla.group_norm_backward(dev(raw_q), dq.flatten(2), H, **norm_qk)[0]
    draw_k = hla.group_norm_backward(dev(raw_k), dk.flatten(2), H, **norm_qk)[0]
    xs = [x.double().requires_grad_() for x in (raw_q, raw_k, v, g, beta, gate, w)]
    Q, K = (od.group_norm(x, H, unit, eps=1e-6, center=False) for x in xs[:2])
    O, _ = od.forward(*(heads(x).transpose(1, 2) for x in (Q, K, xs[2])), *(x.transpose(1, 2) for x in xs[3:5]), d ** -0.5)
    y = od.group_norm(O.transpose(1, 2).flatten(2), H, xs[6], None, xs[5], activation="silu", center=False)
    want = torch.autograd.grad((y * dy.double()).sum(), xs)
    for got, ref in zip((draw_q, draw_k, dv.flatten(2), dg, db, dgate, dw), want):
        close(got, ref, 1e-4)
