"""bf16 calls of the gated delta rule where large terms cancel: what is left shows how many bits the
terms had before the result's one rounding.

x has 24 bits and y = x in the first two bf16 terms (16 bits), so that r = x - y, 2^-18 to 2^-17 of x,
is what a sum of x and -y leaves.  Room: the result's rounding (2^-8 of its value), and for terms of fp32
2^-21 of the sum of their sizes: an approximate power of two (2^-22), four roundings (2^-24 each) and the
sums' cuts (at most 24 of 2^-23 of one term, 2^-21 of eight).  Terms of 16 bits leave all of r.
"""
import pytest

torch = pytest.importorskip("torch")
import higher_order_linear_chunked_b200 as hla  # noqa: E402
from oracle import delta as od  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def short(x):
    """x in two bf16 terms."""
    hi = x.bfloat16().float()
    return hi + (x - hi).bfloat16().float()


def residues(n, seed):
    """n values in [1, 1.5) whose two terms leave 2^-18 or more of them."""
    x = 1 + 0.5 * torch.rand(64 * n, generator=torch.Generator().manual_seed(seed))
    x = x[(x - short(x)) > 2.0 ** -18][:n]
    assert len(x) == n
    return x


def near(got, want, terms, name):
    got = got.cpu().double()
    off, room = (got - want).abs(), 2.0 ** -8 * want.abs() + 2.0 ** -21 * terms
    assert bool((off <= room).all()), f"{name}: {float((off / room).max()):.3g} times the tolerance"


def on(*xs):
    return [x.to(DEV) for x in xs]


@pytest.mark.parametrize("d", [32, 64, 128])
def test_state_in_the_outputs(d):
    """o = sum over pairs of keys of x - y, both elements of the carried state."""
    x = residues(32, d)
    S = torch.stack([x, short(x)]).repeat(d // 2, 1)[None, None].contiguous()
    q = torch.tensor([1.0, -1.0]).repeat(d // 2)[None, None, None].bfloat16()
    zero, none = torch.zeros(1, 1, 1, d).bfloat16(), torch.zeros(1, 1, 1)
    v = torch.zeros(1, 1, 1, 32).bfloat16()
    o = hla.gated_delta(*on(q, zero, v, none, none), scale=1.0, initial_state=S.to(DEV))
    want, _ = od.forward(q, zero, v, none, none, 1.0, S)
    assert float(want.abs().min()) > 2.0 ** -18 * d / 2
    near(o, want, d * 1.5, "o")


@pytest.mark.parametrize("d", [32, 64, 128])
def test_writes_in_the_outputs(d):
    """Orthogonal keys, v = 1: token t writes beta_t, and the last token's output is the sum of
    x - y over the tokens' pairs."""
    x = residues(16, d + 1)
    beta = torch.stack([x, short(x)], 1).reshape(1, 1, 32)
    k = torch.eye(32, d)[None, None].bfloat16()
    q = torch.zeros(1, 1, 32, d)
    q[0, 0, 31, :32] = torch.tensor([1.0, -1.0]).repeat(16)
    q, v, g = q.bfloat16(), torch.ones(1, 1, 32, 32).bfloat16(), torch.zeros(1, 1, 32)
    o = hla.gated_delta(*on(q, k, v, g, beta), scale=1.0)
    want, _ = od.forward(q, k, v, g, beta, 1.0)
    assert float(want[0, 0, 31].min()) > 2.0 ** -18 * 16
    near(o[0, 0, 31], want[0, 0, 31], 32 * 1.5, "o")


@pytest.mark.parametrize("d", [32, 64, 128])
def test_decayed_products_in_the_outputs(d):
    """The same with decays: token 2m + 1 writes e^g of what token 2m writes, so that their terms in the
    last token's output, of different decays, cancel to fp32; the pairs' signs add up what 16 bits of
    the decays would leave."""
    gen = torch.Generator().manual_seed(d + 2)
    g = -0.05 * torch.rand(1, 1, 32, generator=gen)
    beta = torch.ones(1, 1, 32)
    beta[..., 1::2] = g[..., 1::2].double().exp().float()
    c = g.double().cumsum(-1)
    decay = (c[..., -1:] - c).exp().float()[0, 0]
    left = ((decay - short(decay)) * beta[0, 0]).double()
    sign = torch.where(left[0::2] >= left[1::2], 1.0, -1.0)
    terms = float((decay * beta[0, 0]).sum())
    assert float((sign * (left[0::2] - left[1::2])).sum()) > 2 * 2.0 ** -21 * terms
    k = torch.eye(32, d)[None, None].bfloat16()
    q = torch.zeros(1, 1, 32, d)
    q[0, 0, 31, 0:32:2], q[0, 0, 31, 1:32:2] = sign, -sign
    q, v = q.bfloat16(), torch.ones(1, 1, 32, 32).bfloat16()
    o = hla.gated_delta(*on(q, k, v, g, beta), scale=1.0)
    want, _ = od.forward(q, k, v, g, beta, 1.0)
    near(o[0, 0, 31], want[0, 0, 31], terms, "o")


def test_pairs_in_dq():
    """dq of the last token = the sum of w_j k_j, where w_j is what token j wrote: x and y in turn, on
    keys with a small common part of alternating sign."""
    d, T, n = 64, 32, 30
    x = residues(n // 2, 7)
    target = torch.stack([x, short(x)], 1).reshape(n).double()
    k = torch.zeros(T, d)
    k[:n, :n] = torch.eye(n)
    k[:n, d - 1] = 2.0 ** -6 * torch.tensor([1.0, -1.0]).repeat(n // 2)
    # beta_j such that token j writes its target, by the recurrence in 64 bits
    beta, s = torch.zeros(T), torch.zeros(d, dtype=torch.float64)
    for j in range(n):
        beta[j] = float(target[j] / (1 - s @ k[j].double()))
        s = s + float(beta[j]) * k[j].double() * (1 - s @ k[j].double())
    v, dout = torch.zeros(1, 1, T, 32), torch.zeros(1, 1, T, 32)
    v[0, 0, :n, 0], dout[0, 0, T - 1, 0] = 1.0, 1.0
    q, k, v, dout = torch.zeros(1, 1, T, d).bfloat16(), k[None, None].bfloat16(), v.bfloat16(), dout.bfloat16()
    g, beta = torch.zeros(1, 1, T), beta[None, None]
    got = hla.gated_delta_backward(*on(q, k, v, g, beta, dout), scale=1.0)
    want = od.backward(q, k, v, g, beta, 1.0, dout)["dq"][0, 0, T - 1]
    assert float(want[d - 1]) > 2.0 ** -6 * 2.0 ** -18 * n / 2
    near(got[0][0, 0, T - 1, d - 1], want[d - 1], 2.0 ** -6 * 1.5 * n, "dq")
    near(got[0][0, 0, T - 1, :n], want[:n], 1.5, "dq")


@pytest.mark.parametrize("d", [32, 64, 128])
def test_pairs_in_dk(d):
    """Token 0 writes (x, y) into two columns, and the gradients at the next output are 1 and -1 there."""
    x = residues(1, 9)[0]
    S = torch.zeros(1, 1, d, 32)
    S[0, 0, 0, 0], S[0, 0, 0, 1] = -x, -short(x)
    q, k, v, dout = (torch.zeros(1, 1, 2, w) for w in (d, d, 32, 32))
    k[0, 0, 0, 0] = q[0, 0, 1, 1] = dout[0, 0, 1, 0] = 1.0
    dout[0, 0, 1, 1] = -1.0
    q, k, v, dout = (t.bfloat16() for t in (q, k, v, dout))
    g, beta = torch.zeros(1, 1, 2), torch.ones(1, 1, 2)
    got = hla.gated_delta_backward(*on(q, k, v, g, beta, dout), scale=1.0, initial_state=S.to(DEV))
    want = od.backward(q, k, v, g, beta, 1.0, dout, S)["dk"][0, 0, 0]
    assert float(want[1]) > 2.0 ** -18
    near(got[1][0, 0, 0], want, 2 * 1.5, "dk")


@pytest.mark.parametrize("d", [32, 64, 128])
def test_shared_heads_in_dk(d):
    """The same over two value heads of one key head: x of the first, -y of the second."""
    x = residues(1, 9)[0]
    S = torch.zeros(1, 2, d, 32)
    S[0, 0, 0, 0], S[0, 1, 0, 0] = -x, -short(x)
    q, k, v, dout = (torch.zeros(1, h, 2, w) for h, w in ((1, d), (1, d), (2, 32), (2, 32)))
    k[0, 0, 0, 0] = q[0, 0, 1, 1] = dout[0, 0, 1, 0] = 1.0
    dout[0, 1, 1, 0] = -1.0
    q, k, v, dout = (t.bfloat16() for t in (q, k, v, dout))
    g, beta = torch.zeros(1, 2, 2), torch.ones(1, 2, 2)
    got = hla.gated_delta_backward(*on(q, k, v, g, beta, dout), scale=1.0, initial_state=S.to(DEV))
    want = od.backward(q, k, v, g, beta, 1.0, dout, S)["dk"][0, 0, 0]
    assert float(want[1]) > 2.0 ** -18
    near(got[1][0, 0, 0], want, 2 * 1.5, "dk")
