"""States that forget slowly, over many chunks and in one walk (so many heads that the sequence is not cut).

Tolerance.  A chunk of 32 tokens changes a state's elements by two roundings (the decay's product, the sum
with the chunk's own products) of 2^-24 each and by the roundings of its products, which are of the size of
the change, not of the state.  Over n chunks: 2 n 2^-24 of the largest value, 6.1e-5 for 512 chunks.
"""
import pytest

torch = pytest.importorskip("torch")
import higher_order_linear_chunked_b200 as hla  # noqa: E402
from higher_order_linear_chunked_b200 import delta  # noqa: E402
from oracle import delta as od  # noqa: E402
from test_gpu_delta import DEV, leaves  # noqa: E402

pytestmark = pytest.mark.gpu


def slow(dtype, T, d, seed):
    q, k, v, g, beta, S = leaves(dtype, 1, 1, 1, T, d, d, seed, state=True)
    gen = torch.Generator().manual_seed(seed + 1)
    g = -1e-6 * torch.rand(1, 1, T, generator=gen)
    return [q, k, v, g, 1e-3 * (0.5 + torch.rand(1, 1, T, generator=gen)), 3 * S]


def heads(x, n):
    return x.expand(-1, n, *x.shape[2:]).contiguous().to(DEV)


def off(got, want):
    return float((got.cpu().double() - want).abs().max() / want.abs().max())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_state(dtype, d):
    T, H = 16384, 64
    x = slow(dtype, T, d, d)
    code = hla.HLA_BF16 if dtype == "bf16" else hla.HLA_F32
    while delta._library().hla_delta_kernel_launches(code, 1, H, H, T, d, d) != 2:
        H += 32
    _, S = hla.gated_delta(*(heads(t, H) for t in x[:5]), initial_state=heads(x[5], H), return_state=True)
    _, want = od.forward(*x[:5], d ** -0.5, x[5])
    assert off(S[:, :1], want) <= 2 * (T // 32) * 2.0 ** -24


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_state_gradient(dtype, d):
    T, H = 8192, 64
    x = slow(dtype, T, d, d + 1)
    code = hla.HLA_BF16 if dtype == "bf16" else hla.HLA_F32
    while delta._library().hla_delta_backward_kernel_launches(code, 1, H, H, T, d, d) != 4:
        H += 32
    gen = torch.Generator().manual_seed(d + 2)
    dout = torch.randn(x[2].shape, generator=gen).to(x[2].dtype)
    dS = 30 * torch.randn(x[5].shape, generator=gen)
    got = hla.gated_delta_backward(*(heads(t, H) for t in x[:5]), heads(dout, H), initial_state=heads(x[5], H),
                                   dstate=heads(dS, H))
    want = od.backward(*x[:5], d ** -0.5, dout, x[5], dS)
    assert off(got[5][:, :1], want["dstate"]) <= 2 * (T // 32) * 2.0 ** -24
