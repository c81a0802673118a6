"""A NaN or an infinity in a live token: what stands before it in the sequence is what it is without."""
import math

import pytest

torch = pytest.importorskip("torch")
import higher_order_linear_chunked_b200 as hla  # noqa: E402
from oracle import delta as od  # noqa: E402
from test_gpu_delta import DEV, leaves  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("which", ["q", "k", "v", "g", "beta"])
@pytest.mark.parametrize("t", [0, 5, 31, 44, 79])
def test_earlier_outputs_stay(dtype, d, bad, which, t):
    x = [y.to(DEV) for y in leaves(dtype, 1, 2, 2, 80, d, 64, seed=d, state=True)]
    ref = hla.gated_delta(*x[:5], initial_state=x[5])
    i = "q k v g beta".split().index(which)
    x[i] = x[i].clone()
    if which in ("g", "beta"):
        x[i][0, 1, t] = bad
    else:
        x[i][0, 1, t, 7] = bad
    o = hla.gated_delta(*x[:5], initial_state=x[5])
    assert torch.equal(o[:, 0], ref[:, 0])                      # the other head
    assert torch.equal(o[:, 1, :t], ref[:, 1, :t])              # the tokens before
    hit = ~torch.isfinite(o[0, 1])
    if which == "v":
        other = [c for c in range(64) if c != 7]
        assert torch.equal(o[:, 1][..., other], ref[:, 1][..., other])
        assert bool(hit[t:, 7].all())
    elif which == "q":
        assert torch.equal(o[:, 1, t + 1:], ref[:, 1, t + 1:]) and bool(hit[t].all())
    else:
        assert bool(hit[t:].all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("which", ["k", "v", "beta"])
@pytest.mark.parametrize("t", [3, 1000, 1999])
def test_earlier_segments_stay(dtype, which, t):
    """A sequence walked in segments."""
    x = [y.to(DEV) for y in leaves(dtype, 1, 1, 1, 2000, 64, 64, seed=2, state=True, slow=4.0)]
    ref, S = hla.gated_delta(*x[:5], initial_state=x[5], return_state=True)
    i = "q k v g beta".split().index(which)
    x[i] = x[i].clone()
    x[i][(0, 0, t) if which == "beta" else (0, 0, t, 7)] = math.nan
    o, last = hla.gated_delta(*x[:5], initial_state=x[5], return_state=True)
    assert torch.equal(o[:, :, :t], ref[:, :, :t])
    if which == "v":
        other = [c for c in range(64) if c != 7]
        assert torch.equal(o[..., other], ref[..., other]) and torch.equal(last[..., other], S[..., other])
        assert bool(torch.isnan(o[0, 0, t:, 7]).all()) and bool(torch.isnan(last[..., 7]).all())
    else:
        assert bool(torch.isnan(o[:, :, t:]).all()) and bool(torch.isnan(last).all())


def test_a_state_that_is_not_finite():
    """One column of it: the other columns' outputs and state are what they are without."""
    x = [y.to(DEV) for y in leaves("bf16", 1, 1, 1, 70, 64, 64, seed=4, state=True)]
    ref, S = hla.gated_delta(*x[:5], initial_state=x[5], return_state=True)
    x[5][0, 0, 3, 9] = math.inf
    o, last = hla.gated_delta(*x[:5], initial_state=x[5], return_state=True)
    other = [c for c in range(64) if c != 9]
    assert torch.equal(o[..., other], ref[..., other]) and torch.equal(last[..., other], S[..., other])
    assert not bool(torch.isfinite(o[..., 9]).any())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,dv", [(32, 128), (64, 64), (128, 64)])
@pytest.mark.parametrize("layout", ["bhtd", "bthd"])
def test_many_bad_values(dtype, d, dv, layout):
    """NaN in v at scattered places, another first token in every column (both halves of a chunk, several in
    one column), a bad key behind them and NaN behind the end of one sequence."""
    B, H, T = 3, 2, 100
    x = leaves(dtype, B, 1, H, T, d, dv, seed=d + dv, state=True)
    lens = torch.tensor([100, 61, 100], dtype=torch.int32)
    gen = torch.Generator().manual_seed(d)
    first = torch.full((B, H, dv), T)
    spoilt = x[2].clone()
    for b in range(B):
        for h in range(H):
            for c in range(dv):
                ts = torch.randint(0, T, (int(torch.randint(0, 4, (1,), generator=gen)),), generator=gen)
                spoilt[b, h, ts, c] = math.nan if c % 2 else -math.inf
                if len(ts):
                    first[b, h, c] = int(ts.min())
    key = x[1].clone()
    key[2, 0, 77, 3] = math.nan
    first[2] = first[2].clamp(max=77)
    put = lambda t: (t.transpose(1, 2).contiguous() if layout == "bthd" else t).to(DEV)  # noqa: E731
    how = dict(initial_state=x[5].to(DEV), lengths=lens.to(DEV), layout=layout)
    ref = hla.gated_delta(put(x[0]), put(x[1]), put(x[2]), put(x[3]), put(x[4]), **how)
    o = hla.gated_delta(put(x[0]), put(key), put(spoilt), put(x[3]), put(x[4]), **how)
    if layout == "bthd":
        ref, o = ref.transpose(1, 2), o.transpose(1, 2)
    t = torch.arange(T)[None, None, :, None]
    live = t < lens[:, None, None, None]
    hit = (t >= first[:, :, None, :]) & live
    assert torch.equal(~torch.isfinite(o.cpu()), hit)
    assert torch.equal(o.cpu()[~hit], ref.cpu()[~hit])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_an_overflow_stays_out_of_earlier_tokens(dtype, d):
    """Keys of squared length 40 multiply the state by -39 a token, which overflows behind the 23rd: what
    stands before is what the same call over fewer tokens gives."""
    x = leaves(dtype, 1, 1, 1, 60, d, 32, seed=d, state=False)[:5]
    x[1][:] = math.sqrt(40) * x[1][:, :, :1].clone()
    x[3][:], x[4][:] = 0.0, 1.0
    want, S = od.forward(*x[:5], 1.0)
    dev = [t.to(DEV) for t in x]
    full = hla.gated_delta(*dev, scale=1.0)
    assert not bool(torch.isfinite(full[:, :, 40:]).any())
    for n in (3, 17, 21):
        assert float(want[:, :, :n].abs().max()) < 1e36
        part = hla.gated_delta(*dev, scale=1.0, lengths=torch.tensor([n], dtype=torch.int32, device=DEV))
        assert bool(torch.isfinite(part).all()) and torch.equal(full[:, :, :n], part[:, :, :n])
