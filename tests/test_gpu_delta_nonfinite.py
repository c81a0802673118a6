"""A NaN or an infinity in a live token: what stands before it in the sequence is what it is without."""
import math

import pytest

torch = pytest.importorskip("torch")
import higher_order_linear_chunked_b200 as hla  # noqa: E402
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
