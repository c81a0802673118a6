"""fp32 gradients of the gated delta rule against differences of the GPU forward, along the gradient itself,
where the slope is the gradient's norm.

Tolerance.  The slope over +-h is off by what the loss curves (taken from the 64-bit recurrence at the same
points) and by the outputs' own errors: each output within 2e-5 of the largest (tests/test_gpu_delta.py),
independent of one another, so over N outputs sqrt(N) of them times the largest dout, twice over 2 h; the
gradient's own error is within 3e-5 of its largest element for each of n elements (tests/test_gpu_delta_backward.py),
sqrt(n) of them along a unit direction.  The whole has to stay below 1% of the slope.
"""
import math

import pytest

torch = pytest.importorskip("torch")
import higher_order_linear_chunked_b200 as hla  # noqa: E402
from oracle import delta as od  # noqa: E402
from test_gpu_delta import DEV  # noqa: E402
from test_gpu_delta_backward import inputs, run  # noqa: E402

pytestmark = pytest.mark.gpu
# o is linear in q, v and the state: any step will do
STEP = {"dq": 1.0, "dk": 0.2, "dv": 1.0, "dg": 0.2, "dbeta": 0.2, "dstate": 1.0}


@pytest.mark.parametrize("i,name", list(enumerate(STEP)))
@pytest.mark.parametrize("noise", [0.0, 1.0])
def test_slope_along_the_gradient(i, name, noise):
    x, dout, dstate = inputs("f32", 1, 1, 2, 70, 32, 32, seed=6)
    got = run(x, dout, dstate, 0.4)[name].double()
    exact = od.backward(*x[:5], 0.4, dout, x[5], dstate)[name]
    way = got / got.norm()
    if noise:
        other = torch.randn(got.shape, generator=torch.Generator().manual_seed(i), dtype=torch.float64)
        way = way + noise * other / other.norm()
        way = way / way.norm()
    h = STEP[name]
    ends = [[(t.double() + s * h * way).float() if j == i else t for j, t in enumerate(x)] for s in (1, -1)]
    way = (ends[0][i].double() - ends[1][i].double()) / (2 * h)             # as fp32 holds it

    def loss(o, S):
        return float((o.double() * dout.double()).sum() + (S.double() * dstate.double()).sum())

    def here(y):
        o, S = hla.gated_delta(*(t.to(DEV) for t in y[:5]), scale=0.4, initial_state=y[5].to(DEV), return_state=True)
        return loss(o.cpu(), S.cpu())

    slope = (here(ends[0]) - here(ends[1])) / (2 * h)
    at = [od.forward(*y[:5], 0.4, y[5]) for y in ends]
    curve = abs((loss(*at[0]) - loss(*at[1])) / (2 * h) - float((exact * way).sum()))
    room = sum(math.sqrt(o.numel()) * 2e-5 * float(o.abs().max()) * float(d.abs().max()) for o, d in zip(at[0], (dout, dstate))) / h
    room += curve + 3e-5 * float(exact.abs().max()) * math.sqrt(got.numel())
    assert room < 0.01 * abs(slope), (room, slope)
    assert abs(slope - float((got * way).sum())) <= room, (slope, float((got * way).sum()), room)
