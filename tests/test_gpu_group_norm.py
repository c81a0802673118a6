"""Group norm on the GPU against its formulas in 64 bits (oracle/delta.py).

Tolerances.  Statistics are sums of at most 512 terms taken in pieces of at most 16 and a tree of
five levels: (16 + 5 + 10) 2^-24 = 2e-6 of the terms' size; the output passes them through a few
products: 1e-5 of the largest value.  The gradient of x is the difference
r (e - n mean(e n) - mean(e)) of terms of size r |e| (e = dz w) that may cancel, entirely so in a
group of one channel: each term carries its own roundings, so the room is 2e-5 of the largest r |e|,
with |n| <= 1 in a group of one and the mean |e n| <= max |e| max |n| elsewhere.  The
sums over rows add at most (rows / slots + slots / 8 + 8) terms one after another, below 400 here:
400 2^-24 = 2.4e-5 of the sum of the terms' absolute values.  A bf16 result is rounded once more:
2^-8 of its value.
"""
import pytest

torch = pytest.importorskip("torch")
import higher_order_linear_chunked_b200 as hla  # noqa: E402
from oracle import delta as od  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def inputs(dtype, rows, groups, width, gated, affine, seed):
    gen = torch.Generator().manual_seed(seed)
    C = groups * width
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    x, dy = (r(rows, C) * 0.7 + 0.2).to(DT[dtype]), r(rows, C).to(DT[dtype])
    gate = r(rows, C).to(DT[dtype]) if gated else None
    return x, dy, gate, 1 + 0.3 * r(C) if affine else None, 0.2 * r(C) if affine else None


def check(got, want, room, name):
    got = got.cpu()
    assert got.shape == want.shape, name
    rounding = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    room = rounding * want.abs() + room
    off = (got.double() - want).abs()
    assert bool((off <= room).all()), f"{name}: {float((off / room).max()):.3g} times the tolerance"


def both(dtype, rows, groups, width, gated, affine, activation, center, seed=0):
    x, dy, gate, w, b = inputs(dtype, rows, groups, width, gated, affine, seed)
    how = dict(eps=1e-5, activation=activation, center=center)
    dev = lambda t: t.to(DEV) if t is not None else None  # noqa: E731
    y = hla.group_norm(dev(x), groups, dev(w), dev(b), dev(gate), **how)
    got = hla.group_norm_backward(dev(x), dev(dy), groups, dev(w), dev(b), dev(gate), **how)
    torch.cuda.synchronize()
    want = od.group_norm(x, groups, w, b, gate, **how)
    check(y, want, 1e-5 * float(want.abs().max()), "y")
    dx, dgate, dw, db = od.group_norm_backward(x, dy, groups, w, b, gate, **how)
    size = dy.double().abs() * (2.0 if gate is None else 1.0)     # |act'| <= 1.1
    if gated:
        size = size * gate.double().abs().clamp(min=1.0)
    xg = x.double().reshape(rows, groups, width)
    xg = xg - xg.mean(-1, keepdim=True) if center else xg
    r = 1 / torch.sqrt((xg * xg).mean(-1, keepdim=True) + 1e-5)
    e = (size * (w.double().abs() if affine else 1.0)).reshape(rows, groups, width)
    check(got[0], dx, 2e-5 * float((r * e).max()), "dx")
    assert (got[1] is None) == (dgate is None) and (got[2] is None) == (dw is None) == (got[3] is None)
    if gated:
        check(got[1], dgate, 1e-5 * float(dgate.abs().max()), "dgate")
    if affine:
        # the sizes of the summed terms: |dz n| and |dz|, from the same formulas
        n = od.group_norm(x, groups, eps=1e-5, center=center).abs()
        check(got[2], dw, 2.4e-5 * (size * n).sum(0), "dweight")
        check(got[3], db, 2.4e-5 * size.sum(0), "dbias")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 3, 130])
@pytest.mark.parametrize("groups,width", [(1, 1), (3, 1), (16, 64), (7, 33), (5, 100), (2, 200), (1, 257), (2, 512),
                                          (33, 32), (3, 12)])
def test_widths(dtype, rows, groups, width):
    both(dtype, rows, groups, width, True, True, "silu", False, seed=rows + width)
    both(dtype, rows, groups, width, False, True, "silu", True, seed=rows + width + 1)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("affine", [True, False])
@pytest.mark.parametrize("activation", ["none", "silu"])
@pytest.mark.parametrize("center", [True, False])
def test_forms(dtype, gated, affine, activation, center):
    both(dtype, 70, 6, 64, gated, affine, activation, center, seed=7)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_many_rows(dtype):
    both(dtype, 5003, 4, 64, True, True, "silu", False, seed=11)


def test_one_of_weight_and_bias():
    x, dy, _, w, b = inputs("f32", 20, 3, 40, False, True, 2)
    dx, _, dw, db = hla.group_norm_backward(x.to(DEV), dy.to(DEV), 3, weight=w.to(DEV))
    want = od.group_norm_backward(x, dy, 3, w, None)
    assert db is None
    check(dw, want[2], 2.4e-5 * float(dy.abs().sum(0).max() * 5), "dweight")
    y = hla.group_norm(x.to(DEV), 3, bias=b.to(DEV))
    check(y, od.group_norm(x, 3, None, b), 1e-4, "y")


def test_extreme_rows():
    """A row of zeros, a constant row, a huge and a tiny one: finite, and what 64 bits give."""
    x = torch.randn(6, 64, generator=torch.Generator().manual_seed(1))
    x[0], x[1], x[2], x[3] = 0.0, 3.0, x[2] * 1e15, x[3] * 1e-15
    for center in (True, False):
        y = hla.group_norm(x.to(DEV), 2, center=center)
        want = od.group_norm(x, 2, center=center)
        # the constant row: the mean's own rounding of 2^-24 x 3 over sqrt(eps) = 1.8e-7 / 3.2e-3
        check(y, want, 1e-4 if center else 2e-5, "y")
        assert not y[0].any()


def test_nan_stays_in_its_group():
    x, dy, gate, w, b = inputs("bf16", 40, 4, 64, True, True, 3)
    ref = hla.group_norm(x.to(DEV), 4, w.to(DEV), b.to(DEV), gate.to(DEV), activation="silu")
    x[7, 70] = float("nan")
    y = hla.group_norm(x.to(DEV), 4, w.to(DEV), b.to(DEV), gate.to(DEV), activation="silu")
    bad = torch.zeros(40, 256, dtype=torch.bool)
    bad[7, 64:128] = True
    assert torch.equal(torch.isnan(y.cpu()), bad)
    assert torch.equal(y.cpu()[~bad], ref.cpu()[~bad])


def test_in_place_and_guards():
    """out= x or gate; nothing outside the rows is written."""
    x, _, gate, w, b = inputs("bf16", 33, 4, 64, True, True, 5)
    ref = hla.group_norm(x.to(DEV), 4, w.to(DEV), b.to(DEV), gate.to(DEV))
    a, c = x.to(DEV), gate.to(DEV)
    hla.group_norm(a, 4, w.to(DEV), b.to(DEV), c, out=a)
    assert torch.equal(a, ref)
    a = x.to(DEV)
    hla.group_norm(a, 4, w.to(DEV), b.to(DEV), c, out=c)
    assert torch.equal(c, ref)
    big = torch.full((33 + 8, 256), 7.0, dtype=torch.bfloat16, device=DEV)
    hla.group_norm(x.to(DEV), 4, w.to(DEV), b.to(DEV), gate.to(DEV), out=big[4:37])
    assert torch.equal(big[4:37], ref) and bool((big[:4] == 7).all()) and bool((big[37:] == 7).all())


def test_gradients_in_a_graph_repeat_their_bits():
    x, dy, gate, w, b = (t.to(DEV) for t in inputs("bf16", 2000, 8, 64, True, True, 6))
    ref = hla.group_norm_backward(x, dy, 8, w, b, gate, activation="silu")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = hla.group_norm_backward(x, dy, 8, w, b, gate, activation="silu")
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for r, t in zip(ref, got):
            assert torch.equal(r, t)


def test_refusals():
    x = torch.zeros(4, 64, device=DEV)
    with pytest.raises(ValueError, match="do not divide"):
        hla.group_norm(x, 3)
    with pytest.raises(ValueError, match="activation"):
        hla.group_norm(x, 2, activation="relu")
    with pytest.raises(TypeError, match="gate must be"):
        hla.group_norm(x, 2, gate=x.bfloat16())
    with pytest.raises(ValueError, match="weight must be"):
        hla.group_norm(x, 2, weight=torch.ones(63, device=DEV))
    with pytest.raises(ValueError, match="contiguous"):
        hla.group_norm(x.t(), 2)
    with pytest.raises(hla.HLAError, match="SHAPE"):
        hla.group_norm(x[:0], 2)
    with pytest.raises(hla.HLAError, match="UNSUPPORTED"):
        hla.group_norm(torch.zeros(1, 513, device=DEV), 1)
    with pytest.raises(hla.HLAError, match="WORKSPACE"):
        hla.group_norm_backward(x, x, 2, weight=torch.ones(64, device=DEV),
                                workspace=torch.empty(0, dtype=torch.uint8, device=DEV))
