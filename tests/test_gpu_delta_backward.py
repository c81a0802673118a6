"""Gradients of the gated delta rule on the GPU against the 64-bit adjoint recurrence.

Tolerances.  The fp32 part as for the forward (tests/test_gpu_delta.py): a gradient passes three
chains of such sums (states, their gradients, the block's products), each within 1e-5 of the largest
value: 3e-5 of the largest value of dq, dk, dv, dbeta, dstate.  dg is a difference of terms
q . dq, k . dk and <dS, S>, then a sum over at most 64 tokens: its room is 3e-5 of the largest of
those terms' sizes, taken as max |S| |dS| summed by the norms of the rows.  A bf16 result is rounded
once: 2^-8 of its value.
"""
import math

import pytest

torch = pytest.importorskip("torch")
import higher_order_linear_chunked_b200 as hla  # noqa: E402
from oracle import delta as od  # noqa: E402
from test_gpu_delta import DEV, DT, back, leaves, put  # noqa: E402

pytestmark = pytest.mark.gpu
ROOM = 3.0e-5


def inputs(dtype, B, Hk, H, T, d, dv, seed, state=True, dstate=True, **kw):
    x = leaves(dtype, B, Hk, H, T, d, dv, seed, state=state, **kw)
    gen = torch.Generator().manual_seed(seed + 1000)
    dout = torch.randn(B, H, T, dv, generator=gen).to(DT[dtype])
    return x, dout, torch.randn(B, H, d, dv, generator=gen) * 0.3 if dstate else None


def run(x, dout, dstate, scale, lengths=None, layout="bhtd", **kw):
    q, k, v, g, beta, S0 = x
    got = hla.gated_delta_backward(*(put(t, layout) for t in (q, k, v, g, beta)), put(dout, layout), scale=scale,
                                   initial_state=S0.to(DEV) if S0 is not None else None,
                                   dstate=dstate.to(DEV) if dstate is not None else None,
                                   lengths=lengths.to(DEV) if lengths is not None else None, layout=layout, **kw)
    torch.cuda.synchronize()
    out = {n: back(t, layout) for n, t in zip(("dq", "dk", "dv", "dg", "dbeta"), got)}
    assert (got[5] is None) == (S0 is None)
    if got[5] is not None:
        out["dstate"] = got[5].cpu()
    return out


def compare(x, dout, dstate, scale, lengths=None, layout="bhtd"):
    got = run(x, dout, dstate, scale, lengths, layout)
    want = od.backward(*x[:5], scale, dout, x[5], dstate, lengths)
    # the size of the terms of dg: every one is at most |q||dq| or |k||dk| of a token, 64 of them summed
    norm = lambda t: float(t.double().norm(dim=-1).max())  # noqa: E731
    terms = norm(x[0]) * norm(want["dq"]) + norm(x[1]) * norm(want["dk"])
    if dstate is not None and x[5] is not None:
        terms += float((want["dstate"] * x[5].double()).abs().sum((-1, -2)).max())
    for name, ref in want.items():
        if name not in got:
            continue
        t = got[name]
        assert t.shape == ref.shape, name
        rounding = 2.0 ** -8 if t.dtype == torch.bfloat16 else 0.0
        size = max(terms, float(ref.abs().max())) if name == "dg" else float(ref.abs().max())
        room = rounding * ref.abs() + ROOM * max(size, 1e-30)
        off = (t.double() - ref).abs()
        assert bool((off <= room).all()), f"{name}: {float((off / room).max()):.3g} times the tolerance"
    return got, want


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 31, 33, 64, 65, 96, 150])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_lengths_and_widths(dtype, T, d):
    compare(*inputs(dtype, 2, 2, 2, T, d, d, seed=T + d), d ** -0.5)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,dv", [(32, 64), (32, 128), (64, 32), (64, 128), (128, 32), (128, 64)])
@pytest.mark.parametrize("layout", ["bhtd", "bthd"])
def test_unequal_widths_shared_heads_and_layouts(dtype, d, dv, layout):
    compare(*inputs(dtype, 2, 2, 6, 77, d, dv, seed=d + dv), 0.3, layout=layout)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["bhtd", "bthd"])
@pytest.mark.parametrize("Hk", [1, 2])
def test_padded_batch(dtype, layout, Hk):
    lens = torch.tensor([0, 1, 45, 96, 130, 500, -3], dtype=torch.int32)
    B, H, T = len(lens), 2, 130
    x, dout, dstate = inputs(dtype, B, Hk, H, T, 64, 64, seed=3)
    want = od.backward(*x[:5], 0.2, dout, x[5], dstate, lens)
    assert all(torch.isfinite(w).all() for w in want.values())
    clean = run(x, dout, dstate, 0.2, lens, layout)
    for b, n in enumerate(lens.clamp(0, T).tolist()):
        for t in (*x[:5], dout):
            t[b, :, n:] = math.nan
    got = run(x, dout, dstate, 0.2, lens, layout)
    for name, t in got.items():
        assert torch.equal(t, clean[name]), name               # what is behind an end is not used
    for b, n in enumerate(lens.clamp(0, T).tolist()):
        for t in x[:5]:
            t[b, :, n:] = 0.0
        dout[b, :, n:] = 0.0
        for name in ("dq", "dk", "dv", "dg", "dbeta"):
            assert not got[name][b, :, n:].any(), name
    compare(x, dout, dstate, 0.2, lens, layout)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("state,dstate", [(False, False), (True, False), (False, True)])
def test_with_and_without_states(dtype, state, dstate):
    compare(*inputs(dtype, 1, 2, 2, 100, 64, 64, seed=4, state=state, dstate=dstate), 0.125)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_resets_strong_decays_and_idle_tokens(dtype):
    x, dout, dstate = inputs(dtype, 1, 2, 2, 150, 64, 64, seed=8)
    g, beta = x[3], x[4]
    g[0, 0, 0], g[0, 0, 37], g[0, 0, 38], g[0, 1, 64] = -math.inf, -math.inf, -math.inf, -1000.0
    g[0, 1, 100:130:2] = -110.0
    beta[0, :, 5:20] = 0.0
    beta[0, 1, 70] = 1.0
    # the oracle's 0 * -inf has no place here: exp(-1000) is 0 as well
    ref = [t.clone() for t in x[:5]]
    ref[3][torch.isinf(ref[3])] = -1000.0
    got = run(x, dout, dstate, 1.0)
    same = run((*ref, x[5]), dout, dstate, 1.0)
    for name in got:
        assert torch.equal(got[name], same[name]), name
    compare((*ref, x[5]), dout, dstate, 1.0)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_and_many(dtype):
    compare(*inputs(dtype, 1, 1, 2, 1500, 64, 64, seed=12, slow=5.0), 0.125)
    compare(*inputs(dtype, 20, 2, 4, 70, 32, 64, seed=13), 0.2)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,dv", [(32, 64), (64, 64), (128, 128)])
def test_segments_of_a_padded_batch(dtype, d, dv):
    """Few heads and many tokens: both walks go in segments, some of them behind an end."""
    lens = torch.tensor([2000, 630, 0], dtype=torch.int32)
    x, dout, dstate = inputs(dtype, 3, 1, 1, 2000, d, dv, seed=15, slow=4.0)
    assert hla.delta._library().hla_delta_backward_kernel_launches(1 if dtype == "bf16" else 0, 3, 1, 1, 2000, d, dv) == 8
    for b, n in enumerate(lens.tolist()):
        for t in (*x[:5], dout):
            t[b, :, n:] = 0.0
    compare(x, dout, dstate, 0.2, lens)


@pytest.mark.parametrize("d,dv,B,Hk,H,T,layout", [(64, 64, 6, 4, 8, 150, "bhtd"), (32, 64, 6, 8, 8, 97, "bthd"),
                                                  (64, 128, 5, 2, 6, 70, "bthd")])
def test_walks_side_by_side_in_wide_blocks(d, dv, B, Hk, H, T, layout):
    """So many heads that narrow blocks of the two walks would share SMs, and wide ones do not."""
    lens = torch.tensor([T, 0, 33, 64, 1, T + 5][:B], dtype=torch.int32)
    x, dout, dstate = inputs("bf16", B, Hk, H, T, d, dv, seed=21)
    for b, n in enumerate(lens.tolist()):
        for t in (*x[:5], dout):
            t[b, :, n:] = 0.0
    compare(x, dout, dstate, 0.2, lens, layout)
    one, two = run(x, dout, dstate, 0.2, lens, layout), run(x, dout, dstate, 0.2, lens, layout)
    assert all(torch.equal(one[n], two[n]) for n in one)


@pytest.mark.parametrize("dtype,B,H,T,d", [("bf16", 6, 8, 100, 64), ("bf16", 1, 2, 1500, 64), ("f32", 1, 2, 1500, 32),
                                           ("f32", 9, 16, 70, 64)])
def test_walks_side_by_side_in_a_graph(dtype, B, H, T, d):
    """Every replay waits for both walks: new inputs in the captured buffers, the same bits as eager calls."""
    x, dout, dstate = inputs(dtype, B, H, H, T, d, d, seed=22)
    held = [t.to(DEV) for t in (*x[:5], dout, x[5], dstate)]

    def call():
        return hla.gated_delta_backward(*held[:6], scale=0.2, initial_state=held[6], dstate=held[7])

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for seed in (23, 24):
        y, dy, ds = inputs(dtype, B, H, H, T, d, d, seed=seed)
        for to, t in zip(held, (*y[:5], dy, y[5], ds)):
            to.copy_(t)
        for _ in range(3):
            graph.replay()
        want = call()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_against_differences():
    """fp32: the slope of the GPU forward along a direction, by a central difference.  The loss's own
    rounding (2^-24 of its terms' sizes, about 1e-6 of the loss's scale) over the step of 1e-2, and the
    step's square times third derivatives of order one: 1e-4 + 1e-4 of the scale."""
    x, dout, dstate = inputs("f32", 1, 1, 2, 70, 32, 32, seed=6)
    got = run(x, dout, dstate, 0.4)
    gen = torch.Generator().manual_seed(1)

    def loss(y):
        o, S = hla.gated_delta(*(t.to(DEV) for t in y[:5]), scale=0.4, initial_state=y[5].to(DEV), return_state=True)
        return float((o.cpu().double() * dout.double()).sum() + (S.cpu().double() * dstate.double()).sum())

    h = 1e-2
    for i, name in enumerate(("dq", "dk", "dv", "dg", "dbeta", "dstate")):
        way = torch.randn(x[i].shape, generator=gen)
        way = way / way.norm()
        up, down = ([t + s * h * way if j == i else t for j, t in enumerate(x)] for s in (1, -1))
        slope = (loss(up) - loss(down)) / (2 * h)
        scale = max(1.0, float(got[name].double().norm()))
        assert abs(slope - float((got[name].double() * way.double()).sum())) < 2e-3 * scale, name


def test_same_bits_graph_and_streams():
    x, dout, dstate = inputs("bf16", 2, 1, 2, 200, 64, 64, seed=9)
    dev = [t.to(DEV) for t in x]
    do, ds = dout.to(DEV), dstate.to(DEV)
    f = lambda **kw: hla.gated_delta_backward(*dev[:5], do, initial_state=dev[5], dstate=ds, **kw)  # noqa: E731
    ref = f()
    for a, b in zip(ref, f()):
        assert torch.equal(a, b)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = f(stream=side)
    side.synchronize()
    for a, b in zip(ref, got):
        assert torch.equal(a, b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = hla.gated_delta(*dev[:5], initial_state=dev[5])
        got = f()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(ref, got):
            assert torch.equal(a, b)
    assert torch.equal(o, hla.gated_delta(*dev[:5], initial_state=dev[5]))


def test_nothing_beside_the_workspace_is_written():
    x, dout, dstate = inputs("bf16", 2, 1, 2, 75, 64, 32, seed=33)
    dev, do, ds = [t.to(DEV) for t in x], dout.to(DEV), dstate.to(DEV)
    n = hla.gated_delta_backward_workspace_bytes(torch.bfloat16, 2, 1, 2, 75, 64, 32)
    ws = torch.full((n + 8192,), 7, dtype=torch.uint8, device=DEV)
    ref = hla.gated_delta_backward(*dev[:5], do, initial_state=dev[5], dstate=ds)
    got = hla.gated_delta_backward(*dev[:5], do, initial_state=dev[5], dstate=ds, workspace=ws[4096:4096 + n])
    torch.cuda.synchronize()
    for a, b in zip(ref, got):
        assert torch.equal(a, b)
    assert bool((ws[:4096] == 7).all()) and bool((ws[4096 + n:] == 7).all())


def test_refusals():
    x, dout, dstate = inputs("bf16", 1, 2, 4, 8, 64, 64, seed=1)
    dev, do = [t.to(DEV) for t in x], dout.to(DEV)
    with pytest.raises(TypeError, match="dout must be"):
        hla.gated_delta_backward(*dev[:5], do.float())
    with pytest.raises(ValueError, match="dout must be"):
        hla.gated_delta_backward(*dev[:5], do[:, :2])
    with pytest.raises(ValueError, match="dstate must be"):
        hla.gated_delta_backward(*dev[:5], do, dstate=torch.zeros(1, 4, 64, 32, device=DEV))
    with pytest.raises(hla.HLAError, match="WORKSPACE"):
        hla.gated_delta_backward(*dev[:5], do, workspace=torch.empty(1024, dtype=torch.uint8, device=DEV))
