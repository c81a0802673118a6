"""Gated delta rule on the GPU against the 64-bit recurrence (oracle/delta.py).

Tolerances.  fp32 part: an output is a dot product of at most 128 terms of a state whose errors
decay with it (the transitions are contractions here: |k| = 1, beta <= 1, g <= 0), each token adding
a few roundings of 2^-24 per term: (128 + 40) 2^-24 = 1.0e-5 of the largest value bounds it, taken
twice for outputs that pass two such sums (state, then output).  A bf16 result is then rounded once:
at most 2^-8 of its own value.
"""
import math

import pytest

torch = pytest.importorskip("torch")
import higher_order_linear_chunked_b200 as hla  # noqa: E402
from oracle import delta as od  # noqa: E402

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F32 = 2.0e-5
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def leaves(dtype, B, Hk, H, T, d, dv, seed, state=False, slow=2.0):
    gen = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=gen)  # noqa: E731
    unit = lambda x: torch.nn.functional.normalize(torch.nn.functional.silu(x), dim=-1)  # noqa: E731
    q, k, v = unit(r(B, Hk, T, d)).to(DT[dtype]), unit(r(B, Hk, T, d)).to(DT[dtype]), r(B, H, T, dv).to(DT[dtype])
    g = -torch.nn.functional.softplus(r(B, H, T) - slow)
    beta = torch.sigmoid(r(B, H, T))
    return q, k, v, g, beta, r(B, H, d, dv) * 0.3 if state else None


def put(x, layout="bhtd"):
    if x is None:
        return None
    return (x.transpose(1, 2).contiguous() if layout == "bthd" else x.contiguous()).to(DEV)


def back(x, layout="bhtd"):
    return (x.transpose(1, 2) if layout == "bthd" else x).cpu()


def check(got, want, name=""):
    got = got.detach().cpu()
    assert got.shape == want.shape, (name, got.shape, want.shape)
    rounding = 2.0 ** -8 if got.dtype == torch.bfloat16 else 0.0
    room = rounding * want.abs() + F32 * max(float(want.abs().max()), 1e-30)
    off = (got.double() - want).abs()
    assert bool((off <= room).all()), f"{name}: {float((off / room).max()):.3g} times the tolerance"


def run(x, scale, lengths=None, layout="bhtd"):
    q, k, v, g, beta, S0 = x
    o, S = hla.gated_delta(*(put(t, layout) for t in (q, k, v, g, beta)), scale=scale,
                           initial_state=S0.to(DEV) if S0 is not None else None,
                           lengths=lengths.to(DEV) if lengths is not None else None, layout=layout, return_state=True)
    torch.cuda.synchronize()
    return back(o, layout), S.cpu()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T", [1, 2, 31, 32, 33, 64, 65, 200])
@pytest.mark.parametrize("d", [32, 64, 128])
def test_forward_lengths_and_widths(dtype, T, d):
    x = leaves(dtype, 2, 2, 2, T, d, d, seed=T + d, state=T % 2 == 1)
    o, S = run(x, d ** -0.5)
    want, last = od.forward(*x[:5], d ** -0.5, x[5])
    check(o, want, "o")
    check(S, last, "state")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,dv", [(32, 64), (32, 128), (64, 32), (64, 128), (128, 32), (128, 64)])
@pytest.mark.parametrize("layout", ["bhtd", "bthd"])
def test_unequal_widths_shared_heads_and_layouts(dtype, d, dv, layout):
    x = leaves(dtype, 2, 2, 6, 77, d, dv, seed=d + dv, state=True)
    o, S = run(x, 0.3, layout=layout)
    want, last = od.forward(*x[:5], 0.3, x[5])
    check(o, want, "o")
    check(S, last, "state")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("layout", ["bhtd", "bthd"])
def test_padded_batch(dtype, layout):
    """Lengths 0, 1, mid-chunk, exactly T, beyond T and negative; NaN behind every end."""
    lens = torch.tensor([0, 1, 45, 96, 130, 500, -3], dtype=torch.int32)
    B, H, T, d = len(lens), 2, 130, 64
    x = leaves(dtype, B, 1, H, T, d, d, seed=3, state=True)
    want, last = od.forward(*x[:5], 0.2, x[5], lens)
    for b, n in enumerate(lens.clamp(0, T).tolist()):
        for t in x[:5]:
            t[b, :, n:] = math.nan
    o, S = run(x, 0.2, lens, layout)
    check(o, want, "o")
    check(S, last, "state")
    for b, n in enumerate(lens.clamp(0, T).tolist()):
        assert not o[b, :, n:].any()
        if n == 0:
            assert torch.equal(S[b], x[5][b])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_resets_strong_decays_and_idle_tokens(dtype):
    """Log decays of -inf and -1000 start a head anew (packed documents); beta = 0 writes nothing;
    a chunk whose decays sum to thousands keeps the small gaps exact."""
    x = leaves(dtype, 1, 2, 2, 150, 64, 64, seed=8, state=True)
    g, beta = x[3], x[4]
    g[0, 0, 0], g[0, 0, 37], g[0, 0, 38], g[0, 1, 64] = -math.inf, -math.inf, -math.inf, -1000.0
    g[0, 1, 100:130:2] = -110.0
    beta[0, :, 5:20] = 0.0
    beta[0, 1, 70] = 1.0
    o, S = run(x, 1.0)
    want, last = od.forward(*x[:5], 1.0, x[5])
    check(o, want, "o")
    check(S, last, "state")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_equal_keys(dtype):
    """All keys the same and beta = 1: the triangular systems of this case are the worst conditioned."""
    x = leaves(dtype, 1, 1, 2, 100, 64, 64, seed=5)
    x[1][:] = x[1][:, :, :1].clone()
    x[4][:] = 1.0
    x[3][:] = 0.0
    o, S = run(x, 1.0)
    want, last = od.forward(*x[:5], 1.0)
    check(o, want, "o")
    check(S, last, "state")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_long_few_heads(dtype):
    x = leaves(dtype, 1, 1, 1, 4100, 64, 64, seed=12, state=True, slow=5.0)
    o, S = run(x, 0.125)
    want, last = od.forward(*x[:5], 0.125, x[5])
    check(o, want, "o")
    check(S, last, "state")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,dv", [(32, 64), (64, 64), (128, 32), (128, 128)])
def test_segments_of_a_padded_batch(dtype, d, dv):
    """Few heads and many tokens: the sequence is walked in segments, some of them behind an end."""
    lens = torch.tensor([2000, 630, 0], dtype=torch.int32)
    x = leaves(dtype, 3, 1, 1, 2000, d, dv, seed=14, state=True, slow=4.0)
    assert hla.delta._library().hla_delta_kernel_launches(1 if dtype == "bf16" else 0, 3, 1, 1, 2000, d, dv) == 4
    want, last = od.forward(*x[:5], 0.2, x[5], lens)
    for b, n in enumerate(lens.tolist()):
        for t in x[:5]:
            t[b, :, n:] = math.nan
    o, S = run(x, 0.2, lens, "bthd")
    check(o, want, "o")
    check(S, last, "state")
    assert torch.equal(S[2], x[5][2])


def test_many_heads():
    x = leaves("bf16", 40, 4, 8, 70, 64, 64, seed=13)
    o, S = run(x, 0.125)
    want, last = od.forward(*x[:5], 0.125)
    check(o, want, "o")
    check(S, last, "state")


def test_more_heads_than_a_grid_axis():
    """70400 heads (a grid's second axis ends at 65535): every head's result, by a repeated batch."""
    x = leaves("bf16", 4, 1, 64, 2, 32, 32, seed=31, state=True)
    many = [t.repeat(275, *([1] * (t.dim() - 1))).to(DEV) for t in x]
    o, S = hla.gated_delta(*many[:5], scale=0.5, initial_state=many[5], return_state=True)
    want, last = od.forward(*x[:5], 0.5, x[5])
    check(o[-4:], want, "o")
    check(S[-4:], last, "state")
    assert torch.equal(o.view(275, 4, 64, 2, 32), o[:4].expand(275, 4, 64, 2, 32))
    assert torch.equal(S.view(275, 4, 64, 32, 32), S[:4].expand(275, 4, 64, 32, 32))
    step = hla.gated_delta_step(many[5], *(t[:, :, 0].contiguous() for t in many[:5]), scale=0.5)
    check(step[-4:], want[:, :, 0], "step")


def test_nothing_beside_the_outputs_is_written():
    """Outputs, state and workspace in the middle of larger buffers: the rest keeps its values."""
    x = [t.to(DEV) for t in leaves("bf16", 2, 1, 2, 75, 64, 32, seed=32)[:5]]
    n = hla.gated_delta_workspace_bytes(torch.bfloat16, 2, 1, 2, 75, 64, 32)
    big = [torch.full((4, 2, 75, 32), 7.0, dtype=torch.bfloat16, device=DEV), torch.full((4, 2, 64, 32), 7.0, device=DEV),
           torch.full((n + 8192,), 7, dtype=torch.uint8, device=DEV)]
    ref, last = hla.gated_delta(*x, return_state=True)
    hla.gated_delta(*x, out=big[0][1:3], state_out=big[1][1:3], workspace=big[2][4096:4096 + n])
    torch.cuda.synchronize()
    assert torch.equal(big[0][1:3], ref) and torch.equal(big[1][1:3], last)
    for t in (big[0][0], big[0][3], big[1][0], big[1][3], big[2][:4096], big[2][4096 + n:]):
        assert bool((t == 7).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("d,dv", [(32, 32), (64, 64), (128, 128), (64, 128), (128, 32)])
@pytest.mark.parametrize("B,Hk,H", [(1, 1, 1), (5, 2, 6)])
def test_step(dtype, d, dv, B, Hk, H):
    x = leaves(dtype, B, Hk, H, 3, d, dv, seed=d, state=True)
    S = x[5].to(DEV)
    outs = [hla.gated_delta_step(S, *(t[:, :, i].contiguous().to(DEV) for t in x[:5]), scale=0.5) for i in range(3)]
    torch.cuda.synchronize()
    want, last = od.forward(*x[:5], 0.5, x[5])
    check(torch.stack(outs, 2), want, "o")
    check(S, last, "state")


def test_prefill_in_pieces_then_decode_is_the_whole():
    """A prompt in two pieces, the state updated in its own buffer, then steps: the one pass."""
    x = leaves("bf16", 2, 2, 4, 150, 64, 64, seed=21)
    S = torch.zeros(2, 4, 64, 64, device=DEV)
    outs = []
    for lo, hi in ((0, 90), (90, 147)):
        o, S2 = hla.gated_delta(*(t[:, :, lo:hi].contiguous().to(DEV) for t in x[:5]), initial_state=S, state_out=S,
                                return_state=True)
        assert S2.data_ptr() == S.data_ptr()
        outs.append(o)
    for t in range(147, 150):
        outs.append(hla.gated_delta_step(S, *(y[:, :, t].contiguous().to(DEV) for y in x[:5]))[:, :, None])
    torch.cuda.synchronize()
    want, last = od.forward(*x[:5], 64 ** -0.5)
    check(torch.cat(outs, 2), want, "o")
    check(S, last, "state")


def test_long_prompt_from_its_own_state_buffer():
    x = leaves("bf16", 1, 1, 2, 3000, 64, 64, seed=22, state=True, slow=5.0)
    S = x[5].to(DEV)
    o = hla.gated_delta(*(t.to(DEV) for t in x[:5]), initial_state=S, state_out=S)
    torch.cuda.synchronize()
    want, last = od.forward(*x[:5], 64 ** -0.5, x[5])
    check(o, want, "o")
    check(S, last, "state")


def test_side_stream_and_graph():
    x = leaves("bf16", 2, 2, 2, 300, 64, 64, seed=23, state=True)
    dev = [t.to(DEV) for t in x]
    ref, last = hla.gated_delta(*dev[:5], initial_state=dev[5], return_state=True)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o = hla.gated_delta(*dev[:5], initial_state=dev[5], stream=side)
    side.synchronize()
    assert torch.equal(o, ref)
    ws = torch.empty(hla.gated_delta_workspace_bytes(torch.bfloat16, 2, 2, 2, 300, 64, 64), dtype=torch.uint8, device=DEV)
    out, S = torch.empty_like(ref), torch.empty_like(last)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hla.gated_delta(*dev[:5], initial_state=dev[5], out=out, state_out=S, workspace=ws)
        hla.gated_delta_step(S, *(t[:, :, 0].contiguous() for t in dev[:5]))
    want_o, want_S = ref.clone(), last.clone()
    hla.gated_delta_step(want_S, *(t[:, :, 0].contiguous() for t in dev[:5]))
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want_o) and torch.equal(S, want_S)


def test_same_inputs_same_bits():
    x = [t.to(DEV) for t in leaves("bf16", 1, 2, 4, 2500, 64, 64, seed=24)[:5]]
    a, S = hla.gated_delta(*x, return_state=True)
    b, S2 = hla.gated_delta(*x, return_state=True)
    assert torch.equal(a, b) and torch.equal(S, S2)


def test_refusals():
    x = [t.to(DEV) for t in leaves("bf16", 1, 2, 4, 8, 64, 64, seed=1)[:5]]
    q, k, v, g, beta = x
    with pytest.raises(TypeError, match="k must be"):
        hla.gated_delta(q, k.float(), v, g, beta)
    with pytest.raises(TypeError, match="g must be"):
        hla.gated_delta(q, k, v, g.bfloat16(), beta)
    with pytest.raises(ValueError, match="beta must be"):
        hla.gated_delta(q, k, v, g, beta[..., :7])
    with pytest.raises(ValueError, match="v must be contiguous"):
        hla.gated_delta(q, k, v.transpose(2, 3).contiguous().transpose(2, 3), g, beta)
    with pytest.raises(ValueError, match="cannot share"):
        hla.gated_delta(q, k, v[:, :3].contiguous(), g[:, :3].contiguous(), beta[:, :3].contiguous())
    with pytest.raises(ValueError, match="layout"):
        hla.gated_delta(q, k, v, g, beta, layout="tbhd")
    with pytest.raises(TypeError, match="lengths"):
        hla.gated_delta(q, k, v, g, beta, lengths=torch.tensor([4], device=DEV))
    with pytest.raises(ValueError, match="lengths must be a CUDA"):
        hla.gated_delta(q, k, v, g, beta, lengths=torch.tensor([4], dtype=torch.int32))
    with pytest.raises(ValueError, match="initial_state"):
        hla.gated_delta(q, k, v, g, beta, initial_state=torch.zeros(1, 2, 64, 64, device=DEV))
    with pytest.raises(hla.HLAError, match="WORKSPACE"):
        hla.gated_delta(q, k, v, g, beta, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(hla.HLAError):
        hla.gated_delta(q[..., :48].contiguous(), k[..., :48].contiguous(), v, g, beta)
    odd = torch.zeros(v.numel() + 1, dtype=v.dtype, device=DEV)[1:].view_as(v)
    with pytest.raises(hla.HLAError, match="ALIGN"):
        hla.gated_delta(q, k, odd, g, beta)
    with pytest.raises(hla.HLAError, match="SHAPE"):
        hla.gated_delta(q[:, :, :0], k[:, :, :0], v[:, :, :0], g[:, :, :0], beta[:, :, :0])
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        hla.gated_delta(q.half(), k.half(), v.half(), g, beta)
