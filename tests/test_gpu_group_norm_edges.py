"""Group norm on the GPU where eps or the activation's argument is at its edge (oracle/delta.py in 64 bits)."""
import pytest

torch = pytest.importorskip("torch")
import higher_order_linear_chunked_b200 as hla  # noqa: E402
from higher_order_linear_chunked_b200 import delta  # noqa: E402
from oracle import delta as od  # noqa: E402
from test_gpu_group_norm import DEV, DT, check, inputs  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gated", [True, False])
@pytest.mark.parametrize("activation", ["none", "silu"])
@pytest.mark.parametrize("center", [True, False])
def test_no_eps(dtype, gated, activation, center):
    """eps = 0 over more rows than the gradient kernel walks at once, and not a multiple of them.
    Tolerances as in test_gpu_group_norm.py: the sums' terms are |dz n| and |dz|."""
    rows, groups, width = 1000, 64, 32
    x, dy, gate, w, b = inputs(dtype, rows, groups, width, gated, True, 17)
    C = groups * width
    slots = delta._library().hla_group_norm_backward_workspace_bytes(hla.HLA_BF16 if dtype == "bf16" else hla.HLA_F32, rows,
                                                                     C, groups) // (8 * C)
    assert rows > slots and rows % slots
    how = dict(eps=0.0, activation=activation, center=center)
    dev = [t.to(DEV) if t is not None else None for t in (x, dy, w, b, gate)]
    got = hla.group_norm_backward(dev[0], dev[1], groups, *dev[2:], **how)
    want = od.group_norm_backward(x, dy, groups, w, b, gate, **how)
    size = dy.double().abs() * (gate.double().abs().clamp(min=1.0) if gated else 2.0)
    n = od.group_norm(x, groups, eps=0.0, center=center).abs()
    check(got[2], want[2], 2.4e-5 * (size * n).sum(0), "dweight")
    check(got[3], want[3], 2.4e-5 * size.sum(0), "dbias")
    xg = x.double().reshape(rows, groups, width)
    xg = xg - xg.mean(-1, keepdim=True) if center else xg
    r = 1 / torch.sqrt((xg * xg).mean(-1, keepdim=True))
    check(got[0], want[0], 2e-5 * float((r * (size * w.double().abs()).reshape(xg.shape)).max()), "dx")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_activation_in_a_weight_gradient(dtype):
    """One row of pairs (1, -1): n is 1 and -1, so that dweight, fp32 for either type, is +-silu(gate).
    Relative room: rsqrt and exp 2^-22 each, six roundings of 2^-24."""
    gate = torch.linspace(-80, 20, 4096).to(DT[dtype])[None]
    x = torch.tensor([1.0, -1.0]).repeat(2048).to(DT[dtype])[None]
    w = torch.ones(4096)
    how = dict(eps=0.0, activation="silu", center=False)
    dw = hla.group_norm_backward(x.to(DEV), torch.ones_like(x).to(DEV), 2048, weight=w.to(DEV), gate=gate.to(DEV), **how)[2]
    want = od.group_norm_backward(x, torch.ones_like(x), 2048, w, None, gate, **how)[2]
    off = ((dw.cpu().double() - want).abs() / want.abs().clamp(min=1e-300))[gate[0] != 0]
    assert float(off.max()) <= 14 * 2.0 ** -24


def test_many_channels():
    """2^30 channels, whose two column sums together are more than an int counts: without weight, gate and
    activation the gradient of the bias is dy, and each group's dx sums to nothing."""
    C = 1 << 30
    x = torch.ones(1, C, dtype=torch.bfloat16, device=DEV)
    x[0, ::2] = -1.0
    dy = torch.ones_like(x)
    dy[0, ::3] = 2.0
    dx, _, dw, db = hla.group_norm_backward(x, dy, C // 64, bias=torch.zeros(C, device=DEV))
    assert dw is None
    for lo in range(0, C, 1 << 27):
        hi = lo + (1 << 27)
        assert torch.equal(db[lo:hi], dy[0, lo:hi].float())
    last = od.group_norm_backward(x[:, -64:].cpu(), dy[:, -64:].cpu(), 1)[0]
    check(dx[:, -64:], last, 1e-5, "dx")
    del x, dy, dx, db
    torch.cuda.empty_cache()
