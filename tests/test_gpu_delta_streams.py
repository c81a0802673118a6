"""Calls on a stream beside a busy current one: what they allocate is not what queued work still writes."""
import pytest

torch = pytest.importorskip("torch")
import higher_order_linear_chunked_b200 as hla  # noqa: E402
from test_gpu_delta import DEV, leaves  # noqa: E402

pytestmark = pytest.mark.gpu


def test_memory_freed_with_work_queued():
    x = [t.to(DEV) for t in leaves("bf16", 4, 4, 4, 512, 64, 64, seed=1)[:5]]
    want, S = hla.gated_delta(*x, return_state=True)
    grads = hla.gated_delta_backward(*x, x[2])
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        # blocks of the sizes that the calls need, written late and freed at once
        late = [torch.empty_like(t) for t in (want, S, *grads[:5])]
        torch.cuda._sleep(40_000_000)
        for t in late:
            t.fill_(7.0)
        blocks = {t.data_ptr() for t in late}
        del late, t
        o, last = hla.gated_delta(*x, return_state=True, stream=side)
        got = hla.gated_delta_backward(*x, x[2], stream=side)
        assert not blocks & {t.data_ptr() for t in (o, last, *got[:5])}
        torch.cuda.synchronize()
        assert torch.equal(o, want) and torch.equal(last, S)
        assert all(torch.equal(a, b) for a, b in zip(got[:5], grads[:5]))


@pytest.mark.parametrize("op", ["hla2n", "ahla", "hla3"])
def test_memory_freed_with_work_queued_hla(op):
    """The same of the HLA family's calls; a workspace freed while its call is still queued."""
    gen = torch.Generator().manual_seed(3)
    q, k, v = ((torch.randn(2, 4, 1024, 64, generator=gen) / 8).bfloat16().to(DEV) for _ in range(3))
    want = hla.forward(op, q, k, v)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        late = torch.empty_like(want)
        torch.cuda._sleep(40_000_000)
        late.fill_(7.0)
        block = late.data_ptr()
        del late
        side.wait_stream(torch.cuda.current_stream())           # the call is queued, not yet running
        o = hla.forward(op, q, k, v, stream=side)
        assert o.data_ptr() != block
        junk = [torch.full((n,), 255, dtype=torch.uint8, device=DEV) for n in (1 << 16, 1 << 20, 1 << 22, 1 << 24)]
        torch.cuda.synchronize()
        assert torch.equal(o, want)
        del junk
