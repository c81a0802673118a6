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
