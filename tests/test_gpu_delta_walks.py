"""The gradients' two walks side by side and one after the other: the rule's three ranges of heads, the same
bits from repeated calls and from a graph, and the 64-bit gradients."""
import pytest

torch = pytest.importorskip("torch")
import higher_order_linear_chunked_b200 as hla  # noqa: E402
from test_gpu_delta import DEV  # noqa: E402
from test_gpu_delta_backward import compare, inputs  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H", [74, 75, 148, 149])     # 148, 150, 296, 298 blocks of 32 columns a walk
def test_ranges_of_heads(H):
    x, dout, dstate = inputs("bf16", 1, H, H, 70, 64, 64, seed=H)
    compare(x, dout, dstate, 0.2)
    dev = [t.to(DEV) for t in (*x[:5], dout, x[5], dstate)]
    call = lambda: hla.gated_delta_backward(*dev[:6], scale=0.2, initial_state=dev[6], dstate=dev[7])  # noqa: E731
    want = call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for _ in range(3):
        for t in got:
            t.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
