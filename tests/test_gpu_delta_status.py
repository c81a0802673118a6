"""The device status word of a gated delta call's workspace: cleared by the call, as in the library's other calls."""
import pytest

torch = pytest.importorskip("torch")
import higher_order_linear_chunked_b200 as hla  # noqa: E402
from test_gpu_delta import DEV, leaves  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("H,T,lengths", [(2, 70, None), (2, 70, [0]), (1, 4096, None)])
def test_status_is_cleared(dtype, H, T, lengths):
    x = [t.to(DEV) for t in leaves("bf16" if dtype == torch.bfloat16 else "f32", 1, H, H, T, 64, 64, seed=1)[:5]]
    n = torch.tensor(lengths, dtype=torch.int32, device=DEV) if lengths else None
    for size in (hla.gated_delta_workspace_bytes, hla.gated_delta_backward_workspace_bytes):
        ws = torch.full((size(dtype, 1, H, H, T, 64, 64),), 0x55, dtype=torch.uint8, device=DEV)
        if size is hla.gated_delta_workspace_bytes:
            hla.gated_delta(*x, lengths=n, workspace=ws)
        else:
            hla.gated_delta_backward(*x, torch.ones_like(x[2]), lengths=n, workspace=ws)
        assert hla.read_device_status(ws) == 0
