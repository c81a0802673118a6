"""What the Python calls over include/hla_delta.h check and allocate, on tensors without memory (no GPU)."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import higher_order_linear_chunked_b200 as hla


def fake(*shape, dtype=torch.float32, device="cuda:0"):
    return torch.empty(*shape, dtype=dtype, device=device)


def delta_leaves():
    return [fake(1, 2, 8, 64, dtype=torch.bfloat16) for _ in range(3)] + [fake(1, 2, 8) for _ in range(2)]


def calls():
    x = delta_leaves()
    y, w = fake(4, 64), fake(64)
    return {"gated_delta": lambda ws: hla.gated_delta(*x, workspace=ws),
            "gated_delta_backward": lambda ws: hla.gated_delta_backward(*x, x[2], workspace=ws),
            "group_norm_backward": lambda ws: hla.group_norm_backward(y, y, 2, weight=w, workspace=ws)}


@pytest.mark.parametrize("name", ["gated_delta", "gated_delta_backward", "group_norm_backward"])
def test_workspace_of_another_kind(name):
    n = 1 << 24
    with FakeTensorMode():
        call = calls()[name]
        for ws, what in ((fake(n, dtype=torch.uint8, device="cpu"), "workspace must be a CUDA tensor"),
                         (fake(n, dtype=torch.uint8, device="cuda:1"), "workspace is on cuda:1"),
                         (fake(1, dtype=torch.uint8).expand(n), "workspace must be contiguous"),
                         (fake(2 * n, dtype=torch.uint8)[::2], "workspace must be contiguous")):
            with pytest.raises(ValueError, match=what):
                call(ws)
