"""A caller's workspace that the library's calls cannot use is refused, on tensors without memory (no GPU)."""
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import higher_order_linear_chunked_b200 as hla


def fake(*shape, dtype=torch.float32, device="cuda:0"):
    return torch.empty(*shape, dtype=dtype, device=device)


@pytest.mark.parametrize("name", ["hla2", "hla2_normalized", "ahla", "hla3", "hla2_unmasked", "hla2_backward", "ahla_backward",
                                  "state", "forward_profiled"])
def test_workspace_of_another_kind(name):
    n = 1 << 24
    with FakeTensorMode():
        x = [fake(1, 2, 8, 64) for _ in range(3)]
        more = {"hla2_backward": [x[2]], "ahla_backward": [x[2]], "forward_profiled": [()]}.get(name, [])
        first = {"state": ["hla2"], "forward_profiled": ["hla2"]}.get(name, [])
        for ws, what in ((fake(n, dtype=torch.uint8, device="cpu"), "workspace must be a CUDA tensor"),
                         (fake(n, dtype=torch.uint8, device="cuda:1"), "workspace is on cuda:1"),
                         (fake(1, dtype=torch.uint8).expand(n), "workspace must be contiguous")):
            with pytest.raises(ValueError, match=what):
                getattr(hla, name)(*first, *x, *more, workspace=ws)
