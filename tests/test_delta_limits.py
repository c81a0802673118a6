"""The largest sizes that include/hla_delta.h names: counts of chunks and blocks stay in range (no GPU)."""
import pytest

import higher_order_linear_chunked_b200 as hla
from higher_order_linear_chunked_b200 import delta


@pytest.mark.parametrize("dtype", [hla.HLA_F32, hla.HLA_BF16])
def test_longest_sequence(dtype):
    lib, most = delta._library(), 2 ** 31 - 64
    for size, launches, token in ((lib.hla_delta_workspace_bytes, lib.hla_delta_kernel_launches, 200),
                                  (lib.hla_delta_backward_workspace_bytes, lib.hla_delta_backward_kernel_launches, 800)):
        assert size(dtype, 1, 1, 1, most, 32, 32) > token * most and launches(dtype, 1, 1, 1, most, 32, 32) > 0
        for T in (most + 1, 2 ** 31 - 31, 2 ** 31 - 1):
            assert size(dtype, 1, 1, 1, T, 32, 32) == 0 and launches(dtype, 1, 1, 1, T, 32, 32) == 0
