"""The int8 layers at the ends of their range, against values that do not come from
the kernels."""

import pytest
import torch

from test_gpu_int8 import _ops, dev  # noqa: F401

pytestmark = pytest.mark.gpu


def test_outputs_of_an_empty_k_past_32_bits(dev):
    """An empty sum, alone and with its tail, of 2^32 + 2^16 elements."""
    m, n = 2 ** 16 + 1, 2 ** 16
    x = torch.zeros(m, 0, dtype=torch.bfloat16, device=dev)
    cache = torch.empty(0, dtype=torch.uint8, device=dev)
    y = torch.full((m, n), 7.0, device=dev)
    assert not _ops().linear_int8(x, cache, n, out=y).any()
    bias = torch.arange(n, dtype=torch.float32, device=dev)
    row = torch.arange(m, dtype=torch.float32, device=dev)[:, None]
    y.copy_(row.expand(m, n))
    _ops().linear_int8_epilogue(x, cache, n, bias, y, out=y)   # sums below 2^18: exact
    for i in range(0, m, 8192):
        assert torch.equal(y[i:i + 8192], row[i:i + 8192] + bias)
    del y
    y = _ops().linear_int8_epilogue_bf16(x, cache, n, bias)
    for i in range(0, m, 8192):
        assert torch.equal(y[i:i + 8192], bias.to(torch.bfloat16).expand_as(y[i:i + 8192]))
