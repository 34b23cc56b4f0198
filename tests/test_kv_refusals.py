"""What the package's cache calls refuse before they reach the C entries."""
import pytest
import torch

import speculative_decoding_verification_15_gb300 as pkg
from speculative_decoding_verification_15_gb300 import binding


@pytest.fixture(scope="module")
def tensors():
    c = pkg.kv_cache(4, 2, 64, 64, device="cpu")
    i = torch.zeros(2, dtype=torch.int32)
    return c, torch.zeros(1, 4, 64), i[:1].view(1, 1), i[:1], i


@pytest.mark.parametrize("value", [1 << 31, 1 << 32, (1 << 32) + 5, -(1 << 31) - 1, -(1 << 32)])
def test_counts_past_32_bits(tensors, value):
    """Cut to 32 bits, a window of 2^32 would be none at all, and one of 2^32 + 5 five."""
    c, q, table, one, cu = tensors
    for name, at in (("max_query", 5), ("window", 7), ("sinks", 8)):
        args = [q, c, table, one, cu, 1, 0.1, 0, 0, q, None, one, torch.zeros(1, dtype=torch.uint8)]
        args[at] = value
        with pytest.raises(ValueError, match=name):
            binding.spec_cache_attention(*args)
    kv = q[:, :2]
    with pytest.raises(ValueError, match="max_new"):
        binding.spec_kv_append(c, kv, kv, table, one, cu, value, one)


def test_tensors_that_are_not_on_a_gpu(tensors):
    """All three calls refuse them alike."""
    c, q, table, one, cu = tensors
    kv = q[:, :2]
    for call in (lambda: pkg.kv_append(c, kv, kv, table, one, cu, 1), lambda: pkg.kv_gather(c, table, cu, 1),
                 lambda: pkg.cache_attention(q, c, table, one, cu, 1)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
