"""Statuses of thousands of prompts, some of whose offsets are wrong."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("B", [1, 383, 385, 5000])
def test_wrong_offsets_among_many(B, dtype):
    import speculative_decoding_verification_15_gb300 as pkg

    g = np.random.default_rng(B)
    cu = np.cumsum(np.concatenate([[0], g.integers(0, 4, B)])).astype(np.int32)
    n = int(cu[-1]) + 1
    wrong = g.integers(1, B + 1, B // 7)
    cu[wrong] = np.where(g.random(len(wrong)) < 0.5, -1, n + 5)
    q = torch.randn((n, 2, 16), device="cuda").to(dtype)
    status = pkg.prompt_attention(q, q[:, :1], q[:, 1:], cu_query=torch.from_numpy(cu).cuda(), max_query=3)["status"]
    bad = (cu[:-1] < 0) | (cu[1:] < cu[:-1]) | (cu[1:] > n) | (cu[1:] - cu[:-1] > 3)
    np.testing.assert_array_equal(status.cpu().numpy(), np.where(bad, 2, 0))
