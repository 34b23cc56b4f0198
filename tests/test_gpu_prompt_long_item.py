"""A request over hundreds of millions of keys: a CTA works on it for seconds, and its other
requests wait that long without a failure."""
import pytest
import torch

pytestmark = pytest.mark.gpu
BF16 = torch.bfloat16


def test_one_long_request_before_hundreds_of_short_ones():
    import speculative_decoding_verification_15_gb300 as pkg

    B, m, D = 700, 400_000_000, 16  # more requests than are put in order of length: the long one comes first
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 52 GB")
    k = torch.full((m + B - 1, 1, D), -30.0, dtype=BF16, device="cuda")
    v = torch.full((m + B - 1, 1, D), 3.0, dtype=BF16, device="cuda")
    k[m - 1024:] = 0.0  # the last keys have all the weight
    v[m - 512:m] = 5.0
    short = torch.randn((B - 1, 1, D), device="cuda").to(BF16)
    v[m:] = short
    q = torch.ones((B, 1, D), dtype=BF16, device="cuda")
    cu_q = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    cu_k = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), m + cu_q[:B]])
    got = pkg.prompt_attention(q, k, v, cu_q, 1, cu_key=cu_k)
    assert (got["status"] == 0).all()
    assert (got["out"][0] == 4.0).all() and torch.equal(got["out"][1:], short)


def test_hundreds_of_millions_of_queries_without_keys():
    """Seconds without a tile to copy are no failure either: every head of every request gets 0."""
    import speculative_decoding_verification_15_gb300 as pkg

    B, H, D = 8192, 65535, 16
    if torch.cuda.mem_get_info()[0] < 48 << 30:
        pytest.skip("needs 40 GB")
    q = torch.ones((B, H, D), dtype=BF16, device="cuda")
    kv = torch.ones((1, H, D), dtype=BF16, device="cuda")
    cu_k = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    got = pkg.prompt_attention(q, kv, kv, torch.arange(B + 1, dtype=torch.int32, device="cuda"), 1, cu_key=cu_k)
    assert (got["status"] == 0).all()
    assert not bool(got["out"].view(torch.int32).any())
