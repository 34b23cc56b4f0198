"""Rotary positions whose rows are one and the same, or overlap."""
import pytest
import torch

from test_gpu_rotary import BF16, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import speculative_decoding_verification_15_gb300 as pkg

    return pkg


@pytest.mark.parametrize("T", [1, 50, 3000])
@pytest.mark.parametrize("kind", [torch.int32, torch.int64])
def test_expanded_positions(pkg, T, kind):
    """One row of positions for every axis, as a prompt of text has them, without a copy of it;
    and rows that overlap otherwise."""
    q, k, pos = inputs(9, T, 4, 2, 64, BF16, 1, 9999)
    freq, axis = pkg.rotary_frequencies(64, sections=(16, 8, 8))
    one = torch.from_numpy(pos[0]).cuda().to(kind)
    want = pkg.rotary(q, k, one, freq)
    got = pkg.rotary(q, k, one[None].expand(3, -1), freq, axis)
    assert torch.equal(got["q"], want["q"]) and torch.equal(got["k"], want["k"])
    long = torch.arange(2 * T + 8, device="cuda").to(kind)
    slid = torch.as_strided(long, (3, T), (1, 1))
    assert torch.equal(pkg.rotary(q, None, slid, freq, axis)["q"], pkg.rotary(q, None, slid.contiguous(), freq, axis)["q"])


@pytest.mark.parametrize("T", [3, 3000])
def test_no_pairs_and_several_axes(pkg, T):
    """Nothing rotates: what comes in is copied."""
    q, k, pos = inputs(10, T, 3, 1, 32, BF16, 2, 99)
    freq, axis = pkg.rotary_frequencies(0, sections=(0, 0))
    got = pkg.rotary(q, k, torch.from_numpy(pos).cuda(), freq, axis)
    assert torch.equal(got["q"], q) and torch.equal(got["k"], k)
