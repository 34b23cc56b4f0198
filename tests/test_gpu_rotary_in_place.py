"""Long prompts rotated in place."""
import pytest
import torch

from test_gpu_rotary import BF16, F32, check, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import speculative_decoding_verification_15_gb300 as pkg

    return pkg


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,rot", [(3001, 6, 2, 64, 64), (2500, 40, 8, 128, 128), (2600, 12, 4, 256, 96),
                                           (2700, 100, 4, 128, 64), (2450, 3, 1, 80, 48)])
def test_long_prompts_in_place(pkg, T, Hq, Hk, D, rot, adjacent, dtype):
    """In place on slices of a fused product, with copies of later tokens under way: one share of
    a token a warp or several.  What lies beside the slices stays."""
    _, _, pos = inputs(5, T, 1, 1, 16, dtype, 2, 30000)
    g = torch.Generator(device="cuda").manual_seed(D)
    wide = torch.randn((T, Hq + 2 * Hk, D), generator=g, device="cuda").to(dtype)
    before = wide.clone()
    q, k = wide[:, :Hq], wide[:, Hq:Hq + Hk]
    freq, axis = pkg.rotary_frequencies(rot, sections=(rot // 8, rot // 2 - rot // 8))
    got = pkg.rotary(q, k, torch.from_numpy(pos).cuda(), freq, axis, adjacent, out_q=q, out_k=k)
    assert got["q"] is q and got["k"] is k
    apart = pkg.rotary(before[:, :Hq].contiguous(), before[:, Hq:Hq + Hk].contiguous(), torch.from_numpy(pos).cuda(), freq, axis, adjacent)
    assert torch.equal(q, apart["q"]) and torch.equal(k, apart["k"])
    assert torch.equal(wide[:, Hq + Hk:], before[:, Hq + Hk:])
    some = slice(T // 2, T // 2 + 40)
    check(q[some], before[some, :Hq], pos[:, some], freq, axis, adjacent)
    check(k[some], before[some, Hq:Hq + Hk], pos[:, some], freq, axis, adjacent)
