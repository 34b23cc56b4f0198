"""Rotary positions with frequencies that are none, and with huge ones."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import prompt_util as U
from test_gpu_rotary import BF16, F32, check, inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import speculative_decoding_verification_15_gb300 as pkg

    return pkg


# tokens, head_dim, pairs: a few tokens, many, and columns that no vector covers
FORMS = [(40, 64, 32), (3000, 64, 32), (40, 36, 17)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,D,pairs", FORMS)
@pytest.mark.parametrize("adjacent", [False, True])
def test_frequencies_that_are_none(pkg, T, D, pairs, adjacent, dtype):
    """A pair whose frequency is NaN, infinite or 2^64 and more is NaN; the others turn as ever."""
    q, k, pos = inputs(T, T, 4, 2, D, dtype, 1, 5000)
    freq = torch.from_numpy(1e4 ** -(np.arange(pairs) / pairs)).cuda()
    bad = {0: float("nan"), 3: float("inf"), 4: -float("inf"), 9: 1e300, 12: -2.0 ** 64, 16: 2.0 ** 117}
    for i, f in bad.items():
        freq[i] = f
    got = pkg.rotary(q, k, torch.from_numpy(pos[0]).cuda(), freq, adjacent=adjacent)
    spoilt = torch.zeros(D, dtype=torch.bool, device="cuda")
    for i in bad:
        spoilt[[2 * i, 2 * i + 1] if adjacent else [i, i + pairs]] = True
    clean = torch.where(freq.isfinite() & (freq.abs() < 2.0 ** 64), freq, 0.0)
    for name, x in (("q", q), ("k", k)):
        assert got[name][..., spoilt].isnan().all() and not got[name][..., ~spoilt].isnan().any()
        check(torch.where(spoilt, x, got[name]), x, pos, clean, None, adjacent)  # a frequency of 0 leaves x


@pytest.mark.parametrize("T", [40, 3000])
def test_huge_frequencies(pkg, T):
    """Below 2^64 the angle is right at every position, by whole numbers."""
    q, _, pos = inputs(2, T, 1, 1, 64, F32, 1, 2 ** 31 - 1)
    freq = np.array([1.5 * 2.0 ** 63, -2.0 ** 60 - 2.0 ** 9, 1e18, 12345678912345.678] * 8)
    two_pi = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899862803482534")
    got = pkg.rotary(q, None, torch.from_numpy(pos[0]).cuda(), torch.from_numpy(freq).cuda())["q"].double().cpu().numpy()
    turn = np.array([[float((int(p) * Fraction(f) / two_pi) % 1) for f in freq[:4]] for p in pos[0]]) * 2 * np.pi
    turn = np.tile(turn, (1, 8))[:, None, :]
    x = q.double().cpu().numpy()
    a, b = x[..., :32], x[..., 32:]
    want = np.concatenate([a * np.cos(turn) - b * np.sin(turn), b * np.cos(turn) + a * np.sin(turn)], -1)
    tol = 10 * U.U32 * np.tile(np.abs(a) + np.abs(b), 2) + U.U32 * np.abs(want)
    assert (np.abs(got - want) <= tol).all()
