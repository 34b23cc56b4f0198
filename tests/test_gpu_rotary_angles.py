"""How near the angles of rotary positions are."""
import numpy as np
import pytest
import torch

import prompt_util as U

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import speculative_decoding_verification_15_gb300 as pkg

    return pkg


@pytest.mark.parametrize("T", [200, 20000])
def test_angles_near_half_turns(pkg, T):
    """x = 1, y = 0 gives the sine itself.  Near a half turn it is below a quarter, so that its own
    rounding is 2^-26 at most (one unit in the last place, in [1/8, 1/4)).  The phase is off by
    2^-32 turns and, as a float of at most an eighth of a turn, by 2^-28 turns: 2 pi (2^-32 + 2^-28)
    is less than 0.42 2^-24.  In all less than 0.7 2^-24."""
    g = np.random.default_rng(1)
    pos = g.integers(1, 2 ** 31 - 1, T).astype(np.int32)
    freq = np.array(0.5 + 3 * g.random(32))
    turns = pos.astype(np.longdouble)[:, None] * (freq.astype(np.longdouble) / (2 * U.PI))
    sine = np.sin(((turns - np.rint(turns)) * 2 * U.PI).astype(np.float64))
    near = (np.abs(sine) < 0.25) & (np.abs(turns - np.rint(turns)) > 0.25)
    assert near.sum() > T
    x = torch.zeros(T, 1, 64, device="cuda")
    x[..., :32] = 1.0
    got = pkg.rotary(x, None, torch.from_numpy(pos).cuda(), torch.from_numpy(freq).cuda())["q"]
    err = np.abs(got[:, 0, 32:].double().cpu().numpy() - sine)[near]
    assert (err <= 0.7 * U.U32).all(), float(err.max() / U.U32)
