"""GPU tests of appends into pages whose present scale, left by another writer, is not a
power of two: every code is the nearest one to the exact quotient, rounded once."""
import numpy as np
import pytest
import torch

import kv_util as U

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _run(x, k, v, cached):
    import speculative_decoding_verification_15_gb300 as pkg

    c = x.cache()
    st = pkg.kv_append(c, k, v, x.i32(x.table), x.i32(cached), x.i32(x.cu), int(x.new.max()))["status"]
    assert (st == 0).all()
    grown = 0
    for codes, scale, c0, s0, new in ((c.k, c.k_scale, x.kc, x.ks, k), (c.v, c.v_scale, x.vc, x.vs, v)):
        want_c, want_s = U.append(c0, s0, new.double().cpu().numpy(), x.table, cached, x.cu)
        np.testing.assert_array_equal(scale.double().cpu().numpy(), want_s)
        np.testing.assert_array_equal(U.codes_of(codes), want_c)
        grown += int((want_s > s0).sum())
    return grown


def _any_scales(x, g, lo, hi):
    for name in ("ks", "vs"):
        s = getattr(x, name)
        setattr(x, name, np.float32(2.0 ** g.uniform(lo, hi, s.shape)).astype(np.float64))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("size", [1e-4, 1.0, 1e4])  # of the new entries: no page's scale grows, some do, all do
def test_random_entries(dtype, size):
    new, cached = [7, 3, 50, 1, 20], np.array([5, 30, 13, 63, 1])
    x = U.Inputs(80, cached + new, new, 2, 2, 128, 64, dtype)
    _any_scales(x, np.random.default_rng(80), -9, -3)
    grown = _run(x, x.k_new * size, x.v_new * size, cached)
    assert (grown > 0) if size > 1e-4 else True


@pytest.mark.parametrize("power", [-99.5, -60.0, -39.5, 0.0, 60.0, 118.0])
def test_entries_next_to_ties(power):
    """Entries that are a scale times the midpoint of two codes, rounded to fp32, and the
    numbers beside them: the exact quotient is on one side of the tie, or on it."""
    g = np.random.default_rng(81)
    cached, new = np.array([3, 9, 14]), np.array([29, 23, 18])
    x = U.Inputs(81, cached + new, new, 2, 2, 64, 32, F32)
    _any_scales(x, g, power, power + 0.9)
    finite = np.sort(U.VALUE[:127])
    ties = (finite[1:] + finite[:-1]) / 2
    ties = np.concatenate([ties[ties < 200], finite[finite < 200]])  # below where the scale would grow

    def entries(scale):
        out = np.zeros((int(x.cu[-1]), 2, 64), np.float32)
        for b in range(3):
            rows = slice(x.cu[b], x.cu[b + 1])
            s = scale[x.table[b, 0]]  # each request lies in its first page
            t = np.float32(g.choice(ties, (new[b], 2, 64)) * s[None, :, None])
            t = np.where(g.random(t.shape) < 0.3, np.nextafter(t, np.float32(np.inf)), t)
            t = np.where(g.random(t.shape) < 0.3, np.nextafter(t, np.float32(0)), t)
            out[rows] = t * g.choice(np.float32([-1, 1]), t.shape)
        return x.tensor(out)

    _run(x, entries(x.ks), entries(x.vs), cached)


def test_kept_codes_of_any_scale_are_rounded_once():
    """The page's scale grows by every ratio of 1 to 2^12: kept codes times it."""
    g = np.random.default_rng(82)
    B = 60
    cached, new = np.full(B, 15), np.full(B, 1)
    x = U.Inputs(82, cached + new, new, 1, 1, 256, 16, F32)
    _any_scales(x, g, -12, 0)
    x.kc, x.vc = g.integers(0, 256, x.kc.shape).astype(np.uint8), g.integers(0, 256, x.vc.shape).astype(np.uint8)
    x.kc[(x.kc & 127) == 127] = 126
    x.vc[(x.vc & 127) == 127] = 254
    # scales whose product with a code is a tie but for their last bits
    x.ks[::2] = np.float32((1 + 2.0 ** -4 * g.integers(1, 16, x.ks[::2].shape)) * 2.0 ** -7 * (1 + 2.0 ** -22)).astype(np.float64)
    assert _run(x, x.k_new * 448, x.v_new * 448, cached) > B
