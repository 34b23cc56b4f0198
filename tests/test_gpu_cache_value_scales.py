"""GPU tests of the attention over the 8-bit cache where the pages' value scales lie far
apart, against 64-bit results with a bound that knows what each row sees: neither a page
that a row does not see, nor an improbable one, may cost the others' probabilities their
bits."""
import numpy as np
import pytest
import torch

import kv_util as U

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
TILE = 128


def expected(x, scale, window=0, sinks=0):
    """out, lse and their error bounds in 64 bits (u = 2^-24).

    Scores: D products summed in fp32 and a few roundings, 2 (D + 8) u of the row's
    largest sum of magnitudes; log2 of a value's scale joins them, below 256, so 512 u
    more.  bf16 queries are off by 2^-16 of the row's largest entry.  A probability times
    its value's scale, z, is off by 2^-8 of z or, where that is more, by 2^-17 of the
    largest z among the tokens of the tile that the row sees.  Sums of n tokens in fp32:
    (n + 32) u.  The output's rounding: 2^-9 of it (fp32: 4 u), and 2^-126."""
    u, bf16 = 2.0 ** -24, x.dtype == BF16
    q, (T, Hq, D), H = x.q64(), tuple(x.q.shape), x.kc.shape[1]
    G, bs = Hq // H, x.page
    out, lse = np.zeros((T, Hq, D)), np.full((T, Hq), -np.inf)
    tol, tol_lse = np.full((T, Hq, D), 2.0 ** -126), np.zeros((T, Hq))
    for b, length in enumerate(x.lens):
        n = int(x.cu[b + 1] - x.cu[b])
        for t in range(n):
            P, row = int(length) - n + t, int(x.cu[b]) + t
            j = np.arange(P + 1)
            if window:
                j = j[(j > P - window) | (j < sinks)]
            K, page = U.read(x.kc, x.ks, x.table[b], j), x.table[b][j // bs]
            code, vs = U.VALUE[x.vc[page, :, j % bs]], x.vs[page]
            for h in range(H):
                r = slice(h * G, (h + 1) * G)
                s = q[row, r] @ K[:, h].T * scale
                m = s.max(1, keepdims=True)
                p = np.exp(s - m)
                l = p.sum(1, keepdims=True)
                z = p * vs[:, h]
                out[row, r], lse[row, r] = z @ code[:, h] / l, (m + np.log(l))[:, 0]
                dx = 2 * (D + 8) * u * (np.abs(q[row, r]) @ np.abs(K[:, h]).T * scale).max(1, keepdims=True) + 512 * u
                if bf16:
                    dx = dx + 2.0 ** -16 * np.abs(q[row, r]).max(1, keepdims=True) * np.abs(K[:, h]).sum(1).max() * scale
                rel = 2 * dx + (j.size + 32) * u
                A = z @ np.abs(code[:, h]) / l
                tol[row, r] += A * (rel + (2.0 ** -8 if bf16 else 0)) + (2.0 ** -9 if bf16 else 4 * u) * np.abs(out[row, r])
                tol_lse[row, r] = (dx + (j.size + 32) * u + 4 * u * np.abs(m + np.log(l)))[:, 0]
                if bf16:
                    for tile in np.unique(j // TILE):
                        w = j // TILE == tile
                        tol[row, r] += z[:, w].max(1, keepdims=True) * 2.0 ** -17 / l * np.abs(code[w, h]).sum(0)
    return out, lse, tol, tol_lse


def check(x, scale=None, window=0, sinks=0):
    import speculative_decoding_verification_15_gb300 as pkg

    scale = x.q.shape[2] ** -0.5 if scale is None else scale
    got = pkg.cache_attention(x.q, x.cache(), x.i32(x.table), x.i32(x.lens), x.i32(x.cu), int(x.new.max()), scale=scale,
                              window=window, sinks=sinks, want_lse=True)
    assert (got["status"] == 0).all()
    out, lse, tol, tol_lse = expected(x, scale, window, sinks)
    g, gl = got["out"].double().cpu().numpy(), got["lse"].double().cpu().numpy()
    assert np.isfinite(g).all()
    assert (np.abs(g - out) <= tol).all(), (np.abs(g - out) / tol).max()
    assert (np.abs(gl - lse) <= tol_lse).all()
    return got


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("power", [4, 8, 12, 15, 16, 17, 20, 40, 90])
def test_a_later_drafts_page_has_larger_values(dtype, power):
    """Six drafts whose last two open a page with values 2^power above the others': the
    earlier rows do not see that page, and the later ones do."""
    x = U.Inputs(50, [98], [6], 8, 2, 64, 16, dtype)
    x.vs[:] = 2.0 ** -6 * 2.0 ** (np.arange(x.vs.size).reshape(x.vs.shape) % 2)
    x.vs[x.table[0, 6]] = 2.0 ** (power - 6)
    check(x)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("power", [8, 14, 18, 30, 100])
def test_an_improbable_page_has_larger_values(dtype, power):
    """Every row sees a page with values 2^power above the others', with scores so low
    that it adds nothing of weight, or something."""
    x = U.Inputs(51, [100, 270], [3, 2], 4, 2, 64, 16, dtype)
    x.vs[:] = 2.0 ** -7
    q = x.q64()
    for b in range(2):
        page = x.table[b, 3]
        x.vs[page] = 2.0 ** (power - 7)
        for h in range(2):
            x.ks[page, h] = 2.0 ** -4
            x.kc[page, h] = U.encode(-np.sign(q[x.cu[b], 2 * h]) * (20.0 + 10.0 * b))
    check(x)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("power", [10, 20, 60])
def test_a_page_that_has_left_the_window(dtype, power):
    """Rows whose windows start within a tile, behind a page of large values that the
    first rows still see."""
    x = U.Inputs(52, [400, 150], [8, 8], 6, 3, 128, 16, dtype)
    x.vs[:] = 2.0 ** -8
    for b, length in enumerate((400, 150)):
        x.vs[x.table[b, (length - 8 - 60) // 16]] = 2.0 ** (power - 8)
    check(x, window=62, sinks=3)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("zero", [2.0 ** -100, 2.0 ** -30])
@pytest.mark.parametrize("other", [2.0 ** -5, 1.0, 2.0 ** 100])
def test_pages_of_zeros(dtype, zero, other):
    """Pages of zeros, whose scale an append leaves at 2^-100, with most of the weight:
    the weights count, and the small contributions of the other pages keep their bits."""
    x = U.Inputs(53, [200, 61], [4, 1], 4, 1, 64, 16, dtype)
    x.vs[:] = other
    q = x.q64()
    for b in range(2):
        for i in (0, 2):
            page = x.table[b, i]
            x.vs[page], x.vc[page] = zero, 0
            x.ks[page] = 2.0 ** -4
            x.kc[page] = U.encode(np.sign(q[x.cu[b], 0]) * 3.0)
    check(x)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scales_wander_over_a_long_context(dtype):
    """Near and far tiles in turn, an item cut over many CTAs, references that move: the
    scales drift over 2^160 along the context, and so do the scores."""
    x = U.Inputs(54, [9000], [3], 4, 1, 64, 32, dtype)
    g = np.random.default_rng(54)
    i = np.arange(x.table.shape[1])
    x.vs[x.table[0], 0] = 2.0 ** np.round(80 * np.sin(i / 40.0) + g.integers(-9, 10, i.size))
    x.ks[x.table[0], 0] = 2.0 ** (-8 + np.round(3 * np.cos(i / 17.0)))
    check(x)
    x.vs[x.table[0], 0] = x.vs[x.table[0][::-1], 0].copy()
    check(x, window=5000, sinks=40)


@pytest.mark.parametrize("Hq", [1, 4, 8])  # row tiles of 16, 32 and 64
@pytest.mark.parametrize("page", [16, 128])
def test_every_row_tile(Hq, page):
    """Drafts of large values in every shape of row tile, whole items and cut ones."""
    g = np.random.default_rng(55)
    lens = np.array([130, 700, 8, 515, 64, 129])
    x = U.Inputs(55, lens, np.full(6, 8), Hq, 1, 128, page, BF16)
    x.vs[:] = 2.0 ** g.integers(-9, 12, x.vs.shape)
    for b, length in enumerate(lens):
        x.vs[x.table[b, (length - 1) // page]] = 2.0 ** 20
    check(x)
    check(x, window=100, sinks=2)


def test_an_unseen_pages_scale_changes_no_more_than_rounding():
    """The same request with a later draft's page at 2^-6 and at 2^30: the rows before it
    agree to a step of bf16."""
    x = U.Inputs(56, [98], [6], 8, 2, 64, 16, BF16)
    x.vs[:] = 2.0 ** -6
    a = check(x)["out"][:4].double()
    x.vs[x.table[0, 6]] = 2.0 ** 30
    b = check(x)["out"][:4].double()
    assert ((a - b).abs() <= 2.0 ** -7 * a.abs() + 2.0 ** -12 * a.abs().max()).all()
