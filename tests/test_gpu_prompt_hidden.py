"""Values that are not finite in rows that a query does not see: results and statuses stay as
they are, whatever the length; those that it sees join its sums."""
import numpy as np
import pytest
import torch

import prompt_util as U

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def pkg():
    import speculative_decoding_verification_15_gb300 as pkg

    return pkg


def tensors(seed, n, m, Hq, H, D, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randn((t, h, D), generator=g, device="cuda").to(dtype) for t, h in ((n, Hq), (m, H), (m, H))]


def offsets(*lengths):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(lengths)]).astype(np.int32)).cuda()


def last_rows(q, k, v, n, m, rows, dtype, **mask):
    """The oracle's answer for the last `rows` of the first n queries over the first m keys."""
    a, b, c = (t.double().cpu().numpy() for t in (q[n - rows:n], k[:m], v[:m]))
    return U.attention(a, b, c, [0, rows], [0, m], q.shape[2] ** -0.5, bf16=dtype == BF16, **mask)


def near(got, want, tol):
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), (float(np.nanmax(err - tol)), np.argwhere(~(err <= tol))[:3])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,H,old", [(64, 2, 0), (128, 2, 0), (256, 1, 0), (192, 1, 0), (128, 2, 3000)])
def test_values_behind_a_long_prompt(pkg, D, H, old, dtype):
    """Padding rows behind the last request, and the next request's values, are not finite."""
    n = 2500 - old // 2 if old else 3050
    q, k, v = tensors(D + old, n + 20, n + old + 60, 2 * H, H, D, dtype)
    m = n + old
    want, lse, tol, tol_lse = last_rows(q, k, v, n, m, 130, dtype)
    v[m:m + 20] = NAN
    v[m + 20:] = INF
    k[m + 30:] = NAN
    got = pkg.prompt_attention(q, k, v, offsets(n, 20), n, cu_key=offsets(m, 20), want_lse=True)
    near(got["out"][n - 130:n], want, tol)
    near(got["lse"][n - 130:n], lse, tol_lse)
    assert got["out"][:n].isfinite().all() and got["status"].tolist() == [0, 0]
    assert got["out"][n:].isnan().all()  # every row of the second one sees its first value


def test_values_behind_hundreds_of_thousands_of_keys(pkg):
    """The rows that share a tile with the padding cost no more than others: no wait runs out."""
    n, m, D = 40000, 399940, 16
    q, k, v = tensors(1, n, m + 50, 2, 2, D, BF16)
    want, _, tol, _ = last_rows(q, k, v, n, m, 40, BF16)
    v[m:] = NAN
    got = pkg.prompt_attention(q, k, v, offsets(n), n, cu_key=offsets(m))
    assert got["status"].tolist() == [0]
    assert got["out"].isfinite().all()
    near(got["out"][n - 40:], want, tol)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 0), (140, 5), (260, 150)])
@pytest.mark.parametrize("new,total,Hq,H,D", [([500], [500], 6, 2, 64), ([333, 200], [400, 200], 4, 1, 128),
                                              ([300, 70], [300, 500], 4, 2, 256), ([150], [400], 3, 3, 80),
                                              ([90], [4000], 4, 2, 64), ([60], [3500], 2, 1, 192)])
def test_which_columns_are_not_finite(pkg, new, total, Hq, H, D, window, sinks, dtype):
    """Infinities of both signs and NaN in single columns, all over the keys: an output is
    infinite or NaN just where the formula's is, and as near to it as ever elsewhere."""
    g = np.random.default_rng(D + window)
    q, k, v = tensors(D + sinks, sum(new), sum(total), Hq, H, D, dtype)
    q *= 0.25  # no weight underflows
    cu_q, cu_k = offsets(*new), offsets(*total)
    cq, ck = cu_q.cpu().numpy(), cu_k.cpu().numpy()
    clean = [t.double().cpu().numpy() for t in (q, k, v)]
    scale = D ** -0.5
    mask = dict(window=window, sinks=sinks)
    for value in (INF, -INF, NAN):
        at = g.integers(0, sum(total), 14), g.integers(0, H, 14), g.integers(0, D, 14)
        v[at] = torch.tensor(value, device="cuda").to(dtype)
    got = pkg.prompt_attention(q, k, v, cu_q, max(new), cu_key=cu_k, want_lse=True, **mask)
    assert (got["status"] == 0).all()
    x = v.double().cpu().numpy()
    # the finite part, and for each class how many of its values a row sees
    clean[2] = np.where(np.isfinite(x), x, 0.0)
    want, lse, tol, tol_lse = U.attention(*clean, cq, ck, scale, bf16=dtype == BF16, **mask)
    zero = [np.zeros_like(clean[0]), np.zeros_like(clean[1])]
    seen = [U.attention(*zero, kind.astype(np.float64), cq, ck, scale, **mask)[0] > 0
            for kind in (x == INF, x == -INF, np.isnan(x))]
    up, down, nan = seen
    nan = nan | (up & down)
    out = got["out"].double().cpu().numpy()
    np.testing.assert_array_equal(np.isnan(out), nan)
    np.testing.assert_array_equal(out == INF, up & ~nan)
    np.testing.assert_array_equal(out == -INF, down & ~nan)
    fine = ~(up | down | nan)
    assert fine.any() and (~fine).any()
    assert (np.abs(out - want)[fine] <= tol[fine]).all()
    near(got["lse"], lse, tol_lse)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 256])
def test_nothing_but_nan(pkg, D, dtype):
    """Values that are all NaN, in prompts and in a chunk over many keys."""
    q, k, v = tensors(3, 2100, 5300, 4, 2, D, dtype)
    v[:] = NAN
    for new, total in (((2000, 100), (2000, 100)), ((100, 200), (5000, 300))):
        got = pkg.prompt_attention(q, k, v, offsets(*new), max(new), cu_key=offsets(*total))
        assert (got["status"] == 0).all() and got["out"][:sum(new)].isnan().all()


def test_many_items_of_one_sm(pkg):
    """Thousands of short requests of many heads, every other one's first value not finite: the
    others, which share their tiles, are what they are without."""
    g = torch.Generator().manual_seed(4)
    new = torch.randint(1, 4, (6000,), generator=g)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), new.cumsum(0)])
    n = int(cu[-1])
    q, k, v = tensors(5, n, n, 32, 32, 16, BF16)
    want = pkg.prompt_attention(q, k, v, cu, 3)["out"]
    odd = torch.arange(6000) % 2 == 1
    v[cu[:-1][odd].cuda()] = NAN
    got = pkg.prompt_attention(q, k, v, cu, 3)
    assert (got["status"] == 0).all()
    rows = odd.repeat_interleave(new).cuda()
    assert got["out"][rows].isnan().all() and torch.equal(got["out"][~rows], want[~rows])
