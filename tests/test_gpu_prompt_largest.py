"""Counts of tokens, rows and pages near what an int32 holds."""
import pytest
import torch

pytestmark = pytest.mark.gpu
I32 = torch.int32
MOST = 2 ** 31 - 1


@pytest.fixture(scope="module")
def pkg():
    import speculative_decoding_verification_15_gb300 as pkg

    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 60 GB")
    yield pkg
    torch.cuda.empty_cache()


def test_rotary_of_two_billion_tokens(pkg):
    q = torch.ones((MOST, 1, 2), dtype=torch.bfloat16, device="cuda")
    position = torch.zeros(MOST, dtype=I32, device="cuda")
    at = torch.tensor([0, 1, MOST // 2, MOST - 3, MOST - 1], device="cuda")
    position[at] = 1
    freq = torch.full((1,), 3.141592653589793 / 2, dtype=torch.float64, device="cuda")
    pkg.rotary(q, None, position, freq, out_q=q)
    assert torch.equal(q[at].float().round(), torch.tensor([[[-1.0, 1.0]]], device="cuda").expand(5, 1, 2))
    q[at] = 1.0
    assert bool((q == 1).all())


def test_plan_of_two_billion_rows(pkg):
    """Most of them behind the last token, as a padded batch has them."""
    pool = pkg.kv_pool(9)
    table, held = torch.full((2, 4), -1, dtype=I32, device="cuda"), torch.zeros(2, dtype=I32, device="cuda")
    got = pkg.kv_plan(pool, table, held, held.clone(), torch.tensor([20, 30], device="cuda"), 16, MOST)
    assert got["status"].tolist() == [0, 0] and held.tolist() == [2, 2] and int(pool.count) == 5
    assert got["position"][:50].tolist() == [*range(20), *range(30)] and bool((got["position"][50:] == -1).all())
    assert (got["slot"][:50] >= 0).all() and bool((got["slot"][50:] == -1).all())


def test_two_billion_pages_go_back(pkg):
    pages = MOST - 1
    free, count = torch.full((pages,), -7, dtype=I32, device="cuda"), torch.zeros(1, dtype=I32, device="cuda")
    table = torch.arange(pages, dtype=I32, device="cuda")[None]
    held, none = torch.full((1,), pages, dtype=I32, device="cuda"), torch.zeros(1, dtype=I32, device="cuda")
    got = pkg.kv_plan(pkg.PagePool(free, count), table, held, none, none, 16, 0)
    assert got["status"].tolist() == [0] and held.tolist() == [0] and count.tolist() == [pages]
    assert bool((table == -1).all()) and torch.equal(free, torch.arange(pages, dtype=I32, device="cuda"))


@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 30 + 3000, 2 ** 30 + 5000])
def test_windows_of_a_billion_keys(pkg, window):
    """One query over 2^30 + 5000 keys, of which the first 6000 have all the weight."""
    if torch.cuda.mem_get_info()[0] < 80 << 30:
        pytest.skip("needs 70 GB")
    m, D = 2 ** 30 + 5000, 16
    k = torch.full((m, 1, D), -30.0, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros((m, 1, D), dtype=torch.bfloat16, device="cuda")
    k[:6000] = 0.0
    v[:2000], v[2000:6000] = 1.0, 4.0  # 3 on average
    q = torch.ones((1, 1, D), dtype=torch.bfloat16, device="cuda")
    cu = torch.tensor([[0, 1], [0, m]], dtype=I32, device="cuda")
    got = pkg.prompt_attention(q, k, v, cu[0], 1, cu_key=cu[1], window=window)
    want = 4.0 if m - window >= 2000 else 3.0  # 2000 keys, or none, are too far back
    assert got["status"].tolist() == [0] and (got["out"] == want).all()


def test_lengths_past_an_int32(pkg):
    """A request's length must fit; up to that a plan is right, in its last page too."""
    pages, page = 2 ** 24, 128
    pool = pkg.PagePool(torch.arange(pages, 2 * pages, dtype=I32, device="cuda"), torch.full((1,), pages, dtype=I32, device="cuda"))
    table = torch.full((2, pages + 9), -1, dtype=I32, device="cuda")
    table[0, :pages] = torch.arange(pages, dtype=I32, device="cuda")
    held = torch.tensor([pages, 0], dtype=I32, device="cuda")
    keep = torch.tensor([MOST - 3, 0], dtype=I32, device="cuda")
    for new, status in ((3, 0), (4, 2), (MOST, 2)):
        got = pkg.kv_plan(pool, table, held, keep, torch.tensor([new, 0], device="cuda"), page, min(new, 10))
        assert got["status"].tolist() == [status, 2 if new > 10 else 0]  # the second one's row would be past n_out
        assert got["seq_len"].tolist() == [MOST if status == 0 else MOST - 3, 0]
        assert held.tolist() == [pages, 0] and int(pool.count) == pages
        if status == 0:
            assert got["position"].tolist() == [MOST - 3, MOST - 2, MOST - 1]
            assert got["slot"].tolist() == [MOST - 3, MOST - 2, MOST - 1]  # page i is the table's i-th
