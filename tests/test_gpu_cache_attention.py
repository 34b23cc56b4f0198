"""GPU tests of the attention over the 8-bit paged cache against the 64-bit oracle, with
the error bound that kv_util.attention derives element by element."""
import numpy as np
import pytest
import torch

import kv_util as U

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _run(x, cache=None, scale=None, window=0, sinks=0, table=None, seq_len=None, max_query=None, **kw):
    import speculative_decoding_verification_15_gb300 as pkg

    n = x.cu[1:] - x.cu[:-1]
    out = pkg.cache_attention(x.q, cache or x.cache(), x.i32(x.table if table is None else table),
                              x.i32(x.lens if seq_len is None else seq_len), x.i32(x.cu),
                              int(n.max(initial=0)) if max_query is None else max_query, scale=scale, window=window,
                              sinks=sinks, want_lse=True, **kw)
    torch.cuda.synchronize()
    return out


def _check(x, got, scale=None, window=0, sinks=0, only=None, **kw):
    D = x.q.shape[2]
    out, lse, tol, tol_lse = U.attention(x.q64(), x.kc, x.vc, x.ks, x.vs, x.table, x.lens, x.cu,
                                         D ** -0.5 if scale is None else scale, window, sinks, bf16=x.dtype == BF16, **kw)
    g, gl = got["out"].double().cpu().numpy(), got["lse"].double().cpu().numpy()
    rows = slice(None) if only is None else only
    np.testing.assert_array_equal(np.isnan(g[rows]), np.isnan(out[rows]))
    err = np.abs(g - out)[rows]
    assert (np.nan_to_num(err) <= np.nan_to_num(tol[rows])).all(), np.nanmax(err / np.maximum(tol[rows], 1e-30))
    empty = np.isneginf(lse[rows])
    assert (np.isneginf(gl[rows]) == empty).all()
    fine = np.isfinite(lse[rows])
    assert (np.abs(gl - lse)[rows][fine] <= tol_lse[rows][fine]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,page,Hq,Hkv", [(128, 64, 8, 2), (64, 16, 4, 4), (80, 32, 6, 2), (16, 128, 5, 1),
                                           (96, 64, 16, 1), (256, 64, 4, 2), (192, 16, 3, 1), (128, 128, 20, 2)])
def test_matches_oracle(dtype, D, page, Hq, Hkv):
    """Ragged lengths and verify widths, page and tile edges among them."""
    lens = [1, 127, 128, 129, 300, 8, 511, 640, 17]
    new = [1, 8, 1, 3, 5, 8, 0, 2, 4]
    x = U.Inputs(10, lens, new, Hq, Hkv, D, page, dtype)
    out = _run(x)
    assert (out["status"] == 0).all()
    _check(x, out)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (5, 4), (128, 0), (130, 129), (200, 300), (1000, 4),
                                          (2 ** 31 - 1, 2 ** 31 - 1)])
def test_window_and_sinks(dtype, window, sinks):
    lens, new = [700, 129, 40, 1000, 3], [8, 4, 8, 1, 3]
    x = U.Inputs(11, lens, new, 4, 2, 64, 32, dtype)
    out = _run(x, window=window, sinks=sinks)
    assert (out["status"] == 0).all()
    _check(x, out, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_queries_that_see_nothing(dtype):
    """An empty cache, and more queries than cached tokens: zeros and -inf."""
    x = U.Inputs(12, [0, 3, 5, 0], [2, 8, 5, 0], 6, 3, 128, 16, dtype)
    out = _run(x)
    assert (out["status"] == 0).all()
    _check(x, out)
    assert (out["out"][:7] == 0).all() and torch.isneginf(out["lse"][:7]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_unseen_entries_never_matter(dtype):
    """NaN codes after the last token, NaN codes and missing pages before the window,
    NaN among the drafts that earlier queries do not see."""
    lens, new, window, sinks = [200, 150, 517], [4, 8, 2], 64, 5
    x = U.Inputs(13, lens, new, 8, 2, 128, 16, dtype)
    clean = (x.kc.copy(), x.vc.copy(), x.table.copy())
    for b, n in enumerate(lens):
        last = x.table[b, (n - 1) // 16]
        x.kc[last, :, (n - 1) % 16 + 1:] = 127
        x.vc[last, :, (n - 1) % 16 + 1:] = 255
        low = n - new[b] - window + 1
        for j in range(sinks, low):
            page = x.table[b, j // 16]
            if j // 16 > 0 and j // 16 < low // 16:
                x.table[b, j // 16] = -7
            else:
                x.kc[page, :, j % 16] = 255
                x.vc[page, :, j % 16] = 127
    out = _run(x, window=window, sinks=sinks)
    assert (out["status"] == 0).all()
    x.kc, x.vc, x.table = clean
    _check(x, out, window=window, sinks=sinks)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("which", ["kc", "vc"])
def test_nan_reaches_only_the_queries_that_see_it(dtype, which):
    """A NaN code at the third draft's position: the anchor and two drafts stay finite,
    the later ones are NaN (in the channels that hold it at least)."""
    x = U.Inputs(14, [135, 260], [6, 5], 8, 2, 64, 64, dtype)
    pos = 135 - 6 + 3
    page = x.table[0, pos // 64]
    getattr(x, which)[page, 0, pos % 64, 7] = 127
    out = _run(x)
    hit = np.zeros((11, 8), bool)
    hit[3:6, :4] = True  # the queries of key head 0 from that position on
    g = out["out"].double().cpu().numpy()
    assert np.isnan(g[hit][:, 7]).all()
    bad = getattr(x, which)
    bad[page, 0, pos % 64, 7] = 0
    ref, _, tol, _ = U.attention(x.q64(), x.kc, x.vc, x.ks, x.vs, x.table, x.lens, x.cu, 64 ** -0.5,
                                 bf16=dtype == BF16)
    assert (np.abs(g - ref)[~hit] <= tol[~hit]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_nan_deep_in_the_context(dtype):
    """A NaN value code that every query sees: that channel is NaN in all of them, and
    the other key head's results are untouched."""
    x = U.Inputs(15, [400], [3], 4, 2, 64, 32, dtype)
    x.vc[x.table[0, 1], 1, 3, 20] = 127
    g = _run(x)["out"].double().cpu().numpy()
    assert np.isnan(g[:, 2:, 20]).all() and np.isfinite(g[:, :2]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_layouts(dtype):
    """Queries sliced from a fused projection, token-major pages, shared pages."""
    x = U.Inputs(16, [333, 333, 64], [5, 2, 1], 6, 2, 128, 64, dtype, token_major=True, fused=True)
    x.table[1, :5] = x.table[0, :5]  # a shared prefix
    assert not x.q.is_contiguous()
    _check(x, _run(x))


@pytest.mark.parametrize("dtype,L,n,Hq", [(BF16, 50021, 1, 2), (BF16, 70001, 8, 4), (F32, 20011, 2, 2)])
def test_long_contexts(dtype, L, n, Hq):
    """One long request, cut across every SM; results repeat bit for bit."""
    x = U.Inputs(17, [L], [n], Hq, 1, 64, 128, dtype)
    c = x.cache()
    a, b = _run(x, c), _run(x, c)
    assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])
    _check(x, a)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_sink_token_takes_most_of_the_mass(dtype):
    """One token far above a long flat tail, as trained models' first tokens are: the
    tail's small probabilities must still add up."""
    x = U.Inputs(18, [6000], [2], 4, 1, 64, 64, dtype)
    x.kc[:] = U.encode(U.VALUE[x.kc] / 64)
    q = x.q64()
    x.kc[x.table[0, 0], 0, 0] = U.encode(np.sign(q[:, :].sum((0, 1))) * 300)
    x.ks[:] = 2.0 ** -5
    _check(x, _run(x))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_many_small_requests(dtype):
    g = np.random.default_rng(19)
    new = g.integers(0, 9, 400)
    lens = new + g.integers(0, 150, 400)
    x = U.Inputs(19, lens, new, 4, 2, 64, 16, dtype)
    out = _run(x)
    assert (out["status"] == 0).all()
    _check(x, out)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_wide_queries(dtype):
    """More rows than one row tile holds: a prompt's chunk of 150 tokens."""
    x = U.Inputs(20, [400, 150], [150, 33], 6, 2, 64, 64, dtype)
    _check(x, _run(x))
    _check(x, _run(x, window=70, sinks=3), window=70, sinks=3)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scales_far_apart(dtype):
    """Pages of one tile whose scales differ by many powers of two, large scores."""
    x = U.Inputs(21, [250, 90], [4, 2], 4, 2, 128, 16, dtype)
    g = np.random.default_rng(21)
    x.vs[:] = 2.0 ** g.integers(-30, 10, x.vs.shape)
    x.ks[:] = 2.0 ** g.integers(-12, -4, x.ks.shape)
    x.vs[x.table[0, 2]] = 2.0 ** -100  # a page of nothing but zeros
    x.vc[x.table[0, 2]] = 0
    _check(x, _run(x, scale=0.9), scale=0.9)


def test_statuses():
    x = U.Inputs(22, [100, 100, 100, 100, 20], [2, 2, 2, 2, 2], 4, 2, 64, 16, BF16)
    table, lens = x.table.copy(), x.lens.copy()
    table[1, 3] = 10 ** 6
    lens[2] = -1
    lens[3] = 16 * table.shape[1] + 1
    out = _run(x, table=table, seq_len=lens)
    assert out["status"].tolist() == [0, 6, 2, 2, 0]
    _check(x, out, only=np.r_[0:2, 8:10])
    out = _run(x, max_query=1)
    assert (out["status"] == 2).all()
    x.cu = np.array([0, 2, 1, 6, 8, 11], np.int32)
    assert _run(x, max_query=5)["status"].tolist() == [0, 2, 0, 0, 2]


def test_other_stream_and_graph():
    """A call on another stream, and one captured in a CUDA graph and replayed on new
    queries and a longer cache."""
    import speculative_decoding_verification_15_gb300 as pkg

    x = U.Inputs(23, [300, 40], [4, 4], 8, 2, 128, 64, BF16)
    c = x.cache()
    want = _run(x, c)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = _run(x, c, stream=s)
    assert torch.equal(want["out"], got["out"])
    q, seq = x.q.clone(), x.i32([200, 30])
    args = (q, c, x.i32(x.table), seq, x.i32(x.cu), 4)
    with torch.cuda.stream(s):
        pkg.cache_attention(*args)
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            out = pkg.cache_attention(*args)
    q.copy_(x.q)
    seq.copy_(x.i32(x.lens))
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out["out"], want["out"])


def test_pages_past_4_gib():
    import speculative_decoding_verification_15_gb300 as pkg

    x = U.Inputs(24, [260], [3], 4, 2, 128, 128, BF16)
    P = (5 << 30) // (2 * 128 * 128)
    k, v = (torch.empty((P, 2, 128, 128), dtype=torch.uint8, device="cuda") for _ in "kv")
    at = torch.tensor([P - 1, P - 40000, P - 2], device="cuda")
    held = x.table[0, :3]
    k[at], v[at] = x.tensor(x.kc[held]), x.tensor(x.vc[held])
    ks, vs = torch.ones((P, 2), device="cuda"), torch.ones((P, 2), device="cuda")
    ks[at], vs[at] = x.tensor(x.ks[held].astype(np.float32)), x.tensor(x.vs[held].astype(np.float32))
    c = pkg.KVCache(k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn), ks, vs)
    out = _run(x, c, table=at.cpu().numpy()[None])
    _check(x, out)


@pytest.mark.parametrize("Hq,Hkv,n", [(8, 2, 8), (2, 2, 8), (16, 2, 8)])
def test_many_tiles_a_cta(Hq, Hkv, n):
    """Enough tiles for every CTA to hold several items and cut two: row tiles of 16, 32
    and 64 rows."""
    lens = 700 + (np.arange(60) * 97) % 900
    x = U.Inputs(25, lens, np.full(60, n), Hq, Hkv, 64, 64, BF16)
    c = x.cache()
    a, b = _run(x, c), _run(x, c)
    assert torch.equal(a["out"], b["out"])
    _check(x, a)
    w = _run(x, c, window=300, sinks=20)
    _check(x, w, window=300, sinks=20)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_queries_at_any_element(dtype):
    """Query rows that are not 16-byte aligned."""
    x = U.Inputs(26, [90, 300], [3, 4], 6, 2, 80, 32, dtype)
    flat = torch.empty(7 * 491 + 1, dtype=dtype, device="cuda")
    q = flat[1:].view(7, 491)[:, :480].view(7, 6, 80)
    q.copy_(x.q)
    x.q = q
    _check(x, _run(x))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_any_scales(dtype):
    """Scales that are not powers of two, as another writer of the cache may have left."""
    x = U.Inputs(27, [400, 77], [2, 5], 8, 2, 128, 16, dtype)
    g = np.random.default_rng(27)
    x.ks = np.float32(x.ks * g.uniform(0.6, 1.7, x.ks.shape)).astype(np.float64)
    x.vs = np.float32(x.vs * g.uniform(0.6, 1.7, x.vs.shape)).astype(np.float64)
    _check(x, _run(x))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_bad_query_stays_in_its_row(dtype, bad):
    x = U.Inputs(28, [300], [5], 8, 2, 64, 64, dtype)
    clean = x.q64()
    x.q = x.q.clone()
    x.q[2, 3, 9] = bad
    g = _run(x)["out"].double().cpu().numpy()
    assert np.isnan(g[2, 3]).all()
    ref, _, tol, _ = U.attention(clean, x.kc, x.vc, x.ks, x.vs, x.table, x.lens, x.cu, 64 ** -0.5, bf16=dtype == BF16)
    keep = np.ones(g.shape[:2], bool)
    keep[2, 3] = False
    assert (np.abs(g - ref)[keep] <= tol[keep]).all()


def test_large_and_small_query_rows_together():
    """Rows of one row tile whose magnitudes differ by 2^40: each keeps its own scale."""
    x = U.Inputs(29, [200], [4], 8, 1, 128, 64, BF16)
    x.q = (x.q.float() * (2.0 ** torch.arange(-20, 12, device="cuda").float()).view(4, 8, 1)).to(BF16)
    x.q[0, 0] = 0
    _check(x, _run(x))


def test_more_requests_than_threads():
    g = np.random.default_rng(30)
    new = g.integers(0, 3, 5000)
    lens = new + g.integers(0, 20, 5000)
    x = U.Inputs(30, lens, new, 2, 1, 16, 16, BF16)
    out = _run(x)
    assert (out["status"] == 0).all()
    _check(x, out)


@pytest.mark.parametrize("group,page", [(1, 16), (1, 64), (4, 32), (8, 16)])  # 6, 6, 24 and 48 rows
@pytest.mark.parametrize("batch", [30, 75, 151, 153])  # 60 to 306 items of 2 heads, on 304 CTAs of 152 SMs
def test_few_items_and_some_more(batch, group, page):
    """Items as many as the CTAs, somewhat fewer and more: whole CTAs an item, or the line."""
    g = np.random.default_rng(31 + batch)
    new = g.integers(0, 7, batch)
    lens = new + np.where(g.random(batch) < 0.2, g.integers(0, 3000, batch), g.integers(300, 900, batch))
    lens[:2] = new[:2]
    x = U.Inputs(32, lens, new, 2 * group, 2, 32, page, BF16)
    _check(x, _run(x))
    _check(x, _run(x, window=260, sinks=5), window=260, sinks=5)


@pytest.mark.parametrize("long", [3000, 20000])
def test_one_long_item_among_short_ones(long):
    """A fair share of the tiles that one item passes by far, the others by far below it."""
    x = U.Inputs(33, [long] + [40] * 60 + [long // 2], [3] * 62, 8, 4, 64, 16, BF16)
    _check(x, _run(x))
