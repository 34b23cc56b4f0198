"""Prompt attention against 64-bit formulas."""
import numpy as np
import pytest
import torch

import prompt_util as U

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def pkg():
    import speculative_decoding_verification_15_gb300 as pkg

    return pkg


class Inputs:
    """Packed queries, keys and values of requests with n new of m tokens, and `behind` rows
    after the last one."""

    def __init__(self, seed, new, total, Hq, H, D, dtype, behind=0, spread=1.0):
        g = np.random.default_rng(seed)
        self.cu_q = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.cu_k = np.concatenate([[0], np.cumsum(total)]).astype(np.int32)
        T, L = int(self.cu_q[-1]) + behind, int(self.cu_k[-1]) + behind

        def tensor(*shape, scale=1.0):
            return torch.from_numpy(g.normal(size=shape) * scale).to(dtype).cuda()

        self.q = tensor(T, Hq, D, scale=spread)
        self.k = tensor(L, H, D)
        self.v = tensor(L, H, D)
        self.max_new, self.dtype = int(max(new, default=0)), dtype

    def want(self, scale=None, window=0, sinks=0):
        q, k, v = (t.double().cpu().numpy() for t in (self.q, self.k, self.v))
        scale = self.q.shape[2] ** -0.5 if scale is None else scale
        return U.attention(q, k, v, self.cu_q, self.cu_k, scale, window, sinks, self.dtype == BF16)

    def call(self, pkg, same=False, **kw):
        cu = dict(cu_key=torch.from_numpy(self.cu_k).cuda()) if not same else {}
        return pkg.prompt_attention(self.q, self.k, self.v, torch.from_numpy(self.cu_q).cuda(), self.max_new, **cu, **kw)


def close(got, want, rows=None):
    out, lse, tol, tol_lse = want
    n = out.shape[0] if rows is None else rows
    g = got["out"].double().cpu().numpy()[:n]
    err = np.abs(g - out[:n])
    assert (err <= tol[:n]).all(), (float((err - tol[:n]).max()), np.argwhere(~(err <= tol[:n]))[:3])
    if got["lse"] is not None:
        gl = got["lse"].double().cpu().numpy()[:n]
        seen = lse[:n] > -np.inf
        assert (gl[~seen] == -np.inf).all()
        assert (np.abs(gl[seen] - lse[:n][seen]) <= tol_lse[:n][seen]).all()
    assert (got["status"] == 0).all()


SHAPES = [  # queries, of tokens, query heads, key heads, head_dim
    ([1], [1], 1, 1, 16), ([1], [700], 8, 2, 128), ([300], [300], 4, 4, 64), ([129, 1, 64, 257], None, 8, 2, 128),
    ([5, 0, 33, 128, 0], None, 6, 2, 96), ([40, 200], [333, 200], 10, 2, 80), ([70, 8], [70, 400], 7, 1, 112),
    ([64, 65], [64, 900], 3, 1, 48), ([17, 100], None, 8, 1, 256), ([90], [150], 4, 2, 192), ([30, 31], None, 5, 5, 144),
    ([3, 9], None, 130, 1, 32), ([513], None, 2, 1, 128), ([20], None, 128, 1, 64)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new,total,Hq,H,D", SHAPES)
def test_against_64_bits(pkg, new, total, Hq, H, D, dtype):
    x = Inputs(len(new) + D, new, total or new, Hq, H, D, dtype)
    close(x.call(pkg, same=total is None, want_lse=True), x.want())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (50, 0), (64, 5), (200, 40), (128, 300), (1000, 4), (1 << 30, 0)])
@pytest.mark.parametrize("new,total,Hq,H,D", [([400, 90], None, 6, 2, 64), ([200, 33], [700, 300], 4, 1, 128)])
def test_windows(pkg, new, total, Hq, H, D, window, sinks, dtype):
    x = Inputs(window + sinks, new, total or new, Hq, H, D, dtype)
    close(x.call(pkg, want_lse=True, window=window, sinks=sinks), x.want(window=window, sinks=sinks))


@pytest.mark.parametrize("new,total,Hq,H,D", [([33, 5, 0, 100], [5000, 40, 700, 7000], 4, 2, 128), ([70], [4000], 6, 2, 64),
                                              ([1, 2], [9000, 3000], 8, 1, 256), ([40], [2600], 3, 3, 16)])
@pytest.mark.parametrize("window,sinks", [(0, 0), (2500, 300)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_few_queries_over_many_keys(pkg, new, total, Hq, H, D, window, sinks, dtype):
    """Items whose tiles are cut into parts, some of them without a tile."""
    x = Inputs(D, new, total, Hq, H, D, dtype)
    L, code = int(x.cu_k[-1]), int(dtype == F32)
    assert pkg.spec_prompt_attention_workspace_size(int(x.cu_q[-1]), L, len(new), Hq, H, D, code, window, sinks) > 0
    close(x.call(pkg, want_lse=True, window=window, sinks=sinks), x.want(window=window, sinks=sinks))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_parts_with_spoilt_keys(pkg, dtype):
    """A NaN value behind a row, in the tile that it shares with the row's own last key."""
    x = Inputs(31, [60], [5000], 4, 2, 64, dtype)
    want = x.want()
    x.v[4970] = float("nan")
    x.k[4990] = float("nan")
    got = x.call(pkg, want_lse=True)
    out, lse, tol, tol_lse = want
    g, gl = got["out"].double().cpu().numpy(), got["lse"].double().cpu().numpy()
    assert (np.abs(g[:30] - out[:30]) <= tol[:30]).all() and (np.abs(gl[:50] - lse[:50]) <= tol_lse[:50]).all()
    assert np.isnan(g[30:]).all() and np.isnan(gl[50:]).all()


@pytest.mark.parametrize("total", [300, 6000])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_visible_nan_of_no_weight(pkg, total, dtype):
    """Its weight underflows, in its tile or as a whole part's: NaN all the same."""
    x = Inputs(32, [40], [total], 4, 2, 64, dtype)
    x.q[:] = 8.0
    x.k[:total // 2] = -100.0
    x.k[total // 2:] = 0.0
    x.v[10, 0, 5] = float("nan")
    got = x.call(pkg)["out"]
    bad = torch.zeros_like(got, dtype=torch.bool)
    bad[:, :2, 5] = True
    assert torch.equal(torch.isnan(got), bad)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_queries_that_see_nothing(pkg, D, dtype):
    """More queries than keys: the first ones come before every key."""
    x = Inputs(3, [300, 5, 7], [100, 0, 7], 4, 2, D, dtype)
    got = x.call(pkg, want_lse=True)
    close(got, x.want())
    blind = torch.ones(312, dtype=torch.bool, device="cuda")
    blind[200:300] = blind[305:] = False
    assert (got["out"][blind] == 0).all() and (got["lse"][blind] == float("-inf")).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_what_a_query_does_not_see_never_matters(pkg, value, D, dtype):
    """Keys and values behind a row, outside its window, in other requests and in rows that
    belong to none are NaN or infinite; rows that see them are the same as ever, or not finite."""
    x = Inputs(5, [150, 60, 200], [150, 200, 200], 4, 2, D, dtype, behind=9)
    want = x.want(window=70, sinks=3)
    spoilt = [100, 149, 150 + 30, 350 + 77, 350 + 199, 550, 558]
    for t in (x.k, x.v):
        t[spoilt] = value
    x.q[410:] = value
    got = x.call(pkg, want_lse=True, window=70, sinks=3)
    out, lse, tol, tol_lse = want
    g, gl = got["out"].double().cpu().numpy(), got["lse"].double().cpu().numpy()
    sees = np.zeros(g.shape[0], dtype=bool)
    for b in range(3):
        for t in range(x.cu_q[b], x.cu_q[b + 1]):
            P = (x.cu_k[b + 1] - x.cu_k[b]) - (x.cu_q[b + 1] - x.cu_q[b]) + t - x.cu_q[b]
            for s in spoilt:
                j = s - x.cu_k[b]
                sees[t] |= 0 <= j <= P and s < x.cu_k[b + 1] and (j > P - 70 or j < 3)
    ok = ~sees
    ok[410:] = False
    assert ok[:410].sum() > 100
    assert (np.abs(g[ok] - out[ok]) <= tol[ok]).all() and (np.abs(gl[ok] - lse[ok]) <= tol_lse[ok]).all()
    if np.isnan(value):
        assert np.isnan(g[sees]).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_of_no_request_stay(pkg, dtype):
    """Rows before the first offset and behind the last one are not written, nor are those of
    a request whose offsets are wrong."""
    from speculative_decoding_verification_15_gb300 import binding

    g = np.random.default_rng(6)
    q = torch.from_numpy(g.normal(size=(400, 4, 64))).to(dtype).cuda()
    kv = torch.from_numpy(g.normal(size=(400, 2, 64))).to(dtype).cuda()
    cu = np.array([10, 130, 120, 300, 401, 350, 360], np.int32)  # 1: backwards; 3 past the rows; 4 from there
    out = torch.full_like(q, 7.0)
    lse = torch.full((400, 4), 7.0, device="cuda")
    status = torch.empty(6, dtype=torch.int32, device="cuda")
    dcu = torch.from_numpy(cu).cuda()
    binding.spec_prompt_attention(q, kv, kv, dcu, 180, None, 0.125, 0, 0, out, lse, status)
    assert status.tolist() == [0, 2, 0, 2, 2, 0]
    written = torch.zeros(400, dtype=torch.bool, device="cuda")
    written[10:300] = written[350:360] = True
    assert (out[~written] == 7).all() and (lse[~written] == 7).all()
    q64, kv64 = q.double().cpu().numpy(), kv.double().cpu().numpy()
    for a, b in ((120, 300), (350, 360)):  # 10 .. 120 is request 0's too; 120 .. 130 both's
        c = np.array([a, b])
        want, _, tol, _ = U.attention(q64, kv64, kv64, c, c, 0.125, bf16=dtype == BF16)
        rows = slice(130 if a == 120 else a, b)
        assert (np.abs(out.double().cpu().numpy() - want) <= tol)[rows].all()
    binding.spec_prompt_attention(q, kv, kv, dcu[:2].contiguous(), 100, None, 0.125, 0, 0, out, lse, status[:1])
    assert status[0] == 2  # 120 rows, at most 100 told


@pytest.mark.parametrize("D", [64, 128, 192])
def test_slices_of_a_fused_product(pkg, D):
    """Queries, keys and values as slices, and the same from memory that no tensor map takes."""
    new, Hq, H = [200, 77], 6, 2
    x = Inputs(9, new, new, Hq, H, D, BF16)
    want = x.want()
    wide = torch.cat([x.q, x.k, x.v], 1)
    x.q, x.k, x.v = wide[:, :Hq], wide[:, Hq:Hq + H], wide[:, Hq + H:]
    close(x.call(pkg), want)

    def strided(t, offset):
        n, h, d = t.shape
        s = torch.as_strided(torch.zeros(n * (h * d + 1) + 8, dtype=BF16, device="cuda"), (n, h, d), (h * d + 1, d, 1), offset)
        s.copy_(t)
        return s

    x.q, x.k, x.v = strided(x.q, 1), strided(x.k, 0), strided(x.v, 3)
    close(x.call(pkg), want)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("spread,scale", [(60.0, None), (1.0, 1e-6), (30.0, 2.0)])
def test_steep_and_flat_scores(pkg, spread, scale, dtype):
    """Scores far above the exponential's range, rising and falling along the keys, and scores
    that are nearly equal."""
    x = Inputs(12, [300], [600], 4, 2, 128, dtype, spread=spread)
    x.k *= torch.linspace(0.01, 1.5, 600, device="cuda").to(dtype)[:, None, None]
    close(x.call(pkg, want_lse=True, scale=scale), x.want(scale=scale))


def test_many_short_prompts(pkg):
    new = (np.arange(1500) * 7 % 11).tolist()
    x = Inputs(13, new, new, 2, 1, 64, BF16)
    close(x.call(pkg, same=True), x.want())


def test_no_prompts(pkg):
    x = Inputs(14, [], [], 2, 1, 64, BF16)
    assert x.call(pkg)["out"].shape == (0, 2, 64)
    x = Inputs(15, [0, 0], [0, 5], 2, 1, 64, BF16)
    assert x.call(pkg)["status"].tolist() == [0, 0]


@pytest.mark.parametrize("D", [128, 256])
def test_captured_and_on_another_stream(pkg, D):
    """Two captured calls and eager ones between them, on streams of their own, agree bit for
    bit: nothing is shared and sums have a fixed order."""
    x, y = Inputs(16, [333, 40], [900, 4000], 8, 2, D, BF16), Inputs(17, [50], [7000], 8, 1, D, BF16)
    first, second = (z.call(pkg, want_lse=True) for z in (x, y))
    cu = [(torch.from_numpy(z.cu_q).cuda(), torch.from_numpy(z.cu_k).cuda()) for z in (x, y)]
    graphs, got = [], []
    torch.cuda.synchronize()
    for z, (a, b) in zip((x, y), cu):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            got.append(pkg.prompt_attention(z.q, z.k, z.v, a, z.max_new, cu_key=b, want_lse=True))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        eager = y.call(pkg, want_lse=True)
    torch.cuda.synchronize()
    for a, b in ((first, got[0]), (second, got[1]), (second, eager)):
        assert torch.equal(a["out"], b["out"]) and torch.equal(a["lse"], b["lse"])


def test_same_as_the_cache_attention_reads(pkg):
    """Over keys and values that the 8-bit cache holds exactly, both attentions agree."""
    D, H, page = 64, 2, 16
    x = Inputs(18, [100, 37], [100, 237], 4, H, D, BF16)
    x.k, x.v = (t.to(torch.float8_e4m3fn).to(BF16) for t in (x.k, x.v))
    cache = pkg.kv_cache(40, H, page, D)
    pool, table = pkg.kv_pool(40), torch.full((2, 20), -1, dtype=torch.int32, device="cuda")
    held, none = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")
    lens = torch.tensor([100, 237], dtype=torch.int32, device="cuda")
    plan = pkg.kv_plan(pool, table, held, none, lens, page, 337)
    assert (pkg.kv_append(cache, x.k, x.v, table, none, plan["cu_new"], 237)["status"] == 0).all()
    a = x.call(pkg)["out"]
    b = pkg.cache_attention(x.q, cache, table, plan["seq_len"], torch.from_numpy(x.cu_q).cuda(), 100)["out"]
    want = x.want()
    close(dict(out=a, lse=None, status=plan["status"]), want)
    err = (a.double() - b.double()).abs().cpu().numpy()
    # each within its own bound of the formula: the cache's kernel adds at most 2^-16 of a
    # query's largest entry (under a quarter of this bound here) and small terms of 2^-17
    assert (err <= 3 * want[2]).all()
