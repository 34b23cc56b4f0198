"""GPU tests of the 8-bit paged cache's append and gather against the 64-bit oracle:
codes, scales and read-back values are equal, not close."""
import numpy as np
import pytest
import torch

import kv_util as U

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def _append(x, cache, k, v, cached, max_new=None, **kw):
    import speculative_decoding_verification_15_gb300 as pkg

    n = x.cu[1:] - x.cu[:-1]
    out = pkg.kv_append(cache, k, v, x.i32(x.table), x.i32(cached), x.i32(x.cu),
                        int(n.max(initial=0)) if max_new is None else max_new, **kw)
    torch.cuda.synchronize()
    return out["status"].cpu().numpy()


def _check(x, cache, k, v, cached):
    for codes, scale, c0, s0, new in ((cache.k, cache.k_scale, x.kc, x.ks, k), (cache.v, cache.v_scale, x.vc, x.vs, v)):
        want_c, want_s = U.append(c0, s0, new.double().cpu().numpy(), x.table, cached, x.cu)
        np.testing.assert_array_equal(scale.double().cpu().numpy(), want_s)
        np.testing.assert_array_equal(U.codes_of(codes), want_c)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("page,D,H", [(16, 64, 1), (32, 80, 3), (64, 128, 2), (128, 256, 2), (16, 16, 5)])
def test_append_matches_oracle(dtype, page, D, H):
    new = [1, 8, 0, 3, page, page + 1, 2 * page + 5, 1]
    cached = np.array([0, 5, page, page - 1, page, 1, page - 2, 3 * page - 1])
    x = U.Inputs(1, cached + new, new, H, H, D, page, dtype)
    c = x.cache()
    assert (_append(x, c, x.k_new, x.v_new, cached) == 0).all()
    _check(x, c, x.k_new, x.v_new, cached)


@pytest.mark.parametrize("shift", [0, 1])
def test_append_strides_and_alignment(shift):
    """Rows of a fused projection, token-major pages, and rows at an odd element."""
    new, cached = [3, 1, 40], np.array([14, 0, 7])
    x = U.Inputs(2, cached + new, new, 4, 2, 96, 32, BF16, token_major=True, fused=True)
    T = int(x.cu[-1])
    flat = torch.empty(T * 1000 + 8, dtype=BF16, device="cuda")
    k = flat[shift:shift + T * 1000].view(T, 1000)[:, :192].view(T, 2, 96)
    k.copy_(x.k_new)
    c = x.cache()
    assert (_append(x, c, k, x.v_new, cached) == 0).all()
    _check(x, c, k, x.v_new, cached)


def test_append_extremes():
    """Zeros, the type's largest and smallest values, NaN and infinities: non-finite
    entries become NaN codes and leave the scale to the others; the scale's limits."""
    new, cached = [4, 4, 4, 4, 4], np.array([0, 3, 0, 0, 0])
    x = U.Inputs(3, cached + new, new, 1, 1, 16, 16, F32)
    k, v = x.k_new.clone(), x.v_new.clone()
    k[0:4] = 0
    k[4:8] = 1e30                       # a kept page's scale grows past its codes' range
    k[8:12] = 3.4e38
    k[12:16] = torch.tensor([1e-45, -1e-38, 1e-33, 0.0], device="cuda")[:, None, None]
    k[16] = float("nan")
    k[17] = float("inf")
    k[18, 0, :8] = float("-inf")
    v[0:4] = -448.0
    v[4:8] = -0.0
    v[16:20] = float("nan")
    c = x.cache()
    assert (_append(x, c, k, v, cached) == 0).all()
    _check(x, c, k, v, cached)


def test_append_is_idempotent_and_rolls_back():
    """Appending the same tokens at the same length again changes nothing; appending
    others at a shorter length forgets what followed."""
    new, cached = [8, 8, 5], np.array([10, 60, 33])
    x = U.Inputs(4, cached + new, new, 2, 2, 64, 64, BF16)
    c = x.cache()
    _append(x, c, x.k_new * 3, x.v_new, cached)
    first = [t.clone() for t in (c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale)]
    _append(x, c, x.k_new * 3, x.v_new, cached)
    for a, b in zip(first, (c.k.view(torch.uint8), c.v.view(torch.uint8), c.k_scale, c.v_scale)):
        assert torch.equal(a, b)
    x.kc, x.vc = U.codes_of(c.k), U.codes_of(c.v)
    x.ks, x.vs = c.k_scale.double().cpu().numpy(), c.v_scale.double().cpu().numpy()
    back = cached - np.array([3, 0, 1])
    _append(x, c, x.v_new * 9, x.k_new, back)
    _check(x, c, x.v_new * 9, x.k_new, back)


def test_append_statuses():
    new, cached = [2, 2, 2, 2, 2], np.array([14, 3, 3, 3, 3])
    x = U.Inputs(5, cached + new, new, 1, 1, 32, 16, BF16)
    x.table[1, 0] = x.kc.shape[0]  # not a page
    bad = cached.copy()
    bad[2] = -1
    bad[3] = 16 * x.table.shape[1] - 1  # its two tokens do not fit the table
    c = x.cache()
    st = _append(x, c, x.k_new, x.v_new, bad)
    assert st.tolist() == [0, 6, 2, 2, 0]
    keep = x.cu.copy()
    x.table[1, 0] = x.free[0]  # the oracle: requests 0 and 4 only
    want_c, want_s = x.kc, x.ks
    for b in (0, 4):
        x.cu = keep[b:b + 2] - keep[b]
        want_c, want_s = U.append(want_c, want_s, x.k_new[keep[b]:keep[b + 1]].double().cpu().numpy(),
                                  x.table[b:b + 1], cached[b:b + 1], x.cu)
    np.testing.assert_array_equal(U.codes_of(c.k), want_c)
    np.testing.assert_array_equal(c.k_scale.double().cpu().numpy(), want_s)
    x.cu = np.array([0, 2, 1, 4, 6, 99], np.int32)  # decreasing, and past the rows
    c = x.cache()
    st = _append(x, c, x.k_new, x.v_new, cached, max_new=2)
    assert st[1] == 2 and st[4] == 2 and st[2] == 2  # three tokens where at most two were promised


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("page,D,H", [(16, 64, 1), (32, 80, 3), (64, 128, 8), (128, 256, 2)])
def test_gather_matches_oracle(dtype, page, D, H):
    import speculative_decoding_verification_15_gb300 as pkg

    lens = np.array([5, 0, 3 * page, 200, 1, 77])
    new = np.array([5, 0, 2 * page + 1, 130, 1, 0])
    x = U.Inputs(6, lens, new, H, H, D, page, dtype)
    x.kc[x.table[3, 1], 0, 0, :4] = 127  # a NaN code reads as NaN
    c = x.cache()
    first = lens - new
    T = int(x.cu[-1])
    out = pkg.kv_gather(c, x.i32(x.table), x.i32(x.cu), T, first=x.i32(first), dtype=dtype)
    assert (out["status"] == 0).all()
    for name, codes, scale in (("k", x.kc, x.ks), ("v", x.vc, x.vs)):
        got = out[name].double().cpu().numpy()
        for b in range(len(lens)):
            want = U.read(codes, scale, x.table[b], np.arange(first[b], lens[b]))
            np.testing.assert_array_equal(got[x.cu[b]:x.cu[b + 1]], want)


def test_gather_statuses_and_untouched_rows():
    import speculative_decoding_verification_15_gb300 as pkg
    from speculative_decoding_verification_15_gb300 import binding

    x = U.Inputs(7, [20, 20, 20, 20], [4, 4, 4, 4], 2, 2, 32, 16, BF16)
    x.table[1, 1] = -5
    c = x.cache()
    k = torch.full((30, 2, 32), 7.0, dtype=BF16, device="cuda")
    v, st = k.clone(), torch.empty(4, dtype=torch.int32, device="cuda")
    first = np.array([0, 14, -1, 29])
    binding.spec_kv_gather(c, x.i32(x.table), x.i32(x.cu + 3), x.i32(first), k, v, st)
    assert st.tolist() == [0, 6, 2, 2]
    assert (k[:3] == 7).all() and (k[11:] == 7).all() and (v[11:] == 7).all()
    assert torch.isnan(k[9:11]).all() and torch.isnan(v[9:11]).all() and torch.isfinite(k[7:9].float()).all()
    want = U.read(x.kc, x.ks, x.table[0], np.arange(4))
    np.testing.assert_array_equal(k[3:7].double().cpu().numpy(), want)
    assert pkg.kv_gather(c, x.i32(x.table), x.i32([0] * 5), 0)["k"].shape[0] == 0


def test_append_then_gather_round_trip():
    """What is read back is within half a code step of what was written: 2^-4 of it,
    or half the smallest step of its page's scale."""
    import speculative_decoding_verification_15_gb300 as pkg

    new = [33, 100]
    x = U.Inputs(8, new, new, 2, 2, 128, 64, BF16)
    c = x.cache()
    _append(x, c, x.k_new, x.v_new, np.array([0, 0]))
    out = pkg.kv_gather(c, x.i32(x.table), x.i32(x.cu), int(x.cu[-1]))
    want, got = x.k_new.double(), out["k"].double()
    assert ((got - want).abs() <= torch.maximum(want.abs() * 2.0 ** -4, c.k_scale.max().double() * 2.0 ** -10)).all()


def test_pages_past_4_gib():
    """Entries whose byte offset passes 32 bits."""
    import speculative_decoding_verification_15_gb300 as pkg

    H, bs, D = 4, 128, 128
    P = (5 << 30) // (H * bs * D)
    k, v = (torch.empty((P, H, bs, D), dtype=torch.uint8, device="cuda") for _ in "kv")
    c = pkg.KVCache(k.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn),
                    torch.ones((P, H), device="cuda"), torch.ones((P, H), device="cuda"))
    g = torch.Generator(device="cuda").manual_seed(3)
    new = torch.randn((200, H, D), generator=g, device="cuda").to(BF16)
    table = torch.tensor([[P - 1, P // 2 + 1]], dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, 200], dtype=torch.int32, device="cuda")
    zero = torch.zeros(1, dtype=torch.int32, device="cuda")
    pkg.kv_append(c, new, new, table, zero, cu, 200)
    out = pkg.kv_gather(c, table, cu, 200, dtype=F32)
    assert ((out["k"] - new.float()).abs() <= torch.maximum(new.float().abs() / 16, c.k_scale[P - 1].max() / 1024)).all()
    assert torch.equal(out["k"], out["v"])
