"""The 8-bit paged cache's entry points without a GPU: bad arguments are refused before
anything is launched, and the oracle's e4m3 is torch's."""
import ctypes

import numpy as np
import pytest
import torch

import __graft_entry__
import kv_util as U

EINVAL, EUNSUP, EWS = 1, 3, 4
P = ctypes.c_void_p(256)


@pytest.fixture(scope="module")
def binding():
    __graft_entry__.build()
    from speculative_decoding_verification_15_gb300 import binding

    binding.load()
    return binding


def _cache(binding, **kw):
    a = dict(k=256, v=256, k_scale=256, v_scale=256, page_stride=4 * 64 * 128, head_stride=64 * 128, token_stride=128,
             num_pages=10, page_size=64, num_heads=4, head_dim=128)
    a.update(kw)
    return binding._CacheStruct(*(a[f] for f, _ in binding._CacheStruct._fields_))


def _append(binding, cache=None, **kw):
    a = dict(k=P, v=P, dtype=0, ldk=512, ldv=512, n=8, B=2, cu=P, max_new=4, cached=P, table=P, width=3, status=P)
    a.update(kw)
    c = _cache(binding) if cache is None else cache
    return binding.load().spec_kv_append(ctypes.byref(c), *a.values(), None)


def _gather(binding, cache=None, **kw):
    a = dict(B=2, cu=P, n=8, first=P, table=P, width=3, k=P, v=P, dtype=0, status=P)
    a.update(kw)
    c = _cache(binding) if cache is None else cache
    return binding.load().spec_kv_gather(ctypes.byref(c), *a.values(), None)


def _attend(binding, cache=None, **kw):
    a = dict(q=P, dtype=0, ldq=8 * 128, Hq=8, n=8, B=2, cu=P, max_query=4, seq=P, table=P, width=3, scale=0.1, window=0,
             sinks=0, out=P, lse=None, status=P, ws=P, ws_bytes=1 << 30)
    a.update(kw)
    c = _cache(binding) if cache is None else cache
    return binding.load().spec_cache_attention(ctypes.byref(c), *a.values(), None)


@pytest.mark.parametrize("call", [_append, _gather, _attend])
def test_cache_description(binding, call):
    assert call(binding, B=0) == 0
    for bad in (dict(k=None), dict(v=None), dict(k_scale=None), dict(v_scale=None), dict(num_pages=0), dict(num_heads=0),
                dict(head_dim=0), dict(k=8), dict(v=264), dict(k_scale=2), dict(token_stride=112), dict(token_stride=136),
                dict(head_stride=-128), dict(page_stride=0), dict(page_stride=1 << 40)):
        assert call(binding, _cache(binding, **bad)) == EINVAL, bad
    for bad in (dict(page_size=48), dict(page_size=256), dict(head_dim=72, token_stride=128),
                dict(head_dim=272, token_stride=272)):
        assert call(binding, _cache(binding, **bad)) == EUNSUP, bad
    assert call(binding, B=-1) == EINVAL and call(binding, n=-1) == EINVAL and call(binding, dtype=2) == EINVAL
    assert call(binding, B=8193) == EUNSUP
    assert call(binding, cu=None) == EINVAL and call(binding, status=None) == EINVAL
    assert call(binding, table=None) == EINVAL and call(binding, width=-1) == EINVAL


def test_append_arguments(binding):
    for bad in (dict(k=None), dict(v=None), dict(ldk=511), dict(ldv=0), dict(max_new=-1), dict(cached=None),
                dict(k=ctypes.c_void_p(257))):
        assert _append(binding, **bad) == EINVAL, bad


def test_gather_arguments(binding):
    for bad in (dict(k=None), dict(v=None), dict(k=ctypes.c_void_p(264))):
        assert _gather(binding, **bad) == EINVAL, bad


def test_attention_arguments(binding):
    for bad in (dict(q=None), dict(out=None), dict(ldq=1023), dict(Hq=6), dict(Hq=0), dict(seq=None), dict(scale=0.0),
                dict(scale=-1.0), dict(scale=float("nan")), dict(scale=float("inf")), dict(window=-1), dict(sinks=-1),
                dict(max_query=-1), dict(lse=ctypes.c_void_p(258)), dict(q=ctypes.c_void_p(257))):
        assert _attend(binding, **bad) == EINVAL, bad
    need = binding.spec_cache_attention_workspace_size(8, 4, 128, 0)
    assert need > 0
    for bad in (dict(ws=None), dict(ws_bytes=need - 1), dict(ws=ctypes.c_void_p(264))):
        assert _attend(binding, **bad) == EWS, bad
    for bad in ((6, 4, 128, 0), (8, 4, 72, 0), (8, 4, 272, 0), (8, 4, 128, 5), (0, 4, 128, 0)):
        assert binding.spec_cache_attention_workspace_size(*bad) == 0, bad


def test_package_refuses_bad_tensors(binding):
    import speculative_decoding_verification_15_gb300 as pkg

    with pytest.raises(ValueError):
        pkg.kv_cache(4, 2, 48, 64, device="cpu")
    with pytest.raises(ValueError):
        pkg.kv_cache(4, 2, 64, 72, device="cpu")
    c = pkg.kv_cache(4, 2, 64, 64, device="cpu")
    i = torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):  # not on a GPU
        pkg.kv_append(c, torch.zeros(1, 2, 64), torch.zeros(1, 2, 64), i.view(1, 2), i[:1], i, 1)


def test_oracle_e4m3_is_torchs():
    g = torch.Generator().manual_seed(0)
    x = torch.cat([torch.randn(20000, generator=g) * s for s in (200.0, 1.0, 2.0 ** -7)])
    x = torch.cat([x, torch.tensor([448.0, 449.0, 464.0, 1e9, 0.0, -0.0, 2.0 ** -9, 2.0 ** -10, 3 * 2.0 ** -11])])
    want = x.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(U.encode(x.double().numpy()), want)
    torch_values = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(U.VALUE, torch_values)


def test_oracle_scale_covers_and_is_smallest():
    for x in (1e-3, 1.0, 447.9, 448.0, 448.1, 896.0, 1e30):
        s = U.wanted_scale(x)
        assert x <= 448 * s and x > 448 * s / 2
    assert U.wanted_scale(0.0) == 2.0 ** -100 and U.wanted_scale(3.4e38) == 2.0 ** 119
