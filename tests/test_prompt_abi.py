"""Page planning, rotary positions and prompt attention without a GPU: bad arguments are
refused before anything is launched."""
import ctypes

import pytest
import torch

import __graft_entry__

EINVAL, EUNSUP = 1, 3
P = ctypes.c_void_p(256)


@pytest.fixture(scope="module")
def binding():
    __graft_entry__.build()
    from speculative_decoding_verification_15_gb300 import binding

    binding.load()
    return binding


def _plan(binding, **kw):
    a = dict(free=P, count=P, num_pages=9, page_size=16, table=P, width=3, held=P, B=2, keep=P, new=P, n_out=8, cu=P, seq=P,
             slot=P, position=P, status=P)
    a.update(kw)
    return binding.load().spec_kv_plan(*a.values(), None)


def _rotary(binding, **kw):
    a = dict(q=P, k=P, dtype=0, ldq=512, ldk=128, Hq=8, H=2, D=64, n=4, position=P, ldp=4, axes=2, freq=P, axis=P, pairs=32,
             adjacent=0, scale=1.0, oq=P, ok=P, ldoq=512, ldok=128)
    a.update(kw)
    return binding.load().spec_rotary(*a.values(), None)


def _prompt(binding, **kw):
    a = dict(q=P, k=P, v=P, dtype=0, ldq=512, ldk=128, ldv=128, Hq=8, H=2, D=64, n=4, m=4, B=2, cu=P, max_query=4, cuk=None,
             scale=0.1, window=0, sinks=0, out=P, lse=None, status=P, ws=None, ws_bytes=0)
    a.update(kw)
    return binding.load().spec_prompt_attention(*a.values(), None)


def test_plan_arguments(binding):
    for bad in (dict(free=None), dict(count=None), dict(num_pages=0), dict(table=None), dict(held=None), dict(keep=None),
                dict(new=None), dict(cu=None), dict(seq=None), dict(slot=None), dict(position=None), dict(status=None),
                dict(B=-1), dict(n_out=-1), dict(width=-1), dict(slot=ctypes.c_void_p(260)), dict(held=ctypes.c_void_p(258))):
        assert _plan(binding, **bad) == EINVAL, bad
    for bad in (dict(page_size=8), dict(page_size=48), dict(B=8193), dict(B=8000, width=1 << 20)):
        assert _plan(binding, **bad) == EUNSUP, bad


def test_rotary_arguments(binding):
    assert _rotary(binding, n=0) == 0
    for bad in (dict(q=None), dict(k=None), dict(oq=None), dict(ok=None), dict(position=None), dict(freq=None), dict(axis=None),
                dict(dtype=2), dict(ldq=511), dict(ldk=127), dict(ldoq=0), dict(ldok=0), dict(ldp=3), dict(axes=0), dict(Hq=0),
                dict(H=-1), dict(n=-1), dict(pairs=33), dict(pairs=-1), dict(scale=float("inf")), dict(scale=float("nan")),
                dict(q=ctypes.c_void_p(257)), dict(freq=ctypes.c_void_p(260))):
        assert _rotary(binding, **bad) == EINVAL, bad
    assert _rotary(binding, D=257, pairs=32) == EUNSUP and _rotary(binding, Hq=65535) == EUNSUP


def test_prompt_arguments(binding):
    assert _prompt(binding, B=0) == 0
    for bad in (dict(q=None), dict(k=None), dict(v=None), dict(out=None), dict(cu=None), dict(status=None), dict(dtype=2),
                dict(ldq=511), dict(ldk=127), dict(ldv=0), dict(Hq=0), dict(H=0), dict(Hq=7), dict(D=0), dict(n=-1), dict(m=-1),
                dict(B=-1), dict(max_query=-1), dict(m=5), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
                dict(scale=3e38), dict(window=-1), dict(sinks=-1), dict(out=ctypes.c_void_p(264)), dict(q=ctypes.c_void_p(257)),
                dict(cu=ctypes.c_void_p(258)), dict(lse=ctypes.c_void_p(258))):
        assert _prompt(binding, **bad) == EINVAL, bad
    for bad in (dict(D=72), dict(D=272), dict(B=8193), dict(max_query=0x7fffffff), dict(H=65536, Hq=65536)):
        assert _prompt(binding, **bad) == EUNSUP, bad


def test_prompt_workspace(binding):
    size = binding.spec_prompt_attention_workspace_size
    assert size(500, 500, 1, 32, 8, 128, 0) == size(500, 500, 1, 32, 8, 128, 1) == 0  # short
    # what the package does not ask about needs none
    assert not any(size(n, 2047, 1, 4, 1, 64, 0) or size(n, 383, 1, 4, 1, 64, 1) for n in (1, 100, 383))
    need = size(64, 60000, 1, 32, 8, 128, 1)
    assert need > 0 and need % (64 * 32 * 130 * 4) == 0 and size(64, 60000, 1, 32, 8, 128, 1, 300, 4) == 0
    assert size(64, 60000, 1, 32, 8, 128, 2) == 0
    need = size(64, 60000, 1, 32, 8, 128, 0)
    assert need > 0 and need % (64 * 32 * 130 * 4) == 0
    assert size(64, 60000, 1, 32, 8, 128, 0, 500, 4) == 0  # the window leaves little to cut
    assert size(-1, 60000, 1, 32, 8, 128, 0) == size(64, 60000, 1, 32, 7, 128, 0) == size(64, 60000, 0, 32, 8, 128, 0) == 0
    many = dict(n=64, m=60000, Hq=32, H=8, D=128, ldq=4096, ldk=1024, ldv=1024, B=1, cuk=P, max_query=64)
    assert _prompt(binding, **many) == 4
    assert _prompt(binding, **many, ws=P, ws_bytes=need - 1) == 4
    assert _prompt(binding, **many, ws=ctypes.c_void_p(264), ws_bytes=need) == 4


def test_refusals_of_the_package():
    import speculative_decoding_verification_15_gb300 as pkg

    x, i = torch.zeros(4, 2, 64), torch.zeros(3, dtype=torch.int32)
    freq, axis = pkg.rotary_frequencies(64, device="cpu")
    pool = pkg.kv_pool(4, device="cpu")
    for call in (lambda: pkg.rotary(x, x, i, freq), lambda: pkg.prompt_attention(x, x, x, i, 4),
                 lambda: pkg.kv_plan(pool, torch.zeros(2, 3, dtype=torch.int32), i[:2], i[:2], i[:2], 16, 4)):
        with pytest.raises(ValueError, match="CUDA device"):
            call()
    for sections in ((3, 4), (40, -8), (33,)):
        with pytest.raises(ValueError, match="sections"):
            pkg.rotary_frequencies(64, sections=sections, device="cpu")
    for name, at in (("max_query", 4), ("window", 7), ("sinks", 8)):
        args = [x, x, x, i, 4, None, 0.1, 0, 0, x, None, i[:2]]
        args[at] = 1 << 32
        with pytest.raises(ValueError, match=name):
            pkg.spec_prompt_attention(*args)


def test_frequencies():
    import speculative_decoding_verification_15_gb300 as pkg

    freq, axis = pkg.rotary_frequencies(12, 64.0, device="cpu")
    assert axis is None and freq.tolist() == [64.0 ** (-i / 6) for i in range(6)]
    freq, axis = pkg.rotary_frequencies(12, 64.0, (3, 1, 2), device="cpu")
    assert axis.tolist() == [0, 0, 0, 1, 2, 2] and freq.tolist() == [64.0 ** (-i / 6) for i in range(6)]
    freq, axis = pkg.rotary_frequencies(12, 64.0, (3, 1, 2), interleaved=True, per_axis=True, device="cpu")
    assert axis.tolist() == [0, 1, 2, 0, 2, 0]
    assert freq.tolist() == [64.0 ** -x for x in (0.0, 0.0, 0.0, 1 / 3, 0.5, 2 / 3)]
