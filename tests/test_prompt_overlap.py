"""Calls whose arrays overlap are refused before anything is launched."""
import ctypes

import pytest

import __graft_entry__

EINVAL, OK = 1, 0
B, WIDTH, PAGES, ROWS = 5, 3, 40, 70


@pytest.fixture(scope="module")
def lib():
    __graft_entry__.build()
    from speculative_decoding_verification_15_gb300 import binding

    return binding.load()


SIZES = dict(free=4 * PAGES, count=4, table=4 * B * WIDTH, held=4 * B, keep=4 * B, new=4 * B, cu=4 * B + 4, seq=4 * B,
             slot=8 * ROWS, position=4 * ROWS, status=4 * B)


def plan(lib, **places):
    """spec_kv_plan with its arrays one right behind the other, but for those in `places`."""
    at, a = 4096, {}
    for name in ("slot", *(n for n in SIZES if n != "slot")):
        a[name] = at
        at += SIZES[name]
    a.update(places)
    p = {n: ctypes.c_void_p(x) for n, x in a.items()}
    return lib.spec_kv_plan(p["free"], p["count"], PAGES, 16, p["table"], WIDTH, p["held"], B, p["keep"], p["new"], ROWS, p["cu"],
                            p["seq"], p["slot"], p["position"], p["status"], None), a


def test_plan_arrays_that_overlap(lib):
    rc, a = plan(lib)
    assert rc != EINVAL  # neighbours do not overlap (there is no such memory: the call ends at the device)
    assert plan(lib, new=a["keep"])[0] != EINVAL  # both are only read
    written = [n for n in SIZES if n not in ("keep", "new")]
    for one in written:
        for other in SIZES:
            if one == other:
                continue
            assert plan(lib, **{one: a[other] // 8 * 8 if one == "slot" else a[other]})[0] == EINVAL, (one, other)
            if one != "slot":
                assert plan(lib, **{one: a[other] + SIZES[other] - 4})[0] == EINVAL, (one, other)
            assert plan(lib, **{other: a[one] + SIZES[one] - (8 if other == "slot" else 4)})[0] == EINVAL, (one, other)
    assert plan(lib, seq=a["keep"])[0] == EINVAL  # a length advanced in place
