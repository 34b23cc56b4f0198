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


@pytest.mark.parametrize("esz,code", [(2, 0), (4, 1)])
def test_prompt_output_over_its_inputs(lib, esz, code):
    """out may not lie on q, k or v (which may be slices of one product); next to them it may."""
    n, m, Hq, H, D = 6, 9, 4, 2, 16
    ld = (Hq + 2 * H) * D

    def call(out, k=None):
        q = 1 << 20
        k = q + Hq * D * esz if k is None else k
        p = [ctypes.c_void_p(x) for x in (q, k, k + H * D * esz)]
        other = ctypes.c_void_p(1 << 30)
        return lib.spec_prompt_attention(*p, code, ld, ld, ld, Hq, H, D, n, m, 1, other, n, other, 0.25, 0, 0, ctypes.c_void_p(out), None,
                                         other, None, 0, None)

    q = 1 << 20
    apart = 1 << 24
    q_end, k_end = q + ((n - 1) * ld + Hq * D) * esz, apart + ((m - 1) * ld + H * D) * esz
    v_end = k_end + H * D * esz
    size = n * Hq * D * esz
    for out in (q, q - size + 16, q_end - 16, apart, k_end - 16, v_end - 16, apart - size + 16):
        assert call(out, apart) == EINVAL, hex(out)
    for out in (q - size, (q_end + 15) // 16 * 16, (v_end + 15) // 16 * 16, apart - size):
        assert call(out, apart) != EINVAL, hex(out)
