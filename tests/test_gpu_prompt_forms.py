"""Forms of keys and values that neither tensor maps nor 16-byte copies take, whole and in parts."""
import numpy as np
import pytest
import torch

from test_gpu_prompt_attention import BF16, F32, Inputs, close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def pkg():
    import speculative_decoding_verification_15_gb300 as pkg

    return pkg


def strided(t, gap, offset):
    """The same rows `gap` elements further apart, from an address that is off by `offset`."""
    n, h, d = t.shape
    s = torch.as_strided(torch.zeros(n * (h * d + gap) + 8, dtype=t.dtype, device="cuda"), (n, h, d), (h * d + gap, d, 1), offset)
    s.copy_(t)
    return s


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("gaps,offsets", [((1, 1, 1), (1, 0, 3)), ((0, 0, 0), (0, 1, 0)), ((4, 2, 8), (2, 0, 2))])
@pytest.mark.parametrize("new,total,Hq,H,D", [([200, 77], None, 6, 2, 64), ([33, 1], [300, 90], 4, 1, 144),
                                              ([130], None, 3, 3, 96), ([40], [260], 2, 1, 256)])
def test_odd_strides(pkg, new, total, Hq, H, D, gaps, offsets, dtype):
    x = Inputs(D, new, total or new, Hq, H, D, dtype)
    want = x.want(window=100, sinks=2)
    x.q, x.k, x.v = (strided(t, g, o) for t, g, o in zip((x.q, x.k, x.v), gaps, offsets))
    close(x.call(pkg, want_lse=True, window=100, sinks=2), want)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("new,total,Hq,H,D", [([40], [5000], 4, 2, 64), ([5, 0, 60], [3500, 50, 9000], 4, 1, 128),
                                              ([1, 30], [9000, 3000], 2, 2, 192)])
def test_odd_strides_in_parts(pkg, new, total, Hq, H, D, dtype):
    x = Inputs(D + 1, new, total, Hq, H, D, dtype)
    need = pkg.spec_prompt_attention_workspace_size(sum(new), sum(total), len(new), Hq, H, D, int(dtype == F32), 0, 0)
    assert need > 0
    want = x.want()
    x.k, x.v = strided(x.k, 1, 1), strided(x.v, 3, 0)
    close(x.call(pkg, want_lse=True), want)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_odd_strides_with_spoilt_keys(pkg, dtype):
    """What a row does not see is NaN: in its request, behind it, and in rows of none."""
    x = Inputs(8, [90, 40], [90, 40], 4, 2, 64, dtype, behind=9)
    want = x.want(window=30, sinks=1)
    for t in (x.k, x.v):
        t[60] = float("nan")
        t[130:] = float("nan")
    x.k, x.v = strided(x.k, 1, 0), strided(x.v, 1, 1)
    got = x.call(pkg, want_lse=True, window=30, sinks=1)
    out, _, tol, _ = want
    g = got["out"].double().cpu().numpy()[:130]
    sees = np.zeros(130, dtype=bool)
    sees[60:90] = True  # the window is 30 long
    assert np.isnan(g[sees]).all() and (np.abs(g - out[:130]) <= tol[:130])[~sees].all()
    assert (got["status"] == 0).all()
