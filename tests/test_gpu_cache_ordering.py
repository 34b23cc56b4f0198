"""GPU tests of what a CTA of the attention over the 8-bit cache hands from one item to the
next: many short items a CTA, whose rows must all land in their own places."""
import numpy as np
import pytest
import torch

import kv_util as U

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("group,n", [(1, 8), (4, 8), (8, 8), (2, 3)])  # row tiles of 16, 32, 64 and 16 rows
@pytest.mark.parametrize("page", [16, 64])
def test_many_items_of_one_tile(group, n, page):
    """3000 requests of up to 128 tokens, four key heads: about 40 items of one tile a CTA.
    Every row is written (the output starts as NaN), equals the oracle's, and repeats."""
    from speculative_decoding_verification_15_gb300 import binding

    g = np.random.default_rng(40)
    B, H, D = 3000, 4, 64
    new = g.integers(1, n + 1, B)
    new[::7] = n
    lens = np.minimum(128, new + g.integers(0, 128, B))
    x = U.Inputs(41, lens, new, H * group, H, D, page, torch.bfloat16)
    c, T = x.cache(), int(x.cu[-1])
    table, seq, cu = x.i32(x.table), x.i32(x.lens), x.i32(x.cu)
    status = torch.empty(B, dtype=torch.int32, device="cuda")
    ws = torch.zeros(binding.spec_cache_attention_workspace_size(H * group, H, D, 0), dtype=torch.uint8, device="cuda")
    first = None
    for _ in range(20):
        out = torch.full((T, H * group, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        lse = torch.full((T, H * group), float("nan"), device="cuda")
        binding.spec_cache_attention(x.q, c, table, seq, cu, n, D ** -0.5, 0, 0, out, lse, status, ws)
        assert (status == 0).all() and not torch.isnan(out).any() and not torch.isnan(lse).any()
        if first is None:
            first = out, lse
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1])
    pick = np.sort(g.choice(B, 250, replace=False))  # the oracle is slow: every twelfth request
    rows = np.concatenate([np.arange(x.cu[b], x.cu[b + 1]) for b in pick])
    q, x.table, x.lens, x.cu = x.q64()[rows], x.table[pick], x.lens[pick], np.concatenate([[0], np.cumsum(x.new[pick])])
    want, want_lse, tol, tol_lse = U.attention(q, x.kc, x.vc, x.ks, x.vs, x.table, x.lens, x.cu, D ** -0.5, bf16=True)
    got, got_lse = first[0].double().cpu().numpy()[rows], first[1].double().cpu().numpy()[rows]
    assert (np.abs(got - want) <= tol).all() and (np.abs(got_lse - want_lse) <= tol_lse).all()
