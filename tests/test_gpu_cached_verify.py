"""The serving loop of examples/cached_verify.py: append, attention over the cache and
verify together, with drafts rejected and their slots written again."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("cached_verify", os.path.join(ROOT, "examples", "cached_verify.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("window,sinks,temperature", [(0, 0, 0.8), (32, 4, 0.8), (0, 0, 0.0)])
def test_rounds_leave_the_committed_tokens_cached(example, window, sinks, temperature):
    import speculative_decoding_verification_15_gb300 as pkg

    got = example.run(rounds=6, batch=9, drafts=4, window=window, sinks=sinks, temperature=temperature)
    text, cached = got["text"], got["cached"]
    assert [len(t) - 1 for t in text] == cached.tolist()  # all but the last token, the next anchor
    cu = torch.cat([torch.zeros(1, device="cuda"), cached.cumsum(0)]).to(torch.int32)
    out = pkg.kv_gather(got["cache"], got["table"], cu, int(cu[-1]))
    assert (out["status"] == 0).all()
    tokens = torch.cat([torch.tensor(t[:-1]) for t in text]).cuda()
    _, _, k, v = got["target"].projections(tokens)
    # an entry is rounded once, or once more where its page's scale grew: 2^-4 of it each
    # time, and never less than half a step of the largest scale
    for name, want, scale in (("k", k, got["cache"].k_scale), ("v", v, got["cache"].v_scale)):
        err = (out[name].double() - want.double()).abs()
        assert (err <= want.double().abs() / 8 + scale.max().double() * 2.0 ** -9).all()
    assert 0 < got["accepted"] < 4
