"""examples/paged_serving.py: page planning, rotary positions, prompt attention and the cache's
calls together, with drafts rejected and pages handed on."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import prompt_util as U

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("paged_serving", os.path.join(ROOT, "examples", "paged_serving.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("window,sinks,temperature,page", [(0, 0, 0.8, 16), (64, 4, 0.8, 32), (0, 0, 0.0, 128)])
def test_what_is_cached_is_the_committed_text(example, window, sinks, temperature, page):
    import speculative_decoding_verification_15_gb300 as pkg

    got = example.run(rounds=6, batch=9, drafts=4, window=window, sinks=sinks, temperature=temperature, page_size=page)
    text, cached, target = got["text"], got["cached"], got["target"]
    assert [len(t) - 1 for t in text] == cached.tolist()  # all but the last token, the next anchor
    # every page is free or some request's, once
    count, table, held = int(got["pool"].count), got["table"].cpu().numpy(), got["held"].cpu().numpy()
    owned = np.concatenate([table[b, :held[b]] for b in range(9)] + [got["pool"].free[:count].cpu().numpy()])
    assert sorted(owned.tolist()) == list(range(len(owned))) and len(owned) == got["pool"].free.numel()
    live = np.flatnonzero(~got["ended"].cpu().numpy())
    assert (held == np.where(got["ended"].cpu().numpy(), 0, -(-cached.cpu().numpy() // page))).all()
    # the keys of the live requests: turned by their positions, then rounded once or (where a
    # page's scale grew) once more, 2^-4 of an entry each time and never less than half a step
    # of the largest scale
    n = cached[live]
    cu = torch.cat([torch.zeros(1, device="cuda"), n.cumsum(0)]).to(torch.int32)
    out = pkg.kv_gather(got["cache"], got["table"][live].contiguous(), cu, int(cu[-1]))
    assert (out["status"] == 0).all()
    tokens = torch.cat([torch.tensor(text[b][:-1]) for b in live]).cuda()
    x, q, k, v = target.projections(tokens)
    position = torch.cat([torch.arange(m, dtype=torch.int32) for m in n.tolist()]).cuda()
    turned = pkg.rotary(q, k, position, got["freq"])
    for name, want, scale in (("k", turned["k"], got["cache"].k_scale), ("v", v, got["cache"].v_scale)):
        err = (out[name].double() - want.double()).abs()
        assert (err <= want.double().abs() / 8 + scale.max().double() * 2.0 ** -9).all()
    # and the prompt's attention over the whole text is the formula's
    att = pkg.prompt_attention(turned["q"], turned["k"], v, cu, int(n.max()), window=window, sinks=sinks)
    want, _, tol, _ = U.attention(*(t.double().cpu().numpy() for t in (turned["q"], turned["k"], v)), cu.cpu().numpy(),
                                  cu.cpu().numpy(), 64 ** -0.5, window, sinks, bf16=True)
    assert (np.abs(att["out"].double().cpu().numpy() - want) <= tol).all()
    assert 0 < got["accepted"] < 4


def test_no_rounds(example):
    got = example.run(rounds=0, batch=3)
    assert got["cached"].tolist() == got["prompts"].tolist()
