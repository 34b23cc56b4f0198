"""Whose workspace a call of the attention over the 8-bit cache gets, without a GPU."""
import pytest
import torch

CPU = torch.device("cpu")


@pytest.fixture
def api(monkeypatch):
    from speculative_decoding_verification_15_gb300 import api

    state = {"stream": 7, "capturing": False}
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: state["stream"])
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["capturing"])
    monkeypatch.setattr(api, "_attn_ws", {})
    api.state = state
    return api


def test_calls_on_a_stream_share_one(api):
    a = api._attention_workspace(CPU, None, 5000)
    assert api._attention_workspace(CPU, None, 4000) is a
    api.state["stream"] = 8
    assert api._attention_workspace(CPU, None, 4000) is not a
    api.state["stream"] = 7
    assert api._attention_workspace(CPU, None, 9000).numel() == 9000


def test_a_captured_call_has_its_own(api):
    """Whether its stream has one already or not: nothing else may write to what a graph
    holds, and nothing may free it."""
    a = api._attention_workspace(CPU, None, 5000)
    api.state["capturing"] = True
    b, c = api._attention_workspace(CPU, None, 5000), api._attention_workspace(CPU, None, 5000)
    assert len({a.data_ptr(), b.data_ptr(), c.data_ptr()}) == 3
    api.state["capturing"] = False
    assert api._attention_workspace(CPU, None, 5000) is a


@pytest.mark.parametrize("capturing", [False, True])
def test_only_the_counters_are_zeroed(api, monkeypatch, capturing):
    """They are a few KB, the whole is some 20 MB, and a captured call zeroes them in every
    replay."""
    from speculative_decoding_verification_15_gb300 import binding

    monkeypatch.setattr(torch, "empty", lambda n, **kw: torch.full((n,), 0xA5, **kw))
    api.state["capturing"] = capturing
    ws = api._attention_workspace(CPU, None, 50000)
    n = binding.CACHE_ATTENTION_COUNTERS
    assert n <= 4096 and (ws[:n] == 0).all() and (ws[n:] == 0xA5).all()
