"""GPU tests of the workspaces of the attention over the 8-bit cache: graphs, streams."""
import numpy as np
import pytest
import torch

import kv_util as U

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def _args(x):
    return x.q, x.cache(), x.i32(x.table), x.i32(x.lens), x.i32(x.cu), int(x.new.max())


def _cut(seed, D, B=40):
    """Requests whose items are cut between CTAs, so that counters and slots are used."""
    return U.Inputs(seed, 900 + (np.arange(B) * 131) % 700, np.full(B, 4), 8, 2, D, 64, BF16)


def _capture(args, stream, calls=1):
    import speculative_decoding_verification_15_gb300 as pkg

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = [pkg.cache_attention(*args, want_lse=True) for _ in range(calls)]
    return graph, out


def test_graph_outlives_its_streams_workspace():
    """Warm up and capture heads of 64, call heads of 128 on the same stream (a larger
    workspace), take the freed memory, replay: the graph's results are right and nobody
    else's memory has changed."""
    import speculative_decoding_verification_15_gb300 as pkg

    small, large = _args(_cut(60, 64)), _args(_cut(61, 128))
    want = pkg.cache_attention(*small, want_lse=True)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        pkg.cache_attention(*small)
        s.synchronize()
        graph, (out,) = _capture(small, s)
        pkg.cache_attention(*large)
        s.synchronize()
        taken = [torch.full((4 << 20,), 0x55, dtype=torch.uint8, device="cuda") for _ in range(16)]
        for _ in range(3):
            out["out"].fill_(float("nan"))
            graph.replay()
            s.synchronize()
            assert (out["status"] == 0).all()
            assert torch.equal(out["out"], want["out"]) and torch.equal(out["lse"], want["lse"])
        assert all((t == 0x55).all() for t in taken)


def test_replays_next_to_calls_on_the_capture_stream():
    """A graph replayed on another stream while its capture stream makes calls of its own,
    and a second graph captured there: every result is that of a call alone."""
    import speculative_decoding_verification_15_gb300 as pkg

    a, b = _args(_cut(62, 128)), _args(_cut(63, 128))
    want_a, want_b = pkg.cache_attention(*a), pkg.cache_attention(*b)
    s, t, u = (torch.cuda.Stream() for _ in range(3))
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        pkg.cache_attention(*a)
        s.synchronize()
        one, out_one = _capture(a, s, calls=3)
        two, out_two = _capture(b, s, calls=3)
    torch.cuda.synchronize()
    eager = []
    for _ in range(20):
        with torch.cuda.stream(t):
            one.replay()
        with torch.cuda.stream(u):
            two.replay()
        eager.append(pkg.cache_attention(*b, stream=s))
        eager.append(pkg.cache_attention(*a))
    torch.cuda.synchronize()
    for got in out_one:
        assert (got["status"] == 0).all() and torch.equal(got["out"], want_a["out"])
    for got in out_two:
        assert (got["status"] == 0).all() and torch.equal(got["out"], want_b["out"])
    for i, got in enumerate(eager):
        assert torch.equal(got["out"], (want_a if i % 2 else want_b)["out"])


def test_two_streams_at_once():
    import speculative_decoding_verification_15_gb300 as pkg

    a, b = _args(_cut(64, 64)), _args(_cut(65, 64))
    want = pkg.cache_attention(*a)["out"], pkg.cache_attention(*b)["out"]
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = [[pkg.cache_attention(*args, stream=s)["out"] for args, s in zip((a, b), streams)] for _ in range(20)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for pair in got for o, w in zip(pair, want))


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
def test_only_the_counters_need_to_be_zero(dtype):
    """The rest of a workspace may hold anything (here NaN), and a second call finds the
    counters as the first did."""
    from speculative_decoding_verification_15_gb300 import binding

    x = U.Inputs(66, 900 + (np.arange(40) * 131) % 700, np.full(40, 4), 8, 2, 64, 64, dtype)
    q, c, table, seq, cu, n = _args(x)
    need = binding.spec_cache_attention_workspace_size(8, 2, 64, binding._dtype_code(q))
    first = None
    for fill in (0, 0xFF):
        ws = torch.full((need,), fill, dtype=torch.uint8, device="cuda")
        ws[:binding.CACHE_ATTENTION_COUNTERS] = 0
        for _ in range(2):
            out, status = torch.empty_like(q), torch.empty(40, dtype=torch.int32, device="cuda")
            binding.spec_cache_attention(q, c, table, seq, cu, n, 0.125, 0, 0, out, None, status, ws)
            assert (status == 0).all() and (ws[:binding.CACHE_ATTENTION_COUNTERS] == 0).all()
            first = out if first is None else first
            assert torch.equal(out, first)


def _call(args, ws, scale=0.125):
    from speculative_decoding_verification_15_gb300 import binding

    q, c, table, seq, cu, n = args
    out, status = torch.empty_like(q), torch.full((len(seq),), -1, dtype=torch.int32, device="cuda")
    binding.spec_cache_attention(q, c, table, seq, cu, n, scale, 0, 0, out, None, status, ws)
    return out, status


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
@pytest.mark.parametrize("B", [1, 40, 1000])
def test_a_failed_call_fails_for_every_request(dtype, B):
    """A CTA whose wait ran out sets the word at the end of the counters: CTAs that write
    their statuses only afterwards do not hide it (here all of them: the word is there
    before the call), nor does any later call, until the counters are zeroed."""
    from speculative_decoding_verification_15_gb300 import binding

    x = U.Inputs(67, 300 + (np.arange(B) * 131) % 700, np.full(B, 2), 8, 2, 64, 64, dtype)
    args = _args(x)
    ws = torch.zeros(binding.spec_cache_attention_workspace_size(8, 2, 64, binding._dtype_code(x.q)), dtype=torch.uint8,
                     device="cuda")
    want, status = _call(args, ws)
    assert (status == 0).all()
    counters = ws[:binding.CACHE_ATTENTION_COUNTERS]
    counters.view(torch.int32)[-1] = 1
    for _ in range(2):
        assert (_call(args, ws)[1] == 5).all()
    counters.zero_()
    out, status = _call(args, ws)
    assert (status == 0).all() and torch.equal(out, want)


@pytest.mark.parametrize("dtype", [BF16, torch.float32])
@pytest.mark.parametrize("word", [1, 2, 5, 300, 1 << 20, -1, 1 + (1 << 32), (3 << 32) + 2])
def test_counters_that_were_not_zero_are_reported(dtype, word):
    """Two long requests, their items split between all CTAs: a counter that starts at
    anything else would have a part join too early, or never."""
    from speculative_decoding_verification_15_gb300 import binding

    x = U.Inputs(68, [9000, 7777], [3, 1], 8, 2, 64, 64, dtype)
    args = _args(x)
    ws = torch.zeros(binding.spec_cache_attention_workspace_size(8, 2, 64, binding._dtype_code(x.q)), dtype=torch.uint8,
                     device="cuda")
    counters = ws[:binding.CACHE_ATTENTION_COUNTERS]
    want, status = _call(args, ws)
    assert (status == 0).all() and (counters == 0).all()
    counters[:320 * 8].view(torch.int64).fill_(word)
    for _ in range(2):
        assert (_call(args, ws)[1] == 5).all()
    counters.zero_()
    out, status = _call(args, ws)
    assert (status == 0).all() and torch.equal(out, want)


def test_the_package_can_be_told_to_start_over():
    import speculative_decoding_verification_15_gb300 as pkg
    from speculative_decoding_verification_15_gb300 import api, binding

    args = _args(_cut(69, 64))
    want = pkg.cache_attention(*args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    pkg.cache_attention(*args, stream=s)
    torch.cuda.synchronize()
    for ws in api._attn_ws.values():
        ws[:binding.CACHE_ATTENTION_COUNTERS].fill_(1)
    torch.cuda.synchronize()
    for stream in (None, s):
        assert (pkg.cache_attention(*args, stream=stream)["status"].cpu() == 5).all()
    pkg.cache_attention_reset("cuda:0")
    for stream in (None, s):
        got = pkg.cache_attention(*args, stream=stream)
        torch.cuda.synchronize()
        assert (got["status"] == 0).all() and torch.equal(got["out"], want["out"])
