"""Rotary positions against 64-bit formulas."""
import numpy as np
import pytest
import torch

import prompt_util as U

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def pkg():
    import speculative_decoding_verification_15_gb300 as pkg

    return pkg


def inputs(seed, T, Hq, Hk, D, dtype, axes, far, fused=False):
    g = np.random.default_rng(seed)
    wide = torch.from_numpy(g.normal(size=(T, Hq + 2 * Hk, D))).to(dtype).cuda()
    q, k = wide[:, :Hq], wide[:, Hq:Hq + Hk]
    if not fused:
        q, k = q.contiguous(), k.contiguous()
    return q, k, g.integers(-far if far < 2 ** 31 - 1 else -2 ** 31, far + 1, (axes, T)).astype(np.int32)


def check(got, x, position, freq, axis, adjacent=False, scale=1.0):
    n = freq.numel()
    a = np.zeros(n, np.int64) if axis is None else axis.cpu().numpy().astype(np.int64)
    want, tol = U.rotary(x.double().cpu().numpy(), position, freq.cpu().numpy(), a, adjacent, scale)
    tol = tol + (U.U16 if x.dtype == BF16 else U.U32) * (np.abs(want) + tol)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), float((err - tol).max())
    assert torch.equal(got[..., 2 * n:], x[..., 2 * n:])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("adjacent", [False, True])
@pytest.mark.parametrize("T,Hq,Hk,D,rot,sections", [
    (1, 32, 8, 128, 128, None), (8, 4, 1, 64, 64, (16, 8, 8)), (301, 3, 3, 80, 80, (20, 20)), (57, 5, 1, 96, 32, (4, 6, 6)),
    (5, 64, 8, 256, 256, (1, 2, 3, 122)), (33, 2, 2, 16, 16, None), (19, 7, 1, 36, 20, (3, 7)), (3, 1, 1, 2, 2, None),
    (1001, 8, 2, 128, 64, (12, 10, 10)), (4, 2, 1, 24, 0, None),
    # many tokens: whole tokens a warp, lanes that meet one unit of each head or several
    (3001, 4, 1, 128, 128, (24, 20, 20)), (2600, 3, 1, 80, 48, None), (2500, 5, 2, 96, 96, None), (2700, 1, 1, 256, 0, None),
    (2433, 12, 4, 256, 256, (100, 28))])
def test_against_64_bits(pkg, T, Hq, Hk, D, rot, sections, adjacent, dtype):
    axes = 1 if sections is None else len(sections)
    q, k, pos = inputs(T + D, T, Hq, Hk, D, dtype, axes, 100000)
    freq, axis = pkg.rotary_frequencies(rot, 10000.0, sections, interleaved=adjacent)
    got = pkg.rotary(q, k, torch.from_numpy(pos).cuda(), freq, axis, adjacent)
    check(got["q"], q, pos, freq, axis, adjacent)
    check(got["k"], k, pos, freq, axis, adjacent)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_far_positions_and_large_frequencies(pkg, dtype):
    """Every int32 keeps its angle, also where a position turns more than once."""
    q, k, pos = inputs(3, 40, 4, 2, 64, dtype, 1, 2 ** 31 - 1)
    pos[0, :3] = 2 ** 31 - 1, -2 ** 31, 0
    freq = torch.from_numpy(np.concatenate([1e6 ** -(np.arange(24) / 24), [3.1, -2.0, 6.2831853, 12.5, 0.0, 1e-9, np.pi, 100.0]]))
    freq = freq.cuda()
    got = pkg.rotary(q, k, torch.from_numpy(pos).cuda(), freq, scale=1.25)
    check(got["q"], q, pos, freq, None, scale=1.25)
    check(got["k"], k, pos, freq, None, scale=1.25)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("offset", [0, 1])
def test_in_place_on_slices(pkg, dtype, offset):
    """In place on the slices of a fused product, aligned to 16 bytes or not; the values
    between them stay."""
    T, Hq, Hk, D = 77, 6, 2, 64
    g = np.random.default_rng(4)
    flat = torch.from_numpy(g.normal(size=T * (Hq + 2 * Hk) * D + 8)).to(dtype).cuda()
    wide = flat[offset:offset + T * (Hq + 2 * Hk) * D].view(T, Hq + 2 * Hk, D)
    q, k = wide[:, :Hq], wide[:, Hq:Hq + Hk]
    before, rest = wide.clone(), flat.clone()
    pos = np.arange(T, dtype=np.int32)[None] + 5
    freq, _ = pkg.rotary_frequencies(D)
    got = pkg.rotary(q, k, torch.from_numpy(pos[0]).cuda(), freq, out_q=q, out_k=k)
    assert got["q"] is q and got["k"] is k
    check(q, before[:, :Hq], pos, freq, None)
    check(k, before[:, Hq:Hq + Hk], pos, freq, None)
    assert torch.equal(wide[:, Hq + Hk:], before[:, Hq + Hk:])
    assert torch.equal(flat[:offset], rest[:offset]) and torch.equal(flat[offset + wide.numel():], rest[offset + wide.numel():])


def test_queries_alone_positions_of_another_type_and_strided_axes(pkg):
    q, _, _ = inputs(6, 50, 4, 1, 64, BF16, 1, 9)
    pos = np.arange(150, dtype=np.int32).reshape(3, 50)
    freq, axis = pkg.rotary_frequencies(64, sections=(10, 11, 11), per_axis=True)
    got = pkg.rotary(q, None, torch.from_numpy(pos).cuda().long(), freq, axis)
    assert got["k"] is None
    check(got["q"], q, pos, freq, axis)
    wide = torch.from_numpy(np.concatenate([pos, pos], 1)).cuda()[:, :50]
    assert torch.equal(pkg.rotary(q, None, wide, freq, axis)["q"], got["q"])


def test_infinities_stay_in_their_pairs(pkg):
    q, k, pos = inputs(7, 9, 2, 1, 64, BF16, 1, 99)
    q[4, 1, 3], k[2, 0, 40] = float("inf"), float("nan")
    freq, _ = pkg.rotary_frequencies(64)
    got = pkg.rotary(q, k, torch.from_numpy(pos[0]).cuda(), freq)
    bad = torch.zeros_like(q, dtype=torch.bool)
    bad[4, 1, [3, 35]] = True
    assert torch.equal(~torch.isfinite(got["q"]), bad)
    bad = torch.zeros_like(k, dtype=torch.bool)
    bad[2, 0, [8, 40]] = True
    assert torch.equal(~torch.isfinite(got["k"]), bad)


def test_no_tokens_a_captured_call_and_another_stream(pkg):
    freq, _ = pkg.rotary_frequencies(64)
    q, k, pos = inputs(8, 30, 4, 2, 64, BF16, 1, 999)
    none = pkg.rotary(q[:0], k[:0], torch.zeros(0, dtype=torch.int32, device="cuda"), freq)
    assert none["q"].shape == (0, 4, 64)
    dp = torch.zeros(30, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        got = pkg.rotary(q, k, dp, freq)
    dp.copy_(torch.from_numpy(pos[0]))
    graph.replay()
    check(got["q"], q, pos, freq, None)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    other = pkg.rotary(q, k, dp, freq, stream=stream)
    torch.cuda.synchronize()
    assert torch.equal(other["q"], got["q"]) and torch.equal(other["k"], got["k"])
