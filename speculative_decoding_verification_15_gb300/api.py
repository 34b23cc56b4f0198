"""Convenience layer over the C ABI: allocates outputs and a cached workspace.

Every call goes through the C entry points in ``binding``; this module only
manages tensors.  Shapes follow the C ABI: target logits [B, K+1, V], draft logits
[B, K, V] (bfloat16 or float32), draft tokens [B, K] int32.
"""
from __future__ import annotations

import functools
import threading

import torch

from . import binding
from .binding import KVCache, PagePool

_ws_lock = threading.Lock()
_ws_cache: dict[int, torch.Tensor] = {}


def workspace(device: torch.device, nbytes: int) -> torch.Tensor:
    """A cached uint8 workspace of at least nbytes on device (grown on demand).

    It is zero-filled when allocated: the verify calls need a zeroed workspace
    before its first use and leave it ready for the next call."""
    idx = torch.device(device).index
    if idx is None:
        idx = torch.cuda.current_device()
    with _ws_lock:
        ws = _ws_cache.get(idx)
        if ws is None or ws.numel() < nbytes:
            ws = torch.zeros(max(nbytes, 1), dtype=torch.uint8, device=torch.device("cuda", idx))
            _ws_cache[idx] = ws
        return ws


def _as_i32(t, device):
    return None if t is None else t.to(device=device, dtype=torch.int32).contiguous()


def verify_sample(target, draft, draft_tokens, temperature, seed: int, step: int, num_draft=None,
                  stream=None, want_probs: bool = True) -> dict:
    dev = target.device
    B, K1, V = target.shape
    K = K1 - 1
    x = _as_i32(draft_tokens, dev)
    nd = _as_i32(num_draft, dev)
    T = temperature.to(device=dev, dtype=torch.float32).contiguous()
    out = dict(tokens=torch.empty((B, K1), dtype=torch.int32, device=dev),
               accepted=torch.empty(B, dtype=torch.int32, device=dev),
               status=torch.empty(B, dtype=torch.int32, device=dev),
               p=torch.empty((B, K), dtype=torch.float32, device=dev) if want_probs else None,
               q=torch.empty((B, K), dtype=torch.float32, device=dev) if want_probs else None)
    ws = workspace(dev, binding.spec_verify_workspace_size(B, K, V, binding._dtype_code(target)))
    binding.spec_verify_sample(target, draft, x, nd, T, seed, step, out["tokens"], out["accepted"], out["p"],
                               out["q"], out["status"], ws, stream)
    return out


def verify_greedy(target, draft_tokens, num_draft=None, stream=None) -> dict:
    dev = target.device
    B, K1, V = target.shape
    x = _as_i32(draft_tokens, dev)
    nd = _as_i32(num_draft, dev)
    out = dict(tokens=torch.empty((B, K1), dtype=torch.int32, device=dev),
               accepted=torch.empty(B, dtype=torch.int32, device=dev),
               status=torch.empty(B, dtype=torch.int32, device=dev))
    ws = workspace(dev, binding.spec_verify_workspace_size(B, K1 - 1, V, binding._dtype_code(target)))
    binding.spec_verify_greedy(target, x, nd, out["tokens"], out["accepted"], out["status"], ws, stream)
    return out


def schedule_verify_len(conf, step_time_us, budget: int, min_len: int, max_len=None, stream=None):
    dev = conf.device
    B = conf.shape[0]
    out_len = torch.empty(B, dtype=torch.int32, device=dev)
    info = torch.empty(3, dtype=torch.float64, device=dev)
    binding.spec_schedule_verify_len(conf.to(torch.float32).contiguous(), _as_i32(max_len, dev),
                                     step_time_us.to(device=dev, dtype=torch.float32).contiguous(), budget,
                                     min_len, out_len, info, stream)
    return out_len, info


def verify_sample_early_exit(target, draft, draft_tokens, temperature, seed: int, step: int, num_draft=None,
                             stream=None) -> dict:
    """Sampling verify that stops reading at each request's first rejection."""
    dev = target.device
    B, K1, V = target.shape
    K = K1 - 1
    out = dict(tokens=torch.empty((B, K1), dtype=torch.int32, device=dev),
               accepted=torch.empty(B, dtype=torch.int32, device=dev),
               p=torch.empty((B, K), dtype=torch.float32, device=dev),
               q=torch.empty((B, K), dtype=torch.float32, device=dev),
               status=torch.empty(B, dtype=torch.int32, device=dev))
    binding.spec_verify_sample_early_exit(target, draft, _as_i32(draft_tokens, dev), _as_i32(num_draft, dev),
                                          temperature.to(device=dev, dtype=torch.float32).contiguous(), seed, step,
                                          out["tokens"], out["accepted"], out["p"], out["q"], out["status"],
                                          stream)
    return out


def verify_greedy_early_exit(target, draft_tokens, num_draft=None, stream=None) -> dict:
    """Greedy verify that stops reading at each request's first mismatch."""
    dev = target.device
    B, K1, V = target.shape
    out = dict(tokens=torch.empty((B, K1), dtype=torch.int32, device=dev),
               accepted=torch.empty(B, dtype=torch.int32, device=dev),
               status=torch.empty(B, dtype=torch.int32, device=dev))
    binding.spec_verify_greedy_early_exit(target, _as_i32(draft_tokens, dev), _as_i32(num_draft, dev),
                                          out["tokens"], out["accepted"], out["status"], stream)
    return out


def markov_draft(base, anchor, emb, proj, temperature=None, seed: int = 0, step: int = 0, stream=None) -> dict:
    """Markov-head drafting of one block: tokens [B, K], corrected logits [B, K, V]
    (float32) and status [B]."""
    dev = base.device
    B, K, V = base.shape
    out = dict(tokens=torch.empty((B, K), dtype=torch.int32, device=dev),
               logits=torch.empty((B, K, V), dtype=torch.float32, device=dev),
               status=torch.empty(B, dtype=torch.int32, device=dev))
    T = None if temperature is None else temperature.to(device=dev, dtype=torch.float32).contiguous()
    binding.spec_markov_draft(base, _as_i32(anchor, dev), emb, proj, T, seed, step, out["tokens"], out["logits"],
                              out["status"], stream)
    return out


def markov_draft_topk(base, anchor, emb, proj, topk: int, temperature=None, seed: int = 0, step: int = 0,
                      want_logits: bool = True, stream=None) -> dict:
    """Top-K Markov-head drafting of one block: tokens [B, K], corrected logits
    [B, K, V] (float32, -inf outside each position's topk candidates; None unless
    want_logits) and status [B]."""
    dev = base.device
    B, K, V = base.shape
    out = dict(tokens=torch.empty((B, K), dtype=torch.int32, device=dev),
               logits=torch.empty((B, K, V), dtype=torch.float32, device=dev) if want_logits else None,
               status=torch.empty(B, dtype=torch.int32, device=dev))
    T = None if temperature is None else temperature.to(device=dev, dtype=torch.float32).contiguous()
    ws = torch.empty(max(binding.spec_markov_topk_workspace_size(B, K, V, topk), 16), dtype=torch.uint8, device=dev)
    binding.spec_markov_draft_topk(base, _as_i32(anchor, dev), emb, proj, T, seed, step, topk, out["tokens"],
                                   out["logits"], out["status"], ws, stream)
    return out


def verify_sample_flat(target, draft, cu_draft, draft_tokens, temperature, seed: int, step: int, Kmax: int,
                       stream=None) -> dict:
    """Flattened ragged layout (no padding rows): target [sum_b (k_b + 1), V], draft
    [sum_b k_b, V], cu_draft [B + 1] offsets of the draft positions, draft_tokens
    [sum_b k_b]; Kmax bounds every k_b.  Outputs are flattened the same way."""
    dev = target.device
    cu = _as_i32(cu_draft, dev)
    B = cu.numel() - 1
    n_tok = target.shape[0]
    out = dict(tokens=torch.empty(n_tok, dtype=torch.int32, device=dev),
               accepted=torch.empty(B, dtype=torch.int32, device=dev),
               p=torch.empty(draft.shape[0], dtype=torch.float32, device=dev),
               q=torch.empty(draft.shape[0], dtype=torch.float32, device=dev),
               status=torch.empty(B, dtype=torch.int32, device=dev))
    ws = workspace(dev, binding.spec_verify_workspace_size(B, Kmax, target.shape[1], binding._dtype_code(target)))
    binding.spec_verify_sample_flat(target, draft, cu, _as_i32(draft_tokens, dev),
                                    temperature.to(device=dev, dtype=torch.float32).contiguous(), seed, step,
                                    out["tokens"], out["accepted"], out["p"], out["q"], out["status"], ws, Kmax,
                                    stream)
    return out


def verify_greedy_flat(target, cu_draft, draft_tokens, Kmax: int, stream=None) -> dict:
    """Greedy verify in the flattened ragged layout (see verify_sample_flat)."""
    dev = target.device
    cu = _as_i32(cu_draft, dev)
    B = cu.numel() - 1
    out = dict(tokens=torch.empty(target.shape[0], dtype=torch.int32, device=dev),
               accepted=torch.empty(B, dtype=torch.int32, device=dev),
               status=torch.empty(B, dtype=torch.int32, device=dev))
    ws = workspace(dev, binding.spec_verify_workspace_size(B, Kmax, target.shape[1], binding._dtype_code(target)))
    binding.spec_verify_greedy_flat(target, cu, _as_i32(draft_tokens, dev), out["tokens"], out["accepted"],
                                    out["status"], ws, Kmax, stream)
    return out


def schedule_verify_len_stale(conf_stale, conf, step_time_us, budget: int, min_len: int, max_len=None,
                              stream=None):
    dev = conf.device
    B = conf.shape[0]
    out_len = torch.empty(B, dtype=torch.int32, device=dev)
    info = torch.empty(3, dtype=torch.float64, device=dev)
    binding.spec_schedule_verify_len_stale(conf_stale.to(device=dev, dtype=torch.float32).contiguous(),
                                           conf.to(torch.float32).contiguous(), _as_i32(max_len, dev),
                                           step_time_us.to(device=dev, dtype=torch.float32).contiguous(), budget,
                                           min_len, out_len, info, stream)
    return out_len, info


def schedule_threshold(conf, threshold: float, max_len=None, stream=None):
    dev = conf.device
    out_len = torch.empty(conf.shape[0], dtype=torch.int32, device=dev)
    binding.spec_schedule_threshold(conf.to(torch.float32).contiguous(), _as_i32(max_len, dev), threshold,
                                    out_len, stream)
    return out_len


def verify_sample_host(target_h, draft_h, tokens_h, temperature_h, seed: int, step: int, num_draft_h=None,
                       device=None, dev_buffers: dict | None = None) -> dict:
    """End-to-end call from host (ideally pinned) tensors: copy in, verify, copy the
    emitted tokens, accepted counts and statuses back.  Returns host tensors."""
    device = torch.device(device or "cuda")
    bufs = dev_buffers if dev_buffers is not None else {}

    def dev_copy(name, t):
        if t is None:
            return None
        d = bufs.get(name)
        if d is None or d.shape != t.shape or d.dtype != t.dtype:
            d = torch.empty(t.shape, dtype=t.dtype, device=device)
            bufs[name] = d
        d.copy_(t, non_blocking=True)
        return d

    t = dev_copy("target", target_h)
    d = dev_copy("draft", draft_h)
    x = dev_copy("tokens", tokens_h)
    T = dev_copy("temperature", temperature_h)
    nd = dev_copy("num_draft", num_draft_h)
    out = verify_sample(t, d, x, T, seed, step, num_draft=nd, want_probs=False)
    host = {k: v.to("cpu", non_blocking=True) for k, v in out.items() if v is not None}
    torch.cuda.current_stream().synchronize()
    return host


# ------------------------------------------------------------------ 8-bit paged key/value cache
_attn_ws: dict[tuple[int, int], torch.Tensor] = {}
_I32, _F32 = torch.int32, torch.float32


def _on_its_stream(call):
    """What the call itself allocates and converts belongs to the stream it launches on."""
    @functools.wraps(call)
    def run(*args, stream=None, **kw):
        if stream is None:
            return call(*args, stream=None, **kw)
        with torch.cuda.stream(stream):
            return call(*args, stream=stream, **kw)
    return run


def _i32(t, device):
    """int32 and contiguous on the device; as it is where it already is that."""
    if t is None or (t.dtype is _I32 and t.is_contiguous() and t.device == device):
        return t
    return _as_i32(t, device)


def _new_attention_workspace(device: torch.device, nbytes: int) -> torch.Tensor:
    ws = torch.empty(nbytes, dtype=torch.uint8, device=device)
    ws[:binding.CACHE_ATTENTION_COUNTERS].zero_()  # the rest, some 20 MB, is written before it is read
    return ws


def _attention_workspace(device: torch.device, stream, nbytes: int) -> torch.Tensor:
    """One workspace for each device and stream: calls on one stream run in order and may
    share it, calls on two streams may not.  A call that a graph captures gets its own,
    out of the graph's memory: the graph keeps its address, and may be replayed on any
    stream, next to this one's calls and after their workspace has been replaced by a
    larger one."""
    if torch.cuda.is_current_stream_capturing():
        return _new_attention_workspace(device, nbytes)
    raw = torch._C._cuda_getCurrentRawStream(device.index) if stream is None else stream.cuda_stream
    with _ws_lock:
        ws = _attn_ws.get((device.index, raw))
        if ws is None or ws.numel() < nbytes:
            ws = _attn_ws[(device.index, raw)] = _new_attention_workspace(device, nbytes)
        return ws


def cache_attention_reset(device=None) -> None:
    """Forget the workspaces kept for cache_attention's calls on the device (None: on
    every one).  After a call that reported status 5 (an internal wait ran out) the
    later calls on its stream report it too, until this one: they get a new workspace.
    (A graph's calls zero their own in every replay.)"""
    index = None if device is None else torch.device(device).index
    if device is not None and index is None:
        index = torch.cuda.current_device()
    with _ws_lock:
        for key in [k for k in _attn_ws if index is None or k[0] == index]:
            del _attn_ws[key]


def kv_cache(num_pages: int, num_heads: int, page_size: int, head_dim: int, device="cuda") -> KVCache:
    """An empty cache: codes [num_pages, num_heads, page_size, head_dim] and scales
    [num_pages, num_heads] for keys and values.  Any tensors of that form serve (a
    token-major pool transposed to it, for instance): KVCache(k, v, k_scale, v_scale)."""
    if page_size not in binding.KV_PAGE_SIZES or head_dim % 16 or not 16 <= head_dim <= binding.KV_MAX_HEAD_DIM:
        raise ValueError(f"page_size must be one of {binding.KV_PAGE_SIZES}, head_dim a multiple of 16 of at most "
                         f"{binding.KV_MAX_HEAD_DIM}")
    codes = [torch.zeros((num_pages, num_heads, page_size, head_dim), dtype=torch.uint8, device=device) for _ in "kv"]
    scales = [torch.ones((num_pages, num_heads), dtype=torch.float32, device=device) for _ in "kv"]
    return KVCache(*(c.view(torch.float8_e4m3fn) for c in codes), *scales)


@_on_its_stream
def kv_append(cache: KVCache, k, v, page_table, cached_len, cu_new, max_new: int, stream=None) -> dict:
    """Quantise the new tokens' keys and values k, v [tokens, heads, head_dim] (bfloat16
    or float32) into the cache in place: request b's rows cu_new[b] .. cu_new[b+1] - 1
    become its positions cached_len[b] ..; max_new bounds the rows of any request.
    Returns status [B]."""
    dev = k.device
    status = torch.empty(page_table.shape[0], dtype=_I32, device=dev)
    binding.spec_kv_append(cache, k, v, _i32(page_table, dev), _i32(cached_len, dev), _i32(cu_new, dev), max_new, status,
                           stream)
    return {"status": status}


@_on_its_stream
def kv_gather(cache: KVCache, page_table, cu_out, n_out: int, first=None, dtype=torch.bfloat16, stream=None) -> dict:
    """Read the cache back: rows cu_out[b] .. cu_out[b+1] - 1 of k and v [n_out, heads,
    head_dim] are request b's positions from first[b] (None: 0).  Returns k, v, status."""
    dev = cache.k.device
    _, heads, _, dim = cache.k.shape
    k = torch.empty((n_out, heads, dim), dtype=dtype, device=dev)
    v = torch.empty((n_out, heads, dim), dtype=dtype, device=dev)
    status = torch.empty(page_table.shape[0], dtype=_I32, device=dev)
    binding.spec_kv_gather(cache, _i32(page_table, dev), _i32(cu_out, dev), _i32(first, dev), k, v, status, stream)
    return {"k": k, "v": v, "status": status}


@_on_its_stream
def cache_attention(q, cache: KVCache, page_table, seq_len, cu_query, max_query: int, scale: float | None = None,
                    window: int = 0, sinks: int = 0, want_lse: bool = False, stream=None) -> dict:
    """Attention of the new tokens' queries q [tokens, query heads, head_dim] over the
    cache, causal among the new tokens: request b's queries are rows cu_query[b] ..
    cu_query[b+1] - 1 and sit at the last of its seq_len[b] cached positions.  window
    limits each query to the last `window` positions and the first `sinks`; scale
    defaults to head_dim ** -0.5.  Returns out, lse (None unless want_lse), status; after
    a status of 5, see cache_attention_reset."""
    dev = q.device
    if dev.type != "cuda":  # before its workspace is looked up
        raise ValueError("the cache and the call's tensors must be on one CUDA device")
    n, heads, dim = q.shape
    out = torch.empty((n, heads, dim), dtype=q.dtype, device=dev)
    lse = torch.empty((n, heads), dtype=_F32, device=dev) if want_lse else None
    status = torch.empty(page_table.shape[0], dtype=_I32, device=dev)
    nbytes = binding.spec_cache_attention_workspace_size(heads, cache.k.shape[1], dim, binding._dtype_code(q))
    binding.spec_cache_attention(q, cache, _i32(page_table, dev), _i32(seq_len, dev), _i32(cu_query, dev), max_query,
                                 dim ** -0.5 if scale is None else scale, window, sinks, out, lse, status,
                                 _attention_workspace(dev, stream, nbytes), stream)
    return {"out": out, "lse": lse, "status": status}


# ------------------------------------------------------------------ prompts into the cache
def kv_pool(num_pages: int, device="cuda") -> PagePool:
    """A pool in which every page is free; page 0 is handed out last."""
    free = torch.arange(num_pages, dtype=torch.int32, device=device)
    return PagePool(free, torch.full((1,), num_pages, dtype=torch.int32, device=device))


@_on_its_stream
def kv_plan(pool: PagePool, page_table, held, keep_len, new_len, page_size: int, n_out: int, stream=None) -> dict:
    """Build the cache calls' tables on the GPU.  Request b keeps keep_len[b] cached tokens
    and gets new_len[b] more: it takes pages from the pool, or gives back those it needs no
    longer (a rejected draft's; all of them for two zeros).  pool, page_table [B, pages] and
    held [B] (int32, contiguous) are updated in place.  Returns cu_new [B + 1], seq_len [B],
    slot [n_out] (int64: page * page_size + place in it), position [n_out] and status [B];
    n_out bounds the new tokens, and rows behind the last one hold -1."""
    dev, B = page_table.device, page_table.shape[0]
    if n_out < 0:
        raise ValueError(f"n_out must not be negative, got {n_out}")
    ints = torch.empty(3 * B + 1 + n_out, dtype=_I32, device=dev)  # one allocation for what is int32
    slot = torch.empty(n_out, dtype=torch.int64, device=dev)
    at = ints.data_ptr()
    binding._plan(pool, page_table, held, _i32(keep_len, dev), _i32(new_len, dev), page_size, at, at + 4 * B + 4,
                  slot.data_ptr(), at + 12 * B + 4, at + 8 * B + 4, n_out, stream)
    cu, seq_len, status, position = ints.split_with_sizes((B + 1, B, B, n_out))
    return {"cu_new": cu, "seq_len": seq_len, "slot": slot, "position": position, "status": status}


def rotary_frequencies(rotary_dim: int, base: float = 10000.0, sections=None, interleaved: bool = False,
                       per_axis: bool = False, device="cuda"):
    """freq (float64 [rotary_dim / 2], radians a position) and axis (int32, None for one
    axis) of each pair for rotary().  sections: how many pairs each axis has, in blocks one
    after another, or by turns (interleaved: one pair of each axis that has some left).
    freq is base ** (-i / pairs) of the pair, or with per_axis base ** (-n / section) of the
    axis's n-th one.  Long contexts' scalings are changes of freq."""
    pairs = rotary_dim // 2
    parts = [pairs] if sections is None else [int(n) for n in sections]
    if rotary_dim % 2 or rotary_dim < 0 or sum(parts) != pairs or min(parts, default=0) < 0:
        raise ValueError(f"sections must sum to the {rotary_dim} // 2 pairs of columns, got {parts}")
    if interleaved:
        axis = [a for turn in range(max(parts)) for a, n in enumerate(parts) if turn < n]
    else:
        axis = [a for a, n in enumerate(parts) for _ in range(n)]
    nth, seen = [], [0] * len(parts)
    for i, a in enumerate(axis):
        nth.append(seen[a] / parts[a] if per_axis else i / pairs)
        seen[a] += 1
    freq = torch.tensor([float(base) ** -x for x in nth], dtype=torch.float64, device=device)
    return freq, None if len(parts) == 1 else torch.tensor(axis, dtype=_I32, device=device)


@_on_its_stream
def rotary(q, k, position, freq, axis=None, adjacent: bool = False, scale: float = 1.0, out_q=None, out_k=None,
           stream=None) -> dict:
    """Rotate queries q and keys k (or None) [tokens, heads, head_dim] by their positions:
    position int32 [tokens], or [axes, tokens] with the axis of each pair (see
    rotary_frequencies); a prompt of text, with one position for every axis, may expand it.
    A pair is columns (i, i + pairs), or (2 i, 2 i + 1) if adjacent; columns past the pairs
    are copied; scale multiplies what is rotated.  A pair whose frequency is infinite or NaN
    becomes NaN.  out_q and out_k may be q and k themselves (slices of a fused projection's
    output, for instance).  Returns q and k."""
    dev = q.device
    if out_q is None:
        out_q = torch.empty(q.shape, dtype=q.dtype, device=dev)
    if out_k is None and k is not None:
        out_k = torch.empty(k.shape, dtype=k.dtype, device=dev)
    binding.spec_rotary(q, k, _i32_rows(position, dev), freq, axis, adjacent, scale, out_q, out_k, stream)
    return {"q": out_q, "k": out_k}


def _i32_rows(t, device):
    """int32 on the device, with contiguous rows that are one and the same or do not overlap;
    as it is where it already is that."""
    n, strides = t.shape[-1], t.stride()
    apart = len(strides) != 2 or strides[0] == 0 or strides[0] >= n
    if t.dtype is _I32 and t.device == device and (strides[-1] == 1 or n <= 1) and apart:
        return t
    return _as_i32(t, device)


PROMPT_SPLIT_KEYS = {torch.bfloat16: 2048, torch.float32: 384}  # calls with fewer keys need no workspace


@_on_its_stream
def prompt_attention(q, k, v, cu_query, max_query: int, cu_key=None, scale: float | None = None, window: int = 0,
                     sinks: int = 0, want_lse: bool = False, stream=None) -> dict:
    """Causal attention of packed prompts: q [queries, query heads, head_dim] over k, v
    [keys, heads, head_dim]; request b's queries are rows cu_query[b] .. cu_query[b+1] - 1,
    and the last of its keys, rows cu_key[b] .. (None: the same rows).  window limits each
    query to the last `window` positions and the first `sinks`; scale defaults to
    head_dim ** -0.5.  Returns out, lse (None unless want_lse), status."""
    dev = q.device
    n, heads, dim = q.shape
    out = torch.empty((n, heads, dim), dtype=q.dtype, device=dev)
    lse = torch.empty((n, heads), dtype=_F32, device=dev) if want_lse else None
    cu_query = _i32(cu_query, dev)
    status = torch.empty(max(0, cu_query.numel() - 1), dtype=_I32, device=dev)
    ws, nbytes = None, 0
    if k.dim() == 3 and k.shape[0] >= PROMPT_SPLIT_KEYS.get(q.dtype, 0):
        nbytes = binding.spec_prompt_attention_workspace_size(n, k.shape[0], status.numel(), heads, k.shape[1], dim,
                                                              binding._dtype_code(q), window, sinks)
        if nbytes:  # from the allocator in stream order: calls share none, a graph keeps its own
            ws = torch.empty(nbytes, dtype=torch.uint8, device=dev)
    binding._prompt(q, k, v, cu_query, max_query, _i32(cu_key, dev), dim ** -0.5 if scale is None else scale, window, sinks,
                    out.data_ptr(), None if lse is None else lse.data_ptr(), status.data_ptr(),
                    None if ws is None else ws.data_ptr(), nbytes, stream)
    return {"out": out, "lse": lse, "status": status}
