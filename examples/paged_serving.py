"""Prompts into the 8-bit paged cache and speculative rounds after them, with pages handed
out on the GPU.

The toy target of cached_verify.py, with rotary positions:
  1. kv_plan gives the prompts their pages, positions and offsets,
  2. rotary turns their queries and keys in place, prompt_attention attends, kv_append
     writes the cache; the last tokens' logits give the first anchors;
  3. each round plans K + 1 tokens a request (the pages of rejected drafts are reused or go
     back), turns, appends, attends over the cache, verifies, and advances;
  4. requests that end give their pages back.
Between the prompts and the end nothing is read by the host but the tokens it keeps.

    python examples/paged_serving.py [--rounds 8] [--batch 8] [--drafts 5]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path[:0] = [os.path.dirname(os.path.abspath(__file__)), os.path.dirname(os.path.dirname(os.path.abspath(__file__)))]

import speculative_decoding_verification_15_gb300 as spec  # noqa: E402
from cached_verify import Target  # noqa: E402


def run(rounds=8, batch=8, drafts=5, vocab=1000, heads=8, kv_heads=2, head_dim=64, page_size=16, max_len=512,
        temperature=0.8, window=0, sinks=0, longest=200, seed=0, device="cuda"):
    """Returns the committed tokens of every request, the target, the cache, the tables and
    the pool; the requests of even number have ended."""
    g = torch.Generator(device=device).manual_seed(seed + 1)
    target = Target(vocab, heads, kv_heads, head_dim, device, seed)
    width = -(-max_len // page_size)
    num_pages = batch * width
    cache, pool = spec.kv_cache(num_pages, kv_heads, page_size, head_dim, device), spec.kv_pool(num_pages, device)
    table = torch.full((batch, width), -1, dtype=torch.int32, device=device)
    held = torch.zeros(batch, dtype=torch.int32, device=device)
    none = torch.zeros_like(held)
    freq, _ = spec.rotary_frequencies(head_dim, device=device)
    mask = dict(window=window, sinks=sinks)

    lengths = torch.randint(3, longest, (batch,), generator=g, device=device).to(torch.int32)
    total, most = int(lengths.sum()), int(lengths.max())
    prompt = torch.randint(0, vocab, (total,), generator=g, device=device)
    text = [p.tolist() for p in prompt.split(lengths.tolist())]
    plan = spec.kv_plan(pool, table, held, none, lengths, page_size, total)
    x, q, k, v = target.projections(prompt)
    spec.rotary(q, k, plan["position"], freq, out_q=q, out_k=k)
    att = spec.prompt_attention(q, k, v, plan["cu_new"], most, **mask)
    wrote = spec.kv_append(cache, k, v, table, none, plan["cu_new"], most)
    ok = plan["status"] | att["status"] | wrote["status"]
    last = plan["cu_new"][1:].long() - 1
    anchor = target.logits(x[last], att["out"][last]).argmax(-1)
    cached = plan["seq_len"].clone()
    kept = [anchor[:, None].to(torch.int32)]

    new = torch.full_like(held, drafts + 1)
    temps = torch.full((batch,), float(temperature), device=device)
    accepted_all = []
    for step in range(rounds):
        tokens, draft_logits = [anchor], []
        for _ in range(drafts):
            z = target.logits(target.emb[tokens[-1]])
            draft_logits.append(z)
            noise = -torch.log(-torch.log(torch.rand(z.shape, generator=g, device=device).clamp(1e-9, 1 - 1e-7)))
            tokens.append((z / max(temperature, 1e-6) + (noise if temperature > 0 else 0)).argmax(-1))
        block = torch.stack(tokens, 1)
        plan = spec.kv_plan(pool, table, held, cached, new, page_size, batch * (drafts + 1))
        x, q, k, v = target.projections(block.reshape(-1))
        spec.rotary(q, k, plan["position"], freq, out_q=q, out_k=k)
        wrote = spec.kv_append(cache, k, v, table, cached, plan["cu_new"], drafts + 1)
        att = spec.cache_attention(q, cache, table, plan["seq_len"], plan["cu_new"], drafts + 1, **mask)
        logits = target.logits(x, att["out"]).view(batch, drafts + 1, vocab)
        got = spec.verify_sample(logits, torch.stack(draft_logits, 1), block[:, 1:], temps, seed=seed, step=step)
        ok = ok | plan["status"] | wrote["status"] | att["status"] | got["status"]
        cached = cached + got["accepted"] + 1
        anchor = got["tokens"].gather(1, got["accepted"][:, None].long())[:, 0].long()
        kept.append(got["tokens"])
        accepted_all.append(got["accepted"])
    # every other request ends; the others give back what their last round did not need
    ended = torch.arange(batch, device=device) % 2 == 0
    plan = spec.kv_plan(pool, table, held, torch.where(ended, 0, cached), none, page_size, 0)
    ok = ok | plan["status"]
    if int(ok.abs().max()):
        raise RuntimeError(f"a request failed: statuses {ok.tolist()}")
    for rows in kept:
        for b, row in enumerate(rows.tolist()):
            text[b] += [t for t in row if t >= 0]
    return dict(text=text, target=target, cache=cache, table=table, held=held, pool=pool, cached=cached, freq=freq,
                ended=ended, prompts=lengths, accepted=float(torch.stack(accepted_all).float().mean()) if rounds else 0.0)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rounds", type=int, default=8)
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--drafts", type=int, default=5)
    a = ap.parse_args()
    got = run(a.rounds, a.batch, a.drafts)
    print(f"{a.rounds} rounds, {a.batch} requests: {got['accepted']:.2f} of {a.drafts} drafts accepted a round; "
          f"{int(got['cached'].sum())} tokens cached, {int(got['pool'].count)} pages free after half of them ended")


if __name__ == "__main__":
    main()
