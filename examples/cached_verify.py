"""Speculative decoding rounds over the 8-bit paged cache, as a serving loop makes them.

A toy target (one attention layer over an embedding, random weights) and a cheap draft
(the target without its attention) decode a batch of requests.  Each round
  1. drafts K tokens a request,
  2. appends the keys and values of the anchor and the drafts to the cache,
  3. runs the target's attention over everything cached,
  4. verifies the drafts against the target's logits,
  5. advances the cached length by accepted + 1: the rejected drafts' slots are written
     again by the next round.

    python examples/cached_verify.py [--rounds 8] [--batch 8] [--drafts 5]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import speculative_decoding_verification_15_gb300 as spec  # noqa: E402


class Target:
    def __init__(self, vocab, heads, kv_heads, head_dim, device, seed=0):
        g = torch.Generator(device=device).manual_seed(seed)
        width = heads * head_dim
        self.heads, self.kv_heads, self.head_dim = heads, kv_heads, head_dim

        def normal(*shape, scale):
            return (torch.randn(shape, generator=g, device=device) * scale).to(torch.bfloat16)

        self.emb = normal(vocab, width, scale=1.0)
        self.qkv = normal(width, (heads + 2 * kv_heads) * head_dim, scale=width ** -0.5)
        self.out = normal(width, width, scale=2 * width ** -0.5)
        self.head = normal(vocab, width, scale=2 * width ** -0.5)

    def projections(self, tokens):
        """q, k, v [tokens, heads, head_dim]: slices of one product, not copied."""
        x = self.emb[tokens]
        y = (x @ self.qkv).view(len(tokens), self.heads + 2 * self.kv_heads, self.head_dim)
        return x, y[:, :self.heads], y[:, self.heads:self.heads + self.kv_heads], y[:, self.heads + self.kv_heads:]

    def logits(self, x, attended=None):
        h = x if attended is None else x + attended.reshape(len(x), -1) @ self.out
        return (h @ self.head.T).float()


def run(rounds=8, batch=8, drafts=5, vocab=1000, heads=8, kv_heads=2, head_dim=64, page_size=16, max_len=512,
        temperature=0.8, window=0, sinks=0, seed=0, device="cuda"):
    """Returns the committed tokens of every request, the target, the cache and its table."""
    g = torch.Generator(device=device).manual_seed(seed + 1)
    target = Target(vocab, heads, kv_heads, head_dim, device, seed)
    pages = -(-max_len // page_size)
    cache = spec.kv_cache(batch * pages, kv_heads, page_size, head_dim, device)
    table = torch.randperm(batch * pages, generator=g, device=device).to(torch.int32).view(batch, pages)

    # prompts of ragged lengths enter the empty cache; their last token is the first anchor
    lengths = torch.randint(3, 40, (batch,), generator=g, device=device)
    prompt = torch.randint(0, vocab, (int(lengths.sum()),), generator=g, device=device)
    text = [p.tolist() for p in prompt.split(lengths.tolist())]
    cached = (lengths - 1).to(torch.int32)
    body = torch.cat([torch.tensor(t[:-1], device=device) for t in text]).long()
    cu = torch.cat([torch.zeros(1, device=device), cached.cumsum(0)]).to(torch.int32)
    _, _, k, v = target.projections(body)
    ok = spec.kv_append(cache, k, v, table, torch.zeros_like(cached), cu, int(cached.max()))["status"]
    anchor = torch.tensor([t[-1] for t in text], device=device)

    cu_step = torch.arange(batch + 1, device=device, dtype=torch.int32) * (drafts + 1)
    temps = torch.full((batch,), float(temperature), device=device)
    accepted_total = 0
    for step in range(rounds):
        tokens, draft_logits = [anchor], []
        for _ in range(drafts):
            z = target.logits(target.emb[tokens[-1]])
            draft_logits.append(z)
            noise = -torch.log(-torch.log(torch.rand(z.shape, generator=g, device=device).clamp(1e-9, 1 - 1e-7)))
            tokens.append((z / max(temperature, 1e-6) + (noise if temperature > 0 else 0)).argmax(-1))
        block = torch.stack(tokens, 1)  # [batch, drafts + 1]: the anchor and its drafts
        x, q, k, v = target.projections(block.reshape(-1))
        ok = ok | spec.kv_append(cache, k, v, table, cached, cu_step, drafts + 1)["status"]
        att = spec.cache_attention(q, cache, table, cached + (drafts + 1), cu_step, drafts + 1, window=window, sinks=sinks)
        logits = target.logits(x, att["out"]).view(batch, drafts + 1, vocab)
        got = spec.verify_sample(logits, torch.stack(draft_logits, 1), block[:, 1:], temps, seed=seed, step=step)
        ok = ok | att["status"] | got["status"]
        accepted = got["accepted"]
        cached = cached + accepted + 1
        anchor = got["tokens"].gather(1, accepted[:, None].long())[:, 0].long()
        for b, (n, row) in enumerate(zip(accepted.tolist(), got["tokens"].tolist())):
            text[b] += row[:n + 1]
            accepted_total += n
    if int(ok.abs().max()):
        raise RuntimeError(f"a request failed: statuses {ok.tolist()}")
    return dict(text=text, target=target, cache=cache, table=table, cached=cached,
                accepted=accepted_total / (rounds * batch))


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--rounds", type=int, default=8)
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--drafts", type=int, default=5)
    a = ap.parse_args()
    got = run(a.rounds, a.batch, a.drafts)
    print(f"{a.rounds} rounds, {a.batch} requests: {got['accepted']:.2f} of {a.drafts} drafts accepted a round; "
          f"{int(got['cached'].sum())} tokens cached")


if __name__ == "__main__":
    main()
