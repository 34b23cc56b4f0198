"""Measured cases of the operators that take a prompt, and each later step, into the cache.

  plan    block tables on the GPU: pages of the cache are taken and given back as the
          requests' lengths change, and every new token learns its position and its slot
  rotary  queries and keys rotated by positions of one or several axes (time, height,
          width); frequencies and angles keep their bits at far positions
  prompt  causal attention of packed prompts of different lengths with grouped heads;
          optionally more keys than queries (a chunk after earlier ones), a sliding
          window with a few first tokens kept visible, and the log of the sums

`own = False` computes them with elementary torch operations in 32 bits (angles in 64);
`own = True` makes the calls of the package's public entry points.
"""
import math

import numpy as np
import torch

own = False

NEG = float("-inf")
BAD_LENGTH, NO_PAGES = 2, 7  # statuses of a planned request


# ------------------------------------------------------------------ cases
def _plan(name=None, **kw):
    c = dict(op="plan", B=1, page=64, keep_lo=0, keep_hi=0, new_lo=1, new_hi=1, leaving=0, short=0)
    c.update(kw)
    return c | ({"name": name} if name else {})


def _rotary(name=None, **kw):
    c = dict(op="rotary", T=1, Hq=32, Hkv=8, D=128, rot=128, base=1e6, sections="", interleaved=False, per_axis=False,
             adjacent=False, far=0, dtype="bf16")
    c.update(kw)
    return c | ({"name": name} if name else {})


def _prompt(name=None, **kw):
    c = dict(op="prompt", B=1, new_lo=1, new_hi=1, old_lo=0, old_hi=0, Hq=32, Hkv=8, D=128, window=0, sinks=0,
             dtype="bf16", lse=False)
    c.update(kw)
    return c | ({"name": name} if name else {})


def listed():
    return [
        # a verify round of a full batch: the anchor and seven drafts of 64 requests
        _plan("plan_round", B=64, keep_lo=100, keep_hi=8000, new_lo=8, new_hi=8),
        # thousands of requests: some leave, some enter with their prompts, small pages,
        # and the pool runs out before the last ones are served
        _plan("plan_churn", B=4096, page=16, keep_lo=0, keep_hi=2500, new_lo=1, new_hi=60, leaving=7, short=150),
        # one request's verify step: nothing but latency
        _rotary("rotary_step", T=8, far=70000),
        # prompts of text and images: axes take turns among the pairs
        _rotary("rotary_prompts", T=16411, sections="24,20,20", interleaved=True, far=30000),
        # video: a ladder of frequencies for each axis, neighbouring columns paired, fp32
        _rotary("rotary_video", T=5003, Hq=12, Hkv=12, base=1e4, sections="22,21,21", per_axis=True, adjacent=True,
                dtype="f32"),
        # one short prompt: latency
        _prompt("prompt_single", new_lo=203, new_hi=203),
        # a batch of prompts of very different lengths
        _prompt("prompt_packed", B=24, new_lo=40, new_hi=3300),
        # one long document
        _prompt("prompt_long", new_lo=24571, new_hi=24571, Hq=16, Hkv=2),
        # a model with windowed layers, small heads in groups of three
        _prompt("prompt_window", B=8, new_lo=2000, new_hi=7000, Hq=12, Hkv=4, D=64, window=1024, sinks=4),
        # chunks of two long prompts: a few hundred queries over everything before them
        _prompt("prompt_chunk", B=2, new_lo=300, new_hi=512, old_lo=30000, old_hi=60000, Hq=32, Hkv=4),
        # fp32, an odd head size and group, the statistics returned too
        _prompt("prompt_f32", B=5, new_lo=60, new_hi=1700, Hq=10, Hkv=2, D=80, dtype="f32", lse=True),
        # wide heads that all share one key head
        _prompt("prompt_wide", B=3, new_lo=300, new_hi=2500, Hq=8, Hkv=1, D=256, lse=True),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["plan", "rotary", "prompt", "prompt", "prompt"])
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    Hkv = rng.choice([1, 2, 3, 4, 8])
    G = rng.choice([1, 2, 3, 4, 5, 7, 8])
    if op == "plan":
        B = log(1, 4096)
        keep, new = log(1, 2500), min(log(1, 4000), max(1, 120000 // B))
        return _plan(B=B, page=rng.choice([16, 32, 64, 128]), keep_lo=rng.randint(0, keep), keep_hi=keep,
                     new_lo=rng.randint(0, new), new_hi=new, leaving=rng.choice([0, 0, 3, 11]),
                     short=rng.choice([0, 0, 5, 60]))
    if op == "rotary":
        D = rng.choice([64, 80, 96, 128, 256])
        rot = rng.choice([D, D, D // 2, 32])
        T = log(1, max(1, int(7e7 / ((G + 1) * Hkv * D * (2 if dtype == "f32" else 1)))))
        sections = ""
        if rng.random() < 0.6:
            a = rng.randint(1, rot // 4)
            b = rng.randint(1, rot // 4 - 1) if rng.random() < 0.7 else 0
            sections = ",".join(str(n) for n in ([rot // 2 - a - b, a] + [b] * (b > 0)))
        return _rotary(T=T, Hq=G * Hkv, Hkv=Hkv, D=D, rot=rot, base=rng.choice([1e4, 5e5, 1e6]), sections=sections,
                       interleaved=rng.random() < 0.5, per_axis=rng.random() < 0.3, adjacent=rng.random() < 0.3,
                       far=log(1, 1000000), dtype=dtype)
    D = rng.choice([64, 64, 80, 96, 128, 128, 128, 128, 192, 256])
    new = log(1, 16000 if dtype == "bf16" else 3000)
    old = log(1, 40000) if rng.random() < 0.3 else 0
    windowed = rng.random() < 0.3
    # no more work than the longest listed case, and no larger tables of scores
    most = int(min(6.4e9 / (new * (new + old) * G * Hkv), 24, 100000 / (new + old)))
    if most < 1:
        new, old, most = max(1, new // 16), old // 16, 1
    if dtype == "f32":
        new, old = min(new, 1500), min(old, 2000)
    return _prompt(B=rng.randint(1, max(1, most)), new_lo=max(1, new // rng.randint(1, 8)), new_hi=new,
                   old_lo=old // rng.randint(1, 4), old_hi=old, Hq=G * Hkv, Hkv=Hkv, D=D,
                   window=log(32, 4096) if windowed else 0, sinks=rng.randint(0, 40) if windowed else 0, dtype=dtype,
                   lse=rng.random() < 0.4)


# ------------------------------------------------------------------ inputs
def _spread(lo, hi, n, a):
    """n numbers of lo .. hi, the same for every seed, so that work() knows them."""
    i = np.arange(n, dtype=np.int64)
    return lo + (i * a + a // 3) % (hi - lo + 1) if n > 1 else np.array([hi], dtype=np.int64)


def _planned(case):
    """Tokens kept and new ones of each request in the pass's first call."""
    keep = _spread(case["keep_lo"], case["keep_hi"], case["B"], 2654435761)
    new = _spread(case["new_lo"], case["new_hi"], case["B"], 1640531513)
    gone = np.arange(case["B"]) % case["leaving"] == 1 if case["leaving"] else np.zeros(case["B"], dtype=bool)
    return keep, new, gone


def _lengths(case):
    new = _spread(case["new_lo"], case["new_hi"], case["B"], 2654435761)
    return new, new + _spread(case["old_lo"], case["old_hi"], case["B"], 1640531513)


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _frequencies(case):
    """Radians a position and the axis of each pair of columns."""
    pairs, base = case["rot"] // 2, case["base"]
    parts = [int(n) for n in case["sections"].split(",")] if case["sections"] else [pairs]
    axis = np.repeat(np.arange(len(parts)), parts)
    if case["interleaved"]:  # the axes take turns until each has its share
        turn = np.concatenate([np.arange(n) for n in parts])
        axis = axis[np.lexsort((axis, turn))]
    if case["per_axis"]:  # the n-th pair of an axis among its own
        nth = np.zeros(pairs)
        for a, n in enumerate(parts):
            nth[axis == a] = np.arange(n) / n
    else:
        nth = np.arange(pairs) / pairs
    return base ** -nth, axis.astype(np.int32), len(parts)


def _prepare_plan(case, g, dev):
    keep, new, gone = _planned(case)
    page, B = case["page"], case["B"]
    before = np.where(gone, keep + new, keep)  # what the requests hold at the start
    held = -(-before // page)
    first_keep, first_new = np.where(gone, 0, keep), np.where(gone, 0, new)
    need = -(-(first_keep + first_new) // page)
    wanted = int(np.maximum(need - held, 0).sum())
    back = int(np.maximum(held - need, 0).sum())
    spare = max(1, wanted - back) if not case["short"] else max(0, wanted - back - case["short"])
    width = int(max(need.max(), held.max())) + 1
    P = int(held.sum()) + spare + 1
    order = torch.randperm(P, generator=g, device=dev).to(torch.int32)
    start = np.concatenate([[0], np.cumsum(held)[:-1]])
    at = np.minimum(start[:, None] + np.arange(width)[None, :], P - 1)
    owns = np.arange(width)[None, :] < held[:, None]
    table = torch.where(torch.from_numpy(owns).to(dev), order[torch.from_numpy(at).to(dev)], -1).contiguous()
    free = torch.full((P,), -1, dtype=torch.int32, device=dev)
    n = int(held.sum())
    free[:spare] = order[n:n + spare]

    def i32(a):
        return torch.from_numpy(np.asarray(a).astype(np.int32)).to(dev)

    # the first call serves the requests; the second one gives everything back, and lets
    # those that left enter again, so that every pass finds the same lengths
    return dict(case=case, table=table, held=i32(held), free=free, count=i32([spare]), n_out=int(first_new.sum()),
                n_back=int(np.where(gone, before, 0).sum()), keep=i32(first_keep), new=i32(first_new),
                keep_back=i32(np.where(gone, 0, keep)), new_back=i32(np.where(gone, before, 0)))


def _prepare_rotary(case, g, dev):
    T, Hq, Hkv, D = case["T"], case["Hq"], case["Hkv"], case["D"]
    freq, axis, axes = _frequencies(case)
    # slices of a fused projection's output, as a layer has them
    wide = torch.randn((T, Hq + 2 * Hkv, D), generator=g, device=dev).to(_dtype(case))
    t = torch.arange(T, device=dev)
    if axes == 1:
        pos = (t + case["far"])[None]
    else:  # a picture's or a film's grid, after earlier text
        side = int(max(2, math.isqrt(T) // 3))
        grid = [t // (side * side), t // side % side, t % side][:axes]
        pos = torch.stack(grid) + case["far"]
    jump = torch.randint(0, 50, (1,), generator=g, device=dev)
    return dict(case=case, q=wide[:, :Hq], k=wide[:, Hq:Hq + Hkv], pos=(pos + jump).to(torch.int32).contiguous(),
                freq=torch.from_numpy(freq).to(dev), axis=torch.from_numpy(axis).to(dev))


def _prepare_prompt(case, g, dev):
    new, total = _lengths(case)
    Hq, Hkv, D, dt = case["Hq"], case["Hkv"], case["D"], _dtype(case)
    cu_q = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    cu_k = np.concatenate([[0], np.cumsum(total)]).astype(np.int32)
    T, L = int(cu_q[-1]), int(cu_k[-1])
    channel = torch.exp(0.5 * torch.randn((1, Hkv, D), generator=g, device=dev))  # some channels are large
    q = (1.2 * torch.randn((T, Hq, D), generator=g, device=dev)).to(dt)
    k = (torch.randn((L, Hkv, D), generator=g, device=dev) * channel).to(dt)
    v = torch.randn((L, Hkv + 1, D), generator=g, device=dev).to(dt)[:, :Hkv]  # a slice of a wider product
    return dict(case=case, q=q, k=k, v=v, cu_q=torch.from_numpy(cu_q).to(dev), cu_k=torch.from_numpy(cu_k).to(dev),
                T=T, L=L, max_new=int(new.max()), max_total=int(total.max()))


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    return {"plan": _prepare_plan, "rotary": _prepare_rotary, "prompt": _prepare_prompt}[case["op"]](case, g, dev)


# ------------------------------------------------------------------ plain forms
def _plain_plan_call(st, keep, new, n_out):
    page = st["case"]["page"]
    table, held, free, count = st["table"], st["held"], st["free"], st["count"]
    W, total = table.shape[1], keep + new
    cu = torch.cat([torch.zeros_like(count), new.clamp(min=0).cumsum(0).to(torch.int32)])
    bad = (keep < 0) | (new < 0) | (total > W * page) | (keep > held * page) | (cu[1:] > n_out)
    need = torch.where(bad, held, (total + page - 1) // page)
    take = (need - held).clamp(min=0)
    i = torch.arange(W, device=table.device)
    leaves = (i >= need[:, None]) & (i < held[:, None])
    back = table[leaves]
    top = count[0].long()
    free[top + torch.arange(back.numel(), device=table.device)] = back
    table[leaves] = -1
    top = top + back.numel()
    refused = (take.cumsum(0) > top) & (take > 0)
    need = torch.where(refused, held, need)
    enters = (i >= held[:, None]) & (i < need[:, None])
    n = enters.sum()
    nth = enters.flatten().cumsum(0).view_as(enters) - 1
    got = free[(top - n + nth).clamp(min=0)]
    table.copy_(torch.where(enters, got, table))
    held.copy_(need)
    count.copy_((top - n).to(torch.int32)[None])
    status = torch.where(bad, BAD_LENGTH, torch.where(refused, NO_PAGES, 0)).to(torch.int32)
    r = torch.arange(n_out, device=table.device)
    b = torch.searchsorted(cu[1:].contiguous(), r, right=True, out_int32=True).long()
    inside = r < cu[-1]
    b = b.clamp(max=keep.numel() - 1)
    position = torch.where(inside, keep[b] + r - cu[b], -1).to(torch.int32)
    p = table[b, (position // page).clamp(min=0, max=W - 1).long()].long()
    slot = torch.where(inside & (status[b] == 0), p * page + position % page, -1)
    return dict(cu_new=cu, seq_len=torch.where(status == 0, total, keep), slot=slot, position=position, status=status)


def _plain_plan(st):
    got = _plain_plan_call(st, st["keep"], st["new"], st["n_out"])
    back = _plain_plan_call(st, st["keep_back"], st["new_back"], st["n_back"])
    return dict(got=got, back=back, table=st["table"], held=st["held"], count=st["count"])


def _plain_rotary(st):
    case, R = st["case"], st["case"]["rot"]
    angle = st["pos"][st["axis"].long()].T.double() * st["freq"]  # [T, pairs]
    c, s = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def turn(x):
        y = x.float()
        if case["adjacent"]:
            a, b = y[..., 0:R:2], y[..., 1:R:2]
            turned = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
        else:
            a, b = y[..., :R // 2], y[..., R // 2:R]
            turned = torch.cat([a * c - b * s, b * c + a * s], -1)
        return torch.cat([turned, y[..., R:]], -1).to(x.dtype)

    return dict(q=turn(st["q"]), k=turn(st["k"]))


def _plain_prompt(st):
    case, q = st["case"], st["q"]
    dev, D, H, W = q.device, case["D"], case["Hkv"], case["window"]
    G, N, L = case["Hq"] // H, st["max_new"], st["max_total"]
    cu_q, cu_k = st["cu_q"].long(), st["cu_k"].long()
    n, m = cu_q[1:] - cu_q[:-1], cu_k[1:] - cu_k[:-1]
    B = n.numel()
    t, j = torch.arange(N, device=dev), torch.arange(L, device=dev)
    pos = (m - n)[:, None, None] + t[:, None]  # [B, N, 1]
    seen = (j <= pos) & (t[:, None] < n[:, None, None])
    if W:
        seen &= (j > pos - W) | (j < case["sinks"])
    at = (cu_k[:-1, None] + j).clamp(max=st["L"] - 1)
    K, V = st["k"][at].float(), st["v"][at].float()  # [B, L, H, D]
    Q = q[(cu_q[:-1, None] + t).clamp(max=st["T"] - 1)].float()
    Q = Q.view(B, N, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * N, D)
    s = torch.matmul(Q, K.permute(0, 2, 3, 1)).mul_(D ** -0.5).view(B, H, G, N, L)
    s.masked_fill_(~seen[:, None, None], NEG)
    top = s.amax(-1, keepdim=True)
    top = torch.where(top == NEG, 0.0, top)
    p = s.sub_(top).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, H, G * N, L), V.transpose(1, 2)).view(B, H, G, N, D) / torch.where(l == 0, 1.0, l)
    r = torch.arange(st["T"], device=dev)
    b = torch.searchsorted(cu_q[1:].contiguous(), r, right=True)
    t = r - cu_q[b]
    out = {"out": o[b, :, :, t].reshape(st["T"], H * G, D).to(q.dtype)}
    if case["lse"]:
        out["lse"] = (top + l.log())[b, :, :, t].reshape(st["T"], H * G)
    return out


def run(st):
    case, op = st["case"], st["case"]["op"]
    if not own:
        return {"plan": _plain_plan, "rotary": _plain_rotary, "prompt": _plain_prompt}[op](st)
    import speculative_decoding_verification_15_gb300 as pkg

    if op == "plan":
        pool = pkg.PagePool(st["free"], st["count"])

        def call(keep, new, n_out):
            return pkg.kv_plan(pool, st["table"], st["held"], keep, new, case["page"], n_out)

        got = call(st["keep"], st["new"], st["n_out"])
        back = call(st["keep_back"], st["new_back"], st["n_back"])
        return dict(got=got, back=back, table=st["table"], held=st["held"], count=st["count"])
    if op == "rotary":
        return pkg.rotary(st["q"], st["k"], st["pos"], st["freq"], axis=st["axis"], adjacent=case["adjacent"])
    chunk = dict(cu_key=st["cu_k"]) if case["old_hi"] else {}
    got = pkg.prompt_attention(st["q"], st["k"], st["v"], st["cu_q"], st["max_new"], **chunk, window=case["window"],
                               sinks=case["sinks"], want_lse=case["lse"])
    return {"out": got["out"], "lse": got["lse"]} if case["lse"] else {"out": got["out"]}


# ------------------------------------------------------------------ work
def _pairs(case):
    """Visible (query, key) pairs of one head, and the keys that some query sees."""
    pairs = held = 0
    for n, m in zip(*(x.tolist() for x in _lengths(case))):
        pos = np.arange(m - n, m, dtype=np.int64)
        low = np.maximum(pos - case["window"] + 1, 0) if case["window"] else np.zeros_like(pos)
        sinks = np.minimum(case["sinks"], low) if case["window"] else low
        pairs += int((pos + 1 - low + sinks).sum())
        held += int(m - low[0] + sinks[0])
    return pairs, held


def work(case):
    if case["op"] == "plan":
        keep, new, gone = _planned(case)
        before = np.where(gone, keep + new, keep)
        first = np.where(gone, 0, keep + new)
        moved = int(np.abs(-(-before // case["page"]) + -first // case["page"]).sum())
        rows = int(np.where(gone, 0, new).sum()) + int(np.where(gone, before, 0).sum())
        # both calls: lengths and counts in, counts, offsets, lengths and statuses out;
        # a page's id from one list to the other; a slot and a position for each token
        return {"bytes": 2 * 4 * case["B"] * 7 + 2 * 8 * moved + 12 * rows, "flops": 2 * 10 * case["B"] + 4 * rows}
    esz = 2 if case["dtype"] == "bf16" else 4
    if case["op"] == "rotary":
        columns = case["T"] * (case["Hq"] + case["Hkv"])
        axes = len(case["sections"].split(","))
        return {"bytes": 2 * columns * case["D"] * esz + 4 * case["T"] * axes + 6 * case["rot"], "flops": 3 * columns * case["rot"]}
    pairs, held = _pairs(case)
    T = int(_lengths(case)[0].sum())
    return {"bytes": 2 * T * case["Hq"] * case["D"] * esz + 2 * held * case["Hkv"] * case["D"] * esz +
                     (4 * T * case["Hq"] if case["lse"] else 0),
            "flops": 4 * pairs * case["Hq"] * case["D"]}


# ------------------------------------------------------------------ in 64 bits
def _exact_rotary(case, st):
    """Pairs of columns as complex numbers, times exp(i angle)."""
    pos, freq, axis = (st[n].cpu().numpy() for n in ("pos", "freq", "axis"))
    turn = np.exp(1j * (pos.astype(np.float64)[axis] * freq[:, None]).T)[:, None, :]
    half, R, res = case["rot"] // 2, case["rot"], {}
    one, other = (slice(0, R, 2), slice(1, R, 2)) if case["adjacent"] else (slice(0, half), slice(half, R))
    for name in ("q", "k"):
        x = st[name].double().cpu().numpy().copy()
        z = (x[:, :, one] + 1j * x[:, :, other]) * turn
        x[:, :, one], x[:, :, other] = z.real, z.imag
        res[name] = x
    return res


def _exact_prompt(case, st):
    new, total = _lengths(case)
    if 4 * float((new * total).sum()) * case["Hq"] * case["D"] > 6e12:
        return None
    dev, D, G, W = st["q"].device, case["D"], case["Hq"] // case["Hkv"], case["window"]
    out = torch.zeros(st["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.zeros(st["q"].shape[:2], dtype=torch.float64, device=dev)
    a = c = 0
    for n, m in zip(new.tolist(), total.tolist()):
        i = torch.arange(m - n, m, device=dev)[:, None]
        j = torch.arange(m, device=dev)[None, :]
        hidden = j > i
        if W:
            hidden |= (j <= i - W) & (j >= case["sinks"])
        for h in range(case["Hq"]):
            x = st["q"][a:a + n, h].double() @ st["k"][c:c + m, h // G].double().T
            x = (x / math.sqrt(D)).masked_fill(hidden, NEG)
            total_log = torch.logsumexp(x, 1)
            lse[a:a + n, h] = total_log
            out[a:a + n, h] = torch.exp(x - total_log[:, None]) @ st["v"][c:c + m, h // G].double()
        a, c = a + n, c + m
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}


def exact(case, seed):
    if case["op"] == "plan":
        return None  # whole numbers
    st = prepare(case, seed)
    return _exact_rotary(case, st) if case["op"] == "rotary" else _exact_prompt(case, st)
