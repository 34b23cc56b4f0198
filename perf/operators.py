"""Measured cases of the 8-bit paged key/value cache operators.

The verify step scores K + 1 positions of every request with the target model, and what
that forward pass reads is the cache of keys and values.  Three operators share one
paged cache whose entries are e4m3 codes with one power-of-two scale for each page and
head:

  append     quantises the keys and values of the new tokens as they are written; the
             tokens a page already holds are rescaled when the page's scale grows
  attention  the new tokens' queries against everything cached (causal among the new
             tokens; optionally a sliding window with a few first tokens kept visible)
  gather     reads ranges of the cache back as bf16 or fp32 values

`own = False` computes them with elementary torch operations in 32 bits; `own = True`
makes the calls of the package's public entry points.
"""
import math

import numpy as np
import torch

own = False

EXP_MIN, EXP_MAX = -100, 119  # exponents a page's scale may take
NEG = float("-inf")


# ------------------------------------------------------------------ cases
def _case(op, name=None, **kw):
    c = dict(op=op, B=1, new_lo=1, new_hi=1, len_lo=0, len_hi=0, Hq=8, Hkv=8, D=128, page=64, window=0, sinks=0,
             dtype="bf16", lse=False)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one request decoding one token at a time: nothing but latency
        _case("append", "append_single", B=1, len_lo=777, len_hi=777),
        # the verify step of a full batch: the anchor and seven drafts of 64 requests
        _case("append", "append_verify", B=64, new_lo=8, new_hi=8, len_lo=100, len_hi=1000),
        # prompts entering an empty cache, of ragged lengths, fp32 activations
        _case("append", "append_prompts", B=6, new_lo=700, new_hi=8000, Hkv=4, D=96, page=32, dtype="f32"),
        # one request, one token, a short context: latency again
        _case("attention", "attend_single", B=1, len_lo=1003, len_hi=1003, Hq=32),
        # the verify step of the main batch: 64 requests, seven drafts and the anchor
        _case("attention", "attend_verify", B=64, new_lo=8, new_hi=8, len_lo=500, len_hi=8000, Hq=32),
        # scheduled verify lengths: 256 requests that verify one to eight tokens each,
        # small heads and small pages
        _case("attention", "attend_ragged", B=256, new_lo=1, new_hi=8, len_lo=60, len_hi=3000, Hq=16, Hkv=4, D=64,
              page=16),
        # two long documents, single tokens, eight query heads to a key head
        _case("attention", "attend_long", B=2, len_lo=120000, len_hi=131071, Hq=64, page=128),
        # a model with windowed layers: 32 requests deep into their contexts
        _case("attention", "attend_window", B=32, new_lo=8, new_hi=8, len_lo=9000, len_hi=24000, Hq=24, page=32,
              window=1024, sinks=4),
        # fp32 queries, an odd head size and an odd group, the statistics returned too
        _case("attention", "attend_f32", B=9, new_lo=1, new_hi=5, len_lo=40, len_hi=1500, Hq=10, Hkv=2, D=80, page=16,
              dtype="f32", lse=True),
        # the end of a few requests' caches read back for inspection
        _case("gather", "gather_tails", B=3, new_lo=50, new_hi=200, len_lo=300, len_hi=900, Hkv=2, D=64, page=16,
              dtype="f32"),
        # whole prompts' caches read back for a model that takes bf16
        _case("gather", "gather_prompts", B=16, new_lo=2000, new_hi=8000, len_lo=0, len_hi=300),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["append", "attention", "attention", "attention", "gather"])
    D = rng.choice([64, 64, 80, 96, 128, 128, 128])
    page = rng.choice([16, 32, 64, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    if op == "attention":
        length = log(16, 131071)
        most = max(1, min(256, int(2.0e8 / (length * Hkv * D))))  # no larger than the listed cases' caches
        B = log(1, most)
        dtype = "f32" if rng.random() < 0.15 else "bf16"
        if dtype == "f32":
            length = min(length, 4000)
        new = rng.randint(1, 8)
        windowed = rng.random() < 0.3
        return _case(op, B=B, new_lo=rng.randint(1, new), new_hi=new, len_lo=max(1, length // rng.randint(1, 8)),
                     len_hi=length, Hq=Hkv * rng.choice([1, 2, 3, 4, 5, 8]), Hkv=Hkv, D=D, page=page,
                     window=log(32, 4096) if windowed else 0, sinks=rng.randint(0, 40) if windowed else 0, dtype=dtype,
                     lse=dtype == "f32" and rng.random() < 0.5)
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "append" and rng.random() < 0.5:
        return _case(op, B=log(1, 256), new_lo=1, new_hi=rng.randint(1, 8), len_lo=0, len_hi=log(1, 1000), Hkv=Hkv, D=D,
                     page=page, dtype=dtype)
    new = log(9, 8000)
    most = max(1, min(64, int((1.2e7 if op == "append" else 6e7) / (new * Hkv * D))))
    return _case(op, B=log(1, most), new_lo=max(1, new // 5), new_hi=new, len_lo=0, len_hi=log(1, 500), Hkv=Hkv, D=D,
                 page=page, dtype=dtype)


# ------------------------------------------------------------------ inputs
def _lengths(case):
    """New tokens and tokens already cached, per request: set by the case alone, so that
    work() knows them; the values and the pages' order come from the seed."""
    i = np.arange(case["B"], dtype=np.int64)
    def spread(lo, hi, a):
        return lo + (i * a + a // 3) % (hi - lo + 1) if case["B"] > 1 else np.array([hi])
    return spread(case["new_lo"], case["new_hi"], 2654435761), spread(case["len_lo"], case["len_hi"], 1640531513)


def _positions(case):
    new, old = _lengths(case)
    return new, old, old + new


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(int(seed))
    new, old, total = _positions(case)
    B, H, D, bs = case["B"], case["Hkv"], case["D"], case["page"]
    pages = (total + bs - 1) // bs
    width = int(pages.max())
    P = int(pages.sum()) + 3
    order = torch.randperm(P, generator=g, device=dev).to(torch.int32)
    first = np.concatenate([[0], np.cumsum(pages)[:-1]])
    at = np.minimum(first[:, None] + np.arange(width)[None, :], P - 1)
    held = np.arange(width)[None, :] < pages[:, None]
    table = torch.where(torch.from_numpy(held).to(dev), order[torch.from_numpy(at).to(dev)], -1).contiguous()

    # what an earlier run wrote: per page and head a scale, and codes that fill its range;
    # some channels of the keys are much larger than others, as trained models' are
    def contents(outliers):
        codes = torch.empty((P, H, bs, D), dtype=torch.float8_e4m3fn, device=dev)
        scale = torch.empty((P, H), dtype=torch.float32, device=dev)
        channel = torch.exp(0.8 * torch.randn((1, H, 1, D), generator=g, device=dev)) if outliers else 1.0
        step = max(1, (1 << 26) // (H * bs * D))
        for p in range(0, P, step):
            x = torch.randn((min(step, P - p), H, bs, D), generator=g, device=dev) * channel
            s = _scale_of(x.abs().amax(dim=(2, 3)))
            codes[p:p + step] = (x / s[:, :, None, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
            scale[p:p + step] = s
        return codes, scale, channel

    k, k_scale, channel = contents(True)
    v, v_scale, _ = contents(False)
    cu = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    T = int(cu[-1])
    st = dict(case=case, k=k, v=v, k_scale=k_scale, v_scale=v_scale, table=table, T=T, width=width,
              cu=torch.from_numpy(cu).to(dev), old=torch.from_numpy(old.astype(np.int32)).to(dev),
              total=torch.from_numpy(total.astype(np.int32)).to(dev), max_new=int(new.max()), max_total=int(total.max()))
    dt = _dtype(case)
    if case["op"] == "append":
        # the scales of the new tokens wander, so that some pages' scales grow
        wander = torch.exp(0.5 * torch.randn((T, H, 1), generator=g, device=dev))
        st["new_k"] = (torch.randn((T, H, D), generator=g, device=dev) * wander * channel[:, :, 0]).to(dt)
        st["new_v"] = (torch.randn((T, H, D), generator=g, device=dev) * wander).to(dt)
    elif case["op"] == "attention":
        st["q"] = (1.2 * torch.randn((T, case["Hq"], D), generator=g, device=dev)).to(dt)
    return st


# ------------------------------------------------------------------ plain forms
def _scale_of(amax):
    """The smallest power of two 2^e with amax <= 448 * 2^e (e within its limits)."""
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(amax > 0, e, EXP_MIN).clamp(EXP_MIN, EXP_MAX)
    return torch.ldexp(torch.ones_like(amax), e)


def _plain_append_one(st, codes, scale, x):
    case = st["case"]
    bs, old, cu = case["page"], st["old"].long(), st["cu"].long()
    n = cu[1:] - cu[:-1]
    J = (st["max_new"] + bs - 2) // bs + 1
    page_at = old[:, None] // bs + torch.arange(J, device=x.device)  # [B, J] touched pages of each request
    b, j = torch.nonzero(page_at * bs < (old + n)[:, None], as_tuple=True)
    at = page_at[b, j]
    page = st["table"][b, at].long()
    pos = at[:, None] * bs + torch.arange(bs, device=x.device)  # [U, bs]
    kept = pos < old[b, None]
    fresh = ~kept & (pos < (old + n)[b, None])
    row = (cu[b, None] + pos - old[b, None]).clamp(0, st["T"] - 1)
    val = x[row].float().transpose(1, 2)  # [U, H, bs, D]
    val = torch.where(fresh[:, None, :, None], val, 0.0)
    before = codes.view(torch.uint8)[page].view(torch.float8_e4m3fn)
    want = _scale_of(val.abs().amax(dim=(2, 3)))
    had = scale[page]
    s = torch.where(kept.any(dim=1)[:, None], torch.maximum(want, had), want)
    again = before.float() * (had / s)[:, :, None, None]
    new = torch.where(fresh[:, None, :, None], (val / s[:, :, None, None]).clamp(-448, 448), again)
    out = new.to(torch.float8_e4m3fn).view(torch.uint8)
    touched = (kept | fresh)[:, None, :, None]
    codes.view(torch.uint8)[page] = torch.where(touched, out, before.view(torch.uint8))
    scale[page] = s


def _plain_append(st):
    _plain_append_one(st, st["k"], st["k_scale"], st["new_k"])
    _plain_append_one(st, st["v"], st["v_scale"], st["new_v"])
    return {"k": st["k"], "v": st["v"], "k_scale": st["k_scale"], "v_scale": st["v_scale"]}


def _read(codes, scale, page, slot):
    """Cached values [..., H, D] in fp32 at pages and slots of equal shape."""
    c = codes.view(torch.uint8).transpose(1, 2)[page, slot].view(torch.float8_e4m3fn)
    return c.float() * scale[page].unsqueeze(-1)


def _plain_gather(st):
    bs, dt = st["case"]["page"], _dtype(st["case"])
    r = torch.arange(st["T"], device=st["k"].device)
    b = torch.searchsorted(st["cu"][1:].long(), r, right=True)
    pos = r - st["cu"].long()[b] + st["old"].long()[b]
    page, slot = st["table"][b, pos // bs].long(), pos % bs
    return {"k": _read(st["k"], st["k_scale"], page, slot).to(dt), "v": _read(st["v"], st["v_scale"], page, slot).to(dt)}


def _plain_attention(st):
    case, q = st["case"], st["q"]
    dev, bs, D, H = q.device, case["page"], case["D"], case["Hkv"]
    G, N, W = case["Hq"] // H, st["max_new"], case["window"]
    cu, total = st["cu"].long(), st["total"].long()
    n = cu[1:] - cu[:-1]
    B = n.numel()
    t = torch.arange(N, device=dev)
    pos = (total - n)[:, None] + t  # [B, N] positions of the queries
    if W:
        near = torch.arange(W + N - 1, device=dev) + (total - n - W + 1)[:, None]
        col = torch.cat([torch.arange(case["sinks"], device=dev).expand(B, -1), near], 1)  # [B, L]
        once = torch.cat([torch.ones((B, case["sinks"]), dtype=torch.bool, device=dev), near >= case["sinks"]], 1)
    else:
        col = torch.arange(st["max_total"], device=dev).expand(B, -1)
        once = torch.ones_like(col, dtype=torch.bool)
    c = col[:, None, :]
    seen = once[:, None, :] & (c <= pos[:, :, None]) & (t < n[:, None])[:, :, None] & (c >= 0)
    if W:
        seen = seen & ((c > pos[:, :, None] - W) | (c < case["sinks"]))
    safe = col.clamp(min=0).minimum((total - 1).clamp(min=0)[:, None])
    page, slot = st["table"].gather(1, safe // bs).long(), safe % bs
    K = _read(st["k"], st["k_scale"], page, slot).permute(0, 2, 3, 1)  # [B, H, D, L]
    V = _read(st["v"], st["v_scale"], page, slot).transpose(1, 2)  # [B, H, L, D]
    rows = (cu[:-1, None] + t).clamp(max=st["T"] - 1)
    Q = q[rows].float().view(B, N, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, N * G, D)
    s = torch.matmul(Q, K).mul_(D ** -0.5).view(B, H, N, G, -1)
    s = s.masked_fill_(~seen[:, None, :, None, :], NEG)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == NEG, 0.0, m)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, H, N * G, -1), V).view(B, H, N, G, D) / torch.where(l == 0, 1.0, l)
    r = torch.arange(st["T"], device=dev)
    b = torch.searchsorted(cu[1:], r, right=True)
    at = r - cu[b]
    out = {"out": o[b, :, at].reshape(st["T"], H * G, D).to(q.dtype)}
    if case["lse"]:
        out["lse"] = (m + l.log())[b, :, at].reshape(st["T"], H * G)
    return out


def run(st):
    op = st["case"]["op"]
    if not own:
        return {"append": _plain_append, "attention": _plain_attention, "gather": _plain_gather}[op](st)
    import speculative_decoding_verification_15_gb300 as pkg

    case, cache = st["case"], pkg.KVCache(st["k"], st["v"], st["k_scale"], st["v_scale"])
    if op == "append":
        pkg.kv_append(cache, st["new_k"], st["new_v"], st["table"], st["old"], st["cu"], st["max_new"])
        return {"k": cache.k, "v": cache.v, "k_scale": cache.k_scale, "v_scale": cache.v_scale}
    if op == "gather":
        out = pkg.kv_gather(cache, st["table"], st["cu"], st["T"], first=st["old"], dtype=_dtype(case))
        return {"k": out["k"], "v": out["v"]}
    out = pkg.cache_attention(st["q"], cache, st["table"], st["total"], st["cu"], st["max_new"],
                              scale=case["D"] ** -0.5, window=case["window"], sinks=case["sinks"], want_lse=case["lse"])
    return {"out": out["out"], "lse": out["lse"]} if case["lse"] else {"out": out["out"]}


# ------------------------------------------------------------------ work
def work(case):
    new, old, total = _positions(case)
    H, D, bs, W, S = case["Hkv"], case["D"], case["page"], case["window"], case["sinks"]
    esz = 2 if case["dtype"] == "bf16" else 4
    T = int(new.sum())
    if case["op"] == "append":
        touched = int(((total + bs - 1) // bs - old // bs).sum())
        # new values in, their codes out, the touched pages' scales in and out, page ids;
        # then a division and a rounding each
        return {"bytes": 2 * T * H * D * (esz + 1) + 16 * touched * H + 4 * touched, "flops": 4 * T * H * D}
    if case["op"] == "gather":
        pages = int(((total + bs - 1) // bs - old // bs).sum())
        return {"bytes": 2 * T * H * D * (esz + 1) + 8 * pages * H + 4 * pages, "flops": 2 * T * H * D}
    held = pairs = pages = 0
    for n, length in zip(new.tolist(), total.tolist()):
        pos = np.arange(length - n, length)
        if W:
            lo = np.maximum(pos - W + 1, 0)
            pairs += int((pos + 1 - lo + np.minimum(S, lo)).sum())
            held += int(length - lo[0] + min(S, lo[0]))
            pages += int((length + bs - 1) // bs - lo[0] // bs + (min(S, lo[0]) + bs - 1) // bs)
        else:
            pairs += int((pos + 1).sum())
            held += length
            pages += (length + bs - 1) // bs
    return {"bytes": 2 * held * H * D + 8 * pages * H + 4 * pages + 2 * T * case["Hq"] * D * esz,
            "flops": 4 * pairs * case["Hq"] * D}


# ------------------------------------------------------------------ in 64 bits
def _code_values():
    """What each of the 256 e4m3 codes stands for."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    x = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    x = np.where((c & 127) == 127, np.nan, x)
    return np.where(c >> 7, -x, x)


def _round_e4m3(x):
    """x to the nearest e4m3 value, ties to the even one, values past 448 to 448."""
    a = np.minimum(np.abs(x), 448.0)
    step = 2.0 ** (np.maximum(np.frexp(a)[1] - 1, -6) - 3.0)
    return np.copysign(np.minimum(np.rint(a / step) * step, 448.0), x)


def _host(st, *names):
    out = []
    for n in names:
        t = st[n]
        out.append(t.view(torch.uint8).cpu().numpy() if t.dtype == torch.float8_e4m3fn else
                   t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy())
    return out


def exact(case, seed):
    if work(case)["flops"] > 1.2e11:
        return None
    st = prepare(case, seed)
    H, D, bs = case["Hkv"], case["D"], case["page"]
    new, old, total = _positions(case)
    start = np.concatenate([[0], np.cumsum(new)])
    table, kc, vc, ks, vs = _host(st, "table", "k", "v", "k_scale", "v_scale")
    value = _code_values()

    if case["op"] == "append":
        res = {}
        for name, codes, scale, fresh in (("k", kc, ks, "new_k"), ("v", vc, vs, "new_v")):
            x = st[fresh].double().cpu().numpy()
            codes, scale = value[codes], scale.copy()
            for b in range(case["B"]):
                at = int(old[b])
                while at < total[b]:
                    page, slot = int(table[b, at // bs]), at % bs
                    end = min(bs, slot + int(total[b]) - at)
                    src = x[start[b] + at - old[b]:start[b] + at - old[b] + end - slot]  # [tokens, H, D]
                    for h in range(H):
                        top = np.abs(src[:, h]).max()
                        e = EXP_MIN if top == 0 else int(np.clip(math.ceil(math.log2(top / 448.0)), EXP_MIN, EXP_MAX))
                        s = 2.0 ** e
                        if slot:
                            s = max(s, scale[page, h])
                            codes[page, h, :slot] = _round_e4m3(codes[page, h, :slot] * (scale[page, h] / s))
                        codes[page, h, slot:end] = _round_e4m3(src[:, h] / s)
                        scale[page, h] = s
                    at += end - slot
            res[name], res[name + "_scale"] = codes, scale
        return res

    def held(codes, scale, b, lo, hi):
        at = np.arange(lo, hi)
        page, slot = table[b, at // bs], at % bs
        return value[codes[page, :, slot]] * scale[page][:, :, None]  # [tokens, H, D]

    if case["op"] == "gather":
        both = {}
        for name, codes, scale in (("k", kc, ks), ("v", vc, vs)):
            both[name] = np.concatenate([held(codes, scale, b, int(old[b]), int(total[b])) for b in range(case["B"])])
        return both

    q = st["q"].double().cpu().numpy()
    G = case["Hq"] // H
    out, lse = np.zeros(q.shape), np.zeros(q.shape[:2])
    for b in range(case["B"]):
        last = int(total[b])
        pos = np.arange(int(old[b]), last)
        if case["window"]:
            low = max(0, int(pos[0]) - case["window"] + 1)
            sinks = min(case["sinks"], low)
            at = np.concatenate([np.arange(sinks), np.arange(low, last)])
            K, V = (np.concatenate([held(c, s, b, 0, sinks), held(c, s, b, low, last)]) for c, s in ((kc, ks), (vc, vs)))
        else:
            at, K, V = np.arange(last), held(kc, ks, b, 0, last), held(vc, vs, b, 0, last)
        hidden = at[None, :] > pos[:, None]
        if case["window"]:
            hidden |= (at[None, :] <= pos[:, None] - case["window"]) & (at[None, :] >= case["sinks"])
        rows = slice(int(start[b]), int(start[b + 1]))
        for h in range(H):
            Q = q[rows, h * G:(h + 1) * G].reshape(-1, D)
            s = (Q @ np.ascontiguousarray(K[:, h]).T) * D ** -0.5
            s[np.repeat(hidden, G, axis=0)] = NEG
            m = s.max(axis=1, keepdims=True)
            p = np.exp(s - m)
            l = p.sum(axis=1, keepdims=True)
            out[rows, h * G:(h + 1) * G] = (p @ np.ascontiguousarray(V[:, h]) / l).reshape(-1, G, D)
            lse[rows, h * G:(h + 1) * G] = (m + np.log(l)).reshape(-1, G)
    return {"out": out, "lse": lse} if case["lse"] else {"out": out}
