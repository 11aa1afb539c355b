"""Cases of the paged-cache operators for normed heads and for a cache held in 8
bits: appending with the norms of queries and keys, quantising a cache as it is
written and reading it back, and attention over such a cache.

An 8-bit cache holds E4M3 codes and, for every 16 places of a page and head, one
exponent e (a byte, e + 127): a value is code * 2^e.  e is the least with
amax <= 448 * 2^e, in -64 .. 63; a block that tokens are added to keeps the
larger of its own and the new tokens', and its earlier codes follow.

Each case is real work of a decoding or prefilling step: the smallest calls,
where latency counts, ordinary ones and the largest.  Head layouts are those of
the 70B-shaped stack (64 query heads over 8 key/value heads of 128) and of the
7B-shaped stack (32 heads of 128, one key/value head each), and two generic
ones with 64-wide heads and with 7 query heads per key/value head.

`run` computes one pass: in plain torch operations, in 32 bits, or (`own`)
through the package's entry points.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
EPS = 1e-6
BLOCK = 16                       # places of one scale
E_MIN, E_MAX = -64, 63


def _append(name, B, max_q, heads_q, heads_kv, dim, prefix, max_kv, page, **kw):
    c = dict(name=name, op="append", B=B, max_q=max_q, ragged_q=False, heads_q=heads_q, heads_kv=heads_kv, dim=dim,
             prefix=prefix, max_kv=max_kv, page=page, heads_first=True, dtype="bf16", x_dtype="bf16", rot=dim,
             interleaved=False, norm=True)
    c.update(kw)
    return c


def _attend(name, B, max_q, heads_q, heads_kv, dim, prefix, max_kv, page, **kw):
    c = dict(name=name, op="attend8", B=B, max_q=max_q, ragged_q=False, heads_q=heads_q, heads_kv=heads_kv, dim=dim,
             prefix=prefix, max_kv=max_kv, page=page, heads_first=True, dtype="bf16")
    c.update(kw)
    return c


def listed():
    return [
        # a decoding step of a large batch, one token a sequence, heads normed and turned
        _append("norm decode batch", 256, 1, 64, 8, 128, 2048, 512, 64),
        # the product's fp32 output into an fp16 cache, half of each head turned, adjacent pairs, odd lengths
        _append("norm fp32 ragged", 13, 97, 32, 32, 128, 100, 333, 16, ragged_q=True, dtype="f16", x_dtype="f32",
                rot=64, interleaved=True, heads_first=False),
        # prompts of several sequences written at once: bandwidth
        _append("norm prompts", 8, 1024, 64, 8, 128, 4096, 1500, 64),
        # one token into a short 8-bit sequence, which is read back: nothing but latency
        _append("write8 one token", 1, 1, 64, 8, 128, 512, 40, 16, op="write8", norm=False),
        # a decoding step of a large batch into 8 bits; the sequences are read back to be moved elsewhere
        _append("write8 decode batch", 256, 1, 64, 8, 128, 2048, 512, 64, op="write8"),
        # prompts of odd lengths behind earlier turns, quantised as they are written, 64-wide heads
        _append("write8 prompts", 8, 1024, 32, 8, 64, 4096, 1500, 64, op="write8", ragged_q=True, dtype="f16",
                heads_first=False),
        # two sequences over a short system prompt: the smallest attention call
        _attend("two short sequences", 2, 1, 64, 8, 128, 200, 37, 16),
        # long histories, nothing shared: what half the bytes are for
        _attend("decode 32 long histories", 32, 1, 64, 8, 128, 0, 16384, 64),
        # one key/value head per query head, fp16
        _attend("decode 32 one-to-one", 32, 1, 32, 32, 128, 2011, 700, 32, dtype="f16", heads_first=False),
        # several tokens a sequence to check at once (drafted ahead), 64-wide heads
        _attend("drafted tokens", 48, 5, 32, 8, 64, 6000, 1000, 64, dtype="f16", ragged_q=True),
        # many sequences, each with a history of its own
        _attend("decode 256", 256, 1, 64, 8, 128, 8192, 1024, 64),
        # prompts of several sequences behind a shared prefix
        _attend("prompts behind a prefix", 4, 512, 64, 8, 128, 8192, 1200, 64, ragged_q=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        heads_q, heads_kv, dim = rng.choice([(64, 8, 128), (64, 8, 128), (32, 32, 128), (32, 8, 64), (28, 4, 128)])
        c = dict(op=rng.choice(["append", "write8", "attend8", "attend8"]), heads_q=heads_q, heads_kv=heads_kv, dim=dim,
                 page=rng.choice([16, 32, 64, 128]), heads_first=rng.random() < 0.6,
                 dtype=rng.choice(["bf16", "bf16", "f16"]))
        if c["op"] != "attend8":
            c.update(x_dtype=rng.choice(["bf16", "f16", "f32"]), rot=rng.choice([dim, dim, dim // 2]),
                     interleaved=rng.random() < 0.3, norm=c["op"] == "append" or rng.random() < 0.6,
                     B=_log_int(rng, 1, 256), prefix=_log_int(rng, 1, 8192))
            c["max_q"] = 1 if rng.random() < 0.5 else _log_int(rng, 2, 1024)
        else:
            c.update(B=_log_int(rng, 1, 256), prefix=0 if rng.random() < 0.2 else _log_int(rng, 1, 65536))
            c["max_q"] = rng.choice([1, 1, 1, rng.randint(2, 8), _log_int(rng, 9, 512)])
        c["ragged_q"] = c["max_q"] > 1 and rng.random() < 0.7
        c["max_kv"] = max(c["max_q"], _log_int(rng, 1, 16384 if c["op"] == "attend8" else 2048))
        tokens = c["B"] * c["max_q"]
        # the plain form keeps all scores of a pass in memory, and pads the sequences to the longest
        scores = tokens * heads_q * (c["prefix"] + c["max_kv"]) if c["op"] == "attend8" else 0
        room = 300000 if c["op"] == "attend8" else 140000
        if scores <= 1.1e9 and tokens <= 8192 and c["B"] * c["max_kv"] <= room and _cost(c) <= most:
            return c


def _lengths(case):
    """New tokens and length of each sequence: of the case alone, the first at the bounds."""
    r = random.Random(repr([case[k] for k in ("B", "max_q", "max_kv", "prefix", "page")]))
    n_q = [r.randint(1, case["max_q"]) if case["ragged_q"] else case["max_q"] for _ in range(case["B"])]
    n_q[0] = case["max_q"]
    kv = [r.randint(n, case["max_kv"]) for n in n_q]
    kv[0] = case["max_kv"]
    return n_q, kv


def work(case):
    n_q, kv = _lengths(case)
    T, D, hq, hk = sum(n_q), case["dim"], case["heads_q"], case["heads_kv"]
    tables = 4 * (2 * case["B"] + 1)
    if case["op"] != "attend8":
        x, y = 4 if case["x_dtype"] == "f32" else 2, 1 if case["op"] == "write8" else 2
        b = T * (hq * D * (x + 2) + 2 * hk * D * (x + y)) + T * case["rot"] * 4 + tables + 4 * T
        f = T * (hq + hk) * (3 * case["rot"] + 4 * D * case["norm"])
        if case["op"] == "write8":     # the sequences read back, with their scales
            b += 2 * hk * sum(D * k + -(-k // BLOCK) + 2 * D * k for k in kv)
            f += 2 * T * hk * D * 2 + 2 * sum(kv) * hk * D
        return {"bytes": b, "flops": f}
    pages = sum(-(-k // case["page"]) for k in kv) + -(-case["prefix"] // case["page"])
    keys = [case["prefix"]] + kv
    seen = sum(n * (case["prefix"] + k) - n * (n - 1) // 2 for n, k in zip(n_q, kv))
    return {"bytes": 4 * T * hq * D + 2 * hk * sum(D * k + -(-k // BLOCK) for k in keys) + tables + 4 * pages,
            "flops": 4 * D * hq * seen}


def _cost(case):
    w = work(case)
    return w["bytes"] + w["flops"] / 280   # bytes, at the card's rates


def _pow2(e):
    """2^e in 32 bits, exactly."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _exponent(amax):
    """The least e with amax <= 448 * 2^e, in E_MIN .. E_MAX."""
    m, x = torch.frexp(amax)      # m in [0.5, 1); 448 is 0.875 * 2^9
    e = x - 9 + (m > 0.875).to(x.dtype)
    return torch.where(amax > 0, e, E_MIN).clamp(E_MIN, E_MAX)


def _e4m3(x):
    return x.to(torch.float8_e4m3fn).view(torch.uint8)


def _values(codes):
    return codes.view(torch.float8_e4m3fn).float()


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev, dt = "cuda", DTYPES[case["dtype"]]
    n_q, kv = _lengths(case)
    B, T, Hq, Hkv, D, page = case["B"], sum(n_q), case["heads_q"], case["heads_kv"], case["dim"], case["page"]
    eight = case["op"] != "append"

    def values(*shape, dtype=dt):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).to(dtype)

    # pages of the sequences and of the prefix, in no order, a few of them unused
    width = -(-case["max_kv"] // page)
    shared = -(-case["prefix"] // page)
    n_pages = B * width + shared + 3
    order = torch.randperm(n_pages, generator=g, device=dev).to(torch.int32)
    if case["heads_first"]:
        shape, turn = (n_pages, Hkv, page, D), (0, 2, 1, 3)
    else:
        shape, turn = (n_pages, page, Hkv, D), (0, 1, 2, 3)
    caches, scales = [], []
    for _ in range(2):
        pages = torch.empty(shape, device=dev, dtype=torch.uint8 if eight else dt).permute(turn)   # [page, place, head, dim]
        exps = torch.empty((n_pages, page // BLOCK, Hkv), device=dev, dtype=torch.uint8)
        gain = torch.exp2(2 * torch.randn((Hkv, 1), generator=g, device=dev)) if eight else 1.0
        for at in range(0, n_pages, 4096):
            part = pages[at:at + 4096]
            x = torch.randn(part.shape, generator=g, device=dev, dtype=torch.float32) * gain
            if eight:
                x = x.unflatten(1, (-1, BLOCK))                                         # [page, block, place, head, dim]
                e = _exponent(x.abs().amax((2, 4)))
                exps[at:at + 4096] = (e + 127).to(torch.uint8)
                x = _e4m3(x * _pow2(-e)[:, :, None, :, None]).flatten(1, 2)
            part.copy_(x)
        caches.append(pages)
        scales.append(exps)
    s = dict(case=dict(case), T=T, k_cache=caches[0], v_cache=caches[1], k_scale=scales[0], v_scale=scales[1],
             table=order[:B * width].view(B, width), prefix_table=order[B * width:B * width + shared],
             kv_len=torch.tensor(kv, dtype=torch.int32, device=dev),
             cu_q=torch.tensor([0] + np.cumsum(n_q).tolist(), dtype=torch.int32, device=dev))
    if case["op"] == "attend8":
        s["q"] = (1.5 / 4 * torch.randn((T, Hq, D), generator=g, device=dev, dtype=torch.float32)).to(dt)
    else:
        # one row a token, as the fused q/k/v product leaves it
        xd = DTYPES[case["x_dtype"]]
        s["qkv"] = values(T, (Hq + 2 * Hkv) * D, dtype=xd)
        at = torch.arange(case["prefix"] + case["max_kv"], device=dev, dtype=torch.float64)
        freq = 10000.0 ** (-torch.arange(0, case["rot"], 2, device=dev, dtype=torch.float64) / case["rot"])
        angle = at[:, None] * freq[None, :]
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float()   # [position, cosines then sines]
        s["q_norm"], s["k_norm"] = (1 + 0.2 * values(D, dtype=torch.float32) for _ in range(2))
        if case["op"] == "write8":
            s["cu_all"] = torch.tensor([0] + np.cumsum(kv).tolist(), dtype=torch.int32, device=dev)
            s["all"] = sum(kv)
    if own:
        import bit_weight_only_group_gb300 as qg
        codes = [s[n].view(torch.float8_e4m3fn) if eight else s[n] for n in ("k_cache", "v_cache")]
        s["cache"] = qg.KVCache8(*codes, s["k_scale"], s["v_scale"]) if eight else qg.KVCache(*codes)
        s["batch"] = qg.KVBatch(s["table"], s["kv_len"], max_kv=case["max_kv"], cu_q=s["cu_q"], max_q=case["max_q"],
                                tokens=T, prefix_table=s["prefix_table"], prefix_len=case["prefix"])
        if case["op"] == "write8":
            s["batch_all"] = qg.KVBatch(s["table"], s["kv_len"], max_kv=case["max_kv"], cu_q=s["cu_all"],
                                        max_q=case["max_kv"], tokens=s["all"])
        if case["op"] == "attend8":
            need = qg.qattn_workspace_size(s["cache"], s["batch"], Hq)
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device=dev)
    return s


def _heads(s):
    c = s["case"]
    Hq, Hkv, D = c["heads_q"], c["heads_kv"], c["dim"]
    q, k, v = s["qkv"].split([Hq * D, Hkv * D, Hkv * D], 1)
    return q.view(-1, Hq, D), k.view(-1, Hkv, D), v.view(-1, Hkv, D)


def run(state):
    s, c = state, state["case"]
    if own:
        import bit_weight_only_group_gb300 as qg
        if c["op"] == "attend8":
            return qg.qattn_forward(s["q"], s["cache"], s["batch"], workspace=s["workspace"])
        q, k, v = _heads(s)
        norms = dict(q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS) if c["norm"] else {}
        if c["op"] == "append":
            q = qg.qkv_append(s["cache"], s["batch"], k, v, q=q, rope=s["rope"], interleaved=c["interleaved"], **norms)
            return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        q = qg.qkv_append(s["cache"], s["batch"], k, v, q=q, rope=s["rope"], interleaved=c["interleaved"],
                          q_dtype=DTYPES[c["dtype"]], **norms)
        k, v = qg.qkv_read(s["cache"], s["batch_all"])
        return {"q": q, "k": k, "v": v}
    return {"append": _plain_append, "write8": _plain_write, "attend8": _plain_attend}[c["op"]](s, c)


def _places(cu, kv, T):
    """Sequence of each token, and its place among the sequence's own tokens."""
    t = torch.arange(T, device="cuda")
    cu, kv = cu.long(), kv.long()
    seq = torch.searchsorted(cu, t, right=True) - 1
    return seq, kv[seq] - cu[seq + 1] + t


def _normed(x, w, norm):
    x = x.float()
    return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w if norm else x


def _rotate(x, rows, rot, interleaved):
    cos, sin = rows[:, None, :rot // 2], rows[:, None, rot // 2:]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _new_tokens(s, c):
    """Queries and keys normed and turned, values, all in 32 bits; sequence, place, page and place in it of each token."""
    q, k, v = _heads(s)
    seq, place = _places(s["cu_q"], s["kv_len"], s["T"])
    rows = s["rope"][c["prefix"] + place]
    q, k = (_rotate(_normed(x, w, c["norm"]), rows, c["rot"], c["interleaved"]) for x, w in ((q, s["q_norm"]), (k, s["k_norm"])))
    return q, k, v.float(), seq, place, s["table"][seq, place // c["page"]].long(), place % c["page"]


def _plain_append(s, c):
    q, k, v, _, _, page, at = _new_tokens(s, c)
    dt = s["k_cache"].dtype
    s["k_cache"][page, at], s["v_cache"][page, at] = k.to(dt), v.to(dt)
    return {"q": q.to(dt), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_write(s, c):
    q, k, v, seq, place, page, at = _new_tokens(s, c)
    per = c["page"] // BLOCK
    n = s["k_cache"].shape[0] * per
    block = page * per + at // BLOCK
    # the sequence's first block may hold earlier tokens
    cu, kv = s["cu_q"].long(), s["kv_len"].long()
    start = kv - (cu[1:] - cu[:-1])
    first_page = s["table"].gather(1, (start // c["page"])[:, None].clamp(max=s["table"].shape[1] - 1))[:, 0].long()
    first = first_page * per + start % c["page"] // BLOCK
    kept = (start % BLOCK > 0)[:, None]                                                      # of the first block
    for x, codes, scale in ((k, s["k_cache"], s["k_scale"]), (v, s["v_cache"], s["v_scale"])):
        flat = scale.view(n, -1)
        amax = torch.zeros(flat.shape, device="cuda")
        amax.scatter_reduce_(0, block[:, None].expand(-1, flat.shape[1]), x.abs().amax(-1), "amax")
        e = _exponent(amax)
        old = flat[first].int() - 127
        grown = torch.where(kept, torch.maximum(e[first], old), e[first])
        e[first] = grown
        # earlier codes of the first blocks, in the new scale (those of new tokens are written below)
        rows = (first % per * BLOCK)[:, None] + torch.arange(BLOCK, device="cuda")
        was = codes[first_page[:, None], rows]                                               # [sequence, place, head, dim]
        follow = _e4m3(_values(was) * _pow2(old - grown)[:, None, :, None])
        codes[first_page[:, None], rows] = torch.where(kept[:, :, None, None], follow, was)
        flat[block] = (e[block] + 127).to(torch.uint8)
        codes[page, at] = _e4m3(x * _pow2(-e[block])[:, :, None])
    seq, place = _places(s["cu_all"], s["kv_len"], s["all"])
    page, at = s["table"][seq, place // c["page"]].long(), place % c["page"]
    k, v = ((_values(codes[page, at]) * _pow2(scale[page, at // BLOCK].int() - 127)[:, :, None]).bfloat16()
            for codes, scale in ((s["k_cache"], s["k_scale"]), (s["v_cache"], s["v_scale"])))
    return {"q": q.to(DTYPES[c["dtype"]]), "k": k, "v": v}


def _gather(codes, scale, rows):
    """The values of pages `rows` [..., n] in 32 bits: [..., n * page, head, dim]."""
    e = scale[rows].flatten(-3, -2).int() - 127                                               # [..., blocks, head]
    x = _values(codes[rows]).flatten(-4, -3).unflatten(-3, (-1, BLOCK))
    return (x * _pow2(e)[..., :, None, :, None]).flatten(-4, -3)


def _plain_attend(s, c):
    B, T, Hq, Hkv, D, n, L, P = c["B"], s["T"], c["heads_q"], c["heads_kv"], c["dim"], c["max_q"], c["max_kv"], c["prefix"]
    G, scale = Hq // Hkv, 1 / math.sqrt(D)
    q = s["q"].float().view(T, Hkv, G, D) * scale
    cu, kv = s["cu_q"].long(), s["kv_len"].long()
    # the prefix, once for all: [head, token and query head, place]
    kp = _gather(s["k_cache"], s["k_scale"], s["prefix_table"].long())[:P].permute(1, 2, 0)
    vp = _gather(s["v_cache"], s["v_scale"], s["prefix_table"].long())[:P].permute(1, 0, 2)
    sp = torch.matmul(q.permute(1, 0, 2, 3).reshape(Hkv, T * G, D), kp).view(Hkv, T, G, P)
    # each sequence's own tokens, padded to the longest: [sequence, head, query, query head, place]
    seq, place = _places(s["cu_q"], s["kv_len"], T)
    ko = _gather(s["k_cache"], s["k_scale"], s["table"].long())[:, :L].permute(0, 2, 3, 1)
    vo = _gather(s["v_cache"], s["v_scale"], s["table"].long())[:, :L].permute(0, 2, 1, 3)
    there = torch.arange(L, device="cuda") < kv[:, None]
    vo = torch.where(there[:, None, :, None], vo, 0.0)
    at = torch.arange(T, device="cuda") - cu[seq]
    qo = torch.zeros((B, n, Hkv, G, D), device="cuda")
    qo[seq, at] = q
    so = torch.matmul(qo.permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, D), ko).view(B, Hkv, n, G, L)
    so = so[seq, :, at]                                                     # [token, head, query head, place]
    seen = torch.arange(L, device="cuda")[None, :] <= place[:, None]
    so = torch.where(seen[:, None, None, :], so, -math.inf)
    m = so.amax(-1, keepdim=True)
    sp = sp.permute(1, 0, 2, 3)                                             # [token, head, query head, place]
    if P:
        m = torch.maximum(m, sp.amax(-1, keepdim=True))
    m = torch.where(m > -math.inf, m, 0.0)
    ep, eo = torch.exp(sp - m), torch.exp(so - m)
    total = ep.sum(-1, keepdim=True) + eo.sum(-1, keepdim=True)
    o = torch.matmul(ep.permute(1, 0, 2, 3).reshape(Hkv, T * G, P), vp).view(Hkv, T, G, D).permute(1, 0, 2, 3)
    w = torch.zeros((B, n, Hkv, G, L), device="cuda")
    w[seq, at] = eo
    own_part = torch.matmul(w.permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * G, L), vo).view(B, Hkv, n, G, D)
    o = (o + own_part[seq, :, at]) / torch.where(total > 0, total, 1.0)
    return o.reshape(T, Hq, D).to(s["q"].dtype)


def _nearest8(z):
    """E4M3's nearest value of z (64 bits), ties to even, |z| at most 448."""
    step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(z / step) * step


def exact(case, seed):
    """The definition in 64 bits, one head or one sequence at a time."""
    s = prepare(case, seed)
    n_q, kv = _lengths(case)
    Hq, Hkv, D, P, page = case["heads_q"], case["heads_kv"], case["dim"], case["prefix"], case["page"]
    G = Hq // Hkv
    starts = [0] + np.cumsum(n_q).tolist()
    if case["op"] == "attend8":
        return _exact_attention(s, n_q, kv, Hq, Hkv, G, D, P, page, starts)
    rot, x = case["rot"], s["qkv"].double()
    new = {"q": x[:, :Hq * D].reshape(-1, Hq, D).clone(), "k": x[:, Hq * D:(Hq + Hkv) * D].reshape(-1, Hkv, D).clone(),
           "v": x[:, (Hq + Hkv) * D:].reshape(-1, Hkv, D)}
    if case["norm"]:
        for name in ("q", "k"):
            y = new[name]
            y /= (torch.linalg.vector_norm(y, dim=-1, keepdim=True) ** 2 / D + EPS).sqrt()
            y *= s[name + "_norm"].double()
    half = torch.arange(rot // 2, device="cuda")
    first, second = (2 * half, 2 * half + 1) if case["interleaved"] else (half, half + rot // 2)
    # the table's own 32-bit cosines and sines are the inputs
    where = torch.tensor([P + kv[b] - n_q[b] + i for b in range(case["B"]) for i in range(n_q[b])], device="cuda")
    turn = torch.complex(s["rope"][where, :rot // 2].double(), s["rope"][where, rot // 2:].double())[:, None, :]
    for y in (new["q"], new["k"]):
        z = torch.complex(y[:, :, first], y[:, :, second]) * turn
        y[:, :, first], y[:, :, second] = z.real, z.imag
    if case["op"] == "append":
        out = {"q": new["q"], "k_cache": s["k_cache"].double(), "v_cache": s["v_cache"].double()}
        for b in range(case["B"]):
            spots = torch.arange(kv[b] - n_q[b], kv[b], device="cuda")
            pages = s["table"][b].long()[spots // page]
            for name in ("k", "v"):
                out[name + "_cache"][pages, spots % page] = new[name][starts[b]:starts[b + 1]]
        return out
    out = {"q": new["q"], "k": [], "v": []}
    for b in range(case["B"]):
        rows, lo = s["table"][b, :-(-kv[b] // page)].long(), kv[b] - n_q[b]
        for name in ("k", "v"):
            codes = s[name + "_cache"][rows].view(torch.float8_e4m3fn).double().reshape(-1, Hkv, D)
            e = s[name + "_scale"][rows].double().reshape(-1, Hkv) - 127
            have = codes[:kv[b]].clone()                      # the codes there are, then the values of the new ones
            have[lo:] = new[name][starts[b]:starts[b + 1]]
            pad = -kv[b] % BLOCK
            blocks = torch.cat([have, have.new_zeros(pad, Hkv, D)]).view(-1, BLOCK, Hkv, D)
            place = torch.arange(kv[b] + pad, device="cuda").view(-1, BLOCK)
            fresh = (place >= lo)[:, :, None, None]
            mant, ex = torch.frexp((blocks * fresh).abs().amax((1, 3)))
            want = torch.where(mant > 0, ex - 9 + (mant > 0.875).to(ex.dtype), E_MIN).clamp(E_MIN, E_MAX).double()
            old = e[:want.shape[0]]
            holds = (place[:, 0] < lo)[:, None]               # the block has earlier tokens
            scale = torch.where(holds, torch.maximum(torch.where((place[:, -1] >= lo)[:, None], want, old), old), want)
            power = torch.exp2(torch.where(fresh[:, :, 0], -scale[:, None], (old - scale)[:, None]))[..., None]
            value = _nearest8(blocks * power) * torch.exp2(scale)[:, None, :, None]
            out[name].append(value.reshape(-1, Hkv, D)[:kv[b]])
    return {"q": out["q"], "k": torch.cat(out["k"]), "v": torch.cat(out["v"])}


def _exact_attention(s, n_q, kv, Hq, Hkv, G, D, P, page, starts):
    def values(name, rows, h, n):
        codes = s[name + "_cache"][rows, :, h].view(torch.float8_e4m3fn).double().reshape(-1, D)
        e = s[name + "_scale"][rows, :, h].double().reshape(-1) - 127
        return (codes * torch.exp2(e).repeat_interleave(BLOCK)[:, None])[:n]

    out = torch.empty((starts[-1], Hq, D), dtype=torch.float64, device="cuda")
    # per head: logits of all tokens against the prefix, per sequence against its own, joined by their log-sums
    for h in range(Hkv):
        q = s["q"][:, h * G:(h + 1) * G].double()
        kp, vp = (values(name, s["prefix_table"].long(), h, P) for name in ("k", "v"))
        z = q.reshape(-1, D) @ kp.T / math.sqrt(D)
        lp = torch.logsumexp(z, -1) if P else torch.full((q.shape[0] * G,), -math.inf, dtype=torch.float64, device="cuda")
        op = torch.exp_(z.sub_(lp[:, None])) @ vp if P else torch.zeros((q.shape[0] * G, D), dtype=torch.float64, device="cuda")
        lp, op = lp.view(-1, G), op.view(-1, G, D)
        for b in range(len(n_q)):
            a, e, n = starts[b], starts[b + 1], n_q[b]
            rows = s["table"][b].long()
            kb, vb = (values(name, rows, h, kv[b]) for name in ("k", "v"))
            z = torch.einsum("igd,jd->igj", q[a:e], kb) / math.sqrt(D)
            later = torch.arange(kv[b], device="cuda")[None, :] > torch.arange(kv[b] - n, kv[b], device="cuda")[:, None]
            z = z.masked_fill(later[:, None, :], -math.inf)
            lo = torch.logsumexp(z, -1)
            ob = torch.einsum("igj,jd->igd", torch.exp(z - lo[..., None]), vb)
            both = torch.logaddexp(lo, lp[a:e])
            out[a:e, h * G:(h + 1) * G] = torch.exp(lo - both)[..., None] * ob + torch.exp(lp[a:e] - both)[..., None] * op[a:e]
    return out
