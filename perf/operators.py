"""Cases of the paged-cache operators: appending keys and values with the
position rotation, and attention over a batch that shares a prefix.

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


def _append(name, B, max_q, heads_q, heads_kv, dim, prefix, max_kv, page, **kw):
    c = dict(name=name, op="append", B=B, max_q=max_q, ragged_q=False, heads_q=heads_q, heads_kv=heads_kv, dim=dim,
             prefix=prefix, max_kv=max_kv, page=page, heads_first=True, dtype="bf16", x_dtype="bf16", rot=dim,
             interleaved=False)
    c.update(kw)
    return c


def _attend(name, B, max_q, heads_q, heads_kv, dim, prefix, max_kv, page, **kw):
    c = dict(name=name, op="attend", B=B, max_q=max_q, ragged_q=False, heads_q=heads_q, heads_kv=heads_kv, dim=dim,
             prefix=prefix, max_kv=max_kv, page=page, heads_first=True, dtype="bf16")
    c.update(kw)
    return c


def listed():
    return [
        # one new token of one sequence: nothing but the call's latency
        _append("append one token", 1, 1, 64, 8, 128, 512, 40, 16),
        # a decoding step of a large batch, one token a sequence
        _append("append decode batch", 256, 1, 64, 8, 128, 2048, 512, 64),
        # the product's fp32 output into an fp16 cache, half of each head rotated, adjacent pairs, odd lengths
        _append("append fp32 ragged", 13, 97, 32, 32, 128, 100, 333, 16, ragged_q=True, dtype="f16", x_dtype="f32",
                rot=64, interleaved=True, heads_first=False),
        # prompts of several sequences written at once: bandwidth
        _append("append prompts", 8, 1024, 64, 8, 128, 4096, 1500, 64),
        # two sequences over a short system prompt: the smallest attention call
        _attend("two short sequences", 2, 1, 64, 8, 128, 200, 37, 16),
        # an ordinary decoding step
        _attend("decode 16", 16, 1, 64, 8, 128, 4096, 512, 64),
        # one key/value head per query head, fp16
        _attend("decode 32 one-to-one", 32, 1, 32, 32, 128, 2011, 700, 32, dtype="f16", heads_first=False),
        # several tokens a sequence to check at once (drafted ahead), 64-wide heads
        _attend("drafted tokens", 48, 5, 32, 8, 64, 6000, 1000, 64, dtype="f16", ragged_q=True),
        # a large batch over a long document
        _attend("decode 64 long prefix", 64, 1, 64, 8, 128, 32768, 2048, 64),
        # many sequences, each with a history of its own
        _attend("decode 256", 256, 1, 64, 8, 128, 8192, 1024, 64),
        # prompts of several sequences behind a shared prefix
        _attend("prompts behind a prefix", 4, 512, 64, 8, 128, 8192, 1200, 64, ragged_q=True),
        # the largest step: a batch over a prefix of 128 Ki tokens
        _attend("decode 128 longest prefix", 128, 1, 64, 8, 128, 131072, 2048, 128),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        heads_q, heads_kv, dim = rng.choice([(64, 8, 128), (64, 8, 128), (32, 32, 128), (32, 8, 64), (28, 4, 128)])
        c = dict(op="attend", heads_q=heads_q, heads_kv=heads_kv, dim=dim, page=rng.choice([16, 32, 64, 128]),
                 heads_first=rng.random() < 0.6, dtype=rng.choice(["bf16", "bf16", "f16"]))
        if rng.random() < 0.3:
            c.update(op="append", x_dtype=rng.choice(["bf16", "f16", "f32"]), rot=rng.choice([dim, dim, dim // 2]),
                     interleaved=rng.random() < 0.3, B=_log_int(rng, 1, 256), prefix=_log_int(rng, 1, 8192))
            c["max_q"] = 1 if rng.random() < 0.5 else _log_int(rng, 2, 1024)
        else:
            c.update(B=_log_int(rng, 1, 256), prefix=0 if rng.random() < 0.1 else _log_int(rng, 1, 131072))
            c["max_q"] = rng.choice([1, 1, 1, rng.randint(2, 8), _log_int(rng, 9, 512)])
        c["ragged_q"] = c["max_q"] > 1 and rng.random() < 0.7
        c["max_kv"] = max(c["max_q"], _log_int(rng, 1, 4096))
        tokens = c["B"] * c["max_q"]
        # the plain form keeps all scores of a pass in memory, and pads the sequences to the longest
        scores = tokens * heads_q * (c["prefix"] + c["max_kv"]) if c["op"] == "attend" else 0
        if scores <= 1.1e9 and tokens <= 8192 and c["B"] * c["max_kv"] <= 300000 and _cost(c) <= most:
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
    T, D, size = sum(n_q), case["dim"], 2
    token = case["heads_kv"] * D * 2          # values of K and V of one cached token
    tables = 4 * (2 * case["B"] + 1)
    if case["op"] == "append":
        x = 4 if case["x_dtype"] == "f32" else 2
        values = T * (case["heads_q"] * D + token)
        return {"bytes": values * (x + size) + T * case["rot"] * 4 + tables + 4 * T, "flops": 3 * T * (case["heads_q"] + case["heads_kv"]) * case["rot"]}
    pages = sum(-(-k // case["page"]) for k in kv) + -(-case["prefix"] // case["page"])
    seen = sum(n * (case["prefix"] + k) - n * (n - 1) // 2 for n, k in zip(n_q, kv))
    return {"bytes": (2 * T * case["heads_q"] * D + (case["prefix"] + sum(kv)) * token) * size + tables + 4 * pages,
            "flops": 4 * D * case["heads_q"] * seen}


def _cost(case):
    w = work(case)
    return w["bytes"] + w["flops"] / 280   # bytes, at the card's rates


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev, dt = "cuda", DTYPES[case["dtype"]]
    n_q, kv = _lengths(case)
    B, T, Hq, Hkv, D, page = case["B"], sum(n_q), case["heads_q"], case["heads_kv"], case["dim"], case["page"]

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
    caches = []
    for _ in range(2):
        pages = torch.empty(shape, device=dev, dtype=dt)
        for at in range(0, n_pages, 4096):
            part = pages[at:at + 4096]
            part.copy_(torch.randn(part.shape, generator=g, device=dev, dtype=torch.float32))
        caches.append(pages.permute(turn))      # [page, place in it, head, dim]
    s = dict(case=dict(case), T=T, k_cache=caches[0], v_cache=caches[1], table=order[:B * width].view(B, width),
             prefix_table=order[B * width:B * width + shared],
             kv_len=torch.tensor(kv, dtype=torch.int32, device=dev),
             cu_q=torch.tensor([0] + np.cumsum(n_q).tolist(), dtype=torch.int32, device=dev))
    if case["op"] == "append":
        # one row a token, as the fused q/k/v product leaves it
        xd = DTYPES[case["x_dtype"]]
        s["qkv"] = values(T, (Hq + 2 * Hkv) * D, dtype=xd)
        at = torch.arange(case["prefix"] + case["max_kv"], device=dev, dtype=torch.float64)
        freq = 10000.0 ** (-torch.arange(0, case["rot"], 2, device=dev, dtype=torch.float64) / case["rot"])
        angle = at[:, None] * freq[None, :]
        s["rope"] = torch.cat([angle.cos(), angle.sin()], 1).float()   # [position, cosines then sines]
    else:
        s["q"] = (1.5 * torch.randn((T, Hq, D), generator=g, device=dev, dtype=torch.float32)).to(dt)
    if own:
        import bit_weight_only_group_gb300 as qg
        s["cache"] = qg.KVCache(s["k_cache"], s["v_cache"])
        s["batch"] = qg.KVBatch(s["table"], s["kv_len"], max_kv=case["max_kv"], cu_q=s["cu_q"], max_q=case["max_q"],
                                tokens=T, prefix_table=s["prefix_table"], prefix_len=case["prefix"])
        if case["op"] == "attend":
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
        if c["op"] == "append":
            q, k, v = _heads(s)
            q = qg.qkv_append(s["cache"], s["batch"], k, v, q=q, rope=s["rope"], interleaved=c["interleaved"])
            return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
        return qg.qattn_forward(s["q"], s["cache"], s["batch"], workspace=s["workspace"])
    return _plain_append(s, c) if c["op"] == "append" else _plain_attend(s, c)


def _places(s, c, T):
    """Sequence of each token, and its place among the sequence's own tokens."""
    t = torch.arange(T, device="cuda")
    cu, kv = s["cu_q"].long(), s["kv_len"].long()
    seq = torch.searchsorted(cu, t, right=True) - 1
    return seq, kv[seq] - cu[seq + 1] + t


def _rotate(x, rows, rot, interleaved):
    x = x.float()
    cos, sin = rows[:, None, :rot // 2], rows[:, None, rot // 2:]
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_append(s, c):
    q, k, v = _heads(s)
    seq, place = _places(s, c, s["T"])
    rows = s["rope"][c["prefix"] + place]
    page, at = s["table"][seq, place // c["page"]].long(), place % c["page"]
    dt = s["k_cache"].dtype
    s["k_cache"][page, at] = _rotate(k, rows, c["rot"], c["interleaved"]).to(dt)
    s["v_cache"][page, at] = v.to(dt)
    return {"q": _rotate(q, rows, c["rot"], c["interleaved"]).to(dt), "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def _plain_attend(s, c):
    B, T, Hq, Hkv, D, n, L, P = c["B"], s["T"], c["heads_q"], c["heads_kv"], c["dim"], c["max_q"], c["max_kv"], c["prefix"]
    G, scale = Hq // Hkv, 1 / math.sqrt(D)
    q = s["q"].float().view(T, Hkv, G, D) * scale
    cu, kv = s["cu_q"].long(), s["kv_len"].long()
    # the prefix, once for all: [head, token and query head, place]
    kp = s["k_cache"][s["prefix_table"].long()].flatten(0, 1)[:P].float().permute(1, 2, 0)
    vp = s["v_cache"][s["prefix_table"].long()].flatten(0, 1)[:P].float().permute(1, 0, 2)
    sp = torch.matmul(q.permute(1, 0, 2, 3).reshape(Hkv, T * G, D), kp).view(Hkv, T, G, P)
    # each sequence's own tokens, padded to the longest: [sequence, head, query, query head, place]
    seq, place = _places(s, c, T)
    ko = s["k_cache"][s["table"].long()].flatten(1, 2)[:, :L].float().permute(0, 2, 3, 1)
    vo = s["v_cache"][s["table"].long()].flatten(1, 2)[:, :L].permute(0, 2, 1, 3)
    there = torch.arange(L, device="cuda") < kv[:, None]
    vo = torch.where(there[:, None, :, None], vo, torch.zeros((), dtype=vo.dtype, device="cuda")).float()
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


def exact(case, seed):
    """The definition in 64 bits, one head or one sequence at a time."""
    s = prepare(case, seed)
    n_q, kv = _lengths(case)
    Hq, Hkv, D, P, page = case["heads_q"], case["heads_kv"], case["dim"], case["prefix"], case["page"]
    G = Hq // Hkv
    starts = [0] + np.cumsum(n_q).tolist()
    table = s["table"].tolist()
    if case["op"] == "append":
        rot = case["rot"]
        x = s["qkv"].double()
        out = {"q": x[:, :Hq * D].reshape(-1, Hq, D).clone(), "k_cache": s["k_cache"].double(), "v_cache": s["v_cache"].double()}
        keys = x[:, Hq * D:(Hq + Hkv) * D].reshape(-1, Hkv, D).clone()
        vals = x[:, (Hq + Hkv) * D:].reshape(-1, Hkv, D)
        half = torch.arange(rot // 2, device="cuda")
        first, second = (2 * half, 2 * half + 1) if case["interleaved"] else (half, half + rot // 2)
        # the table's own 32-bit cosines and sines are the inputs
        where = torch.tensor([P + kv[b] - n_q[b] + i for b in range(case["B"]) for i in range(n_q[b])], device="cuda")
        turn = torch.complex(s["rope"][where, :rot // 2].double(), s["rope"][where, rot // 2:].double())[:, None, :]
        for y in (out["q"], keys):
            z = torch.complex(y[:, :, first], y[:, :, second]) * turn
            y[:, :, first], y[:, :, second] = z.real, z.imag
        for b in range(case["B"]):
            lo = kv[b] - n_q[b]
            spots = torch.arange(lo, kv[b], device="cuda")
            pages = s["table"][b].long()[spots // page]
            out["k_cache"][pages, spots % page] = keys[starts[b]:starts[b + 1]]
            out["v_cache"][pages, spots % page] = vals[starts[b]:starts[b + 1]]
        return out
    out = torch.empty((starts[-1], Hq, D), dtype=torch.float64, device="cuda")
    # per head: logits of all tokens against the prefix, per sequence against its own, joined by their log-sums
    for h in range(Hkv):
        q = s["q"][:, h * G:(h + 1) * G].double()
        kp = s["k_cache"][s["prefix_table"].long(), :, h].reshape(-1, D)[:P].double()
        vp = s["v_cache"][s["prefix_table"].long(), :, h].reshape(-1, D)[:P].double()
        z = q.reshape(-1, D) @ kp.T / math.sqrt(D)
        lp = torch.logsumexp(z, -1) if P else torch.full((q.shape[0] * G,), -math.inf, dtype=torch.float64, device="cuda")
        op = torch.exp_(z.sub_(lp[:, None])) @ vp if P else torch.zeros((q.shape[0] * G, D), dtype=torch.float64, device="cuda")
        lp, op = lp.view(-1, G), op.view(-1, G, D)
        for b in range(case["B"]):
            a, e, n = starts[b], starts[b + 1], n_q[b]
            rows = s["table"][b].long()
            kb = s["k_cache"][rows, :, h].reshape(-1, D)[:kv[b]].double()
            vb = s["v_cache"][rows, :, h].reshape(-1, D)[:kv[b]].double()
            z = torch.einsum("igd,jd->igj", q[a:e], kb) / math.sqrt(D)
            later = torch.arange(kv[b], device="cuda")[None, :] > torch.arange(kv[b] - n, kv[b], device="cuda")[:, None]
            z = z.masked_fill(later[:, None, :], -math.inf)
            lo = torch.logsumexp(z, -1)
            ob = torch.einsum("igj,jd->igd", torch.exp(z - lo[..., None]), vb)
            both = torch.logaddexp(lo, lp[a:e])
            out[a:e, h * G:(h + 1) * G] = torch.exp(lo - both)[..., None] * ob + torch.exp(lp[a:e] - both)[..., None] * op[a:e]
    return out
