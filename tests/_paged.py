"""Paged-cache test helpers: seeded batches over a cache, and the operators'
definitions in 64 bits with the error bounds that follow from the kernels'
roundings."""
import math

import torch

# unit roundoffs: bf16 keeps 8 significant bits, fp16 11, fp32 24
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}


class Case:
    """n_q new tokens and own cached tokens kv of each sequence behind a prefix, in pages in no order; whatever lies
    past a length holds NaN."""

    def __init__(self, n_q, kv, prefix=0, heads_q=8, heads_kv=2, dim=128, page=16, dtype=torch.bfloat16,
                 heads_first=True, seed=0, spread=1.5, spare_tokens=0, garbage=float("nan"), poison=True):
        g = torch.Generator(device="cpu").manual_seed(seed)
        self.n_q, self.kv, self.prefix, self.page, self.dtype = list(n_q), list(kv), prefix, page, dtype
        self.heads_q, self.heads_kv, self.dim = heads_q, heads_kv, dim
        B, self.B = len(n_q), len(n_q)
        self.T = sum(n_q) + spare_tokens
        width = max(1, max((-(-k // page) for k in kv), default=1))
        shared = -(-prefix // page)
        n_pages = B * width + shared + 2
        order = torch.randperm(n_pages, generator=g).to(torch.int32)
        shape = (n_pages, heads_kv, page, dim) if heads_first else (n_pages, page, heads_kv, dim)
        turn = (0, 2, 1, 3) if heads_first else (0, 1, 2, 3)
        pages = [torch.full(shape, garbage).permute(turn) for _ in range(2)]
        table, prefix_table = order[:B * width].view(B, width), order[B * width:B * width + shared]
        for t in pages:
            for rows, lens in [(prefix_table[None], [prefix]), (table, kv)]:
                for b, n in enumerate(lens):
                    for e in range(-(-n // page)):
                        part = min(page, n - e * page)
                        t[rows[b, e].item(), :part] = torch.randn((part, heads_kv, dim), generator=g)
        self.q = (spread * torch.randn((self.T, heads_q, dim), generator=g)).to(dtype).cuda()
        self.k, self.v = (t.to(dtype).cuda() for t in pages)
        # entries that no length reaches point nowhere
        self.table_host = table.clone()
        if poison:
            for b in range(B):
                self.table_host[b, -(-kv[b] // page):] = 0x7FFFFFFF
        self.table, self.prefix_table = self.table_host.cuda(), prefix_table.cuda()
        self.kv_len = torch.tensor(kv, dtype=torch.int32).cuda()
        cu = [0]
        for n in n_q:
            cu.append(cu[-1] + n)
        self.cu = cu
        self.cu_q = torch.tensor(cu, dtype=torch.int32).cuda()

    def cache(self, qg):
        return qg.KVCache(self.k, self.v)

    def batch(self, qg, **kw):
        args = dict(max_kv=max(self.kv, default=0), cu_q=self.cu_q, max_q=max(max(self.n_q, default=1), 1), tokens=self.T,
                    prefix_table=self.prefix_table if self.prefix else None, prefix_len=self.prefix)
        args.update(kw)
        return qg.KVBatch(self.table, self.kv_len, **args)

    def _gather(self, pages, rows, n):
        return pages[rows.long()].flatten(0, 1)[:n].double()      # [n, heads_kv, dim]

    def reference(self, scale=None):
        """out, lse [T, heads_q(, dim)] in 64 bits, and the bound of |out error| per element before the last rounding."""
        G, D = self.heads_q // self.heads_kv, self.dim
        scale = D ** -0.5 if scale is None else scale
        u = UNIT[self.dtype]
        out = torch.zeros((self.T, self.heads_q, D), dtype=torch.float64, device="cuda")
        lse = torch.full((self.T, self.heads_q), -math.inf, dtype=torch.float64, device="cuda")
        bound = torch.zeros_like(out)
        lse_bound = torch.zeros_like(lse)
        kp, vp = (self._gather(t, self.prefix_table, self.prefix) for t in (self.k, self.v))
        for b in range(self.B):
            n, L = self.n_q[b], self.kv[b]
            pages = self.table[b, :-(-L // self.page)]
            ks, vs = (torch.cat([p, self._gather(t, pages, L)]) for p, t in ((kp, self.k), (vp, self.v)))
            for i in range(n):
                t = self.cu[b] + i
                seen = self.prefix + max(0, L - n + i + 1)
                if seen <= 0:
                    continue
                q = self.q[t].double().view(self.heads_kv, G, D)
                k, v = ks[:seen].transpose(0, 1), vs[:seen].transpose(0, 1)          # [heads_kv, seen, dim]
                s = scale * q @ k.transpose(1, 2)
                m = s.amax(-1, keepdim=True)
                e = torch.exp(s - m)
                total = e.sum(-1, keepdim=True)
                p = e / total
                out[t] = (p @ v).view(self.heads_q, D)
                lse[t] = (m + total.log()).view(self.heads_q)
                # each logit: D fp32 products summed, |error| <= D 2^-24 scale |q||k|; 2^-21 covers the exponential and
                # its argument's rounding (|s - m| log2 e up to 64 in fp32); seen 2^-24 the sums over keys
                size = scale * q.norm(dim=-1, keepdim=True) * k.norm(dim=-1).amax(-1)[:, None, None]
                rel = 2 * (D * 2.0 ** -24 * size + 2.0 ** -18) + 2 * seen * 2.0 ** -24
                pv = p @ v.abs()
                # p rounded to the cache's type: relative u, and in fp16 at least half its smallest step
                floor = 2.0 ** -25 * v.abs().sum(1, keepdim=True) / total if self.dtype == torch.float16 else 0.0
                bound[t] = ((u + rel) * pv + floor).view(self.heads_q, D)
                lse_bound[t] = (rel + 2.0 ** -22 * (m.abs() + total.log() + 1)).view(self.heads_q)
        return out, lse, bound, lse_bound


def check_attention(case, out, lse=None, scale=None):
    ref, ref_lse, bound, lse_bound = case.reference(scale)
    used = case.cu[-1]
    got = out[:used].double()
    assert torch.isfinite(got).all()
    err = (got - ref[:used]).abs()
    room = bound[:used] + UNIT[out.dtype] * (ref[:used].abs() + bound[:used]) + 2.0 ** -25
    worst = (err / room).max().item() if err.numel() else 0.0
    assert worst <= 1.0, worst
    if lse is not None:
        none = torch.isinf(ref_lse[:used])
        assert torch.equal(torch.isinf(lse[:used]), none) and (lse[:used][none] < 0).all()
        off = (lse[:used].double() - ref_lse[:used])[~none].abs()
        assert (off <= lse_bound[:used][~none]).all()
