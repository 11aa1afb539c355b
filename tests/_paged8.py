"""8-bit paged-cache test helpers: the codec's definition in 64 bits, and seeded
batches over such a cache with attention's definition and error bounds."""
import math

import torch

from _paged import UNIT, Case

E4M3 = torch.float8_e4m3fn
BLOCK, E_MIN, E_MAX = 16, -64, 63
NAN_CODE = 0x7F


def exponent(amax):
    """The least e with amax <= 448 * 2^e, within E_MIN .. E_MAX (64 bits)."""
    m, x = torch.frexp(amax.double())          # m in [0.5, 1); 448 = 0.875 * 2^9
    e = x - 9 + (m > 0.875).to(x.dtype)
    return torch.where(amax > 0, e, E_MIN).clamp(E_MIN, E_MAX)


def nearest(z):
    """The nearest E4M3 value of z (64 bits, |z| at most 448 or NaN), ties to even."""
    step = torch.exp2(torch.floor(torch.log2(z.abs().clamp(min=2.0 ** -6))) - 3)
    return torch.round(z / step) * step


def pow2(e):
    return torch.exp2(e.double())


def quantised(x):
    """codes (uint8, of x's shape) and scale bytes of x [pages, page, heads, dim]; NaN values become NaN codes."""
    b = x.double().unflatten(1, (-1, BLOCK))
    fine = torch.isfinite(b)
    e = exponent(torch.where(fine, b, 0.0).abs().amax((2, 4)))
    z = torch.where(fine, nearest(torch.where(fine, b, 0.0) * pow2(-e)[:, :, None, :, None]), math.nan)
    codes = z.flatten(1, 2).float().to(E4M3).view(torch.uint8)
    return codes, torch.where(fine.any(4).any(2), e + 127, 255).to(torch.uint8)


def values(codes, scale):
    """What codes [pages, page, heads, dim] and scale bytes [pages, blocks, heads] stand for (64 bits)."""
    x = codes.view(E4M3).double().unflatten(1, (-1, BLOCK))
    return (x * pow2(scale.int() - 127)[:, :, None, :, None]).flatten(1, 2)


class Case8(Case):
    """A Case over an 8-bit cache: heads of magnitudes 2^gain apart and blocks of magnitudes 2^swing apart, codes and
    scales past a length NaN and 255.  k and v hold what the cache stands for."""

    def __init__(self, *args, dtype=torch.bfloat16, gain=1.5, swing=1.0, **kw):
        args = list(args)
        if len(args) > 7:
            dtype = args.pop(7)
        heads_first = args.pop(7) if len(args) > 7 else kw.pop("heads_first", True)
        super().__init__(*args, dtype=torch.float32, heads_first=heads_first, **kw)
        g = torch.Generator(device="cpu").manual_seed(kw.get("seed", 0) + 1000)
        self.dtype, self.q = dtype, self.q.to(dtype)
        for name in ("k", "v"):
            x = getattr(self, name)
            pages, page, heads, dim = x.shape
            amount = gain * torch.randn((1, 1, heads), generator=g) + swing * torch.randn((pages, page // BLOCK, heads), generator=g)
            x = x * torch.exp2(amount).cuda().repeat_interleave(BLOCK, 1)[..., None]
            codes, scale = quantised(x)
            if heads_first:
                codes, scale = (t.transpose(1, 2).contiguous().transpose(1, 2) for t in (codes, scale))
            setattr(self, name + "_codes", codes)
            setattr(self, name + "_scale", scale)
        self.refresh()

    def refresh(self):
        self.k, self.v = values(self.k_codes, self.k_scale), values(self.v_codes, self.v_scale)

    def cache(self, qg):
        return qg.KVCache8(self.k_codes.view(E4M3), self.v_codes.view(E4M3), self.k_scale, self.v_scale)

    def _scales(self, rows, n):
        return pow2(self.v_scale[rows.long()].flatten(0, 1).repeat_interleave(BLOCK, 0)[:n].int() - 127)   # [n, heads_kv]

    def reference(self, scale=None):
        G, D, H = self.heads_q // self.heads_kv, self.dim, self.heads_kv
        scale = D ** -0.5 if scale is None else scale
        out = torch.zeros((self.T, self.heads_q, D), dtype=torch.float64, device="cuda")
        lse = torch.full((self.T, self.heads_q), -math.inf, dtype=torch.float64, device="cuda")
        bound, lse_bound = torch.zeros_like(out), torch.zeros_like(lse)
        kp, vp = (self._gather(t, self.prefix_table, self.prefix) for t in (self.k, self.v))
        ep = self._scales(self.prefix_table, self.prefix)
        for b in range(self.B):
            n, L = self.n_q[b], self.kv[b]
            if n == 0:
                continue
            pages = self.table[b, :-(-L // self.page)]
            k, v = (torch.cat([p, self._gather(t, pages, L)]).transpose(0, 1) for p, t in ((kp, self.k), (vp, self.v)))
            ev = torch.cat([ep, self._scales(pages, L)]).T[:, None, None]                      # [heads_kv, 1, 1, keys]
            t0 = self.cu[b]
            q = self.q[t0:t0 + n].double().view(n, H, G, D).permute(1, 0, 2, 3)                # [heads_kv, n, G, D]
            s = scale * torch.einsum("hngd,hkd->hngk", q, k)
            seen = self.prefix + (L - n + 1 + torch.arange(n, device="cuda")).clamp(min=0)     # keys each token sees
            keys = k.shape[1]
            there = torch.arange(keys, device="cuda") < seen[:, None]                          # [n, keys]
            if keys == 0:
                continue
            s = torch.where(there[None, :, None], s, -math.inf)
            m = s.amax(-1, keepdim=True)
            m0 = torch.where(m > -math.inf, m, 0.0)
            e = torch.exp(s - m0)
            total = e.sum(-1, keepdim=True)
            some = total > 0
            p = torch.where(some, e / torch.where(some, total, 1.0), 0.0)
            o = torch.einsum("hngk,hkd->hngd", p, v)
            # each logit: D fp32 products summed, |error| <= D 2^-24 scale |q||k| (and the scalings' roundings); 2^-18 covers
            # the exponential and its argument's rounding (|s - m| log2 e up to 64, the exponents' share 128, in fp32)
            size = scale * q.norm(dim=-1, keepdim=True) * k.norm(dim=-1).amax(-1)[:, None, None, None]
            rel = 2 * (D * 2.0 ** -24 * size + 2.0 ** -17) + 2 * keys * 2.0 ** -24
            pv = torch.einsum("hngk,hkd->hngd", p, v.abs())
            # the probabilities weighted with their V scales are rounded to fp16: 2^-11 of each, or 2^-25 of the row's largest
            # (the reference of any part the keys are split into is no larger)
            most = (p * ev).amax(-1, keepdim=True)
            floor = 2.0 ** -25 * most * torch.einsum("nk,hkd->hnd", there.double(), (v / ev[:, 0, 0, :, None]).abs())[:, :, None]
            room = (UNIT[torch.float16] + rel) * pv + floor
            out[t0:t0 + n] = o.permute(1, 0, 2, 3).reshape(n, self.heads_q, D)
            bound[t0:t0 + n] = room.permute(1, 0, 2, 3).reshape(n, self.heads_q, D)
            row = lambda t: t[..., 0].permute(1, 0, 2).reshape(n, self.heads_q)
            some_ln = torch.where(some, total, 1.0).log()
            lse[t0:t0 + n] = row(torch.where(some, m0 + some_ln, -math.inf))
            # an fp32 number of size |lse| in powers of two, weighted by exponents up to 64 more
            lse_bound[t0:t0 + n] = row(rel + 2.0 ** -22 * (m0.abs() + some_ln.abs() + 64))
        return out, lse, bound, lse_bound
