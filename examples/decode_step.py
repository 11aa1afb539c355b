"""The attention half of a decoder layer, one decoding step: the fused q/k/v
product over 4-bit weights, the new tokens appended to the paged cache with the
position rotation, attention over a prefix that all sequences share and their
own tokens, and the o product.

    python examples/decode_step.py [8]

With 8 the cache holds 8-bit codes, and the heads of q and k are normed before
the rotation.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_weight_only_group_gb300 as qg  # noqa: E402


def rope_table(positions: int, dim: int, base: float = 10000.0) -> torch.Tensor:
    """fp32 [positions, dim]: the cosines, then the sines of each position's angles."""
    freq = base ** (-torch.arange(0, dim, 2, dtype=torch.float64) / dim)
    angle = torch.arange(positions, dtype=torch.float64)[:, None] * freq
    return torch.cat([angle.cos(), angle.sin()], 1).float().cuda()


class AttentionLayer:
    """Quantized q/k/v/o matrices [out, in] of one layer, and its cache."""

    def __init__(self, wq, wk, wv, wo, heads_q, heads_kv, head_dim, num_pages, page_size=64, bits=4, group=128,
                 cache_bits=16, q_norm=None, k_norm=None):
        self.qkv = [qg.qpack_quantize(w, bits, group) for w in (wq, wk, wv)]
        self.o = qg.qpack_quantize(wo, bits, group)
        self.heads_q, self.heads_kv, self.head_dim = heads_q, heads_kv, head_dim
        self.cache = (qg.KVCache8 if cache_bits == 8 else qg.KVCache).empty(num_pages, page_size, heads_kv, head_dim)
        self.norms = dict(q_norm=q_norm, k_norm=k_norm)

    def step(self, x: torch.Tensor, batch: "qg.KVBatch", rope: torch.Tensor) -> torch.Tensor:
        """x [T, hidden] (bf16), the new tokens of the batch -> [T, hidden] (bf16).  The batch's lengths count them."""
        q, k, v = qg.qgemm_forward_multi(x, self.qkv, out_dtype=torch.bfloat16)
        q, k, v = (y.view(x.shape[0], -1, self.head_dim) for y in (q, k, v))
        q = qg.qkv_append(self.cache, batch, k, v, q=q, rope=rope, **self.norms)
        y = qg.qattn_forward(q, self.cache, batch)
        return qg.qgemm_forward(y.flatten(1), self.o, out_dtype=torch.bfloat16)


def build(hidden=1024, heads_q=8, heads_kv=2, head_dim=128, sequences=6, prefix=300, room=128, page_size=64, seed=0,
          cache_bits=16):
    """A layer with random weights, its pages dealt out, and the prefix already in the cache."""
    g = torch.Generator().manual_seed(seed)
    w = lambda n, k: (torch.randn((n, k), generator=g) * 0.02).half().cuda()
    width, shared = -(-room // page_size), -(-prefix // page_size)
    layer = AttentionLayer(w(heads_q * head_dim, hidden), w(heads_kv * head_dim, hidden), w(heads_kv * head_dim, hidden),
                           w(hidden, heads_q * head_dim), heads_q, heads_kv, head_dim, sequences * width + shared, page_size,
                           cache_bits=cache_bits, **({n: torch.ones(head_dim, device="cuda") for n in ("q_norm", "k_norm")}
                                                     if cache_bits == 8 else {}))
    pages = torch.randperm(sequences * width + shared, generator=g).to(torch.int32).cuda()
    table, prefix_table = pages[:sequences * width].view(sequences, width), pages[sequences * width:]
    rope = rope_table(prefix + room, head_dim)
    # the prefix goes through the layer once, as one sequence over its own pages
    x = torch.randn((prefix, hidden), generator=g).bfloat16().cuda()
    layer.step(x, qg.KVBatch(prefix_table.view(1, -1), torch.tensor([prefix], dtype=torch.int32).cuda(), max_kv=prefix,
                             cu_q=torch.tensor([0, prefix], dtype=torch.int32).cuda(), max_q=prefix, tokens=prefix), rope)
    return layer, table, prefix_table, rope, x


def main(steps: int = 4, cache_bits: int = 16):
    sequences, prefix, room, hidden = 6, 300, 128, 1024
    layer, table, prefix_table, rope, _ = build(hidden, sequences=sequences, prefix=prefix, room=room, cache_bits=cache_bits)
    kv_len = torch.zeros(sequences, dtype=torch.int32, device="cuda")
    batch = qg.KVBatch(table, kv_len, max_kv=room, prefix_table=prefix_table, prefix_len=prefix)
    x = torch.randn((sequences, hidden), device="cuda").bfloat16()
    for i in range(steps):
        kv_len += 1
        x = x + layer.step(x, batch, rope)
        print(f"step {i}: {sequences} tokens at position {prefix + i}, |x| = {x.float().norm().item():.3f}")
    if qg.qgemm_device_status() != 0:
        raise SystemExit("the device status word reports an error")


if __name__ == "__main__":
    main(cache_bits=8 if sys.argv[1:] == ["8"] else 16)
