"""The example's decoding step over an 8-bit cache with normed heads: the append,
the attention and the o product follow from what the cache holds."""
import pytest
import torch

from test_gpu_decode_step import _dense, _turn, example  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sequences,prefix", [(6, 300), (40, 1100)])
def test_steps_follow_from_the_cache(example, sequences, prefix):  # noqa: F811
    import bit_weight_only_group_gb300 as qg
    hidden, hq, hkv, d, room = 1024, 8, 2, 128, 128
    layer, table, prefix_table, rope, _ = example.build(hidden, hq, hkv, d, sequences, prefix, room, seed=sequences, cache_bits=8)
    wq, wo = _dense(layer.qkv[0]), _dense(layer.o)
    ints = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
    kv_len = torch.zeros(sequences, dtype=torch.int32, device="cuda")
    batch = qg.KVBatch(table, kv_len, max_kv=room, prefix_table=prefix_table, prefix_len=prefix)
    whole = qg.KVBatch(prefix_table.view(1, -1), ints(prefix), max_kv=prefix, cu_q=ints(0, prefix), max_q=prefix, tokens=prefix)
    kp, vp = (t.double()[None].expand(sequences, -1, -1, -1) for t in qg.qkv_read(layer.cache, whole, dtype=torch.float32))
    x = torch.randn((sequences, hidden), device="cuda").bfloat16()
    for i in range(3):
        kv_len += 1
        y = layer.step(x, batch, rope)
        own = qg.KVBatch(table, kv_len, max_kv=room, cu_q=(i + 1) * torch.arange(sequences + 1, dtype=torch.int32, device="cuda"),
                         max_q=i + 1, tokens=sequences * (i + 1))
        k, v = (torch.cat([p, t.double().view(sequences, i + 1, hkv, d)], 1)
                for p, t in zip((kp, vp), qg.qkv_read(layer.cache, own, dtype=torch.float32)))
        q = (x.double() @ wq.T).view(-1, hq, d)
        q = q / (q.square().mean(-1, keepdim=True) + 1e-6).sqrt()
        q = _turn(q, rope, torch.full((sequences,), prefix + i, device="cuda")).view(sequences, hkv, hq // hkv, d)
        p = torch.softmax(torch.einsum("shgd,skhd->shgk", q, k) / d ** 0.5, -1)
        ref = torch.einsum("shgk,skhd->shgd", p, v).reshape(sequences, -1) @ wo.T
        # roundings to bf16 on the way (the q product's output, q, the attention's and the last output; x is given), each at
        # most 2^-8 of a value and of either sign; a norm's error in the product's output counts twice: their root sum of
        # squares, 6 of them, bounds the relative norm
        off = (y.double() - ref).norm() / ref.norm()
        assert off <= 6 ** 0.5 * 2.0 ** -8, off
        x = (x.float() + y.float()).bfloat16()
    torch.cuda.synchronize()
    assert qg.qgemm_device_status() == 0


def test_example_runs(example, capsys):  # noqa: F811
    example.main(2, cache_bits=8)
    assert "step 1" in capsys.readouterr().out
