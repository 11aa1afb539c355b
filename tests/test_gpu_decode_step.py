"""The example's decoding step against the same step computed in 64 bits from
the dequantized weights: products, append, attention and the o product together."""
import importlib.util
import os

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def example():
    spec = importlib.util.spec_from_file_location("decode_step", os.path.join(ROOT, "examples", "decode_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _dense(qw):
    """The weights a 4-bit QWeight stands for, fp64."""
    b = qw.packed.cpu().numpy()
    q = np.stack([b & 15, b >> 4], -1).reshape(qw.N, qw.K).astype(np.float64)
    scale = qw.scale.cpu().numpy().view(np.float16).astype(np.float64)
    zp = qw.zp.cpu().numpy().astype(np.float64)
    rep = lambda a: np.repeat(a, qw.group, 1)
    return torch.from_numpy((q - rep(zp)) * rep(scale)).cuda()


def _turn(x, rope, at):
    half = x.shape[-1] // 2
    cos, sin = rope[at, :half].double()[:, None], rope[at, half:].double()[:, None]
    a, b = x[..., :half], x[..., half:]
    return torch.cat([a * cos - b * sin, b * cos + a * sin], -1)


@pytest.mark.parametrize("sequences,prefix", [(6, 300), (3, 20), (40, 1100)])
def test_steps_follow_the_definition(example, sequences, prefix):
    import bit_weight_only_group_gb300 as qg
    hidden, hq, hkv, d, steps = 1024, 8, 2, 128, 3
    layer, table, prefix_table, rope, xp = example.build(hidden, hq, hkv, d, sequences, prefix, seed=sequences)
    wq, wk, wv, wo = (_dense(w) for w in (*layer.qkv, layer.o))
    kv_len = torch.zeros(sequences, dtype=torch.int32, device="cuda")
    batch = qg.KVBatch(table, kv_len, max_kv=128, prefix_table=prefix_table, prefix_len=prefix)
    heads = lambda x, w, n: (x.double() @ w.T).view(-1, n, d)
    at = torch.arange(prefix, device="cuda")
    keys = [_turn(heads(xp, wk, hkv), rope, at)[None].expand(sequences, -1, -1, -1)]
    vals = [heads(xp, wv, hkv)[None].expand(sequences, -1, -1, -1)]
    x = torch.randn((sequences, hidden), device="cuda").bfloat16()
    for i in range(steps):
        kv_len += 1
        y = layer.step(x, batch, rope)
        at = torch.full((sequences,), prefix + i, device="cuda")
        keys.append(_turn(heads(x, wk, hkv), rope, at)[:, None])
        vals.append(heads(x, wv, hkv)[:, None])
        k, v = torch.cat(keys, 1), torch.cat(vals, 1)
        q = _turn(heads(x, wq, hq), rope, at).view(sequences, hkv, hq // hkv, d)
        p = torch.softmax(torch.einsum("shgd,skhd->shgk", q, k) / d ** 0.5, -1)
        ref = torch.einsum("shgk,skhd->shgd", p, v).reshape(sequences, -1) @ wo.T
        # roundings to bf16 on the way (q, k, v and their products' outputs, p, the attention's and the last output), each
        # at most 2^-8 of a value and of either sign: their root sum of squares, 8 of them, bounds the relative norm
        off = (y.double() - ref).norm() / ref.norm()
        assert off <= 8 ** 0.5 * 2.0 ** -8, off
        x = (x.float() + y.float()).bfloat16()
    torch.cuda.synchronize()
    assert qg.qgemm_device_status() == 0


def test_example_runs(example, capsys):
    example.main(2)
    assert "step 1" in capsys.readouterr().out
