"""The paged-cache entry points without a GPU: every refusal is made on the
host before anything is launched, and the size query answers there."""
import ctypes
import math

import pytest


@pytest.fixture(scope="module")
def qg():
    from bit_weight_only_group_gb300 import build
    build.build()
    import bit_weight_only_group_gb300 as qg
    return qg


def _cache(qg, **kw):
    # 100 pages of 64 tokens, 8 heads of 128, heads first
    d = dict(k=0x100000, v=0x200000, dtype=1, num_pages=100, page_size=64, heads_kv=8, head_dim=128,
             page_stride=8 * 64 * 128, token_stride=128, head_stride=64 * 128)
    d.update(kw)
    return qg.QgKvCache(*d.values())


def _batch(qg, **kw):
    d = dict(sequences=4, tokens=4, max_q=1, max_kv=200, table_ld=4, prefix_len=1000, table=0x300000, kv_len=0x310000,
             cu_q=0x320000, prefix_table=0x330000)
    d.update(kw)
    return qg.QgKvBatch(*d.values())


Q, OUT, WS = 0x400000, 0x500000, 0x600000


def _attn(qg, cache=None, batch=None, q=Q, ldq=64 * 128, heads_q=64, scale=0.1, out=OUT, ldo=64 * 128, ot=1, lse=None,
          ws=None, ws_bytes=0):
    cache, batch = cache or _cache(qg), batch or _batch(qg)
    return qg.lib().qattn_forward(ctypes.byref(cache), ctypes.byref(batch), q, ldq, heads_q, scale, out, ldo, ot, lse, ws,
                                  ws_bytes, None)


def _append(qg, cache=None, batch=None, rope=None, q=Q, ldq=64 * 128, heads_q=64, k=0x410000, ldk=1024, v=0x420000, ldv=1024,
            xt=1, q_out=OUT, ldq_out=64 * 128):
    cache, batch = cache or _cache(qg), batch or _batch(qg)
    return qg.lib().qkv_append(ctypes.byref(cache), ctypes.byref(batch), ctypes.byref(rope) if rope else None, q, ldq, heads_q,
                               k, ldk, v, ldv, xt, q_out, ldq_out, None)


BAD_CACHES = [(dict(k=None), -1), (dict(v=None), -1), (dict(dtype=0), -2), (dict(dtype=7), -2), (dict(head_dim=96), -2),
              (dict(head_dim=256), -2), (dict(page_size=8), -2), (dict(page_size=48), -2), (dict(page_size=2048), -2),
              (dict(num_pages=0), -1), (dict(heads_kv=0), -1), (dict(k=0x100008), -3), (dict(v=0x200002), -3),
              (dict(token_stride=100), -1), (dict(token_stride=132), -3), (dict(head_stride=0), -1),
              (dict(page_stride=1 << 38), -1), (dict(page_stride=8 * 64 * 128 + 4), -3)]
BAD_BATCHES = [(dict(sequences=-1), -1), (dict(tokens=-1), -1), (dict(max_kv=-1), -1), (dict(prefix_len=-5), -1),
               (dict(max_q=0), -1), (dict(kv_len=None), -1), (dict(table=None), -1), (dict(table_ld=3), -1),
               (dict(prefix_table=None), -1), (dict(cu_q=None, tokens=5), -1), (dict(cu_q=None, max_q=2), -1),
               (dict(kv_len=0x310002), -3), (dict(table=0x300001), -3), (dict(prefix_len=1 << 30), -2)]


@pytest.mark.parametrize("change,expect", BAD_CACHES)
def test_bad_caches(qg, change, expect):
    c = _cache(qg, **change)
    assert _attn(qg, cache=c) == expect, qg.last_error()
    assert _append(qg, cache=c) == expect, qg.last_error()


@pytest.mark.parametrize("change,expect", BAD_BATCHES)
def test_bad_batches(qg, change, expect):
    b = _batch(qg, **change)
    assert _attn(qg, batch=b) == expect, qg.last_error()
    assert _append(qg, batch=b) == expect, qg.last_error()


def test_null_descriptors(qg):
    L = qg.lib()
    assert L.qattn_forward(None, None, Q, 0, 1, 1.0, OUT, 0, 1, None, None, 0, None) == -1
    assert L.qkv_append(None, None, None, None, 0, 0, None, 0, None, 0, 1, None, 0, None) == -1
    assert L.qattn_workspace_size(None, None, 1, None) == -1


@pytest.mark.parametrize("change,expect", [
    (dict(heads_q=60), -1), (dict(heads_q=0), -1), (dict(scale=0.0), -1), (dict(scale=-1.0), -1), (dict(scale=math.nan), -1),
    (dict(scale=math.inf), -1), (dict(scale=3e38), -1), (dict(ot=3), -1), (dict(q=None), -1), (dict(out=None), -1),
    (dict(ldq=64 * 128 - 8), -1), (dict(ldq=64 * 128 + 4), -3), (dict(q=Q + 8), -3), (dict(out=OUT + 4), -3),
    (dict(ldo=64 * 128 + 2, ot=0), -3), (dict(lse=0x700002), -3), ({}, -4), (dict(ws=WS + 16, ws_bytes=1 << 40), -3)])
def test_bad_attention_arguments(qg, change, expect):
    assert _attn(qg, **change) == expect, qg.last_error()


@pytest.mark.parametrize("change,expect", [
    (dict(xt=3), -1), (dict(heads_q=-1), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(q=None), -1), (dict(q_out=None), -1),
    (dict(ldk=1000), -1), (dict(ldv=1028), -3), (dict(k=0x410008), -3), (dict(q_out=OUT + 2), -3)])
def test_bad_append_arguments(qg, change, expect):
    assert _append(qg, **change) == expect, qg.last_error()


@pytest.mark.parametrize("rope,expect", [
    (dict(table=None), -1), (dict(dim=8), -2), (dict(dim=24), -2), (dict(dim=144), -2), (dict(positions=0), -1),
    (dict(table=0x800004), -3), (dict(at=0x810002), -3)])
def test_bad_rotations(qg, rope, expect):
    d = dict(table=0x800000, at=None, positions=100, dim=128, interleaved=0)
    d.update(rope)
    assert _append(qg, rope=qg.QgRope(*d.values())) == expect, qg.last_error()


def test_nothing_to_do(qg):
    # no sequences or no tokens: accepted without a GPU, nothing is launched
    for kw in (dict(sequences=0), dict(tokens=0)):
        assert _attn(qg, batch=_batch(qg, **kw)) == 0
        assert _append(qg, batch=_batch(qg, **kw)) == 0


def test_workspace_size_on_the_host(qg):
    def need(**kw):
        b, n = _batch(qg, **kw), ctypes.c_size_t()
        assert qg.lib().qattn_workspace_size(ctypes.byref(_cache(qg)), ctypes.byref(b), 64, ctypes.byref(n)) == 0
        return n.value

    assert need(sequences=0) == 0 and need(tokens=0) == 0
    assert need(prefix_len=0, max_kv=10) == 0                      # one part: results are written at once
    row = 64 * (128 * 4 + 8)                                      # one part of one token
    assert need() >= 2 * 4 * row and need() % 256 == 0
    assert need(tokens=2000, max_q=600, max_kv=256) >= 2 * 2000 * row
    assert need(tokens=2000, max_q=600, max_kv=256) < 8 * 2000 * row


def test_workspace_of_long_prompts_does_not_grow_with_them(qg):
    # only the pieces at the ends of the CTAs' runs are kept there
    def need(tokens):
        b, n = _batch(qg, sequences=1, tokens=tokens, max_q=tokens, max_kv=tokens, table_ld=-(-tokens // 64), prefix_len=0), ctypes.c_size_t()
        assert qg.lib().qattn_workspace_size(ctypes.byref(_cache(qg)), ctypes.byref(b), 64, ctypes.byref(n)) == 0
        return n.value

    row = 128 * 4 + 8
    layout = lambda tokens: 64 + 16 * (tokens // 32 + 2) + 2048   # a few words a pair of tiles
    for tokens in (4096, 8192, 65536, 131072):
        assert need(tokens) <= (1 << 18) * row + layout(tokens)
    assert need(20) <= 2 * 20 * 64 * row + 16 * 256 * row + layout(20)
