"""The 8-bit paged cache's entry points and the norms without a GPU: every
refusal is made on the host before anything is launched, and the size query
answers there; the Python checks with stand-ins for tensors."""
import ctypes
import math

import pytest
import torch

from test_kv_devices_cpu import Fake, qg as devices_qg  # noqa: F401  (the fixture with a library that counts its calls)


@pytest.fixture(scope="module")
def qg():
    from bit_weight_only_group_gb300 import build
    build.build()
    import bit_weight_only_group_gb300 as qg
    return qg


def _cache(qg, **kw):
    # 100 pages of 64 tokens, 8 heads of 128, heads first
    d = dict(k=0x100000, v=0x200000, k_scale=0x300001, v_scale=0x310003, num_pages=100, page_size=64, heads_kv=8,
             head_dim=128, page_stride=8 * 64 * 128, token_stride=128, head_stride=64 * 128, scale_page_stride=32,
             scale_block_stride=1, scale_head_stride=4)
    d.update(kw)
    return qg.QgKv8Cache(*d.values())


def _batch(qg, **kw):
    d = dict(sequences=4, tokens=4, max_q=1, max_kv=200, table_ld=4, prefix_len=1000, table=0x400000, kv_len=0x410000,
             cu_q=0x420000, prefix_table=0x430000)
    d.update(kw)
    return qg.QgKvBatch(*d.values())


Q, OUT, WS = 0x500000, 0x600000, 0x700000


def _attn(qg, cache=None, batch=None, q=Q, ldq=64 * 128, heads_q=64, qt=1, scale=0.1, out=OUT, ldo=64 * 128, ot=1, lse=None,
          ws=None, ws_bytes=0):
    cache, batch = cache or _cache(qg), batch or _batch(qg)
    return qg.lib().qattn8_forward(ctypes.byref(cache), ctypes.byref(batch), q, ldq, heads_q, qt, scale, out, ldo, ot, lse,
                                   ws, ws_bytes, None)


def _append(qg, cache=None, batch=None, norm=None, rope=None, q=Q, ldq=64 * 128, heads_q=64, k=0x510000, ldk=1024, v=0x520000,
            ldv=1024, xt=1, q_out=OUT, ldq_out=64 * 128, qt=1):
    cache, batch = cache or _cache(qg), batch or _batch(qg)
    ref = lambda x: ctypes.byref(x) if x is not None else None
    return qg.lib().qkv8_append(ctypes.byref(cache), ctypes.byref(batch), ref(norm), ref(rope), q, ldq, heads_q, k, ldk, v, ldv,
                                xt, q_out, ldq_out, qt, None)


def _read(qg, cache=None, batch=None, k=0x510000, ldk=1024, v=0x520000, ldv=1024, ot=1):
    cache, batch = cache or _cache(qg), batch or _batch(qg)
    return qg.lib().qkv8_read(ctypes.byref(cache), ctypes.byref(batch), k, ldk, v, ldv, ot, None)


@pytest.mark.parametrize("change,expect", [
    (dict(k=None), -1), (dict(v=None), -1), (dict(k_scale=None), -1), (dict(v_scale=None), -1), (dict(head_dim=96), -2),
    (dict(page_size=8), -2), (dict(page_size=48), -2), (dict(page_size=2048), -2), (dict(num_pages=0), -1), (dict(heads_kv=0), -1),
    (dict(k=0x100008), -3), (dict(v=0x200002), -3), (dict(token_stride=100), -1), (dict(token_stride=136), -3),
    (dict(head_stride=0), -1), (dict(page_stride=1 << 38), -1), (dict(page_stride=8 * 64 * 128 + 8), -3),
    (dict(scale_page_stride=0), -1), (dict(scale_block_stride=-1), -1), (dict(scale_head_stride=1 << 38), -1)])
def test_bad_caches(qg, change, expect):
    c = _cache(qg, **change)
    for call in (_attn, _append, _read):
        assert call(qg, cache=c) == expect, qg.last_error()


@pytest.mark.parametrize("change,expect", [
    (dict(sequences=-1), -1), (dict(tokens=-1), -1), (dict(max_kv=-1), -1), (dict(max_q=0), -1), (dict(kv_len=None), -1),
    (dict(table=None), -1), (dict(table_ld=3), -1), (dict(prefix_table=None), -1), (dict(cu_q=None, tokens=5), -1),
    (dict(cu_q=None, max_q=2), -1), (dict(kv_len=0x410002), -3), (dict(prefix_len=1 << 30), -2)])
def test_bad_batches(qg, change, expect):
    b = _batch(qg, **change)
    for call in (_attn, _append, _read):
        assert call(qg, batch=b) == expect, qg.last_error()


@pytest.mark.parametrize("change,expect", [
    (dict(heads_q=60), -1), (dict(heads_q=0), -1), (dict(qt=0), -1), (dict(qt=3), -1), (dict(scale=0.0), -1),
    (dict(scale=math.nan), -1), (dict(scale=math.inf), -1), (dict(ot=3), -1), (dict(q=None), -1), (dict(out=None), -1),
    (dict(ldq=64 * 128 - 8), -1), (dict(ldq=64 * 128 + 4), -3), (dict(q=Q + 8), -3), (dict(ldo=64 * 128 + 2, ot=0), -3),
    (dict(lse=0x700002), -3), ({}, -4), (dict(ws=WS + 16, ws_bytes=1 << 40), -3)])
def test_bad_attention_arguments(qg, change, expect):
    assert _attn(qg, **change) == expect, qg.last_error()


@pytest.mark.parametrize("change,expect", [
    (dict(xt=3), -1), (dict(qt=0), -1), (dict(heads_q=-1), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(q=None), -1),
    (dict(q_out=None), -1), (dict(ldk=1000), -1), (dict(ldv=1028), -3), (dict(k=0x510008), -3), (dict(q_out=OUT + 2), -3)])
def test_bad_append_arguments(qg, change, expect):
    assert _append(qg, **change) == expect, qg.last_error()


@pytest.mark.parametrize("change,expect", [(dict(ot=3), -1), (dict(k=None), -1), (dict(v=None), -1), (dict(ldk=1000), -1),
                                           (dict(ldk=1026, ot=0), -3), (dict(v=0x520004), -3)])
def test_bad_read_arguments(qg, change, expect):
    assert _read(qg, **change) == expect, qg.last_error()


@pytest.mark.parametrize("change,expect", [(dict(dtype=3), -1), (dict(eps=-1.0), -1), (dict(eps=math.nan), -1),
                                           (dict(eps=math.inf), -1), (dict(q=0x800004), -3), (dict(k=0x810008), -3)])
def test_bad_norms(qg, change, expect):
    d = dict(q=0x800000, k=0x810000, dtype=0, eps=1e-6)
    d.update(change)
    n = qg.QgHeadNorm(*d.values())
    assert _append(qg, norm=n) == expect, qg.last_error()
    c = qg.QgKvCache(0x100000, 0x200000, 1, 100, 64, 8, 128, 8 * 64 * 128, 128, 64 * 128)
    b = _batch(qg)
    assert qg.lib().qkv_append_norm(ctypes.byref(c), ctypes.byref(b), ctypes.byref(n), None, Q, 64 * 128, 64, 0x510000, 1024,
                                    0x520000, 1024, 1, OUT, 64 * 128, None) == expect, qg.last_error()


def test_nothing_to_do_and_null_descriptors(qg):
    for kw in (dict(sequences=0), dict(tokens=0)):
        for call in (_attn, _append, _read):
            assert call(qg, batch=_batch(qg, **kw)) == 0
    L = qg.lib()
    assert L.qattn8_forward(None, None, Q, 0, 1, 1, 1.0, OUT, 0, 1, None, None, 0, None) == -1
    assert L.qkv8_append(None, None, None, None, None, 0, 0, None, 0, None, 0, 1, None, 0, 1, None) == -1
    assert L.qkv8_read(None, None, None, 0, None, 0, 1, None) == -1
    assert L.qattn8_workspace_size(None, None, 1, None) == -1


def test_workspace_size_on_the_host(qg):
    def need(**kw):
        b, n = _batch(qg, **kw), ctypes.c_size_t()
        assert qg.lib().qattn8_workspace_size(ctypes.byref(_cache(qg)), ctypes.byref(b), 64, ctypes.byref(n)) == 0
        return n.value

    assert need(sequences=0) == 0 and need(tokens=0) == 0
    assert need(prefix_len=0, max_kv=10) == 0                      # one part: results are written at once
    row = 64 * (128 * 4 + 8)                                      # one part of one token
    assert need() >= 2 * 4 * row and need() % 256 == 0
    # long prompts: only the pieces at the ends of the CTAs' runs are kept there
    for tokens in (8192, 131072):
        size = need(sequences=1, tokens=tokens, max_q=tokens, max_kv=tokens, table_ld=-(-tokens // 64), prefix_len=0)
        assert size <= (1 << 18) * (128 * 4 + 8) + 64 + 16 * (tokens // 32 + 2) + 2048


# ------------------------------------------------------------------ the Python checks
E4M3, U8, BF = torch.float8_e4m3fn, torch.uint8, torch.bfloat16


def _fake_cache(qg, **dev):
    at = lambda name: dev.get(name, "cuda:0")
    return qg.KVCache8(Fake(10, 64, 2, 128, dtype=E4M3, device=at("k")), Fake(10, 64, 2, 128, dtype=E4M3, device=at("v")),
                       Fake(10, 4, 2, dtype=U8, device=at("k_scale")), Fake(10, 4, 2, dtype=U8, device=at("v_scale")))


@pytest.fixture
def counted(devices_qg, monkeypatch):  # noqa: F811
    qg = devices_qg
    lib = qg.lib()
    for name in ("qkv8_append", "qkv8_read", "qattn8_forward", "qkv_append_norm"):
        setattr(lib, name, lambda *a, name=name: qg.calls.append(name) or 0)
    return qg


def _fake_batch(qg):
    ints = lambda *s: Fake(*s, dtype=torch.int32)
    return qg.KVBatch(ints(3, 4), ints(3), max_kv=200, prefix_table=ints(5), prefix_len=300)


def test_one_device_is_accepted(counted):
    qg = counted
    c, b = _fake_cache(qg), _fake_batch(qg)
    qg.qkv_append(c, b, Fake(3, 2, 128), Fake(3, 2, 128), q=Fake(3, 8, 128), q_out=Fake(3, 8, 128), q_norm=Fake(128), k_norm=Fake(128))
    qg.qkv_read(c, b, k_out=Fake(3, 2, 128), v_out=Fake(3, 2, 128))
    qg.qattn_forward(Fake(3, 8, 128), c, b, out=Fake(3, 8, 128), workspace=Fake(1 << 20, dtype=U8))
    assert qg.calls == ["qkv8_append", "qkv8_read", "qattn8_forward"]


@pytest.mark.parametrize("device", ["cuda:1", "cpu"])
def test_another_device_is_refused(counted, device):
    qg = counted
    for name in ("k", "v", "k_scale", "v_scale"):
        with pytest.raises(ValueError):
            _fake_cache(qg, **{name: device})
    c, b = _fake_cache(qg), _fake_batch(qg)
    far = lambda *s, **kw: Fake(*s, device=device, **kw)
    k = Fake(3, 2, 128)
    for kw in (dict(q_norm=far(128)), dict(k_norm=far(128))):
        with pytest.raises(ValueError):
            qg.qkv_append(c, b, k, k, q=Fake(3, 8, 128), q_out=Fake(3, 8, 128), **kw)
    with pytest.raises(ValueError):
        qg.qkv_read(c, b, k_out=far(3, 2, 128), v_out=k)
    with pytest.raises(ValueError):
        qg.qattn_forward(far(3, 8, 128), c, b, out=Fake(3, 8, 128), workspace=Fake(1 << 20, dtype=U8))
    assert qg.calls == []


def test_a_cache_that_is_not_on_the_current_device_is_refused(counted, monkeypatch):
    qg = counted
    c, b, k = _fake_cache(qg), _fake_batch(qg), Fake(3, 2, 128)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in (lambda: qg.qkv_append(c, b, k, k), lambda: qg.qkv_read(c, b, k_out=k, v_out=k),
                 lambda: qg.qattn_forward(Fake(3, 8, 128), c, b, out=Fake(3, 8, 128), workspace=Fake(1 << 20, dtype=U8))):
        with pytest.raises(ValueError):
            call()
    assert qg.calls == []
