"""The paged-cache calls refuse tensors of another device than the cache's and
a cache that is not on the current device, before anything is launched: shown
with stand-ins for tensors, without a GPU."""
import math
import types

import pytest
import torch

BF = torch.bfloat16


class Fake:
    """What the checks see of a tensor."""

    def __init__(self, *shape, dtype=BF, device="cuda:0", contiguous=True):
        self.shape, self.dtype, self.device = torch.Size(shape), dtype, torch.device(device)
        self.is_cuda, self._contiguous = self.device.type == "cuda", contiguous

    def get_device(self):
        return self.device.index if self.is_cuda else -1

    def dim(self):
        return len(self.shape)

    def numel(self):
        return math.prod(self.shape)

    def stride(self, i=None):
        st = tuple(math.prod(self.shape[j + 1:]) for j in range(len(self.shape)))
        return st if i is None else st[i]

    def data_ptr(self):
        return 0x100000

    def element_size(self):
        return self.dtype.itemsize

    def is_contiguous(self):
        return self._contiguous


@pytest.fixture
def qg(monkeypatch):
    """The package with the library replaced by one that counts its calls, and device 0 current."""
    import bit_weight_only_group_gb300 as qg
    calls = []
    lib = types.SimpleNamespace(qkv_append=lambda *a: calls.append("append") or 0,
                                qattn_forward=lambda *a: calls.append("attention") or 0)
    monkeypatch.setattr(qg, "lib", lambda: lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0)
    monkeypatch.setattr(qg, "calls", calls, raising=False)
    return qg


def _cache(qg, device="cuda:0"):
    return qg.KVCache(*(Fake(10, 64, 2, 128, device=device) for _ in range(2)))


def _ints(*shape, **kw):
    return Fake(*shape, dtype=torch.int32, **kw)


def _batch(qg, device="cuda:0"):
    return qg.KVBatch(_ints(3, 4, device=device), _ints(3, device=device), max_kv=200, prefix_table=_ints(5, device=device),
                      prefix_len=300)


def _append(qg, **kw):
    a = dict(k=Fake(3, 2, 128), v=Fake(3, 2, 128), q=Fake(3, 8, 128), q_out=Fake(3, 8, 128),
             rope=Fake(600, 128, dtype=torch.float32), positions=_ints(3))
    a.update(kw)
    return qg.qkv_append(_cache(qg), _batch(qg), **a)


def _attend(qg, cache=None, batch=None, **kw):
    a = dict(q=Fake(3, 8, 128), out=Fake(3, 8, 128), lse=Fake(3, 8, dtype=torch.float32),
             workspace=Fake(1 << 20, dtype=torch.uint8))
    a.update(kw)
    return qg.qattn_forward(a.pop("q"), cache or _cache(qg), batch or _batch(qg), **a)


def test_one_device_is_accepted(qg):
    _append(qg)
    _attend(qg)
    assert qg.calls == ["append", "attention"]


@pytest.mark.parametrize("device", ["cuda:1", "cpu"])
@pytest.mark.parametrize("name", ["k", "v", "q", "q_out", "rope", "positions"])
def test_append_refuses_another_device(qg, name, device):
    shapes = dict(q=(3, 8, 128), q_out=(3, 8, 128), rope=(600, 128), positions=(3,))
    dtypes = dict(rope=torch.float32, positions=torch.int32)
    with pytest.raises(ValueError):
        _append(qg, **{name: Fake(*shapes.get(name, (3, 2, 128)), dtype=dtypes.get(name, BF), device=device)})
    assert qg.calls == []


@pytest.mark.parametrize("device", ["cuda:1", "cpu"])
@pytest.mark.parametrize("name", ["q", "out", "lse", "workspace"])
def test_attention_refuses_another_device(qg, name, device):
    fake = dict(q=Fake(3, 8, 128, device=device), out=Fake(3, 8, 128, device=device),
                lse=Fake(3, 8, dtype=torch.float32, device=device),
                workspace=Fake(1 << 20, dtype=torch.uint8, device=device))[name]
    with pytest.raises(ValueError):
        _attend(qg, **{name: fake})
    assert qg.calls == []


def test_a_batch_or_a_cache_on_two_devices_is_refused(qg):
    with pytest.raises(ValueError):
        qg.KVCache(Fake(10, 64, 2, 128), Fake(10, 64, 2, 128, device="cuda:1"))
    for bad in range(3):
        t = [_ints(3, 4), _ints(4), _ints(5)]
        t[bad] = _ints(*t[bad].shape, device="cuda:1")
        with pytest.raises(ValueError):
            qg.KVBatch(t[0], _ints(3), max_kv=200, cu_q=t[1], tokens=3, prefix_table=t[2], prefix_len=300)
    with pytest.raises(ValueError):
        _attend(qg, batch=_batch(qg, "cuda:1"))
    assert qg.calls == []


def test_a_cache_that_is_not_on_the_current_device_is_refused(qg, monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    for call in (_append, _attend):
        with pytest.raises(ValueError):
            call(qg)
    assert qg.calls == []


def test_a_workspace_with_gaps_is_refused(qg):
    with pytest.raises(ValueError):
        _attend(qg, workspace=Fake(1 << 20, dtype=torch.uint8, contiguous=False))
    assert qg.calls == []
