"""The 8-bit cache's calls on a stream that is not the current one: results and
scratch memory are that stream's; and calls of several threads at once."""
import threading

import pytest
import torch

from _paged import check_attention
from _paged8 import Case8
from test_gpu_streams import HOLD, _other, _tensors

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


@pytest.fixture(scope="module")
def calls():
    """name -> (call with a stream, bytes of its scratch memory)."""
    import bit_weight_only_group_gb300 as qg
    qg.lib()
    shared = Case8([1] * 5, [20, 30, 64, 65, 130], 700, 16, 2, 128, 32, seed=12)
    prompts = Case8([130, 90], [130, 191], 333, 16, 2, 128, 32, seed=13)
    att = [(c, c.cache(qg), c.batch(qg)) for c in (shared, prompts)]
    kq = torch.randn((5, 20, 128), device="cuda").to(BF)
    w = torch.ones(128, device="cuda")
    ws = qg.qattn_workspace_size
    return {
        "append": (lambda s: qg.qkv_append(att[0][1], att[0][2], kq[:, 16:18], kq[:, 18:], q=kq[:, :16], q_norm=w, k_norm=w,
                                           stream=s), 0),
        "read": (lambda s: qg.qkv_read(att[1][1], att[1][2], stream=s), 0),
        "attention": (lambda s: qg.qattn_forward(shared.q, att[0][1], att[0][2], stream=s), ws(att[0][1], att[0][2], 16)),
        "attention of prompts": (lambda s: qg.qattn_forward(prompts.q, att[1][1], att[1][2], stream=s),
                                 ws(att[1][1], att[1][2], 16)),
    }


NAMES = ["append", "read", "attention", "attention of prompts"]


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("raw", [False, True])
def test_results_are_not_written_by_the_current_stream(calls, name, raw):
    call, scratch = calls[name]
    want = [t.clone() for t in _tensors(call(None))]
    s = _other()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda._sleep(HOLD)
    blocks = [torch.empty(max(n, 1), dtype=torch.uint8, device="cuda") for n in [t.nbytes for t in want] + [scratch] for _ in range(2)]
    for b in blocks:
        b.fill_(0xFF)
    del blocks, b
    got = _tensors(call(s.cuda_stream if raw else s))
    torch.cuda.synchronize()
    assert len(got) == len(want) and all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("name", NAMES)
def test_scratch_is_not_given_to_the_current_stream(calls, name):
    call, scratch = calls[name]
    want = [t.clone() for t in _tensors(call(None))]
    s = _other()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(s):
        torch.cuda._sleep(HOLD)
    got = _tensors(call(s))
    blocks = [torch.zeros(max(scratch, 1), dtype=torch.uint8, device="cuda") for _ in range(2)]
    torch.cuda.synchronize()
    assert not any(b.any() for b in blocks)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_layers_without_a_wait_on_one_workspace_and_threads_at_once():
    # append, attention and reading of one layer after another, by three threads on three streams
    import bit_weight_only_group_gb300 as qg
    failed = []

    def work(seed):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                cases = [Case8(n_q, kv, prefix, 16, 2, 128, 32, seed=seed + i) for i, (n_q, kv, prefix) in enumerate(
                    [([1] * 40, [70] * 40, 2500), ([130, 90], [130, 191], 333), ([1, 1], [900, 33], 0), ([1] * 5, [64] * 5, 700)])]
                need = max(qg.qattn_workspace_size(c.cache(qg), c.batch(qg), 16) for c in cases)
                ws = torch.empty(need, dtype=torch.uint8, device="cuda")
                steps = []
                for c in cases:
                    x = torch.randn((c.T, 20, 128), device="cuda").to(BF)
                    steps.append((c, c.cache(qg), c.batch(qg), x))
                s.synchronize()
                outs = []
                for c, cache, batch, x in steps:
                    c.q = qg.qkv_append(cache, batch, x[:, 16:18], x[:, 18:], q=x[:, :16])
                    outs.append(qg.qattn_forward(c.q, cache, batch, workspace=ws))
                s.synchronize()
                for (c, *_), out in zip(steps, outs):
                    c.refresh()
                    check_attention(c, out)
        except Exception as e:   # told to the test
            failed.append(e)

    threads = [threading.Thread(target=work, args=(100 * i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    assert qg.qgemm_device_status() == 0
