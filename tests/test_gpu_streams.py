"""Calls on a stream that is not the current one: what a call allocates itself,
results and scratch memory, is that stream's, so work of the current stream
neither overwrites it nor is overwritten by it."""
import pytest
import torch

import workloads as wl
from _paged import Case

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
HOLD = 200_000_000   # clocks a stream is held busy, about a tenth of a second


@pytest.fixture(scope="module")
def qg():
    import bit_weight_only_group_gb300 as qg
    qg.lib()
    return qg


def _tensors(r):
    """The tensors of a result."""
    if isinstance(r, torch.Tensor):
        return [r]
    if isinstance(r, dict):
        return _tensors(list(r.values()))
    if isinstance(r, (list, tuple)):
        return [t for x in r for t in _tensors(x)]
    if hasattr(r, "packed"):
        return _tensors([v for v in vars(r).values() if v is not None])
    return []


def _calls(qg):
    """name -> (call with a stream, bytes of its scratch memory)."""
    N, K, T, k, E = 256, 1024, 24, 2, 4
    W = wl.gen_weight(N, K, seed=1, outlier_frac=0.002, outlier_seed=2).cuda()
    turned = wl.gen_weight(K, N, seed=3).cuda().t()          # quantized from a copy that the call makes
    qw, q8 = qg.qpack_quantize(W, 4, 128, 0.002), qg.qpack_quantize(W, 8, 128, 0.0)
    tiles = qg.qrepack_tiles(qw)
    x, few = wl.gen_x(64, K, seed=4).cuda(), wl.gen_x(9, K, seed=5).cuda()
    experts = [qg.qpack_quantize(wl.gen_weight(N, K, seed=6 + e).cuda(), 4, 128) for e in range(E)]
    topk, xt = wl.gen_topk(T, k, E, seed=10).cuda(), wl.gen_x(T, K, seed=11).cuda()
    shared = Case([1] * 5, [20, 30, 64, 65, 130], 700, 16, 2, 128, 32, BF, seed=12)
    prompts = Case([130, 90], [130, 191], 333, 16, 2, 128, 32, BF, seed=13)
    att = [(c, c.cache(qg), c.batch(qg)) for c in (shared, prompts)]
    kq = torch.randn((5, 20, 128), device="cuda").to(BF)
    ws = qg.qpack_workspace_size
    return {
        "quantize": (lambda s: qg.qpack_quantize(turned, 4, 128, 0.002, stream=s), ws(N, K)),
        "quantize noalloc": (lambda s: qg.qpack_quantize_noalloc(W, 4, 128, 0.002, stream=s), 0),
        "forward": (lambda s: qg.qgemm_forward(x, qw, stream=s), qg.qgemm_workspace_size(64, qw)),
        "forward few": (lambda s: qg.qgemm_forward(few, qw, stream=s), qg.qgemm_workspace_size(9, qw)),
        "multi": (lambda s: qg.qgemm_forward_multi(x, [qw, qw], stream=s), qg.qgemm_workspace_size(64, qw)),
        "moe": (lambda s: qg.qgemm_moe_grouped(xt, topk, experts, stream=s), qg.qgemm_moe_workspace_size(T, k, experts)),
        "moe multi": (lambda s: qg.qgemm_moe_grouped_multi(xt, topk, [experts, experts], stream=s),
                      qg.qgemm_moe_workspace_size(T, k, experts)),
        "w8a8": (lambda s: qg.qgemm_forward_w8a8(few, q8, stream=s), 16 * K),
        "repack": (lambda s: qg.qrepack_tiles(qw, stream=s), 0),
        "tiles": (lambda s: qg.qgemm_forward_tiles(x, qw, tiles, stream=s), qg.qgemm_workspace_size(64, qw)),
        "diagnostics": (lambda s: torch.tensor(qg.qdiag_layer(W, qw, stream=s)["rmse"]), 1 << 16),
        "append": (lambda s: qg.qkv_append(att[0][1], att[0][2], kq[:, 16:18], kq[:, 18:], q=kq[:, :16], stream=s), 0),
        "attention": (lambda s: qg.qattn_forward(shared.q, att[0][1], att[0][2], stream=s),
                      qg.qattn_workspace_size(att[0][1], att[0][2], 16)),
        "attention of prompts": (lambda s: qg.qattn_forward(prompts.q, att[1][1], att[1][2], stream=s),
                                 qg.qattn_workspace_size(att[1][1], att[1][2], 16)),
    }


NAMES = ["quantize", "quantize noalloc", "forward", "forward few", "multi", "moe", "moe multi", "w8a8", "repack", "tiles",
         "diagnostics", "append", "attention", "attention of prompts"]


@pytest.fixture(scope="module")
def calls(qg):
    c = _calls(qg)
    assert list(c) == NAMES
    return c


def _other():
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    return s


@pytest.mark.parametrize("name", NAMES)
@pytest.mark.parametrize("raw", [False, True])
def test_results_are_not_written_by_the_current_stream(calls, name, raw):
    # the current stream is held, and what it will write then is in freed blocks of the results' and the scratch's sizes
    call, scratch = calls[name]
    want = [t.clone() for t in _tensors(call(None))]
    s = _other()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda._sleep(HOLD)
    blocks = [torch.empty(max(n, 1), dtype=torch.uint8, device="cuda")
              for n in [t.nbytes for t in want] + [scratch] + [1024 * 256 * 2] for _ in range(2)]
    for b in blocks:
        b.fill_(0xFF)
    del blocks, b
    got = _tensors(call(s.cuda_stream if raw else s))
    torch.cuda.synchronize()
    assert len(got) == len(want)
    for a, b in zip(got, want):
        assert a.dtype == b.dtype and torch.equal(a.view(-1).view(torch.uint8), b.view(-1).view(torch.uint8))


@pytest.mark.parametrize("name", [n for n in NAMES if n != "diagnostics"])   # which reads its result before it returns
def test_scratch_is_not_given_to_the_current_stream(calls, name):
    # the call's stream is held, and the current stream takes blocks of the scratch's size after the call has returned
    call, scratch = calls[name]
    want = [t.clone() for t in _tensors(call(None))]
    s = _other()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    with torch.cuda.stream(s):
        torch.cuda._sleep(HOLD)
    got = _tensors(call(s))
    blocks = [torch.zeros(max(n, 1), dtype=torch.uint8, device="cuda") for n in (scratch, 1024 * 256 * 2) for _ in range(2)]
    torch.cuda.synchronize()
    for b in blocks:
        assert not b.any()
    for a, b in zip(got, want):
        assert torch.equal(a.view(-1).view(torch.uint8), b.view(-1).view(torch.uint8))


def test_default_stream_handles(calls):
    # the legacy default stream's handles, 0 and 1, and a stream given by position
    call, _ = calls["forward"]
    want = call(None)
    for handle in (0, 1):
        assert torch.equal(call(handle), want)
    s = _other()
    with torch.cuda.stream(s):
        got = call(0)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
