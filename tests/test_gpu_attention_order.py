"""The paged-cache calls one after another without a wait between them, on one
workspace, in captured graphs, from several streams and threads, and with the
dependent launch on and off: in each way an attention call is run the outputs
are those of the same calls run alone."""
import threading

import pytest
import torch

from _paged import Case, check_attention

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16

# new tokens, own lengths, prefix: each way a call of 64 query heads over 8 key/value heads is run
WAYS = {
    "alone": ([1, 1, 1], [70, 400, 33], 0),
    "rows shared": ([1] * 5, [9, 300, 5, 64, 65], 700),
    "tiles shared": ([1] * 36, [40 + 7 * b for b in range(36)], 2500),
    "tiles shared, several tokens": ([3, 1, 5, 0, 2] * 9, [60 + 5 * b for b in range(45)], 2431),
    "prompts": ([130, 1, 90], [150, 65, 191], 333),
    "prompts in pieces": ([40], [3000], 0),
}


@pytest.fixture(scope="module")
def qg():
    import bit_weight_only_group_gb300 as qg
    qg.lib()
    assert qg.qgemm_device_status(reset=True) in (0, -6, -7)
    yield qg
    assert qg.qgemm_device_status() == 0


def _case(way, seed=50, **kw):
    n_q, kv, prefix = WAYS[way]
    return Case(n_q, kv, prefix, 64, 8, 128, 64, BF, seed=seed, **kw)


class Step:
    """One layer of a step: its cache, its new tokens, the append and the attention after it."""

    def __init__(self, qg, way, seed):
        self.qg, self.c = qg, _case(way, seed)
        g = torch.Generator().manual_seed(seed)
        T = self.c.T
        qkv = torch.randn((T, 80 * 128), generator=g).to(BF).cuda()
        self.q, self.k, self.v = (t.unflatten(1, (-1, 128)) for t in qkv.split([64 * 128, 8 * 128, 8 * 128], 1))
        angle = torch.rand((self.c.prefix + max(self.c.kv), 64), generator=g) * 6
        self.rope = torch.cat([angle.cos(), angle.sin()], 1).cuda()
        self.cache, self.batch = self.c.cache(qg), self.c.batch(qg)
        self.need = qg.qattn_workspace_size(self.cache, self.batch, 64)
        self.turned, self.out = torch.empty_like(self.c.q), torch.empty_like(self.c.q)
        # the new tokens' places hold NaN until the append has run
        self.where = [(self.c.table_host[b, own // 64].item(), own % 64)
                      for b in range(self.c.B) for own in range(self.c.kv[b] - self.c.n_q[b], self.c.kv[b])]

    def forget(self):
        page, place = (torch.tensor(x, device="cuda") for x in zip(*self.where))
        self.c.k[page, place] = self.c.v[page, place] = float("nan")
        self.out.fill_(7.0)
        self.turned.fill_(7.0)

    def run(self, ws, stream=None):
        self.qg.qkv_append(self.cache, self.batch, self.k, self.v, q=self.q, rope=self.rope, q_out=self.turned, stream=stream)
        self.qg.qattn_forward(self.turned, self.cache, self.batch, out=self.out, workspace=ws, stream=stream)


def _alone(steps, ws):
    """Each step's output when the device is waited for after each call."""
    want = []
    for s in steps:
        s.forget()
        torch.cuda.synchronize()
        s.qg.qkv_append(s.cache, s.batch, s.k, s.v, q=s.q, rope=s.rope, q_out=s.turned)
        torch.cuda.synchronize()
        s.qg.qattn_forward(s.turned, s.cache, s.batch, out=s.out, workspace=ws)
        torch.cuda.synchronize()
        s.c.q = s.turned
        check_attention(s.c, s.out)
        want.append(s.out.clone())
    return want


def _workspace(steps):
    return torch.full((max(max(s.need for s in steps), 1),), 0xFF, dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("way", list(WAYS))
def test_append_and_attention_of_several_layers_without_a_wait(qg, way):
    steps = [Step(qg, way, seed) for seed in range(60, 64)]
    ws = _workspace(steps)
    want = _alone(steps, ws)
    for on in (True, False):
        qg.qgemm_set_dependent_launch(on)
        try:
            for _ in range(3):
                for s in steps:
                    s.forget()
                for s in steps:
                    s.run(ws)
                torch.cuda.synchronize()
                for s, w in zip(steps, want):
                    assert torch.equal(s.out, w)
        finally:
            qg.qgemm_set_dependent_launch(True)


def test_layers_run_in_different_ways_without_a_wait(qg):
    # one workspace for all: what one call has not yet joined is not overwritten by the next
    steps = [Step(qg, way, 70 + i) for i, way in enumerate(list(WAYS) + list(WAYS)[::-1])]
    ws = _workspace(steps)
    want = _alone(steps, ws)
    for _ in range(3):
        for s in steps:
            s.forget()
        for s in steps:
            s.run(ws)
        torch.cuda.synchronize()
        for s, w in zip(steps, want):
            assert torch.equal(s.out, w)


@pytest.mark.parametrize("way", list(WAYS))
def test_graph_replayed_with_new_lengths(qg, way):
    n_q, kv, prefix = WAYS[way]
    c = _case(way, 80, poison=False)
    cache, batch = c.cache(qg), c.batch(qg)
    ws = torch.full((max(qg.qattn_workspace_size(cache, batch, 64), 1),), 0xFF, dtype=torch.uint8, device="cuda")
    out, lse = torch.empty_like(c.q), torch.empty((c.T, 64), dtype=torch.float32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        qg.qattn_forward(c.q, cache, batch, out=out, lse=lse, workspace=ws)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            qg.qattn_forward(c.q, cache, batch, out=out, lse=lse, workspace=ws)
    fewer = [max(0, n - b % 2) for b, n in enumerate(n_q)]
    for n_now, kv_now in ((n_q, kv), (n_q, [max(n, k - 9) for n, k in zip(n_q, kv)]), (n_q, [max(n, 1) for n in n_q]),
                          (fewer, [max(n, k // 2) for n, k in zip(fewer, kv)])):
        c.n_q, c.kv, c.cu = n_now, kv_now, [sum(n_now[:b]) for b in range(c.B + 1)]
        c.kv_len.copy_(torch.tensor(kv_now, dtype=torch.int32))
        c.cu_q.copy_(torch.tensor(c.cu, dtype=torch.int32))
        out.fill_(7.0)
        lse.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        check_attention(c, out, lse)
        assert (out[c.cu[-1]:] == 7.0).all() and (lse[c.cu[-1]:] == 7.0).all()
    assert qg.qgemm_device_status() == 0


def test_streams_and_threads_at_once(qg):
    # every thread has its stream, its workspace and its layers, in all the ways; the card is theirs together
    mine = [[Step(qg, way, 90 + 10 * i + j) for j, way in enumerate(list(WAYS)[i:] + list(WAYS)[:i])] for i in range(3)]
    spaces = [_workspace(steps) for steps in mine]
    want = [_alone(steps, ws) for steps, ws in zip(mine, spaces)]
    for steps in mine:
        for s in steps:
            s.forget()
    torch.cuda.synchronize()
    streams, errors = [torch.cuda.Stream() for _ in mine], []

    def work(i):
        try:
            for _ in range(3):
                for s in mine[i]:
                    s.run(spaces[i], streams[i])
        except Exception as e:   # noqa: BLE001 - shown by the test's own thread
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(mine))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for steps, ws in zip(mine, want):
        for s, w in zip(steps, ws):
            assert torch.equal(s.out, w)


@pytest.mark.parametrize("way", list(WAYS))
@pytest.mark.parametrize("bad", [-1, 1 << 20, 0x7FFFFFFF])
def test_page_numbers_outside_the_cache_are_not_followed(qg, way, bad):
    c = _case(way, 120)
    want = qg.qattn_forward(c.q, c.cache(qg), c.batch(qg))
    assert qg.qgemm_device_status(reset=True) == 0
    b = next(i for i in range(c.B) if c.n_q[i] and c.kv[i] > 64)
    others = [t for t in range(c.T) if not c.cu[b] <= t < c.cu[b + 1]]
    kept = c.table[b, 0].item()
    c.table[b, 0] = bad
    out = qg.qattn_forward(c.q, c.cache(qg), c.batch(qg))
    assert qg.qgemm_device_status(reset=True) == -7
    assert torch.equal(out[others], want[others])   # the other sequences are as they were
    c.table[b, 0] = kept
    if c.prefix:
        kept = c.prefix_table[2].item()
        c.prefix_table[2] = bad
        qg.qattn_forward(c.q, c.cache(qg), c.batch(qg))
        assert qg.qgemm_device_status(reset=True) == -7
        c.prefix_table[2] = kept
    assert torch.equal(qg.qattn_forward(c.q, c.cache(qg), c.batch(qg)), want)
    assert qg.qgemm_device_status() == 0


@pytest.mark.parametrize("way", list(WAYS))
def test_offsets_that_descend_end_and_a_sound_call_follows(qg, way):
    c = _case(way, 130)
    want = qg.qattn_forward(c.q, c.cache(qg), c.batch(qg))
    sound = c.cu_q.clone()
    c.cu_q[1::2] = c.T
    c.cu_q[2::2] = 0
    c.cu_q[-1] = c.T
    qg.qattn_forward(c.q, c.cache(qg), c.batch(qg))
    assert qg.qgemm_device_status(reset=True) == (-7 if c.B > 1 else 0)
    c.cu_q.copy_(sound)
    assert torch.equal(qg.qattn_forward(c.q, c.cache(qg), c.batch(qg)), want)
    assert qg.qgemm_device_status() == 0


@pytest.mark.parametrize("way", list(WAYS))
def test_bounds_above_the_lengths(qg, way):
    # more places, new tokens and rows allowed than there are, in each way
    c = _case(way, 140, spare_tokens=70)
    wide = torch.full((c.B, 200), 0x7FFFFFFF, dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide
    for bounds in (dict(max_kv=200 * 64), dict(max_q=max(c.n_q) + 60), dict(max_kv=12000, max_q=max(c.n_q) + 7)):
        lse = torch.empty((c.T, 64), dtype=torch.float32, device="cuda")
        out = qg.qattn_forward(c.q, c.cache(qg), c.batch(qg, **bounds), lse=lse)
        check_attention(c, out, lse)
        assert qg.qgemm_device_status() == 0


@pytest.mark.parametrize("heads_q,heads_kv,dim,dtype", [(136, 1, 128, BF), (320, 2, 64, FP), (129, 1, 64, BF)])
@pytest.mark.parametrize("n_q,kv,prefix", [([1, 1], [70, 9], 0), ([1] * 4, [1, 64, 65, 130], 3000), ([5, 0, 9], [5, 3, 200], 400)])
def test_more_query_heads_than_a_tile_has_rows(qg, heads_q, heads_kv, dim, dtype, n_q, kv, prefix):
    c = Case(n_q, kv, prefix, heads_q, heads_kv, dim, 32, dtype, seed=150, spare_tokens=1)
    lse = torch.empty((c.T, heads_q), dtype=torch.float32, device="cuda")
    out = qg.qattn_forward(c.q, c.cache(qg), c.batch(qg), lse=lse)
    check_attention(c, out, lse)
