"""Attention over the paged cache against its definition in 64 bits: head
layouts, page sizes, lengths from one token on, shared prefixes, several new
tokens a sequence, and everything past a length poisoned with NaN."""
import math

import pytest
import torch

from _paged import Case, check_attention

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def qg():
    import bit_weight_only_group_gb300 as qg
    qg.lib()
    assert qg.qgemm_device_status(reset=True) in (0, -6, -7)
    yield qg
    assert qg.qgemm_device_status() == 0


def _run(qg, c, scale=None, **kw):
    out = torch.full((c.T, c.heads_q, c.dim), 7.0, dtype=kw.pop("out_dtype", c.dtype), device="cuda")
    lse = torch.full((c.T, c.heads_q), 7.0, dtype=torch.float32, device="cuda")
    cache, batch = c.cache(qg), c.batch(qg, **kw)
    ws = torch.full((qg.qattn_workspace_size(cache, batch, c.heads_q),), 0xFF, dtype=torch.uint8, device="cuda")
    qg.qattn_forward(c.q, cache, batch, scale=scale, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    assert qg.qgemm_device_status() == 0
    # rows of no sequence are left alone
    assert (out[c.cu[-1]:] == 7.0).all() and (lse[c.cu[-1]:] == 7.0).all()
    return out, lse


HEADS = [(8, 8, 128), (8, 1, 128), (16, 2, 64), (28, 4, 128), (9, 3, 64), (64, 8, 128)]


@pytest.mark.parametrize("heads_q,heads_kv,dim", HEADS)
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("page,heads_first", [(16, True), (64, False), (256, True)])
def test_decode_heads_and_pages(qg, heads_q, heads_kv, dim, dtype, page, heads_first):
    c = Case([1, 1, 1], [1, 77, 200], 0, heads_q, heads_kv, dim, page, dtype, heads_first, seed=heads_q + page)
    check_attention(c, *_run(qg, c))


@pytest.mark.parametrize("prefix", [1, 63, 64, 65, 255, 256, 257, 1000])
@pytest.mark.parametrize("dtype,dim", [(BF, 128), (FP, 64)])
def test_shared_prefix_lengths(qg, prefix, dtype, dim):
    c = Case([1] * 5, [1, 2, 64, 65, 130], prefix, 16, 2, dim, 32, dtype, seed=prefix)
    check_attention(c, *_run(qg, c))


@pytest.mark.parametrize("own", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 500, 1025])
def test_own_lengths(qg, own):
    c = Case([1, 1], [own, max(1, own - 1)], 300, 8, 2, 128, 16, BF, False, seed=own)
    check_attention(c, *_run(qg, c))


@pytest.mark.parametrize("B", [1, 2, 3, 7, 16, 17, 33, 40])
def test_batch_sizes(qg, B):
    c = Case([1] * B, [1 + (37 * b) % 90 for b in range(B)], 700, 16, 2, 128, 64, BF, seed=B)
    check_attention(c, *_run(qg, c))


@pytest.mark.parametrize("heads_q,heads_kv,dim,dtype,page,heads_first", [
    (64, 8, 128, BF, 64, True), (64, 8, 128, FP, 16, False), (32, 8, 64, FP, 128, True), (28, 4, 128, BF, 32, False),
    (32, 32, 128, BF, 64, True), (48, 1, 64, BF, 256, True), (100, 1, 128, FP, 64, True)])
@pytest.mark.parametrize("n_q,prefix", [([1] * 33, 2500), ([1] * 90, 2049), ([3, 1, 5, 0, 2] * 9, 2431)])
def test_much_shared_prefix(qg, heads_q, heads_kv, dim, dtype, page, heads_first, n_q, prefix):
    # enough rows and keys that the prefix is worked on in tiles: pairs of tiles, a single one, a cut last block
    kv = [max(n, 1) + (31 * b) % 150 for b, n in enumerate(n_q)]
    c = Case(n_q, kv, prefix, heads_q, heads_kv, dim, page, dtype, heads_first, seed=len(n_q) + page, spare_tokens=2)
    check_attention(c, *_run(qg, c))


@pytest.mark.parametrize("heads_q,heads_kv,dim", [(16, 2, 128), (32, 8, 64)])
def test_rows_packed_across_sequences(qg, heads_q, heads_kv, dim):
    # more than 64 rows a sequence and head, few of its own keys: the prefix's tiles hold rows of several sequences
    n_q = [20, 17, 1, 19] * 10
    c = Case(n_q, [n + b for b, n in enumerate(n_q)], 4000, heads_q, heads_kv, dim, 64, BF, seed=30)
    check_attention(c, *_run(qg, c))


@pytest.mark.parametrize("n_q,kv", [([1, 5, 2], [1, 9, 200]), ([8, 8], [8, 64]), ([3, 0, 4, 1], [70, 50, 4, 1]),
                                    ([17, 33], [17, 129]), ([64], [300]), ([130, 1, 90], [130, 65, 191]),
                                    ([257, 3], [400, 3])])
@pytest.mark.parametrize("heads_q,heads_kv,dim", [(16, 2, 128), (7, 1, 64), (4, 4, 128)])
@pytest.mark.parametrize("prefix", [0, 333])
def test_several_tokens(qg, n_q, kv, heads_q, heads_kv, dim, prefix):
    c = Case(n_q, kv, prefix, heads_q, heads_kv, dim, 16, BF, seed=sum(n_q) + prefix, spare_tokens=3)
    check_attention(c, *_run(qg, c))


@pytest.mark.parametrize("prefix", [0, 400])
def test_rows_that_see_nothing(qg, prefix):
    # own lengths below the count of new tokens: the first rows see no own token (and without a prefix nothing)
    c = Case([4, 2, 70, 1], [2, 0, 33, 0], prefix, 8, 2, 128, 16, BF, seed=3)
    out, lse = _run(qg, c)
    check_attention(c, out, lse)
    if prefix == 0:
        assert (out[:2] == 0).all() and (out[4:6] == 0).all() and torch.isinf(lse[:2]).all()


@pytest.mark.parametrize("garbage", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("n_q,kv", [([1, 1], [33, 70]), ([9, 100], [33, 170])])
def test_whatever_lies_past_a_length(qg, garbage, n_q, kv):
    c = Case(n_q, kv, 270, 16, 2, 128, 128, FP, seed=5, garbage=garbage)
    check_attention(c, *_run(qg, c))


@pytest.mark.parametrize("n_q,kv,prefix", [([1, 1, 1], [70, 2000, 33], 0), ([1] * 5, [9, 300, 1, 64, 65], 700),
                                           ([1] * 33, [200] * 33, 2500), ([4] * 20, [70] * 20, 2500),
                                           ([130, 90, 70], [130, 200, 70], 333)])
def test_not_finite_stays_not_finite_and_in_its_place(qg, n_q, kv, prefix):
    # a NaN key makes the rows that see it NaN in any way a call is split, and changes no bit of any other row
    c = Case(n_q, kv, prefix, 64, 8, 128, 16, BF, seed=40)
    clean, lse0 = _run(qg, c)
    check_attention(c, clean, lse0)
    rows = torch.arange(c.cu[1], c.cu[2], device="cuda")

    def places(key):   # of sequence 1
        return c.table[1, key // c.page].item(), key % c.page

    def expect(seen, out, lse, heads):
        bad = torch.zeros((c.T, c.heads_q), dtype=torch.bool, device="cuda")
        bad[seen[:, None], torch.tensor(heads, device="cuda")] = True
        assert out[bad].isnan().all() and lse[bad].isnan().all()
        assert torch.equal(out[~bad], clean[~bad]) and torch.equal(lse[~bad], lse0[~bad])

    for key, seen in ((0, rows), (kv[1] - 1, rows[-1:])):   # seen by all of the sequence's tokens, by its last alone
        page, at = places(key)
        kept = c.k[page, at, 2, 5].clone()
        c.k[page, at, 2, 5] = math.nan
        expect(seen, *_run(qg, c), list(range(16, 24)))
        c.k[page, at, 2, 5] = kept
    if prefix:
        page = c.prefix_table[prefix // 2 // c.page].item()
        kept = c.k[page, 0, 7, 100].clone()
        c.k[page, 0, 7, 100] = math.nan
        expect(torch.arange(c.T, device="cuda"), *_run(qg, c), list(range(56, 64)))
        c.k[page, 0, 7, 100] = kept
    # an infinite value of the first own key: that column of its rows alone
    page, at = places(0)
    c.v[page, at, 0, 9] = math.inf
    out, lse = _run(qg, c)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[c.cu[1]:c.cu[2], :8, 9] = True
    assert (~torch.isfinite(out[bad])).all() and torch.equal(out[~bad], clean[~bad]) and torch.equal(lse, lse0)


@pytest.mark.parametrize("out_dtype", [torch.float32, BF, FP])
def test_output_types_and_scale(qg, out_dtype):
    c = Case([1, 1, 40], [50, 3, 90], 500, 8, 4, 128, 32, BF, seed=8)
    for scale in (0.25, 1e-3):
        out, lse = _run(qg, c, scale=scale, out_dtype=out_dtype)
        check_attention(c, out, lse, scale)


def test_large_logits(qg):
    # logits in the hundreds: the softmax is all but one-hot, and only the running maximum keeps it finite
    c = Case([1, 1, 6], [200, 900, 130], 800, 8, 2, 128, 16, BF, seed=9, spread=60.0)
    check_attention(c, *_run(qg, c))


def test_rising_and_falling_logits(qg):
    # keys in order of their logit, both ways: the running maximum changes at every tile, or never again
    for sign in (1.0, -1.0):
        c = Case([1, 1], [640, 640], 640, 4, 1, 128, 64, BF, seed=10)
        ramp = sign * torch.linspace(-4, 4, 640, device="cuda")
        direction = torch.randn(128, device="cuda")
        direction /= direction.norm()
        for rows in (c.table[0], c.table[1], c.prefix_table):
            c.k[rows.long()] = (ramp.view(-1, 64)[:, :, None, None] * direction * 11.3).to(BF)
        c.q[:] = (direction * 11.3).to(BF)
        check_attention(c, *_run(qg, c))


def test_strided_arrays(qg):
    # q inside the fused product's rows, out inside wider rows, K and V interleaved page by page
    c = Case([1, 3, 1], [40, 20, 99], 290, 16, 2, 128, 16, BF, False, seed=12)
    both = torch.empty((c.k.shape[0], 2, *c.k.shape[1:]), dtype=BF, device="cuda")
    both[:, 0], both[:, 1] = c.k, c.v
    c.k, c.v = both[:, 0], both[:, 1]
    wide = torch.randn((c.T, 20 * 128), device="cuda").to(BF)
    wide[:, :16 * 128] = c.q.flatten(1)
    c.q = wide[:, :16 * 128].view(c.T, 16, 128)
    into = torch.zeros((c.T, 17 * 128), dtype=BF, device="cuda")
    out = into[:, :16 * 128].view(c.T, 16, 128)
    qg.qattn_forward(c.q, c.cache(qg), c.batch(qg), out=out)
    check_attention(c, out)
    assert (into[:, 16 * 128:] == 0).all()


@pytest.mark.parametrize("n_q,kv,heads_q,heads_kv,dim", [
    ([16], [20000], 8, 1, 128), ([9, 30], [9000, 31], 9, 1, 64), ([40, 33, 70], [4000, 33, 70], 28, 4, 128),
    ([300], [2500], 16, 2, 64), ([3], [5000], 100, 1, 128)])
def test_prompts_in_many_pieces(qg, n_q, kv, heads_q, heads_kv, dim):
    # few items of many keys: cut to pieces over many CTAs.  Nothing past the workspace is written.
    c = Case(n_q, kv, 0, heads_q, heads_kv, dim, 64, BF, seed=27)
    cache, batch = c.cache(qg), c.batch(qg)
    need = qg.qattn_workspace_size(cache, batch, heads_q)
    ws = torch.full((need + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    lse = torch.empty((c.T, heads_q), dtype=torch.float32, device="cuda")
    out = qg.qattn_forward(c.q, cache, batch, lse=lse, workspace=ws)
    check_attention(c, out, lse)
    assert (ws[need:] == 0x5A).all()


def _time(f):
    """Least time of some calls, in microseconds."""
    for _ in range(3):
        f()
    times = []
    for _ in range(10):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(4):
            f()
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) * 250)
    return min(times)


def _loose(qg, n_q, kv, prefix, bound):
    """Times of a call with its bound of own tokens far above the lengths, and at them."""
    c = Case(n_q, kv, prefix, 64, 8, 128, 64, BF, seed=28)
    wide = torch.zeros((len(n_q), -(-bound // 64)), dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = c.table
    tight, c.table = c.table, wide
    cache, batches = c.cache(qg), [c.batch(qg, max_kv=bound)]
    c.table = tight
    batches.append(c.batch(qg))
    times = []
    for b in batches:
        ws = torch.empty(qg.qattn_workspace_size(cache, b, 64), dtype=torch.uint8, device="cuda")
        out = torch.empty_like(c.q)
        times.append(_time(lambda: qg.qattn_forward(c.q, cache, b, out=out, workspace=ws)))
        check_attention(c, out)
    assert qg.qgemm_device_status() == 0
    return times


def test_prompts_are_dealt_by_their_lengths(qg):
    # 512 tokens where 131072 might be: the blocks there are go to all CTAs (run by run of the bound they all went to one,
    # 24 times as long)
    loose, tight = _loose(qg, [512], [512], 0, 131072)
    assert loose < 3 * tight, (loose, tight)


def test_parts_are_dealt_by_the_lengths(qg):
    # 4096 tokens where 131072 might be: cut to parts of the bound only 2 of 57 had keys, 3.6 times as long
    loose, tight = _loose(qg, [1], [4096], 0, 131072)
    assert loose < 2.5 * tight, (loose, tight)


def test_a_loose_bound_leaves_the_prefix_its_share_of_the_card(qg):
    # 40 own histories of 300 where 32768 might be, over 20000: SMs kept for own tokens that are not there stay idle
    loose, tight = _loose(qg, [1] * 40, [300] * 40, 20000, 32768)
    assert loose < 3 * tight, (loose, tight)


def test_one_token_each_without_offsets(qg):
    c = Case([1] * 6, [3, 1, 20, 64, 65, 18], 260, 8, 2, 64, 16, FP, seed=13)
    out, lse = _run(qg, c, cu_q=None)
    check_attention(c, out, lse)


def test_looser_bounds_change_nothing(qg):
    # bounds above the lengths: the same result within the error of both
    c = Case([1, 4, 2], [70, 4, 33], 270, 8, 2, 128, 16, BF, seed=14)
    wide = torch.zeros((3, 64), dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide
    check_attention(c, *_run(qg, c, max_kv=1000, max_q=9))


@pytest.mark.parametrize("n_q,kv,prefix", [([1] * 20, [300] * 20, 5000), ([1] * 60, [300] * 60, 20000), ([200, 200], [200, 500], 700), ([1], [9000], 0)])
def test_repeatable_bit_for_bit(qg, n_q, kv, prefix):
    c = Case(n_q, kv, prefix, 16, 2, 128, 64, BF, seed=15)
    a, la = _run(qg, c)
    for _ in range(3):
        b, lb = _run(qg, c)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_long_prefix_and_long_own(qg):
    c = Case([1, 1, 2], [4500, 17, 9000], 20000, 16, 2, 128, 64, BF, seed=16)
    check_attention(c, *_run(qg, c))


def test_offsets_past_32_bits(qg):
    # pages 2^21 elements apart in a cache of 6.4 GB each: the last ones start past 2^31 elements and 2^32 bytes
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    c = Case([1, 2], [40, 130], 300, 8, 2, 128, 16, BF, seed=17, poison=False)
    n = c.k.shape[0]
    far = 1500 + torch.arange(n, device="cuda")
    caches = []
    for t in (c.k, c.v):
        big = torch.empty((1600, 2, 8192, 128), dtype=BF, device="cuda")[:, :, :16].transpose(1, 2)
        big[far] = t
        caches.append(big)
    c.k, c.v = caches
    c.table, c.prefix_table = c.table + 1500, c.prefix_table + 1500
    check_attention(c, *_run(qg, c))
    del c, caches, big
    torch.cuda.empty_cache()


@pytest.mark.parametrize("prefix", [0, 400, 3000])
def test_fewer_tokens_than_rows(qg, prefix):
    # a batch that has shrunk: most rows belong to no sequence, in each of the ways a call is run
    for n_q in ([1, 1], [100, 3], [0, 0], [0, 7]):
        c = Case(n_q, [n + 5 for n in n_q], prefix, 64, 8, 128, 64, BF, seed=43, spare_tokens=200)
        check_attention(c, *_run(qg, c))
    c = Case([1, 0, 1] + [0] * 60, [9] * 63, prefix, 64, 8, 128, 64, BF, seed=44, spare_tokens=61)
    check_attention(c, *_run(qg, c))


def test_captured_graph_with_new_lengths(qg):
    # lengths and tables are read when the graph runs
    c = Case([1] * 4, [10, 60, 100, 128], 300, 8, 2, 128, 16, BF, seed=18, poison=False)
    cache, batch = c.cache(qg), c.batch(qg)
    ws = torch.empty(qg.qattn_workspace_size(cache, batch, 8), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(c.q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        qg.qattn_forward(c.q, cache, batch, out=out, workspace=ws)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            qg.qattn_forward(c.q, cache, batch, out=out, workspace=ws)
    for kv in ([10, 60, 100, 128], [9, 59, 99, 127], [1, 2, 3, 4]):
        c.kv = kv
        c.kv_len.copy_(torch.tensor(kv, dtype=torch.int32))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        check_attention(c, out)


def test_other_stream(qg):
    c = Case([1, 1], [100, 30], 500, 8, 2, 128, 16, BF, seed=19)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(c.q)
    qg.qattn_forward(c.q, c.cache(qg), c.batch(qg), out=out, stream=s)
    s.synchronize()
    check_attention(c, out)


def test_dependent_launch_off_gives_the_same(qg):
    c = Case([1] * 9, [100] * 9, 700, 8, 2, 128, 16, BF, seed=20)
    a, _ = _run(qg, c)
    qg.qgemm_set_dependent_launch(False)
    try:
        b, _ = _run(qg, c)
    finally:
        qg.qgemm_set_dependent_launch(True)
    assert torch.equal(a, b)


def test_bad_lengths_and_pages_are_reported(qg):
    # on the device: a length above its bound is cut, a page number outside the cache is not followed
    assert qg.qgemm_device_status(reset=True) == 0

    def status(c, **kw):
        qg.qattn_forward(c.q, c.cache(qg), c.batch(qg, **kw))
        return qg.qgemm_device_status(reset=True)

    make = lambda: Case([1, 1], [40, 30], 300, 8, 2, 128, 16, BF, seed=21)
    assert status(make()) == 0
    assert status(make(), max_kv=30) == -7
    c = make()
    c.kv_len[1] = -1
    assert status(c) == -7
    for bad in (-1, 1 << 20, 0x7FFFFFFF):
        c = make()
        c.table[0, 1] = bad
        assert status(c) == -7
        c = make()
        c.prefix_table[3] = bad
        assert status(c) == -7
    # more new tokens than max_q says
    c = Case([5, 1], [40, 30], 300, 8, 2, 128, 16, BF, seed=22)
    assert status(c, max_q=1) == -7
    # offsets that are not ascending, in each of the ways a call is run
    for n_q, prefix in (([1, 1, 1], 0), ([1] * 40, 2500), ([100, 90, 70], 300)):
        c = Case(n_q, [n + 100 for n in n_q], prefix, 64, 8, 128, 64, BF, seed=24)
        c.cu_q[1::2] = c.T
        c.cu_q[2::2] = 0
        c.cu_q[-1] = c.T
        status(c)   # finishes, whatever it reports
    # a sound call afterwards
    c = make()
    check_attention(c, *_run(qg, c))


@pytest.mark.parametrize("n_q,prefix", [([1, 1, 1], 0), ([1] * 5, 700), ([1] * 40, 2500), ([100, 90, 70], 300)])
def test_offsets_past_the_rows_are_reported(qg, n_q, prefix):
    # the last sequence claims rows that are not there, in each of the ways a call is run: the others are as they were
    assert qg.qgemm_device_status(reset=True) == 0
    c = Case(n_q, [n + 30 for n in n_q], prefix, 64, 8, 128, 64, BF, seed=26)
    want, _ = _run(qg, c)
    for past in (c.T + 1, 0x7FFFFFFF):
        c.cu_q[-1] = past
        out = qg.qattn_forward(c.q, c.cache(qg), c.batch(qg))
        assert qg.qgemm_device_status(reset=True) == -7
        assert torch.equal(out[:c.cu[-2]], want[:c.cu[-2]])
    # and one without rows, past their end
    c.cu_q[-2:] = c.T + 5
    qg.qattn_forward(c.q, c.cache(qg), c.batch(qg))
    assert qg.qgemm_device_status(reset=True) == -7


def test_offsets_whose_pairs_of_tiles_pass_32_bits(qg):
    # every other sequence claims all 2^16 tokens, a tile holds one of them: the pairs of tiles add up to 2^31
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    assert qg.qgemm_device_status(reset=True) == 0
    T, B = 1 << 16, (1 << 17) + 1
    cache = qg.KVCache.empty(1, 16, 1, 64)
    cache.k.fill_(1.0)
    cache.v.fill_(2.0)
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu[1::2] = T
    batch = qg.KVBatch(torch.zeros((B, 1), dtype=torch.int32, device="cuda"), torch.ones(B, dtype=torch.int32, device="cuda"),
                       max_kv=1, cu_q=cu, max_q=1, tokens=T)
    q = torch.zeros((T + 2, 128, 64), dtype=BF, device="cuda")
    out = torch.full_like(q, 7.0)
    qg.qattn_forward(q[1:-1], cache, batch, out=out[1:-1])
    assert qg.qgemm_device_status(reset=True) == -7
    assert (out[0] == 7.0).all() and (out[-1] == 7.0).all()
    del q, out
    torch.cuda.empty_cache()
    c = Case([100, 90], [100, 90], 0, 16, 2, 128, 16, BF, seed=25)
    check_attention(c, *_run(qg, c))


def test_refusals(qg):
    c = Case([1, 1], [40, 30], 300, 8, 2, 128, 16, BF, seed=23)
    cache, batch = c.cache(qg), c.batch(qg)
    with pytest.raises(ValueError):
        qg.qattn_forward(c.q.half(), cache, batch)
    with pytest.raises(ValueError):
        qg.qattn_forward(c.q[:1], cache, batch)
    with pytest.raises(qg.QgError) as e:
        qg.qattn_forward(c.q[:, :7].contiguous(), cache, batch)
    assert e.value.status == -1
    for scale in (0.0, -1.0, math.inf, math.nan):
        with pytest.raises(qg.QgError):
            qg.qattn_forward(c.q, cache, batch, scale=scale)
    with pytest.raises(ValueError):
        qg.qattn_forward(c.q, cache, c.batch(qg, max_kv=10000))
    with pytest.raises(ValueError):
        qg.qattn_forward(c.q, cache, c.batch(qg, prefix_len=10000))
    with pytest.raises(qg.QgError) as e:
        qg.qattn_forward(c.q, cache, batch, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert e.value.status == -4
