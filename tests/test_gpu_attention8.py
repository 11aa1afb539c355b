"""Attention over the 8-bit paged cache against its definition in 64 bits: head
layouts, page sizes, lengths from one token on, shared prefixes, several new
tokens a sequence, and everything past a length poisoned."""
import math

import pytest
import torch

from _paged import check_attention
from _paged8 import BLOCK, NAN_CODE, Case8

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
    need = qg.qattn_workspace_size(cache, batch, c.heads_q)
    ws = torch.full((need + 1024,), 0xFF, dtype=torch.uint8, device="cuda")
    qg.qattn_forward(c.q, cache, batch, scale=scale, out=out, lse=lse, workspace=ws)
    torch.cuda.synchronize()
    assert qg.qgemm_device_status() == 0
    # rows of no sequence are left alone, and so is what follows the workspace
    assert (out[c.cu[-1]:] == 7.0).all() and (lse[c.cu[-1]:] == 7.0).all() and (ws[need:] == 0xFF).all()
    return out, lse


HEADS = [(8, 8, 128), (8, 1, 128), (16, 2, 64), (28, 4, 128), (9, 3, 64), (64, 8, 128)]


@pytest.mark.parametrize("heads_q,heads_kv,dim", HEADS)
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("page,heads_first", [(16, True), (64, False), (256, True)])
def test_decode_heads_and_pages(qg, heads_q, heads_kv, dim, dtype, page, heads_first):
    c = Case8([1, 1, 1], [1, 77, 200], 0, heads_q, heads_kv, dim, page, dtype, heads_first, seed=heads_q + page)
    check_attention(c, *_run(qg, c))


@pytest.mark.parametrize("prefix", [1, 15, 16, 17, 63, 64, 65, 255, 256, 257, 1000])
@pytest.mark.parametrize("dtype,dim", [(BF, 128), (FP, 64)])
def test_shared_prefix_lengths(qg, prefix, dtype, dim):
    c = Case8([1] * 5, [1, 2, 64, 65, 130], prefix, 16, 2, dim, 32, dtype, seed=prefix)
    check_attention(c, *_run(qg, c))


@pytest.mark.parametrize("own", [1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 128, 129, 500, 1025])
def test_own_lengths(qg, own):
    c = Case8([1, 1], [own, max(1, own - 1)], 300, 8, 2, 128, 16, BF, False, seed=own)
    check_attention(c, *_run(qg, c))


@pytest.mark.parametrize("B", [1, 2, 3, 7, 16, 17, 33, 40])
def test_batch_sizes(qg, B):
    c = Case8([1] * B, [1 + (37 * b) % 90 for b in range(B)], 700, 16, 2, 128, 64, BF, seed=B)
    check_attention(c, *_run(qg, c))


@pytest.mark.parametrize("heads_q,heads_kv,dim,dtype,page,heads_first", [
    (64, 8, 128, BF, 64, True), (64, 8, 128, FP, 16, False), (32, 8, 64, FP, 128, True), (28, 4, 128, BF, 32, False),
    (32, 32, 128, BF, 64, True), (48, 1, 64, BF, 256, True), (100, 1, 128, FP, 64, True)])
@pytest.mark.parametrize("n_q,prefix", [([1] * 33, 2500), ([1] * 90, 2049), ([3, 1, 5, 0, 2] * 9, 2431)])
def test_much_shared_prefix(qg, heads_q, heads_kv, dim, dtype, page, heads_first, n_q, prefix):
    # enough rows and keys that the prefix is worked on in tiles: pairs of tiles, a single one, a cut last block
    kv = [max(n, 1) + (31 * b) % 150 for b, n in enumerate(n_q)]
    c = Case8(n_q, kv, prefix, heads_q, heads_kv, dim, page, dtype, heads_first, seed=len(n_q) + page, spare_tokens=2)
    check_attention(c, *_run(qg, c))


@pytest.mark.parametrize("heads_q,heads_kv,dim", [(16, 2, 128), (32, 8, 64)])
def test_rows_packed_across_sequences(qg, heads_q, heads_kv, dim):
    # more than 64 rows a sequence and head, few of its own keys: the prefix's tiles hold rows of several sequences
    n_q = [20, 17, 1, 19] * 10
    c = Case8(n_q, [n + b for b, n in enumerate(n_q)], 4000, heads_q, heads_kv, dim, 64, BF, seed=30)
    check_attention(c, *_run(qg, c))


@pytest.mark.parametrize("n_q,kv", [([1, 5, 2], [1, 9, 200]), ([8, 8], [8, 64]), ([3, 0, 4, 1], [70, 50, 4, 1]),
                                    ([17, 33], [17, 129]), ([64], [300]), ([130, 1, 90], [130, 65, 191]),
                                    ([257, 3], [400, 3])])
@pytest.mark.parametrize("heads_q,heads_kv,dim", [(16, 2, 128), (7, 1, 64), (4, 4, 128), (136, 1, 128)])
@pytest.mark.parametrize("prefix", [0, 333])
def test_several_tokens(qg, n_q, kv, heads_q, heads_kv, dim, prefix):
    c = Case8(n_q, kv, prefix, heads_q, heads_kv, dim, 16, BF, seed=sum(n_q) + prefix, spare_tokens=3)
    check_attention(c, *_run(qg, c))


@pytest.mark.parametrize("prefix", [0, 400])
def test_rows_that_see_nothing(qg, prefix):
    # own lengths below the count of new tokens: the first rows see no own token (and without a prefix nothing)
    c = Case8([4, 2, 70, 1], [2, 0, 33, 0], prefix, 8, 2, 128, 16, BF, seed=3)
    out, lse = _run(qg, c)
    check_attention(c, out, lse)
    if prefix == 0:
        assert (out[:2] == 0).all() and (out[4:6] == 0).all() and torch.isinf(lse[:2]).all()


WAYS = [([1, 1, 1], [70, 2000, 33], 0), ([1] * 5, [9, 300, 1, 64, 65], 700), ([1] * 33, [200] * 33, 2500),
        ([4] * 20, [70] * 20, 2500), ([130, 90, 70], [130, 200, 70], 333)]


@pytest.mark.parametrize("n_q,kv,prefix", WAYS)
def test_not_finite_stays_not_finite_and_in_its_place(qg, n_q, kv, prefix):
    # a NaN key makes the rows that see it NaN in any way a call is split, and changes no bit of any other row
    c = Case8(n_q, kv, prefix, 64, 8, 128, 16, BF, seed=40)
    clean, lse0 = _run(qg, c)
    check_attention(c, clean, lse0)
    rows = torch.arange(c.cu[1], c.cu[2], device="cuda")

    def expect(seen, out, lse, heads):
        bad = torch.zeros((c.T, c.heads_q), dtype=torch.bool, device="cuda")
        bad[seen[:, None], torch.tensor(heads, device="cuda")] = True
        assert out[bad].isnan().all() and lse[bad].isnan().all()
        assert torch.equal(out[~bad], clean[~bad]) and torch.equal(lse[~bad], lse0[~bad])

    for key, seen in ((0, rows), (kv[1] - 1, rows[-1:])):   # seen by all of the sequence's tokens, by its last alone
        page, at = c.table[1, key // c.page].item(), key % c.page
        kept = c.k_codes[page, at, 2, 5].clone()
        c.k_codes[page, at, 2, 5] = NAN_CODE
        expect(seen, *_run(qg, c), list(range(16, 24)))
        c.k_codes[page, at, 2, 5] = kept
    if prefix:
        page = c.prefix_table[prefix // 2 // c.page].item()
        kept = c.k_codes[page, 0, 7, 100].clone()
        c.k_codes[page, 0, 7, 100] = NAN_CODE
        expect(torch.arange(c.T, device="cuda"), *_run(qg, c), list(range(56, 64)))
        c.k_codes[page, 0, 7, 100] = kept
    # a NaN in the first own value: that column of its rows alone
    page = c.table[1, 0].item()
    c.v_codes[page, 0, 0, 9] = 0x80 | NAN_CODE
    out, lse = _run(qg, c)
    bad = torch.zeros_like(out, dtype=torch.bool)
    bad[c.cu[1]:c.cu[2], :8, 9] = True
    assert out[bad].isnan().all() and torch.equal(out[~bad], clean[~bad]) and torch.equal(lse, lse0)


@pytest.mark.parametrize("out_dtype", [torch.float32, BF, FP])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_output_types_and_scale(qg, out_dtype, dtype):
    c = Case8([1, 1, 40], [50, 3, 90], 500, 8, 4, 128, 32, dtype, seed=8)
    for scale in (0.25, 1e-3):
        out, lse = _run(qg, c, scale=scale, out_dtype=out_dtype)
        check_attention(c, out, lse, scale)


@pytest.mark.parametrize("n_q,kv,prefix", WAYS)
def test_large_logits(qg, n_q, kv, prefix):
    # logits in the hundreds: the softmax is all but one-hot, and only the running maximum keeps it finite
    c = Case8(n_q, kv, prefix, 16, 2, 128, 16, BF, seed=9, spread=60.0)
    check_attention(c, *_run(qg, c))


@pytest.mark.parametrize("n_q,kv,prefix", WAYS)
@pytest.mark.parametrize("shift", [0, 20, -30])
def test_scales_far_apart(qg, n_q, kv, prefix, shift):
    # blocks of V (and of K) many powers of two apart, all of them far from 1, and blocks of zeros: what a row sees may
    # come from any of them
    c = Case8(n_q, kv, prefix, 16, 2, 128, 16, BF, seed=50, swing=0.5)
    g = torch.Generator(device="cpu").manual_seed(51)
    move = torch.randint(-6, 7, c.v_scale.shape, generator=g).cuda()
    c.v_scale = torch.where(c.v_scale == 255, 255, (c.v_scale.int() + move + shift).clamp(1, 254)).to(torch.uint8)
    c.k_scale = torch.where(c.k_scale == 255, 255, (c.k_scale.int() + shift).clamp(1, 254)).to(torch.uint8)
    c.q = (c.q.float() * 2.0 ** -shift).to(BF)
    page = c.table[1, 0].item()
    c.v_codes[page, :min(BLOCK, kv[1])] = 0
    c.v_scale[page, 0] = 127 - 64
    c.refresh()
    check_attention(c, *_run(qg, c, out_dtype=torch.float32))


@pytest.mark.parametrize("magnitude", [2.0 ** -100, 2.0 ** -20, 2.0 ** 60])
def test_queries_of_any_magnitude(qg, magnitude):
    # rows of q are scaled to fp16's range: far outside it, and with rows of zeros among them
    for n_q, kv, prefix in WAYS:
        c = Case8(n_q, kv, prefix, 16, 2, 128, 16, BF, seed=52)
        c.q = (c.q.float() * magnitude).to(BF)
        c.q[0, 3] = 0
        scale = min(0.09 / magnitude, 1e38)
        check_attention(c, *_run(qg, c, scale=scale), scale)


def test_strided_arrays(qg):
    # q inside the fused product's rows, out inside wider rows, K and V (and their scales) interleaved page by page
    c = Case8([1, 3, 1], [40, 20, 99], 290, 16, 2, 128, 16, BF, False, seed=12)
    for names in (("k_codes", "v_codes"), ("k_scale", "v_scale")):
        k, v = (getattr(c, n) for n in names)
        both = torch.empty((k.shape[0], 2, *k.shape[1:]), dtype=torch.uint8, device="cuda")
        both[:, 0], both[:, 1] = k, v
        setattr(c, names[0], both[:, 0])
        setattr(c, names[1], both[:, 1])
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
    # few items of many keys: cut to pieces over many CTAs.  Nothing past the workspace is written (_run looks).
    c = Case8(n_q, kv, 0, heads_q, heads_kv, dim, 64, BF, seed=27)
    check_attention(c, *_run(qg, c))


def test_one_token_each_without_offsets(qg):
    c = Case8([1] * 6, [3, 1, 20, 64, 65, 18], 260, 8, 2, 64, 16, FP, seed=13)
    check_attention(c, *_run(qg, c, cu_q=None))


def test_looser_bounds_change_nothing(qg):
    # bounds above the lengths: the same result within the error of both
    c = Case8([1, 4, 2], [70, 4, 33], 270, 8, 2, 128, 16, BF, seed=14)
    wide = torch.zeros((3, 64), dtype=torch.int32, device="cuda")
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide
    check_attention(c, *_run(qg, c, max_kv=1000, max_q=9))


@pytest.mark.parametrize("n_q,kv,prefix", [([1] * 20, [300] * 20, 5000), ([1] * 60, [300] * 60, 20000),
                                           ([200, 200], [200, 500], 700), ([1], [9000], 0)])
def test_repeatable_bit_for_bit(qg, n_q, kv, prefix):
    c = Case8(n_q, kv, prefix, 16, 2, 128, 64, BF, seed=15)
    a, la = _run(qg, c)
    for _ in range(3):
        b, lb = _run(qg, c)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_long_prefix_and_long_own(qg):
    c = Case8([1, 1, 2], [4500, 17, 9000], 20000, 16, 2, 128, 64, BF, seed=16)
    check_attention(c, *_run(qg, c))


def test_offsets_past_32_bits(qg):
    # pages 2^22 codes apart: the last ones start past 2^32 bytes, and so do their scales, 2^21 bytes and more apart
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB")
    c = Case8([1, 2], [40, 130], 300, 8, 2, 128, 16, BF, seed=17, poison=False)
    n, first = c.k_codes.shape[0], 1500
    far = first + torch.arange(n, device="cuda")
    for name in ("k", "v"):
        big = torch.empty((1600, 2, 16384, 128), dtype=torch.uint8, device="cuda")[:, :, :16].transpose(1, 2)
        big[far] = getattr(c, name + "_codes")
        scale = torch.empty((1600, 2, 1 << 21), dtype=torch.uint8, device="cuda")[:, :, :1].transpose(1, 2)
        scale[far] = getattr(c, name + "_scale")
        setattr(c, name + "_codes", big)
        setattr(c, name + "_scale", scale)
    c.table, c.prefix_table = c.table + first, c.prefix_table + first
    out, lse = _run(qg, c)
    for name in ("k", "v"):   # the reference from the pages alone
        setattr(c, name + "_codes", getattr(c, name + "_codes")[far].contiguous())
        setattr(c, name + "_scale", getattr(c, name + "_scale")[far].contiguous())
    c.table, c.prefix_table = c.table - first, c.prefix_table - first
    c.refresh()
    check_attention(c, out, lse)
    del big, scale
    torch.cuda.empty_cache()


@pytest.mark.parametrize("prefix", [0, 400, 3000])
def test_fewer_tokens_than_rows(qg, prefix):
    # a batch that has shrunk: most rows belong to no sequence, in each of the ways a call is run
    for n_q in ([1, 1], [100, 3], [0, 0], [0, 7]):
        c = Case8(n_q, [n + 5 for n in n_q], prefix, 64, 8, 128, 64, BF, seed=43, spare_tokens=200)
        check_attention(c, *_run(qg, c))
    c = Case8([1, 0, 1] + [0] * 60, [9] * 63, prefix, 64, 8, 128, 64, BF, seed=44, spare_tokens=61)
    check_attention(c, *_run(qg, c))


@pytest.mark.parametrize("n_q,kv,prefix", WAYS)
def test_captured_graphs_with_new_lengths(qg, n_q, kv, prefix):
    # lengths, tables and scales are read when the graph runs; two graphs share a workspace
    c = Case8(n_q, kv, prefix, 16, 2, 128, 16, BF, seed=18, poison=False)
    cache, batch = c.cache(qg), c.batch(qg)
    ws = torch.empty(qg.qattn_workspace_size(cache, batch, 16), dtype=torch.uint8, device="cuda")
    outs = [torch.empty_like(c.q) for _ in range(2)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graphs = []
    with torch.cuda.stream(s):
        qg.qattn_forward(c.q, cache, batch, out=outs[0], workspace=ws)
        s.synchronize()
        for out in outs:
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                qg.qattn_forward(c.q, cache, batch, out=out, workspace=ws)
            graphs.append(g)
    for less in (0, 1, 5):
        c.kv = [max(n, k - less) for n, k in zip(n_q, kv)]
        c.kv_len.copy_(torch.tensor(c.kv, dtype=torch.int32))
        for g, out in zip(graphs, outs):
            out.zero_()
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for out in outs:
            check_attention(c, out)


def test_other_stream(qg):
    c = Case8([1, 1], [100, 30], 500, 8, 2, 128, 16, BF, seed=19)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.empty_like(c.q)
    qg.qattn_forward(c.q, c.cache(qg), c.batch(qg), out=out, stream=s)
    s.synchronize()
    check_attention(c, out)


@pytest.mark.parametrize("n_q,kv,prefix", WAYS)
def test_dependent_launch_off_gives_the_same(qg, n_q, kv, prefix):
    c = Case8(n_q, kv, prefix, 16, 2, 128, 16, BF, seed=20)
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

    for n_q, kv, prefix in WAYS:
        make = lambda: Case8(n_q, kv, prefix, 16, 2, 128, 16, BF, seed=21)
        assert status(make()) == 0
        assert status(make(), max_kv=max(kv) - 1) == -7
        c = make()
        c.kv_len[1] = -1
        assert status(c) == -7
        for bad in (-1, 1 << 20, 0x7FFFFFFF):
            c = make()
            c.table[1, 0] = bad
            assert status(c) == -7
            if prefix:
                c = make()
                c.prefix_table[3] = bad
                assert status(c) == -7
        # offsets that are not ascending, or past the rows
        c = make()
        c.cu_q[1::2] = c.T
        c.cu_q[2::2] = 0
        c.cu_q[-1] = c.T
        status(c)   # finishes, whatever it reports
        c = make()
        want, _ = _run(qg, c)
        c.cu_q[-1] = c.T + 1
        out = qg.qattn_forward(c.q, c.cache(qg), c.batch(qg))
        assert qg.qgemm_device_status(reset=True) == -7
        assert torch.equal(out[:c.cu[-2]], want[:c.cu[-2]])
    # more new tokens than max_q says
    c = Case8([5, 1], [40, 30], 300, 8, 2, 128, 16, BF, seed=22)
    assert status(c, max_q=1) == -7
    # a sound call afterwards
    c = make()
    check_attention(c, *_run(qg, c))


def test_refusals(qg):
    c = Case8([1, 1], [40, 30], 300, 8, 2, 128, 16, BF, seed=23)
    cache, batch = c.cache(qg), c.batch(qg)
    with pytest.raises(ValueError):
        qg.qattn_forward(c.q.float(), cache, batch)
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
    with pytest.raises(qg.QgError) as e:
        qg.qattn_forward(c.q, cache, batch, workspace=torch.empty(0, dtype=torch.uint8, device="cuda"))
    assert e.value.status == -4
    for bad in (c.k_scale[:, :0], c.k_scale.float(), c.k_scale[1:]):
        with pytest.raises(ValueError):
            qg.KVCache8(cache.k, cache.v, bad, c.v_scale)
    with pytest.raises(ValueError):
        qg.KVCache8(c.k_codes, c.v_codes, c.k_scale, c.v_scale)
