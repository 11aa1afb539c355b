"""Appending to the paged cache against its definition in 64 bits: types,
rotations, layouts, lengths, and every value the call must leave alone."""
import pytest
import torch

from _paged import UNIT, Case

pytestmark = pytest.mark.gpu
F32, BF, FP = torch.float32, torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def qg():
    import bit_weight_only_group_gb300 as qg
    qg.lib()
    qg.qgemm_device_status(reset=True)
    yield qg
    assert qg.qgemm_device_status() == 0


def _rope(positions, rot):
    at = torch.arange(positions, dtype=torch.float64)
    angle = at[:, None] * 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64) / rot)
    return torch.cat([angle.cos(), angle.sin()], 1).float().cuda()


def _turned(x, rope, at, interleaved):
    """x [T, heads, dim] in 64 bits with row at[t] of the table applied, and the sum of the absolute terms."""
    y, size = x.clone(), x.abs()
    if rope is None:
        return y, size
    rot = rope.shape[1]
    cos, sin = rope[at, :rot // 2].double()[:, None], rope[at, rot // 2:].double()[:, None]
    a = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
    b = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
    y[..., a], y[..., b] = x[..., a] * cos - x[..., b] * sin, x[..., b] * cos + x[..., a] * sin
    both = x[..., a].abs() + x[..., b].abs()
    size[..., a] = both
    size[..., b] = both
    return y, size


def _close(got, ref, size):
    # a product, a fused product and sum (fp32), one rounding to the type; fp16 results below 2^-14 have steps of 2^-24
    room = UNIT[got.dtype] * ref.abs() + 2 * 2.0 ** -23 * size + (2.0 ** -25 if got.dtype == FP else 0.0)
    assert ((got.double() - ref).abs() <= room).all()


def _check(qg, c, xt, rot=None, interleaved=False, positions=None, with_q=True, split=False):
    T, D, used = c.T, c.dim, c.cu[-1]
    g = torch.Generator(device="cpu").manual_seed(99)
    width = (c.heads_q + 2 * c.heads_kv) * D
    qkv = torch.randn((T, width), generator=g).to(xt).cuda()
    if split:   # arrays of their own, not columns of one
        q, k, v = (t.contiguous().view(T, -1, D) for t in qkv.split([c.heads_q * D, c.heads_kv * D, c.heads_kv * D], 1))
    else:
        q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([c.heads_q * D, c.heads_kv * D, c.heads_kv * D], 1))
    rope = _rope(c.prefix + max(c.kv) + 5, rot) if rot else None
    before_k, before_v = c.k.clone(), c.v.clone()
    q_out = torch.full((T, c.heads_q, D), 7.0, dtype=c.dtype, device="cuda")
    got = qg.qkv_append(c.cache(qg), c.batch(qg), k, v, q=q if with_q else None, rope=rope, interleaved=interleaved,
                        positions=positions, q_out=q_out if with_q else None)
    torch.cuda.synchronize()
    assert qg.qgemm_device_status() == 0
    where, at = [], []
    for b in range(c.B):
        for i in range(c.n_q[b]):
            own = c.kv[b] - c.n_q[b] + i
            where.append((c.table_host[b, own // c.page].item(), own % c.page))
            at.append(c.prefix + own)
    at = torch.tensor(at, device="cuda", dtype=torch.long) if positions is None else positions[:used].long()
    if with_q:
        assert got is q_out and (q_out[used:] == 7.0).all()
        _close(q_out[:used], *_turned(q[:used].double(), rope, at, interleaved))
    page, place = (torch.tensor(x, device="cuda") for x in zip(*where))
    _close(c.k[page, place], *_turned(k[:used].double(), rope, at, interleaved))
    assert torch.equal(c.v[page, place], v[:used].to(c.dtype))
    # everything else as it was
    before_k[page, place], before_v[page, place] = c.k[page, place], c.v[page, place]
    for a, b in ((before_k, c.k), (before_v, c.v)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("xt", [F32, BF, FP])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(128, 128), (128, 32), (128, 16), (64, 64), (64, 48), (128, None)])
def test_types_and_rotations(qg, xt, dtype, interleaved, dim, rot):
    c = Case([3, 1, 2], [3, 40, 65], 21, 6, 2, dim, 16, dtype, seed=1, garbage=3.0)
    _check(qg, c, xt, rot, interleaved)


@pytest.mark.parametrize("heads_q,heads_kv", [(1, 1), (64, 8), (32, 32), (28, 4), (71, 1), (128, 16)])
@pytest.mark.parametrize("heads_first", [True, False])
@pytest.mark.parametrize("page", [16, 128])
def test_layouts(qg, heads_q, heads_kv, heads_first, page):
    c = Case([1, 5], [200, 16], 0, heads_q, heads_kv, 128, page, BF, heads_first, seed=2, garbage=3.0)
    _check(qg, c, BF, 128)


@pytest.mark.parametrize("B", [1, 2, 31, 32, 33, 100, 1100])
def test_batch_sizes_and_empty_sequences(qg, B):
    n_q = [(b * 7) % 4 for b in range(B)]
    n_q[B // 2] = 2
    c = Case(n_q, [n + (b % 5) for b, n in enumerate(n_q)], 9, 2, 1, 64, 16, BF, seed=B, spare_tokens=4, garbage=3.0)
    _check(qg, c, BF, 64)


@pytest.mark.parametrize("used", [0, 1, 5])
def test_fewer_tokens_than_rows(qg, used):
    # rows of no sequence, as in a captured step whose batch has shrunk: nothing is read or written for them
    c = Case([1] * used or [0], [3] * max(used, 1), 9, 4, 2, 128, 16, BF, seed=40, spare_tokens=300, garbage=3.0)
    if used:
        _check(qg, c, BF, 128)
    else:
        before = c.k.clone()
        k = torch.randn((c.T, 2, 128), device="cuda").to(BF)
        qg.qkv_append(c.cache(qg), c.batch(qg), k, k, rope=_rope(20, 128))
        torch.cuda.synchronize()
        assert qg.qgemm_device_status() == 0 and torch.equal(before.view(torch.int16), c.k.view(torch.int16))


def test_many_tokens_a_cta(qg):
    # more than 32 units a CTA, over sequences of all lengths, heads that take several units a token
    n_q = [(37 * b) % 61 for b in range(330)]
    c = Case(n_q, [n + b % 7 for b, n in enumerate(n_q)], 5, 2, 2, 64, 16, FP, seed=41, garbage=3.0)
    _check(qg, c, F32, 32)
    n_q = [150, 0, 211, 3]
    c = Case(n_q, [n + 3 for n in n_q], 5, 128, 32, 128, 64, BF, False, seed=42, garbage=3.0)
    _check(qg, c, F32, 128, interleaved=True)


def test_given_positions(qg):
    c = Case([3, 2], [3, 40], 10, 4, 2, 128, 16, BF, seed=4, garbage=3.0)
    _check(qg, c, BF, 128, positions=torch.tensor([0, 44, 7, 7, 1], dtype=torch.int32, device="cuda"))


def test_without_queries_and_separate_arrays(qg):
    c = Case([3, 2], [3, 40], 10, 4, 2, 128, 16, FP, seed=5, garbage=3.0)
    _check(qg, c, F32, 64, with_q=False)
    _check(qg, c, BF, 64, split=True)


def test_positions_and_places_outside_are_reported(qg):
    assert qg.qgemm_device_status(reset=True) == 0
    c = Case([2, 1], [1, 20], 0, 4, 2, 128, 16, BF, seed=6, garbage=3.0)   # sequence 0: the first token has no place
    k = torch.randn((3, 2, 128), device="cuda").to(BF)
    before = c.k.clone()
    qg.qkv_append(c.cache(qg), c.batch(qg), k, k)
    assert qg.qgemm_device_status(reset=True) == -7
    p0, p1 = c.table_host[0, 0].item(), c.table_host[1, 1].item()
    before[p0, 0], before[p1, 3] = k[1], k[2]
    assert torch.equal(before, c.k)
    # a position past the rotation table: the token is not written
    c = Case([1, 1], [5, 20], 0, 4, 2, 128, 16, BF, seed=7, garbage=3.0)
    before = c.k.clone()
    qg.qkv_append(c.cache(qg), c.batch(qg), k[:2], k[:2], rope=_rope(10, 128))
    assert qg.qgemm_device_status(reset=True) == -7
    before[c.table_host[0, 0].item(), 4] = c.k[c.table_host[0, 0].item(), 4]
    assert torch.equal(before, c.k)
    # a page outside the cache
    c.table[0, 0] = 1 << 20
    before = c.k.clone()
    qg.qkv_append(c.cache(qg), c.batch(qg), k[:2], k[:2])
    assert qg.qgemm_device_status(reset=True) == -7
    before[c.table_host[1, 1].item(), 3] = k[1]
    assert torch.equal(before, c.k)


@pytest.mark.parametrize("heads_first", [True, False])
def test_lengths_outside_their_bounds_leave_the_cache_alone(qg, heads_first):
    # the sequence's keys so far are still there after a call that counted its tokens wrongly; other sequences are written
    assert qg.qgemm_device_status(reset=True) == 0
    c = Case([2, 1, 1], [40, 20, 33], 0, 4, 2, 128, 16, BF, heads_first, seed=10, garbage=3.0)
    k, q = torch.randn((4, 2, 128), device="cuda").to(BF), torch.randn((4, 4, 128), device="cuda").to(BF)
    where = [[(c.table_host[b, own // 16].item(), own % 16) for own in range(c.kv[b] - c.n_q[b], c.kv[b])] for b in range(3)]

    def check(written, **bounds):
        before_k, before_v = c.k.clone(), c.v.clone()
        q_out = qg.qkv_append(c.cache(qg), c.batch(qg, **bounds), k, -k, q=q)
        assert qg.qgemm_device_status(reset=True) == -7
        for b in written:
            for i, (page, place) in enumerate(where[b]):
                before_k[page, place], before_v[page, place] = k[c.cu[b] + i], -k[c.cu[b] + i]
        for a, b in ((before_k, c.k), (before_v, c.v)):
            assert torch.equal(a.view(torch.int16), b.view(torch.int16))
        assert all(torch.equal(q_out[c.cu[b]:c.cu[b + 1]], q[c.cu[b]:c.cu[b + 1]]) for b in written)

    check([1, 2], max_kv=39)          # sequence 0 is longer than its bound
    check([1], max_kv=32)             # and sequence 2
    check([1, 2], max_q=1)            # sequence 0 has more new tokens than its bound
    for bad in (-1, -(1 << 31), 1 << 30, 0x7FFFFFFF):
        c.kv_len[1] = bad
        check([0, 2])
    c.kv_len[1] = 20


def test_offsets_past_the_rows_are_reported(qg):
    # the last sequence claims a row that is not there: it is not cached, the others are
    assert qg.qgemm_device_status(reset=True) == 0
    c = Case([2, 1, 2], [40, 20, 33], 0, 4, 2, 128, 16, BF, seed=11, garbage=3.0)
    k = torch.randn((5, 2, 128), device="cuda").to(BF)
    c.cu_q[3] = 6
    before = c.k.clone()
    qg.qkv_append(c.cache(qg), c.batch(qg), k, k)
    assert qg.qgemm_device_status(reset=True) == -7
    for t, (b, own) in enumerate([(0, 38), (0, 39), (1, 19)]):
        before[c.table_host[b, own // 16].item(), own % 16] = k[t]
    assert torch.equal(before, c.k)


def test_append_then_attend(qg):
    """The two calls as a decoding step uses them: the appended tokens are what the attention sees."""
    from _paged import check_attention
    c = Case([1, 3, 1], [18, 40, 65], 300, 8, 2, 128, 16, BF, seed=8)
    used = c.T
    qkv = torch.randn((used, 12 * 128), device="cuda").to(BF)
    q, k, v = (t.unflatten(1, (-1, 128)) for t in qkv.split([8 * 128, 2 * 128, 2 * 128], 1))
    cache, batch = c.cache(qg), c.batch(qg)
    c.q = qg.qkv_append(cache, batch, k, v, q=q, rope=_rope(400, 128))
    out = qg.qattn_forward(c.q, cache, batch)
    check_attention(c, out)


def test_refusals(qg):
    c = Case([1, 1], [5, 20], 0, 4, 2, 128, 16, BF, seed=9)
    cache, batch = c.cache(qg), c.batch(qg)
    k = torch.zeros((2, 2, 128), dtype=BF, device="cuda")
    with pytest.raises(ValueError):
        qg.qkv_append(cache, batch, k, k.half())
    with pytest.raises(ValueError):
        qg.qkv_append(cache, batch, k[:, :1], k)
    with pytest.raises(ValueError):
        qg.qkv_append(cache, batch, k.transpose(0, 1).contiguous().transpose(0, 1), k)
    for bad in (24, 144):
        with pytest.raises(qg.QgError) as e:
            qg.qkv_append(cache, batch, k, k, rope=torch.zeros((30, bad), device="cuda"))
        assert e.value.status == -2
    with pytest.raises(ValueError):
        qg.qkv_append(cache, batch, k, k, rope=torch.zeros((30, 128), device="cuda"),
                      positions=torch.zeros(3, dtype=torch.int32, device="cuda"))
