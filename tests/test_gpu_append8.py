"""Appending with the norms of queries and keys, appending to the 8-bit paged
cache and reading it back, against their definitions in 64 bits: types,
rotations, layouts, lengths, blocks that grow, and every value the calls must
leave alone."""
import math

import pytest
import torch

from _paged import UNIT, Case, check_attention
from _paged8 import BLOCK, E4M3, E_MAX, E_MIN, Case8, exponent, nearest, pow2, values

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


def _turned(x, w, eps, rope, at, interleaved):
    """x [T, heads, dim] in 64 bits normed (w) and turned by rows at[t] of the table, and a bound of the fp32 error."""
    y, rel = x.clone(), 0.0
    if w is not None:
        y = y / (y.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
        # the sum of squares (at most dim roundings, halved by the root), rsqrtf (2^-22), its argument and two products
        rel = 2.0 ** -22 + (x.shape[-1] / 2 + 4) * 2.0 ** -24
    size = y.abs()
    room = rel * size
    if rope is not None:
        rot = rope.shape[1]
        cos, sin = rope[at, :rot // 2].double()[:, None], rope[at, rot // 2:].double()[:, None]
        a = slice(0, rot, 2) if interleaved else slice(0, rot // 2)
        b = slice(1, rot, 2) if interleaved else slice(rot // 2, rot)
        s, c = y[..., a].clone(), y[..., b].clone()
        y[..., a], y[..., b] = s * cos - c * sin, c * cos + s * sin
        # a product, a fused product and sum
        room[..., a] = room[..., b] = (rel + 2 * 2.0 ** -23) * (s.abs() + c.abs())
    return y, room


def _close(got, ref, room):
    # one rounding to the type; fp16 results below 2^-14 have steps of 2^-24
    room = UNIT[got.dtype] * (ref.abs() + room) + room + (2.0 ** -25 if got.dtype == FP else 0.0)
    assert ((got.double() - ref).abs() <= room).all()


def _inputs(c, xt, seed=99, magnitude=1.0):
    g = torch.Generator(device="cpu").manual_seed(seed)
    D = c.dim
    qkv = (magnitude * torch.randn((c.T, (c.heads_q + 2 * c.heads_kv) * D), generator=g)).to(xt).cuda()
    return [t.unflatten(1, (-1, D)) for t in qkv.split([c.heads_q * D, c.heads_kv * D, c.heads_kv * D], 1)]


def _where(c):
    """Sequence, own place, page and place in it of each token."""
    rows = [(b, c.kv[b] - c.n_q[b] + i) for b in range(c.B) for i in range(c.n_q[b])]
    return [(b, own, c.table_host[b, own // c.page].item(), own % c.page) for b, own in rows]


def _norms(c, wt, which):
    g = torch.Generator(device="cpu").manual_seed(5)
    w = [(1 + 0.3 * torch.randn(c.dim, generator=g)).to(wt).cuda() for _ in range(2)]
    return w[0] if "q" in which else None, w[1] if "k" in which else None


# ------------------------------------------------------------------ norms, 16-bit cache
def _check_norm(qg, c, xt, rot=None, interleaved=False, wt=F32, which="qk", eps=1e-6, magnitude=1.0, zero=False):
    q, k, v = _inputs(c, xt, magnitude=magnitude)
    if zero:
        q[0, 0] = 0
        k[0, 0] = 0
    rope = _rope(c.prefix + max(c.kv) + 5, rot) if rot else None
    qw, kw = _norms(c, wt, which)
    before_k, before_v = c.k.clone(), c.v.clone()
    q_out = torch.full((c.T, c.heads_q, c.dim), 7.0, dtype=c.dtype, device="cuda")
    qg.qkv_append(c.cache(qg), c.batch(qg), k, v, q=q, rope=rope, interleaved=interleaved, q_out=q_out, q_norm=qw, k_norm=kw,
                  eps=eps)
    torch.cuda.synchronize()
    assert qg.qgemm_device_status() == 0
    where, used = _where(c), c.cu[-1]
    at = torch.tensor([c.prefix + w[1] for w in where], device="cuda")
    page, place = (torch.tensor([w[i] for w in where], device="cuda") for i in (2, 3))
    assert (q_out[used:] == 7.0).all()
    _close(q_out[:used], *_turned(q[:used].double(), qw, eps, rope, at, interleaved))
    _close(c.k[page, place], *_turned(k[:used].double(), kw, eps, rope, at, interleaved))
    assert torch.equal(c.v[page, place], v[:used].to(c.dtype))
    before_k[page, place], before_v[page, place] = c.k[page, place], c.v[page, place]
    for a, b in ((before_k, c.k), (before_v, c.v)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("xt", [F32, BF, FP])
@pytest.mark.parametrize("dtype,wt", [(BF, F32), (FP, FP), (BF, BF)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(128, 128), (128, 32), (64, 64), (64, 48), (128, None)])
def test_norms_types_and_rotations(qg, xt, dtype, wt, interleaved, dim, rot):
    c = Case([3, 1, 2], [3, 40, 65], 21, 6, 2, dim, 16, dtype, seed=1, garbage=3.0, spare_tokens=2)
    _check_norm(qg, c, xt, rot, interleaved, wt)


@pytest.mark.parametrize("which", ["q", "k"])
@pytest.mark.parametrize("heads_q,heads_kv", [(1, 1), (64, 8), (28, 4), (71, 1)])
def test_one_norm_alone_and_head_counts(qg, which, heads_q, heads_kv):
    c = Case([1, 5], [200, 16], 0, heads_q, heads_kv, 128, 16, BF, False, seed=2, garbage=3.0)
    _check_norm(qg, c, BF, 128, which=which)


@pytest.mark.parametrize("magnitude,eps", [(1e-4, 1e-6), (1e-4, 0.0), (300.0, 1e-5), (1.0, 0.5)])
def test_norms_of_small_and_large_heads(qg, magnitude, eps):
    c = Case([3, 1, 2], [3, 40, 65], 21, 6, 2, 128, 16, BF, seed=3, garbage=3.0)
    _check_norm(qg, c, BF, 128, eps=eps, magnitude=magnitude, zero=eps > 0)


def test_norms_of_many_tokens(qg):
    n_q = [(37 * b) % 61 for b in range(330)]
    c = Case(n_q, [n + b % 7 for b, n in enumerate(n_q)], 5, 2, 2, 64, 16, FP, seed=41, garbage=3.0)
    _check_norm(qg, c, F32, 32)


# ------------------------------------------------------------------ 8 bits
def _check8(qg, c, xt, rot=None, interleaved=False, which="", wt=F32, qt=BF, magnitude=1.0, positions=None, with_q=True,
            change=None):
    """One call, compared with its definition; returns nothing, the cache is as the call left it."""
    q, k, v = _inputs(c, xt, magnitude=magnitude)
    if change is not None:
        change(k, v)
    rope = _rope(c.prefix + max(c.kv) + 5, rot) if rot else None
    qw, kw = _norms(c, wt, which)
    was = {n: getattr(c, n).clone() for n in ("k_codes", "v_codes", "k_scale", "v_scale")}
    q_out = torch.full((c.T, c.heads_q, c.dim), 7.0, dtype=qt, device="cuda")
    got = qg.qkv_append(c.cache(qg), c.batch(qg), k, v, q=q if with_q else None, rope=rope, interleaved=interleaved,
                        positions=positions, q_out=q_out if with_q else None, q_norm=qw if with_q else None, k_norm=kw)
    torch.cuda.synchronize()
    assert qg.qgemm_device_status() == 0
    where, used = _where(c), c.cu[-1]
    at = torch.tensor([c.prefix + w[1] for w in where], device="cuda", dtype=torch.long)
    if positions is not None:
        at = positions[:used].long()
    if with_q:
        assert got is q_out and (q_out[used:] == 7.0).all()
        _close(q_out[:used], *_turned(q[:used].double(), qw, 1e-6, rope, at, interleaved))
    # the blocks the new tokens lie in, the tokens of each, and whether it had any before
    blocks = {}
    for t, (b, own, page, place) in enumerate(where):
        blocks.setdefault((page, place // BLOCK), [own - own % BLOCK < c.kv[b] - c.n_q[b], []])[1].append((t, place))
    for name, x, w in (("k", k, kw), ("v", v, None)):
        y, room = _turned(x[:used].double(), w, 1e-6, rope if name == "k" else None, at, interleaved)
        codes, scale = getattr(c, name + "_codes"), getattr(c, name + "_scale")
        want_codes, want_scale = was[name + "_codes"], was[name + "_scale"]
        for (page, block), (older, tokens) in blocks.items():
            rows = torch.tensor([t for t, _ in tokens], device="cuda")
            places = torch.tensor([p for _, p in tokens], device="cuda")
            z, r = y[rows], room[rows]                                        # [tokens, heads, dim]
            fine = torch.isfinite(z) & (z.abs() <= 448 * 2.0 ** E_MAX)
            amax = torch.where(fine, z, 0.0).abs().amax((0, 2))
            off = torch.where(fine, r, 0.0).amax((0, 2))
            low, high = exponent(amax - off), exponent(amax + off)            # fp32's roundings may cross a border
            e = scale[page, block].int() - 127
            old = want_scale[page, block].int() - 127
            if older:
                low, high = torch.maximum(low, old), torch.maximum(high, old)
            assert ((e >= low) & (e <= high)).all()
            if older:   # earlier codes follow the scale
                kept = torch.arange(block * BLOCK, places.min().item(), device="cuda")
                follow = nearest(want_codes[page, kept].view(E4M3).double() * pow2(old - e)[None, :, None])
                assert torch.equal(codes[page, kept].view(E4M3).double(), follow)
                want_codes[page, kept] = codes[page, kept]
            have = codes[page, places].view(E4M3).double()
            up = pow2(-e)[None, :, None]
            if r.max() == 0:    # nothing is computed before the rounding: the nearest code itself
                assert torch.equal(have[fine], nearest(torch.where(fine, z, 0.0) * up)[fine])
            # half a step: 2^-4 of the value, or 2^-10 where codes are subnormal
            step = torch.maximum(2.0 ** -4 * (z.abs() + r) * up, torch.full_like(z, 2.0 ** -10))
            assert ((have - z * up).abs() <= step + r * up)[fine].all()
            assert have[~fine].isnan().all()
            want_codes[page, places] = codes[page, places]
            want_scale[page, block] = scale[page, block]
        assert torch.equal(codes, want_codes) and torch.equal(scale, want_scale)


@pytest.mark.parametrize("xt", [F32, BF, FP])
@pytest.mark.parametrize("which,qt,wt", [("", BF, F32), ("qk", FP, BF), ("k", BF, FP)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(128, 128), (128, 32), (64, 64), (64, 48), (128, None)])
def test_types_and_rotations(qg, xt, which, qt, wt, interleaved, dim, rot):
    for n_q, kv in (([3, 1, 20], [3, 40, 65]), ([1, 1, 1], [1, 40, 49])):
        c = Case8(n_q, kv, 21, 6, 2, dim, 16, seed=1, spare_tokens=3 if max(n_q) > 1 else 0)
        _check8(qg, c, xt, rot, interleaved, which, wt, qt)


@pytest.mark.parametrize("heads_q,heads_kv", [(1, 1), (64, 8), (32, 32), (28, 4), (71, 1), (128, 16)])
@pytest.mark.parametrize("heads_first", [True, False])
@pytest.mark.parametrize("page", [16, 128])
def test_layouts(qg, heads_q, heads_kv, heads_first, page):
    for n_q in ([1, 5], [1, 1]):
        c = Case8(n_q, [200, 16], 0, heads_q, heads_kv, 128, page, BF, heads_first, seed=2)
        _check8(qg, c, BF, 128)


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 70])
@pytest.mark.parametrize("start", [0, 1, 15, 16, 30])
def test_any_start_in_a_block(qg, n, start):
    c = Case8([n, 1, 0, n], [start + n, 33, 40, start + n + 5], 9, 3, 2, 64, 32, seed=n + start)
    _check8(qg, c, BF, 64, which="qk")


@pytest.mark.parametrize("B", [1, 2, 31, 32, 33, 100, 1100])
def test_batch_sizes_and_empty_sequences(qg, B):
    n_q = [(b * 7) % 4 for b in range(B)]
    n_q[B // 2] = 2
    c = Case8(n_q, [n + (b % 5) for b, n in enumerate(n_q)], 9, 2, 1, 64, 16, seed=B, spare_tokens=4)
    _check8(qg, c, BF, 64)
    n_q = [b % 2 for b in range(B)]   # at most one token a sequence
    n_q[B // 2] = 1
    c = Case8(n_q, [n + (b % 35) for b, n in enumerate(n_q)], 9, 2, 1, 64, 16, seed=B, spare_tokens=1)
    _check8(qg, c, BF, 64)


@pytest.mark.parametrize("used", [0, 1, 5])
def test_fewer_tokens_than_rows(qg, used):
    c = Case8([1] * used or [0], [3] * max(used, 1), 9, 4, 2, 128, 16, seed=40, spare_tokens=300)
    before = c.k_codes.clone()
    if used:
        _check8(qg, c, BF, 128)
    else:
        k = torch.randn((c.T, 2, 128), device="cuda").to(BF)
        qg.qkv_append(c.cache(qg), c.batch(qg), k, k, rope=_rope(20, 128))
        torch.cuda.synchronize()
        assert qg.qgemm_device_status() == 0 and torch.equal(before, c.k_codes)


@pytest.mark.parametrize("n_q", [[3, 2], [1, 1]])
def test_given_positions_without_queries(qg, n_q):
    c = Case8(n_q, [3, 40], 10, 4, 2, 128, 16, seed=4)
    at = torch.tensor([0, 44, 7, 7, 1][:sum(n_q)], dtype=torch.int32, device="cuda")
    _check8(qg, c, BF, 128, positions=at)
    _check8(qg, c, F32, 64, with_q=False)


@pytest.mark.parametrize("magnitude", [1e-30, 1e-18, 1e-5, 1e4, 1e20])
def test_magnitudes(qg, magnitude):
    # below the smallest scale (zeros or subnormal codes), far from 1, up to near the largest scale
    for n_q, kv in (([3, 1, 20], [3, 40, 65]), ([1, 1, 1], [1, 40, 49])):
        c = Case8(n_q, kv, 0, 6, 2, 128, 16, seed=6)
        _check8(qg, c, F32, magnitude=magnitude)


def test_a_block_grows_token_by_token(qg):
    # 20 steps of one token, each 4 times the last, then smaller ones: earlier codes follow the scale, and what is read back
    # is each token within half a step of the block's largest so far
    c = Case8([1, 1], [0, 0], 0, 2, 2, 128, 16, seed=7, poison=False)
    c.table_host = torch.tensor([[0, 1, 2], [3, 4, 5]], dtype=torch.int32)
    codes = torch.zeros((6, 16, 2, 128), dtype=torch.uint8, device="cuda")
    c.k_codes, c.v_codes = codes, codes.clone()
    c.k_scale, c.v_scale = (torch.full((6, 1, 2), 255, dtype=torch.uint8, device="cuda") for _ in range(2))
    c.table = c.table_host.cuda()
    cache, batch = c.cache(qg), c.batch(qg, max_kv=48)
    told = [[], []]
    for i in range(40):
        k = (torch.randn((2, 2, 128), device="cuda") * 2.0 ** (2 * min(i, 39 - i))).to(BF)
        c.kv_len.add_(1)
        qg.qkv_append(cache, batch, k, -k)
        told[0].append(k)
    torch.cuda.synchronize()
    assert qg.qgemm_device_status() == 0
    true = torch.stack(told[0], 1).double()                          # [sequence, place, head, dim]
    for b in range(2):
        v = values(c.k_codes, c.k_scale)[c.table[b].long()].flatten(0, 1)[:40]
        w = values(c.v_codes, c.v_scale)[c.table[b].long()].flatten(0, 1)[:40]
        assert torch.equal(v, -w)
        for first in range(0, 40, BLOCK):
            x, y = true[b, first:first + BLOCK], v[first:first + BLOCK]
            e = c.k_scale[c.table[b, first // BLOCK].item(), 0].int() - 127
            assert torch.equal(e, exponent(x.abs().amax((0, 2))).int())
            # half a step, and where a code became subnormal on the way another half of the steps since: 1/2 + 1/4 + ..
            room = 2.0 ** -4 * x.abs() + 2 * 2.0 ** -10 * pow2(e)[None, :, None]
            assert ((y - x).abs() <= room).all()


def test_not_finite_values(qg):
    def change(k, v):
        k[0, 0, 3], k[2, 1, 5], v[0, 1, 7], v[1, 0, 0] = math.nan, math.inf, -math.inf, math.nan

    for n_q, kv in (([3, 1, 20], [3, 40, 65]), ([1, 1, 1], [1, 40, 49])):
        c = Case8(n_q, kv, 0, 6, 2, 128, 16, seed=8)
        _check8(qg, c, BF, change=change)


# ------------------------------------------------------------------ reading back
@pytest.mark.parametrize("dtype", [F32, BF, FP])
@pytest.mark.parametrize("heads_kv,dim,page,heads_first", [(2, 128, 16, True), (8, 128, 64, False), (1, 64, 256, True), (33, 64, 32, True)])
def test_read(qg, dtype, heads_kv, dim, page, heads_first):
    for n_q, kv in (([3, 1, 20, 0], [3, 40, 65, 7]), ([1, 1, 1], [1, 40, 49]), ([33, 200, 16], [33, 200, 16])):
        c = Case8(n_q, kv, 21, heads_kv, heads_kv, dim, page, BF, heads_first, seed=dim + page, spare_tokens=2 if max(n_q) > 1 else 0)
        wide = [torch.full((c.T, heads_kv + 1, dim), 7.0, dtype=dtype, device="cuda") for _ in range(2)]
        k, v = (w[:, :heads_kv] for w in wide)
        got = qg.qkv_read(c.cache(qg), c.batch(qg), k_out=k, v_out=v)
        torch.cuda.synchronize()
        assert qg.qgemm_device_status() == 0 and got[0] is k and got[1] is v
        where, used = _where(c), c.cu[-1]
        page_at, place = (torch.tensor([w[i] for w in where], device="cuda") for i in (2, 3))
        assert torch.equal(k[:used], c.k[page_at, place].to(dtype)) and torch.equal(v[:used], c.v[page_at, place].to(dtype))
        for w in wide:
            assert (w[used:] == 7.0).all() and (w[:, heads_kv:] == 7.0).all()
    k, v = qg.qkv_read(c.cache(qg), c.batch(qg))
    assert k.dtype == v.dtype == BF


def test_read_the_prefix(qg):
    # as a sequence over its own pages
    c = Case8([1], [5], 150, 2, 2, 128, 32, seed=12)
    batch = qg.KVBatch(c.prefix_table.view(1, -1), torch.tensor([150], dtype=torch.int32, device="cuda"), max_kv=150,
                       cu_q=torch.tensor([0, 150], dtype=torch.int32, device="cuda"), max_q=150, tokens=150)
    k, v = qg.qkv_read(c.cache(qg), batch, dtype=F32)
    for got, x in ((k, c.k), (v, c.v)):
        assert torch.equal(got.double(), x[c.prefix_table.long()].flatten(0, 1)[:150])


# ------------------------------------------------------------------ together
@pytest.mark.parametrize("n_q,kv,prefix", [([1, 1, 1], [18, 40, 65], 300), ([4, 1, 20], [18, 40, 65], 0), ([130], [190], 40)])
def test_append_then_attend(qg, n_q, kv, prefix):
    """The calls as a step uses them: normed and turned, quantised, and what was appended is what the attention sees."""
    c = Case8(n_q, kv, prefix, 16, 2, 128, 16, seed=8)
    q, k, v = _inputs(c, BF)
    qw, kw = _norms(c, BF, "qk")
    cache, batch = c.cache(qg), c.batch(qg)
    c.q = qg.qkv_append(cache, batch, k, v, q=q, rope=_rope(prefix + max(kv), 128), q_norm=qw, k_norm=kw)
    out = qg.qattn_forward(c.q, cache, batch)
    torch.cuda.synchronize()
    c.refresh()
    check_attention(c, out)


def test_steps_captured_in_a_graph(qg):
    """Append, attention and reading back in one graph, replayed with new lengths."""
    c = Case8([1, 1], [10, 30], 40, 8, 2, 128, 16, seed=9, poison=False)
    q, k, v = _inputs(c, BF)
    cache, batch = c.cache(qg), c.batch(qg, max_kv=c.table.shape[1] * 16)
    ws = torch.empty(qg.qattn_workspace_size(cache, batch, 8), dtype=torch.uint8, device="cuda")
    q_out, out = torch.empty_like(q, memory_format=torch.contiguous_format), torch.empty((2, 8, 128), dtype=BF, device="cuda")
    back = [torch.empty((2, 2, 128), dtype=BF, device="cuda") for _ in range(2)]
    rope = _rope(100, 128)

    def step():
        qg.qkv_append(cache, batch, k, v, q=q, rope=rope, q_out=q_out)
        qg.qattn_forward(q_out, cache, batch, out=out, workspace=ws)
        qg.qkv_read(cache, batch, k_out=back[0], v_out=back[1])

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            step()
    for kv in ([10, 30], [11, 31], [12, 32]):
        c.kv = kv
        c.kv_len.copy_(torch.tensor(kv, dtype=torch.int32))
        fresh = torch.randn((2, 12 * 128), device="cuda").to(BF)
        for t, at in ((q, 0), (k, 8), (v, 10)):
            t.copy_(fresh[:, at * 128:(at + t.shape[1]) * 128].unflatten(1, (-1, 128)))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert qg.qgemm_device_status() == 0
        c.refresh()
        c.q = q_out
        check_attention(c, out)
        for got, x in ((back[0], c.k), (back[1], c.v)):
            want = torch.stack([x[c.table[b, (kv[b] - 1) // 16].item(), (kv[b] - 1) % 16] for b in range(2)])
            assert torch.equal(got, want.to(BF))


def test_dependent_launch_off_and_other_streams_give_the_same(qg):
    for n_q, kv in (([3, 1, 20], [3, 40, 65]), ([1, 1, 1], [1, 40, 49])):
        results = []
        for way in range(3):
            c = Case8(n_q, kv, 21, 6, 2, 128, 16, seed=10)
            q, k, v = _inputs(c, BF)
            s = torch.cuda.Stream() if way == 2 else None
            if s:
                s.wait_stream(torch.cuda.current_stream())
            qg.qgemm_set_dependent_launch(way != 1)
            try:
                out = qg.qkv_append(c.cache(qg), c.batch(qg), k, v, q=q, stream=s)
                back = qg.qkv_read(c.cache(qg), c.batch(qg), stream=s)
            finally:
                qg.qgemm_set_dependent_launch(True)
            torch.cuda.synchronize()
            results.append((out, *back, c.k_codes, c.v_codes, c.k_scale, c.v_scale))
        for other in results[1:]:
            assert all(torch.equal(a, b) for a, b in zip(results[0], other))


# ------------------------------------------------------------------ outside the bounds
@pytest.mark.parametrize("heads_first", [True, False])
@pytest.mark.parametrize("n_q", [[2, 1, 1], [1, 1, 1]])
def test_lengths_outside_their_bounds_leave_the_cache_alone(qg, heads_first, n_q):
    # the sequence's codes and scales so far are still there; other sequences are written
    assert qg.qgemm_device_status(reset=True) == 0
    kv = [40, 20, 33]

    def check(written, spoil=None, **bounds):
        a, b = (Case8(n_q, kv, 0, 4, 2, 128, 16, BF, heads_first, seed=10) for _ in range(2))
        q, k, v = _inputs(a, BF)
        qg.qkv_append(b.cache(qg), b.batch(qg), k, v, q=q)
        assert qg.qgemm_device_status(reset=True) == 0
        was = {n: getattr(a, n).clone() for n in ("k_codes", "v_codes", "k_scale", "v_scale")}
        if spoil:
            spoil(a)
        qg.qkv_append(a.cache(qg), a.batch(qg, **bounds), k, v, q=q)
        assert qg.qgemm_device_status(reset=True) == -7
        for s in range(3):
            pages = a.table_host[s, :-(-kv[s] // 16)].long().cuda()
            for n, x in was.items():
                assert torch.equal(getattr(a, n)[pages], getattr(b if s in written else None, n)[pages] if s in written else x[pages])

    check([1, 2], max_kv=39)          # sequence 0 is longer than its bound
    check([1], max_kv=32)             # and sequence 2
    if n_q[0] > 1:
        check([1, 2], max_q=1)        # sequence 0 has more new tokens than its bound

    def length(bad):
        def f(c):
            c.kv_len[1] = bad
        return f

    for bad in (-1, -(1 << 31), 1 << 30, 0x7FFFFFFF):
        check([0, 2], length(bad))

    def page(c):
        c.table[2, 2] = 1 << 20       # the page its new token belongs to

    check([0, 1], page)

    def offsets(c):
        c.cu_q[3] = c.T + 1

    check([0, 1], offsets)


def test_offsets_in_no_order_write_nothing_outside(qg):
    # offsets that go up and down, and past the rows: reported, and nothing is written but places of the sequences' pages
    assert qg.qgemm_device_status(reset=True) == 0
    c = Case8([40, 30, 20, 10], [70, 60, 50, 40], 0, 4, 2, 64, 16, seed=13, spare_tokens=100)
    q, k, v = _inputs(c, BF)
    for bad in ([0, 200, 0, 200, 100], [50, 10, 50, 10, 50], [-5, 3, 1 << 30, -(1 << 31), 0x7FFFFFFF], [200, 200, 200, 200, 0]):
        c.cu_q.copy_(torch.tensor(bad, dtype=torch.int32))
        qg.qkv_append(c.cache(qg), c.batch(qg), k, v, q=q)
        qg.qkv_read(c.cache(qg), c.batch(qg))
        assert qg.qgemm_device_status(reset=True) == -7
    unused = sorted(set(range(c.k_codes.shape[0])) - set(c.table_host[c.table_host < c.k_codes.shape[0]].tolist()))
    assert (c.k_codes[unused] == 0x7F).all()


def test_positions_and_places_outside_are_reported(qg):
    assert qg.qgemm_device_status(reset=True) == 0
    c = Case8([2, 1], [1, 20], 0, 4, 2, 128, 16, seed=6)   # sequence 0: the first token has no place
    k = torch.randn((3, 2, 128), device="cuda").to(BF)
    qg.qkv_append(c.cache(qg), c.batch(qg), k, k)
    assert qg.qgemm_device_status(reset=True) == -7
    c.refresh()
    p0, p1 = c.table_host[0, 0].item(), c.table_host[1, 1].item()
    assert (c.k[p0, 0] - k[1].double()).abs().max() < 0.3 and (c.k[p1, 3] - k[2].double()).abs().max() < 0.3
    # a position past the rotation table: the token is not written
    for n_q in ([1, 1], [3, 1]):
        c = Case8(n_q, [5, 20], 0, 4, 2, 128, 16, seed=7)
        before = c.k_codes.clone()
        qg.qkv_append(c.cache(qg), c.batch(qg), k[:1].expand(c.T, -1, -1).contiguous(), k[:1].expand(c.T, -1, -1).contiguous(),
                      rope=_rope(10, 128))
        assert qg.qgemm_device_status(reset=True) == -7
        assert torch.equal(before[c.table_host[1, 1].item()], c.k_codes[c.table_host[1, 1].item()])
    # reading a place that is not there leaves the row
    c = Case8([2, 1], [1, 20], 0, 4, 2, 128, 16, seed=6)
    out = torch.full((3, 2, 128), 7.0, dtype=BF, device="cuda")
    qg.qkv_read(c.cache(qg), c.batch(qg), k_out=out)
    assert qg.qgemm_device_status(reset=True) == -7
    assert (out[0] == 7.0).all() and torch.equal(out[1], c.k[c.table_host[0, 0].item(), 0].to(BF))


def test_refusals(qg):
    c = Case8([1, 1], [5, 20], 0, 4, 2, 128, 16, seed=9)
    cache, batch = c.cache(qg), c.batch(qg)
    k = torch.zeros((2, 2, 128), dtype=BF, device="cuda")
    q = torch.zeros((2, 4, 128), dtype=BF, device="cuda")
    w = torch.ones(128, device="cuda")
    with pytest.raises(ValueError):
        qg.qkv_append(cache, batch, k, k.half())
    with pytest.raises(ValueError):
        qg.qkv_append(cache, batch, k, k, q=q, q_dtype=F32)
    with pytest.raises(ValueError):
        qg.qkv_append(cache, batch, k, k, q=q, q_out=q.float())
    with pytest.raises(ValueError):
        qg.qkv_append(cache, batch, k, k, q_norm=w)                       # q_norm without q
    with pytest.raises(ValueError):
        qg.qkv_append(cache, batch, k, k, q=q, q_norm=w, k_norm=w.half())
    for bad in (w[:64], w.cpu(), w.double(), torch.ones(256, device="cuda")[::2]):
        with pytest.raises(ValueError):
            qg.qkv_append(cache, batch, k, k, k_norm=bad)
    for eps in (-1e-6, math.inf, math.nan):
        with pytest.raises(qg.QgError) as e:
            qg.qkv_append(cache, batch, k, k, k_norm=w, eps=eps)
        assert e.value.status == -1
    with pytest.raises(qg.QgError) as e:
        qg.qkv_append(cache, batch, k, k, k_norm=torch.ones(129, device="cuda")[1:])
    assert e.value.status == -3
    d = Case([1, 1], [5, 20], 0, 4, 2, 128, 16, BF, seed=9)
    with pytest.raises(ValueError):
        qg.qkv_append(d.cache(qg), d.batch(qg), k, k, q=q, q_dtype=FP)    # a 16-bit cache's queries have its type
    with pytest.raises(ValueError):
        qg.qkv_read(d.cache(qg), d.batch(qg))
    with pytest.raises(ValueError):
        qg.qkv_read(cache, batch, k_out=torch.empty((2, 2, 128), dtype=BF, device="cuda"), v_out=torch.empty((2, 2, 128), device="cuda"))
    with pytest.raises(ValueError):
        qg.qkv_read(cache, batch, k_out=torch.empty((3, 2, 128), dtype=BF, device="cuda"))
