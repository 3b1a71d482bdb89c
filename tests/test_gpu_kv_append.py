"""GPU: keys normed and rotated on their way into the paged cache, values beside them, queries in
the same launch, against a 64-bit evaluation."""
import math

import pytest
import torch

import attn_ref
import gated_deltanet_linear_prefill_amd as gdn
import rope_ref
from test_gpu_kv_cache import BF, DEV, F8, F32, Cache, ints, offsets, same, values
from test_gpu_qk_norm_rope import freqs, per_pair, positions, rows, weights

pytestmark = pytest.mark.gpu


def check_cache(cache, pool, scale, before, where, want, bound):
    """Rows that were written against want [total, h, d] (64 bits) and its error bound; all others as before."""
    got = values(cache, pool, scale)
    for i, at in enumerate(where):
        if at is None:
            continue
        x, w, b = got[at[0], :, at[1]], want[i], bound[i]
        nan = torch.isnan(w)
        if cache.store == F8:
            # half a step of e4m3, 2^-4 of the value; below the smallest normal code half of 2^-9 units, of
            # a scale that is the next one where the row's largest is within its error of the border
            unit = torch.exp2((scale[at[0], :, at[1]].cpu().double() - 127))[:, None]
            tol = b + 2.0 ** -4 * (w.abs() + b) + 2.0 ** -10 * unit
            top = torch.where(torch.isfinite(w), w.abs(), 0.0).amax(-1, keepdim=True)
            assert bool((top <= 448 * unit * (1 + 2.0 ** -18)).all()) and bool(((top > 224 * unit * (1 - 2.0 ** -18)) | (top == 0)).all())
        else:
            tol = b + torch.finfo(cache.store).eps / 2 * w.abs() + 2.0 ** -126
        assert torch.equal(torch.isnan(x), nan), i
        assert bool(((x - w).abs() <= tol)[~nan].all()), (i, ((x - w).abs() / tol)[~nan].max())
        before[at[0], :, at[1]] = x
    assert same(got, before)


def run(n, lens, start, hq, h, d, page, rot, axes, inter, norm, dtype, store, given=False, first=0, behind=0, cache=None, scale=1.0):
    """`first` and `behind`: rows before and after the sequences', which belong to none."""
    cache = cache or Cache([max(a + b, 1) for a, b in zip(start, lens)], page, h, d, store, seed=n)
    total = first + sum(lens) + behind
    k, v, q = rows(total, h, d, dtype, 1), rows(total, h, d, dtype, 2), rows(total, hq, d, dtype, 3) if hq else None
    freq = freqs(rot) if rot else None
    axis = (torch.arange(rot // 2) % axes).to(torch.uint8) if rot and axes > 1 else None
    place = torch.zeros(1, total, dtype=torch.int32)
    where, mine = [None] * total, [False] * total
    at = first
    for s in range(n):
        for i in range(lens[s]):
            where[at], mine[at], place[0, at] = cache.place(s, start[s] + i), True, start[s] + i
            at += 1
    pos = positions(axes, total, 5) if axes > 1 or given else None
    wk = weights(d, dtype, 6) if norm else None
    wq = weights(d, dtype, 7) if norm and hq else None
    before_k, before_v = values(cache, cache.k, cache.ks).clone(), values(cache, cache.v, cache.vs).clone()
    q_out = torch.full(q.shape, 7.0, dtype=dtype, device=DEV) if hq else None
    dv = lambda x: None if x is None else x.to(DEV)
    cu = [first + x for x in offsets(lens)]
    got = gdn.gdn_kv_append(k.to(DEV), v.to(DEV), *cache.args(), ints(start), ints(cu), positions=dv(pos if axes > 1 else pos[0] if given else None) if rot else None,
                            freq=dv(freq), axis=dv(axis), interleaved=inter, rope_scale=scale, k_weight=dv(wk), q=dv(q), q_weight=dv(wq),
                            weight_bias=1.0, q_out=q_out, **cache.scales())
    pp = per_pair(place if pos is None else pos, axis, rot // 2) if rot else None
    want, bound = rope_ref.norm_rope(k, wk, 1.0, 1e-6, freq, pp, inter, scale)
    check_cache(cache, cache.k, cache.ks, before_k, where, want, bound)
    check_cache(cache, cache.v, cache.vs, before_v, where, v.double(), torch.zeros(v.shape, dtype=torch.float64))
    if hq:
        assert got is q_out
        m = torch.tensor(mine)
        want, bound = rope_ref.norm_rope(q, wq, 1.0, 1e-6, freq, pp, inter, scale)
        rope_ref.check(got.cpu()[m], want[m], bound[m], "q")
        assert bool((got.cpu()[~m] == 7.0).all())
    else:
        assert got is None
    return cache


CASES = [  # n, lens, start, h_q, h_kv, d, page, rot, axes, interleaved, norm, dtype, store
    (1, [1], [0], 16, 2, 256, 64, 64, 1, False, True, BF, F8), (3, [1, 7, 40], [5, 0, 31], 0, 3, 64, 16, 64, 1, False, False, BF, BF),
    (2, [33, 2], [15, 16], 2, 1, 128, 32, 48, 1, True, True, F32, F32), (4, [0, 5, 0, 17], [3, 64, 9, 1], 4, 2, 128, 64, 128, 3, False, True, F32, F8),
    (2, [100, 64], [0, 1000], 8, 8, 128, 1024, 112, 2, True, True, BF, F8), (3, [16, 16, 1], [16, 48, 0], 5, 5, 256, 16, 256, 1, False, True, BF, BF),
    (2, [9, 4], [0, 3], 3, 1, 64, 16, 0, 1, False, True, BF, F8), (5, [1, 1, 1, 1, 1], [4000, 0, 16, 31, 77], 20, 1, 64, 16, 16, 1, False, False, BF, BF),
    (1, [2500], [100000], 2, 1, 64, 16, 32, 1, False, True, BF, F8),
]


@pytest.mark.parametrize("n,lens,start,hq,h,d,page,rot,axes,inter,norm,dtype,store", CASES)
def test_against_64_bits(n, lens, start, hq, h, d, page, rot, axes, inter, norm, dtype, store):
    run(n, lens, start, hq, h, d, page, rot, axes, inter, norm, dtype, store)


@pytest.mark.parametrize("store", [BF, F8])
def test_given_positions_and_rows_of_nobody(store):
    run(2, [30, 17], [10, 3], 4, 2, 64, 16, 32, 1, False, True, BF, store, given=True, first=4, behind=6, scale=1.5)


def test_places_that_are_not_there():
    """Keys and values of absent pages and of positions outside the table are dropped; queries are not."""
    cache = Cache([40, 20], 16, 2, 64, BF, extra_width=0)
    cache.page_table[0, 1] = -1
    cache.page_table[1, 0] = cache.pages + 5
    cache.table[0][1], cache.table[1][0] = -1, -1
    run(2, [30, 40], [10, -3], 4, 2, 64, 16, 32, 1, False, True, BF, BF, cache=cache, first=2, behind=3)


def test_one_token_each_without_offsets():
    n, h, d = 9, 2, 128
    start = [0, 1, 15, 16, 17, 40, 2, 31, 32]
    a, b = (Cache([x + 1 for x in start], 16, h, d, F8) for _ in range(2))
    k, v, q = rows(n, h, d, BF, 1).to(DEV), rows(n, h, d, BF, 2).to(DEV), rows(n, 4, d, BF, 3).to(DEV)
    w, f = weights(d, BF, 4).to(DEV), freqs(64).to(DEV)
    kw = dict(freq=f, k_weight=w, q=q, q_weight=w, weight_bias=1.0)
    qa = gdn.gdn_kv_append(k, v, *a.args(), ints(start), None, **kw, **a.scales())
    qb = gdn.gdn_kv_append(k, v, *b.args(), ints(start), ints(list(range(n + 1))), **kw, **b.scales())
    assert torch.equal(qa, qb)
    for x, y in ((a.k, b.k), (a.v, b.v)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert torch.equal(a.ks, b.ks) and torch.equal(a.vs, b.vs)


@pytest.mark.parametrize("dtype,store", [(BF, BF), (F32, F32), (BF, F8), (F32, F8)])
def test_without_norm_and_rotation_it_is_a_write(dtype, store):
    """The same bytes as gdn_kv_write, NaN and infinities among the rows."""
    lens, start, h, d = [20, 1, 9], [3, 0, 40], 2, 128
    a, b = (Cache([x + y for x, y in zip(lens, start)], 16, h, d, store) for _ in range(2))
    k, v = rows(30, h, d, dtype, 1), rows(30, h, d, dtype, 2)
    k[3, 1, 7], v[4, 0, 100], k[9, 0, 0] = math.nan, math.inf, -math.inf
    k, v, cu = k.to(DEV), v.to(DEV), ints(offsets(lens))
    gdn.gdn_kv_append(k, v, *a.args(), ints(start), cu, **a.scales())
    gdn.gdn_kv_write(k, v, *b.args(), ints(start), cu, **b.scales())
    for x, y in ((a.k, b.k), (a.v, b.v)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    if store == F8:
        assert torch.equal(a.ks, b.ks) and torch.equal(a.vs, b.vs)


def test_the_same_rows_as_the_packed_call():
    """What goes into a cache of the rows' type is what gdn_qk_norm_rope gives, bit for bit."""
    lens, start, h, d = [40, 3], [100, 0], 2, 256
    cache = Cache([x + y for x, y in zip(lens, start)], 64, h, d, BF)
    k, v, q = rows(43, h, d, BF, 1).to(DEV), rows(43, h, d, BF, 2).to(DEV), rows(43, 16, d, BF, 3).to(DEV)
    pos = torch.cat([torch.arange(100, 140), torch.arange(3)]).to(torch.int32).to(DEV)
    w, f, cu = weights(d, BF, 4).to(DEV), freqs(64).to(DEV), ints(offsets(lens))
    qo = gdn.gdn_kv_append(k, v, *cache.args(), ints(start), cu, freq=f, k_weight=w, q=q, q_weight=w, weight_bias=1.0)
    qp, kp = gdn.gdn_qk_norm_rope(q, k, pos, freq=f, q_weight=w, k_weight=w, weight_bias=1.0)
    kc, vc = gdn.gdn_kv_read(*cache.args(), ints(start), cu, 43)
    assert torch.equal(qo, qp) and torch.equal(kc, kp) and torch.equal(vc, v)


def test_strided_slices_of_a_projection():
    n, lens, start, hq, h, d = 2, [9, 20], [3, 0], 4, 2, 64
    f = rows(29, hq + 2 * h, d, BF, 1).to(DEV)
    a, b = (Cache([x + y for x, y in zip(lens, start)], 16, h, d, F8) for _ in range(2))
    w, fr, cu = weights(d, BF, 4).to(DEV), freqs(32).to(DEV), ints(offsets(lens))
    parts = [f[:, :hq], f[:, hq:hq + h], f[:, hq + h:]]
    out = []
    for c, (q, k, v) in ((a, parts), (b, [x.contiguous() for x in parts])):
        out.append(gdn.gdn_kv_append(k, v, *c.args(), ints(start), cu, freq=fr, k_weight=w, q=q, q_weight=w, **c.scales()))
    assert torch.equal(out[0], out[1]) and torch.equal(a.k.view(torch.uint8), b.k.view(torch.uint8))
    assert torch.equal(a.v.view(torch.uint8), b.v.view(torch.uint8)) and torch.equal(a.ks, b.ks)


def test_captured_and_replayed():
    """A decode step's append in a graph, its starts moved on between replays."""
    n, h, d = 5, 2, 128
    cache, ref = (Cache([40] * n, 16, h, d, F8) for _ in range(2))
    k, v, q = rows(n, h, d, BF, 1).to(DEV), rows(n, h, d, BF, 2).to(DEV), rows(n, 4, d, BF, 3).to(DEV)
    w, f, start = weights(d, BF, 4).to(DEV), freqs(64).to(DEV), ints([0, 3, 9, 14, 15])
    qo = torch.empty_like(q)
    call = lambda c, out: gdn.gdn_kv_append(k, v, *c.args(), start, None, freq=f, k_weight=w, q=q, q_weight=w, q_out=out, **c.scales())
    call(cache, qo)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call(cache, qo)
    call(ref, torch.empty_like(q))
    for i in range(4):
        k.mul_(1.25)
        start.add_(1)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(call(ref, None), qo), i
        assert torch.equal(cache.k.view(torch.uint8), ref.k.view(torch.uint8)) and torch.equal(cache.ks, ref.ks), i


def test_offsets_past_32_bits():
    """The last page of a pool of more than 4 GiB."""
    h, d, page = 8, 256, 64
    pages = (1 << 32) // (h * page * d * 2) + 40
    k, v = (torch.empty(pages, h, page, d, dtype=BF, device=DEV) for _ in range(2))
    for x in (k, v):
        x[0], x[-1] = 3.0, 3.0
    a, b = rows(20, h, d, BF, 9).to(DEV), rows(20, h, d, BF, 10).to(DEV)
    f = freqs(64).to(DEV)
    gdn.gdn_kv_append(a, b, k, v, ints([[pages - 1]]), ints([30]), ints([0, 20]), freq=f)
    want = gdn.gdn_qk_norm_rope(a, None, torch.arange(30, 50, dtype=torch.int32, device=DEV), freq=f)[0]
    assert torch.equal(k[-1, :, 30:50].transpose(0, 1), want) and bool((k[0] == 3.0).all())
    assert torch.equal(v[-1, :, 30:50].transpose(0, 1), b) and bool((k[-1, :, :30] == 3.0).all())


def test_refusals():
    cache = Cache([20], 16, 2, 64, BF)
    k = rows(20, 2, 64, BF, 1).to(DEV)
    cu, st, f, w = ints([0, 20]), ints([0]), freqs(32).to(DEV), weights(64, BF, 1).to(DEV)
    before = cache.k.clone()
    bad = [dict(k=k[:, :1]), dict(q=k.float()), dict(q=k[:19]), dict(start=st.long()), dict(cu_seqlens=cu[:1]), dict(freq=f.double()),
           dict(positions=ints([0] * 19)), dict(k_weight=w.float()), dict(q_out=k), dict(q_weight=w[:32]), dict(axis=f), dict(freq=None, positions=ints([0] * 20))]
    for over in bad:
        a = dict(k=k, v=k, k_cache=cache.k, v_cache=cache.v, page_table=cache.page_table, start=st, cu_seqlens=cu, freq=f)
        a.update(over)
        with pytest.raises(ValueError):
            gdn.gdn_kv_append(**a)
    for over, status in ((dict(k=cache.k.view(-1, 2, 64)[:20]), 5), (dict(q=k, q_out=k), 5), (dict(q=k, q_out=cache.v.view(-1, 2, 64)[:20]), 5),
                         (dict(positions=torch.zeros(5, 20, dtype=torch.int32, device=DEV)), 2), (dict(freq=freqs(24).to(DEV)), 2)):
        a = dict(k=k, v=k, k_cache=cache.k, v_cache=cache.v, page_table=cache.page_table, start=st, cu_seqlens=cu, freq=f)
        a.update(over)
        with pytest.raises(gdn.GdnError) as e:
            gdn.gdn_kv_append(**a)
        assert e.value.status == status
    torch.cuda.synchronize()
    assert torch.equal(cache.k, before)
