"""GPU: attention of one new token over the paged cache against a 64-bit evaluation
(tests/attn_ref.py)."""
import math

import pytest
import torch

import attn_ref
import gated_deltanet_linear_prefill_amd as gdn
from test_gpu_kv_cache import BF, DEV, F8, F32, Cache, ints, values

pytestmark = pytest.mark.gpu


def fill(cache, seed, nan_behind=None):
    """Random rows in every page; with nan_behind (lengths), the rows past each length are NaN."""
    g = torch.Generator().manual_seed(seed)
    for name in ("k", "v"):
        pool = getattr(cache, name)
        x = torch.randn(pool.shape, generator=g)
        if cache.store == F8:
            x = (x * 40).clamp(-448, 448).to(F8)
            getattr(cache, name + "s").copy_(torch.randint(118, 124, pool.shape[:3], generator=g).to(torch.uint8))
        pool.view(torch.uint8).copy_(x.to(cache.store).view(torch.uint8)) if cache.store == F8 else pool.copy_(x)
    if nan_behind is not None:
        code = 0x7f if cache.store == F8 else None
        for s, length in enumerate(nan_behind):
            for pos in range(length, len(cache.table[s]) * cache.page):
                at = cache.place(s, pos)
                if at is None:
                    continue
                for name in ("k", "v"):
                    pool = getattr(cache, name)
                    if code is not None:
                        pool.view(torch.uint8)[at[0], :, at[1]] = code
                        getattr(cache, name + "s")[at[0], :, at[1]] = 255
                    else:
                        pool[at[0], :, at[1]] = math.nan


def dense(cache, s, length):
    """[length, h, d] K and V of a sequence, and which of its positions are on pages that exist."""
    k, v = values(cache, cache.k, cache.ks), values(cache, cache.v, cache.vs)
    at = [cache.place(s, p) for p in range(length)]
    there = torch.tensor([x is not None for x in at], dtype=torch.bool)
    pick = lambda x: torch.stack([x[a[0], :, a[1]] if a else torch.zeros(cache.h, cache.d).double() for a in at]) \
        if length else torch.zeros(0, cache.h, cache.d).double()
    return pick(k), pick(v), there


def compare(cache, q, lens, out, lse, scale):
    g = q.shape[1] // cache.h
    for s, length in enumerate(lens):
        k, v, there = dense(cache, s, max(length, 0))
        for h in range(q.shape[1]):
            ref = attn_ref.attend(q[s:s + 1, h], k[:, h // g], v[:, h // g], scale, there[None])
            attn_ref.check(out[s:s + 1, h], None if lse is None else lse[s:s + 1, h], *ref, what=f"sequence {s} head {h}")


def queries(n, hq, d, dtype, seed=1):
    return (1.5 * torch.randn(n, hq, d, generator=torch.Generator().manual_seed(seed))).to(dtype)


CASES = [
    ([1], 1, 1, 64, 16, BF, BF), ([333], 16, 2, 256, 64, BF, BF), ([17, 1, 0, 200, 31, 32, 33], 8, 2, 128, 16, BF, BF),
    ([500, 3], 6, 2, 64, 32, BF, F8), ([129, 128, 127], 16, 1, 256, 128, BF, F8), ([64, 65], 20, 1, 64, 16, BF, F8),
    ([90, 2], 4, 4, 64, 16, F32, F32), ([40], 33, 1, 128, 16, F32, F8), ([70, 7], 6, 3, 256, 64, F32, F32),
    ([300], 2, 1, 256, 1024, F32, F8), ([5000, 100], 3, 1, 128, 64, BF, BF), ([2500], 17, 1, 64, 16, BF, BF),
]


@pytest.mark.parametrize("lens,hq,hk,d,page,dtype,store", CASES)
def test_against_64_bits(lens, hq, hk, d, page, dtype, store):
    cache = Cache(lens, page, hk, d, store)
    fill(cache, 5, nan_behind=lens)
    q = queries(len(lens), hq, d, dtype)
    lse = torch.full(q.shape[:2], 5.0, device=DEV)
    out = gdn.gdn_attn_decode(q.to(DEV), *cache.args(), ints(lens), lse=lse, **cache.scales())
    compare(cache, q, lens, out, lse, d ** -0.5)


@pytest.mark.parametrize("store,dtype", [(BF, BF), (F8, BF), (F32, F32)])
def test_absent_pages_and_bounds(store, dtype):
    """Pages that are not there are skipped, whole ranges of them too; lengths past the table or
    past max_len are cut, negative ones are empty."""
    lens, page = [400, 300, 700, 100], 16
    cache = Cache(lens, page, 2, 64, store, extra_width=0)
    fill(cache, 6)
    for s, gone in ((0, [0, 3, 24]), (1, list(range(len(cache.table[1])))), (2, list(range(8, 30)))):
        for x in gone:
            if x < len(cache.table[s]) and cache.table[s][x] >= 0:
                cache.table[s][x] = -1
                cache.page_table[s, x] = -1 if x % 2 else cache.pages + 1
    q = queries(4, 4, 64, dtype)
    lse = torch.zeros(4, 4, device=DEV)
    width = cache.page_table.shape[1] * page
    out = gdn.gdn_attn_decode(q.to(DEV), *cache.args(), ints([400, 300, 10 ** 6, -5]), lse=lse, **cache.scales())
    compare(cache, q, [400, 300, width, 0], out, lse, 64 ** -0.5)
    out = gdn.gdn_attn_decode(q.to(DEV), *cache.args(), ints([400, 300, 10 ** 6, 100]), max_len=130, lse=lse, **cache.scales())
    compare(cache, q, [130, 130, 130, 100], out, lse, 64 ** -0.5)
    out = gdn.gdn_attn_decode(q.to(DEV), *cache.args(), ints(lens), max_len=0, lse=lse, **cache.scales())
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_strided_queries_scale_and_used_workspace():
    lens = [260, 31]
    cache = Cache(lens, 32, 2, 128, BF)
    fill(cache, 7)
    f = torch.randn(2, 12, 128, dtype=BF, generator=torch.Generator().manual_seed(2))
    q = f[:, 4:8]
    need = gdn.gdn_attn_decode_workspace_bytes(2, cache.page_table.shape[1], 32, 4, 2, 128, 260)
    ws = torch.full((need + 64,), 0xff, dtype=torch.uint8, device=DEV)
    out = gdn.gdn_attn_decode(f.to(DEV)[:, 4:8], *cache.args(), ints(lens), max_len=260, scale=0.5, workspace=ws)
    compare(cache, q, lens, out, None, 0.5)
    assert bool((ws[need:] == 0xff).all())


def test_large_scores():
    lens = [600]
    cache = Cache(lens, 16, 1, 64, BF)
    fill(cache, 8)
    at = cache.place(0, 555)
    cache.k[at[0], :, at[1]] *= 30
    q = queries(1, 4, 64, BF) * 6
    out = gdn.gdn_attn_decode(q.to(DEV), *cache.args(), ints(lens))
    compare(cache, q, lens, out, None, 64 ** -0.5)


def test_bad_values_that_are_seen_reach_the_output():
    lens = [50]
    cache = Cache(lens, 16, 1, 64, BF)
    fill(cache, 9)
    at = cache.place(0, 20)
    cache.v[at[0], 0, at[1], 5] = math.inf
    q = queries(1, 2, 64, BF)
    out = gdn.gdn_attn_decode(q.to(DEV), *cache.args(), ints(lens))
    compare(cache, q, lens, out, None, 64 ** -0.5)
    assert bool(torch.isinf(out[0, :, 5].float()).all())


def test_offsets_past_32_bits():
    h, d, page = 8, 256, 64
    pages = (1 << 32) // (h * page * d * 2) + 8
    g = torch.Generator().manual_seed(3)
    k, v = (torch.empty(pages, h, page, d, dtype=BF, device=DEV) for _ in range(2))
    kk, vv = (torch.randn(2, h, page, d, generator=g).to(BF) for _ in range(2))
    k[-2:], v[-2:] = kk.to(DEV), vv.to(DEV)
    q = queries(1, 16, d, BF)
    out = gdn.gdn_attn_decode(q.to(DEV), k, v, ints([[pages - 1, pages - 2]]), ints([100]))
    for x in range(16):
        row = lambda t: torch.cat([t[1, x // 2], t[0, x // 2]])[:100]
        ref = attn_ref.attend(q[:, x], row(kk), row(vv), d ** -0.5, torch.ones(1, 100, dtype=torch.bool))
        attn_ref.check(out[:, x], None, *ref, what=f"head {x}")


def test_the_same_twice_and_in_a_graph():
    """Eager runs agree bit for bit, and so does every replay of a captured call, with other
    work between the replays and the inputs changed in place."""
    lens = [3000, 100, 7]
    cache = Cache(lens, 64, 2, 128, F8)
    fill(cache, 10)
    q = queries(3, 16, 128, BF).to(DEV)
    ln = ints(lens)
    out = torch.empty_like(q)
    need = gdn.gdn_attn_decode_workspace_bytes(3, cache.page_table.shape[1], 64, 16, 2, 128, 3000, store=F8)
    ws = torch.empty(max(need, 1), dtype=torch.uint8, device=DEV)
    call = lambda o: gdn.gdn_attn_decode(q, *cache.args(), ln, max_len=3000, out=o, workspace=ws, **cache.scales())
    call(out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call(out)
    for step in range(4):
        q.mul_(1.0 + 0.1 * step)
        ln[1] = 100 + step
        want = torch.empty_like(q)
        call(want)
        torch.cuda.synchronize()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), step


def test_memory_of_a_call_on_another_stream():
    """With stream=, the outputs and workspace that a call makes are that stream's: what the current
    stream allocates and writes while the call waits there does not reach them, and the call
    does not write what the current stream has freed and still reads."""
    lens = [3000, 2000]
    cache = Cache(lens, 64, 2, 128, BF)
    fill(cache, 12)
    q = queries(2, 16, 128, BF).to(DEV)
    ln, start, cu = ints(lens), ints([0, 0]), ints([0, 3000, 5000])
    want = gdn.gdn_attn_decode(q, *cache.args(), ln, max_len=3000)
    wk, wv = gdn.gdn_kv_read(*cache.args(), start, cu, 5000)
    wp = gdn.gdn_attn_prefill(wk.repeat(1, 8, 1), wk, wv, cu)
    long_q = wk.repeat(1, 8, 1)
    torch.cuda.synchronize()
    need = gdn.gdn_attn_decode_workspace_bytes(2, cache.page_table.shape[1], 64, 16, 2, 128, 3000)
    assert need > 0
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(10_000_000)  # some milliseconds: the calls below wait behind it
    out = gdn.gdn_attn_decode(q, *cache.args(), ln, max_len=3000, stream=s)
    k, v = gdn.gdn_kv_read(*cache.args(), start, cu, 5000, stream=s)
    p = gdn.gdn_attn_prefill(long_q, wk, wv, cu, stream=s)
    bad = [torch.full((size,), 0xff, dtype=torch.uint8, device=DEV)
           for size in (need, need, out.numel() * 2, k.numel() * 2, k.numel() * 2, p.numel() * 2)]
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(k, wk) and torch.equal(v, wv) and torch.equal(p, wp)
    assert all(bool((x == 0xff).all()) for x in bad)


def test_refusals():
    cache = Cache([40], 16, 2, 64, BF)
    q = torch.zeros(1, 4, 64, dtype=BF, device=DEV)
    ln = ints([40])
    for over in (dict(q=q.float().cpu()), dict(q=q[:, :, :32]), dict(q=torch.zeros(2, 4, 64, dtype=BF, device=DEV)),
                 dict(lens=ln.long()), dict(lens=ints([1, 2])), dict(out=q.float()), dict(k_cache=cache.k[1:]),
                 dict(workspace=torch.zeros(4, device=DEV))):
        a = dict(q=q, k_cache=cache.k, v_cache=cache.v, page_table=cache.page_table, lens=ln)
        a.update(over)
        with pytest.raises(ValueError):
            gdn.gdn_attn_decode(**a)
    for over, name in ((dict(q=q[:, :3]), "SHAPE"), (dict(q=q.float()), "UNSUPPORTED"), (dict(max_len=-1), "SHAPE"),
                       (dict(out=q), "ALIAS"), (dict(scale=math.nan), "SHAPE")):
        a = dict(q=q, k_cache=cache.k, v_cache=cache.v, page_table=cache.page_table, lens=ln)
        a.update(over)
        with pytest.raises(gdn.GdnError, match=name):
            gdn.gdn_attn_decode(**a)
    long = Cache([5000], 16, 2, 64, BF)
    with pytest.raises(gdn.GdnError, match="WORKSPACE"):
        gdn.gdn_attn_decode(q, *long.args(), ints([5000]), workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
