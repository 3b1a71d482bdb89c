"""GPU: attention of new tokens over the paged cache, with and without a window, against a 64-bit
evaluation (tests/attn_ref.py)."""
import math

import pytest
import torch

import attn_ref
import gated_deltanet_linear_prefill_amd as gdn
from test_gpu_attn_decode import dense, fill
from test_gpu_kv_cache import BF, DEV, F8, F32, Cache, ints, offsets

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True, params=["as they are", "among empty sequences"])
def batch(request, monkeypatch):
    """Every test twice: small calls take tiles of 16 rows, the same sequences among 70 empty ones larger tiles."""
    if request.param == "as they are":
        return
    plain = gdn.gdn_attn_extend

    def call(q, k_cache, v_cache, page_table, lens, cu_q=None, **kw):
        tensors = all(isinstance(x, torch.Tensor) and x.is_cuda and x.dtype == torch.int32 for x in (page_table, lens, cu_q))
        if tensors and "workspace" not in kw and kw.get("max_q") != 1:
            with torch.cuda.stream(kw.get("stream")):
                page_table = torch.cat([page_table, page_table.new_full((70, page_table.shape[1]), -1)])
                lens = torch.cat([lens, lens.new_zeros(70)])
                cu_q = torch.cat([cu_q, cu_q[-1:].expand(70)])
        return plain(q, k_cache, v_cache, page_table, lens, cu_q, **kw)

    monkeypatch.setattr(gdn, "gdn_attn_extend", call)


def queries(total, hq, d, dtype, seed=1):
    return (1.5 * torch.randn(total, hq, d, generator=torch.Generator().manual_seed(seed))).to(dtype)


def sight(lq, length, window, sinks):
    """[lq, length] of the definition."""
    p, j = torch.arange(lq)[:, None] + length - lq, torch.arange(length)[None]
    ok = j <= p
    if window:
        ok &= (p - j < window) | (j < sinks)
    return ok


def compare(cache, q, lens_q, lens, out, lse, scale, window=0, sinks=0, first=0):
    g, at = q.shape[1] // cache.h, first
    for s, (lq, length) in enumerate(zip(lens_q, lens)):
        k, v, there = dense(cache, s, max(length, 0))
        allowed = sight(lq, max(length, 0), window, sinks) & there[None]
        for h in range(q.shape[1]):
            ref = attn_ref.attend(q[at:at + lq, h], k[:, h // g], v[:, h // g], scale, allowed)
            attn_ref.check(out[at:at + lq, h], None if lse is None else lse[at:at + lq, h], *ref, what=f"sequence {s} head {h}")
        at += lq


def go(lens_q, lens, hq, hk, d, page, dtype, store, window=0, sinks=0, seed=5, scale=None, **kw):
    cache = Cache(lens, page, hk, d, store, seed=seed)
    fill(cache, seed, nan_behind=lens)
    q = queries(sum(lens_q), hq, d, dtype)
    lse = torch.full(q.shape[:2], 5.0, device=DEV)
    out = gdn.gdn_attn_extend(q.to(DEV), *cache.args(), ints(lens), ints(offsets(lens_q)), window=window, sinks=sinks, lse=lse,
                              scale=scale, **cache.scales(), **kw)
    compare(cache, q, lens_q, lens, out, lse, d ** -0.5 if scale is None else scale, window, sinks)
    return out


CASES = [  # rows per sequence, lengths, h_q, h_kv, d, page, dtype, store
    ([1], [1], 1, 1, 64, 16, BF, BF), ([4], [333], 16, 2, 256, 64, BF, BF), ([3, 1, 0, 17, 2, 5, 1], [17, 1, 0, 200, 31, 32, 33], 8, 2, 128, 16, BF, BF),
    ([33, 3], [500, 3], 6, 2, 64, 32, BF, F8), ([2, 9, 1], [129, 128, 127], 16, 1, 256, 128, BF, F8), ([64, 65], [64, 65], 20, 1, 64, 16, BF, F8),
    ([7, 2], [90, 2], 4, 4, 64, 16, F32, F32), ([5], [40], 33, 1, 128, 16, F32, F8), ([11, 7], [70, 7], 6, 3, 256, 64, F32, F32),
    ([6], [300], 2, 1, 256, 1024, F32, F8), ([4, 100], [5000, 100], 3, 1, 128, 64, BF, BF), ([8], [2500], 17, 1, 64, 16, BF, BF),
    ([150], [700], 4, 2, 128, 16, BF, BF), ([300, 20], [300, 1000], 2, 1, 256, 64, BF, BF), ([130], [400], 8, 1, 256, 32, BF, F8),
    ([90, 1], [100, 90], 3, 3, 64, 16, F32, F32), ([70], [257], 4, 1, 128, 64, F32, F8), ([200], [333], 2, 2, 64, 16, BF, F8),
]


@pytest.mark.parametrize("lens_q,lens,hq,hk,d,page,dtype,store", CASES)
def test_against_64_bits(lens_q, lens, hq, hk, d, page, dtype, store):
    go(lens_q, lens, hq, hk, d, page, dtype, store)


WINDOWS = [(1, 0), (1, 1), (5, 3), (16, 16), (17, 4), (100, 0), (64, 33), (130, 700)]


@pytest.mark.parametrize("window,sinks", WINDOWS)
@pytest.mark.parametrize("lens_q,lens,hq,hk,d,page,dtype,store", [
    ([3, 1, 0, 40], [300, 90, 5, 555], 8, 2, 128, 16, BF, BF), ([150], [700], 4, 2, 64, 32, BF, F8), ([5, 70], [333, 71], 6, 3, 256, 64, BF, BF),
    ([9, 2], [260, 400], 3, 1, 64, 16, F32, F32), ([20], [310], 16, 1, 256, 16, BF, F8), ([33], [290], 2, 1, 128, 64, F32, F8),
])
def test_windows(window, sinks, lens_q, lens, hq, hk, d, page, dtype, store):
    go(lens_q, lens, hq, hk, d, page, dtype, store, window, sinks)


@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (33, 4), (1000, 70)])
@pytest.mark.parametrize("lens,hq,hk,d,page,dtype,store", [
    ([1, 333, 0, 2000], 16, 2, 256, 64, BF, BF), ([17, 5000], 8, 2, 128, 16, BF, F8), ([40, 41, 900], 33, 1, 64, 16, F32, F32), ([1500], 20, 1, 64, 32, F32, F8),
])
def test_one_token_per_sequence(window, sinks, lens, hq, hk, d, page, dtype, store):
    cache = Cache(lens, page, hk, d, store)
    fill(cache, 5, nan_behind=lens)
    n = len(lens)
    q = queries(n, hq, d, dtype)
    lse = torch.full(q.shape[:2], 5.0, device=DEV)
    out = gdn.gdn_attn_extend(q.to(DEV), *cache.args(), ints(lens), window=window, sinks=sinks, lse=lse, **cache.scales())
    compare(cache, q, [1] * n, lens, out, lse, d ** -0.5, window, sinks)
    same = gdn.gdn_attn_extend(q.to(DEV), *cache.args(), ints(lens), ints(list(range(n + 1))), max_q=1, window=window, sinks=sinks, **cache.scales())
    assert torch.equal(out, same)
    # some of the sequences bring no token
    some = [i % 2 for i in range(n)]
    out = gdn.gdn_attn_extend(q[:sum(some)].to(DEV), *cache.args(), ints(lens), ints(offsets(some)), max_q=1, window=window, sinks=sinks, **cache.scales())
    compare(cache, q[:sum(some)], some, lens, out, None, d ** -0.5, window, sinks)


@pytest.mark.parametrize("store,dtype", [(BF, BF), (F8, BF), (F32, F32)])
@pytest.mark.parametrize("rows", [1, 6, 90])
def test_absent_pages_and_bounds(store, dtype, rows):
    """Pages that are not there are skipped, whole ranges of them too; lengths past the table or past
    max_len are cut, negative ones are empty; sequences with more rows than positions."""
    lens, page, lens_q = [400, 300, 700, 100], 16, [rows, rows, rows + 1, rows]
    cache = Cache(lens, page, 2, 64, store, extra_width=0)
    fill(cache, 6)
    for s, gone in ((0, [0, 3, 24]), (1, list(range(len(cache.table[1])))), (2, list(range(8, 30)))):
        for x in gone:
            if x < len(cache.table[s]) and cache.table[s][x] >= 0:
                cache.table[s][x] = -1
                cache.page_table[s, x] = -1 if x % 2 else cache.pages + 1
    q = queries(sum(lens_q), 4, 64, dtype)
    lse = torch.zeros(sum(lens_q), 4, device=DEV)
    width = cache.page_table.shape[1] * page
    cu = ints(offsets(lens_q))
    for window, sinks in ((0, 0), (50, 5)):
        kw = dict(lse=lse, window=window, sinks=sinks, **cache.scales())
        out = gdn.gdn_attn_extend(q.to(DEV), *cache.args(), ints([400, 300, 10 ** 6, -5]), cu, **kw)
        compare(cache, q, lens_q, [400, 300, width, 0], out, lse, 64 ** -0.5, window, sinks)
        out = gdn.gdn_attn_extend(q.to(DEV), *cache.args(), ints([400, 300, 10 ** 6, 3]), cu, max_len=130, **kw)
        compare(cache, q, lens_q, [130, 130, 130, 3], out, lse, 64 ** -0.5, window, sinks)
    out = gdn.gdn_attn_extend(q.to(DEV), *cache.args(), ints(lens), cu, max_len=0, lse=lse, **cache.scales())
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


@pytest.mark.parametrize("rows", [4, 80])
def test_pages_behind_the_window_are_given_away(rows):
    """With a window the pages that no row sees are not looked at: absent, or full of NaN."""
    lens, page, window, sinks = [900], 16, 100, 20
    cache = Cache(lens, page, 2, 128, BF)
    fill(cache, 7)
    low = 900 - rows - window
    q = queries(rows, 8, 128, BF)
    ref = gdn.gdn_attn_extend(q.to(DEV), *cache.args(), ints(lens), ints([0, rows]), window=window, sinks=sinks)
    for x in range(2, low // page):
        page_id = int(cache.page_table[0, x])
        if x % 2:
            cache.page_table[0, x] = -1
        else:
            cache.k[page_id] = math.nan
            cache.v[page_id] = math.nan
    out = gdn.gdn_attn_extend(q.to(DEV), *cache.args(), ints(lens), ints([0, rows]), window=window, sinks=sinks)
    assert torch.equal(out, ref)


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("store,dtype,d", [(BF, BF, 128), (F8, BF, 64), (F32, F32, 64), (BF, BF, 256), (F8, F32, 128), (F8, BF, 256)])
@pytest.mark.parametrize("rows", [12, 100])
def test_what_a_row_may_not_see(bad, store, dtype, d, rows):
    """NaN and infinities in keys and values that some rows see and others do not: after a row, before its
    window, between the sinks and it."""
    lens, page, window, sinks = [200], 16, 30, 5
    for name in ("k", "v"):
        for w, s in ((0, 0), (window, sinks)):
            cache = Cache(lens, page, 1, d, store)
            fill(cache, 8)
            for pos in ([199, 195] if w == 0 else [195, 3, 6, 200 - rows - 5, 199 - rows // 2, 160]):
                at = cache.place(0, max(pos, 0))
                pool = getattr(cache, name)
                if store == F8:
                    if not math.isnan(bad):
                        continue
                    pool.view(torch.uint8)[at[0], :, at[1], pos % 7] = 0x7f
                else:
                    pool[at[0], :, at[1], pos % 7] = bad
            q = queries(rows, 2, d, dtype)
            lse = torch.zeros(rows, 2, device=DEV)
            out = gdn.gdn_attn_extend(q.to(DEV), *cache.args(), ints(lens), ints([0, rows]), window=w, sinks=s, lse=lse, **cache.scales())
            if name == "v":
                compare(cache, q, [rows], lens, out, lse, d ** -0.5, w, s)
            else:  # rows that see no such key
                k, _, _ = dense(cache, 0, 200)
                clean = ~(sight(rows, 200, w, s) & ~torch.isfinite(k).all(-1)[:, 0][None]).any(1)
                k = torch.nan_to_num(k, 0.0, 0.0, 0.0)
                _, v, _ = dense(cache, 0, 200)
                for h in range(2):
                    ref = attn_ref.attend(q[:, h], k[:, 0], v[:, 0], d ** -0.5, sight(rows, 200, w, s))
                    ref = [x[clean] for x in ref]
                    attn_ref.check(out[clean, h], lse[clean, h], *ref, what=f"head {h}")
                if math.isnan(bad):
                    assert bool(torch.isnan(out[~clean]).all()) and bool(torch.isnan(lse[~clean]).all())


def test_nan_in_a_query():
    cache = Cache([300], 16, 2, 64, BF)
    fill(cache, 9)
    q = queries(40, 4, 64, BF)
    q[7, 2, 5] = math.nan
    lse = torch.zeros(40, 4, device=DEV)
    out = gdn.gdn_attn_extend(q.to(DEV), *cache.args(), ints([300]), ints([0, 40]), lse=lse)
    want = torch.zeros(40, 4, dtype=torch.bool)
    want[7, 2] = True
    assert torch.equal(torch.isnan(out.cpu()).all(-1), want) and torch.equal(torch.isnan(out.cpu()).any(-1), want)
    assert torch.equal(torch.isnan(lse.cpu()), want)


@pytest.mark.parametrize("layout", ["fused", "head_major"])
@pytest.mark.parametrize("rows", [3, 70])
def test_strided_queries_scale_and_used_workspace(layout, rows):
    lens = [2600, 71]
    cache = Cache(lens, 32, 2, 128, BF)
    fill(cache, 7)
    f = torch.randn(2 * rows, 12, 128, dtype=BF, generator=torch.Generator().manual_seed(2))
    q = f[:, 4:8]
    qd = f.to(DEV)[:, 4:8] if layout == "fused" else q.transpose(0, 1).contiguous().to(DEV).transpose(0, 1)
    sizes = dict(max_q=rows, max_len=2600)
    need = gdn.gdn_attn_extend_workspace_bytes(2, cache.page_table.shape[1], 32, 2 * rows, 4, 2, 128, **sizes)
    assert need > 0
    ws = torch.full((need + 64,), 0xff, dtype=torch.uint8, device=DEV)
    out = gdn.gdn_attn_extend(qd, *cache.args(), ints(lens), ints([0, rows, 2 * rows]), scale=-0.5, workspace=ws, **sizes)
    compare(cache, q, [rows, rows], lens, out, None, -0.5)
    assert bool((ws[need:] == 0xff).all())
    with pytest.raises(gdn.GdnError, match="WORKSPACE"):
        gdn.gdn_attn_extend(qd, *cache.args(), ints(lens), ints([0, rows, 2 * rows]), workspace=ws[:need - 16], **sizes)


@pytest.mark.parametrize("rows", [5, 90])
def test_rows_that_are_not_computed(rows):
    """Rows of no sequence and rows from max_q on are left as they are in out and lse."""
    cache = Cache([200, 100], 16, 1, 64, BF)
    fill(cache, 3)
    total = rows + 20
    q = queries(total, 2, 64, BF)
    out, lse = torch.full((total, 2, 64), 7.0, dtype=BF, device=DEV), torch.full((total, 2), 7.0, device=DEV)
    cu = [4, 4 + rows, 4 + rows + 6]
    gdn.gdn_attn_extend(q.to(DEV), *cache.args(), ints([200, 100]), ints(cu), out=out, lse=lse, max_q=rows - 2)
    whole = gdn.gdn_attn_extend(q.to(DEV), *cache.args(), ints([200, 100]), ints(cu))
    done = [i for i in range(4, cu[1] - 2)] + [i for i in range(cu[1], min(cu[2], cu[1] + rows - 2))]
    rest = [i for i in range(total) if i not in done]
    assert bool((out[rest] == 7.0).all()) and bool((lse[rest] == 7.0).all())
    # another bound may divide the keys otherwise: the same to a rounding of each
    tol = 2 * (2.0 ** -7 + 2.0 ** -10) * cache.v.float().abs().max()
    assert bool(((out[done].float() - whole[done].float()).abs() <= tol).all())
    compare(cache, q[done], [rows - 2], [198], out[done][:rows - 2], None, 64 ** -0.5)


def test_large_scores_and_scales():
    lens, lens_q = [600, 300], [20, 40]
    cache = Cache(lens, 16, 1, 64, BF)
    fill(cache, 9)
    q = 40 * queries(60, 3, 64, BF)
    for scale in (1.0, 0.0, 1e-30, -2.0):
        out = gdn.gdn_attn_extend(q.to(DEV), *cache.args(), ints(lens), ints(offsets(lens_q)), scale=scale)
        compare(cache, q, lens_q, lens, out, None, scale)


def test_the_same_as_the_other_calls():
    """A whole prompt against gdn_attn_prefill, a last token against gdn_attn_decode: one formula."""
    length, hq, hk, d = 333, 8, 2, 128
    cache = Cache([length], 16, hk, d, BF)
    fill(cache, 4)
    q = queries(length, hq, d, BF).to(DEV)
    k, v = gdn.gdn_kv_read(*cache.args(), ints([0]), ints([0, length]), length)
    top = float(v.abs().max())
    a = gdn.gdn_attn_extend(q, *cache.args(), ints([length]), ints([0, length]))
    b = gdn.gdn_attn_prefill(q, k, v, ints([0, length]))
    assert float((a.float() - b.float()).abs().max()) <= 2 * (2.0 ** -7 + 2.0 ** -10) * top
    a = gdn.gdn_attn_extend(q[-1:], *cache.args(), ints([length]))
    b = gdn.gdn_attn_decode(q[-1:], *cache.args(), ints([length]))
    assert float((a.float() - b.float()).abs().max()) <= 2 * (2.0 ** -7 + 2.0 ** -10) * top


def test_repeats_and_streams():
    lens, lens_q = [3000, 800, 70], [5, 40, 1]
    cache = Cache(lens, 64, 2, 128, F8)
    fill(cache, 4)
    q, cu, ln = queries(46, 8, 128, BF).to(DEV), ints(offsets(lens_q)), ints(lens)
    call = lambda **kw: gdn.gdn_attn_extend(q, *cache.args(), ln, cu, window=700, sinks=4, max_q=40, **cache.scales(), **kw)
    ref = call()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    outs = [call(stream=s) for _ in range(3)]
    s.synchronize()
    for x in outs + [call()]:
        assert torch.equal(x, ref)


@pytest.mark.parametrize("lens_q", [[1, 1, 1], [4, 2, 6], [50, 1, 90]])
def test_captured_and_replayed(lens_q):
    """Two graphs with workspaces of their own, the lengths moved on between replays."""
    lens = [3000, 2100, 900]
    cache = Cache([x + 40 for x in lens], 16, 2, 128, BF)
    fill(cache, 4)
    q, cu, ln = queries(sum(lens_q), 8, 128, BF).to(DEV), ints(offsets(lens_q)), ints(lens)
    kw = dict(max_q=max(lens_q), max_len=3040)
    graphs, outs = [], []
    for window in (0, 500):
        call = lambda out: gdn.gdn_attn_extend(q, *cache.args(), ln, cu, window=window, sinks=8 if window else 0, out=out, **kw)
        out = torch.empty_like(q)
        call(out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            call(out)
        graphs.append(g)
        outs.append(out)
    for i in range(4):
        q.mul_(1.125)
        ln.add_(i)
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for window, out in zip((0, 500), outs):
            ref = gdn.gdn_attn_extend(q, *cache.args(), ln, cu, window=window, sinks=8 if window else 0, **kw)
            assert torch.equal(ref, out), (i, window)


def test_empty_calls():
    cache = Cache([20], 16, 2, 64, BF)
    none = torch.empty(0, 4, 64, dtype=BF, device=DEV)
    assert gdn.gdn_attn_extend(none, *cache.args(), ints([20]), ints([0, 0])).shape == none.shape
    q = queries(3, 4, 64, BF).to(DEV)
    out = torch.full_like(q, 7.0)
    gdn.gdn_attn_extend(q, *cache.args(), ints([20]), ints([0, 3]), out=out, max_q=0)
    assert bool((out == 7.0).all())
    # an empty pool: rows that see nothing
    pool = torch.empty(0, 2, 16, 64, dtype=BF, device=DEV)
    lse = torch.zeros(3, 4, device=DEV)
    out = gdn.gdn_attn_extend(q, pool, pool, cache.page_table, ints([20]), ints([0, 3]), lse=lse)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_offsets_past_32_bits():
    """Pages past the 4 GiB of a pool."""
    h, d, page = 8, 256, 64
    pages = (1 << 32) // (h * page * d * 2) + 40
    k, v = (torch.zeros(pages, h, page, d, dtype=BF, device=DEV) for _ in range(2))
    g = torch.Generator().manual_seed(3)
    last = [pages - 1, pages - 5, pages - 30]
    small_k, small_v = (torch.randn(3, h, page, d, generator=g).to(BF).to(DEV) for _ in range(2))
    for i, x in enumerate(last):
        k[x], v[x] = small_k[i], small_v[i]
    for rows in (2, 60):
        q = queries(rows, 16, d, BF).to(DEV)
        a = gdn.gdn_attn_extend(q, k, v, ints([last]), ints([170]), ints([0, rows]))
        b = gdn.gdn_attn_extend(q, small_k, small_v, ints([[0, 1, 2]]), ints([170]), ints([0, rows]))
        assert torch.equal(a, b)


def test_refusals():
    cache = Cache([20], 16, 2, 64, BF)
    q, ln, cu = queries(3, 4, 64, BF).to(DEV), ints([20]), ints([0, 3])
    bad = [dict(q=q.half()), dict(q=q.cpu()), dict(q=q[..., :32]), dict(lens=ln.long()), dict(cu_q=cu[:1]), dict(cu_q=None),
           dict(out=q[:2]), dict(lse=torch.zeros(3, 4, device=DEV, dtype=BF)), dict(workspace=q)]
    for over in bad:
        a = dict(q=q, k_cache=cache.k, v_cache=cache.v, page_table=cache.page_table, lens=ln, cu_q=cu)
        a.update(over)
        with pytest.raises(ValueError):
            gdn.gdn_attn_extend(**a)
    for over, status in ((dict(window=-1), 2), (dict(sinks=-1), 2), (dict(max_len=-1), 2), (dict(max_q=-1), 2), (dict(scale=math.inf), 2),
                         (dict(q=q[:, :3]), 2), (dict(out=q), 5), (dict(q=q.float()), 3)):
        a = dict(q=q, k_cache=cache.k, v_cache=cache.v, page_table=cache.page_table, lens=ln, cu_q=cu)
        a.update(over)
        with pytest.raises(gdn.GdnError) as e:
            gdn.gdn_attn_extend(**a)
        assert e.value.status == status, over
