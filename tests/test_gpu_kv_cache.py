"""GPU: the paged key-value cache. What gdn_kv_write stores, and what gdn_kv_read gives back,
are compared bit for bit with a 64-bit evaluation: no step of either is inexact but the one
rounding to the store's type."""
import math

import pytest
import torch

import attn_ref
import gated_deltanet_linear_prefill_amd as gdn

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32, F8 = torch.bfloat16, torch.float32, torch.float8_e4m3fn


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def offsets(lens):
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    return cu


class Cache:
    """Pools filled with a byte pattern, pages handed out in shuffled order."""

    def __init__(self, lens, page, h, d, store, spare=3, seed=0, extra_width=1):
        g = torch.Generator().manual_seed(seed)
        per = [-(-x // page) for x in lens]
        self.pages = sum(per) + spare
        order = torch.randperm(self.pages, generator=g).tolist()
        width = max(per + [0]) + extra_width
        rows, at = [], 0
        for p in per:
            rows.append(order[at:at + p] + [-1] * (width - p))
            at += p
        self.table = rows
        self.page_table = ints(rows).reshape(len(lens), width)
        self.page, self.h, self.d, self.store = page, h, d, store
        size = {F32: 4, BF: 2, F8: 1}[store]
        shape = (self.pages, h, page, d)
        mk = lambda: torch.full((math.prod(shape) * size,), 0x2b, dtype=torch.uint8, device=DEV).view(store).view(shape)
        self.k, self.v = mk(), mk()
        self.ks = self.vs = None
        if store == F8:
            self.ks = torch.full(shape[:3], 120, dtype=torch.uint8, device=DEV)
            self.vs = torch.full(shape[:3], 121, dtype=torch.uint8, device=DEV)

    def args(self):
        return self.k, self.v, self.page_table

    def scales(self):
        return dict(k_scale=self.ks, v_scale=self.vs)

    def place(self, s, pos):
        page = self.table[s][pos // self.page] if 0 <= pos // self.page < len(self.table[s]) and pos >= 0 else -1
        return (page, pos % self.page) if page >= 0 else None


def expected(cache, pool, scale, rows, where):
    """The pool (as float64 values) and scales after rows[i] went to where[i] (None: dropped)."""
    raw = pool.view(torch.uint8).cpu().clone().view(cache.store).double() if cache.store == F8 else pool.cpu().double()
    sc = None if scale is None else scale.cpu().clone()
    if cache.store == F8:
        raw = raw * torch.ldexp(torch.ones(()).double(), sc.int() - 127)[..., None]
    for x, at in zip(rows, where):
        if at is None:
            continue
        if cache.store == F8:
            q, b = attn_ref.quantise(x)
            raw[at[0], :, at[1]] = q
            sc[at[0], :, at[1]] = b
        else:
            raw[at[0], :, at[1]] = x.to(cache.store).double()
    return raw, sc


def values(cache, pool, scale):
    x = pool.view(torch.uint8).cpu().view(cache.store).double() if cache.store == F8 else pool.cpu().double()
    return x if scale is None else x * torch.ldexp(torch.ones(()).double(), scale.cpu().int() - 127)[..., None]


def same(a, b):
    return torch.equal(torch.isnan(a), torch.isnan(b)) and torch.equal(torch.nan_to_num(a, 0.0, 1e300, -1e300),
                                                                       torch.nan_to_num(b, 0.0, 1e300, -1e300))


def rows_of(total, h, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(total, h, d, generator=g) * torch.exp(3 * torch.randn(total, h, 1, generator=g))
    return x.to(dtype)


CASES = [(1, [1], [0], 2, 256, 64, BF, F8), (3, [1, 7, 40], [5, 0, 31], 3, 64, 16, BF, BF),
         (2, [33, 2], [15, 16], 1, 128, 32, F32, F32), (4, [0, 5, 0, 17], [3, 64, 9, 1], 2, 128, 64, F32, F8),
         (2, [100, 64], [0, 1000], 8, 128, 1024, BF, F8), (3, [16, 16, 1], [16, 48, 0], 5, 256, 16, BF, BF)]


@pytest.mark.parametrize("n,lens,start,h,d,page,dtype,store", CASES)
def test_write_and_read_back(n, lens, start, h, d, page, dtype, store):
    cache = Cache([a + b for a, b in zip(start, lens)], page, h, d, store, seed=n)
    total = sum(lens)
    k, v = rows_of(total, h, d, dtype, 1), rows_of(total, h, d, dtype, 2)
    where = [cache.place(s, start[s] + i) for s in range(n) for i in range(lens[s])]
    want_k = expected(cache, cache.k, cache.ks, k, where)
    want_v = expected(cache, cache.v, cache.vs, v, where)
    st, cu = ints(start), ints(offsets(lens))
    gdn.gdn_kv_write(k.to(DEV), v.to(DEV), *cache.args(), st, cu, **cache.scales())
    for pool, sc, (raw, by) in ((cache.k, cache.ks, want_k), (cache.v, cache.vs, want_v)):
        assert sc is None or torch.equal(sc.cpu(), by)
        assert same(values(cache, pool, sc), raw)  # rows that were not written among them
    ko, vo = gdn.gdn_kv_read(*cache.args(), st, cu, total, dtype=dtype, **cache.scales())
    for x, out in ((k, ko), (v, vo)):
        ref = attn_ref.quantise(x)[0] if store == F8 else x.double()
        assert torch.equal(out.cpu(), ref.to(dtype))


@pytest.mark.parametrize("store", [BF, F8])
def test_one_token_each_without_offsets(store):
    n, h, d, page = 9, 2, 128, 16
    start = [0, 1, 15, 16, 17, 40, 2, 31, 32]
    cache = Cache([x + 1 for x in start], page, h, d, store)
    k, v = rows_of(n, h, d, BF, 3), rows_of(n, h, d, BF, 4)
    want = expected(cache, cache.k, cache.ks, k, [cache.place(s, start[s]) for s in range(n)])[0]
    gdn.gdn_kv_write(k.to(DEV), v.to(DEV), *cache.args(), ints(start), **cache.scales())
    assert same(values(cache, cache.k, cache.ks), want)
    ko, vo = gdn.gdn_kv_read(*cache.args(), ints(start), None, n, **cache.scales())
    ref = attn_ref.quantise(v)[0].to(BF) if store == F8 else v
    assert torch.equal(vo.cpu(), ref)


@pytest.mark.parametrize("layout", ["fused", "head_major", "one_head"])
@pytest.mark.parametrize("dtype,store", [(BF, F8), (F32, F32)])
def test_strided_rows(layout, dtype, store):
    n, lens, start, d, page = 2, [9, 20], [3, 0], 64, 16
    h = 1 if layout == "one_head" else 3
    total = sum(lens)
    k, v = rows_of(total, h, d, dtype, 5), rows_of(total, h, d, dtype, 6)
    if layout == "head_major":
        kd = k.transpose(0, 1).contiguous().to(DEV).transpose(0, 1)
        vd = v.transpose(0, 1).contiguous().to(DEV).transpose(0, 1)
    else:  # slices of a fused projection's output
        f = torch.full((total, 5 + 2 * h, d), math.nan, dtype=dtype, device=DEV)
        f[:, 5:5 + h], f[:, 5 + h:] = k.to(DEV), v.to(DEV)
        kd, vd = f[:, 5:5 + h], f[:, 5 + h:]
    assert h == 1 or not kd.is_contiguous()
    cache = Cache([a + b for a, b in zip(start, lens)], page, h, d, store)
    gdn.gdn_kv_write(kd, vd, *cache.args(), ints(start), ints(offsets(lens)), **cache.scales())
    ko, vo = gdn.gdn_kv_read(*cache.args(), ints(start), ints(offsets(lens)), total, dtype=dtype, **cache.scales())
    for x, out in ((k, ko), (v, vo)):
        assert torch.equal(out.cpu(), (attn_ref.quantise(x)[0] if store == F8 else x.double()).to(dtype))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_fp8_edges(dtype):
    """Zeros, the ends of the scale's range, ties, subnormal codes, NaN and infinities."""
    d, fi = 64, torch.finfo(dtype)
    rows = [torch.zeros(d), torch.full((d,), 448.0), torch.full((d,), 448.0 * 2 ** -9), torch.full((d,), 450.0),
            torch.full((d,), fi.max), torch.full((d,), fi.tiny), torch.full((d,), -fi.tiny * 2 ** -3),
            torch.linspace(-1, 1, d), torch.arange(d) * 1.0, 2.0 ** -torch.arange(d).double(),
            256 + 8.0 * torch.arange(d), torch.full((d,), 1.0625), -torch.full((d,), 1.1875)]
    for bad in (math.nan, math.inf, -math.inf):
        x = torch.linspace(-3, 5, d)
        x[7] = bad
        rows.append(x)
    rows.append(torch.full((d,), math.inf))
    k = torch.stack([r.double() for r in rows]).to(dtype)[:, None]
    total = k.shape[0]
    cache = Cache([total], 16, 1, d, F8)
    gdn.gdn_kv_write(k.to(DEV), (-k).to(DEV), *cache.args(), ints([0]), ints([0, total]), **cache.scales())
    ko, vo = gdn.gdn_kv_read(*cache.args(), ints([0]), ints([0, total]), total, dtype=F32, **cache.scales()) \
        if dtype == F32 else gdn.gdn_kv_read(*cache.args(), ints([0]), ints([0, total]), total, **cache.scales())
    ref = attn_ref.quantise(k)[0]
    tiny = 2.0 ** -126  # a value below the normal range may be rounded again, or flushed
    for sign, out in ((1, ko), (-1, vo)):
        # in the type read: the largest may round up past its end
        got, want = out.double().cpu(), (sign * ref).to(dtype).double()
        big = ~(want.abs() < tiny)
        assert same(got[big], want[big])
        assert bool(((got[~big] - want[~big]).abs() <= tiny).all())


def test_places_that_are_not_there():
    """Absent pages, positions past the table or before it, rows outside the offsets."""
    h, d, page = 2, 64, 16
    cache = Cache([40, 20], page, h, d, BF, extra_width=0)
    cache.page_table[0, 1] = -1
    cache.page_table[1, 0] = cache.pages + 5
    cache.table[0][1], cache.table[1][0] = -1, -1
    lens, start = [30, 40], [10, -3]
    first, total = 4, 4 + sum(lens) + 6  # rows 0..3 and the last 6 belong to nobody
    cu = [first, first + lens[0], first + sum(lens)]
    k, v = rows_of(total, h, d, BF, 7), rows_of(total, h, d, BF, 8)
    where = [None] * first + [cache.place(s, start[s] + i) for s in range(2) for i in range(lens[s])] + [None] * 6
    want = expected(cache, cache.k, None, k, where)[0]
    gdn.gdn_kv_write(k.to(DEV), v.to(DEV), *cache.args(), ints(start), ints(cu))
    assert same(values(cache, cache.k, None), want)
    ko = torch.full((total, h, d), 7.0, dtype=BF, device=DEV)
    vo = torch.full((total, h, d), 7.0, dtype=BF, device=DEV)
    gdn.gdn_kv_read(*cache.args(), ints(start), ints(cu), total, k_out=ko, v_out=vo)
    for i in range(total):
        for x, out in ((k, ko), (v, vo)):
            if i < first or i >= total - 6:
                assert bool((out[i] == 7.0).all()), i
            else:
                assert torch.equal(out[i].cpu(), x[i] if where[i] is not None else torch.zeros_like(x[i])), i


def test_offsets_past_32_bits():
    """A pool of more than 4 GiB: its last page is written and read, its first is not touched."""
    h, d, page = 8, 256, 64
    pages = (1 << 32) // (h * page * d * 2) + 40
    k, v = (torch.empty(pages, h, page, d, dtype=BF, device=DEV) for _ in range(2))
    for x in (k, v):
        x[0], x[-1] = 3.0, 3.0
    table = ints([[pages - 1]])
    a, b = rows_of(20, h, d, BF, 9), rows_of(20, h, d, BF, 10)
    gdn.gdn_kv_write(a.to(DEV), b.to(DEV), k, v, table, ints([30]), ints([0, 20]))
    assert torch.equal(k[-1, :, 30:50].cpu(), a.transpose(0, 1)) and bool((k[0] == 3.0).all())
    ko, vo = gdn.gdn_kv_read(k, v, table, ints([30]), ints([0, 20]), 20)
    assert torch.equal(ko.cpu(), a) and torch.equal(vo.cpu(), b)


def test_on_another_stream_and_empty_calls():
    cache = Cache([20], 16, 2, 64, F8)
    k = rows_of(20, 2, 64, BF, 11).to(DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    cu = ints([0, 20])
    with torch.cuda.stream(s):
        gdn.gdn_kv_write(k, k, *cache.args(), ints([0]), cu, **cache.scales())
        ko, _ = gdn.gdn_kv_read(*cache.args(), ints([0]), cu, 20, **cache.scales())
    s.synchronize()
    assert torch.equal(ko.cpu(), attn_ref.quantise(k.cpu())[0].to(BF))
    none = torch.empty(0, 2, 64, dtype=BF, device=DEV)
    gdn.gdn_kv_write(none, none, *cache.args(), ints([0]), ints([0, 0]), **cache.scales())
    ko, vo = gdn.gdn_kv_read(*cache.args(), ints([0]), ints([0, 0]), 0, **cache.scales())
    assert ko.shape == (0, 2, 64)


def test_refusals():
    cache = Cache([20], 16, 2, 64, BF)
    k = torch.zeros(20, 2, 64, dtype=BF, device=DEV)
    cu, st = ints([0, 20]), ints([0])
    before = cache.k.clone()
    bad = [dict(k=k[:, :1]), dict(k=k.float()), dict(k=k.cpu()), dict(k=k.transpose(1, 2)), dict(start=st.long()),
           dict(cu=cu[:1]), dict(cu=cu.cpu()), dict(page_table=cache.page_table.long()), dict(v_cache=cache.v[1:]),
           dict(k_cache=cache.k.half(), v_cache=cache.v.half()), dict(start=ints([0, 0]))]
    for over in bad:
        a = dict(k=k, v=k, k_cache=cache.k, v_cache=cache.v, page_table=cache.page_table, start=st, cu=cu)
        a.update(over)
        with pytest.raises(ValueError):
            gdn.gdn_kv_write(*a.values())
    with pytest.raises(ValueError):  # an fp8 cache without its scales
        f8 = Cache([20], 16, 2, 64, F8)
        gdn.gdn_kv_write(k, k, *f8.args(), st, cu)
    with pytest.raises(gdn.GdnError, match="ALIAS"):
        gdn.gdn_kv_write(cache.k.view(-1, 2, 64)[:20], k, *cache.args(), st, cu)
    with pytest.raises(gdn.GdnError, match="ALIAS"):
        gdn.gdn_kv_read(cache.k, cache.k, cache.page_table, st, cu, 20, k_out=cache.k.view(-1, 2, 64)[:20])
    torch.cuda.synchronize()
    assert torch.equal(cache.k, before)
