"""CPU tests of the attention entry points: every refusal returns its status before any HIP call,
and the binding rejects what the library must not see. Addresses are fake; nothing is launched."""
import ctypes
import random

import pytest
import torch

import gated_deltanet_linear_prefill_amd as gdn

OK, NULL, SHAPE, UNSUP, ALIGN, ALIAS, WS, HIP = range(8)
BASE, STEP = 0x7F0000000000, 1 << 32


@pytest.fixture(scope="module")
def lib():
    return gdn._load()


def addr(i):
    return BASE + i * STEP


def cache(**over):
    a = dict(n=2, num_pages=8, max_pages=4, page_size=16, h_kv=2, d=64, store=gdn.GDN_BF16, k=addr(1), v=addr(2),
             k_scale=addr(3), v_scale=addr(4), page_table=addr(5))
    a.update(over)
    return gdn.KvCache(*[a[f] for f, _ in gdn.KvCache._fields_])


def write(lib, c=None, **over):
    a = dict(total=10, dtype=gdn.GDN_BF16, k=addr(6), kt=128, kh=64, v=addr(7), vt=128, vh=64, start=addr(8), cu=addr(9))
    a.update(over)
    c = cache() if c is None else c
    return lib.gdn_kv_write(ctypes.byref(c), *a.values(), None)


def read(lib, c=None, **over):
    a = dict(total=10, dtype=gdn.GDN_BF16, k=addr(6), v=addr(7), start=addr(8), cu=addr(9))
    a.update(over)
    c = cache() if c is None else c
    return lib.gdn_kv_read(ctypes.byref(c), *a.values(), None)


BAD_CACHES = [
    (dict(n=-1), SHAPE), (dict(num_pages=-1), SHAPE), (dict(max_pages=-1), SHAPE), (dict(page_size=0), SHAPE),
    (dict(h_kv=0), SHAPE), (dict(d=0), SHAPE), (dict(n=1 << 31), SHAPE), (dict(max_pages=1 << 30), SHAPE),
    (dict(num_pages=(1 << 31) - 1, h_kv=1 << 30, page_size=1024), SHAPE),
    (dict(d=32), UNSUP), (dict(d=80), UNSUP), (dict(page_size=8), UNSUP), (dict(page_size=48), UNSUP),
    (dict(page_size=2048), UNSUP), (dict(store=gdn.GDN_F32), UNSUP), (dict(store=7), UNSUP),
    (dict(k=None), NULL), (dict(v=None), NULL), (dict(page_table=None), NULL),
    (dict(store=gdn.GDN_FP8, k_scale=None), NULL), (dict(store=gdn.GDN_FP8, v_scale=None), NULL),
    (dict(k=addr(1) + 8), ALIGN), (dict(v=addr(2) + 4), ALIGN), (dict(page_table=addr(5) + 2), ALIGN),
    (dict(store=gdn.GDN_FP8, k_scale=addr(3) + 1), ALIGN),
]


@pytest.mark.parametrize("over,status", BAD_CACHES)
def test_bad_caches(lib, over, status):
    c = cache(**over)
    assert write(lib, c) == status
    assert read(lib, c) == status
    q = dict(h_q=4, dtype=gdn.GDN_BF16, scale=0.1, max_len=64, q=addr(6), qt=256, qh=64, lens=addr(8), out=addr(9))
    assert lib.gdn_attn_decode(ctypes.byref(c), *q.values(), None, None, 0, None) == status
    if status in (SHAPE, UNSUP) and "store" not in over:
        assert lib.gdn_attn_decode_workspace_bytes(ctypes.byref(c), 4, 100000) == 0


@pytest.mark.parametrize("over,status", [
    (dict(total=-1), SHAPE), (dict(total=1 << 31), SHAPE), (dict(dtype=gdn.GDN_FP8), UNSUP), (dict(dtype=9), UNSUP),
    (dict(kt=60), SHAPE), (dict(kt=132), SHAPE), (dict(kh=0), SHAPE), (dict(vh=-64), SHAPE), (dict(kh=32), SHAPE),
    (dict(kt=64, kh=64), SHAPE), (dict(vt=1 << 22), SHAPE), (dict(k=None), NULL), (dict(v=None), NULL),
    (dict(start=None), NULL), (dict(k=addr(6) + 2), ALIGN), (dict(start=addr(8) + 1), ALIGN), (dict(cu=addr(9) + 2), ALIGN),
    (dict(cu=None), SHAPE), (dict(k=addr(1) + 1024), ALIAS), (dict(v=addr(2)), ALIAS), (dict(start=addr(1) + 64), ALIAS),
])
def test_write_refusals(lib, over, status):
    assert write(lib, **over) == status


def test_pools_that_overlap(lib):
    assert write(lib, cache(v=addr(1) + 1024)) == ALIAS
    assert write(lib, cache(store=gdn.GDN_FP8, k_scale=addr(1))) == ALIAS
    assert write(lib, cache(page_table=addr(2))) == ALIAS


@pytest.mark.parametrize("over,status", [
    (dict(total=-1), SHAPE), (dict(dtype=3), UNSUP), (dict(k=None), NULL), (dict(start=None), NULL),
    (dict(v=addr(7) + 8), ALIGN), (dict(k=addr(7)), ALIAS), (dict(k=addr(1)), ALIAS), (dict(v=addr(5)), ALIAS),
    (dict(cu=None), SHAPE), (dict(k=addr(8)), ALIAS),
])
def test_read_refusals(lib, over, status):
    assert read(lib, **over) == status


def test_calls_without_work(lib):
    """No sequences, no tokens, an empty pool: accepted, nothing to do, no pointers needed."""
    assert write(lib, cache(n=0), total=0, k=None, v=None, start=None) == OK
    assert write(lib, total=0, k=None, v=None) == OK
    assert write(lib, cache(num_pages=0, k=None, v=None)) == OK
    assert read(lib, cache(n=0), total=0, k=None, v=None, start=None, cu=None) == OK


def prefill(lib, lse=None, ws=None, ws_bytes=0, out=addr(4), q=addr(1), k=addr(2), v=addr(3), cu_q=addr(5), cu_k=addr(6), **over):
    a = dict(n=2, total_q=10, total_k=20, h_q=4, h_kv=2, d=64, dtype=gdn.GDN_BF16, causal=1, scale=0.125, q_token=256,
             q_head=64, k_token=128, k_head=64, v_token=128, v_head=64)
    a.update(over)
    d = gdn.AttnDims(*[a[f] for f, _ in gdn.AttnDims._fields_])
    return lib.gdn_attn_prefill(ctypes.byref(d), q, k, v, cu_q, cu_k, out, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("over,status", [
    (dict(n=-1), SHAPE), (dict(total_q=-1), SHAPE), (dict(total_k=-2), SHAPE), (dict(h_q=3), SHAPE), (dict(h_kv=0), SHAPE),
    (dict(h_q=0), SHAPE), (dict(causal=2), SHAPE), (dict(scale=float("nan")), SHAPE), (dict(scale=float("inf")), SHAPE),
    (dict(total_q=(1 << 31) - 1), SHAPE), (dict(total_k=1 << 31), SHAPE), (dict(n=1 << 31), SHAPE),
    (dict(d=96), UNSUP), (dict(dtype=gdn.GDN_FP8), UNSUP), (dict(cu_k=None), SHAPE),
    (dict(q_token=250), SHAPE), (dict(k_head=8), SHAPE), (dict(v_token=0), SHAPE), (dict(q_token=128), SHAPE),
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(out=None), NULL), (dict(cu_q=None), NULL),
    (dict(q=addr(1) + 8), ALIGN), (dict(lse=addr(7) + 2), ALIGN), (dict(cu_k=addr(6) + 1), ALIGN),
    (dict(out=addr(1)), ALIAS), (dict(out=addr(3) + 256), ALIAS), (dict(lse=addr(2)), ALIAS), (dict(lse=addr(4)), ALIAS),
    (dict(out=addr(5)), ALIAS), (dict(ws=addr(8) + 4), ALIGN), (dict(total_k=9000), WS),
    (dict(total_k=9000, ws=addr(8), ws_bytes=1000), WS),
    (dict(total_k=9000, ws=addr(1), ws_bytes=1 << 30), ALIAS), (dict(total_k=9000, ws=addr(5), ws_bytes=1 << 30), ALIAS),
])
def test_prefill_refusals(lib, over, status):
    assert prefill(lib, **over) == status


def test_prefill_without_work(lib):
    assert prefill(lib, n=0, q=None, k=None, v=None, out=None, cu_q=None, cu_k=None, total_k=10) == OK
    assert prefill(lib, total_q=0, q=None, out=None) == OK
    assert lib.gdn_attn_prefill(None, None, None, None, None, None, None, None, None, 0, None) == NULL


def decode(lib, c=None, ws=None, ws_bytes=0, lse=None, **over):
    a = dict(h_q=4, dtype=gdn.GDN_BF16, scale=0.1, max_len=64, q=addr(6), qt=256, qh=64, lens=addr(8), out=addr(9))
    a.update(over)
    c = cache() if c is None else c
    return lib.gdn_attn_decode(ctypes.byref(c), *a.values(), lse, ws, ws_bytes, None)


@pytest.mark.parametrize("over,status", [
    (dict(h_q=3), SHAPE), (dict(h_q=0), SHAPE), (dict(max_len=-1), SHAPE), (dict(scale=float("inf")), SHAPE),
    (dict(dtype=gdn.GDN_F32), UNSUP), (dict(qt=100), SHAPE), (dict(qh=4), SHAPE), (dict(q=None), NULL),
    (dict(lens=None), NULL), (dict(out=None), NULL), (dict(q=addr(6) + 4), ALIGN), (dict(lens=addr(8) + 2), ALIGN),
    (dict(lse=addr(10) + 1), ALIGN), (dict(out=addr(6)), ALIAS), (dict(out=addr(1)), ALIAS), (dict(lse=addr(9)), ALIAS),
    (dict(lse=addr(5)), ALIAS),
])
def test_decode_refusals(lib, over, status):
    assert decode(lib, **over) == status


def test_decode_workspace(lib):
    c = cache(num_pages=1000, max_pages=400)
    need = lib.gdn_attn_decode_workspace_bytes(ctypes.byref(c), 4, 6400)
    assert need > 0
    assert lib.gdn_attn_decode_workspace_bytes(ctypes.byref(c), 4, 100) == 0  # nothing to split
    assert lib.gdn_attn_decode_workspace_bytes(ctypes.byref(c), 3, 6400) == 0
    assert lib.gdn_attn_decode_workspace_bytes(None, 4, 6400) == 0
    # max_len beyond the table asks for no more than the table does
    assert lib.gdn_attn_decode_workspace_bytes(ctypes.byref(c), 4, 1 << 40) == need
    assert decode(lib, c, max_len=6400) == WS
    assert decode(lib, c, max_len=6400, ws=addr(11), ws_bytes=need - 1) == WS
    assert decode(lib, c, max_len=6400, ws=addr(11) + 8, ws_bytes=need) == ALIGN
    assert decode(lib, c, max_len=6400, ws=addr(9), ws_bytes=need) == ALIAS
    assert decode(lib, c, max_len=6400, ws=addr(1), ws_bytes=need) == ALIAS


def test_decode_without_sequences(lib):
    assert decode(lib, cache(n=0, page_table=None, max_pages=0), q=None, lens=None, out=None) == OK


def test_binding_rejects_cpu_tensors():
    z = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    pool = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: gdn.gdn_kv_write(z, z, pool, pool, i[:, None], i, i), lambda: gdn.gdn_attn_prefill(z, z, z, i),
                 lambda: gdn.gdn_kv_read(pool, pool, i[:, None], i, i, 4),
                 lambda: gdn.gdn_attn_decode(z[:2], pool, pool, i[:, None], i)):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(ValueError):
        gdn.gdn_attn_prefill(z.tolist(), z, z, i)


def test_workspaces_stay_below_their_bounds(lib):
    """What the header says is enough for any call, over random sizes."""
    rng = random.Random(5)
    size = lambda top: int(2 ** rng.uniform(0, top))
    seen = 0
    for _ in range(20000):
        hk, g, n, d = rng.choice([1, 2, 3, 8]), rng.choice([1, 3, 8, 16, 20]), size(9), rng.choice([64, 128, 256])
        f32 = rng.random() < 0.4
        need = gdn.gdn_attn_prefill_workspace_bytes(n, size(16), size(22), hk * g, hk, d,
                                                    torch.float32 if f32 else torch.bfloat16)
        assert need <= 64 * 1024 * (4 * d + 16) * (2 if f32 and d == 256 else 1)
        seen += need > 0
        page = rng.choice([16, 64, 1024])
        units = n * hk * -(-g // 16)
        need = gdn.gdn_attn_decode_workspace_bytes(n, size(12), page, hk * g, hk, d, size(22))
        assert need <= (4096 + units) * 16 * (4 * d + 16)
        seen += need > 0
    assert seen > 4000
