"""CPU tests of the entry points around the attention layers: every refusal returns its status before
any HIP call, and the binding rejects what the library must not see. Addresses are fake; nothing is
launched."""
import ctypes
import random

import pytest
import torch

import gated_deltanet_linear_prefill_amd as gdn
from test_attn_checks import ALIAS, ALIGN, BAD_CACHES, NULL, OK, SHAPE, UNSUP, WS, addr, cache, lib  # noqa: F401


def norm(**over):
    a = dict(eps=1e-6, weight_bias=1.0, q_weight=addr(20), k_weight=addr(21), rot=32, interleaved=0, axes=1, rope_scale=1.0,
             freq=addr(22), axis=None, pos=addr(23))
    a.update(over)
    return gdn.NormRope(*[a[f] for f, _ in gdn.NormRope._fields_])


NORMS = [
    (dict(eps=-1.0), SHAPE), (dict(eps=float("nan")), SHAPE), (dict(eps=float("inf")), SHAPE), (dict(weight_bias=float("inf")), SHAPE),
    (dict(rot=8), SHAPE), (dict(rot=-16), SHAPE), (dict(rot=80), SHAPE), (dict(rot=24), SHAPE), (dict(interleaved=2), SHAPE),
    (dict(axes=0), SHAPE), (dict(axes=5), SHAPE), (dict(rope_scale=float("nan")), SHAPE), (dict(freq=None), NULL),
    (dict(q_weight=addr(20) + 8), ALIGN), (dict(k_weight=addr(21) + 2), ALIGN), (dict(freq=addr(22) + 2), ALIGN), (dict(pos=addr(23) + 1), ALIGN),
]


def rope(lib, f=None, **over):
    a = dict(total=10, h_q=4, h_kv=2, d=64, dtype=gdn.GDN_BF16, q=addr(1), qt=256, qh=64, k=addr(2), kt=128, kh=64, q_out=addr(3),
             k_out=addr(4))
    a.update(over)
    f = norm() if f is None else f
    return lib.gdn_qk_norm_rope(ctypes.byref(f), *a.values(), None)


@pytest.mark.parametrize("over,status", NORMS + [(dict(pos=None), NULL)])
def test_rope_norms(lib, over, status):
    assert rope(lib, norm(**over)) == status


@pytest.mark.parametrize("over,status", [
    (dict(total=-1), SHAPE), (dict(total=1 << 31), SHAPE), (dict(total=1 << 30), SHAPE), (dict(h_q=-1), SHAPE), (dict(h_kv=-2), SHAPE), (dict(d=0), SHAPE),
    (dict(d=96), UNSUP), (dict(dtype=gdn.GDN_FP8), UNSUP), (dict(qt=100), SHAPE), (dict(kh=8), SHAPE), (dict(kt=64), SHAPE), (dict(qt=1 << 22), SHAPE),
    (dict(q=None), NULL), (dict(k=None), NULL), (dict(q_out=None), NULL), (dict(k_out=None), NULL), (dict(q=addr(1) + 8), ALIGN),
    (dict(k_out=addr(4) + 4), ALIGN), (dict(q_out=addr(1)), ALIAS), (dict(k_out=addr(2) + 256), ALIAS), (dict(k_out=addr(3)), ALIAS),
    (dict(q_out=addr(20)), ALIAS), (dict(q_out=addr(22)), ALIAS), (dict(k_out=addr(23)), ALIAS), (dict(q_out=addr(2)), ALIAS),
])
def test_rope_refusals(lib, over, status):
    assert rope(lib, **over) == status


def test_rope_without_work(lib):
    assert rope(lib, total=0, q=None, k=None, q_out=None, k_out=None) == OK
    assert rope(lib, h_q=0, h_kv=0, q=None, k=None, q_out=None, k_out=None) == OK
    assert lib.gdn_qk_norm_rope(None, 1, 1, 1, 64, gdn.GDN_BF16, None, 0, 0, None, 0, 0, None, None, None) == NULL
    # strides of what is not there are not looked at; what is there still is
    assert rope(lib, h_kv=0, k=None, kt=0, kh=0, k_out=None, q=addr(1) + 8) == ALIGN
    # without a rotation its tensors are not looked at
    assert rope(lib, norm(rot=0, axes=0, rope_scale=float("nan"), freq=None, pos=None, axis=addr(1)), q_out=addr(1)) == ALIAS


def append(lib, c=None, f=None, **over):
    a = dict(total=10, dtype=gdn.GDN_BF16, k=addr(6), kt=128, kh=64, v=addr(7), vt=128, vh=64, start=addr(8), cu=addr(9), h_q=4, q=addr(10),
             qt=256, qh=64, q_out=addr(11))
    a.update(over)
    c = cache() if c is None else c
    f = norm() if f is None else f
    return lib.gdn_kv_append(ctypes.byref(c), ctypes.byref(f), *a.values(), None)


@pytest.mark.parametrize("over,status", NORMS + [(dict(pos=None, axes=2), SHAPE)])
def test_append_norms(lib, over, status):
    assert append(lib, None, norm(**over)) == status


@pytest.mark.parametrize("over,status", BAD_CACHES)
def test_bad_caches(lib, over, status):
    assert append(lib, cache(**over)) == status
    assert extend(lib, cache(**over)) == status


@pytest.mark.parametrize("over,status", [
    (dict(total=-1), SHAPE), (dict(total=1 << 31), SHAPE), (dict(total=1 << 28), SHAPE), (dict(dtype=gdn.GDN_FP8), UNSUP), (dict(kt=60), SHAPE),
    (dict(vh=-64), SHAPE), (dict(qh=32), SHAPE), (dict(h_q=-1), SHAPE), (dict(k=None), NULL), (dict(v=None), NULL), (dict(q=None), NULL),
    (dict(q_out=None), NULL), (dict(start=None), NULL), (dict(q=addr(10) + 2), ALIGN), (dict(q_out=addr(11) + 8), ALIGN),
    (dict(start=addr(8) + 1), ALIGN), (dict(cu=None), SHAPE), (dict(k=addr(1) + 1024), ALIAS), (dict(q=addr(2)), ALIAS), (dict(q_out=addr(1)), ALIAS),
    (dict(q_out=addr(5)), ALIAS), (dict(q_out=addr(6)), ALIAS), (dict(q_out=addr(10)), ALIAS), (dict(q_out=addr(23)), ALIAS), (dict(start=addr(1)), ALIAS),
])
def test_append_refusals(lib, over, status):
    assert append(lib, **over) == status


def test_append_aliases_of_the_rotation(lib):
    assert append(lib, None, norm(freq=addr(1))) == ALIAS
    assert append(lib, None, norm(k_weight=addr(2) + 64)) == ALIAS
    assert append(lib, cache(store=gdn.GDN_FP8, k_scale=addr(23))) == ALIAS
    assert append(lib, cache(v=addr(1) + 1024)) == ALIAS


def test_append_without_work(lib):
    assert append(lib, cache(n=0), total=0, k=None, v=None, q=None, q_out=None, start=None) == OK
    assert append(lib, total=0, k=None, v=None, q=None, q_out=None) == OK
    assert append(lib, cache(num_pages=0, k=None, v=None), h_q=0, q=None, q_out=None) == OK
    assert append(lib, cache(max_pages=0, page_table=None), h_q=0, q=None, q_out=None, qt=0, qh=0) == OK


def dims(**over):
    a = dict(total_q=10, max_q=8, max_len=64, window=0, sinks=0, h_q=4, dtype=gdn.GDN_BF16, scale=0.1, q_token=256, q_head=64)
    a.update(over)
    return gdn.ExtendDims(*[a[f] for f, _ in gdn.ExtendDims._fields_])


def extend(lib, c=None, q=addr(6), cu=addr(7), lens=addr(8), out=addr(9), lse=None, ws=None, ws_bytes=0, **over):
    c = cache() if c is None else c
    d = dims(**over)
    return lib.gdn_attn_extend(ctypes.byref(c), ctypes.byref(d), q, cu, lens, out, lse, ws, ws_bytes, None)


@pytest.mark.parametrize("over,status", [
    (dict(total_q=-1), SHAPE), (dict(max_q=-1), SHAPE), (dict(max_len=-1), SHAPE), (dict(window=-1), SHAPE), (dict(sinks=-1), SHAPE),
    (dict(h_q=3), SHAPE), (dict(h_q=0), SHAPE), (dict(scale=float("nan")), SHAPE), (dict(scale=3e38), SHAPE), (dict(total_q=1 << 31), SHAPE),
    (dict(total_q=1 << 30), SHAPE), (dict(dtype=gdn.GDN_F32), UNSUP), (dict(q_token=100), SHAPE), (dict(q_head=4), SHAPE), (dict(q=None), NULL),
    (dict(lens=None), NULL), (dict(out=None), NULL), (dict(q=addr(6) + 4), ALIGN), (dict(lens=addr(8) + 2), ALIGN), (dict(cu=addr(7) + 2), ALIGN),
    (dict(lse=addr(10) + 1), ALIGN), (dict(ws=addr(10) + 4), ALIGN), (dict(out=addr(6)), ALIAS), (dict(out=addr(1)), ALIAS), (dict(lse=addr(9)), ALIAS),
    (dict(lse=addr(5)), ALIAS), (dict(out=addr(7)), ALIAS), (dict(out=addr(8)), ALIAS), (dict(cu=None), SHAPE), (dict(cu=None, total_q=2, max_q=2), SHAPE),
    (dict(cu=None, total_q=2, max_q=1, q=None), NULL),
])
def test_extend_refusals(lib, over, status):
    assert extend(lib, **over) == status


def test_extend_lengths(lib):
    """The kernels count positions in 32 bits and step past the end by less than 2^16."""
    c = cache(max_pages=(1 << 21) - 1, page_size=1024)
    assert extend(lib, c, max_len=(1 << 31) - (1 << 16)) == SHAPE
    assert extend(lib, c, max_len=1 << 40) == SHAPE
    assert extend(lib, c, max_len=(1 << 31) - (1 << 16) - 1) == WS


def test_extend_workspace(lib):
    c = cache(num_pages=1000, max_pages=400)
    of = lambda **over: lib.gdn_attn_extend_workspace_bytes(ctypes.byref(c), ctypes.byref(dims(**over)))
    need = of(max_len=6400)
    assert need > 0
    assert of(max_len=100) == 0  # nothing to split
    assert of(max_len=6400, h_q=3) == 0 and of(max_len=6400, total_q=0) == 0 and of(max_len=6400, max_q=0) == 0
    assert of(max_len=1 << 40) == need  # max_len beyond the table asks for no more than the table does
    assert of(max_len=6400, window=6400) == need and of(max_len=6400, window=10, sinks=1 << 50) == need
    assert of(max_len=6400, window=100) == 0
    assert lib.gdn_attn_extend_workspace_bytes(None, ctypes.byref(dims())) == 0
    assert lib.gdn_attn_extend_workspace_bytes(ctypes.byref(c), None) == 0
    assert extend(lib, c, max_len=6400) == WS
    assert extend(lib, c, max_len=6400, ws=addr(11), ws_bytes=need - 1) == WS
    assert extend(lib, c, max_len=6400, ws=addr(11) + 8, ws_bytes=need) == ALIGN
    for i in (9, 1, 6, 7, 8):
        assert extend(lib, c, max_len=6400, ws=addr(i), ws_bytes=need) == ALIAS


def test_extend_without_work(lib):
    assert extend(lib, cache(n=0, page_table=None, max_pages=0), q=None, lens=None, out=None) == OK
    assert extend(lib, total_q=0, q=None, out=None, lens=None) == OK
    assert extend(lib, max_q=0, q=None, out=None) == OK
    assert lib.gdn_attn_extend(None, ctypes.byref(dims()), None, None, None, None, None, None, 0, None) == NULL
    c = cache()
    assert lib.gdn_attn_extend(ctypes.byref(c), None, None, None, None, None, None, None, 0, None) == NULL


def test_binding_rejects_cpu_tensors():
    z = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    pool = torch.zeros(3, 2, 16, 64, dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    for call in (lambda: gdn.gdn_qk_norm_rope(z, z), lambda: gdn.gdn_kv_append(z, z, pool, pool, i[:, None], i, i),
                 lambda: gdn.gdn_attn_extend(z, pool, pool, i[:, None], i, i), lambda: gdn.gdn_qk_norm_rope(z.tolist())):
        with pytest.raises(ValueError):
            call()


def test_workspace_sizes_stay_reasonable(lib):
    """Over random sizes: no overflow, and never more than a sixteenth of the chip's memory for what is divided."""
    rng = random.Random(5)
    size = lambda top: int(2 ** rng.uniform(0, top))
    seen = 0
    for _ in range(20000):
        hk, g, n, d = rng.choice([1, 2, 3, 8]), rng.choice([1, 3, 8, 16, 20]), size(9), rng.choice([64, 128, 256])
        f32, total = rng.random() < 0.4, size(16)
        dtype = torch.float32 if f32 else torch.bfloat16
        need = gdn.gdn_attn_extend_workspace_bytes(
            n, size(12), rng.choice([16, 64, 1024]), total, hk * g, hk, d, max_q=rng.choice([1, size(10), total]),
            max_len=size(22), window=rng.choice([0, size(14)]), sinks=size(8), dtype=dtype,
            store=rng.choice([dtype, torch.float8_e4m3fn]))
        assert 0 <= need <= 18 << 30
        seen += need > 0
    assert seen > 2000
