"""GPU: norms and rotary positions of queries and keys against a 64-bit evaluation
(tests/rope_ref.py)."""
import math

import pytest
import torch

import gated_deltanet_linear_prefill_amd as gdn
import rope_ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def rows(total, h, d, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(total, h, d, generator=g) * torch.exp(torch.randn(total, h, 1, generator=g))).to(dtype)


def weights(d, dtype, seed):
    return (0.3 * torch.randn(d, generator=torch.Generator().manual_seed(seed))).to(dtype)


def freqs(rot, base=1e6):
    half = rot // 2
    return (base ** (-torch.arange(half, dtype=torch.float64) / half)).float()


def positions(axes, total, seed, top=200000):
    return torch.randint(0, top, (axes, total), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)


def per_pair(pos, axis, half):
    """[total, half]: the position that each pair turns by."""
    a = torch.zeros(half, dtype=torch.long) if axis is None else axis.long().clamp(max=pos.shape[0] - 1)
    return pos[a].t()


def dev(x):
    return None if x is None else x.to(DEV)


def compare(q, k, pos, freq=None, axis=None, inter=False, scale=1.0, wq=None, wk=None, bias=0.0, eps=1e-6, qd=None, kd=None):
    p = None if pos is None else (pos[0] if pos.shape[0] == 1 and axis is None else pos)
    qo, ko = gdn.gdn_qk_norm_rope(dev(q) if qd is None else qd, dev(k) if kd is None else kd, dev(p), freq=dev(freq),
                                  axis=dev(axis), interleaved=inter, rope_scale=scale, q_weight=dev(wq), k_weight=dev(wk),
                                  weight_bias=bias, eps=eps)
    at = None if freq is None else per_pair(pos, axis, freq.shape[0])
    for name, x, w, out in (("q", q, wq, qo), ("k", k, wk, ko)):
        if x is not None:
            assert out.shape == x.shape and out.dtype == x.dtype and out.is_contiguous()
            rope_ref.check(out, *rope_ref.norm_rope(x, w, bias, eps, freq, at, inter, scale), what=name)
    return qo, ko


CASES = [  # total, h_q, h_kv, d, rot, axes, interleaved, norm, dtype
    (1, 1, 1, 64, 16, 1, False, True, BF), (1, 16, 2, 256, 64, 1, False, True, BF), (5, 6, 3, 64, 48, 2, True, False, F32),
    (77, 8, 1, 128, 128, 3, False, True, BF), (33, 3, 3, 128, 112, 3, True, True, F32), (130, 4, 2, 256, 240, 1, False, False, BF),
    (64, 2, 1, 256, 256, 4, False, True, F32), (257, 20, 1, 64, 64, 1, True, True, BF), (19, 5, 5, 256, 0, 1, False, True, BF),
    (3000, 1, 1, 64, 32, 1, False, True, BF), (40, 7, 1, 128, 16, 2, False, False, F32), (9, 40, 8, 128, 128, 1, False, True, BF),
]


@pytest.mark.parametrize("total,hq,hk,d,rot,axes,inter,norm,dtype", CASES)
def test_against_64_bits(total, hq, hk, d, rot, axes, inter, norm, dtype):
    q, k = rows(total, hq, d, dtype, 1), rows(total, hk, d, dtype, 2)
    freq = freqs(rot) if rot else None
    axis = (torch.arange(rot // 2) % axes).to(torch.uint8) if rot and axes > 1 else None
    pos = positions(axes, total, 3) if rot else None
    wq, wk = (weights(d, dtype, 4), weights(d, dtype, 5)) if norm else (None, None)
    compare(q, k, pos, freq, axis, inter, 1.0, wq, wk, 1.0)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_only_one_weight_and_only_queries(dtype):
    q, k = rows(21, 4, 128, dtype, 1), rows(21, 2, 128, dtype, 2)
    pos, freq = positions(1, 21, 3), freqs(64)
    compare(q, k, pos, freq, wq=weights(128, dtype, 4))
    compare(q, k, pos, freq, wk=weights(128, dtype, 4), bias=0.5, eps=0.1, scale=1.25)
    compare(q, None, pos, freq, wq=weights(128, dtype, 4), bias=1.0, scale=-0.5)


@pytest.mark.parametrize("layout", ["fused", "head_major"])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_strided_rows(layout, dtype):
    total, hq, hk, d = 37, 4, 2, 64
    q, k = rows(total, hq, d, dtype, 1), rows(total, hk, d, dtype, 2)
    if layout == "head_major":
        qd, kd = (x.transpose(0, 1).contiguous().to(DEV).transpose(0, 1) for x in (q, k))
    else:
        f = torch.full((total, 3 + hq + hk, d), math.nan, dtype=dtype, device=DEV)
        f[:, 3:3 + hq], f[:, 3 + hq:] = q.to(DEV), k.to(DEV)
        qd, kd = f[:, 3:3 + hq], f[:, 3 + hq:]
    assert not qd.is_contiguous()
    compare(q, k, positions(1, total, 3), freqs(32), None, False, 1.0, weights(d, dtype, 4), weights(d, dtype, 5), 1.0, qd=qd, kd=kd)


def test_far_positions_and_large_frequencies():
    """Angles of 2^31 and frequencies above a turn per position."""
    total = 64
    q = rows(total, 2, 64, F32, 1)
    pos = (torch.arange(total, dtype=torch.int64) * 0x2000001 + (1 << 30)).clamp(max=(1 << 31) - 1).to(torch.int32)[None]
    compare(q, None, pos, freqs(64))
    compare(q, None, -pos, freqs(64))
    compare(q, None, positions(1, total, 2, 5000), freqs(64) * 37.5)


def test_turns_that_are_known():
    """Position 0 leaves rows as they are; quarter turns exchange the elements of a pair."""
    q = rows(4, 1, 64, F32, 1)
    freq = torch.full((32,), math.pi / 2)
    out, _ = gdn.gdn_qk_norm_rope(q.to(DEV), None, torch.arange(4, dtype=torch.int32, device=DEV), freq=freq.to(DEV))
    a, b, o = q[..., :32], q[..., 32:], out.cpu()
    assert torch.equal(o[0], q[0])
    for t, (x, y) in ((1, (-b, a)), (2, (-a, -b)), (3, (b, -a))):
        # float32's pi / 2 is off by 4.4e-8, times up to 3
        tol = (a.abs() + b.abs()) * 2.0 ** -21
        assert bool(((o[t, :, :32] - x[t]).abs() <= tol[t]).all()) and bool(((o[t, :, 32:] - y[t]).abs() <= tol[t]).all())


@pytest.mark.parametrize("dtype", [BF, F32])
def test_norms_at_the_ends_of_the_range(dtype):
    """Squares past either end of fp32, rows of zeros, NaN and infinities."""
    d, fi = 128, torch.finfo(dtype)
    x = torch.randn(8, 1, d, generator=torch.Generator().manual_seed(1)).double()
    x[0] = x[0] / x[0].abs().max() * fi.max
    x[1] *= 1e30
    x[2] *= 1e-30
    x[3] = 0
    x[4, 0, 5] = math.nan
    x[5, 0, 100] = math.inf
    x[6] *= 1e-36
    q = x.to(dtype)
    w = weights(d, dtype, 2)
    compare(q[[0, 1, 2, 3, 4, 5, 7]], None, None, wq=w, bias=1.0)
    # eps far below the squares, and below 2^-100
    compare(q[[0, 1, 2, 6, 7]], None, None, wq=w, bias=1.0, eps=1e-38)
    compare(q[[0, 1, 2, 6, 7]], None, None, wq=w, bias=1.0, eps=0.0)


def test_nan_stays_in_its_pair_without_a_norm():
    q = rows(6, 2, 64, BF, 1)
    q[2, 1, 3] = math.nan
    out, _ = compare(q, None, positions(1, 6, 2), freqs(32))
    assert int(torch.isnan(out).sum()) == 2
    q[2, 1, 3] = 0
    q[4, 0, 50] = math.nan  # past the rotated elements
    out, _ = compare(q, None, positions(1, 6, 2), freqs(32))
    assert int(torch.isnan(out).sum()) == 1


def test_axes_past_the_last_count_as_the_last():
    q = rows(12, 1, 64, F32, 1)
    axis = torch.arange(16, dtype=torch.uint8) * 17
    compare(q, None, positions(3, 12, 2), freqs(32), axis)


def test_streams_outputs_and_repeats():
    """Given outputs, another stream, the same bits each time, nothing past the outputs."""
    total, hq, hk, d = 50, 4, 2, 128
    q, k = rows(total, hq, d, BF, 1).to(DEV), rows(total, hk, d, BF, 2).to(DEV)
    pos, freq, w = positions(1, total, 3)[0].to(DEV), freqs(64).to(DEV), weights(d, BF, 4).to(DEV)
    kw = dict(freq=freq, q_weight=w, k_weight=w, weight_bias=1.0)
    ref = gdn.gdn_qk_norm_rope(q, k, pos, **kw)
    big = [torch.full((total + 2, h, d), 7.0, dtype=BF, device=DEV) for h in (hq, hk)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = gdn.gdn_qk_norm_rope(q, k, pos, q_out=big[0][1:-1], k_out=big[1][1:-1], stream=s, **kw)
    new = gdn.gdn_qk_norm_rope(q, k, pos, stream=s, **kw)
    s.synchronize()
    for a, b, c, f in zip(ref, out, new, big):
        assert torch.equal(a, b) and torch.equal(a, c)
        assert bool((f[0] == 7.0).all()) and bool((f[-1] == 7.0).all())


def test_captured_and_replayed():
    total, d = 40, 256
    q, k = rows(total, 4, d, BF, 1).to(DEV), rows(total, 2, d, BF, 2).to(DEV)
    pos, freq, w = positions(1, total, 3)[0].to(DEV), freqs(64).to(DEV), weights(d, BF, 4).to(DEV)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    call = lambda: gdn.gdn_qk_norm_rope(q, k, pos, freq=freq, q_weight=w, k_weight=w, q_out=qo, k_out=ko)
    call()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for i in range(3):
        q.mul_(1.5)
        pos.add_(7)
        g.replay()
        torch.cuda.synchronize()
        a, b = gdn.gdn_qk_norm_rope(q, k, pos, freq=freq, q_weight=w, k_weight=w)
        assert torch.equal(a, qo) and torch.equal(b, ko), i


def test_empty_and_refusals():
    q = torch.zeros(0, 2, 64, dtype=BF, device=DEV)
    a, b = gdn.gdn_qk_norm_rope(q, q, torch.zeros(0, dtype=torch.int32, device=DEV), freq=freqs(32).to(DEV))
    assert a.shape == q.shape and b.shape == q.shape
    x = rows(4, 2, 64, BF, 1).to(DEV)
    pos, freq, w = torch.zeros(4, dtype=torch.int32, device=DEV), freqs(32).to(DEV), weights(64, BF, 1).to(DEV)
    bad = [dict(positions=None), dict(positions=pos.long()), dict(positions=pos[:3]), dict(freq=freq.double()),
           dict(freq=freq.cpu()), dict(freq=None), dict(axis=pos), dict(q_weight=w.float()), dict(k_weight=w[:32]),
           dict(q=x.half()), dict(q=x.transpose(1, 2)), dict(k=x[:3]), dict(q_out=x[:, :1]), dict(k=None, k_out=x)]
    for over in bad:
        a = dict(q=x, k=x, positions=pos, freq=freq)
        a.update(over)
        with pytest.raises(ValueError):
            gdn.gdn_qk_norm_rope(**a)
    for over, what in ((dict(freq=freqs(24).to(DEV)), "SHAPE"), (dict(freq=freqs(80).to(DEV)), "SHAPE"), (dict(eps=-1.0), "SHAPE"),
                       (dict(rope_scale=math.inf), "SHAPE"), (dict(weight_bias=math.nan), "SHAPE"), (dict(q_out=x), "ALIAS"),
                       (dict(positions=torch.zeros(5, 4, dtype=torch.int32, device=DEV)), "SHAPE")):
        a = dict(q=x, k=x, positions=pos, freq=freq)
        a.update(over)
        with pytest.raises(gdn.GdnError) as e:
            gdn.gdn_qk_norm_rope(**a)
        assert gdn.gdn_status_str(e.value.status) == str(e.value).split(": ", 1)[1]
        assert e.value.status == {"SHAPE": 2, "ALIAS": 5}[what]


def test_many_tokens():
    """Several tokens a workgroup, and a last one that is not full."""
    total = 40001
    q, k = rows(total, 2, 64, BF, 1), rows(total, 1, 64, BF, 2)
    compare(q, k, positions(3, total, 3), freqs(64), (torch.arange(32) * 3 // 32).to(torch.uint8), False, 1.0,
            weights(64, BF, 4), weights(64, BF, 5), 1.0)
