"""GPU: attention over packed prompts against a 64-bit evaluation (tests/attn_ref.py, which also
derives the error each element may have)."""
import math

import pytest
import torch

import attn_ref
import gated_deltanet_linear_prefill_amd as gdn

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def offsets(lens):
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    return cu


def make(lq, lk, hq, hk, d, dtype, seed=0, spread=1.5):
    g = torch.Generator().manual_seed(seed)
    q = (spread * torch.randn(sum(lq), hq, d, generator=g)).to(dtype)
    k = torch.randn(sum(lk), hk, d, generator=g).to(dtype)
    v = torch.randn(sum(lk), hk, d, generator=g).to(dtype)
    return q, k, v


def compare(q, k, v, lq, lk, causal, scale, out, lse, what=""):
    cq, ck, g = offsets(lq), offsets(lk), q.shape[1] // k.shape[1]
    for s in range(len(lq)):
        allowed = attn_ref.causal_mask(lq[s], lk[s], causal)
        for h in range(q.shape[1]):
            a, b = slice(cq[s], cq[s + 1]), slice(ck[s], ck[s + 1])
            ref = attn_ref.attend(q[a, h], k[b, h // g], v[b, h // g], scale, allowed)
            attn_ref.check(out[a, h], None if lse is None else lse[a, h], *ref, what=f"{what} sequence {s} head {h}")


def run(q, k, v, lq, lk, causal=True, scale=None, with_lse=True):
    lse = torch.full(q.shape[:2], 5.0, device=DEV) if with_lse else None
    out = gdn.gdn_attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), ints(offsets(lq)), ints(offsets(lk)), causal=causal,
                               scale=scale, lse=lse)
    return out, lse


SHAPES = [
    ([1], [1], 1, 1, 64), ([1], [1], 16, 2, 256), ([31], [31], 4, 4, 64), ([64], [64], 2, 1, 128),
    ([65], [65], 8, 1, 256), ([129], [129], 3, 1, 128), ([200], [200], 6, 2, 64),
    ([1, 2, 33, 127, 64], [1, 2, 33, 127, 64], 8, 2, 128),            # packed, ragged
    ([5, 0, 70], [300, 17, 70], 4, 2, 64),                             # context, an empty sequence
    ([17], [400], 16, 2, 256), ([1, 1, 1], [63, 64, 65], 16, 1, 128),  # few queries, long keys
    ([40, 9], [7, 0], 4, 2, 64),                                       # rows that see no key
    ([257], [257], 20, 1, 64), ([90], [90], 5, 5, 256),
]


@pytest.mark.parametrize("lq,lk,hq,hk,d", SHAPES)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("causal", [True, False])
def test_against_64_bits(lq, lk, hq, hk, d, dtype, causal):
    q, k, v = make(lq, lk, hq, hk, d, dtype, seed=len(lq) + d)
    out, lse = run(q, k, v, lq, lk, causal)
    compare(q, k, v, lq, lk, causal, d ** -0.5, out, lse)


# Few rows over many keys: the keys are divided over workgroups. Ragged, so that some sequences have
# fewer ranges than others, one or none; rows whose last keys lie in the middle of a range.
FEW = [([8], [5000], 8, 2, 64), ([1, 3, 0, 40], [3000, 700, 900, 41], 4, 2, 128), ([70], [2500], 16, 2, 256),
       ([2, 5, 30], [4100, 0, 20], 3, 1, 256), ([200, 1], [1700, 1900], 2, 2, 64), ([16, 16], [2049, 255], 6, 1, 128)]


@pytest.mark.parametrize("lq,lk,hq,hk,d", FEW)
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("causal", [True, False])
def test_few_rows_over_many_keys(lq, lk, hq, hk, d, dtype, causal):
    q, k, v = make(lq, lk, hq, hk, d, dtype, seed=d + len(lk))
    dims = gdn.AttnDims(len(lq), sum(lq), sum(lk), hq, hk, d, gdn.GDN_BF16 if dtype == BF else gdn.GDN_F32, int(causal),
                        d ** -0.5, hq * d, d, hk * d, d, hk * d, d)
    need = gdn._load().gdn_attn_prefill_workspace_bytes(dims)
    assert need > 0
    out, lse = run(q, k, v, lq, lk, causal)
    compare(q, k, v, lq, lk, causal, d ** -0.5, out, lse)
    # the same from run to run, also with a workspace that held something else, and without lse
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device=DEV)
    again = gdn.gdn_attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), ints(offsets(lq)), ints(offsets(lk)), causal=causal,
                                 workspace=ws)
    assert torch.equal(out, again)
    with pytest.raises(gdn.GdnError, match="WORKSPACE"):
        gdn.gdn_attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), ints(offsets(lq)), ints(offsets(lk)), causal=causal,
                             workspace=ws[:need - 1])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_few_rows_masked_values_and_large_scores(dtype):
    """NaN and infinities that a row may not see, in the range of its last keys, change nothing; the
    largest score in any of the ranges."""
    lq, lk, d = [6], [3000], 128
    for at in (0, 700, 2990):
        q, k, v = make(lq, lk, 2, 1, d, dtype, seed=at)
        k[at] *= 30.0
        out, lse = run(q, k, v, lq, lk)
        compare(q, k, v, lq, lk, True, d ** -0.5, out, lse, f"large at {at}")
        bad_k, bad_v = k.clone(), v.clone()
        bad_k[2998:], bad_v[2997:] = math.nan, math.inf
        bad, bad_lse = run(q, bad_k, bad_v, lq, lk)
        assert torch.equal(bad[:3], out[:3]) and torch.equal(bad_lse[:3], lse[:3])


def test_few_rows_in_a_graph():
    lq, lk, d = [9, 2], [4000, 1000], 128
    q, k, v = (x.to(DEV) for x in make(lq, lk, 4, 2, d, BF, seed=21))
    cq, ck = ints(offsets(lq)), ints(offsets(lk))
    out = torch.empty_like(q)
    call = lambda o: gdn.gdn_attn_prefill(q, k, v, cq, ck, out=o)
    call(out)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        call(out)
    for step in range(4):
        q.mul_(1.0 + 0.1 * step)
        want = torch.empty_like(q)
        call(want)
        torch.cuda.synchronize()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want), step


@pytest.mark.parametrize("dtype,d,n", [(BF, 128, 1500), (BF, 256, 700), (BF, 64, 1100), (F32, 128, 300)])
def test_longer(dtype, d, n):
    lq = lk = [n]
    q, k, v = make(lq, lk, 2, 1, d, dtype, seed=3)
    out, lse = run(q, k, v, lq, lk)
    compare(q, k, v, lq, lk, True, d ** -0.5, out, lse)


def test_same_packing_and_no_lse():
    lq = [30, 50]
    q, k, v = make(lq, lq, 4, 2, 64, BF)
    out = gdn.gdn_attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), ints(offsets(lq)), scale=0.3)
    compare(q, k, v, lq, lq, True, 0.3, out, None)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale", [-0.1, 0.0, 3.0])
def test_scales_and_large_scores(dtype, scale):
    """Scores of hundreds, one key far above the rest late in the row, and a uniform row."""
    lq = [150]
    q, k, v = make(lq, lq, 2, 1, 64, dtype, spread=4.0)
    k[140] *= 20
    out, lse = run(q, k, v, lq, lq, True, scale)
    compare(q, k, v, lq, lq, True, scale, out, lse)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("layout", ["fused", "head_major"])
def test_strides(dtype, layout):
    lq, hq, hk, d = [37, 80], 6, 2, 64
    q, k, v = make(lq, lq, hq, hk, d, dtype)
    if layout == "fused":
        f = torch.cat([q, k, v], 1).to(DEV)
        a, b, c = f[:, :hq], f[:, hq:hq + hk], f[:, hq + hk:]
    else:
        a, b, c = (x.transpose(0, 1).contiguous().to(DEV).transpose(0, 1) for x in (q, k, v))
    assert not a.is_contiguous()
    out = gdn.gdn_attn_prefill(a, b, c, ints(offsets(lq)))
    compare(q, k, v, lq, lq, True, d ** -0.5, out, None)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_masked_keys_may_hold_anything(dtype, d, bad):
    """NaN and infinities in keys and values that a row does not see leave the row as it is; the
    neighbours of a sequence in the packing are such rows too."""
    lq, lk, hq, hk = [70, 50], [70, 90], 4, 2
    q, k, v = make(lq, lk, hq, hk, d, dtype)
    k[40], v[45, :, 3] = bad, bad           # seen by rows 40.. and 45.. of sequence 0 only
    v[69] = bad                             # the last key of sequence 0
    k[70 + 89], v[70 + 60] = math.nan, bad  # sequence 1: seen by its last row, by rows 20..
    out, _ = run(q, k, v, lq, lk, True, None, False)
    # rows that see nothing bad
    cq, ck, g = offsets(lq), offsets(lk), hq // hk
    for s, rows in ((0, 40), (1, 20)):
        allowed = attn_ref.causal_mask(lq[s], lk[s], True)[:rows]
        for h in range(hq):
            b = slice(ck[s], ck[s + 1])
            kk, vv = k[b, h // g].clone(), v[b, h // g].clone()
            kk[~allowed.any(0)], vv[~allowed.any(0)] = 0, 0
            ref = attn_ref.attend(q[cq[s]:cq[s] + rows, h], kk, vv, d ** -0.5, allowed)
            attn_ref.check(out[cq[s]:cq[s] + rows, h], None, *ref, what=f"{s} {h}")
    # and what a row does see reaches it
    assert bool(torch.isnan(out[69].float()).all())
    x = out[45:69, :, 3].float()
    assert not bool(torch.isfinite(x).any())


def test_rows_of_no_sequence_stay():
    lq = [20, 33]
    q, k, v = make(lq, lq, 4, 2, 128, BF)
    pad = torch.zeros(7, 4, 128, dtype=BF)
    qq = torch.cat([pad, q, pad]).to(DEV)
    out = torch.full(qq.shape, 9.0, dtype=BF, device=DEV)
    lse = torch.full(qq.shape[:2], 9.0, device=DEV)
    gdn.gdn_attn_prefill(qq, k.to(DEV), v.to(DEV), ints([7, 27, 60]), ints(offsets(lq)), out=out, lse=lse)
    assert bool((out[:7] == 9).all()) and bool((out[60:] == 9).all()) and bool((lse[60:] == 9).all())
    compare(q, k, v, lq, lq, True, 128 ** -0.5, out[7:60], lse[7:60])


def test_offsets_out_of_range_are_clamped():
    """Offsets that do not fit the tensors: nothing outside them is read or written."""
    q, k, v = make([64], [64], 4, 2, 64, BF)
    big = torch.full((128, 4, 64), 9.0, dtype=BF, device=DEV)
    out = big[32:96]
    for cu in ([0, 1000], [-50, 64], [60, 3], [2 ** 31 - 1, 2 ** 31 - 1], [-2 ** 31, 2 ** 31 - 1]):
        gdn.gdn_attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), ints(cu), ints([0, 64]), out=out)
        torch.cuda.synchronize()
        assert bool((big[:32] == 9).all()) and bool((big[96:] == 9).all())


def test_the_same_twice_and_on_another_stream():
    lq = [300, 41]
    q, k, v = (x.to(DEV) for x in make(lq, lq, 16, 2, 128, BF))
    cu = ints(offsets(lq))
    a = gdn.gdn_attn_prefill(q, k, v, cu)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b = gdn.gdn_attn_prefill(q, k, v, cu)
    s.synchronize()
    assert torch.equal(a, b)


def test_empty_calls():
    z = torch.empty(0, 4, 64, dtype=BF, device=DEV)
    assert gdn.gdn_attn_prefill(z, z, z, ints([0, 0])).shape == (0, 4, 64)
    assert gdn.gdn_attn_prefill(z, z, z, ints([0])).shape == (0, 4, 64)
    q = torch.ones(3, 4, 64, dtype=BF, device=DEV)
    lse = torch.zeros(3, 4, device=DEV)
    out = gdn.gdn_attn_prefill(q, z, z, ints([0, 3]), ints([0, 0]), lse=lse)
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())


def test_refusals():
    q, k, v = (x.to(DEV) for x in make([20], [20], 4, 2, 64, BF))
    cu = ints([0, 20])
    out = torch.full((20, 4, 64), 7.0, dtype=BF, device=DEV)
    for over in (dict(q=q.float()), dict(k=k.cpu()), dict(v=v[:19]), dict(q=q[..., ::2]), dict(q=q.half()),
                 dict(cu_q=cu.long()), dict(cu_k=ints([0, 5, 20])), dict(cu_q=cu.cpu()), dict(k=k[0]),
                 dict(lse=torch.zeros(20, 3, device=DEV)), dict(out=out[:19]), dict(out=out.float())):
        a = dict(q=q, k=k, v=v, cu_q=cu, cu_k=cu, out=out)
        a.update(over)
        with pytest.raises(ValueError):
            gdn.gdn_attn_prefill(**a)
    for over, name in ((dict(q=q[:, :3], out=None), "SHAPE"), (dict(scale=math.inf), "SHAPE"), (dict(out=q), "ALIAS"),
                       (dict(q=q[..., :32], k=k[..., :32], v=v[..., :32], out=None), "UNSUPPORTED"),
                       (dict(q=q.expand(20, 4, 64)[:, :1].expand(20, 4, 64)), "SHAPE")):
        a = dict(q=q, k=k, v=v, cu_q=cu, cu_k=cu, out=out)
        a.update(over)
        with pytest.raises(gdn.GdnError, match=name):
            gdn.gdn_attn_prefill(**a)
    torch.cuda.synchronize()
    assert bool((out == 7).all())
