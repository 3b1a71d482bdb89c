"""One-token rows of the attention calls. torch gives a dimension of one entry any stride; the binding
hands the library one that every layout allows, so that a token taken out of a head-major tensor
is accepted however far its heads lie apart."""
import ctypes

import pytest
import torch

import attn_ref
import gated_deltanet_linear_prefill_amd as gdn

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("heads,tokens,d,at", [(16, 4096, 256, 5), (8, 4096, 128, 0), (1, 100, 64, 99), (3, 7, 64, 6)])
def test_strides_that_the_library_takes(heads, tokens, d, at):
    """On the CPU: the strides of x[:, t:t + 1] of a head-major x pass the library's checks."""
    x = torch.empty(heads, tokens, d, dtype=BF)[:, at:at + 1].transpose(0, 1)
    ptr, token, head = gdn._rows("x", x, BF, -1)
    assert ptr == x.data_ptr() and (heads == 1 or head == tokens * d)
    # the check of strides runs before anything else that this call gets wrong (no queries' pointer)
    dims = gdn.AttnDims(1, 1, 1, heads, heads, d, gdn.GDN_BF16, 1, 1.0, token, head, token, head, token, head)
    name = [None] * 8
    st = gdn._load().gdn_attn_prefill(ctypes.byref(dims), *name, 0, None)
    assert gdn.gdn_status_str(st) == gdn.gdn_status_str(1), gdn.gdn_status_str(st)  # 1: a null pointer


def test_rows_without_tokens():
    x = torch.empty(3, 8, 64, dtype=BF)[:, 4:4].transpose(0, 1)
    _, token, head = gdn._rows("x", x, BF, -1)
    dims = gdn.AttnDims(1, 0, 0, 3, 3, 64, gdn.GDN_BF16, 1, 1.0, token, head, token, head, token, head)
    assert gdn._load().gdn_attn_prefill(ctypes.byref(dims), *[None] * 8, 0, None) == 0


def far(heads, tokens, d, dtype, seed):
    """A head-major tensor on the GPU and one token of it as rows, with the same values dense."""
    whole = torch.zeros(heads, tokens, d, dtype=dtype, device=DEV)
    t = tokens // 2
    row = torch.randn(heads, d, generator=torch.Generator().manual_seed(seed)).to(dtype).to(DEV)
    whole[:, t] = row
    view = whole[:, t:t + 1].transpose(0, 1)
    assert view.shape == (1, heads, d) and not view.is_contiguous()
    return view, row[None].clone()


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
def test_one_token_of_head_major_tensors(dtype):
    """Written, attended to and attended from: the same as with dense rows, bit for bit."""
    hq, hk, tokens, d = 16, 2, 16384, 256
    q, qd = far(hq, tokens, d, dtype, 1)
    k, kd = far(hk, tokens, d, dtype, 2)
    v, vd = far(hk, tokens, d, dtype, 3)
    assert q.stride(1) * hq >= 1 << 22 and k.stride(1) * hk >= 1 << 22
    caches = []
    for a, b in ((k, v), (kd, vd)):
        kc, vc = (torch.zeros(4, hk, 16, d, dtype=dtype, device=DEV) for _ in range(2))
        table, at = ints([[2, 1, 3, 0]]), ints([33])
        gdn.gdn_kv_write(a, b, kc, vc, table, at)
        caches.append((kc, vc, table))
    assert torch.equal(caches[0][0], caches[1][0]) and torch.equal(caches[0][1], caches[1][1])
    assert bool((caches[0][0][3, :, 1] == kd[0]).all())
    a = gdn.gdn_attn_decode(q, *caches[0], ints([34]))
    b = gdn.gdn_attn_decode(qd, *caches[0], ints([34]))
    assert torch.equal(a, b)
    cu = ints([0, 1])
    a = gdn.gdn_attn_prefill(q, k, v, cu)
    assert torch.equal(a, gdn.gdn_attn_prefill(qd, kd, vd, cu))
    for h in range(hq):  # one key: its value
        x = slice(h // (hq // hk), h // (hq // hk) + 1)
        ref = attn_ref.attend(qd[0, h:h + 1].cpu(), kd[0, x].cpu(), vd[0, x].cpu(), d ** -0.5, torch.ones(1, 1, dtype=torch.bool))
        attn_ref.check(a[:, h], None, *ref, what=f"head {h}")
