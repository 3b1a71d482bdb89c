"""GPU: sizes within the stated limits whose launches hold 2^32 threads and more, which one grid
dimension does not."""
import pytest
import torch

import attn_ref
import gated_deltanet_linear_prefill_amd as gdn
from test_gpu_kv_cache import BF, DEV, ints

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _memory():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def test_decode_of_many_sequences():
    n, d, page = (1 << 24) + 5, 64, 16
    g = torch.Generator().manual_seed(1)
    kc, vc = (torch.randn(3, 1, page, d, generator=g).to(BF) for _ in range(2))
    at = [0, 1, 70000, (1 << 22) - 1, 1 << 22, (1 << 24) - 1, 1 << 24, n - 1]
    table = torch.zeros(n, 1, dtype=torch.int32, device=DEV)
    lens = torch.zeros(n, dtype=torch.int32, device=DEV)
    table[at, 0] = ints([x % 3 for x in range(len(at))])
    lens[at] = ints([1 + 2 * x for x in range(len(at))])
    q = torch.zeros(n, 1, d, dtype=BF, device=DEV)
    qs = torch.randn(len(at), 1, d, generator=g).to(BF)
    q[at] = qs.to(DEV)
    out = torch.full((n, 1, d), 3.0, dtype=BF, device=DEV)
    gdn.gdn_attn_decode(q, kc.to(DEV), vc.to(DEV), table, lens, out=out)
    got = out[at].clone()
    for x in range(len(at)):
        length = 1 + 2 * x
        ref = attn_ref.attend(qs[x], kc[x % 3, 0, :length], vc[x % 3, 0, :length], d ** -0.5, torch.ones(1, length, dtype=torch.bool))
        attn_ref.check(got[x], None, *ref, what=f"sequence {at[x]}")
    out[at] = 0
    assert not bool(out.any())


def test_prefill_of_many_sequences():
    n, h, d, total = (1 << 23) + 3, 2, 64, 41
    g = torch.Generator().manual_seed(2)
    q, k, v = (torch.randn(total, h, d, generator=g).to(BF) for _ in range(3))
    # 40 rows in the first sequence, one in the last
    cu = torch.full((n + 1,), 40, dtype=torch.int32, device=DEV)
    cu[0], cu[-1] = 0, total
    out = gdn.gdn_attn_prefill(q.to(DEV), k.to(DEV), v.to(DEV), cu)
    for x in range(h):
        ref = attn_ref.attend(q[:40, x], k[:40, x], v[:40, x], d ** -0.5, attn_ref.causal_mask(40, 40, True))
        attn_ref.check(out[:40, x], None, *ref, what=f"head {x}")
    assert torch.equal(out[40].cpu(), v[40])


def test_cache_rows_of_64_gib():
    """Packed rows of 64 GiB of K, of which the first and last few belong to sequences."""
    d, page, total = 256, 16, (1 << 27) + 9
    if torch.cuda.mem_get_info()[0] < 150 << 30:
        pytest.skip("needs 150 GiB of free memory")
    g = torch.Generator().manual_seed(3)
    rows = torch.randn(10, 1, d, generator=g).to(BF).to(DEV)
    x = torch.empty(total, 1, d, dtype=BF, device=DEV)
    x[:4], x[-6:] = rows[:4], rows[4:]
    kc, vc = (torch.zeros(2, 1, page, d, dtype=BF, device=DEV) for _ in range(2))
    # sequence 1 has the rows between, none of whose pages exist
    table, cu, start = ints([[0], [-1], [1]]), ints([0, 4, total - 6, total]), ints([2, 0, 9])
    gdn.gdn_kv_write(x, x, kc, vc, table, start, cu)
    want = torch.zeros(2, 1, page, d, dtype=BF, device=DEV)
    want[0, 0, 2:6], want[1, 0, 9:15] = rows[:4, 0], rows[4:, 0]
    assert torch.equal(kc, want) and torch.equal(vc, want)
    vo = torch.empty_like(x)
    gdn.gdn_kv_read(kc, vc, table, start, cu, total, k_out=x, v_out=vo)
    for y in (x, vo):
        assert torch.equal(y[:4], rows[:4]) and torch.equal(y[-6:], rows[4:])
        assert not bool(y[4:100000].any()) and not bool(y[-100000:-6].any())
