"""GPU: a packed call's lookup of sequences does not walk the empty ones. A batch of slots of which few
have new tokens is an ordinary one for a server; the lookup is logarithmic in the slots."""
import pytest
import torch

import gated_deltanet_linear_prefill_amd as gdn
from test_gpu_kv_cache import BF, DEV, ints

pytestmark = pytest.mark.gpu

N = 1 << 18


def slots(full):
    """Offsets of N sequences of which those in `full` have one token."""
    one = torch.zeros(N, dtype=torch.int32)
    one[full] = 1
    return torch.cat([torch.zeros(1, dtype=torch.int32), one.cumsum(0, dtype=torch.int32)]).to(DEV)


def seconds(call):
    call()
    times = []
    for _ in range(5):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        call()
        b.record()
        b.synchronize()
        times.append(a.elapsed_time(b) * 1e-3)
    return min(times)


@pytest.mark.parametrize("full", [[0, N - 1], [5, 6, 70000, 70001, 200000, N - 2], list(range(1, N, 40000)),
                                  [N // 2], list(range(63, 64 * 40, 64))])
def test_rows_around_empty_sequences(full):
    """The right rows, and no more time than where the same tokens lie in neighbouring sequences."""
    h, d, page = 1, 64, 16
    g = torch.Generator().manual_seed(1)
    total = len(full)
    k, v = (torch.randn(total, h, d, generator=g).to(BF).to(DEV) for _ in range(2))
    table = torch.full((N, 1), -1, dtype=torch.int32)
    table[full, 0] = torch.arange(total, dtype=torch.int32)
    table = table.to(DEV)
    start = torch.full((N,), 7, dtype=torch.int32, device=DEV)
    kc, vc = (torch.zeros(total, h, page, d, dtype=BF, device=DEV) for _ in range(2))
    cu = slots(full)
    write = lambda at: gdn.gdn_kv_write(k, v, kc, vc, table, start, at)
    write(cu)
    assert torch.equal(kc[:, :, 7], k) and torch.equal(vc[:, :, 7], v)
    assert int((kc != 0).any(-1).sum()) == total  # and nothing else
    ko, vo = gdn.gdn_kv_read(kc, vc, table, start, cu, total)
    assert torch.equal(ko, k) and torch.equal(vo, v)
    near = slots(list(range(total)))
    slow, quick = seconds(lambda: write(cu)), seconds(lambda: write(near))
    # a walk over the empty sequences takes tens of milliseconds; the lookup some microseconds
    assert slow < 20 * quick + 5e-4, (slow, quick)


def test_random_slots():
    """Random lengths with many zeros: every row goes to its own sequence."""
    g = torch.Generator().manual_seed(3)
    n = 5000
    lens = torch.randint(0, 40, (n,), generator=g) * (torch.rand(n, generator=g) < 0.02)
    cu = torch.cat([torch.zeros(1, dtype=torch.int64), lens.cumsum(0)]).to(torch.int32)
    total = int(cu[-1])
    assert total > 500
    k, v = (torch.randn(total, 2, 64, generator=g).to(BF) for _ in range(2))
    pages = int(((lens + 15) // 16).sum())
    table = torch.full((n, 3), -1, dtype=torch.int32)
    at = 0
    for s in torch.nonzero(lens)[:, 0].tolist():
        for x in range(-(-int(lens[s]) // 16)):
            table[s, x] = at
            at += 1
    assert at == pages
    kc, vc = (torch.zeros(pages, 2, 16, 64, dtype=BF, device=DEV) for _ in range(2))
    args = kc, vc, table.to(DEV), ints([0] * n)
    gdn.gdn_kv_write(k.to(DEV), v.to(DEV), *args, cu.to(DEV))
    seq = torch.repeat_interleave(torch.arange(n), lens)
    pos = torch.arange(total) - cu[:-1].long()[seq]
    where = table[seq, pos // 16].long(), pos % 16
    assert torch.equal(kc.cpu()[where[0], :, where[1]], k) and torch.equal(vc.cpu()[where[0], :, where[1]], v)
    ko, vo = gdn.gdn_kv_read(*args, cu.to(DEV), total)
    assert torch.equal(ko.cpu(), k) and torch.equal(vo.cpu(), v)
