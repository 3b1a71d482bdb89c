"""GPU: attention of new tokens over the cache stays within its workspace where the offsets ask for more rows than
there are (tests/test_extend_parts_cpu.py replays which parts are written)."""
import random

import pytest
import torch

import gated_deltanet_linear_prefill_amd as gdn
from test_gpu_attn_extend import BF, DEV, F32, F8, Cache, fill, ints, offsets, queries
from test_gpu_extend_shapes import sampled

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("store,dtype", [(F32, F32), (BF, BF), (F8, BF)])
def test_overlapping_sequences_stay_in_the_workspace(store, dtype):
    """Every other sequence has all 128 rows, four times what the plan counts on."""
    lens, n, total = [128, 1, 128, 1, 7168, 1, 128, 1], 8, 128
    cache = Cache(lens, 16, 2, 256, store, extra_width=0)
    fill(cache, 4)
    q = queries(total, 16, 256, dtype).to(DEV)
    need = gdn.gdn_attn_extend_workspace_bytes(n, cache.page_table.shape[1], 16, total, 16, 2, 256, max_q=total, max_len=7168, dtype=dtype, store=store)
    assert need > 0
    room = torch.full((need + (8 << 20),), 7, dtype=torch.uint8, device=DEV)  # where parts past the end would lie
    for _ in range(2):
        gdn.gdn_attn_extend(q, *cache.args(), ints(lens), ints([0, 128] * 4 + [0]), max_q=total, max_len=7168, workspace=room[:need], **cache.scales())
    assert bool((room[need:] == 7).all())
    # the same buffers with offsets that are right
    cu = [0, 16, 16, 32, 32, 100, 100, 128, 128]
    out = gdn.gdn_attn_extend(q, *cache.args(), ints(lens), ints(cu), max_q=total, max_len=7168, workspace=room[:need], **cache.scales())
    new = gdn.gdn_attn_extend(q, *cache.args(), ints(lens), ints(cu), max_q=total, max_len=7168, **cache.scales())
    assert torch.equal(out, new) and bool((room[need:] == 7).all())


@pytest.mark.parametrize("store,dtype", [(F32, F32), (BF, BF), (F8, BF)])
@pytest.mark.parametrize("n,hq,hk,d", [(40, 8, 2, 128), (200, 4, 1, 256), (300, 8, 2, 64)])
def test_a_long_piece_among_many_tokens(n, hq, hk, d, store, dtype):
    """Tiles of many rows whose keys are divided, in a workspace of just the size that is asked for."""
    rng = random.Random(n)
    lens_q = [1] * n
    lens = [rng.randint(1, 60) for _ in range(n)]
    lens_q[n // 3], lens[n // 3] = 150, 9000
    lens_q[n // 2], lens[n // 2] = 70, 2500
    cache = Cache(lens, 16, hk, d, store, extra_width=0)
    fill(cache, 2, nan_behind=lens)
    q = queries(sum(lens_q), hq, d, dtype)
    need = gdn.gdn_attn_extend_workspace_bytes(n, cache.page_table.shape[1], 16, len(q), hq, hk, d, max_q=150, max_len=9000, dtype=dtype, store=store)
    assert need > 0
    room = torch.full((need + (8 << 20),), 7, dtype=torch.uint8, device=DEV)
    lse = torch.full(q.shape[:2], 5.0, device=DEV)
    out = gdn.gdn_attn_extend(q.to(DEV), *cache.args(), ints(lens), ints(offsets(lens_q)), max_q=150, max_len=9000, lse=lse, workspace=room[:need],
                              **cache.scales())
    sampled(cache, q, lens_q, lens, out, lse, 0, 0, rng, heads=1)
    assert bool((room[need:] == 7).all())


@pytest.mark.parametrize("store,dtype", [(F32, F32), (BF, BF), (F8, BF)])
def test_captured_with_other_lengths_later(store, dtype):
    """Two graphs that share a workspace, their offsets and lengths changed between replays: the divided tiles' rows move."""
    n, total, width = 12, 240, 500
    cache = Cache([8000] * n, 16, 2, 128, store, extra_width=0)
    fill(cache, 2)
    q = queries(total, 8, 128, dtype).to(DEV)
    need = gdn.gdn_attn_extend_workspace_bytes(n, width, 16, total, 8, 2, 128, max_q=200, max_len=8000, dtype=dtype, store=store)
    assert need > 0 and cache.page_table.shape[1] == width
    room = torch.empty(need, dtype=torch.uint8, device=DEV)
    cu, lens, outs, graphs = ints([0] * n + [total]), ints([8000] * n), [torch.empty_like(q) for _ in range(2)], []
    call = lambda out, **kw: gdn.gdn_attn_extend(q, *cache.args(), lens, cu, max_q=200, max_len=8000, out=out, **kw, **cache.scales())
    call(outs[0], workspace=room)
    torch.cuda.synchronize()
    for out in outs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call(out, workspace=room)
    rng = random.Random(3)
    for step in range(4):
        lens_q = [1] * n
        lens_q[rng.randrange(n)] += total - n - 30 - (step == 2) * 10
        lens_q[rng.randrange(n)] += 30
        cu.copy_(ints(offsets(lens_q)))
        lens.copy_(ints([max(m, rng.randint(1, 8000)) for m in lens_q]))
        for out, graph in zip(outs, graphs):
            out.fill_(3.0)
            graph.replay()
        torch.cuda.synchronize()
        new = call(torch.full_like(q, 3.0))
        assert torch.equal(outs[0], new) and torch.equal(outs[1], new), step
