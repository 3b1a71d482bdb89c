"""GPU: attention of new tokens over the cache stays within its workspace where the offsets ask for more rows than
there are (tests/test_extend_parts_cpu.py replays which parts are written)."""
import pytest
import torch

import gated_deltanet_linear_prefill_amd as gdn
from test_gpu_attn_extend import BF, DEV, F32, F8, Cache, fill, ints, queries

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
