"""GPU: norms of rows down to the smallest numbers of their type, without an eps and with the smallest one."""
import pytest
import torch

import gated_deltanet_linear_prefill_amd as gdn
import rope_ref
from test_gpu_qk_norm_rope import BF, DEV, F32, weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("eps", [0.0, 2.0 ** -149, 2.0 ** -110])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_against_64_bits(dtype, d, eps):
    least = 2.0 ** (-149 if dtype == F32 else -133)
    whole = torch.randint(-3, 4, (8, 2, d), generator=torch.Generator().manual_seed(1)).double()
    whole[..., 0] = 1  # no row of zeros
    x = torch.stack([whole[i] * least * 2.0 ** (3 * i * i) for i in range(8)])  # to about 2^0
    x[0, 1] = 0
    x[0, 1, 7] = least
    q, w = x.to(dtype), weights(d, dtype, 2)
    assert torch.equal(q.double(), x)
    out, _ = gdn.gdn_qk_norm_rope(q.to(DEV), q_weight=w.to(DEV), weight_bias=1.0, eps=eps)
    assert bool(torch.isfinite(out).all())
    rope_ref.check(out, *rope_ref.norm_rope(q, w, 1.0, eps, None, None, False, 1.0), what=f"eps {eps}")
