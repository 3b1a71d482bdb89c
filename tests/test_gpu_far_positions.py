"""GPU: sines and cosines of far positions, against the angle reduced in whole numbers.

A row of pairs (1, 0) without a norm comes back as (cos t, sin t). Of the error, the library's sincospi has 2 ulp
(2^-23 for values up to 1), the added term of the reduced angle's rest rounds once more (2^-25), and all else is
below 2^-40: less than 1.5 * 2^-23."""
import math
from fractions import Fraction

import pytest
import torch

import gated_deltanet_linear_prefill_amd as gdn

pytestmark = pytest.mark.gpu
DEV = "cuda"
PI = Fraction(31415926535897932384626433832795028841971693993751, 10 ** 49)
MOST = 1.5 * 2.0 ** -23


def exact(pos, freq):
    """(cos, sin) of pos * freq, the reduced angle exact to 1e-35."""
    t = Fraction(pos) * Fraction(freq) / (2 * PI)
    t = float(2 * PI * (t - round(t)))
    return math.cos(t), math.sin(t)


def draw(lo, hi, seed, axes=1, total=96):
    g = torch.Generator().manual_seed(seed)
    pos = torch.randint(lo, hi, (axes, total), generator=g, dtype=torch.int64).to(torch.int32)
    freq = torch.cat([torch.rand(24, generator=g) * 0.7 + 0.3, 1e4 ** -torch.rand(8, generator=g)])
    freq[0] = 1.0
    return pos, freq


def check(out, pos, freq):
    for t in range(pos.shape[-1]):
        for p in range(freq.shape[0]):
            c, s = exact(int(pos[t]), float(freq[p]))
            assert abs(float(out[t, p]) - c) <= MOST and abs(float(out[t, freq.shape[0] + p]) - s) <= MOST, (int(pos[t]), float(freq[p]))


@pytest.mark.parametrize("lo,hi", [(0, 5000), (1 << 23, 1 << 25), (1 << 30, (1 << 31) - 1), (-(1 << 31), -(1 << 30)), ((1 << 31) - 100, (1 << 31) - 1)])
def test_angles(lo, hi):
    pos, freq = draw(lo, hi, 1)
    x = torch.zeros(96, 1, 64)
    x[..., :32] = 1
    out, _ = gdn.gdn_qk_norm_rope(x.to(DEV), None, pos[0].to(DEV), freq=freq.to(DEV))
    check(out[:, 0].cpu(), pos[0], freq)


def test_angles_of_appended_keys():
    """Positions given and fp32 pages: the same angles on the way into the cache."""
    pos, freq = draw(1 << 30, (1 << 31) - 1, 2)
    x = torch.zeros(96, 1, 64, device=DEV)
    x[..., :32] = 1
    pool = torch.zeros(6, 1, 16, 64, device=DEV)
    table = torch.arange(6, dtype=torch.int32, device=DEV)[None].contiguous()
    at = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)
    gdn.gdn_kv_append(x, x, pool, pool.clone(), table, at(0), at(0, 96), positions=pos[0].to(DEV), freq=freq.to(DEV))
    check(pool.view(96, 64).cpu(), pos[0], freq)
