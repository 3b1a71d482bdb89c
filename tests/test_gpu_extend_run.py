"""GPU: an attention layer served through the norm, rotation, append and attention calls together:
prompts in pieces beside single tokens and drafted ones, a window layer, and a captured decode step.

Each call's queries are checked against the 64-bit norm and rotation (tests/rope_ref.py), its outputs
against 64-bit attention (tests/attn_ref.py) from those queries over the rows that the cache stands for,
whose own writing tests/test_gpu_kv_append.py checks. The example's bar is that of its other path
(tests/test_gpu_hybrid_example.py): both of its runs see the same keys, values and queries."""
import importlib.util
import os

import pytest
import torch

import gated_deltanet_linear_prefill_amd as gdn
import rope_ref
from test_gpu_attn_decode import fill
from test_gpu_attn_extend import compare
from test_gpu_kv_cache import BF, DEV, F8, F32, Cache, ints, offsets

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Layer:
    """One attention layer, its cache, and the tokens that its projections would give."""

    def __init__(self, capacity, hq, h, d, rot, dtype, store, window=0, sinks=0, page=16):
        self.cache = Cache(capacity, page, h, d, store, seed=3)
        fill(self.cache, 3, nan_behind=[0] * len(capacity))
        g = torch.Generator().manual_seed(4)
        self.weights = {x: (0.2 * torch.randn(d, generator=g)).to(dtype) for x in ("q_weight", "k_weight")}
        self.freq = 1e4 ** (-torch.arange(rot // 2).float() / max(rot // 2, 1))
        self.hq, self.h, self.d, self.dtype, self.g = hq, h, d, dtype, g
        self.sight = dict(window=window, sinks=sinks)
        self.norm = dict(freq=self.freq.to(DEV), weight_bias=1.0, **{x: w.to(DEV) for x, w in self.weights.items()})

    def projection(self, total):
        """q, k and v as views of one product, [total, h_q + 2 h_kv, d]."""
        x = torch.randn(total, self.hq + 2 * self.h, self.d, generator=self.g).to(self.dtype)
        return x, x.to(DEV)

    def parts(self, x):
        return x[:, :self.hq], x[:, self.hq:self.hq + self.h], x[:, self.hq + self.h:]

    def call(self, x, start, lens, cu, out=None, q_out=None, **bounds):
        q, k, v = self.parts(x)
        qn = gdn.gdn_kv_append(k, v, *self.cache.args(), start, cu, q=q, q_out=q_out, **self.norm, **self.cache.scales())
        return qn, gdn.gdn_attn_extend(qn, *self.cache.args(), lens, cu, out=out, **self.sight, **bounds, **self.cache.scales())

    def check(self, x, qn, out, new, lens):
        pos = torch.cat([torch.arange(b - a, b) for a, b in zip(new, lens)])[:, None].expand(-1, self.freq.shape[0])
        q, bound = rope_ref.norm_rope(self.parts(x)[0], self.weights["q_weight"], 1.0, 1e-6, self.freq, pos, False, 1.0)
        rope_ref.check(qn, q, bound, "q")
        compare(self.cache, qn.cpu(), new, lens, out, None, self.d ** -0.5, **self.sight)


LAYERS = [  # h_q, h_kv, d, rot, dtype, store, window, sinks
    (16, 2, 256, 64, BF, BF, 0, 0), (8, 2, 128, 128, BF, F8, 0, 0), (8, 4, 64, 64, BF, BF, 60, 4), (4, 2, 128, 32, F32, F32, 0, 0), (6, 2, 256, 64, BF, F8, 100, 0),
]


@pytest.mark.parametrize("hq,h,d,rot,dtype,store,window,sinks", LAYERS)
def test_a_batch_is_served(hq, h, d, rot, dtype, store, window, sinks):
    """Four sequences: prompts in pieces, some waiting, some generating, one with drafted tokens of which
    a part is taken back (written again by the next call)."""
    layer = Layer([500, 160, 40, 300], hq, h, d, rot, dtype, store, window, sinks)
    length = [0, 0, 0, 0]
    for new, back in (([130, 40, 0, 1], 0), ([130, 1, 33, 1], 0), ([70, 1, 1, 200], 0), ([1, 5, 1, 1], 3), ([1, 5, 0, 1], 0), ([1, 1, 1, 1], 0)):
        start = list(length)
        length = [a + b for a, b in zip(length, new)]
        x, xd = layer.projection(sum(new))
        qn, out = layer.call(xd, ints(start), ints(length), ints(offsets(new)), max_q=max(new), max_len=max(length))
        layer.check(x, qn, out, new, length)
        length[1] -= back


@pytest.mark.parametrize("hq,h,d,rot,dtype,store,window,sinks", LAYERS)
def test_a_captured_decode_step(hq, h, d, rot, dtype, store, window, sinks):
    """The graph moves the lengths on by itself; its replays give the eager calls' bits, and eager work of
    the same layer runs between them."""
    runs = []
    for captured in (False, True):
        layer = Layer([400, 90, 20], hq, h, d, rot, dtype, store, window, sinks)
        fill(layer.cache, 5)
        lens = ints([380, 60, 0])
        steps = [layer.projection(3) for _ in range(6)]
        x, qn, out = steps[0][1].clone(), torch.empty(3, hq, d, dtype=dtype, device=DEV), torch.empty(3, hq, d, dtype=dtype, device=DEV)
        start = torch.empty_like(lens)

        def step():
            start.copy_(lens)
            lens.add_(1)
            layer.call(x, start, lens, None, out=out, q_out=qn, max_len=400)

        got = []
        if captured:
            step()  # what is allocated or loaded on first use
            lens.sub_(1)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
        for i, (host, dev) in enumerate(steps):
            x.copy_(dev)
            if captured and i % 3 != 2:
                graph.replay()
            else:
                step()
            if not captured:
                layer.check(host, qn, out, [1] * 3, [380 + i + 1, 60 + i + 1, i + 1])
            got.append((qn.clone(), out.clone()))
        runs.append(got)
    for a, b in zip(*runs):
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("tokens,segment,steps,store", [(700, 256, 3, "fp8"), (300, 128, 5, "bf16")])
def test_the_example(tokens, segment, steps, store):
    spec = importlib.util.spec_from_file_location("hybrid_layers", os.path.join(ROOT, "examples", "hybrid_layers.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    off = m.run(tokens, segment, steps, store, attention="joined")
    assert off["recurrent"] <= 1e-3 and off["state"] <= 1e-3, off
    assert off["attention"] <= 9e-3, off
