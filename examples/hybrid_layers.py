"""One recurrent layer and one attention layer of a hybrid stack, side by side, through a prompt in
segments and then token by token -- the way the library's entry points are used together.

    python examples/hybrid_layers.py [--tokens 4096] [--segment 1024] [--steps 8] [--store fp8|bf16]
                                     [--attention apart|joined]

Projections and MLPs are left out: each layer gets its own random q, k, v (and gates), as
its projections would give them. Per segment of the prompt:
  recurrent layer   gdn_prefill, its state carried from segment to segment
  attention layer   gdn_kv_write puts the segment's K and V into the paged cache (quantised as
                    they are written), gdn_kv_read hands back the context so far, and
                    gdn_attn_prefill attends from the segment's queries to all of it
and per generated token:
  recurrent layer   gdn_decode_step, the state updated in place
  attention layer   gdn_kv_write appends the token, gdn_attn_decode attends over the cache

With --attention joined the attention layer also norms its queries and keys for each head and turns
them to their positions, and reads the cache where it is, both per segment and per token:
  gdn_kv_append     norms and rotates K and Q, and puts K and V into the cache
  gdn_attn_extend   attends from the new tokens to all of the cache

At the end the segmented run is compared with the whole prompt in one call of each layer.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gated_deltanet_linear_prefill_amd as gdn  # noqa: E402
import gdn_inputs  # noqa: E402

H_Q, H_KV, D, PAGE = 16, 2, 256, 64  # the attention layer's heads; the recurrent layer has 16/32 of 128


def ints(x, dev):
    return torch.tensor(x, dtype=torch.int32, device=dev)


class PagedCache:
    """The pools and page table of one sequence, as a serving program would keep them."""

    def __init__(self, capacity, store, dev, gen):
        pages = -(-capacity // PAGE)
        dtype = torch.float8_e4m3fn if store == "fp8" else torch.bfloat16
        self.k, self.v = (torch.empty(pages, H_KV, PAGE, D, dtype=dtype, device=dev) for _ in range(2))
        self.scales = {}
        if store == "fp8":
            self.scales = {name: torch.empty(pages, H_KV, PAGE, dtype=torch.uint8, device=dev)
                           for name in ("k_scale", "v_scale")}
        self.table = torch.randperm(pages, generator=gen, device=dev).to(torch.int32)[None].contiguous()

    def args(self):
        return self.k, self.v, self.table


def rotation(dev):
    """Norm weights of d, and angles per token of the first quarter of a head's elements."""
    ramp = torch.linspace(-0.5, 0.5, D, device=dev).to(torch.bfloat16)
    freq = 1e4 ** (-torch.arange(0, D // 4, 2, device=dev, dtype=torch.float64) / (D // 4))
    return {"freq": freq.float(), "q_weight": ramp, "k_weight": -ramp, "weight_bias": 1.0}


def run(tokens=4096, segment=1024, steps=8, store="fp8", device="cuda", attention="apart"):
    """Returns the differences from the whole-prompt outputs, relative to them (2-norms)."""
    if attention not in ("apart", "joined"):
        raise ValueError('attention must be "apart" or "joined"')
    dev = torch.device(device)
    gen = torch.Generator(device=dev)
    gen.manual_seed(1)
    total = tokens + steps
    rec = gdn_inputs.make_case(gdn_inputs.Shape(1, total, 16, 32, 128), seed=2, device=dev)
    normal = lambda h: torch.randn(total, h, D, generator=gen, device=dev).to(torch.bfloat16)
    q, k, v = normal(H_Q), normal(H_KV), normal(H_KV)
    part = lambda a, b: {x: rec[x][:, a:b].contiguous() for x in ("q", "k", "v", "g", "beta")}

    cache = PagedCache(total, store, dev, gen)
    rope = rotation(dev)

    def joined(a, b):
        """Tokens a to b - 1 of the attention layer, whatever their number."""
        at, cu = ints([a], dev), ints([0, b - a], dev)
        qn = gdn.gdn_kv_append(k[a:b], v[a:b], *cache.args(), at, cu, q=q[a:b], **rope, **cache.scales)
        return gdn.gdn_attn_extend(qn, *cache.args(), ints([b], dev), cu, max_q=b - a, max_len=b, **cache.scales)

    rec_out, att_out, state = [], [], None
    for a in range(0, tokens, segment):
        b = min(a + segment, tokens)
        o, state = gdn.gdn_prefill(**part(a, b), state_in=state)
        rec_out.append(o[0])
        if attention == "joined":
            att_out.append(joined(a, b))
            continue
        gdn.gdn_kv_write(k[a:b], v[a:b], *cache.args(), ints([a], dev), ints([0, b - a], dev), **cache.scales)
        upto = ints([0, b], dev)
        kc, vc = gdn.gdn_kv_read(*cache.args(), ints([0], dev), upto, b, **cache.scales)
        att_out.append(gdn.gdn_attn_prefill(q[a:b], kc, vc, ints([0, b - a], dev), upto))
    for t in range(tokens, total):
        o, state = gdn.gdn_decode_step(**part(t, t + 1), state_in=state, state_out=state)
        rec_out.append(o[0])
        if attention == "joined":
            att_out.append(joined(t, t + 1))
            continue
        at = ints([t], dev)
        gdn.gdn_kv_write(k[t:t + 1], v[t:t + 1], *cache.args(), at, **cache.scales)
        att_out.append(gdn.gdn_attn_decode(q[t:t + 1], *cache.args(), at + 1, max_len=total, **cache.scales))

    whole_rec, whole_state = gdn.gdn_prefill(**part(0, total))
    # the same keys and values as the cache stands for, in one causal call
    kc, vc = gdn.gdn_kv_read(*cache.args(), ints([0], dev), ints([0, total], dev), total, **cache.scales)
    if attention == "joined":
        q, _ = gdn.gdn_qk_norm_rope(q, positions=torch.arange(total, dtype=torch.int32, device=dev), **rope)
    whole_att = gdn.gdn_attn_prefill(q, kc, vc, ints([0, total], dev))

    def off(x, y):
        x, y = x.float(), y.float()
        return float((x - y).norm() / y.norm())

    return {"recurrent": off(torch.cat(rec_out), whole_rec[0]), "state": off(state, whole_state),
            "attention": off(torch.cat(att_out), whole_att)}


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n\n")[0])
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--segment", type=int, default=1024)
    ap.add_argument("--steps", type=int, default=8)
    ap.add_argument("--store", choices=("fp8", "bf16"), default="fp8")
    ap.add_argument("--attention", choices=("apart", "joined"), default="apart")
    a = ap.parse_args()
    for name, x in run(a.tokens, a.segment, a.steps, a.store, attention=a.attention).items():
        print(f"{name:10s} segments and steps against the whole prompt: relative difference {x:.2e}")


if __name__ == "__main__":
    main()
