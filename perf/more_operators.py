"""Performance cases of the operators around the attention layers: norms and rotary positions of
queries and keys, appending rotated keys and values to the paged cache, and attention of a chunk of
new tokens (or of one per sequence) over the cache, with a sliding window and first tokens that
stay visible.

Each case is one pass of one operator. `run` computes it either in its plain form (elementary
torch operations in 32 bits, angles in 64, rounded once at the end) or, with `own` set, through the
package's entry points. `exact` evaluates the definition in 64 bits.

The cache is that of perf/operators.py: a store is f32, bf16 or fp8 (e4m3 codes with one
power-of-two scale per token and KV head, kept as the biased exponent); position p of sequence s
lies in page page_table[s][p // page], row p % page; pages are in no particular order.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f32": 4, "fp8": 1}
EPS = 1e-6
# what no drawn case exceeds: about the largest listed ones' bytes and operations
MOST_BYTES, MOST_FLOPS, MOST_SCORES = 6.5e8, 5e11, 1 << 32


def listed():
    return [
        # Patches of a small image in 32 bits: two axes, no norm, odd sizes, neighbouring pairs.
        dict(name="norm_rope_small_f32", op="norm_rope", tokens=77, h_q=6, h_kv=3, d=64, rot=48, axes=2, pairs=True,
             norm=False, fused=False, dtype="f32"),
        # The 4096-token prompt of the benchmark at the source page's attention layout: a quarter of
        # each head is rotated; q and k are slices of the fused projection.
        dict(name="norm_rope_prompt", op="norm_rope", tokens=4096, h_q=16, h_kv=2, d=256, rot=64, axes=1, pairs=False,
             norm=True, fused=True, dtype="bf16"),
        # Packed prompts with video: whole heads rotated, positions in time, height and width.
        dict(name="norm_rope_video", op="norm_rope", tokens=30001, h_q=32, h_kv=8, d=128, rot=128, axes=3, pairs=False,
             norm=True, fused=True, dtype="bf16"),
        # A decode step of 64 sequences: queries normed and rotated, keys as well on the way into the cache.
        dict(name="append_step", op="append", n=64, lo=1, hi=1, start=8000, h_q=16, h_kv=2, d=256, page=64, rot=64,
             axes=1, pairs=False, norm=True, dtype="bf16", store="bf16"),
        # Prompts of very different lengths, packed, each after a context of its own: keys and values only.
        dict(name="append_packed", op="append", n=24, lo=1, hi=2600, start=1500, h_q=0, h_kv=8, d=128, page=16, rot=128,
             axes=1, pairs=False, norm=False, dtype="bf16", store="bf16"),
        # A long segment into an 8-bit cache, its queries too, and the keys and values read back.
        dict(name="append_read_fp8", op="append", n=1, lo=16384, hi=16384, start=40000, h_q=16, h_kv=2, d=256, page=64,
             rot=64, axes=3, pairs=False, norm=True, dtype="bf16", store="fp8"),
        # A few short 32-bit rows behind a window: the smallest attention call.
        dict(name="extend_small_f32", op="extend", n=3, lo=1, hi=5, context=300, window=100, sinks=4, h_q=4, h_kv=2,
             d=64, page=16, dtype="f32", store="f32"),
        # Drafted tokens of a served batch are checked, four a sequence.
        dict(name="extend_draft", op="extend", n=16, lo=4, hi=4, context=8192, window=0, sinks=0, h_q=32, h_kv=8,
             d=128, page=16, dtype="bf16", store="bf16"),
        # The next 512 tokens of a long prompt over an 8-bit cache.
        dict(name="extend_chunk_fp8", op="extend", n=1, lo=512, hi=512, context=32256, window=0, sinks=0, h_q=16, h_kv=2,
             d=256, page=64, dtype="bf16", store="fp8"),
        # A batch in which some sequences decode and some bring a piece of their prompt.
        dict(name="extend_mixed", op="extend", n=24, lo=1, hi=700, context=4096, window=0, sinks=0, h_q=32, h_kv=8,
             d=128, page=16, dtype="bf16", store="bf16"),
        # Half of a long prompt through a layer with a window, its first tokens in sight.
        dict(name="extend_window", op="extend", n=1, lo=8192, hi=8192, context=8192, window=4096, sinks=64, h_q=16,
             h_kv=2, d=128, page=64, dtype="bf16", store="bf16"),
        # A decode step of 32 sequences in such a layer.
        dict(name="extend_step_window", op="extend", n=32, lo=1, hi=1, context=16000, window=4096, sinks=4, h_q=16,
             h_kv=2, d=256, page=64, dtype="bf16", store="bf16"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["norm_rope", "append", "extend", "extend"])
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        d = rng.choice([64, 128, 256])
        h_kv = rng.choice([1, 2, 3, 4, 8])
        group = rng.choice([1, 2, 3, 4, 6, 8, 16])
        case = dict(op=op, h_q=h_kv * group, h_kv=h_kv, d=d, dtype=dtype)
        if op != "extend":
            case.update(rot=rng.choice([16, d // 4, 48, d // 2, d - 16, d]), axes=rng.choice([1, 1, 2, 3]),
                        pairs=rng.random() < 0.3, norm=rng.random() < 0.6)
        if op == "norm_rope":
            case.update(tokens=_log_int(rng, 1, 65536), fused=rng.random() < 0.7)
        else:
            store, page = rng.choice([dtype, "fp8"]), rng.choice([16, 32, 64, 128])
            n = _log_int(rng, 1, 64)
            case.update(n=n, page=page, store=store)
            if op == "append":
                hi = rng.choice([1, _log_int(rng, 1, 16384)])
                case.update(lo=rng.randint(1, hi), hi=hi, start=rng.choice([0, _log_int(rng, 1, 65536)]),
                            h_q=rng.choice([0, h_kv * group]))
                if n * (hi + case["start"]) * h_kv * d > 1 << 28:
                    continue
            else:
                hi = rng.choice([1, _log_int(rng, 1, 16), _log_int(rng, 1, 8192)])
                window = rng.choice([0, _log_int(rng, 1, 8192)])
                case.update(lo=rng.randint(1, hi), hi=hi, context=rng.choice([0, _log_int(rng, 1, 65536)]), window=window,
                            sinks=rng.choice([0, _log_int(rng, 1, 128)]) if window else 0)
                rows = hi + case["context"]
                if n * rows * h_kv * d > 1 << 28 or n * case["h_q"] * hi * rows > MOST_SCORES:
                    continue
        w = work(case)
        if w["bytes"] <= MOST_BYTES and w["flops"] <= MOST_FLOPS / (16 if dtype == "f32" else 1):
            return case


# ---------------------------------------------------------------- sizes

def _lens(case):
    """The sequences' new tokens: from lo to hi by a fixed law, so that work(case) and prepare(case)
    agree; the first is the longest."""
    n, lo, hi = case["n"], case["lo"], case["hi"]
    return [hi if i == 0 else lo + int((hi - lo) * ((i * 0.6180339887498949) % 1.0) ** 1.5) for i in range(n)]


def _before(case):
    """Tokens that each sequence has in the cache before this call; a single one has them all."""
    n, most = case["n"], case.get("start", case.get("context"))
    return [most if n == 1 else int(most * ((i * 0.7548776662466927 + 0.37) % 1.0)) for i in range(n)]


def _seen(case, p):
    """Keys that the row at position p sees."""
    w, s = case["window"], case["sinks"]
    return p + 1 if w == 0 or p < w else w + min(s, p + 1 - w)


def work(case):
    h, d, e = case["h_kv"], case["d"], BYTES[case["dtype"]]
    if case["op"] == "norm_rope":
        elems = case["tokens"] * (case["h_q"] + h) * d
        return {"bytes": 2 * elems * e + 4 * case["tokens"] * case["axes"], "flops": 8 * elems}
    lens, before, row = _lens(case), _before(case), d * BYTES[case["store"]] + (1 if case["store"] == "fp8" else 0)
    tokens = sum(lens)
    if case["op"] == "append":
        moved = 2 * tokens * case["h_q"] * d * e + 2 * tokens * h * (d * e + row)
        if case["store"] == "fp8":  # and read back
            moved += 2 * tokens * h * (d * e + row)
        return {"bytes": moved, "flops": 8 * tokens * (case["h_q"] + h) * d}
    pairs = keys = 0
    for m, c in zip(lens, before):
        w, end = case["window"], c + m
        first = max(0, c + 1 - w) if w else 0  # of the first row's window
        keys += end - first + min(case["sinks"], first)
        if w == 0 or end <= w:
            pairs += m * c + m * (m + 1) // 2
        else:
            pairs += sum(_seen(case, p) for p in range(c, end))
    return {"bytes": 2 * tokens * case["h_q"] * d * e + 2 * keys * h * row, "flops": 4 * d * case["h_q"] * pairs}


# ---------------------------------------------------------------- inputs

def _offsets(lens):
    cu = [0]
    for x in lens:
        cu.append(cu[-1] + x)
    return cu


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def _normal(gen, *size):
    return torch.randn(*size, generator=gen, device=DEV)


def _pool(gen, case, ends):
    """An empty cache with room for `ends` positions a sequence: the pages' order is shuffled."""
    page, h, d = case["page"], case["h_kv"], case["d"]
    per = [-(-e // page) for e in ends]
    pages, width = max(sum(per), 1), max(max(per), 1)
    order = torch.randperm(pages, generator=gen, device=DEV).to(torch.int32)
    at = torch.tensor(_offsets(per)[:-1], device=DEV)[:, None] + torch.arange(width, device=DEV)[None]
    used = torch.arange(width, device=DEV)[None] < torch.tensor(per, device=DEV)[:, None]
    s = dict(page_table=torch.where(used, order[at.clamp(max=pages - 1)], torch.full_like(order[:1], -1)).contiguous())
    shape, fp8 = (pages, h, page, d), case["store"] == "fp8"
    for x in ("k", "v"):
        s[x + "_cache"] = torch.zeros(shape, dtype=torch.uint8, device=DEV).view(TYPES["fp8"]) if fp8 else \
            torch.zeros(shape, dtype=TYPES[case["store"]], device=DEV)
        s[x + "_scale"] = torch.full(shape[:3], 127, dtype=torch.uint8, device=DEV) if fp8 else None
    return s


def _fill(gen, case, s):
    """A cache in use: every row of every page holds keys (values) as a program wrote them."""
    for x in ("k", "v"):
        pool = s[x + "_cache"]
        channel = torch.exp(0.5 * _normal(gen, 1, pool.shape[1], 1, pool.shape[3]))
        if case["store"] == "fp8":
            # rows whose largest code lies between 224 and 448, at scales around 2^-7
            s[x + "_cache"] = (_normal(gen, *pool.shape) * channel * 40).clamp_(-448, 448).to(torch.float8_e4m3fn)
            s[x + "_scale"] = torch.randint(119, 122, pool.shape[:3], generator=gen, device=DEV).to(torch.uint8)
        else:
            s[x + "_cache"] = (_normal(gen, *pool.shape) * channel).to(pool.dtype)


def _positions(gen, case, total):
    """[axes, total]: text, which advances on every axis, then frames of 24 x 24 patches."""
    if case["axes"] == 1:
        return torch.arange(total, device=DEV, dtype=torch.int32) + int(torch.randint(0, 100000, (), generator=gen, device=DEV))
    text = total // 8
    base = int(torch.randint(0, 30000, (), generator=gen, device=DEV))
    i = torch.arange(total, device=DEV)
    j = (i - text).clamp(min=0)
    axes = [torch.where(i < text, i, text + x) + base for x in (j // 576, j // 24 % 24, j % 24)]
    return torch.stack(axes[-case["axes"]:]).to(torch.int32).contiguous()


def _rotation(gen, case, total, dtype):
    """What a model keeps for its norms and rotation, and the tokens' positions."""
    half, d = case["rot"] // 2, case["d"]
    freq = (1e6 ** (-torch.arange(half, device=DEV, dtype=torch.float64) / half)).float()
    p = torch.arange(half, device=DEV)
    # pairs of one axis lie together, or take turns
    axis = (p * case["axes"] // half if case["pairs"] else p % case["axes"]).to(torch.uint8)
    s = dict(freq=freq, axis=axis if case["axes"] > 1 else None, positions=_positions(gen, case, total),
             pairs=case["pairs"], q_weight=None, k_weight=None, bias=1.0 if d == 256 else 0.0)
    if case["norm"]:  # weights about 1, held as the distance from it where the bias is 1
        for x in ("q_weight", "k_weight"):
            s[x] = (1.0 - s["bias"] + 0.2 * _normal(gen, d)).to(dtype)
    return s


def _projected(gen, total, h, d, dtype, into=None):
    """Rows with the uneven channels that trained projections have."""
    x = (_normal(gen, total, h, d) * torch.exp(0.5 * _normal(gen, 1, h, d))).to(dtype)
    return x if into is None else into.copy_(x)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    h_q, h, d, dtype = case["h_q"], case["h_kv"], case["d"], TYPES[case["dtype"]]
    s = dict(op=case["op"], dtype=dtype)
    if case["op"] == "norm_rope":
        total = case["tokens"]
        s.update(_rotation(gen, case, total, dtype))
        if case["fused"]:
            f = torch.zeros(total, h_q + 2 * h, d, dtype=dtype, device=DEV)
            s.update(q=_projected(gen, total, h_q, d, dtype, f[:, :h_q]), k=_projected(gen, total, h, d, dtype, f[:, h_q:h_q + h]))
        else:
            s.update(q=_projected(gen, total, h_q, d, dtype), k=_projected(gen, total, h, d, dtype))
        return s
    lens, before = _lens(case), _before(case)
    total, ends = sum(lens), [a + b for a, b in zip(lens, before)]
    s.update(lens_host=lens, ends_host=ends, total=total, cu=_ints(_offsets(lens)))
    s.update(_pool(gen, case, ends))
    if case["op"] == "extend":
        _fill(gen, case, s)
        s.update(q=(1.5 * _normal(gen, total, h_q, d)).to(dtype), lens=_ints(ends), max_len=max(ends), max_q=max(lens),
                 window=case["window"], sinks=case["sinks"], single=case["hi"] == 1)
        return s
    s.update(_rotation(gen, case, total, dtype))
    s.update(start=_ints(before), read=case["store"] == "fp8")
    if case["axes"] == 1:  # keys are rotated by the place that they take
        s["positions"] = None
    f = torch.empty(total, h_q + 2 * h, d, dtype=dtype, device=DEV)
    s.update(q=_projected(gen, total, h_q, d, dtype, f[:, :h_q]) if h_q else None,
             k=_projected(gen, total, h, d, dtype, f[:, h_q:h_q + h]), v=_projected(gen, total, h, d, dtype, f[:, h_q + h:]))
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import gated_deltanet_linear_prefill_amd as gdn
    if s["op"] == "norm_rope":
        return gdn.gdn_qk_norm_rope(s["q"], s["k"], s["positions"], freq=s["freq"], axis=s["axis"], interleaved=s["pairs"],
                                    q_weight=s["q_weight"], k_weight=s["k_weight"], weight_bias=s["bias"], eps=EPS)
    if s["op"] == "extend":
        return gdn.gdn_attn_extend(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["lens"],
                                   None if s["single"] else s["cu"], window=s["window"], sinks=s["sinks"], max_q=s["max_q"],
                                   max_len=s["max_len"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    q = gdn.gdn_kv_append(s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"], s["start"], s["cu"], q=s["q"],
                          positions=s["positions"], freq=s["freq"], axis=s["axis"], interleaved=s["pairs"],
                          q_weight=s["q_weight"], k_weight=s["k_weight"], weight_bias=s["bias"], eps=EPS,
                          k_scale=s["k_scale"], v_scale=s["v_scale"])
    out = (s["k_cache"], s["v_cache"])
    if s["read"]:
        out = gdn.gdn_kv_read(s["k_cache"], s["v_cache"], s["page_table"], s["start"], s["cu"], s["total"],
                              dtype=s["dtype"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    return out if q is None else (*out, q)


def _plain_norm_rope(s, x, weight, positions):
    """Rows [total, h, d] normed (where there is a weight) and rotated, in 32 bits."""
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * (s["bias"] + weight.float())
    freq, half = s["freq"].double(), s["freq"].shape[0]
    at = positions[None] if positions.dim() == 1 else positions
    at = at[:1].expand(half, -1) if s["axis"] is None else at[s["axis"].long()]  # [pairs, total]
    angle = (at.double() * freq[:, None]).t()[:, None]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    r = x[..., :2 * half]
    a, b = (r[..., 0::2], r[..., 1::2]) if s["pairs"] else (r[..., :half], r[..., half:])
    a, b = a * cos - b * sin, b * cos + a * sin
    r = torch.stack((a, b), -1).flatten(-2) if s["pairs"] else torch.cat((a, b), -1)
    return torch.cat((r, x[..., 2 * half:]), -1)


def _places(s):
    """(page, row, position) of each packed token."""
    page = s["k_cache"].shape[2]
    token = torch.arange(s["total"], device=DEV, dtype=torch.int32)
    seq = torch.searchsorted(s["cu"], token, right=True) - 1
    pos = s["start"][seq] + token - s["cu"][seq]
    return s["page_table"][seq, pos // page].long(), (pos % page).long(), pos


def _two_to(e):
    """2^e in 32 bits, from the exponent's bits: exact for -126 <= e <= 127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _plain_store(x, cache, scale, page, row):
    if scale is None:
        cache[page, :, row] = x.to(cache.dtype)
        return
    top = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
    m, e = torch.frexp(top)  # top = m 2^e with m in [1/2, 1), and 448 = 0.875 * 2^9
    e = torch.where(top > 0, (e - 9 + (m > 0.875)).clamp(min=-126), 0)
    scale[page, :, row] = (e + 127).to(torch.uint8)
    cache.view(torch.uint8)[page, :, row] = (x * _two_to(-e)[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_load(cache, scale, page, row, dtype):
    x = cache.view(torch.uint8)[page, :, row].view(torch.float8_e4m3fn).float()
    return (x * _two_to(scale[page, :, row].to(torch.int32) - 127)[..., None]).to(dtype)


def _run_plain(s):
    if s["op"] == "extend":
        return _plain_extend(s)
    if s["op"] == "norm_rope":
        return tuple(_plain_norm_rope(s, s[x], s[x + "_weight"], s["positions"]).to(s["dtype"]) for x in ("q", "k"))
    page, row, pos = _places(s)
    at = pos if s["positions"] is None else s["positions"]
    _plain_store(_plain_norm_rope(s, s["k"], s["k_weight"], at), s["k_cache"], s["k_scale"], page, row)
    _plain_store(s["v"].float(), s["v_cache"], s["v_scale"], page, row)
    out = (s["k_cache"], s["v_cache"])
    if s["read"]:
        out = tuple(_plain_load(s[x + "_cache"], s[x + "_scale"], page, row, s["dtype"]) for x in ("k", "v"))
    return out if s["q"] is None else (*out, _plain_norm_rope(s, s["q"], s["q_weight"], at).to(s["dtype"]))


def _plain_cache(cache, scale, table):
    """The whole cache of each sequence: [n, h, positions, d] in 32 bits."""
    n, width = table.shape
    at = table.clamp(min=0).long()
    x = cache.view(torch.uint8)[at].view(cache.dtype).float() if scale is not None else cache[at].float()
    if scale is not None:
        x = x * _two_to(scale[at].to(torch.int32) - 127)[..., None]
    h, page, d = cache.shape[1:]
    return x.permute(0, 2, 1, 3, 4).reshape(n, h, width * page, d)


def _visible(pos, keys, window, sinks):
    """Which keys a row at position pos sees: both broadcast."""
    ok = keys <= pos
    if window:
        ok = ok & ((pos - keys < window) | (keys < sinks))
    return ok


def _plain_extend(s):
    q, cu, table = s["q"], s["cu"], s["page_table"]
    n, hq, d = table.shape[0], q.shape[1], q.shape[2]
    k = _plain_cache(s["k_cache"], s["k_scale"], table)
    v = _plain_cache(s["v_cache"], s["v_scale"], table)
    h, length, lq = k.shape[1], k.shape[2], max(s["lens_host"])
    i = torch.arange(lq, device=DEV)
    have = cu[1:] - cu[:-1]
    ok = i[None] < have[:, None]
    rows = torch.where(ok, cu[:-1, None] + i[None], 0).long()
    pos = (s["lens"] - have)[:, None] + i[None]
    mask = _visible(pos[..., None], torch.arange(length, device=DEV), s["window"], s["sinks"])  # [n, lq, length]
    g = hq // h
    qp = (q.float() / math.sqrt(d))[rows].view(n, lq, h, g, d).permute(0, 2, 3, 1, 4).reshape(n * h, g * lq, d)
    scores = torch.bmm(qp, k.transpose(2, 3).reshape(n * h, d, length))
    scores.view(n, h, g, lq, length).masked_fill_(~mask[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True).clamp_(min=-3e38)
    p = scores.sub_(top).exp_()
    o = torch.bmm(p, v.view(n * h, length, d)) / p.sum(-1, keepdim=True).clamp_(min=1e-37)
    return o.view(n, h, g, lq, d).permute(0, 3, 1, 2, 4).reshape(n, lq, hq, d)[ok].to(q.dtype)


# ---------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "extend":
        return _exact_extend(case, s)
    if case["op"] == "norm_rope":
        return tuple(_exact_rows(case, s, s[x], s[x + "_weight"], s["positions"]) for x in ("q", "k"))
    return _exact_append(case, s)


def _exact_rows(case, s, x, weight, positions):
    """Rows as the definition has them: a pair is a complex number that is turned by its angle."""
    out, half = x.double().clone(), case["rot"] // 2
    if weight is not None:
        out *= (weight.double() + s["bias"]) / torch.sqrt(out.square().sum(-1, keepdim=True) / case["d"] + EPS)
    step = 2 if case["pairs"] else 1
    for p in range(half):
        of = positions if positions.dim() == 1 else positions[int(s["axis"][p]) if s["axis"] is not None else 0]
        turn = torch.polar(torch.ones_like(of, dtype=torch.float64), of.double() * s["freq"][p].double())[:, None]
        a, b = p * step, p * step + 1 if case["pairs"] else p + half
        z = torch.complex(out[..., a].contiguous(), out[..., b].contiguous()) * turn
        out[..., a], out[..., b] = z.real, z.imag
    return out


def _two_to_64(e):
    """2^e in 64 bits, from the exponent's bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_fp8(x):
    """The values an fp8 row stands for after it is written: the nearest multiples of the code's
    step (ties to even) at the smallest power of two that brings the largest within 448."""
    top = x.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(torch.where(top > 0, top, 448.0) / 448) - 1).clamp(min=-126)
    for _ in range(2):  # the logarithm may be off by a rounding: the comparison is not
        e = torch.where(top > 448 * _two_to_64(e), e + 1, e)
    y = x / _two_to_64(e)
    step = _two_to_64(torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 4)
    return torch.round(y / step) * step * _two_to_64(e)


def _exact_append(case, s):
    before, cu, page = _before(case), _offsets(s["lens_host"]), case["page"]
    at = s["positions"]
    if at is None:
        at = torch.cat([torch.arange(a, a + m, device=DEV) for a, m in zip(before, s["lens_host"])])
    new = (_exact_rows(case, s, s["k"], s["k_weight"], at), s["v"].double())
    if s["read"]:
        out = tuple(_exact_fp8(x) for x in new)
    else:
        out = (s["k_cache"].double(), s["v_cache"].double())
        for pool, x in zip(out, new):
            for b, m in enumerate(s["lens_host"]):
                pages = s["page_table"][b, : -(-(before[b] + m) // page)].long()
                whole = pool[pages].transpose(1, 2).reshape(-1, case["h_kv"], case["d"])
                whole[before[b]:before[b] + m] = x[cu[b]:cu[b + 1]]
                pool[pages] = whole.view(len(pages), page, case["h_kv"], case["d"]).transpose(1, 2)
    return out if s["q"] is None else (*out, _exact_rows(case, s, s["q"], s["q_weight"], at))


def _exact_cache(cache, scale, pages, upto):
    """The first `upto` positions of one sequence: [h, upto, d]."""
    x = cache.view(torch.uint8)[pages].view(cache.dtype).double() if scale is not None else cache[pages].double()
    if scale is not None:
        x = x * _two_to_64(scale[pages].to(torch.int64) - 127)[..., None]
    return x.transpose(0, 1).reshape(cache.shape[1], -1, cache.shape[3])[:, :upto]


def _exact_extend(case, s):
    if case["n"] * case["h_q"] * case["hi"] * (case["hi"] + case["context"]) > MOST_SCORES:
        return None
    g, cu = case["h_q"] // case["h_kv"], _offsets(s["lens_host"])
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    for b, (m, end) in enumerate(zip(s["lens_host"], s["ends_host"])):
        pages = s["page_table"][b, : -(-end // case["page"])].long()
        k = _exact_cache(s["k_cache"], s["k_scale"], pages, end)
        v = _exact_cache(s["v_cache"], s["v_scale"], pages, end)
        p, j = torch.arange(end - m, end, device=DEV)[:, None], torch.arange(end, device=DEV)[None]
        unseen = j > p
        if case["window"]:
            unseen |= (j <= p - case["window"]) & (j >= case["sinks"])
        for y in range(case["h_q"]):
            x = s["q"][cu[b]:cu[b + 1], y].double() @ k[y // g].t().contiguous() / math.sqrt(case["d"])
            out[cu[b]:cu[b + 1], y] = torch.softmax(x.masked_fill_(unseen, -math.inf), -1) @ v[y // g]
    return out
