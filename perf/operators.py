"""Performance cases of the attention operators: the paged key-value cache (write, read back),
packed causal attention over prompts, and attention of one new token over the cache.

Each case is one pass of one operator. `run` computes it either in its plain form (elementary
torch operations in 32 bits, rounded once at the end) or, with `own` set, through the
package's entry points. `exact` evaluates the definition in 64 bits.

A cache store is f32, bf16 or fp8 (e4m3 codes with one power-of-two scale per token and KV
head, kept as the biased exponent). Position p of sequence s lies in page
page_table[s][p // page], row p % page; the pages of a sequence are in no particular order.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f32": torch.float32, "fp8": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "f32": 4, "fp8": 1}
LARGEST = 2.0e12  # multiply-adds x 2 of the largest listed case, which no drawn one exceeds


def listed():
    return [
        # One decode step of 32 sequences appends its tokens: the smallest write.
        dict(name="write_step", op="write", n=32, lo=1, hi=1, start=4000, h_kv=2, d=256, page=64,
             dtype="bf16", store="bf16"),
        # Prompts of very different lengths, packed, each after a context of its own.
        dict(name="write_packed", op="write", n=24, lo=1, hi=2600, start=1500, h_kv=8, d=128, page=16,
             dtype="bf16", store="bf16"),
        # A 4096-token prompt is quantised as it is written, and read back for its next segment.
        dict(name="write_read_fp8", op="write_read", n=1, lo=4096, hi=4096, start=0, h_kv=2, d=256,
             page=64, dtype="bf16", store="fp8"),
        # The context of a long prompt is read back before its next segment.
        dict(name="read_long_fp8", op="read", n=1, lo=65536, hi=65536, start=0, h_kv=2, d=256, page=64,
             dtype="bf16", store="fp8"),
        # A few short 32-bit rows, odd heads: the smallest read.
        dict(name="read_short_f32", op="read", n=5, lo=1, hi=90, start=33, h_kv=3, d=64, page=16,
             dtype="f32", store="f32"),
        # Short prompts in 32 bits, where the call's latency counts.
        dict(name="prefill_short_f32", op="prefill", n=3, lo=1, hi=200, context=0, h_q=4, h_kv=2, d=64,
             dtype="f32", causal=True),
        # The 4096-token prompt of the benchmark, at the source page's attention layout.
        dict(name="prefill_prompt", op="prefill", n=1, lo=4096, hi=4096, context=0, h_q=16, h_kv=2,
             d=256, dtype="bf16", causal=True),
        # A batch of prompts of very different lengths, packed.
        dict(name="prefill_packed", op="prefill", n=16, lo=1, hi=2500, context=0, h_q=32, h_kv=8, d=128,
             dtype="bf16", causal=True),
        # The last 4096-token segment of a long prompt, attending to all that came before.
        dict(name="prefill_segment", op="prefill", n=1, lo=4096, hi=4096, context=28672, h_q=16, h_kv=2,
             d=256, dtype="bf16", causal=True),
        # One sequence early in its answer: a decode step where latency counts.
        dict(name="decode_short", op="decode", n=1, lo=333, hi=333, h_q=16, h_kv=2, d=256, page=64,
             dtype="bf16", store="bf16"),
        # A served batch: 64 sequences of very different lengths.
        dict(name="decode_batch", op="decode", n=64, lo=17, hi=8192, h_q=32, h_kv=8, d=128, page=16,
             dtype="bf16", store="bf16"),
        # One sequence with a 131072-token context in an 8-bit cache.
        dict(name="decode_long_fp8", op="decode", n=1, lo=131072, hi=131072, h_q=16, h_kv=2, d=256,
             page=64, dtype="bf16", store="fp8"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    while True:
        op = rng.choice(["write", "write_read", "read", "prefill", "prefill", "decode", "decode"])
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        d = rng.choice([64, 128, 256])
        h_kv = rng.choice([1, 2, 3, 4, 8])
        group = rng.choice([1, 2, 3, 4, 6, 8, 16])
        n = _log_int(rng, 1, 64)
        if op == "prefill":
            hi = _log_int(rng, 1, 8192)
            case = dict(op=op, n=n, lo=rng.randint(1, hi), hi=hi, context=rng.choice([0, _log_int(rng, 1, 16384)]),
                        h_q=h_kv * group, h_kv=h_kv, d=d, dtype=dtype, causal=rng.random() < 0.8)
            # the plain form keeps all scores: stay below 16 GiB of them
            if n * h_kv * group * hi * (hi + case["context"]) > 1 << 32:
                continue
        else:
            store = rng.choice([dtype, "fp8"])
            page = rng.choice([16, 32, 64, 128])
            if op == "decode":
                hi = _log_int(rng, 1, 131072)
                case = dict(op=op, n=n, lo=rng.randint(1, hi), hi=hi, h_q=h_kv * group, h_kv=h_kv, d=d, page=page,
                            dtype=dtype, store=store)
            else:
                hi = _log_int(rng, 1, 16384)
                if op == "write":
                    store = dtype
                case = dict(op=op, n=n, lo=rng.randint(1, hi), hi=hi, start=rng.choice([0, _log_int(rng, 1, 8192)]),
                            h_kv=h_kv, d=d, page=page, dtype=dtype, store=store)
            if n * (hi + case.get("start", 0)) * h_kv * d > 1 << 28:
                continue
        if work(case)["flops"] <= LARGEST / (16 if dtype == "f32" else 1):
            return case


# ---------------------------------------------------------------- sizes

def _lens(case):
    """The sequences' lengths: from lo to hi by a fixed law, so that work(case) and prepare(case)
    agree; the longest is hi."""
    n, lo, hi = case["n"], case["lo"], case["hi"]
    # low-discrepancy fractions, skewed so that short sequences are more frequent than long ones
    return [hi if i == 0 else lo + int((hi - lo) * ((i * 0.6180339887498949) % 1.0) ** 1.5) for i in range(n)]


def _starts(case):
    """Tokens that each sequence has in the cache before this call."""
    return [int(case["start"] * ((i * 0.7548776662466927 + 0.37) % 1.0)) for i in range(case["n"])]


def _pairs(lq, lk, causal):
    """(query, key) pairs that count, per head; lk >= lq."""
    return lq * (lk - lq) + lq * (lq + 1) // 2 if causal else lq * lk


def work(case):
    lens, d, h = _lens(case), case["d"], case["h_kv"]
    tokens, e = sum(lens), BYTES[case["dtype"]]
    if case["op"] == "prefill":
        keys = tokens + case["context"] * case["n"]
        pairs = sum(_pairs(x, x + case["context"], case["causal"]) for x in lens)
        return {"bytes": 2 * tokens * case["h_q"] * d * e + 2 * keys * h * d * e, "flops": 4 * d * case["h_q"] * pairs}
    row = d * BYTES[case["store"]] + (1 if case["store"] == "fp8" else 0)
    if case["op"] == "decode":
        return {"bytes": 2 * tokens * h * row + 2 * case["n"] * case["h_q"] * d * e, "flops": 4 * d * case["h_q"] * tokens}
    moved = 2 * tokens * h * (d * e + row)
    return {"bytes": moved * (2 if case["op"] == "write_read" else 1), "flops": 2 * tokens * h * d}


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


def _keys(gen, rows, h, d, dtype):
    """Keys (or values) with the uneven channels that trained projections have."""
    channel = torch.exp(0.5 * _normal(gen, 1, h, d))
    return (_normal(gen, rows, h, d) * channel).to(dtype)


def _pool(gen, case, ends):
    """An empty cache with room for `ends` positions a sequence: the pages' order is shuffled."""
    page, h, d = case["page"], case["h_kv"], case["d"]
    per = [-(-e // page) for e in ends]
    pages, width = sum(per), max(max(per), 1)
    order = torch.randperm(max(pages, 1), generator=gen, device=DEV).to(torch.int32)
    first = _offsets(per)
    at = torch.tensor(first[:-1], device=DEV)[:, None] + torch.arange(width, device=DEV)[None]
    used = torch.arange(width, device=DEV)[None] < torch.tensor(per, device=DEV)[:, None]
    table = torch.where(used, order[at.clamp(max=max(pages, 1) - 1)], torch.full_like(order[:1], -1))
    shape = (max(pages, 1), h, page, d)
    s = dict(page_table=table.contiguous())
    for x in ("k", "v"):
        s[x + "_cache"] = torch.zeros(shape, dtype=torch.float32 if case["store"] == "f32" else torch.bfloat16,
                                      device=DEV) if case["store"] != "fp8" else \
            torch.zeros(shape, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn)
        s[x + "_scale"] = torch.full(shape[:3], 127, dtype=torch.uint8, device=DEV) if case["store"] == "fp8" else None
    return s


def _fill(gen, case, s):
    """A cache in use: every row of every page holds keys (values) as a program wrote them."""
    for x in ("k", "v"):
        pool = s[x + "_cache"]
        channel = torch.exp(0.5 * _normal(gen, 1, pool.shape[1], 1, pool.shape[3]))
        if case["store"] == "fp8":
            # rows whose largest code lies between 224 and 448, at scales around 2^-7
            body = (_normal(gen, *pool.shape) * channel * 40).clamp_(-448, 448)
            s[x + "_cache"] = body.to(torch.float8_e4m3fn)
            s[x + "_scale"] = torch.randint(119, 122, pool.shape[:3], generator=gen, device=DEV).to(torch.uint8)
        else:
            s[x + "_cache"] = (_normal(gen, *pool.shape) * channel).to(pool.dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    lens, h, d, dtype = _lens(case), case["h_kv"], case["d"], TYPES[case["dtype"]]
    total = sum(lens)
    s = dict(op=case["op"], dtype=dtype, lens_host=lens, total=total)
    if case["op"] == "prefill":
        keys = [x + case["context"] for x in lens]
        s.update(q=(1.5 * _normal(gen, total, case["h_q"], d)).to(dtype), k=_keys(gen, sum(keys), h, d, dtype),
                 v=_keys(gen, sum(keys), h, d, dtype), cu_q=_ints(_offsets(lens)), cu_k=_ints(_offsets(keys)),
                 keys_host=keys, causal=case["causal"])
        return s
    if case["op"] == "decode":
        s.update(_pool(gen, case, lens))
        _fill(gen, case, s)
        s.update(q=(1.5 * _normal(gen, case["n"], case["h_q"], d)).to(dtype), lens=_ints(lens), max_len=max(lens))
        return s
    starts = _starts(case)
    s.update(_pool(gen, case, [a + b for a, b in zip(starts, lens)]))
    s.update(start=_ints(starts), cu=_ints(_offsets(lens)))
    if case["op"] == "read":
        _fill(gen, case, s)
    else:
        s.update(k=_keys(gen, total, h, d, dtype), v=_keys(gen, total, h, d, dtype))
    return s


# ---------------------------------------------------------------- one pass

def run(state):
    return _run_own(state) if own else _run_plain(state)


def _run_own(s):
    import gated_deltanet_linear_prefill_amd as gdn
    op = s["op"]
    if op == "prefill":
        return gdn.gdn_attn_prefill(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=s["causal"])
    if op == "decode":
        return gdn.gdn_attn_decode(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["lens"],
                                   max_len=s["max_len"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    if op != "read":
        gdn.gdn_kv_write(s["k"], s["v"], s["k_cache"], s["v_cache"], s["page_table"], s["start"], s["cu"],
                         k_scale=s["k_scale"], v_scale=s["v_scale"])
        if op == "write":
            return s["k_cache"], s["v_cache"]
    return gdn.gdn_kv_read(s["k_cache"], s["v_cache"], s["page_table"], s["start"], s["cu"], s["total"],
                           dtype=s["dtype"], k_scale=s["k_scale"], v_scale=s["v_scale"])


def _places(s):
    """(page, row) of each packed token."""
    page = s["k_cache"].shape[2]
    token = torch.arange(s["total"], device=DEV, dtype=torch.int32)
    seq = torch.searchsorted(s["cu"], token, right=True) - 1
    pos = s["start"][seq] + token - s["cu"][seq]
    return s["page_table"][seq, pos // page].long(), (pos % page).long()


def _two_to(e):
    """2^e in 32 bits, from the exponent's bits: exact for -126 <= e <= 127."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _plain_store(x, cache, scale, page, row):
    x = x.float()
    if scale is not None:
        top = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
        m, e = torch.frexp(top)  # top = m 2^e with m in [1/2, 1), and 448 = 0.875 * 2^9
        e = torch.where(top > 0, (e - 9 + (m > 0.875)).clamp(min=-126), 0)
        x = x * _two_to(-e)[..., None]
        scale[page, :, row] = (e + 127).to(torch.uint8)
        cache.view(torch.uint8)[page, :, row] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        cache[page, :, row] = x.to(cache.dtype)


def _plain_load(cache, scale, page, row, dtype):
    if scale is None:
        return cache[page, :, row].float().to(dtype)
    x = cache.view(torch.uint8)[page, :, row].view(torch.float8_e4m3fn).float()
    return (x * _two_to(scale[page, :, row].to(torch.int32) - 127)[..., None]).to(dtype)


def _softmax_av(scores, v):
    """softmax of [b, m, l] scores over the last axis, times v [b, l, d]; rows with nothing but
    -inf give 0."""
    top = scores.amax(-1, keepdim=True).clamp_(min=-3e38)
    p = scores.sub_(top).exp_()
    return torch.bmm(p, v) / p.sum(-1, keepdim=True).clamp_(min=1e-37)


def _rows(cu, lens, width):
    """Indices of each sequence's packed rows, padded to `width`, and which of them exist."""
    j = torch.arange(width, device=DEV)
    ok = j[None] < (cu[1:] - cu[:-1])[:, None]
    return torch.where(ok, cu[:-1, None] + j[None], 0).long(), ok


def _run_plain(s):
    op = s["op"]
    if op == "prefill":
        return _plain_prefill(s)
    if op == "decode":
        return _plain_decode(s)
    page, row = _places(s)
    if op != "read":
        _plain_store(s["k"], s["k_cache"], s["k_scale"], page, row)
        _plain_store(s["v"], s["v_cache"], s["v_scale"], page, row)
        if op == "write":
            return s["k_cache"], s["v_cache"]
    return (_plain_load(s["k_cache"], s["k_scale"], page, row, s["dtype"]),
            _plain_load(s["v_cache"], s["v_scale"], page, row, s["dtype"]))


def _plain_prefill(s):
    q, k, v = s["q"], s["k"], s["v"]
    n, hq, d, h = len(s["lens_host"]), q.shape[1], q.shape[2], k.shape[1]
    lq, lk = max(s["lens_host"]), max(s["keys_host"])
    iq, okq = _rows(s["cu_q"], s["lens_host"], lq)
    ik, okk = _rows(s["cu_k"], s["keys_host"], lk)
    g = hq // h
    # [n, h, g, lq, d] x [n, h, d, lk]: the heads of a group share their keys
    qp = (q.float() / math.sqrt(d))[iq].view(n, lq, h, g, d).permute(0, 2, 3, 1, 4).reshape(n * h, g * lq, d)
    kt = k.float()[ik].permute(0, 2, 3, 1).reshape(n * h, d, lk)
    vp = v.float()[ik].permute(0, 2, 1, 3).reshape(n * h, lk, d)
    mask = okk[:, None, :].expand(n, lq, lk)
    if s["causal"]:
        shift = (s["cu_k"][1:] - s["cu_k"][:-1]) - (s["cu_q"][1:] - s["cu_q"][:-1])
        i, j = torch.arange(lq, device=DEV), torch.arange(lk, device=DEV)
        mask = mask & (j[None, None, :] <= i[None, :, None] + shift[:, None, None])
    scores = torch.bmm(qp, kt)
    scores.view(n, h, g, lq, lk).masked_fill_(~mask[:, None, None], -math.inf)
    o = _softmax_av(scores, vp).view(n, h, g, lq, d).permute(0, 3, 1, 2, 4).reshape(n, lq, hq, d)
    return o[okq].to(q.dtype)


def _plain_cache(cache, scale, table):
    """The whole cache of each sequence: [n, h, positions, d] in 32 bits."""
    n, width = table.shape
    at = table.clamp(min=0).long()
    x = cache.view(torch.uint8)[at].view(cache.dtype).float() if scale is not None else cache[at].float()
    if scale is not None:
        x = x * _two_to(scale[at].to(torch.int32) - 127)[..., None]
    h, page, d = cache.shape[1:]
    return x.permute(0, 2, 1, 3, 4).reshape(n, h, width * page, d)


def _plain_decode(s):
    q, table = s["q"], s["page_table"]
    n, hq, d = q.shape
    k = _plain_cache(s["k_cache"], s["k_scale"], table)
    v = _plain_cache(s["v_cache"], s["v_scale"], table)
    h, length = k.shape[1], k.shape[2]
    qp = (q.float() / math.sqrt(d)).view(n * h, hq // h, d)
    scores = torch.bmm(qp, k.transpose(2, 3).reshape(n * h, d, length))
    mask = torch.arange(length, device=DEV)[None] < s["lens"][:, None]
    scores.view(n, h, -1, length).masked_fill_(~mask[:, None, None], -math.inf)
    return _softmax_av(scores, v.view(n * h, length, d)).reshape(n, hq, d).to(q.dtype)


# ---------------------------------------------------------------- the definition, in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "prefill":
        return _exact_prefill(case, s)
    if case["op"] == "decode":
        return _exact_decode(case, s)
    return _exact_cache(case, s)


def _exact_attend(q, k, v, allowed):
    """q [g, m, d], k and v [l, d], allowed [m, l] or None: softmax(q k^T / sqrt d) v."""
    x = q.double() @ k.double().t().contiguous() / math.sqrt(q.shape[-1])
    if allowed is not None:
        x.masked_fill_(~allowed, -math.inf)
    return torch.softmax(x, -1) @ v.double()


def _exact_prefill(case, s):
    g, d = case["h_q"] // case["h_kv"], case["d"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    cq, ck = _offsets(s["lens_host"]), _offsets(s["keys_host"])
    for b in range(case["n"]):
        lq, lk = s["lens_host"][b], s["keys_host"][b]
        allowed = torch.ones(lq, lk, dtype=torch.bool, device=DEV).tril(lk - lq) if case["causal"] else None
        for x in range(case["h_kv"]):
            k, v = s["k"][ck[b]:ck[b + 1], x], s["v"][ck[b]:ck[b + 1], x]
            for y in range(x * g, (x + 1) * g):
                out[cq[b]:cq[b + 1], y] = _exact_attend(s["q"][None, cq[b]:cq[b + 1], y], k, v, allowed)[0]
    return out


def _two_to_64(e):
    """2^e in 64 bits, from the exponent's bits."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_rows(cache, scale, pages, upto):
    """The first `upto` positions of one sequence: [h, upto, d]."""
    x = cache.view(torch.uint8)[pages].view(cache.dtype).double() if scale is not None else cache[pages].double()
    if scale is not None:
        x = x * _two_to_64(scale[pages].to(torch.int64) - 127)[..., None]
    return x.transpose(0, 1).reshape(cache.shape[1], -1, cache.shape[3])[:, :upto]


def _exact_decode(case, s):
    g = case["h_q"] // case["h_kv"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=DEV)
    for b, length in enumerate(s["lens_host"]):
        pages = s["page_table"][b, : -(-length // case["page"])].long()
        k = _exact_rows(s["k_cache"], s["k_scale"], pages, length)
        v = _exact_rows(s["v_cache"], s["v_scale"], pages, length)
        for x in range(case["h_kv"]):
            out[b, x * g:(x + 1) * g] = _exact_attend(s["q"][b, x * g:(x + 1) * g], k[x], v[x], None)
    return out


def _exact_fp8(x):
    """The values an fp8 row stands for after it is written: the nearest multiples of the code's
    step (ties to even) at the smallest power of two that brings the largest within 448."""
    x = x.double()
    top = x.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(torch.where(top > 0, top, 448.0) / 448) - 1).clamp(min=-126)
    for _ in range(2):  # the logarithm may be off by a rounding: the comparison is not
        e = torch.where(top > 448 * _two_to_64(e), e + 1, e)
    y = x / _two_to_64(e)
    binade = torch.frexp(y.abs().clamp(min=2.0 ** -6))[1] - 1
    step = _two_to_64(binade - 3)
    return torch.round(y / step) * step * _two_to_64(e)


def _exact_cache(case, s):
    starts, cu, page = _starts(case), _offsets(s["lens_host"]), case["page"]
    got = []
    for x in ("k", "v"):
        pool = s[x + "_cache"].double() if case["op"] == "write" else None
        back = torch.empty(s["total"], case["h_kv"], case["d"], dtype=torch.float64, device=DEV)
        for b, length in enumerate(s["lens_host"]):
            if length == 0:
                continue
            at = slice(cu[b], cu[b + 1])
            pages = s["page_table"][b, : -(-(starts[b] + length) // page)].long()
            if case["op"] == "read":
                rows = _exact_rows(s[x + "_cache"], s[x + "_scale"], pages, starts[b] + length)
                back[at] = rows[:, starts[b]:].transpose(0, 1)
            elif case["op"] == "write_read":
                back[at] = _exact_fp8(s[x][at]) if case["store"] == "fp8" else s[x][at].double()
            else:
                whole = pool[pages].transpose(1, 2).reshape(-1, case["h_kv"], case["d"])
                whole[starts[b]:starts[b] + length] = s[x][at].double()
                pool[pages] = whole.view(len(pages), page, case["h_kv"], case["d"]).transpose(1, 2)
        got.append(pool if case["op"] == "write" else back)
    return tuple(got)
