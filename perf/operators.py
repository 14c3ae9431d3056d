"""Cases and plain forms of the 4-bit key/value cache operators.

Three operators are measured: writing keys and values into a paged cache held
in 4 bits (NF4 or FP4 codes, one scale of the cache's 16-bit type per block
of a head's row), reading rows of it back, and attention of new queries over
it -- one token per sequence (decode), a few (a verified draft), or a chunk
of a prompt (prefill).

The cache's layout (shared by both forms): codes are uint8
[pages, kv heads, page size, D / 2], two per byte, the first in the high
nibble; scales are [pages, kv heads, page size, D / blocksize].  A row's D
values are stored in 8 strips: strip g holds, block after block, values
[g w, (g + 1) w) of each block, w = blocksize / 8 (a row of one block is in
its natural order).  A cached value is table[code] * scale.  Slot s of the
cache is row s % page_size of page s // page_size.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# ------------------------------------------------------------------- cases
def listed():
    def attn(name, b, hq, hkv, d, bs, qt, dtype, page, kv, q=(1, 1), window=0, mix=1):
        return {"name": name, "kind": "attn", "b": b, "hq": hq, "hkv": hkv, "d": d, "bs": bs,
                "qt": qt, "dtype": dtype, "page": page, "kv_lo": kv[0], "kv_hi": kv[1],
                "q_lo": q[0], "q_hi": q[1], "window": window, "mix": mix}

    def rows(name, kind, tokens, hkv, d, bs, qt, dtype, page, spread=False):
        return {"name": name, "kind": kind, "tokens": tokens, "hkv": hkv, "d": d, "bs": bs,
                "qt": qt, "dtype": dtype, "page": page, "spread": spread}

    return [
        # one decode step of 16 sequences, 32 heads of 128 (a 7B layer): the
        # new tokens, each on a page of its own, are written and read back --
        # latency is everything
        rows("append 16 tokens", "write", 16, 32, 128, 64, "nf4", "bf16", 64, True),
        # a 2048-token prompt of the same layer
        rows("append a 2048-token prompt", "write", 2048, 32, 128, 64, "nf4", "bf16", 64),
        # several prompts packed together, grouped heads, odd count, small head
        rows("append 12345 packed tokens", "write", 12345, 8, 64, 32, "fp4", "f16", 16),
        # a cached prefix is read back, e.g. to hand it to another layout
        rows("read a 777-token prefix", "read", 777, 8, 128, 128, "nf4", "f16", 16),
        # the whole cache of one layer, 16 sequences of 4096
        rows("read 65536 tokens", "read", 65536, 32, 128, 64, "nf4", "bf16", 64),
        # decode: one sequence, short context, the interactive case
        attn("decode 1 x 257", 1, 32, 32, 128, 64, "nf4", "bf16", 64, (257, 257)),
        # decode: a serving batch with grouped heads and ragged lengths
        attn("decode 24 ragged grouped", 24, 32, 8, 128, 64, "nf4", "bf16", 64, (100, 8192)),
        # decode: a 7B layer's heads, full batch
        attn("decode 16 x 4096", 16, 32, 32, 128, 64, "nf4", "bf16", 64, (4096, 4096)),
        # decode: two very long documents, work has to be split over the axis
        attn("decode 2 x 131072", 2, 32, 8, 128, 128, "fp4", "f16", 256, (120001, 131072)),
        # four draft tokens verified at once
        attn("verify 4 tokens x 12", 12, 32, 8, 128, 32, "nf4", "f16", 32, (500, 6000), (4, 4)),
        # chunks of prompts against what is cached, a sliding window
        attn("chunks 4 ragged, window", 4, 32, 8, 128, 64, "nf4", "bf16", 64, (700, 5000),
             (33, 700), 2000),
        # a whole 2048-token prompt, a 7B layer's heads
        attn("prompt 2048", 2, 32, 32, 128, 64, "nf4", "bf16", 64, (2048, 2048), (2048, 2048)),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    d = rng.choice([64, 128, 128])
    c = {"kind": rng.choice(["write", "read", "attn", "attn", "attn"]), "hkv": rng.choice([1, 2, 4, 8, 8, 32]),
         "d": d, "bs": rng.choice([b for b in (32, 64, 128) if b <= d]),
         "qt": rng.choice(["nf4", "nf4", "fp4"]), "dtype": rng.choice(["bf16", "bf16", "f16"]),
         "page": rng.choice([16, 32, 48, 64, 128, 256])}
    if c["kind"] != "attn":
        c["tokens"] = log(1, 60000 if c["kind"] == "read" else 15000)
        c["spread"] = c["tokens"] < 100 and rng.random() < 0.5
        return c
    g = rng.choice([1, 2, 4, 5, 7, 8, 16]) if c["hkv"] < 32 else 1
    c["hq"], c["mix"] = c["hkv"] * g, rng.randrange(1 << 20)
    form = rng.choice(["decode", "decode", "verify", "chunk"])
    c["b"] = log(1, 64) if form != "chunk" else log(1, 6)
    most = min(131072, 2000000 // (c["b"] * c["hkv"]))  # rows of codes read by a pass
    if form == "chunk":
        c["q_hi"] = log(17, 1500)
        c["q_lo"] = rng.randint(1, c["q_hi"])
        most = min(most, int(4e8 / (c["b"] * c["hq"] * c["q_hi"])), 12000)
    else:
        c["q_lo"] = c["q_hi"] = 1 if form == "decode" else rng.randint(2, 9)
        most = min(most, int(1e9 / (c["b"] * c["hq"] * c["q_hi"])))
    c["kv_hi"] = log(64, max(65, most))
    c["kv_lo"] = rng.randint(0, c["kv_hi"]) if c["b"] > 1 else c["kv_hi"]
    c["window"] = rng.choice([0, 0, 0, log(16, 4096)])
    return c


def lengths(case):
    """The sequences' query and context lengths (the context ends with the
    queries' own tokens; one shorter than its queries leaves rows empty)."""
    r = random.Random(case["mix"])
    b = case["b"]
    q = [r.randint(case["q_lo"], case["q_hi"]) for _ in range(b)]
    kv = [r.randint(case["kv_lo"], case["kv_hi"]) for _ in range(b)]
    q[0], kv[0] = case["q_hi"], case["kv_hi"]
    return q, kv


# ------------------------------------------------------------------ inputs
def table(qt, dtype=torch.float32, device="cpu"):
    """The 16 values of a code."""
    if qt == "nf4":  # normal quantiles: 7 below zero, zero, 8 above, over the largest
        hexes = ("-0x1p+0 -0x1.647362p-1 -0x1.0cd65cp-1 -0x1.94653cp-2 -0x1.234496p-2 "
                 "-0x1.7a6a7ap-3 -0x1.74f0d2p-4 0x0p+0 0x1.45f602p-4 0x1.4995bep-3 "
                 "0x1.f809b4p-3 0x1.5a066cp-2 0x1.c3496ap-2 0x1.200f52p-1 0x1.722760p-1 0x1p+0")
        t = [float.fromhex(h) for h in hexes.split()]
    else:  # sign and E2M1 magnitudes over 6, in fp32
        m = np.array([0, .5, 1, 1.5, 2, 3, 4, 6], np.float32) / np.float32(6)
        t = [float(x) for x in m] + [-float(x) for x in m]
    return torch.tensor(t, dtype=torch.float64).to(device=device, dtype=dtype)


def strips(x, bs):
    """[..., D] from its natural order to the stored one."""
    d = x.shape[-1]
    w = bs // 8
    return x.unflatten(-1, (d // bs, 8, w)).transpose(-3, -2).flatten(-3)


def unstrips(x, bs):
    d = x.shape[-1]
    w = bs // 8
    return x.unflatten(-1, (8, d // bs, w)).transpose(-3, -2).flatten(-3)


def _codes(v, qt, t):
    """Codes of scaled values v: the number of midpoints of neighbouring
    table values strictly below v (FP4: of magnitudes below |v|, and the sign
    of a value with a magnitude)."""
    if qt == "nf4":
        mid = (t[:-1] + t[1:]) * 0.5
        return (v.unsqueeze(-1) > mid).sum(-1)
    mid = (t[:7] + t[1:8]) * 0.5
    m = (v.abs().unsqueeze(-1) > mid).sum(-1)
    return m + 8 * ((v < 0) & (m > 0))


def _quantize(x, bs, qt):
    """(packed codes in stored order, scales) of rows x [..., D]."""
    blk = x.float().unflatten(-1, (-1, bs))
    a = blk.abs().amax(-1)
    r = torch.where(a == 0, torch.zeros_like(a), 1.0 / a)
    c = _codes(blk * r.unsqueeze(-1), qt, table(qt, device=x.device))
    c = strips(c.flatten(-2), bs).to(torch.uint8)
    return (c[..., 0::2] << 4) | c[..., 1::2], a.to(x.dtype)


def _values(codes, scales, bs, qt, dtype):
    """Rows [..., D] of packed codes [..., D / 2] and scales, in dtype."""
    c = torch.stack([codes >> 4, codes & 15], -1).flatten(-2)
    t = table(qt, torch.float32, codes.device).to(dtype)
    v = unstrips(t[c.int()], bs).unflatten(-1, (-1, bs))
    return (v * scales.to(dtype).unsqueeze(-1)).flatten(-2)


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    dt, d, bs, h, page = DTYPES[case["dtype"]], case["d"], case["bs"], case["hkv"], case["page"]

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=g, device=dev, dtype=torch.float32).mul_(std).to(dt)

    # keys have a few channels that run larger than the others
    chan = torch.ones(h, d, device=dev)
    chan[torch.rand(h, d, generator=g, device=dev) < 0.03] = 4.0
    st = {"case": case}
    if case["kind"] == "attn":
        q_len, kv_len = lengths(case)
        per = max(1, -(-max(kv_len) // page))
        pages = case["b"] * per
    else:
        pages = (case["tokens"] if case["spread"] else -(-case["tokens"] // page)) + 3
    shape = (pages, h, page)
    filled = case["kind"] != "write"
    make = torch.empty if filled else torch.zeros
    for n in "kv":
        st[n + "_codes"] = make(*shape, d // 2, dtype=torch.uint8, device=dev)
        st[n + "_absmax"] = make(*shape, d // bs, dtype=dt, device=dev)
    if filled:  # what was written before, piece by piece
        step = max(1, (1 << 22) // (h * page * d))
        for p in range(0, pages, step):
            n = min(step, pages - p)
            k = (normal(n, h, page, d).float() * chan[:, None]).to(dt)
            st["k_codes"][p:p + n], st["k_absmax"][p:p + n] = _quantize(k, bs, case["qt"])
            st["v_codes"][p:p + n], st["v_absmax"][p:p + n] = _quantize(
                normal(n, h, page, d), bs, case["qt"])
    order = torch.randperm(pages, generator=g, device=dev)
    if case["kind"] == "attn":
        total = sum(q_len)
        st["q"] = normal(total, case["hq"], d, std=1.3)
        st["block_table"] = order.view(case["b"], per).int()
        st["seq_lens"] = torch.tensor(kv_len, dtype=torch.int32, device=dev)
        st["cu_q"] = torch.tensor(np.concatenate([[0], np.cumsum(q_len)]), dtype=torch.int32,
                                  device=dev)
        st["max_q"], st["max_kv"], st["total_q"] = max(q_len), max(kv_len), total
        return st
    t = torch.arange(case["tokens"], device=dev)
    st["slots"] = order[t] * page + t * 7 % page if case["spread"] else \
        order[t // page] * page + t % page
    if case["kind"] == "write":
        # keys and values as a fused projection leaves them: parts of one row
        qkv = normal(case["tokens"], 3 * h * d).view(case["tokens"], 3, h, d)
        qkv[:, 1] *= chan.to(dt)
        st["k"], st["v"] = qkv[:, 1], qkv[:, 2]
    return st


# ------------------------------------------------------------- plain forms
def _plain_read(s):
    c = s["case"]
    page, slot = s["slots"] // c["page"], s["slots"] % c["page"]
    return tuple(_values(s[n + "_codes"][page, :, slot], s[n + "_absmax"][page, :, slot], c["bs"],
                         c["qt"], torch.float32).to(DTYPES[c["dtype"]]) for n in "kv")


def _plain_write(s):
    c = s["case"]
    page, slot = s["slots"] // c["page"], s["slots"] % c["page"]
    kc, ka = _quantize(s["k"], c["bs"], c["qt"])
    vc, va = _quantize(s["v"], c["bs"], c["qt"])
    s["k_codes"][page, :, slot], s["k_absmax"][page, :, slot] = kc, ka
    s["v_codes"][page, :, slot], s["v_absmax"][page, :, slot] = vc, va
    return _plain_read(s)


def _plain_attn(s):
    c = s["case"]
    q, bt, cu, lens = s["q"], s["block_table"].long(), s["cu_q"].long(), s["seq_lens"].long()
    b, h, d, mq, mkv = c["b"], c["hkv"], c["d"], s["max_q"], s["max_kv"]
    g = c["hq"] // h
    # [b, h, context, d] of every sequence, as long as the longest
    k, v = (_values(s[n + "_codes"][bt], s[n + "_absmax"][bt], c["bs"], c["qt"], torch.float32)
            .transpose(1, 2).flatten(2, 3)[:, :, :mkv] for n in "kv")
    i = torch.arange(mq, device=q.device)
    n = cu[1:] - cu[:-1]
    real = i < n[:, None]  # [b, mq]
    row = torch.where(real, cu[:-1, None] + i, torch.zeros_like(cu[:-1, None]))
    qp = q[row].float().view(b, mq, h, g, d).permute(0, 2, 3, 1, 4)  # [b, h, g, mq, d]
    score = (qp.reshape(b, h, g * mq, d) @ k.transpose(-1, -2)).view(b, h, g, mq, mkv)
    score = score * (1.0 / math.sqrt(d))
    pos = (lens[:, None] - n[:, None] + i)[:, :, None]  # a query's place in its sequence
    j = torch.arange(mkv, device=q.device)
    see = (j <= pos) & (j < lens[:, None, None])
    if c["window"]:
        see = see & (j > pos - c["window"])
    see = see[:, None, None]
    score = torch.where(see, score, torch.full_like(score[:1, :1, :1, :1, :1], -math.inf))
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p = torch.exp(score - top)
    total = p.sum(-1, keepdim=True)
    o = (p.view(b, h, g * mq, mkv) @ v).view(b, h, g, mq, d)
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    out = torch.zeros(s["total_q"] + 1, c["hq"], d, dtype=q.dtype, device=q.device)
    at = torch.where(real, row, torch.full_like(row, s["total_q"]))
    out[at] = o.permute(0, 3, 1, 2, 4).reshape(b, mq, c["hq"], d).to(q.dtype)
    return out[:-1]


# -------------------------------------------------------------------- runs
def run(state):
    kind = state["case"]["kind"]
    if not own:
        return {"write": _plain_write, "read": _plain_read, "attn": _plain_attn}[kind](state)
    import bit_blockwise_weight_nf4_b200 as bnb4
    c = state["case"]
    cache = bnb4.KVCache4bit(state["k_codes"], state["v_codes"], state["k_absmax"],
                             state["v_absmax"], c["bs"], bnb4.NF4 if c["qt"] == "nf4" else bnb4.FP4)
    if kind == "write":
        bnb4.kv_write_4bit(state["k"], state["v"], cache, state["slots"])
    if kind in ("write", "read"):
        return bnb4.kv_read_4bit(cache, state["slots"])
    return bnb4.attn_4bit(state["q"], cache, state["block_table"], state["seq_lens"],
                          cu_seqlens_q=state["cu_q"], max_q_len=state["max_q"],
                          max_seq_len=state["max_kv"], causal=True, window=c["window"])


# -------------------------------------------------------------------- work
def work(case):
    d, h = case["d"], case["hkv"]
    row = d // 2 + 2 * (d // case["bs"])  # bytes of a cached row
    if case["kind"] != "attn":
        n = 2 * case["tokens"] * h
        b = n * (row + 2 * d) + 8 * case["tokens"]
        if case["kind"] == "read":
            return {"bytes": b, "flops": n * d}
        # written and read back: the codes stay on the chip at best
        return {"bytes": b + n * 2 * d, "flops": 4 * n * d}
    q_len, kv_len = lengths(case)
    seen = rows = 0  # (query, key) pairs; cached tokens any query sees
    for n, kv in zip(q_len, kv_len):
        w = case["window"] or kv + n
        first = kv - n
        rows += min(kv, max(0, kv - max(0, first - w + 1)))
        seen += sum(max(0, min(w, p + 1)) for p in range(first, kv))
    t = sum(q_len)
    return {"bytes": 2 * rows * h * row + 4 * t * case["hq"] * d + 4 * (rows // case["page"] + 3 * case["b"]),
            "flops": 4 * seen * case["hq"] * d}


# ------------------------------------------------------------------- exact
def _decode64(codes, scales, case):
    """float64 rows of uint8 codes [..., D / 2], element by element from the
    stored place of each value."""
    d, bs = case["d"], case["bs"]
    w = bs // 8
    e = torch.arange(d, device=codes.device)
    blk, i = e // bs, e % bs
    place = (i // w) * (d // 8) + blk * w + i % w
    byte = codes[..., place // 2].int()
    c = torch.where(place % 2 == 0, byte // 16, byte % 16)
    return table(case["qt"], torch.float64, codes.device)[c] * scales.double()[..., blk]


def exact(case, seed):
    s = prepare(case, seed)
    d, bs, h, page = case["d"], case["bs"], case["hkv"], case["page"]
    if case["kind"] == "read":
        at = s["slots"]
        return tuple(_decode64(s[n + "_codes"].transpose(1, 2).flatten(0, 1)[at],
                               s[n + "_absmax"].transpose(1, 2).flatten(0, 1)[at], case)
                     for n in "kv")
    if case["kind"] == "write":  # the nearest table value, the lower one where two are as near
        t = table(case["qt"], torch.float64, "cuda")
        t = torch.sort(t.unique()).values
        got = []
        for x in (s["k"], s["v"]):
            x = x.double().unflatten(-1, (-1, bs))
            a = x.abs().amax(-1, keepdim=True)
            v = torch.where(a > 0, x / a, torch.zeros_like(x))
            near = torch.searchsorted(t, v.contiguous()).clamp(1, t.numel() - 1)
            lo, hi = t[near - 1], t[near]
            if case["qt"] == "fp4":  # ties go to the smaller magnitude
                up = torch.where(v < 0, (hi - v) <= (v - lo), (hi - v) < (v - lo))
            else:
                up = (hi - v) < (v - lo)
            got.append((torch.where(up, hi, lo) * a).flatten(-2))
        return tuple(got)
    q_len, kv_len = lengths(case)
    g = case["hq"] // h
    out, at = [], 0
    for b in range(case["b"]):
        n, kv = q_len[b], kv_len[b]
        q = s["q"][at:at + n].double().view(n, h, g, d)
        at += n
        o = torch.zeros(n, h, g, d, dtype=torch.float64, device="cuda")
        pages = s["block_table"][b, :-(-kv // page)].long()
        for head in range(h if kv else 0):
            k, v = (_decode64(s[m + "_codes"][pages, head], s[m + "_absmax"][pages, head], case)
                    .flatten(0, 1)[:kv] for m in "kv")
            logit = torch.einsum("ngd,jd->ngj", q[:, head], k) / math.sqrt(d)
            place = torch.arange(kv - n, kv, device="cuda")[:, None, None]
            j = torch.arange(kv, device="cuda")
            hide = j > place
            if case["window"]:
                hide = hide | (j <= place - case["window"])
            logit = logit.masked_fill(hide, -math.inf)
            o[:, head] = torch.nan_to_num(torch.softmax(logit, -1), nan=0.0) @ v
        out.append(o.view(n, case["hq"], d))
    return torch.cat(out)
