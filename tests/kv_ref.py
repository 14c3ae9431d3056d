"""Plain 64-bit reference of the 4-bit key/value cache: rows quantized by the
CPU oracle, the stored order written out value by value, and attention over
the cached values in float64.

Tolerance of attention (o against the float64 o64 over the same cached
values).  For one output o = sum_j p_j V_jd with normalised weights p:
  * a code's table value is off by at most et of itself (NF4 3e-4: half an
    fp16 step of the smallest entries under the kernel's scaling is below it;
    FP4 0, its values are exact), in the scores and in the values;
  * fp32 sums: the scores' by at most (D + 4) 2^-23 of sum |q K|, the
    weighted sum's by at most (n + 64) 2^-23 of sum p |V| for n tokens, any
    order; exp2 by 2^-22 of the weight plus the rounding of its argument,
    2^-23 of |s|;
  * a weight is rounded to fp16: 2^-11 of itself (fp16 caches: both halves
    kept, 2^-22);
  * so with ds = the largest score error of the row, every weight is off by a
    factor within exp(2 ds) and
    |o - o64| <= (2 ds + et + ew + (n + 64) 2^-23) sum_j p_j |V_jd| * 1.1 + f
                 + u (|o64| + the same),
    u = 2^-8 (bf16) or 2^-11 (fp16) of the last rounding;
  * the kernel for more than 16 rows multiplies table and scale before the
    product, one rounding more of NF4's keys and values in fp16, 2^-11 (bf16
    caches; FP4's 3 bits times a scale's 8 are exact, and fp16 caches keep what
    is rounded away in a second term): added to et;
  * f = n 2^-39 max|V|: fp16 weights have an absolute step too.  A weight
    times its scale, p_j a_j <= a_max < 2^(e + 1), is rounded as p_j a_j 2^(14
    - e), below 2^-14 by at most half the subnormal step, 2^-25, that is
    2^(e - 39) <= 2^-39 a_max; times |t| <= 1 for each of n tokens, and p is
    relative to the largest weight, so the sum it is divided by is >= 1.  (The
    kernel for more than 16 rows holds p_j 2^7, so its step is 2^-25 2^-7 =
    2^-32 of V.)  (It shows where the tokens that carry the row have a zero in a dimension.)
On at least 1024 outputs the errors' root mean square adds in quadrature: bf16
1.66e-3 (last rounding), 2.0e-4 (weights), 1e-4 (tables) < 2e-3; fp16 2.1e-4
and 2.1e-4 (weights), 1.5e-4 (tables; scores of a size around one) < 5e-4:
the relative Frobenius error is held to those."""
import math

import numpy as np
import torch

import bit_blockwise_weight_nf4_b200 as bnb4
import oracle

TORCH = {oracle.BF16: torch.bfloat16, oracle.F16: torch.float16}
UNIT = {oracle.BF16: 2.0 ** -8, oracle.F16: 2.0 ** -11}
FROB = {oracle.BF16: 2e-3, oracle.F16: 5e-4}
TABLE_ERR = {bnb4.NF4: 3e-4, bnb4.FP4: 0.0}


def stored_place(D, bs):
    """place[d]: where value d of a row lies among the stored ones."""
    w = bs // 8
    place = np.zeros(D, np.int64)
    for d in range(D):
        b, i = d // bs, d % bs
        place[d] = (i // w) * (D // 8) + b * w + i % w
    return place


def quantize_rows(x, bs, qtype):
    """(codes [..., D / 2] in the stored order, absmax [..., D / bs], code
    numbers [..., D] in natural order) of a CPU bf16 / fp16 tensor [..., D]."""
    D = x.shape[-1]
    flat = x.contiguous().view(-1)
    host = flat.numpy() if x.dtype == torch.float16 else \
        flat.view(torch.int16).numpy().view(np.uint16)
    st = oracle.quantize(host, bs, qtype, False)
    c = np.stack([st["codes"] >> 4, st["codes"] & 15], -1).reshape(-1, D)
    s = np.zeros_like(c)
    s[:, stored_place(D, bs)] = c
    packed = (s[:, 0::2] << 4 | s[:, 1::2]).astype(np.uint8)
    a = torch.from_numpy(st["absmax"]).to(x.dtype)
    assert torch.equal(a.float(), torch.from_numpy(st["absmax"])) or torch.isnan(a).any()
    lead = x.shape[:-1]
    return (torch.from_numpy(packed).view(*lead, D // 2), a.view(*lead, D // bs),
            torch.from_numpy(c.astype(np.int64)).view(*lead, D))


def values64(codes, absmax, D, bs, qtype):
    """float64 cached values [..., D] of stored codes and scales (CPU)."""
    c = torch.stack([codes >> 4, codes & 15], -1).flatten(-2).long()
    c = c[..., torch.from_numpy(stored_place(D, bs))]
    t = torch.from_numpy(oracle.codebook(qtype).astype(np.float64))
    return (t[c].unflatten(-1, (-1, bs)) * absmax.double().unsqueeze(-1)).flatten(-2)


class Case:
    """A filled cache with sequences spread over shuffled pages."""

    def __init__(self, kv_lens, page, heads, D, bs, qtype, dtype, seed=0, spare=2, v_std=1.0,
                 k_std=1.0, sink=False):
        g = torch.Generator().manual_seed(seed)
        self.kv_lens, self.page, self.heads, self.D, self.bs = kv_lens, page, heads, D, bs
        self.qtype, self.dtype = qtype, dtype
        tdt = TORCH[dtype]
        self.width = max(1, -(-max(kv_lens) // page))
        pages = len(kv_lens) * self.width + spare
        rnd = lambda: torch.randn(pages, heads, page, D, generator=g)
        k, v = rnd() * k_std, rnd() * v_std
        k[..., 3] *= 5
        if sink:  # value scales that span many binades
            v *= torch.exp2(torch.randint(-12, 6, (pages, heads, page, 1), generator=g).float())
        self.k_codes, self.k_absmax, _ = quantize_rows(k.to(tdt), bs, qtype)
        self.v_codes, self.v_absmax, _ = quantize_rows(v.to(tdt), bs, qtype)
        perm = torch.randperm(pages, generator=g)[:len(kv_lens) * self.width]
        self.block_table = perm.view(len(kv_lens), self.width).int()
        self.gen = g

    def cache(self):
        return bnb4.KVCache4bit(self.k_codes.cuda(), self.v_codes.cuda(), self.k_absmax.cuda(),
                                self.v_absmax.cuda(), self.bs, self.qtype)

    def queries(self, n, n_heads, std=1.0):
        return (torch.randn(n, n_heads, self.D, generator=self.gen) * std).to(TORCH[self.dtype])

    def kv64(self, b):
        """float64 keys and values [heads, len, D] of sequence b; tokens of a
        page out of range are NaN."""
        out = []
        for codes, absmax in ((self.k_codes, self.k_absmax), (self.v_codes, self.v_absmax)):
            pages = self.block_table[b].long()
            bad = (pages < 0) | (pages >= codes.shape[0])
            x = values64(codes[pages.clamp(0, codes.shape[0] - 1)],
                         absmax[pages.clamp(0, codes.shape[0] - 1)], self.D, self.bs, self.qtype)
            x[bad] = float("nan")
            out.append(x.transpose(0, 1).flatten(1, 2)[:, :self.kv_lens[b]])
        return out


def attention64(case, q, q_lens, causal=True, window=0, scale=None, rounded=2.0 ** -11):
    """(o64, bound, lse64, lse bound): float64 attention of q [T, n_heads, D] and
    the elementwise bounds of the module docstring."""
    scale = case.D ** -0.5 if scale is None else scale
    T, nh, D = q.shape
    group = nh // case.heads
    o = torch.zeros(T, nh, D, dtype=torch.float64)
    bound = torch.zeros_like(o)
    lse = torch.full((T, nh), -math.inf, dtype=torch.float64)
    lse_b = torch.zeros_like(lse)
    wide = group * max(q_lens) > 16
    et = TABLE_ERR[case.qtype]
    if wide and case.qtype == bnb4.NF4 and case.dtype == oracle.BF16:
        et += 2.0 ** -11
    step = 2.0 ** (-32 if wide else -39)
    u = UNIT[case.dtype]
    at = 0
    for b, n in enumerate(q_lens):
        kv = case.kv_lens[b]
        k, v = case.kv64(b)
        j = torch.arange(kv)
        for i in range(n):
            pos = kv - n + i
            see = ~torch.isnan(k[0, :, 0])
            if causal:
                see &= j <= pos
            if window:
                see &= j > pos - window
            idx = see.nonzero().view(-1)
            if idx.numel():
                for h in range(case.heads):
                    qq = q[at + i, h * group:(h + 1) * group].double()
                    kk, vv = k[h, idx], v[h, idx]
                    s = qq @ kk.T * scale
                    mag = qq.abs() @ kk.abs().T * scale
                    ds = (mag * (et + (D + 4) * 2.0 ** -23) + s.abs() * 2.0 ** -22).amax(-1) + \
                        2.0 ** -22
                    p = torch.softmax(s, -1)
                    o[at + i, h * group:(h + 1) * group] = p @ vv
                    rel = (2 * ds + et + rounded + (idx.numel() + 64) * 2.0 ** -23)[:, None]
                    e = rel * (p @ vv.abs()) * 1.1 + idx.numel() * step * vv.abs().max()
                    y = o[at + i, h * group:(h + 1) * group]
                    bound[at + i, h * group:(h + 1) * group] = e + u * (y.abs() + e)
                    lse[at + i, h * group:(h + 1) * group] = torch.logsumexp(s, -1)
                    lse_b[at + i, h * group:(h + 1) * group] = \
                        ds * 1.1 + (idx.numel() + 64) * 2.0 ** -23 + 2.0 ** -20
        at += n
    lse_b += torch.nan_to_num(lse.abs(), posinf=0.0) * 2.0 ** -22
    return o, bound, lse, lse_b


def check(out, o64, bound, dtype, min_size=1024):
    y = out.detach().cpu().double()
    err = (y - o64).abs()
    # subnormal outputs round by an absolute half step
    tiny = 2.0 ** -134 if dtype == oracle.BF16 else 2.0 ** -25
    bad = ~(err <= bound + tiny)
    assert not bad.any(), "%d outputs past the bound; worst %g of it" % (
        int(bad.sum()), float((err / (bound + tiny)).max()))
    norm = float(o64.norm())
    if o64.numel() >= min_size and norm > 0:
        rel = float((y - o64).norm()) / norm
        assert rel <= FROB[dtype], "relative Frobenius error %.3g" % rel
