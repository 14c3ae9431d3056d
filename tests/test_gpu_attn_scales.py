"""Keys and scores of very different sizes in one call."""
import pytest
import torch

import bit_blockwise_weight_nf4_b200 as bnb4
import oracle
from kv_ref import TORCH, Case, attention64, check, quantize_rows
from test_gpu_attn import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,small,binades", [(oracle.BF16, 1.0, 8), (oracle.BF16, 1.0, 16),
                                                 (oracle.BF16, 2.0 ** -40, 24),
                                                 (oracle.F16, 2.0 ** -6, 16)])
@pytest.mark.parametrize("qtype", [bnb4.NF4, bnb4.FP4])
@pytest.mark.parametrize("q_len,window", [(3, 0), (40, 0), (40, 30), (200, 150)])
def test_a_large_key_that_a_row_does_not_see(q_len, window, qtype, dtype, small, binades):
    """Two tokens' keys are up to 2^24 times the others': the rows before them,
    and those whose window has left them, are as exact as without them.  (A
    key in the chunk kernel is normal fp16 over 24 binades below the largest
    of its tile, so the module's bounds hold as they stand.)"""
    lens = [333, 61]
    case = Case(lens, 32, 2, 128, 64, qtype, dtype, seed=binades, k_std=small)
    untouched = []  # rows that see neither of the two
    for kv in lens:
        large = (kv - 1, max(0, kv - 170) if q_len == 200 else kv - q_len // 2 - 1)
        b = lens.index(kv)
        for j in large:
            page, at = int(case.block_table[b, j // 32]), j % 32
            row = torch.randn(2, 128, generator=case.gen) * small * 2.0 ** binades
            case.k_codes[page, :, at], case.k_absmax[page, :, at], _ = \
                quantize_rows(row.to(TORCH[dtype]), 64, qtype)
        for pos in range(kv - q_len, kv):
            untouched.append(not any(j <= pos and (not window or j > pos - window)
                                     for j in large))
    untouched = torch.tensor(untouched)
    assert untouched.any()
    q = case.queries(2 * q_len, 4, std=1.0 if dtype == oracle.F16 else 1.0 / small)
    out, lse = run(case, q, [q_len] * 2, window=window)
    o64, bound, l64, lb = attention64(case, q, [q_len] * 2, window=window)
    # (of the other rows only the log-sum-exp is checked: the bound of an output is
    # linear in the scores' error, which is not small next to a score of 2^24)
    assert torch.isfinite(out).all()
    check(out.cpu()[untouched], o64[untouched], bound[untouched], case.dtype)
    seen = ~torch.isinf(l64)
    assert ((lse.cpu().double() - l64).abs()[seen] <= lb[seen]).all()


@pytest.mark.parametrize("dtype", [oracle.BF16, oracle.F16])
@pytest.mark.parametrize("qtype", [bnb4.NF4, bnb4.FP4])
@pytest.mark.parametrize("q_len,n_heads,max_seq_len",
                         [(1, 2, 64), (1, 2, None), (3, 4, None), (40, 4, 64), (40, 4, None)])
@pytest.mark.parametrize("log2", [10, 20, 24, 27, 35, 100])
def test_huge_scores_choose_a_token(log2, q_len, n_heads, max_seq_len, qtype, dtype):
    """Scores up to 2^108, whose own last place is many binades of a weight: the
    largest ones share the weight all the same.

    A key is +-2^e in one dimension, a query +-2^n, a value +-1: codes, scales,
    products and values are exact, so equal scores stay equal and the weights of
    different ones differ by their own rounding only.  An output is then off by
    a weight's rounding to fp16, 2^-11 of sum p |V| = 1, its last rounding, u of
    itself, and a few fp32 roundings (2^-18).  The log-sum-exp is a score after
    five fp32 roundings and three rounded constants, 2^-21 of itself, plus a
    logarithm (2^-18)."""
    lens = [900, 130]
    case = Case(lens, 32, 1, 128, 64, qtype, dtype, seed=31)
    g, tdt = case.gen, TORCH[dtype]
    signs = lambda *shape: torch.randint(0, 2, shape, generator=g).float() * 2 - 1
    rows = tuple(case.k_codes.shape[:3])
    k = torch.zeros(*rows, 128)
    k[..., 70] = torch.exp2(torch.randint(-8, 9, rows, generator=g).float()) * signs(*rows)
    case.k_codes, case.k_absmax, _ = quantize_rows(k.to(tdt), 64, qtype)
    case.v_codes, case.v_absmax, _ = quantize_rows(signs(*rows, 128).to(tdt), 64, qtype)
    up = log2 if dtype == oracle.BF16 else min(log2, 12)
    q = torch.zeros(2 * q_len, n_heads, 128)
    q[..., 70] = 2.0 ** up * signs(2 * q_len, n_heads)
    q = q.to(tdt)
    scale = 2.0 ** min(log2 - up, 26)
    out, lse = run(case, q, [q_len] * 2, max_seq_len=max_seq_len, scale=scale)
    o64, _, l64, _ = attention64(case, q, [q_len] * 2, scale=scale)
    u = 2.0 ** -8 if dtype == oracle.BF16 else 2.0 ** -11
    assert ((out.cpu().double() - o64).abs() <= u * o64.abs() + 2.0 ** -11 + 2.0 ** -18).all()
    assert ((lse.cpu().double() - l64).abs() <= l64.abs() * 2.0 ** -21 + 2.0 ** -18).all()
