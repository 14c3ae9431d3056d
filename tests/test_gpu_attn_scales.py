"""Keys and scores of very different sizes in one call."""
import pytest
import torch

import bit_blockwise_weight_nf4_b200 as bnb4
import oracle
from kv_ref import TORCH, Case, attention64, quantize_rows
from test_gpu_attn import run

pytestmark = pytest.mark.gpu


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
