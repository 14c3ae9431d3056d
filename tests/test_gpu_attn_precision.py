"""What the attention kernels round, held to the figures that include/bnb4.h
states: tight limits for fp16 caches with few rows, and scores of large size."""
import math

import numpy as np
import pytest
import torch

import bit_blockwise_weight_nf4_b200 as bnb4
import oracle
from kv_ref import Case, attention64, stored_place
from test_gpu_attn import run

pytestmark = pytest.mark.gpu

# Half a step of an output, 2^-11 / m (fp16) or 2^-8 / m (bf16) of a value of
# mantissa m, uniform: 2^-11 / sqrt(3) sqrt(E m^-2), E m^-2 = 3 / (8 ln 2) for
# evenly spread logarithms.
LAST = {oracle.F16: 2.07e-4, oracle.BF16: 1.66e-3}
NF4_SCALE = 1613.0 / 1024.0  # the table's constant (csrc/attn.cuh)


def table16():
    """NF4's table as one fp16 term holds it, in float64."""
    t = oracle.codebook(bnb4.NF4).astype(np.float32) * np.float32(NF4_SCALE)
    return t.astype(np.float16).astype(np.float64) / NF4_SCALE


def test_table_error():
    """One fp16 term of NF4's table is within 3.1e-4 of a value, 8.5e-5 of the scale
    and 3.7e-5 of it in the root mean square, its ends exact."""
    t = oracle.codebook(bnb4.NF4).astype(np.float64)
    e = np.abs(table16() - t)
    assert e[0] == e[-1] == 0 and e.max() <= 8.5e-5 and np.sqrt((e ** 2).mean()) <= 3.7e-5
    assert (e[t != 0] / np.abs(t[t != 0])).max() <= 3.1e-4


class OneTerm(Case):
    """A case whose values (not keys) come from the table in one fp16 term."""

    def kv64(self, b):
        k, v = super().kv64(b)
        if self.qtype != bnb4.NF4:
            return k, v
        pages = self.block_table[b].long()
        c = torch.stack([self.v_codes[pages] >> 4, self.v_codes[pages] & 15], -1).flatten(-2)
        c = c[..., torch.from_numpy(stored_place(self.D, self.bs))].long()
        a = self.v_absmax[pages].double().unsqueeze(-1)
        v = (torch.from_numpy(table16())[c].unflatten(-1, (-1, self.bs)) * a).flatten(-2)
        return k, v.transpose(0, 1).flatten(1, 2)[:, :self.kv_lens[b]]


@pytest.mark.parametrize("D,bs", [(64, 32), (128, 32), (128, 64), (128, 128)])
@pytest.mark.parametrize("qtype", [bnb4.NF4, bnb4.FP4])
@pytest.mark.parametrize("q_len,n_heads", [(1, 2), (1, 8), (2, 8), (3, 10), (4, 8)])
def test_fp16_few_rows_lose_only_the_last_rounding(q_len, n_heads, qtype, D, bs):
    """1 to 16 rows per key/value head, fp16: keys and weights are held in two fp16
    terms, values in one of the table's (exact for FP4), which the reference has
    too; so the error is the output's last rounding, and 10% for samples that
    are not quite that and for fp32 sums.  Weights in one term would add
    2.07e-4 in quadrature (2.9e-4 in all), keys in one term 1e-4 of a score's
    size, 4 to 5 here."""
    case = OneTerm([600, 450, 301, 64] * 4, 32, 2, D, bs, qtype, oracle.F16, seed=q_len + bs)
    q = case.queries(16 * q_len, n_heads, std=3.0)
    out, _ = run(case, q, [q_len] * 16)
    o64, _, _, _ = attention64(case, q, [q_len] * 16)
    rel = float((out.cpu().double() - o64).norm() / o64.norm())
    assert rel <= 1.1 * LAST[oracle.F16], rel


@pytest.mark.parametrize("dtype", [oracle.BF16, oracle.F16])
@pytest.mark.parametrize("qtype", [bnb4.NF4, bnb4.FP4])
@pytest.mark.parametrize("q_len,n_heads", [(1, 2), (4, 8), (40, 2)])
@pytest.mark.parametrize("size", [1.0, 10.0, 30.0])
def test_large_scores(size, q_len, n_heads, qtype, dtype):
    """Scores of a standard deviation of 1, 10 and 30; 1, 16 and 40 rows.

    In the root mean square, relative: the last rounding; weights in one fp16
    term (bf16 caches) 2.07e-4; the values' table in one term (NF4 but for fp16
    chunks) 1e-4, rounded with its scale to fp16 (chunks, bf16 caches) 2.07e-4;
    and a key element's error r makes one of r times a score's root sum of
    squares, here the scores' standard deviation s, in the exponent: r s of the
    output where weights lie on few tokens, r from the table and the rounding of
    the product as for the values (FP4's products are exact).  These add in
    quadrature; 15% for samples."""
    lens = [600, 450, 301, 64] * (4 if q_len < 40 else 1)
    case = Case(lens, 32, 2, 128, 64, qtype, dtype, seed=60)
    q = case.queries(len(lens) * q_len, n_heads)
    k = torch.cat([case.kv64(b)[0] for b in range(4)], 1)
    now = float((q[:, :2].double().transpose(0, 1) @ k.transpose(1, 2)).std()) / math.sqrt(128)
    scale = size / now / math.sqrt(128)
    out, _ = run(case, q, [q_len] * len(lens), scale=scale)
    o64, _, _, _ = attention64(case, q, [q_len] * len(lens), scale=scale)
    rel = float((out.cpu().double() - o64).norm() / o64.norm())
    chunk, nf4 = q_len == 40, qtype == bnb4.NF4
    two = dtype == oracle.F16
    table = 1e-4 if nf4 else 0.0
    product = 2.07e-4 if chunk and nf4 and not two else 0.0
    key = math.hypot(0.0 if two else table, product) * size
    limit = math.sqrt(LAST[dtype] ** 2 + (0.0 if two else 2.07e-4) ** 2 +
                      (0.0 if two and chunk else table) ** 2 + product ** 2 + key ** 2)
    assert rel <= 1.15 * limit, (rel, limit)
