"""Calls of attention over the 4-bit cache that are allowed and out of the
ordinary."""
import pytest
import torch

import bit_blockwise_weight_nf4_b200 as bnb4
from bit_blockwise_weight_nf4_b200 import torch_ops  # noqa: F401
import oracle
from kv_ref import Case
from test_gpu_attn import ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch", [0, 3])
@pytest.mark.parametrize("ragged", [False, True])
def test_no_queries_is_an_empty_call(ragged, batch):
    case = Case([90, 33, 1], 16, 2, 128, 64, bnb4.NF4, oracle.BF16, seed=50)
    c, bt, sl = case.cache(), case.block_table.cuda()[:batch], ints(case.kv_lens[:batch])
    q = torch.empty(0, 4, 128, dtype=torch.bfloat16, device="cuda")
    cu = ints([0] * (batch + 1)) if ragged else None
    for kw in (dict(), dict(max_q_len=0), dict(max_q_len=5), dict(max_seq_len=100000)):
        out = torch.empty_like(q)
        lse = torch.empty(0, 4, device="cuda")
        assert bnb4.attn_4bit(q, c, bt, sl, cu, **kw).shape == (0, 4, 128)
        assert bnb4.attn_4bit(q, c, bt, sl, cu, out=out, lse=lse, **kw) is out
    for max_q in (0, 1):
        y = torch.ops.bnb4.attn_4bit(q, c.k_codes, c.v_codes, c.k_absmax, c.v_absmax, bt, sl, cu,
                                     max_q, 90, 0.1, True, 0, 64, bnb4.NF4)
        assert y.shape == (0, 4, 128)
    torch.cuda.synchronize()
