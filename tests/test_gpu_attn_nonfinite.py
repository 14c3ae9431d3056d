"""Rows that see no token, whatever stands in their query."""
import pytest
import torch

import bit_blockwise_weight_nf4_b200 as bnb4
import oracle
from kv_ref import Case
from test_gpu_attn import run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [oracle.BF16, oracle.F16])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("q_len,n_heads,max_seq_len",
                         [(1, 2, 64), (1, 2, None), (5, 4, 64), (5, 4, None), (40, 4, 64),
                          (40, 4, None), (70, 8, None)])
def test_rows_that_see_nothing_are_zero_whatever_their_query(q_len, n_heads, max_seq_len, dtype,
                                                             value):
    """Empty sequences, sequences shorter than their queries and sequences all
    of whose pages are missing, next to a long one, few rows (both row tiles)
    and chunks, split over the SMs and not: a NaN or an infinity in the query of a
    row that sees nothing changes nothing."""
    case = Case([0, 3, 5000, 33], 32, 2, 128, 64, bnb4.NF4, dtype, seed=23)
    case.block_table[3] = -1
    q_lens = [q_len] * 4
    q = case.queries(4 * q_len, n_heads)
    clean, l0 = run(case, q, q_lens, max_seq_len=max_seq_len)
    empty = torch.isinf(l0).cpu()
    assert empty[:q_len].all() and empty[3 * q_len:].all()
    assert (clean.cpu()[empty] == 0).all()
    x = q.clone()
    x[empty] = torch.where(torch.arange(case.D) % 7 == 3, torch.full((), value, dtype=q.dtype),
                           x[empty])
    dirty, l1 = run(case, x, q_lens, max_seq_len=max_seq_len)
    assert torch.equal(clean, dirty) and torch.equal(l0, l1)
