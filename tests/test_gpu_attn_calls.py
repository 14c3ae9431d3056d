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


def test_workspaces_of_any_element_type():
    """A workspace's size is its bytes, whatever its elements are."""
    case = Case([5000, 333], 64, 2, 128, 64, bnb4.NF4, oracle.BF16, seed=51)
    q, c = case.queries(2, 4).cuda(), case.cache()
    bt, sl = case.block_table.cuda(), ints(case.kv_lens)
    want = bnb4.attn_4bit(q, c, bt, sl)
    a = bnb4.Attn(0, 0, 0, 0, 0, 0, None, bnb4.ctypes.pointer(c.struct), 0, bt.shape[1], 0, None,
                  None, 0, 2, 2, 4, 1, bt.shape[1] * 64, bt.shape[1], 1, 0, 0.1, 0)
    rc, need = bnb4.bnb4_attn_workspace(a)
    assert rc == bnb4.OK and need > 0
    for dtype in (torch.uint8, torch.float32, torch.int64):
        ws = torch.empty(-(-need // dtype.itemsize), dtype=dtype, device="cuda")
        assert torch.equal(bnb4.attn_4bit(q, c, bt, sl, workspace=ws), want)
    with pytest.raises(bnb4.Bnb4Error):
        bnb4.attn_4bit(q, c, bt, sl, workspace=torch.empty(need - 1, dtype=torch.uint8,
                                                           device="cuda"))
    with pytest.raises(ValueError):
        bnb4.attn_4bit(q, c, bt, sl, workspace=torch.empty(need, dtype=torch.uint8))
