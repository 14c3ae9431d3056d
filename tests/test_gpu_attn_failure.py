"""Failure detection of the attention kernels on the GPU without a fault: a copy
that a wait counts on is never made (few rows), or an arrival (many); the wait
runs out, the kernel sets the library's device error word and ends,
bnb4_device_status reports it, and the context stays usable.  Nothing traps or
hangs."""
import ctypes

import pytest
import torch

import bit_blockwise_weight_nf4_b200 as bnb4
import oracle
from kv_ref import Case, attention64, check
from test_gpu_attn import ints, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D,bs,qtype,dtype", [(128, 64, bnb4.NF4, oracle.BF16),
                                              (64, 32, bnb4.NF4, oracle.F16),
                                              (128, 128, bnb4.FP4, oracle.F16)])
@pytest.mark.parametrize("q_len,n_heads,max_seq_len",
                         [(1, 2, 64), (1, 2, 5000), (4, 8, 64), (4, 8, 5000), (40, 4, 64),
                          (200, 4, 5000)])
def test_withheld_operand_times_out_and_context_survives(q_len, n_heads, max_seq_len, D, bs, qtype,
                                                         dtype):
    lens = [4000, 1000]
    case = Case(lens, 64, 2, D, bs, qtype, dtype, seed=41)
    q = case.queries(2 * q_len, n_heads)
    qd, c, bt, sl = q.cuda(), case.cache(), case.block_table.cuda(), ints(lens)
    out, ws = torch.empty_like(qd), torch.empty(1 << 26, dtype=torch.uint8, device="cuda")
    a = bnb4.Attn(qd.data_ptr(), n_heads * D, D, out.data_ptr(), n_heads * D, D, None,
                  ctypes.pointer(c.struct), bt.data_ptr(), bt.shape[1], sl.data_ptr(), None,
                  ws.data_ptr(), ws.numel(), 2 * q_len, 2, n_heads, q_len, max_seq_len,
                  bt.shape[1], 1, 0, D ** -0.5, 0)
    stream = torch.cuda.current_stream().cuda_stream
    assert bnb4.bnb4_device_status(stream, True) == bnb4.OK
    assert bnb4.bnb4_debug_attn_withhold(a, 20000, stream) == bnb4.OK
    assert bnb4.bnb4_device_status(stream, True) == bnb4.ERR_DEVICE_TIMEOUT
    assert bnb4.bnb4_device_status(stream, True) == bnb4.OK  # cleared
    # the context is still usable: the same call is right
    got, _ = run(case, q, [q_len] * 2, cache=c, max_seq_len=max_seq_len)
    o64, bound, _, _ = attention64(case, q, [q_len] * 2)
    check(got, o64, bound, dtype)
