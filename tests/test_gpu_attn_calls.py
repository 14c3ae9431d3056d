"""Calls of attention over the 4-bit cache that are allowed and out of the
ordinary."""
import pytest
import torch

import bit_blockwise_weight_nf4_b200 as bnb4
from bit_blockwise_weight_nf4_b200 import torch_ops  # noqa: F401
import oracle
from kv_ref import Case
from test_gpu_attn import ints, run, verify

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


@pytest.mark.parametrize("q_len", [1, 3, 50])
def test_windows_without_causality(q_len):
    case = Case([75, 1030, 20, 0], 48, 2, 64, 32, bnb4.FP4, oracle.BF16, seed=52)
    for window in (1, 30, 1 << 30, 0x7fffffff):
        verify(case, 4, [q_len] * 4, causal=False, window=window)


@pytest.mark.parametrize("q_len", [1, 30])
def test_pages_past_32_bits_of_bytes(q_len):
    """A cache of 5 GB per tensor of codes whose sequences lie on its last pages."""
    case = Case([700, 80], 256, 8, 128, 64, bnb4.NF4, oracle.BF16, seed=53, spare=0)
    q = case.queries(2 * q_len, 8)
    want, lse = run(case, q, [q_len] * 2)
    n = case.k_codes.shape[0]
    pages = 5 * (1 << 30) // (256 * 8 * 64)
    big = bnb4.KVCache4bit.empty(pages, 256, 8, 128, torch.bfloat16, 64, bnb4.NF4)
    big.k_codes[-n:], big.v_codes[-n:] = case.k_codes.cuda(), case.v_codes.cuda()
    big.k_absmax[-n:], big.v_absmax[-n:] = case.k_absmax.cuda(), case.v_absmax.cuda()
    case.block_table += pages - n
    got, lse2 = run(case, q, [q_len] * 2, cache=big)
    assert torch.equal(want, got) and torch.equal(lse, lse2)


@pytest.mark.parametrize("q_len", [1, 20])
def test_rows_past_32_bits_of_bytes(q_len):
    """Keys, values, queries and outputs whose rows lie 2^31 + 64 elements (4 GB)
    apart: written, attended to and read back."""
    T, step = 3 * q_len, (1 << 31) + 64 if q_len == 1 else (1 << 27) + 64
    case = Case([700, 80, 65], 16, 1, 64, 64, bnb4.NF4, oracle.F16, seed=54)
    q = case.queries(T, 1).cuda()
    c, bt, sl = case.cache(), case.block_table.cuda(), ints(case.kv_lens)
    room = torch.empty((T - 1) * step + 64, dtype=torch.float16, device="cuda")
    far = room.as_strided((T, 1, 64), (step, 64, 1))
    want = bnb4.attn_4bit(q, c, bt, sl)
    far.copy_(q)
    assert torch.equal(bnb4.attn_4bit(far, c, bt, sl), want)
    far.fill_(7)
    bnb4.attn_4bit(q, c, bt, sl, out=far)
    assert torch.equal(far, want)
    slots = torch.arange(T, device="cuda")
    a, b = (bnb4.KVCache4bit.empty(8, 16, 1, 64, torch.float16, 64) for _ in range(2))
    far.copy_(q)
    bnb4.kv_write_4bit(far, far, a, slots)
    bnb4.kv_write_4bit(q, q, b, slots)
    k = bnb4.kv_read_4bit(b, slots)[0]
    bnb4.kv_read_4bit(a, slots, out=(far, None))
    assert torch.equal(far, k)
    assert torch.equal(a.v_codes.view(-1, 32)[:T], b.v_codes.view(-1, 32)[:T])
