"""Calls of the 4-bit key/value cache that are settled on the host, without a
GPU: what they refuse, and what they answer at once."""
import numpy as np
import pytest
import torch

import bit_blockwise_weight_nf4_b200 as bnb4
from test_kv_abi import A, attn, cache


@pytest.fixture(scope="module", autouse=True)
def lib():
    from bit_blockwise_weight_nf4_b200 import build
    build.build()
    return bnb4.load()


def test_failure_diagnostic_checks_its_limit_and_arguments():
    for limit in (0, -1, 1000001):
        assert bnb4.bnb4_debug_attn_withhold(attn(), limit, None) == bnb4.ERR_INVALID_ARG
    assert bnb4.bnb4_debug_attn_withhold(attn(out=None), 1000, None) == bnb4.ERR_INVALID_ARG
    assert bnb4.bnb4_debug_attn_withhold(attn(window=-1), 1000, None) == bnb4.ERR_SHAPE
    assert bnb4.bnb4_debug_attn_withhold(attn(batch=0, total_q=0), 1000, None) == bnb4.OK


# (tokens, heads, token stride, head stride) in elements, rows of 128: do any two
# rows share an element?
OVERLAPS = [(2, 2, 128, 128, True), (2, 2, 256, 128, False), (2, 2, 128, 256, False),
            (3, 2, 128, 256, True), (3, 2, 128, 384, False), (2, 3, 256, 128, True),
            (2, 3, 384, 128, False), (2, 2, 384, 256, False), (3, 3, 384, 256, False),
            (3, 4, 384, 256, True),
            (3, 2, 384, 512, False), (2, 2, 256, 248, True), (2, 2, 256, 136, True),
            (1, 8, 0, 128, False), (8, 1, 128, 0, False), (5, 4, 128, 136, True),
            (4, 5, 136, 128, True), (1000, 2, 128, 128000, False), (1001, 2, 128, 128000, True),
            (2, 2, 1 << 62, (1 << 62) + 64, True), (2, 3, (1 << 62) + 64, 1 << 61, True),
            (2, 2, 1 << 62, (1 << 62) + 128, False), (70, 50, 49 * 128, 50 * 128, True),
            (50, 49, 49 * 128, 50 * 128, False)]


@pytest.mark.parametrize("tokens,heads,ts,hs,shared", OVERLAPS)
def test_rows_that_are_written_do_not_overlap(tokens, heads, ts, hs, shared):
    rows = np.add.outer(np.arange(tokens, dtype=object) * ts, np.arange(heads, dtype=object) * hs)
    rows = sorted(rows.ravel())
    assert shared == any(b - a < 128 for a, b in zip(rows, rows[1:]))
    c = cache(n_kv_heads=heads)
    read = lambda *kv: bnb4.bnb_kv_read_4bit(c, A, tokens, *kv, bnb4.BF16, None)
    fine = (A, heads * 128, 128)
    got = [read(A, ts, hs, A + (1 << 30), *fine[1:]), read(A + (1 << 30), *fine[1:], A, ts, hs),
           read(None, 0, 0, A, ts, hs),
           bnb4.bnb_attn_4bit(attn(cache=c, n_heads=heads, total_q=tokens, batch=tokens,
                                   out_stride_t=ts, out_stride_h=hs), None)]
    assert [rc == bnb4.ERR_SHAPE for rc in got] == [shared] * 4, got


def test_keys_and_values_are_not_read_into_one_place():
    got = bnb4.bnb_kv_read_4bit(cache(), A, 2, A, 256, 128, A, 256, 128, bnb4.BF16, None)
    assert got == bnb4.ERR_SHAPE


def test_no_queries_is_an_empty_call():
    """Sequences without new queries: nothing to do, with and without offsets."""
    for kw in (dict(), dict(cu_seqlens_q=A)):
        a = attn(total_q=0, batch=3, q=None, out=None, workspace=None, workspace_bytes=0, **kw)
        assert bnb4.bnb4_attn_workspace(a) == (bnb4.OK, 0)
        assert bnb4.bnb_attn_4bit(a, None) == bnb4.OK
    assert bnb4.bnb_attn_4bit(attn(total_q=0, batch=3, scale=0.0), None) == bnb4.ERR_INVALID_ARG


def cpu_call(**kw):
    """attn_4bit on CPU tensors: a call without a fault fails for the device."""
    c = bnb4.KVCache4bit.empty(40, 64, 2, 128, torch.bfloat16, 64, bnb4.NF4, device="cpu")
    q = torch.zeros(3, 4, 128, dtype=torch.bfloat16)
    bt, sl = torch.zeros(3, 40, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    cu = torch.zeros(4, dtype=torch.int32) if "max_q_len" in kw else None
    return bnb4.attn_4bit(q, c, bt, sl, cu, **kw)


@pytest.mark.parametrize("name", ["window", "max_q_len", "max_seq_len"])
@pytest.mark.parametrize("value", [(1 << 32) + 5, 1 << 31, -(1 << 32) + 1, 1 << 70])
def test_numbers_past_32_bits_are_refused(name, value):
    """They would be cut to their low 32 bits on the way: another window, rows left out."""
    with pytest.raises(ValueError, match="CUDA device"):
        cpu_call(**{name: 5})
    with pytest.raises(ValueError, match=name):
        cpu_call(**{name: value})


def test_code_types_past_32_bits_are_refused():
    c = bnb4.KVCache4bit.empty(4, 16, 2, 128, torch.bfloat16, 64, bnb4.NF4, device="cpu")
    for qtype in (1 << 32, (1 << 32) + 1, 2, -1):
        with pytest.raises(ValueError, match="qtype"):
            bnb4.KVCache4bit(c.k_codes, c.v_codes, c.k_absmax, c.v_absmax, 64, qtype)


def test_workspaces_are_checked():
    """A workspace is memory on the cache's device, counted in bytes."""
    ok = torch.empty(1 << 24, dtype=torch.uint8)
    with pytest.raises(ValueError, match="CUDA device"):
        cpu_call(workspace=ok)
    with pytest.raises(ValueError, match="CUDA device"):  # as many bytes in other elements
        cpu_call(workspace=ok.view(torch.float32))
    small = torch.empty(16, dtype=torch.uint8)
    for bad in (small.expand(1 << 20, 16), ok[::2], ok.view(4096, 4096).t(),
                torch.empty(1 << 24, dtype=torch.uint8, device="meta")):
        with pytest.raises(ValueError, match="workspace"):
            cpu_call(workspace=bad)
