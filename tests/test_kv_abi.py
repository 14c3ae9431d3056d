"""The 4-bit key/value cache without a GPU: the C entry points refuse bad
arguments with the documented status before any CUDA call, the Python calls
refuse bad tensors, the workspace query is a host function, the operators'
fakes give shapes, and the stored order is a permutation that every part of
the layout's description agrees with."""
import numpy as np
import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

import bit_blockwise_weight_nf4_b200 as bnb4
from bit_blockwise_weight_nf4_b200 import torch_ops  # noqa: F401
from kv_ref import stored_place

A = 0x10000  # never dereferenced: every call below fails its checks first


@pytest.fixture(scope="module", autouse=True)
def lib():
    from bit_blockwise_weight_nf4_b200 import build
    build.build()
    return bnb4.load()


def cache(**kw):
    c = bnb4.KvCache(A, A, A, A, 4, 16, 2, 128, 64, bnb4.NF4, bnb4.BF16, 0)
    for k, v in kw.items():
        setattr(c, k, v)
    return c


CACHE_ERRORS = [
    (dict(k_codes=None), bnb4.ERR_INVALID_ARG), (dict(v_codes=None), bnb4.ERR_INVALID_ARG),
    (dict(k_absmax=None), bnb4.ERR_INVALID_ARG), (dict(v_absmax=None), bnb4.ERR_INVALID_ARG),
    (dict(reserved=1), bnb4.ERR_INVALID_ARG), (dict(qtype=2), bnb4.ERR_INVALID_ARG),
    (dict(dtype=bnb4.F32), bnb4.ERR_UNSUPPORTED), (dict(head_dim=96), bnb4.ERR_UNSUPPORTED),
    (dict(head_dim=256), bnb4.ERR_UNSUPPORTED), (dict(blocksize=16), bnb4.ERR_UNSUPPORTED),
    (dict(blocksize=256), bnb4.ERR_UNSUPPORTED),
    (dict(head_dim=64, blocksize=128), bnb4.ERR_UNSUPPORTED),
    (dict(num_pages=0), bnb4.ERR_SHAPE), (dict(page_size=8), bnb4.ERR_SHAPE),
    (dict(page_size=40), bnb4.ERR_SHAPE), (dict(n_kv_heads=0), bnb4.ERR_SHAPE),
    (dict(num_pages=1 << 28), bnb4.ERR_SHAPE), (dict(k_codes=A + 8), bnb4.ERR_ALIGNMENT),
    (dict(v_absmax=A + 2), bnb4.ERR_ALIGNMENT),
]


@pytest.mark.parametrize("kw,want", CACHE_ERRORS)
def test_cache_errors(kw, want):
    c = cache(**kw)
    assert bnb4.bnb_kv_write_4bit(A, 256, 128, A, 256, 128, 1, A, c, None) == want
    assert bnb4.bnb_kv_read_4bit(c, A, 1, A, 256, 128, A, 256, 128, bnb4.BF16, None) == want
    assert bnb4.bnb_attn_4bit(attn(cache=c), None) == want
    assert bnb4.bnb4_attn_workspace(attn(cache=c))[0] == want


def test_write_errors():
    def call(k=A, kt=256, kh=128, v=A, vt=256, vh=128, n=1, slots=A):
        return bnb4.bnb_kv_write_4bit(k, kt, kh, v, vt, vh, n, slots, cache(), None)
    assert call(n=-1) == bnb4.ERR_SHAPE
    assert call(n=0, k=None, slots=None) == bnb4.OK
    assert call(k=None) == bnb4.ERR_INVALID_ARG and call(v=None) == bnb4.ERR_INVALID_ARG
    assert call(slots=None) == bnb4.ERR_INVALID_ARG
    assert call(slots=A + 4) == bnb4.ERR_ALIGNMENT
    assert call(kt=-256) == bnb4.ERR_SHAPE and call(vh=-8) == bnb4.ERR_SHAPE
    assert call(kt=252) == bnb4.ERR_ALIGNMENT and call(vh=4) == bnb4.ERR_ALIGNMENT
    assert call(k=A + 8) == bnb4.ERR_ALIGNMENT and call(v=A + 2) == bnb4.ERR_ALIGNMENT
    assert call(n=1 << 30) == bnb4.ERR_SHAPE


def test_read_errors():
    def call(k=A, kt=256, kh=128, v=A, vt=256, vh=128, n=1, slots=A, dt=bnb4.F32):
        return bnb4.bnb_kv_read_4bit(cache(), slots, n, k, kt, kh, v, vt, vh, dt, None)
    assert call(n=-1) == bnb4.ERR_SHAPE and call(n=0, k=None, v=None) == bnb4.OK
    assert call(dt=5) == bnb4.ERR_UNSUPPORTED
    assert call(k=None, v=None) == bnb4.ERR_INVALID_ARG
    assert call(slots=None) == bnb4.ERR_INVALID_ARG
    assert call(kt=250) == bnb4.ERR_ALIGNMENT and call(kt=-4) == bnb4.ERR_SHAPE
    assert call(kt=252, dt=bnb4.BF16) == bnb4.ERR_ALIGNMENT
    assert call(k=None, kt=3, v=A + 4) == bnb4.ERR_ALIGNMENT
    # rows that would lie over one another
    assert call(n=2, kt=64) == bnb4.ERR_SHAPE and call(vh=64) == bnb4.ERR_SHAPE
    assert call(n=1 << 30) == bnb4.ERR_SHAPE


def attn(**kw):
    d = dict(q=A, q_stride_t=1024, q_stride_h=128, out=A, out_stride_t=1024, out_stride_h=128,
             lse=None, cache=cache(), block_table=A, block_table_stride=8, seq_lens=A,
             cu_seqlens_q=None, workspace=A, workspace_bytes=1 << 30, total_q=3, batch=3,
             n_heads=8, max_q_len=1, max_seq_len=100000, block_table_width=8, causal=1, window=0,
             scale=0.1, reserved=0)
    d.update(kw)
    a = bnb4.Attn()
    a._keep = d["cache"]
    for k, v in d.items():
        setattr(a, k, bnb4.ctypes.pointer(v) if k == "cache" else v)
    return a


@pytest.mark.parametrize("kw,want", [
    (dict(q=None), bnb4.ERR_INVALID_ARG), (dict(out=None), bnb4.ERR_INVALID_ARG),
    (dict(block_table=None), bnb4.ERR_INVALID_ARG), (dict(seq_lens=None), bnb4.ERR_INVALID_ARG),
    (dict(reserved=1), bnb4.ERR_INVALID_ARG), (dict(causal=2), bnb4.ERR_INVALID_ARG),
    (dict(scale=0.0), bnb4.ERR_INVALID_ARG), (dict(scale=float("nan")), bnb4.ERR_INVALID_ARG),
    (dict(scale=-1.0), bnb4.ERR_INVALID_ARG), (dict(scale=float("inf")), bnb4.ERR_INVALID_ARG),
    (dict(batch=-1), bnb4.ERR_SHAPE), (dict(total_q=-1), bnb4.ERR_SHAPE),
    (dict(max_q_len=0), bnb4.ERR_SHAPE), (dict(window=-1), bnb4.ERR_SHAPE),
    (dict(max_seq_len=-1), bnb4.ERR_SHAPE), (dict(n_heads=7), bnb4.ERR_SHAPE),
    (dict(n_heads=0), bnb4.ERR_SHAPE), (dict(total_q=4), bnb4.ERR_SHAPE),
    (dict(block_table_width=0), bnb4.ERR_SHAPE), (dict(block_table_stride=7), bnb4.ERR_SHAPE),
    (dict(q_stride_t=-8), bnb4.ERR_SHAPE), (dict(q_stride_t=12), bnb4.ERR_ALIGNMENT),
    (dict(out_stride_h=0), bnb4.ERR_SHAPE), (dict(out_stride_t=64), bnb4.ERR_SHAPE),
    (dict(out_stride_h=4), bnb4.ERR_ALIGNMENT), (dict(q=A + 8), bnb4.ERR_ALIGNMENT),
    (dict(out=A + 2), bnb4.ERR_ALIGNMENT), (dict(lse=A + 2), bnb4.ERR_ALIGNMENT),
    (dict(seq_lens=A + 1), bnb4.ERR_ALIGNMENT), (dict(cu_seqlens_q=A + 2), bnb4.ERR_ALIGNMENT),
    (dict(workspace=None), bnb4.ERR_WORKSPACE), (dict(workspace_bytes=64), bnb4.ERR_WORKSPACE),
    (dict(workspace=A + 4), bnb4.ERR_ALIGNMENT),
    (dict(batch=0, total_q=0), bnb4.OK), (dict(total_q=0, batch=2, cu_seqlens_q=A), bnb4.OK),
])
def test_attn_errors(kw, want):
    assert bnb4.bnb_attn_4bit(attn(**kw), None) == want


def test_workspace_is_a_host_function():
    rc, n = bnb4.bnb4_attn_workspace(attn(workspace=None, workspace_bytes=0))
    assert rc == 0 and n > 0
    assert bnb4.load().bnb4_attn_workspace(bnb4.ctypes.byref(attn()), None) == \
        bnb4.ERR_INVALID_ARG


@pytest.mark.parametrize("D,bs", [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)])
def test_stored_order(D, bs):
    place = stored_place(D, bs)
    assert sorted(place) == list(range(D))
    if D == bs:
        assert (place == np.arange(D)).all()
    # strip s of a row holds values [s w, (s + 1) w) of each block
    w = bs // 8
    for s in range(8):
        dims = [d for d in range(D) if place[d] // (D // 8) == s]
        assert dims == [b * bs + s * w + i for b in range(D // bs) for i in range(w)]


def test_tensors_are_checked():
    c = bnb4.KVCache4bit.empty(4, 16, 2, 128, torch.bfloat16, 64, bnb4.NF4, device="cpu")
    assert c.nbytes == 2 * 4 * 2 * 16 * (64 + 4) and c.head_dim == 128
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int64)
    for bad in ((k.half(), k, slots), (k, k[:2], slots), (k[:, :1], k[:, :1], slots),
                (k[..., :64], k, slots), (k, k, slots.int()), (k, k, slots[:2]),
                (k.transpose(1, 2), k, slots)):
        with pytest.raises((ValueError, RuntimeError)):
            bnb4.kv_write_4bit(bad[0], bad[1], c, bad[2])
    with pytest.raises(TypeError):
        bnb4.kv_read_4bit(c, slots, out=(k.double(), None))
    with pytest.raises(ValueError):
        bnb4.kv_read_4bit(c, slots, out=(None, None))
    q = torch.zeros(3, 4, 128, dtype=torch.bfloat16)
    bt, sl = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    for bad in ((q.half(), bt, sl, None), (q, bt.long(), sl, None), (q, bt, sl[:2], None),
                (q[:2], bt, sl, None), (q, bt, sl, sl), (q, bt[0], sl, None),
                (q[..., :64], bt, sl, None)):
        with pytest.raises((ValueError, RuntimeError)):
            bnb4.attn_4bit(bad[0], c, bad[1], bad[2], bad[3])
    with pytest.raises(ValueError):
        bnb4.attn_4bit(q, c, bt, sl, lse=torch.zeros(3, 4, dtype=torch.float64))
    with pytest.raises(ValueError):
        bnb4.KVCache4bit(c.k_codes, c.v_codes[:2], c.k_absmax, c.v_absmax, 64)
    with pytest.raises(ValueError):
        bnb4.KVCache4bit(c.k_codes, c.v_codes, c.k_absmax, c.v_absmax, 32)
    with pytest.raises(TypeError):
        bnb4.KVCache4bit(c.k_codes, c.v_codes, c.k_absmax.float(), c.v_absmax.float(), 64)


def test_fakes():
    with FakeTensorMode():
        codes = [torch.empty(4, 2, 16, 64, dtype=torch.uint8, device="cuda") for _ in range(2)]
        scales = [torch.empty(4, 2, 16, 2, dtype=torch.float16, device="cuda") for _ in range(2)]
        slots = torch.empty(5, dtype=torch.int64, device="cuda")
        k = torch.empty(5, 2, 128, dtype=torch.float16, device="cuda")
        torch.ops.bnb4.kv_write_4bit(k, k, *codes, *scales, slots, 64, bnb4.NF4)
        a, b = torch.ops.bnb4.kv_read_4bit(*codes, *scales, slots, 64, bnb4.NF4, torch.float32)
        q = torch.empty(3, 8, 128, dtype=torch.float16, device="cuda")
        bt = torch.empty(3, 2, dtype=torch.int32, device="cuda")
        sl = torch.empty(3, dtype=torch.int32, device="cuda")
        o = torch.ops.bnb4.attn_4bit(q, *codes, *scales, bt, sl, None, 1, 32, 0.1, True, 0, 64,
                                     bnb4.NF4)
    assert a.shape == b.shape == (5, 2, 128) and a.dtype == torch.float32
    assert o.shape == q.shape and o.dtype == torch.float16 and o.device.type == "cuda"
