"""Writing rows into the 4-bit key/value cache and reading them back: codes
and scales bit for bit against the CPU oracle, values bit for bit against the
rounding of table * scale, at every head size, block size, code table and
type, odd token counts, strided inputs, shuffled and missing slots, and
special values."""
import numpy as np
import pytest
import torch

import bit_blockwise_weight_nf4_b200 as bnb4
import oracle
from kv_ref import TORCH, quantize_rows, stored_place

pytestmark = pytest.mark.gpu

SHAPES = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)]


def empty_cache(pages, page, heads, D, bs, qtype, dtype):
    c = bnb4.KVCache4bit.empty(pages, page, heads, D, TORCH[dtype], bs, qtype)
    for t in (c.k_codes, c.v_codes):
        t.fill_(0xA5)
    for t in (c.k_absmax, c.v_absmax):
        t.fill_(7.0)
    return c


def bits(t):
    return t.contiguous().view(torch.int16) if t.dtype in (torch.bfloat16, torch.float16) else \
        t.contiguous().view(torch.int32) if t.dtype == torch.float32 else t


def check_write(k, v, slots, page, pages, bs, qtype, dtype, kd=None, vd=None):
    """k, v: CPU [T, H, D]; kd, vd: the device tensors handed to the call."""
    T, H, D = k.shape
    c = empty_cache(pages, page, H, D, bs, qtype, dtype)
    before = [t.cpu().clone() for t in (c.k_codes, c.v_codes, c.k_absmax, c.v_absmax)]
    bnb4.kv_write_4bit(k.cuda() if kd is None else kd, v.cuda() if vd is None else vd, c,
                       slots.cuda())
    for x, codes, absmax, c0, a0 in ((k, c.k_codes, c.k_absmax, before[0], before[2]),
                                     (v, c.v_codes, c.v_absmax, before[1], before[3])):
        want_c, want_a, _ = quantize_rows(x, bs, qtype)
        ok = (slots >= 0) & (slots < pages * page)
        pg, sl = slots[ok] // page, slots[ok] % page
        c0[pg, :, sl] = want_c[ok]
        a0[pg, :, sl] = want_a[ok]
        assert torch.equal(codes.cpu(), c0)
        assert torch.equal(bits(absmax.cpu()), bits(a0))
    return c


@pytest.mark.parametrize("D,bs", SHAPES)
@pytest.mark.parametrize("qtype", [bnb4.NF4, bnb4.FP4])
@pytest.mark.parametrize("dtype", [oracle.BF16, oracle.F16])
@pytest.mark.parametrize("T,H,page", [(1, 1, 16), (7, 3, 48), (333, 2, 64)])
def test_write_and_read_every_format(D, bs, qtype, dtype, T, H, page):
    g = torch.Generator().manual_seed(T + D + bs)
    k, v = (torch.randn(T, H, D, generator=g).to(TORCH[dtype]) for _ in range(2))
    pages = -(-T // page) + 2
    slots = torch.randperm(pages * page, generator=g)[:T]
    c = check_write(k, v, slots, page, pages, bs, qtype, dtype)
    t = torch.from_numpy(oracle.codebook(qtype))
    for od in (torch.float32, torch.bfloat16, torch.float16):
        got = bnb4.kv_read_4bit(c, slots.cuda(), od)
        for x, y in zip((k, v), got):
            _, a, codes = quantize_rows(x, bs, qtype)
            want = (t[codes].unflatten(-1, (-1, bs)) * a.float().unsqueeze(-1)).flatten(-2).to(od)
            assert torch.equal(bits(y.cpu()), bits(want))


@pytest.mark.parametrize("dtype", [oracle.BF16, oracle.F16])
def test_write_strided_padded_and_out_of_range_slots(dtype):
    """Keys and values as parts of a fused projection's rows; slots of -1,
    behind the cache and far behind it leave their tokens out."""
    T, H, D, page, pages = 130, 4, 128, 32, 9
    qkv = torch.randn(T, 6 + 2 * H, D, generator=torch.Generator().manual_seed(3)).to(TORCH[dtype])
    k, v = qkv[:, 6:6 + H], qkv[:, 6 + H:]
    slots = torch.randperm(pages * page, generator=torch.Generator().manual_seed(4))[:T]
    slots[5], slots[17], slots[63], slots[129] = -1, pages * page, 1 << 40, -(1 << 50)
    d = qkv.cuda()
    c = check_write(k, v, slots, page, pages, 64, bnb4.NF4, dtype, d[:, 6:6 + H], d[:, 6 + H:])
    # rows of such slots are left as they were when reading, too
    out = [torch.full((T, H + 1, D), 3.5, dtype=TORCH[dtype], device="cuda") for _ in range(2)]
    bnb4.kv_read_4bit(c, slots.cuda(), out=(out[0][:, :H], out[1][:, 1:]))
    for i in (5, 17, 63, 129):
        assert (out[0][i] == 3.5).all() and (out[1][i] == 3.5).all()
    assert (out[0][:, H] == 3.5).all() and (out[1][:, 0] == 3.5).all()
    ref = bnb4.kv_read_4bit(c, slots.cuda())
    ok = torch.tensor([i not in (5, 17, 63, 129) for i in range(T)])
    assert torch.equal(out[0][:, :H].cpu()[ok], ref[0].cpu()[ok])
    assert torch.equal(out[1][:, 1:].cpu()[ok], ref[1].cpu()[ok])
    only = torch.empty(T, H, D, dtype=torch.float32, device="cuda")
    bnb4.kv_read_4bit(c, slots.cuda(), out=(None, only))
    assert torch.equal(only.to(TORCH[dtype]).cpu()[ok], ref[1].cpu()[ok])


@pytest.mark.parametrize("qtype", [bnb4.NF4, bnb4.FP4])
@pytest.mark.parametrize("dtype", [oracle.BF16, oracle.F16])
def test_write_special_values(qtype, dtype):
    """Zero, subnormal, huge, infinite and NaN blocks, and every value of the
    type against a block maximum of one (the decision points' neighbours)."""
    D, bs, page = 128, 64, 16
    tdt = TORCH[dtype]
    every = torch.arange(-32768, 32768, dtype=torch.int32).to(torch.int16).view(tdt)
    every = every[(every.float().abs() <= 1)]
    rows = -(-every.numel() // 63)
    x = torch.zeros(rows * 63, dtype=tdt)
    x[:every.numel()] = every
    x = torch.cat([torch.ones(rows, 1, dtype=tdt), x.view(rows, 63)], 1)
    x = torch.cat([x, torch.zeros(-rows % 2 + 16, 64, dtype=tdt)])
    x[-1, 3] = float("inf")
    x[-2, 5] = float("nan")
    x[-2, 6] = 2.0
    x[-3] = float("nan")
    x[-4, 0] = torch.finfo(tdt).tiny
    x[-4, 1] = -torch.finfo(tdt).tiny / 2
    x[-5, 7] = torch.finfo(tdt).smallest_normal / 64
    x[-5, 8] = -torch.finfo(tdt).smallest_normal / 128
    x[-6, 9] = torch.finfo(tdt).max
    x[-6, 10] = -torch.finfo(tdt).max / 3
    x[-7, 9] = -float("inf")
    x[-7, 10] = float("nan")
    x = x.view(-1, 1, D)
    T = x.shape[0]
    check_write(x, x.flip(0).contiguous(), torch.arange(T), page, -(-T // page), bs, qtype, dtype)


def test_write_equals_weight_quantizer():
    """A cache row is bnb_quantize_4bit's block codes in the stored order."""
    T, H, D, bs = 64, 2, 128, 64
    x = torch.randn(T, H, D, generator=torch.Generator().manual_seed(9)).to(torch.bfloat16).cuda()
    c = empty_cache(4, 16, H, D, bs, bnb4.NF4, oracle.BF16)
    bnb4.kv_write_4bit(x, x, c, torch.arange(T, device="cuda"))
    st = bnb4.quantize_4bit(x.view(-1), bs, bnb4.NF4, False)
    nat = torch.stack([st.codes >> 4, st.codes & 15], -1).view(T, H, D)
    sto = c.k_codes.transpose(1, 2).reshape(T, H, D // 2)
    sto = torch.stack([sto >> 4, sto & 15], -1).flatten(-2)
    assert torch.equal(sto[..., torch.from_numpy(stored_place(D, bs)).cuda()], nat)
    assert torch.equal(c.k_absmax.transpose(1, 2).reshape(-1).float(), st.absmax)


def test_empty_calls_and_large_strides():
    c = empty_cache(2, 16, 2, 64, 32, bnb4.NF4, oracle.F16)
    z = torch.zeros(0, 2, 64, dtype=torch.float16, device="cuda")
    none = torch.zeros(0, dtype=torch.int64, device="cuda")
    bnb4.kv_write_4bit(z, z, c, none)
    assert bnb4.kv_read_4bit(c, none)[0].shape == (0, 2, 64)
    assert (c.k_codes == 0xA5).all()
    # one token repeated through a zero stride, and a row stride of 4 GB
    x = torch.randn(1, 2, 64, generator=torch.Generator().manual_seed(5)).half().cuda()
    bnb4.kv_write_4bit(x.expand(5, 2, 64), x.expand(5, 2, 64), c, torch.arange(5, device="cuda"))
    k, _ = bnb4.kv_read_4bit(c, torch.arange(5, device="cuda"))
    assert all(torch.equal(k[i], k[0]) for i in range(5))


def test_offsets_past_32_bits():
    """A cache whose last page lies 5 GB in: codes and scales land there."""
    page, H, D, bs = 256, 32, 128, 64
    pages = 5 * (1 << 30) // (page * H * D // 2)
    c = bnb4.KVCache4bit.empty(pages, page, H, D, torch.bfloat16, bs, bnb4.NF4)
    last = pages * page - 1
    slots = torch.tensor([last, 0, last - 300], device="cuda")
    x = torch.randn(3, H, D, generator=torch.Generator().manual_seed(6)).to(torch.bfloat16)
    bnb4.kv_write_4bit(x.cuda(), x.flip(0).cuda(), c, slots)
    want, a, _ = quantize_rows(x, bs, bnb4.NF4)
    assert torch.equal(c.k_codes[pages - 1, :, page - 1].cpu(), want[0])
    assert torch.equal(c.k_absmax[pages - 1, :, page - 1].cpu(), a[0])
    assert torch.equal(c.v_codes[0, :, 0].cpu(), want[1])
    k, v = bnb4.kv_read_4bit(c, slots)
    small = bnb4.KVCache4bit.empty(1, 16, H, D, torch.bfloat16, bs, bnb4.NF4)
    at = torch.arange(3, device="cuda")
    bnb4.kv_write_4bit(x.cuda(), x.flip(0).cuda(), small, at)
    k2, v2 = bnb4.kv_read_4bit(small, at)
    assert torch.equal(k, k2) and torch.equal(v, v2)


def test_captured_write_then_read():
    """A captured write and read (programmatic launches) replayed on new
    inputs, on another stream than the default one."""
    T, H, D, bs = 40, 4, 128, 32
    c = empty_cache(4, 16, H, D, bs, bnb4.FP4, oracle.F16)
    x = torch.zeros(T, H, D, dtype=torch.float16, device="cuda")
    slots = torch.randperm(64, device="cuda")[:T]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        bnb4.kv_write_4bit(x, x, c, slots)
        out = bnb4.kv_read_4bit(c, slots)
    s.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        y = x * 2
        bnb4.kv_write_4bit(y, x, c, slots)
        out = bnb4.kv_read_4bit(c, slots)
    for seed in (1, 2):
        x.copy_(torch.randn(T, H, D, generator=torch.Generator().manual_seed(seed)))
        gr.replay()
        e = empty_cache(4, 16, H, D, bs, bnb4.FP4, oracle.F16)
        bnb4.kv_write_4bit(x * 2, x, e, slots)
        want = bnb4.kv_read_4bit(e, slots)
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
