"""Attention over the 4-bit key/value cache against the 64-bit reference: one
token per sequence, a few, and chunks; every format; ragged, empty and
one-token sequences; windows; missing pages; unseen garbage; captured graphs;
streams; and the run write -> attend -> read of a decoder."""
import math

import pytest
import torch

import bit_blockwise_weight_nf4_b200 as bnb4
from bit_blockwise_weight_nf4_b200 import torch_ops  # noqa: F401
import oracle
from kv_ref import Case, attention64, check

pytestmark = pytest.mark.gpu

SHAPES = [(64, 32), (64, 64), (128, 32), (128, 64), (128, 128)]


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def cu_of(q_lens):
    return ints([0] + list(torch.tensor(q_lens).cumsum(0)))


def run(case, q, q_lens, cache=None, **kw):
    same = len(set(q_lens)) == 1 and "cu" not in kw
    cu = kw.pop("cu", None)
    lse = torch.full(q.shape[:2], 123.0, device="cuda")
    out = bnb4.attn_4bit(q.cuda(), cache or case.cache(), case.block_table.cuda(),
                         ints(case.kv_lens), cu_seqlens_q=None if same else
                         (cu_of(q_lens) if cu is None else cu),
                         max_q_len=max(1, max(q_lens)), lse=lse, **kw)
    torch.cuda.synchronize()
    assert bnb4.bnb4_device_status(torch.cuda.current_stream().cuda_stream) == 0
    return out, lse


def verify(case, n_heads, q_lens, std=1.0, causal=True, window=0, scale=None, **kw):
    q = case.queries(sum(q_lens), n_heads, std)
    out, lse = run(case, q, q_lens, causal=causal, window=window, scale=scale, **kw)
    o64, bound, l64, lb = attention64(case, q, q_lens, causal, window, scale)
    check(out, o64, bound, case.dtype)
    lse = lse.cpu().double()
    empty = torch.isinf(l64)
    assert torch.equal(torch.isinf(lse), empty)
    assert (out.cpu()[empty] == 0).all()
    assert ((lse - l64).abs()[~empty] <= lb[~empty]).all()
    return out


@pytest.mark.parametrize("D,bs", SHAPES)
@pytest.mark.parametrize("qtype", [bnb4.NF4, bnb4.FP4])
@pytest.mark.parametrize("dtype", [oracle.BF16, oracle.F16])
@pytest.mark.parametrize("group,q_len", [(1, 1), (4, 1), (5, 3), (4, 11)])
def test_every_format(D, bs, qtype, dtype, group, q_len):
    """1, 4, 15 and 44 rows per key/value head; ragged contexts."""
    case = Case([131, 16, 77], 32, 2, D, bs, qtype, dtype, seed=D + bs + group)
    verify(case, 2 * group, [q_len] * 3)


@pytest.mark.parametrize("page", [16, 48, 64, 256])
@pytest.mark.parametrize("dtype", [oracle.BF16, oracle.F16])
def test_lengths_from_nothing_to_long(page, dtype):
    """Empty sequences, one token, tile and page borders, and a context that
    many runs share."""
    lens = [0, 1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 511, 512, 513, 2999]
    case = Case(lens, page, 1, 128, 64, bnb4.NF4, dtype, seed=page)
    verify(case, 2, [1] * len(lens))


@pytest.mark.parametrize("n_heads,heads", [(8, 8), (8, 1), (16, 1), (14, 2)])
def test_long_contexts_are_split(n_heads, heads):
    case = Case([20011, 5], 64, heads, 128, 128, bnb4.NF4, oracle.BF16, seed=3)
    verify(case, n_heads, [1, 1])


@pytest.mark.parametrize("max_seq_len", [0, 1, 100000, None])
def test_bound_of_lengths_changes_nothing_but_the_split(max_seq_len):
    case = Case([700, 1300, 40], 32, 2, 64, 64, bnb4.FP4, oracle.BF16, seed=4)
    verify(case, 8, [1, 1, 1], max_seq_len=max_seq_len)


@pytest.mark.parametrize("q_lens", [[3, 0, 1, 4], [0, 0, 0, 2], [17, 1, 40, 0]])
@pytest.mark.parametrize("causal", [True, False])
def test_ragged_queries(q_lens, causal):
    """Sequences with and without queries, and one shorter than its queries
    (rows that see nothing)."""
    case = Case([90, 50, 700, 1], 16, 2, 128, 32, bnb4.NF4, oracle.BF16, seed=5)
    verify(case, 8, q_lens, causal=causal)


@pytest.mark.parametrize("window", [1, 7, 16, 100, 1000])
@pytest.mark.parametrize("q_len", [1, 4, 70])
def test_windows(window, q_len):
    case = Case([75, 1030, 20], 48, 1, 128, 64, bnb4.NF4, oracle.F16, seed=window)
    verify(case, 4, [q_len] * 3, window=window)


def test_sequence_shorter_than_its_queries():
    case = Case([3, 0, 20], 16, 1, 64, 32, bnb4.NF4, oracle.BF16, seed=8)
    verify(case, 2, [5, 5, 25])


def test_many_sequences():
    """More sequences than the schedule's search takes in one step."""
    lens = [(37 * i) % 91 for i in range(100)]
    lens[70] = 1500
    case = Case(lens, 16, 1, 64, 64, bnb4.NF4, oracle.BF16, seed=9)
    verify(case, 2, [1] * 100)
    verify(case, 2, [i % 3 for i in range(100)])


@pytest.mark.parametrize("std,scale", [(30.0, None), (1e-3, None), (1.0, 2.0), (0.0, None)])
def test_peaked_and_flat_scores(std, scale):
    case = Case([400, 33], 32, 2, 128, 128, bnb4.FP4, oracle.BF16, seed=10)
    verify(case, 4, [1, 1], std=std, scale=scale)


@pytest.mark.parametrize("dtype", [oracle.BF16, oracle.F16])
@pytest.mark.parametrize("q_len", [1, 24])
def test_value_scales_of_many_sizes(dtype, q_len):
    case = Case([600], 64, 1, 128, 32, bnb4.NF4, dtype, seed=11, sink=True)
    verify(case, 4, [q_len])


def test_very_large_and_small_inputs():
    for ks, vs, qs in ((2.0 ** 60, 2.0 ** -60, 2.0 ** -60), (2.0 ** -70, 2.0 ** 90, 2.0 ** 70)):
        case = Case([100], 16, 1, 64, 32, bnb4.NF4, oracle.BF16, seed=12, k_std=ks, v_std=vs)
        verify(case, 2, [1], std=qs)
        verify(case, 2, [20], std=qs)


@pytest.mark.parametrize("q_len", [1, 3, 40])
def test_what_no_query_sees_may_be_anything(q_len):
    """Pages behind the end, before the window and of no sequence hold NaN
    and infinite scales and any code: outputs do not change."""
    case = Case([205, 130], 16, 2, 128, 64, bnb4.NF4, oracle.BF16, seed=13, spare=4)
    q = case.queries(2 * q_len, 4)
    kw = dict(window=60)
    clean, lse = run(case, q, [q_len] * 2, **kw)
    bad = torch.tensor([float("nan"), float("inf"), 3e38, -float("inf")], dtype=torch.bfloat16)
    for absmax, codes in ((case.k_absmax, case.k_codes), (case.v_absmax, case.v_codes)):
        used = torch.zeros(absmax.shape[0], case.page, dtype=torch.bool)
        for b, kv in enumerate(case.kv_lens):
            first = max(0, kv - q_len - 60 + 1)
            for j in range(first, kv):
                used[case.block_table[b, j // case.page], j % case.page] = True
        hit = ~used[:, None, :].expand(absmax.shape[:3])
        n = int(hit.sum())
        absmax[hit] = bad[torch.arange(n) % 4][:, None].expand(n, absmax.shape[-1])
        codes[hit] = 0xff
    dirty, lse2 = run(case, q, [q_len] * 2, **kw)
    assert torch.equal(clean, dirty) and torch.equal(lse, lse2)


def test_pages_out_of_range_are_not_seen():
    case = Case([150, 64, 40], 16, 1, 64, 64, bnb4.NF4, oracle.BF16, seed=14)
    case.block_table[0, 2] = -1
    case.block_table[0, 7] = case.k_codes.shape[0]
    case.block_table[1, :] = 1 << 30
    case.block_table[2, 0] = -(1 << 31)
    for T in (3, 60):  # few rows, and a chunk
        q = case.queries(T, 2)
        o64, bound, l64, _ = attention64(case, q, [T // 3] * 3)
        out, lse = run(case, q, [T // 3] * 3)
        # the second sequence's pages are all missing: it sees nothing
        check(out, o64, bound, case.dtype)
        n = T // 3
        assert (out[n:2 * n] == 0).all() and torch.isinf(lse[n:2 * n]).all()
        assert torch.equal(torch.isinf(lse.cpu()), torch.isinf(l64))


def test_lengths_past_the_block_table_are_cut():
    case = Case([64, 64], 16, 1, 64, 64, bnb4.NF4, oracle.BF16, seed=15)
    q = case.queries(2, 2)
    want, _ = run(case, q, [1, 1])
    case.kv_lens = [64, 64]
    got = bnb4.attn_4bit(q.cuda(), case.cache(), case.block_table.cuda(), ints([1 << 30, 2147483647]))
    none = bnb4.attn_4bit(q.cuda(), case.cache(), case.block_table.cuda(), ints([-5, -(1 << 31)]))
    assert torch.equal(want, got) and (none == 0).all()


def test_rows_of_no_sequence_are_left_alone():
    case = Case([90, 33], 16, 2, 128, 64, bnb4.NF4, oracle.BF16, seed=16)
    for q_lens in ([1, 1], [3, 2], [30, 9]):
        T = sum(q_lens)
        q = case.queries(T + 5, 4)
        out = torch.full((T + 5, 4, 128), 9.0, dtype=torch.bfloat16, device="cuda")
        cu = cu_of(q_lens)
        bnb4.attn_4bit(q.cuda(), case.cache(), case.block_table.cuda(), ints(case.kv_lens), cu,
                       max(q_lens), out=out)
        assert (out[T:] == 9).all()
        o64, bound, _, _ = attention64(case, q[:T], q_lens)
        check(out[:T], o64, bound, case.dtype)
        # offsets that point outside q stay inside it
        out.fill_(9)
        bnb4.attn_4bit(q.cuda(), case.cache(), case.block_table.cuda(), ints(case.kv_lens),
                       ints([-7, q_lens[0], 1 << 30]), max(q_lens), out=out)
        torch.cuda.synchronize()


def test_strided_queries_and_outputs():
    """q as part of a fused projection's rows, out with gaps and heads apart."""
    case = Case([260, 31], 32, 2, 128, 64, bnb4.NF4, oracle.BF16, seed=17)
    for n in (1, 12):
        qkv = torch.randn(2 * n, 12, 128, generator=case.gen).to(torch.bfloat16)
        q = qkv[:, 1:9]
        big = torch.full((8, 2 * n, 2, 128), 5.0, dtype=torch.bfloat16, device="cuda")
        out = big[:, :, 1].transpose(0, 1)
        bnb4.attn_4bit(qkv.cuda()[:, 1:9], case.cache(), case.block_table.cuda(),
                       ints(case.kv_lens), out=out)
        o64, bound, _, _ = attention64(case, q, [n, n])
        check(out, o64, bound, case.dtype)
        assert (big[:, :, 0] == 5).all()


@pytest.mark.parametrize("q_len,n_heads", [(1, 2), (2, 8), (50, 4)])
def test_results_repeat(q_len, n_heads):
    case = Case([3000, 777, 12], 64, 2, 128, 64, bnb4.NF4, oracle.BF16, seed=18)
    q = case.queries(3 * q_len, n_heads)
    c = case.cache()
    a, la = run(case, q, [q_len] * 3, cache=c)
    for _ in range(3):
        b, lb = run(case, q, [q_len] * 3, cache=c)
        assert torch.equal(a, b) and torch.equal(la, lb)


@pytest.mark.parametrize("q_len", [1, 2, 33])
def test_nan_and_infinite_inputs_stay_in_their_rows(q_len):
    case = Case([200, 64], 32, 2, 64, 32, bnb4.NF4, oracle.BF16, seed=19)
    q = case.queries(2 * q_len, 4)
    want, _ = run(case, q, [q_len] * 2)
    for value in (float("nan"), float("inf"), -float("inf")):
        x = q.clone()
        x[0, 1, 5] = value
        out, _ = run(case, x, [q_len] * 2)
        assert torch.isnan(out[0, 1].float()).all()
        keep = torch.ones(out.shape[:2], dtype=torch.bool)
        keep[0, 1] = False
        assert torch.equal(out.cpu()[keep], want.cpu()[keep])


@pytest.mark.parametrize("q_len", [1, 3, 40])
def test_captured_decode_with_other_lengths(q_len):
    """One capture serves later lengths, pages and queries; two captured
    graphs with workspaces of their own may run at once."""
    lens = [300, 2000, 64]
    case = Case(lens, 32, 2, 128, 64, bnb4.NF4, oracle.BF16, seed=20)
    c = case.cache()
    bt = case.block_table.cuda()
    graphs = []
    for _ in range(2):
        q = case.queries(3 * q_len, 8).cuda()
        sl = ints([1, 1, 1])
        bnb4.attn_4bit(q, c, bt, sl, max_seq_len=2000)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = q * 1
            out = bnb4.attn_4bit(y, c, bt, sl, max_seq_len=2000)
        graphs.append((g, q, sl, out))
    streams = [torch.cuda.Stream() for _ in graphs]
    for lens2 in ([300, 2000, 64], [7, 0, 33], [250, 1999, 1]):
        for (g, q, sl, out), s in zip(graphs, streams):
            sl.copy_(ints(lens2))
        torch.cuda.synchronize()
        for (g, q, sl, out), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for g, q, sl, out in graphs:
            want = bnb4.attn_4bit(q, c, bt, sl, max_seq_len=2000)
            assert torch.equal(out, want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_decoder_write_attend_read(dtype):
    """A prompt in two chunks, then single tokens, as a decoder runs them: the
    4-bit linears' projections are written, attended to and read back."""
    H, HK, D, hidden, page = 8, 2, 128, 512, 16
    g = torch.Generator().manual_seed(21)
    W = torch.randn((H + 2 * HK) * D, hidden, generator=g).mul_(0.05).to(dtype).cuda()
    st = bnb4.quantize_4bit(W.view(-1), 64, bnb4.NF4, True)
    cache = bnb4.KVCache4bit.empty(16, page, HK, D, dtype)
    bt = torch.randperm(16, generator=g).int().view(1, 16).cuda()
    pos, outs, qs = 0, [], []
    for n in (37, 60, 1, 1, 2):
        x = torch.randn(n, hidden, generator=g).to(dtype).cuda()
        qkv = bnb4.linear_4bit(x, st, (H + 2 * HK) * D).view(n, H + 2 * HK, D)
        at = torch.arange(pos, pos + n, device="cuda")
        slots = bt[0, at // page].long() * page + at % page
        bnb4.kv_write_4bit(qkv[:, H:H + HK], qkv[:, H + HK:], cache, slots)
        pos += n
        outs.append(bnb4.attn_4bit(qkv[:, :H], cache, bt, ints([pos])))
        qs.append(qkv[:, :H].cpu())
    at = torch.arange(pos, device="cuda")
    slots = bt[0, at // page].long() * page + at % page
    k, v = (x.double().cpu() for x in bnb4.kv_read_4bit(cache, slots, torch.float32))
    q = torch.cat(qs).double().view(pos, HK, H // HK, D)
    s = torch.einsum("ihgd,jhd->hgij", q, k) / math.sqrt(D)
    s.masked_fill_(torch.ones(pos, pos, dtype=torch.bool).triu(1), -math.inf)
    want = torch.einsum("hgij,jhd->ihgd", torch.softmax(s, -1), v).reshape(pos, H, D)
    got = torch.cat(outs).double().cpu()
    rel = float((got - want).norm() / want.norm())
    assert rel <= (2e-3 if dtype == torch.bfloat16 else 5e-4)


def test_operators():
    """The calls as torch operators: schema, fake against real, mutation."""
    case = Case([90, 33], 16, 2, 64, 32, bnb4.FP4, oracle.F16, seed=22)
    c = case.cache()
    ts = (c.k_codes, c.v_codes, c.k_absmax, c.v_absmax)
    bt, sl = case.block_table.cuda(), ints(case.kv_lens)
    k, v = (case.queries(4, 2).cuda() for _ in range(2))
    slots = torch.tensor([3, 40, 11, 2], device="cuda")
    torch.library.opcheck(torch.ops.bnb4.kv_write_4bit.default, (k, v, *ts, slots, 32, bnb4.FP4))
    torch.ops.bnb4.kv_write_4bit(k, v, *ts, slots, 32, bnb4.FP4)
    a = bnb4.kv_read_4bit(c, slots, torch.float32)
    b = torch.ops.bnb4.kv_read_4bit(*ts, slots, 32, bnb4.FP4, torch.float32)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    torch.library.opcheck(torch.ops.bnb4.kv_read_4bit.default,
                          (*ts, slots, 32, bnb4.FP4, torch.bfloat16))
    q = case.queries(2, 4).cuda()
    args = (q, *ts, bt, sl, None, 1, 90, 0.125, True, 0, 32, bnb4.FP4)
    torch.library.opcheck(torch.ops.bnb4.attn_4bit.default, args)
    assert torch.equal(torch.ops.bnb4.attn_4bit(*args), bnb4.attn_4bit(q, c, bt, sl))
    cu = ints([0, 0, 1])
    y = torch.ops.bnb4.attn_4bit(q, *ts, bt, sl, cu, 1, 90, 0.125, True, 0, 32, bnb4.FP4)
    assert (y[1] == 0).all() and not (y[0] == 0).all()


@pytest.mark.parametrize("D,bs", [(64, 32), (128, 64)])
@pytest.mark.parametrize("qtype", [bnb4.NF4, bnb4.FP4])
def test_fp16_chunks_lose_only_the_last_rounding(D, bs, qtype):
    """fp16, many rows, weights on a few tokens: keys, values and weights are held
    in two fp16 terms (2^-22 each), so the error is the output's last rounding.
    Half a step is 2^-11 / m of a value with mantissa m, uniform: 2^-11 / sqrt(3)
    sqrt(E m^-2) = 2^-11 * 0.577 * 0.736 = 2.07e-4 in the mean square for evenly
    spread logarithms (E m^-2 = 3 / (8 ln 2)); 10% more for 10240 samples that
    are not quite that, and for the fp32 sums."""
    case = Case([600], 32, 2, D, bs, qtype, oracle.F16, seed=D + bs)
    q = case.queries(40, 4, std=2.0)
    out, _ = run(case, q, [40])
    o64, _, _, _ = attention64(case, q, [40])
    rel = float((out.cpu().double() - o64).norm() / o64.norm())
    assert rel <= 2.28e-4, rel
