"""The paged 8-bit cache on the GPU: write and read bit for bit against their
plain forms, attention against 64 bits within the bound that paged_util
derives, and the four together as a generation uses them."""
import math

import pytest
import torch

from paged_util import DTYPES, FORMATS, QMAX, Case, check

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def kvq():
    from kv_cache_quantization_02_b200 import kvq
    return kvq


@pytest.fixture(autouse=True)
def no_faults(kvq):
    kvq.kvq_fault_status(clear=True)
    yield
    assert kvq.kvq_fault_status(clear=True) == 0


def same(a, b):
    return torch.equal(a.cpu().view(torch.uint8 if a.element_size() == 1 else torch.int32 if a.element_size() == 4
                                    else torch.int16),
                       b.cpu().view(torch.uint8 if b.element_size() == 1 else torch.int32 if b.element_size() == 4
                                    else torch.int16))


def same_cache(c, d):
    return all(same(x, y) for x, y in zip(c.cache(), d.cache()))


WRITES = [
    # D, Hkv, block, fmt, dtype, ctx, new
    (128, 8, 64, "int8", "bf16", [0, 63, 64, 100], [1, 1, 1, 1]),
    (128, 2, 32, "int8", "fp16", [0, 31, 5], [100, 33, 2]),
    (64, 1, 16, "int8", "fp16", [0, 7, 15, 3], [0, 9, 1, 40]),
    (64, 3, 128, "e4m3", "bf16", [200, 0, 128], [1, 300, 128]),
    (128, 4, 16, "e4m3", "fp16", [1, 16, 0, 90], [17, 15, 1, 0]),
    (256, 1, 128, "int8", "fp16", [127, 0], [130, 257]),
    (256, 2, 16, "e4m3", "bf16", [0, 3, 500], [16, 1, 31]),
    (256, 1, 64, "int8", "bf16", [10] * 40, [1] * 39 + [0]),
    (64, 5, 32, "int8", "bf16", list(range(70)), [3] * 70),
    (128, 2, 32, "e4m3", "fp16", [0, 9, 31] + [4] * 27, [50, 0, 3] + [0] * 27),       # few tokens, most of them one's
]


@pytest.mark.parametrize("D,Hkv,block,fmt,dtype,ctx,new", WRITES)
@pytest.mark.parametrize("gain", [0.25, 30.0])          # mostly below, and above, the scales there
def test_write_and_read(kvq, D, Hkv, block, fmt, dtype, ctx, new, gain):
    c = Case(D, Hkv, block, fmt, ctx, new, seed=len(ctx) * D + block)
    k, v = c.rows(Hkv, dtype, gain, tail=5), c.rows(Hkv, dtype, gain / 3, tail=5)
    d = c.cuda()
    kvq.paged_write(k.cuda(), v.cuda(), d.cu, d.start, d.table, *d.cache())
    c.write(k, v)
    assert same_cache(c, d)
    for out in ("fp16", "bf16"):
        ko = torch.full((c.n + 5, Hkv, D), 7.0, dtype=DTYPES[out], device="cuda")
        vo = ko.clone()
        kvq.paged_read(d.cu, d.start, d.table, *d.cache(), n_tokens=c.n + 5, dtype=DTYPES[out], k_out=ko, v_out=vo)
        for got, want in zip((ko, vo), c.read(out)):
            assert same(got[:c.n], want)
            assert bool((got[c.n:] == 7.0).all())       # rows behind the last sequence stay


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_token_by_token(kvq, fmt):
    """Growing magnitudes: every token raises its block's scale, and the earlier codes are rounded again each time."""
    D, Hkv, block, T = 128, 2, 16, 40
    c = Case(D, Hkv, block, fmt, [0, 0], [T, T], seed=5)
    d = c.cuda()
    k, v = c.rows(Hkv, "fp16"), c.rows(Hkv, "fp16")
    k *= torch.linspace(0.1, 4.0, 2 * T)[:, None, None].half()
    at = torch.tensor([0, 1, 2], dtype=torch.int32)
    for t in range(T):
        kt, vt = k[[t, T + t]].contiguous(), v[[t, T + t]].contiguous()
        start = torch.tensor([t, t], dtype=torch.int32)
        kvq.paged_write(kt.cuda(), vt.cuda(), at.cuda(), start.cuda(), d.table, *d.cache())
        c.ctx, c.new, c.cu = [t, t], [1, 1], at
        c.write(kt, vt)
    assert same_cache(c, d)


def test_write_sliced_rows(kvq):
    """k and v as slices of one fused projection, and a single token whose stride says nothing."""
    D, Hkv, Hq = 128, 2, 6
    for new in ([3, 5], [1, 0]):
        c = Case(D, Hkv, 32, "int8", [30, 0], new, seed=6)
        d = c.cuda()
        qkv = c.rows(Hq + 2 * Hkv, "bf16")
        _, k, v = qkv.cuda().split([Hq, Hkv, Hkv], 1)
        kvq.paged_write(k, v, d.cu, d.start, d.table, *d.cache())
        c.write(qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:])
        assert same_cache(c, d)


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_write_special_values(kvq, fmt, dtype):
    """Zeros, subnormals, the largest values, infinities and NaN; a scale that was NaN."""
    D, Hkv, block = 64, 1, 16
    t = DTYPES[dtype]
    c = Case(D, Hkv, block, fmt, [0] * 8 + [5], [16] * 8 + [3], seed=7)
    k, v = c.rows(1, dtype), c.rows(1, dtype)
    big, least = torch.finfo(t).max, 2.0 ** -24 if dtype == "fp16" else 2.0 ** -133
    k[:16] = 0
    k[16:32] *= least * 3
    k[32] = big
    k[48, 0, 3], k[50, 0, 5] = math.inf, -math.inf
    k[64, 0, 1] = math.nan
    k[80:96] = math.nan
    k[96, 0] = -big
    k[112:128] = -0.0
    c.ks[int(c.table[8, 0])] = math.nan
    d = c.cuda()
    kvq.paged_write(k.cuda(), v.cuda(), d.cu, d.start, d.table, *d.cache())
    # the plain form's old scale: NaN counts as none
    c.ks[int(c.table[8, 0])] = 0.0
    page = int(c.table[8, 0])
    before = c.kc[page, :, :5].clone()
    c.write(k, v)
    # the earlier slots of that block: code * (NaN / S) is NaN, and counts as 0, or is left
    got = d.kc.cpu()[page, :, :5].float()
    assert bool(((got == 0) | (got == before.float())).all())
    c.kc.view(torch.uint8)[page, :, :5] = d.kc.cpu().view(torch.uint8)[page, :, :5]
    assert same_cache(c, d)
    assert torch.isfinite(d.ks).all() and torch.isfinite(d.kc.float()).all()


def test_write_leaves_the_rest(kvq):
    """Slots behind the new tokens, other blocks and other scales keep their bits (the plain form touches none)."""
    c = Case(128, 2, 64, "int8", [10], [3], seed=8, spare=9)
    d = c.cuda()
    k = c.rows(2, "fp16")
    before = d.kc.clone()
    kvq.paged_write(k.cuda(), k.cuda(), d.cu, d.start, d.table, *d.cache())
    page = int(c.table[0, 0])
    changed = (d.kc != before).any(-1).any(1).cpu()               # [blocks, slots]
    changed[page, :13] = False
    assert not changed.any()


ATTENDS = [
    # D, Hkv, R, block, fmt, dtype, lens (of one-token queries)
    (128, 2, 4, 32, "int8", "fp16", [1, 33, 64, 100]),
    (128, 8, 4, 64, "int8", "bf16", [300, 0, 17, 64, 65]),
    (128, 1, 1, 16, "e4m3", "fp16", [15, 16, 17, 2000]),
    (128, 2, 8, 128, "e4m3", "bf16", [127, 128, 129, 700]),
    (128, 1, 6, 64, "int8", "fp16", [5000]),
    (128, 1, 12, 32, "int8", "bf16", [77, 513]),
    (128, 2, 16, 16, "e4m3", "fp16", [31, 260]),
    (64, 3, 5, 16, "int8", "bf16", [1, 2, 3, 500]),
    (64, 4, 2, 64, "e4m3", "fp16", [4000, 1]),
    (64, 1, 8, 128, "int8", "fp16", [129]),
    (256, 1, 4, 32, "int8", "bf16", [400, 31]),
    (256, 2, 8, 16, "e4m3", "bf16", [1, 50, 333]),
    (256, 1, 3, 128, "int8", "fp16", [3000]),
    (256, 1, 1, 64, "e4m3", "fp16", [64]),
    (64, 1, 40, 16, "int8", "fp16", [70, 9]),
    (128, 4, 7, 32, "int8", "fp16", [n * 13 % 97 for n in range(70)]),
]


@pytest.mark.parametrize("D,Hkv,R,block,fmt,dtype,lens", ATTENDS)
@pytest.mark.parametrize("window", [0, 40])
def test_decode(kvq, D, Hkv, R, block, fmt, dtype, lens, window):
    c = Case(D, Hkv, block, fmt, [max(0, n - 1) for n in lens], [min(1, n) for n in lens], seed=D + R + len(lens), R=R)
    lens = torch.tensor(lens, dtype=torch.int32)
    q = (torch.randn((c.B, Hkv * R, D), generator=c.g) * 1.5).to(DTYPES[dtype])
    d = c.cuda()
    scale = 1.0 / math.sqrt(D)
    want, bound = c.attend(q, range(c.B + 1), lens, scale, window)
    args = (q.cuda(), lens.cuda(), d.table, *d.cache())
    got = kvq.paged_attention_decode(*args, sm_scale=scale, window=window)
    check(got, want, bound)
    again = kvq.paged_attention_decode(*args, sm_scale=scale, window=window)
    assert same(got, again)
    unsplit = kvq.paged_attention_decode(*args, sm_scale=scale, window=window, workspace=False)
    check(unsplit, want, bound)


PREFILLS = [
    # D, Hkv, R, block, fmt, dtype, ctx, new
    (128, 2, 4, 64, "int8", "fp16", [0, 0], [200, 1]),
    (128, 1, 4, 32, "int8", "bf16", [100, 0, 31], [130, 0, 300]),
    (128, 2, 6, 16, "e4m3", "fp16", [17, 500, 0], [45, 3, 129]),
    (128, 1, 8, 128, "e4m3", "bf16", [1000], [257]),
    (128, 3, 1, 64, "int8", "fp16", [5], [600]),
    (128, 1, 12, 32, "int8", "bf16", [64, 3], [11, 50]),
    (64, 2, 5, 16, "int8", "bf16", [0, 700], [333, 2]),
    (64, 1, 8, 64, "e4m3", "fp16", [128], [128]),
    (64, 4, 1, 128, "int8", "fp16", [0, 1, 2], [1, 127, 128]),
    (256, 1, 4, 32, "int8", "bf16", [200, 0], [100, 70]),
    (256, 2, 2, 16, "e4m3", "fp16", [0, 33], [65, 200]),
    (256, 1, 7, 128, "int8", "fp16", [640], [90]),
    (256, 1, 1, 64, "e4m3", "bf16", [0], [300]),
    (128, 2, 2, 32, "int8", "fp16", list(range(60)), [n % 5 for n in range(60)]),
    (64, 1, 40, 16, "int8", "bf16", [9, 0], [20, 7]),
]


@pytest.mark.parametrize("D,Hkv,R,block,fmt,dtype,ctx,new", PREFILLS)
@pytest.mark.parametrize("window", [0, 50])
def test_prefill(kvq, D, Hkv, R, block, fmt, dtype, ctx, new, window):
    c = Case(D, Hkv, block, fmt, ctx, new, seed=D + R + len(ctx), R=R)
    q = c.rows(Hkv * R, dtype, 1.5, tail=3)
    d = c.cuda()
    scale = 1.0 / math.sqrt(D)
    want, bound = c.attend(q[:c.n], c.cu, c.seq_len, scale, window)
    out = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    args = (q.cuda(), d.cu, d.seq_len, d.table, *d.cache())
    kvq.paged_attention_prefill(*args, sm_scale=scale, window=window, out=out)
    check(out[:c.n], want, bound)
    assert bool((out[c.n:] == 7.0).all())               # rows behind the last sequence stay
    again = kvq.paged_attention_prefill(*args, sm_scale=scale, window=window)
    assert same(out[:c.n], again[:c.n])
    unsplit = kvq.paged_attention_prefill(*args, sm_scale=scale, window=window, workspace=False)
    check(unsplit[:c.n], want, bound)


# Few queries over long sequences: the keys of a tile are split by the lengths.
MIXES = [
    # 32 sequences, some without new tokens, some without any before them; 33 are split without the lengths
    (64, 2, 3, 16, "e4m3", "bf16", [97 * i % 1700 if i % 5 else 0 for i in range(32)], [i * 7 % 10 for i in range(32)]),
    (64, 2, 3, 16, "e4m3", "bf16", [97 * i % 1700 if i % 5 else 0 for i in range(33)], [i * 7 % 10 for i in range(33)]),
    (128, 1, 8, 64, "int8", "fp16", [9000, 40, 0], [1, 33, 2]),
    (128, 3, 2, 128, "e4m3", "fp16", [5000], [300]),
    # more tiles than thread blocks run at once: only those that are left over are split
    (256, 16, 1, 32, "int8", "bf16", [1500, 1300, 1700], [500, 400, 257]),
]


@pytest.mark.parametrize("D,Hkv,R,block,fmt,dtype,ctx,new", MIXES)
@pytest.mark.parametrize("window", [0, 600])
def test_prefill_split_by_lengths(kvq, D, Hkv, R, block, fmt, dtype, ctx, new, window):
    test_prefill(kvq, D, Hkv, R, block, fmt, dtype, ctx, new, window)


def test_the_largest_window(kvq):
    """A window beyond the table is none, also for queries that stand before their sequence."""
    c = Case(128, 2, 32, "int8", [1300, 0], [40, 30], seed=22, R=2)
    lens = torch.tensor([1340, 10], dtype=torch.int32)
    q = c.rows(4, "fp16")
    d = c.cuda()
    for window in (2**31 - 1, c.table.shape[1] * 32):
        args = (q.cuda(), d.cu, lens.cuda(), d.table, *d.cache())
        want, bound = c.attend(q, c.cu, lens, 0.1)
        check(kvq.paged_attention_prefill(*args, sm_scale=0.1, window=window), want, bound)
        check(kvq.paged_attention_prefill(*args, sm_scale=0.1, window=window, workspace=False), want, bound)
        want, bound = c.attend(q[:2], range(3), lens, 0.1)
        check(kvq.paged_attention_decode(q[:2].cuda(), *args[2:], sm_scale=0.1, window=window), want, bound)


def test_prefill_lengths_change_between_replays(kvq):
    """A captured call splits by the lengths of each replay."""
    c = Case(128, 2, 32, "int8", [1500, 20, 900], [10, 120, 70], seed=21, R=4)
    q = c.rows(8, "fp16")
    d, qd = c.cuda(), q.cuda()
    cu, lens = d.cu.clone(), d.seq_len.clone()
    out = torch.zeros_like(qd)
    run = lambda: kvq.paged_attention_prefill(qd, cu, lens, d.table, *d.cache(), sm_scale=0.1, out=out)
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    n = c.n
    for offsets, lengths in (([0, 10, 130, 200], [1510, 140, 970]), ([0, 200, 200, 200], [1510, 140, 970]),
                             ([0, 1, 2, 3], [1510, 33, 500]), ([0, 0, 140, 140], [0, 140, 0])):
        cu.copy_(torch.tensor(offsets, dtype=torch.int32))
        lens.copy_(torch.tensor(lengths, dtype=torch.int32))
        out.fill_(7.0)
        g.replay()
        want, bound = c.attend(q[:offsets[-1]], torch.tensor(offsets, dtype=torch.int32),
                               torch.tensor(lengths, dtype=torch.int32), 0.1)
        check(out[:offsets[-1]], want, bound)
        assert n == 200 and bool((out[offsets[-1]:] == 7.0).all())


@pytest.mark.parametrize("D,block", [(64, 16), (128, 64), (256, 32)])
def test_queries_without_keys(kvq, D, block):
    """More queries than positions: the first ones stand before the sequence and give zeros; so do empty sequences."""
    c = Case(D, 2, block, "int8", [0, 0, 0], [70, 20, 5], seed=11, R=2)
    lens = torch.tensor([30, 0, 5], dtype=torch.int32)
    q = c.rows(4, "fp16")
    d = c.cuda()
    want, bound = c.attend(q, c.cu, lens, 0.1)
    got = kvq.paged_attention_prefill(q.cuda(), d.cu, lens.cuda(), d.table, *d.cache(), sm_scale=0.1)
    check(got, want, bound)
    assert not got[:40].any() and not got[70:90].any()
    got = kvq.paged_attention_decode(q[:3].cuda(), torch.zeros(3, dtype=torch.int32, device="cuda"), d.table,
                                     *d.cache(), sm_scale=0.1)
    assert not got.any()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_what_is_masked_does_not_matter(kvq, D, fmt):
    """Slots behind the last position, blocks of nobody and their scales: whatever they hold, outputs are the same bits."""
    c = Case(D, 1, 16, fmt, [37, 70, 3], [9, 21, 1], seed=12, R=3)
    q = c.rows(3, "bf16")
    outs = []
    for fill, scale in ((0, 1.0), (0x7F, math.nan), (0x81, math.inf), (0xFF, -1.0)):
        d = c.cuda()
        live = torch.zeros((c.num_blocks, 16), dtype=torch.bool)
        for b in range(3):
            for p in range(int(c.seq_len[b])):
                live[int(c.table[b, p // 16]), p % 16] = True
        for codes, s in ((d.kc, d.ks), (d.vc, d.vs)):
            codes.view(torch.uint8).masked_fill_(~live.cuda()[:, None, :, None], fill)
            s.masked_fill_(~live.any(1).cuda()[:, None], scale)
        a = kvq.paged_attention_prefill(q.cuda(), d.cu, d.seq_len, d.table, *d.cache(), sm_scale=0.2)
        b = kvq.paged_attention_decode(q[:3].cuda(), d.seq_len, d.table, *d.cache(), sm_scale=0.2)
        outs.append((a, b))
    for a, b in outs[1:]:
        assert same(a, outs[0][0]) and same(b, outs[0][1])


@pytest.mark.parametrize("D", [64, 128, 256])
def test_odd_scales_and_queries(kvq, D):
    """Blocks whose value scales lie 2^18 apart, queries of very different size, a negative softmax scale; one query
    row that holds NaN touches its own output alone."""
    c = Case(D, 1, 16, "int8", [0, 0], [150, 90], seed=13, R=2)
    c.vs *= torch.exp2(torch.randint(-9, 10, c.vs.shape, generator=c.g).float())
    q = c.rows(2, "bf16")
    q *= torch.exp2(torch.randint(-6, 3, (c.n, 1, 1), generator=c.g).float()).bfloat16()
    d = c.cuda()
    for scale in (0.05, -0.05, 0.0):
        want, bound = c.attend(q, c.cu, c.seq_len, scale)
        check(kvq.paged_attention_prefill(q.cuda(), d.cu, d.seq_len, d.table, *d.cache(), sm_scale=scale), want, bound)
        want, bound = c.attend(q[:2], range(3), c.seq_len, scale)
        check(kvq.paged_attention_decode(q[:2].cuda(), d.seq_len, d.table, *d.cache(), sm_scale=scale), want, bound)
    want, bound = c.attend(q, c.cu, c.seq_len, 0.05)
    bad = q.clone()
    bad[20, 1, 5] = math.nan
    got = kvq.paged_attention_prefill(bad.cuda(), d.cu, d.seq_len, d.table, *d.cache(), sm_scale=0.05).cpu()
    assert got[20, 1].isnan().all()
    got[20, 1] = want[20, 1].bfloat16()
    check(got, want, bound)
    want, bound = c.attend(q[:2], range(3), c.seq_len, 0.05)
    bad = q[:2].clone()
    bad[1, 0, 0] = math.nan
    got = kvq.paged_attention_decode(bad.cuda(), d.seq_len, d.table, *d.cache(), sm_scale=0.05).cpu()
    assert got[1, 0].isnan().all()
    got[1, 0] = want[1, 0].bfloat16()
    check(got, want, bound)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_large_scores(kvq, D):
    """Scores in the thousands, of either sign: the softmax is nearly one key, and nothing overflows."""
    c = Case(D, 2, 32, "e4m3", [120, 0], [40, 99], seed=14, R=4)
    q = c.rows(8, "fp16", 40.0)
    d = c.cuda()
    want, bound = c.attend(q, c.cu, c.seq_len, 1.0)
    check(kvq.paged_attention_prefill(q.cuda(), d.cu, d.seq_len, d.table, *d.cache(), sm_scale=1.0), want, bound)
    want, bound = c.attend(q[:2], range(3), c.seq_len, 1.0)
    check(kvq.paged_attention_decode(q[:2].cuda(), d.seq_len, d.table, *d.cache(), sm_scale=1.0), want, bound)


def test_zero_values(kvq):
    """Blocks of zeros carry the least scale; their keys still count in the softmax."""
    c = Case(128, 1, 16, "int8", [0], [60], seed=15, R=2)
    k, v = c.rows(1, "fp16"), c.rows(1, "fp16")
    v[16:32] = 0
    q = c.rows(2, "fp16")
    d = c.cuda()
    kvq.paged_write(k.cuda(), v.cuda(), d.cu, d.start, d.table, *d.cache())
    c.write(k, v)
    want, bound = c.attend(q, c.cu, c.seq_len, 0.1)
    check(kvq.paged_attention_prefill(q.cuda(), d.cu, d.seq_len, d.table, *d.cache(), sm_scale=0.1), want, bound)
    want, bound = c.attend(q[:1], range(2), c.seq_len, 0.1)
    check(kvq.paged_attention_decode(q[:1].cuda(), d.seq_len, d.table, *d.cache(), sm_scale=0.1), want, bound)


@pytest.mark.parametrize("D,block", [(64, 64), (128, 16), (256, 32)])
@pytest.mark.parametrize("up", [60, -60])
def test_queries_far_from_one(kvq, D, block, up):
    """bf16 queries around 2^60 and 2^-60, the softmax scale around 2^-60 and 2^60: beyond fp16, which holds the rows."""
    c = Case(D, 1, block, "int8", [0, 40], [100, 30], seed=21, R=2)
    q = (c.rows(2, "bf16").float() * 2.0 ** up).bfloat16()
    d = c.cuda()
    scale = 2.0 ** -up / math.sqrt(D)
    want, bound = c.attend(q, c.cu, c.seq_len, scale)
    check(kvq.paged_attention_prefill(q.cuda(), d.cu, d.seq_len, d.table, *d.cache(), sm_scale=scale), want, bound)
    want, bound = c.attend(q[:2], range(3), c.seq_len, scale)
    check(kvq.paged_attention_decode(q[:2].cuda(), d.seq_len, d.table, *d.cache(), sm_scale=scale), want, bound)


@pytest.mark.parametrize("D,block,fmt", [(128, 16, "e4m3"), (128, 64, "int8"), (64, 32, "int8"), (256, 128, "e4m3")])
@pytest.mark.parametrize("window", [1, 17, 64, 130])
def test_blocks_before_the_window(kvq, D, block, fmt, window):
    """Blocks that lie wholly before every window are given up: their table entries may be anything, and none is reported."""
    c = Case(D, 1, block, fmt, [700, 300, 0], [20, 1, 3], seed=22, R=4)
    for b in range(3):
        first = max(0, c.ctx[b] - window + 1) // block               # the first block that a new token sees
        c.table[b, :first] = -1 if b == 0 else 2 ** 30
    q = c.rows(4, "bf16")
    d = c.cuda()
    want, bound = c.attend(q, c.cu, c.seq_len, 0.2, window)
    check(kvq.paged_attention_prefill(q.cuda(), d.cu, d.seq_len, d.table, *d.cache(), sm_scale=0.2, window=window),
          want, bound)
    last = q[(c.cu[1:] - 1).long()]
    want, bound = c.attend(last, range(4), c.seq_len, 0.2, window)
    check(kvq.paged_attention_decode(last.cuda(), d.seq_len, d.table, *d.cache(), sm_scale=0.2, window=window),
          want, bound)


@pytest.mark.parametrize("B", [33, 128, 129, 300])
def test_many_sequences(kvq, B):
    """Searches and scans over more sequences than a warp, or a block, looks at at once; empty ones among them."""
    D, Hkv, block = 64, 2, 16
    new = [(7 * b) % 5 for b in range(B)]
    new[B // 2] = 40
    c = Case(D, Hkv, block, "int8", [(5 * b) % 19 for b in range(B)], new, seed=B, R=2)
    d = c.cuda()
    k, v, q = c.rows(Hkv, "fp16"), c.rows(Hkv, "fp16"), c.rows(2 * Hkv, "fp16")
    kvq.paged_write(k.cuda(), v.cuda(), d.cu, d.start, d.table, *d.cache())
    c.write(k, v)
    assert same_cache(c, d)
    for got, want in zip(kvq.paged_read(d.cu, d.start, d.table, *d.cache(), n_tokens=c.n), c.read("fp16")):
        assert same(got, want)
    want, bound = c.attend(q, c.cu, c.seq_len, 0.1)
    check(kvq.paged_attention_prefill(q.cuda(), d.cu, d.seq_len, d.table, *d.cache(), sm_scale=0.1), want, bound)
    one = (torch.randn((B, 2 * Hkv, D), generator=c.g)).half()
    want, bound = c.attend(one, range(B + 1), c.seq_len, 0.1)
    check(kvq.paged_attention_decode(one.cuda(), d.seq_len, d.table, *d.cache(), sm_scale=0.1), want, bound)


def test_thousands_of_sequences(kvq):
    """4500 sequences in one call are what they are in calls of 30."""
    B, D, Hkv, block = 4500, 64, 1, 16
    new = [(3 * b) % 4 for b in range(B)]
    c = Case(D, Hkv, block, "e4m3", [(11 * b) % 37 for b in range(B)], new, seed=23, R=2)
    k, v, q = c.rows(Hkv, "bf16").cuda(), c.rows(Hkv, "bf16").cuda(), c.rows(2, "bf16").cuda()
    d, e = c.cuda(), c.cuda()
    e.kc, e.vc, e.ks, e.vs = (x.clone() for x in d.cache())
    kvq.paged_write(k, v, d.cu, d.start, d.table, *d.cache())
    pieces = [(b, min(B, b + 30)) for b in range(0, B, 30)]
    part = lambda x, b0, b1: x[int(c.cu[b0]):int(c.cu[b1])]
    cus = [(d.cu[b0:b1 + 1] - d.cu[b0]).contiguous() for b0, b1 in pieces]
    for (b0, b1), cu in zip(pieces, cus):
        kvq.paged_write(part(k, b0, b1), part(v, b0, b1), cu, e.start[b0:b1], e.table[b0:b1], *e.cache())
    assert same_cache(d, e)
    out = kvq.paged_attention_prefill(q, d.cu, d.seq_len, d.table, *d.cache(), sm_scale=0.2, workspace=False)
    one = torch.randn((B, 2, D), generator=c.g).bfloat16().cuda()
    dec = kvq.paged_attention_decode(one, d.seq_len, d.table, *d.cache(), sm_scale=0.2, workspace=False)
    for (b0, b1), cu in zip(pieces, cus):
        lens, table = d.seq_len[b0:b1], d.table[b0:b1]
        assert same(part(out, b0, b1), kvq.paged_attention_prefill(part(q, b0, b1), cu, lens, table, *d.cache(),
                                                                   sm_scale=0.2, workspace=False))
        assert same(dec[b0:b1], kvq.paged_attention_decode(one[b0:b1], lens, table, *d.cache(), sm_scale=0.2,
                                                           workspace=False))
    c.kc, c.vc, c.ks, c.vs = (x.cpu() for x in d.cache())
    want, bound = c.attend(one.cpu(), range(B + 1), c.seq_len, 0.2)
    check(kvq.paged_attention_decode(one, d.seq_len, d.table, *d.cache(), sm_scale=0.2), want, bound)


def test_positions_behind_the_table(kvq):
    """New tokens that the table has no block for are reported and left out, the others written."""
    c = Case(128, 1, 16, "int8", [10, 0], [20, 40], seed=24, extra=0)
    c.table = c.table[:, :2].contiguous()
    d = c.cuda()
    k = c.rows(1, "fp16")
    kvq.paged_write(k.cuda(), k.cuda(), d.cu, d.start, d.table, *d.cache())
    assert kvq.kvq_fault_status(clear=True) == 4
    c.write(k, k)
    assert same_cache(c, d)


def test_first_call_in_a_capture():
    """A process whose first calls are captured into a graph, and replayed."""
    import subprocess
    import sys
    code = """
import torch
from kv_cache_quantization_02_b200 import kvq
torch.manual_seed(0)
kc, vc = (torch.zeros((9, 2, 16, 128), dtype=torch.int8, device="cuda") for _ in range(2))
ks, vs = (torch.ones((9, 2), device="cuda") for _ in range(2))
table = torch.arange(8, dtype=torch.int32, device="cuda").view(1, 8)
cu = torch.tensor([0, 100], dtype=torch.int32, device="cuda")
zero, lens = torch.zeros(1, dtype=torch.int32, device="cuda"), torch.full((1,), 100, dtype=torch.int32, device="cuda")
k, v, q = (torch.randn((100, h, 128), device="cuda").half() for h in (2, 2, 8))
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
def run():
    kvq.paged_write(k, v, cu, zero, table, kc, vc, ks, vs)
    a, _ = kvq.paged_read(cu, zero, table, kc, vc, ks, vs, n_tokens=100)
    b = kvq.paged_attention_prefill(q, cu, lens, table, kc, vc, ks, vs, sm_scale=0.1)
    return a, b, kvq.paged_attention_decode(q[:1], lens, table, kc, vc, ks, vs, sm_scale=0.1)
with torch.cuda.graph(g):
    out = run()
g.replay()
torch.cuda.synchronize()
assert all(torch.equal(x, y) for x, y in zip(out, run()))
assert kvq.kvq_fault_status() == 0
"""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def _generate(kvq, c, d, fmt, steps, prompt, Hq, Hkv, D, graph):
    """A prompt in two chunks, then single tokens, on the GPU and plainly; yields (got, want, bound)."""
    B = len(prompt)
    scale = 1.0 / math.sqrt(D)
    at = [0] * B
    for chunk in (prompt, [7] * B):
        n = sum(chunk)
        c.ctx, c.new, c.n = list(at), list(chunk), n
        c.cu = torch.tensor([0] + list(chunk)).cumsum(0).to(torch.int32)
        c.start = torch.tensor(at, dtype=torch.int32)
        at = [a + m for a, m in zip(at, chunk)]
        lens = torch.tensor(at, dtype=torch.int32)
        qkv = c.rows(Hq + 2 * Hkv, "bf16")
        q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
        gq, gk, gv = qkv.cuda().split([Hq, Hkv, Hkv], 1)
        kvq.paged_write(gk, gv, c.cu.cuda(), c.start.cuda(), d.table, *d.cache())
        got = kvq.paged_attention_prefill(gq, c.cu.cuda(), lens.cuda(), d.table, *d.cache(), sm_scale=scale)
        c.write(k, v)
        yield (got, *c.attend(q.contiguous(), c.cu, lens, scale))
    one = torch.arange(B + 1, dtype=torch.int32)
    gone, start, lens = one.cuda(), torch.zeros(B, dtype=torch.int32).cuda(), torch.zeros(B, dtype=torch.int32).cuda()
    qkv = torch.zeros((B, Hq + 2 * Hkv, D), dtype=torch.bfloat16, device="cuda")

    def step():
        q, k, v = qkv.split([Hq, Hkv, Hkv], 1)
        kvq.paged_write(k, v, gone, start, d.table, *d.cache())
        return kvq.paged_attention_decode(q, lens, d.table, *d.cache(), sm_scale=scale)

    replay = None
    if graph:
        start.fill_(0)                                   # no keys yet: the warm-up writes position 0, put back below
        keep = [x.clone() for x in d.cache()]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            res = step()
        for x, y in zip(d.cache(), keep):
            x.view(torch.uint8).copy_(y.view(torch.uint8))
        replay = g
    for _ in range(steps):
        c.ctx, c.new, c.n, c.cu = list(at), [1] * B, B, one
        c.start = torch.tensor(at, dtype=torch.int32)
        at = [a + 1 for a in at]
        x = c.rows(Hq + 2 * Hkv, "bf16")
        q, k, v = x.split([Hq, Hkv, Hkv], 1)
        qkv.copy_(x)
        start.copy_(c.start)
        lens.copy_(torch.tensor(at, dtype=torch.int32))
        if replay is not None:
            replay.replay()
            got = res
        else:
            got = step()
        c.write(k, v)
        yield (got, *c.attend(q.contiguous(), one, torch.tensor(at), scale))


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("D,block,fmt", [(128, 16, "int8"), (64, 32, "e4m3"), (256, 16, "e4m3")])
def test_generation(kvq, D, block, fmt, graph):
    """Write, prompt attention, append and decode attention in a row, eager and with the step captured in a graph."""
    prompt = [50, 3, 129]
    Hkv, R = 2, 3
    c = Case(D, Hkv, block, fmt, [0] * 3, [p + 7 + 20 for p in prompt], seed=16, R=R)
    d = c.cuda()
    for got, want, bound in _generate(kvq, c, d, fmt, 20, prompt, Hkv * R, Hkv, D, graph):
        check(got, want, bound)
    assert same_cache(c, d)


def test_other_stream_and_two_calls_at_once(kvq):
    """Calls on two streams with nothing between them give what each gives alone."""
    c = Case(128, 1, 64, "int8", [6000, 5000], [1, 1], seed=17, R=4)
    d = c.cuda()
    qs = [c.rows(4, "fp16").cuda() for _ in range(2)]
    alone = [kvq.paged_attention_decode(q, d.seq_len, d.table, *d.cache(), sm_scale=0.1) for q in qs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in qs]
    outs = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            outs[i].append(kvq.paged_attention_decode(qs[i], d.seq_len, d.table, *d.cache(), sm_scale=0.1, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(same(o, alone[i]) for o in outs[i])


def test_far_blocks(kvq):
    """Codes past 4 GiB: the last blocks of a large cache, written, read and attended over."""
    D, Hkv, block = 256, 8, 128
    num_blocks = (9 << 29) // (Hkv * block * D)                   # 4.5 GiB of codes for K, and for V
    c = Case(D, Hkv, block, "int8", [100], [150], seed=18)
    small = c.cuda()
    k, v = c.rows(Hkv, "fp16"), c.rows(Hkv, "fp16")
    q = c.rows(Hkv, "fp16").cuda()
    kc, vc = (torch.zeros((num_blocks, Hkv, block, D), dtype=torch.int8, device="cuda") for _ in range(2))
    ks, vs = (torch.ones((num_blocks, Hkv), device="cuda") for _ in range(2))
    n = c.num_blocks
    kc[-n:], vc[-n:], ks[-n:], vs[-n:] = small.kc, small.vc, small.ks, small.vs
    table = torch.where(small.table >= 0, small.table + (num_blocks - n), small.table)
    far = (kc, vc, ks, vs)
    kvq.paged_write(k.cuda(), v.cuda(), small.cu, small.start, small.table, *small.cache())
    kvq.paged_write(k.cuda(), v.cuda(), small.cu, small.start, table, *far)
    assert all(same(x[-n:], y) for x, y in zip(far, small.cache()))
    for x, y in zip(kvq.paged_read(small.cu, small.start, table, *far, n_tokens=c.n),
                    kvq.paged_read(small.cu, small.start, small.table, *small.cache(), n_tokens=c.n)):
        assert same(x, y)
    near = kvq.paged_attention_prefill(q, small.cu, small.seq_len, small.table, *small.cache(), sm_scale=0.1)
    assert same(kvq.paged_attention_prefill(q, small.cu, small.seq_len, table, *far, sm_scale=0.1), near)
    near = kvq.paged_attention_decode(q[:1], small.seq_len, small.table, *small.cache(), sm_scale=0.1)
    assert same(kvq.paged_attention_decode(q[:1], small.seq_len, table, *far, sm_scale=0.1), near)


def test_bad_tables_and_lengths(kvq):
    """Entries outside the cache, positions outside the table and lengths out of range: skipped or clamped, reported,
    and everything else is right."""
    c = Case(128, 2, 16, "int8", [20, 40, 0], [30, 9, 25], seed=19, R=2, extra=0)
    for bad in (-1, c.num_blocks, 2 ** 31 - 1):
        d = c.cuda()
        e = Case(128, 2, 16, "int8", c.ctx, c.new, seed=19, R=2, extra=0)
        e.table = c.table.clone()
        e.table[0, 2] = bad
        table = e.table.cuda()
        k, v = e.rows(2, "fp16"), e.rows(2, "fp16")
        kvq.paged_write(k.cuda(), v.cuda(), d.cu, d.start, table, *d.cache())
        assert kvq.kvq_fault_status(clear=True) == 4
        e.write(k, v)
        assert same_cache(e, d)
        out = torch.full((e.n, 2, 128), 3.0, dtype=torch.float16, device="cuda")
        ko, _ = kvq.paged_read(d.cu, d.start, table, *d.cache(), n_tokens=e.n, k_out=out, v_out=out.clone())
        assert kvq.kvq_fault_status(clear=True) == 4
        hole = torch.zeros(e.n, dtype=torch.bool)
        hole[12:28] = True                                       # positions 32 .. 47 of sequence 0
        assert bool((ko.cpu()[hole] == 3.0).all())
        q = e.rows(4, "fp16")
        want, bound = e.attend(q, e.cu, e.seq_len, 0.1)
        check(kvq.paged_attention_prefill(q.cuda(), d.cu, d.seq_len, table, *d.cache(), sm_scale=0.1), want, bound)
        assert kvq.kvq_fault_status(clear=True) == 4
        want, bound = e.attend(q[:3], range(4), e.seq_len, 0.1)
        check(kvq.paged_attention_decode(q[:3].cuda(), d.seq_len, table, *d.cache(), sm_scale=0.1), want, bound)
        assert kvq.kvq_fault_status(clear=True) == 4
    # lengths outside the table are clamped: sequence 2's negative one to nothing, sequence 1's to the whole table row
    d = c.cuda()
    width = c.table.shape[1]
    table = c.table.clamp(min=0)
    lens = torch.tensor([50, 10 ** 9, -5], dtype=torch.int32)
    e = Case(128, 2, 16, "int8", c.ctx, c.new, seed=19, R=2, extra=0)
    e.table = table
    q = e.rows(4, "fp16")
    want, bound = e.attend(q[:3], range(4), torch.tensor([50, width * 16, 0]), 0.1)
    check(kvq.paged_attention_decode(q[:3].cuda(), lens.cuda(), table.cuda(), *d.cache(), sm_scale=0.1), want, bound)
    assert kvq.kvq_fault_status(clear=True) == 8
    want, bound = e.attend(q, c.cu, torch.tensor([50, width * 16, 0]), 0.1)
    check(kvq.paged_attention_prefill(q.cuda(), d.cu, lens.cuda(), table.cuda(), *d.cache(), sm_scale=0.1), want, bound)
    assert kvq.kvq_fault_status(clear=True) == 8
    # offsets beyond the rows and negative starts: their sequences are skipped
    d = c.cuda()
    before = [x.clone() for x in d.cache()]
    k = e.rows(2, "fp16").cuda()
    cu = torch.tensor([0, 10 ** 6, 10 ** 6, 10 ** 6], dtype=torch.int32).cuda()
    kvq.paged_write(k, k, cu, d.start, d.table, *d.cache())
    assert kvq.kvq_fault_status(clear=True) & 8
    kvq.paged_write(k, k, d.cu, -1 - d.start, d.table, *d.cache())
    assert kvq.kvq_fault_status(clear=True) & 8
    assert all(same(x, y) for x, y in zip(before, d.cache()))


@pytest.mark.parametrize("B", [3, 33])                  # split by the lengths, and without them
def test_bad_lengths_and_offsets_of_long_sequences(kvq, B):
    ctx, new = [2000, 1500, 40] + [3] * (B - 3), [9, 20, 30] + [0] * (B - 3)
    c = Case(64, 2, 64, "int8", ctx, new, seed=23, R=2)
    q = c.rows(4, "fp16")
    c.table = c.table.clamp(min=0)
    d = c.cuda()
    run = lambda cu, lens: kvq.paged_attention_prefill(
        q.cuda(), torch.tensor(cu, dtype=torch.int32).cuda(), lens.cuda(), d.table, *d.cache(), sm_scale=0.1,
        out=torch.full_like(q, 7.0).cuda())
    rest = [3] * (B - 3)
    lens = torch.tensor([2009, 10 ** 9, -5] + rest, dtype=torch.int32)
    clamped = torch.tensor([2009, c.table.shape[1] * 64, 0] + rest, dtype=torch.int32)
    want, bound = c.attend(q, c.cu, clamped, 0.1)
    check(run(c.cu.tolist(), lens), want, bound)
    assert kvq.kvq_fault_status(clear=True) == 8
    want, bound = c.attend(q, c.cu, c.seq_len, 0.1)
    end = [59] * (B - 3)
    for cu, right in (([0, 9, 10 ** 6, 59], range(0, 9)), ([-5, 9, 29, 59], range(9, 59))):
        got = run(cu + end, c.seq_len)
        assert kvq.kvq_fault_status(clear=True) == 8
        check(got[right.start:right.stop], want[right.start:right.stop], bound[right.start:right.stop])
        assert all(bool((got[i] == 7.0).all()) for i in range(59) if i not in right)
    # sequences that share rows: whichever is last, those of one alone are right
    got = run([0, 59, 9, 59] + end, c.seq_len)
    assert kvq.kvq_fault_status(clear=True) == 8
    want, bound = c.attend(q, torch.tensor([0, 59, 59, 59] + end, dtype=torch.int32), c.seq_len, 0.1)
    check(got[:9], want[:9], bound[:9])


def test_empty_calls(kvq):
    c = Case(128, 2, 16, "int8", [], [], seed=20, extra=4)
    d = c.cuda()
    none = torch.empty((0, 2, 128), dtype=torch.float16, device="cuda")
    kvq.paged_write(none, none, d.cu, d.start, d.table, *d.cache())
    k, v = kvq.paged_read(d.cu, d.start, d.table, *d.cache(), n_tokens=0)
    assert k.shape == v.shape == (0, 2, 128)
    assert kvq.paged_attention_decode(none, d.start, d.table, *d.cache(), sm_scale=1.0).shape == (0, 2, 128)
    assert kvq.paged_attention_prefill(none, d.cu, d.start, d.table, *d.cache(), sm_scale=1.0).shape == (0, 2, 128)


def test_wrong_tensors(kvq):
    """Each wrong argument is refused by name; small workspaces are not used, and statuses become KvqError."""
    c = Case(128, 2, 16, "int8", [3, 40], [5, 6], seed=25, R=2)
    d = c.cuda()
    k, q = c.rows(2, "fp16").cuda(), c.rows(4, "fp16").cuda()
    before = [x.clone() for x in d.cache()]
    cache = list(d.cache())

    def swapped(i, x):
        return [x if j == i else y for j, y in enumerate(cache)]

    bad_caches = [
        ("k_cache", swapped(0, d.kc.view(torch.uint8))), ("k_cache", swapped(0, d.kc[0])),
        ("v_cache", swapped(1, d.vc[1:])), ("v_cache", swapped(1, d.vc.view(torch.float8_e4m3fn))),
        ("v_cache", swapped(1, d.vc.transpose(1, 2).contiguous().transpose(1, 2))), ("v_cache", swapped(1, d.vc.cpu())),
        ("k_scales", swapped(2, d.ks.double())), ("v_scales", swapped(3, d.vs[:, :1])), ("k_scales", swapped(2, d.ks.cpu())),
    ]
    for name, bad in bad_caches:
        for call in (lambda: kvq.paged_write(k, k, d.cu, d.start, d.table, *bad),
                     lambda: kvq.paged_read(d.cu, d.start, d.table, *bad, n_tokens=11),
                     lambda: kvq.paged_attention_decode(q[:2], d.seq_len, d.table, *bad, sm_scale=1.0),
                     lambda: kvq.paged_attention_prefill(q, d.cu, d.seq_len, d.table, *bad, sm_scale=1.0)):
            with pytest.raises(ValueError, match=name):
                call()
    for name, args in (("cu_tokens", (k, k, d.cu.long(), d.start, d.table)), ("cu_tokens", (k, k, d.cu[1:], d.start, d.table)),
                       ("start", (k, k, d.cu, d.start.cpu(), d.table)), ("block_table", (k, k, d.cu, d.start, d.table.long())),
                       ("block_table", (k, k, d.cu, d.start, d.table[0])), ("k and v", (k, k[1:], d.cu, d.start, d.table)),
                       ("k and v", (k, k.bfloat16(), d.cu, d.start, d.table)), ("k and v", (q, q, d.cu, d.start, d.table)),
                       ("k must", (k.float(), k, d.cu, d.start, d.table)), ("v must", (k, k[:, :, :64], d.cu, d.start, d.table)),
                       ("k: the channels", (k.transpose(0, 1).contiguous().transpose(0, 1), k, d.cu, d.start, d.table)),
                       ("k must", (k.cpu(), k, d.cu, d.start, d.table))):
        with pytest.raises(ValueError, match=name):
            kvq.paged_write(*args, *cache)
    for name, kw in (("out", dict(out=q[:2].float())), ("out", dict(out=q[:3])), ("out", dict(out=q[:2].cpu())),
                     ("workspace", dict(workspace=torch.empty(9, device="cuda")))):
        with pytest.raises(ValueError, match=name):
            kvq.paged_attention_decode(q[:2], d.seq_len, d.table, *cache, sm_scale=1.0, **kw)
    with pytest.raises(ValueError, match="q must have one row"):
        kvq.paged_attention_decode(q, d.seq_len, d.table, *cache, sm_scale=1.0)
    with pytest.raises(ValueError, match="torch.Tensor"):
        kvq.paged_attention_decode(None, d.seq_len, d.table, *cache, sm_scale=1.0)
    with pytest.raises(ValueError, match="dtype"):
        kvq.paged_read(d.cu, d.start, d.table, *cache, n_tokens=11, dtype=torch.float32)
    with pytest.raises(ValueError, match="n_tokens"):
        kvq.paged_read(d.cu, d.start, d.table, *cache, n_tokens=-1)
    with pytest.raises(TypeError):
        kvq.paged_attention_decode(q[:2], d.seq_len, d.table, *cache, sm_scale="1")
    for kw, status in ((dict(window=-1), -5), (dict(sm_scale=math.nan), -5)):
        with pytest.raises(kvq.KvqError) as e:
            kvq.paged_attention_decode(q[:2], d.seq_len, d.table, *cache, **dict(dict(sm_scale=1.0), **kw))
        assert e.value.status == status
    with pytest.raises(kvq.KvqError) as e:
        kvq.paged_read(d.cu, d.start, d.table, *(x[:, :, :8].contiguous() for x in cache[:2]), *cache[2:], n_tokens=11)
    assert e.value.status == -7                                   # blocks of 8 tokens
    want = kvq.paged_attention_decode(q[:2], d.seq_len, d.table, *cache, sm_scale=1.0, workspace=False)
    small = torch.empty(64, dtype=torch.uint8, device="cuda")
    assert same(kvq.paged_attention_decode(q[:2], d.seq_len, d.table, *cache, sm_scale=1.0, workspace=small), want)
    assert all(same(x, y) for x, y in zip(before, d.cache()))


def test_formats_are_named(kvq):
    assert set(FORMATS.values()) == set(QMAX)


@pytest.mark.parametrize("D,block,fmt", [(64, 16, "int8"), (128, 32, "e4m3"), (256, 16, "int8"), (128, 16, "int8")])
def test_scales_that_no_write_makes(kvq, D, block, fmt):
    """A cache that other code filled may hold key and value scales that are NaN, negative, infinite below, zero or
    tiny: both attentions read max(scale, 2^-40)."""
    c = Case(D, 1, block, fmt, [0, 3], [170, 90], seed=26, R=2)
    odd = [math.nan, -0.01, 0.0, -math.inf, 2.0 ** -50]
    for i, x in enumerate(odd):
        c.ks[int(c.table[i % 2, i // 2])] = x
        c.vs[int(c.table[i % 2, (i + 1) // 2 % 3])] = x
    d = c.cuda()
    for s in (c.ks, c.vs):
        s.copy_(torch.nan_to_num(s, nan=0.0).clamp(min=2.0 ** -40))
    q = c.rows(2, "bf16")
    for scale in (0.3, -0.3):
        want, bound = c.attend(q, c.cu, c.seq_len, scale)
        check(kvq.paged_attention_prefill(q.cuda(), d.cu, d.seq_len, d.table, *d.cache(), sm_scale=scale), want, bound)
        want, bound = c.attend(q[:2], range(3), c.seq_len, scale)
        check(kvq.paged_attention_decode(q[:2].cuda(), d.seq_len, d.table, *d.cache(), sm_scale=scale), want, bound)


def test_out_of_memory(kvq):
    """Outputs that do not fit the GPU raise what torch's own allocations raise, and the next call works."""
    c = Case(128, 8, 16, "int8", [3], [5], seed=27)
    d = c.cuda()
    with pytest.raises(torch.OutOfMemoryError):
        kvq.paged_read(d.cu, d.start, d.table, *d.cache(), n_tokens=2 ** 31 - 1)           # 4 TiB
    for got, want in zip(kvq.paged_read(d.cu, d.start, d.table, *d.cache(), n_tokens=c.n), c.read("fp16")):
        assert same(got, want)


def test_more_tokens_than_a_call_takes(kvq):
    """2^31 tokens and more are refused by name, not by what their outputs would need."""
    c = Case(128, 2, 16, "int8", [3], [5], seed=28)
    d = c.cuda()
    for n in (2 ** 31, 2 ** 40, 2 ** 62):
        with pytest.raises(ValueError, match="n_tokens"):
            kvq.paged_read(d.cu, d.start, d.table, *d.cache(), n_tokens=n)


def _empty_cache(num_blocks, fmt):
    return (*(torch.zeros((num_blocks, 2, 16, 128), dtype=FORMATS[fmt], device="cuda") for _ in range(2)),
            *(torch.ones((num_blocks, 2), device="cuda") for _ in range(2)))


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
@pytest.mark.parametrize("B", [3, 40])
def test_tables_without_columns(kvq, B, fmt):
    """Sequences that have no block yet, in a cache with and without blocks: nothing is seen, and nothing reported."""
    table = torch.zeros((B, 0), dtype=torch.int32, device="cuda")
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    one = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    x, q = (torch.ones((B, h, 128), dtype=torch.float16, device="cuda") for h in (2, 6))
    for num_blocks in (5, 0):
        cache = _empty_cache(num_blocks, fmt)
        kvq.paged_write(x, x, cu, zero, table, *cache)
        k, v = kvq.paged_read(cu, zero, table, *cache, n_tokens=2, k_out=x[:2].clone(), v_out=x[:2].clone())
        assert bool((k == 1).all()) and bool((v == 1).all())
        for ws in (True, False):
            assert not kvq.paged_attention_decode(q, zero, table, *cache, sm_scale=1.0, workspace=ws).any()
            assert not kvq.paged_attention_prefill(q, one, zero, table, *cache, sm_scale=1.0, workspace=ws).any()
    # tokens and lengths that the table has no room for are reported
    kvq.paged_write(x, x, one, zero, table, *cache)
    assert kvq.kvq_fault_status(clear=True) == 4
    assert not kvq.paged_attention_decode(q, zero + 1, table, *cache, sm_scale=1.0).any()
    assert kvq.kvq_fault_status(clear=True) == 8
    # and so is a table whose blocks the cache has not
    table = torch.zeros((B, 300), dtype=torch.int32, device="cuda")
    for ws in (True, False):
        assert not kvq.paged_attention_decode(q, zero + 4700, table, *cache, sm_scale=1.0, workspace=ws).any()
        assert kvq.kvq_fault_status(clear=True) == 4
        assert not kvq.paged_attention_prefill(q, one, zero + 4700, table, *cache, sm_scale=1.0, workspace=ws).any()
        assert kvq.kvq_fault_status(clear=True) == 4


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("part", ["k", "v"])
def test_the_nan_pattern(kvq, D, part):
    """e4m3's NaN pattern, which no write makes, reads as NaN; in attention it stays in its sequence and KV head."""
    c = Case(D, 2, 16, "e4m3", [40, 330], [3, 4], seed=30, R=2)
    page = int(c.table[0, 1])
    (c.kc if part == "k" else c.vc).view(torch.uint8)[page, 0, 5, 7] = 0xFF       # position 21, head 0, channel 7
    d = c.cuda()
    q = c.rows(4, "fp16")
    every = torch.tensor([0, 43, 377], dtype=torch.int32, device="cuda")
    got = kvq.paged_read(every, torch.zeros_like(d.start), d.table, *d.cache(), n_tokens=377)
    for x, name in zip(got, "kv"):
        assert x.isnan().nonzero().tolist() == ([[21, 0, 7]] if name == part else [])
    clean = (c.kc if part == "k" else c.vc).view(torch.uint8)
    clean[page, 0, 5, 7] = 0
    for ws in (True, False):
        want, bound = c.attend(q, c.cu, c.seq_len, 0.1)
        out = kvq.paged_attention_prefill(q.cuda(), d.cu, d.seq_len, d.table, *d.cache(), sm_scale=0.1, workspace=ws)
        hit = out[:3, :2] if part == "k" else out[:3, :2, 7]
        assert hit.isnan().all()
        check(out[:3, 2:], want[:3, 2:], bound[:3, 2:])
        check(out[3:], want[3:], bound[3:])
        want, bound = c.attend(q[2:4], range(3), c.seq_len, 0.1)
        out = kvq.paged_attention_decode(q[2:4].cuda(), d.seq_len, d.table, *d.cache(), sm_scale=0.1, workspace=ws)
        assert (out[0, :2] if part == "k" else out[0, :2, 7]).isnan().all()
        check(out[0, 2:], want[0, 2:], bound[0, 2:])
        check(out[1], want[1], bound[1])


def test_prompts_on_two_streams_at_once(kvq):
    """Split prompt calls, each with the workspace that it allocates, and a write beside them, give what each gives
    alone."""
    c = Case(128, 2, 32, "int8", [4000, 900], [20, 70], seed=31, R=4)
    e = Case(128, 2, 32, "int8", [10, 30], [50, 9], seed=32)
    d, f = c.cuda(), e.cuda()
    qs = [c.rows(8, "bf16").cuda() for _ in range(2)]
    k = e.rows(2, "fp16")
    run = lambda q, **kw: kvq.paged_attention_prefill(q, d.cu, d.seq_len, d.table, *d.cache(), sm_scale=0.1, **kw)
    assert kvq.kvq_paged_prefill_workspace_bytes(2, c.table.shape[1], c.n, 8, 2, 128, 32) > 0
    alone, k_gpu = [run(q) for q in qs], k.cuda()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = [[], []]
    for _ in range(20):
        for i in range(2):
            outs[i].append(run(qs[i], stream=streams[i]))
        kvq.paged_write(k_gpu, k_gpu, f.cu, f.start, f.table, *f.cache(), stream=streams[2])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(same(o, alone[i]) for o in outs[i])
    e.write(k, k)
    assert same_cache(e, f)
