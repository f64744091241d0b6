"""How the paged attentions share out their keys: every way of dividing a call
over thread blocks against 64 bits, each case with the condition that makes it
one of that kind, and the workspaces that the caller brings."""
import math

import pytest
import torch

from paged_util import DTYPES, Case, check
from test_paged import kvq, no_faults, same         # noqa: F401  (fixtures)

pytestmark = pytest.mark.gpu


def exact(d, q, cu, lens, scale, window=0):
    """Case.attend on the GPU, whose 64-bit arithmetic these sizes want."""
    with torch.device("cuda"):
        return tuple(x.cpu() for x in d.attend(q.cuda(), cu, lens, scale, window))


def decode_blocks(kvq, c, R, window):
    """Thread blocks of a split decode call, from its workspace: two sets of eight heads' sums and a record each."""
    n = kvq.kvq_paged_decode_workspace_bytes(c.B, c.table.shape[1], c.Hkv * R, c.Hkv, c.D, c.block, window)
    each = 2 * 8 * (c.D + 4) * 4 + 16
    assert n % each == 0
    return n // each


def decode_tiles(c, lens, R, window):
    """(sequence, KV head, up to 8 heads) items' 32-key tiles, each item's as whole rounds of four."""
    tiles = 0
    for n in lens:
        lo = max(0, n - window) // 32 * 32 if window else 0
        tiles += -(-(-(-(n - lo) // 32)) // 4) * 4
    return tiles * c.Hkv * -(-R // 8)


def decode_case(kvq, D, Hkv, R, block, fmt, dtype, lens, window, equal):
    c = Case(D, Hkv, block, fmt, [max(0, n - 1) for n in lens], [min(1, n) for n in lens], seed=D + R + len(lens), R=R)
    blocks, rounds = decode_blocks(kvq, c, R, window), decode_tiles(c, lens, R, window)
    assert blocks > 0                               # split
    assert (rounds > 4 * blocks) is equal           # into equal shares of the line, or rounds inside items
    lens = torch.tensor(lens, dtype=torch.int32)
    q = (torch.randn((c.B, Hkv * R, D), generator=c.g) * 1.5).to(DTYPES[dtype])
    d = c.cuda()
    scale = 1.0 / math.sqrt(D)
    want, bound = exact(d, q, range(c.B + 1), lens, scale, window)
    args = (q.cuda(), lens.cuda(), d.table, *d.cache())
    got = kvq.paged_attention_decode(*args, sm_scale=scale, window=window)
    check(got, want, bound)
    assert same(got, kvq.paged_attention_decode(*args, sm_scale=scale, window=window))
    check(kvq.paged_attention_decode(*args, sm_scale=scale, window=window, workspace=False), want, bound)


def ragged(B, most, seed):
    """Lengths of which some are 0, 1 or a tile's border."""
    g = torch.Generator().manual_seed(seed)
    lens = (torch.rand(B, generator=g) * most).int().tolist()
    for i, n in zip(range(3, B, 7), [0, 1, 32, 0, 33, most, 0, 128, 129] * B):
        lens[i] = n
    return lens


EQUAL = [
    # D, Hkv, R, block, fmt, dtype, B, longest: up to 32 sequences each warp scans for itself, more the block does
    (64, 8, 4, 16, "int8", "bf16", 24, 2500),
    (128, 8, 4, 64, "e4m3", "fp16", 24, 2500),
    (256, 8, 2, 128, "int8", "bf16", 24, 2500),
    (256, 8, 3, 32, "e4m3", "fp16", 32, 1500),
    (128, 8, 7, 32, "int8", "bf16", 40, 2100),
    (64, 4, 12, 64, "e4m3", "bf16", 40, 2500),
    (256, 4, 16, 16, "int8", "fp16", 33, 1700),
    (128, 8, 1, 16, "int8", "fp16", 140, 900),
    (64, 8, 5, 32, "e4m3", "fp16", 140, 1100),
    (256, 8, 9, 64, "e4m3", "bf16", 140, 700),
]


@pytest.mark.parametrize("D,Hkv,R,block,fmt,dtype,B,most", EQUAL)
@pytest.mark.parametrize("window", [0, 600])
def test_decode_in_equal_shares(kvq, D, Hkv, R, block, fmt, dtype, B, most, window):
    decode_case(kvq, D, Hkv, R, block, fmt, dtype, ragged(B, most, D + B), window, True)


@pytest.mark.parametrize("D,R,fmt,n", [(64, 4, "int8", 90001), (128, 8, "e4m3", 70000), (256, 2, "int8", 62003)])
def test_decode_of_one_item_in_hundreds_of_shares(kvq, D, R, fmt, n):
    """One KV head whose line is cut everywhere: one join takes all the stretches' sums."""
    decode_case(kvq, D, 1, R, 64, fmt, "fp16", [n], 0, True)


FEW = [
    (64, 2, 4, 16, "int8", "bf16", 9, 900), (128, 1, 12, 32, "e4m3", "fp16", 20, 700),
    (256, 1, 4, 16, "e4m3", "bf16", 32, 1200), (128, 1, 3, 64, "int8", "bf16", 40, 700),
    (64, 1, 9, 128, "e4m3", "fp16", 70, 500), (256, 1, 1, 64, "int8", "fp16", 140, 300),
]


@pytest.mark.parametrize("D,Hkv,R,block,fmt,dtype,B,most", FEW)
@pytest.mark.parametrize("window", [0, 400])
def test_decode_in_rounds_inside_items(kvq, D, Hkv, R, block, fmt, dtype, B, most, window):
    decode_case(kvq, D, Hkv, R, block, fmt, dtype, ragged(B, most, D + B), window, False)


def prompt_pieces(kvq, c, R, window, rows):
    """Pieces that the workspace of a prompt call has room for, and the call's row tiles."""
    n = kvq.kvq_paged_prefill_workspace_bytes(c.B, c.table.shape[1], c.n, c.Hkv * R, c.Hkv, c.D, c.block, window)
    each = rows * (c.D + 2) * 4
    assert n % each == 0
    return n // each, (c.n * R // rows + c.B) * c.Hkv


def prompt_case(kvq, D, Hkv, R, block, fmt, dtype, ctx, new, window, kind):
    c = Case(D, Hkv, block, fmt, ctx, new, seed=D + R + len(ctx), R=R)
    pieces, tiles = prompt_pieces(kvq, c, R, window, 128 if D == 256 else 256)
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    if kind == "rest":                              # full rounds whole, the tiles after them in two pieces or more
        assert tiles > sms and 2 * (tiles % sms) <= pieces and pieces % (tiles % sms) == 0
    else:                                           # every tile in two pieces or more
        assert tiles < 2 * sms and 2 * tiles <= pieces and pieces % tiles == 0
    q = c.rows(Hkv * R, dtype, 1.5)
    d = c.cuda()
    scale = 1.0 / math.sqrt(D)
    want, bound = exact(d, q, c.cu, c.seq_len, scale, window)
    args = (q.cuda(), d.cu, d.seq_len, d.table, *d.cache())
    got = kvq.paged_attention_prefill(*args, sm_scale=scale, window=window)
    check(got, want, bound)
    assert same(got, kvq.paged_attention_prefill(*args, sm_scale=scale, window=window))
    check(kvq.paged_attention_prefill(*args, sm_scale=scale, window=window, workspace=False), want, bound)


def behind(B, most, seed):
    """Contexts, and few new tokens behind them; one chunk of 40, some sequences without any."""
    ctx = ragged(B, most, seed)
    new = [(3 * b) % 4 for b in range(B)]
    new[B // 3] = 40
    ctx[B // 3] = most
    return ctx, new


PROMPTS = [
    # whole prompts whose longest tile is split (the tiles see anything from nothing to all)
    ("all", 128, 2, 4, 64, "int8", "bf16", [0], [4096], 0),
    ("all", 64, 2, 4, 32, "e4m3", "fp16", [0], [4001], 0),
    ("all", 256, 2, 4, 16, "int8", "fp16", [0], [2047], 0),
    ("all", 128, 1, 6, 128, "e4m3", "bf16", [3, 0], [2500, 1500], 0),
    # more than 32 sequences behind contexts: every tile split
    ("all", 128, 2, 3, 16, "int8", "bf16", *behind(33, 3000, 1), 0),
    ("all", 256, 1, 4, 64, "e4m3", "fp16", *behind(40, 2500, 2), 0),
    ("all", 256, 2, 2, 32, "int8", "bf16", *behind(34, 3000, 3), 700),
    # and their tiles more than thread blocks run at once
    ("rest", 128, 4, 4, 64, "int8", "bf16", *behind(40, 4000, 4), 0),
    ("rest", 256, 4, 4, 16, "e4m3", "bf16", *behind(39, 3000, 5), 0),
    ("rest", 64, 4, 5, 32, "e4m3", "fp16", *behind(76, 4000, 6), 0),
    ("rest", 256, 8, 1, 128, "int8", "fp16", *behind(40, 2500, 7), 0),
    ("rest", 128, 4, 8, 32, "e4m3", "fp16", *behind(39, 4000, 8), 1500),
]


@pytest.mark.parametrize("kind,D,Hkv,R,block,fmt,dtype,ctx,new,window", PROMPTS)
def test_prompts_split_from_the_host(kvq, kind, D, Hkv, R, block, fmt, dtype, ctx, new, window):
    prompt_case(kvq, D, Hkv, R, block, fmt, dtype, ctx, new, window, kind)


WORKSPACES = [
    # D, Hkv, R, block, fmt, ctx, new
    (128, 2, 4, 64, "int8", [5000, 3], [1, 1], "decode"),
    (64, 8, 12, 32, "e4m3", [2000] * 20, [1] * 20, "decode"),
    (256, 4, 4, 32, "int8", [1800] * 40, [1] * 40, "decode"),
    (128, 2, 4, 64, "int8", [0], [4096], "prompt"),
    (256, 1, 4, 16, "e4m3", [1500, 40, 900], [40, 3, 100], "prompt"),
    (64, 2, 3, 64, "int8", [900] * 33, [2] * 33, "prompt"),
]


@pytest.mark.parametrize("D,Hkv,R,block,fmt,ctx,new,kind", WORKSPACES)
def test_the_callers_workspace(kvq, D, Hkv, R, block, fmt, ctx, new, kind):
    """Exactly the bytes asked for, used by one call after another and by two captured graphs, and none behind them
    touched; what is too small or not aligned leaves the call unsplit."""
    c = Case(D, Hkv, block, fmt, ctx, new, seed=29, R=R)
    d = c.cuda()
    qs = [c.rows(Hkv * R, "bf16").cuda() for _ in range(2)]
    W = c.table.shape[1]
    if kind == "decode":
        need = kvq.kvq_paged_decode_workspace_bytes(c.B, W, Hkv * R, Hkv, D, block)
        call = lambda q, **kw: kvq.paged_attention_decode(q, d.seq_len, d.table, *d.cache(), sm_scale=0.1, **kw)
    else:
        need = kvq.kvq_paged_prefill_workspace_bytes(c.B, W, c.n, Hkv * R, Hkv, D, block)
        call = lambda q, **kw: kvq.paged_attention_prefill(q, d.cu, d.seq_len, d.table, *d.cache(), sm_scale=0.1, **kw)
    assert need > 0
    alone, unsplit = [call(q) for q in qs], [call(q, workspace=False) for q in qs]
    room = torch.full((need + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        for q, want in zip(qs, alone):
            assert same(call(q, workspace=room[:need]), want)
    graphs, outs = [], [torch.empty_like(x) for x in alone]
    for q, out in zip(qs, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call(q, workspace=room[:need], out=out)
    for _ in range(3):
        for out in outs:
            out.fill_(7.0)
        for g in graphs:
            g.replay()
        assert all(same(out, want) for out, want in zip(outs, alone))
    assert bool((room[need:] == 0xA5).all())
    room.fill_(0xA5)
    for short in (room[:need - 16], room[8:need + 8], room[:0]):
        assert same(call(qs[0], workspace=short), unsplit[0])
    assert bool((room == 0xA5).all())
