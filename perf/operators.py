"""The paged 8-bit cache: its write, its read, and attention over it, as calls on one set of inputs.

Cache: codes [num_blocks, Hkv, block, D] of 8 bits (int8 or e4m3) for K and for V, with one fp32 scale per
(block, KV head); ``table`` [B, max_blocks] maps position p of a sequence to slot p % block of block
table[b, p // block].  New tokens lie packed behind one another, sequence b's at cu[b] .. cu[b+1], and begin at
position start[b].
"""
import math
import random

import torch

own = False

QMAX = {"int8": 127.0, "e4m3": 448.0}
FLOAT = {"fp16": torch.float16, "bf16": torch.bfloat16}
SMALLEST, LARGEST = 2.0 ** -40, 2.0 ** 40      # the range of a scale


def listed():
    c = []

    def add(name, op, B, Hkv, R, D, block, fmt, dtype, new, ctx, ragged, window=0, strided=False):
        c.append(dict(name=name, op=op, B=B, Hkv=Hkv, R=R, D=D, block=block, fmt=fmt, dtype=dtype, new=new,
                      ctx=ctx, ragged=ragged, window=window, strided=strided))

    # one decode step's new token of 64 sequences, sliced out of the fused projection: latency
    add("write_append", "write", 64, 8, 4, 128, 64, "int8", "bf16", 1, 1000, 1, strided=True)
    # one long prompt (32K tokens, 8 KV heads) as it is written: bandwidth
    add("write_prompt", "write", 1, 8, 4, 128, 32, "int8", "fp16", 32768, 0, 0)
    # chunks of odd lengths behind odd contexts: every first block is continued, most are recoded
    add("write_chunks", "write", 17, 1, 4, 256, 128, "e4m3", "bf16", 701, 900, 2, strided=True)
    # four caches of 32K tokens read back whole
    add("read_long", "read", 4, 8, 4, 128, 64, "int8", "bf16", 32768, 0, 0)
    # a few ragged stretches read back for a check or a transfer
    add("read_ragged", "read", 9, 2, 6, 64, 16, "e4m3", "fp16", 333, 500, 3)
    # one user's token, 12 query heads on 2 KV heads, 4096 tokens: latency
    add("decode_one", "decode", 1, 2, 6, 128, 32, "int8", "fp16", 1, 4095, 0)
    # 64 users of ragged lengths up to 4096, 32 query heads on 8 KV heads
    add("decode_batch", "decode", 64, 8, 4, 128, 64, "int8", "bf16", 1, 4095, 4)
    # 16 users with 32K tokens each
    add("decode_long", "decode", 16, 8, 4, 128, 64, "e4m3", "fp16", 1, 32767, 0)
    # 1 KV head of 256 channels, a sliding window of 512 in 8 long sequences
    add("decode_window", "decode", 8, 1, 4, 256, 16, "e4m3", "bf16", 1, 16383, 5, window=512)
    # a whole prompt of 8192 tokens: tensor-core rate
    add("prefill_prompt", "prefill", 1, 8, 4, 128, 64, "int8", "bf16", 8192, 0, 0, strided=True)
    # chunks of odd lengths behind contexts of odd lengths, 12 query heads on 2 KV heads, small blocks
    add("prefill_chunks", "prefill", 6, 2, 6, 128, 16, "e4m3", "fp16", 600, 3500, 6)
    # 256 channels, a sliding window of 512
    add("prefill_window", "prefill", 2, 1, 4, 256, 32, "int8", "bf16", 4096, 1000, 7, window=512)
    return c


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["write", "read", "decode", "prefill"])
    Hkv, R = rng.choice([1, 2, 3, 4, 8]), rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    D, block = rng.choice([64, 128, 256]), rng.choice([16, 32, 64, 128])
    fmt, dtype = rng.choice(["int8", "e4m3"]), rng.choice(["fp16", "bf16"])
    row = Hkv * D                                   # channels of one token
    window = 0
    if op in ("write", "read"):
        new = log(1, 32768)
        B = log(1, max(1, min(64, (32768 * 1024) // (new * row))))
        ctx = log(1, 2000) if op == "write" else log(1, 500)
    elif op == "decode":
        new = 1
        ctx = log(1, 32767)
        B = log(1, max(1, min(128, (16 * 32768 * 1024) // ((ctx + 1) * row))))
    else:
        new = log(1, 8192)
        ctx = log(1, 8192)
        pairs = new * (ctx + new) * R * row         # the padded products of one sequence
        B = log(1, max(1, min(32, (8192 * 8192 * 4096) // pairs)))
    if op in ("decode", "prefill") and rng.random() < 0.25:
        window = log(16, 4096)
    return dict(op=op, B=B, Hkv=Hkv, R=R, D=D, block=block, fmt=fmt, dtype=dtype, new=new, ctx=ctx,
                ragged=rng.randrange(1, 1 << 20) if rng.random() < 0.8 else 0, window=window,
                strided=rng.random() < 0.5)


def _lengths(case):
    """(tokens before the new ones, new tokens) of each sequence."""
    B, new, ctx = case["B"], case["new"], case["ctx"]
    if not case["ragged"]:
        return [ctx] * B, [new] * B
    r = random.Random(case["ragged"])
    return [r.randint(ctx // 4, ctx) for _ in range(B)], [r.randint(max(1, new // 8), new) for _ in range(B)]


def _visible(case):
    """(query, key) pairs that are computed, and keys that some query of their sequence sees."""
    pairs = keys = 0
    w = case["window"]
    for c, n in zip(*_lengths(case)):
        if w <= 0:
            pairs += n * c + n * (n + 1) // 2
            keys += c + n
        else:
            full = max(0, min(n, c + n - w + 1 if c < w else n))     # queries with a whole window before them
            part = n - full
            pairs += full * w + part * (c + 1) + part * (part - 1) // 2
            keys += min(c + n, w + n - 1)
    return pairs, keys


def work(case):
    Hkv, D, R, block = case["Hkv"], case["D"], case["R"], case["block"]
    ctx, new = _lengths(case)
    n = sum(new)
    row = Hkv * D
    if case["op"] in ("write", "read"):
        return {"bytes": 2 * n * row * 3 + 8 * Hkv * (n // block + len(new)), "flops": 4 * n * row}
    pairs, keys = _visible(case)
    return {"bytes": 2 * keys * row + 8 * Hkv * (keys // block + len(new)) + 4 * n * R * row,
            "flops": 4 * pairs * R * row}


def _f8(x):
    """x rounded to the nearest e4m3 value."""
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


def _encode(x, fmt):
    return torch.round(x).clamp(-127.0, 127.0).to(torch.int8) if fmt == "int8" else _f8(x)


def _filled(gen, blocks, Hkv, block, D, fmt, gain):
    """Codes and scales of `blocks` blocks of Gaussian rows whose tokens differ in size."""
    codes = torch.empty((blocks, Hkv, block, D), dtype=torch.int8 if fmt == "int8" else torch.float8_e4m3fn,
                        device="cuda")
    scales = torch.empty((blocks, Hkv), dtype=torch.float32, device="cuda")
    step = max(1, (1 << 26) // (Hkv * block * D))
    for b0 in range(0, blocks, step):
        m = min(step, blocks - b0)
        x = torch.randn((m, Hkv, block, D), generator=gen, device="cuda") * gain
        x *= torch.exp(0.3 * torch.randn((m, Hkv, block, 1), generator=gen, device="cuda"))
        s = x.abs().amax((2, 3)) / QMAX[fmt]
        codes[b0:b0 + m] = _encode(x / s[:, :, None, None], fmt)
        scales[b0:b0 + m] = s
    return codes, scales


def prepare(case, seed):
    """The inputs: keys with four channels that stand out, values without; blocks in random order."""
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed) * 7919 + 17)
    B, Hkv, R, D, block, fmt = (case[k] for k in ("B", "Hkv", "R", "D", "block", "fmt"))
    dtype = FLOAT[case["dtype"]]
    ctx, new = _lengths(case)
    used = [-(-(c + n) // block) for c, n in zip(ctx, new)]
    n, total, width = sum(new), sum(used), max(used) + 1
    blocks = total + 3
    order = torch.randperm(blocks, generator=gen, device="cuda")[:total].to(torch.int32).cpu()
    table = torch.zeros((B, width), dtype=torch.int32)
    at = 0
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        at += u
    cu = torch.tensor([0] + new).cumsum(0).to(torch.int32)
    gain = torch.ones(D, device="cuda")
    gain[torch.randperm(D, generator=gen, device="cuda")[:4]] = 8.0
    kc, ks = _filled(gen, blocks, Hkv, block, D, fmt, gain)
    vc, vs = _filled(gen, blocks, Hkv, block, D, fmt, torch.ones(D, device="cuda"))
    s = dict(case=case, table=table.cuda(), cu=cu.cuda(), start=torch.tensor(ctx, dtype=torch.int32).cuda(),
             seq_len=torch.tensor([c + m for c, m in zip(ctx, new)], dtype=torch.int32).cuda(),
             kc=kc, ks=ks, vc=vc, vs=vs, n=n, max_new=max(new), max_len=max(c + m for c, m in zip(ctx, new)),
             sm_scale=1.0 / math.sqrt(D))
    if case["op"] == "read":
        return s
    # q, k and v of the new tokens, out of one fused projection or each on its own
    heads = [R * Hkv, Hkv, Hkv] if case["op"] == "write" or case["strided"] else [R * Hkv]
    parts = []
    for i, h in enumerate(heads):
        x = torch.randn((n, h, D), generator=gen, device="cuda")
        if i:
            x *= torch.exp(0.3 * torch.randn((n, h, 1), generator=gen, device="cuda"))
        parts.append((x * gain if i == 1 else x).to(dtype))
    if case["strided"]:
        parts = list(torch.cat(parts, 1).split(heads, 1))
    s["q"] = parts[0]
    if case["op"] == "write":
        s["k"], s["v"] = parts[1], parts[2]
    return s


# ---- the plain forms ------------------------------------------------------------------------------

def _places(s):
    """Sequence, position, block and slot of every new token."""
    i = torch.arange(s["n"], device="cuda")
    b = torch.searchsorted(s["cu"].long(), i, right=True) - 1
    pos = s["start"].long()[b] + i - s["cu"].long()[b]
    block = s["case"]["block"]
    return b, pos, s["table"].long()[b, pos // block], pos % block


def _write(s, x, codes, scales):
    case = s["case"]
    fmt, block = case["fmt"], case["block"]
    b, pos, page, slot = _places(s)
    x = x.float()
    # every sequence's first block, if it is continued, keeps its scale unless the new tokens need a larger one
    start = s["start"].long()
    first = s["table"].long().gather(1, (start // block)[:, None])[:, 0]
    kept = start % block
    old = torch.where((kept > 0)[:, None], scales[first], torch.zeros_like(scales[first]))
    most = torch.zeros_like(scales).index_reduce_(0, page, x.abs().amax(2), "amax")
    need = (most / QMAX[fmt]).clamp(SMALLEST, LARGEST)
    touched = torch.zeros(scales.shape[0], dtype=torch.bool, device="cuda").index_fill_(0, page, True)
    scales.copy_(torch.where(touched[:, None], need, scales))
    now = torch.maximum(old, need[first])
    scales[first] = now
    # its earlier tokens take the larger scale
    before = codes[first]
    again = _encode(before.float() * (old / now)[:, :, None, None], fmt)
    mine = (torch.arange(block, device="cuda")[None] < kept[:, None])[:, None, :, None] & (now > old)[:, :, None, None]
    bits = torch.where(mine, again.view(torch.uint8), before.view(torch.uint8))
    codes.view(torch.uint8)[first] = bits
    r = 1.0 / scales[page]
    codes.view(torch.uint8)[page, :, slot] = _encode(x * r[:, :, None], fmt).view(torch.uint8)


def _read(s, codes, scales, dtype):
    _, _, page, slot = _places(s)
    x = codes.view(torch.uint8)[page, :, slot].view(codes.dtype).float()
    return (x * scales[page][:, :, None]).to(dtype)


def _attend(s, q, cu, new):
    """q [n, Hq, D] in packed rows; `new` the longest sequence's."""
    case = s["case"]
    B, Hkv, R, D, block, w = (case[k] for k in ("B", "Hkv", "R", "D", "block", "window"))
    T = s["max_len"]
    pages = s["table"].long()[:, :-(-T // block)]

    def rows(codes, scales):                        # [B, Hkv, T, D]
        x = codes.view(torch.uint8)[pages].view(codes.dtype).float() * scales[pages][..., None, None]
        return x.transpose(1, 2).reshape(B, Hkv, -1, D)[:, :, :T]

    cu, length = cu.long(), s["seq_len"].long()
    count = cu[1:] - cu[:-1]
    j = torch.arange(new, device="cuda")
    src = (cu[:-1, None] + j).clamp(max=q.shape[0] - 1)
    x = q[src].float().view(B, new, Hkv, R, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, R * new, D)
    score = torch.matmul(x, rows(s["kc"], s["ks"]).transpose(2, 3)).view(B, Hkv, R, new, T)
    score *= s["sm_scale"]
    t = torch.arange(T, device="cuda")
    at = length[:, None] - count[:, None] + j       # the queries' positions
    seen = t <= at[:, :, None]
    if w > 0:
        seen &= t > at[:, :, None] - w
    score.masked_fill_(~seen[:, None, None], float("-inf"))
    score -= score.amax(-1, keepdim=True)
    score.exp_()
    total = score.sum(-1, keepdim=True)
    o = torch.matmul(score.view(B, Hkv, R * new, T), rows(s["vc"], s["vs"])).view(B, Hkv, R, new, D) / total
    o = o.permute(0, 3, 1, 2, 4).reshape(B, new, Hkv * R, D)
    b, k, _, _ = _places(s)
    return o[b, k - s["start"].long()[b]].to(q.dtype)


def run(s):
    case = s["case"]
    op, dtype = case["op"], FLOAT[case["dtype"]]
    if own:
        from kv_cache_quantization_02_b200 import kvq
        cache = (s["kc"], s["vc"], s["ks"], s["vs"])
        if op == "write":
            kvq.paged_write(s["k"], s["v"], s["cu"], s["start"], s["table"], *cache)
            return {"k": s["kc"], "v": s["vc"], "k_scales": s["ks"], "v_scales": s["vs"]}
        if op == "read":
            k, v = kvq.paged_read(s["cu"], s["start"], s["table"], *cache, n_tokens=s["n"], dtype=dtype)
            return {"k": k, "v": v}
        if op == "decode":
            return kvq.paged_attention_decode(s["q"], s["seq_len"], s["table"], *cache, sm_scale=s["sm_scale"],
                                              window=case["window"])
        return kvq.paged_attention_prefill(s["q"], s["cu"], s["seq_len"], s["table"], *cache,
                                           sm_scale=s["sm_scale"], window=case["window"])
    if op == "write":
        _write(s, s["k"], s["kc"], s["ks"])
        _write(s, s["v"], s["vc"], s["vs"])
        return {"k": s["kc"], "v": s["vc"], "k_scales": s["ks"], "v_scales": s["vs"]}
    if op == "read":
        return {"k": _read(s, s["kc"], s["ks"], dtype), "v": _read(s, s["vc"], s["vs"], dtype)}
    return _attend(s, s["q"], s["cu"], s["max_new"])


# ---- from the definition, in 64 bits ----------------------------------------------------------------

def exact(case, seed):
    op, block, D, R = case["op"], case["block"], case["D"], case["R"]
    s = prepare(case, seed)
    ctx, new = _lengths(case)
    table = s["table"].tolist()
    if op == "write":
        # codes have no value off their grid; the scales do
        out = {}
        for name, x, sc in (("k_scales", s["k"], s["ks"]), ("v_scales", s["v"], s["vs"])):
            if len(new) + sum(new) // block > 20000:
                return None
            sc = sc.double()
            row = 0
            for b, (c, n) in enumerate(zip(ctx, new)):
                size = x[row:row + n].double().abs().amax(2)
                for p in range(c // block, (c + n - 1) // block + 1):
                    lo, hi = max(c, p * block), min(c + n, (p + 1) * block)
                    a = (size[lo - c:hi - c].amax(0) / QMAX[case["fmt"]]).clamp(SMALLEST, LARGEST)
                    page = table[b][p]
                    sc[page] = torch.maximum(sc[page], a) if lo > p * block else a
                row += n
            out[name] = sc
        return {"k": None, "v": None, **out}

    def tokens(b, codes, scales, lo, hi):           # positions lo .. hi of sequence b: [hi - lo, Hkv, D]
        first = lo // block
        at = torch.tensor(table[b][first:-(-hi // block)], device="cuda")
        x = codes.view(torch.uint8)[at].view(codes.dtype).double() * scales[at].double()[:, :, None, None]
        return x.transpose(1, 2).reshape(-1, case["Hkv"], D)[lo - first * block:hi - first * block]

    if op == "read":
        every = range(case["B"])
        return {"k": torch.cat([tokens(b, s["kc"], s["ks"], ctx[b], ctx[b] + new[b]) for b in every]),
                "v": torch.cat([tokens(b, s["vc"], s["vs"], ctx[b], ctx[b] + new[b]) for b in every])}
    if 4.0 * case["Hkv"] * R * D * sum(n * (c + n) for c, n in zip(ctx, new)) > 6e12:
        return None
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    row = 0
    for b, (c, n) in enumerate(zip(ctx, new)):
        k, v = (tokens(b, x, y, 0, c + n).permute(1, 0, 2) for x, y in ((s["kc"], s["ks"]), (s["vc"], s["vs"])))
        for q0 in range(0, n, 256):
            m = min(256, n - q0)
            for h in range(case["Hkv"]):
                q = s["q"][row + q0:row + q0 + m, h * R:(h + 1) * R].double()
                z = torch.einsum("mrd,td->mrt", q, k[h]) / math.sqrt(D)
                pos = torch.arange(c + q0, c + q0 + m, device="cuda")[:, None]
                t = torch.arange(c + n, device="cuda")[None]
                hide = t > pos
                if case["window"] > 0:
                    hide = hide | (t <= pos - case["window"])
                p = torch.softmax(z.masked_fill(hide[:, None], float("-inf")), -1)
                out[row + q0:row + q0 + m, h * R:(h + 1) * R] = torch.einsum("mrt,td->mrd", p, v[h])
        row += n
    return out
