"""Plain forms of the paged 8-bit cache for the tests: its write in fp32, one
operation at a time as include/kvq.h defines it, its read, and attention in
64 bits with the bound that each output has to keep."""
from __future__ import annotations

import math

import torch

QMAX = {torch.int8: 127.0, torch.float8_e4m3fn: 448.0}
FORMATS = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
SMALLEST, LARGEST = 2.0 ** -40, 2.0 ** 40


def encode(x, fmt):
    x = torch.nan_to_num(x, nan=0.0, posinf=math.inf, neginf=-math.inf)
    if fmt == torch.int8:
        return torch.round(x).clamp(-127.0, 127.0).to(torch.int8)
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)


class Case:
    """A cache on the CPU with `ctx[b]` positions before `new[b]` new tokens of
    each sequence, blocks in random order, everything that nothing may read
    filled with codes and scales that would show."""

    def __init__(self, D, Hkv, block, fmt, ctx, new, seed, R=1, spare=3, extra=2):
        g = torch.Generator().manual_seed(seed)
        self.D, self.Hkv, self.block, self.fmt, self.R = D, Hkv, block, FORMATS[fmt], R
        self.ctx, self.new = list(ctx), list(new)
        self.B = len(self.ctx)
        used = [-(-(c + n) // block) for c, n in zip(ctx, new)]
        self.num_blocks = sum(used) + spare
        width = max(used + [0]) + extra
        order = torch.randperm(self.num_blocks, generator=g)[:sum(used)].to(torch.int32)
        self.table = torch.full((self.B, width), -7, dtype=torch.int32)      # not to be used
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = order[at:at + u]
            at += u
        self.cu = torch.tensor([0] + self.new).cumsum(0).to(torch.int32)
        self.start = torch.tensor(self.ctx, dtype=torch.int32)
        self.seq_len = torch.tensor([c + n for c, n in zip(ctx, new)], dtype=torch.int32)
        self.n = sum(self.new)
        shape = (self.num_blocks, Hkv, block, D)
        bits = torch.randint(0, 256, shape, generator=g).to(torch.uint8)
        if fmt == "e4m3":
            bits[(bits & 0x7F) == 0x7F] = 0x7E                               # never the NaN pattern
        self.kc, self.vc = (x.clone().view(self.fmt) for x in (bits, bits.flip(0)))
        span = 0.02 if fmt == "int8" else 0.006
        self.ks, self.vs = (torch.rand((self.num_blocks, Hkv), generator=g) * span + span / 8 for _ in range(2))
        self.g = g

    def rows(self, heads, dtype, gain=1.0, tail=0):
        """Token rows for the new tokens and `tail` more."""
        return (torch.randn((self.n + tail, heads, self.D), generator=self.g) * gain).to(DTYPES[dtype])

    def cuda(self):
        import copy
        c = copy.copy(self)
        for name in ("table", "cu", "start", "seq_len", "kc", "vc", "ks", "vs"):
            setattr(c, name, getattr(self, name).cuda())
        return c

    def cache(self):
        return self.kc, self.vc, self.ks, self.vs

    # ---- plain forms -------------------------------------------------------------

    def write(self, k, v):
        """In place, token by token range; blocks outside the table are skipped."""
        for x, codes, scales in ((k, self.kc, self.ks), (v, self.vc, self.vs)):
            q = QMAX[self.fmt]
            for b in range(self.B):
                c, n, row = self.ctx[b], self.new[b], int(self.cu[b])
                for j in range(c // self.block, -(-(c + n) // self.block) if n else 0):
                    lo, hi = max(c, j * self.block), min(c + n, (j + 1) * self.block)
                    if j >= self.table.shape[1] or not 0 <= int(self.table[b, j]) < self.num_blocks:
                        continue
                    page, slot = int(self.table[b, j]), lo - j * self.block
                    y = x[row + lo - c:row + hi - c].float()                 # [m, Hkv, D]
                    a = torch.nan_to_num(y.abs(), nan=0.0, posinf=math.inf).amax((0, 2))
                    s = (a * (1.0 / torch.tensor(q))).clamp(SMALLEST, LARGEST)
                    old = scales[page].clone()
                    S = torch.maximum(old, s) if slot else s
                    if slot:
                        again = encode(codes[page, :, :slot].float() * (old / S)[:, None, None], self.fmt)
                        grew = (S > old)[:, None, None]
                        now = torch.where(grew, again.view(torch.uint8), codes[page, :, :slot].view(torch.uint8))
                        codes.view(torch.uint8)[page, :, :slot] = now
                    scales[page] = S
                    z = encode(y * (1.0 / S)[None, :, None], self.fmt)
                    codes.view(torch.uint8)[page, :, slot:slot + hi - lo] = z.transpose(0, 1).view(torch.uint8)

    def read(self, dtype):
        """[n, Hkv, D] of K and of V."""
        out = []
        for codes, scales in ((self.kc, self.ks), (self.vc, self.vs)):
            rows = []
            for b in range(self.B):
                for p in range(self.ctx[b], self.ctx[b] + self.new[b]):
                    page = int(self.table[b, p // self.block])
                    rows.append(codes[page, :, p % self.block].float() * scales[page][:, None])
            out.append(torch.stack(rows).to(DTYPES[dtype]) if rows else torch.empty((0, self.Hkv, self.D)))
        return out

    def keys(self, b, L):
        """K and V of sequence b's first L positions in 64 bits, [L, Hkv, D], the value scales [L, Hkv], and
        which of the positions are in the table."""
        t = torch.arange(L)
        j = t // self.block
        page = torch.where(j < self.table.shape[1], self.table[b].long()[j.clamp(max=self.table.shape[1] - 1)], -1)
        ok = (page >= 0) & (page < self.num_blocks)
        page, slot = page.clamp(0, self.num_blocks - 1), t % self.block
        k, v = (c.view(torch.uint8)[page, :, slot].view(self.fmt).double() * s[page].double()[:, :, None]
                for c, s in ((self.kc, self.ks), (self.vc, self.vs)))
        return k, v, self.vs[page].double(), ok

    def attend(self, q, cu, lens, sm_scale, window=0):
        """Attention in 64 bits of packed query rows, and the bound on each output's distance from it.

        The kernels hold scores and sums in fp32 (u = 2^-24) and round each softmax weight to fp16 before the
        value product.  With z the largest sum_d |q_d k_d| sm_scale over the keys, a score is off by at most
        e = (D + 8) u z (D products added in any order, the scales and the exponent's argument), plus a few u
        of the argument itself, |s| <= z; the value scale's logarithm b (|b| <= y) joins the argument,
        four roundings of it and a reference at most y + z away; the exponential adds 2^-21.  So each weight is off
        by r = 2 e + 2^-21 + 8 u (z + y) relative (numerator and denominator), then by 2^-11 from fp16 or, below fp16's normal
        range, by 2^-25 of the largest weight times value scale of the row, which is at least 1 as the kernels
        hold it: 2^-25 Q for each of the L keys.  L additions in fp32 add (L + 64) 2 u.  With A = sum_t p_t |v_t|
        for the output's channel:
            |out - o| <= eps/2 |o| (1 + 2^-8) + A (2^-11 + r + (L + 64) 2 u) + L 2^-25 Q max_t(p_t S_t)
        and the least subnormal of the output's type."""
        total, Hq, D = q.shape
        out = torch.zeros((total, Hq, D), dtype=torch.float64)
        bound = torch.zeros((total, Hq, D), dtype=torch.float64)
        u, eps = 2.0 ** -24, torch.finfo(q.dtype).eps
        least = 2.0 ** -24 if q.dtype == torch.float16 else 2.0 ** -133
        R = Hq // self.Hkv
        for b in range(len(lens)):
            L, r0, r1 = int(lens[b]), int(cu[b]), int(cu[b + 1])
            if L <= 0 or r1 <= r0:
                continue
            k, v, sv, ok = self.keys(b, L)
            pos = L - (r1 - r0) + torch.arange(r1 - r0)
            t = torch.arange(L)
            seen = (t[None] <= pos[:, None]) & ok[None]
            if window > 0:
                seen &= t[None] > pos[:, None] - window
            x = q[r0:r1].double().view(r1 - r0, self.Hkv, R, D)
            s = torch.einsum("nhrd,thd->nhrt", x, k) * sm_scale
            big = torch.einsum("nhrd,thd->nhrt", x.abs(), k.abs()) * abs(sm_scale)
            hide = ~seen[:, None, None, :]
            p = torch.softmax(s.masked_fill(hide, -math.inf), -1)
            p = torch.nan_to_num(p, nan=0.0)                                 # rows that see nothing
            z = big.masked_fill(hide, 0.0).amax(-1)
            o = torch.einsum("nhrt,thd->nhrd", p, v)
            A = torch.einsum("nhrt,thd->nhrd", p, v.abs())
            y = sv.log2().abs().max()
            r = 2 * (D + 8) * u * z + 8 * u * (z + y) + 2.0 ** -21
            top = (p * sv.t()[None, :, None, :]).amax(-1)
            e = o.abs() * (eps / 2 * (1 + 2.0 ** -8)) + A * (2.0 ** -11 + r + (L + 64) * 2 * u)[..., None]
            e = e + (L * 2.0 ** -25 * QMAX[self.fmt] * top)[..., None] + least
            out[r0:r1] = o.reshape(r1 - r0, Hq, D)
            bound[r0:r1] = e.reshape(r1 - r0, Hq, D)
        return out, bound


def check(got, want, bound):
    got = got.double().cpu()
    assert torch.isfinite(got).all()
    off = (got - want).abs() - bound
    worst = int(off.argmax())
    assert (off <= 0).all(), (f"{int((off > 0).sum())} of {off.numel()} outputs; at {worst}: got "
                              f"{got.flatten()[worst].item()}, want {want.flatten()[worst].item()} "
                              f"within {bound.flatten()[worst].item()}")
