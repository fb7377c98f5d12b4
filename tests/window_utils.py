"""The 4-bit cache and attention with a window from their definitions in 64 bits, for the tests of the operators.

4 bits: a = max|y| over 32 columns, s = a / 7 rounded to five significant bits, code = y / s rounded (both to nearest
even); a group below 2^-120 is zero, one with a value that is not finite has a NaN for s.  Both are exact here: a / 7
in 64 bits is no closer than 2^-3 of a step of s to a border unless it is one, and y / s no closer than 2^-10.

Attention: the allowances of attention_utils, of the keys that a row sees.  The 4-bit decode adds to them: a weight is
rounded to fp16, and its product with a group's scale again (2 * 2^-11 A, the second one at most 2^-25 2^7 of the largest
weight times scale below fp16's normal range); its sums hold codes + 8, which are at most 15 where the code is 1 at least or
stands for nothing, less 8 times the sum of the weights: fp32 sums over n keys, n 2^-24 * (15 + 8) sum_j p_j s_j each.
Sums of products with codes, which are denormal numbers to the tensor cores, keep 2^-14 of the largest weight times
scale (measured 2^-13.8 of their sum); the allowance for weights below fp16's range, 15 * 2^-17 of the largest, holds that.
A logit's sums are over (code + 8) q: 130 * 2^-24 * (15 + 8) * scale sum_d |q_d| s_d.
"""
import torch

from attention_utils import BF16, D, F16, F32, quantise, values

GROUP = 32


def quantise_int4(y):
    """(packed codes [..., 64] uint8, scales [..., 4] bf16) of y [..., 128], computed in 64 bits."""
    y = y.double().unflatten(-1, (D // GROUP, GROUP))
    a = y.abs().amax(-1)
    fine = torch.isfinite(a)
    live = fine & (a >= 2.0 ** -120)
    m, e = torch.frexp(torch.where(live, a, 1.0) / 7)  # m in [1/2, 1)
    s = torch.ldexp(torch.round(m * 32), e - 5).bfloat16().double()  # ldexp's power of two may be an ulp off
    c = torch.where(live[..., None], torch.round(y / s[..., None]), 0.0).long().flatten(-2)
    s = torch.where(fine, torch.where(live, s, 0.0), float("nan"))
    return ((c[..., 0::2] & 15) | ((c[..., 1::2] & 15) << 4)).to(torch.uint8), s.to(torch.bfloat16)


def codes_of(packed):
    n = torch.stack((packed & 15, packed >> 4), -1).flatten(-2).long()
    return torch.where(n > 7, n - 16, n)


def values_int4(packed, scale):
    return codes_of(packed).double() * scale.double().repeat_interleave(GROUP, -1)


def numbers(kind, codes, scale):
    """What entries of a cache of a kind stand for, fp64."""
    return values_int4(codes, scale) if kind == "int4" else values(codes, scale)


class AnyCache:
    """A paged cache (bf16, fp8 or int4) with random contents, pages given out in no order; cells that no sequence uses hold
    `fill` (scales, and bf16 entries) and, in their codes, E4M3's NaN or ones."""

    def __init__(self, lens, kv, page, kind, seed=0, extra=2, max_pages=None, fill=None, std=1.0):
        g = torch.Generator().manual_seed(seed)
        need = [-(-max(n, 0) // page) for n in lens]
        self.lens, self.kv, self.page, self.kind = list(lens), kv, page, kind
        self.pages = sum(need) + extra
        width = max_pages or max(max(need), 1)
        order = torch.randperm(self.pages, generator=g).to(torch.int32)
        table = torch.zeros(len(lens), width, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        self.table = table.cuda()
        self.seq_lens = torch.tensor(lens, dtype=torch.int32).cuda()
        shape = (self.pages, kv, page, D)
        k, v = ((torch.randn(shape, generator=g) * std).bfloat16().cuda() for _ in range(2))
        self.ks = self.vs = None
        if kind != "bf16":
            q = quantise if kind == "fp8" else quantise_int4
            (k, self.ks), (v, self.vs) = q(k), q(v)
        if fill is not None:
            free = torch.ones(self.pages, page, dtype=torch.bool)
            for b, n in enumerate(lens):
                j = torch.arange(max(n, 0))
                free[table[b].long()[j // page], j % page] = False
            free = free.cuda()[:, None].expand(-1, kv, -1)
            for t in (k, v):
                t[free] = fill if kind == "bf16" else 0x7F if kind == "fp8" else 0x77
            if kind != "bf16":
                for t in (self.ks, self.vs):
                    t[free] = fill
        self.k, self.v = k, v

    def args(self):
        return self.k, self.v, self.table, self.seq_lens

    def scales(self):
        return {"k_page_scale": self.ks, "v_page_scale": self.vs}

    def sequence(self, b, n=None):
        """(k, v) of sequence b, [kv heads, tokens, 128] fp64."""
        n = self.lens[b] if n is None else n
        j = torch.arange(n, device="cuda")
        at, slot = self.table[b].long()[j // self.page], j % self.page
        k = numbers(self.kind, self.k[at, :, slot], None if self.ks is None else self.ks[at, :, slot])
        v = numbers(self.kind, self.v[at, :, slot], None if self.vs is None else self.vs[at, :, slot])
        return k.transpose(0, 1), v.transpose(0, 1)

    def value_scales(self, b):
        """Of each value of sequence b, [kv heads, tokens, 128] fp64 (4 bits)."""
        j = torch.arange(self.lens[b], device="cuda")
        at, slot = self.table[b].long()[j // self.page], j % self.page
        return [s[at, :, slot].double().repeat_interleave(GROUP, -1).transpose(0, 1) for s in (self.ks, self.vs)]


def visible(query, key, window, sinks):
    seen = key <= query
    return seen & ((key > query - window) | (key < sinks)) if window else seen


def attend_window(q, k, v, scale, window, sinks, weight_step, key_step=0.0, powers=None, scales=None):
    """q [heads, n, 128], the last n tokens of k and v [kv heads, tokens, 128] (fp64); scales: (of K, of V) where the sums hold
    codes + 8.  Returns (o, tolerance), both [heads, n, 128]; zeros for a row that sees nothing."""
    g = q.shape[0] // k.shape[0]
    k, v = k.repeat_interleave(g, 0), v.repeat_interleave(g, 0)
    n, tokens = q.shape[1], k.shape[1]
    i = torch.arange(n, device=q.device)[:, None] + tokens - n
    hide = ~visible(i, torch.arange(tokens, device=q.device)[None], window, sinks)
    nothing = hide.all(-1)[None, :, None]
    x = (q @ k.transpose(1, 2) * scale).masked_fill(hide, float("-inf"))
    mag = (q.abs() @ k.abs().transpose(1, 2) * scale).masked_fill(hide, 0.0)
    p = torch.softmax(x, -1).nan_to_num(0.0) if bool(nothing.any()) else torch.softmax(x, -1)
    v_seen = v
    o, a = p @ v_seen, p @ v_seen.abs()
    wide = 0.0
    if scales is not None:
        ks, vs = (s.repeat_interleave(g, 0) for s in scales)
        mag = torch.maximum(mag, (23 * q.abs() @ ks.transpose(1, 2) * scale).masked_fill(hide, 0.0))
        wide = 2 * tokens * F32 * 23 * (p @ vs) + 2.0 ** -17 * 15 * (p[..., None] * vs[:, None]).amax(2)
    d = (130 * F32 + key_step) * mag.amax(-1, keepdim=True) + 2.0 ** -21 + F32
    tol = BF16 * o.abs() + (weight_step + torch.expm1(2 * d) + 2 * tokens * F32) * a + wide
    if powers is not None:
        two_b = torch.exp2(powers.repeat_interleave(g, 0))
        heavy = p * two_b[:, None]
        tol += 2.0 ** -32 * heavy.amax(-1, keepdim=True) * ((~hide).double() @ (v.abs() / two_b[..., None]))
        tol += 2.0 ** -25 * heavy.sum(-1, keepdim=True)
    return torch.where(nothing, 0.0, o), torch.where(nothing, 0.0, tol * (1 + 2 * BF16) + 1e-30)
