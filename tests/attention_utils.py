"""The attention operators from their definition in 64 bits, with the error that the kernels' arithmetic
allows, element by element.

Notation: p_j = exp(x_j - max x), x_j = scale q.k_j, o = sum p_j v_j / sum p_j, A = sum p_j |v_j| / sum p_j.

- The output is rounded to bf16 once: 2^-8 |o|.
- Prefill rounds each weight p_j to bf16 for the tensor cores: each term moves by at most 2^-8 of itself, so o by
  at most 2^-8 A.  Scaled E4M3 keys are rounded to bf16 first: held against the definition with these rounded keys
  that adds nothing; against the exact ones a logit moves by at most 2^-8 scale sum_d |q_d k_d|.  With E4M3 the
  weights and the scaled values become fp16: each is rounded by at most 2^-11 (2^-10 A together), or below fp16's
  normal range by at most 2^-25.  Weights are 2^(7 + b_j - m) p_j there and values 2^-b_j v_j, b_j the power of the key's
  tile and 2^m at most the largest 2^b_j p_j of the row: so a weight p_j moves by at most 2^-32 2^-b_j max 2^b p and the
  output by 2^-32 (max 2^b p) sum_j 2^-b_j |v_j|, over the keys that the row sees; the values' part is
  2^-25 sum_j 2^b_j p_j (p as a part of the row's sum in both).  Decode rounds the weights to fp16 (E4M3 cache) or splits them
  into two bf16 values (bf16 cache): 2^-11 A covers both (2^-16 for the split).
- A logit is a sum of 128 exact products in fp32: |dx| <= 130 * 2^-24 * scale sum_d |q_d k_d| (the
  accumulation, the scaling and the multiplication by log2 e), plus 2^-21 for exp2 itself and 2^-24 |x_j - max|
  for the rounding of its argument (|x_j - max| p_j < 1 for every j, so 2^-24 of the whole).  Logits that move by
  at most d move every p_j / sum p_j by a factor within exp(+-2d), so o by at most (exp(2d) - 1) A.
- fp32 sums over n keys: n 2^-24 relative at most in each of numerator and denominator, 2 n 2^-24 A.
"""
import torch

BF16, F16, F32 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24
D = 128


def quantise(y):
    """E4M3 bytes and scales of y [..., 128] (one scale per head of a token) in the library's fp32 arithmetic:
    s = max * fl(1/448), codes = e4m3(y * fl(448 / max)).  The quotient of two tensors is rounded once; with a
    Python number on either side torch multiplies by a reciprocal instead.  Below 2^-100, where 448 / max leaves
    fp32, y and max are both taken times 2^64 (exact) before."""
    y = y.double().float()
    m = y.abs().amax(-1)
    s = m * torch.tensor(1.0 / 448.0, dtype=torch.float32, device=y.device)
    lift = torch.where(m < 2.0 ** -100, 2.0 ** 64, 1.0).to(m.dtype)
    q = torch.where(m > 0, torch.full_like(m, 448.0) / torch.where(m > 0, m * lift, 1.0), 0.0)
    return (y * lift[..., None] * q[..., None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8), s


def values(codes, scale=None):
    if scale is None:
        return codes.double()
    return codes.view(torch.float8_e4m3fn).double() * scale.double()[..., None]


def rounded(x):
    """To bf16 by way of fp32, as the kernel does (a code times an fp32 scale is rounded to fp32 on the way)."""
    return x.float().bfloat16().double()


def tile_powers(scales):
    """b of each key and head, [kv heads, tokens], from the scales [tokens, kv heads] of a sequence's values: two to the b
    is 2^-4 of the largest scale's power of two in the key's tile of 128."""
    n = scales.shape[0]
    tiles = torch.nn.functional.pad(scales.double(), (0, 0, 0, -n % 128)).view(-1, 128, scales.shape[1]).amax(1)
    b = torch.where(tiles > 0, torch.floor(torch.log2(tiles)) - 4, 0.0)
    return b.repeat_interleave(128, 0)[:n].T


def attend(q, k, v, scale, weight_step, causal=False, key_step=0.0, powers=None):
    """q [heads, n, 128]; k, v [kv heads, tokens, 128] (fp64).  Returns (o, tolerance), both [heads, n, 128]."""
    g = q.shape[0] // k.shape[0]
    k, v = k.repeat_interleave(g, 0), v.repeat_interleave(g, 0)
    n, tokens = q.shape[1], k.shape[1]
    seen = torch.ones(n, tokens, dtype=torch.double, device=q.device)
    x = q @ k.transpose(1, 2) * scale
    mag = q.abs() @ k.abs().transpose(1, 2) * scale
    if causal:
        i = torch.arange(n, device=q.device)[:, None] + tokens - n
        hide = torch.arange(tokens, device=q.device)[None] > i
        seen.masked_fill_(hide, 0.0)
        x = x.masked_fill(hide, float("-inf"))
        mag = mag.masked_fill(hide, 0.0)
    p = torch.softmax(x, -1)
    o, a = p @ v, p @ v.abs()
    d = (130 * F32 + key_step) * mag.amax(-1, keepdim=True) + 2.0 ** -21 + F32
    tol = BF16 * o.abs() + (weight_step + torch.expm1(2 * d) + 2 * tokens * F32) * a
    if powers is not None:
        two_b = torch.exp2(powers.repeat_interleave(g, 0))
        heavy = p * two_b[:, None]
        tol += 2.0 ** -32 * heavy.amax(-1, keepdim=True) * (seen @ (v.abs() / two_b[..., None]))
        tol += 2.0 ** -25 * heavy.sum(-1, keepdim=True)
    return o, tol * (1 + 2 * BF16) + 1e-30  # products of two of the errors


def assert_within(got, ref, tol, what=""):
    got = got.double()
    err = (got - ref).abs()
    bad = ~(err <= tol)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.numel()} outside, worst {(err / tol).max().item():.3g} of "
                           f"the allowed error at {bad.nonzero()[0].tolist()}")


class Cache:
    """A paged cache with random contents, pages given out in no order; `used` pages of each sequence."""

    def __init__(self, lens, kv, page, fp8, seed=0, extra=2, max_pages=None, fill=None):
        g = torch.Generator().manual_seed(seed)
        need = [-(-max(n, 0) // page) for n in lens]
        self.lens, self.kv, self.page, self.fp8 = lens, kv, page, fp8
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
        k, v = (torch.randn(shape, generator=g).bfloat16().cuda() for _ in range(2))
        self.ks = self.vs = None
        if fp8:
            (k, self.ks), (v, self.vs) = quantise(k), quantise(v)
        if fill is not None:  # every cell that no sequence uses
            free = torch.ones(self.pages, page, dtype=torch.bool)
            for b, n in enumerate(lens):
                for j in range(n):
                    free[table[b, j // page], j % page] = False
            free = free.cuda()[:, None].expand(-1, kv, -1)
            for t in (k, v):
                t[free] = 0x7F if fp8 else fill
            if fp8:
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
        k = values(self.k[at, :, slot], None if self.ks is None else self.ks[at, :, slot])
        v = values(self.v[at, :, slot], None if self.vs is None else self.vs[at, :, slot])
        return k.transpose(0, 1), v.transpose(0, 1)


def check_decode(q, cache, out, scale=D ** -0.5, what="", skip=()):
    heads = q.shape[1] // D
    for b, n in enumerate(cache.lens):
        if b in skip:
            continue
        got = out[b].view(heads, 1, D)
        if n == 0:
            assert (got == 0).all(), f"{what}: sequence {b} is empty"
            continue
        k, v = cache.sequence(b)
        ref, tol = attend(q[b].double().view(heads, 1, D), k, v, scale, F16)
        assert_within(got, ref, tol, f"{what} sequence {b} of {n}")


def check_prefill(q, k, v, ks, vs, lens, out, causal, scale=D ** -0.5, what=""):
    heads, kv = q.shape[1] // D, k.shape[1] // D
    first = 0
    for b, n in enumerate(lens):
        rows = slice(first, first + n)
        first += n
        if n == 0:
            continue
        kk = values(k[rows].reshape(n, kv, D), None if ks is None else ks[rows]).transpose(0, 1)
        vv = values(v[rows].reshape(n, kv, D), None if vs is None else vs[rows]).transpose(0, 1)
        qq, got = q[rows].double().reshape(n, heads, D).transpose(0, 1), out[rows].view(n, heads, D).transpose(0, 1)
        if ks is not None:
            powers = tile_powers(vs[rows])
            ref, tol = attend(qq, kk, vv, scale, 2 * F16, causal, BF16, powers)
            assert_within(got, ref, tol, f"{what} sequence {b} of {n}")
            kk = rounded(kk)
            ref, tol = attend(qq, kk, vv, scale, 2 * F16, causal, powers=powers)
        else:
            ref, tol = attend(qq, kk, vv, scale, BF16, causal)
        assert_within(got, ref, tol, f"{what} sequence {b} of {n}")


def cu(lens):
    c = [0]
    for n in lens:
        c.append(c[-1] + n)
    return torch.tensor(c, dtype=torch.int32).cuda()
