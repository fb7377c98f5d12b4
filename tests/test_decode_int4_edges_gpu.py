"""Decode over a 4-bit cache where its kernel's own arithmetic and its ring have their edges: waits that run out, scales at both
ends of their range, long flat attention, pages of many tokens, lengths that no count holds."""
import pytest
import torch

import gemm_epilogue_tcgen05_gb300 as fl
from attention_utils import BF16, D, assert_within, cu
from test_attention_window_gpu import KINDS, STEP, check_decode, randn
from window_utils import AnyCache, attend_window, quantise_int4, values_int4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("page", [16, 3])  # tensor copies, copies by 16 bytes
def test_ring_serves_on_after_waits_that_ran_out(page):
    """A sequence behind a hundred empty ones: the warp that fills the ring is through with these at once and waits some hundred
    microseconds for a free stage, with a limit of one.  What the call could not finish is NaN, the rest is right, and the
    workspace serves on."""
    lens = ([0] * 100 + [640]) * 1000
    c = AnyCache([640], 1, page, "int4", seed=1)
    pages = c.table.shape[1]
    table = c.table.expand(len(lens), pages)  # all sequences have the same tokens
    seq_lens = torch.tensor(lens, dtype=torch.int32).cuda()
    q = randn(1, D, seed=2).expand(len(lens), D).contiguous()
    ws = fl.attention_decode_workspace()
    full = seq_lens > 0

    def call():
        return fl.attention_decode_window(q, c.k, c.v, table.contiguous(), seq_lens, workspace=ws, **c.scales())

    want = call()
    assert fl.check_device_status(ws) == fl.FL_OK
    check_decode(q[:1], c, want[100:101])
    assert (want[~full] == 0).all()
    for _ in range(2):
        try:
            fl.set_wait_timeout_ns(1000)
            out = call()
            status = fl.check_device_status(ws)
        finally:
            fl.set_wait_timeout_ns(0)
        assert status == fl.FL_ERR_TIMEOUT
        nan = torch.isnan(out).any(1)
        assert nan.any() and not nan[~full].all()
        assert torch.equal(out[~nan], want[~nan])
        assert torch.equal(call(), want)
        assert fl.check_device_status(ws) == fl.FL_OK


# ---------------------------------------------------------------- scales at the low end
def check_small_values(q, cache, out, up):
    """As check_decode, with everything 2^up times as large so that its absolute allowance means nothing; the output is
    rounded to bf16's smallest step, 2^-133, where it is below the normal range, and to fp32's, 2^-149, before."""
    heads = q.shape[1] // D
    for b in range(len(cache.lens)):
        k, v = cache.sequence(b)
        scales = cache.value_scales(b) if cache.kind == "int4" else None
        if scales is not None:
            scales = scales[0], scales[1] * 2.0 ** up
        ref, tol = attend_window(q[b].double().view(heads, 1, D), k, v * 2.0 ** up, D ** -0.5, 0, 0, STEP[cache.kind], scales=scales)
        assert (tol < 0.1 * ref.abs().amax()).all()  # zeros do not pass
        assert_within(out[b].double().view(heads, 1, D) * 2.0 ** up, ref, tol + (2.0 ** -134 + 2.0 ** -149) * 2.0 ** up, f"sequence {b}")


@pytest.mark.parametrize("power", [-110, -116, -118, -119, -121, -124])
@pytest.mark.parametrize("lens", [[200, 33], [1500]])  # finished by one CTA, joined from pieces
def test_decode_over_4_bits_of_the_smallest_scales(power, lens):
    """Scales of some 2^-1 to 2^-2 times 2^power, down to bf16's smallest normal ones: the values are normal bf16 numbers."""
    c = AnyCache(lens, 2, 16, "int4", seed=10)
    c.vs *= torch.tensor(2.0 ** power, device="cuda").bfloat16()
    q = randn(len(lens), 12 * D, seed=11)
    check_small_values(q, c, fl.attention_decode_window(q, *c.args(), **c.scales()), -power)


@pytest.mark.parametrize("power", [-110, -118, -122, -126])
@pytest.mark.parametrize("lens", [[200, 33], [1500]])
def test_decode_over_e4m3_of_the_smallest_scales(power, lens):
    """Scales of some 2^-7 times 2^power, below fp32's normal range in the end; the values are not."""
    c = AnyCache(lens, 2, 16, "fp8", seed=10)
    c.vs = (c.vs.double() * 2.0 ** power).float()
    q = randn(len(lens), 12 * D, seed=11)
    check_small_values(q, c, fl.attention_decode_window(q, *c.args(), **c.scales()), -power)
    check_small_values(q, c, fl.attention_decode(q, *c.args(), **c.scales()), -power)


# ---------------------------------------------------------------- long sums
def shared(cache, batch):
    """Many sequences with the tokens of one: each CTA walks most of a (sequence, head) by itself."""
    return (cache.k, cache.v, cache.table.expand(batch, -1).contiguous(), cache.seq_lens.expand(batch).contiguous())


def test_decode_over_4_bits_flat_attention_over_many_tokens():
    """All weights are alike: these, and their products with the scales, are exact.  A sum of 16 products with a running sum r is
    truncated to 2^-23 of the larger of |r| and what it adds, 16 * 15 weights times scale for the codes + 8 of one product,
    and the sum of the eights is taken off once in two products (2^-24).  So a warp that walks a quarter of n tokens leaves
    (n / 64) 1.25 2^-23 (max |r| + 480 s), 2^-27 1.25 (max |r| + 480 s) of the output for all four; values are random signs of
    some 1, so |r| stays below 5 sqrt(n / 4).  (With all eights taken off at the end: 2 % of the output.)"""
    n, kv, batch = 400000, 8, 64
    c = AnyCache([n], kv, 64, "int4", seed=21)
    q = torch.zeros(batch, 2 * kv * D, dtype=torch.bfloat16, device="cuda")
    out = fl.attention_decode_window(q, *shared(c, batch), **c.scales()).view(batch, kv, 2, D).double()
    ref = c.sequence(0)[1].mean(1)
    s = c.value_scales(0)[1].amax(1)
    tol = BF16 * ref.abs() + 1.25 * 2.0 ** -27 * (5 * (n / 4) ** 0.5 + 480 * s) + 2.0 ** -20 * ref.abs()
    err = (out - ref[:, None]).abs()
    assert (err <= tol[:, None]).all(), f"worst {(err / tol[:, None]).max():.3f} of the allowance"


@pytest.mark.parametrize("n", [9000, 40000])
def test_decode_over_4_bits_nearly_flat_attention_over_many_tokens(n):
    """Over all elements: the output's rounding is 2^-8 / sqrt(3) of them at most, the two of the weights and their products with
    scales 2^-11 each of values that average out as they do (a quarter of 2^-8), and what 16 products drop, 2^-14 of a weight
    times scale, 2^-18 of the sum p s, and again for the running sums."""
    kv, batch = 8, 64
    c = AnyCache([n], kv, 64, "int4", seed=22)
    q = randn(1, 2 * kv * D, seed=23, std=0.05).expand(batch, -1).contiguous()
    out = fl.attention_decode_window(q, *shared(c, batch), **c.scales()).view(batch, 2 * kv, 1, D).double()
    k, v = c.sequence(0)
    ref = attend_window(q[0].double().view(2 * kv, 1, D), k, v, D ** -0.5, 0, 0, 0.0)[0]
    s = c.value_scales(0)[1].mean()
    err = (out - ref).square().mean().sqrt()
    assert err <= BF16 * ref.square().mean().sqrt() + 2.0 ** -17 * s, f"{err:.3e} of outputs of {ref.square().mean().sqrt():.3e}"


# ---------------------------------------------------------------- scales of -0
def test_scales_of_minus_zero_are_zeros():
    for spread in (False, True):
        c = AnyCache([300, 700], 2, 16, "int4", seed=31)
        g = torch.Generator().manual_seed(32)
        if spread:
            c.vs *= torch.exp2(torch.randint(-30, 31, c.vs.shape, generator=g).float().cuda()).bfloat16()
        for s in (c.ks, c.vs):
            s[torch.rand(s.shape, generator=g).cuda() < 0.2] = 0.0
        q = randn(2, 8 * D, seed=33)
        want = fl.attention_decode_window(q, *c.args(), **c.scales())
        check_decode(q, c, want)
        for s in (c.ks, c.vs):
            s[s == 0] = -0.0
        assert torch.equal(fl.attention_decode_window(q, *c.args(), **c.scales()), want)


# ---------------------------------------------------------------- pages of many tokens
@pytest.mark.parametrize("last", [1, 6])
def test_a_page_whose_bytes_pass_32_bits(last):
    """One page of 2^25 tokens and some more: rows behind 2^31 bytes of codes come back, are attended to, and nothing else is written."""
    page, n = (1 << 25) + 64, 9
    k, v = (torch.zeros(1, 1, page, D // 2, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(1, 1, page, 4, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.zeros(1, 1, dtype=torch.int32, device="cuda")
    seq_lens = torch.tensor([page - last], dtype=torch.int32, device="cuda")
    y, z = randn(n, D, seed=41), randn(n, D, seed=42)
    fl.paged_kv_append_int4(y, z, k, v, ks, vs, table, seq_lens, cu_seqlens=cu([n]))
    scales = dict(k_page_scale=ks, v_page_scale=vs)
    back = fl.paged_kv_read(k, v, table, seq_lens, cu_seqlens=cu([n]), rows=n, **scales)
    end = page - last
    for out, x, codes, s in zip(back, (y, z), (k, v), (ks, vs)):
        want, ws = quantise_int4(x)
        assert torch.equal(out.double(), values_int4(want, ws))
        assert torch.equal(codes[0, 0, end - n:end], want) and torch.equal(s[0, 0, end - n:end], ws)
        assert not codes[0, 0, :end - n].any() and not codes[0, 0, end:].any() and not s[0, 0, :end - n].any()
    q = randn(1, 2 * D, seed=43)
    out = fl.attention_decode_window(q, k, v, table, seq_lens, window=n, **scales)
    ref, tol = attend_window(q.double().view(2, 1, D), *(t.double()[None] for t in back), D ** -0.5, 0, 0, STEP["int4"],
                             scales=[s[0, 0, end - n:end].double().repeat_interleave(32, -1)[None] for s in (ks, vs)])
    assert_within(out.view(2, 1, D), ref, tol, "decode")


# ---------------------------------------------------------------- lengths up to 2^31
@pytest.mark.parametrize("kind", KINDS)
def test_lengths_next_to_the_end_of_32_bits(kind):
    """A table with room for 2^31 tokens (its entries are all one page): up to 2^31 - 1024 of them a sequence is served, longer
    ones are refused like those that pass the table."""
    page, window, sinks, longest = 1 << 20, 100, 5, (1 << 31) - 1024
    lens = [longest, (1 << 31) - 1, 300, longest + 1]
    small = AnyCache([window + sinks, 300], 2, 400, kind, seed=51)  # the tokens that are seen, of sequence 0 and of sequence 2

    def paged(x):
        if x is None:
            return None
        big = torch.zeros((1, x.shape[1], page) + x.shape[3:], dtype=x.dtype, device="cuda")
        first, second = (x[small.table[b, 0].long()] for b in (0, 1))
        big[0, :, :300] = second[:, :300]
        end = longest % page
        big[0, :, end - window:end] = first[:, sinks:sinks + window]
        return big

    k, v, ks, vs = (paged(x) for x in (small.k, small.v, small.ks, small.vs))
    for x, y in ((small.k, k), (small.v, v), (small.ks, ks), (small.vs, vs)):
        if x is not None:
            x[small.table[0, 0].long(), :, :sinks] = y[0, :, :sinks]  # the sinks are the other sequence's first tokens
    table = torch.zeros(4, 2048, dtype=torch.int32, device="cuda")
    seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q = randn(4, 8 * D, seed=52)
    ws = fl.attention_decode_workspace()
    scales = dict(k_page_scale=ks, v_page_scale=vs)
    out = fl.attention_decode_window(q, k, v, table, seq_lens, window=window, sinks=sinks, workspace=ws, **scales)
    assert fl.check_device_status(ws) == fl.FL_ERR_INVALID_ARG
    assert torch.isnan(out[[1, 3]]).all()
    check_decode(q[[0, 2]], small, out[[0, 2]], window + sinks, 0, what="sequence 0 with its tokens side by side", skip=(1,))
    check_decode(q[[0, 2]], small, out[[0, 2]], window, sinks, skip=(0,))
    if kind != "int4":
        out = fl.attention_decode(q[1:3], k, v, table[1:3], seq_lens[1:3], workspace=ws, **scales)
    else:
        out = fl.attention_decode_window(q[1:3], k, v, table[1:3], seq_lens[1:3], workspace=ws, **scales)
    assert fl.check_device_status(ws) == fl.FL_ERR_INVALID_ARG
    assert torch.isnan(out[0]).all()
    check_decode(q[1:3], small, out, skip=(0,))
