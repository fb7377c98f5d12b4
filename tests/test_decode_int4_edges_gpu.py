"""Decode over a 4-bit cache where its kernel's own arithmetic and its ring have their edges: waits that run out, scales at both
ends of their range, long flat attention, pages of many tokens, lengths that no count holds."""
import pytest
import torch

import gemm_epilogue_tcgen05_gb300 as fl
from attention_utils import D, assert_within
from test_attention_window_gpu import STEP, check_decode, randn
from window_utils import AnyCache, attend_window

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
