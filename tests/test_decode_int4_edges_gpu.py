"""Decode over a 4-bit cache where its kernel's own arithmetic and its ring have their edges: waits that run out, scales at both
ends of their range, long flat attention, pages of many tokens, lengths that no count holds."""
import pytest
import torch

import gemm_epilogue_tcgen05_gb300 as fl
from attention_utils import D
from test_attention_window_gpu import check_decode, randn
from window_utils import AnyCache

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
