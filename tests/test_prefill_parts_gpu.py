"""Which calls of attention_prefill_window are cut along their keys, and which rows of a cache a prompt's next part needs."""
import pytest
import torch

import gemm_epilogue_tcgen05_gb300 as fl
from attention_utils import cu
from test_attention_window_gpu import check_prefill, keys_of, rows_of
from window_utils import AnyCache

pytestmark = pytest.mark.gpu


def space(m, m_k, batch, heads, kv, window=0, sinks=0):
    return fl.load().fl_attention_prefill_window_scratch_bytes(m, m_k, batch, heads, kv, window, sinks)


def test_batches_of_short_sequences_stay_whole():
    """However many keys they have together; one of the same rows alone, or among others that leave it long, is cut."""
    assert space(80, 2000, 4, 32, 8) == 0 and space(32, 2000, 8, 16, 4) == 0 and space(320, 8000, 16, 16, 2) == 0
    assert space(80, 2000, 1, 32, 8) > 0 and space(80, 3180, 4, 32, 8) > 0 and space(320, 9750, 16, 16, 2) > 0
    assert space(80, 2499, 4, 32, 8) == 0 and space(80, 2500, 4, 32, 8) > 0


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens_k", [[500] * 4, [900, 0, 1, 1598], [2440, 20, 20, 20], [2200, 150, 149, 0]])
def test_batches_on_both_sides_of_the_rule(lens_k, fp8):
    lens = [20, 7, 0, 20]
    q = rows_of(sum(lens) + 3, 8, seed=1)
    k, v, ks, vs = keys_of(sum(lens_k), 2, fp8, seed=2)
    out = fl.attention_prefill_window(q, k, v, cu_seqlens=cu(lens), cu_seqlens_k=cu(lens_k), k_scale=ks, v_scale=vs)
    check_prefill(q, k, v, ks, vs, lens, out, lens_k=lens_k)
    assert (out[sum(lens):] == 0).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_parts_serve_on_after_waits_that_ran_out(fp8):
    """With a limit of a microsecond the waits for the first unit give up while its sequence is looked for among 2000, which takes
    some ten microseconds and more: the call ends, the status record says so, and workspace and scratch buffer serve on."""
    batch, n, rows = 2000, 5000, 1001000
    q = rows_of(33, 4, seed=3)
    k, v, ks, vs = keys_of(n, 1, fp8, seed=4)
    wide = [torch.zeros((rows,) + x.shape[1:], dtype=x.dtype, device="cuda") if x is not None else None for x in (k, v, ks, vs)]
    for x, y in zip(wide, (k, v, ks, vs)):
        if x is not None:
            x[:n] = y
    offsets, offsets_k = (torch.zeros(batch + 1, dtype=torch.int32, device="cuda") for _ in range(2))
    offsets[batch], offsets_k[batch] = 33, n  # the last sequence's; the keys behind it are nobody's
    assert space(33, rows, batch, 4, 1) > 0
    ws = fl.attention_prefill_workspace(rows, 1, fp8)

    def call():
        out = torch.full_like(q, 7.0)
        fl.attention_prefill_window(q, wide[0], wide[1], cu_seqlens=offsets, cu_seqlens_k=offsets_k, k_scale=wide[2],
                                    v_scale=wide[3], O=out, workspace=ws)
        return out

    want = call()
    check_prefill(q, k, v, ks, vs, [33], want, lens_k=[n])
    assert fl.check_device_status(ws) == fl.FL_OK
    for _ in range(2):
        try:
            fl.set_wait_timeout_ns(1000)
            call()
            status = fl.check_device_status(ws)
        finally:
            fl.set_wait_timeout_ns(0)
        assert status == fl.FL_ERR_TIMEOUT
        for _ in range(2):
            assert torch.equal(call(), want)
        assert fl.check_device_status(ws) == fl.FL_OK


@pytest.mark.parametrize("kind", ["bf16", "int4"])
@pytest.mark.parametrize("sinks", [0, 4, 70])
def test_rows_of_sinks_and_window_alone(kind, sinks):
    """A prompt's next part needs the first `sinks` tokens and those from window - 1 in front of its own on: read as two sequences
    one behind the other, they give what all rows give."""
    lens, lens_k, window, kv = [33, 1, 80], [2000, 700, 1500], 200, 2
    c = AnyCache(lens_k, kv, 16, kind, seed=5)
    q = rows_of(sum(lens), 8, seed=6)
    keep = [window - 1 + n for n in lens]
    table = c.table.repeat_interleave(2, 0)
    seq_lens = torch.tensor([x for n in lens_k for x in (sinks, n)], dtype=torch.int32, device="cuda")
    total = sum(keep) + sinks * len(lens)
    k, v = fl.paged_kv_read(c.k, c.v, table, seq_lens, cu_seqlens=cu([x for n in keep for x in (sinks, n)]), rows=total, **c.scales())
    out = fl.attention_prefill_window(q, k, v, cu_seqlens=cu(lens), cu_seqlens_k=cu([sinks + n for n in keep]), window=window,
                                      sinks=sinks)
    k, v = fl.paged_kv_read(*c.args(), cu_seqlens=cu(lens_k), rows=sum(lens_k), **c.scales())
    check_prefill(q, k, v, None, None, lens, out, window, sinks, lens_k)
