"""Calls of the 4-bit cache and of attention with a window that their documentation allows and that lie at its edges: offsets
beyond 32 bits, outputs in the place of the queries, a capture as the first call, two graphs with one workspace, waits that ran
out, pages that sequences share, spans longer than anything."""
import os
import subprocess
import sys

import pytest
import torch

import gemm_epilogue_tcgen05_gb300 as fl
from attention_utils import D, cu
from test_attention_window_gpu import KINDS, check_decode, check_prefill, keys_of, randn, rows_of
from window_utils import AnyCache

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


# ---------------------------------------------------------------- decode
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads", [8, 24])
def test_output_in_the_place_of_the_queries(kind, heads):
    """24 heads of 2: the heads of a kv head in two parts over 4 bits, one after the other in the same rows."""
    c = AnyCache([3000, 70, 0, 900, 130], 2, 16, kind, seed=101)
    q = randn(5, heads * D, seed=102)
    for window, sinks in ((0, 0), (200, 8)):
        want = fl.attention_decode_window(q, *c.args(), window=window, sinks=sinks, **c.scales())
        place = q.clone()
        out = fl.attention_decode_window(place, *c.args(), window=window, sinks=sinks, O=place, **c.scales())
        assert out is place and torch.equal(place, want)


@pytest.mark.parametrize("batch", [56, 57, 58, 61, 64, 115])
def test_decode_runs_that_end_with_the_beginning_of_a_sequence(batch):
    """8 heads of about as many (sequence, head) pairs as there are CTAs, of one to three units: some shares hold no more of
    their last one than what its beginning counts as, some begin behind it."""
    lens = [1 + (37 * b) % 128 + 128 * (b % 3) for b in range(batch)]
    c = AnyCache(lens, 8, 16, "int4", seed=103)
    q = randn(batch, 8 * D, seed=104)
    ws = fl.attention_decode_workspace()
    for window, sinks in ((0, 0), (100, 3)):
        for _ in range(2):
            out = torch.full_like(q, 7.0)
            fl.attention_decode_window(q, *c.args(), window=window, sinks=sinks, O=out, workspace=ws, **c.scales())
            check_decode(q, c, out, window, sinks)
    assert fl.check_device_status(ws) == fl.FL_OK


@pytest.mark.parametrize("kind", KINDS)
def test_sequences_that_share_pages(kind):
    """The same prefix in several sequences, the same page twice in one."""
    c = AnyCache([130, 130, 100, 64], 2, 16, kind, seed=105)
    c.table[1, :5] = c.table[0, :5]
    c.table[2, 3] = c.table[2, 0]
    q = randn(4, 8 * D, seed=106)
    for window, sinks in ((0, 0), (50, 20)):
        out = fl.attention_decode_window(q, *c.args(), window=window, sinks=sinks, **c.scales())
        check_decode(q, c, out, window, sinks)
    k, v = fl.paged_kv_read(*c.args(), cu_seqlens=cu(c.lens), rows=sum(c.lens), **c.scales())
    first = 0
    for b, n in enumerate(c.lens):
        for got, want in zip((k, v), c.sequence(b)):
            assert torch.equal(got[first:first + n].view(n, 2, D).transpose(0, 1), want.to(torch.bfloat16))
        first += n


@pytest.mark.parametrize("kind", KINDS)
def test_spans_longer_than_anything(kind):
    c = AnyCache([300, 1, 70], 2, 16, kind, seed=107)
    q = randn(3, 8 * D, seed=108)
    want = fl.attention_decode_window(q, *c.args(), **c.scales())
    for window, sinks in ((1 << 40, 0), ((1 << 31) - 1, (1 << 31) - 1), (1, 1 << 40), (0, 1 << 40)):
        got = fl.attention_decode_window(q, *c.args(), window=window, sinks=sinks, **c.scales())
        assert torch.equal(got, want)
    p = rows_of(371, 8, seed=109)
    k, v, ks, vs = keys_of(371, 2, kind == "fp8", seed=110)
    call = dict(cu_seqlens=cu([300, 1, 70]), k_scale=ks, v_scale=vs)
    want = fl.attention_prefill_window(p, k, v, **call)
    for window, sinks in ((1 << 40, 0), ((1 << 31) - 1, (1 << 31) - 1), (0, 1 << 40)):
        assert torch.equal(fl.attention_prefill_window(p, k, v, window=window, sinks=sinks, **call), want)
    out = fl.attention_prefill_window(p, k, v, window=1, sinks=1 << 40, **call)  # everything by the sinks alone
    check_prefill(p, k, v, ks, vs, [300, 1, 70], out, 1, 1 << 40)


def test_two_graphs_with_one_workspace():
    """Replayed one after the other in any order: each leaves the workspace as it found it."""
    c = AnyCache([3000, 900, 40], 2, 16, "int4", seed=111)
    q, ws = randn(3, 8 * D, seed=112), fl.attention_decode_workspace()
    p = rows_of(900, 8, seed=113)
    k, v, ks, vs = keys_of(900, 2, True, seed=114)
    wp = fl.attention_prefill_workspace(900, 2, True)
    graphs, outs, wants = [], [], []
    for window in (0, 250):
        call = dict(window=window, sinks=4)
        wants.append((fl.attention_decode_window(q, *c.args(), **call, **c.scales()),
                      fl.attention_prefill_window(p, k, v, k_scale=ks, v_scale=vs, **call)))
        outs.append((torch.empty_like(q), torch.empty_like(p)))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fl.attention_decode_window(q, *c.args(), **call, **c.scales(), O=outs[-1][0], workspace=ws)
            fl.attention_prefill_window(p, k, v, k_scale=ks, v_scale=vs, **call, O=outs[-1][1], workspace=wp)
        graphs.append(g)
    for i in (0, 1, 1, 0, 1, 0, 0):
        for o in outs[i]:
            o.fill_(7)
        graphs[i].replay()
        assert all(torch.equal(o, w) for o, w in zip(outs[i], wants[i]))


# ---------------------------------------------------------------- prefill
@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_window_beyond_32_bits(fp8):
    """Rows of Q, K, V, O and the workspace behind their 2^31st element and 2^32nd byte: the last sequences count."""
    kv, tail, n = 64, [130, 300, 200], 100
    rows = (1 << 31) // (kv * D) // n * n + 2 * n
    total = rows + sum(tail)
    q = torch.zeros(total, kv * D, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros(total, kv * D, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda") for _ in range(2))
    ks = vs = None
    q_tail = rows_of(sum(tail), kv, seed=115)
    k_tail, v_tail, ks_tail, vs_tail = keys_of(sum(tail), kv, fp8, seed=116)
    q[rows:], k[rows:], v[rows:] = q_tail, k_tail, v_tail
    if fp8:
        ks, vs = torch.zeros(total, kv, device="cuda"), torch.zeros(total, kv, device="cuda")
        ks[rows:], vs[rows:] = ks_tail, vs_tail
    out = torch.empty_like(q)
    fl.attention_prefill_window(q, k, v, cu_seqlens=cu([n] * (rows // n) + tail), k_scale=ks, v_scale=vs, window=90, sinks=3, O=out)
    check_prefill(q_tail, k_tail, v_tail, ks_tail, vs_tail, tail, out[rows:], 90, 3)
    assert (out[:rows] == 0).all()


@pytest.mark.parametrize("window,sinks", [(150, 40), (300, 0), (40, 130), (129, 1)])
def test_prefill_window_tiles_of_very_different_scales(window, sinks):
    """E4M3: the scales of V change by up to 2^40 from one 128 keys to the next, and a unit's key tiles hold parts of two or
    three such stretches."""
    lens, lens_k = [700, 90, 333], [700, 1300, 400]
    q = rows_of(sum(lens), 8, seed=117)
    k, v, ks, vs = keys_of(sum(lens_k), 2, True, seed=118)
    first = 0
    for b, n in enumerate(lens_k):
        for i, j in enumerate(range(0, n, 128)):
            vs[first + j:first + min(j + 128, n)] *= 2.0 ** (-20, 0, 20)[(i + b) % 3]
        first += n
    out = fl.attention_prefill_window(q, k, v, cu_seqlens=cu(lens), cu_seqlens_k=cu(lens_k), window=window, sinks=sinks,
                                      k_scale=ks, v_scale=vs)
    check_prefill(q, k, v, ks, vs, lens, out, window, sinks, lens_k)


@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_window_serves_on_after_waits_that_ran_out(fp8):
    """With a limit of a microsecond the waits for units of tens of microseconds give up: the call ends, the status record says
    so, and the workspace serves on though nobody zeroes it."""
    n, m = 65536, 24000
    q = rows_of(n, 2, seed=119)
    k, v, ks, vs = keys_of(n, 2, fp8, seed=120)
    ws = fl.attention_prefill_workspace(n, 2, fp8)
    cut = (q[:m], k[:m], v[:m])
    scales = dict(k_scale=ks[:m], v_scale=vs[:m]) if fp8 else {}
    want = fl.attention_prefill_window(*cut, **scales, window=5000, sinks=70)
    for times in (1, 2):
        try:
            fl.set_wait_timeout_ns(1000)
            for _ in range(times):
                fl.attention_prefill_window(q, k, v, k_scale=ks, v_scale=vs, window=20000, sinks=70, workspace=ws)
            status = fl.check_device_status(ws)
        finally:
            fl.set_wait_timeout_ns(0)
        assert status == fl.FL_ERR_TIMEOUT
        for _ in range(2):
            out = torch.full((m, 2 * D), 7.0, dtype=torch.bfloat16, device="cuda")
            fl.attention_prefill_window(*cut, **scales, window=5000, sinks=70, O=out, workspace=ws)
            assert torch.equal(out, want)
        assert fl.check_device_status(ws) == fl.FL_OK


# ---------------------------------------------------------------- the first calls of a process
FIRST = """
import sys
sys.path[:0] = {paths}
import torch
import gemm_epilogue_tcgen05_gb300 as fl
from test_attention_window_gpu import D, check_decode, check_prefill, keys_of, randn, rows_of
from window_utils import AnyCache
c = AnyCache([100, 700], 2, 16, "int4", seed=1)
q, (k, v, _, _) = rows_of(300, 8), keys_of(300, 2, False)
rows = torch.empty(2, 2, 2 * D, dtype=torch.bfloat16, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    fl.paged_kv_append_int4(k[:2], v[:2], c.k, c.v, c.ks, c.vs, c.table, c.seq_lens)
    one = fl.attention_decode_window(q[:2], *c.args(), window=90, sinks=2, **c.scales())
    fl.paged_kv_read(*c.args(), K=rows[0], V=rows[1], **c.scales())
    whole = fl.attention_prefill_window(q, k, v, window=90, sinks=2)
for _ in range(3):
    one.fill_(3), whole.fill_(3), rows.fill_(3)
    g.replay()
    check_decode(q[:2], c, one, 90, 2)
    check_prefill(q, k, v, None, None, [300], whole, 90, 2)
    for b, n in enumerate(c.lens):
        assert all(torch.equal(rows[i, b].view(2, D), x[:, n - 1].bfloat16()) for i, x in enumerate(c.sequence(b)))
print("captured first")
"""


def test_first_calls_of_a_process_are_captured():
    """Nothing is left to a call outside the capture, and workspaces made inside it are the graph's."""
    code = FIRST.format(paths=[os.path.dirname(HERE), HERE])
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stdout + r.stderr
