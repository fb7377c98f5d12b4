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


# ---------------------------------------------------------------- few queries behind many keys, cut along these
LONG = [([33], [5000]), ([1], [1700]), ([70, 1, 0, 64], [3000, 1, 900, 2500]), ([5, 300], [4000, 200]), ([200], [130 * 128])]


def space_of(q, k, lens, window, sinks):
    return fl.load().fl_attention_prefill_window_scratch_bytes(q.shape[0], k.shape[0], len(lens), q.shape[1] // D, k.shape[1] // D,
                                                               window, sinks)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window,sinks", [(0, 0), (2100, 100), (1000, 0)])
@pytest.mark.parametrize("heads,kv", [(8, 2), (4, 4), (48, 1)])
@pytest.mark.parametrize("lens,lens_k", LONG, ids=lambda x: "-".join(map(str, x)))
def test_prefill_parts_match_the_definition(lens, lens_k, heads, kv, window, sinks, fp8):
    """Also queries in front of the first key (5 of 300 behind 200), a sequence without rows, a key tile that ends inside."""
    q = rows_of(sum(lens) + 3, heads, seed=121)
    k, v, ks, vs = keys_of(sum(lens_k) + 5, kv, fp8, seed=122)
    assert space_of(q, k, lens, window, sinks) > 0 or heads == 48 or 0 < window < 2000 or sum(lens) > 300
    out = torch.full_like(q, 7.0)
    call = dict(cu_seqlens=cu(lens), cu_seqlens_k=cu(lens_k), window=window, sinks=sinks, k_scale=ks, v_scale=vs)
    ws = fl.attention_prefill_workspace(k.shape[0], kv, fp8)
    for _ in range(2):
        fl.attention_prefill_window(q, k, v, O=out, workspace=ws, **call)
        check_prefill(q, k, v, ks, vs, lens, out, window, sinks, lens_k)
        assert (out[sum(lens):] == 7.0).all()
    assert torch.equal(fl.attention_prefill_window(q, k, v, **call)[:sum(lens)], out[:sum(lens)])


def test_prefill_parts_are_used():
    """What the cases above count on; one window as long as a few tiles, and many units, stay whole."""
    def space(m, m_k, batch, heads, kv, window=0, sinks=0):
        return fl.load().fl_attention_prefill_window_scratch_bytes(m, m_k, batch, heads, kv, window, sinks)
    assert space(33, 5000, 1, 8, 2) > 0 and space(1, 2000, 1, 8, 2) > 0 and space(512, 5000, 1, 4, 4, 3000, 10) > 0
    assert space(33, 5000, 1, 8, 2, 500, 4) == 0 and space(4096, 8000, 2, 32, 8) == 0 and space(33, 1500, 1, 8, 2) == 0
    assert space(0, 10, 1, 8, 2) == 0 and space(10, 0, 1, 8, 2) == 0 and space(10, 10, 0, 8, 2) == 0 and space(9, 9, 1, 8, 3) == 0


@pytest.mark.parametrize("scale", [2.0 ** 30, 2.0 ** -30])
def test_prefill_parts_of_very_different_scales(scale):
    """E4M3: a part whose values are far larger or smaller than the others', and one of zeros."""
    q = rows_of(40, 8, seed=123)
    k, v, ks, vs = keys_of(5000, 2, True, seed=124)
    vs[1000:2000] *= scale
    vs[2500:3700] = 0
    out = fl.attention_prefill_window(q, k, v, cu_seqlens=cu([40]), cu_seqlens_k=cu([5000]), k_scale=ks, v_scale=vs)
    check_prefill(q, k, v, ks, vs, [40], out, lens_k=[5000])


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_prefill_parts_values_that_are_not_finite(bad, fp8):
    """In a value that all rows see, in one that the last rows see, and behind them all."""
    q = rows_of(60, 8, seed=125)
    k, v, ks, vs = keys_of(5000, 2, fp8, seed=126)
    call = dict(cu_seqlens=cu([60]), cu_seqlens_k=cu([4960]))
    want = fl.attention_prefill_window(q, k, v, k_scale=ks, v_scale=vs, **call)
    for at, seen in ((1234, 0), (4950, 50), (4965, 60)):  # key 4900 + r is row r's own
        if fp8:
            scales = vs.clone()
            scales[at, 1] = bad
            got = fl.attention_prefill_window(q, k, v, k_scale=ks, v_scale=scales, **call)
        else:
            values = v.clone()
            values[at, D + 5] = bad
            got = fl.attention_prefill_window(q, k, values, **call)
        first = got.view(60, 8, D)[:, :4]
        assert torch.equal(first, want.view(60, 8, D)[:, :4])  # the other kv head's
        mine = got.view(60, 8, D)[:, 4:]
        assert torch.isfinite(mine[:seen]).all()
        assert seen == 60 or (~torch.isfinite(mine[seen:, :, 5])).all()
        if not fp8 and seen < 60:
            assert torch.isfinite(mine[seen:, :, :5]).all() and torch.isfinite(mine[seen:, :, 6:]).all()
            assert torch.isnan(mine[seen:, :, 5]).all() if bad != bad else (mine[seen:, :, 5] == bad).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_parts_captured_and_replayed_with_other_offsets(fp8):
    q = rows_of(100, 8, seed=127)
    k, v, ks, vs = keys_of(6000, 2, fp8, seed=128)
    offsets, offsets_k = cu([40, 60]), cu([3000, 3000])
    out = torch.empty_like(q)
    ws = fl.attention_prefill_workspace(6000, 2, fp8)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fl.attention_prefill_window(q, k, v, cu_seqlens=offsets, cu_seqlens_k=offsets_k, k_scale=ks, v_scale=vs, O=out, workspace=ws)
    for lens, lens_k in (([40, 60], [3000, 3000]), ([1, 99], [5800, 200]), ([100, 0], [100, 5000]), ([64, 36], [10, 5990])):
        offsets.copy_(cu(lens)), offsets_k.copy_(cu(lens_k))
        out.fill_(3)
        g.replay()
        check_prefill(q, k, v, ks, vs, lens, out, lens_k=lens_k)


def test_prefill_parts_bad_offsets_stay_inside():
    """Offsets that give the same rows to many sequences make more units than there is room for: they stay whole, and nothing
    behind the scratch buffer or outside the rows is written."""
    heads, kv, m, m_k, batch = 8, 2, 60, 5000, 9
    q = rows_of(m, heads, seed=133)
    k, v, _, _ = keys_of(m_k, kv, False, seed=134)
    ws = fl.attention_prefill_workspace(m_k, kv, False)
    size = fl.load().fl_attention_prefill_window_scratch_bytes(m, m_k, batch, heads, kv, 0, 0)
    assert size > 0
    scratch = torch.full((size + 65536,), 0x5A, dtype=torch.uint8, device="cuda")
    out = torch.full((m + 8, heads * D), 7.0, dtype=torch.bfloat16, device="cuda")
    for rows in ([0, 60] * 5, [0, 60, 0, 60, -5, 70, 3, 1 << 30, 0, 60], [0, 1, 2, 3, 4, 5, 6, 7, 8, 60]):
        for keys in ([0, 5000] * 5, [0, 5000, -9, 5000, 0, 1 << 30, 7, 5000, 0, 4000]):
            offsets, offsets_k = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (rows, keys))
            st = fl.load().attention_prefill_window(
                q.data_ptr(), k.data_ptr(), v.data_ptr(), None, None, offsets.data_ptr(), offsets_k.data_ptr(), out.data_ptr(), m,
                m_k, batch, heads, kv, D, 1, heads * D, kv * D, 0, heads * D, D ** -0.5, 0, 0, fl.FL_BF16, ws.data_ptr(),
                ws.numel(), scratch.data_ptr(), size, torch.cuda.current_stream().cuda_stream)
            assert st == fl.FL_OK
            torch.cuda.synchronize()
            assert (scratch[size:] == 0x5A).all() and (out[m:] == 7.0).all()
    # the workspace serves on, with the scratch buffer as it is
    offsets, offsets_k = cu([60]), cu([5000])
    want = fl.attention_prefill_window(q, k, v, cu_seqlens=offsets, cu_seqlens_k=offsets_k)
    assert torch.equal(fl.attention_prefill_window(q, k, v, cu_seqlens=offsets, cu_seqlens_k=offsets_k, workspace=ws), want)


def test_prefill_parts_of_two_calls_at_once():
    q = rows_of(60, 8, seed=131)
    k, v, _, _ = keys_of(5000, 2, False, seed=132)
    calls = [dict(cu_seqlens=cu([60]), cu_seqlens_k=cu([n])) for n in (5000, 3000)]
    wants = [fl.attention_prefill_window(q, k, v, **c) for c in calls]
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, c in enumerate(calls):
            got[i].append(fl.attention_prefill_window(q, k, v, stream=streams[i], **c))
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for outs, w in zip(got, wants) for o in outs)


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
