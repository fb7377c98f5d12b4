"""Calls of the attention operators that their documentation allows and that lie at its edges: offsets beyond 32 bits,
outputs in the place of the queries, caches without pages, a capture as the first call, a stream of one's own."""
import os
import subprocess
import sys

import pytest
import torch

import gemm_epilogue_tcgen05_gb300 as fl
from attention_utils import D, Cache, check_decode, check_prefill, cu, quantise

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def randn(*shape, seed=0):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()


def prompt(rows, heads, kv, fp8, seed=0):
    q, k, v = randn(rows, heads * D, seed=seed), randn(rows, kv, D, seed=seed + 1), randn(rows, kv, D, seed=seed + 2)
    ks = vs = None
    if fp8:
        (k, ks), (v, vs) = quantise(k), quantise(v)
    return q, k.view(rows, -1), v.view(rows, -1), ks, vs


# ---------------------------------------------------------------- offsets beyond 32 bits
@pytest.mark.parametrize("fp8", [False, True])
def test_cache_beyond_32_bits(fp8):
    """Pages whose elements lie behind the 2^32nd of their array (and scales whose bytes do), written and read."""
    kv, page, lens = 8, 64, [150, 64, 1, 700]
    small = Cache(lens, kv, page, fp8, seed=90)
    pages = (1 << 32) // (kv * page * D) + 40
    big = [torch.empty((pages,) + t.shape[1:], dtype=t.dtype, device="cuda") for t in (small.k, small.v)]
    first = pages - small.pages
    for t, from_ in zip(big, (small.k, small.v)):
        t[first:] = from_
    if fp8:  # scales with a pitch that takes them behind 2^32 bytes, too
        pitch = (1 << 32) // (4 * first) + 1
        room = [torch.empty(pages * pitch, device="cuda").as_strided((pages, kv, page), (pitch, page, 1)) for _ in range(2)]
        for t, from_ in zip(room, (small.ks, small.vs)):
            t[first:] = from_
        small.ks, small.vs = room
    small.k, small.v = big
    small.table += first
    q = randn(len(lens), 32 * D, seed=91)
    check_decode(q, small, fl.attention_decode(q, *small.args(), **small.scales()))
    _, k, v, ks, vs = prompt(sum(lens), 8, kv, fp8, seed=92)
    fl.paged_kv_append(k, v, *small.args(), cu_seqlens=cu(lens), k_scale=ks, v_scale=vs, **small.scales())
    at = 0
    for b, n in enumerate(lens):
        pos = torch.arange(n, device="cuda")
        page_of, slot = small.table[b].long()[pos // page], pos % page
        assert torch.equal(small.k[page_of, :, slot], k[at:at + n].view(n, kv, D))
        assert torch.equal(small.v[page_of, :, slot], v[at:at + n].view(n, kv, D))
        if fp8:
            assert torch.equal(small.vs[page_of, :, slot], vs[at:at + n])
        at += n
    check_decode(q, small, fl.attention_decode(q, *small.args(), **small.scales()))


@pytest.mark.parametrize("fp8", [False, True])
def test_prompts_beyond_32_bits(fp8):
    """Rows of Q, K, V, O and the workspace behind their 2^31st element and 2^32nd byte: the last sequences count."""
    kv, tail, n = 64, [130, 77, 200], 100
    rows = (1 << 31) // (kv * D) // n * n + 2 * n
    total = rows + sum(tail)
    q = torch.zeros(total, kv * D, dtype=torch.bfloat16, device="cuda")
    k, v = (torch.zeros(total, kv * D, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda") for _ in range(2))
    ks = vs = None
    last = prompt(sum(tail), kv, kv, fp8, seed=93)
    q[rows:], k[rows:], v[rows:] = last[:3]
    if fp8:
        ks, vs = torch.zeros(total, kv, device="cuda"), torch.zeros(total, kv, device="cuda")
        ks[rows:], vs[rows:] = last[3:]
        vs[rows + 5] *= 2.0 ** 30  # a key on its own, with its codes and scale read back there
        last[4][5] *= 2.0 ** 30
    out = torch.empty_like(q)
    offsets = cu([n] * (rows // n) + tail)
    fl.attention_prefill(q, k, v, cu_seqlens=offsets, k_scale=ks, v_scale=vs, O=out)
    check_prefill(*last, tail, out[rows:], True)
    assert (out[:rows] == 0).all()


# ---------------------------------------------------------------- O in the place of Q
@pytest.mark.parametrize("fp8", [False, True])
def test_output_in_the_place_of_the_queries(fp8):
    c = Cache([3000, 70, 0, 900], 2, 16, fp8, seed=94)
    q = randn(4, 24 * D, seed=94)
    want = fl.attention_decode(q, *c.args(), **c.scales())
    place = q.clone()
    assert torch.equal(fl.attention_decode(place, *c.args(), **c.scales(), O=place), want)
    lens = [700, 1, 333, 64, 2000, 90]
    q, k, v, ks, vs = prompt(sum(lens), 12, 4, fp8, seed=95)
    for causal in (True, False):
        call = dict(cu_seqlens=cu(lens), k_scale=ks, v_scale=vs, causal=causal)
        want = fl.attention_prefill(q, k, v, **call)
        place = q.clone()
        assert torch.equal(fl.attention_prefill(place, k, v, O=place, **call), want)


# ---------------------------------------------------------------- nothing there
@pytest.mark.parametrize("fp8", [False, True])
def test_nothing_to_attend_to(fp8):
    """No pages, no table columns, no sequences, no rows, no heads."""
    kind = torch.uint8 if fp8 else torch.bfloat16
    none = [torch.empty(0, 2, 16, D, dtype=kind, device="cuda") for _ in range(2)]
    scales = {}
    if fp8:
        scales = {n: torch.empty(0, 2, 16, device="cuda") for n in ("k_page_scale", "v_page_scale")}
    lens = torch.zeros(3, dtype=torch.int32, device="cuda")
    for width in (0, 4):
        table = torch.zeros(3, width, dtype=torch.int32, device="cuda")
        out = torch.full((3, 8 * D), 5.0, dtype=torch.bfloat16, device="cuda")
        fl.attention_decode(randn(3, 8 * D), *none, table, lens, O=out, **scales)
        assert (out == 0).all()
    empty = torch.empty(0, 8 * D, dtype=torch.bfloat16, device="cuda")
    assert fl.attention_decode(empty, *none, torch.empty(0, 4, dtype=torch.int32, device="cuda"), lens[:0],
                               **scales).shape == (0, 8 * D)
    rows, rs = torch.empty(0, 2 * D, dtype=kind, device="cuda"), torch.empty(0, 2, device="cuda") if fp8 else None
    assert fl.attention_prefill(empty, rows, rows, k_scale=rs, v_scale=rs).shape == (0, 8 * D)
    assert fl.attention_prefill(empty, rows, rows, cu_seqlens=lens, k_scale=rs, v_scale=rs).shape == (0, 8 * D)
    fl.paged_kv_append(rows, rows, *none, torch.zeros(3, 4, dtype=torch.int32, device="cuda"), lens, cu_seqlens=cu([0, 0, 0]),
                       k_scale=rs, v_scale=rs, **scales)
    q, k, v, ks, vs = prompt(9, 4, 2, fp8, seed=96)
    out = torch.full_like(q, 5.0)
    fl.attention_prefill(q, k, v, cu_seqlens=cu([0, 0]), k_scale=ks, v_scale=vs, O=out)
    assert (out == 5.0).all() and fl.device_status() == fl.FL_OK


# ---------------------------------------------------------------- graphs and streams
FIRST = """
import sys
sys.path[:0] = {paths!r}
import torch
import gemm_epilogue_tcgen05_gb300 as fl
from attention_utils import Cache, check_decode, check_prefill
from test_attention_use_gpu import D, prompt
fp8 = {fp8}
c = Cache([100, 700], 2, 16, fp8, seed=1)
q, k, v, ks, vs = prompt(300, 8, 2, fp8)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    fl.paged_kv_append(k[:2], v[:2], *c.args(), k_scale=ks if ks is None else ks[:2], v_scale=vs if vs is None else vs[:2],
                       **c.scales())
    one = fl.attention_decode(q[:2], *c.args(), **c.scales())
    whole = fl.attention_prefill(q, k, v, k_scale=ks, v_scale=vs)
for _ in range(3):
    one.fill_(3), whole.fill_(3)
    g.replay()
    check_decode(q[:2], c, one)
    check_prefill(q, k, v, ks, vs, [300], whole, True)
    assert torch.equal(c.k[c.table[0, 99 // 16].long(), :, 99 % 16], k[0].view(2, D))
print("captured first")
"""


@pytest.mark.parametrize("fp8", [False, True])
def test_first_calls_of_a_process_are_captured(fp8):
    """Nothing is left to a call outside the capture, and workspaces made inside it are the graph's."""
    code = FIRST.format(paths=[os.path.dirname(HERE), HERE], fp8=fp8)
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stdout + r.stderr


@pytest.mark.parametrize("fp8", [False, True])
def test_append_on_a_given_stream(fp8):
    """The current stream is busy, the given one is not: the rows are there once the given one is done."""
    c = Cache([40, 3], 2, 16, fp8, seed=97)
    _, k, v, ks, vs = prompt(2, 8, 2, fp8, seed=98)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        torch.cuda._sleep(20000000)
        fl.paged_kv_append(k, v, *c.args(), k_scale=ks, v_scale=vs, **c.scales(), stream=other)
        with torch.cuda.stream(other):
            got = [c.v[c.table[b, (n - 1) // 16].long(), :, (n - 1) % 16].clone() for b, n in enumerate(c.lens)]
        other.synchronize()
    for b in range(2):
        assert torch.equal(got[b], v[b].view(2, D))
