"""attention_decode_window and attention_prefill_window against their definition in 64 bits (window_utils derives the
tolerances), at the lengths, windows and layouts where they can go wrong."""
import pytest
import torch

import gemm_epilogue_tcgen05_gb300 as fl
from attention_utils import D, F16, assert_within, cu
from window_utils import AnyCache, attend_window

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")
KINDS = ["bf16", "fp8", "int4"]
STEP = {"bf16": F16, "fp8": F16, "int4": 2 * F16}


def randn(*shape, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).bfloat16().cuda()


def check_decode(q, cache, out, window=0, sinks=0, scale=D ** -0.5, what="", skip=()):
    heads = q.shape[1] // D
    for b, n in enumerate(cache.lens):
        if b in skip:
            continue
        got = out[b].view(heads, 1, D)
        if n == 0:
            assert (got == 0).all(), f"{what}: sequence {b} is empty"
            continue
        k, v = cache.sequence(b)
        ref, tol = attend_window(q[b].double().view(heads, 1, D), k, v, scale, window, sinks, STEP[cache.kind],
                                 scales=cache.value_scales(b) if cache.kind == "int4" else None)
        assert_within(got, ref, tol, f"{what} sequence {b} of {n}")


# ---------------------------------------------------------------- decode over 4 bits
@pytest.mark.parametrize("lens,heads,kv,page", [
    ([1], 1, 1, 16), ([2, 1, 3], 4, 4, 1), ([33], 8, 1, 32), ([64, 0, 129], 12, 2, 16), ([500, 31, 32, 127, 128], 32, 8, 64),
    ([257], 16, 1, 128), ([77, 700], 24, 2, 24), ([130], 40, 2, 8), ([90, 5], 33, 1, 16), ([1100], 7, 1, 100),
    ([3000, 1], 14, 2, 64), ([64] * 9, 2, 1, 64), ([1025], 128, 1, 16), ([255], 65, 5, 5)])
def test_decode_over_4_bits_matches_the_definition(lens, heads, kv, page):
    c = AnyCache(lens, kv, page, "int4", seed=sum(lens), fill=NAN)
    q = randn(len(lens), heads * D, seed=1)
    check_decode(q, c, fl.attention_decode_window(q, *c.args(), **c.scales()))


def test_decode_over_4_bits_of_a_large_ragged_batch():
    lens = [(37 * i * i + 11) % 3000 for i in range(90)] + [9000]
    c = AnyCache(lens, 4, 16, "int4", seed=2)
    q = randn(len(lens), 16 * D, seed=3)
    check_decode(q, c, fl.attention_decode_window(q, *c.args(), **c.scales()))


@pytest.mark.parametrize("batch", [1, 31, 33, 128, 129, 300])
def test_decode_batch_sizes(batch):
    lens = [(i * 53 + 7) % 400 for i in range(batch)]
    c = AnyCache(lens, 2, 16, "int4", seed=batch)
    q = randn(batch, 8 * D, seed=4)
    check_decode(q, c, fl.attention_decode_window(q, *c.args(), **c.scales()))
    check_decode(q, c, fl.attention_decode_window(q, *c.args(), window=50, sinks=3, **c.scales()), 50, 3)


@pytest.mark.parametrize("heads,kv", [(8, 2), (24, 2)])
def test_decode_over_4_bits_long_sequence(heads, kv):
    c = AnyCache([40000], kv, 64, "int4", seed=5)
    q = randn(1, heads * D, seed=6, std=2.0)
    check_decode(q, c, fl.attention_decode_window(q, *c.args(), **c.scales()))


def test_decode_over_4_bits_wide_range_of_scales():
    """Groups of one token, tokens and sequences whose values lie powers of two apart, zeros among them."""
    lens = [300, 70, 129]
    c = AnyCache(lens, 2, 16, "int4", seed=7)
    g = torch.Generator().manual_seed(8)
    shift = torch.randint(-40, 41, c.vs.shape, generator=g).cuda()
    c.vs *= torch.exp2(shift.float()).bfloat16()
    c.vs[torch.rand(c.vs.shape, generator=g).cuda() < 0.1] = 0
    c.ks *= torch.exp2(torch.randint(-20, 1, c.ks.shape, generator=g).float().cuda()).bfloat16()
    q = randn(3, 8 * D, seed=9)
    check_decode(q, c, fl.attention_decode_window(q, *c.args(), **c.scales()))


@pytest.mark.parametrize("power", [-118, -60, 60, 110])
def test_decode_over_4_bits_scales_at_the_ends_of_the_range(power):
    c = AnyCache([200, 33], 2, 16, "int4", seed=10)
    c.vs *= torch.tensor(2.0 ** power, device="cuda").bfloat16()
    q = randn(2, 12 * D, seed=11)
    check_decode(q, c, fl.attention_decode_window(q, *c.args(), **c.scales()))
    c = AnyCache([200, 33], 2, 16, "int4", seed=10)  # keys, against queries that make up for it
    c.ks *= torch.tensor(2.0 ** power, device="cuda").bfloat16()
    q = (randn(2, 12 * D, seed=11).float() * 2.0 ** -power).bfloat16()
    check_decode(q, c, fl.attention_decode_window(q, *c.args(), **c.scales()))


def test_decode_over_4_bits_peaked_flat_and_large():
    c = AnyCache([900, 64], 2, 32, "int4", seed=12)
    for std in (1e-4, 1.0, 30.0):
        q = randn(2, 8 * D, seed=13, std=std)
        check_decode(q, c, fl.attention_decode_window(q, *c.args(), **c.scales()), what=f"std {std}")
    q = torch.full((2, 8 * D), 100.0, dtype=torch.bfloat16, device="cuda")  # sums of q far from zero
    check_decode(q, c, fl.attention_decode_window(q, *c.args(), scale=1e-3, **c.scales()), scale=1e-3)
    q = torch.zeros(2, 8 * D, dtype=torch.bfloat16, device="cuda")
    check_decode(q, c, fl.attention_decode_window(q, *c.args(), **c.scales()))


def test_decode_over_4_bits_entries_that_are_not_finite():
    """A value's group reaches its own 32 columns only, a key's the whole of its heads; other heads and sequences neither."""
    c = AnyCache([300, 300, 300], 2, 16, "int4", seed=14)
    page, slot = c.table[0, 5].long(), 3
    c.vs[page, 1, slot, 2] = NAN
    page = c.table[1, 18].long()
    c.ks[page, 0, 11, 1] = NAN
    q = randn(3, 8 * D, seed=15)
    out = fl.attention_decode_window(q, *c.args(), **c.scales())
    o = out.view(3, 8, D)
    bad = torch.zeros(3, 8, D, dtype=torch.bool, device="cuda")
    bad[0, 4:, 64:96] = True
    bad[1, :4] = True
    assert torch.equal(torch.isnan(o), bad)
    fine = c.vs.nan_to_num(0.0), c.ks.nan_to_num(0.0)
    keep = AnyCache([300] * 3, 2, 16, "int4", seed=14)
    keep.vs, keep.ks = fine
    ref = fl.attention_decode_window(q, *keep.args(), **keep.scales()).view(3, 8, D)
    # a scale of zero in the place of the NaN takes one part of one token away: other columns keep their value
    assert torch.equal(o[0, 4:, :64], ref[0, 4:, :64]) and torch.equal(o[0, :4], ref[0, :4]) and torch.equal(o[2], ref[2])
    assert torch.equal(o[1, 4:], ref[1, 4:])


# ---------------------------------------------------------------- decode with a window
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("page", [1, 5, 16, 64, 200])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (17, 4), (64, 0), (128, 16), (100, 130), (300, 1), (1000, 64), (2000, 0)])
def test_decode_window_matches_the_definition(kind, page, window, sinks):
    """Everything that is not seen holds NaN, and pages without a token that is seen are not there."""
    lens = [1, 2, window, window + 1, window + sinks, window + sinks + 1, 0, 700, 1300]
    c = AnyCache(lens, 2, page, kind, seed=window + sinks, fill=NAN)
    for b, n in enumerate(lens):
        hidden = torch.arange(sinks, max(n - window, sinks), device="cuda")
        at, slot = c.table[b].long()[hidden // page], hidden % page
        for t in (c.ks, c.vs) if c.ks is not None else (c.k, c.v):
            t[at, :, slot] = NAN
        if kind == "fp8":
            c.k[at, :, slot], c.v[at, :, slot] = 0x7F, 0x7F
        first = -(-sinks // page)
        pages = torch.arange(first, max(max(n - window, 0) // page, first))
        c.table[b, pages.cuda()] = -5
    q = randn(len(lens), 8 * D, seed=16)
    ws = fl.attention_decode_workspace()
    out = fl.attention_decode_window(q, *c.args(), window=window, sinks=sinks, workspace=ws, **c.scales())
    assert fl.check_device_status(ws) == fl.FL_OK
    heads = 8
    for b, n in enumerate(lens):
        if n == 0:
            assert (out[b] == 0).all()
            continue
        j = torch.arange(n, device="cuda")
        seen = (j >= n - window) | (j < sinks)
        t, c.table[b] = c.table[b].clone(), c.table[b].clamp_min(0)
        k, v = (x[:, seen] for x in c.sequence(b))
        scales = [x[:, seen] for x in c.value_scales(b)] if kind == "int4" else None
        c.table[b] = t
        ref, tol = attend_window(q[b].double().view(heads, 1, D), k, v, D ** -0.5, 0, 0, STEP[kind], scales=scales)
        assert_within(out[b].view(heads, 1, D), ref, tol, f"sequence {b} of {n}")


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads,kv", [(3, 1), (24, 2), (16, 16), (40, 2)])
def test_decode_window_head_layouts(kind, heads, kv):
    lens = [2500, 90, 1, 600]
    c = AnyCache(lens, kv, 16, kind, seed=17)
    q = randn(len(lens), heads * D, seed=18)
    check_decode(q, c, fl.attention_decode_window(q, *c.args(), window=333, sinks=5, **c.scales()), 333, 5)


@pytest.mark.parametrize("kind", KINDS)
def test_decode_window_that_hides_nothing(kind):
    """A window of 0 or as long as the table is the whole sequence, bit for bit what attention_decode gives."""
    c = AnyCache([700, 3, 64, 1000], 2, 16, kind, seed=19)
    q = randn(4, 8 * D, seed=20)
    whole = fl.attention_decode_window(q, *c.args(), **c.scales())
    for window, sinks in ((0, 7), (1 << 40, 0), (c.table.shape[1] * 16, 0), (990, 10), (1000, 1 << 31), (2 ** 31 - 1, 2 ** 31 - 1)):
        assert torch.equal(whole, fl.attention_decode_window(q, *c.args(), window=window, sinks=sinks, **c.scales()))
    if kind != "int4":
        assert torch.equal(whole, fl.attention_decode(q, *c.args(), **c.scales()))
    # all is seen, but the table has room for more: the windowed kernel, the same sums
    wide = AnyCache([700, 3, 64, 1000], 2, 16, kind, seed=19, max_pages=100)
    assert torch.equal(whole, fl.attention_decode_window(q, *wide.args(), window=1000, **wide.scales()))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 8)])
def test_decode_reports_bad_entries(kind, window, sinks):
    c = AnyCache([100, 100, 100, 100, 100], 2, 16, kind, seed=21)
    c.table[1, 6], c.table[2, 0] = c.pages, -1
    c.lens[3], c.lens[4] = -1, 10000
    c.seq_lens = torch.tensor(c.lens, dtype=torch.int32).cuda()
    q = randn(5, 8 * D, seed=22)
    ws = fl.attention_decode_workspace()
    out = fl.attention_decode_window(q, *c.args(), window=window, sinks=sinks, workspace=ws, **c.scales())
    assert fl.check_device_status(ws) == fl.FL_ERR_INVALID_ARG and fl.check_device_status(ws) == fl.FL_OK
    assert torch.isnan(out[1:]).all()
    check_decode(q, c, out, window, sinks, skip=(1, 2, 3, 4))


@pytest.mark.parametrize("kind", KINDS)
def test_decode_window_strides_streams_and_repeats(kind):
    lens = [1200, 77, 400]
    c = AnyCache(lens, 2, 16, kind, seed=23)
    q = randn(3, 12 * D, seed=24)
    want = fl.attention_decode_window(q, *c.args(), window=200, sinks=4, **c.scales())
    check_decode(q, c, want, 200, 4)
    wide = torch.full((3, 13 * D), 9.0, dtype=torch.bfloat16, device="cuda")
    wide[:, :12 * D] = q
    out = torch.full((3, 14 * D), 9.0, dtype=torch.bfloat16, device="cuda")
    table = torch.cat([c.table, torch.full_like(c.table, -3)], 1)[:, :c.table.shape[1]]
    fl.attention_decode_window(wide[:, :12 * D], c.k, c.v, table, c.seq_lens, window=200, sinks=4, O=out[:, :12 * D], **c.scales())
    assert torch.equal(out[:, :12 * D], want) and (out[:, 12 * D:] == 9).all()
    # pages that are parts of larger blocks
    def apart(t, more):
        room = torch.zeros((t.shape[0], t[0].numel() + more), dtype=t.dtype, device="cuda")
        room[:, :t[0].numel()] = t.flatten(1)
        return room[:, :t[0].numel()].unflatten(1, t.shape[1:])
    scales = {n: None if t is None else apart(t, 8) for n, t in c.scales().items()}
    assert torch.equal(fl.attention_decode_window(q, apart(c.k, 64), apart(c.v, 64), c.table, c.seq_lens, window=200, sinks=4,
                                                  **scales), want)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        torch.cuda._sleep(20000000)
        got = fl.attention_decode_window(q, *c.args(), window=200, sinks=4, **c.scales(), stream=other)
        other.synchronize()
    assert torch.equal(got, want)
    place = q.clone()
    assert torch.equal(fl.attention_decode_window(place, *c.args(), window=200, sinks=4, O=place, **c.scales()), want)
    ws = fl.attention_decode_workspace()
    for _ in range(5):
        assert torch.equal(fl.attention_decode_window(q, *c.args(), window=200, sinks=4, workspace=ws, **c.scales()), want)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 20)])
def test_decode_captured_and_replayed_as_sequences_grow(kind, window, sinks):
    """Through the lengths at which the window's first unit moves on."""
    c = AnyCache([400, 700, 30], 2, 16, kind, seed=25)
    q, ws = randn(3, 8 * D, seed=26), fl.attention_decode_workspace()
    out = torch.empty_like(q)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fl.attention_decode_window(q, *c.args(), window=window, sinks=sinks, O=out, workspace=ws, **c.scales())
    full = [400, 700, 30]
    for step in (250, 240, 130, 129, 128, 127, 64, 1, 0):
        c.lens = [max(n - step, 0) for n in full]
        c.seq_lens.copy_(torch.tensor(c.lens, dtype=torch.int32))
        g.replay()
        check_decode(q, c, out, window, sinks)


def test_two_calls_at_once_with_a_workspace_each():
    c = AnyCache([3000, 900], 2, 16, "int4", seed=27)
    q = randn(2, 8 * D, seed=28)
    want = [fl.attention_decode_window(q, *c.args(), window=w, sinks=4, **c.scales()) for w in (0, 500)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [fl.attention_decode_workspace() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(fl.attention_decode_window(q, *c.args(), window=(0, 500)[i], sinks=4, workspace=spaces[i],
                                                         **c.scales()))
    torch.cuda.synchronize()
    assert all(torch.equal(o, w) for outs, w in zip(got, want) for o in outs)


def test_decode_offsets_beyond_32_bits():
    kv, page, lens = 8, 64, [150, 64, 1, 700]
    c = AnyCache(lens, kv, page, "int4", seed=29)
    pages = (1 << 32) // (kv * page * D // 2) + 40
    first = pages - c.pages
    q = randn(len(lens), 32 * D, seed=30)
    want = [fl.attention_decode_window(q, *c.args(), window=w, sinks=2, **c.scales()) for w in (0, 100)]
    pitch = ((1 << 32) // (2 * first) // 4 + 1) * 4
    for name in ("k", "v"):
        big = torch.zeros((pages,) + c.k.shape[1:], dtype=torch.uint8, device="cuda")
        big[first:] = getattr(c, name)
        setattr(c, name, big)
    for name in ("ks", "vs"):
        big = torch.zeros(pages * pitch, dtype=torch.bfloat16, device="cuda").as_strided((pages, kv, page, 4), (pitch, page * 4, 4, 1))
        big[first:] = getattr(c, name)
        setattr(c, name, big)
    c.table += first
    for w, o in zip((0, 100), want):
        assert torch.equal(fl.attention_decode_window(q, *c.args(), window=w, sinks=2, **c.scales()), o)


def test_projection_append_and_decode_steps_over_4_bits():
    """The path as it is used: projection, append, one token after the other; against the rows that are read back."""
    hidden, lens = 256, [70, 1, 130]
    x = randn(sum(lens), hidden, seed=31)
    w = randn(3 * 4 * D, hidden, seed=32, std=hidden ** -0.5)
    c = AnyCache([n + 3 for n in lens], 4, 16, "int4", seed=33)
    held = torch.tensor(lens, dtype=torch.int32).cuda()
    positions = torch.cat([torch.arange(n) for n in lens]).int().cuda()
    _, k, v = fl.fused_qkv_rope(x, w, None, n_heads=4, positions=positions)
    fl.paged_kv_append_int4(k, v, c.k, c.v, c.ks, c.vs, c.table, held, cu_seqlens=cu(lens))
    for step in range(3):
        q, k, v = fl.fused_qkv_rope(randn(3, hidden, seed=34 + step), w, None, n_heads=4, positions=held.clone())
        held += 1
        fl.paged_kv_append_int4(k, v, c.k, c.v, c.ks, c.vs, c.table, held)
        now = [n + step + 1 for n in lens]
        kk, vv = fl.paged_kv_read(c.k, c.v, c.table, held, cu_seqlens=cu(now), rows=sum(now), **c.scales())
        for window, sinks in ((0, 0), (40, 2)):
            out = fl.attention_decode_window(q, c.k, c.v, c.table, held, window=window, sinks=sinks, **c.scales())
            at = 0
            for b, n in enumerate(now):
                rows = slice(at, at + n)
                at += n
                c.lens[b] = n
                ref, tol = attend_window(q[b].double().view(4, 1, D), kk[rows].double().view(n, 4, D).transpose(0, 1),
                                         vv[rows].double().view(n, 4, D).transpose(0, 1), D ** -0.5, window, sinks, 2 * F16,
                                         scales=c.value_scales(b))
                assert_within(out[b].view(4, 1, D), ref, tol, f"step {step}, sequence {b}")
