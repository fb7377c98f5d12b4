"""attention_decode_window and attention_prefill_window against their definition in 64 bits (window_utils derives the
tolerances), at the lengths, windows and layouts where they can go wrong."""
import pytest
import torch

import gemm_epilogue_tcgen05_gb300 as fl
from attention_utils import BF16, D, F16, assert_within, cu, quantise, rounded, tile_powers, values
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


@pytest.mark.parametrize("std", [2.0, 4.0, 8.0])
def test_decode_over_4_bits_heavy_tokens_with_small_codes(std):
    """A few tokens have all the weight, and in many columns codes of zero: what is left of their codes + 8 and the eights."""
    for seed in range(12):
        c = AnyCache([16, 40, 100, 7, 33, 300, 12, 20, 2, 1], 1, 16, "int4", seed=140 + seed)
        q = randn(10, 8 * D, seed=160 + seed, std=std)
        out = fl.attention_decode_window(q, *c.args(), **c.scales())
        check_decode(q, c, out)


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


# ---------------------------------------------------------------- prefill
def rows_of(n, heads, seed=0, std=1.0):
    return randn(n, heads * D, seed=seed, std=std)


def keys_of(rows, kv, fp8, seed=0):
    k, v = randn(rows, kv, D, seed=seed + 1), randn(rows, kv, D, seed=seed + 2)
    ks = vs = None
    if fp8:
        (k, ks), (v, vs) = quantise(k), quantise(v)
    return k.view(rows, -1), v.view(rows, -1), ks, vs


def check_prefill(q, k, v, ks, vs, lens, out, window=0, sinks=0, lens_k=None, scale=D ** -0.5, what="", first=0, first_k=0):
    heads, kv = q.shape[1] // D, k.shape[1] // D
    for b, (n, n_k) in enumerate(zip(lens, lens_k or lens)):
        rows, keys = slice(first, first + n), slice(first_k, first_k + n_k)
        first, first_k = first + n, first_k + n_k
        if n == 0:
            continue
        got = out[rows].view(n, heads, D).transpose(0, 1)
        if n_k == 0:
            assert (got == 0).all(), f"{what}: sequence {b} has no keys"
            continue
        kk = values(k[keys].reshape(n_k, kv, D), None if ks is None else ks[keys]).transpose(0, 1)
        vv = values(v[keys].reshape(n_k, kv, D), None if vs is None else vs[keys]).transpose(0, 1)
        qq = q[rows].double().reshape(n, heads, D).transpose(0, 1)
        if ks is not None:
            kk = rounded(kk)
            ref, tol = attend_window(qq, kk, vv, scale, window, sinks, 2 * F16, powers=tile_powers(vs[keys]))
        else:
            ref, tol = attend_window(qq, kk, vv, scale, window, sinks, BF16)
        assert_within(got, ref, tol, f"{what} sequence {b} of {n} behind {n_k - n}")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 3), (64, 0), (100, 4), (128, 128), (129, 1), (200, 200), (500, 64), (1000, 0)])
@pytest.mark.parametrize("heads,kv", [(4, 1), (3, 3), (24, 2), (48, 1), (80, 1)])
def test_prefill_window_matches_the_definition(heads, kv, window, sinks, fp8):
    lens = [1, 700, 0, 130, 128, 333]
    q = rows_of(sum(lens), heads, seed=40)
    k, v, ks, vs = keys_of(sum(lens), kv, fp8, seed=41)
    out = fl.attention_prefill_window(q, k, v, cu_seqlens=cu(lens), window=window, sinks=sinks, k_scale=ks, v_scale=vs)
    check_prefill(q, k, v, ks, vs, lens, out, window, sinks)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 3), (300, 150)])
@pytest.mark.parametrize("heads,kv", [(8, 2), (16, 16), (20, 4)])
def test_prefill_behind_cached_rows_matches_the_definition(heads, kv, window, sinks, fp8):
    """Histories of every kind: none, shorter and longer than the new rows, with and without whole tiles."""
    lens, lens_k = [1, 33, 128, 0, 200, 5, 300, 64], [900, 33, 129, 70, 328, 1200, 301, 192]
    q = rows_of(sum(lens), heads, seed=42)
    k, v, ks, vs = keys_of(sum(lens_k), kv, fp8, seed=43)
    out = fl.attention_prefill_window(q, k, v, cu_seqlens=cu(lens), cu_seqlens_k=cu(lens_k), window=window, sinks=sinks,
                                      k_scale=ks, v_scale=vs)
    check_prefill(q, k, v, ks, vs, lens, out, window, sinks, lens_k)


@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_rows_in_front_of_the_first_key_are_zeros(fp8):
    """More queries than keys, no keys at all; what lies in the rows of K there reaches nothing."""
    lens, lens_k = [5, 300, 129, 40], [2, 0, 128, 41]
    q = rows_of(sum(lens), 8, seed=44)
    k, v, ks, vs = keys_of(sum(lens_k) + 200, 2, fp8, seed=45)
    if fp8:
        ks[sum(lens_k):], vs[sum(lens_k):] = NAN, INF
    else:
        k[sum(lens_k):], v[sum(lens_k):] = NAN, INF
    for window, sinks in ((0, 0), (3, 1), (200, 7)):
        out = torch.full((sum(lens), 8 * D), 5.0, dtype=torch.bfloat16, device="cuda")
        fl.attention_prefill_window(q, k, v, cu_seqlens=cu(lens), cu_seqlens_k=cu(lens_k), window=window, sinks=sinks,
                                    k_scale=ks, v_scale=vs, O=out)
        check_prefill(q, k, v, ks, vs, lens, out, window, sinks, lens_k)
        assert (out[:3] == 0).all() and (out[5:305] == 0).all() and (out[305] == 0).all()
    # a query alone, without a key, in front of everything
    out = fl.attention_prefill_window(q[:1], k, v, cu_seqlens=cu([1]), cu_seqlens_k=cu([0]), k_scale=ks, v_scale=vs)
    assert (out == 0).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_window_of_long_and_many_sequences(fp8):
    lens = [3000, 20] + [(7 * i * i + 3) % 97 for i in range(150)] + [1100]
    q = rows_of(sum(lens), 4, seed=46)
    k, v, ks, vs = keys_of(sum(lens), 2, fp8, seed=47)
    for window, sinks in ((256, 4), (1024, 64), (40, 500)):
        out = fl.attention_prefill_window(q, k, v, cu_seqlens=cu(lens), window=window, sinks=sinks, k_scale=ks, v_scale=vs)
        check_prefill(q, k, v, ks, vs, lens, out, window, sinks)


@pytest.mark.parametrize("seq_len,rows", [(64, 256), (300, 1000), (0, 450)])
def test_prefill_window_of_equal_sequences(seq_len, rows):
    q = rows_of(rows, 8, seed=48)
    k, v, _, _ = keys_of(rows, 4, False, seed=49)
    n = seq_len or rows
    lens = [n] * (rows // n) + ([rows % n] if rows % n else [])
    out = fl.attention_prefill_window(q, k, v, seq_len=seq_len, window=150, sinks=2)
    check_prefill(q, k, v, None, None, lens, out, 150, 2)


@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_window_that_hides_nothing(fp8):
    lens = [700, 3, 128]
    q = rows_of(sum(lens), 8, seed=50)
    k, v, ks, vs = keys_of(sum(lens), 2, fp8, seed=51)
    call = dict(cu_seqlens=cu(lens), k_scale=ks, v_scale=vs)
    want = fl.attention_prefill(q, k, v, **call)
    for window, sinks in ((0, 0), (0, 5), (sum(lens), 0), (1 << 40, 1 << 33)):
        assert torch.equal(want, fl.attention_prefill_window(q, k, v, window=window, sinks=sinks, **call))
    for window, sinks in ((700, 0), (600, 100), (1, 830)):  # the windowed kernel
        out = fl.attention_prefill_window(q, k, v, window=window, sinks=sinks, **call)
        check_prefill(q, k, v, ks, vs, lens, out, window, sinks)
    out = fl.attention_prefill_window(q, k, v, cu_seqlens_k=cu(lens), **call)
    check_prefill(q, k, v, ks, vs, lens, out)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("window,sinks", [(100, 3), (0, 0)])
def test_prefill_window_leaves_other_rows_and_ignores_their_contents(fp8, window, sinks):
    lens, lens_k, first, first_k = [150, 70], [400, 70], 20, 33
    rows, rows_k = 300, 600
    q = rows_of(rows, 8, seed=52)
    k, v, ks, vs = keys_of(rows_k, 2, fp8, seed=53)
    q[:first], q[first + 220:] = NAN, INF
    for r in (slice(0, first_k), slice(first_k + 470, None)):
        k[r], v[r] = (0x7F, 0x7F) if fp8 else (INF, NAN)
        if fp8:
            ks[r], vs[r] = NAN, INF
    out = torch.full((rows, 8 * D), 3.0, dtype=torch.bfloat16, device="cuda")
    fl.attention_prefill_window(q, k, v, cu_seqlens=cu(lens) + first, cu_seqlens_k=cu(lens_k) + first_k, window=window,
                                sinks=sinks, k_scale=ks, v_scale=vs, O=out)
    check_prefill(q, k, v, ks, vs, lens, out, window, sinks, lens_k, first=first, first_k=first_k)
    assert (out[:first] == 3).all() and (out[first + 220:] == 3).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_prefill_window_values_that_are_not_finite_reach_only_who_sees_them(which, bad, fp8):
    """In the sinks, in a window, and at keys that most rows do not see any more."""
    n, window, sinks = 900, 130, 40
    lens = [n, 64]
    at = [7, 39, 300, 511, 512]
    q = rows_of(sum(lens), 4, seed=54)
    k, v, ks, vs = keys_of(sum(lens), 1, fp8, seed=55)
    clean = [k.clone(), v.clone(), None if ks is None else ks.clone(), None if vs is None else vs.clone()]
    for j in at[2:]:
        if fp8:
            (ks if which == "k" else vs)[j] = abs(bad)  # scales are not negative
        else:
            (k if which == "k" else v)[j, 5] = bad
    call = dict(cu_seqlens=cu(lens), window=window, sinks=sinks)
    out = fl.attention_prefill_window(q, k, v, k_scale=ks, v_scale=vs, **call)
    i = torch.arange(n, device="cuda")
    sees = torch.zeros(n, dtype=torch.bool, device="cuda")
    for j in at[2:]:
        sees |= (i >= j) & (i < j + window)
    hidden = torch.cat([~sees, torch.ones(64, dtype=torch.bool, device="cuda")])
    assert torch.isfinite(out[hidden]).all()
    ref = fl.attention_prefill_window(q, *clean[:2], k_scale=clean[2], v_scale=clean[3], **call)
    if not fp8 or which == "k":
        assert torch.equal(out[hidden], ref[hidden])
    seen = out[:n][sees]
    if which == "v" and not fp8:
        assert (~torch.isfinite(seen.view(-1, 4, D)[..., 5])).all()
        keep = torch.arange(D, device="cuda") != 5
        assert torch.equal(seen.view(-1, 4, D)[..., keep], ref[:n][sees].view(-1, 4, D)[..., keep])
    # in the sinks every row behind sees them
    k, v, ks, vs = clean
    for j in at[:2]:
        if fp8:
            (ks if which == "k" else vs)[j] = abs(bad)  # scales are not negative
        else:
            (k if which == "k" else v)[j, 5] = bad
    out = fl.attention_prefill_window(q, k, v, k_scale=ks, v_scale=vs, **call)
    assert torch.isfinite(out[:7]).all() and torch.isfinite(out[n:]).all()
    if which == "v":
        col = out[7:n].view(-1, 4, D)[..., 5]
        assert (~torch.isfinite(col)).all()


@pytest.mark.parametrize("shift", [2.0 ** 20, 2.0 ** 40, 2.0 ** -40, 0.0])
def test_prefill_window_single_keys(shift):
    """E4M3 keys whose scale of V lies far from the others', in the sinks, at the window's edges, and out of sight."""
    lens, window, sinks = [800, 130], 200, 5
    q = rows_of(sum(lens), 8, seed=56)
    k, v, ks, vs = keys_of(sum(lens), 2, True, seed=57)
    for j in (0, 3, 4, 6, 255, 256, 600, 799, 801):
        vs[j] *= shift
    out = fl.attention_prefill_window(q, k, v, cu_seqlens=cu(lens), window=window, sinks=sinks, k_scale=ks, v_scale=vs)
    first = 0
    for b, n in enumerate(lens):
        r = slice(first, first + n)
        first += n
        kk = rounded(values(k[r].view(n, 2, D), ks[r]).transpose(0, 1))
        vv = values(v[r].view(n, 2, D), vs[r]).transpose(0, 1)
        ref, tol = attend_window(q[r].double().view(n, 8, D).transpose(0, 1), kk, vv, D ** -0.5, window, sinks, 2 * F16)
        # a weight below fp16's range is off by 2^-32 of the row's largest weight times scale (attention_utils); 210 keys, and a
        # value is below 2^9 of its scale's power: 2^-15 of that together
        i = torch.arange(n, device="cuda")
        seen = ((i[None] <= i[:, None]) & ((i[None] > i[:, None] - window) | (i[None] < sinks))).double()
        x = (q[r].double().view(n, 8, D).transpose(0, 1) @ kk.repeat_interleave(4, 0).transpose(1, 2) * D ** -0.5)
        p = torch.softmax(x.masked_fill(seen == 0, -INF), -1)
        part = (p * vv.abs().amax(-1).repeat_interleave(4, 0)[:, None]).amax(-1, keepdim=True)
        assert_within(out[r].view(n, 8, D).transpose(0, 1), ref, tol + 2.0 ** -14 * part, f"sequence {b}")


@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_window_strides_place_streams_and_repeats(fp8):
    lens, lens_k = [300, 1, 64, 150], [700, 1, 200, 150]
    q = rows_of(sum(lens), 12, seed=58)
    k, v, ks, vs = keys_of(sum(lens_k), 4, fp8, seed=59)
    call = dict(cu_seqlens=cu(lens), cu_seqlens_k=cu(lens_k), window=180, sinks=9, k_scale=ks, v_scale=vs, scale=0.11)
    want = fl.attention_prefill_window(q, k, v, **call)
    check_prefill(q, k, v, ks, vs, lens, want, 180, 9, lens_k, scale=0.11)

    def wide(t, more):
        room = torch.zeros((t.shape[0], t.shape[1] + more), dtype=t.dtype, device="cuda")
        room[:, :t.shape[1]] = t
        return room[:, :t.shape[1]]
    out = wide(torch.zeros_like(q), 2 * D)
    moved = dict(call, k_scale=None if ks is None else wide(ks, 3), v_scale=None if vs is None else wide(vs, 3))
    fl.attention_prefill_window(wide(q, D), wide(k, 64), wide(v, 64), O=out, **moved)
    assert torch.equal(out, want)
    place = q.clone()
    assert torch.equal(fl.attention_prefill_window(place, k, v, O=place, **call), want)
    ws = fl.attention_prefill_workspace(sum(lens_k), 4, fp8)
    for _ in range(5):
        assert torch.equal(fl.attention_prefill_window(q, k, v, workspace=ws, **call), want)
        fl.attention_prefill(q[:150], k[:150], v[:150], k_scale=ks if ks is None else ks[:150],
                             v_scale=vs if vs is None else vs[:150], workspace=ws)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        torch.cuda._sleep(20000000)
        got = fl.attention_prefill_window(q, k, v, **call, stream=other)
        other.synchronize()
    assert torch.equal(got, want) and fl.check_device_status(ws) == fl.FL_OK


@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_window_captured_and_replayed_with_other_offsets(fp8):
    rows, rows_k = 600, 1500
    q = rows_of(rows, 8, seed=60)
    k, v, ks, vs = keys_of(rows_k, 2, fp8, seed=61)
    offsets, offsets_k = cu([300, 300]), cu([700, 800])
    out = torch.zeros_like(q)
    ws = fl.attention_prefill_workspace(rows_k, 2, fp8)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fl.attention_prefill_window(q, k, v, cu_seqlens=offsets, cu_seqlens_k=offsets_k, window=250, sinks=4, k_scale=ks,
                                    v_scale=vs, O=out, workspace=ws)
    for lens, lens_k in (([300, 300], [700, 800]), ([1, 599], [900, 600]), ([0, 64], [100, 1400]), ([600, 0], [600, 0])):
        offsets.copy_(cu(lens)), offsets_k.copy_(cu(lens_k))
        out.fill_(2)
        g.replay()
        check_prefill(q, k, v, ks, vs, lens, out, 250, 4, lens_k)
        assert (out[sum(lens):] == 2).all()


def test_prefill_window_bad_offsets_stay_inside():
    """Offsets that fall or leave the rows give some rows or none, never a fault."""
    q = rows_of(200, 4, seed=62)
    k, v, _, _ = keys_of(300, 2, False, seed=63)
    for a, b in (([0, 500, 100], [0, 300, 300]), ([-5, 50, 20], [10, 400, 350]), ([0, 100, 200], [300, 0, 900]),
                 ([0, 100, 200], [-9, -4, -1]), ([200, 300, 400], [0, 100, 200])):
        fl.attention_prefill_window(q, k, v, cu_seqlens=torch.tensor(a, dtype=torch.int32).cuda(),
                                    cu_seqlens_k=torch.tensor(b, dtype=torch.int32).cuda(), window=40, sinks=2)
    torch.cuda.synchronize()
    assert fl.device_status() == fl.FL_OK


@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 4)])
def test_a_prompt_in_parts_over_a_4_bit_cache(window, sinks):
    """The run as it is used: each part of two prompts is projected, appended, the context read back, and attended to; the
    last token once more by decode.  Parts of another cut give the same bits in the cache and agree within the rounding."""
    hidden, total = 256, [333, 64]
    x = randn(sum(total), hidden, seed=64)
    w = randn(3 * 4 * D, hidden, seed=65, std=hidden ** -0.5)
    kept = None
    for parts in ([(333, 64)], [(100, 64), (200, 0), (33, 0)], [(128, 1), (128, 62), (77, 1)]):
        c = AnyCache(total, 4, 16, "int4", seed=66)
        done, outs = [0, 0], [[], []]
        for part in parts:
            rows = torch.cat([x[sum(total[:b]) + done[b]:sum(total[:b]) + done[b] + part[b]] for b in range(2)])
            pos = torch.cat([torch.arange(done[b], done[b] + part[b]) for b in range(2)]).int().cuda()
            q, k, v = fl.fused_qkv_rope(rows, w, None, n_heads=4, positions=pos)
            done = [done[b] + part[b] for b in range(2)]
            held = torch.tensor(done, dtype=torch.int32).cuda()
            fl.paged_kv_append_int4(k, v, c.k, c.v, c.ks, c.vs, c.table, held, cu_seqlens=cu(part))
            kk, vv = fl.paged_kv_read(c.k, c.v, c.table, held, cu_seqlens=cu(done), rows=sum(done), **c.scales())
            o = fl.attention_prefill_window(q, kk, vv, cu_seqlens=cu(part), cu_seqlens_k=cu(done), window=window, sinks=sinks)
            check_prefill(q, kk, vv, None, None, part, o, window, sinks, done)
            outs[0].append(o[:part[0]]), outs[1].append(o[part[0]:])
            last = q[[part[0] - 1, part[0] + part[1] - 1]] if min(part) > 0 else None
        if last is not None:
            one = fl.attention_decode_window(last, c.k, c.v, c.table, c.seq_lens, window=window, sinks=sinks, **c.scales())
            check_decode(last, c, one, window, sinks)
        whole = torch.cat([torch.cat(o) for o in outs])
        if kept is None:
            kept = whole, kk, vv
        assert torch.equal(kept[1], kk) and torch.equal(kept[2], vv)
        # both are within 2^-8 |o| + 2^-8 A of one value, and A is at most the largest value
        assert ((whole - kept[0]).double().abs() <= 2 * BF16 * (kept[0].double().abs() + vv.double().abs().max())).all()
