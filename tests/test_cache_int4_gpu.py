"""paged_kv_append_int4 and paged_kv_read against their definition in 64 bits, bit for bit: the 4-bit codes and scales have
one right value each, and what is read back of bf16 and 4-bit entries is what they stand for."""
import pytest
import torch

import gemm_epilogue_tcgen05_gb300 as fl
from attention_utils import D, cu, quantise
from window_utils import AnyCache, codes_of, numbers, quantise_int4

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def randn(*shape, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).bfloat16().cuda()


def cells(cache, b, first, n):
    pos = torch.arange(first, first + n, device="cuda")
    return cache.table[b].long()[pos // cache.page], pos % cache.page


def bits(t):
    return t.view(torch.int16)


@pytest.mark.parametrize("page", [1, 3, 16, 64])
@pytest.mark.parametrize("kv", [1, 2, 3, 8, 11])
def test_append_puts_codes_and_scales_in_their_slots(page, kv):
    lens, new = [70, 5, 33, 200, 1], [1, 5, 0, 130, 1]
    c = AnyCache(lens, kv, page, "int4", seed=1)
    rows = sum(new)
    k, v = randn(rows + 3, kv * D, seed=2), randn(rows + 3, kv * D, seed=3)
    want = [t.clone() for t in (c.k, c.v, c.ks, c.vs)]
    at = 0
    for b, n in enumerate(new):
        p, s = cells(c, b, lens[b] - n, n)
        for i, y in ((0, k), (1, v)):
            want[i][p, :, s], want[2 + i][p, :, s] = quantise_int4(y[at:at + n].view(n, kv, D))
        at += n
    fl.paged_kv_append_int4(k, v, c.k, c.v, c.ks, c.vs, c.table, c.seq_lens, cu_seqlens=cu(new))
    for got, w in zip((c.k, c.v, c.ks, c.vs), want):
        assert torch.equal(got.view(torch.uint8), w.view(torch.uint8))


@pytest.mark.parametrize("std", [1e-38, 1e-30, 1e-3, 1.0, 300.0, 1e30, 3.9e37])
def test_append_rounds_to_the_nearest_code(std):
    """Also where bf16's range ends, and with groups of zeros, of one value, and of exact halves of a step."""
    n = 600
    y = randn(n, 2 * D, seed=int(std) % 1000 + 7, std=1.0).float()
    y[0] = 0
    y[1, 5] = 0
    y[2, :] = 1.75  # a group of one value: s = 1/4, codes 7
    y[3, :32] = torch.arange(32) / 2 - 7.0  # up to 8.5: the largest stays in range
    y[4, ::2] = 0
    y = (y * std).bfloat16()
    assert torch.isfinite(y).all()
    c = AnyCache([1] * n, 2, 4, "int4", seed=8)
    z = -y.flip(0)
    fl.paged_kv_append_int4(y, z, c.k, c.v, c.ks, c.vs, c.table, c.seq_lens)
    at, slot = c.table[:, 0].long(), torch.zeros(n, dtype=torch.long, device="cuda")
    for got, scale, x in ((c.k, c.ks, y), (c.v, c.vs, z)):
        code, s = quantise_int4(x.view(n, 2, D))
        assert torch.equal(bits(scale[at, :, slot]), bits(s)) and torch.equal(got[at, :, slot], code)
        assert (codes_of(code).abs() <= 7).all()


def test_append_every_largest_value_and_every_quotient():
    """All 128 significands of a group's largest value against all 256 values of another, both signs: every border."""
    big = (torch.arange(128, 256).float() / 128)[:, None].expand(128, 256)
    other = torch.cat([torch.arange(128, 256).float() / 128 * 2.0 ** -e for e in (0, 1)])[None].expand(128, 256)
    other = torch.minimum(other, big)
    y = torch.zeros(128 * 256, 32)
    y[:, 3], y[:, 9], y[:, 10] = big.reshape(-1), other.reshape(-1), -other.reshape(-1) / 4
    y[:, 11], y[:, 12] = other.reshape(-1) / 2, -other.reshape(-1)
    y = y.view(-1, D).bfloat16().cuda()
    n = y.shape[0]
    c = AnyCache([1] * n, 1, 1, "int4", seed=9)
    fl.paged_kv_append_int4(y, y, c.k, c.v, c.ks, c.vs, c.table, c.seq_lens)
    code, s = quantise_int4(y.view(n, 1, D))
    at = c.table[:, 0].long()
    assert torch.equal(c.k[at, :, 0], code) and torch.equal(bits(c.ks[at, :, 0]), bits(s))
    assert torch.equal(c.v[at, :, 0], code) and torch.equal(bits(c.vs[at, :, 0]), bits(s))


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_append_groups_with_values_that_are_not_finite(bad):
    n = 5
    y = randn(n, 3 * D, seed=10)
    y[1, 40], y[2, D + 127], y[3, 2 * D:] = bad, bad, bad
    c = AnyCache([1] * n, 3, 8, "int4", seed=11)
    fl.paged_kv_append_int4(y, -y, c.k, c.v, c.ks, c.vs, c.table, c.seq_lens)
    code, s = quantise_int4(y.view(n, 3, D))
    at = c.table[:, 0].long()
    assert torch.equal(c.k[at, :, 0], code) and torch.equal(torch.isnan(c.ks[at, :, 0]), torch.isnan(s))
    fine = ~torch.isnan(s)
    assert torch.equal(c.ks[at, :, 0][fine], s[fine]) and int((~fine).sum()) == 1 + 1 + 4
    assert torch.equal(torch.isnan(c.vs[at, :, 0]), ~fine)


def test_append_ignores_rows_without_a_place():
    """Behind the sequences, in front of a sequence's first token, beyond the table, and with a bad page."""
    c = AnyCache([40, 40, 40, 40], 2, 8, "int4", seed=12)
    before = [t.clone() for t in (c.k, c.v, c.ks, c.vs)]
    c.seq_lens = torch.tensor([3, 45, 2 ** 31 - 1, 40], dtype=torch.int32).cuda()
    c.table[3, 4] = -1
    offsets = torch.tensor([2, 8, 13, 15, 18], dtype=torch.int32).cuda()
    k, v = randn(25, 2 * D, seed=13), randn(25, 2 * D, seed=14)
    fl.paged_kv_append_int4(k, v, c.k, c.v, c.ks, c.vs, c.table, c.seq_lens, cu_seqlens=offsets)
    p, s = cells(c, 0, 0, 3)  # six rows for three tokens: the first three have no place
    code, scale = quantise_int4(k[5:8].view(3, 2, D))
    assert torch.equal(c.k[p, :, s], code) and torch.equal(c.ks[p, :, s], scale)
    before[0][p, :, s], before[2][p, :, s] = code, scale
    before[1][p, :, s], before[3][p, :, s] = quantise_int4(v[5:8].view(3, 2, D))
    for t, b in zip((c.k, c.v, c.ks, c.vs), before):
        assert torch.equal(t, b)


# ---------------------------------------------------------------- read
@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
@pytest.mark.parametrize("page,kv", [(1, 1), (5, 3), (16, 8), (64, 2), (128, 9)])
def test_read_gives_what_the_entries_stand_for(kind, page, kv):
    """Ends, whole sequences and parts from the middle; rows in front of, between and behind the sequences stay."""
    c = AnyCache([300, 7, 0, 129, 64, 1], kv, page, kind, seed=20, fill=NAN)
    ends, n, first = [300, 7, 0, 100, 64, 1], [300, 2, 0, 33, 64, 1], 4
    rows = first + sum(n) + 5
    k, v = (torch.full((rows, kv * D), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    got = fl.paged_kv_read(c.k, c.v, c.table, torch.tensor(ends, dtype=torch.int32).cuda(), cu_seqlens=cu(n) + first, K=k, V=v,
                           **c.scales())
    assert got[0] is k and got[1] is v
    at = first
    for b, (e, m) in enumerate(zip(ends, n)):
        p, s = cells(c, b, e - m, m)
        for out, codes, scale in ((k, c.k, c.ks), (v, c.v, c.vs)):
            want = numbers(kind, codes[p, :, s], None if scale is None else scale[p, :, s])
            # E4M3: the product in fp32, then bf16; else exact
            assert torch.equal(out[at:at + m].view(m, kv, D), want.float().bfloat16())
            if kind != "fp8":
                assert torch.equal(out[at:at + m].view(m, kv, D).double(), want)
        at += m
    for out in (k, v):
        assert (out[:first] == 3).all() and (out[at:] == 3).all()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
def test_read_last_tokens_strides_and_allocated_outputs(kind):
    c = AnyCache([17, 1, 40], 2, 16, kind, seed=21)
    k, v = fl.paged_kv_read(*c.args(), **c.scales())
    for b in range(3):
        p, s = cells(c, b, c.lens[b] - 1, 1)
        for out, codes, scale in ((k, c.k, c.ks), (v, c.v, c.vs)):
            assert torch.equal(out[b:b + 1].view(1, 2, D), numbers(kind, codes[p, :, s], None if scale is None else
                                                                    scale[p, :, s]).float().bfloat16())
    wide = [torch.full((70, 3 * D), 2.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    fl.paged_kv_read(*c.args(), cu_seqlens=cu(c.lens), K=wide[0][:, :2 * D], V=wide[1][:, :2 * D], **c.scales())
    dense = fl.paged_kv_read(*c.args(), cu_seqlens=cu(c.lens), rows=70, **c.scales())
    for w, t in zip(wide, dense):
        assert torch.equal(w[:58, :2 * D], t[:58]) and (w[58:] == 2).all() and (w[:, 2 * D:] == 2).all() and (t[58:] == 0).all()


@pytest.mark.parametrize("kind", ["bf16", "fp8", "int4"])
def test_read_rows_without_a_place_are_nan(kind):
    c = AnyCache([40, 40, 40], 2, 8, kind, seed=22)
    c.table[1, 2], c.table[2, 1] = c.pages, -7
    ends = torch.tensor([2, 40, 60], dtype=torch.int32).cuda()
    k, v = fl.paged_kv_read(c.k, c.v, c.table, ends, cu_seqlens=cu([4, 40, 60]), rows=104, **c.scales())
    bad = torch.zeros(104, dtype=torch.bool, device="cuda")
    bad[:2] = True                     # in front of the first token
    bad[4 + 16:4 + 24] = True          # a page that is not there
    bad[44 + 8:44 + 16] = True         # a negative one
    bad[44 + 40:] = True               # beyond the table
    for t in (k, v):
        assert torch.isnan(t[bad]).all() and torch.isfinite(t[~bad]).all()


def test_read_many_sequences_and_repeated_ones():
    """More sequences than a search can do without, empty ones among them; two sequences that share their pages."""
    lens = [0 if i % 7 == 3 else 1 + i % 5 for i in range(900)]
    c = AnyCache(lens, 1, 4, "int4", seed=23)
    k, v = fl.paged_kv_read(*c.args(), cu_seqlens=cu(lens), rows=sum(lens), **c.scales())
    want = torch.cat([c.sequence(b)[0][0] for b in range(900)])
    assert torch.equal(k.double(), want)
    c.table[1] = c.table[0]
    both = fl.paged_kv_read(c.k, c.v, c.table[:2], c.seq_lens[:1].repeat(2), cu_seqlens=cu([lens[0]] * 2), rows=2 * lens[0],
                            **c.scales())[1]
    assert torch.equal(both[:lens[0]], both[lens[0]:])


@pytest.mark.parametrize("kind", ["int4", "fp8"])
def test_rows_come_back_as_they_were_cached(kind):
    """What an append writes a read returns: 4-bit entries quantise to themselves, E4M3 ones to their rounding."""
    lens = [150, 1, 64]
    c = AnyCache(lens, 4, 16, kind, seed=24)
    k, v = randn(215, 4 * D, seed=25), randn(215, 4 * D, seed=26)

    def append(k, v):
        if kind == "int4":
            fl.paged_kv_append_int4(k, v, c.k, c.v, c.ks, c.vs, c.table, c.seq_lens, cu_seqlens=cu(lens))
        else:
            fl.paged_kv_append(k, v, *c.args(), cu_seqlens=cu(lens), **c.scales())

    append(k, v)
    for out, y in zip(fl.paged_kv_read(*c.args(), cu_seqlens=cu(lens), rows=215, **c.scales()), (k, v)):
        code, s = (quantise_int4 if kind == "int4" else quantise)(y.view(215, 4, D))
        assert torch.equal(out, numbers(kind, code, s).float().bfloat16().view(215, -1))
        # half a step of 1/7 (and of the scale's rounding), or of E4M3's eight steps and bf16
        part = (1 / 14 + 1 / 28) if kind == "int4" else 2.0 ** -4 + 2.0 ** -8
        largest = y.float().view(215, -1, 32 if kind == "int4" else D).abs().amax(-1, keepdim=True)
        assert ((out.float() - y.float()).view(largest.shape[0], largest.shape[1], -1).abs() <= part * largest).all()
    assert fl.device_status() == fl.FL_OK


def test_captured_and_replayed_on_growing_sequences():
    lens = torch.tensor([15, 31], dtype=torch.int32).cuda()
    c = AnyCache([40, 40], 2, 16, "int4", seed=27)
    k, v = randn(2, 2 * D, seed=28), randn(2, 2 * D, seed=29)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fl.paged_kv_append_int4(k, v, c.k, c.v, c.ks, c.vs, c.table, lens)
        back = fl.paged_kv_read(c.k, c.v, c.table, lens, **c.scales())
    for step in range(4):
        k.copy_(randn(2, 2 * D, seed=30 + step))
        v.copy_(-k)
        lens += 1
        g.replay()
        code, s = quantise_int4(k.view(2, 2, D))
        want = numbers("int4", code, s).bfloat16().view(2, -1)
        assert torch.equal(back[0], want) and torch.equal(back[1], -want)
        for b in range(2):
            p, slot = cells(c, b, int(lens[b]) - 1, 1)
            assert torch.equal(c.k[p, :, slot][0], code[b])


def test_given_streams_and_another_stream_than_the_tensors():
    c = AnyCache([40, 3], 2, 16, "int4", seed=31)
    k, v = randn(2, 2 * D, seed=32), randn(2, 2 * D, seed=33)
    other = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        torch.cuda._sleep(20000000)
        fl.paged_kv_append_int4(k, v, c.k, c.v, c.ks, c.vs, c.table, c.seq_lens, stream=other)
        got = fl.paged_kv_read(*c.args(), **c.scales(), stream=other)
        other.synchronize()
    code, s = quantise_int4(k.view(2, 2, D))
    assert torch.equal(got[0], numbers("int4", code, s).bfloat16().view(2, -1))


def test_offsets_beyond_32_bits():
    """Pages whose bytes lie behind 2^32 of their arrays, scales by their pitch, too."""
    kv, page, lens = 8, 64, [150, 64, 1, 300]
    small = AnyCache(lens, kv, page, "int4", seed=34)
    pages = (1 << 32) // (kv * page * D // 2) + 40
    first = pages - small.pages
    pitch = ((1 << 32) // (2 * first) // 4 + 1) * 4
    k, v = (torch.zeros(pages, kv, page, D // 2, dtype=torch.uint8, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(pages * pitch, dtype=torch.bfloat16, device="cuda").as_strided((pages, kv, page, 4), (pitch, page * 4, 4, 1))
              for _ in range(2))
    table = small.table + first
    y, z = randn(sum(lens), kv * D, seed=35), randn(sum(lens), kv * D, seed=36)
    fl.paged_kv_append_int4(y, z, k, v, ks, vs, table, small.seq_lens, cu_seqlens=cu(lens))
    back = fl.paged_kv_read(k, v, table, small.seq_lens, cu_seqlens=cu(lens), rows=sum(lens), k_page_scale=ks, v_page_scale=vs)
    for out, x in zip(back, (y, z)):
        code, s = quantise_int4(x.view(-1, kv, D))
        assert torch.equal(out.double(), numbers("int4", code, s).view(out.shape))
    assert (k[:4] == 0).all() and (vs[:4] == 0).all()


def test_nothing_to_do():
    c = AnyCache([5, 5], 2, 16, "int4", seed=37)
    before = c.k.clone()
    empty = torch.empty(0, 2 * D, dtype=torch.bfloat16, device="cuda")
    fl.paged_kv_append_int4(empty, empty, c.k, c.v, c.ks, c.vs, c.table, c.seq_lens, cu_seqlens=cu([0, 0]))
    assert torch.equal(c.k, before)
    k, v = fl.paged_kv_read(*c.args(), cu_seqlens=cu([0, 0]), rows=0, **c.scales())
    assert k.shape == v.shape == (0, 2 * D)
    none = [torch.empty(0, 2, 16, 64, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scales = [torch.empty(0, 2, 16, 4, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    k, v = fl.paged_kv_read(*none, c.table, c.seq_lens, k_page_scale=scales[0], v_page_scale=scales[1])
    assert torch.isnan(k).all() and torch.isnan(v).all()
    fl.paged_kv_append_int4(k, v, *none, *scales, c.table, c.seq_lens)
