"""paged_kv_append, attention_prefill and attention_decode against their definition in 64 bits
(attention_utils derives the tolerances), at the sizes, masks and layouts where they can go wrong, and a
run of them together behind the library's QKV projection."""
import pytest
import torch

import gemm_epilogue_tcgen05_gb300 as fl
from attention_utils import (BF16, D, F16, Cache, assert_within, attend, check_decode, check_prefill, cu, quantise,
                             rounded, values)

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def randn(*shape, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).bfloat16().cuda()


def prompt(rows, heads, kv, fp8, seed=0, std=1.0):
    q, k, v = randn(rows, heads * D, seed=seed, std=std), randn(rows, kv * D, seed=seed + 1), randn(rows, kv * D,
                                                                                                    seed=seed + 2)
    if not fp8:
        return q, k, v, None, None
    (k, ks), (v, vs) = quantise(k.view(rows, kv, D)), quantise(v.view(rows, kv, D))
    return q, k.view(rows, -1), v.view(rows, -1), ks, vs


# ---------------------------------------------------------------- prefill
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,heads,kv", [
    ([1], 1, 1), ([2], 4, 1), ([77], 8, 2), ([128], 2, 2), ([129, 127], 2, 1), ([0, 5, 0, 0, 300, 0], 4, 4),
    ([257, 1, 64, 256], 6, 2), ([513], 16, 1), ([40, 41], 20, 4), ([100], 7, 1), ([33, 260], 24, 2),
    ([1] * 37, 4, 2), ([130], 48, 1), ([70], 80, 1), ([1100, 30], 8, 1), ([9], 129, 1), ([640], 3, 3)])
def test_prefill_matches_the_definition(lens, heads, kv, causal, fp8):
    rows = sum(lens)
    q, k, v, ks, vs = prompt(rows, heads, kv, fp8, seed=rows)
    out = fl.attention_prefill(q, k, v, cu_seqlens=cu(lens), k_scale=ks, v_scale=vs, causal=causal)
    check_prefill(q, k, v, ks, vs, lens, out, causal)


@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_many_sequences(fp8):
    lens = [(7 * i * i + 3) % 97 for i in range(300)]
    q, k, v, ks, vs = prompt(sum(lens), 4, 2, fp8, seed=5)
    out = fl.attention_prefill(q, k, v, cu_seqlens=cu(lens), k_scale=ks, v_scale=vs)
    check_prefill(q, k, v, ks, vs, lens, out, True)


@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_of_a_thousand_short_sequences(fp8):
    """More sequences than a warp probes twice, empty ones and longer ones among them, rows behind the last."""
    lens = [0 if i % 9 == 4 else 129 + i % 3 if i % 200 == 7 else 1 + i % 2 for i in range(1100)]
    rows = sum(lens)
    q, k, v, ks, vs = prompt(rows + 40, 2, 1, fp8, seed=72)
    out = fl.attention_prefill(q, k, v, cu_seqlens=cu(lens), k_scale=ks, v_scale=vs)
    long = [i for i, n in enumerate(lens) if n > 2]
    first = [sum(lens[:i]) for i in range(len(lens) + 1)]
    for i in long + list(range(0, 1100, 29)):
        r = slice(first[i], first[i + 1])
        check_prefill(q[r], k[r], v[r], None if ks is None else ks[r], None if vs is None else vs[r], [lens[i]], out[r], True,
                      what=f"of {i}:")
    assert (out[rows:] == 0).all()
    values_of = values(v[:rows].view(rows, 1, D), None if vs is None else vs[:rows]).view(rows, D)
    alone = torch.tensor([first[i] for i, n in enumerate(lens) if n == 1], device="cuda")
    ref = values_of[alone].repeat(1, 2)  # one key: its value, rounded to fp16 (E4M3) and bf16
    assert ((out[alone].double() - ref).abs() <= (BF16 + 2 * F16) * ref.abs() * (1 + BF16) + 1e-6).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_of_more_sequences_than_rows(fp8):
    lens = [0] * 700 + [3] + [0] * 60 + [1, 140] + [0] * 9
    q, k, v, ks, vs = prompt(sum(lens), 4, 2, fp8, seed=73)
    check_prefill(q, k, v, ks, vs, lens, fl.attention_prefill(q, k, v, cu_seqlens=cu(lens), k_scale=ks, v_scale=vs), True)


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("batch", [32, 33, 64, 65, 150])
def test_prefill_order_of_the_tiles(batch, causal):
    """Around the batches from which on the tiles come in another order; a long sequence last, first or in the middle."""
    for at in (0, batch // 2, batch - 1):
        lens = [1 + 37 * i % 150 for i in range(batch)]
        lens[at] = 2100
        q, k, v, _, _ = prompt(sum(lens), 4, 2, False, seed=batch)
        out = fl.attention_prefill(q, k, v, cu_seqlens=cu(lens), causal=causal)
        check_prefill(q, k, v, None, None, lens, out, causal)


def test_prefill_more_tiles_than_a_wave():
    lens = [700, 1, 333, 1025, 512, 90, 256, 255]
    q, k, v, _, _ = prompt(sum(lens), 32, 32, False, seed=6)
    out = fl.attention_prefill(q, k, v, cu_seqlens=cu(lens))
    check_prefill(q, k, v, None, None, lens, out, True)


@pytest.mark.parametrize("seq_len,rows", [(64, 256), (100, 333), (0, 150), (500, 150), (1, 9)])
def test_prefill_of_equal_sequences(seq_len, rows):
    q, k, v, _, _ = prompt(rows, 8, 4, False, seed=7)
    n = seq_len or rows
    lens = [n] * (rows // n) + ([rows % n] if rows % n else [])
    out = fl.attention_prefill(q, k, v, seq_len=seq_len)
    check_prefill(q, k, v, None, None, lens, out, True)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("causal", [True, False])
def test_prefill_leaves_other_rows_and_ignores_their_contents(fp8, causal):
    """NaN and infinities before, between and behind the sequences reach nothing; rows of O there stay."""
    lens, rows, first = [150, 70], 400, 20
    q, k, v, ks, vs = prompt(rows, 8, 2, fp8, seed=8)
    other = torch.ones(rows, dtype=torch.bool, device="cuda")
    other[first:first + 220] = False
    q[other] = NAN
    for t, bad in ((k, INF), (v, NAN)):
        t[other] = 0x7F if fp8 else bad
    if fp8:
        ks[other], vs[other] = NAN, INF
    out = torch.full((rows, 8 * D), 3.0, dtype=torch.bfloat16, device="cuda")
    fl.attention_prefill(q, k, v, cu_seqlens=cu(lens) + first, k_scale=ks, v_scale=vs, causal=causal, O=out)
    assert (out[other] == 3.0).all()
    mine = slice(first, first + 220)
    check_prefill(q[mine], k[mine], v[mine], None if ks is None else ks[mine], None if vs is None else vs[mine], lens,
                  out[mine], causal)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_prefill_masked_values_of_the_own_sequence(which, bad, fp8):
    """A row never sees what a later token holds, finite or not; rows that do see a NaN value get it."""
    if fp8 and bad != NAN:
        pytest.skip("E4M3 has no infinities")
    n, at = 300, 210
    q, k, v, ks, vs = prompt(n, 4, 1, fp8, seed=9)
    (k if which == "k" else v)[at, 5] = 0x7F if fp8 else bad
    out = fl.attention_prefill(q, k, v, k_scale=ks, v_scale=vs)
    cut = slice(0, at)
    check_prefill(q[cut], k[cut], v[cut], None if ks is None else ks[cut], None if vs is None else vs[cut], [at],
                  out[cut], True)
    seen = out[at:].view(n - at, 4, D)
    if which == "v":
        assert (seen[:, :, 5].isnan() if bad != bad else seen[:, :, 5] == bad).all()
        keep = [d for d in range(D) if d != 5]
        kk, vv = values(k.view(n, 1, D), ks).transpose(0, 1), values(v.view(n, 1, D), vs).transpose(0, 1).clone()
        vv[:, at, 5] = 0.0
        ref, tol = attend(q.double().view(n, 4, D).transpose(0, 1), rounded(kk) if fp8 else kk, vv, D ** -0.5, BF16, True)
        assert_within(seen.transpose(0, 1)[..., keep], ref[:, at:, keep], tol[:, at:, keep])
    elif bad != bad:
        assert seen.isnan().all()


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("at", [5, 127, 128, 210, 299])
def test_prefill_masked_scales_of_the_own_sequence(which, bad, at):
    """The same for a scale that is not finite: rows before it do not meet it, rows behind a NaN one do."""
    n = 300
    q, k, v, ks, vs = prompt(n, 4, 1, True, seed=9)
    (ks if which == "k" else vs)[at] = bad
    out = fl.attention_prefill(q, k, v, k_scale=ks, v_scale=vs)
    check_prefill(q[:at], k[:at], v[:at], ks[:at], vs[:at], [at], out[:at], True)
    if bad != bad:
        assert out[at:].isnan().all()
    elif which == "v":  # an infinite scale of K gives logits of both signs: weight 0 or NaN
        assert not out[at:].isfinite().all(-1).any()


def test_prefill_peaked_and_flat_rows():
    """Logits of many hundreds (the running maximum jumps late) and of one value."""
    for std, seed in ((60.0, 10), (0.0, 11)):
        q, k, v, _, _ = prompt(500, 4, 2, False, seed=seed, std=std)
        k[400] = k[400] * 3
        out = fl.attention_prefill(q, k, v)
        check_prefill(q, k, v, None, None, [500], out, True)


def test_prefill_rising_maximum():
    """Keys that grow along the sequence: nearly every tile raises the maximum."""
    n = 900
    q, k, v, _, _ = prompt(n, 2, 1, False, seed=12)
    q[:] = q.abs()
    k = (k.abs() * torch.linspace(0, 6, n, device="cuda")[:, None]).bfloat16()
    for causal in (True, False):
        check_prefill(q, k, v, None, None, [n], fl.attention_prefill(q, k, v, causal=causal), causal)


def test_prefill_scale_and_strides():
    """Q, K, V and O as columns of wider tensors, E4M3 scales as columns, and a scale of one's own."""
    n, heads, kv = 200, 8, 2
    wide = randn(n, (heads + 2 * kv) * D + 64, seed=13)
    q, k, v = wide[:, 8:8 + heads * D], wide[:, heads * D + 16:(heads + kv) * D + 16], wide[:, (heads + kv) * D + 64:]
    out = torch.zeros(n, heads * D + 24, dtype=torch.bfloat16, device="cuda")[:, 8:8 + heads * D]
    fl.attention_prefill(q, k, v, O=out, scale=0.02)
    check_prefill(q, k, v, None, None, [n], out, True, scale=0.02)
    (k8, ks), (v8, vs) = quantise(k.reshape(n, kv, D)), quantise(v.reshape(n, kv, D))
    codes = torch.zeros(n, 2 * kv * D + 32, dtype=torch.uint8, device="cuda")
    scales = torch.full((n, 2 * kv + 1), NAN, device="cuda")
    k8v, v8v = codes[:, 16:16 + kv * D], codes[:, 32 + kv * D:]
    k8v.copy_(k8.view(n, -1)), v8v.copy_(v8.view(n, -1))
    ksv, vsv = scales[:, :kv], scales[:, kv + 1:]
    ksv.copy_(ks), vsv.copy_(vs)
    out = fl.attention_prefill(q, k8v, v8v, k_scale=ksv, v_scale=vsv, scale=0.3)
    check_prefill(q, k8v, v8v, ksv, vsv, [n], out, True, scale=0.3)


@pytest.mark.parametrize("shift", [-40, -20, 20, 40])
def test_prefill_scales_far_apart(shift):
    """Values of the first 128 keys 2^shift times as large as the others; every row looks at its own key or at one of
    150 tokens before, by some 80 in the exponent, so both sides count for somebody and neither may swamp the other."""
    n = 500
    q, k, v, ks, vs = prompt(n, 2, 1, True, seed=70)
    at = torch.arange(n, device="cuda")
    at = torch.where(at % 2 == 0, at, (at - 150).clamp(min=0))
    q = (8 * values(k.view(n, 1, D), ks).view(n, D)[at]).bfloat16().repeat(1, 2)
    vs[:128] *= 2.0 ** shift
    for causal in (True, False):
        check_prefill(q, k, v, ks, vs, [n], fl.attention_prefill(q, k, v, k_scale=ks, v_scale=vs, causal=causal), causal)


@pytest.mark.parametrize("shift", [-40, 40])
def test_prefill_scales_along_a_long_sequence(shift):
    """The same over more key tiles than a warp's lanes hold powers for, the scales growing or falling all the way."""
    n = 4500
    q, k, v, ks, vs = prompt(n, 1, 1, True, seed=71)
    at = torch.arange(n, device="cuda")
    at = torch.where(at % 2 == 0, at, (at - 2000).clamp(min=0))
    q = (8 * values(k.view(n, 1, D), ks).view(n, D)[at]).bfloat16()
    vs *= torch.exp2(torch.linspace(0, shift, n, device="cuda").round())[:, None]
    check_prefill(q, k, v, ks, vs, [n], fl.attention_prefill(q, k, v, k_scale=ks, v_scale=vs), True)


def test_prefill_zero_scales_and_codes():
    """Heads of zeros (scale 0) beside ordinary ones."""
    n = 150
    q, k, v, ks, vs = prompt(n, 4, 2, True, seed=14)
    for t, s in ((k, ks), (v, vs)):
        t[3:40], s[3:40] = 0, 0.0
    out = fl.attention_prefill(q, k, v, k_scale=ks, v_scale=vs)
    check_prefill(q, k, v, ks, vs, [n], out, True)


def test_prefill_bad_offsets_stay_inside():
    """Offsets that decrease or point outside: clipped to the tensors, other sequences unharmed."""
    q, k, v, _, _ = prompt(120, 4, 2, False, seed=15)
    out = torch.full_like(q, 2.0)
    c = torch.tensor([0, 50, 30, -7, 50, 120000], dtype=torch.int32, device="cuda")
    fl.attention_prefill(q, k, v, cu_seqlens=c, O=out)
    torch.cuda.synchronize()
    check_prefill(q[:50], k[:50], v[:50], None, None, [50], out[:50], True)


@pytest.mark.parametrize("fp8", [False, True])
def test_prefill_captured_replayed_and_reused(fp8):
    """One graph, replayed as lengths and inputs change, its workspace shared with eager calls between."""
    rows, heads, kv = 500, 8, 4
    q, k, v, ks, vs = prompt(rows, heads, kv, fp8, seed=16)
    ws = fl.attention_prefill_workspace(rows, kv, fp8)
    offsets, out = cu([100, 200, 150]), torch.zeros(rows, heads * D, dtype=torch.bfloat16, device="cuda")
    call = dict(cu_seqlens=offsets, k_scale=ks, v_scale=vs, O=out, workspace=ws)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        fl.attention_prefill(q, k, v, **call)
    torch.cuda.current_stream().wait_stream(s)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fl.attention_prefill(q, k, v, **call)
    for lens in ([100, 200, 150], [1, 0, 499], [300, 130, 3]):
        offsets.copy_(cu(lens))
        q.copy_(randn(rows, heads * D, seed=lens[0]))
        for _ in range(3):
            g.replay()
        check_prefill(q, k, v, ks, vs, lens, out, True)
        small = prompt(60, heads, kv, fp8, seed=17)
        eager = fl.attention_prefill(small[0], small[1], small[2], k_scale=small[3], v_scale=small[4], workspace=ws)
        check_prefill(*small, [60], eager, True)
    assert fl.check_device_status(ws) == fl.FL_OK


def test_prefill_same_results_every_time():
    q, k, v, ks, vs = prompt(2000, 16, 4, True, seed=18)
    first = fl.attention_prefill(q, k, v, seq_len=700, k_scale=ks, v_scale=vs)
    for _ in range(5):
        assert torch.equal(first, fl.attention_prefill(q, k, v, seq_len=700, k_scale=ks, v_scale=vs))


def test_prefill_wait_that_runs_out():
    """With a limit of a microsecond the wait for a unit of work of some hundred microseconds (two heads of 65536
    tokens give every CTA three) gives up: the call ends, the status record says so, and after zeroing it the
    workspace serves again."""
    n = 65536
    q, k, v = (randn(n, 2 * D, seed=s) for s in (51, 52, 53))
    ws = fl.attention_prefill_workspace(n, 2, False)
    try:
        fl.set_wait_timeout_ns(1000)
        fl.attention_prefill(q, k, v, workspace=ws)
        status = fl.check_device_status(ws)
    finally:
        fl.set_wait_timeout_ns(0)
    assert status == fl.FL_ERR_TIMEOUT
    ws[:512] = 0
    out = fl.attention_prefill(q[:700], k[:700], v[:700], workspace=ws)
    check_prefill(q[:700], k[:700], v[:700], None, None, [700], out, True)
    assert fl.check_device_status(ws) == fl.FL_OK


# ---------------------------------------------------------------- decode
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,heads,kv,page", [
    ([1], 1, 1, 16), ([0], 4, 2, 16), ([17], 8, 1, 8), ([64, 63, 65, 0, 1], 8, 2, 64), ([300], 32, 8, 64),
    ([1000, 3], 6, 2, 1), ([511, 513], 7, 1, 7), ([200], 16, 1, 24), ([90, 91], 12, 1, 32), ([77], 40, 2, 16),
    ([4000], 4, 4, 128), ([129, 4097, 2], 5, 1, 256), ([100], 129, 1, 16), ([5000], 9, 9, 16)])
def test_decode_matches_the_definition(lens, heads, kv, page, fp8):
    c = Cache(lens, kv, page, fp8, seed=heads)
    q = randn(len(lens), heads * D, seed=1)
    check_decode(q, c, fl.attention_decode(q, *c.args(), **c.scales()))


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_large_ragged_batch(fp8):
    lens = [(37 * i * i + 11) % 1500 if i % 7 else i % 3 for i in range(200)]
    c = Cache(lens, 2, 16, fp8, seed=2)
    q = randn(len(lens), 8 * D, seed=2)
    check_decode(q, c, fl.attention_decode(q, *c.args(), **c.scales()))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("batch", [32, 33, 128, 129, 257])
def test_decode_batch_sizes(batch, fp8):
    """Around a warp's and a block's share of the lengths; most of the last sequences are short or empty."""
    lens = [300 if i % 31 == 0 else (i * 7) % 5 for i in range(batch - 1)] + [513]
    c = Cache(lens, 3, 16, fp8, seed=batch)
    q = randn(batch, 6 * D, seed=batch)
    check_decode(q, c, fl.attention_decode(q, *c.args(), **c.scales()))


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_wide_page_table(fp8):
    """A table so wide that the units of all lengths it allows pass 31 bits, with ordinary sequences in it."""
    lens, width = [700, 0, 65], 1 << 21
    c = Cache(lens, 32, 1024, fp8, seed=7, max_pages=width)
    q = randn(3, 64 * D, seed=7)
    check_decode(q, c, fl.attention_decode(q, *c.args(), **c.scales()))


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_long_sequence(fp8):
    c = Cache([70001], 2, 64, fp8, seed=3)
    q = randn(1, 8 * D, seed=3)
    check_decode(q, c, fl.attention_decode(q, *c.args(), **c.scales()))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("page", [16, 5, 64])
def test_decode_ignores_what_lies_behind_a_sequence(page, fp8):
    c = Cache([1, 20, 77, 0, 64], 2, page, fp8, seed=4, fill=NAN)
    q = randn(5, 8 * D, seed=4)
    check_decode(q, c, fl.attention_decode(q, *c.args(), **c.scales()))


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_reports_bad_entries(fp8):
    """Pages outside the cache, lengths outside the table: NaN rows and a status, nothing else touched; an
    entry behind the length is not looked at."""
    lens = [100, 700, 50, 20, 64, 10]
    c = Cache(lens, 2, 16, fp8, seed=5)
    c.table[0, 3] = c.pages
    c.table[1, 40] = -1
    c.table[2, 4] = 1 << 30  # position 64 and later: behind the length
    c.table[4, 4:] = -5
    c.seq_lens[3] = -4
    c.seq_lens[5] = c.table.shape[1] * 16 + 1
    q = randn(6, 8 * D, seed=5)
    ws = fl.attention_decode_workspace()
    out = fl.attention_decode(q, *c.args(), **c.scales(), workspace=ws)
    for b in (0, 1, 3, 5):
        assert out[b].isnan().all()
    check_decode(q, c, out, skip=(0, 1, 3, 5))
    assert fl.check_device_status(ws) == fl.FL_ERR_INVALID_ARG
    assert fl.check_device_status(ws) == fl.FL_OK
    good = Cache(lens, 2, 16, fp8, seed=6)
    check_decode(q, good, fl.attention_decode(q, *good.args(), **good.scales(), workspace=ws))
    assert fl.check_device_status(ws) == fl.FL_OK


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_non_finite_keys_and_values_in_use(fp8):
    """A NaN that the sequence does hold reaches its own heads only."""
    c = Cache([100, 90], 2, 16, fp8, seed=7)
    c.v[c.table[0, 2], 1, 3, 7] = 0x7F if fp8 else NAN
    q = randn(2, 8 * D, seed=7)
    out = fl.attention_decode(q, *c.args(), **c.scales())
    assert out[0].view(8, D)[4:, 7].isnan().all()
    assert out[0].view(8, D)[:4].isfinite().all() and out[1].isfinite().all()
    check_decode(q, c, out, skip=(0,))


def test_decode_wide_range_of_scales():
    """V's scales over many orders of magnitude, K's zero for some tokens, values and scale of zero."""
    c = Cache([600], 2, 32, True, seed=8)
    c.vs *= torch.exp(torch.randn(c.vs.shape, generator=torch.Generator().manual_seed(1)) * 4).cuda()
    c.ks[:, :, ::5] = 0.0
    c.vs[:, 1] = 0.0
    q = randn(1, 16 * D, seed=8)
    out = fl.attention_decode(q, *c.args(), **c.scales())
    check_decode(q, c, out)
    assert (out.view(16, D)[8:] == 0).all()


def test_decode_peaked_and_flat_rows():
    for std, seed in ((60.0, 9), (0.0, 10)):
        for fp8 in (False, True):
            c = Cache([1500, 40], 2, 16, fp8, seed=seed)
            q = randn(2, 8 * D, seed=seed, std=std)
            check_decode(q, c, fl.attention_decode(q, *c.args(), **c.scales()))


def test_decode_small_queries():
    """Queries of 1e-20 and 1e20: no intermediate type may narrow their range."""
    for std in (1e-20, 1e20):
        for fp8 in (False, True):
            c = Cache([150], 1, 16, fp8, seed=11)
            q = randn(1, 4 * D, seed=11, std=std)
            check_decode(q, c, fl.attention_decode(q, *c.args(), **c.scales(), scale=0.1 / std), scale=0.1 / std)


def test_decode_strides_and_shared_pages():
    """Keys and values as halves of one allocation, table and queries as parts of wider tensors, two
    sequences with a common prefix."""
    lens, kv, page = [100, 130, 100], 2, 16
    for fp8 in (False, True):
        c = Cache(lens, kv, page, fp8, seed=12)
        both = torch.zeros((c.pages, 2) + c.k.shape[1:], dtype=c.k.dtype, device="cuda")
        both[:, 0], both[:, 1] = c.k, c.v
        c.k, c.v = both[:, 0], both[:, 1]
        if fp8:
            sc = torch.stack((c.ks, c.vs), 1).contiguous()
            c.ks, c.vs = sc[:, 0], sc[:, 1]
        c.table[2, :4] = c.table[0, :4]
        wide = torch.full((3, c.table.shape[1] + 5), -1, dtype=torch.int32, device="cuda")
        wide[:, 2:2 + c.table.shape[1]] = c.table
        c.table = wide[:, 2:2 + c.table.shape[1]]
        q = randn(3, 8 * D + 16, seed=12)[:, 8:8 + 8 * D]
        out = torch.full((3, 8 * D + 8), 5.0, dtype=torch.bfloat16, device="cuda")
        fl.attention_decode(q, *c.args(), **c.scales(), O=out[:, :8 * D])
        check_decode(q, c, out[:, :8 * D])
        assert (out[:, 8 * D:] == 5.0).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_captured_replayed_and_reused(fp8):
    """One graph over growing sequences; the workspace also serves other shapes between, and the results do
    not depend on the run."""
    c = Cache([3000, 900, 2500, 1], 2, 16, fp8, seed=13)
    q = randn(4, 8 * D, seed=13)
    ws, out = fl.attention_decode_workspace(), torch.empty_like(q)
    fl.attention_decode(q, *c.args(), **c.scales(), O=out, workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fl.attention_decode(q, *c.args(), **c.scales(), O=out, workspace=ws)
    other = Cache([5, 800] * 40, 1, 32, fp8, seed=14)
    qo = randn(80, 16 * D, seed=14)
    for lens in ([1, 1, 1, 1], [100, 899, 2500, 0], [3000, 900, 1700, 1]):
        c.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        c.lens = lens
        g.replay()
        check_decode(q, c, out)
        again = out.clone()
        g.replay()
        assert torch.equal(out, again)
        check_decode(qo, other, fl.attention_decode(qo, *other.args(), **other.scales(), workspace=ws))
    assert fl.check_device_status(ws) == fl.FL_OK


def test_calls_on_two_streams_at_once():
    c = [Cache([2000, 50 + i], 4, 16, bool(i), seed=15 + i) for i in range(2)]
    q = [randn(2, 16 * D, seed=15 + i) for i in range(2)]
    p = [prompt(600, 8, 2, bool(i), seed=17 + i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                outs[i].append((fl.attention_decode(q[i], *c[i].args(), **c[i].scales()),
                                fl.attention_prefill(*p[i][:3], k_scale=p[i][3], v_scale=p[i][4])))
    torch.cuda.synchronize()
    for i in range(2):
        for d, f in outs[i]:
            check_decode(q[i], c[i], d)
            check_prefill(*p[i], [600], f, True)


@pytest.mark.parametrize("fp8", [False, True])
def test_stream_given_without_workspace_or_output(fp8):
    """What a call makes itself belongs to the stream it is given: the current stream is busy, the other one is not."""
    c = Cache([3000, 70], 2, 16, fp8, seed=60)
    q = randn(2, 8 * D, seed=60)
    p = prompt(500, 8, 2, fp8, seed=61)
    offsets, other = cu([300, 200]), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        for _ in range(4):
            junk = torch.full((64 << 20,), 255, dtype=torch.uint8, device="cuda")  # memory that is given out again
            del junk
            torch.cuda._sleep(2000000)
            out = fl.attention_decode(q, *c.args(), **c.scales(), stream=other)
            whole = fl.attention_prefill(p[0], p[1], p[2], cu_seqlens=offsets, k_scale=p[3], v_scale=p[4], stream=other)
            other.synchronize()
            check_decode(q, c, out)
            check_prefill(*p, [300, 200], whole, True)


# ---------------------------------------------------------------- append
def place(cache, b, pos, pages):
    at, slot = cache.table[b].long()[pos // cache.page], pos % cache.page
    return pages[at, :, slot]


@pytest.mark.parametrize("rows8,cache8", [(False, False), (True, True), (False, True)])
@pytest.mark.parametrize("page,kv", [(16, 8), (7, 1), (64, 3), (1, 2)])
def test_append_puts_rows_in_their_slots(page, kv, rows8, cache8):
    before, new = [0, 5, 40, 16, 9], [33, 1, 0, 17, 100]
    c = Cache([a + n for a, n in zip(before, new)], kv, page, cache8, seed=20)
    T = sum(new)
    k, v = randn(T + 6, kv * D, seed=21), randn(T + 6, kv * D, seed=22)
    k[3], v[5, :D] = 0, 0
    k[7, 3] = 1e-30
    ks = vs = None
    if rows8:
        (k, ks), (v, vs) = quantise(k.view(-1, kv, D)), quantise(v.view(-1, kv, D))
        k, v = k.view(-1, kv * D), v.view(-1, kv * D)
    old = [None if t is None else t.clone() for t in (c.k, c.v, c.ks, c.vs)]
    fl.paged_kv_append(k, v, *c.args(), cu_seqlens=cu(new), k_scale=ks, v_scale=vs, **c.scales())
    if cache8 and not rows8:
        (k, ks), (v, vs) = quantise(k.view(-1, kv, D)), quantise(v.view(-1, kv, D))
    first = 0
    for b, n in enumerate(new):
        pos = torch.arange(before[b], before[b] + n, device="cuda")
        for pages, was, rows in ((c.k, old[0], k), (c.v, old[1], v), (c.ks, old[2], ks), (c.vs, old[3], vs)):
            if pages is None:
                continue
            want = rows[first:first + n].reshape(n, kv, *pages.shape[3:])
            assert torch.equal(place(c, b, pos, pages), want)
            at, slot = c.table[b].long()[pos // page], pos % page
            was[at, :, slot] = want
        first += n
    for pages, was in zip((c.k, c.v, c.ks, c.vs), old):  # everything else, rows behind the last sequence too
        assert pages is None or torch.equal(pages, was)


@pytest.mark.parametrize("std", [1.0, 1e-36, 1e30])
def test_append_quantises_to_the_nearest_code(std):
    """code * s is within half a step of the value: 2^-4 of it, or half of the smallest step 2^-9 s below the
    normal range (2^-6 s); one part in 2^20 more for the fp32 arithmetic of s and 448 / max."""
    kv, page = 2, 16
    c = Cache([64], kv, page, True, seed=19)
    k, v = randn(64, kv * D, seed=19, std=std), randn(64, kv * D, seed=18, std=std)
    fl.paged_kv_append(k, v, *c.args(), cu_seqlens=cu([64]), **c.scales())
    for got, want in zip(c.sequence(0), (k, v)):
        want = want.double().view(64, kv, D).transpose(0, 1)
        s = want.abs().amax(-1, keepdim=True) / 448.0
        tiny = 2.0 ** -149 * 448  # the scale itself may be subnormal
        assert_within(got, want, torch.maximum(want.abs() * 2.0 ** -4, s * 2.0 ** -10) * (1 + 2.0 ** -20) + tiny)


@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_append_quantises_rows_with_values_that_are_not_finite(bad):
    """NaN stays NaN and leaves the other codes of its head alone; an infinity takes its head's scale with it.  Heads of
    values near fp32's smallest beside ordinary ones keep their own factors."""
    kv, page = 5, 16
    c = Cache([40], kv, page, True, seed=50)
    k, v = randn(40, kv * D, seed=51), randn(40, kv * D, seed=52)
    k.view(40, kv, D)[::3, 1] *= 1e-36
    v.view(40, kv, D)[1::3, 4] *= 1e-37
    clean_k, clean_v = k.clone(), v.clone()
    for t, clean, row, head, d in ((k, clean_k, 3, 0, 5), (v, clean_v, 17, 4, 127), (v, clean_v, 18, 0, 64)):
        t.view(40, kv, D)[row, head, d] = bad
        clean.view(40, kv, D)[row, head, d] = 0
    fl.paged_kv_append(k, v, *c.args(), cu_seqlens=cu([40]), **c.scales())
    pos = torch.arange(40, device="cuda")
    for pages, scales, t, clean in ((c.k, c.ks, k, clean_k), (c.v, c.vs, v, clean_v)):
        got, scale = place(c, 0, pos, pages), place(c, 0, pos, scales)
        spoiled = ~t.view(40, kv, D).isfinite()
        codes, want = quantise(clean.view(40, kv, D))
        if bad != bad:
            assert torch.equal(scale, want) and torch.equal(got[~spoiled], codes[~spoiled])
            assert (got[spoiled] & 0x7F == 0x7F).all()
        else:
            heads = spoiled.any(-1)
            assert (scale[heads] == INF).all() and torch.equal(scale[~heads], want[~heads])
            assert torch.equal(got[~heads], codes[~heads])


def test_append_one_token_each_with_strides():
    """Decode steps: no offsets, rows as columns of a projection's output, the cache as halves of one block."""
    kv, page = 2, 16
    c = Cache([1, 16, 17, 300], kv, page, False, seed=23)
    both = torch.zeros((c.pages, 2) + c.k.shape[1:], dtype=torch.bfloat16, device="cuda")
    c.k, c.v = both[:, 0], both[:, 1]
    wide = randn(4, 2 * kv * D + 64, seed=24)
    k, v = wide[:, 32:32 + kv * D], wide[:, 64 + kv * D:]
    fl.paged_kv_append(k, v, *c.args())
    for b, n in enumerate(c.lens):
        pos = torch.tensor([n - 1], device="cuda")
        assert torch.equal(place(c, b, pos, c.k)[0], k[b].view(kv, D))
        assert torch.equal(place(c, b, pos, c.v)[0], v[b].view(kv, D))
    assert int((both != 0).any(-1).sum()) == 4 * 2 * kv


def test_append_ignores_rows_without_a_place():
    """Lengths of zero, positions behind the table and pages outside the cache: nothing is written."""
    kv, page = 2, 16
    c = Cache([20, 20, 20, 20], kv, page, False, seed=25)
    c.seq_lens.copy_(torch.tensor([0, 33, 20, 20], dtype=torch.int32))
    c.table[2, 1], c.table[3, 1] = c.pages, -1
    k, v = randn(4, kv * D, seed=26), randn(4, kv * D, seed=27)
    old = c.k.clone(), c.v.clone()
    fl.paged_kv_append(k, v, *c.args())
    torch.cuda.synchronize()
    assert torch.equal(c.k, old[0]) and torch.equal(c.v, old[1])


def test_append_captured_and_replayed():
    kv, page = 2, 16
    c = Cache([64, 64], kv, page, True, seed=28)
    k, v = randn(2, kv * D, seed=29), randn(2, kv * D, seed=30)
    c.seq_lens.fill_(1)
    fl.paged_kv_append(k, v, *c.args(), **c.scales())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fl.paged_kv_append(k, v, *c.args(), **c.scales())
    for n in (1, 2, 16, 17, 64):
        c.seq_lens.fill_(n)
        k.copy_(randn(2, kv * D, seed=n))
        g.replay()
        codes, scale = quantise(k.view(2, kv, D))
        for b in range(2):
            pos = torch.tensor([n - 1], device="cuda")
            assert torch.equal(place(c, b, pos, c.k)[0], codes[b]) and torch.equal(place(c, b, pos, c.ks)[0], scale[b])


# ---------------------------------------------------------------- together
@pytest.mark.parametrize("fp8", [False, True])
def test_projection_prompt_and_decode_steps(fp8):
    """Prompts through the QKV projection, the cache and the prefill attention, then token after token through
    projection, append and decode attention: each step equals the attention of the whole sequence over the
    same keys and values."""
    heads, kv, width, page = 8, (2 if fp8 else 8), 512, 16
    lens, steps = [37, 130, 1], 4
    rows, batch = sum(lens), len(lens)
    n_w = (heads + 2 * kv) * D
    W, X = randn(n_w, width, seed=31, std=width ** -0.5), randn(rows, width, seed=32)
    pos = torch.cat([torch.arange(n) for n in lens]).to(torch.int32).cuda()

    def project(x, positions):
        if fp8:
            return fl.fused_qkv_rope_fp8kv(x, W, None, heads, kv, D, positions=positions)
        return (*fl.fused_qkv_rope(x, W, None, heads, D, positions=positions), None, None)

    q, k, v, ks, vs = project(X, pos)
    out = fl.attention_prefill(q, k, v, cu_seqlens=cu(lens), k_scale=ks, v_scale=vs)
    check_prefill(q, k, v, ks, vs, lens, out, True)
    c = Cache([n + steps for n in lens], kv, page, fp8, seed=33, fill=NAN)
    c.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
    fl.paged_kv_append(k, v, *c.args(), cu_seqlens=cu(lens), k_scale=ks, v_scale=vs, **c.scales())
    ws = fl.attention_decode_workspace()
    for t in range(steps):
        c.seq_lens += 1
        c.lens = [n + t + 1 for n in lens]
        q, k, v, ks, vs = project(randn(batch, width, seed=40 + t), c.seq_lens - 1)
        fl.paged_kv_append(k, v, *c.args(), k_scale=ks, v_scale=vs, **c.scales())
        out = fl.attention_decode(q, *c.args(), **c.scales(), workspace=ws)
        check_decode(q, c, out, what=f"step {t}")
        for b in range(batch):  # the newest entry is the projection's
            kk, vv = c.sequence(b)
            assert torch.equal(kk[:, -1], values(k[b].view(kv, D), None if ks is None else ks[b]))
            assert torch.equal(vv[:, -1], values(v[b].view(kv, D), None if vs is None else vs[b]))
    assert fl.check_device_status(ws) == fl.FL_OK and fl.device_status() == fl.FL_OK


@pytest.mark.parametrize("fp8", [False, True])
def test_workspace_serves_on_after_waits_that_ran_out(fp8):
    """Calls that gave up leave nothing behind that the next one would trip over, though nobody zeroes the workspace: it
    works off all of its tiles (more than there are CTAs)."""
    n, m = 65536, 24000
    q, k, v, ks, vs = prompt(n, 2, 2, fp8, seed=54)
    ws = fl.attention_prefill_workspace(n, 2, fp8)
    cut = (q[:m], k[:m], v[:m])
    scales = dict(k_scale=ks[:m], v_scale=vs[:m]) if fp8 else {}
    want = fl.attention_prefill(*cut, **scales)
    for times in (1, 2):
        try:
            fl.set_wait_timeout_ns(1000)
            for _ in range(times):
                fl.attention_prefill(q, k, v, k_scale=ks, v_scale=vs, workspace=ws)
            status = fl.check_device_status(ws)
        finally:
            fl.set_wait_timeout_ns(0)
        assert status == fl.FL_ERR_TIMEOUT
        for _ in range(2):
            out = torch.full((m, 2 * D), 7.0, dtype=torch.bfloat16, device="cuda")
            fl.attention_prefill(*cut, **scales, O=out, workspace=ws)
            assert torch.equal(out, want)
        assert fl.check_device_status(ws) == fl.FL_OK


@pytest.mark.parametrize("heads,kv", [(4, 4), (8, 2), (24, 2)])
def test_decode_weights_over_a_bf16_cache_keep_sixteen_bits(heads, kv):
    """Sequences of two keys whose second value all but cancels the first one in the first head of each group: v_2 is
    -p_1 v_1 / p_2 rounded to bf16, so |o| <= 2^-8 p_1 |v_1| and the output's rounding hides nothing.  Weights in two bf16
    terms move o by 2^-16 A; in one, by up to 2^-8 A, forty times what is allowed here."""
    batch, group = 64, heads // kv
    c = Cache([2] * batch, kv, 16, False, seed=62)
    q = randn(batch, heads * D, seed=63, std=0.25)
    for b in range(batch):
        k, v = c.sequence(b)
        x = torch.einsum("hd,htd->ht", q[b].view(kv, group, D)[:, 0].double(), k) * D ** -0.5
        p = torch.softmax(x, -1)
        c.v[c.table[b, 0].long(), :, 1] = (-p[:, :1] * v[:, 0] / p[:, 1:]).bfloat16()
    out = fl.attention_decode(q, *c.args())
    for b in range(batch):
        k, v = c.sequence(b)
        ref, tol = attend(q[b].double().view(heads, 1, D), k, v, D ** -0.5, 2.0 ** -16)
        assert_within(out[b].view(heads, 1, D)[::group], ref[::group], tol[::group], f"sequence {b}")
        assert_within(out[b].view(heads, 1, D), ref, tol, f"sequence {b}, all heads")
