"""attention_prefill on E4M3 rows whose scales of V are far apart, against the definition in 64 bits.

The tolerance is the definition's, it knows nothing of how the kernel groups keys.  With p_j the weights of a row (their
sum 1), s_j the scales of V and c_j its codes:
- the output is rounded to bf16 (2^-8 |o|), logits and sums as attention_utils derives them; the keys are taken as rounded
  to bf16;
- values become fp16 times 2^-b_j with 2^-6 <= s_j 2^-b_j < 2^7: the smallest code, 2^-9, is 2^-15 at least there, and
  half a step of fp16's smallest numbers, 2^-25, is 2^-10 of it; larger ones lose less;
- weights become fp16: 2^-11 of each, or half a step of the smallest numbers, 2^-25.  They carry their key's 2^b_j there
  and the largest of a row is held at 2^7 at least.  So the latter moves a weight by at most
  2^-32 2^-b_j max_i(p_i 2^b_i) <= 2^-26 2^-b_j max_i(p_i s_i), and o by 2^-26 max_i(p_i s_i) times the sum of
  |c_j| s_j 2^-b_j <= 2^7 |c_j| over the keys that the row sees: 2^-19 max_i(p_i s_i) sum_j |c_j|.
"""
import pytest
import torch

import gemm_epilogue_tcgen05_gb300 as fl
from attention_utils import D, F16, assert_within, attend, cu, quantise, rounded, values

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


def randn(*shape, seed=0, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * std).bfloat16().cuda()


def prompt(rows, heads, kv, seed=0):
    q, k, v = randn(rows, heads * D, seed=seed), randn(rows, kv, D, seed=seed + 1), randn(rows, kv, D, seed=seed + 2)
    (k, ks), (v, vs) = quantise(k), quantise(v)
    return q, k.view(rows, -1), v.view(rows, -1), ks, vs


def looks_at(k, ks, at, strength=8.0):
    """Queries (one head for each kv head) that single out key at[i] of their sequence."""
    n, kv = ks.shape
    return (strength * values(k.view(n, kv, D), ks)[at]).bfloat16().view(n, kv * D)


def check(q, k, v, ks, vs, out, causal, rows=None, what=""):
    """One sequence; rows: only these (all of them see finite keys and values only)."""
    n, kv = vs.shape
    heads = q.shape[1] // D
    kk = rounded(values(k.reshape(n, kv, D), ks)).transpose(0, 1)
    vv = values(v.reshape(n, kv, D), vs).transpose(0, 1)
    qq = q.double().reshape(n, heads, D).transpose(0, 1)
    ref, tol = attend(qq, kk, vv, D ** -0.5, 3 * F16, causal)
    g = heads // kv
    codes = v.reshape(n, kv, D).view(torch.float8_e4m3fn).double()
    x = qq @ kk.repeat_interleave(g, 0).transpose(1, 2) * D ** -0.5
    seen = torch.ones(n, n, dtype=torch.double, device=q.device)
    if causal:
        seen = seen.tril()
        x = x.masked_fill(seen == 0, -INF)
    largest = (torch.softmax(x, -1) * vs.double().T.repeat_interleave(g, 0)[:, None]).amax(-1, keepdim=True)
    tol += 2.0 ** -19 * largest * (seen @ codes.abs().transpose(0, 1).repeat_interleave(g, 0))
    got = out.view(n, heads, D).transpose(0, 1)
    rows = slice(None) if rows is None else rows
    assert_within(got[:, rows], ref[:, rows], tol[:, rows], what)


def run_and_check(q, k, v, ks, vs, what=""):
    for causal in (True, False):
        out = fl.attention_prefill(q, k, v, k_scale=ks, v_scale=vs, causal=causal)
        check(q, k, v, ks, vs, out, causal, what=f"{what} causal {causal}")


# ---------------------------------------------------------------- tiles whose values are all zero
@pytest.mark.parametrize("std", [1.0, 1e-2, 1e-4, 1e-5, 1e-8])
@pytest.mark.parametrize("first", [0, 128, 256])
def test_a_run_of_keys_without_values(first, std):
    """128 keys with values of zero (scale 0) before, between and behind small ones that other keys carry."""
    n = 384
    q, k, v, ks, vs = prompt(n, 4, 2, seed=100)
    vs *= std
    gone = slice(first, first + 128)
    v[gone], vs[gone] = 0, 0.0
    run_and_check(q, k, v, ks, vs)
    # rows that look at the zeros, by some 80 in the exponent, and rows that look past them
    at = torch.arange(n, device="cuda")
    run_and_check(looks_at(k, ks, torch.where(at % 2 == 0, at, (at - 140).clamp(min=0))), k, v, ks, vs)


def test_no_values_at_all():
    q, k, v, ks, vs = prompt(300, 4, 1, seed=101)
    vs[:] = 0.0
    for causal in (True, False):
        assert (fl.attention_prefill(q, k, v, k_scale=ks, v_scale=vs, causal=causal) == 0).all()


# ---------------------------------------------------------------- keys whose scale is far from the others' of their tile
@pytest.mark.parametrize("factor", [2.0 ** 12, 2.0 ** 28, 2.0 ** 32, 2.0 ** 40, 1e30])
@pytest.mark.parametrize("at", [5, 120, 127, 128, 200])
def test_a_later_scale_reaches_no_earlier_row(at, factor):
    """A huge scale of a key's values: rows before it are what they are without it, to the rounding."""
    n = 260
    q, k, v, ks, vs = prompt(n, 4, 2, seed=110)
    vs[at, 0] *= factor
    out = fl.attention_prefill(q, k, v, k_scale=ks, v_scale=vs)
    c = slice(0, at)
    check(q[c], k[c], v[c], ks[c], vs[c], out[c], True)
    check(q, k, v, ks, vs, out, True)


@pytest.mark.parametrize("factor", [2.0 ** -40, 2.0 ** -13, 2.0 ** -11, 0.0, 2.0 ** 11, 2.0 ** 13, 2.0 ** 16, 2.0 ** 40])
@pytest.mark.parametrize("which", [[0], [0, 1, 127, 128], [130, 131, 255, 256], [299], list(range(0, 300, 3))])
def test_single_keys_far_from_the_others(which, factor):
    """Some keys' scales far above or below the rest of their tile, from one key to a third of all, around tile borders.
    Every row looks at its own key or at one before it by some 80 in the exponent, or at nothing in particular, so each
    kind of key counts for somebody."""
    n = 300
    q, k, v, ks, vs = prompt(n, 2, 2, seed=111)
    vs[which] *= factor
    if factor == 0.0:
        v[which] = 0
    i = torch.arange(n, device="cuda")
    run_and_check(q, k, v, ks, vs, "even")
    run_and_check(looks_at(k, ks, i), k, v, ks, vs, "own")
    run_and_check(looks_at(k, ks, (i - 1 - i % 5).clamp(min=0)), k, v, ks, vs, "near")
    run_and_check(looks_at(k, ks, (i // 2)), k, v, ks, vs, "far")


def test_a_key_that_is_hardly_looked_at():
    """One key whose scale is 2^40 times the others' and whose logit is far below; another key of its tile is looked at a
    little less than the keys of the tile behind."""
    n, big, other, main = 256, 60, 90, 200
    q, k, v, ks, vs = prompt(n, 1, 1, seed=112)
    vs[big] *= 2.0 ** 40
    kk = values(k.view(n, 1, D), ks)[:, 0]
    for part in (0.5, 0.8, 0.95):
        mix = torch.linalg.lstsq(kk[[big, other, main]].cpu(),
                                 torch.tensor([-300.0, part * 400.0, 400.0], dtype=torch.double, device="cpu"),
                                 driver="gelsd").solution.cuda()
        run_and_check(mix.bfloat16()[None].repeat(n, 1), k, v, ks, vs, f"part {part}")


@pytest.mark.parametrize("heads,kv,n", [(1, 1, 1), (4, 4, 3), (5, 5, 130), (24, 4, 270), (70, 35, 140), (33, 33, 40)])
def test_scales_over_many_orders_of_magnitude(heads, kv, n):
    """Scales of V spread over some 2^+-25, different for every head, zeros among them; more heads than a block converts."""
    q, k, v, ks, vs = prompt(n, heads, kv, seed=113)
    vs *= torch.exp2(torch.randn(vs.shape, generator=torch.Generator().manual_seed(1)) * 8).cuda()
    vs.view(-1)[::7] = 0.0
    run_and_check(q, k, v, ks, vs)


def test_many_sequences_with_scales_apart():
    """Short and long sequences beside one another, wide tiles in some of them only, rows behind the last one."""
    lens = [1, 128, 129, 0, 5, 400, 127, 2, 260, 64]
    rows = sum(lens)
    q, k, v, ks, vs = prompt(rows + 9, 4, 2, seed=114)
    vs[0] *= 2.0 ** 30
    vs[1:129:50, 1] *= 2.0 ** 30
    vs[270:300] *= 2.0 ** -30
    vs[rows - 64] = 0.0
    vs[rows:] = NAN
    for causal in (True, False):
        out = fl.attention_prefill(q, k, v, cu_seqlens=cu(lens), k_scale=ks, v_scale=vs, causal=causal)
        first = 0
        for b, n in enumerate(lens):
            r = slice(first, first + n)
            if n:
                check(q[r], k[r], v[r], ks[r], vs[r], out[r], causal, what=f"sequence {b} causal {causal}")
            first += n
        assert (out[rows:] == 0).all()


def test_codes_that_are_not_a_number_under_scales_apart():
    """NaN in a key whose scale is far from the others' reaches the rows that see it, in its dimension, and no other."""
    n, at = 200, 70
    for factor in (2.0 ** 30, 2.0 ** -30, 0.0):
        q, k, v, ks, vs = prompt(n, 2, 1, seed=115)
        vs[at] *= factor
        v[at, 9] = 0x7F
        out = fl.attention_prefill(q, k, v, k_scale=ks, v_scale=vs)
        c = slice(0, at)
        check(q[c], k[c], v[c], ks[c], vs[c], out[c], True)
        assert out[at:].view(n - at, 2, D)[:, :, 9].isnan().all()
        keep = [d for d in range(D) if d != 9]
        assert out[at:].view(n - at, 2, D)[:, :, keep].isfinite().all()


@pytest.mark.parametrize("bad", [NAN, INF])
def test_scales_that_are_not_finite_beside_scales_apart(bad):
    n, at = 200, 90
    q, k, v, ks, vs = prompt(n, 2, 1, seed=116)
    vs[30] *= 2.0 ** 25
    vs[50] *= 2.0 ** -25
    vs[at] = bad
    out = fl.attention_prefill(q, k, v, k_scale=ks, v_scale=vs)
    c = slice(0, at)
    check(q[c], k[c], v[c], ks[c], vs[c], out[c], True)
    assert not out[at:].isfinite().all(-1).any()


def test_scales_apart_captured_and_replayed():
    """One graph whose tiles turn wide and ordinary again between replays; strided codes and scales."""
    n, heads, kv = 300, 4, 2
    q, k, v, ks, vs = prompt(n, heads, kv, seed=117)
    codes = torch.zeros(n, 2 * kv * D + 32, dtype=torch.uint8, device="cuda")
    scales = torch.full((n, 2 * kv + 1), NAN, device="cuda")
    k8, v8, ks8, vs8 = codes[:, 16:16 + kv * D], codes[:, 32 + kv * D:], scales[:, :kv], scales[:, kv + 1:]
    k8.copy_(k), v8.copy_(v), ks8.copy_(ks), vs8.copy_(vs)
    ws = fl.attention_prefill_workspace(n, kv, True)
    out = torch.empty_like(q)
    call = dict(k_scale=ks8, v_scale=vs8, O=out, workspace=ws)
    fl.attention_prefill(q, k8, v8, **call)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        fl.attention_prefill(q, k8, v8, **call)
    for rows, factor in (([], 1.0), ([3, 250], 2.0 ** 30), ([140], 2.0 ** -30), ([], 1.0), ([0], 0.0)):
        vs8.copy_(vs)
        vs8[rows] *= factor
        for _ in range(2):
            g.replay()
        check(q, k8, v8, ks8, vs8, out, True)
    assert fl.check_device_status(ws) == fl.FL_OK


# ---------------------------------------------------------------- tiles whose scales are far from one another
@pytest.mark.parametrize("apart", [60, 100, 130, 160])
@pytest.mark.parametrize("rising", [False, True])
def test_neighbouring_tiles_far_apart(apart, rising):
    """The scales of 128 keys and of those behind them 2^apart apart, around 1: both sides count for the rows that look at
    them, by some 130 powers of two, and the smaller side for those that look past the other one."""
    n = 300
    q, k, v, ks, vs = prompt(n, 2, 2, seed=120)
    step = torch.where(torch.arange(n, device="cuda") < 128, -1.0, 1.0) * (1 if rising else -1)
    vs *= torch.exp2(step * (apart // 2))[:, None]
    i = torch.arange(n, device="cuda")
    run_and_check(q, k, v, ks, vs, "even")
    run_and_check(looks_at(k, ks, i), k, v, ks, vs, "own")
    run_and_check(looks_at(k, ks, (i - 140).clamp(min=0)), k, v, ks, vs, "before")
    run_and_check(looks_at(k, ks, i, 2.0), k, v, ks, vs, "own, less so")


@pytest.mark.parametrize("exponent", [-142, -120, -80, -53, -46, 37, 44, 60, 100])
def test_scales_of_any_size(exponent):
    """All values of one size, down to subnormal scales and up to where bf16 still holds the output; and some of them only."""
    n = 200
    q, k, v, ks, vs = prompt(n, 2, 1, seed=121)
    big = vs * 2.0 ** exponent
    small = vs.clone()
    small[40:60] = big[40:60]
    for scales in (big, small):
        run_and_check(q, k, v, ks, scales, str(exponent))
        out = fl.attention_prefill(q, k, v, k_scale=ks, v_scale=scales)
        assert out.isfinite().all()


def test_large_outlier_hardly_looked_at_keeps_the_sum():
    """A key 2^100 times the others with weights from 2^-30 to 2^-200 of theirs: the sum of the weights is the others', the
    output the key's or theirs."""
    n, big = 256, 60
    q, k, v, ks, vs = prompt(n, 1, 1, seed=122)
    vs[big] *= 2.0 ** 100
    kk = values(k.view(n, 1, D), ks)[:, 0]
    u = kk[big] / kk[big].square().sum()
    for down in (20.0, 40.0, 70.0, 100.0, 140.0):
        row = (-(down / 1.4427) * D ** 0.5) * u
        run_and_check(row.bfloat16()[None].repeat(n, 1), k, v, ks, vs, f"2^-{down}")


# ---------------------------------------------------------------- many units of work
def test_single_keys_in_many_units():
    """Several units of work for each CTA, single keys in some of their tiles; the same results every time."""
    lens, heads, kv = [700, 650, 513, 700, 384, 699, 700, 640, 100, 700], 16, 4
    rows = sum(lens)
    q, k, v, ks, vs = prompt(rows, heads, kv, seed=130)
    pick = torch.rand(vs.shape, generator=torch.Generator().manual_seed(2)).cuda()
    vs[pick < 0.004] *= 2.0 ** 20
    vs[(pick > 0.004) & (pick < 0.008)] *= 2.0 ** -20
    vs[pick > 0.99] = 0.0
    offsets = cu(lens)
    for causal in (True, False):
        out = fl.attention_prefill(q, k, v, cu_seqlens=offsets, k_scale=ks, v_scale=vs, causal=causal)
        first = 0
        for b, n in enumerate(lens):
            r = slice(first, first + n)
            check(q[r], k[r], v[r], ks[r], vs[r], out[r], causal, what=f"sequence {b} causal {causal}")
            first += n
        for _ in range(3):
            assert torch.equal(out, fl.attention_prefill(q, k, v, cu_seqlens=offsets, k_scale=ks, v_scale=vs, causal=causal))


def test_single_keys_of_a_long_sequence():
    """Around the 32 key tiles whose powers a warp's lanes hold at a time."""
    n = 4500
    q, k, v, ks, vs = prompt(n, 1, 1, seed=131)
    for at, factor in ((0, 2.0 ** -20), (4000, 2.0 ** 20), (4095, 0.0), (4096, 2.0 ** -20), (4097, 2.0 ** 25), (4223, 0.0),
                       (4224, 2.0 ** 20), (4499, 2.0 ** -30)):
        vs[at] *= factor
    i = torch.arange(n, device="cuda")
    for q in (q, looks_at(k, ks, torch.where(i % 3 == 0, i, (i - 300).clamp(min=0)))):
        check(q, k, v, ks, vs, fl.attention_prefill(q, k, v, k_scale=ks, v_scale=vs), True)


def test_padded_batch():
    """Sequences of equal length that end in rows of zeros, the last one shorter."""
    n, real, seq = 700, 140, 200
    q, k, v, ks, vs = prompt(n, 8, 2, seed=132)
    at = torch.arange(n, device="cuda") % seq
    for t in (q, k, v, ks, vs):
        t[at >= real] = 0
    out = fl.attention_prefill(q, k, v, seq_len=seq, k_scale=ks, v_scale=vs)
    for first in range(0, n, seq):
        r = slice(first, min(first + seq, n))
        check(q[r], k[r], v[r], ks[r], vs[r], out[r], True)
        r = slice(first, min(first + real, n))
        check(q[r], k[r], v[r], ks[r], vs[r], out[r], True)


@pytest.mark.parametrize("apart", [1.0, 2.0 ** 20])
def test_large_logits(apart):
    """Logits of many hundreds, tiles of different powers, single keys: the maxima of O and of the sum move apart and on."""
    n = 500
    q, k, v, ks, vs = prompt(n, 2, 2, seed=133)
    q = (q.float() * 60).bfloat16()
    ks[400:] *= 3.0
    vs[128:256] *= 2.0 ** -6
    vs[300:310] *= apart
    run_and_check(q, k, v, ks, vs)
    rising = torch.linspace(0, 4, n, device="cuda")[:, None]
    run_and_check(q.abs(), k & 0x7F, v, ks * rising, vs)
