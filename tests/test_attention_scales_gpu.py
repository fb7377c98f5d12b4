"""attention_prefill on E4M3 rows whose scales of V are far apart, against the definition in 64 bits.

The tolerance is the definition's, it knows nothing of how the kernel groups keys.  With p_j the weights of a row (their
sum 1), s_j the scales of V and c_j its codes:
- the output is rounded to bf16 (2^-8 |o|), weights and values to fp16 (2^-11 each), logits and sums as attention_utils
  derives them; the keys are taken as rounded to bf16;
- a weight may also be lost below fp16's range, by half of its smallest step, 2^-25.  Weights carry a power of two of
  their key's scale there: 2^b_j, 2^-4 <= s_j 2^-b_j < 2^7, and the largest of a row is held at 2^7 at least.  So a weight
  moves by at most 2^-32 2^-b_j max_i(p_i 2^b_i) <= 2^-28 2^-b_j max_i(p_i s_i), and o by 2^-28 max_i(p_i s_i) times the
  sum of |c_j| s_j 2^-b_j <= 2^7 |c_j| over the keys that the row sees: 2^-21 max_i(p_i s_i) sum_j |c_j|.
"""
import pytest
import torch

import gemm_epilogue_tcgen05_gb300 as fl
from attention_utils import D, F16, assert_within, attend, quantise, rounded, values

pytestmark = pytest.mark.gpu
INF = float("inf")


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
    ref, tol = attend(qq, kk, vv, D ** -0.5, 2 * F16, causal)
    g = heads // kv
    codes = v.reshape(n, kv, D).view(torch.float8_e4m3fn).double()
    x = qq @ kk.repeat_interleave(g, 0).transpose(1, 2) * D ** -0.5
    seen = torch.ones(n, n, dtype=torch.double, device=q.device)
    if causal:
        seen = seen.tril()
        x = x.masked_fill(seen == 0, -INF)
    largest = (torch.softmax(x, -1) * vs.double().T.repeat_interleave(g, 0)[:, None]).amax(-1, keepdim=True)
    tol += 2.0 ** -21 * largest * (seen @ codes.abs().transpose(0, 1).repeat_interleave(g, 0))
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
