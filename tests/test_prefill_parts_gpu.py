"""Which calls of attention_prefill_window are cut along their keys."""
import pytest

import gemm_epilogue_tcgen05_gb300 as fl
from attention_utils import cu
from test_attention_window_gpu import check_prefill, keys_of, rows_of

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
