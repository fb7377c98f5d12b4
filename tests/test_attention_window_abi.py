"""attention_decode_window and attention_prefill_window on the host (no GPU needed): what they refuse before the device is
touched, through the C ABI and through the binding."""
import ctypes

import pytest
import torch

import gemm_epilogue_tcgen05_gb300 as fl
from gemm_epilogue_tcgen05_gb300 import build as cuda_build

P, F = ctypes.c_void_p, ctypes.c_float
A = P(0x10000)
OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = (fl.FL_OK, fl.FL_ERR_INVALID_ARG, fl.FL_ERR_UNSUPPORTED,
                                                  fl.FL_ERR_ALIGNMENT, fl.FL_ERR_WORKSPACE)


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return fl.load()


def call(fn, defaults, **changes):
    args = dict(defaults)
    assert set(changes) <= set(args)
    args.update(changes)
    return fn(*args.values())


DECODE = dict(Q=A, kp=A, vp=A, kps=A, vps=A, table=A, lens=A, O=A, batch=4, heads=8, n_kv=2, head_dim=128, page=16, pages=9,
              max_pages=5, ldq=1024, ldo=1024, ldt=5, pitch=16 * 128, spitch=128, scale=F(0.1), window=10, sinks=2, cache=3,
              ws=A, bytes=1 << 30, stream=None)
PREFILL = dict(Q=A, K=A, V=A, ks=None, vs=None, cu=A, cu_k=A, O=A, M=10, M_k=30, batch=2, heads=8, n_kv=2, head_dim=128,
               seq_len=0, ldq=1024, ldkv=256, lds=0, ldo=1024, scale=F(0.1), window=10, sinks=2, kv=1, ws=A, bytes=1 << 30,
               scratch=None, scratch_bytes=0, stream=None)


@pytest.mark.parametrize("status,changes", [
    (INVALID, dict(window=-1)), (INVALID, dict(sinks=-1)), (INVALID, dict(batch=-1)), (INVALID, dict(heads=-1)),
    (INVALID, dict(n_kv=0)), (INVALID, dict(n_kv=3)), (INVALID, dict(page=0)), (INVALID, dict(pages=-1)),
    (INVALID, dict(max_pages=-1)), (INVALID, dict(cache=0)), (INVALID, dict(cache=4)), (INVALID, dict(scale=F(0.0))),
    (INVALID, dict(scale=F(float("nan")))), (INVALID, dict(scale=F(3e38))), (UNSUPPORTED, dict(head_dim=64)),
    (UNSUPPORTED, dict(heads=131072)), (INVALID, dict(Q=None)), (INVALID, dict(O=None)), (INVALID, dict(kp=None)),
    (INVALID, dict(kps=None)), (INVALID, dict(vps=None)), (INVALID, dict(table=None)), (INVALID, dict(lens=None)),
    (INVALID, dict(ldq=1016)), (INVALID, dict(ldo=1016)), (INVALID, dict(ldt=4)), (INVALID, dict(pitch=16 * 128 - 16)),
    (INVALID, dict(spitch=124)), (INVALID, dict(cache=2, spitch=31)), (INVALID, dict(cache=1)),
    (ALIGNMENT, dict(Q=P(0x10004))), (ALIGNMENT, dict(O=P(0x10008))), (ALIGNMENT, dict(ldq=1028)),
    (ALIGNMENT, dict(kp=P(0x10008))), (ALIGNMENT, dict(kps=P(0x10004))), (ALIGNMENT, dict(spitch=129)),
    (ALIGNMENT, dict(lens=P(0x10002))), (ALIGNMENT, dict(ws=P(0x10010))), (WORKSPACE, dict(ws=None)),
    (WORKSPACE, dict(bytes=4096)), (OK, dict(batch=0, Q=None)), (OK, dict(heads=0, O=None))])
def test_decode_checks(lib, status, changes):
    assert call(lib.attention_decode_window, DECODE, **changes) == status


@pytest.mark.parametrize("status,changes", [
    (INVALID, dict(window=-1)), (INVALID, dict(sinks=-3)), (INVALID, dict(M=-1)), (INVALID, dict(M_k=-1)),
    (INVALID, dict(M_k=0)), (INVALID, dict(cu_k=None)), (INVALID, dict(cu=None, seq_len=5)), (INVALID, dict(cu=None)),
    (INVALID, dict(batch=-1)), (INVALID, dict(heads=-8)), (INVALID, dict(n_kv=3)), (INVALID, dict(n_kv=0)),
    (INVALID, dict(kv=0)), (INVALID, dict(kv=3)), (INVALID, dict(scale=F(-1.0))), (UNSUPPORTED, dict(head_dim=256)),
    (UNSUPPORTED, dict(heads=131072)), (INVALID, dict(Q=None)), (INVALID, dict(K=None)), (INVALID, dict(V=None)),
    (INVALID, dict(O=None)), (INVALID, dict(kv=2)), (INVALID, dict(ldq=1016)), (INVALID, dict(ldkv=248)),
    (INVALID, dict(kv=2, ks=A, vs=A, lds=1)), (ALIGNMENT, dict(Q=P(0x10008))), (ALIGNMENT, dict(ldkv=260)),
    (ALIGNMENT, dict(cu_k=P(0x10002))), (ALIGNMENT, dict(ws=P(0x10020))), (WORKSPACE, dict(ws=None)),
    (WORKSPACE, dict(bytes=100)), (WORKSPACE, dict(kv=2, ks=A, vs=A, lds=2, bytes=512 + 10 * 2 * 516)),
    (ALIGNMENT, dict(scratch=P(0x10008), scratch_bytes=1 << 20)),
    (OK, dict(M=0, Q=None)), (OK, dict(heads=0)), (OK, dict(batch=0))])
def test_prefill_checks(lib, status, changes):
    assert call(lib.attention_prefill_window, PREFILL, **changes) == status


def test_binding_refuses():
    """CPU tensors, negative spans and mismatched offsets are refused before anything else happens."""
    t = torch.zeros(4, 256, dtype=torch.bfloat16)
    k = torch.zeros(9, 256, dtype=torch.bfloat16)
    c = torch.zeros(3, 2, 16, 64, dtype=torch.uint8)
    s = torch.zeros(3, 2, 16, 4, dtype=torch.bfloat16)
    table, lens = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    offsets = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        fl.attention_decode_window(t, c, c, table, lens, k_page_scale=s, v_page_scale=s)
    with pytest.raises(ValueError):
        fl.attention_prefill_window(t, t, t)
    with pytest.raises(ValueError):
        fl.attention_prefill_window(t, k, k, cu_seqlens=offsets)
    with pytest.raises(ValueError):
        fl.attention_prefill_window(t, k, k, cu_seqlens_k=offsets)
    with pytest.raises(ValueError):
        fl.attention_prefill_window(t, k, k, cu_seqlens=offsets, cu_seqlens_k=lens)
    for bad in (-1, -(1 << 40)):
        with pytest.raises(ValueError):
            fl._span(bad, "window")
    assert fl._span(1 << 40, "window") == 0x7FFFFFFF and fl._span(7, "sinks") == 7


def test_build_checks_the_registers_of_both_prefill_sources():
    assert {"k_attention_prefill.cu", "k_attention_prefill_window.cu"} <= set(cuda_build.REGISTERS)
