"""paged_kv_append_int4 and paged_kv_read on the host (no GPU needed): what they refuse before the device is touched, through
the C ABI and through the binding; and the arithmetic of the 4-bit codes, exhaustively."""
import ctypes

import pytest
import torch

import gemm_epilogue_tcgen05_gb300 as fl
from gemm_epilogue_tcgen05_gb300 import build as cuda_build

P = ctypes.c_void_p
A = P(0x10000)
OK, INVALID, UNSUPPORTED, ALIGNMENT = fl.FL_OK, fl.FL_ERR_INVALID_ARG, fl.FL_ERR_UNSUPPORTED, fl.FL_ERR_ALIGNMENT


@pytest.fixture(scope="module")
def lib():
    cuda_build.build()
    return fl.load()


def call(fn, defaults, **changes):
    args = dict(defaults)
    assert set(changes) <= set(args)
    args.update(changes)
    return fn(*args.values())


APPEND = dict(K=A, V=A, kp=A, vp=A, kps=A, vps=A, table=A, lens=A, cu=A, T=10, batch=4, n_kv=2, head_dim=128, page=16,
              pages=9, max_pages=5, ldkv=256, ldt=5, pitch=16 * 128, spitch=128, stream=None)
READ = dict(kp=A, vp=A, kps=A, vps=A, table=A, lens=A, cu=A, K=A, V=A, T=10, batch=4, n_kv=2, head_dim=128, page=16,
            pages=9, max_pages=5, ldkv=256, ldt=5, pitch=16 * 128, spitch=128, cache=3, stream=None)

BOTH = [
    (INVALID, dict(T=-1)), (INVALID, dict(batch=-1)), (INVALID, dict(n_kv=-1)), (INVALID, dict(page=0)),
    (INVALID, dict(pages=-1)), (INVALID, dict(max_pages=-1)), (UNSUPPORTED, dict(head_dim=64)),
    (UNSUPPORTED, dict(n_kv=65537)), (INVALID, dict(K=None)), (INVALID, dict(V=None)), (INVALID, dict(kp=None)),
    (INVALID, dict(vp=None)), (INVALID, dict(kps=None)), (INVALID, dict(vps=None)), (INVALID, dict(table=None)),
    (INVALID, dict(lens=None)), (INVALID, dict(cu=None)), (INVALID, dict(ldkv=248)), (INVALID, dict(ldt=4)),
    (INVALID, dict(pitch=16 * 128 - 16)), (INVALID, dict(spitch=124)), (ALIGNMENT, dict(K=P(0x10008))),
    (ALIGNMENT, dict(vp=P(0x10008))), (ALIGNMENT, dict(ldkv=260)), (ALIGNMENT, dict(pitch=16 * 128 + 8)),
    (ALIGNMENT, dict(kps=P(0x10004))), (ALIGNMENT, dict(vps=P(0x10002))), (ALIGNMENT, dict(spitch=130)),
    (ALIGNMENT, dict(table=P(0x10002))), (ALIGNMENT, dict(lens=P(0x10001))), (ALIGNMENT, dict(cu=P(0x10001))),
    (OK, dict(T=0, K=None, V=None)), (OK, dict(batch=0, lens=None)), (OK, dict(n_kv=0))]


@pytest.mark.parametrize("status,changes", BOTH)
def test_append_checks(lib, status, changes):
    assert call(lib.paged_kv_append_int4, APPEND, **changes) == status


@pytest.mark.parametrize("status,changes", BOTH + [
    (INVALID, dict(cache=0)), (INVALID, dict(cache=4)), (INVALID, dict(cache=2, spitch=31)), (INVALID, dict(cache=1)),
    (ALIGNMENT, dict(cache=1, pitch=16 * 256 + 4)), (ALIGNMENT, dict(cache=2, pitch=16 * 256, kps=P(0x10002)))])
def test_read_checks(lib, status, changes):
    assert call(lib.paged_kv_read, READ, **changes) == status


def test_other_calls_refuse_the_type(lib):
    """The calls that know bf16 and E4M3 caches."""
    dev = torch.device("cpu")
    c = torch.zeros(3, 2, 16, 64, dtype=torch.uint8, device=dev)
    t = torch.zeros(4, 256, dtype=torch.bfloat16)
    table, lens = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    s = torch.zeros(3, 2, 16, 4, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fl.attention_decode(t, c, c, table, lens, k_page_scale=s, v_page_scale=s)
    with pytest.raises(ValueError):
        fl.paged_kv_append(t, t, c, c, table, lens, k_page_scale=s, v_page_scale=s)


@pytest.mark.parametrize("change", [
    dict(K=torch.zeros(4, 256)), dict(K=torch.zeros(4, 128, dtype=torch.bfloat16)), dict(kps=None),
    dict(kps=torch.zeros(3, 2, 16, 4)), dict(vps=torch.zeros(3, 2, 16, 2, dtype=torch.bfloat16)),
    dict(kp=torch.zeros(3, 2, 16, 128, dtype=torch.uint8)), dict(vp=torch.zeros(3, 2, 8, 64, dtype=torch.uint8)),
    dict(kp=torch.zeros(3, 2, 16, 64, dtype=torch.int8)), dict(table=torch.zeros(3, 2, dtype=torch.int32)),
    dict(lens=torch.zeros(4, dtype=torch.int64)), dict(cu=torch.zeros(4, dtype=torch.int32))])
def test_binding_refuses(change):
    a = dict(K=torch.zeros(4, 256, dtype=torch.bfloat16), V=torch.zeros(4, 256, dtype=torch.bfloat16),
             kp=torch.zeros(3, 2, 16, 64, dtype=torch.uint8), vp=torch.zeros(3, 2, 16, 64, dtype=torch.uint8),
             kps=torch.zeros(3, 2, 16, 4, dtype=torch.bfloat16), vps=torch.zeros(3, 2, 16, 4, dtype=torch.bfloat16),
             table=torch.zeros(4, 2, dtype=torch.int32), lens=torch.zeros(4, dtype=torch.int32), cu=None)
    a.update(change)
    with pytest.raises(ValueError):
        fl.paged_kv_append_int4(a["K"], a["V"], a["kp"], a["vp"], a["kps"], a["vps"], a["table"], a["lens"], cu_seqlens=a["cu"])
    with pytest.raises(ValueError):
        fl.paged_kv_read(a["kp"], a["vp"], a["table"], a["lens"], cu_seqlens=a["cu"], k_page_scale=a["kps"],
                         v_page_scale=a["vps"], K=a["K"], V=a["V"])


def test_the_scale_by_a_product_is_that_by_a_quotient():
    """a * fl(1/7), rounded to five significant bits, is a / 7 rounded to them, for every significand of a bf16 number."""
    a = torch.arange(128, 256).float()
    third = torch.tensor(1.0 / 7.0, dtype=torch.float32)
    b = (a * third).view(torch.int32)
    got = (((b + 0x3FFFF + ((b >> 19) & 1)) >> 19) << 19).view(torch.float32).double()
    m, e = torch.frexp(a.double() / 7)
    assert torch.equal(got, torch.ldexp(torch.round(m * 32), e - 5))
    assert (7 * got < 256).all()  # the largest entry of a group stays in bf16's range


def test_the_codes_by_a_product_are_those_by_a_quotient():
    """(y * fl(1/s) + 768) + (3 * 2^22 - 768), each sum rounded once, is 3 * 2^22 plus y / s rounded to the nearest even
    whole number, for every significand of y and s where |y / s| is at most 7 * 33/32 (fma emulated in 64 bits: the product of
    two fp32 numbers is exact there, and so is its sum with 768 to 2^-29)."""
    y = torch.cat([torch.arange(128, 256).double() * 2.0 ** e for e in range(-8, 1)])[:, None]
    s = torch.arange(16, 32).double()[None] * 2
    y, s = torch.broadcast_tensors(y, s)
    r = (1.0 / s).float()
    q = y / s
    keep = q <= 7 * 33 / 32
    t = (y * r.double() + 768.0).float()
    u = t + torch.tensor(12582912.0 - 768.0, dtype=torch.float32)
    got = u.view(torch.int32) - 0x4B400000
    assert torch.equal(got[keep].double(), torch.round(q[keep])) and int(keep.sum()) > 5000
