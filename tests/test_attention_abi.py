"""The attention entry points on the host (no GPU needed): what they refuse before the device is touched,
through the C ABI and through the binding."""
import ctypes
import os

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


APPEND = dict(K=A, V=A, ks=None, vs=None, kp=A, vp=A, kps=None, vps=None, table=A, lens=A, cu=A, T=10, batch=4, n_kv=2,
              head_dim=128, page=16, pages=9, max_pages=5, ldkv=256, lds=0, ldt=5, pitch=16 * 256, spitch=0, row=1,
              cache=1, stream=None)
DECODE = dict(Q=A, kp=A, vp=A, kps=None, vps=None, table=A, lens=A, O=A, batch=4, heads=8, n_kv=2, head_dim=128, page=16,
              pages=9, max_pages=5, ldq=1024, ldo=1024, ldt=5, pitch=16 * 256, spitch=0, scale=F(0.1), cache=1, ws=A,
              bytes=1 << 30, stream=None)
PREFILL = dict(Q=A, K=A, V=A, ks=None, vs=None, cu=A, O=A, M=10, batch=2, heads=8, n_kv=2, head_dim=128, seq_len=0,
               ldq=1024, ldkv=256, lds=0, ldo=1024, scale=F(0.1), causal=1, kv=1, ws=A, bytes=1 << 30, stream=None)
FP8_CACHE = dict(kps=A, vps=A, spitch=32, cache=2)


@pytest.mark.parametrize("status,changes", [
    (INVALID, dict(T=-1)), (INVALID, dict(batch=-1)), (INVALID, dict(n_kv=-1)), (INVALID, dict(page=0)),
    (INVALID, dict(pages=-1)), (INVALID, dict(max_pages=-1)), (INVALID, dict(row=0)), (INVALID, dict(cache=3)),
    (UNSUPPORTED, dict(head_dim=64)),
    (UNSUPPORTED, dict(n_kv=65537)), (UNSUPPORTED, dict(row=2, ks=A, vs=A, lds=2)), (INVALID, dict(K=None)),
    (INVALID, dict(V=None)), (INVALID, dict(kp=None)), (INVALID, dict(vp=None)), (INVALID, dict(table=None)),
    (INVALID, dict(lens=None)), (INVALID, dict(cu=None)), (INVALID, dict(ldkv=248)), (INVALID, dict(ldt=4)),
    (INVALID, dict(pitch=16 * 256 - 8)), (INVALID, dict(cache=2)), (INVALID, dict(FP8_CACHE, spitch=31)),
    (INVALID, dict(FP8_CACHE, row=2)), (INVALID, dict(FP8_CACHE, row=2, ks=A, vs=A, lds=1)),
    (ALIGNMENT, dict(K=P(0x10008))), (ALIGNMENT, dict(vp=P(0x10002))), (ALIGNMENT, dict(ldkv=260)),
    (ALIGNMENT, dict(pitch=16 * 256 + 4)), (ALIGNMENT, dict(table=P(0x10002))), (ALIGNMENT, dict(cu=P(0x10001))),
    (ALIGNMENT, dict(FP8_CACHE, kps=P(0x10002))),
    (OK, dict(T=0, K=None, V=None)), (OK, dict(batch=0, lens=None)), (OK, dict(n_kv=0))])
def test_append_checks(lib, status, changes):
    assert call(lib.paged_kv_append, APPEND, **changes) == status


@pytest.mark.parametrize("status,changes", [
    (INVALID, dict(batch=-1)), (INVALID, dict(heads=-1)), (INVALID, dict(n_kv=-2)), (INVALID, dict(page=0)),
    (INVALID, dict(pages=-1)), (INVALID, dict(max_pages=-1)), (INVALID, dict(cache=0)), (INVALID, dict(scale=F(0.0))),
    (INVALID, dict(scale=F(-1.0))), (INVALID, dict(scale=F(float("nan")))), (INVALID, dict(scale=F(float("inf")))),
    (INVALID, dict(n_kv=0)), (INVALID, dict(n_kv=3)), (UNSUPPORTED, dict(head_dim=64)),
    (UNSUPPORTED, dict(heads=131072)), (INVALID, dict(Q=None)),
    (INVALID, dict(O=None)), (INVALID, dict(kp=None)), (INVALID, dict(table=None)), (INVALID, dict(lens=None)),
    (INVALID, dict(ldq=1016)), (INVALID, dict(ldo=1016)), (INVALID, dict(ldt=4)), (INVALID, dict(pitch=4088)),
    (INVALID, dict(cache=2)), (INVALID, dict(FP8_CACHE, spitch=30)), (ALIGNMENT, dict(Q=P(0x10004))),
    (ALIGNMENT, dict(O=P(0x10008))), (ALIGNMENT, dict(ldq=1028)), (ALIGNMENT, dict(kp=P(0x10008))),
    (ALIGNMENT, dict(lens=P(0x10002))), (ALIGNMENT, dict(ws=P(0x10010))), (WORKSPACE, dict(ws=None)),
    (WORKSPACE, dict(bytes=4096)), (OK, dict(batch=0, Q=None)), (OK, dict(heads=0, O=None))])
def test_decode_checks(lib, status, changes):
    assert call(lib.attention_decode, DECODE, **changes) == status


@pytest.mark.parametrize("status,changes", [
    (INVALID, dict(M=-1)), (INVALID, dict(batch=-1)), (INVALID, dict(heads=-8)), (INVALID, dict(n_kv=-1)),
    (INVALID, dict(cu=None)), (INVALID, dict(kv=0)), (INVALID, dict(scale=F(0.0))), (INVALID, dict(n_kv=3)),
    (INVALID, dict(n_kv=0)), (UNSUPPORTED, dict(head_dim=256)), (UNSUPPORTED, dict(heads=131072)), (INVALID, dict(Q=None)), (INVALID, dict(K=None)),
    (INVALID, dict(V=None)), (INVALID, dict(O=None)), (INVALID, dict(kv=2)), (INVALID, dict(ldq=1016)),
    (INVALID, dict(ldo=1016)), (INVALID, dict(ldkv=248)), (INVALID, dict(kv=2, ks=A, vs=A, lds=1)),
    (ALIGNMENT, dict(Q=P(0x10008))), (ALIGNMENT, dict(ldkv=260)), (ALIGNMENT, dict(ldo=1028)),
    (ALIGNMENT, dict(cu=P(0x10002))), (ALIGNMENT, dict(ws=P(0x10020))), (WORKSPACE, dict(ws=None)),
    (WORKSPACE, dict(bytes=100)), (WORKSPACE, dict(kv=2, ks=A, vs=A, lds=2, bytes=512)),
    (OK, dict(M=0, Q=None)), (OK, dict(heads=0)), (OK, dict(batch=0))])
def test_prefill_checks(lib, status, changes):
    assert call(lib.attention_prefill, PREFILL, **changes) == status


def test_workspace_sizes(lib):
    n = lib.fl_attention_prefill_workspace_bytes
    assert n(100, 2, fl.FL_BF16) >= 512
    assert n(100, 2, fl.FL_E4M3) - n(100, 2, fl.FL_BF16) >= 100 * 2 * 128 * 2 * 2  # K and V in 16 bits
    assert n(1 << 22, 16, fl.FL_E4M3) > 1 << 32
    assert n(-1, 2, fl.FL_BF16) == 0
    assert lib.fl_attention_decode_workspace_bytes() % 256 == 0


def test_binding_refuses_mixed_types_and_shapes():
    """CPU tensors are refused before anything else happens."""
    t = torch.zeros(4, 256, dtype=torch.bfloat16)
    c = torch.zeros(3, 2, 16, 128, dtype=torch.bfloat16)
    table, lens = torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        fl.attention_prefill(t, t, t)
    with pytest.raises(ValueError):
        fl.attention_decode(t, c, c, table, lens)
    with pytest.raises(ValueError):
        fl.paged_kv_append(t, t, c, c, table, lens)
    with pytest.raises(ValueError):
        fl.paged_kv_append(t, t, c, c, table, lens, k_scale=torch.zeros(4, 2))


def test_kernels_launched_as_dependents_read_by_ordinary_loads():
    """Every attention kernel begins while the kernel in front may still write its inputs, which rules out loads for data
    that is read-only as long as the kernel lives: by intrinsic, in PTX, or by a pointer that promises it."""
    files = [f for f in cuda_build._deps() if os.path.dirname(f) == cuda_build.ATTENTION]
    assert len(files) >= 5
    for f in files:
        with open(f, encoding="utf-8") as src:
            code = "".join(line.split("//")[0] + "\n" for line in src)
        for word in ("__ldg", "ld.global.nc", "__restrict__", "ldu."):
            assert word not in code, (f, word)


def test_build_refuses_another_register_count():
    """The prefill kernel's warps share out the registers of its launch: a compiler that takes another number than the
    source counts on ends the build, not the first call."""
    src = os.path.join(cuda_build.ATTENTION, "k_attention_prefill.cu")
    report = ("ptxas info    : Compiling entry function '_ZN2fl24attention_prefill_kernelILb{}EEEvNS_13PrefillParamsE' for "
              "'sm_103a'\nptxas info    : Function properties for x\n    0 bytes stack frame\n"
              "ptxas info    : Used {} registers, used 1 barriers\n")
    other = "ptxas info    : Compiling entry function '_ZN2fl5otherEv' for 'sm_103a'\nptxas info    : Used 64 registers\n"
    with open(os.path.join(cuda_build.ATTENTION, "prefill_attention_kernel.cuh"), encoding="utf-8") as f:
        want = int(f.read().split("kPreRegs = ")[1].split(",")[0])
    cuda_build.check_registers(src, report.format(0, want) + other + report.format(1, want))
    for bad in (other, report.format(0, want) + report.format(1, want - 8), report.format(1, want + 8) + other, ""):
        with pytest.raises(RuntimeError):
            cuda_build.check_registers(src, bad)


@pytest.mark.parametrize("device", [0, 1, "cuda:0", None])
def test_workspaces_are_made_on_the_device_that_is_asked_for(lib, monkeypatch, device):
    """An index of 0 is a device of its own, not the current one."""
    made, empty = [], torch.empty
    monkeypatch.setattr(fl.torch, "empty", lambda n, dtype, device: (made.append(device), empty(n, dtype=dtype))[1])
    fl.attention_decode_workspace(device)
    fl.attention_prefill_workspace(10, 2, True, device)
    assert made == ["cuda" if device is None else device] * 2


@pytest.mark.parametrize("scale", [2.4e38, 3.4e38])
def test_scales_that_base_two_does_not_hold(lib, scale):
    """The kernels work to base 2: a finite scale whose product with log2 e is not is refused, as an infinite one is."""
    assert call(lib.attention_decode, DECODE, scale=F(scale)) == INVALID
    assert call(lib.attention_prefill, PREFILL, scale=F(scale)) == INVALID
    assert call(lib.attention_decode, DECODE, scale=F(2.3e38), ws=None) == WORKSPACE


def test_decode_linear_kernels_read_by_ordinary_loads():
    """The same for the decode kernels of the linear layers, and for the loader that they share with nobody else."""
    def code(name):
        with open(os.path.join(cuda_build.CSRC, name), encoding="utf-8") as src:
            return "".join(line.split("//")[0] + "\n" for line in src)

    loader = code("gemm_kernel.cuh").split("void load_bf16x4(")[1].split("__device__")[0]
    kernels = [code(f) for f in os.listdir(cuda_build.CSRC) if "decode" in f and f.endswith(".cuh")]
    assert len(kernels) >= 3 and any("griddep_wait();" in k for k in kernels)
    for text in [loader] + kernels:
        for word in ("__ldg", "ld.global.nc", "__restrict__", "ldu."):
            assert word not in text
