"""GB300 (sm_103a) fused Linear + epilogue library: Python binding.

This module only marshals arguments: it turns torch CUDA tensors into device
pointers, leading dimensions and a stream handle, and calls the C ABI of
``libfusedlinear.so`` (declared in ``include/fused_linear.h``), whose CUDA
kernels do every step of the computation.  There is no other code path: if
the library is not built or cannot be loaded, every call raises.

Functions carry the C names: :func:`fused_linear_gelu` (and its host-buffer
form :func:`fused_linear_gelu_host`), :func:`fused_qkv_rope`,
:func:`fused_qkv_rope_fp8kv`, :func:`fused_swiglu`,
:func:`fused_linear_residual_rmsnorm_fp8` (and
:func:`fused_linear_residual_rmsnorm_fp8_noalloc`, which takes no workspace),
the deferred-scale chain :func:`fused_linear_residual_gamma` and
:func:`fused_linear_rms_rowscale`, :func:`fused_linear_cross_entropy`,
:func:`fused_linear_quant`, and the backward epilogues
:func:`fused_dgrad_gelu` and :func:`fused_swiglu_bwd`; for the attention behind
the QKV projections :func:`paged_kv_append`, :func:`attention_prefill` and
:func:`attention_decode`.
"""
from __future__ import annotations

import ctypes
import os
import re

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
LIB_PATH = os.path.join(HERE, "libfusedlinear.so")
HEADER = os.path.join(ROOT, "include", "fused_linear.h")

FL_OK, FL_ERR_INVALID_ARG, FL_ERR_UNSUPPORTED, FL_ERR_ALIGNMENT, FL_ERR_WORKSPACE, FL_ERR_CUDA, \
    FL_ERR_TIMEOUT, FL_ERR_ARCH = range(8)
FL_F32, FL_BF16, FL_E4M3 = 0, 1, 2
FL_GELU_ERF, FL_GELU_TANH = 0, 1

_lib = None


class FusedLinearError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        super().__init__(f"{fn}: {status_string(status)} (status {status})")


def load() -> ctypes.CDLL:
    """Loads the in-tree library (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is not built; run gemm_epilogue_tcgen05_gb300.build.build()")
    lib = ctypes.CDLL(LIB_PATH)
    P, I, I64, F, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
    lib.fused_linear_gelu.argtypes = [P, P, P, P, I, I, I, I64, I64, I64, I, I, P]
    lib.fused_qkv_rope.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, F, I64, I64, I64, P]
    lib.fused_swiglu.argtypes = [P, P, P, P, P, P, I, I, I, I64, I64, I64, P]
    lib.fused_linear_residual_rmsnorm_fp8.argtypes = [P, P, P, P, P, F, P, P, P, I, I, I, I64, I64, I64, I64,
                                                      P, SZ, P]
    for f in (lib.fused_linear_gelu, lib.fused_qkv_rope, lib.fused_swiglu,
              lib.fused_linear_residual_rmsnorm_fp8):
        f.restype = I
    lib.fused_linear_residual_gamma.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I64, I64, I64, I64, P]
    lib.fused_linear_rms_rowscale.argtypes = [P, P, P, P, I, F, P, I, I, I, I64, I64, I64, P]
    lib.fused_linear_residual_gamma.restype = I
    lib.fused_linear_rms_rowscale.restype = I
    lib.fused_linear_cross_entropy.argtypes = [P, P, P, P, P, P, I, I, I, I64, I64, I64, P, SZ, P]
    lib.fused_linear_cross_entropy.restype = I
    lib.fused_qkv_rope_fp8kv.argtypes = [P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, I64, I64, I64, I64, I64, P]
    lib.fused_qkv_rope_fp8kv.restype = I
    lib.fused_dgrad_gelu.argtypes = [P, P, P, P, I, I, I, I64, I64, I64, I64, I, P]
    lib.fused_dgrad_gelu.restype = I
    lib.fused_swiglu_bwd.argtypes = [P, P, P, P, P, I, I, I, I64, I64, I64, I64, P]
    lib.fused_swiglu_bwd.restype = I
    lib.fused_linear_gelu_host.argtypes = [P, P, P, P, I, I, I, I, P, SZ, P]
    lib.fused_linear_gelu_host.restype = I
    lib.fl_linear_gelu_host_buffer_bytes.argtypes = [I, I, I]
    lib.fl_linear_gelu_host_buffer_bytes.restype = SZ
    lib.fused_linear_quant.argtypes = [P, P, P, P, P, P, I, I, I, I64, I64, I64, I64, I, P]
    lib.fused_linear_quant.restype = I
    lib.paged_kv_append.argtypes = [P] * 11 + [I] * 7 + [I64] * 5 + [I, I, P]
    lib.paged_kv_append.restype = I
    lib.attention_decode.argtypes = [P] * 8 + [I] * 7 + [I64] * 5 + [F, I, P, SZ, P]
    lib.attention_decode.restype = I
    lib.fl_attention_decode_workspace_bytes.argtypes = []
    lib.fl_attention_decode_workspace_bytes.restype = SZ
    lib.attention_prefill.argtypes = [P] * 7 + [I] * 6 + [I64] * 4 + [F, I, I, P, SZ, P]
    lib.attention_prefill.restype = I
    lib.fl_attention_prefill_workspace_bytes.argtypes = [I, I, I]
    lib.fl_attention_prefill_workspace_bytes.restype = SZ
    lib.fl_cross_entropy_workspace_bytes.argtypes = [I, I]
    lib.fl_cross_entropy_workspace_bytes.restype = SZ
    lib.fl_rms_partials_per_row.argtypes = [I]
    lib.fl_rms_partials_per_row.restype = I
    lib.fused_linear_residual_rmsnorm_fp8_noalloc.argtypes = [P, P, P, P, P, F, P, P, I, I, I, I64, I64, I64,
                                                              I64, P]
    lib.fused_linear_residual_rmsnorm_fp8_noalloc.restype = I
    lib.fl_rmsnorm_fp8_workspace_bytes.argtypes = [I, I, I]
    lib.fl_rmsnorm_fp8_workspace_bytes.restype = SZ
    lib.fl_device_status.argtypes = [P]
    lib.fl_device_status.restype = I
    lib.fl_check_device_status.argtypes = [P, P]
    lib.fl_check_device_status.restype = I
    lib.fl_set_cooperative_launch.argtypes = [I]
    lib.fl_set_cooperative_launch.restype = None
    lib.fl_set_descriptor_cache.argtypes = [I]
    lib.fl_set_descriptor_cache.restype = None
    lib.fl_descriptor_cache_stats.argtypes = [P, P]
    lib.fl_descriptor_cache_stats.restype = None
    lib.fl_set_wait_timeout_ns.argtypes = [ctypes.c_uint64]
    lib.fl_set_wait_timeout_ns.restype = None
    lib.fl_set_max_ctas.argtypes = [I]
    lib.fl_set_max_ctas.restype = None
    lib.fl_set_cta_pairing.argtypes = [I]
    lib.fl_set_cta_pairing.restype = None
    lib.fl_set_linear_decode.argtypes = [I]
    lib.fl_set_linear_decode.restype = None
    lib.fl_linear_decode_shape.argtypes = [I, I, I, I, P, P, P]
    lib.fl_linear_decode_shape.restype = I
    lib.fl_status_string.argtypes = [I]
    lib.fl_status_string.restype = ctypes.c_char_p
    lib.fl_version.argtypes = []
    lib.fl_version.restype = I
    _lib = lib
    return lib


def header_symbols() -> list[str]:
    """Names of every entry point declared (FL_API) in include/fused_linear.h."""
    with open(HEADER) as f:
        text = f.read()
    return re.findall(r"^FL_API\s+[\w\s\*]+?\b(\w+)\s*\(", text, flags=re.M)


def status_string(status: int) -> str:
    return load().fl_status_string(int(status)).decode()


def version() -> int:
    return load().fl_version()


def _check(fn: str, status: int):
    if status != FL_OK:
        raise FusedLinearError(fn, status)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _mat(t, name, dtype):
    if t.dim() != 2 or t.dtype != dtype or not t.is_cuda or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name}: expected a 2-D {dtype} CUDA tensor with unit column stride")
    return t.stride(0) if t.shape[0] > 1 else max(t.shape[1], 1)


def _vec(t, name, dtype, n):
    if t is None:
        return None
    if t.dtype != dtype or not t.is_cuda or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous {dtype} CUDA vector of length {n}")
    return t


def _out(rows: int, cols: int, dtype, device):
    """An output [rows, cols] whose row pitch is rounded up to 16 bytes (the TMA store rule)."""
    per = 16 // torch.empty((), dtype=dtype).element_size()
    return torch.empty((rows, -(-cols // per) * per), dtype=dtype, device=device)[:, :cols]


def _ld(t, width, fallback):
    # Leading dimension of a [rows, width] row-major matrix.  A one-row matrix
    # never reads past its first row, so any pitch >= width works; take one
    # that satisfies the 16-byte pitch rule.
    if t.shape[0] > 1:
        return t.stride(0)
    return max(-(-fallback // 16) * 16, 16)


def fused_linear_gelu(X, W, b=None, Y=None, mode: str = "tanh", stream=None):
    """Y = GELU(X W^T + b); bf16 (tcgen05) or fp32 operands."""
    dtype = X.dtype
    if dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("X must be bf16 or fp32")
    M, K = X.shape
    N = W.shape[0]
    _mat(X, "X", dtype)
    _mat(W, "W", dtype)
    _vec(b, "b", dtype, N)
    if Y is None:
        Y = _out(M, N, dtype, X.device)
    _mat(Y, "Y", dtype)
    m = {"erf": FL_GELU_ERF, "tanh": FL_GELU_TANH}[mode]
    st = load().fused_linear_gelu(_ptr(X), _ptr(W), _ptr(b), _ptr(Y), M, N, K, _ld(X, K, K), _ld(W, K, K),
                                  _ld(Y, N, N), FL_BF16 if dtype == torch.bfloat16 else FL_F32, m,
                                  _stream(stream))
    _check("fused_linear_gelu", st)
    return Y


def linear_gelu_host_buffer(M: int, N: int, K: int, device=None) -> torch.Tensor:
    """Device buffer for fused_linear_gelu_host (256-byte aligned, as torch allocates)."""
    n = int(load().fl_linear_gelu_host_buffer_bytes(M, N, K))
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def fused_linear_gelu_host(X, W, b=None, Y=None, mode: str = "tanh", dev_buf=None, stream=None):
    """fused_linear_gelu on host (CPU, ideally pinned) bf16 tensors, copies overlapped with the GEMM.

    Returns Y (host); it is complete once `stream` (default: the current stream) has finished.
    """
    M, K = X.shape
    N = W.shape[0]
    for t, nm in ((X, "X"), (W, "W"), (b, "b"), (Y, "Y")):
        if t is not None and (t.is_cuda or t.dtype != torch.bfloat16 or not t.is_contiguous()):
            raise ValueError(f"{nm}: expected a contiguous bf16 host tensor")
    if b is not None and b.numel() != N:
        raise ValueError("b must have N elements")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, pin_memory=True)
    if tuple(Y.shape) != (M, N):
        raise ValueError("Y must be [M, N]")
    if dev_buf is None:
        dev_buf = linear_gelu_host_buffer(M, N, K)
    if mode not in ("tanh", "erf"):
        raise ValueError("mode must be 'tanh' or 'erf'")
    st = load().fused_linear_gelu_host(_ptr(X), _ptr(W), _ptr(b), _ptr(Y), M, N, K,
                                       FL_GELU_TANH if mode == "tanh" else FL_GELU_ERF, _ptr(dev_buf),
                                       dev_buf.numel(), _stream(stream))
    _check("fused_linear_gelu_host", st)
    return Y


def fused_qkv_rope(X, Wqkv, bqkv=None, n_heads: int = 32, head_dim: int = 128, seq_len: int = 2048,
                   theta: float = 10000.0, positions=None, out=None, stream=None):
    """Returns (Q, K, V), Q and K already rotated (RoPE on adjacent pairs)."""
    M, K = X.shape
    d = n_heads * head_dim
    _mat(X, "X", torch.bfloat16)
    _mat(Wqkv, "Wqkv", torch.bfloat16)
    _vec(bqkv, "bqkv", torch.bfloat16, 3 * d)
    if positions is not None and (positions.dtype != torch.int32 or positions.numel() != M
                                  or not positions.is_cuda or not positions.is_contiguous()):
        raise ValueError("positions must be a contiguous int32 CUDA vector of length M")
    if out is None:
        out = tuple(torch.empty((M, d), dtype=torch.bfloat16, device=X.device) for _ in range(3))
    Q, Ko, V = out
    lds = {_ld(t, d, d) for t in out}
    for t, nm in zip(out, "QKV"):
        _mat(t, nm, torch.bfloat16)
    if len(lds) != 1:
        raise ValueError("Q, K and V must share one leading dimension")
    st = load().fused_qkv_rope(_ptr(X), _ptr(Wqkv), _ptr(bqkv), _ptr(Q), _ptr(Ko), _ptr(V), _ptr(positions),
                               M, K, n_heads, head_dim, seq_len, float(theta), _ld(X, K, K), _ld(Wqkv, K, K),
                               lds.pop(), _stream(stream))
    _check("fused_qkv_rope", st)
    return Q, Ko, V


def fused_qkv_rope_fp8kv(X, Wqkv, bqkv=None, n_heads: int = 32, n_kv_heads: int = 8, head_dim: int = 128,
                         seq_len: int = 2048, theta: float = 10000.0, positions=None, out=None, stream=None):
    """QKV + RoPE with the K/V cache entry in FP8; returns (Q, Kq, Vq, k_scale, v_scale).

    Q bf16 [M, n_heads*head_dim] (rotated); Kq (rotated) and Vq E4M3 bytes
    [M, n_kv_heads*head_dim]; k_scale, v_scale fp32 [M, n_kv_heads].
    """
    M, K = X.shape
    dq, dkv = n_heads * head_dim, n_kv_heads * head_dim
    _mat(X, "X", torch.bfloat16)
    _mat(Wqkv, "Wqkv", torch.bfloat16)
    _vec(bqkv, "bqkv", torch.bfloat16, dq + 2 * dkv)
    if positions is not None and (positions.dtype != torch.int32 or positions.numel() != M
                                  or not positions.is_cuda or not positions.is_contiguous()):
        raise ValueError("positions must be a contiguous int32 CUDA vector of length M")
    if out is None:
        out = (torch.empty((M, dq), dtype=torch.bfloat16, device=X.device),
               torch.empty((M, dkv), dtype=torch.uint8, device=X.device),
               torch.empty((M, dkv), dtype=torch.uint8, device=X.device),
               torch.empty((M, n_kv_heads), dtype=torch.float32, device=X.device),
               torch.empty((M, n_kv_heads), dtype=torch.float32, device=X.device))
    Q, Kq, Vq, ks, vs = out
    _mat(Q, "Q", torch.bfloat16)
    for t, nm in ((Kq, "Kq"), (Vq, "Vq")):
        _mat(t, nm, torch.uint8)
    for t, nm in ((ks, "k_scale"), (vs, "v_scale")):
        _mat(t, nm, torch.float32)
    ldkv = {_ld(Kq, dkv, dkv), _ld(Vq, dkv, dkv)}
    lds = {_ld(ks, n_kv_heads, n_kv_heads), _ld(vs, n_kv_heads, n_kv_heads)}
    if len(ldkv) != 1 or len(lds) != 1:
        raise ValueError("Kq and Vq (and their scales) must share one leading dimension")
    st = load().fused_qkv_rope_fp8kv(_ptr(X), _ptr(Wqkv), _ptr(bqkv), _ptr(Q), _ptr(Kq), _ptr(Vq), _ptr(ks),
                                     _ptr(vs), _ptr(positions), M, K, n_heads, n_kv_heads, head_dim, seq_len,
                                     float(theta), _ld(X, K, K), _ld(Wqkv, K, K), _ld(Q, dq, dq), ldkv.pop(),
                                     lds.pop(), _stream(stream))
    _check("fused_qkv_rope_fp8kv", st)
    return Q, Kq, Vq, ks, vs


def fused_swiglu(X, Wgate, Wup, bgate=None, bup=None, Y=None, stream=None):
    """Y = SiLU(X Wgate^T + bgate) * (X Wup^T + bup)."""
    M, K = X.shape
    N = Wgate.shape[0]
    _mat(X, "X", torch.bfloat16)
    ldg = _mat(Wgate, "Wgate", torch.bfloat16)
    ldu = _mat(Wup, "Wup", torch.bfloat16)
    if Wup.shape != Wgate.shape or (N > 1 and ldg != ldu):
        raise ValueError("Wgate and Wup must have the same shape and leading dimension")
    _vec(bgate, "bgate", torch.bfloat16, N)
    _vec(bup, "bup", torch.bfloat16, N)
    if Y is None:
        Y = _out(M, N, torch.bfloat16, X.device)
    _mat(Y, "Y", torch.bfloat16)
    st = load().fused_swiglu(_ptr(X), _ptr(Wgate), _ptr(Wup), _ptr(bgate), _ptr(bup), _ptr(Y), M, N, K,
                             _ld(X, K, K), _ld(Wgate, K, K), _ld(Y, N, N), _stream(stream))
    _check("fused_swiglu", st)
    return Y


def rmsnorm_fp8_workspace_bytes(M: int, N: int, K: int) -> int:
    return load().fl_rmsnorm_fp8_workspace_bytes(M, N, K)


def rmsnorm_fp8_workspace(M: int, N: int, K: int, device=None) -> torch.Tensor:
    """A zero-filled workspace of the size the library asks for (torch allocation)."""
    n = max(rmsnorm_fp8_workspace_bytes(M, N, K), 1)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def fused_linear_residual_rmsnorm_fp8(X, W, b, Z, gamma, eps: float = 1e-6, Yq=None, row_scale=None,
                                      workspace=None, h_out=None, stream=None):
    """Returns (Yq, row_scale): E4M3 codes as uint8 [M, N] and fp32 scales [M].

    h_out: None (default), True (allocate one) or a bf16 [M, N] tensor with Z's row pitch;
    when given, h = X W^T + b + Z is written there too and (Yq, row_scale, h_out) is returned."""
    M, K = X.shape
    N = W.shape[0]
    _mat(X, "X", torch.bfloat16)
    _mat(W, "W", torch.bfloat16)
    _mat(Z, "Z", torch.bfloat16)
    _vec(b, "b", torch.bfloat16, N)
    _vec(gamma, "gamma", torch.bfloat16, N)
    if Yq is None:  # row pitch rounded up to 16 bytes, as the TMA store needs
        Yq = _out(M, N, torch.uint8, X.device)
    if Yq.dtype != torch.uint8:
        Yq = Yq.view(torch.uint8)
    _mat(Yq, "Yq", torch.uint8)
    if row_scale is None:
        row_scale = torch.empty(M, dtype=torch.float32, device=X.device)
    _vec(row_scale, "row_scale", torch.float32, M)
    want_h = h_out is not None
    if h_out is True:
        h_out = torch.empty_strided((M, N), (_ld(Z, N, N), 1), dtype=torch.bfloat16, device=X.device)
    if want_h:
        _mat(h_out, "h_out", torch.bfloat16)
        if tuple(h_out.shape) != (M, N) or (M > 1 and h_out.stride(0) != Z.stride(0)):
            raise ValueError("h_out must be [M, N] with Z's row pitch")
    if workspace is None:
        workspace = rmsnorm_fp8_workspace(M, N, K, X.device)
    st = load().fused_linear_residual_rmsnorm_fp8(
        _ptr(X), _ptr(W), _ptr(b), _ptr(Z), _ptr(gamma), float(eps), _ptr(Yq), _ptr(row_scale),
        _ptr(h_out) if want_h else None, M, N, K, _ld(X, K, K), _ld(W, K, K), _ld(Z, N, N), _ld(Yq, N, N),
        _ptr(workspace), workspace.numel(), _stream(stream))
    _check("fused_linear_residual_rmsnorm_fp8", st)
    return (Yq, row_scale, h_out) if want_h else (Yq, row_scale)


def fused_linear_residual_rmsnorm_fp8_noalloc(X, W, b, Z, gamma, Yq, row_scale, eps: float = 1e-6,
                                              stream=None):
    """The same codes and scales as :func:`fused_linear_residual_rmsnorm_fp8`, through the entry point
    that needs no workspace (it uses a scratch array built into the library; calls that may overlap
    on the GPU must not be issued).  Yq (uint8 [M, N]) and row_scale (fp32 [M]) are the caller's:
    the call allocates nothing.  Returns (Yq, row_scale)."""
    M, K = X.shape
    N = W.shape[0]
    _mat(X, "X", torch.bfloat16)
    _mat(W, "W", torch.bfloat16)
    _mat(Z, "Z", torch.bfloat16)
    _vec(b, "b", torch.bfloat16, N)
    _vec(gamma, "gamma", torch.bfloat16, N)
    _mat(Yq, "Yq", torch.uint8)
    _vec(row_scale, "row_scale", torch.float32, M)
    st = load().fused_linear_residual_rmsnorm_fp8_noalloc(
        _ptr(X), _ptr(W), _ptr(b), _ptr(Z), _ptr(gamma), float(eps), _ptr(Yq), _ptr(row_scale), M, N, K,
        _ld(X, K, K), _ld(W, K, K), _ld(Z, N, N), _ld(Yq, N, N), _stream(stream))
    _check("fused_linear_residual_rmsnorm_fp8_noalloc", st)
    return Yq, row_scale


def rms_partials_per_row(n_norm: int) -> int:
    return load().fl_rms_partials_per_row(int(n_norm))


def fused_linear_residual_gamma(X, W, b, Z, gamma, store_h1: bool = True, H2=None, H1=None, rms_partials=None,
                                stream=None):
    """Step 1 of GEMM -> residual -> RMSNorm -> GEMM: returns (H2 = h1 * gamma, H1 = h1 or None, partials)."""
    M, K = X.shape
    N = W.shape[0]
    _mat(X, "X", torch.bfloat16)
    _mat(W, "W", torch.bfloat16)
    _mat(Z, "Z", torch.bfloat16)
    _vec(b, "b", torch.bfloat16, N)
    _vec(gamma, "gamma", torch.bfloat16, N)
    if H2 is None:
        H2 = _out(M, N, torch.bfloat16, X.device)
    if H1 is None and store_h1:
        H1 = _out(M, N, torch.bfloat16, X.device)
    _mat(H2, "H2", torch.bfloat16)
    if H1 is not None and (_mat(H1, "H1", torch.bfloat16) != _mat(H2, "H2", torch.bfloat16) and M > 1):
        raise ValueError("H1 and H2 must share one leading dimension")
    npart = rms_partials_per_row(N)
    if rms_partials is None:
        rms_partials = torch.empty((npart, M), dtype=torch.float32, device=X.device)
    if rms_partials.dtype != torch.float32 or rms_partials.numel() < npart * M or not rms_partials.is_contiguous():
        raise ValueError("rms_partials must be a contiguous fp32 tensor of [ceil(N/256), M] entries")
    st = load().fused_linear_residual_gamma(_ptr(X), _ptr(W), _ptr(b), _ptr(Z), _ptr(gamma), _ptr(H2), _ptr(H1),
                                            _ptr(rms_partials), M, N, K, _ld(X, K, K), _ld(W, K, K), _ld(Z, N, N),
                                            _ld(H2, N, N), _stream(stream))
    _check("fused_linear_residual_gamma", st)
    return H2, H1, rms_partials


def fused_linear_rms_rowscale(H2, W1, b1, rms_partials, n_norm: int, eps: float = 1e-6, Y=None, stream=None):
    """Step 2: Y = r * (H2 W1^T) + b1, r = 1/sqrt(sum of the row's partials / n_norm + eps)."""
    M, K = H2.shape
    N = W1.shape[0]
    _mat(H2, "H2", torch.bfloat16)
    _mat(W1, "W1", torch.bfloat16)
    _vec(b1, "b1", torch.bfloat16, N)
    if Y is None:
        Y = _out(M, N, torch.bfloat16, H2.device)
    _mat(Y, "Y", torch.bfloat16)
    st = load().fused_linear_rms_rowscale(_ptr(H2), _ptr(W1), _ptr(b1), _ptr(rms_partials), int(n_norm), float(eps),
                                          _ptr(Y), M, N, K, _ld(H2, K, K), _ld(W1, K, K), _ld(Y, N, N),
                                          _stream(stream))
    _check("fused_linear_rms_rowscale", st)
    return Y


def cross_entropy_workspace(M: int, V: int, device=None) -> torch.Tensor:
    n = max(load().fl_cross_entropy_workspace_bytes(int(M), int(V)), 1)
    return torch.zeros(n, dtype=torch.uint8, device=device or "cuda")


def fused_linear_cross_entropy(X, W, b, labels, loss=None, logits=None, store_logits: bool = False,
                               workspace=None, stream=None):
    """Per-row loss logsumexp(X W^T + b) - (X W^T + b)[label]; returns (loss, logits or None)."""
    M, K = X.shape
    V = W.shape[0]
    _mat(X, "X", torch.bfloat16)
    _mat(W, "W", torch.bfloat16)
    _vec(b, "b", torch.bfloat16, V)
    if labels.dtype != torch.int32 or labels.numel() != M or not labels.is_cuda or not labels.is_contiguous():
        raise ValueError("labels must be a contiguous int32 CUDA vector of length M")
    if loss is None:
        loss = torch.empty(M, dtype=torch.float32, device=X.device)
    _vec(loss, "loss", torch.float32, M)
    if logits is None and store_logits:
        logits = _out(M, V, torch.bfloat16, X.device)
    ldl = 0
    if logits is not None:
        _mat(logits, "logits", torch.bfloat16)
        ldl = _ld(logits, V, V)
    if workspace is None:
        workspace = cross_entropy_workspace(M, V, X.device)
    st = load().fused_linear_cross_entropy(_ptr(X), _ptr(W), _ptr(b), _ptr(labels), _ptr(loss), _ptr(logits), M, V, K,
                                           _ld(X, K, K), _ld(W, K, K), ldl, _ptr(workspace), workspace.numel(),
                                           _stream(stream))
    _check("fused_linear_cross_entropy", st)
    return loss, logits


QUANT_FP8_1X128, QUANT_INT4_G32, QUANT_NVFP4_G16 = 0, 1, 2
QUANT_BLOCK = {QUANT_FP8_1X128: 128, QUANT_INT4_G32: 32, QUANT_NVFP4_G16: 16}


def fused_linear_quant(X, W, b=None, fmt: int = QUANT_FP8_1X128, Yq=None, scales=None, inv_smooth=None,
                       stream=None):
    """Block-scaled quantised Linear output; returns (codes uint8, scales).

    inv_smooth: optional fp32 [N] inverse smoothing factor, multiplied into each output
    column before the block maxima (the optional correction step of the quantised write-back).
    FP8 1x128: codes [M, N] E4M3, scales fp32 [M, ceil(N/128)].
    INT4 g32:  codes [M, N/2] (column 2j in the low nibble of byte j), scales fp32 [M, ceil(N/32)].
    NVFP4 g16: codes [M, N/2] E2M1 pairs, scales E4M3 bytes (uint8) [M, ceil(N/16)].
    """
    if fmt not in QUANT_BLOCK:
        raise ValueError(f"unknown quantisation format {fmt}")
    M, K = X.shape
    N = W.shape[0]
    _mat(X, "X", torch.bfloat16)
    _mat(W, "W", torch.bfloat16)
    _vec(b, "b", torch.bfloat16, N)
    _vec(inv_smooth, "inv_smooth", torch.float32, N)
    qbytes = N if fmt == QUANT_FP8_1X128 else N // 2
    nblocks = -(-N // QUANT_BLOCK[fmt])
    sdt = torch.uint8 if fmt == QUANT_NVFP4_G16 else torch.float32
    if Yq is None:  # row pitch rounded up to 16 bytes, as the TMA store needs
        Yq = _out(M, qbytes, torch.uint8, X.device)
    if scales is None:
        scales = torch.empty((M, nblocks), dtype=sdt, device=X.device)
    _mat(Yq, "Yq", torch.uint8)
    _mat(scales, "scales", sdt)
    st = load().fused_linear_quant(_ptr(X), _ptr(W), _ptr(b), _ptr(inv_smooth), _ptr(Yq), _ptr(scales), M, N, K,
                                   _ld(X, K, K),
                                   _ld(W, K, K), _ld(Yq, qbytes, qbytes), _ld(scales, nblocks, nblocks), int(fmt),
                                   _stream(stream))
    _check("fused_linear_quant", st)
    return Yq, scales


def fused_dgrad_gelu(dZ, W, H, mode: str = "tanh", dH=None, stream=None):
    """dH = (dZ W) * GELU'(H): the next layer's weight W [K, N] as stored, H the saved pre-activation."""
    M, K = dZ.shape
    if W.shape[0] != K:
        raise ValueError("W must be [K, N] with K = dZ.shape[1]")
    N = W.shape[1]
    _mat(dZ, "dZ", torch.bfloat16)
    _mat(W, "W", torch.bfloat16)
    _mat(H, "H", torch.bfloat16)
    if tuple(H.shape) != (M, N):
        raise ValueError("H must be [M, N]")
    if dH is None:
        dH = _out(M, N, torch.bfloat16, dZ.device)
    _mat(dH, "dH", torch.bfloat16)
    if mode not in ("tanh", "erf"):
        raise ValueError("mode must be 'tanh' or 'erf'")
    st = load().fused_dgrad_gelu(_ptr(dZ), _ptr(W), _ptr(H), _ptr(dH), M, N, K, _ld(dZ, K, K), _ld(W, N, N),
                                 _ld(H, N, N), _ld(dH, N, N), FL_GELU_TANH if mode == "tanh" else FL_GELU_ERF,
                                 _stream(stream))
    _check("fused_dgrad_gelu", st)
    return dH


def fused_swiglu_bwd(dO, Wd, G, U, dGU=None, stream=None):
    """SwiGLU backward through the down projection Wd [K, N] (as stored): returns dGU [M, 2N]
    with dg at column 2n and du at column 2n + 1."""
    M, K = dO.shape
    if Wd.shape[0] != K:
        raise ValueError("Wd must be [K, N] with K = dO.shape[1]")
    N = Wd.shape[1]
    _mat(dO, "dO", torch.bfloat16)
    _mat(Wd, "Wd", torch.bfloat16)
    _mat(G, "G", torch.bfloat16)
    _mat(U, "U", torch.bfloat16)
    if tuple(G.shape) != (M, N) or tuple(U.shape) != (M, N) or _ld(G, N, N) != _ld(U, N, N):
        raise ValueError("G and U must be [M, N] with one shared pitch")
    if dGU is None:
        dGU = _out(M, 2 * N, torch.bfloat16, dO.device)
    _mat(dGU, "dGU", torch.bfloat16)
    st = load().fused_swiglu_bwd(_ptr(dO), _ptr(Wd), _ptr(G), _ptr(U), _ptr(dGU), M, N, K, _ld(dO, K, K),
                                 _ld(Wd, N, N), _ld(G, N, N), _ld(dGU, 2 * N, 2 * N), _stream(stream))
    _check("fused_swiglu_bwd", st)
    return dGU


HEAD_DIM = 128
_BF16, _U8, _I32, _F32 = torch.bfloat16, torch.uint8, torch.int32, torch.float32

# The attention calls are made once per layer and token, so their checks are written for few Python steps: a device
# is an index, pointers go to ctypes as plain integers, a contiguous tensor is asked for nothing further, and the
# device is switched only where the tensors are not on the current one.


def _addr(t):
    return None if t is None else t.data_ptr()


def _on(dev, call, args, stream):
    """Runs call(*args, stream) on device `dev` (an index) and its current stream, or on the stream given."""
    if dev < 0:
        raise ValueError("expected CUDA tensors")
    if torch._C._cuda_getDevice() == dev:
        return call(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)
    with torch.cuda.device(dev):
        return call(*args, torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream)


def _pitch(a, b, rows, width, what):
    """The shared leading dimension of two [rows, width] tensors with unit column stride."""
    if a.is_contiguous() and b.is_contiguous():
        return width
    (ld, one), (ld_b, one_b) = a.stride(), b.stride()
    if width > 1 and (one != 1 or one_b != 1) or rows > 1 and ld != ld_b:
        raise ValueError(f"{what}: expected unit column stride and one shared pitch")
    return ld if rows > 1 else width


def _kv_pair(K, V, k_scale, v_scale, dev):
    """Checks K and V rows: bf16 without scales, or E4M3 bytes (uint8) with fp32 [rows, n_kv_heads] scales; returns
    (rows, width, leading dimension, that of the scales, type)."""
    shape, dt = K.shape, K.dtype
    if len(shape) != 2 or shape[1] % HEAD_DIM or V.shape != shape or V.dtype is not dt or V.get_device() != dev or \
            K.get_device() != dev:
        raise ValueError(f"K and V: expected two tensors [rows, n_kv_heads * {HEAD_DIM}] of one type on the call's "
                         "device")
    rows, width = shape
    ld = _pitch(K, V, rows, width, "K and V")
    if dt is _BF16:
        if k_scale is not None or v_scale is not None:
            raise ValueError("bf16 rows have no scales")
        return rows, width, ld, 0, FL_BF16
    if dt is not _U8 or k_scale is None or v_scale is None:
        raise ValueError("K and V: expected bf16 rows, or uint8 (E4M3) rows with k_scale and v_scale")
    heads = width // HEAD_DIM
    if k_scale.dtype is not _F32 or v_scale.dtype is not _F32 or k_scale.shape != (rows, heads) or \
            v_scale.shape != (rows, heads) or k_scale.get_device() != dev or v_scale.get_device() != dev:
        raise ValueError("k_scale and v_scale: expected fp32 [rows, n_kv_heads] on the call's device")
    return rows, width, ld, _pitch(k_scale, v_scale, rows, heads, "k_scale and v_scale"), FL_E4M3


def _ints(t, name, dev):
    if t.dtype is not _I32 or t.dim() != 1 or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous int32 vector on the call's device")
    return t.numel()


def _page_pitch(a, b, shape, per_page, what):
    """The shared pitch of two page arrays whose pages are contiguous blocks of per_page elements."""
    if a.is_contiguous() and b.is_contiguous():
        return per_page
    n, pitch = shape[0], a.stride(0) if shape[0] > 1 else per_page
    inner, size = [], 1
    for d in reversed(shape[1:]):
        inner.insert(0, size)
        size *= d
    for t in (a, b):
        if n and (t.stride()[1:] != tuple(inner) or (n > 1 and t.stride(0) != pitch)):
            raise ValueError(f"{what}: expected contiguous pages with one shared pitch")
    return pitch


def _cache(k_pages, v_pages, page_table, seq_lens, ks, vs, dev):
    """Checks the paged cache; returns (batch, n_kv_heads, page_size, num_pages, max_pages, ldt, page_pitch,
    scale_pitch, type)."""
    shape, dt = k_pages.shape, k_pages.dtype
    if len(shape) != 4 or shape[3] != HEAD_DIM or v_pages.shape != shape or v_pages.dtype is not dt or \
            k_pages.get_device() != dev or v_pages.get_device() != dev:
        raise ValueError(f"k_pages and v_pages: expected two tensors [num_pages, n_kv_heads, page_size, {HEAD_DIM}] "
                         "of one type on the call's device")
    n_pages, n_kv, page, _ = shape
    pitch = _page_pitch(k_pages, v_pages, shape, n_kv * page * HEAD_DIM, "k_pages and v_pages")
    spitch, kind = 0, FL_BF16
    if dt is _U8:
        kind = FL_E4M3
        if ks is None or vs is None:
            raise ValueError("an E4M3 cache needs k_page_scale and v_page_scale")
        if ks.dtype is not _F32 or vs.dtype is not _F32 or ks.shape != shape[:3] or vs.shape != shape[:3] or \
                ks.get_device() != dev or vs.get_device() != dev:
            raise ValueError("k_page_scale and v_page_scale: expected fp32 [num_pages, n_kv_heads, page_size] on the "
                             "call's device")
        spitch = _page_pitch(ks, vs, shape[:3], n_kv * page, "k_page_scale and v_page_scale")
    elif dt is not _BF16:
        raise ValueError("k_pages and v_pages: expected bf16 or uint8 (E4M3)")
    elif ks is not None or vs is not None:
        raise ValueError("a bf16 cache has no scales")
    batch, t_shape = _ints(seq_lens, "seq_lens", dev), page_table.shape
    if page_table.dtype is not _I32 or len(t_shape) != 2 or t_shape[0] != batch or page_table.get_device() != dev:
        raise ValueError("page_table: expected int32 [batch, max_pages] on the call's device")
    ldt = max_pages = t_shape[1]
    if not page_table.is_contiguous():
        ldt, one = page_table.stride()
        if one != 1 and max_pages > 1:
            raise ValueError("page_table: expected unit column stride")
        if batch <= 1:
            ldt = max_pages
    return batch, n_kv, page, n_pages, max_pages, ldt, pitch, spitch, kind


def _query(t, name, dev):
    """Checks Q or O, bf16 [rows, n_heads * 128]; returns (rows, width, leading dimension)."""
    shape = t.shape
    if t.dtype is not _BF16 or len(shape) != 2 or shape[1] % HEAD_DIM or t.get_device() != dev:
        raise ValueError(f"{name}: expected bf16 [rows, n_heads * {HEAD_DIM}] on the call's device")
    rows, width = shape
    if t.is_contiguous():
        return rows, width, width
    ld, one = t.stride()
    if one != 1 and width > 1:
        raise ValueError(f"{name}: expected unit column stride")
    return rows, width, ld if rows > 1 else width


def _space(t, dev):
    if t.dtype is not _U8 or t.get_device() != dev or not t.is_contiguous():
        raise ValueError("workspace: expected a contiguous uint8 tensor on the call's device")
    return t.numel()


def paged_kv_append(K, V, k_pages, v_pages, page_table, seq_lens, cu_seqlens=None, k_scale=None, v_scale=None,
                    k_page_scale=None, v_page_scale=None, stream=None):
    """Puts K/V rows [T, n_kv_heads * 128] into the pages of a cache [num_pages, n_kv_heads, page_size, 128].

    The rows of sequence b (cu_seqlens[b] .. cu_seqlens[b + 1] - 1; without cu_seqlens row b alone) become its
    last tokens: seq_lens holds the lengths after the call.  bf16 rows go into a bf16 cache as they are and into
    an E4M3 cache (uint8 pages with fp32 page scales) quantised with one scale per (token, kv head); uint8 rows
    with k_scale and v_scale (as fused_qkv_rope_fp8kv returns them) go into an E4M3 cache as they are."""
    dev = K.get_device()
    T, width, ld, lds, rows_dt = _kv_pair(K, V, k_scale, v_scale, dev)
    batch, n_kv, page, n_pages, max_pages, ldt, pitch, spitch, dt = _cache(k_pages, v_pages, page_table, seq_lens,
                                                                          k_page_scale, v_page_scale, dev)
    if width != n_kv * HEAD_DIM:
        raise ValueError("the rows must have the cache's n_kv_heads")
    if cu_seqlens is not None and _ints(cu_seqlens, "cu_seqlens", dev) != batch + 1:
        raise ValueError("cu_seqlens must have batch + 1 entries")
    st = _on(dev, load().paged_kv_append,
             (K.data_ptr(), V.data_ptr(), _addr(k_scale), _addr(v_scale), k_pages.data_ptr(), v_pages.data_ptr(),
              _addr(k_page_scale), _addr(v_page_scale), page_table.data_ptr(), seq_lens.data_ptr(), _addr(cu_seqlens),
              T, batch, n_kv, HEAD_DIM, page, n_pages, max_pages, ld, lds, ldt, pitch, spitch, rows_dt, dt), stream)
    if st:
        _check("paged_kv_append", st)


def _fresh(n: int, head: int, device) -> torch.Tensor:
    """A workspace of n bytes, its first `head` bytes (status and counters; the rest is written before it is read) zero."""
    t = torch.empty(n, dtype=torch.uint8, device="cuda" if device is None else device)
    t[:head].zero_()
    return t


def attention_decode_workspace(device=None) -> torch.Tensor:
    """A workspace for attention_decode calls of any shape (one for each set of calls that may overlap)."""
    return _fresh(load().fl_attention_decode_workspace_bytes(), 4096, device)


def attention_decode(Q, k_pages, v_pages, page_table, seq_lens, k_page_scale=None, v_page_scale=None, scale=None,
                     O=None, workspace=None, stream=None):
    """Attention of one new token per sequence, Q bf16 [batch, n_heads * 128], over the paged cache.

    scale: of the logits, 1 / sqrt(128) by default.  Returns O bf16 [batch, n_heads * 128]."""
    if stream is not None and (O is None or workspace is None):  # what is made here belongs to that stream, too
        with torch.cuda.stream(stream):
            return attention_decode(Q, k_pages, v_pages, page_table, seq_lens, k_page_scale, v_page_scale, scale, O,
                                    workspace)
    dev = Q.get_device()
    rows, width, ldq = _query(Q, "Q", dev)
    batch, n_kv, page, n_pages, max_pages, ldt, pitch, spitch, dt = _cache(k_pages, v_pages, page_table, seq_lens,
                                                                          k_page_scale, v_page_scale, dev)
    if rows != batch:
        raise ValueError("Q: expected one row for each sequence")
    if O is None:
        O = torch.empty((rows, width), dtype=_BF16, device=Q.device)
    o_rows, o_width, ldo = _query(O, "O", dev)
    if o_rows != rows or o_width != width:
        raise ValueError("O must have Q's shape")
    if workspace is None:
        workspace = attention_decode_workspace(Q.device)
    st = _on(dev, load().attention_decode,
             (Q.data_ptr(), k_pages.data_ptr(), v_pages.data_ptr(), _addr(k_page_scale), _addr(v_page_scale),
              page_table.data_ptr(), seq_lens.data_ptr(), O.data_ptr(), batch, width // HEAD_DIM, n_kv, HEAD_DIM, page,
              n_pages, max_pages, ldq, ldo, ldt, pitch, spitch, HEAD_DIM ** -0.5 if scale is None else scale, dt,
              workspace.data_ptr(), _space(workspace, dev)), stream)
    if st:
        _check("attention_decode", st)
    return O


def attention_prefill_workspace(rows: int, n_kv_heads: int, fp8: bool, device=None) -> torch.Tensor:
    """A workspace for attention_prefill calls of up to `rows` rows."""
    n = load().fl_attention_prefill_workspace_bytes(int(rows), int(n_kv_heads), FL_E4M3 if fp8 else FL_BF16)
    return _fresh(n, 512, device)


def attention_prefill(Q, K, V, cu_seqlens=None, seq_len: int = 0, k_scale=None, v_scale=None, causal: bool = True,
                      scale=None, O=None, workspace=None, stream=None):
    """Attention over whole prompts, Q bf16 [M, n_heads * 128], K and V [M, n_kv_heads * 128] bf16 or uint8 (E4M3
    codes with fp32 [M, n_kv_heads] scales, as fused_qkv_rope_fp8kv returns them).

    Sequence b is rows cu_seqlens[b] .. cu_seqlens[b + 1] - 1; without cu_seqlens the rows are sequences of
    seq_len tokens laid end to end (0: one sequence).  Rows of O in no sequence stay as they were (zeros where O
    is allocated here).  scale: of the logits, 1 / sqrt(128) by default.  Returns O bf16 [M, n_heads * 128].

    A wait in the kernel that runs out (set_wait_timeout_ns) leaves O incomplete: check_device_status(workspace)
    says so once, and the workspace serves the next call as it is."""
    if stream is not None and (O is None or workspace is None):
        with torch.cuda.stream(stream):
            return attention_prefill(Q, K, V, cu_seqlens, seq_len, k_scale, v_scale, causal, scale, O, workspace)
    dev = Q.get_device()
    M, width, ldq = _query(Q, "Q", dev)
    rows, kv_width, ldkv, lds, dt = _kv_pair(K, V, k_scale, v_scale, dev)
    if rows != M:
        raise ValueError("Q, K and V must have the same number of rows")
    n_kv = kv_width // HEAD_DIM
    batch = 0 if cu_seqlens is None else _ints(cu_seqlens, "cu_seqlens", dev) - 1
    if batch < 0:
        raise ValueError("cu_seqlens must have batch + 1 entries")
    if O is None:
        O = (torch.empty if cu_seqlens is None else torch.zeros)((M, width), dtype=_BF16, device=Q.device)
    o_rows, o_width, ldo = _query(O, "O", dev)
    if o_rows != M or o_width != width:
        raise ValueError("O must have Q's shape")
    if workspace is None:
        workspace = attention_prefill_workspace(M, n_kv, dt == FL_E4M3, Q.device)
    st = _on(dev, load().attention_prefill,
             (Q.data_ptr(), K.data_ptr(), V.data_ptr(), _addr(k_scale), _addr(v_scale), _addr(cu_seqlens),
              O.data_ptr(), M, batch, width // HEAD_DIM, n_kv, HEAD_DIM, min(seq_len, M) or max(M, 1), ldq, ldkv, lds, ldo,
              HEAD_DIM ** -0.5 if scale is None else scale, 1 if causal else 0, dt, workspace.data_ptr(),
              _space(workspace, dev)), stream)
    if st:
        _check("attention_prefill", st)
    return O


def device_status(stream=None) -> int:
    """Synchronises the stream; returns (and clears) the device-wide failure code."""
    return load().fl_device_status(_stream(stream))


def check_device_status(workspace=None, stream=None) -> int:
    """Synchronises the stream; returns (and clears) the failure code recorded in `workspace`
    (a workspace of the RMSNorm + FP8, cross-entropy or attention calls); None: the device-wide word."""
    return load().fl_check_device_status(_ptr(workspace), _stream(stream))


def set_cooperative_launch(enable: bool) -> None:
    """Cooperative attribute on the RMSNorm prefill launch (default on); off only for profilers
    that refuse cooperative launches of clusters."""
    load().fl_set_cooperative_launch(1 if enable else 0)


def set_descriptor_cache(enable: bool) -> None:
    """Tensor-map descriptor cache on (default) or off (and emptied)."""
    load().fl_set_descriptor_cache(1 if enable else 0)


def descriptor_cache_stats() -> tuple[int, int]:
    """(hits, misses) of the tensor-map descriptor cache since the process started."""
    h, m = ctypes.c_ulonglong(0), ctypes.c_ulonglong(0)
    load().fl_descriptor_cache_stats(ctypes.byref(h), ctypes.byref(m))
    return h.value, m.value


def set_wait_timeout_ns(ns: int) -> None:
    load().fl_set_wait_timeout_ns(int(ns))


def set_max_ctas(n: int) -> None:
    load().fl_set_max_ctas(int(n))


def set_cta_pairing(enable: bool) -> None:
    """Two-CTA (cta_group::2) prefill tiles on (default) or off; results are the same."""
    load().fl_set_cta_pairing(1 if enable else 0)


DECODE_GELU, DECODE_SWIGLU, DECODE_QKV, DECODE_QKV_FP8KV, DECODE_QUANT = 0, 1, 2, 3, 4
DECODE_RESID_GAMMA, DECODE_ROWSCALE = 5, 6


def linear_decode_shape(kind: int, M: int, N: int, K: int) -> tuple[int, int, int]:
    """(CTAs per W-row tile, CTAs per SM, launches) that a decode-shaped call would use on the current
    device; (0, 0, 0) when it would run on the GEMM kernel.  N: the rows of W (SwiGLU: d_ff; QKV:
    3 * d_model; QKV + FP8 K/V: (n_heads + 2 * n_kv_heads) * head_dim; block-scaled and the chain: N)."""
    out = [ctypes.c_int(0) for _ in range(3)]
    _check("fl_linear_decode_shape", load().fl_linear_decode_shape(kind, M, N, K, *(ctypes.byref(o) for o in out)))
    return tuple(o.value for o in out)


def set_linear_decode(enable: bool) -> None:
    """Decode kernels for M <= 32 calls of fused_linear_gelu (bf16), fused_swiglu, fused_qkv_rope,
    fused_qkv_rope_fp8kv, fused_linear_quant and both chain steps on (default) or off (the prefill
    GEMM kernel then takes them)."""
    load().fl_set_linear_decode(1 if enable else 0)
