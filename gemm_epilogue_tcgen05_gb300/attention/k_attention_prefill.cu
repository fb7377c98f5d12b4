// attention_prefill: argument checks, tensor maps and launch (the kernel: prefill_attention_kernel.cuh).
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <mutex>

#include "prefill_attention_kernel.cuh"

namespace fl {
namespace {

constexpr int64_t kL2Share = 32 << 20;  // keys and values of the heads worked off together
// The order of the tiles: by falling cost, with a walk over the sequences for each tier of blocks, or in the order of the
// sequences, with one walk.  Up to 32 sequences stay in a warp's lanes and a tier costs little.  Measured, causal | full
// mask, 32 query and 8 kv heads (tiers -> one walk): 4 x 2048 108 -> 113 | 176 -> 177 us, 32 of 200-2000 tokens and one
// of 8000 523 -> 539 | 894 -> 899, 64 of 20-1500 154 -> 158 | 207 -> 214, 64 of 200-2000 and one of 8000 916 -> 686 |
// 1143 -> 1184, 128 of 20-1500 and one of 4000 765 -> 356 | 623 -> 520, 1024 of 20-100 and one of 8000 9945 -> 634 |
// 5180 -> 863.
constexpr int kTierBatch = 32, kTierBatchFull = 64;

// 3-D tiled map over Q [rows][heads][128] bf16 with a row pitch of ld elements.
bool encode_q(CUtensorMap* map, const void* base, int heads, int rows, int64_t ld, int hp, int tq) {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) == cudaSuccess &&
        r == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {kHeadDim, static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {kHeadDim * 2, static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(hp), static_cast<cuuint32_t>(tq)}, step[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class Kernel, class... Args>
bool launch_dependent(Kernel* kernel, dim3 grid, int threads, int smem, cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;  // see griddep_wait in the kernels
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

template <bool FP8>
int launch_prefill(const PrefillParams& p, long long tiles, const DeviceInfo& di, cudaStream_t s) {
  using T = PrefillTraits;
  const void* fn = reinterpret_cast<const void*>(&attention_prefill_kernel<FP8>);
  if (!ensure_smem_attr(fn, di.device, T::kSmem)) return FL_ERR_CUDA;
  // the warps share out the registers of the launch: with any other number of them the kernel would not start
  static std::atomic<int> regs{0};
  if (regs.load() == 0) {
    cudaFuncAttributes a;
    if (cudaFuncGetAttributes(&a, fn) != cudaSuccess) return FL_ERR_CUDA;
    regs.store(a.numRegs);
  }
  if (regs.load() != kPreRegs) return FL_ERR_UNSUPPORTED;
  const int grid = tiles < di.num_sms ? static_cast<int>(tiles) : di.num_sms;
  return launch_dependent(attention_prefill_kernel<FP8>, grid, kPreThreads, T::kSmem, s, p) ? FL_OK : FL_ERR_CUDA;
}

}  // namespace
}  // namespace fl

extern "C" size_t fl_attention_prefill_workspace_bytes(int M, int n_kv_heads, int kv_dtype) {
  using namespace fl;
  if (M < 0 || n_kv_heads < 0) return 0;
  // the status record and the work counters; for E4M3 also K as bf16, V as fp16 and a power for each key tile (kept at
  // its first row; where it has single keys, the other rows hold which)
  const size_t rows = static_cast<size_t>(M) * n_kv_heads;
  return 2 * kWsStatusBytes + (kv_dtype == FL_E4M3 ? rows * (kHeadDim * (sizeof(__nv_bfloat16) + sizeof(__half)) + sizeof(float)) : 0);
}

extern "C" int attention_prefill(const void* Q, const void* K, const void* V, const float* k_scale,
                                 const float* v_scale, const int32_t* cu_seqlens, void* O, int M, int batch,
                                 int n_heads, int n_kv_heads, int head_dim, int seq_len, int64_t ldq, int64_t ldkv,
                                 int64_t lds, int64_t ldo, float scale, int causal, int kv_dtype, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  using namespace fl;
  if (M < 0 || n_heads < 0 || n_kv_heads < 0 || (cu_seqlens != nullptr ? batch < 0 : seq_len < 1))
    return FL_ERR_INVALID_ARG;
  const bool fp8 = kv_dtype == FL_E4M3;
  float scale_log2;
  if ((kv_dtype != FL_BF16 && !fp8) || !scale_to_base_2(scale, &scale_log2)) return FL_ERR_INVALID_ARG;
  if (M == 0 || n_heads == 0 || (cu_seqlens != nullptr && batch == 0)) return FL_OK;
  if (n_kv_heads == 0 || n_heads % n_kv_heads != 0) return FL_ERR_INVALID_ARG;
  if (head_dim != kHeadDim) return FL_ERR_UNSUPPORTED;
  if (n_heads > kMaxHeads) return FL_ERR_UNSUPPORTED;
  if (Q == nullptr || K == nullptr || V == nullptr || O == nullptr) return FL_ERR_INVALID_ARG;
  if (fp8 && (k_scale == nullptr || v_scale == nullptr)) return FL_ERR_INVALID_ARG;
  const int64_t width = static_cast<int64_t>(n_heads) * kHeadDim, kv_width = static_cast<int64_t>(n_kv_heads) * kHeadDim;
  if (ldq < width || ldo < width || ldkv < kv_width || (fp8 && lds < n_kv_heads)) return FL_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(O)) return FL_ERR_ALIGNMENT;
  if (!pitch_ok(ldq, 2) || !pitch_ok(ldo, 2) || !pitch_ok(ldkv, fp8 ? 1 : 2)) return FL_ERR_ALIGNMENT;
  if (((reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale) |
        reinterpret_cast<uintptr_t>(cu_seqlens)) & 3u) != 0)
    return FL_ERR_ALIGNMENT;
  if (workspace == nullptr || workspace_bytes < fl_attention_prefill_workspace_bytes(M, n_kv_heads, kv_dtype))
    return FL_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & (kWsStatusBytes - 1)) != 0) return FL_ERR_ALIGNMENT;
  DeviceInfo di;
  const int st = current_device(&di);
  if (st != FL_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);

  PrefillParams p;
  std::memset(&p, 0, sizeof(p));
  p.group = n_heads / n_kv_heads;
  // heads of a tile: the largest part of the group that leaves room for two tokens
  p.hp = p.group < 64 ? p.group : 64;
  while (p.group % p.hp != 0) --p.hp;
  p.tq = kPreTile / p.hp;
  p.pairs = n_heads / p.hp;
  const int64_t kv_bytes = static_cast<int64_t>(M) * kHeadDim * 4;  // of one kv head, as bf16
  const int64_t at_once = std::max<int64_t>(kL2Share / kv_bytes, 1);
  const int64_t groups = (n_kv_heads + at_once - 1) / at_once;
  p.pairs_at_once = static_cast<int>((n_kv_heads + groups - 1) / groups) * (p.group / p.hp);
  p.batch = cu_seqlens == nullptr ? (M - 1) / seq_len + 1 : batch;
  p.seq_len = seq_len;
  const long long per_cta = 2 * p.tq;
  const long long blocks = cu_seqlens == nullptr
                               ? (M / seq_len) * ((seq_len - 1) / per_cta + 1) + (M % seq_len + per_cta - 1) / per_cta
                               : M / per_cta + batch;  // an upper bound: the lengths are on the device
  if (blocks * p.pairs > (1ll << 30)) return FL_ERR_UNSUPPORTED;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const void* k16 = K;
  const void* v16 = V;
  int64_t ld16 = ldkv;
  if (fp8) {
    __nv_bfloat16* kw = reinterpret_cast<__nv_bfloat16*>(ws + 2 * kWsStatusBytes);
    __half* vw = reinterpret_cast<__half*>(kw + static_cast<size_t>(M) * kv_width);
    p.powers = reinterpret_cast<const float*>(vw + static_cast<size_t>(M) * kv_width);
    k16 = kw, v16 = vw, ld16 = kv_width;
    p.codes = static_cast<const uint8_t*>(V);
    p.v_scale = v_scale;
    p.ld_codes = ldkv;
    p.ld_scale = lds;
  }
  if (!encode_q(&p.map_q, Q, n_heads, M, ldq, p.hp, p.tq) ||
      !encode_2d(&p.map_k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, k16, kv_width, M, ld16, 64, kPreTile,
                 CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_2d(&p.map_v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, v16, kv_width, M, ld16, 64, kPreTile,
                 CU_TENSOR_MAP_SWIZZLE_128B))
    return FL_ERR_CUDA;
  p.V = static_cast<const __nv_bfloat16*>(v16);
  p.ldv = ld16;
  p.n_kv = n_kv_heads;
  p.cu = cu_seqlens;
  p.O = static_cast<__nv_bfloat16*>(O);
  p.ldo = ldo;
  p.M = M;
  p.causal = causal != 0;
  p.flat = p.batch > (p.causal ? kTierBatch : kTierBatchFull);
  p.scale_log2 = scale_log2;
  p.status = reinterpret_cast<int*>(ws);
  p.work = reinterpret_cast<unsigned*>(ws + kWsStatusBytes);
  p.timeout_ns = wait_timeout_ns();
  if (!fp8) return launch_prefill<false>(p, blocks * p.pairs, di, s);
  const long long key_tiles =
      cu_seqlens == nullptr
          ? static_cast<long long>(M / seq_len) * ((seq_len - 1) / kPreTile + 1) + (M % seq_len + kPreTile - 1) / kPreTile
          : static_cast<long long>(M) / kPreTile + batch;  // the numbers that tiles can have
  const long long parts = key_tiles * (kPreTile / kCodesRows);
  if (parts > INT32_MAX) return FL_ERR_UNSUPPORTED;
  if (!launch_dependent(e4m3_tiles_kernel, dim3(static_cast<unsigned>(parts), (n_kv_heads - 1) / kCodesHeads + 1), 256, 0, s,
                        static_cast<const uint8_t*>(K),
                        static_cast<const uint8_t*>(V), k_scale, v_scale, static_cast<long long>(ldkv),
                        static_cast<long long>(lds), cu_seqlens, p.batch, seq_len, M, n_kv_heads,
                        static_cast<__nv_bfloat16*>(const_cast<void*>(k16)), static_cast<__half*>(const_cast<void*>(v16)),
                        const_cast<float*>(p.powers)))
    return FL_ERR_CUDA;
  return launch_prefill<true>(p, blocks * p.pairs, di, s);
}
