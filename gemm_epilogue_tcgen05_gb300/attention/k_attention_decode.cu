// attention_decode: argument checks and launch (the kernel and its design: decode_attention_kernel.cuh).
#include <algorithm>
#include <cstdint>

#include "decode_attention_kernel.cuh"

namespace fl {
namespace {

constexpr size_t kDecWorkspace = kWsStatusBytes + kDecMaxCtas * sizeof(unsigned) +
                                 static_cast<size_t>(kDecMaxCtas) * 2 * kDecPartFloats * sizeof(float);

template <bool FP8, int NT>
int launch_decode(const DecodeParams& p, const DeviceInfo& di, cudaStream_t s) {
  using T = DecodeTraits<FP8, NT>;
  const void* fn = reinterpret_cast<const void*>(&attention_decode_kernel<FP8, NT>);
  if (!ensure_smem_attr(fn, di.device, T::kSmem)) return FL_ERR_CUDA;
  const int grid = T::kCtas * di.num_sms < kDecMaxCtas ? T::kCtas * di.num_sms : kDecMaxCtas;
  // programmatic dependent launch: only the launch itself overlaps the kernel in front (griddep_wait)
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kDecThreads);
  cfg.dynamicSmemBytes = T::kSmem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attention_decode_kernel<FP8, NT>, p) == cudaSuccess ? FL_OK : FL_ERR_CUDA;
}

}  // namespace
}  // namespace fl

extern "C" size_t fl_attention_decode_workspace_bytes(void) {
  return fl::kDecWorkspace;
}

extern "C" int attention_decode(const void* Q, const void* k_pages, const void* v_pages, const float* k_page_scale,
                                const float* v_page_scale, const int32_t* page_table, const int32_t* seq_lens, void* O,
                                int batch, int n_heads, int n_kv_heads, int head_dim, int page_size, int num_pages,
                                int max_pages, int64_t ldq, int64_t ldo, int64_t ldt, int64_t page_pitch,
                                int64_t scale_pitch, float scale, int cache_dtype, void* workspace,
                                size_t workspace_bytes, void* stream) {
  using namespace fl;
  if (batch < 0 || n_heads < 0 || n_kv_heads < 0 || page_size < 1 || num_pages < 0 || max_pages < 0)
    return FL_ERR_INVALID_ARG;
  const bool fp8 = cache_dtype == FL_E4M3;
  float scale_log2;
  if ((cache_dtype != FL_BF16 && !fp8) || !scale_to_base_2(scale, &scale_log2)) return FL_ERR_INVALID_ARG;
  if (batch == 0 || n_heads == 0) return FL_OK;
  if (n_kv_heads == 0 || n_heads % n_kv_heads != 0) return FL_ERR_INVALID_ARG;
  if (head_dim != kHeadDim) return FL_ERR_UNSUPPORTED;
  if (n_heads > kMaxHeads) return FL_ERR_UNSUPPORTED;
  if (Q == nullptr || O == nullptr) return FL_ERR_INVALID_ARG;
  const int64_t width = static_cast<int64_t>(n_heads) * kHeadDim;
  if (batch > 1 && (ldq < width || ldo < width)) return FL_ERR_INVALID_ARG;
  int st = check_cache(k_pages, v_pages, k_page_scale, v_page_scale, page_table, seq_lens, batch, n_kv_heads,
                       page_size, num_pages, max_pages, ldt, page_pitch, scale_pitch, fp8);
  if (st != FL_OK) return st;
  if (!aligned16(Q) || !aligned16(O) || (batch > 1 && (!pitch_ok(ldq, 2) || !pitch_ok(ldo, 2)))) return FL_ERR_ALIGNMENT;
  if (workspace == nullptr || workspace_bytes < fl_attention_decode_workspace_bytes()) return FL_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & (kWsStatusBytes - 1)) != 0) return FL_ERR_ALIGNMENT;
  DeviceInfo di;
  st = current_device(&di);
  if (st != FL_OK) return st;
  DecodeParams p;
  p.c = CacheView{k_pages, v_pages, k_page_scale, v_page_scale, page_table, seq_lens, page_pitch, scale_pitch, ldt,
                  n_kv_heads, page_size, num_pages, max_pages, batch};
  p.Q = static_cast<const __nv_bfloat16*>(Q);
  p.O = static_cast<__nv_bfloat16*>(O);
  p.ldq = ldq;
  p.ldo = ldo;
  p.group = n_heads / n_kv_heads;
  p.chunks = (p.group + 15) / 16;
  p.chunk_heads = (p.group + p.chunks - 1) / p.chunks;
  p.page_shift = (page_size & (page_size - 1)) == 0 ? __builtin_ctz(static_cast<unsigned>(page_size)) : -1;
  // units of all lengths that the table allows (64 tokens at least), for all heads
  const int64_t longest = std::min<int64_t>(static_cast<int64_t>(max_pages) * page_size, INT32_MAX) / 64 + 1;
  p.small = batch <= 128 && longest * batch < (int64_t{1} << 31) / (static_cast<int64_t>(n_kv_heads) * p.chunks);
  p.scale_log2 = scale_log2;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.status = reinterpret_cast<int*>(ws);
  p.counters = reinterpret_cast<unsigned*>(ws + kWsStatusBytes);
  p.parts = reinterpret_cast<float*>(ws + kWsStatusBytes + kDecMaxCtas * sizeof(unsigned));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (p.chunk_heads <= 8) return fp8 ? launch_decode<true, 1>(p, di, s) : launch_decode<false, 1>(p, di, s);
  return fp8 ? launch_decode<true, 2>(p, di, s) : launch_decode<false, 2>(p, di, s);
}
