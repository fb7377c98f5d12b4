// Launch of the decode kernel (decode_attention_kernel.cuh), for the translation units that hold its variants.
#pragma once
#include "decode_attention_kernel.cuh"

namespace fl {

template <int KIND, int NT, bool WIN>
int launch_decode(const DecodeParams& p, const DeviceInfo& di, cudaStream_t s) {
  using T = DecodeTraits<KIND, NT>;
  const void* fn = reinterpret_cast<const void*>(&attention_decode_kernel<KIND, NT, WIN>);
  if (!ensure_smem_attr(fn, di.device, T::kSmem)) return FL_ERR_CUDA;
  const int grid = T::kCtas * di.num_sms < kDecMaxCtas ? T::kCtas * di.num_sms : kDecMaxCtas;
  return launch_dependent(attention_decode_kernel<KIND, NT, WIN>, dim3(grid), kDecThreads, T::kSmem, s, p) ? FL_OK : FL_ERR_CUDA;
}

// Of a group of up to 16 query heads: one column tile or two.
template <int KIND, bool WIN>
int launch_decode_tiles(const DecodeParams& p, const DeviceInfo& di, cudaStream_t s) {
  return p.chunk_heads <= 8 ? launch_decode<KIND, 1, WIN>(p, di, s) : launch_decode<KIND, 2, WIN>(p, di, s);
}

// bf16 and E4M3 with a window (k_attention_decode_window.cu), 4 bits without and with one (k_attention_decode_int4.cu).
int launch_decode_window(const DecodeParams& p, bool fp8, const DeviceInfo& di, cudaStream_t s);
int launch_decode_int4(const DecodeParams& p, bool window, const DeviceInfo& di, cudaStream_t s);

}  // namespace fl
