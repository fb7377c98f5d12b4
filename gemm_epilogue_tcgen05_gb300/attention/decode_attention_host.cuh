// Launch of the decode kernels, for the translation units that hold their variants.
#pragma once
#include "decode_attention_common.cuh"

namespace fl {

// Traits: kCtas (on an SM), kThreads, kSmem.
template <class Traits, class Kernel>
int launch_decode(Kernel* kernel, const DecodeParams& p, const DeviceInfo& di, cudaStream_t s) {
  if (!ensure_smem_attr(reinterpret_cast<const void*>(kernel), di.device, Traits::kSmem)) return FL_ERR_CUDA;
  const int grid = Traits::kCtas * di.num_sms < kDecMaxCtas ? Traits::kCtas * di.num_sms : kDecMaxCtas;
  return launch_dependent(kernel, dim3(grid), Traits::kThreads, Traits::kSmem, s, p) ? FL_OK : FL_ERR_CUDA;
}

// bf16 and E4M3 with a window (k_attention_decode_window.cu), 4 bits without and with one (k_attention_decode_int4.cu).
int launch_decode_window(const DecodeParams& p, bool fp8, const DeviceInfo& di, cudaStream_t s);
int launch_decode_int4(const DecodeParams& p, bool window, const DeviceInfo& di, cudaStream_t s);

}  // namespace fl
