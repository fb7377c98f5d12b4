// Launch of the prefill kernel (prefill_attention_kernel.cuh), for the translation units that hold its variants.
#pragma once
#include <atomic>

#include "prefill_attention_kernel.cuh"

namespace fl {

template <bool FP8, bool WIN, bool CUT = false>
int launch_prefill(const PrefillParams& p, long long tiles, const DeviceInfo& di, cudaStream_t s) {
  using T = PrefillTraits;
  const void* fn = reinterpret_cast<const void*>(&attention_prefill_kernel<FP8, WIN, CUT>);
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
  return launch_dependent(attention_prefill_kernel<FP8, WIN, CUT>, grid, kPreThreads, T::kSmem, s, p) ? FL_OK : FL_ERR_CUDA;
}

// The variants with a window or with offsets of their own for the keys (k_attention_prefill_window.cu), and those whose units are
// cut along the keys, with the kernel that joins the parts (k_attention_prefill_parts.cu).
int launch_prefill_window(const PrefillParams& p, bool fp8, long long tiles, const DeviceInfo& di, cudaStream_t s);
int launch_prefill_parts(const PrefillParams& p, bool fp8, long long numbers, const DeviceInfo& di, cudaStream_t s);

}  // namespace fl
