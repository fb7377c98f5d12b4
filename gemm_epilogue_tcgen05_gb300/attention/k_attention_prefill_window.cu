// The prefill kernel's variants with a window or with offsets of their own for the keys (attention_prefill_window).
#include "prefill_attention_host.cuh"

namespace fl {

int launch_prefill_window(const PrefillParams& p, bool fp8, long long tiles, const DeviceInfo& di, cudaStream_t s) {
  return fp8 ? launch_prefill<true, true>(p, tiles, di, s) : launch_prefill<false, true>(p, tiles, di, s);
}

}  // namespace fl
