// The decode kernel's variants with a window over bf16 and E4M3 caches (attention_decode_window).
#include "decode_attention_host.cuh"
#include "decode_attention_kernel.cuh"

namespace fl {

int launch_decode_window(const DecodeParams& p, bool fp8, const DeviceInfo& di, cudaStream_t s) {
  auto launch = [&](auto traits, auto* kernel) { return launch_decode<decltype(traits)>(kernel, p, di, s); };
  return fp8 ? decode_tiles<true, true>(p, launch) : decode_tiles<false, true>(p, launch);
}

}  // namespace fl
