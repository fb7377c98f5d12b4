// The decode kernel's variants with a window over bf16 and E4M3 caches (attention_decode_window).
#include "decode_attention_host.cuh"

namespace fl {

int launch_decode_window(const DecodeParams& p, bool fp8, const DeviceInfo& di, cudaStream_t s) {
  return fp8 ? launch_decode_tiles<FL_E4M3, true>(p, di, s) : launch_decode_tiles<FL_BF16, true>(p, di, s);
}

}  // namespace fl
