// The decode kernel's variants over a 4-bit cache (attention_decode_window).
#include "decode_attention_host.cuh"

namespace fl {

int launch_decode_int4(const DecodeParams& p, bool window, const DeviceInfo& di, cudaStream_t s) {
  return window ? launch_decode_tiles<FL_INT4, true>(p, di, s) : launch_decode_tiles<FL_INT4, false>(p, di, s);
}

}  // namespace fl
