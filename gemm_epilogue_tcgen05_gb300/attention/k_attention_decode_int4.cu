// The decode kernel's variants over a 4-bit cache (attention_decode_window).
#include "decode_attention_host.cuh"
#include "decode_int4_kernel.cuh"

namespace fl {

int launch_decode_int4(const DecodeParams& p, bool window, const DeviceInfo& di, cudaStream_t s) {
  return window ? launch_decode<DecodeInt4Traits>(attention_decode_int4_kernel<true>, p, di, s)
                : launch_decode<DecodeInt4Traits>(attention_decode_int4_kernel<false>, p, di, s);
}

}  // namespace fl
