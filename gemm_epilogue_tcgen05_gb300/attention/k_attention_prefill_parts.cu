// The prefill kernel's variants whose units are cut along their keys, and the join of the parts (attention_prefill_window).
#include "prefill_attention_host.cuh"

namespace fl {

int launch_prefill_parts(const PrefillParams& p, bool fp8, long long numbers, const DeviceInfo& di, cudaStream_t s) {
  const int st = fp8 ? launch_prefill<true, true, true>(p, numbers, di, s) : launch_prefill<false, true, true>(p, numbers, di, s);
  if (st != FL_OK) return st;
  const PrefillJoinParams join{p.parts, p.cuts, p.hp, p.tq, p.O, p.ldo};
  return launch_dependent(fp8 ? attention_prefill_join_kernel<true> : attention_prefill_join_kernel<false>,
                          dim3(static_cast<unsigned>(numbers), 2, kHeadDim / 32), kPreTile, 0, s, join)
             ? FL_OK
             : FL_ERR_CUDA;
}

}  // namespace fl
