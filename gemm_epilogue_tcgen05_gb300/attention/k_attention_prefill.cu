// attention_prefill: attention over whole prompts, packed one behind the other.
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = exp(scale * q_i . k_j - max_j), over the keys j of i's own
//   sequence (causal: j <= i).
// One warp takes one (row, query head) and walks the keys once with the running maximum and sum; a lane
// holds 4 of the 128 dimensions.
#include "attention_common.h"

namespace fl {
namespace {

struct PrefillParams {
  const __nv_bfloat16* Q;
  const void* K;
  const void* V;
  const float* ks;
  const float* vs;
  const int* cu;
  __nv_bfloat16* O;
  long long ldq, ldkv, lds, ldo;
  int M, batch, n_heads, group, seq_len, causal;
  float scale;
};

template <bool FP8>
__device__ __forceinline__ float4 load4(const void* base, long long i) {
  if (FP8) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(base) + i);
    return make_float4(e4m3_to_f32(w & 255u), e4m3_to_f32((w >> 8) & 255u), e4m3_to_f32((w >> 16) & 255u),
                       e4m3_to_f32(w >> 24));
  }
  const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(base) + i);
  return make_float4(bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y));
}

template <bool FP8>
__global__ void __launch_bounds__(128) attention_prefill_kernel(const PrefillParams p) {
  const int lane = threadIdx.x & 31;
  const long long item = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (item >= static_cast<long long>(p.M) * p.n_heads) return;
  const int r = static_cast<int>(item / p.n_heads), head = static_cast<int>(item % p.n_heads), kvh = head / p.group;
  int first = 0, last = 0;
  for (int b = 0; b < p.batch; ++b) {
    sequence_rows(p.cu, b, p.seq_len, p.M, first, last);
    if (r >= first && r < last) break;
  }
  if (r < first || r >= last) return;  // a row of no sequence stays as it is
  const int end = p.causal ? r + 1 : last;
  const float4 q = load4<false>(p.Q, r * p.ldq + head * kHeadDim + lane * 4);
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j = first; j < end; ++j) {
    const long long at = j * p.ldkv + kvh * kHeadDim + lane * 4;
    const float4 k = load4<FP8>(p.K, at), v = load4<FP8>(p.V, at);
    float s = q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
    float vs = 1.f;
    if (FP8) {
      s *= p.ks[j * p.lds + kvh];
      vs = p.vs[j * p.lds + kvh];
    }
    s *= p.scale;
    const float mn = fmaxf(m, s), ref = mn == -INFINITY ? 0.f : mn;
    const float a = expf(m - ref), w = expf(s - ref);
    m = mn;
    l = l * a + w;
    o.x = o.x * a + w * vs * v.x;
    o.y = o.y * a + w * vs * v.y;
    o.z = o.z * a + w * vs * v.z;
    o.w = o.w * a + w * vs * v.w;
  }
  const float inv = 1.f / l;
  uint2 w;
  w.x = pack_bf16x2(o.x * inv, o.y * inv);
  w.y = pack_bf16x2(o.z * inv, o.w * inv);
  *reinterpret_cast<uint2*>(p.O + r * p.ldo + head * kHeadDim + lane * 4) = w;
}

}  // namespace
}  // namespace fl

extern "C" size_t fl_attention_prefill_workspace_bytes(int M, int n_kv_heads, int kv_dtype) {
  using namespace fl;
  if (M < 0 || n_kv_heads < 0) return 0;
  // the status record, and the E4M3 codes of K and V as bf16
  return 2 * kWsStatusBytes +
         (kv_dtype == FL_E4M3 ? static_cast<size_t>(M) * n_kv_heads * kHeadDim * 2 * sizeof(__nv_bfloat16) : 0);
}

extern "C" int attention_prefill(const void* Q, const void* K, const void* V, const float* k_scale,
                                 const float* v_scale, const int32_t* cu_seqlens, void* O, int M, int batch,
                                 int n_heads, int n_kv_heads, int head_dim, int seq_len, int64_t ldq, int64_t ldkv,
                                 int64_t lds, int64_t ldo, float scale, int causal, int kv_dtype, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  using namespace fl;
  if (M < 0 || n_heads < 0 || n_kv_heads < 0 || (cu_seqlens != nullptr ? batch < 0 : seq_len < 1))
    return FL_ERR_INVALID_ARG;
  const bool fp8 = kv_dtype == FL_E4M3;
  if ((kv_dtype != FL_BF16 && !fp8) || !positive_finite(scale)) return FL_ERR_INVALID_ARG;
  if (M == 0 || n_heads == 0 || (cu_seqlens != nullptr && batch == 0)) return FL_OK;
  if (n_kv_heads == 0 || n_heads % n_kv_heads != 0) return FL_ERR_INVALID_ARG;
  if (head_dim != kHeadDim) return FL_ERR_UNSUPPORTED;
  if (Q == nullptr || K == nullptr || V == nullptr || O == nullptr) return FL_ERR_INVALID_ARG;
  if (fp8 && (k_scale == nullptr || v_scale == nullptr)) return FL_ERR_INVALID_ARG;
  const int64_t width = static_cast<int64_t>(n_heads) * kHeadDim, kv_width = static_cast<int64_t>(n_kv_heads) * kHeadDim;
  if (ldq < width || ldo < width || ldkv < kv_width || (fp8 && lds < n_kv_heads)) return FL_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(O)) return FL_ERR_ALIGNMENT;
  if (!pitch_ok(ldq, 2) || !pitch_ok(ldo, 2) || !pitch_ok(ldkv, fp8 ? 1 : 2)) return FL_ERR_ALIGNMENT;
  if (((reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale) |
        reinterpret_cast<uintptr_t>(cu_seqlens)) & 3u) != 0)
    return FL_ERR_ALIGNMENT;
  if (workspace == nullptr || workspace_bytes < fl_attention_prefill_workspace_bytes(M, n_kv_heads, kv_dtype))
    return FL_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & (kWsStatusBytes - 1)) != 0) return FL_ERR_ALIGNMENT;
  const long long items = static_cast<long long>(M) * n_heads;
  if ((items + 3) / 4 > 0x7FFFFFFFll) return FL_ERR_UNSUPPORTED;
  DeviceInfo di;
  const int st = current_device(&di);
  if (st != FL_OK) return st;
  if (cu_seqlens == nullptr) batch = (M - 1) / seq_len + 1;
  const PrefillParams p{static_cast<const __nv_bfloat16*>(Q), K, V, k_scale, v_scale, cu_seqlens,
                        static_cast<__nv_bfloat16*>(O), ldq, ldkv, lds, ldo, M, batch, n_heads,
                        n_heads / n_kv_heads, seq_len, causal, scale};
  const int grid = static_cast<int>((items + 3) / 4);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (fp8) attention_prefill_kernel<true><<<grid, 128, 0, s>>>(p);
  else attention_prefill_kernel<false><<<grid, 128, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? FL_OK : FL_ERR_CUDA;
}
