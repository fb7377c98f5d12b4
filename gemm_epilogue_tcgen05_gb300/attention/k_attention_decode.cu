// attention_decode: attention of one new token per sequence over a paged key-value cache.
//   o_h = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale * q_h . k_j - max_j), over j < seq_lens[b].
// One warp takes one (sequence, query head) and walks the cache once with the running maximum and sum;
// a lane holds 4 of the 128 dimensions.
#include "attention_common.h"

namespace fl {
namespace {

struct DecodeParams {
  CacheView c;
  const __nv_bfloat16* Q;
  __nv_bfloat16* O;
  long long ldq, ldo;
  int n_heads, group;
  float scale;
  int* status;
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
__global__ void __launch_bounds__(128) attention_decode_kernel(const DecodeParams p) {
  const int lane = threadIdx.x & 31;
  const long long item = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  if (item >= static_cast<long long>(p.c.batch) * p.n_heads) return;
  const int b = static_cast<int>(item / p.n_heads), head = static_cast<int>(item % p.n_heads), kvh = head / p.group;
  const int len = p.c.lens[b];
  bool bad = len < 0 || len > static_cast<long long>(p.c.max_pages) * p.c.page_size;
  const float4 q = load4<false>(p.Q, b * p.ldq + head * kHeadDim + lane * 4);
  float m = -INFINITY, l = 0.f;
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int j = 0; j < len && !bad; ++j) {
    const int page = p.c.table[b * p.c.ldt + j / p.c.page_size];
    if (page < 0 || page >= p.c.num_pages) {
      bad = true;
      break;
    }
    const long long cell = static_cast<long long>(kvh) * p.c.page_size + j % p.c.page_size;
    const long long at = page * p.c.page_pitch + cell * kHeadDim + lane * 4;
    const float4 k = load4<FP8>(p.c.k, at), v = load4<FP8>(p.c.v, at);
    float s = q.x * k.x + q.y * k.y + q.z * k.z + q.w * k.w;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(~0u, s, d);
    float vs = 1.f;
    if (FP8) {
      s *= p.c.ks[page * p.c.scale_pitch + cell];
      vs = p.c.vs[page * p.c.scale_pitch + cell];
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
  float inv = len == 0 ? 0.f : 1.f / l;
  if (bad) {
    inv = NAN;
    if (lane == 0 && atomicCAS(p.status + ST_CODE, 0, static_cast<int>(FL_ERR_INVALID_ARG)) == 0) p.status[ST_DETAIL] = b;
  }
  uint2 w;
  w.x = pack_bf16x2(o.x * inv, o.y * inv);
  w.y = pack_bf16x2(o.z * inv, o.w * inv);
  *reinterpret_cast<uint2*>(p.O + b * p.ldo + head * kHeadDim + lane * 4) = w;
}

}  // namespace
}  // namespace fl

extern "C" size_t fl_attention_decode_workspace_bytes(void) {
  return fl::kWsStatusBytes + 640 * 4 + 640 * 2 * 16 * 132 * sizeof(float);
}

extern "C" int attention_decode(const void* Q, const void* k_pages, const void* v_pages, const float* k_page_scale,
                                const float* v_page_scale, const int32_t* page_table, const int32_t* seq_lens, void* O,
                                int batch, int n_heads, int n_kv_heads, int head_dim, int page_size, int num_pages,
                                int max_pages, int64_t ldq, int64_t ldo, int64_t ldt, int64_t page_pitch,
                                int64_t scale_pitch, float scale, int cache_dtype, void* workspace,
                                size_t workspace_bytes, void* stream) {
  using namespace fl;
  if (batch < 0 || n_heads < 0 || n_kv_heads < 0 || page_size < 1 || num_pages < 0 || max_pages < 0)
    return FL_ERR_INVALID_ARG;
  const bool fp8 = cache_dtype == FL_E4M3;
  if ((cache_dtype != FL_BF16 && !fp8) || !positive_finite(scale)) return FL_ERR_INVALID_ARG;
  if (batch == 0 || n_heads == 0) return FL_OK;
  if (n_kv_heads == 0 || n_heads % n_kv_heads != 0) return FL_ERR_INVALID_ARG;
  if (head_dim != kHeadDim) return FL_ERR_UNSUPPORTED;
  if (Q == nullptr || O == nullptr) return FL_ERR_INVALID_ARG;
  const int64_t width = static_cast<int64_t>(n_heads) * kHeadDim;
  if (batch > 1 && (ldq < width || ldo < width)) return FL_ERR_INVALID_ARG;
  int st = check_cache(k_pages, v_pages, k_page_scale, v_page_scale, page_table, seq_lens, batch, n_kv_heads,
                       page_size, num_pages, max_pages, ldt, page_pitch, scale_pitch, fp8);
  if (st != FL_OK) return st;
  if (!aligned16(Q) || !aligned16(O) || (batch > 1 && (!pitch_ok(ldq, 2) || !pitch_ok(ldo, 2)))) return FL_ERR_ALIGNMENT;
  if (workspace == nullptr || workspace_bytes < fl_attention_decode_workspace_bytes()) return FL_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & (kWsStatusBytes - 1)) != 0) return FL_ERR_ALIGNMENT;
  const long long items = static_cast<long long>(batch) * n_heads;
  if ((items + 3) / 4 > 0x7FFFFFFFll) return FL_ERR_UNSUPPORTED;
  DeviceInfo di;
  st = current_device(&di);
  if (st != FL_OK) return st;
  DecodeParams p;
  p.c = CacheView{k_pages, v_pages, k_page_scale, v_page_scale, page_table, seq_lens, page_pitch, scale_pitch, ldt,
                  n_kv_heads, page_size, num_pages, max_pages, batch};
  p.Q = static_cast<const __nv_bfloat16*>(Q);
  p.O = static_cast<__nv_bfloat16*>(O);
  p.ldq = ldq;
  p.ldo = ldo;
  p.n_heads = n_heads;
  p.group = n_heads / n_kv_heads;
  p.scale = scale;
  p.status = static_cast<int*>(workspace);
  const int grid = static_cast<int>((items + 3) / 4);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (fp8) attention_decode_kernel<true><<<grid, 128, 0, s>>>(p);
  else attention_decode_kernel<false><<<grid, 128, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? FL_OK : FL_ERR_CUDA;
}
