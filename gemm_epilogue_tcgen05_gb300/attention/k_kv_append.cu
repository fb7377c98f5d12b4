// paged_kv_append: rows of keys and values into the pages of a cache.
//
// Row r of sequence b goes to position seq_lens[b] - n_b + (r - first row of b), with n_b the rows that b
// brings: to slot position % page_size of page page_table[b][position / page_size].  bf16 rows into a bf16
// cache and E4M3 rows (with their scales) into an E4M3 cache are moved as they are; bf16 rows into an E4M3
// cache are quantised with one scale per (token, kv head), the rule of fused_qkv_rope_fp8kv:
// s = max|y| / 448, code = e4m3(y / s), a head of zeros gets s = 0 and zero codes.
//
// Bound by memory: each row is read once and written once.  One warp moves one (row, kv head), K and V:
// a warp's lanes cover a head's 128 values (4 values a lane), so its maximum is five shuffles.
#include "attention_common.h"

namespace fl {
namespace {

struct AppendParams {
  const void* K;
  const void* V;
  const float* ks;
  const float* vs;
  void* kp;
  void* vp;
  float* kps;
  float* vps;
  const int* table;
  const int* lens;
  const int* cu;
  long long ldkv, lds, ldt, page_pitch, scale_pitch;
  int T, batch, n_kv, page_size, num_pages, max_pages;
};

enum AppendMode : int { APPEND_BF16 = 0, APPEND_FP8 = 1, APPEND_QUANT = 2 };

// The sequence that row r belongs to: the last b with cu[b] <= r (sequences without rows are skipped);
// -1 for rows before the first and behind the last sequence.
__device__ __forceinline__ int sequence_of_row(const int* cu, int batch, int r) {
  int lo = 0, hi = batch;  // cu[lo] <= r < cu[hi] once both ends are checked
  if (r < cu[0] || r >= cu[batch]) return -1;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (cu[mid] <= r) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ uint32_t quantise4(const uint2 raw, float& scale) {
  float y0 = bf16_lo(raw.x), y1 = bf16_hi(raw.x), y2 = bf16_lo(raw.y), y3 = bf16_hi(raw.y);
  float a = fmaxf(fmaxf(fabsf(y0), fabsf(y1)), fmaxf(fabsf(y2), fabsf(y3)));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) a = fmaxf(a, __shfl_xor_sync(~0u, a, o));
  scale = a * (1.f / 448.f);
  float qs = a > 0.f ? 448.f / a : 0.f;  // the projection's arithmetic, so that both give the same codes
  if (a < 0x1p-100f) {                   // where 448 / a leaves fp32: both factors stay in range
    y0 *= 0x1p64f, y1 *= 0x1p64f, y2 *= 0x1p64f, y3 *= 0x1p64f;
    qs = a > 0.f ? 448.f / (a * 0x1p64f) : 0.f;
  }
  return f32x2_to_e4m3x2(y0 * qs, y1 * qs) | (f32x2_to_e4m3x2(y2 * qs, y3 * qs) << 16);
}

template <int MODE>
__global__ void __launch_bounds__(256) kv_append_kernel(const AppendParams p) {
  const int lane = threadIdx.x & 31;
  const long long item = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (item >= static_cast<long long>(p.T) * p.n_kv) return;
  const int r = static_cast<int>(item / p.n_kv), h = static_cast<int>(item % p.n_kv);
  int b, pos;
  if (p.cu == nullptr) {
    b = r;
    pos = p.lens[b] - 1;
  } else {
    b = sequence_of_row(p.cu, p.batch, r);
    if (b < 0) return;
    pos = p.lens[b] - p.cu[b + 1] + r;
  }
  if (pos < 0) return;
  const int pi = pos / p.page_size, slot = pos - pi * p.page_size;
  if (pi >= p.max_pages) return;
  const int page = p.table[b * p.ldt + pi];
  if (page < 0 || page >= p.num_pages) return;
  const long long cell = static_cast<long long>(h) * p.page_size + slot;
  const long long dst = page * p.page_pitch + cell * kHeadDim + lane * 4;
  const long long src = r * p.ldkv + h * kHeadDim + lane * 4;
  if (MODE == APPEND_FP8) {
    const uint32_t k = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p.K) + src);
    const uint32_t v = *reinterpret_cast<const uint32_t*>(static_cast<const uint8_t*>(p.V) + src);
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.kp) + dst) = k;
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.vp) + dst) = v;
    if (lane < 2) {
      const float s = (lane == 0 ? p.ks : p.vs)[r * p.lds + h];
      (lane == 0 ? p.kps : p.vps)[page * p.scale_pitch + cell] = s;
    }
    return;
  }
  const uint2 k = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.K) + src);
  const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(p.V) + src);
  if (MODE == APPEND_BF16) {
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.kp) + dst) = k;
    *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.vp) + dst) = v;
  } else {
    float sk, sv;
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.kp) + dst) = quantise4(k, sk);
    *reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.vp) + dst) = quantise4(v, sv);
    if (lane < 2) (lane == 0 ? p.kps : p.vps)[page * p.scale_pitch + cell] = lane == 0 ? sk : sv;
  }
}

}  // namespace
}  // namespace fl

extern "C" int paged_kv_append(const void* K, const void* V, const float* k_scale, const float* v_scale,
                               void* k_pages, void* v_pages, float* k_page_scale, float* v_page_scale,
                               const int32_t* page_table, const int32_t* seq_lens, const int32_t* cu_seqlens, int T,
                               int batch, int n_kv_heads, int head_dim, int page_size, int num_pages, int max_pages,
                               int64_t ldkv, int64_t lds, int64_t ldt, int64_t page_pitch, int64_t scale_pitch,
                               int row_dtype, int cache_dtype, void* stream) {
  using namespace fl;
  if (T < 0 || batch < 0 || n_kv_heads < 0 || page_size < 1 || num_pages < 0 || max_pages < 0)
    return FL_ERR_INVALID_ARG;
  const bool rows8 = row_dtype == FL_E4M3, cache8 = cache_dtype == FL_E4M3;
  if ((row_dtype != FL_BF16 && !rows8) || (cache_dtype != FL_BF16 && !cache8)) return FL_ERR_INVALID_ARG;
  if (T == 0 || batch == 0 || n_kv_heads == 0) return FL_OK;
  if (head_dim != kHeadDim || (rows8 && !cache8)) return FL_ERR_UNSUPPORTED;
  if (cu_seqlens == nullptr && T > batch) return FL_ERR_INVALID_ARG;
  if (K == nullptr || V == nullptr || (rows8 && (k_scale == nullptr || v_scale == nullptr))) return FL_ERR_INVALID_ARG;
  if (T > 1 && (ldkv < static_cast<int64_t>(n_kv_heads) * kHeadDim || (rows8 && lds < n_kv_heads)))
    return FL_ERR_INVALID_ARG;
  int st = check_cache(k_pages, v_pages, k_page_scale, v_page_scale, page_table, seq_lens, batch, n_kv_heads,
                       page_size, num_pages, max_pages, ldt, page_pitch, scale_pitch, cache8);
  if (st != FL_OK) return st;
  if (!aligned16(K) || !aligned16(V) || (T > 1 && !pitch_ok(ldkv, rows8 ? 1 : 2))) return FL_ERR_ALIGNMENT;
  if (((reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale) |
        reinterpret_cast<uintptr_t>(cu_seqlens)) & 3u) != 0)
    return FL_ERR_ALIGNMENT;
  const long long items = static_cast<long long>(T) * n_kv_heads;
  if ((items + 7) / 8 > 0x7FFFFFFFll) return FL_ERR_UNSUPPORTED;
  DeviceInfo di;
  st = current_device(&di);
  if (st != FL_OK) return st;
  const AppendParams p{K, V, k_scale, v_scale, k_pages, v_pages, k_page_scale, v_page_scale, page_table, seq_lens,
                       cu_seqlens, ldkv, lds, ldt, page_pitch, scale_pitch, T, batch, n_kv_heads, page_size,
                       num_pages, max_pages};
  const int grid = static_cast<int>((items + 7) / 8);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (!cache8) kv_append_kernel<APPEND_BF16><<<grid, 256, 0, s>>>(p);
  else if (rows8) kv_append_kernel<APPEND_FP8><<<grid, 256, 0, s>>>(p);
  else kv_append_kernel<APPEND_QUANT><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError() == cudaSuccess ? FL_OK : FL_ERR_CUDA;
}
