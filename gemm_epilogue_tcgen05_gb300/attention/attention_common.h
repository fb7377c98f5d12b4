// Shared by the attention entry points (paged_kv_append, attention_decode, attention_prefill): argument
// checks, the cache's layout, and small device helpers.
#pragma once
#include <cmath>

#include "host_common.h"

namespace fl {

constexpr int kHeadDim = 128;  // the width the QKV projections of this library write
constexpr int kMaxHeads = 1 << 16;

// The E4M3 or bf16 cache: k_pages and v_pages are [num_pages] blocks `page_pitch` elements apart, each
// [n_kv_heads][page_size][128]; the scales are [num_pages] blocks `scale_pitch` floats apart, each
// [n_kv_heads][page_size].  page_table[b * ldt + i] is the page that holds positions
// [i * page_size, (i + 1) * page_size) of sequence b.
struct CacheView {
  const void* k;
  const void* v;
  const float* ks;
  const float* vs;
  const int* table;
  const int* lens;
  long long page_pitch, scale_pitch, ldt;
  int n_kv, page_size, num_pages, max_pages, batch;
};

inline int check_cache(const void* k_pages, const void* v_pages, const void* ks, const void* vs,
                       const void* page_table, const void* seq_lens, int batch, int n_kv_heads, int page_size,
                       int num_pages, int max_pages, int64_t ldt, int64_t page_pitch, int64_t scale_pitch, bool fp8) {
  if (num_pages > 0 && (k_pages == nullptr || v_pages == nullptr)) return FL_ERR_INVALID_ARG;
  if (page_table == nullptr && max_pages > 0) return FL_ERR_INVALID_ARG;
  if (seq_lens == nullptr) return FL_ERR_INVALID_ARG;
  if (batch > 1 && ldt < max_pages) return FL_ERR_INVALID_ARG;
  const int64_t tokens = static_cast<int64_t>(n_kv_heads) * page_size;
  if (num_pages > 1 && page_pitch < tokens * kHeadDim) return FL_ERR_INVALID_ARG;
  if (fp8) {
    if (num_pages > 0 && (ks == nullptr || vs == nullptr)) return FL_ERR_INVALID_ARG;
    if (num_pages > 1 && scale_pitch < tokens) return FL_ERR_INVALID_ARG;
  }
  if (!aligned16(k_pages) || !aligned16(v_pages)) return FL_ERR_ALIGNMENT;
  if (num_pages > 1 && !pitch_ok(page_pitch, fp8 ? 1 : 2)) return FL_ERR_ALIGNMENT;
  if (((reinterpret_cast<uintptr_t>(ks) | reinterpret_cast<uintptr_t>(vs) | reinterpret_cast<uintptr_t>(page_table) |
        reinterpret_cast<uintptr_t>(seq_lens)) & 3u) != 0)
    return FL_ERR_ALIGNMENT;
  return FL_OK;
}

// The factor of the logits to base 2: positive and finite, or the scale is refused.
inline bool scale_to_base_2(float scale, float* out) {
  *out = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  return *out > 0.f && std::isfinite(*out);
}

// The kernels are launched as dependents: they may begin while the kernel in front still writes what they read behind
// griddep_wait.  So they read it by ordinary loads: the read-only path (ld.global.nc) asks for data that nobody writes
// as long as the kernel lives.  Measured no difference in any case.

// First and one-past-last row of sequence b: cu_seqlens clipped to [0, M] (a decreasing or out-of-range
// entry gives an empty sequence, never a row outside the tensors), or runs of seq_len rows.
__device__ __forceinline__ void sequence_rows(const int* cu, int b, int seq_len, int M, int& first, int& last) {
  if (cu != nullptr) {
    first = min(max(cu[b], 0), M);
    last = min(max(cu[b + 1], first), M);
  } else {
    first = static_cast<int>(min(static_cast<long long>(b) * seq_len, static_cast<long long>(M)));
    last = static_cast<int>(min(static_cast<long long>(first) + seq_len, static_cast<long long>(M)));
  }
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float e4m3_to_f32(uint32_t code) {
  uint32_t h;
  asm("{\n\t.reg .b32 t;\n\tcvt.rn.f16x2.e4m3x2 t, %1;\n\tmov.b32 %0, t;\n\t}" : "=r"(h) : "h"(static_cast<uint16_t>(code)));
  return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xFFFFu)));
}

}  // namespace fl
