// Shared by the attention entry points (paged_kv_append, paged_kv_read, attention_decode, attention_prefill and
// their forms): argument checks, the cache's layout, and small device helpers.
#pragma once
#include <cmath>

#include "host_common.h"

namespace fl {

constexpr int kHeadDim = 128;  // the width the QKV projections of this library write
constexpr int kMaxHeads = 1 << 16;
constexpr int kInt4Group = 32;  // values of the 4-bit cache that share a scale
constexpr int kInt4Groups = kHeadDim / kInt4Group;

// The bf16 or E4M3 cache: k_pages and v_pages are [num_pages] blocks `page_pitch` elements apart, each
// [n_kv_heads][page_size][128]; the scales are [num_pages] blocks `scale_pitch` floats apart, each
// [n_kv_heads][page_size].  The 4-bit cache: the same with 64 bytes of codes for a head and token and four bf16 scales.
// page_table[b * ldt + i] is the page that holds positions [i * page_size, (i + 1) * page_size) of sequence b.
struct CacheView {
  const void* k;
  const void* v;
  const void* ks;
  const void* vs;
  const int* table;
  const int* lens;
  long long page_pitch, scale_pitch, ldt;
  int n_kv, page_size, num_pages, max_pages, batch;
};

// What a cache of one type holds for one head of a token.
struct CacheCell {
  int elems, bytes;         // codes, and their bytes
  int scales, scale_bytes;  // scales, and the bytes of one
};
inline bool cache_cell(int cache_dtype, CacheCell* out) {
  switch (cache_dtype) {
    case FL_BF16: *out = {kHeadDim, 2 * kHeadDim, 0, 0}; return true;
    case FL_E4M3: *out = {kHeadDim, kHeadDim, 1, 4}; return true;
    case FL_INT4: *out = {kHeadDim / 2, kHeadDim / 2, kInt4Groups, 2}; return true;
    default: return false;
  }
}

inline int check_cache(const void* k_pages, const void* v_pages, const void* ks, const void* vs,
                       const void* page_table, const void* seq_lens, int batch, int n_kv_heads, int page_size,
                       int num_pages, int max_pages, int64_t ldt, int64_t page_pitch, int64_t scale_pitch,
                       const CacheCell& cell) {
  if (num_pages > 0 && (k_pages == nullptr || v_pages == nullptr)) return FL_ERR_INVALID_ARG;
  if (page_table == nullptr && max_pages > 0) return FL_ERR_INVALID_ARG;
  if (seq_lens == nullptr) return FL_ERR_INVALID_ARG;
  if (batch > 1 && ldt < max_pages) return FL_ERR_INVALID_ARG;
  const int64_t tokens = static_cast<int64_t>(n_kv_heads) * page_size;
  if (num_pages > 1 && page_pitch < tokens * cell.elems) return FL_ERR_INVALID_ARG;
  if (cell.scales > 0) {
    if (num_pages > 0 && (ks == nullptr || vs == nullptr)) return FL_ERR_INVALID_ARG;
    if (num_pages > 1 && scale_pitch < tokens * cell.scales) return FL_ERR_INVALID_ARG;
  }
  if (!aligned16(k_pages) || !aligned16(v_pages)) return FL_ERR_ALIGNMENT;
  if (num_pages > 1 && !pitch_ok(page_pitch, cell.bytes / cell.elems)) return FL_ERR_ALIGNMENT;
  // the scales of a head and token are read at once
  const int at_once = cell.scales > 0 ? cell.scales * cell.scale_bytes : 4;
  if (((reinterpret_cast<uintptr_t>(ks) | reinterpret_cast<uintptr_t>(vs)) & (at_once - 1)) != 0) return FL_ERR_ALIGNMENT;
  if (num_pages > 1 && cell.scales > 0 && scale_pitch % cell.scales != 0) return FL_ERR_ALIGNMENT;
  if (((reinterpret_cast<uintptr_t>(page_table) | reinterpret_cast<uintptr_t>(seq_lens)) & 3u) != 0)
    return FL_ERR_ALIGNMENT;
  return FL_OK;
}

// Division by the page size as a product: pos / page_size = pos * mul >> shift for pos below 2^31.  With 2^bits the first power
// of two that page_size does not pass, mul = ceil(2^(31 + bits) / page_size) fits 32 bits and is less than 2^bits / page_size
// <= 1 part in 2^31 too large.
struct PageDivisor {
  uint32_t mul;
  int shift;
  __device__ __forceinline__ int operator()(int pos) const {
    return static_cast<int>(static_cast<uint64_t>(static_cast<uint32_t>(pos)) * mul >> shift);
  }
};
inline PageDivisor page_divisor(int page_size) {
  const int bits = page_size == 1 ? 0 : 32 - __builtin_clz(static_cast<unsigned>(page_size) - 1);
  return {static_cast<uint32_t>(((uint64_t{1} << (31 + bits)) + page_size - 1) / page_size), 31 + bits};
}

// The factor of the logits to base 2: positive and finite, or the scale is refused.
inline bool scale_to_base_2(float scale, float* out) {
  *out = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634);
  return *out > 0.f && std::isfinite(*out);
}

// The kernels are launched as dependents: they may begin while the kernel in front still writes what they read behind
// griddep_wait.  So they read it by ordinary loads: the read-only path (ld.global.nc) asks for data that nobody writes
// as long as the kernel lives.  Measured no difference in any case.

// Programmatic dependent launch: only the launch itself overlaps the kernel in front (griddep_wait).
template <class Kernel, class... Args>
bool launch_dependent(Kernel* kernel, dim3 grid, int threads, int smem, cudaStream_t s, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess;
}

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

// The same by all lanes of a warp, 32 probes at a time: two loads one behind the other for up to 1000 sequences.
__device__ __forceinline__ int sequence_of_row(const int* cu, int batch, int r, int lane) {
  int lo = 0;
  for (int n = batch + 1; n > 1;) {  // the last of cu[lo .. lo + n - 1] that is not above r
    const int step = (n - 1) / 32 + 1;
    const unsigned below = __ballot_sync(~0u, lane * step < n && cu[lo + lane * step] <= r);
    if (below == 0) return -1;
    const int past = (31 - __clz(below)) * step;
    lo += past;
    n = min(step, n - past);
  }
  return lo < batch ? lo : -1;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two fp32 lanes in one 64-bit register.
__device__ __forceinline__ uint64_t f2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_split(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

}  // namespace fl
