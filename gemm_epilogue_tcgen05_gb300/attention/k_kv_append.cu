// paged_kv_append: rows of keys and values into the pages of a cache.
//
// Row r of sequence b goes to position seq_lens[b] - n_b + (r - first row of b), with n_b the rows that b
// brings: to slot position % page_size of page page_table[b][position / page_size].  bf16 rows into a bf16
// cache and E4M3 rows (with their scales) into an E4M3 cache are moved as they are; bf16 rows into an E4M3
// cache are quantised with one scale per (token, kv head), the rule of fused_qkv_rope_fp8kv:
// s = max|y| / 448, code = e4m3(y / s), a head of zeros gets s = 0 and zero codes.
//
// Bound by memory: each row is read once and written once.  One warp moves one row, all its heads: finding the row's
// place takes a search over the offsets and three dependent loads, some 2 us, which a warp for each (row, head) paid
// for each head (26.0 us for 12500 rows of 8 heads, bf16 to E4M3).  The row is on its way meanwhile.  A lane takes 16
// bytes, 16 lanes a bf16 head (8 an E4M3 one), and four of a warp's loads for K and four for V are in flight.  With a
// reduction and a division for each head the same rows took 14.9 us, with one of each for eight heads 13.4.
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

__device__ __forceinline__ uint32_t bf16x2_max(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Largest magnitudes (NaN aside) of 8 bf16 values of K and of V: one bf16 each, K's in the low half.
__device__ __forceinline__ uint32_t magnitudes(const uint4 k, const uint4 v) {
  constexpr uint32_t kAbs = 0x7FFF7FFFu;
  const uint32_t a = bf16x2_max(bf16x2_max(k.x & kAbs, k.y & kAbs), bf16x2_max(k.z & kAbs, k.w & kAbs));
  const uint32_t b = bf16x2_max(bf16x2_max(v.x & kAbs, v.y & kAbs), bf16x2_max(v.z & kAbs, v.w & kAbs));
  return bf16x2_max(bf16x2_max(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632)), 0u);
}
// 8 bf16 values times lift times factor to E4M3 codes.
template <bool LIFT>
__device__ __forceinline__ uint2 codes8(const uint4 raw, float factor, float lift) {
  float y[8] = {bf16_lo(raw.x), bf16_hi(raw.x), bf16_lo(raw.y), bf16_hi(raw.y),
                bf16_lo(raw.z), bf16_hi(raw.z), bf16_lo(raw.w), bf16_hi(raw.w)};
  if (LIFT) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] *= lift;
  }
  uint2 c;
  c.x = f32x2_to_e4m3x2(y[0] * factor, y[1] * factor) | (f32x2_to_e4m3x2(y[2] * factor, y[3] * factor) << 16);
  c.y = f32x2_to_e4m3x2(y[4] * factor, y[5] * factor) | (f32x2_to_e4m3x2(y[6] * factor, y[7] * factor) << 16);
  return c;
}

constexpr int kAppendWarps = 4;

template <int MODE>
__global__ void __launch_bounds__(32 * kAppendWarps) kv_append_kernel(const AppendParams p) {
  griddep_wait();  // launched as a dependent: nothing is read before the kernel in front has finished
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5);
  if (row >= p.T) return;
  const int r = static_cast<int>(row);
  constexpr int kInBytes = MODE == APPEND_FP8 ? 1 : 2, kOutBytes = MODE == APPEND_BF16 ? 2 : 1;
  constexpr int kLanes = kHeadDim * kInBytes / 16, kHeads = 32 / kLanes;  // lanes of a head, heads of a warp's load
  constexpr int kEach = 16 / kInBytes;                                   // values of a lane
  const int part = lane % kLanes, h0 = lane / kLanes;
  const uint8_t* k_src = static_cast<const uint8_t*>(p.K) + (r * p.ldkv + part * kEach) * kInBytes;
  const uint8_t* v_src = static_cast<const uint8_t*>(p.V) + (r * p.ldkv + part * kEach) * kInBytes;
  constexpr int kTogether = 4;
  uint4 k[kTogether], v[kTogether];
  auto fetch = [&](int first) {
#pragma unroll
    for (int i = 0; i < kTogether; ++i) {
      const int h = first + i * kHeads + h0;
      k[i] = v[i] = make_uint4(0, 0, 0, 0);
      if (h < p.n_kv) {
        k[i] = *reinterpret_cast<const uint4*>(k_src + h * (kHeadDim * kInBytes));
        v[i] = *reinterpret_cast<const uint4*>(v_src + h * (kHeadDim * kInBytes));
      }
    }
  };
  fetch(0);  // on their way while the row's place is looked up
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
  const long long dst = (page * p.page_pitch + static_cast<long long>(slot) * kHeadDim + part * kEach) * kOutBytes;
  uint8_t* k_dst = static_cast<uint8_t*>(p.kp) + dst;
  uint8_t* v_dst = static_cast<uint8_t*>(p.vp) + dst;
  const long long head_step = static_cast<long long>(p.page_size) * kHeadDim * kOutBytes;
  const long long scale_dst = page * p.scale_pitch + slot;
  for (int first = 0; first < p.n_kv; first += kTogether * kHeads) {
    if (first > 0) fetch(first);
    if constexpr (MODE == APPEND_QUANT) {
      // The maxima of four heads of K and of V over 16 lanes each, by halves: every lane ends with one of the eight
      // (head 2 * bit 3 + bit 2 of the lane; bit 0: V), does that one's division and hands the factor round.
      uint32_t top[kTogether];
#pragma unroll
      for (int i = 0; i < kTogether; ++i) top[i] = magnitudes(k[i], v[i]);
      const bool b3 = (lane & 8) != 0, b2 = (lane & 4) != 0;
      const uint32_t t0 = bf16x2_max(b3 ? top[2] : top[0], __shfl_xor_sync(~0u, b3 ? top[0] : top[2], 8));
      const uint32_t t1 = bf16x2_max(b3 ? top[3] : top[1], __shfl_xor_sync(~0u, b3 ? top[1] : top[3], 8));
      uint32_t t = bf16x2_max(b2 ? t1 : t0, __shfl_xor_sync(~0u, b2 ? t0 : t1, 4));
      t = bf16x2_max(t, __shfl_xor_sync(~0u, t, 2));
      t = bf16x2_max(t, __shfl_xor_sync(~0u, t, 1));
      const float a = (lane & 1) != 0 ? bf16_hi(t) : bf16_lo(t);
      // the projection's arithmetic, so that both give the same codes; where 448 / a leaves fp32 both factors are lifted
      const bool tiny = a > 0.f && a < 0x1p-100f;
      const float lift = tiny ? 0x1p64f : 1.f, factor = a > 0.f ? 448.f / (a * lift) : 0.f;
      const int h_mine = first + ((b3 ? 2 : 0) + (b2 ? 1 : 0)) * kHeads + h0;
      if ((lane & 2) == 0 && h_mine < p.n_kv)
        ((lane & 1) != 0 ? p.vps : p.kps)[scale_dst + static_cast<long long>(h_mine) * p.page_size] = a * (1.f / 448.f);
      const bool any_tiny = __any_sync(~0u, tiny);
#pragma unroll
      for (int i = 0; i < kTogether; ++i) {
        const int h = first + i * kHeads + h0, from = (lane & 16) | (i << 2);
        const float fk = __shfl_sync(~0u, factor, from), fv = __shfl_sync(~0u, factor, from | 1);
        uint2 ck, cv;
        if (any_tiny) {
          ck = codes8<true>(k[i], fk, __shfl_sync(~0u, lift, from));
          cv = codes8<true>(v[i], fv, __shfl_sync(~0u, lift, from | 1));
        } else {
          ck = codes8<false>(k[i], fk, 1.f);
          cv = codes8<false>(v[i], fv, 1.f);
        }
        if (h >= p.n_kv) continue;
        *reinterpret_cast<uint2*>(k_dst + h * head_step) = ck;
        *reinterpret_cast<uint2*>(v_dst + h * head_step) = cv;
      }
    } else {
#pragma unroll
      for (int i = 0; i < kTogether; ++i) {
        const int h = first + i * kHeads + h0;
        if (h >= p.n_kv) continue;
        *reinterpret_cast<uint4*>(k_dst + h * head_step) = k[i];
        *reinterpret_cast<uint4*>(v_dst + h * head_step) = v[i];
        if (MODE == APPEND_FP8 && part < 2)
          (part == 0 ? p.kps : p.vps)[scale_dst + static_cast<long long>(h) * p.page_size] =
              (part == 0 ? p.ks : p.vs)[r * p.lds + h];
      }
    }
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
  if (n_kv_heads > kMaxHeads) return FL_ERR_UNSUPPORTED;
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
  DeviceInfo di;
  st = current_device(&di);
  if (st != FL_OK) return st;
  const AppendParams p{K, V, k_scale, v_scale, k_pages, v_pages, k_page_scale, v_page_scale, page_table, seq_lens,
                       cu_seqlens, ldkv, lds, ldt, page_pitch, scale_pitch, T, batch, n_kv_heads, page_size,
                       num_pages, max_pages};
  // programmatic dependent launch: only the launch itself overlaps the kernel in front (griddep_wait)
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((T - 1) / kAppendWarps + 1);
  cfg.blockDim = dim3(32 * kAppendWarps);
  cfg.stream = static_cast<cudaStream_t>(stream);
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  const cudaError_t e = !cache8 ? cudaLaunchKernelEx(&cfg, kv_append_kernel<APPEND_BF16>, p)
                        : rows8 ? cudaLaunchKernelEx(&cfg, kv_append_kernel<APPEND_FP8>, p)
                                : cudaLaunchKernelEx(&cfg, kv_append_kernel<APPEND_QUANT>, p);
  return e == cudaSuccess ? FL_OK : FL_ERR_CUDA;
}
