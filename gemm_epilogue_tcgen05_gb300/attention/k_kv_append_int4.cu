// paged_kv_append_int4: bf16 rows of keys and values into the pages of a 4-bit cache.
//
// For 32 consecutive values y of a head, a = max|y|:
//   s = a / 7 rounded to five significant bits (nearest even), code = y / s rounded to the nearest even whole number.
// |y / s| <= 7 * (1 + 2^-5), so codes lie in [-7, 7] and fit 4 bits (two's complement, the even column in the low half
// of a byte), and a code times s has eight significant bits at most: what the cache stands for are bf16 numbers.  A
// group whose largest magnitude is below 2^-120 becomes zeros (no denormal number has to be dealt with, here or where
// the cache is read), a group with a value that is not finite gets a NaN for s and zero codes.
//
// Both roundings are exact although no division is made.  a / 7 is half way between two five-bit numbers only for significands
// 231 and 245 (33 and 35 times 7; of the other multiples of 7 the quotients are five-bit numbers themselves), whose product
// with fl(1/7) is the quotient exactly; else it is 1/14 of a step or more from there, and the product is off by 2^-18 of one at
// most (fl(1/7) is off by 2^-24.4 of itself, its rounding 2^-24).  y / s has a denominator of at most 2 * 31 * 16 beside a power of
// two, so it is k + 1/2 exactly or 2^-10 off: y times an approximate 1/s, plus 768, in one rounding is its nearest multiple of 2^-14,
// and the next addition rounds that to a whole number.
//
// Bound by memory: 512 bytes in and 144 out for each head of a token.  One warp moves a row, all its heads, as in
// paged_kv_append; a lane takes 8 values, four lanes a group.  10075 rows of 8 heads: 13.1 us, 4.0 TB/s: a chain of loads (offsets,
// length, table entry) behind a row's own, and the ramp of a short kernel.  (Several rows a warp: 16.5 us and more.)
#include "attention_common.h"

namespace fl {
namespace {

struct AppendInt4Params {
  const __nv_bfloat16* K;
  const __nv_bfloat16* V;
  uint8_t* kp;
  uint8_t* vp;
  __nv_bfloat16* kps;
  __nv_bfloat16* vps;
  const int* table;
  const int* lens;
  const int* cu;
  long long ldkv, ldt, page_pitch, scale_pitch;
  int T, batch, n_kv, page_size, num_pages, max_pages;
  PageDivisor page_of;
};

__device__ __forceinline__ uint32_t bf16x2_max_nan(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Largest magnitudes of 8 bf16 values of K and of V: one bf16 each, K's in the low half; NaN where there is one.
__device__ __forceinline__ uint32_t magnitudes_nan(const uint4 k, const uint4 v) {
  constexpr uint32_t kAbs = 0x7FFF7FFFu;
  const uint32_t a = bf16x2_max_nan(bf16x2_max_nan(k.x & kAbs, k.y & kAbs), bf16x2_max_nan(k.z & kAbs, k.w & kAbs));
  const uint32_t b = bf16x2_max_nan(bf16x2_max_nan(v.x & kAbs, v.y & kAbs), bf16x2_max_nan(v.z & kAbs, v.w & kAbs));
  return bf16x2_max_nan(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
}
// s of a group from the bf16 bits of its largest magnitude, as an fp32 number: 0 for a group of zeros, NaN for one with
// a value that is not finite.
__device__ __forceinline__ float int4_scale(uint32_t largest) {
  const uint32_t b = __float_as_uint(__uint_as_float(largest << 16) * (1.f / 7.f));
  const uint32_t s = largest < (127u - 120u) << 7 ? 0u : (b + 0x3FFFFu + ((b >> 19) & 1u)) & 0xFFF80000u;
  return __uint_as_float(largest >= 0x7F80u ? 0x7FFF0000u : s);
}
// 1/s to 2^-22 of itself, 0 for 0 and NaN: the fastest will do, for y * inverse(s) is off by 2^-19 at most.
__device__ __forceinline__ float inverse(float s) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(s));
  return s > 0.f ? r : 0.f;
}
// 8 values over s as codes, value i in bits 4 i; zeros for a group of zeros, and where s is NaN.
__device__ __forceinline__ uint32_t int4_codes(const uint4 raw, float s) {
  const float r = inverse(s);
  const float y[8] = {bf16_lo(raw.x), bf16_hi(raw.x), bf16_lo(raw.y), bf16_hi(raw.y),
                      bf16_lo(raw.z), bf16_hi(raw.z), bf16_lo(raw.w), bf16_hi(raw.w)};
  // 3 * 2^22 + 8 + code: the last bits of the sum are code + 8, whose weighted sum has no carries
  constexpr uint32_t kBase = 0x4B400000u;
  const uint64_t r2 = f2(r, r), part = f2(768.f, 768.f), whole = f2(12582912.f - 768.f + 8.f, 12582912.f - 768.f + 8.f);
  uint32_t word = 0;
#pragma unroll
  for (int i = 6; i >= 0; i -= 2) {
    float a, b;
    f2_split(f2_add(f2_fma(f2(y[i], y[i + 1]), r2, part), whole), a, b);
    word = (word * 16 + __float_as_uint(b)) * 16 + __float_as_uint(a);
  }
  return s >= 0.f ? (word - kBase * 0x11111111u) ^ 0x88888888u : 0u;  // zeros where s is NaN
}

constexpr int kAppendWarps = 4;

__global__ void __launch_bounds__(32 * kAppendWarps) kv_append_int4_kernel(const AppendInt4Params p) {
  griddep_wait();  // launched as a dependent: nothing is read before the kernel in front has finished
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * kAppendWarps + (threadIdx.x >> 5);
  if (row >= p.T) return;
  const int r = static_cast<int>(row);
  const int part = lane & 15, h0 = lane >> 4;  // 16 lanes a head, two heads a load
  const uint4* k_src = reinterpret_cast<const uint4*>(p.K + r * p.ldkv) + part;
  const uint4* v_src = reinterpret_cast<const uint4*>(p.V + r * p.ldkv) + part;
  constexpr int kTogether = 4;
  uint4 k[kTogether], v[kTogether];
  auto fetch = [&](int first) {
#pragma unroll
    for (int i = 0; i < kTogether; ++i) {
      const int h = first + i * 2 + h0;
      k[i] = v[i] = make_uint4(0, 0, 0, 0);
      if (h < p.n_kv) k[i] = k_src[h * 16], v[i] = v_src[h * 16];
    }
  };
  fetch(0);  // on their way while the row's place is looked up
  int b, pos;
  if (p.cu == nullptr) {
    b = r;
    pos = p.lens[b] - 1;
  } else {
    b = sequence_of_row(p.cu, p.batch, r, lane);
    if (b < 0) return;
    const long long at = static_cast<long long>(p.lens[b]) - p.cu[b + 1] + r;
    pos = at > INT32_MAX ? -1 : static_cast<int>(max(at, -1ll));
  }
  if (pos < 0) return;
  const int pi = p.page_of(pos);
  const long long slot = pos - pi * p.page_size;  // its bytes may pass 32 bits
  if (pi >= p.max_pages) return;
  const int page = p.table[b * p.ldt + pi];
  if (page < 0 || page >= p.num_pages) return;
  const long long head_step = static_cast<long long>(p.page_size) * (kHeadDim / 2);  // bytes; of the scales an eighth
  const long long at = page * p.page_pitch + slot * (kHeadDim / 2) + part * 4 + h0 * head_step;
  // of each four lanes the first writes the scale of K, the second that of V
  __nv_bfloat16* s_dst = ((lane & 1) != 0 ? p.vps : p.kps) + page * p.scale_pitch + slot * kInt4Groups + (part >> 2) +
                         h0 * (head_step / 16);
  for (int first = 0; first < p.n_kv; first += kTogether * 2) {
    if (first > 0) fetch(first);
#pragma unroll
    for (int i = 0; i < kTogether; ++i) {
      uint32_t top = magnitudes_nan(k[i], v[i]);
      top = bf16x2_max_nan(top, __shfl_xor_sync(~0u, top, 1));
      top = bf16x2_max_nan(top, __shfl_xor_sync(~0u, top, 2));
      const float sk = int4_scale(top & 0xFFFFu), sv = int4_scale(top >> 16);
      if (first + i * 2 + h0 >= p.n_kv) continue;
      const long long ahead = (first + i * 2) * head_step;
      *reinterpret_cast<uint32_t*>(p.kp + at + ahead) = int4_codes(k[i], sk);
      *reinterpret_cast<uint32_t*>(p.vp + at + ahead) = int4_codes(v[i], sv);
      if ((lane & 2) == 0) s_dst[ahead / 16] = __float2bfloat16_rn((lane & 1) != 0 ? sv : sk);
    }
  }
}

}  // namespace
}  // namespace fl

extern "C" int paged_kv_append_int4(const void* K, const void* V, void* k_pages, void* v_pages, void* k_page_scale,
                                    void* v_page_scale, const int32_t* page_table, const int32_t* seq_lens,
                                    const int32_t* cu_seqlens, int T, int batch, int n_kv_heads, int head_dim,
                                    int page_size, int num_pages, int max_pages, int64_t ldkv, int64_t ldt,
                                    int64_t page_pitch, int64_t scale_pitch, void* stream) {
  using namespace fl;
  if (T < 0 || batch < 0 || n_kv_heads < 0 || page_size < 1 || num_pages < 0 || max_pages < 0)
    return FL_ERR_INVALID_ARG;
  if (T == 0 || batch == 0 || n_kv_heads == 0) return FL_OK;
  if (head_dim != kHeadDim || n_kv_heads > kMaxHeads) return FL_ERR_UNSUPPORTED;
  if (cu_seqlens == nullptr && T > batch) return FL_ERR_INVALID_ARG;
  if (K == nullptr || V == nullptr) return FL_ERR_INVALID_ARG;
  if (T > 1 && ldkv < static_cast<int64_t>(n_kv_heads) * kHeadDim) return FL_ERR_INVALID_ARG;
  CacheCell cell;
  cache_cell(FL_INT4, &cell);
  int st = check_cache(k_pages, v_pages, k_page_scale, v_page_scale, page_table, seq_lens, batch, n_kv_heads,
                       page_size, num_pages, max_pages, ldt, page_pitch, scale_pitch, cell);
  if (st != FL_OK) return st;
  if (!aligned16(K) || !aligned16(V) || (T > 1 && !pitch_ok(ldkv, 2))) return FL_ERR_ALIGNMENT;
  if ((reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) != 0) return FL_ERR_ALIGNMENT;
  DeviceInfo di;
  st = current_device(&di);
  if (st != FL_OK) return st;
  const AppendInt4Params p{static_cast<const __nv_bfloat16*>(K), static_cast<const __nv_bfloat16*>(V),
                           static_cast<uint8_t*>(k_pages), static_cast<uint8_t*>(v_pages),
                           static_cast<__nv_bfloat16*>(k_page_scale), static_cast<__nv_bfloat16*>(v_page_scale),
                           page_table, seq_lens, cu_seqlens, ldkv, ldt, page_pitch, scale_pitch, T, batch, n_kv_heads,
                           page_size, num_pages, max_pages, page_divisor(page_size)};
  return launch_dependent(kv_append_int4_kernel, dim3((T - 1) / kAppendWarps + 1), 32 * kAppendWarps, 0,
                          static_cast<cudaStream_t>(stream), p)
             ? FL_OK
             : FL_ERR_CUDA;
}
