// paged_kv_read: tokens of a cache back as bf16 rows of keys and values.
//
// Row r of sequence b is position seq_lens[b] - n_b + (r - first row of b), with n_b the rows that b gets: the
// counterpart of the appends.  bf16 entries are moved as they are, E4M3 codes are multiplied by their scale in fp32 and
// rounded, 4-bit codes times theirs are bf16 numbers (three and five significant bits).
//
// Bound by memory: a row is written once, its entries read once.  One warp does one row, all its heads; a lane writes
// 16 bytes.  32768 tokens of 8 heads in 4 bits: 29.9 us, 5.8 TB/s; 7437 in E4M3: 10.1 us, 4.6 TB/s, the same chain of loads as the
// append's in front of it.
#include "attention_common.h"

namespace fl {
namespace {

struct ReadParams {
  CacheView c;
  const int* cu;
  __nv_bfloat16* K;
  __nv_bfloat16* V;
  long long ldkv;
  int T;
  PageDivisor page_of;
};

enum ReadMode : int { READ_BF16 = 0, READ_E4M3 = 1, READ_INT4 = 2 };

__device__ __forceinline__ uint32_t bf16x2_sub(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t bf16x2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// What a lane loads of an entry, and the 8 bf16 values that it stands for.
template <int MODE>
struct Piece;
template <>
struct Piece<READ_BF16> {
  uint4 x;
  __device__ __forceinline__ void load(const void* codes, const void*, long long cell, int part) {
    x = reinterpret_cast<const uint4*>(codes)[cell * 16 + part];
  }
  __device__ __forceinline__ uint4 values() const { return x; }
};
template <>
struct Piece<READ_E4M3> {
  uint2 x;
  float s;
  __device__ __forceinline__ void load(const void* codes, const void* scales, long long cell, int part) {
    x = reinterpret_cast<const uint2*>(codes)[cell * 16 + part];
    s = reinterpret_cast<const float*>(scales)[cell];
  }
  __device__ __forceinline__ uint4 values() const {
    uint32_t out[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t two;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(two) : "h"(static_cast<uint16_t>((e < 2 ? x.x : x.y) >> ((e & 1) * 16))));
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&two));
      out[e] = pack_bf16x2(f.x * s, f.y * s);
    }
    return make_uint4(out[0], out[1], out[2], out[3]);
  }
};
template <>
struct Piece<READ_INT4> {
  uint32_t x;
  unsigned short s;
  __device__ __forceinline__ void load(const void* codes, const void* scales, long long cell, int part) {
    x = reinterpret_cast<const uint32_t*>(codes)[cell * 16 + part];
    s = reinterpret_cast<const unsigned short*>(scales)[cell * kInt4Groups + (part >> 2)];
  }
  __device__ __forceinline__ uint4 values() const {
    const uint32_t ss = __byte_perm(s, s, 0x5410), u = x ^ 0x88888888u;
    const uint32_t even = u & 0x0F0F0F0Fu, odd = u >> 4 & 0x0F0F0F0Fu;
    const uint32_t low = __byte_perm(even, odd, 0x5140), high = __byte_perm(even, odd, 0x7362);  // columns 0-3 | 4-7, a byte each
    constexpr uint32_t k128 = 0x43434343u;  // with a byte u below it: 128 + u as bf16
    uint32_t out[4] = {__byte_perm(low, k128, 0x4140), __byte_perm(low, k128, 0x4342), __byte_perm(high, k128, 0x4140),
                       __byte_perm(high, k128, 0x4342)};
#pragma unroll
    for (int e = 0; e < 4; ++e) out[e] = bf16x2_mul(bf16x2_sub(out[e], 0x43084308u), ss);  // less 136: exact, and so is the product
    return make_uint4(out[0], out[1], out[2], out[3]);
  }
};

constexpr int kReadWarps = 4;

template <int MODE>
__global__ void __launch_bounds__(32 * kReadWarps) kv_read_kernel(const ReadParams p) {
  griddep_wait();  // launched as a dependent: nothing is read before the kernel in front has finished
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const long long row = static_cast<long long>(blockIdx.x) * kReadWarps + (threadIdx.x >> 5);
  if (row >= p.T) return;
  const int r = static_cast<int>(row);
  int b, pos;
  if (p.cu == nullptr) {
    b = r;
    pos = p.c.lens[b] - 1;
  } else {
    b = sequence_of_row(p.cu, p.c.batch, r, lane);
    if (b < 0) return;
    const long long at = static_cast<long long>(p.c.lens[b]) - p.cu[b + 1] + r;
    pos = at > INT32_MAX ? -1 : static_cast<int>(max(at, -1ll));
  }
  const int pi = pos < 0 ? -1 : p.page_of(pos), slot = pos - pi * p.c.page_size;
  const int entry = pi < 0 || pi >= p.c.max_pages ? -1 : p.c.table[b * p.c.ldt + pi];
  const bool ok = entry >= 0 && entry < p.c.num_pages;
  const long long page = ok ? entry : 0;
  constexpr int kBytes = MODE == READ_BF16 ? 2 : 1, kScale = MODE == READ_E4M3 ? 4 : 2;
  const uint8_t* k_src = static_cast<const uint8_t*>(p.c.k) + page * p.c.page_pitch * kBytes;
  const uint8_t* v_src = static_cast<const uint8_t*>(p.c.v) + page * p.c.page_pitch * kBytes;
  const uint8_t* ks_src = static_cast<const uint8_t*>(p.c.ks) + page * p.c.scale_pitch * kScale;
  const uint8_t* vs_src = static_cast<const uint8_t*>(p.c.vs) + page * p.c.scale_pitch * kScale;
  const int part = lane & 15, h0 = lane >> 4;  // 16 lanes a head, two heads at a time
  uint4* k_dst = reinterpret_cast<uint4*>(p.K + r * p.ldkv) + part;
  uint4* v_dst = reinterpret_cast<uint4*>(p.V + r * p.ldkv) + part;
  constexpr int kTogether = 4;
  for (int first = 0; first < p.c.n_kv; first += kTogether * 2) {
    Piece<MODE> k[kTogether], v[kTogether];
#pragma unroll
    for (int i = 0; i < kTogether; ++i) {
      const int h = first + i * 2 + h0;
      if (!ok || h >= p.c.n_kv) continue;
      const long long cell = static_cast<long long>(h) * p.c.page_size + slot;
      k[i].load(k_src, ks_src, cell, part);
      v[i].load(v_src, vs_src, cell, part);
    }
#pragma unroll
    for (int i = 0; i < kTogether; ++i) {
      const int h = first + i * 2 + h0;
      if (h >= p.c.n_kv) continue;
      const uint4 none = make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
      k_dst[h * 16] = ok ? k[i].values() : none;
      v_dst[h * 16] = ok ? v[i].values() : none;
    }
  }
}

template <int MODE>
bool launch_read(const ReadParams& p, cudaStream_t s) {
  return launch_dependent(kv_read_kernel<MODE>, dim3((p.T - 1) / kReadWarps + 1), 32 * kReadWarps, 0, s, p);
}

}  // namespace
}  // namespace fl

extern "C" int paged_kv_read(const void* k_pages, const void* v_pages, const void* k_page_scale,
                             const void* v_page_scale, const int32_t* page_table, const int32_t* seq_lens,
                             const int32_t* cu_seqlens, void* K, void* V, int T, int batch, int n_kv_heads,
                             int head_dim, int page_size, int num_pages, int max_pages, int64_t ldkv, int64_t ldt,
                             int64_t page_pitch, int64_t scale_pitch, int cache_dtype, void* stream) {
  using namespace fl;
  if (T < 0 || batch < 0 || n_kv_heads < 0 || page_size < 1 || num_pages < 0 || max_pages < 0)
    return FL_ERR_INVALID_ARG;
  CacheCell cell;
  if (!cache_cell(cache_dtype, &cell)) return FL_ERR_INVALID_ARG;
  if (T == 0 || batch == 0 || n_kv_heads == 0) return FL_OK;
  if (head_dim != kHeadDim || n_kv_heads > kMaxHeads) return FL_ERR_UNSUPPORTED;
  if (cu_seqlens == nullptr && T > batch) return FL_ERR_INVALID_ARG;
  if (K == nullptr || V == nullptr) return FL_ERR_INVALID_ARG;
  if (T > 1 && ldkv < static_cast<int64_t>(n_kv_heads) * kHeadDim) return FL_ERR_INVALID_ARG;
  int st = check_cache(k_pages, v_pages, k_page_scale, v_page_scale, page_table, seq_lens, batch, n_kv_heads,
                       page_size, num_pages, max_pages, ldt, page_pitch, scale_pitch, cell);
  if (st != FL_OK) return st;
  if (!aligned16(K) || !aligned16(V) || (T > 1 && !pitch_ok(ldkv, 2))) return FL_ERR_ALIGNMENT;
  if ((reinterpret_cast<uintptr_t>(cu_seqlens) & 3u) != 0) return FL_ERR_ALIGNMENT;
  DeviceInfo di;
  st = current_device(&di);
  if (st != FL_OK) return st;
  const ReadParams p{CacheView{k_pages, v_pages, k_page_scale, v_page_scale, page_table, seq_lens, page_pitch,
                               scale_pitch, ldt, n_kv_heads, page_size, num_pages, max_pages, batch},
                     cu_seqlens, static_cast<__nv_bfloat16*>(K), static_cast<__nv_bfloat16*>(V), ldkv, T,
                     page_divisor(page_size)};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool done = cache_dtype == FL_BF16   ? launch_read<READ_BF16>(p, s)
                    : cache_dtype == FL_E4M3 ? launch_read<READ_E4M3>(p, s)
                                             : launch_read<READ_INT4>(p, s);
  return done ? FL_OK : FL_ERR_CUDA;
}
