// attention_decode and attention_decode_window: argument checks and dispatch (the kernels and their design:
// decode_attention_kernel.cuh, decode_int4_kernel.cuh).
#include <algorithm>
#include <cstdint>

#include "decode_attention_host.cuh"
#include "decode_attention_kernel.cuh"

namespace fl {
namespace {

constexpr size_t kDecWorkspace = kWsStatusBytes + kDecMaxCtas * sizeof(unsigned) +
                                 static_cast<size_t>(kDecMaxCtas) * 2 * kDecPartFloats * sizeof(float);

int enqueue_decode(const void* Q, const void* k_pages, const void* v_pages, const void* k_page_scale,
                   const void* v_page_scale, const int32_t* page_table, const int32_t* seq_lens, void* O, int batch,
                   int n_heads, int n_kv_heads, int head_dim, int page_size, int num_pages, int max_pages, int64_t ldq,
                   int64_t ldo, int64_t ldt, int64_t page_pitch, int64_t scale_pitch, float scale, int window, int sinks,
                   int cache_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (batch < 0 || n_heads < 0 || n_kv_heads < 0 || page_size < 1 || num_pages < 0 || max_pages < 0)
    return FL_ERR_INVALID_ARG;
  CacheCell cell;
  float scale_log2;
  if (!cache_cell(cache_dtype, &cell) || !scale_to_base_2(scale, &scale_log2)) return FL_ERR_INVALID_ARG;
  if (batch == 0 || n_heads == 0) return FL_OK;
  if (n_kv_heads == 0 || n_heads % n_kv_heads != 0) return FL_ERR_INVALID_ARG;
  if (head_dim != kHeadDim) return FL_ERR_UNSUPPORTED;
  if (n_heads > kMaxHeads) return FL_ERR_UNSUPPORTED;
  if (Q == nullptr || O == nullptr) return FL_ERR_INVALID_ARG;
  const int64_t width = static_cast<int64_t>(n_heads) * kHeadDim;
  if (batch > 1 && (ldq < width || ldo < width)) return FL_ERR_INVALID_ARG;
  int st = check_cache(k_pages, v_pages, k_page_scale, v_page_scale, page_table, seq_lens, batch, n_kv_heads,
                       page_size, num_pages, max_pages, ldt, page_pitch, scale_pitch, cell);
  if (st != FL_OK) return st;
  if (!aligned16(Q) || !aligned16(O) || (batch > 1 && (!pitch_ok(ldq, 2) || !pitch_ok(ldo, 2)))) return FL_ERR_ALIGNMENT;
  if (workspace == nullptr || workspace_bytes < kDecWorkspace) return FL_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & (kWsStatusBytes - 1)) != 0) return FL_ERR_ALIGNMENT;
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
  p.group = n_heads / n_kv_heads;
  const int at_once = cache_dtype == FL_INT4 ? 8 : 16;  // query heads of one pass over the cache
  p.chunks = (p.group + at_once - 1) / at_once;
  p.chunk_heads = (p.group + p.chunks - 1) / p.chunks;
  p.page_of = page_divisor(page_size);
  // units of all lengths that the table allows (64 tokens at least), for all heads
  const int64_t longest = std::min<int64_t>(static_cast<int64_t>(max_pages) * page_size, INT32_MAX) / 64 + 2;
  p.small = batch <= 128 && longest * batch < (int64_t{1} << 31) / (static_cast<int64_t>(n_kv_heads) * p.chunks);
  p.window = window;
  p.sinks = sinks;
  p.eights = 0x00080008u;
  p.box = 0;
  p.timeout_ns = wait_timeout_ns();
  p.scale_log2 = scale_log2;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.status = reinterpret_cast<int*>(ws);
  p.counters = reinterpret_cast<unsigned*>(ws + kWsStatusBytes);
  p.parts = reinterpret_cast<float*>(ws + kWsStatusBytes + kDecMaxCtas * sizeof(unsigned));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // a window that no sequence can pass hides nothing
  const bool windowed = window > 0 && static_cast<int64_t>(window) + sinks < static_cast<int64_t>(max_pages) * page_size;
  const bool fp8 = cache_dtype == FL_E4M3;
  if (cache_dtype == FL_INT4) {
    // Tensor copies of 32, 16 or 8 tokens need whole boxes in a page, pages one behind the other (one index finds a row) and
    // scales that begin on 16 bytes; other caches are copied by 16 bytes.
    const int64_t rows = static_cast<int64_t>(num_pages) * n_kv_heads * page_size;
    const int box = page_size % 32 == 0 ? 32 : page_size % 16 == 0 ? 16 : page_size % 8 == 0 ? 8 : 0;
    const bool packed = num_pages == 1 || (page_pitch == static_cast<int64_t>(n_kv_heads) * page_size * cell.elems &&
                                           scale_pitch % 8 == 0);
    p.box = packed && rows > 0 && rows <= INT32_MAX && aligned16(k_page_scale) && aligned16(v_page_scale) ? box : 0;
    if (p.box > 0 && (!encode_2d(&p.map_k, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, k_pages, cell.elems, rows, cell.elems, cell.elems,
                                 p.box, CU_TENSOR_MAP_SWIZZLE_64B) ||
                      !encode_2d(&p.map_v, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, v_pages, cell.elems, rows, cell.elems, cell.elems,
                                 p.box, CU_TENSOR_MAP_SWIZZLE_64B)))
      return FL_ERR_CUDA;
    return launch_decode_int4(p, windowed, di, s);
  }
  if (windowed) return launch_decode_window(p, fp8, di, s);
  auto launch = [&](auto traits, auto* kernel) { return launch_decode<decltype(traits)>(kernel, p, di, s); };
  return fp8 ? decode_tiles<true, false>(p, launch) : decode_tiles<false, false>(p, launch);
}

}  // namespace
}  // namespace fl

extern "C" size_t fl_attention_decode_workspace_bytes(void) {
  return fl::kDecWorkspace;
}

extern "C" int attention_decode(const void* Q, const void* k_pages, const void* v_pages, const float* k_page_scale,
                                const float* v_page_scale, const int32_t* page_table, const int32_t* seq_lens, void* O,
                                int batch, int n_heads, int n_kv_heads, int head_dim, int page_size, int num_pages,
                                int max_pages, int64_t ldq, int64_t ldo, int64_t ldt, int64_t page_pitch,
                                int64_t scale_pitch, float scale, int cache_dtype, void* workspace,
                                size_t workspace_bytes, void* stream) {
  if (cache_dtype != FL_BF16 && cache_dtype != FL_E4M3) return FL_ERR_INVALID_ARG;
  return fl::enqueue_decode(Q, k_pages, v_pages, k_page_scale, v_page_scale, page_table, seq_lens, O, batch, n_heads,
                            n_kv_heads, head_dim, page_size, num_pages, max_pages, ldq, ldo, ldt, page_pitch, scale_pitch,
                            scale, 0, 0, cache_dtype, workspace, workspace_bytes, stream);
}

extern "C" int attention_decode_window(const void* Q, const void* k_pages, const void* v_pages, const void* k_page_scale,
                                       const void* v_page_scale, const int32_t* page_table, const int32_t* seq_lens,
                                       void* O, int batch, int n_heads, int n_kv_heads, int head_dim, int page_size,
                                       int num_pages, int max_pages, int64_t ldq, int64_t ldo, int64_t ldt,
                                       int64_t page_pitch, int64_t scale_pitch, float scale, int window, int sinks,
                                       int cache_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  if (window < 0 || sinks < 0) return FL_ERR_INVALID_ARG;
  return fl::enqueue_decode(Q, k_pages, v_pages, k_page_scale, v_page_scale, page_table, seq_lens, O, batch, n_heads,
                            n_kv_heads, head_dim, page_size, num_pages, max_pages, ldq, ldo, ldt, page_pitch, scale_pitch,
                            scale, window, sinks, cache_dtype, workspace, workspace_bytes, stream);
}
