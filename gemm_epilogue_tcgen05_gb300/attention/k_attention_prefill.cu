// attention_prefill and attention_prefill_window: argument checks, tensor maps and launch (the kernel:
// prefill_attention_kernel.cuh).
#include <cudaTypedefs.h>

#include <algorithm>
#include <mutex>

#include "e4m3_tiles_kernel.cuh"
#include "prefill_attention_host.cuh"

namespace fl {
namespace {

constexpr int64_t kL2Share = 32 << 20;  // keys and values of the heads worked off together
// The order of the tiles: by falling cost, with a walk over the sequences for each tier of blocks, or in the order of the
// sequences, with one walk.  Up to 32 sequences stay in a warp's lanes and a tier costs little.  Measured, causal | full
// mask, 32 query and 8 kv heads (tiers -> one walk): 4 x 2048 108 -> 113 | 176 -> 177 us, 32 of 200-2000 tokens and one
// of 8000 523 -> 539 | 894 -> 899, 64 of 20-1500 154 -> 158 | 207 -> 214, 64 of 200-2000 and one of 8000 916 -> 686 |
// 1143 -> 1184, 128 of 20-1500 and one of 4000 765 -> 356 | 623 -> 520, 1024 of 20-100 and one of 8000 9945 -> 634 |
// 5180 -> 863.
constexpr int kTierBatch = 32, kTierBatchFull = 64;

// 3-D tiled map over Q [rows][heads][128] bf16 with a row pitch of ld elements.
bool encode_q(CUtensorMap* map, const void* base, int heads, int rows, int64_t ld, int hp, int tq) {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void* f = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &r) == cudaSuccess &&
        r == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
  });
  if (fn == nullptr) return false;
  const cuuint64_t dims[3] = {kHeadDim, static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {kHeadDim * 2, static_cast<cuuint64_t>(ld) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(hp), static_cast<cuuint32_t>(tq)}, step[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Query heads of a tile: the largest part of a group that leaves room for two tokens.
int heads_of_tile(int group) {
  int hp = group < 64 ? group : 64;
  while (group % hp != 0) --hp;
  return hp;
}
// Blocks of per_cta tokens, at most (the lengths are on the device): a sequence of n has (n - 1) / per_cta + 1.
long long packed_blocks(int M, int batch, long long per_cta) {
  const int some = std::min(M, batch);
  return (M - some) / per_cta + some;
}

// Parts that each unit may be cut into where few units go over many keys, 1: none.  A part costs a unit's output, 128 KB into the
// scratch buffer and out of it, and a second kernel joins them, so they pay where SMs would be idle and units be long.  Measured,
// whole units -> parts, 32/8 heads, bf16: 33 tokens behind 5000 58.1 -> 24.8 us, 128 behind 8000 92.9 -> 35.5, 512 behind 8000 96.7
// -> 62.1, 16 behind 1500 (two parts) 20.9 -> 18.1, which the second launch costs the host; E4M3, 33 behind 5000 70.1 -> 34.4.  From
// half as many units as SMs on a part for each is none to spare: 576 behind 8000 93.8 -> 60.2, 577 stay whole with 94.9 (a batch
// of 144 units of up to 33 tiles, all of them cut, 55 -> 62).
// The lengths are on the device: of several sequences the longest is taken to be what it is where they are spread evenly from
// none on, 2 M_k / (batch + 1), and where that is short nothing is cut, for the binding's pass and the kernel, 4 x 20 behind 480
// tokens: 20.3 -> 10.8 us, 13.0 -> 10.5 (16/2 heads, 16 x 20 behind 480: 19.8 -> 11.6, 13.8 -> 11.2).  Above, what even
// lengths lose, 4 x 20 behind 980 16.2 -> 20.2, 15.8 -> 17.0, is less than what uneven ones gain, 60, 60, 60 and 3000 keys: 37.1 ->
// 23.6, 36.9 -> 23.3, fifteen times 250 and once 6000: 67.2 -> 34.6, 66.8 -> 34.3.
constexpr int kCutKeys = 1000;
int parts_of_units(long long units, int M_k, int batch, int window, int sinks, long long per_cta, int num_sms) {
  if (2ll * M_k < kCutKeys * (batch + 1ll)) return 1;
  long long keys = M_k;
  if (window > 0) keys = std::min(keys, static_cast<long long>(window) + sinks + 61 + per_cta);
  const long long longest = (keys - 1) / kPreTile / kPrePartTiles + 1;
  if (longest < 3) return 1;
  return static_cast<int>(std::max<long long>(std::min(longest, num_sms / units), 1));
}
size_t scratch_of(long long numbers) {
  return numbers * kPrePartFloats * sizeof(float) + (numbers + 1) * sizeof(PrefillCut);
}

}  // namespace
}  // namespace fl

extern "C" size_t fl_attention_prefill_window_scratch_bytes(int M, int M_k, int batch, int n_heads, int n_kv_heads, int window,
                                                            int sinks) {
  using namespace fl;
  DeviceInfo di;
  if (M <= 0 || M_k <= 0 || batch <= 0 || n_heads <= 0 || n_kv_heads <= 0 || n_heads % n_kv_heads != 0 || window < 0 ||
      sinks < 0 || current_device(&di) != FL_OK)
    return 0;
  const int hp = heads_of_tile(n_heads / n_kv_heads);
  const long long per_cta = 2 * (kPreTile / hp), units = packed_blocks(M, batch, per_cta) * (n_heads / hp);
  const int parts = parts_of_units(units, M_k, batch, window, sinks, per_cta, di.num_sms);
  return parts > 1 ? scratch_of(units * parts) : 0;
}

extern "C" size_t fl_attention_prefill_workspace_bytes(int M, int n_kv_heads, int kv_dtype) {
  using namespace fl;
  if (M < 0 || n_kv_heads < 0) return 0;
  // the status record and the work counters; for E4M3 also K as bf16, V as fp16 and a power for each key tile (kept at
  // its first row; where it has single keys, the other rows hold which)
  const size_t rows = static_cast<size_t>(M) * n_kv_heads;
  return 2 * kWsStatusBytes + (kv_dtype == FL_E4M3 ? rows * (kHeadDim * (sizeof(__nv_bfloat16) + sizeof(__half)) + sizeof(float)) : 0);
}

namespace fl {
namespace {

int enqueue_prefill(const void* Q, const void* K, const void* V, const float* k_scale, const float* v_scale,
                    const int32_t* cu_seqlens, const int32_t* cu_seqlens_k, void* O, int M, int M_k, int batch, int n_heads,
                    int n_kv_heads, int head_dim, int seq_len, int64_t ldq, int64_t ldkv, int64_t lds, int64_t ldo,
                    float scale, int causal, int window, int sinks, int kv_dtype, void* workspace,
                    size_t workspace_bytes, void* scratch, size_t scratch_bytes, void* stream) {
  if (M < 0 || M_k < 0 || n_heads < 0 || n_kv_heads < 0 || (cu_seqlens != nullptr ? batch < 0 : seq_len < 1))
    return FL_ERR_INVALID_ARG;
  if (cu_seqlens_k != nullptr ? cu_seqlens == nullptr : M_k != M) return FL_ERR_INVALID_ARG;
  const bool fp8 = kv_dtype == FL_E4M3;
  float scale_log2;
  if ((kv_dtype != FL_BF16 && !fp8) || !scale_to_base_2(scale, &scale_log2)) return FL_ERR_INVALID_ARG;
  if (M == 0 || n_heads == 0 || (cu_seqlens != nullptr && batch == 0)) return FL_OK;
  if (M_k == 0 || n_kv_heads == 0 || n_heads % n_kv_heads != 0) return FL_ERR_INVALID_ARG;
  if (head_dim != kHeadDim) return FL_ERR_UNSUPPORTED;
  if (n_heads > kMaxHeads) return FL_ERR_UNSUPPORTED;
  if (Q == nullptr || K == nullptr || V == nullptr || O == nullptr) return FL_ERR_INVALID_ARG;
  if (fp8 && (k_scale == nullptr || v_scale == nullptr)) return FL_ERR_INVALID_ARG;
  const int64_t width = static_cast<int64_t>(n_heads) * kHeadDim, kv_width = static_cast<int64_t>(n_kv_heads) * kHeadDim;
  if (ldq < width || ldo < width || ldkv < kv_width || (fp8 && lds < n_kv_heads)) return FL_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(O)) return FL_ERR_ALIGNMENT;
  if (!pitch_ok(ldq, 2) || !pitch_ok(ldo, 2) || !pitch_ok(ldkv, fp8 ? 1 : 2)) return FL_ERR_ALIGNMENT;
  if (((reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale) |
        reinterpret_cast<uintptr_t>(cu_seqlens) | reinterpret_cast<uintptr_t>(cu_seqlens_k)) & 3u) != 0)
    return FL_ERR_ALIGNMENT;
  if (workspace == nullptr || workspace_bytes < fl_attention_prefill_workspace_bytes(M_k, n_kv_heads, kv_dtype))
    return FL_ERR_WORKSPACE;
  if ((reinterpret_cast<uintptr_t>(workspace) & (kWsStatusBytes - 1)) != 0 || !aligned16(scratch)) return FL_ERR_ALIGNMENT;
  DeviceInfo di;
  const int st = current_device(&di);
  if (st != FL_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);

  PrefillParams p;
  std::memset(&p, 0, sizeof(p));
  p.group = n_heads / n_kv_heads;
  p.hp = heads_of_tile(p.group);
  p.tq = kPreTile / p.hp;
  p.pairs = n_heads / p.hp;
  const int64_t kv_bytes = static_cast<int64_t>(M_k) * kHeadDim * 4;  // of one kv head, as bf16
  const int64_t at_once = std::max<int64_t>(kL2Share / kv_bytes, 1);
  const int64_t groups = (n_kv_heads + at_once - 1) / at_once;
  p.pairs_at_once = static_cast<int>((n_kv_heads + groups - 1) / groups) * (p.group / p.hp);
  p.batch = cu_seqlens == nullptr ? (M - 1) / seq_len + 1 : batch;
  p.seq_len = seq_len;
  const long long per_cta = 2 * p.tq;
  const long long blocks = cu_seqlens == nullptr
                               ? (M / seq_len) * ((seq_len - 1) / per_cta + 1) + (M % seq_len + per_cta - 1) / per_cta
                               : packed_blocks(M, batch, per_cta);
  if (blocks * p.pairs > (1ll << 30)) return FL_ERR_UNSUPPORTED;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const void* k16 = K;
  const void* v16 = V;
  int64_t ld16 = ldkv;
  if (fp8) {
    __nv_bfloat16* kw = reinterpret_cast<__nv_bfloat16*>(ws + 2 * kWsStatusBytes);
    __half* vw = reinterpret_cast<__half*>(kw + static_cast<size_t>(M_k) * kv_width);
    p.powers = reinterpret_cast<const float*>(vw + static_cast<size_t>(M_k) * kv_width);
    k16 = kw, v16 = vw, ld16 = kv_width;
    p.codes = static_cast<const uint8_t*>(V);
    p.v_scale = v_scale;
    p.ld_codes = ldkv;
    p.ld_scale = lds;
  }
  if (!encode_q(&p.map_q, Q, n_heads, M, ldq, p.hp, p.tq) ||
      !encode_2d(&p.map_k, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, k16, kv_width, M_k, ld16, 64, kPreTile,
                 CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_2d(&p.map_v, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, v16, kv_width, M_k, ld16, 64, kPreTile,
                 CU_TENSOR_MAP_SWIZZLE_128B))
    return FL_ERR_CUDA;
  if ((window > 0 || cu_seqlens_k != nullptr) &&
      (!encode_2d(&p.map_k32, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, k16, kv_width, M_k, ld16, 64, 32,
                  CU_TENSOR_MAP_SWIZZLE_128B) ||
       !encode_2d(&p.map_v32, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, v16, kv_width, M_k, ld16, 64, 32,
                  CU_TENSOR_MAP_SWIZZLE_128B)))
    return FL_ERR_CUDA;
  p.V = static_cast<const __nv_bfloat16*>(v16);
  p.ldv = ld16;
  p.n_kv = n_kv_heads;
  p.cu = cu_seqlens;
  p.O = static_cast<__nv_bfloat16*>(O);
  p.ldo = ldo;
  p.M = M;
  p.causal = causal != 0;
  // a window as long as the rows hides nothing
  p.window = window < M_k ? window : 0;
  p.sinks = sinks < M_k ? sinks : M_k;
  p.cu_k = cu_seqlens_k;
  p.M_k = M_k;
  p.flat = p.window > 0 || p.batch > (p.causal ? kTierBatch : kTierBatchFull);
  p.scale_log2 = scale_log2;
  p.status = reinterpret_cast<int*>(ws);
  p.work = reinterpret_cast<unsigned*>(ws + kWsStatusBytes);
  p.timeout_ns = wait_timeout_ns();
  const bool windowed = p.window > 0 || cu_seqlens_k != nullptr;
  const long long units = blocks * p.pairs;
  const int most_parts = cu_seqlens_k == nullptr ? 1 : parts_of_units(units, M_k, batch, p.window, p.sinks, per_cta, di.num_sms);
  const bool cut = most_parts > 1 && scratch != nullptr && scratch_bytes >= scratch_of(units * most_parts);
  if (cut) {
    p.flat = 1;
    p.most_parts = most_parts;
    p.numbers = static_cast<int>(units * most_parts);
    p.cuts = static_cast<PrefillCut*>(scratch);
    p.parts = reinterpret_cast<float*>(p.cuts + 1 + units * most_parts);
  }
  if (!fp8 && cut) return launch_prefill_parts(p, false, units * most_parts, di, s);
  if (!fp8)
    return windowed ? launch_prefill_window(p, false, blocks * p.pairs, di, s)
                    : launch_prefill<false, false>(p, blocks * p.pairs, di, s);
  const int32_t* cu_tiles = cu_seqlens_k != nullptr ? cu_seqlens_k : cu_seqlens;
  const long long key_tiles =
      cu_seqlens == nullptr
          ? static_cast<long long>(M / seq_len) * ((seq_len - 1) / kPreTile + 1) + (M % seq_len + kPreTile - 1) / kPreTile
          : static_cast<long long>(M_k) / kPreTile + batch;  // the numbers that tiles can have
  const long long parts = key_tiles * (kPreTile / kCodesRows);
  if (parts > INT32_MAX) return FL_ERR_UNSUPPORTED;
  if (!launch_dependent(e4m3_tiles_kernel, dim3(static_cast<unsigned>(parts), (n_kv_heads - 1) / kCodesHeads + 1), 256, 0, s,
                        static_cast<const uint8_t*>(K),
                        static_cast<const uint8_t*>(V), k_scale, v_scale, static_cast<long long>(ldkv),
                        static_cast<long long>(lds), cu_tiles, p.batch, seq_len, M_k, n_kv_heads,
                        static_cast<__nv_bfloat16*>(const_cast<void*>(k16)), static_cast<__half*>(const_cast<void*>(v16)),
                        const_cast<float*>(p.powers)))
    return FL_ERR_CUDA;
  if (cut) return launch_prefill_parts(p, true, units * most_parts, di, s);
  return windowed ? launch_prefill_window(p, true, blocks * p.pairs, di, s)
                  : launch_prefill<true, false>(p, blocks * p.pairs, di, s);
}

}  // namespace
}  // namespace fl

extern "C" int attention_prefill(const void* Q, const void* K, const void* V, const float* k_scale,
                                 const float* v_scale, const int32_t* cu_seqlens, void* O, int M, int batch,
                                 int n_heads, int n_kv_heads, int head_dim, int seq_len, int64_t ldq, int64_t ldkv,
                                 int64_t lds, int64_t ldo, float scale, int causal, int kv_dtype, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  return fl::enqueue_prefill(Q, K, V, k_scale, v_scale, cu_seqlens, nullptr, O, M, M, batch, n_heads, n_kv_heads, head_dim,
                             seq_len, ldq, ldkv, lds, ldo, scale, causal, 0, 0, kv_dtype, workspace, workspace_bytes,
                             nullptr, 0, stream);
}

extern "C" int attention_prefill_window(const void* Q, const void* K, const void* V, const float* k_scale,
                                        const float* v_scale, const int32_t* cu_seqlens, const int32_t* cu_seqlens_k,
                                        void* O, int M, int M_k, int batch, int n_heads, int n_kv_heads, int head_dim,
                                        int seq_len, int64_t ldq, int64_t ldkv, int64_t lds, int64_t ldo, float scale,
                                        int window, int sinks, int kv_dtype, void* workspace, size_t workspace_bytes,
                                        void* scratch, size_t scratch_bytes, void* stream) {
  if (window < 0 || sinks < 0) return FL_ERR_INVALID_ARG;
  return fl::enqueue_prefill(Q, K, V, k_scale, v_scale, cu_seqlens, cu_seqlens_k, O, M, M_k, batch, n_heads, n_kv_heads,
                             head_dim, seq_len, ldq, ldkv, lds, ldo, scale, 1, window, sinks, kv_dtype, workspace,
                             workspace_bytes, scratch, scratch_bytes, stream);
}
