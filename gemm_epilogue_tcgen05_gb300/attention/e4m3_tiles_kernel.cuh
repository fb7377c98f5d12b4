// The conversion in front of attention_prefill_kernel for E4M3 keys and values.
#pragma once
#include "prefill_attention_kernel.cuh"

namespace fl {

// E4M3 codes of K and V times their scales, for the prefill kernel: K as bf16, V as fp16 times 2^-b, with b for each key
// tile (128 rows of a sequence, from its first) and head: from V's largest finite scale where the tile's scales lie
// within kPreWindow powers of two, else from the window of that width that holds most of its keys; in either case not
// beyond kPrePowerMin and kPrePowerMax.  The keys outside it are written as zeros and marked as single keys.  Bound by
// memory: 1 byte in and 2 out for each value.  A CTA takes 16 rows of a key tile for up to 32 heads at a time, a thread
// 8 codes (16 bytes out; with 16 codes each store left half sectors to the next one); the scales of the whole tile are
// read by each of its eight CTAs (an eighth more to read, from L2) rather than one CTA turning a tile of one head (18.5
// instead of 11.2 us for 12400 rows of 8 heads, caches cold: too few, too long).
constexpr int kCodesRows = 16, kCodesHeads = 32;

__global__ void __launch_bounds__(256, 4) e4m3_tiles_kernel(
    const uint8_t* K, const uint8_t* V, const float* ks, const float* vs, long long ld, long long lds, const int* cu,
    int batch, int seq_len, int M, int n_kv, __nv_bfloat16* K16, __half* V16, float* powers) {
  __shared__ uint32_t top[kCodesHeads], low[kCodesHeads];  // largest and smallest finite scale of V, as bit patterns
  __shared__ float power[kCodesHeads];
  __shared__ int window[kCodesHeads];  // exponent field of its top; -1: it holds all keys
  __shared__ unsigned most;
  __shared__ short fields[kPreTile];
  const int tid = threadIdx.x, lane = tid & 31;
  if (tid < kCodesHeads) top[tid] = 0, low[tid] = ~0u;
  if (cu != nullptr && tid <= batch) asm volatile("prefetch.global.L2 [%0];" ::"l"(cu + tid));
  griddep_wait();
  griddep_launch_dependents();
  __syncthreads();
  constexpr int kParts = kPreTile / kCodesRows;
  const int tile = static_cast<int>(blockIdx.x / kParts), part = static_cast<int>(blockIdx.x % kParts);
  const int h0 = static_cast<int>(blockIdx.y) * kCodesHeads, heads = min(kCodesHeads, n_kv - h0);
  // Key tile j of sequence b has number cu[b] / 128 + b + j: no two have the same one, and each warp finds the sequence by
  // itself, by 32 probes at a time for the last b whose number is not above the tile's.
  int b = 0, at = tile;
  auto number = [&](int b) { return min(max(cu[b], 0), M) / kPreTile + b; };
  if (cu == nullptr) {
    const int each = (seq_len - 1) / kPreTile + 1;
    b = tile / each, at = tile - b * each;
  } else {
    for (int n = batch; n > 1;) {
      const int step = (n + 31) / 32;
      const unsigned below = __ballot_sync(~0u, lane * step < n && number(b + lane * step) <= tile);
      const int past = (32 - __clz(below) - 1) * step;
      if (below == 0) return;
      b += past;
      n = min(step, n - past);
    }
    at -= number(b);
  }
  int first, last;
  sequence_rows(cu, b, seq_len, M, first, last);
  if (at < 0 || at > (last - first - 1) / kPreTile) return;  // a number that nothing has; the same for all threads
  const int row0 = first + at * kPreTile, rows = min(kPreTile, last - row0);
  if (part * kCodesRows >= rows) return;  // the same for all threads
  const int r = part * kCodesRows + (tid >> 4), c = tid & 15;  // 16 threads a row and head
  const bool there = r < rows;
  const long long row = row0 + (there ? r : 0);
  constexpr int kTogether = 4;
  uint2 k[kTogether], v[kTogether];
  float sk[kTogether], sv[kTogether];
  auto fetch = [&](int j0) {
#pragma unroll
    for (int i = 0; i < kTogether; ++i) {
      if (j0 + i >= heads) break;
      const long long h = h0 + j0 + i;
      k[i] = reinterpret_cast<const uint2*>(K + row * ld + h * kHeadDim)[c];
      v[i] = reinterpret_cast<const uint2*>(V + row * ld + h * kHeadDim)[c];
      sk[i] = ks[row * lds + h];
      sv[i] = vs[row * lds + h];
    }
  };
  fetch(0);
  {
    const int each = 256 / heads, j = tid % heads;
    uint32_t largest = 0, smallest = ~0u;
    if (tid < each * heads)
      for (int q = tid / heads; q < rows; q += each) {
        const float x = fabsf(vs[(row0 + q) * lds + h0 + j]);
        if (x < INFINITY) largest = max(largest, __float_as_uint(x)), smallest = min(smallest, __float_as_uint(x));
      }
    if (smallest != ~0u) atomicMax(&top[j], largest), atomicMin(&low[j], smallest);
  }
  __syncthreads();
  constexpr int kFieldMin = 127 + kPreRoom + kPrePowerMin, kFieldMax = 127 + kPreRoom + kPrePowerMax;
  bool wide = false;
  if (tid < heads) {
    const int field = static_cast<int>(top[tid] >> 23);
    wide = top[tid] != 0 && (field - static_cast<int>(low[tid] >> 23) >= kPreWindow || field < kFieldMin || field > kFieldMax);
    power[tid] = top[tid] == 0 ? kPreZero : static_cast<float>(field - (127 + kPreRoom));
    window[tid] = wide ? field : -1;
  }
  if (__syncthreads_or(wide)) {
#pragma unroll 1
    for (int j = 0; j < heads; ++j) {
      if (window[j] < 0) continue;  // the same for all threads
      if (tid == 0) most = 0;
      if (tid < kPreTile) {
        const uint32_t bits = tid < rows ? __float_as_uint(fabsf(vs[(row0 + tid) * lds + h0 + j])) : 0u;
        fields[tid] = bits == 0 || bits >= 0x7F800000u ? -1 : static_cast<short>(bits >> 23);
      }
      __syncthreads();
      if (tid < rows && fields[tid] >= kFieldMin && fields[tid] <= kFieldMax) {
        const int mine = fields[tid];
        unsigned n = 0;
        for (int q = 0; q < rows; ++q) n += fields[q] > mine - kPreWindow && fields[q] <= mine;
        atomicMax(&most, n << 8 | mine);
      }
      __syncthreads();
      if (tid == 0) {
        window[j] = most != 0 ? static_cast<int>(most & 255u) : 512;  // 512: holds none
        power[j] = most != 0 ? static_cast<float>(window[j] - (127 + kPreRoom)) : 0.f;
      }
    }
    __syncthreads();
  }
  for (int j0 = 0; j0 < heads; j0 += kTogether) {
    if (j0 > 0) fetch(j0);
#pragma unroll
    for (int i = 0; i < kTogether; ++i) {
      if (j0 + i >= heads || !there) break;
      auto codes = [](uint2 in, float scale, auto pack) {
        uint32_t out[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          uint32_t two;
          asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(two) : "h"(static_cast<uint16_t>((e < 2 ? in.x : in.y) >> ((e & 1) * 16))));
          const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&two));
          out[e] = pack(f.x * scale, f.y * scale);
        }
        return make_uint4(out[0], out[1], out[2], out[3]);
      };
      const float b = power[j0 + i];
      const int win = window[j0 + i];
      const uint32_t bits = __float_as_uint(fabsf(sv[i]));
      const int field = static_cast<int>(bits >> 23);
      const bool single = win >= 0 && field < 255 && (bits == 0 || field > win || field <= win - kPreWindow);
      // 448 * scale * 2^-b is below 2^16 * 0.875
      const float down = __uint_as_float(static_cast<uint32_t>(127 - static_cast<int>(b)) << 23);
      const long long to = (row * n_kv + h0 + j0 + i) * (kHeadDim / 8) + c;
      reinterpret_cast<uint4*>(K16)[to] = codes(k[i], sk[i], [](float x, float y) { return pack_bf16x2(x, y); });
      uint4 v16 = codes(v[i], sv[i] * down, [](float x, float y) { return pack_f16x2(x, y); });
      if (single && bits != 0) v16 = make_uint4(0, 0, 0, 0);  // a scale of zero leaves zeros, and what is not a number
      reinterpret_cast<uint4*>(V16)[to] = v16;
      if (c == 0 && (r == 0 || win >= 0))
        powers[row * n_kv + h0 + j0 + i] =
            r == 0 ? b + kPreMark * ((win >= 0 ? PRE_SINGLE : 0) | (single ? PRE_SINGLE_FIRST : 0))
                   : single ? 1.f : 0.f;
    }
  }
}

}  // namespace fl
