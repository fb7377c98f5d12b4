// Attention of one new token per sequence over a paged key-value cache of bf16 or E4M3.
//
//   o_h = sum_j p_j v_j / sum_j p_j,  p_j = 2^(x_j - m),  x_j = scale * log2(e) * q_h . k_j
//
// What bounds it: the cache is read once, 4 * 128 * group multiply-adds for every 256 (E4M3) or 512 (bf16)
// bytes, so it runs at the memory's rate as long as enough loads are in flight and nothing else keeps a warp
// from issuing the next ones.
//
// Units (decode_attention_common.cuh) are 64 (bf16) or 128 (E4M3) tokens long.
//
// Inside a CTA each of four warps streams its own tokens, 16 (bf16) or 32 (E4M3, two independent tiles: the
// conversions make a step longer) at a time, through its own ring of cp.async
// stages: no barrier in the loop, and the ring runs on over the end of a sequence.  Both products run on the
// tensor cores with the tokens on the M side, S^T = K Q^T and O^T = V^T P^T (m16n8k16: 8 query heads of a group
// in the N columns, two column tiles for groups above 8), so a small group wastes little.  The assignment of
// cache columns to MMA k-indexes is free as long as both operands agree: each lane takes 16 consecutive bytes
// of a row, and the query's fragments are loaded in the same order.  V^T needs two tokens of one dimension in a
// register: bytes of two rows interleaved by prmt.  Chunks of 16 bytes are permuted inside a row (xor with bits
// of the row) so that no quarter warp meets a bank twice.
//
// E4M3: codes become fp16 exactly (cvt.f16x2.e4m3x2); a query head is scaled by a power of two to fp16's upper
// range, where its bf16 values are exact down to 2^-29 of the largest; the scales stay in fp32: K's multiplies
// the logit, V's enters the weight as 2^(x_j + log2 vs_j - m').  m' is the running maximum of that exponent, so
// weights lie in [0, 2^15] and are rounded to fp16 (2^-11).
// bf16: weights are split into two bf16 terms (hi + lo, 2^-16) so that the product is as exact as the inputs.
//
// The maxima m and m' rise only when a logit passes them by more than 8 (2^8 fits every type used): then the
// sums are rescaled.  That takes one vote in most steps instead of six shuffles and a rescale of O.
#pragma once
#include "decode_attention_common.cuh"

namespace fl {

constexpr int kDecWarps = 4;
constexpr int kDecThreads = 32 * kDecWarps;

template <bool FP8, int NT>
struct DecodeTraits {
  static constexpr int kThreads = kDecThreads;
  static constexpr int kRowBytes = FP8 ? 128 : 256;
  static constexpr int kSubs = FP8 ? 2 : 1;          // 16-token tiles of one warp's step
  static constexpr int kStep = 16 * kSubs;
  static constexpr int kUnit = kDecWarps * kStep;    // tokens of one unit of work
  static constexpr int kTile = kStep * kRowBytes;
  static constexpr int kStage = 2 * kTile + (FP8 ? 2 * kStep * 4 : 0);
  // CTAs on an SM and stages of a warp's ring.  Measured (64 sequences of 2048-8192 tokens, E4M3): 2 x 3 stages
  // 104.7 us, 3 x 2 108.3 us; (24 sequences of 5-4096 tokens | 3 of 15000-32768, bf16): 2 x 3 25.2 | 87.9 us, 3 x 2
  // 22.2 | 89.1 us.  Two column tiles need the registers of 3 CTAs.
  static constexpr int kCtas = !FP8 && NT == 1 ? 3 : 2;
  static constexpr int kStages = kCtas == 3 ? 2 : 3;
  static_assert(kStage >= NT * 8 * kHeadDim * 4, "a stage takes a warp's piece");
  static constexpr int kSmem = kDecWarps * kStages * kStage + kDecWarps * NT * 8 * 16 + 128;
};

__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}
template <bool FP8, int NT, bool WIN>
__global__ void __launch_bounds__(kDecThreads, DecodeTraits<FP8, NT>::kCtas) attention_decode_kernel(const __grid_constant__ DecodeParams p) {
  using T = DecodeTraits<FP8, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  float4* stats = reinterpret_cast<float4*>(smem + kDecWarps * T::kStages * T::kStage);  // [warp][head]: m, m', l, stage
  long long* plan = reinterpret_cast<long long*>(stats + kDecWarps * NT * 8);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  const DecodeWalk<T::kUnit, WIN> walk(p);
  decode_hints(p, tid);
  griddep_wait();  // launched as a dependent: nothing is read before the kernel in front has finished
  griddep_launch_dependents();
  DecodeShare own;
  DecodeSeg seg;
  if (!decode_plan<kDecThreads>(p, walk, plan, own, seg)) return;
  long long left = own.u1 - own.u0;

  // ---- producer side of this warp's ring
  DecodeSeg ps = seg;
  long long p_left = left;
  int pt = ps.t0 + warp * T::kStep, entry = 0, slot = 0, p_stage = 0;  // slot: in the page that entry is
  uint32_t bad_steps = 0;  // stages whose page-table entry is outside the cache
  bool fresh = true;
  const bool one_page = (p.c.page_size & (T::kStep - 1)) == 0;  // a step's 16 tokens lie in one page
  auto settle = [&]() {  // moves on to this warp's next step and fetches its page-table entry
    while (pt >= ps.t1) {
      p_left -= ps.units;
      if (p_left <= 0) return;
      walk.next(ps, p_left);
      pt = ps.t0 + warp * T::kStep;
      fresh = true;
    }
    if (fresh) {  // the query rows of the segment that begins, into L2
      fresh = false;
      const char* row = reinterpret_cast<const char*>(p.Q + ps.b * p.ldq + static_cast<long long>(ps.kvh) * p.group * kHeadDim);
      if (lane < 2 * p.group) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + lane * 128));
    }
    const int pos = (one_page ? pt : min(pt + (lane & (T::kStep - 1)), ps.t1 - 1)) + walk.shift_of(ps, pt);
    const int page = walk.page_of(pos);
    slot = pos - page * p.c.page_size;
    entry = p.c.table[ps.b * p.c.ldt + page];
  };
  const uint32_t ring = smem_u32(smem) + warp * T::kStages * T::kStage;
  auto issue = [&]() {
    if (p_left > 0) {
      constexpr int kChunks = T::kRowBytes / 16, kRowsPer = 32 / kChunks;
      const uint32_t dst = ring + p_stage * T::kStage;
      const int rows = ps.t1 - pt, shift = walk.shift_of(ps, pt);
      const bool ok = static_cast<unsigned>(entry) < static_cast<unsigned>(p.c.num_pages);
      bool used = true;  // some row of the page is needed
      if (WIN) {
        const int mypos = (one_page ? pt : min(pt + (lane & (T::kStep - 1)), ps.t1 - 1)) + shift;
        used = walk.in_sight(ps, mypos) || (one_page && walk.in_sight(ps, min(pt + T::kStep, ps.t1) - 1 + shift));
      }
      bad_steps = (bad_steps & ~(1u << p_stage)) | (ok || !used ? 0u : 1u << p_stage);
      const int mypage = ok ? entry : 0;
      const int c = lane % kChunks, row0 = lane / kChunks;
      const long long cell = static_cast<long long>(ps.kvh) * p.c.page_size + slot;
      if (one_page) {
        const long long byte = (mypage * p.c.page_pitch + (cell + row0) * kHeadDim) * (FP8 ? 1 : 2) + c * 16;
        const uint8_t* ksrc = static_cast<const uint8_t*>(p.c.k) + byte;
        const uint8_t* vsrc = static_cast<const uint8_t*>(p.c.v) + byte;
#pragma unroll
        for (int i = 0; i < T::kStep / kRowsPer; ++i) {
          const int row = row0 + i * kRowsPer;
          const bool there = ok && row < rows && walk.in_sight(ps, pt + row + shift);
          cp_async_16_or_zero(dst + row * T::kRowBytes + ((c ^ ((row & 1) << 2)) << 4), ksrc + i * 512, there);
          cp_async_16_or_zero(dst + T::kTile + row * T::kRowBytes + ((c ^ (row & 6)) << 4), vsrc + i * 512, there);
        }
      } else {
#pragma unroll
        for (int i = 0; i < T::kStep / kRowsPer; ++i) {
          const int row = row0 + i * kRowsPer;
          const int page = __shfl_sync(~0u, ok ? entry : -1, row), s = __shfl_sync(~0u, slot, row);
          const bool there = page >= 0 && row < rows && walk.in_sight(ps, pt + row + shift);
          const long long at = max(page, 0) * p.c.page_pitch + (static_cast<long long>(ps.kvh) * p.c.page_size + s) * kHeadDim;
          const long long byte = at * (FP8 ? 1 : 2) + c * 16;
          cp_async_16_or_zero(dst + row * T::kRowBytes + ((c ^ ((row & 1) << 2)) << 4),
                              static_cast<const uint8_t*>(p.c.k) + byte, there);
          cp_async_16_or_zero(dst + T::kTile + row * T::kRowBytes + ((c ^ (row & 6)) << 4),
                              static_cast<const uint8_t*>(p.c.v) + byte, there);
        }
      }
      if (FP8) {  // lane = row of the step
        const bool there = ok && lane < rows && walk.in_sight(ps, pt + lane + shift);
        const long long at = mypage * p.c.scale_pitch + cell + (one_page ? lane : 0);
        cp_async_4_or_zero(dst + 2 * T::kTile + lane * 4, static_cast<const float*>(p.c.ks) + at, there);
        cp_async_4_or_zero(dst + 2 * T::kTile + 128 + lane * 4, static_cast<const float*>(p.c.vs) + at, there);
      }
      pt += T::kUnit;
      settle();
    }
    cp_async_commit();
    p_stage = p_stage + 1 == T::kStages ? 0 : p_stage + 1;
  };
  DecodeCuts cuts;
  settle();
#pragma unroll
  for (int i = 0; i < T::kStages - 1; ++i) issue();
  int stage = 0;

  for (;;) {
    // ---- this segment's query fragments (B operand: head g of the column tile, dimensions in the cache's order)
    const int head0 = seg.kvh * p.group + seg.chunk * p.chunk_heads;
    const int n_heads = min(p.chunk_heads, p.group - seg.chunk * p.chunk_heads);
    uint32_t qf[NT][16];
    float fac[NT][2];  // of heads 2q, 2q + 1 of the column tile
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const bool has = nt * 8 + g < n_heads;
      const __nv_bfloat16* src = p.Q + seg.b * p.ldq + static_cast<long long>(head0 + nt * 8 + g) * kHeadDim;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int d = FP8 ? ((i >> 1) * 4 + q) * 16 + (i & 1) * 8 : (i * 4 + q) * 8;
        uint4 w = make_uint4(0, 0, 0, 0);
        if (has) w = *reinterpret_cast<const uint4*>(src + d);
        qf[nt][i * 4] = w.x, qf[nt][i * 4 + 1] = w.y, qf[nt][i * 4 + 2] = w.z, qf[nt][i * 4 + 3] = w.w;
      }
      float f = p.scale_log2;
      if (FP8) {
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) a = fmaxf(a, fmaxf(fabsf(bf16_lo(qf[nt][i])), fabsf(bf16_hi(qf[nt][i]))));
        a = fmaxf(a, __shfl_xor_sync(~0u, a, 1));
        a = fmaxf(a, __shfl_xor_sync(~0u, a, 2));
        // 2^e that takes the largest value to [2^14, 2^15); values that are not finite stay what they are
        const int ex = static_cast<int>(__float_as_uint(a) >> 23);
        const int up = ex == 255 ? 127 : min(max(268 - ex, 1), 253);
        const float lift = __uint_as_float(static_cast<uint32_t>(up) << 23);
        f *= __uint_as_float(static_cast<uint32_t>(254 - up) << 23);
#pragma unroll
        for (int i = 0; i < 16; ++i) qf[nt][i] = pack_f16x2(bf16_lo(qf[nt][i]) * lift, bf16_hi(qf[nt][i]) * lift);
      }
      fac[nt][0] = __shfl_sync(~0u, f, q * 8);
      fac[nt][1] = __shfl_sync(~0u, f, q * 8 + 4);
    }
    bool bad = seg.bad;
    float o[NT][8][4];
    float m[NT][2], mv[NT][2], l[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int t = 0; t < 8; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[nt][t][i] = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) m[nt][i] = mv[nt][i] = kDecNone, l[nt][i] = 0.f;
    }

    for (int t = seg.t0 + warp * T::kStep; t < seg.t1; t += T::kUnit) {
      cp_async_wait<T::kStages - 2>();
      __syncwarp();
      const uint32_t kb = ring + stage * T::kStage, vb = kb + T::kTile;
      float x[NT][T::kSubs * 4];  // logits: lane (g, q) holds tokens g, g + 8 of each tile for heads 2q, 2q + 1
      float lv[T::kSubs * 2];     // binary logarithm of V's scale
      // ---- S^T = K Q^T: tiles of 16 tokens x 8 heads, k = 128
      float s[NT][T::kSubs][2][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < T::kSubs * 8; ++i) s[nt][i >> 3][(i >> 2) & 1][i & 3] = 0.f;
      const uint32_t kr = kb + g * T::kRowBytes;
      const int sw = (g & 1) << 2;
#pragma unroll
      for (int ci = 0; ci < T::kRowBytes / 64; ++ci)
#pragma unroll
        for (int sub = 0; sub < T::kSubs; ++sub) {
          const uint32_t at = kr + sub * 16 * T::kRowBytes + (((ci * 4 + q) ^ sw) << 4);
          const uint4 x = ld_shared_v4(at), y = ld_shared_v4(at + 8 * T::kRowBytes);
          const uint32_t xr[4] = {x.x, x.y, x.z, x.w}, yr[4] = {y.x, y.y, y.z, y.w};
          if (FP8) {
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const uint32_t a0 = e4m3x2_to_f16x2(xr[u] & 0xFFFFu), a2 = e4m3x2_to_f16x2(xr[u] >> 16);
              const uint32_t a1 = e4m3x2_to_f16x2(yr[u] & 0xFFFFu), a3 = e4m3x2_to_f16x2(yr[u] >> 16);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_16816<true>(s[nt][sub][u & 1], a0, a1, a2, a3, qf[nt][ci * 8 + u * 2], qf[nt][ci * 8 + u * 2 + 1]);
            }
          } else {
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_16816<false>(s[nt][sub][u], xr[u * 2], yr[u * 2], xr[u * 2 + 1], yr[u * 2 + 1],
                                 qf[nt][ci * 4 + u * 2], qf[nt][ci * 4 + u * 2 + 1]);
          }
        }
      float ks[T::kSubs * 2];
#pragma unroll
      for (int r = 0; r < T::kSubs * 2; ++r) {
        ks[r] = 1.f, lv[r] = 0.f;
        if (FP8) {
          const float* sc = reinterpret_cast<const float*>(smem + (kb - smem_u32(smem)) + 2 * T::kTile);
          ks[r] = sc[g + r * 8];
          lv[r] = lg2(sc[T::kStep + g + r * 8]);
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < T::kSubs * 4; ++i) {
          x[nt][i] = (s[nt][i >> 2][0][i & 3] + s[nt][i >> 2][1][i & 3]) * fac[nt][i & 1];
          if (FP8) x[nt][i] *= ks[i >> 1];
        }
      // ---- softmax
      bool rise = false;
      const int pos0 = t + walk.shift_of(seg, t);
      bool cut = t + T::kStep > seg.t1;
      if (WIN) cut |= pos0 + T::kStep > p.sinks && pos0 < seg.len - p.window;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < T::kSubs * 4; ++i) {
          float v = x[nt][i];
          if (cut && (t + g + (i >> 1) * 8 >= seg.t1 || !walk.in_sight(seg, pos0 + g + (i >> 1) * 8))) v = -INFINITY;
          x[nt][i] = v;
          rise |= v > m[nt][i & 1] + kDecLazy;
          if (FP8) rise |= v + lv[i >> 1] > mv[nt][i & 1] + kDecLazy;
        }
      if (__any_sync(~0u, rise)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float a = m[nt][i], b = mv[nt][i];
#pragma unroll
            for (int r = 0; r < T::kSubs * 2; ++r) {
              a = fmaxf(a, x[nt][r * 2 + i]);
              if (FP8) b = fmaxf(b, x[nt][r * 2 + i] + lv[r]);
            }
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
              a = fmaxf(a, __shfl_xor_sync(~0u, a, d));
              if (FP8) b = fmaxf(b, __shfl_xor_sync(~0u, b, d));
            }
            const float down = ex2(m[nt][i] - a), down_o = FP8 ? ex2(mv[nt][i] - b) : down;
            m[nt][i] = a;
            mv[nt][i] = b;
            l[nt][i] *= down;
#pragma unroll
            for (int d = 0; d < 8; ++d) o[nt][d][i] *= down_o, o[nt][d][i + 2] *= down_o;
          }
      }
      uint32_t pf[NT][T::kSubs][2], pl[NT][T::kSubs][2];  // P^T (B operand: tokens 2q, 2q + 1 | + 8 of head g)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float w[T::kSubs * 4];
#pragma unroll
        for (int i = 0; i < T::kSubs * 4; ++i) {
          const float e = ex2(x[nt][i] - m[nt][i & 1]);
          l[nt][i & 1] += e;
          w[i] = FP8 ? ex2((x[nt][i] + lv[i >> 1]) - (mv[nt][i & 1] - kDecLift)) : e;
        }
#pragma unroll
        for (int r = 0; r < T::kSubs * 2; ++r) {
          if (FP8) {
            pf[nt][r >> 1][r & 1] = transpose8x8(pack_f16x2(w[r * 2], w[r * 2 + 1]));
          } else {
            const uint32_t hi = pack_bf16x2(w[r * 2], w[r * 2 + 1]);
            pf[nt][r >> 1][r & 1] = transpose8x8(hi);
            pl[nt][r >> 1][r & 1] = transpose8x8(pack_bf16x2(w[r * 2] - bf16_lo(hi), w[r * 2 + 1] - bf16_hi(hi)));
          }
        }
      }
      // ---- O^T += V^T P^T: lane (g, q) brings tokens 2q, 2q + 1, 2q + 8, 2q + 9 of 16 dimensions
#pragma unroll
      for (int sub = 0; sub < T::kSubs; ++sub) {
        const uint32_t vr = vb + (sub * 16 + 2 * q) * T::kRowBytes;
#pragma unroll
        for (int half = 0; half < T::kRowBytes / 128; ++half) {
          const uint32_t off = ((half * 8 + g) ^ (2 * q)) << 4;
          uint32_t v[4][4];
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const uint4 y = ld_shared_v4(vr + ((r & 1) + (r >> 1) * 8) * T::kRowBytes + off);
            v[r][0] = y.x, v[r][1] = y.y, v[r][2] = y.z, v[r][3] = y.w;
          }
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            if (FP8) {
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                const uint32_t lo = __byte_perm(v[0][w], v[1][w], u ? 0x7362 : 0x5140);
                const uint32_t hi = __byte_perm(v[2][w], v[3][w], u ? 0x7362 : 0x5140);
                const uint32_t a0 = e4m3x2_to_f16x2(lo & 0xFFFFu), a1 = e4m3x2_to_f16x2(lo >> 16);
                const uint32_t a2 = e4m3x2_to_f16x2(hi & 0xFFFFu), a3 = e4m3x2_to_f16x2(hi >> 16);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma_16816<true>(o[nt][w * 2 + u], a0, a1, a2, a3, pf[nt][sub][0], pf[nt][sub][1]);
              }
            } else {
              const uint32_t a0 = __byte_perm(v[0][w], v[1][w], 0x5410), a1 = __byte_perm(v[0][w], v[1][w], 0x7632);
              const uint32_t a2 = __byte_perm(v[2][w], v[3][w], 0x5410), a3 = __byte_perm(v[2][w], v[3][w], 0x7632);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                mma_16816<false>(o[nt][half * 4 + w], a0, a1, a2, a3, pf[nt][sub][0], pf[nt][sub][1]);
                mma_16816<false>(o[nt][half * 4 + w], a0, a1, a2, a3, pl[nt][sub][0], pl[nt][sub][1]);
              }
            }
          }
        }
      }
      bad |= (bad_steps >> stage & 1u) != 0;
      __syncwarp();
      stage = stage + 1 == T::kStages ? 0 : stage + 1;
      issue();
    }

    // ---- the CTA's four pieces become one: finished here, or a part of a cut (sequence, head)
    const DecodeOwners owners = decode_owners(p, own, seg);
    const bool spoiled = __any_sync(~0u, bad);
    if (spoiled && lane == 0 && atomicCAS(p.status + ST_CODE, 0, static_cast<int>(FL_ERR_INVALID_ARG)) == 0)
      p.status[ST_DETAIL] = seg.b;
    // The ring always has a stage that is neither read nor on its way, the next to be filled: the warp's piece goes there.
    // o[nt][t][i]: head 2q + (i & 1), dimension 16 g + 2 t + (i >> 1) (E4M3), or for bf16 with t = 4 half + w
    // dimension 64 half + 8 g + 2 w + (i >> 1).  Chunks of 4 dimensions, permuted by q against bank conflicts.
    const int place = (warp * T::kStages + p_stage) * T::kStage;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float sum = l[nt][i];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(~0u, sum, d);
        const int h = nt * 8 + 2 * q + i;
        float* row = reinterpret_cast<float*>(smem + place) + h * kHeadDim;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int chunk4 = FP8 ? g * 4 + c : (c >> 1) * 16 + g * 2 + (c & 1);
          *reinterpret_cast<float4*>(row + ((chunk4 ^ q) << 2)) =
              make_float4(o[nt][c * 2][i], o[nt][c * 2][i + 2], o[nt][c * 2 + 1][i], o[nt][c * 2 + 1][i + 2]);
        }
        if (g == 0)
          stats[warp * NT * 8 + h] = make_float4(m[nt][i], FP8 ? mv[nt][i] - kDecLift : m[nt][i], spoiled ? NAN : sum,
                                                 __int_as_float(place));
      }
    __syncthreads();
    decode_merge<kDecWarps, NT * 8, 1>(p, smem, stats, warp, lane, seg, head0, n_heads, owners);
    __syncthreads();
    if (!owners.whole) cuts.add(seg, owners);
    left -= seg.units;
    if (left <= 0) break;
    own.seg_first += seg.n_units;
    walk.next(seg, left);
  }

  if (cuts.any()) decode_join<kDecWarps>(p, cuts, plan, [] { __syncthreads(); });
}

// Of a group of up to 16 query heads: one column tile or two.
template <bool FP8, bool WIN, class Launch>
int decode_tiles(const DecodeParams& p, Launch&& launch) {
  return p.chunk_heads <= 8 ? launch(DecodeTraits<FP8, 1>(), attention_decode_kernel<FP8, 1, WIN>)
                            : launch(DecodeTraits<FP8, 2>(), attention_decode_kernel<FP8, 2, WIN>);
}

}  // namespace fl
