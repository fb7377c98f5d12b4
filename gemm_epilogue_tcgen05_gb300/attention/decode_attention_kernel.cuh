// Attention of one new token per sequence over a paged key-value cache.
//
//   o_h = sum_j p_j v_j / sum_j p_j,  p_j = 2^(x_j - m),  x_j = scale * log2(e) * q_h . k_j
//
// What bounds it: the cache is read once, 4 * 128 * group multiply-adds for every 256 (E4M3) or 512 (bf16)
// bytes, so it runs at the memory's rate as long as enough loads are in flight and nothing else keeps a warp
// from issuing the next ones.
//
// Split.  The work is cut into units of 64 (bf16) or 128 (E4M3) tokens of one (sequence, kv head); every sequence has at least one.
// The CTAs take runs of units in the order (sequence, kv head, unit) that differ by one unit at most, so every CTA
// streams the same number of bytes whatever the lengths are, and a captured launch adapts to them.  A (sequence, kv
// head) that lies in one CTA is finished there; one that is cut writes (m, l, o) of each piece to the workspace,
// and the last CTA to arrive joins the pieces in the order of the CTAs (the result does not depend on which
// came last).
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
#include "attention_common.h"

namespace fl {

constexpr int kDecWarps = 4;
constexpr int kDecThreads = 32 * kDecWarps;
constexpr int kDecMaxCtas = 640;
constexpr int kDecPartFloats = 16 * (kHeadDim + 4);  // o[16][128], then (m, m', l, 0) of up to 16 heads
constexpr float kDecNone = -3e38f;             // a maximum over nothing: any finite logit passes it
constexpr float kDecLazy = 8.f;
constexpr float kDecLift = 7.f;                // E4M3: weights are lifted by 2^7 in fp16

struct DecodeParams {
  CacheView c;
  const __nv_bfloat16* Q;
  __nv_bfloat16* O;
  long long ldq, ldo;
  int group, chunks, chunk_heads;  // query heads of a kv head, cut into `chunks` of `chunk_heads` (<= 8 NT)
  int page_shift;                  // log2(page_size), -1 if it is no power of two
  bool small;                      // batch <= 128 and no count can pass 31 bits
  float scale_log2;
  int* status;
  unsigned* counters;              // [kDecMaxCtas], by the first CTA of a cut (sequence, kv head)
  float* parts;                    // [kDecMaxCtas][2][kDecPartFloats]
};

template <bool FP8, int NT>
struct DecodeTraits {
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
__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_4_or_zero(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
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
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
template <bool F16>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  if (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// A run of units of one (sequence, head chunk): tokens [t0, t1).
struct DecodeSeg {
  int b, h, t0, t1, units;
  int n_units, len;  // of the whole sequence
  bool bad;          // its length is outside the table
};

template <int UNIT>
__device__ __forceinline__ int decode_units(int len, long long capacity, bool& bad) {
  bad = len < 0 || len > capacity;
  return bad || len == 0 ? 1 : (len - 1) / UNIT + 1;
}

template <bool FP8, int NT>
__global__ void __launch_bounds__(kDecThreads, DecodeTraits<FP8, NT>::kCtas) attention_decode_kernel(const __grid_constant__ DecodeParams p) {
  using T = DecodeTraits<FP8, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  float4* stats = reinterpret_cast<float4*>(smem + kDecWarps * T::kStages * T::kStage);  // [warp][head]: m, m', l, stage
  long long* plan = reinterpret_cast<long long*>(stats + kDecWarps * NT * 8);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  const int heads_v = p.c.n_kv * p.chunks;  // independent (kv head, chunk) pairs of a sequence
  const long long capacity = static_cast<long long>(p.c.max_pages) * p.c.page_size;
  const int cta = blockIdx.x;

  // Only hints go out before the kernel in front has finished: they bring the address translations (plan done after
  // 1900 instead of 2400 cycles).  Planning on lengths that may be old and fetching the first keys with it was slower.
  if (tid < p.c.batch) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p.c.lens + tid));
    if (p.c.max_pages > 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.c.table + tid * p.c.ldt));
  }
  griddep_wait();  // launched as a dependent: nothing is read before the kernel in front has finished
  griddep_launch_dependents();

  // ---- plan: total units, and where this CTA's first unit lies.  CTA i of G starts at unit i * share + min(i, more).
  long long total = 0, share, more, u0, seg_first;  // seg_first: first unit of this (sequence, head) in the whole order
  int G, tile;                                      // tile: the CTA's first unit, inside its (sequence, head)
  DecodeSeg seg;
  bool odd;
  if (p.small) {  // at most 128 sequences, all counts in 32 bits: each warp finds its way alone, without a barrier
    int len[4], mine[4], last[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) len[k] = k * 32 + lane < p.c.batch ? p.c.lens[k * 32 + lane] : 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      last[k] = mine[k] = k * 32 + lane < p.c.batch ? decode_units<T::kUnit>(len[k], capacity, odd) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int y = __shfl_up_sync(~0u, last[k], o);
        if (lane >= o) last[k] += y;
      }
    int sum[5] = {0};
#pragma unroll
    for (int k = 0; k < 4; ++k) sum[k + 1] = sum[k] + __shfl_sync(~0u, last[k], 31);
    const unsigned all = static_cast<unsigned>(sum[4]) * heads_v;
    G = static_cast<int>(min(gridDim.x, all));  // each has a unit at least
    if (cta >= G) return;
    const unsigned each = all / G, rest = all - each * G, first = each * cta + min(static_cast<unsigned>(cta), rest);
    const int at = static_cast<int>(first / heads_v);
    total = all, share = each, more = rest, u0 = first;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (at < sum[k] || at >= sum[k + 1]) continue;  // the same for all lanes
      const int who = __ffs(__ballot_sync(~0u, at < sum[k] + last[k])) - 1;
      const int n = __shfl_sync(~0u, mine[k], who), before = sum[k] + __shfl_sync(~0u, last[k], who) - n;
      const int in = static_cast<int>(first - static_cast<unsigned>(before) * heads_v);
      seg.b = k * 32 + who;
      seg.len = __shfl_sync(~0u, len[k], who);
      seg.h = in / n;
      tile = in - seg.h * n;
    }
  } else {
    int mine;
    long long before;
    auto block_scan = [&](int b0) -> long long {  // of 128 sequences from b0
      const int b = b0 + tid;
      mine = b < p.c.batch ? decode_units<T::kUnit>(p.c.lens[b], capacity, odd) : 0;
      long long x = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(~0u, x, o);
        if (lane >= o) x += y;
      }
      __syncthreads();
      if (lane == 31) plan[warp] = x;
      __syncthreads();
      long long sum = 0;
      before = x - mine;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        if (w < warp) before += plan[w];
        sum += plan[w];
      }
      return sum;
    };
    for (int b0 = 0; b0 < p.c.batch; b0 += kDecThreads) total += block_scan(b0);
    total *= heads_v;
    G = static_cast<int>(min(static_cast<long long>(gridDim.x), total));
    if (cta >= G) return;
    share = total / G, more = total - share * G;
    u0 = share * cta + min(static_cast<long long>(cta), more);
    long long base = 0;
    for (int b0 = 0;; b0 += kDecThreads) {
      const long long sum = block_scan(b0), lo = (base + before) * heads_v;
      if (mine > 0 && u0 >= lo && u0 < lo + static_cast<long long>(mine) * heads_v) {
        plan[8] = b0 + tid;
        plan[9] = u0 - lo;
      }
      base += sum;
      if (base * heads_v > u0) break;
    }
    __syncthreads();
    seg.b = static_cast<int>(plan[8]);
    seg.len = p.c.lens[seg.b];
    const int n = decode_units<T::kUnit>(seg.len, capacity, odd);
    seg.h = static_cast<int>(plan[9] / n);
    tile = static_cast<int>(plan[9] - static_cast<long long>(seg.h) * n);
  }
  const long long u1 = u0 + share + (cta < more ? 1 : 0);
  seg_first = u0 - tile;
  auto cta_of = [&](long long u) {  // the CTA that has unit u
    const long long longer = more * (share + 1);
    return static_cast<int>(u < longer ? u / (share + 1) : more + (u - longer) / share);
  };
  long long left = u1 - u0;
  auto begin_seg = [&](DecodeSeg& s, int tile, long long units_left) {
    if (tile == 0 && s.h == 0) s.len = p.c.lens[s.b];
    s.n_units = decode_units<T::kUnit>(s.len, capacity, s.bad);
    s.units = static_cast<int>(min(static_cast<long long>(s.n_units - tile), units_left));
    const int end = s.bad ? 0 : s.len;
    s.t0 = tile * T::kUnit;
    s.t1 = static_cast<int>(min(static_cast<long long>(end), (static_cast<long long>(tile) + s.units) * T::kUnit));
  };
  auto next_seg = [&](DecodeSeg& s, long long units_left) {
    if (++s.h == heads_v) {
      s.h = 0;
      ++s.b;
    }
    begin_seg(s, 0, units_left);
  };
  begin_seg(seg, tile, left);

  // ---- producer side of this warp's ring
  DecodeSeg ps = seg;
  long long p_left = left;
  int pt = ps.t0 + warp * T::kStep, entry = 0, p_stage = 0;
  uint32_t bad_steps = 0;  // stages whose page-table entry is outside the cache
  bool fresh = true;
  const bool one_page = (p.c.page_size & (T::kStep - 1)) == 0;  // a step's 16 tokens lie in one page
  auto page_of = [&](int pos) { return p.page_shift >= 0 ? pos >> p.page_shift : pos / p.c.page_size; };
  auto settle = [&]() {  // moves on to this warp's next step and fetches its page-table entry
    while (pt >= ps.t1) {
      p_left -= ps.units;
      if (p_left <= 0) return;
      next_seg(ps, p_left);
      pt = ps.t0 + warp * T::kStep;
      fresh = true;
    }
    if (fresh) {  // the query rows of the segment that begins, into L2
      fresh = false;
      const char* row = reinterpret_cast<const char*>(p.Q + ps.b * p.ldq + static_cast<long long>(ps.h / p.chunks) * p.group * kHeadDim);
      if (lane < 2 * p.group) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + lane * 128));
    }
    const int pos = one_page ? pt : min(pt + (lane & (T::kStep - 1)), ps.t1 - 1);
    entry = p.c.table[ps.b * p.c.ldt + page_of(pos)];
  };
  const uint32_t ring = smem_u32(smem) + warp * T::kStages * T::kStage;
  auto issue = [&]() {
    if (p_left > 0) {
      constexpr int kChunks = T::kRowBytes / 16, kRowsPer = 32 / kChunks;
      const uint32_t dst = ring + p_stage * T::kStage;
      const int kvh = ps.h / p.chunks, rows = ps.t1 - pt;
      const bool ok = static_cast<unsigned>(entry) < static_cast<unsigned>(p.c.num_pages);
      bad_steps = (bad_steps & ~(1u << p_stage)) | (ok ? 0u : 1u << p_stage);
      const int mypos = one_page ? pt : min(pt + (lane & (T::kStep - 1)), ps.t1 - 1);
      const int slot = mypos - page_of(mypos) * p.c.page_size, mypage = ok ? entry : 0;
      const int c = lane % kChunks, row0 = lane / kChunks;
      const long long cell = static_cast<long long>(kvh) * p.c.page_size + slot;
      if (one_page) {
        const long long byte = (mypage * p.c.page_pitch + (cell + row0) * kHeadDim) * (FP8 ? 1 : 2) + c * 16;
        const uint8_t* ksrc = static_cast<const uint8_t*>(p.c.k) + byte;
        const uint8_t* vsrc = static_cast<const uint8_t*>(p.c.v) + byte;
#pragma unroll
        for (int i = 0; i < T::kStep / kRowsPer; ++i) {
          const int row = row0 + i * kRowsPer;
          const bool there = ok && row < rows;
          cp_async_16_or_zero(dst + row * T::kRowBytes + ((c ^ ((row & 1) << 2)) << 4), ksrc + i * 512, there);
          cp_async_16_or_zero(dst + T::kTile + row * T::kRowBytes + ((c ^ (row & 6)) << 4), vsrc + i * 512, there);
        }
      } else {
#pragma unroll
        for (int i = 0; i < T::kStep / kRowsPer; ++i) {
          const int row = row0 + i * kRowsPer;
          const int page = __shfl_sync(~0u, ok ? entry : -1, row), s = __shfl_sync(~0u, slot, row);
          const bool there = page >= 0 && row < rows;
          const long long at = max(page, 0) * p.c.page_pitch + (static_cast<long long>(kvh) * p.c.page_size + s) * kHeadDim;
          const long long byte = at * (FP8 ? 1 : 2) + c * 16;
          cp_async_16_or_zero(dst + row * T::kRowBytes + ((c ^ ((row & 1) << 2)) << 4),
                              static_cast<const uint8_t*>(p.c.k) + byte, there);
          cp_async_16_or_zero(dst + T::kTile + row * T::kRowBytes + ((c ^ (row & 6)) << 4),
                              static_cast<const uint8_t*>(p.c.v) + byte, there);
        }
      }
      if (FP8) {  // lane = row of the step
        const bool there = ok && lane < rows;
        const long long at = mypage * p.c.scale_pitch + cell + (one_page ? lane : 0);
        cp_async_4_or_zero(dst + 2 * T::kTile + lane * 4, p.c.ks + at, there);
        cp_async_4_or_zero(dst + 2 * T::kTile + 128 + lane * 4, p.c.vs + at, there);
      }
      pt += T::kUnit;
      settle();
    }
    cp_async_commit();
    p_stage = p_stage + 1 == T::kStages ? 0 : p_stage + 1;
  };
  int cut_b[2] = {0, 0}, cut_h[2] = {0, 0}, cut_first[2] = {-1, -1}, cut_last[2] = {-1, -1};
  settle();
#pragma unroll
  for (int i = 0; i < T::kStages - 1; ++i) issue();
  int stage = 0;

  for (;;) {
    // ---- this segment's query fragments (B operand: head g of the column tile, dimensions in the cache's order)
    const int kvh = seg.h / p.chunks, chunk = seg.h - kvh * p.chunks;
    const int head0 = kvh * p.group + chunk * p.chunk_heads;
    const int n_heads = min(p.chunk_heads, p.group - chunk * p.chunk_heads);
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
      // ---- softmax: lane (g, q) holds tokens g, g + 8 of each tile for heads 2q, 2q + 1
      float ks[T::kSubs * 2], lv[T::kSubs * 2];
#pragma unroll
      for (int r = 0; r < T::kSubs * 2; ++r) {
        ks[r] = 1.f, lv[r] = 0.f;
        if (FP8) {
          const float* sc = reinterpret_cast<const float*>(smem + (kb - smem_u32(smem)) + 2 * T::kTile);
          ks[r] = sc[g + r * 8];
          lv[r] = lg2(sc[T::kStep + g + r * 8]);
        }
      }
      float x[NT][T::kSubs * 4];  // [tile][token half][head]
      bool rise = false;
      const bool cut = t + T::kStep > seg.t1;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < T::kSubs * 4; ++i) {
          float v = (s[nt][i >> 2][0][i & 3] + s[nt][i >> 2][1][i & 3]) * fac[nt][i & 1];
          if (FP8) v *= ks[i >> 1];
          if (cut && t + g + (i >> 1) * 8 >= seg.t1) v = -INFINITY;
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
    const bool whole = seg_first >= u0 && seg_first + seg.n_units <= u1;
    int c_first = cta, c_last = cta;  // the CTAs that share it
    if (!whole) {
      if (seg_first < u0) c_first = cta_of(seg_first);
      if (seg_first + seg.n_units > u1) c_last = cta_of(seg_first + seg.n_units - 1);
    }
    float* part = p.parts + (static_cast<long long>(cta) * 2 + (cta == c_first ? 1 : 0)) * kDecPartFloats;
    const bool spoiled = __any_sync(~0u, bad);
    if (spoiled && lane == 0 && atomicCAS(p.status + ST_CODE, 0, static_cast<int>(FL_ERR_INVALID_ARG)) == 0)
      p.status[ST_DETAIL] = seg.b;
    // The ring always has a stage that is neither read nor on its way, the next to be filled: the warp's piece goes there.
    // o[nt][t][i]: head 2q + (i & 1), dimension 16 g + 2 t + (i >> 1) (E4M3), or for bf16 with t = 4 half + w
    // dimension 64 half + 8 g + 2 w + (i >> 1).  Chunks of 4 dimensions, permuted by q against bank conflicts.
    const int own = (warp * T::kStages + p_stage) * T::kStage;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float sum = l[nt][i];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(~0u, sum, d);
        const int h = nt * 8 + 2 * q + i;
        float* row = reinterpret_cast<float*>(smem + own) + h * kHeadDim;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int chunk4 = FP8 ? g * 4 + c : (c >> 1) * 16 + g * 2 + (c & 1);
          *reinterpret_cast<float4*>(row + ((chunk4 ^ q) << 2)) =
              make_float4(o[nt][c * 2][i], o[nt][c * 2][i + 2], o[nt][c * 2 + 1][i], o[nt][c * 2 + 1][i + 2]);
        }
        if (g == 0)
          stats[warp * NT * 8 + h] = make_float4(m[nt][i], FP8 ? mv[nt][i] - kDecLift : m[nt][i], spoiled ? NAN : sum,
                                                 __int_as_float(own));
      }
    __syncthreads();
    for (int h = warp; h < n_heads; h += kDecWarps) {  // a warp joins whole heads, a lane 4 dimensions
      float4 st[kDecWarps], acc = make_float4(0.f, 0.f, 0.f, 0.f);
      float M = kDecNone, MV = kDecNone, L = 0.f;
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        st[w] = stats[w * NT * 8 + h];
        M = fmaxf(M, st[w].x);
        MV = fmaxf(MV, st[w].y);
      }
      const int at = h * kHeadDim + ((lane ^ ((h >> 1) & 3)) << 2);
#pragma unroll
      for (int w = 0; w < kDecWarps; ++w) {
        const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + __float_as_int(st[w].w)) + at);
        const float f = ex2(st[w].y - MV);
        L += st[w].z * ex2(st[w].x - M);
        acc.x += v.x * f, acc.y += v.y * f, acc.z += v.z * f, acc.w += v.w * f;
      }
      if (whole) {
        const float r = ex2(MV - M) / L;
        uint2 out;
        out.x = pack_bf16x2(acc.x * r, acc.y * r);
        out.y = pack_bf16x2(acc.z * r, acc.w * r);
        if (seg.len == 0) out = make_uint2(0, 0);
        *reinterpret_cast<uint2*>(p.O + seg.b * p.ldo + static_cast<long long>(head0 + h) * kHeadDim + lane * 4) = out;
      } else {
        __stcg(reinterpret_cast<float4*>(part + h * kHeadDim) + lane, acc);
        if (lane == 0) __stcg(reinterpret_cast<float4*>(part + 16 * kHeadDim) + h, make_float4(M, MV, L, 0.f));
      }
    }
    __syncthreads();
    if (!whole) {  // at most two of a CTA's segments are cut: its first and its last
      if (cta == c_first) cut_b[1] = seg.b, cut_h[1] = seg.h, cut_first[1] = c_first, cut_last[1] = c_last;
      else cut_b[0] = seg.b, cut_h[0] = seg.h, cut_first[0] = c_first, cut_last[0] = c_last;
    }
    left -= seg.units;
    if (left <= 0) break;
    seg_first += seg.n_units;
    next_seg(seg, left);
  }

  // ---- pieces of cut (sequence, head) pairs: the CTA that arrives last joins them
  if (cut_first[0] < 0 && cut_first[1] < 0) return;
  __syncthreads();
  if (tid < 2) {
    __threadfence();  // for the whole CTA: the others' stores are behind the barrier
    plan[tid] = 0;
    const int first = tid == 0 ? cut_first[0] : cut_first[1], last = tid == 0 ? cut_last[0] : cut_last[1];
    if (first >= 0 && atomicAdd(p.counters + first, 1u) == static_cast<unsigned>(last - first)) {
      p.counters[first] = 0;
      plan[tid] = 1;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (plan[k] == 0) continue;
    __threadfence();
    const int c_first = cut_first[k], c_last = cut_last[k];
    const int kvh = cut_h[k] / p.chunks, chunk = cut_h[k] - kvh * p.chunks;
    const int head0 = kvh * p.group + chunk * p.chunk_heads;
    const int n_heads = min(p.chunk_heads, p.group - chunk * p.chunk_heads);
    auto src = [&](int c) { return p.parts + (static_cast<long long>(c) * 2 + (c == c_first)) * kDecPartFloats; };
    for (int h = warp; h < n_heads; h += kDecWarps) {  // lane i weighs piece i, then holds 4 dimensions
      float M = kDecNone, MV = kDecNone, L = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int c0 = c_first; c0 <= c_last; c0 += 32) {
        const int n = min(32, c_last - c0 + 1);
        float4 st = make_float4(kDecNone, kDecNone, 0.f, 0.f);
        if (lane < n) st = __ldcg(reinterpret_cast<const float4*>(src(c0 + lane) + 16 * kHeadDim) + h);
        float4 v[8];
        auto fetch = [&](int i0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            v[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i0 + i < n) v[i] = __ldcg(reinterpret_cast<const float4*>(src(c0 + i0 + i) + h * kHeadDim) + lane);
          }
        };
        fetch(0);  // before their weights are known
        float nm = fmaxf(M, st.x), nmv = fmaxf(MV, st.y);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) {
          nm = fmaxf(nm, __shfl_xor_sync(~0u, nm, d));
          nmv = fmaxf(nmv, __shfl_xor_sync(~0u, nmv, d));
        }
        float sum = st.z * ex2(st.x - nm);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(~0u, sum, d);
        L = L * ex2(M - nm) + sum;
        const float w = lane < n ? ex2(st.y - nmv) : 0.f, old = ex2(MV - nmv);
        acc.x *= old, acc.y *= old, acc.z *= old, acc.w *= old;
        M = nm;
        MV = nmv;
        for (int i0 = 0; i0 < n; i0 += 8) {
          if (i0 > 0) fetch(i0);
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float wi = __shfl_sync(~0u, w, i0 + i);
            acc.x += v[i].x * wi, acc.y += v[i].y * wi, acc.z += v[i].z * wi, acc.w += v[i].w * wi;
          }
        }
      }
      const float r = ex2(MV - M) / L;
      uint2 out;
      out.x = pack_bf16x2(acc.x * r, acc.y * r);
      out.y = pack_bf16x2(acc.z * r, acc.w * r);
      *reinterpret_cast<uint2*>(p.O + cut_b[k] * p.ldo + static_cast<long long>(head0 + h) * kHeadDim + lane * 4) = out;
    }
  }
}

}  // namespace fl
