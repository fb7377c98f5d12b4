// What the decode kernels (bf16 and E4M3: decode_attention_kernel.cuh; 4 bits: decode_int4_kernel.cuh) share: the work's
// split, a sequence's walk with a window, the joins of pieces, and matrix instructions.
//
// Split.  The work is cut into units of tokens of one (sequence, kv head); every sequence has at least one.  The CTAs take runs
// of units in the order (sequence, kv head, unit) that differ by one unit at most, so every CTA streams the same number of
// bytes whatever the lengths are, and a captured launch adapts to them.  A (sequence, kv head) that lies in one CTA is finished
// there; one that is cut writes (m, l, o) of each piece to the workspace, and the last CTA to arrive joins the pieces in the
// order of the CTAs (the result does not depend on which came last).
//
// Window.  A token sees the last `window` tokens and the first `sinks`.  The units that hold any of these are counted
// through (virtual tokens: the units between them are left out), so shares stay even; the edges are masked, their rows
// not loaded, and pages that hold none of them are not looked at.  16 sequences of 8192-65536 tokens, window 4096 and 64 sinks,
// bf16, 16/16 heads: 87 us, 6200 GB/s of what is seen.
#pragma once
#include "attention_common.h"

namespace fl {

constexpr int kDecMaxCtas = 640;
constexpr int kDecPartFloats = 16 * (kHeadDim + 4);  // o[16][128], then (m, m', l, 0) of up to 16 heads
constexpr long long kDecLongest = 0x7FFFFC00;  // tokens of a sequence: a warp looks up to 1000 ahead of the last one, in 32 bits
constexpr float kDecNone = -3e38f;             // a maximum over nothing: any finite logit passes it
constexpr float kDecLazy = 8.f;
constexpr float kDecLift = 7.f;                // E4M3 and 4 bits: weights are lifted by 2^7 in fp16

struct alignas(128) DecodeParams {
  CUtensorMap map_k, map_v;        // 4 bits, box > 0: the codes as rows of 64 bytes, box {64, box}
  CacheView c;
  const __nv_bfloat16* Q;
  __nv_bfloat16* O;
  long long ldq, ldo;
  int group, chunks, chunk_heads;  // query heads of a kv head, cut into `chunks` of `chunk_heads` (<= 8 NT)
  PageDivisor page_of;
  bool small;                      // batch <= 128 and no count can pass 31 bits
  int window, sinks;               // of attention_decode_window
  uint32_t eights;                 // 4 bits: 0x00080008, which the compiler is not to know (int4_even)
  int box;                         // 4 bits: rows of a tensor copy, 32, 16 or 8; 0: copies of 16 bytes
  unsigned long long timeout_ns;
  float scale_log2;
  int* status;
  unsigned* counters;              // [kDecMaxCtas], by the first CTA of a cut (sequence, kv head)
  float* parts;                    // [kDecMaxCtas][2][kDecPartFloats]
};

__device__ __forceinline__ void cp_async_16_or_zero(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(there ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_4_or_zero(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(there ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_8_or_zero(uint32_t dst, const void* src, bool there) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(there ? 8 : 0) : "memory");
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

// A run of units of one (sequence, head chunk): virtual tokens [t0, t1); those from jump_at on are `jump` further on.
struct DecodeSeg {
  int b, h, kvh, chunk, t0, t1, units;  // h: kvh * chunks + chunk
  int n_units, len;                     // of the whole sequence
  int jump_at, jump;
  bool bad;                             // its length is outside the table
};

// How segments follow one another, and which of their tokens count.
// OVER: units that the beginning of a (sequence, head) counts as in the split, 0 or 1; they hold no tokens and stand in front.
template <int UNIT, bool WIN, int OVER = 0>
struct DecodeWalk {
  static constexpr int kOver = OVER;
  const DecodeParams& p;
  const int heads_v;         // independent (kv head, chunk) pairs of a sequence
  const long long capacity;  // tokens that the table has room for, kDecLongest at most

  __device__ __forceinline__ explicit DecodeWalk(const DecodeParams& p)
      : p(p), heads_v(p.c.n_kv * p.chunks), capacity(min(static_cast<long long>(p.c.max_pages) * p.c.page_size, kDecLongest)) {}
  // Units of a sequence, and where its virtual tokens jump.
  __device__ __forceinline__ int span(int len, bool& bad, int& jump_at, int& jump) const {
    bad = len < 0 || len > capacity;
    jump_at = jump = 0;
    if (bad || len == 0) return 1;
    if (WIN && len > p.window && len - p.window > p.sinks) {
      // first unit of the window, units of the sinks
      const int from = (len - p.window) / UNIT, to = (static_cast<unsigned>(p.sinks) + UNIT - 1) / UNIT;
      if (from > to) jump_at = to * UNIT, jump = (from - to) * UNIT;
    }
    return (len - jump - 1) / UNIT + 1;
  }
  __device__ __forceinline__ int units_of(int len) const {
    bool bad;
    int at, jump;
    return span(len, bad, at, jump) + OVER;
  }
  __device__ __forceinline__ void begin(DecodeSeg& s, int tile, long long units_left) const {
    if (tile == 0 && s.h == 0) s.len = p.c.lens[s.b];
    s.n_units = span(s.len, s.bad, s.jump_at, s.jump) + OVER;
    s.units = static_cast<int>(min(static_cast<long long>(s.n_units - tile), units_left));
    const int end = s.bad ? 0 : s.len - s.jump;
    s.t0 = max(tile - OVER, 0) * UNIT;
    s.t1 = static_cast<int>(min(static_cast<long long>(end), (static_cast<long long>(tile) + s.units - OVER) * UNIT));
  }
  __device__ __forceinline__ void next(DecodeSeg& s, long long units_left) const {
    ++s.h;
    if (++s.chunk == p.chunks) {
      s.chunk = 0;
      if (++s.kvh == p.c.n_kv) {
        s.h = s.kvh = 0;
        ++s.b;
      }
    }
    begin(s, 0, units_left);
  }
  // Of the tokens of a unit that begins at or in front of virtual token t: position less virtual token.
  __device__ __forceinline__ int shift_of(const DecodeSeg& s, int t) const { return WIN && t >= s.jump_at ? s.jump : 0; }
  __device__ __forceinline__ bool in_sight(const DecodeSeg& s, int pos) const {
    return !WIN || pos < p.sinks || pos >= s.len - p.window;
  }
  __device__ __forceinline__ int page_of(int pos) const { return p.page_of(pos); }
};

// Only hints go out before the kernel in front has finished: they bring the address translations (plan done after
// 1900 instead of 2400 cycles).  Planning on lengths that may be old and fetching the first keys with it was slower.
__device__ __forceinline__ void decode_hints(const DecodeParams& p, int tid) {
  if (tid < p.c.batch) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p.c.lens + tid));
    if (p.c.max_pages > 0) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.c.table + tid * p.c.ldt));
  }
}

// This CTA's run of units.  CTA i of G starts at unit i * share + min(i, more).
struct DecodeShare {
  long long share, more, u0, u1;
  long long seg_first;  // first unit of the current (sequence, head) in the whole order
  __device__ __forceinline__ int cta_of(long long u) const {  // the CTA that has unit u
    const long long longer = more * (share + 1);
    return static_cast<int>(u < longer ? u / (share + 1) : more + (u - longer) / share);
  }
};

// The plan: false if there is nothing for this CTA.  All threads call it; plan: 10 words of shared memory.
template <int THREADS, class Walk>
__device__ __forceinline__ bool decode_plan(const DecodeParams& p, const Walk& walk, long long* plan, DecodeShare& own,
                                            DecodeSeg& seg) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x, heads_v = walk.heads_v;
  int G, tile;  // tile: the CTA's first unit, inside its (sequence, head)
  if (p.small) {  // at most 128 sequences, all counts in 32 bits: each warp finds its way alone, without a barrier
    int len[4], mine[4], last[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) len[k] = k * 32 + lane < p.c.batch ? p.c.lens[k * 32 + lane] : 0;
#pragma unroll
    for (int k = 0; k < 4; ++k)
      last[k] = mine[k] = k * 32 + lane < p.c.batch ? walk.units_of(len[k]) : 0;
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
    if (cta >= G) return false;
    const unsigned each = all / G, rest = all - each * G, first = each * cta + min(static_cast<unsigned>(cta), rest);
    const int at = static_cast<int>(first / heads_v);
    own.share = each, own.more = rest, own.u0 = first;
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
    long long before, total = 0;
    auto block_scan = [&](int b0) -> long long {  // of THREADS sequences from b0
      const int b = b0 + tid;
      mine = b < p.c.batch ? walk.units_of(p.c.lens[b]) : 0;
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
      for (int w = 0; w < THREADS / 32; ++w) {
        if (w < warp) before += plan[w];
        sum += plan[w];
      }
      return sum;
    };
    for (int b0 = 0; b0 < p.c.batch; b0 += THREADS) total += block_scan(b0);
    total *= heads_v;
    G = static_cast<int>(min(static_cast<long long>(gridDim.x), total));
    if (cta >= G) return false;
    own.share = total / G, own.more = total - own.share * G;
    own.u0 = own.share * cta + min(static_cast<long long>(cta), own.more);
    const long long u0 = own.u0;
    long long base = 0;
    for (int b0 = 0;; b0 += THREADS) {
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
    const int n = walk.units_of(seg.len);
    seg.h = static_cast<int>(plan[9] / n);
    tile = static_cast<int>(plan[9] - static_cast<long long>(seg.h) * n);
  }
  own.u1 = own.u0 + own.share + (cta < own.more ? 1 : 0);
  own.seg_first = own.u0 - tile;
  seg.kvh = seg.h / p.chunks;
  seg.chunk = seg.h - seg.kvh * p.chunks;
  walk.begin(seg, tile, own.u1 - own.u0);
  return tile >= Walk::kOver || own.u1 - own.u0 > Walk::kOver;  // more than a beginning
}

// The CTAs that share a (sequence, head).
struct DecodeOwners {
  bool whole;
  int first, last;
  float* part;  // where this CTA's piece goes if not whole
};
template <int OVER = 0>
__device__ __forceinline__ DecodeOwners decode_owners(const DecodeParams& p, const DecodeShare& own, const DecodeSeg& seg) {
  const int cta = blockIdx.x;
  const long long first = own.seg_first + OVER;  // unit with tokens
  DecodeOwners w;
  w.whole = first >= own.u0 && own.seg_first + seg.n_units <= own.u1;
  w.first = w.last = cta;
  if (!w.whole) {
    if (first < own.u0) w.first = own.cta_of(first);
    if (own.seg_first + seg.n_units > own.u1) w.last = own.cta_of(own.seg_first + seg.n_units - 1);
  }
  w.part = p.parts + (static_cast<long long>(cta) * 2 + (cta == w.first ? 1 : 0)) * kDecPartFloats;
  return w;
}

// acc 2^(mv - m) / l as bf16.  mv - m is the power of V's scales, down to 2^-149: below 2^-100 it comes as two factors, for one
// below 2^-126 would be flushed to zero, and the quotient lose bits before that.
__device__ __forceinline__ uint2 decode_output(const float4& acc, float m, float mv, float l) {
  const float e = mv - m, r = ex2(fmaxf(e, -100.f)) / l, rest = ex2(fminf(e + 100.f, 0.f));
  return make_uint2(pack_bf16x2(acc.x * r * rest, acc.y * r * rest), pack_bf16x2(acc.z * r * rest, acc.w * r * rest));
}

// The pieces of a CTA's warps become one: finished, or a part of a cut (sequence, head).  stats [warp][head]: m, m', l and where
// in shared memory the warp's piece is: o[head][128], chunks of 4 permuted by SWIZZLE times the head's pair.
template <int WARPS, int HEADS, int SWIZZLE>
__device__ __forceinline__ void decode_merge(const DecodeParams& p, const uint8_t* smem, const float4* stats, int warp, int lane,
                                             const DecodeSeg& seg, int head0, int n_heads, const DecodeOwners& w) {
  for (int h = warp; h < n_heads; h += WARPS) {  // a warp joins whole heads, a lane 4 dimensions
    float4 st[WARPS], acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float M = kDecNone, MV = kDecNone, L = 0.f;
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
      st[i] = stats[i * HEADS + h];
      M = fmaxf(M, st[i].x);
      MV = fmaxf(MV, st[i].y);
    }
    const int at = h * kHeadDim + ((lane ^ ((h >> 1 & 3) * SWIZZLE)) << 2);
#pragma unroll
    for (int i = 0; i < WARPS; ++i) {
      const float4 v = *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(smem + __float_as_int(st[i].w)) + at);
      const float f = ex2(st[i].y - MV);
      L += st[i].z * ex2(st[i].x - M);
      acc.x += v.x * f, acc.y += v.y * f, acc.z += v.z * f, acc.w += v.w * f;
    }
    if (w.whole) {
      uint2 out = decode_output(acc, M, MV, L);
      if (seg.len == 0) out = make_uint2(0, 0);
      *reinterpret_cast<uint2*>(p.O + seg.b * p.ldo + static_cast<long long>(head0 + h) * kHeadDim + lane * 4) = out;
    } else {
      __stcg(reinterpret_cast<float4*>(w.part + h * kHeadDim) + lane, acc);
      if (lane == 0) __stcg(reinterpret_cast<float4*>(w.part + 16 * kHeadDim) + h, make_float4(M, MV, L, 0.f));
    }
  }
}

// A CTA's cut segments, two at most: its first and its last.
struct DecodeCuts {
  int b[2] = {0, 0}, h[2] = {0, 0}, first[2] = {-1, -1}, last[2] = {-1, -1};
  __device__ __forceinline__ void add(const DecodeSeg& s, const DecodeOwners& w) {
    if (static_cast<int>(blockIdx.x) == w.first) b[1] = s.b, h[1] = s.h, first[1] = w.first, last[1] = w.last;
    else b[0] = s.b, h[0] = s.h, first[0] = w.first, last[0] = w.last;
  }
  __device__ __forceinline__ bool any() const { return first[0] >= 0 || first[1] >= 0; }
};

// Pieces of cut (sequence, head) pairs: the CTA that arrives last joins them.  sync: a barrier of the WARPS warps that call.
template <int WARPS, class Sync>
__device__ __forceinline__ void decode_join(const DecodeParams& p, const DecodeCuts& cuts, long long* plan, Sync&& sync) {
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  sync();
  if (tid < 2) {  // release: for the whole CTA, the others' stores are behind the barrier; acquire: those of the others that came
    plan[tid] = 0;
    const int first = tid == 0 ? cuts.first[0] : cuts.first[1], last = tid == 0 ? cuts.last[0] : cuts.last[1];
    unsigned came = 0;
    if (first >= 0)
      asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(came) : "l"(p.counters + first) : "memory");
    if (first >= 0 && came == static_cast<unsigned>(last - first)) {
      p.counters[first] = 0;
      plan[tid] = 1;
    }
  }
  sync();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    if (plan[k] == 0) continue;
    const int c_first = cuts.first[k], c_last = cuts.last[k];
    const int kvh = cuts.h[k] / p.chunks, chunk = cuts.h[k] - kvh * p.chunks;
    const int head0 = kvh * p.group + chunk * p.chunk_heads;
    const int n_heads = min(p.chunk_heads, p.group - chunk * p.chunk_heads);
    auto src = [&](int c) { return p.parts + (static_cast<long long>(c) * 2 + (c == c_first)) * kDecPartFloats; };
    for (int h = warp; h < n_heads; h += WARPS) {  // lane i weighs piece i, then holds 4 dimensions
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
      uint2 out = decode_output(acc, M, MV, L);
      *reinterpret_cast<uint2*>(p.O + cuts.b[k] * p.ldo + static_cast<long long>(head0 + h) * kHeadDim + lane * 4) = out;
    }
  }
}

}  // namespace fl
