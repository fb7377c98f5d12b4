// Attention of one new token per sequence over a paged key-value cache of 4 bits.
//
//   o_h = sum_j p_j v_j / sum_j p_j,  p_j = 2^(x_j - m),  x_j = scale * log2(e) * q_h . k_j
//
// What bounds it: the cache is read once, 144 bytes for a token and kv head, at the memory's rate if the instructions for
// these 256 codes are few enough: a logic instruction takes two cycles of a scheduler, and an SM has some 25 cycles of each
// of its four for a token and head.  64 sequences of 2048-8192 tokens, 32/8 heads: 81 us, 4440 GB/s; some 350 instructions for
// 16 tokens and a head, 0.53 of them in a cycle of a scheduler.
//
// Codes.  A code xor 8, u = code + 8, is an fp16 number u 2^-24 (a denormal one) as it stands in the low bits of a half, and
// 16 u 2^-24 four bits further up: one logic instruction gives two, and the factor 16 lies in the query's fragments for K, in
// the output's odd dimensions for V.
//   q . k = sum_g s_g (sum_d q_d u_d - 8 sum_d q_d): products of 32 columns with a scale of their own.
//   o_d = sum_j w_j u_jd - 8 sum_j w_j: weights with the scale of the value's group in them, w_j = p_j s_jg, and eight times
//   their sum by one more product for each group, of eights: in its even rows as the even dimensions' codes stand, in its odd ones
//   as the odd dimensions'.  A product of denormal numbers is aligned by the exponent of their format, so sums of these codes keep
//   2^-14 (even) and 2^-18 (odd) of the largest weight, not fp32's 2^-24, and much of what they drop leaves with eights that are
//   aligned alike (one sum of eights for both: 2^-12.6 of the weights' sum where the heavy tokens' codes are zero, now 2^-13.8;
//   1 % of the time).  The eights are taken off every 32 tokens: the tensor cores truncate a running sum, and the sum of u, 8 or so
//   times the weights', would lose more with every product than the eights, rounded to nearest, take off (400000 tokens with
//   like weights in one CTA: an error of 2.3 % of the output, now 0.16 %, its rounding).
// A query head is scaled by a power of two to fp16's upper range, where its bf16 values are exact down to 2^-25 of the largest.
// p_j is 2^(x_j + e_j - m'), 2^e_j next above the token's largest scale and m' the running maximum of that exponent; it is
// rounded to fp16, and its product with s_jg 2^-e_j (at most 1) again.  Where the four scales of a token lie 2^12 and more
// apart, fp16 would lose the small ones' columns: from there on the warp takes a slower step, with p_j s_jg split into two bf16
// numbers (the codes' bits are u 2^-133 there, so both kinds of steps add to the same sums).
//
// Both products run on the tensor cores with the tokens on the M side, S^T = K Q^T and O^T = V^T P^T (m16n8k16: 8 query heads of
// a group in the N columns; of larger groups each 8 read the cache).  V^T comes by ldmatrix: a group's 16 bytes are 8 columns of
// 16 bits, 4 codes each.  The maxima m and m' rise only when a logit passes them by more than 8.
//
// Work.  Units (decode_attention_common.cuh) are 128 tokens, a stage of the CTA's ring; each of four warps takes 32 of them.  A
// fifth warp walks ahead and fills the stages by tensor copies, one for each 32, 16 or 8 tokens of a page and tensor (codes with
// the 64-byte swizzle, so that eight rows of a chunk meet in no bank), and bulk copies for the scales; caches that these
// do not fit are copied by 16 bytes.  With a ring of its own for each warp, filled by itself, finding the pages and issuing the
// copies took 112 of 400 instructions for 16 tokens and a head: 105.7 us for these 64 sequences, 91 with the fifth warp.  In the
// split the beginning of a (sequence, head) counts as a unit: its queries and the join of its pieces take as long (24 sequences
// with a window of 1024: 16.4 us without).
#pragma once
#include "decode_attention_common.cuh"

namespace fl {

// What the warps that compute only look at between segments; in registers it cost spills (90 us for 80).
struct DecodeKept {
  DecodeShare own;
  DecodeSeg seg;
  long long left;  // units
  DecodeCuts cuts;
};

struct DecodeInt4Traits {
  static constexpr int kWarps = 4;  // that compute
  static constexpr int kThreads = 32 * (kWarps + 1);
  static constexpr int kRowBytes = kHeadDim / 2, kScaleBytes = 2 * kInt4Groups;  // of a row
  static constexpr int kSubs = 2, kStep = 16 * kSubs, kUnit = kWarps * kStep;
  static constexpr int kTile = kUnit * kRowBytes, kScales = kUnit * kScaleBytes;
  static constexpr int kStage = 2 * (kTile + kScales);  // K, V, K's scales, V's
  static_assert(kStage % 512 == 0, "the swizzle's pattern");
  static_assert(kWarps == kInt4Groups, "a warp prepares a group of the queries");
  // A warp's tables: parts of V's scales as fp16, [group][q][pairs of tokens 2 q + 8 j]; K's scales and the power of V's, each
  // twice, [group or power][g][tokens g + 8 r].  Its piece of a segment's result comes to the same place.
  static constexpr int kParts = kInt4Groups * kStep * 2, kPairs = kStep * 8, kTables = kParts + (kInt4Groups + 1) * kPairs;
  static constexpr int kPiece = 8 * kHeadDim * 4, kOwn = kPiece > kTables ? kPiece : kTables;
  // The segment's queries, for all warps: fragments of each group, [group][lane], -8 sum q, [group][head], and the
  // logits' factor in two parts, [q][part][head 2 q, 2 q + 1].
  static constexpr int kQuery = kInt4Groups * (32 * 16 + 8 * 4) + 4 * 16;
  static constexpr int kOver = 1;  // units that the beginning of a (sequence, head) counts as
  static constexpr int kCtas = 3, kStages = 3;
  static constexpr int kSmem = 512 /*alignment*/ + kStages * kStage + kWarps * (kOwn + 8 * 16) + kQuery + 128 + 2 * kStages * 8 +
                               16 + sizeof(DecodeKept);
};

template <bool TRANS>
__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
  if (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t u16x2_max(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t u16x2_min(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("min.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t u16x2_add(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("add.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// A bounded wait that looks at the clock only now and then; the first that gives up makes the CTA's others do so, too.
__device__ __forceinline__ bool decode_wait(uint64_t* bar, uint32_t parity, int* abort_flag, unsigned long long timeout_ns) {
  unsigned long long t0 = 0;
#pragma unroll 1
  for (uint32_t i = 0; !mbar_try_wait(bar, parity); ++i) {
    if ((i & 15u) != 15u) continue;
    const unsigned long long now = global_timer_ns();
    t0 = i < 16u ? now : t0;
    if (now - t0 > timeout_ns) atomicExch(abort_flag, 1);
    if (*const_cast<volatile int*>(abort_flag) != 0) return false;
  }
  return true;
}
// d = a b.
template <bool F16>
__device__ __forceinline__ void mma_16816_first(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                                uint32_t b1) {
  if (F16)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
                 : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t f16x2_mul(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// 4-bit codes 0 and 4 (even) or 1 and 5 of a word as fp16 numbers (code + 8) 2^-24, the odd ones times 16: one instruction,
// if the eights come in a register (as two constants they are two instructions).
__device__ __forceinline__ uint32_t int4_even(uint32_t w, uint32_t eights) { return (w & 0x000F000Fu) ^ eights; }
__device__ __forceinline__ uint32_t int4_odd(uint32_t w, uint32_t eights16) { return (w & 0x00F000F0u) ^ eights16; }
enum : int { W_DEC_FULL = 40, W_DEC_EMPTY = 41 };  // where a wait ran out
constexpr float kDecCode = 16777216.f;           // 2^24: one over a code as fp16
constexpr float kDecToBf16 = 6.490371073168535e32f;  // 2^109: that over a code as bf16

// A scale of V (bits of a bf16 number that is not negative) times 2^-e, e = field - 126 with `field` that of the token's
// largest: at most 1; 0 for what is no finite number.
__device__ __forceinline__ float int4_part(uint32_t bits, int field) {
  const float down = __uint_as_float(static_cast<uint32_t>(253 - min(field, 252)) << 23);
  const float more = field > 252 ? (field == 253 ? 0.5f : 0.25f) : 1.f;
  return bits < 0x7F80u ? __uint_as_float(bits << 16) * down * more : 0.f;
}

template <bool WIN>
__global__ void __launch_bounds__(DecodeInt4Traits::kThreads, DecodeInt4Traits::kCtas)
    attention_decode_int4_kernel(const __grid_constant__ DecodeParams p) {
  using T = DecodeInt4Traits;
  extern __shared__ __align__(128) uint8_t smem_raw[];
  uint8_t* const smem = smem_raw + ((512u - (smem_u32(smem_raw) & 511u)) & 511u);
  // [warp][head]: m, m', l, place
  float4* const stats = reinterpret_cast<float4*>(smem + T::kStages * T::kStage + T::kWarps * T::kOwn);
  uint8_t* const query = reinterpret_cast<uint8_t*>(stats + T::kWarps * 8);
  long long* const plan = reinterpret_cast<long long*>(query + T::kQuery);
  uint64_t* const full = reinterpret_cast<uint64_t*>(plan + 16);
  uint64_t* const empty = full + T::kStages;
  int* const stage_bad = reinterpret_cast<int*>(empty + T::kStages);  // the unit in the stage meets a bad table entry
  int* const abort_flag = stage_bad + T::kStages;
  DecodeKept* const kept = reinterpret_cast<DecodeKept*>(plan + 16 + 2 * T::kStages + 2);
  static_assert((T::kStages + 1) * 4 <= 16, "two words");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, q = lane & 3;
  const DecodeWalk<T::kUnit, WIN, T::kOver> walk(p);
  decode_hints(p, tid);
  if (tid == 0) {
    for (int i = 0; i < T::kStages; ++i) mbar_init(&full[i], p.box > 0 ? 1 : 33), mbar_init(&empty[i], T::kWarps);
    *abort_flag = 0;
    fence_mbar_init();
    if (p.box > 0) tma_prefetch_desc(&p.map_k), tma_prefetch_desc(&p.map_v);
  }
  __syncthreads();
  griddep_wait();  // launched as a dependent: nothing is read before the kernel in front has finished
  griddep_launch_dependents();
  DecodeSeg seg;
  long long left;
  {
    DecodeShare own;
    if (!decode_plan<T::kThreads>(p, walk, plan, own, seg)) return;
    left = own.u1 - own.u0;
    if (tid == 0) kept->own = own, kept->seg = seg, kept->left = left, kept->cuts = DecodeCuts();
  }

  if (warp == T::kWarps) {
    // ================================================================ the ring is filled
    int pt = seg.t0, stage = 0;
    uint32_t round = 0;
    auto advance = [&]() -> bool {  // on to the next unit that has tokens
      while (pt >= seg.t1) {
        left -= seg.units;
        if (left <= T::kOver) return false;
        walk.next(seg, left);
        pt = seg.t0;
        const char* row = reinterpret_cast<const char*>(p.Q + seg.b * p.ldq + static_cast<long long>(seg.kvh) * p.group * kHeadDim);
        if (lane < 2 * p.group) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + lane * 128));  // its queries
      }
      return true;
    };
    auto stage_free = [&]() -> bool {
      return __all_sync(~0u, round == 0 || decode_wait(&empty[stage], (round & 1) ^ 1, abort_flag, p.timeout_ns));
    };
    auto filled = [&]() {
      if (++stage == T::kStages) stage = 0, ++round;
    };
    bool more = advance(), ok = true;
    if (p.box > 0) {  // a lane for each box of rows
      const int row0 = lane * p.box;
      int entry = 0, slot = 0;
      auto look_up = [&]() {
        const int pos = min(pt + row0, seg.t1 - 1) + walk.shift_of(seg, pt), page = walk.page_of(pos);
        slot = pos - page * p.c.page_size;
        entry = p.c.table[seg.b * p.c.ldt + page];
      };
      if (more) look_up();
      while (more) {
        const int rows = seg.t1 - pt;
        bool mine = row0 < T::kUnit && row0 < rows;  // a box that no row is needed of stays where it is
        if (WIN && mine) {
          const int first = pt + walk.shift_of(seg, pt);
          mine = walk.in_sight(seg, first + row0) || walk.in_sight(seg, first + min(row0 + p.box, rows) - 1);
        }
        const bool there = static_cast<unsigned>(entry) < static_cast<unsigned>(p.c.num_pages);
        const bool bad = __any_sync(~0u, mine && !there);
        mine = mine && there;
        const int boxes = __popc(__ballot_sync(~0u, mine));
        const long long cell = static_cast<long long>(seg.kvh) * p.c.page_size + slot;
        const int row = static_cast<int>(static_cast<long long>(entry) * p.c.n_kv * p.c.page_size + cell);
        const long long scale = (entry * p.c.scale_pitch + cell * kInt4Groups) * 2;
        pt += T::kUnit;
        more = advance();
        if (more) look_up();  // on its way while the stage is waited for
        if (!(ok = stage_free())) break;
        if (lane == 0) {
          stage_bad[stage] = bad;
          mbar_arrive_expect_tx(&full[stage], static_cast<uint32_t>(boxes * p.box * 2 * (T::kRowBytes + T::kScaleBytes)));
        }
        __syncwarp();
        if (mine) {
          uint8_t* to = smem + stage * T::kStage;
          tma_load_2d(&p.map_k, &full[stage], to + row0 * T::kRowBytes, 0, row);
          tma_load_2d(&p.map_v, &full[stage], to + T::kTile + row0 * T::kRowBytes, 0, row);
          to += 2 * T::kTile + row0 * T::kScaleBytes;
          bulk_load_g2s(to, static_cast<const uint8_t*>(p.c.ks) + scale, p.box * T::kScaleBytes, &full[stage]);
          bulk_load_g2s(to + T::kScales, static_cast<const uint8_t*>(p.c.vs) + scale, p.box * T::kScaleBytes, &full[stage]);
        }
        filled();
      }
    } else {  // four rows a lane
      while (more) {
        if (!(ok = stage_free())) break;
        bool bad = false;
        const uint32_t to = smem_u32(smem) + stage * T::kStage;
        const int shift = walk.shift_of(seg, pt);
#pragma unroll 1
        for (int row = lane; row < T::kUnit && pt + row < seg.t1; row += 32) {
          const int pos = pt + row + shift;
          if (!walk.in_sight(seg, pos)) continue;
          const int page = walk.page_of(pos), entry = p.c.table[seg.b * p.c.ldt + page];
          const bool there = static_cast<unsigned>(entry) < static_cast<unsigned>(p.c.num_pages);
          bad |= !there;
          if (!there) continue;
          const long long cell = static_cast<long long>(seg.kvh) * p.c.page_size + (pos - page * p.c.page_size);
          const long long code = entry * p.c.page_pitch + cell * T::kRowBytes,
                          scale = (entry * p.c.scale_pitch + cell * kInt4Groups) * 2;
#pragma unroll
          for (int c = 0; c < T::kRowBytes / 16; ++c) {
            const uint32_t at = to + (row >> 1) * 128 + ((((row & 1) << 2 | c) ^ (row >> 1 & 3)) << 4);  // as the tensor copies do
            cp_async_16_or_zero(at, static_cast<const uint8_t*>(p.c.k) + code + c * 16, true);
            cp_async_16_or_zero(at + T::kTile, static_cast<const uint8_t*>(p.c.v) + code + c * 16, true);
          }
          const uint32_t scales = to + 2 * T::kTile + row * T::kScaleBytes;
          cp_async_8_or_zero(scales, static_cast<const uint8_t*>(p.c.ks) + scale, true);
          cp_async_8_or_zero(scales + T::kScales, static_cast<const uint8_t*>(p.c.vs) + scale, true);
        }
        bad = __any_sync(~0u, bad);
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&full[stage])) : "memory");
        if (lane == 0) {
          stage_bad[stage] = bad;
          mbar_arrive(&full[stage]);
        }
        filled();
        pt += T::kUnit;
        more = advance();
      }
    }
    if (!ok && lane == 0) record_failure(p.status, W_DEC_EMPTY, stage);
    // Leave no copy in flight, each stage's last one: a warp that gave up waiting for it ends without it.
    for (int i = 0; i < T::kStages; ++i)
      if (round > 0 || i < stage) mbar_wait_quiet(&full[i], (i < stage ? round : round - 1) & 1, 1000000000);
    return;
  }

  // ================================================================ the warps that compute
  uint8_t* const mine = smem + T::kStages * T::kStage + warp * T::kOwn;
  uint8_t* const parts = mine;
  // group 0 of row `lane`, whose address this lane gives to ldmatrix; group c: xor 16 c
  const uint32_t ld_at = (lane >> 1) * 128 + (((lane & 1) << 2 ^ (lane >> 1 & 3)) << 4);
  const uint32_t flip = p.eights, flip16 = flip << 4;
  auto sync = [] { named_bar_sync(1, 32 * T::kWarps); };
  int stage = 0;
  uint32_t parity = 0;
  constexpr uint32_t kSpread = 16, kBad = 32, kFailed = 64;
  uint32_t said = 0;  // kFailed: a wait ran out

  for (;;) {
    // ---- this segment's query fragments (B operand: head g of the column tile, dimensions in the codes' order)
    auto first_head = [&] { return seg.kvh * p.group + seg.chunk * p.chunk_heads; };
    auto heads_here = [&] { return min(p.chunk_heads, p.group - seg.chunk * p.chunk_heads); };
    {
      const int head0 = first_head(), n_heads = heads_here();
      uint4 own_group = make_uint4(0, 0, 0, 0);
      float a = 0.f;
#pragma unroll
      for (int c = 0; c < kInt4Groups; ++c) {
        uint4 w = make_uint4(0, 0, 0, 0);
        if (g < n_heads)
          w = *reinterpret_cast<const uint4*>(p.Q + seg.b * p.ldq + static_cast<long long>(head0 + g) * kHeadDim + c * kInt4Group +
                                              q * 8);
        if (c == warp) own_group = w;
        const uint32_t four[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) a = fmaxf(a, fmaxf(fabsf(bf16_lo(four[i])), fabsf(bf16_hi(four[i]))));
      }
      a = fmaxf(a, __shfl_xor_sync(~0u, a, 1));
      a = fmaxf(a, __shfl_xor_sync(~0u, a, 2));
      // 2^e that takes the largest value to [2^14, 2^15); values that are not finite stay what they are
      const int ex = static_cast<int>(__float_as_uint(a) >> 23);
      const int up = ex == 255 ? 127 : min(max(268 - ex, 1), 253);
      const float lift = __uint_as_float(static_cast<uint32_t>(up) << 23);
      const float f = p.scale_log2 * __uint_as_float(static_cast<uint32_t>(254 - up) << 23);
      // columns 0 and 4, 2 and 6, 1 and 5, 3 and 7 of group `warp`
      uint32_t two[4] = {__byte_perm(own_group.x, own_group.z, 0x5410), __byte_perm(own_group.y, own_group.w, 0x5410),
                         __byte_perm(own_group.x, own_group.z, 0x7632), __byte_perm(own_group.y, own_group.w, 0x7632)};
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float by = i < 2 ? lift : lift * 0.0625f, back = i < 2 ? 1.f : 16.f;
        two[i] = pack_f16x2(bf16_lo(two[i]) * by, bf16_hi(two[i]) * by);
        const float2 used = __half22float2(*reinterpret_cast<const __half2*>(&two[i]));  // what the products see
        sum += (used.x + used.y) * back;
      }
      sum += __shfl_xor_sync(~0u, sum, 1);
      sum += __shfl_xor_sync(~0u, sum, 2);
      *reinterpret_cast<uint4*>(query + (warp * 32 + lane) * 16) = make_uint4(two[0], two[1], two[2], two[3]);
      if (q == 0) reinterpret_cast<float*>(query + kInt4Groups * 512)[warp * 8 + g] = sum * (-8.f / kDecCode);
      // f times 2^24, as two factors the first of which neither overflows nor, where it matters, underflows
      const float f0 = f > 1.f ? kDecCode : f, f1 = f > 1.f ? f : kDecCode;
      // [q]: of heads 2q and 2q + 1 the first, then the second
      if (warp == 0 && q < 2)
        reinterpret_cast<float*>(query + kInt4Groups * (512 + 32))[(g >> 1) * 4 + q * 2 + (g & 1)] = q == 0 ? f0 : f1;
      sync();
    }
    // Of this segment: the table or the length is bad; the scales of some token lie far apart (kSpread); in bits 0-3 the groups of
    // columns in which this lane met a scale of V that is not finite.
    said = (said & kFailed) | (seg.bad ? kBad : 0u);
    float o[8][4];
    float m[2], mv[2];
    uint64_t l;
#pragma unroll
    for (int t = 0; t < 8; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[t][i] = 0.f;
    m[0] = m[1] = mv[0] = mv[1] = kDecNone;
    l = 0;

    for (int unit = seg.t0; unit < seg.t1; unit += T::kUnit) {
      if ((said & kFailed) == 0 && !decode_wait(&full[stage], parity, abort_flag, p.timeout_ns)) {
        said |= kFailed;
        record_failure(p.status, W_DEC_FULL, stage);
      }
      __syncwarp();
      if (stage_bad[stage] != 0) said |= kBad;
      const int t = unit + warp * T::kStep;
      if (t < seg.t1) {
        const uint32_t kb = smem_u32(smem) + stage * T::kStage + warp * (T::kStep * T::kRowBytes), vb = kb + T::kTile;
        const uint8_t* const k_scales = smem + stage * T::kStage + 2 * T::kTile + warp * (T::kStep * T::kScaleBytes);
        const uint8_t* const v_scales = k_scales + T::kScales;
        const int pos0 = t + walk.shift_of(seg, t);
        float x[T::kSubs * 4];    // logits: lane (g, q) holds tokens g, g + 8 of each tile for heads 2q, 2q + 1
        // ---- V's scales, lane = token: their power of two apart, the rest (at most 1) as fp16 by pairs of tokens.  For bf16
        // bits w of exponent E and `field` that of the token's largest, the part's fp16 bits are (w - ((field - 14) << 7)) << 3.
        uint2 sv = *reinterpret_cast<const uint2*>(v_scales + lane * 8);
        bool cut = t + T::kStep > seg.t1;  // some rows are not to be seen; they may hold anything
        if (WIN) cut |= pos0 + T::kStep > p.sinks && pos0 < seg.len - p.window;
        if (cut && (t + lane >= seg.t1 || !walk.in_sight(seg, pos0 + lane))) sv = make_uint2(0, 0);
        uint32_t top, low;  // the token's largest scale, and the smallest that is not zero less 1
        auto ends = [&]() {
          top = u16x2_max(sv.x, sv.y);
          top = max(top & 0xFFFFu, top >> 16);
          low = u16x2_min(u16x2_add(sv.x, 0xFFFFFFFFu), u16x2_add(sv.y, 0xFFFFFFFFu));
          low = min(low & 0xFFFFu, low >> 16);
        };
        // scales that lie far apart, and what the integers do not hold: 2^-111 and below, 2^126 and above
        auto far = [&]() { return top != 0 && (top < 0x0800u || top >= 0x7E80u || low + 1 < top - 0x0600u); };
        ends();
        if (__any_sync(~0u, far())) {
          uint32_t four[4] = {sv.x & 0xFFFFu, sv.x >> 16, sv.y & 0xFFFFu, sv.y >> 16};
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (four[c] >= 0x7F80u) {  // reaches its own columns only, at the segment's end; -0 is a zero
              if (four[c] != 0x8000u) said |= 1u << c;
              four[c] = 0;
            }
          sv = make_uint2(four[0] | four[1] << 16, four[2] | four[3] << 16);
          ends();
          if (__any_sync(~0u, far())) said |= kSpread;
        }
        const float power = __uint_as_float(0x4B000000u + (top >> 7)) - (8388608.f + 126.f);
        uint8_t* const pairs = parts + T::kParts;
        {
          const uint2 sk = *reinterpret_cast<const uint2*>(k_scales + lane * 8);
          const float k[4] = {bf16_lo(sk.x), bf16_hi(sk.x), bf16_lo(sk.y), bf16_hi(sk.y)};
          uint8_t* const to = pairs + (lane & 7) * 32 + (lane >> 3) * 8;
#pragma unroll
          for (int c = 0; c < kInt4Groups; ++c) *reinterpret_cast<float2*>(to + c * T::kPairs) = make_float2(k[c], k[c]);
          *reinterpret_cast<float2*>(to + kInt4Groups * T::kPairs) = make_float2(power, power);
        }
        if ((said & kSpread) == 0) {
          const uint32_t base = (max(top >> 7, 14u) - 14u) * 0x00800080u;
          const uint32_t p01 = (u16x2_max(sv.x, base) - base) << 3, p23 = (u16x2_max(sv.y, base) - base) << 3;
          const bool second = (lane & 1) != 0;  // of a pair of tokens: writes groups 2 and 3, the first one 0 and 1
          const uint32_t other = __shfl_xor_sync(~0u, second ? p01 : p23, 1);
          const uint32_t first_token = second ? other : p01, second_token = second ? p23 : other;
          uint8_t* const to = parts + (lane & 1) * (2 * T::kStep * 2) + (lane >> 1 & 3) * 16 + (lane >> 3) * 4;
          *reinterpret_cast<uint32_t*>(to) = __byte_perm(first_token, second_token, 0x5410);
          *reinterpret_cast<uint32_t*>(to + T::kStep * 2) = __byte_perm(first_token, second_token, 0x7632);
        }
        __syncwarp();
        // ---- S^T = K Q^T: two tiles of 16 tokens x 8 heads, k = 32 for each group
        uint64_t sum[T::kSubs * 2];  // of tokens g + 8 r
#pragma unroll
        for (int c = 0; c < kInt4Groups; ++c) {
          uint32_t kw[4];
          ldmatrix_x4<false>(kw, kb + (ld_at ^ (c << 4)));
          const uint4 qf = *reinterpret_cast<const uint4*>(query + (c * 32 + lane) * 16);
          const uint64_t begin = *reinterpret_cast<const uint64_t*>(query + kInt4Groups * 512 + c * 32 + q * 8);
          const ulonglong2 k01 = *reinterpret_cast<const ulonglong2*>(pairs + c * T::kPairs + g * 32);
          const ulonglong2 k23 = *reinterpret_cast<const ulonglong2*>(pairs + c * T::kPairs + g * 32 + 16);
          const uint64_t ks[4] = {k01.x, k01.y, k23.x, k23.y};
#pragma unroll
          for (int sub = 0; sub < T::kSubs; ++sub) {
            const uint32_t wx = kw[sub * 2], wy = kw[sub * 2 + 1];
            float d[4];
            mma_16816_first<true>(d, int4_even(wx, flip), int4_even(wy, flip), int4_even(wx >> 8, flip), int4_even(wy >> 8, flip),
                                  qf.x, qf.y);
            mma_16816<true>(d, int4_odd(wx, flip16), int4_odd(wy, flip16), int4_odd(wx >> 8, flip16), int4_odd(wy >> 8, flip16),
                            qf.z, qf.w);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int r = sub * 2 + h;
              const uint64_t whole = f2_add(f2(d[h * 2], d[h * 2 + 1]), begin);
              sum[r] = c == 0 ? f2_mul(whole, ks[r]) : f2_fma(whole, ks[r], sum[r]);
            }
          }
        }
        const ulonglong2 fac = *reinterpret_cast<const ulonglong2*>(query + kInt4Groups * (512 + 32) + q * 16);
#pragma unroll
        for (int r = 0; r < T::kSubs * 2; ++r) f2_split(f2_mul(f2_mul(sum[r], fac.x), fac.y), x[r * 2], x[r * 2 + 1]);
        // ---- softmax
        if (cut) {
#pragma unroll
          for (int r = 0; r < T::kSubs * 2; ++r)
            if (t + g + r * 8 >= seg.t1 || !walk.in_sight(seg, pos0 + g + r * 8)) {
              x[r * 2] = x[r * 2 + 1] = -INFINITY;
            }
        }
        float y[T::kSubs * 4];  // logits with the power of V's scale on top
        bool rise = false;
        {
          const ulonglong2 l01 = *reinterpret_cast<const ulonglong2*>(pairs + kInt4Groups * T::kPairs + g * 32);
          const ulonglong2 l23 = *reinterpret_cast<const ulonglong2*>(pairs + kInt4Groups * T::kPairs + g * 32 + 16);
          const uint64_t lv[4] = {l01.x, l01.y, l23.x, l23.y};
#pragma unroll
          for (int r = 0; r < T::kSubs * 2; ++r)
            f2_split(f2_add(f2(x[r * 2], x[r * 2 + 1]), lv[r]), y[r * 2], y[r * 2 + 1]);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float a = fmaxf(max3(x[i], x[i + 2], x[i + 4]), x[i + 6]);
            const float b = fmaxf(max3(y[i], y[i + 2], y[i + 4]), y[i + 6]);
            rise |= a > m[i] + kDecLazy || b > mv[i] + kDecLazy;
          }
        }
        if (__any_sync(~0u, rise)) {
          float down[2], down_o[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float a = m[i], b = mv[i];
#pragma unroll
            for (int r = 0; r < T::kSubs * 2; ++r) a = fmaxf(a, x[r * 2 + i]), b = fmaxf(b, y[r * 2 + i]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
              a = fmaxf(a, __shfl_xor_sync(~0u, a, d));
              b = fmaxf(b, __shfl_xor_sync(~0u, b, d));
            }
            down[i] = ex2(m[i] - a), down_o[i] = ex2(mv[i] - b);
            m[i] = a;
            mv[i] = b;
#pragma unroll
            for (int d = 0; d < 8; ++d) o[d][i] *= down_o[i], o[d][i + 2] *= down_o[i];
          }
          l = f2_mul(l, f2(down[0], down[1]));
        }
        // ---- weights, and O^T += V^T P^T, of a group of 32: dimensions 4 g and 4 g + 2, then 4 g + 1 and 4 g + 3
        // -8 sum w, heads 2q and 2q + 1: d in the units of o's even dimensions, then in those of its odd ones
        const uint32_t less = flip ^ 0x80008000u, less16 = flip16 ^ 0x80008000u;
        auto take_off = [](float (&even)[4], float (&odd)[4], const float (&d)[4]) {
          const uint64_t d2 = f2(d[0], d[1]), d16 = f2(d[2], d[3]);
          f2_split(f2_add(f2(even[0], even[1]), d2), even[0], even[1]);
          f2_split(f2_add(f2(even[2], even[3]), d2), even[2], even[3]);
          f2_split(f2_add(f2(odd[0], odd[1]), d16), odd[0], odd[1]);
          f2_split(f2_add(f2(odd[2], odd[3]), d16), odd[2], odd[3]);
        };
        const uint64_t minus_m = f2(-m[0], -m[1]), minus_mv = f2(kDecLift - mv[0], kDecLift - mv[1]);
#pragma unroll
        for (int r = 0; r < T::kSubs * 2; ++r) {
          float e0, e1;
          f2_split(f2_add(f2(x[r * 2], x[r * 2 + 1]), minus_m), e0, e1);
          l = f2_add(l, f2(ex2(e0), ex2(e1)));
          f2_split(f2_add(f2(y[r * 2], y[r * 2 + 1]), minus_mv), e0, e1);
          y[r * 2] = ex2(e0), y[r * 2 + 1] = ex2(e1);
        }
        if ((said & kSpread) == 0) {
          uint32_t pf[T::kSubs][2];  // P^T (B operand: tokens 2q, 2q + 1 | + 8 of head g)
#pragma unroll
          for (int r = 0; r < T::kSubs * 2; ++r) pf[r >> 1][r & 1] = transpose8x8(pack_f16x2(y[r * 2], y[r * 2 + 1]));
#pragma unroll
          for (int c = 0; c < kInt4Groups; ++c) {
            uint32_t v[4];
            ldmatrix_x4<true>(v, vb + (ld_at ^ (c << 4)));
            const uint4 rc = *reinterpret_cast<const uint4*>(parts + c * (T::kStep * 2) + q * 16);
            const uint32_t b[4] = {f16x2_mul(pf[0][0], rc.x), f16x2_mul(pf[0][1], rc.y), f16x2_mul(pf[1][0], rc.z),
                                   f16x2_mul(pf[1][1], rc.w)};
#pragma unroll
            for (int sub = 0; sub < T::kSubs; ++sub) {
              const uint32_t lo = v[sub * 2], hi = v[sub * 2 + 1], b0 = b[sub * 2], b1 = b[sub * 2 + 1];
              mma_16816<true>(o[c * 2], int4_even(lo, flip), int4_even(lo >> 8, flip), int4_even(hi, flip),
                              int4_even(hi >> 8, flip), b0, b1);
              mma_16816<true>(o[c * 2 + 1], int4_odd(lo, flip16), int4_odd(lo >> 8, flip16), int4_odd(hi, flip16),
                              int4_odd(hi >> 8, flip16), b0, b1);
            }
            float d[4];
            mma_16816_first<true>(d, less, less16, less, less16, b[0], b[1]);
            mma_16816<true>(d, less, less16, less, less16, b[2], b[3]);
            take_off(o[c * 2], o[c * 2 + 1], d);
          }
        } else {
#pragma unroll
          for (int r = 0; r < T::kSubs * 2; ++r) {  // tokens g + 8 r: eight at a time, the other eight with weights of zero
            uint2 raw = *reinterpret_cast<const uint2*>(v_scales + (g + r * 8) * 8);
            if (t + g + r * 8 >= seg.t1 || !walk.in_sight(seg, pos0 + g + r * 8)) raw = make_uint2(0, 0);  // it may hold anything
            const uint32_t four[4] = {raw.x & 0xFFFFu, raw.x >> 16, raw.y & 0xFFFFu, raw.y >> 16};
            uint32_t largest = 0;
#pragma unroll
            for (int c = 0; c < 4; ++c) largest = max(largest, four[c] < 0x7F80u ? four[c] : 0u);
#pragma unroll
            for (int c = 0; c < kInt4Groups; ++c) {
              uint32_t v[4];
              ldmatrix_x4<true>(v, vb + (ld_at ^ (c << 4)));
              const float part = int4_part(four[c], static_cast<int>(largest >> 7)) * kDecToBf16;
              const float w0 = y[r * 2] * part, w1 = y[r * 2 + 1] * part;
              const uint32_t top = pack_bf16x2(w0, w1);
              const uint32_t b[2] = {transpose8x8(top), transpose8x8(pack_bf16x2(w0 - bf16_lo(top), w1 - bf16_hi(top)))};
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                mma_16816<false>(o[c * 2], int4_even(v[r], flip), int4_even(v[r] >> 8, flip), 0u, 0u, b[k], 0u);
                mma_16816<false>(o[c * 2 + 1], int4_odd(v[r], flip16), int4_odd(v[r] >> 8, flip16), 0u, 0u, b[k], 0u);
              }
              float d[4];
              mma_16816_first<false>(d, less, less16, less, less16, b[0], 0u);
              mma_16816<false>(d, less, less16, less, less16, b[1], 0u);
              take_off(o[c * 2], o[c * 2 + 1], d);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[stage]);
      if (++stage == T::kStages) stage = 0, parity ^= 1;
    }

    // ---- the CTA's four pieces become one: finished here, or a part of a cut (sequence, head)
    DecodeShare own = kept->own;
    seg = kept->seg, left = kept->left;
    const DecodeOwners owners = decode_owners<T::kOver>(p, own, seg);
    const bool spoiled = __any_sync(~0u, (said & (kBad | kFailed)) != 0);
    if (spoiled && lane == 0 && atomicCAS(p.status + ST_CODE, 0, static_cast<int>(FL_ERR_INVALID_ARG)) == 0)
      p.status[ST_DETAIL] = seg.b;
    const uint32_t no_number = __reduce_or_sync(~0u, said);  // bits 0-3
    // o[t][i] with t = 2 group + odd: head 2q + (i & 1), dimension 32 group + 4 g + odd + 2 (i >> 1), odd ones times 16.  Chunks of
    // 4 dimensions, permuted by 2 q against bank conflicts.
    {
      float sums[2];
      f2_split(l, sums[0], sums[1]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float sum = sums[i];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(~0u, sum, d);
        const int h = 2 * q + i;
        float* row = reinterpret_cast<float*>(mine) + h * kHeadDim;
#pragma unroll
        for (int c = 0; c < kInt4Groups; ++c) {
          constexpr float kOdd = kDecCode / 16.f;
          float4 four = make_float4(o[c * 2][i] * kDecCode, o[c * 2 + 1][i] * kOdd, o[c * 2][i + 2] * kDecCode,
                                    o[c * 2 + 1][i + 2] * kOdd);
          if ((no_number >> c & 1u) != 0) four = make_float4(NAN, NAN, NAN, NAN);
          *reinterpret_cast<float4*>(row + (((c * 8 + g) ^ (q * 2)) << 2)) = four;
        }
        if (g == 0)
          stats[warp * 8 + h] =
              make_float4(m[i], mv[i] - kDecLift, spoiled ? NAN : sum, __int_as_float(static_cast<int>(mine - smem)));
      }
    }
    sync();
    decode_merge<T::kWarps, 8, 2>(p, smem, stats, warp, lane, seg, first_head(), heads_here(), owners);
    sync();
    if (!owners.whole && tid == 0) kept->cuts.add(seg, owners);
    left -= seg.units;
    if (left <= T::kOver) break;  // another beginning at most
    own.seg_first += seg.n_units;
    walk.next(seg, left);
    if (tid == 0) kept->own.seg_first = own.seg_first, kept->seg = seg, kept->left = left;
  }
  sync();
  if (kept->cuts.any()) decode_join<T::kWarps>(p, kept->cuts, plan, sync);
}

}  // namespace fl
