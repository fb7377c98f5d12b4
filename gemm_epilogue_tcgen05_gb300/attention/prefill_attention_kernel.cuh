// Attention over whole prompts, packed one behind the other, on the tcgen05 tensor cores.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = 2^(x_ij - m_i),  x_ij = scale * log2(e) * q_i . k_j
//
// What bounds it: 4 * 128 multiply-adds for every (query, key, head) on the tensor cores, and one exponential
// for each of the same on the special-function units; HBM traffic is small beside both.
//
// Tile.  A CTA works on two query tiles of 128 rows at once against one stream of 128-key tiles of K and V.  The
// rows of a query tile are (token, head) pairs: the hp query heads that share a kv head lie side by side, so a
// tile holds 128 / hp consecutive tokens.  Short prompts fill their tiles and the causal diagonal cuts off less.
// While one query tile is in its softmax the tensor cores work for the other one:
//   S_s = Q_s K^T (TMEM, 128 columns each)  ->  softmax in registers, one thread a row  ->  P_s as bf16 over S_s
//   (TMEM)  ->  O_s += P_s V (A from TMEM, V as stored: MN-major B; TMEM, 128 columns each).  512 columns in all.
//
// Warps 0-3 and 4-7: softmax of query tile 0 and 1 and its output.  Warp 8: one thread issues the MMAs.  Warp 9:
// one thread issues the TMA loads (Q by a 3-D map over (dimension, head, row); a V tile and the K tile behind it
// into one of two 64 KB stages).  Warp 10: which tile comes next.  Warp 11: V rows in masked tiles.
// One persistent CTA on each SM; the next tile's loads, its first products and the last one's output overlap.
//
// The row maximum is only raised when a logit passes it by more than 2^8 (in the weights); then the thread that
// owns the row scales its O in TMEM, which is complete by the time S of the next key tile is (one commit covers
// all products before it), so no hand-over is needed.
//
// Work: tile (sequence, block of tokens, kv head) by falling block index, so the longest come first whatever the
// sequences' lengths are (without the causal mask by falling length; with many sequences one after the other, each from
// its last block), each taken by the CTA that is free next (an atomic counter, one tile ahead).  Neighbouring ranks are
// the heads of one block: K and V are met again by every block of the sequence, and the keys and values of all heads of all
// sequences can be more than the L2 holds.  So the heads are worked off in groups whose keys and values are at
// most 32 MB.
//
// Masked columns have weight zero, but 0 * NaN is NaN: in tiles where some row masks some key, warp 11 replaces
// values of V that are not finite by zero before the product; rows that do see such a key add it at the end.
//
// E4M3: a first kernel writes K as bf16 (code times scale, 8 bits where the code carries 4) and V as fp16 times 2^-b,
// b from the largest scale of 128 keys and a head, so that the largest possible value is in [2^14, 2^16).  The logits of
// a key tile get b on top: weights are 2^(x + b - m + 7) in fp16, m the running maximum of x + b, and meet V 2^-b in O
// at one common power whatever the tiles' scales are.  The sum l has a maximum mx of its own, of x alone: each tile's
// weights come to it times 2^(m - b - 7 - mx).  A tile whose values are all zero gets a power of 2^-90, and its sum is
// taken at mx: with an ordinary power its logits would raise m and push the weights of small values in other tiles below
// fp16's range (128 such keys in front of values of 1e-5: relative error 0.2).
//
// b stands for the tile's ordinary keys, whose scales lie within kPreWindow powers of two, so that each value keeps its
// bits whatever another key's scale is, be it later in the sequence.  What lies outside (attention sinks with tiny values,
// outliers) are single keys: their V is zero in the tile, and the softmax warps take their columns out of S and add
// p_j v_j in fp32 from the codes to O, which they begin with zeros.  (One power for all keys of a tile lost the bits of
// the small ones: a later scale 2^32 times the others' put an error of 4 % on the rows before it, 2^40 all of them.)
//
// Measured for 4 x 2048 tokens, 32 query and 8 kv heads: 311 us with scales inside the softmax (two multiplications and
// two shared-memory reads for each query and key, reads that the tensor cores need for themselves), 123 us with fp16
// keys (11 bits, but queries that have to become fp16, too), 110.5 us with keys as bf16 and one power for all keys of a
// tile, 105 us with bf16 values and weights, whose roundings make the error 1.8 times that of a bf16 output alone
// instead of 1.4 times.  Single keys cost 1.5 us where there are none (109.2 -> 110.6 in one run), else 3 us for the
// first and 1.5 us for each other one that a unit of work meets in a tile, 0.1 us for those of zeros.
#pragma once
#include <climits>

#include "attention_common.h"

namespace fl {

constexpr int kPreThreads = 384;
// Registers of a thread at launch (the launch checks that the compiler used exactly these), of the softmax
// warps and of the other four: 384 * 168 = 256 * 200 + 128 * 104.
constexpr int kPreRegs = 168, kPreRegsSoftmax = 200, kPreRegsOther = 104;
static_assert(kPreThreads * kPreRegs == 256 * kPreRegsSoftmax + 128 * kPreRegsOther, "register split");
constexpr int kPreTile = 128;                      // query rows of a tile, and keys of a tile
constexpr int kPreTileBytes = kPreTile * kHeadDim * 2;
constexpr int kPreRing = 3;                        // tile descriptors
constexpr float kPreNone = -3e38f;                 // a maximum over nothing: any finite logit passes it
constexpr float kPreLazy = 8.f;
constexpr uint64_t kPreDrainNs = 1000000000;       // for copies and products in flight, whatever the limit of the waits
constexpr float kPreLift = 7.f;                    // E4M3: weights are lifted by 2^7 in fp16 (2^8 more: kPreLazy)
// E4M3: the power of a key tile whose values are all zero, and of a single key of that kind: low enough to leave other
// weights alone, high enough for 2^(m - mx) to stay in fp32's range, and no whole number, so that no other tile has it.
constexpr float kPreZero = -90.5f;
constexpr int kPreWindow = 13;                     // E4M3: powers of two that the scales of a tile's ordinary keys span
constexpr int kPreRoom = 6;                        // E4M3: the largest of these scales times 2^-b is in [2^6, 2^7)
// E4M3: b of any tile with ordinary keys.  m stays within 2^30 of mx then, and no weight that counts for l falls below
// fp32's range: it is 2^(x - mx - 30 - 60 + 7 - 8) at least, 2^-126 for x = mx - 35.
constexpr int kPrePowerMin = -60, kPrePowerMax = 30;
// E4M3: what a tile's power carries on top, times kPreMark: it has single keys, and its first key is one.
constexpr float kPreMark = 65536.f;
enum : int { PRE_SINGLE = 1, PRE_SINGLE_FIRST = 2 };

// Where a wait gave up (recorded in the workspace's status record).
enum : int {
  W_PRE_TILE_FULL = 20, W_PRE_TILE_EMPTY = 21, W_PRE_Q_EMPTY = 22, W_PRE_Q_FULL = 23, W_PRE_KV_EMPTY = 24,
  W_PRE_KV_FULL = 25, W_PRE_S = 26, W_PRE_P = 27, W_PRE_O = 28, W_PRE_V = 29
};

struct alignas(128) PrefillParams {
  CUtensorMap map_q;  // Q [M][n_heads][128] bf16, box {64, hp, tq}
  CUtensorMap map_k;  // K [M][n_kv * 128] bf16, box {64, 128}
  CUtensorMap map_v;  // the same, E4M3: fp16
  const __nv_bfloat16* V;  // the rows map_v covers
  long long ldv;
  const float* powers;  // E4M3: [first row of a key tile][n_kv]: b of V * 2^-b, and marks; other rows: 1 for a single key
  const uint8_t* codes;  // E4M3: V and its scales as given, for single keys
  const float* v_scale;
  long long ld_codes, ld_scale;
  int n_kv;
  const int* cu;
  __nv_bfloat16* O;
  long long ldo;
  int M, batch, seq_len, causal, flat;
  int group, hp, tq;       // query heads of a kv head; heads and tokens of a query tile
  int pairs;               // head packs of a token block: n_kv * group / hp
  int pairs_at_once;       // of which this many are worked off before the next ones begin
  float scale_log2;
  int* status;
  unsigned* work;          // [0] ranks given out beyond the first of each CTA, [1] CTAs that take no more
  unsigned long long timeout_ns;
};

struct PrefillTraits {
  static constexpr int kStages = 2;  // of a V tile and the next K tile, 64 KB
  static constexpr int kBars = 1024;
  // output on its way from a row per thread to whole lines: 32 rows of kOutCols columns for each softmax warp
  static constexpr int kOutCols = 64;
  static constexpr int kOut = 8 * 32 * kOutCols * 2;
  static constexpr int kSmem = (2 + 2 * kStages) * kPreTileBytes + kOut + kBars + 1024 /*alignment*/;
  static_assert(kSmem <= 232448, "shared memory of a CTA");
};

// One unit of work.
struct PrefillTile {
  int row0, len;   // the sequence's first row and length
  int tok0;        // first token of query tile 0 (query tile 1: + tq)
  int n0, n1;      // key tiles that query tiles 0 and 1 meet
  int head0, kvh;
  int bad_lo, bad_hi;  // set by warp 11: first and last key of masked tiles whose V is not finite (none: hi < 0)
};

struct PrefillBars {
  uint64_t tile_full[kPreRing], tile_empty[kPreRing];
  uint64_t q_full[2], q_empty[2];
  uint64_t kv_full[2], kv_empty[2], v_ok[2];
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t drain;
  PrefillTile tile[kPreRing];
  int abort_flag;
  uint32_t tmem;
};
static_assert(sizeof(PrefillBars) <= 1024, "barrier block");

struct PreWait {
  int* abort_flag;      // shared memory: where the first wait gave up, 0 while none has
  uint32_t timeout_ns;  // at most 2^32 - 1: 4 seconds
};

// D[tmem] (+)= A[tmem] * B: A bf16 pairs packed along K in tensor memory.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
__device__ __forceinline__ float tmem_ld1(uint32_t taddr) {
  uint32_t r;
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(taddr));
  tmem_ld_wait();
  return __uint_as_float(r);
}
__device__ __forceinline__ void tmem_st1(uint32_t taddr, float v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x1.b32 [%0], {%1};" ::"r"(taddr), "r"(__float_as_uint(v)));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tma_load_3d(const void* map, uint64_t* bar, uint32_t dst, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}
// A bounded wait that looks at the clock only now and then (reading it takes longer than most of these waits).  One
// that gives up leaves its place in the abort flag, which is recorded at the end: there are many waits, and
// instructions come from a cache that this kernel overflows.
__device__ __forceinline__ bool pre_wait(uint64_t* bar, uint32_t parity, const PreWait& w, int where) {
  uint32_t t0 = 0;
#pragma unroll 1
  for (uint32_t i = 0; !mbar_try_wait(bar, parity); ++i) {
    if ((i & 15u) != 15u) continue;
    uint32_t now;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(now));
    t0 = i < 16u ? now : t0;
    if (now - t0 > w.timeout_ns) atomicCAS(w.abort_flag, 0, where);
    if (*const_cast<volatile int*>(w.abort_flag) != 0) return false;
  }
  return true;
}
// A wait of all lanes of a warp: they go on, or give up, together.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const PreWait& w, int where) {
  return __all_sync(~0u, pre_wait(bar, parity, w, where));
}
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// Two values times zero, plus c: NaN for one that is not finite.
template <bool F16>
__device__ __forceinline__ uint32_t times_zero(uint32_t a, uint32_t c) {
  uint32_t r;
  if (F16) asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(0), "r"(c));
  else asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(0), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two fp32 lanes in one 64-bit register.
__device__ __forceinline__ uint64_t f2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_split(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

template <bool FP8>
__global__ void __launch_bounds__(kPreThreads, 1) attention_prefill_kernel(const __grid_constant__ PrefillParams p) {
  using T = PrefillTraits;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t q_smem = smem_u32(smem), kv_smem = q_smem + 2 * kPreTileBytes;
  constexpr int kOutAt = (2 + 2 * T::kStages) * kPreTileBytes;
  PrefillBars& bar = *reinterpret_cast<PrefillBars*>(smem + kOutAt + T::kOut);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = gridDim.x, cta = blockIdx.x;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kPreRing; ++i) mbar_init(&bar.tile_full[i], 1), mbar_init(&bar.tile_empty[i], 11);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.q_full[i], 1), mbar_init(&bar.q_empty[i], 1);
      mbar_init(&bar.s_full[i], 1), mbar_init(&bar.p_full[i], 4), mbar_init(&bar.o_full[i], 1);
    }
    for (int i = 0; i < T::kStages; ++i)
      mbar_init(&bar.kv_full[i], 1), mbar_init(&bar.kv_empty[i], 2), mbar_init(&bar.v_ok[i], 1);
    mbar_init(&bar.drain, 1);
    bar.abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&p.map_q);
    tma_prefetch_desc(&p.map_k);
    tma_prefetch_desc(&p.map_v);
  }
  if (warp == 8) {
    tmem_alloc(&bar.tmem, 512);
    tmem_relinquish();
  }
  __syncthreads();
  tc_fence_after();
  griddep_wait();
  griddep_launch_dependents();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(&bar.tmem);
  const PreWait wc{&bar.abort_flag, static_cast<uint32_t>(min(p.timeout_ns, 0xFFFFFFFFull))};

  // The tile that descriptor k (counted per CTA) describes; false when there is none or a wait gave up.
  auto get_tile = [&](int k, PrefillTile& t) -> bool {
    if (!pre_wait(&bar.tile_full[k % kPreRing], (k / kPreRing) & 1, wc, W_PRE_TILE_FULL)) return false;
    const volatile PrefillTile& s = bar.tile[k % kPreRing];
    t.row0 = s.row0, t.len = s.len, t.tok0 = s.tok0, t.n0 = s.n0, t.n1 = s.n1, t.head0 = s.head0, t.kvh = s.kvh;
    return t.len > 0;
  };
  auto first_masked = [&](const PrefillTile& t) { return p.causal ? (t.tok0 + 1) / kPreTile : t.len / kPreTile; };

  if (warp >= 8) {
  fewer_registers<kPreRegsOther>();
  if (warp == 10) {
    // ================================================================ tiles
    const int tpc = 2 * p.tq;
    // Tiers: sequences have blocks [0, blocks) of tpc tokens.  Causal: block j costs about j, tier j is block j of
    // each sequence that has one.  Full mask: a block costs as much as its sequence has key tiles, tier j is all
    // blocks of the sequences with j + 1 key tiles.  Flat: all blocks are one tier in the order of the sequences, so
    // that there is one walk over the sequences instead of one a tier.
    auto length_of = [&](int b) {
      int first, last;
      sequence_rows(p.cu, b, p.seq_len, p.M, first, last);
      return last - first;
    };
    const int tier_len = p.causal ? tpc : kPreTile;
    auto measure = [&](int b, int& reach, int& count) {  // tiers of a sequence, and its blocks
      const int len = b < p.batch ? length_of(b) : 0;
      reach = len > 0 ? (len - 1) / tier_len + 1 : 0;
      count = len > 0 ? (len - 1) / tpc + 1 : 0;
    };
    int my_reach = 0, my_count = 0, tiers = 0;  // of sequence `lane`
    unsigned blocks = 0;
#pragma unroll 1
    for (int b = lane; b < p.batch; b += 32) {
      int reach, count;
      measure(b, reach, count);
      if (b == lane) my_reach = reach, my_count = count;
      tiers = max(tiers, reach);
      blocks += count;
    }
    tiers = __reduce_max_sync(~0u, tiers);
    blocks = __reduce_add_sync(~0u, blocks);
    if (p.flat) tiers = 1;
    int tier = tiers - 1;
    unsigned before = 0;                                     // blocks before sequence `from` of this tier
    int from = 0;                                            // where the last block was found: ranks only rise
    int pair0 = 0, n_pairs = min(p.pairs, p.pairs_at_once);  // the group of heads
    unsigned rank0 = 0;                                      // its first rank (the launch keeps ranks below 2^30)
    bool more = true, long_before = false;
    for (int k = 0; more; ++k) {
      if (!warp_wait(&bar.tile_empty[k % kPreRing], ((k / kPreRing) & 1) ^ 1, wc, W_PRE_TILE_EMPTY)) break;
      // behind a long tile the next one is only taken once the tile before it is done: it goes to who is free
      if (k >= 2 && long_before &&
          !warp_wait(&bar.tile_empty[(k - 2) % kPreRing], ((k - 2) / kPreRing) & 1, wc, W_PRE_TILE_EMPTY))
        break;
      unsigned taken = 0;
      if (k > 0 && lane == 0) taken = atomicAdd(p.work, 1u);
      const unsigned rank = k == 0 ? cta : G + __shfl_sync(~0u, taken, 0);
      while (rank >= rank0 + blocks * n_pairs && pair0 + n_pairs < p.pairs) {  // on to the next group
        rank0 += blocks * n_pairs;
        pair0 += n_pairs;
        n_pairs = min(p.pairs - pair0, p.pairs_at_once);
        tier = tiers - 1, before = 0, from = 0;
      }
      const unsigned block = (rank - rank0) / n_pairs;
      const int pair = pair0 + static_cast<int>(rank - rank0 - block * n_pairs);
      // the tier, and in it the sequence, that holds this block: `in` of it
      int seq = -1, in = 0;
#pragma unroll 1
      while (tier >= 0) {
#pragma unroll 1
        for (; from < p.batch; from += 32) {
          int reach = my_reach, count = my_count;
          if (from > 0) measure(from + lane, reach, count);
          const unsigned have = p.flat ? count : p.causal ? reach > tier : reach == tier + 1 ? count : 0;
          const unsigned all = __reduce_add_sync(~0u, have);
          if (block < before + all) {
            unsigned sum = have;  // inclusive sum over the lanes
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
              const unsigned y = __shfl_up_sync(~0u, sum, o);
              if (lane >= o) sum += y;
            }
            const int src = __ffs(__ballot_sync(~0u, before + sum > block)) - 1;
            seq = from + src;
            in = static_cast<int>(block - before - __shfl_sync(~0u, sum - have, src));
            break;
          }
          before += all;
        }
        if (seq >= 0) break;
        from = 0;
        --tier;
      }
      PrefillTile t = {};
      t.bad_lo = INT_MAX, t.bad_hi = -1;
      more = seq >= 0;
      if (more) {
        int first, last;
        sequence_rows(p.cu, seq, p.seq_len, p.M, first, last);
        t.row0 = first;
        t.len = last - first;
        t.tok0 = (!p.causal ? in : p.flat ? (t.len - 1) / tpc - in : tier) * tpc;
        const int packs = p.group / p.hp;
        t.kvh = pair / packs;
        t.head0 = t.kvh * p.group + (pair - t.kvh * packs) * p.hp;
        const int all = (t.len - 1) / kPreTile + 1;
        // tokens [tok0, tok0 + tq) and [tok0 + tq, tok0 + 2 tq), cut off at the sequence's end
        t.n0 = p.causal ? (min(t.tok0 + p.tq, t.len) - 1) / kPreTile + 1 : all;
        t.n1 = t.tok0 + p.tq >= t.len ? 0 : p.causal ? (min(t.tok0 + tpc, t.len) - 1) / kPreTile + 1 : all;
        long_before = max(t.n0, t.n1) >= 4;
      }
      if (lane == 0) {
        bar.tile[k % kPreRing] = t;
        mbar_arrive(&bar.tile_full[k % kPreRing]);
      }
      __syncwarp();
    }
    // Counted on every way out, also where a wait gave up, so that the next launch finds the counters at zero.
    if (lane == 0 && atomicAdd(p.work + 1, 1u) == static_cast<unsigned>(G) - 1) {
      p.work[0] = 0;  // every CTA has taken its last tile
      p.work[1] = 0;
    }
  } else if (warp == 9) {
    // ================================================================ TMA loads
    if (lane == 0) {
      int fills = 0;
      PrefillTile t = {}, next = {};
      uint32_t q_phase = 0;  // a bit for each query tile
      bool q_used[2] = {false, false}, ok = true, more = get_tile(0, next);
      // Stage after stage: key tile i of the current unit's V (none before the first unit), and the K tile behind it,
      // of the same unit or, at its end, the first of the next one, whose queries follow.
#pragma unroll 1
      for (int k = -1, i = 0, n = 1; ok; ++i) {
        const bool last = i == n - 1;
        if (k >= 0 && last) more = get_tile(k + 1, next);
        const bool has_v = k >= 0, has_k = !last || more;
        if (!has_v && !has_k) break;
        const int st = fills & 1;
        if (!(ok = pre_wait(&bar.kv_empty[st], ((fills >> 1) & 1) ^ 1, wc, W_PRE_KV_EMPTY))) break;
        mbar_arrive_expect_tx(&bar.kv_full[st], (has_v + has_k) * kPreTileBytes);
        ++fills;
        const int v_row = t.row0 + i * kPreTile, v_col = t.kvh * kHeadDim;
        const int k_row = last ? next.row0 : v_row + kPreTile, k_col = last ? next.kvh * kHeadDim : v_col;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          uint8_t* to = smem + (2 + 2 * st) * kPreTileBytes + h * (kPreTileBytes / 2);
          if (has_v) tma_load_2d(&p.map_v, &bar.kv_full[st], to, v_col + h * 64, v_row);
          if (has_k) tma_load_2d(&p.map_k, &bar.kv_full[st], to + kPreTileBytes, k_col + h * 64, k_row);
        }
        if (!last) continue;
        if (!more) break;
#pragma unroll 1
        for (int s = 0; s < 2; ++s) {
          if ((s ? next.n1 : next.n0) == 0) continue;
          if (!(ok = pre_wait(&bar.q_empty[s], ((q_phase >> s) & 1) ^ 1, wc, W_PRE_Q_EMPTY))) break;
          q_phase ^= 1u << s;
          q_used[0] |= s == 0, q_used[1] |= s == 1;
          mbar_arrive_expect_tx(&bar.q_full[s], static_cast<uint32_t>(p.hp * p.tq * kHeadDim * 2));
#pragma unroll 1
          for (int h = 0; h < 2; ++h)
            tma_load_3d(&p.map_q, &bar.q_full[s], q_smem + s * kPreTileBytes + h * (kPreTileBytes / 2), h * 64, next.head0,
                        next.row0 + next.tok0 + s * p.tq);
        }
        mbar_arrive(&bar.tile_empty[(k + 1) % kPreRing]);
        t = next;
        ++k;
        i = -1;
        n = max(t.n0, t.n1);
      }
      if (bar.abort_flag) {  // leave no copy in flight
        if (q_used[0]) mbar_wait_quiet(&bar.q_full[0], (q_phase & 1) ^ 1, kPreDrainNs);
        if (q_used[1]) mbar_wait_quiet(&bar.q_full[1], ((q_phase >> 1) & 1) ^ 1, kPreDrainNs);
        for (int i = max(0, fills - T::kStages); i < fills; ++i)
          mbar_wait_quiet(&bar.kv_full[i & 1], (i >> 1) & 1, kPreDrainNs);
      }
    }
    __syncwarp();
  } else if (warp == 8) {
    // ================================================================ MMA issue
    // The whole warp walks the loop, so that descriptors stay in uniform registers, and one elected lane issues.
    constexpr uint32_t kF16 = FP8 ? (1u << 7) | (1u << 10) : 0u;  // P and V: without these bits they are fp16
    constexpr uint32_t idesc_qk = idesc_bf16_f32(kPreTile, kPreTile),
                       idesc_pv = idesc_bf16_f32(kPreTile, kHeadDim, true) & ~kF16;
    constexpr uint32_t kStep16 = kPreTileBytes / 16;  // one tile in descriptor units
    const bool one = elect_one();
    const uint64_t q_desc = sdesc_k_sw128(q_smem), k_desc = sdesc_k_sw128(kv_smem + kPreTileBytes),
                   v_desc = sdesc_mn_sw128(kv_smem, kPreTileBytes / 2);
    uint32_t q_phase = 0, p_phase = 0, v_phase = 0;  // a bit for each barrier
    uint32_t uses = 0;                               // stages waited for: the next one is (uses & 1)
    // Lanes wait on their own and agree once a step: after a wait that gave up, what is still issued works on the
    // CTA's own memory and its results are not used.
    bool ok = true;
    auto wait = [&](uint64_t* b, uint32_t parity, int where) { ok = pre_wait(b, parity, wc, where) && ok; };
    auto stage_wait = [&]() {
      wait(&bar.kv_full[uses & 1], (uses >> 1) & 1, W_PRE_KV_FULL);
      ++uses;
    };
    auto q_wait = [&](int s) {
      wait(&bar.q_full[s], (q_phase >> s) & 1, W_PRE_Q_FULL);
      q_phase ^= 1u << s;
    };
    auto p_wait = [&](int s) {
      wait(&bar.p_full[s], (p_phase >> s) & 1, W_PRE_P);
      p_phase ^= 1u << s;
      tc_fence_after();
    };
    auto qk = [&](int s, int st, bool last) {  // S_s = Q_s K^T
      if (one) {
        const uint64_t ad = q_desc + s * kStep16, bd = k_desc + st * (2 * kStep16);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_bf16(tmem + s * kPreTile, ad + (k >> 2) * (kStep16 / 2) + (k & 3) * 2,
                   bd + (k >> 2) * (kStep16 / 2) + (k & 3) * 2, idesc_qk, k != 0);
        mma_commit(&bar.s_full[s]);
        if (last) mma_commit(&bar.q_empty[s]);
      }
      __syncwarp();
    };
    auto pv = [&](int s, int st, bool first, bool last) {  // O_s (+)= P_s V; E4M3: += always, the softmax warps begin O
      if (one) {
        const uint64_t bd = v_desc + st * (2 * kStep16);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          mma_bf16_ts(tmem + 256 + s * kHeadDim, tmem + s * kPreTile + k * 8, bd + k * 128, idesc_pv, FP8 || !first || k != 0);
        if (last) mma_commit(&bar.o_full[s]);
      }
      __syncwarp();
    };
    PrefillTile t, u = {};
    bool more = __all_sync(~0u, get_tile(0, t));
    if (more) {
      if (one) mbar_arrive(&bar.tile_empty[0]);
      stage_wait();
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int ns = s ? t.n1 : t.n0;
        if (ns > 0) {
          q_wait(s);
          qk(s, 0, ns == 1);
        }
      }
      if (one) mma_commit(&bar.kv_empty[0]);
      stage_wait();
    }
    // The queue behind the tensor cores holds about three instructions (some 190 cycles), so between two products
    // stands one wait at most: the one for a P before its PV, the one for the next stage before the second QK.
    for (int k = 0; more && (ok = __all_sync(~0u, ok)); ++k) {
      const int n = max(t.n0, t.n1), mask0 = first_masked(t);
      const int plain = min(min(t.n0, t.n1) - 1, mask0);  // steps without a mask that both query tiles go on behind
      int i = 0;
#pragma unroll 1
      for (; i < plain; ++i) {
        const int st = (uses - 1) & 1;
        p_wait(0);
        pv(0, st, i == 0, false);
        qk(0, st, i + 2 == t.n0);
        p_wait(1);
        pv(1, st, i == 0, false);
        stage_wait();
        qk(1, st, i + 2 == t.n1);
        if (one) mma_commit(&bar.kv_empty[st]);
        ok = __all_sync(~0u, ok);
        if (!ok) break;
      }
#pragma unroll 1
      for (; i < n && ok; ++i) {
        const bool last = i == n - 1;
        if (last) {
          more = __all_sync(~0u, get_tile(k + 1, u));
          if (more && one) mbar_arrive(&bar.tile_empty[(k + 1) % kPreRing]);
        }
        const bool next = !last || more;  // another key tile, of this unit of work or the next
        const int st = (uses - 1) & 1;
        if (i >= mask0) {
          wait(&bar.v_ok[st], (v_phase >> st) & 1, W_PRE_V);
          v_phase ^= 1u << st;
        }
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          const int ns = s ? t.n1 : t.n0, un = s ? u.n1 : u.n0;
          if (i < ns) {
            p_wait(s);
            pv(s, st, i == 0, i == ns - 1);
          }
          if (s == 1 && next) stage_wait();
          if (last ? more && un > 0 : i + 1 < ns) {
            if (last) q_wait(s);
            qk(s, st, last ? un == 1 : i + 1 == ns - 1);
          }
        }
        if (one) mma_commit(&bar.kv_empty[st]);
        ok = __all_sync(~0u, ok);
      }
      t = u;
    }
    if (one) {
      mma_commit(&bar.drain);  // nothing of this CTA's products or their arrivals is left behind
      mbar_wait_quiet(&bar.drain, 0, kPreDrainNs);
    }
    __syncwarp();
  } else if (warp == 11) {
    // ================================================================ V of masked tiles: finite values only
    PrefillTile t;
    int fills = 1;  // the first holds a K tile only
    bool ok = true;
    for (int k = 0; ok && __all_sync(~0u, get_tile(k, t)); ++k) {
      if (k == 0) {
        if (!(ok = warp_wait(&bar.kv_full[0], 0, wc, W_PRE_KV_FULL))) break;
        if (lane == 0) mbar_arrive(&bar.kv_empty[0]);
      }
      const int n = max(t.n0, t.n1);
      const int mask0 = first_masked(t);
      // Every fill of the ring passes here in order (a parity says nothing about older or newer phases), so
      // a stage is only free once this warp has seen it, too.
      for (int i = 0; i < n; ++i, ++fills) {
        const int st = fills & 1;
        if (!(ok = warp_wait(&bar.kv_full[st], (fills >> 1) & 1, wc, W_PRE_KV_FULL))) break;
        if (i < mask0) {
          if (lane == 0) mbar_arrive(&bar.kv_empty[st]);
          continue;
        }
        const uint32_t base = kv_smem + st * 2 * kPreTileBytes + lane * 16;
        uint32_t seen[4] = {0, 0, 0, 0};  // sums of 0 * v: NaN once a v is not finite
#pragma unroll 8
        for (int c = 0; c < kPreTileBytes / 512; ++c) {
          const uint4 w = ld_shared_v4(base + c * 512);
          seen[0] = times_zero<FP8>(w.x, seen[0]), seen[1] = times_zero<FP8>(w.y, seen[1]);
          seen[2] = times_zero<FP8>(w.z, seen[2]), seen[3] = times_zero<FP8>(w.w, seen[3]);
        }
        if (__any_sync(~0u, ((seen[0] | seen[1] | seen[2] | seen[3]) & 0x7FFF7FFFu) != 0)) {
          int lo = INT_MAX, hi = -1;
          bool bad_chunk = false;
          auto clean = [&](uint32_t w) {  // an exponent of all ones carries into the sign's place
            constexpr uint32_t kExp = FP8 ? 0x7C007C00u : 0x7F807F80u, kOne = FP8 ? 0x04000400u : 0x00800080u;
            const uint32_t bad = ((w & kExp) + kOne) & 0x80008000u;
            bad_chunk |= bad != 0;
            return w & ~((bad >> 15) * 0xFFFFu);
          };
#pragma unroll 1
          for (int c = 0; c < kPreTileBytes / 512; ++c) {
            const uint4 w = ld_shared_v4(base + c * 512);
            bad_chunk = false;
            st_shared_v4(base + c * 512, clean(w.x), clean(w.y), clean(w.z), clean(w.w));
            const int pos = i * kPreTile + (c & 31) * 4 + (lane >> 3);  // half a key's values are 128 bytes
            if (bad_chunk && pos < t.len) lo = min(lo, pos), hi = max(hi, pos);
          }
          lo = __reduce_min_sync(~0u, lo), hi = __reduce_max_sync(~0u, hi);
          if (lane == 0) {
            PrefillTile& to = bar.tile[k % kPreRing];
            to.bad_lo = min(to.bad_lo, lo), to.bad_hi = max(to.bad_hi, hi);
          }
          fence_async_smem();
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.v_ok[st]), mbar_arrive(&bar.kv_empty[st]);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.tile_empty[k % kPreRing]);
    }
  }
  } else {
    more_registers<kPreRegsSoftmax>();
    // ================================================================ softmax of query tile s, and its output
    const int s = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_tmem = tmem + lanes + s * kPreTile, o_tmem = tmem + lanes + 256 + s * kHeadDim;
    const uint32_t hp_inverse = 65536u / p.hp + 1;  // row / hp = row * hp_inverse >> 16 for rows below 128
    const int row_tok = row / p.hp;
    const float c = p.scale_log2;
    auto load_powers = [&](const PrefillTile& t, int n, int i) {
      const long long tile = i + lane;
      return tile < n ? p.powers[(t.row0 + tile * kPreTile) * p.n_kv + t.kvh] : 0.f;
    };
    // E4M3: the single keys of a tile, in fp32 from their codes and scales: into l and O, and out of S.  O is complete: S
    // of this tile was committed behind the products before.
    auto single_keys = [&](const PrefillTile& t, int i, bool first_too, int lim, float& m, float& mx, float& l, bool& begun) {
      const long long key0 = t.row0 + static_cast<long long>(i) * kPreTile;
      const int keys = min(kPreTile, t.len - i * kPreTile);
      uint32_t which[4], scales[4];  // of key 32 h + lane
      float mark[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) {  // all loads on their way together
        const long long at = key0 + min(h * 32 + lane, keys - 1);
        mark[h] = p.powers[at * p.n_kv + t.kvh];
        scales[h] = __float_as_uint(p.v_scale[at * p.ld_scale + t.kvh]);
      }
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int j = h * 32 + lane;
        which[h] = __ballot_sync(~0u, j == 0 ? first_too : j < keys && mark[h] != 0.f);
      }
      tmem_st_wait();  // O may have been begun just now
      float zero_top = -INFINITY;  // of the logits of keys whose values are zero: O learns of them once, behind the last key
#pragma unroll 1
      for (int j = 0; j <= kPreTile; ++j) {
        const bool end = j == kPreTile;
        uint32_t bits = 0;
        float x = zero_top;
        bool sees = false;
        if (end) {
          if (!begun) m = fmaxf(m, zero_top + kPreZero);  // O is zero yet
          if (!__any_sync(~0u, zero_top + kPreZero > m)) break;
        } else {
          const int h = j >> 5;
          const uint32_t w = (h < 2 ? (h == 0 ? which[0] : which[1]) : (h == 2 ? which[2] : which[3])) >> (j & 31);
          if (w == 0) j |= 31;
          if ((w & 1u) == 0) continue;
          bits = __shfl_sync(~0u, h < 2 ? (h == 0 ? scales[0] : scales[1]) : (h == 2 ? scales[2] : scales[3]), j & 31);
          const float logit = tmem_ld1(s_tmem + j) * c;
          tmem_st1(s_tmem + j, -INFINITY);
          sees = i * kPreTile + j <= lim;
          x = sees ? logit : -INFINITY;
          const float up_l = fmaxf(mx, x);
          l = l * ex2(mx - up_l) + ex2(x - up_l);
          mx = up_l;
          if (bits << 1 == 0) {
            zero_top = fmaxf(zero_top, x);
            continue;
          }
        }
        const uint8_t* from = p.codes + (key0 + (end ? 0 : j)) * p.ld_codes + t.kvh * kHeadDim;
        uint4 codes = *reinterpret_cast<const uint4*>(from);
        const int power = max((static_cast<int>(bits >> 23) & 255) - (127 + kPreRoom), -120);
        // m rises by 2^kPrePowerMax at most, for l's sake: fp32 has room for weights of 2^98 (and for 2^(m - mx) from
        // 2^-125 on)
        const float lift = end ? kPreZero : static_cast<float>(min(max(power, -110), kPrePowerMax));
        const float up = fmaxf(m, x + lift), down = ex2(m - up);
        const float weight = ex2((x + static_cast<float>(power)) - (up - kPreLift));
        const float scale = __uint_as_float(bits) * __uint_as_float(static_cast<uint32_t>(127 - power) << 23);
#pragma unroll 2
        for (int d = 0; d < kHeadDim; d += 16) {
          uint32_t o[16];
          tmem_ld16(o_tmem + d, o);
          const uint32_t four[4] = {codes.x, codes.y, codes.z, codes.w};
          if (d + 16 < kHeadDim) codes = *reinterpret_cast<const uint4*>(from + d + 16);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            uint32_t two;
            asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(two) : "h"(static_cast<uint16_t>(four[e >> 1] >> ((e & 1) * 16))));
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&two));
            float y0 = __uint_as_float(o[e * 2]) * down, y1 = __uint_as_float(o[e * 2 + 1]) * down;
            if (sees) y0 = fmaf(weight, f.x * scale, y0), y1 = fmaf(weight, f.y * scale, y1);  // a NaN only for who sees it
            o[e * 2] = __float_as_uint(y0), o[e * 2 + 1] = __float_as_uint(y1);
          }
          tmem_st16(o_tmem + d, o);
        }
        tmem_st_wait();
        m = up;
        begun = true;
      }
      tmem_st_wait();
    };
    float powers_next = 0.f;
    int s_uses = 0, o_uses = 0;
    bool ok = true;
    PrefillTile t = {}, next;
    for (int k = -1; ok; ++k) {  // unit -1 is there for what precedes the first one
      const int n = s ? t.n1 : t.n0, first = t.tok0 + s * p.tq;
      const int tok = first + row_tok;
      const int lim = p.causal ? min(tok, t.len - 1) : t.len - 1;  // last key this row sees
      const int lim_lo = __reduce_min_sync(~0u, lim);              // last key that every row of this warp sees
      float m = kPreNone, l = 0.f;
      float mx = kPreNone;         // E4M3: the maximum that l is held at (m is that of O)
      float powers = powers_next;  // E4M3: of key tile i in lane i % 32
      if (FP8 && n > 0) {  // O begins here, for what single keys bring to it ahead of the first product
        uint32_t none[16] = {0};
#pragma unroll
        for (int j = 0; j < 8; ++j) tmem_st16(o_tmem + j * 16, none);
      }
      int i = 0, single_done = -1;
      bool begun = false;  // E4M3: single keys are in O (it may be before the first product)
      for (;;) {
        for (; i < n; ++i) {
          if (FP8 && i > 0 && (i & 31) == 0) powers = load_powers(t, n, i);
          float b = FP8 ? __shfl_sync(~0u, powers, i & 31) : 0.f;
          if (FP8 && b > kPreMark / 2) {
            if (i != single_done) break;  // its single keys come first, behind this loop: in it they cost 3 % of the time
            b -= rintf(b / kPreMark) * kPreMark;
          }
          if (!(ok = warp_wait(&bar.s_full[s], s_uses & 1, wc, W_PRE_S))) break;
          ++s_uses;
          tc_fence_after();
          uint32_t x[4][32];
#pragma unroll
          for (int j = 0; j < 4; ++j) tmem_ld32(s_tmem + j * 32, x[j]);
          tmem_ld_wait();
          if (i * kPreTile + kPreTile - 1 > lim_lo) {
            const int cols = lim - i * kPreTile, all = lim_lo - i * kPreTile;  // columns up to these count
#pragma unroll
            for (int h = 0; h < 4; ++h)
              if (h * 32 + 31 > all) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                  if (h * 32 + j > cols) x[h][j] = __float_as_uint(-INFINITY);
              }
          }
          float t4[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) t4[j] = __uint_as_float(x[j][0]);
#pragma unroll
          for (int j = 1; j < 31; j += 2)
#pragma unroll
            for (int h = 0; h < 4; ++h)
              t4[h] = max3(t4[h], __uint_as_float(x[h][j]), __uint_as_float(x[h][j + 1]));
#pragma unroll
          for (int h = 0; h < 4; ++h) t4[h] = fmaxf(t4[h], __uint_as_float(x[h][31]));
          const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * c, lifted = FP8 ? top + b : top;
          const bool rise = lifted > m + kPreLazy, rise_l = FP8 && top > mx + kPreLazy;
          if (__any_sync(~0u, rise || rise_l)) {
            const float up = rise ? lifted : m;
            const float down = ex2(m - up);
            m = up;
            if (FP8) {
              const float up_l = rise_l ? top : mx;
              l *= ex2(mx - up_l);
              mx = up_l;
            } else {
              l *= down;
            }
            if (i > 0 || (FP8 && begun)) {  // O of the key tiles before is complete: S of this one was committed behind it
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                uint32_t o[16];
                tmem_ld16(o_tmem + j * 16, o);
                tmem_ld_wait();
#pragma unroll
                for (int h = 0; h < 16; ++h) o[h] = __float_as_uint(__uint_as_float(o[h]) * down);
                tmem_st16(o_tmem + j * 16, o);
              }
            }
          }
          const float at = FP8 && b == kPreZero ? mx : m - b;  // E4M3: what the tile's weights are held at, 2^7 above
          const float minus = FP8 ? kPreLift - at : -m;
          const uint64_t c2 = f2(c, c), m2 = f2(minus, minus);
          uint64_t l0 = 0, l1 = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t w[16];
#pragma unroll
            for (int h = 0; h < 16; h += 2) {
              float w0, w1, w2, w3;
              f2_split(f2_fma(f2(__uint_as_float(x[j][h * 2]), __uint_as_float(x[j][h * 2 + 1])), c2, m2), w0, w1);
              f2_split(f2_fma(f2(__uint_as_float(x[j][h * 2 + 2]), __uint_as_float(x[j][h * 2 + 3])), c2, m2), w2, w3);
              w0 = ex2(w0), w1 = ex2(w1), w2 = ex2(w2), w3 = ex2(w3);
              l0 = f2_add(l0, f2(w0, w1)), l1 = f2_add(l1, f2(w2, w3));
              w[h] = FP8 ? pack_f16x2(w0, w1) : pack_bf16x2(w0, w1);
              w[h + 1] = FP8 ? pack_f16x2(w2, w3) : pack_bf16x2(w2, w3);
            }
            tmem_st16(s_tmem + j * 16, w);
          }
          float s0, s1, s2, s3;
          f2_split(l0, s0, s1);
          f2_split(l1, s2, s3);
          l += FP8 ? ((s0 + s1) + (s2 + s3)) * ex2((at - kPreLift) - mx) : (s0 + s1) + (s2 + s3);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.p_full[s]);
        }
        if (!FP8 || !ok || i >= n) break;
        if (!(ok = warp_wait(&bar.s_full[s], s_uses & 1, wc, W_PRE_S))) break;  // the loop waits for the same phase again
        tc_fence_after();
        const int marks = __float2int_rn(__shfl_sync(~0u, powers, i & 31) / kPreMark);
        begun |= i > 0;
        single_keys(t, i, (marks & PRE_SINGLE_FIRST) != 0, lim, m, mx, l, begun);
        single_done = i;
      }
      if (!ok) break;
      const bool have = __all_sync(~0u, get_tile(k + 1, next));
      if (FP8 && have) powers_next = load_powers(next, s ? next.n1 : next.n0, 0);
      if (n > 0) {
        if (!(ok = warp_wait(&bar.o_full[s], o_uses & 1, wc, W_PRE_O))) break;
        ++o_uses;
        tc_fence_after();
        const float inv = (FP8 ? ex2((m - kPreLift) - mx) : 1.f) / l;  // E4M3: O is held at m - 7, l at mx
        const volatile PrefillTile& said = bar.tile[k % kPreRing];
        const int bad_lo = said.bad_lo, bad_hi = said.bad_hi;
        // A thread has a row; lines of global memory want a few rows each, all of 128 bytes.  So 16-byte pieces go
        // through shared memory, piece j of row r at place j ^ (r's low bits).  (Stored straight from the row's
        // thread, each instruction touched 32 lines: 4000 cycles a tile.)
        constexpr int kPieces = T::kOutCols / 8, kRowsPer = 32 / kPieces, kSwizzle = kPieces - 1;
        const uint32_t out = smem_u32(smem) + kOutAt + warp * (32 * T::kOutCols * 2);
        const int piece = lane % kPieces;
        // rows lane / kPieces, + kRowsPer, ... of the warp's: their token and head step by step
        const int r_first = lane / kPieces, at_first = (warp & 3) * 32 + r_first;
        const int tok_first = static_cast<int>((at_first * hp_inverse) >> 16), head_first = at_first - tok_first * p.hp;
        const int d_tok = kRowsPer / p.hp, d_head = kRowsPer - d_tok * p.hp;
        const long long d_off = d_tok * p.ldo + d_head * kHeadDim, d_wrap = p.ldo - static_cast<long long>(p.hp) * kHeadDim;
        const int toks = min(p.tq, t.len - first);
        __nv_bfloat16* dst = p.O + static_cast<long long>(t.row0 + first + tok_first) * p.ldo +
                             static_cast<long long>(t.head0 + head_first) * kHeadDim + piece * 8;
#pragma unroll 1
        for (int j = 0; j < kHeadDim; j += T::kOutCols) {
#pragma unroll
          for (int h = 0; h < T::kOutCols; h += 32) {
            uint32_t o[32];
            tmem_ld32(o_tmem + j + h, o);
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                w[e] = pack_bf16x2(__uint_as_float(o[q * 8 + e * 2]) * inv, __uint_as_float(o[q * 8 + e * 2 + 1]) * inv);
              st_shared_v4(out + lane * (T::kOutCols * 2) + (((h >> 3) + q) ^ (lane & kSwizzle)) * 16, w[0], w[1], w[2], w[3]);
            }
          }
          __syncwarp();
          __nv_bfloat16* to = dst + j;
          int at_tok = tok_first, at_head = head_first;
#pragma unroll
          for (int r0 = 0; r0 < 32; r0 += kRowsPer) {
            const int r = r_first + r0;
            const uint4 w = ld_shared_v4(out + r * (T::kOutCols * 2) + (piece ^ (r & kSwizzle)) * 16);
            if (at_tok < toks) *reinterpret_cast<uint4*>(to) = w;
            at_tok += d_tok, at_head += d_head, to += d_off;
            if (at_head >= p.hp) at_head -= p.hp, ++at_tok, to += d_wrap;
          }
          __syncwarp();
        }
        tc_fence_before();
        if (bad_lo <= min(bad_hi, lim) && row_tok < p.tq && tok < t.len) {
          // Values of V that are not finite were taken out for the rows that do not see them.  The others get their
          // sum (infinite or NaN), whatever the finite rest is.
          const __nv_bfloat16* v = p.V + static_cast<long long>(t.row0) * p.ldv + static_cast<long long>(t.kvh) * kHeadDim;
          __nv_bfloat16* mine = p.O + static_cast<long long>(t.row0 + tok) * p.ldo +
                                static_cast<long long>(t.head0 + row - row_tok * p.hp) * kHeadDim;
#pragma unroll 1
          for (int d = 0; d < kHeadDim; ++d) {
            float sum = 0.f;
#pragma unroll 1
            for (int pos = bad_lo; pos <= min(bad_hi, lim); ++pos) {
              const __nv_bfloat16 raw = v[static_cast<long long>(pos) * p.ldv + d];
              const float y = FP8 ? __half2float(__ushort_as_half(__bfloat16_as_ushort(raw))) : __bfloat162float(raw);
              if (!isfinite(y)) sum += y;
            }
            if (!isfinite(sum)) mine[d] = __float2bfloat16_rn(sum);
          }
        }
      }
      __syncwarp();
      if (k >= 0 && lane == 0) mbar_arrive(&bar.tile_empty[k % kPreRing]);
      if (!have) break;
      t = next;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_dealloc(tmem, 512);
  if (threadIdx.x == 0 && bar.abort_flag != 0) record_failure(p.status, bar.abort_flag, 0);
}

// E4M3 codes of K and V times their scales, for the kernel above: K as bf16, V as fp16 times 2^-b, with b for each key
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
