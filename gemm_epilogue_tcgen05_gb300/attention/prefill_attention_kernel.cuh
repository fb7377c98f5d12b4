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
// Window (WIN, causal).  Queries are the last tokens of their sequence's keys, which have offsets of their own, and row i sees
// the keys of the last `window` tokens and the first `sinks`.  A unit of work goes over a stream of keys: whole chunks of 32
// that hold the sinks, then the keys from the chunk on that holds the first key its first row sees.  So a key tile is four
// such chunks, loaded as one box where they follow one another and as four in the tile in which the sinks end; E4M3 has a
// power for each (below).  Any tile may be masked.  The blocks of a long prompt cost the same, so they come in the order of
// the sequences.  8192 tokens, a window of 1024 and 4 sinks, 32/8 heads, bf16: 105 us, 1230 TFLOP/s of what the rows see, 9
// key tiles for 64 tokens at the tensor cores' pace and 1.7 us between units.  (Tiles at multiples of 128 keys, the sinks with
// one of their own: 116 us.)
//
// Parts (CUT, WIN).  Few units over many keys (a prompt's next part behind thousands of tokens) leave SMs idle: then a unit's
// stream is cut into parts of 6 key tiles and more, each a unit for itself, whose O, m and l go to a scratch buffer as they are,
// and a second kernel joins them in their order.  A kernel of its own: the mere presence of this code cost E4M3 6 %.
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
constexpr int kPrePartTiles = 6;                   // CUT: key tiles of a part, at least
// A part: of query tiles 0 and 1 O [32 float4][128 rows], then m, mx and l of each row.
constexpr int kPrePartRows = kPreTile * (kHeadDim + 3), kPrePartFloats = 2 * kPrePartRows;
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

// Of a unit's first part: what the join needs; `parts` 0 in the others and where nothing is to be joined.
struct alignas(16) PrefillCut {
  int parts[2], step;  // of query tiles 0 and 1, and how far apart their numbers are
  int row, tokens;     // row of the first token, and how many there are
  int head0, unused[2];
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
  CUtensorMap map_k32, map_v32;  // WIN: the same as map_k and map_v, box {64, 32}
  const int* cu_k;               // WIN: offsets of the keys' rows, of which there are M_k; null: those of the queries
  int M_k, window, sinks;        // WIN; a window of 0 hides nothing
  int most_parts, numbers;       // CUT: numbers that a unit has, and how many there is room for
  float* parts;                  // CUT: [numbers][kPrePartFloats]
  PrefillCut* cuts;              // CUT: [numbers], and in front of them one whose `step` says how many there are
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

struct PrefillJoinParams {
  const float* parts;
  const PrefillCut* cuts;
  int hp, tq;
  __nv_bfloat16* O;
  long long ldo;
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
  int row0, len;   // the sequence's first row of keys, and their number (WIN: it may be none)
  int tok0;        // first token of query tile 0 (query tile 1: + tq), as a position
  int n0, n1;      // key tiles that query tiles 0 and 1 meet
  int head0, kvh;
  int q_row0;          // WIN: row of position 0, as if the queries began there
  int k0, sink_keys;   // WIN: place P of the stream is key P below sink_keys, else k0 + P - sink_keys
  int place0, part;    // CUT: where in the stream the part begins, and its number, -1 for a whole unit
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
// The n lowest bits: none for n below 1, all for more than 31.
__device__ __forceinline__ uint32_t bits_below(int n) {
  uint32_t r;
  asm("shr.u32 %0, %1, %2;" : "=r"(r) : "r"(~0u), "r"(32 - min(max(n, 0), 32)));  // a shift by 32 leaves nothing
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
template <bool FP8, bool WIN, bool CUT = false>
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
    if (WIN) {
      t.q_row0 = s.q_row0, t.k0 = s.k0, t.sink_keys = s.sink_keys;
      if (CUT) t.place0 = s.place0;
      return CUT ? max(t.n0, t.n1) > 0 : t.n0 > 0;  // a tile may have no keys
    }
    return t.len > 0;
  };
  auto first_masked = [&](const PrefillTile& t) { return p.causal ? (t.tok0 + 1) / kPreTile : t.len / kPreTile; };
  // First key of chunk h of a unit's i-th key tile; WIN: and whether all rows see all of the tile, a run of keys.
  auto key_of = [&](const PrefillTile& t, int i, int h) {
    if (!WIN) return i * kPreTile + h * 32;
    const int place = (CUT ? t.place0 : 0) + i * kPreTile + h * 32;
    return place < t.sink_keys ? place : place + t.k0 - t.sink_keys;
  };
  auto run_of_keys = [&](const PrefillTile& t, int i) {
    const int place = (CUT ? t.place0 : 0) + i * kPreTile;
    return !WIN || place >= t.sink_keys || place + kPreTile <= t.sink_keys;
  };
  auto plain_tile = [&](const PrefillTile& t, int i) {
    const int first = key_of(t, i, 0), last = first + kPreTile - 1;
    return run_of_keys(t, i) && last <= t.tok0 && (p.window == 0 || last < p.sinks || first > t.tok0 + 2 * p.tq - 1 - p.window);
  };

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
    // WIN: the stream of the block that begins at position tok0, of a sequence with len_k keys.
    auto stream_of = [&](int tok0, int len_k, PrefillTile& t) {
      const int from = (tok0 - p.window + 1) & ~31, sink_keys = static_cast<int>((static_cast<unsigned>(p.sinks) + 31u) & ~31u);
      const bool gap = p.window > 0 && tok0 - p.window + 1 > 0 && from > sink_keys;
      t.k0 = gap ? from : 0, t.sink_keys = gap ? sink_keys : 0;
      // tiles that end at the last key of query tiles 0 and 1; rows in front of the first key (or without any) have one
      auto tiles = [&](int end) { return max((t.sink_keys + min(end, len_k) - t.k0 - 1) / kPreTile + 1, 1); };
      t.n0 = tiles(tok0 + p.tq);
      t.n1 = tok0 + p.tq >= len_k ? 0 : tiles(tok0 + tpc);
    };
    int parts_here = CUT ? p.most_parts : 1;
    auto measure = [&](int b, int& reach, int& count) {  // tiers of a sequence, and its blocks
      const int len = b < p.batch ? length_of(b) : 0;
      reach = len > 0 ? (len - 1) / tier_len + 1 : 0;
      count = len > 0 ? (len - 1) / tpc + 1 : 0;
      if (CUT) count *= parts_here;
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
    if (CUT && static_cast<unsigned long long>(blocks) * p.pairs > static_cast<unsigned>(p.numbers)) {
      // offsets that give rows to several sequences: more units than rows can make, and they stay whole
      blocks /= parts_here, my_count /= parts_here;
      parts_here = 1;
    }
    if (p.flat) tiers = 1;
    int tier = tiers - 1;
    unsigned before = 0;                                     // blocks before sequence `from` of this tier
    int from = 0;                                            // where the last block was found: ranks only rise
    int pair0 = 0, n_pairs = min(p.pairs, p.pairs_at_once);  // the group of heads
    unsigned rank0 = 0;                                      // its first rank (the launch keeps ranks below 2^30)
    bool more = true, long_before = false, ok = true, again = false;  // again, CUT: a number that stands for nothing
    if (CUT && cta == 0 && lane == 0) p.cuts[0].step = parts_here > 1 ? static_cast<int>(blocks * p.pairs) : 0;
    for (int k = 0; more; ++k) {
      ok = ok && warp_wait(&bar.tile_empty[k % kPreRing], ((k / kPreRing) & 1) ^ 1, wc, W_PRE_TILE_EMPTY);
      // behind a long tile the next one is only taken once the tile before it is done: it goes to who is free
      if (k >= 2 && long_before)
        ok = ok && warp_wait(&bar.tile_empty[(k - 2) % kPreRing], ((k - 2) / kPreRing) & 1, wc, W_PRE_TILE_EMPTY);
      if (!CUT && !ok) break;  // CUT: all numbers are taken, so that the join knows what each is
      unsigned taken = 0;
      if ((k > 0 || again) && lane == 0) taken = atomicAdd(p.work, 1u);
      const unsigned rank = k == 0 && !again ? cta : G + __shfl_sync(~0u, taken, 0);
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
      PrefillCut cut = {};
      t.bad_lo = INT_MAX, t.bad_hi = -1;
      more = seq >= 0;
      again = false;
      if (more) {
        int first, last;
        sequence_rows(p.cu, seq, p.seq_len, p.M, first, last);
        t.row0 = first;
        t.len = last - first;
        const int part = CUT ? in % parts_here : 0;
        if (CUT) in /= parts_here;
        t.tok0 = (!p.causal ? in : p.flat ? (t.len - 1) / tpc - in : tier) * tpc;
        if (WIN) {
          int first_k = first, last_k = last;
          if (p.cu_k != nullptr) sequence_rows(p.cu_k, seq, 0, p.M_k, first_k, last_k);
          const int shift = (last_k - first_k) - t.len;  // position of the first query
          t.row0 = first_k, t.len = last_k - first_k;
          t.q_row0 = first - shift;
          t.tok0 += shift;
          stream_of(t.tok0, t.len, t);
        }
        if (CUT) {
          // part i of c: tiles n i / c .. n (i + 1) / c - 1; query tile s takes part in those that begin before its last key
          const int n = max(t.n0, t.n1), c = min(parts_here, (n - 1) / kPrePartTiles + 1);
          const int begin = static_cast<int>(static_cast<long long>(n) * part / c),
                    end = static_cast<int>(static_cast<long long>(n) * (part + 1) / c);
          auto taking_part = [&](int own) { return own > 0 ? static_cast<int>((static_cast<long long>(own) * c - 1) / n) + 1 : 0; };
          again = part >= c;
          t.place0 = begin * kPreTile;
          t.part = c > 1 ? static_cast<int>(rank) : -1;
          if (c > 1 && part == 0) {
            cut.parts[0] = taking_part(t.n0), cut.parts[1] = taking_part(t.n1), cut.step = n_pairs;
            cut.row = t.q_row0 + t.tok0, cut.tokens = t.len - t.tok0;
          }
          t.n0 = min(max(t.n0 - begin, 0), end - begin), t.n1 = min(max(t.n1 - begin, 0), end - begin);
        }
        const int packs = p.group / p.hp;
        t.kvh = pair / packs;
        t.head0 = t.kvh * p.group + (pair - t.kvh * packs) * p.hp;
        const int all = (t.len - 1) / kPreTile + 1;
        // tokens [tok0, tok0 + tq) and [tok0 + tq, tok0 + 2 tq), cut off at the sequence's end
        if (!WIN) {
          t.n0 = p.causal ? (min(t.tok0 + p.tq, t.len) - 1) / kPreTile + 1 : all;
          t.n1 = t.tok0 + p.tq >= t.len ? 0 : p.causal ? (min(t.tok0 + tpc, t.len) - 1) / kPreTile + 1 : all;
        }
        if (CUT && parts_here > 1 && lane == 0) {
          cut.head0 = t.head0;
          p.cuts[1 + rank] = cut;
        }
        if (CUT && again) {
          --k;  // the next number in its place
          continue;
        }
        long_before = max(t.n0, t.n1) >= 4;
      }
      if (ok && lane == 0) {
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
        const int v_col = t.kvh * kHeadDim, k_col = last ? next.kvh * kHeadDim : v_col;
        if (WIN) {
          auto load = [&](const CUtensorMap& whole, const CUtensorMap& part, const PrefillTile& from, int tile, int col, int at) {
            const bool run = run_of_keys(from, tile);
#pragma unroll 1
            for (int j = 0; j < (run ? 2 : 8); ++j) {  // halves of 64 dimensions, or their chunks of 32 keys
              const int h = run ? j : j >> 2, c = run ? 0 : j & 3;
              tma_load_2d(run ? &whole : &part, &bar.kv_full[st], smem + at + h * (kPreTileBytes / 2) + c * (32 * 128),
                          col + h * 64, from.row0 + key_of(from, tile, c));
            }
          };
          const int at = (2 + 2 * st) * kPreTileBytes;
          if (has_v) load(p.map_v, p.map_v32, t, i, v_col, at);
          if (has_k) load(p.map_k, p.map_k32, last ? next : t, last ? 0 : i + 1, k_col, at + kPreTileBytes);
        } else {
          const int v_row = t.row0 + i * kPreTile, k_row = last ? next.row0 : v_row + kPreTile;
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            uint8_t* to = smem + (2 + 2 * st) * kPreTileBytes + h * (kPreTileBytes / 2);
            if (has_v) tma_load_2d(&p.map_v, &bar.kv_full[st], to, v_col + h * 64, v_row);
            if (has_k) tma_load_2d(&p.map_k, &bar.kv_full[st], to + kPreTileBytes, k_col + h * 64, k_row);
          }
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
                        (WIN ? next.q_row0 : next.row0) + next.tok0 + s * p.tq);
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
      for (;;) {
        // steps that wait for no cleaned V (with a window bf16 gains 1.5 % by this loop, E4M3 loses 4 %)
#pragma unroll 1
        for (; WIN ? !FP8 && i < min(t.n0, t.n1) - 1 && plain_tile(t, i) : i < plain; ++i) {
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
        for (const int end = WIN && !FP8 ? min(i + 1, n) : n; i < end && ok; ++i) {
          const bool last = i == n - 1;
          if (last) {
            more = __all_sync(~0u, get_tile(k + 1, u));
            if (more && one) mbar_arrive(&bar.tile_empty[(k + 1) % kPreRing]);
          }
          const bool next = !last || more;  // another key tile, of this unit of work or the next
          const int st = (uses - 1) & 1;
          if (WIN ? !plain_tile(t, i) : i >= mask0) {
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
        if (i >= n || !ok) break;
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
        if (WIN ? plain_tile(t, i) : i < mask0) {
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
            const int pos = key_of(t, i, (c & 31) >> 3) + (c & 7) * 4 + (lane >> 3);  // half a key's values are 128 bytes
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
    // E4M3: of key tile i + lane, WIN: of chunk lane % 4 of key tile i + lane / 4; and how many tiles that is.
    constexpr int kPowers = WIN ? 8 : 32;
    auto load_powers = [&](const PrefillTile& t, int n, int i) {
      if (WIN) {
        const int tile = i + (lane >> 2), key = key_of(t, tile, lane & 3) & ~(kPreTile - 1);
        return tile < n && key < t.len ? p.powers[(t.row0 + static_cast<long long>(key)) * p.n_kv + t.kvh] : 0.f;
      }
      const long long tile = i + lane;
      return tile < n ? p.powers[(t.row0 + tile * kPreTile) * p.n_kv + t.kvh] : 0.f;
    };
    // E4M3: the single keys of a tile, in fp32 from their codes and scales: into l and O, and out of S.  O is complete: S
    // of this tile was committed behind the products before.
    auto single_keys = [&](const PrefillTile& t, int i, float powers, int lim, int low, float& m, float& mx, float& l,
                           bool& begun) {
      uint32_t which[4], scales[4];  // of key 32 h + lane
      float mark[4];
#pragma unroll
      for (int h = 0; h < 4; ++h) {  // all loads on their way together
        const long long at = t.row0 + static_cast<long long>(min(key_of(t, i, h) + lane, t.len - 1));
        mark[h] = p.powers[at * p.n_kv + t.kvh];
        scales[h] = __float_as_uint(p.v_scale[at * p.ld_scale + t.kvh]);
      }
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int key = key_of(t, i, h) + lane;
        const int marks = __float2int_rn(__shfl_sync(~0u, powers, WIN ? (i % kPowers) * 4 + h : i & 31) / kPreMark);
        const bool first = key % kPreTile == 0, single = first ? (marks & PRE_SINGLE_FIRST) != 0 : marks != 0 && mark[h] != 0.f;
        which[h] = __ballot_sync(~0u, key < t.len && single);
      }
      tmem_st_wait();  // O may have been begun just now
      float zero_top = -INFINITY;  // of the logits of keys whose values are zero: O learns of them once, behind the last key
#pragma unroll 1
      for (int j = 0; j <= kPreTile; ++j) {
        const bool end = j == kPreTile;
        uint32_t bits = 0;
        int from = key_of(t, i, 0);
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
          const int key = key_of(t, i, h) + (j & 31);
          sees = key <= lim && (!WIN || key >= low || key < p.sinks);
          from = key;
          x = sees ? logit : -INFINITY;
          const float up_l = fmaxf(mx, x);
          l = l * ex2(mx - up_l) + ex2(x - up_l);
          mx = up_l;
          if (bits << 1 == 0) {
            zero_top = fmaxf(zero_top, x);
            continue;
          }
        }
        const uint8_t* codes_at = p.codes + (t.row0 + static_cast<long long>(from)) * p.ld_codes + t.kvh * kHeadDim;
        uint4 codes = *reinterpret_cast<const uint4*>(codes_at);
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
          if (d + 16 < kHeadDim) codes = *reinterpret_cast<const uint4*>(codes_at + d + 16);
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
      const int low = WIN && p.window > 0 ? tok - p.window + 1 : 0;  // first key of this row's window
      const int low_hi = WIN ? __reduce_max_sync(~0u, low) : 0;     // from here on every row sees (up to lim_lo)
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
          if (FP8 && i > 0 && i % kPowers == 0) powers = load_powers(t, n, i);
          float b = FP8 && !WIN ? __shfl_sync(~0u, powers, i & 31) : 0.f;
          float b4[4] = {b, b, b, b};  // WIN: of each chunk
          if (FP8 && WIN) {
#pragma unroll
            for (int h = 0; h < 4; ++h) b4[h] = __shfl_sync(~0u, powers, (i % kPowers) * 4 + h);
            if (fmaxf(fmaxf(b4[0], b4[1]), fmaxf(b4[2], b4[3])) > kPreMark / 2) {
              if (i != single_done) break;
#pragma unroll
              for (int h = 0; h < 4; ++h)
                if (b4[h] > kPreMark / 2) b4[h] -= rintf(b4[h] / kPreMark) * kPreMark;
            }
          }
          if (FP8 && !WIN && b > kPreMark / 2) {
            if (i != single_done) break;  // its single keys come first, behind this loop: in it they cost 3 % of the time
            b -= rintf(b / kPreMark) * kPreMark;
          }
          if (!(ok = warp_wait(&bar.s_full[s], s_uses & 1, wc, W_PRE_S))) break;
          ++s_uses;
          tc_fence_after();
          if (WIN) {
            // Where a row does not see all of a chunk, S gets its -inf in tensor memory: few chunks do.  (Masks of the registers
            // below cost more, taken or not: 118-180 us for 107, by how their branches are written.)
            const int first_key = key_of(t, i, 0), last_key = key_of(t, i, 3) + 31;
            if (last_key > lim_lo || (first_key < low_hi && last_key >= p.sinks)) {
#pragma unroll 1
              for (int h = 0; h < 4; ++h) {
                const int key0 = key_of(t, i, h);
                if (key0 + 31 <= lim_lo && (key0 >= low_hi || key0 + 31 < p.sinks)) continue;
                const uint32_t seen = bits_below(lim + 1 - key0) & (~bits_below(low - key0) | bits_below(p.sinks - key0));
                uint32_t y[2][16];
#pragma unroll
                for (int q = 0; q < 2; ++q) tmem_ld16(s_tmem + h * 32 + q * 16, y[q]);
                tmem_ld_wait();
#pragma unroll
                for (int q = 0; q < 2; ++q) {
#pragma unroll
                  for (int j = 0; j < 16; ++j)
                    if ((seen & (1u << (q * 16 + j))) == 0) y[q][j] = __float_as_uint(-INFINITY);
                  tmem_st16(s_tmem + h * 32 + q * 16, y[q]);
                }
              }
              tmem_st_wait();
            }
          }
          uint32_t x[4][32];
#pragma unroll
          for (int j = 0; j < 4; ++j) tmem_ld32(s_tmem + j * 32, x[j]);
          tmem_ld_wait();
          if (!WIN && i * kPreTile + kPreTile - 1 > lim_lo) {
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
          const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * c;
          float lifted = FP8 ? top + b : top;
          if (FP8 && WIN)
            lifted = fmaxf(fmaxf(fmaf(t4[0], c, b4[0]), fmaf(t4[1], c, b4[1])),
                           fmaxf(fmaf(t4[2], c, b4[2]), fmaf(t4[3], c, b4[3])));
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
          // E4M3: what the tile's (WIN: a chunk's) weights are held at, 2^7 above
          auto held_at = [&](float power) { return FP8 && power == kPreZero ? mx : m - power; };
          const float at = held_at(b);
          const float minus = FP8 ? kPreLift - at : -m;
          const uint64_t c2 = f2(c, c), m2 = f2(minus, minus);
          uint64_t l0 = 0, l1 = 0;
          float chunks = 0.f;  // E4M3, WIN: their sums
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t w[16];
            const float at4 = held_at(b4[j]);
            const uint64_t m4 = FP8 && WIN ? f2(kPreLift - at4, kPreLift - at4) : m2;
            if (FP8 && WIN) l0 = l1 = 0;
#pragma unroll
            for (int h = 0; h < 16; h += 2) {
              float w0, w1, w2, w3;
              f2_split(f2_fma(f2(__uint_as_float(x[j][h * 2]), __uint_as_float(x[j][h * 2 + 1])), c2, m4), w0, w1);
              f2_split(f2_fma(f2(__uint_as_float(x[j][h * 2 + 2]), __uint_as_float(x[j][h * 2 + 3])), c2, m4), w2, w3);
              w0 = ex2(w0), w1 = ex2(w1), w2 = ex2(w2), w3 = ex2(w3);
              l0 = f2_add(l0, f2(w0, w1)), l1 = f2_add(l1, f2(w2, w3));
              w[h] = FP8 ? pack_f16x2(w0, w1) : pack_bf16x2(w0, w1);
              w[h + 1] = FP8 ? pack_f16x2(w2, w3) : pack_bf16x2(w2, w3);
            }
            tmem_st16(s_tmem + j * 16, w);
            if (FP8 && WIN) {
              float s0, s1, s2, s3;
              f2_split(l0, s0, s1);
              f2_split(l1, s2, s3);
              chunks += ((s0 + s1) + (s2 + s3)) * ex2((at4 - kPreLift) - mx);
            }
          }
          float s0, s1, s2, s3;
          f2_split(l0, s0, s1);
          f2_split(l1, s2, s3);
          if (FP8 && WIN) l += chunks;
          else l += FP8 ? ((s0 + s1) + (s2 + s3)) * ex2((at - kPreLift) - mx) : (s0 + s1) + (s2 + s3);
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.p_full[s]);
        }
        if (!FP8 || !ok || i >= n) break;
        if (!(ok = warp_wait(&bar.s_full[s], s_uses & 1, wc, W_PRE_S))) break;  // the loop waits for the same phase again
        tc_fence_after();
        begun |= i > 0;
        single_keys(t, i, powers, lim, low, m, mx, l, begun);
        single_done = i;
      }
      if (!ok) break;
      const bool have = __all_sync(~0u, get_tile(k + 1, next));
      if (FP8 && have) powers_next = load_powers(next, s ? next.n1 : next.n0, 0);
      if (n > 0) {
        if (!(ok = warp_wait(&bar.o_full[s], o_uses & 1, wc, W_PRE_O))) break;
        ++o_uses;
        tc_fence_after();
        const volatile PrefillTile& said = bar.tile[k % kPreRing];
        const int bad_lo = said.bad_lo, bad_hi = said.bad_hi;
        const int number = CUT ? said.part : -1;
        float* own_part = nullptr;  // CUT: where this row's columns go as they are
        if (CUT && number >= 0) {
          float* at = p.parts + static_cast<long long>(number) * kPrePartFloats + s * kPrePartRows;
          own_part = at + row * 4;
          at += kPreTile * kHeadDim + row;
          at[0] = m, at[kPreTile] = mx, at[2 * kPreTile] = l;
#pragma unroll 1
          for (int d = 0; d < kHeadDim; d += 16) {
            uint32_t o[16];
            tmem_ld16(o_tmem + d, o);
            tmem_ld_wait();
#pragma unroll
            for (int h = 0; h < 16; h += 4)
              *reinterpret_cast<uint4*>(own_part + (d + h) * kPreTile) = make_uint4(o[h], o[h + 1], o[h + 2], o[h + 3]);
          }
        }
        float inv = (FP8 ? ex2((m - kPreLift) - mx) : 1.f) / l;  // E4M3: O is held at m - 7, l at mx
        if (WIN && l == 0.f) inv = 0.f;  // a row that sees nothing
        const uint64_t inv2 = f2(inv, inv);
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
        const int row_zero = WIN ? t.q_row0 : t.row0;
        __nv_bfloat16* dst = p.O + static_cast<long long>(row_zero + first + tok_first) * p.ldo +
                             static_cast<long long>(t.head0 + head_first) * kHeadDim + piece * 8;
#pragma unroll 1
        for (int j = CUT && number >= 0 ? kHeadDim : 0; j < kHeadDim; j += T::kOutCols) {
#pragma unroll
          for (int h = 0; h < T::kOutCols; h += 32) {
            uint32_t o[32];
            tmem_ld32(o_tmem + j + h, o);
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              uint32_t w[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                float a, b;
                f2_split(f2_mul(f2(__uint_as_float(o[q * 8 + e * 2]), __uint_as_float(o[q * 8 + e * 2 + 1])), inv2), a, b);
                w[e] = pack_bf16x2(a, b);
              }
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
          __nv_bfloat16* mine = p.O + static_cast<long long>(row_zero + tok) * p.ldo +
                                static_cast<long long>(t.head0 + row - row_tok * p.hp) * kHeadDim;
#pragma unroll 1
          for (int d = 0; d < kHeadDim; ++d) {
            float sum = 0.f;
#pragma unroll 1
            for (int pos = bad_lo; pos <= min(bad_hi, lim); ++pos) {
              if (WIN && pos < low && pos >= p.sinks) {  // on to the window
                pos = min(low, bad_hi + 1) - 1;
                continue;
              }
              const __nv_bfloat16 raw = v[static_cast<long long>(pos) * p.ldv + d];
              const float y = FP8 ? __half2float(__ushort_as_half(__bfloat16_as_ushort(raw))) : __bfloat162float(raw);
              if (!isfinite(y)) sum += y;
            }
            if (isfinite(sum)) continue;
            if (CUT && number >= 0) own_part[(d >> 2) * (4 * kPreTile) + (d & 3)] = sum;
            else mine[d] = __float2bfloat16_rn(sum);
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

// The parts of units, in their order: blocks (number, query tile, quarter of the columns) of a thread for each row.  A value that
// is not finite counts as it is, whatever the weight of its part.
template <bool FP8>
__global__ void __launch_bounds__(kPreTile) attention_prefill_join_kernel(const __grid_constant__ PrefillJoinParams p) {
  griddep_wait();
  const int number = blockIdx.x, s = blockIdx.y, d0 = blockIdx.z * 32, row = threadIdx.x;
  if (number >= p.cuts[0].step) return;
  const PrefillCut cut = p.cuts[1 + number];
  const int parts = cut.parts[s], row_tok = row / p.hp, tok = s * p.tq + row_tok;
  if (parts == 0 || row_tok >= p.tq || tok >= cut.tokens) return;
  const float* first = p.parts + static_cast<long long>(number) * kPrePartFloats + s * kPrePartRows;
  const long long apart = static_cast<long long>(cut.step) * kPrePartFloats;
  float m = kPreNone, mx = kPreNone, l = 0.f;
  for (int i = 0; i < parts; ++i) {
    const float* at = first + i * apart + kPreTile * kHeadDim + row;
    m = fmaxf(m, at[0]);
    if (FP8) mx = fmaxf(mx, at[kPreTile]);
  }
  float o[32];
#pragma unroll
  for (int h = 0; h < 32; ++h) o[h] = 0.f;
#pragma unroll 1
  for (int i = 0; i < parts; ++i) {
    const float* at = first + i * apart;
    const float* own = at + kPreTile * kHeadDim + row;
    const float down = ex2(own[0] - m);
    l += own[2 * kPreTile] * (FP8 ? ex2(own[kPreTile] - mx) : down);
    float4 v[8];
#pragma unroll
    for (int h = 0; h < 8; ++h) v[h] = *reinterpret_cast<const float4*>(at + (d0 + h * 4) * kPreTile + row * 4);
#pragma unroll
    for (int h = 0; h < 8; ++h) {
      o[h * 4] = isfinite(v[h].x) ? fmaf(v[h].x, down, o[h * 4]) : o[h * 4] + v[h].x;
      o[h * 4 + 1] = isfinite(v[h].y) ? fmaf(v[h].y, down, o[h * 4 + 1]) : o[h * 4 + 1] + v[h].y;
      o[h * 4 + 2] = isfinite(v[h].z) ? fmaf(v[h].z, down, o[h * 4 + 2]) : o[h * 4 + 2] + v[h].z;
      o[h * 4 + 3] = isfinite(v[h].w) ? fmaf(v[h].w, down, o[h * 4 + 3]) : o[h * 4 + 3] + v[h].w;
    }
  }
  float inv = (FP8 ? ex2((m - kPreLift) - mx) : 1.f) / l;
  if (l == 0.f) inv = 0.f;  // a row that sees nothing
  __nv_bfloat16* to = p.O + static_cast<long long>(cut.row + tok) * p.ldo +
                      static_cast<long long>(cut.head0 + row - row_tok * p.hp) * kHeadDim + d0;
#pragma unroll
  for (int h = 0; h < 32; h += 8)
    *reinterpret_cast<uint4*>(to + h) =
        make_uint4(pack_bf16x2(o[h] * inv, o[h + 1] * inv), pack_bf16x2(o[h + 2] * inv, o[h + 3] * inv),
                   pack_bf16x2(o[h + 4] * inv, o[h + 5] * inv), pack_bf16x2(o[h + 6] * inv, o[h + 7] * inv));
}

}  // namespace fl
