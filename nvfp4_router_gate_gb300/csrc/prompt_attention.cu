// prompt_attention.cu -- softmax attention of packed prompts of different lengths
// over their own 16-bit keys and values (sm_103a): prompt_attention.
// Bound by the tensor cores: 4 D flops for every (query, head) and seen token.  Measured (no
// inputs in L2, bursts of some 30 ms): 8192 tokens of 64 heads of 128 channels 656 us, 1676 TFLOP/s, the
// tensor pipe 72 % busy; 2048 over 8192 keys 309 us, 1557; windows of 1024 over two prompts of 8192 451
// us, 1142; ragged prompts of up to 2500 tokens (32 heads) 216 us, 1230; one prompt of 37 tokens 9.1 us.
// After 0.1 s of nothing else the GPU is at its power limit: 705, 326, 469 and 225 us.
//
// Mathematics: as csrc/kv_prefill.cu -- S = Q K^T and O += P V on tcgen05 with 128
// rows (query, head) of an accumulator in tensor memory, a thread a row; the running
// maximum moves in steps, sums and statistics in fp32, the weights P rounded to the
// values' type.
//
// A block (one per SM) takes 256 rows of a sequence that share a KV head as two row
// tiles (qt queries of Gt heads each) and walks the tokens in tiles of 128:
//   warps 0-3, 4-7  softmax of row tile 0 and 1: read S from tensor memory, write P
//                   over it, rescale O when the maximum moves;
//   warps 8-11      the rows out: O from tensor memory, scaled, joined with the prefix,
//                   stored, while the softmax warps are at the next rows already;
//   warps 12, 13    issue the products of row tile 0 and 1, so that one tile's softmax
//                   runs under the other's products;
//   warp 14         walks the work, hands every role its runs and copies their queries,
//                   keys and values into swizzled shared memory (TMA);
//   warp 15         looks tiles with masked tokens over for infinities and NaNs among
//                   the values: a weight of zero would make NaNs of them.  They become
//                   zeros; the rows that see them get them back at the end.
//
// Tensor memory, 512 columns: S0 | S1 (128 each, P over the first half of its
// S), O0 | O1 (D each).  S of the next tile follows P V of this one in issue
// order, so S is never overwritten early and a complete S implies the earlier
// P V complete.  A run's last products and the next run's first ones follow each other
// in the same way: the pipeline does not drain.
//
// Many keys, or short ones, go to the blocks whole, the longest first (kPaEven).  Others are cut
// as in csrc/kv_attention.cu: all keys' tiles end to end in equal chunks, one per block.  Every
// part of a cut key is written, and the warps that come last to their rows join them, in the
// parts' order:
//   m = max m_i,  w_i = 2^(m_i - m),  out = sum w_i O_i / sum w_i l_i.
// Usually that is the key's first part, the last work of its block (a second kernel took
// 24 to 29 us behind all of them).
#include <algorithm>
#include <type_traits>

#include "../../include/nvfp4_prompt.h"
#include "prompt_attention.cuh"

namespace nvr {

namespace {

constexpr int kPaThreads = 512;
constexpr int kPaPlaces = 2;               // places of a tile in the flat order
// Starting and ending a key counts as this many places.  Three ragged prompts of up to 3500 tokens, 8
// heads, 64 us at 2, 57 at 5, 62 at 9; 1100 tokens over 4000 more 62.6, 64.6 and 67.4, 30 sequences of 9
// queries over 3000 keys 37.3, 38.4, 39.5; 8192 tokens of 8 heads 114, 116, 116, 2048 over 8192 keys 308 at all three.
constexpr int kPaKeyCost = 5;
// Fewest places of a block; of a key of n tiles it has sqrt(n) tiles at least: the parts are
// joined one after the other.
constexpr int kPaMinChunk = 4;
// Keys of at most this many tiles are not cut (a block more or less even then): 2571 tokens of 16
// heads 56 us at 12, 35 at 24 and 40; 3000 tokens that see all 164, 155, 155; 8192 tokens of 8 heads
// 116, 117, 124.
constexpr int kPaWhole = 24;
// Fewer where the longest key is more than two of the blocks' chunks, so that most blocks would wait
// for it: 30 queries of four sequences over 2000 keys 29.6 us whole, 24.5 cut; one query over 2900
// 36.9 and 29.4; a prompt of 3000 tokens, 4 heads, 38.1 and 32.5.  Four queries over 1000 keys (8
// tiles) 17.8 whole, 24.8 cut.
constexpr int kPaWholeFew = 9;
// Keys are shared out whole, as blocks have room for them, where none is longer than that; where a
// block gets this many of the longest; and where it gets one of them at least and they are
// three quarters of it on average, as causal prompts' are (the short ones, last, even the blocks
// out).  In place of equal chunks of the flat order: 8192 tokens of 64 heads (7 a block) 691 to 660 us;
// three ragged prompts of 3500 109 to 84, 4096 tokens of 32 heads 123 to 103; short prompts 25.9
// to 21.8; one token to one key a block 0.3 us slower.  2048 queries over 8192 keys (3 a block,
// 56 tiles of 64 on average) are 318 us in chunks, 325 whole.
constexpr int kPaEven = 4;
// A call has fewer places than this: the chunks' borders in the flat order stay below 2^31.
constexpr int kPaMost = INT32_MAX - (1 << 24) + 1;
// So many sequences are passed by, empty, in a third of the time that a role waits for its next run (1 s).
constexpr int kPaMaxB = 1 << 24;
// A block's stretch of a key at most: tiles take up to 2 us, so half of what a role waits for its end.
constexpr int kPaMostTiles = 1 << 18;
constexpr int kRuns = 3;                   // runs handed out ahead
constexpr int kConsumers = 15;             // warps that read a run: all but the one that walks

struct alignas(16) Run {
  int tiles;                               // -1: the end
  int tile0;                               // first tile of the sequence
  int head;                                // head group
  int q0, k0;                              // first query's row, the sequence's first key row
  int n_q, pos0, kmax;                     // queries, position of the first one, keys that exist
  int first[2], last[2];                   // tiles of each row tile: [first, last)
  int free_to, free_from;                  // tiles inside [free_from, free_to) of the tokens are seen by every row
  int parts, part;                         // of its key (1: all of it), which one
  int block, tail;                         // the block of the first part, whether it is in its second slot
  int bad;                                 // values of the run were not finite
  int pad[2];
};

template <int D>
struct PaSmem {
  static constexpr int kTileBytes = kPaTile * D * 2;         // rows in 128-byte swizzled atoms of 64 channels
  static constexpr int kSlots = D == 128 ? 4 : 8;            // tiles of keys and of values, alternately
  static constexpr int kQ = 0;
  static constexpr int kKV = kQ + 2 * kTileBytes;
  static constexpr int kOut = kKV + kSlots * kTileBytes;     // 128 bytes of each row on their way out
  static constexpr int kStat = kOut + kPaTile * 128;         // per row tile and row: m, l
  static constexpr int kRunsAt = kStat + 2 * 2 * kPaTile * 4;
  static constexpr int kFirstAt = kRunsAt + kRuns * static_cast<int>(sizeof(Run));
  static constexpr int kBarAt = kFirstAt + kPaThreads * 4;
  static constexpr int kTotal = kBarAt + (2 * kRuns + 3 * kSlots + 2 * 7 + 1) * 8 + 64 + 1024;
};

// D fp32 (1 in bits 4-5), A and B bf16 (1) or fp16 (0) in bits 7-9 and 10-12, B
// transposed in bit 16, N >> 3 in bits 17-22, M >> 4 in bits 24-28.
template <bool kF16>
__device__ __forceinline__ uint32_t idesc_16(int M, int N, bool b_mn_major) {
  return (1u << 4) | (kF16 ? 0u : (1u << 7) | (1u << 10)) | (b_mn_major ? 1u << 16 : 0u) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// The two words of a matrix descriptor: 128-byte swizzle, 8-row groups 1024 bytes
// apart; the low one holds the address and the distance of 64-channel atoms (used
// by the transposed operand alone).
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(const void* tile, uint32_t atom_distance) {
  return ((smem_u32(tile) & 0x3FFFFu) >> 4) | ((atom_distance >> 4) << 16);
}

// D[tmem] (+)= A[smem] . B[smem]; descriptors by their low words.
__device__ __forceinline__ void tc_mma_ss(uint32_t d_tmem, uint32_t a_low, uint32_t b_low, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}"
      :: "r"(d_tmem), "r"(a_low), "r"(b_low), "r"(idesc), "r"(static_cast<uint32_t>(add)), "r"(kDescHigh)
      : "memory");
}
// The same with A in tensor memory (two 16-bit values of a row to a column).
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_low, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}"
      :: "r"(d_tmem), "r"(a_tmem), "r"(b_low), "r"(idesc), "r"(static_cast<uint32_t>(add)), "r"(kDescHigh)
      : "memory");
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];"
      :: "r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// 16 columns of this warp's lanes without the wait, and the wait: the registers
// pass through it so that nothing reads them early.
__device__ __forceinline__ void tmem_load16_start(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_load16_finish(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :: "memory");
}

// The same of 32 columns.
__device__ __forceinline__ void tmem_load32_start(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_load32_finish(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29])
               :: "memory");
  asm volatile("" : "+r"(r[30]), "+r"(r[31]) :: "memory");
}

// A key's length in the flat order: its tiles, then places without work.
__device__ __forceinline__ int key_cost(const PromptGroup& g) { return g.n > 0 ? kPaPlaces * g.tiles + kPaKeyCost : 0; }

// Zeros, and an lse of -inf, for the rows that no sequence covers: in front of the first
// one, behind the last one (a batch padded for a captured graph), past max_q in one.
template <int D>
__device__ __forceinline__ void clear_rows(const PromptParams& p, int unit, int units) {
  const int lane = threadIdx.x & 31, T = static_cast<int>(p.T);
  auto row_of = [&](int b) { return min(max(__ldg(p.cu_q + b), 0), T); };
  auto clear = [&](int64_t from, int64_t to, int step) {
#pragma unroll 1
    for (int64_t r = from; r < to; r += step) {
      uint4* o = reinterpret_cast<uint4*>(p.out + r * p.Hq * D);
#pragma unroll 1
      for (int i = lane; i < p.Hq * (D / 8); i += 32) o[i] = make_uint4(0u, 0u, 0u, 0u);
      if (!p.lse) continue;
#pragma unroll 1
      for (int i = lane; i < p.Hq; i += 32) p.lse[r * p.Hq + i] = -INFINITY;
    }
  };
  const int first = row_of(0), last = row_of(p.B);
  clear(unit, first, units);
  clear(static_cast<int64_t>(last) + unit, T, units);
#pragma unroll 1
  for (int64_t b0 = static_cast<int64_t>(unit) * 32; b0 < p.B; b0 += static_cast<int64_t>(units) * 32) {
    const int b = static_cast<int>(min(b0 + lane, static_cast<int64_t>(p.B - 1))), a = row_of(b), e = row_of(b + 1);
    uint32_t over = __ballot_sync(0xFFFFFFFFu, b0 + lane < p.B && e - a > p.max_q);
#pragma unroll 1
    for (; over; over &= over - 1) {
      const int l = __ffs(over) - 1;
      clear(static_cast<int64_t>(__shfl_sync(0xFFFFFFFFu, a, l)) + p.max_q, __shfl_sync(0xFFFFFFFFu, e, l), 1);
    }
  }
}

// Where a block's shared memory has what.
template <int D>
struct Block {
  uint8_t* smem;
  Run* s_runs;
  float* s_stat;                           // [row tile][m, l][row]
  uint64_t *run_full, *run_empty, *kv_full, *kv_empty, *v_clean, *q_full, *q_empty;
  uint64_t *s_full, *p_full, *o_full, *o_empty, *stat_full, *drained;
  uint32_t* tmem_holder;
  volatile int* abort_flag;
  int* s_start;                            // item of the chunk's start, offset inside it
  int* s_first;                            // of each thread's share of the items: those with queries before it

  __device__ __forceinline__ Block() {
    using Sm = PaSmem<D>;
    constexpr int NS = Sm::kSlots;
    extern __shared__ uint8_t smem_raw[];
    smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    s_runs = reinterpret_cast<Run*>(smem + Sm::kRunsAt);
    s_stat = reinterpret_cast<float*>(smem + Sm::kStat);
    s_first = reinterpret_cast<int*>(smem + Sm::kFirstAt);
    run_full = reinterpret_cast<uint64_t*>(smem + Sm::kBarAt);
    run_empty = run_full + kRuns;
    kv_full = run_empty + kRuns;
    kv_empty = kv_full + NS;
    v_clean = kv_empty + NS;
    q_full = v_clean + NS;
    q_empty = q_full + 2;
    s_full = q_empty + 2;
    p_full = s_full + 2;
    o_full = p_full + 2;
    o_empty = o_full + 2;
    stat_full = o_empty + 2;
    drained = stat_full + 2;
    tmem_holder = reinterpret_cast<uint32_t*>(drained + 1);
    abort_flag = reinterpret_cast<int*>(tmem_holder) + 1;
    s_start = reinterpret_cast<int*>(tmem_holder) + 2;
  }
};

// One warp of it.
template <int D>
struct Member : Block<D> {
  int lane = threadIdx.x & 31, n_taken = 0;

  __device__ __forceinline__ bool wait_all(uint64_t* bar, uint32_t parity) {
    return __all_sync(0xFFFFFFFFu, wait_bounded(bar, parity, this->abort_flag)) != 0;
  }
  __device__ __forceinline__ void arrive(uint64_t* bar) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  }
  // the next run, or null; its last reader frees it
  __device__ __forceinline__ const volatile Run* take() {
    const int s = n_taken % kRuns;
    if (!wait_all(this->run_full + s, (n_taken / kRuns) & 1)) return nullptr;
    ++n_taken;
    return this->s_runs + s;
  }
  __device__ __forceinline__ void give_back() { arrive(this->run_empty + (n_taken - 1) % kRuns); }
};

// The roles.  False: gave up waiting.
//
// What is not run all the time is bound by fetching its instructions, about 700 clocks for
// eight of them when they come from L2 (measured: 55000 clocks for joining two parts in
// unrolled code), and sixteen warps of six roles share the instruction cache.  So all but the
// inner loop of the softmax and the issue of the products is in loops of few instructions.

// The products, by a warp for each row tile w: neither waits for the other's softmax.  What
// lies between the arrival of P and the issue of the products is the chain that the tensor
// cores wait for: every other wait comes first, and an elected lane of the whole warp issues
// them (descriptors in uniform registers: 256 rows over 128 tokens took 3900 clocks when one
// lane went through all of it by itself, and take 3000).
template <int D, bool kF16>
__device__ __forceinline__ bool products(uint32_t tmem, int w) {
  using Sm = PaSmem<D>;
  constexpr int NS = Sm::kSlots;
  Member<D> me;
  const uint32_t id_s = idesc_16<kF16>(128, kPaTile, false), id_o = idesc_16<kF16>(128, D, true);
  constexpr uint32_t kTileLow = Sm::kTileBytes >> 4;
  const uint32_t q_low = desc_low(me.smem + Sm::kQ, 16) + w * kTileLow;
  const uint32_t k_low = desc_low(me.smem + Sm::kKV, 16), v_low = desc_low(me.smem + Sm::kKV, kPaTile * 128);
  const uint32_t t_s = tmem + w * kPaTile, t_o = tmem + 2 * kPaTile + w * D;
  auto score = [&](int slot) {
    const uint32_t k = k_low + slot * kTileLow;
#pragma unroll
    for (int i = 0; i < D / 16; ++i) {
      const uint32_t o = ((i / 4) * (kPaTile * 128) + (i % 4) * 32) >> 4;
      tc_mma_ss(t_s, q_low + o, k + o, id_s, i != 0);
    }
  };
  auto weigh = [&](int slot, bool add) {
    const uint32_t v = v_low + slot * kTileLow;
#pragma unroll
    for (int i = 0; i < kPaTile / 16; ++i)
      // 16 tokens: two groups of eight 128-byte rows; 64-channel atoms a tile of rows apart
      tc_mma_ts(t_o, t_s + 8 * i, v + (i * 2048 >> 4), id_o, add || i != 0);
  };
  auto have = [&](uint64_t* bar, uint32_t parity) { return me.wait_all(bar, parity); };
  uint32_t ph_q = 0, ph_p = 0, ph_o = 1, clean = 0;    // (bit i of clean: the phase of slot 2 i + 1)
  int n_tile = 0, n_run = 0;                           // tiles whose scores were issued (or passed by), runs taken
  // the tile whose weights come next: 1, 2 its row tile's first, 4 its last one, 8 masked; 16 passed by
  uint32_t prev = 0;
  int j = 0, n = 0, first = 0, last = 0, tile0 = 0, free_from = 0, free_to = 0;
  for (bool more = true; more || prev;) {
    uint32_t cur = 0;
    while (more && j >= n) {
      if (n_run) me.arrive(me.run_empty + (n_run - 1) % kRuns);
      if (!have(me.run_full + n_run % kRuns, (n_run / kRuns) & 1)) return false;
      const volatile Run* run = me.s_runs + n_run % kRuns;
      ++n_run;
      n = run->tiles;
      j = 0;
      if (n < 0) { more = false; break; }
      first = run->first[w]; last = run->last[w];
      tile0 = run->tile0; free_from = run->free_from; free_to = run->free_to;
      // A run without tiles: the weights before it do not wait for the run behind it.  That one may
      // need the slot of theirs, which the rows' way out gives back after their product.
      if (n == 0 && prev) break;
    }
    if (more && j < n) {
      cur = j >= first && j < last ? 1u | (j == first ? 2u : 0u) | (j + 1 == last ? 4u : 0u) : 16u;
      const int t0 = (tile0 + j) * kPaTile;
      if (t0 < free_from || t0 + kPaTile > free_to) cur |= 8u;
      ++j;
    }
    // everything but P first
    const int v_slot = (2 * n_tile - 1 + NS) % NS, k_slot = (2 * n_tile) % NS;
    if (prev) {
      // (passed by as well: a barrier's phases are told apart by their parity alone)
      if (!have(me.kv_full + v_slot, ((2 * n_tile - 1) / NS) & 1)) return false;
      if (prev & 8u) {
        if (!have(me.v_clean + v_slot, (clean >> (v_slot / 2)) & 1u)) return false;
        clean ^= 1u << (v_slot / 2);
      }
      if (prev & 2u) {
        if (!have(me.o_empty + w, ph_o)) return false;
        ph_o ^= 1u;
      }
    }
    if (cur && !have(me.kv_full + k_slot, ((2 * n_tile) / NS) & 1)) return false;
    if (cur & 2u) {
      // (between runs: the last weights do not wait for the next queries)
      if (prev & 1u) {
        if (!have(me.p_full + w, ph_p)) return false;
        ph_p ^= 1u;
        tc_fence_after();
        if (elect_one()) {
          weigh(v_slot, !(prev & 2u));
          if (prev & 4u) tc_commit(me.o_full + w);
        }
        __syncwarp();
      }
      if (!have(me.q_full + w, ph_q)) return false;
      ph_q ^= 1u;
    } else if (prev & 1u) {
      if (!have(me.p_full + w, ph_p)) return false;
      ph_p ^= 1u;
    }
    tc_fence_after();
    if (elect_one()) {
      if ((prev & 1u) && !(cur & 2u)) {
        weigh(v_slot, !(prev & 2u));
        if (prev & 4u) tc_commit(me.o_full + w);
      }
      if (cur & 1u) {
        score(k_slot);
        tc_commit(me.s_full + w);
        if (cur & 4u) tc_commit(me.q_empty + w);
      }
      // (The softmax frees the slots of the tiles that it sees.  A commit more for each costs the
      // tensor cores a pause: with two more 8192 tokens took 768 us, with one 731, without 709.)
      if (cur & 16u) tc_commit(me.kv_empty + k_slot);
    }
    __syncwarp();
    if (cur) ++n_tile;
    prev = cur;
  }
  me.arrive(me.run_empty + (n_run - 1) % kRuns);
  return true;
}

// How a call's keys are shared out: in chunks of the flat order, or whole (keys of them), as blocks
// have room for one.
struct Share {
  bool whole;
  int f0, f1, chunk;
  int uncut;                               // keys of at most this many tiles are not
  int keys;
};

// The walk, and the queries, keys and values of its runs in.
template <int D>
__device__ __forceinline__ bool walk(const PromptParams& p, const Share& share) {
  using Sm = PaSmem<D>;
  constexpr int NS = Sm::kSlots;
  Member<D> me;
  const int n_items = p.B * p.groups;
  uint32_t sent_q[2] = {0, 0};
  int n_load = 0, n_run = 0;
  auto hand_out = [&](const Run& r) {
    const int s = n_run % kRuns;
    if (!me.wait_all(me.run_empty + s, ((n_run / kRuns) & 1) ^ 1)) return false;
    if (me.lane == 0) {
      me.s_runs[s] = r;
      mbar_arrive(me.run_full + s);
    }
    __syncwarp();
    ++n_run;
    return true;
  };
  // Keys go in where keys were, values where values were: those are done with when the next
  // tile's keys are, whose slot is the next one, and when they have been looked over.
  auto tile = [&](const CUtensorMap* map, int head, int row) {
    const int s = n_load % NS;
    if (!me.wait_all(me.kv_empty + s, ((n_load / NS) & 1) ^ 1)) return false;
    if ((s & 1) && n_load >= NS && !me.wait_all(me.kv_empty + (s + 1) % NS, (((n_load + 1) / NS) & 1) ^ 1)) return false;
    if (me.lane == 0) {
      mbar_arrive_expect_tx(me.kv_full + s, Sm::kTileBytes);
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
        tma_load_3d(me.smem + Sm::kKV + s * Sm::kTileBytes + c * (kPaTile * 128), map, 64 * c, head, row, me.kv_full + s);
    }
    __syncwarp();
    ++n_load;
    return true;
  };
  auto queries = [&](const Run& r, int w) {
    if (r.first[w] >= r.last[w]) return true;
    if (!me.wait_all(me.q_empty + w, (sent_q[w] & 1) ^ 1)) return false;
    if (me.lane == 0) {
      mbar_arrive_expect_tx(me.q_full + w, p.Gt * p.qt * D * 2);
#pragma unroll
      for (int c = 0; c < D / 64; ++c)
        tma_load_3d(me.smem + Sm::kQ + w * Sm::kTileBytes + c * (kPaTile * 128), &p.tm_q, 64 * c, r.head * p.Gt,
                    r.q0 + w * p.qt, me.q_full + w);
    }
    __syncwarp();
    ++sent_q[w];
    return true;
  };
  auto copies = [&](const Run& r) {
    const int row0 = r.k0 + r.tile0 * kPaTile, kv_head = r.head / p.chunks;
    for (int j = 0; j < r.tiles; ++j) {
      if (!tile(&p.tm_k, kv_head, row0 + j * kPaTile)) return false;
      if (j == 0 && (!queries(r, 0) || !queries(r, 1))) return false;
      if (!tile(&p.tm_v, kv_head, row0 + j * kPaTile)) return false;
    }
    return true;
  };
  bool ok = true;
  // A key's stretch [from, to) of its places, from place key_f0 of the flat order on: the
  // tiles whose first place is in it.  (Behind the tiles' come places without work.)  The
  // first place of a key of few tiles stands for all of it.
  auto stretch = [&](const PromptGroup& g, int head, int key_f0, int from, int to) {
    const bool uncut = share.whole || g.tiles <= share.uncut;
    const int ta = uncut ? 0 : min((from + kPaPlaces - 1) / kPaPlaces, g.tiles);
    const int tb = uncut ? g.tiles : min((to + kPaPlaces - 1) / kPaPlaces, g.tiles);
    if (uncut ? from > 0 : ta >= tb) return true;
    Run r = {};
    r.tiles = tb - ta;
    r.tile0 = g.tile0 + ta;
    r.head = head;
    r.q0 = g.q0 + g.i0; r.k0 = g.k0;
    r.n_q = g.n; r.pos0 = g.shift + g.i0; r.kmax = g.kmax;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      r.first[w] = min(max(g.first[w] - ta, 0), r.tiles);
      r.last[w] = max(min(g.last[w] - ta, r.tiles), r.first[w]);
    }
    r.free_to = seen_end(p.causal, r.pos0, g.kmax);
    r.free_from = seen_begin(p.window, r.pos0 + g.n - 1);
    r.parts = 1;
    if (!uncut) {
      r.block = key_f0 / share.chunk;
      r.parts = (key_f0 + kPaPlaces * (g.tiles - 1)) / share.chunk - r.block + 1;
      r.part = static_cast<int>(blockIdx.x) - r.block;
      r.tail = key_f0 > r.block * share.chunk;
    }
    return hand_out(r) && copies(r);
  };
  if (share.whole) {
    // The longest come first, so blocks end within a short one of each other.
    const int starters = min(static_cast<int>(gridDim.x), share.keys), per = (n_items + kPaThreads - 1) / kPaThreads;
    int x = blockIdx.x;
    while (x < share.keys && ok) {
      const int rank = x / p.Hv;
      // the thread whose share of the items has it, the item
      int t = 16 * (__popc(__ballot_sync(0xFFFFFFFFu, me.s_first[16 * me.lane] <= rank)) - 1);
      t += __popc(__ballot_sync(0xFFFFFFFFu, me.lane < 16 && me.s_first[t + (me.lane & 15)] <= rank)) - 1;
      int item = t * per;
      if (per > 1) {
        int skip = rank - me.s_first[t];
#pragma unroll 1
        for (;; item += 32) {
          uint32_t some = __ballot_sync(0xFFFFFFFFu, prompt_group(p, min(item + me.lane, n_items - 1)).n > 0);
          const int n = __popc(some);
          if (skip >= n) {
            skip -= n;
            continue;
          }
#pragma unroll 1
          for (; skip; --skip) some &= some - 1;
          item += __ffs(some) - 1;
          break;
        }
      }
      int next = 0;
      if (me.lane == 0) next = starters + static_cast<int>(atomicAdd(p.handed, 1u));
      ok = stretch(prompt_group(p, item), x - rank * p.Hv, 0, 0, 0);
      // (a key is handed out for each that was done: the last of those that are none)
      if (me.lane == 0 && next == starters + share.keys - 1) *p.handed = 0;
      x = __shfl_sync(0xFFFFFFFFu, next, 0);
    }
  } else {
    int item = me.s_start[0], off = me.s_start[1], f = share.f0;
    PromptGroup next = prompt_group(p, item);
    for (; f < share.f1 && ok; ++item) {
      if (next.n == 0) {
        // (Groups without queries 32 at a time.  Between those of a long sequence lie up to 2 B of them,
        // and the other roles' waits are bounded: 5000 tokens among 4096 empty sequences 1280 us one by one
        // and 230 so, among 262144 78 and 11 ms, most of it to find the blocks' shares.)
        const uint32_t some = __ballot_sync(0xFFFFFFFFu, prompt_group(p, min(item + me.lane, n_items - 1)).n > 0);
        item += some ? __ffs(some) - 1 : 31;
        next = prompt_group(p, min(some ? item : item + 1, n_items - 1));
        if (!some) continue;
      }
      const PromptGroup g = next;
      next = prompt_group(p, min(item + 1, n_items - 1));
      const int cost = key_cost(g);
      while (off < cost * p.Hv && f < share.f1 && ok) {
        const int head = off / cost, at = off - head * cost, n = min(cost - at, share.f1 - f);
        ok = stretch(g, head, f - at, at, at + n);
        off += n;
        f += n;
      }
      off = 0;
    }
  }
  if (ok) {
    Run r = {};
    r.tiles = -1;
    ok = hand_out(r);
  }
  if (!ok || *me.abort_flag) {
    // copies in flight land before the block's memory goes away
    const uint64_t drain = globaltimer_ns() + 1000000000ull;
    for (int i = max(n_load - NS, 0); i < n_load; ++i)
      while (!mbar_try_wait(me.kv_full + i % NS, (i / NS) & 1))
        if (globaltimer_ns() > drain) break;
    for (int w = 0; w < 2; ++w)
      while (sent_q[w] && !mbar_try_wait(me.q_full + w, (sent_q[w] - 1) & 1))
        if (globaltimer_ns() > drain) break;
  }
  return ok;
}

// Values that are not finite, in tiles with masked tokens: to zeros.
template <int D, bool kF16>
__device__ __forceinline__ bool look_over() {
  using Sm = PaSmem<D>;
  constexpr int NS = Sm::kSlots;
  Member<D> me;
  constexpr uint32_t kExp = kF16 ? 0x7C007C00u : 0x7F807F80u;
  int n_tile = 0;
  for (;;) {
    const volatile Run* run = me.take();
    if (!run) return false;
    const int n = run->tiles;
    if (n < 0) break;
    for (int j = 0; j < n; ++j, ++n_tile) {
      const int t0 = (run->tile0 + j) * kPaTile, s = (2 * n_tile + 1) % NS;
      // (every tile in turn: a barrier's phases are told apart by their parity alone)
      if (!me.wait_all(me.kv_full + s, ((2 * n_tile + 1) / NS) & 1)) return false;
      if (t0 >= run->free_from && t0 + kPaTile <= run->free_to) {
        me.arrive(me.kv_empty + s);
        continue;
      }
      uint4* tile = reinterpret_cast<uint4*>(me.smem + Sm::kKV + s * Sm::kTileBytes);
      // A half whose exponent is all ones leaves its top bit clear below
      uint32_t finite = 0x80008000u;
#pragma unroll 8
      for (int i = me.lane; i < Sm::kTileBytes / 16; i += 32) {
        const uint4 u = tile[i];
        finite &= (~u.x & kExp) + kExp;
        finite &= (~u.y & kExp) + kExp;
        finite &= (~u.z & kExp) + kExp;
        finite &= (~u.w & kExp) + kExp;
      }
      if (__any_sync(0xFFFFFFFFu, finite != 0x80008000u)) {
        for (int i = me.lane; i < Sm::kTileBytes / 16; i += 32) {
          uint4 u = tile[i];
          uint32_t* x = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if ((x[k] & kExp & 0xFFFFu) == (kExp & 0xFFFFu)) x[k] &= 0xFFFF0000u;
            if ((x[k] & kExp & 0xFFFF0000u) == (kExp & 0xFFFF0000u)) x[k] &= 0xFFFFu;
          }
          tile[i] = u;
        }
        if (me.lane == 0) const_cast<volatile Run*>(run)->bad = 1;
      }
      fence_proxy_async_smem();
      me.arrive(me.v_clean + s);
      me.arrive(me.kv_empty + s);
    }
    me.give_back();
  }
  me.give_back();
  return true;
}

// The rows out.
template <int D, bool kF16, bool kPrefix>
__device__ __forceinline__ bool rows_out(const PromptParams& p, uint32_t tmem) {
  using Sm = PaSmem<D>;
  Member<D> me;
  const int wl = (threadIdx.x >> 5) & 3, row = threadIdx.x & 127;
  const uint32_t lanes = static_cast<uint32_t>(wl * 32) << 16;
  const int iq = row / p.Gt, g = row - iq * p.Gt;
  uint8_t* rows_at = me.smem + Sm::kOut + wl * 32 * 128;
  uint32_t ph[2] = {0, 0};
  auto put_vector = [&](int i, uint4 v) {
    *reinterpret_cast<uint4*>(rows_at + me.lane * 128 + (((i ^ me.lane) & 7) << 4)) = v;
  };
  for (;;) {
    const volatile Run* run = me.take();
    if (!run) return false;
    if (run->tiles < 0) break;
    if (kPrefix && run->parts == 1) {
      // (read behind the run's last product)
#pragma unroll 1
      for (int w = 0; w < 2; ++w) {
        const int dq = w * p.qt + iq;
        if (iq >= p.qt || dq >= run->n_q) continue;
        const int64_t at = (static_cast<int64_t>(run->q0 + dq) * p.Hq + run->head * p.Gt + g) * D;
#pragma unroll
        for (int c = 0; c < D; c += 64) asm volatile("prefetch.global.L2 [%0];" :: "l"(p.prefix_out + at + c));
      }
    }
    for (int w = 0; w < 2; ++w) {
      const int dq = w * p.qt + iq;                  // the row's query in the group
      const bool on = iq < p.qt && dq < run->n_q;
      if (w * p.qt >= run->n_q) continue;
      const bool any = run->first[w] < run->last[w];
      const uint32_t rows_on = __ballot_sync(0xFFFFFFFFu, on);
      const uint32_t t_o = tmem + lanes + 2 * kPaTile + w * D;
      const int64_t out_row = static_cast<int64_t>(run->q0 + (on ? dq : 0)) * p.Hq + run->head * p.Gt + (on ? g : 0);
      const float z_before = kPrefix && on ? p.prefix_lse[out_row] : -INFINITY;
      // 32 channels of the rows' prefix to where the results leave from, 16 bytes a lane of every eighth row
      auto piece = [&](int u, int r, int v) { return rows_at + (u & 1) * 2048 + r * 64 + (((v ^ (r >> 1)) & 3) << 4); };
      auto fetch = [&](int u) {
        if (u < D / 32) {
          const uint8_t* in = reinterpret_cast<const uint8_t*>(p.prefix_out) + u * 64 + (me.lane % 4) * 16;
#pragma unroll
          for (int r = me.lane / 4; r < 32; r += 8) {
            const int64_t from = __shfl_sync(0xFFFFFFFFu, out_row, r);
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;"
                         :: "r"(smem_u32(piece(u, r, me.lane % 4))), "l"(in + from * (D * 2))
                         : "memory");
          }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
      };
      if (kPrefix && any && run->parts == 1) {
        fetch(0);
        fetch(1);
      }
      float m = -INFINITY, l = 0.0f;
      if (any) {
        if (!me.wait_all(me.stat_full + w, ph[w])) return false;
        m = me.s_stat[w * 2 * kPaTile + row];
        l = me.s_stat[w * 2 * kPaTile + kPaTile + row];
        if (!me.wait_all(me.o_full + w, ph[w])) return false;
        ph[w] ^= 1u;
        tc_fence_after();
      }
      if (any && run->bad) {
        // the infinities and NaNs among the values of masked tiles that the row sees join its O
        const int pos = run->pos0 + dq, kmax = run->kmax;
        const int hi = on ? seen_end(p.causal, pos, kmax) : 0, lo = on ? seen_begin(p.window, pos) : 0;
#pragma unroll 1
        for (int c = 0; c < D; c += 16) {
          uint32_t o[16];
          tmem_load16_start(t_o + c, o);
          tmem_load16_finish(o);
          const uint16_t* v = p.v + static_cast<int64_t>(run->head / p.chunks) * p.v_head + c;
#pragma unroll 1
          for (int t = (run->tile0 + run->first[w]) * kPaTile; t < min((run->tile0 + run->last[w]) * kPaTile, kmax); ++t) {
            const int t0 = t & ~(kPaTile - 1);
            if (t0 >= run->free_from && t0 + kPaTile <= run->free_to) {
              t = t0 + kPaTile - 1;                    // (an unmasked tile's are in O)
              continue;
            }
            const uint4* src = reinterpret_cast<const uint4*>(v + (run->k0 + static_cast<int64_t>(t)) * p.v_stride);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint4 u = __ldg(src + i);
              const uint32_t y[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float2 f2 = unpack_16<kF16>(y[k]);
                uint32_t &a = o[8 * i + 2 * k], &b = o[8 * i + 2 * k + 1];
                const bool sees = t >= lo && t < hi;
                if (sees && !(fabsf(f2.x) < INFINITY)) a = __float_as_uint(__uint_as_float(a) + f2.x);
                if (sees && !(fabsf(f2.y) < INFINITY)) b = __float_as_uint(__uint_as_float(b) + f2.y);
              }
            }
          }
          tmem_store16(t_o + c, o);
        }
        tmem_store_wait();
      }
      // Parts of a cut key: [m 256][l 256][D / 4][256 rows][4 channels]
      constexpr size_t kSlot = static_cast<size_t>(kPaRows) * (D + 2);
      const int parts = run->parts, part = run->part, at = w * kPaTile + row;
      const int first_slot = 2 * run->block + run->tail;
      auto part_of = [&](int i) { return p.partials + static_cast<size_t>(i == 0 ? first_slot : (first_slot & ~1) + 2 * i) * kSlot + at; };
      if (parts > 1) {
        float* dst = part_of(part);
        if (on) {
          dst[0] = m;
          dst[kPaRows] = l;
        }
        float4* o = reinterpret_cast<float4*>(dst + 2 * kPaRows + 3 * at);
#pragma unroll 1
        for (int c = 0; any && c < D; c += 16, o += 4 * kPaRows) {
          uint32_t y[16];
          tmem_load16_start(t_o + c, y);
          tmem_load16_finish(y);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (on)
              o[i * kPaRows] = make_float4(__uint_as_float(y[4 * i]), __uint_as_float(y[4 * i + 1]),
                                           __uint_as_float(y[4 * i + 2]), __uint_as_float(y[4 * i + 3]));
          __syncwarp();
        }
        if (any) {
          tc_fence_before();
          me.arrive(me.o_empty + w);
        }
        // the last to write joins them; back to zero
        __threadfence();
        __syncwarp();
        uint32_t* count = p.arrived + run->block * 8 + w * 4 + wl;
        uint32_t written = 0;
        if (me.lane == 0) {
          written = atomicAdd(count, 1u) + 1;
          if (written == static_cast<uint32_t>(parts)) *count = 0;
        }
        if (__shfl_sync(0xFFFFFFFFu, written, 0) != static_cast<uint32_t>(parts)) continue;
        __threadfence();
        // (a part that the row sees nothing of has a sum of 0: its m and its O do not count)
        m = -INFINITY;
#pragma unroll 4
        for (int i = 0; i < parts; ++i) {
          const float mi = __ldcg(part_of(i)), li = __ldcg(part_of(i) + kPaRows);
          m = li == 0.0f ? m : fmaxf(m, mi);
        }
        const float base = m == -INFINITY ? 0.0f : m;
        l = 0.0f;
#pragma unroll 4
        for (int i = 0; i < parts; ++i) {
          const float mi = __ldcg(part_of(i)), li = __ldcg(part_of(i) + kPaRows);
          l = __fadd_rn(l, li == 0.0f ? 0.0f : __fmul_rn(li, ex2(mi - base)));
        }
        float z = lse_of(m, l), f = out_factor(1.0f, l), f_before = 0.0f;
        if (kPrefix && on) {
          float f_own;
          z = join_prefix(z, z_before, f_own, f_before);
          f *= f_own;
        }
        // Their weighted sum in their order, every step rounded by itself: the same whichever
        // comes last.  A trip to the parts takes 1500 clocks, so four of them are on their way at a
        // time, 16 channels each (a query of 8 heads over 20000 keys of 128 channels: parts one by one 78
        // us, four of 8 channels 66, of 16 49; of 64 channels 49, 43, 34).
        constexpr int kStep = 16;
#pragma unroll 1
        for (int c = 0; c < D; c += kStep) {
          float y[kStep];
#pragma unroll
          for (int x = 0; x < kStep; ++x) y[x] = 0.0f;
#pragma unroll 1
          for (int i0 = 0; i0 < parts; i0 += 4) {
            float4 u[4][kStep / 4];
            float wi[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float* src = part_of(min(i0 + e, parts - 1));
              const float4* v = reinterpret_cast<const float4*>(src + 2 * kPaRows + 3 * at) + (c / 4) * kPaRows;
              const float mi = __ldcg(src), li = __ldcg(src + kPaRows);
              wi[e] = i0 + e < parts && li != 0.0f ? mi : -INFINITY;
#pragma unroll
              for (int k = 0; k < kStep / 4; ++k) u[e][k] = __ldcg(v + k * kPaRows);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float a = wi[e] == -INFINITY ? 0.0f : ex2(wi[e] - base);
              if (a == 0.0f) continue;
#pragma unroll
              for (int k = 0; k < kStep / 4; ++k) {
                y[4 * k] = __fadd_rn(y[4 * k], __fmul_rn(u[e][k].x, a));
                y[4 * k + 1] = __fadd_rn(y[4 * k + 1], __fmul_rn(u[e][k].y, a));
                y[4 * k + 2] = __fadd_rn(y[4 * k + 2], __fmul_rn(u[e][k].z, a));
                y[4 * k + 3] = __fadd_rn(y[4 * k + 3], __fmul_rn(u[e][k].w, a));
              }
            }
          }
#pragma unroll
          for (int i = 0; i < kStep / 8; ++i) {
            uint4 before = make_uint4(0u, 0u, 0u, 0u);
            if (kPrefix && f_before != 0.0f) before = reinterpret_cast<const uint4*>(p.prefix_out + out_row * D + c)[i];
            const uint32_t b4[4] = {before.x, before.y, before.z, before.w};
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 v = unpack_16<kF16>(b4[k]);
              h[k] = pack_16<kF16>(fmaf(v.x, f_before, y[8 * i + 2 * k] * f), fmaf(v.y, f_before, y[8 * i + 2 * k + 1] * f));
            }
            if (on) reinterpret_cast<uint4*>(p.out + out_row * D + c)[i] = make_uint4(h[0], h[1], h[2], h[3]);
          }
        }
        if (on && p.lse) p.lse[out_row] = z;
        continue;
      }
      float z = lse_of(m, l), f = out_factor(1.0f, l), f_before = 0.0f;
      if (kPrefix && on) {
        float f_own;
        z = join_prefix(z, z_before, f_own, f_before);
        f *= f_own;
      }
      // 128 bytes of every row: a lane stores vector lane % 8 of every fourth row
      auto store_rows = [&](int c) {
        __syncwarp();
        uint8_t* out = reinterpret_cast<uint8_t*>(p.out) + c * 2 + (me.lane % 8) * 16;
#pragma unroll 4
        for (int r = me.lane / 8; r < 32; r += 4) {
          const int64_t to = __shfl_sync(0xFFFFFFFFu, out_row, r);
          const uint4 v = *reinterpret_cast<const uint4*>(rows_at + r * 128 + (((me.lane ^ r) & 7) << 4));
          if ((rows_on >> r) & 1u) *reinterpret_cast<uint4*>(out + to * (D * 2)) = v;
        }
        __syncwarp();
      };
      if (!kPrefix && any) {
        // (usually.  The next run's products wait for the accumulator: 64 channels at once, it is
        // read after 1500 clocks; 16 channels at a time on their way out it took 4800.)
#pragma unroll 1
        for (int c = 0; c < D; c += 64) {
          uint32_t y[2][32];
          tmem_load32_start(t_o + c, y[0]);
          tmem_load32_start(t_o + c + 32, y[1]);
          tmem_load32_finish(y[0]);
          tmem_load32_finish(y[1]);
          if (c + 64 == D) {
            tc_fence_before();
            me.arrive(me.o_empty + w);
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint32_t* x = y[i / 4] + 8 * (i % 4);
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) h[k] = pack_16<kF16>(__uint_as_float(x[2 * k]) * f, __uint_as_float(x[2 * k + 1]) * f);
            put_vector(i, make_uint4(h[0], h[1], h[2], h[3]));
          }
          store_rows(c);
        }
        if (on && p.lse) p.lse[out_row] = z;
        continue;
      }
      if (kPrefix && any) {
        // (with a prefix: two pieces of 32 channels of its rows on their way, the first ones since before
        // the products were awaited; five ragged turns of 700 tokens 44 us with 64 channels at a time, 41 so.
        // In registers they cost the warps' other paths spills: ragged prompts 223 us, and 217.)
#pragma unroll 1
        for (int u = 0; u < D / 32; ++u) {
          uint32_t y[32];
          tmem_load32_start(t_o + 32 * u, y);
          asm volatile("cp.async.wait_group 1;" ::: "memory");
          __syncwarp();
          tmem_load32_finish(y);
          if (u == D / 32 - 1) {
            tc_fence_before();
            me.arrive(me.o_empty + w);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint4* at = reinterpret_cast<uint4*>(piece(u, me.lane, i));
            uint4 v = *at;
            // (whatever lies in rows without a prefix)
            if (f_before == 0.0f) v = make_uint4(0u, 0u, 0u, 0u);
            const uint32_t b[4] = {v.x, v.y, v.z, v.w};
            uint32_t h[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 x = unpack_16<kF16>(b[k]);
              const float y0 = __uint_as_float(y[8 * i + 2 * k]) * f, y1 = __uint_as_float(y[8 * i + 2 * k + 1]) * f;
              h[k] = pack_16<kF16>(fmaf(x.x, f_before, y0), fmaf(x.y, f_before, y1));
            }
            *at = make_uint4(h[0], h[1], h[2], h[3]);
          }
          __syncwarp();
          uint8_t* out = reinterpret_cast<uint8_t*>(p.out) + u * 64 + (me.lane % 4) * 16;
#pragma unroll
          for (int r = me.lane / 4; r < 32; r += 8) {
            const int64_t to = __shfl_sync(0xFFFFFFFFu, out_row, r);
            if ((rows_on >> r) & 1u)
              *reinterpret_cast<uint4*>(out + to * (D * 2)) = *reinterpret_cast<const uint4*>(piece(u, r, me.lane % 4));
          }
          __syncwarp();
          fetch(u + 2);
        }
        if (on && p.lse) p.lse[out_row] = z;
        continue;
      }
      // (no tokens: zeros, or the prefix's result)
#pragma unroll 1
      for (int c = 0; c < D; c += 64) {
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
          uint4 u = make_uint4(0u, 0u, 0u, 0u);
          if (kPrefix && f_before != 0.0f) u = reinterpret_cast<const uint4*>(p.prefix_out + out_row * D + c)[i];
          uint32_t* h = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 v = unpack_16<kF16>(h[k]);
            h[k] = pack_16<kF16>(v.x * f_before, v.y * f_before);
          }
          put_vector(i, u);
        }
        store_rows(c);
      }
      if (on && p.lse) p.lse[out_row] = z;
    }
    me.give_back();
  }
  me.give_back();
  return true;
}

// Softmax of a row tile's rows.
template <int D, bool kF16>
__device__ __forceinline__ bool softmax(uint32_t tmem, int Gt, int qt, int causal, int window, float scale) {
  using Sm = PaSmem<D>;
  constexpr int NS = Sm::kSlots;
  Member<D> me;
  // A row's weights are 2^(s - m), m set to its largest score less kRise and set again when
  // those of a tile (128) add up to more than kMostSum: none is above 2^15 with the m of before,
  // none above 2^kRise in the tile that set it, so fp16 holds them.  fp16: as csrc/kv_attention.cuh,
  // most of its range lies below; bf16 has fp32's range, and results need room above the weights.
  constexpr float kRise = kF16 ? kLift : 0.0f;
  constexpr float kMostSum = 32768.0f;
  const int w = threadIdx.x >> 7, wl = (threadIdx.x >> 5) & 3, row = threadIdx.x & 127;
  const uint32_t lanes = static_cast<uint32_t>(wl * 32) << 16;
  const uint32_t t_s = tmem + lanes + w * kPaTile, t_o = tmem + lanes + 2 * kPaTile + w * D;
  const int iq = row / Gt;
  uint32_t ph_s = 0, ph_stat = 1;
  int n_tiles = 0;                                     // of the runs so far
  // What hides a score: -inf once it is scaled.  (A scale of zero hides nothing by itself: its
  // scores are multiplied by zero where the masks are written, NaNs and infinities become NaNs, and
  // then scaled by one.)
  const bool flat = scale == 0.0f;
  const float to_log2 = flat ? 1.0f : scale, hidden = scale < 0.0f ? INFINITY : -INFINITY;
  // ---- a run's tiles
  auto weigh = [&](const volatile Run& run) -> bool {
    const int j0 = run.first[w], j1 = run.last[w];
    if (j0 >= j1) return true;
    const int dq = w * qt + iq, t00 = run.tile0 * kPaTile;
    const bool on = iq < qt && dq < run.n_q, any_on = __any_sync(0xFFFFFFFFu, on);
    // (rows that nobody asked for see all: nothing of theirs matters, nothing is masked for them)
    const int pos = run.pos0 + dq, kmax = run.kmax;
    const int hi = on ? seen_end(causal, pos, kmax) - t00 : 0, lo = on ? seen_begin(window, pos) - t00 : 0;
    // every row of the warp sees all tokens of [all_from, all_to), those of the tiles [full0, full1) among them
    const int all_from = max(__reduce_max_sync(0xFFFFFFFFu, on ? lo : 0), 0);
    const int all_to = max(__reduce_min_sync(0xFFFFFFFFu, on ? hi : INT32_MAX), 0);
    const int full0 = (all_from + kPaTile - 1) / kPaTile, full1 = all_to / kPaTile;
    float m_neg = on ? INFINITY : 0.0f, l = 0.0f;
#pragma unroll 1
    for (int j = j0; j < j1; ++j) {
      if (!me.wait_all(me.s_full + w, ph_s)) return false;
      ph_s ^= 1u;
      tc_fence_after();
      // S is there, so its keys and the values of the tile before have been read
      auto free_slots = [&]() { if (wl == 0 && me.lane == 0) mbar_arrive(me.kv_empty + 2 * (n_tiles + j) % NS); };
      if (any_on) {
        const bool masked = j < full0 || j >= full1 || flat;
        const int from = on ? lo - j * kPaTile : 0, to = on ? hi - j * kPaTile : kPaTile;     // tokens that the row sees
        if (masked) {
          // in place: one loop of weights for all tiles
#pragma unroll 1
          for (int c = 0; c < kPaTile; c += 32) {
            if (j * kPaTile + c >= all_from && j * kPaTile + c + 32 <= all_to && !flat) continue;
            uint32_t y[2][16];
            tmem_load16_start(t_s + c, y[0]);
            tmem_load16_start(t_s + c + 16, y[1]);
            tmem_load16_finish(y[0]);
            tmem_load16_finish(y[1]);
            const uint32_t see = tokens32(c, from, to);
#pragma unroll
            for (int x = 0; x < 32; ++x)
              y[x / 16][x % 16] = !(see & (1u << x)) ? __float_as_uint(hidden) :
                                  flat ? __float_as_uint(__uint_as_float(y[x / 16][x % 16]) * 0.0f) : y[x / 16][x % 16];
            tmem_store16(t_s + c, y[0]);
            tmem_store16(t_s + c + 16, y[1]);
          }
          tmem_store_wait();
        }
        // The maximum is looked for by rows that see tokens here and none before, and again where
        // weights add up to more than kMostSum (or to no number).  (Each row by itself: what lies
        // in one does not change another's roundings.)
        const bool sees = on && from < kPaTile && to > 0;
        bool need = m_neg == INFINITY && sees, moved = !on;
        bool look = (masked || j == j0) && __any_sync(0xFFFFFFFFu, need);
        uint32_t pr[kPaTile / 2];
        float sum;
        bool held = true;
#pragma unroll 1
        for (;;) {
          if (look) {
            // m is set by the largest score so far, this tile's included.  (By those of the first 16
            // tokens of a first tile, many rows needed a second one: pictures 99 us, and 71 so;
            // 8192 tokens 716 and 689.)
            float top = -INFINITY;
#pragma unroll 1
            for (int c = 0; c < kPaTile; c += 32) {
              uint32_t y[2][16];
              tmem_load16_start(t_s + c, y[0]);
              tmem_load16_start(t_s + c + 16, y[1]);
              tmem_load16_finish(y[0]);
              tmem_load16_finish(y[1]);
#pragma unroll
              for (int x = 0; x < 32; ++x) top = fmaxf(top, __uint_as_float(y[x / 16][x % 16]) * to_log2);
            }
            const float now = need ? fminf(m_neg, kRise - top) : m_neg;
            moved = moved || need;
            const float shrink = now < m_neg ? ex2(now - m_neg) : 1.0f;
            m_neg = now;
            l *= shrink;
            if (j > j0) {
              // (earlier tiles are in O: S came after them)
#pragma unroll 1
              for (int c = 0; c < D; c += 16) {
                uint32_t y[16];
                tmem_load16_start(t_o + c, y);
                tmem_load16_finish(y);
#pragma unroll
                for (int x = 0; x < 16; ++x) y[x] = __float_as_uint(__uint_as_float(y[x]) * shrink);
                tmem_store16(t_o + c, y);
              }
            }
          }
          uint32_t s[2][16];
          tmem_load16_start(t_s, s[0]);
          if (held) free_slots();
          held = false;
          uint64_t sum2 = f2_pack(0.0f, 0.0f);
          const float add = m_neg == INFINITY ? 0.0f : m_neg;          // (nothing but -inf seen so far)
          const uint64_t k2 = f2_pack(to_log2, to_log2), m2 = f2_pack(add, add);
#pragma unroll
          for (int c = 0; c < kPaTile; c += 16) {
            uint32_t (&y)[16] = s[c / 16 % 2];
            tmem_load16_finish(y);
            if (c + 16 < kPaTile) tmem_load16_start(t_s + c + 16, s[(c / 16 + 1) % 2]);
#pragma unroll
            for (int x = 0; x < 16; x += 2) {
              const uint64_t v = f2_fma(f2_pack(__uint_as_float(y[x]), __uint_as_float(y[x + 1])), k2, m2);
              const float a = ex2(f2_lo(v)), b = ex2(f2_hi(v));
              sum2 = f2_add(sum2, f2_pack(a, b));
              pr[(c + x) / 2] = pack_16<kF16>(a, b);
            }
          }
          sum = f2_lo(sum2) + f2_hi(sum2);
          need = !moved && (!(sum <= kMostSum) || (m_neg == INFINITY && sees));
          look = __any_sync(0xFFFFFFFFu, need);
          if (!look) break;
        }
        l += sum;
        // P over the columns of S that have been read
#pragma unroll
        for (int c = 0; c < kPaTile / 2; c += 16) {
          uint32_t x[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) x[k] = pr[c + k];
          tmem_store16(t_s + c, x);
        }
        tmem_store_wait();
        tc_fence_before();
        me.arrive(me.p_full + w);
      } else {
        // (rows that nobody asked for: their P may be anything)
        free_slots();
        tc_fence_before();
        me.arrive(me.p_full + w);
      }
    }
    // (me.o_empty: the statistics of the run before have been read as well)
    if (!me.wait_all(me.o_empty + w, ph_stat)) return false;
    ph_stat ^= 1u;
    me.s_stat[w * 2 * kPaTile + row] = -m_neg;
    me.s_stat[w * 2 * kPaTile + kPaTile + row] = l;
    me.arrive(me.stat_full + w);
    return true;
  };
  for (;;) {
    const volatile Run* run = me.take();
    if (!run) return false;
    if (run->tiles < 0) break;
    if (!weigh(*run)) return false;
    n_tiles += run->tiles;
    me.give_back();
  }
  me.give_back();
  return true;
}

// (With a prefix the rows' way out is compiled apart: its registers and instructions cost the calls
// without one 1 to 2 %, 8192 tokens 660 and 647 us, ragged prompts 219 and 214.)
template <int D, bool kF16, bool kPrefix>
__global__ void __launch_bounds__(kPaThreads, 1)
prompt_attention_kernel(const __grid_constant__ PromptParams p) {
  constexpr int NS = PaSmem<D>::kSlots;
  const Block<D> sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < kRuns; ++i) { mbar_init(sh.run_full + i, 1); mbar_init(sh.run_empty + i, kConsumers); }
    for (int i = 0; i < NS; ++i) { mbar_init(sh.kv_full + i, 1); mbar_init(sh.kv_empty + i, 2 - i % 2); mbar_init(sh.v_clean + i, 1); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(sh.q_full + i, 1); mbar_init(sh.q_empty + i, 1); mbar_init(sh.s_full + i, 1);
      mbar_init(sh.p_full + i, 4);
      mbar_init(sh.o_full + i, 1); mbar_init(sh.o_empty + i, 4); mbar_init(sh.stat_full + i, 4);
    }
    mbar_init(sh.drained, 2);
    *sh.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 12) tmem_alloc(sh.tmem_holder, 512);
  if (warp == 14 && lane < 3) tma_prefetch_map(lane == 0 ? &p.tm_q : lane == 1 ? &p.tm_k : &p.tm_v);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");

  // ---- this block's chunk of the flat order
  const int n_items = p.B * p.groups;
  const int per = (n_items + kPaThreads - 1) / kPaThreads;
  // Sums of places stop at 2^31 - 1.  (Offsets that decrease can make more of the same rows than the
  // host allowed for: then nothing is done.  In 64 bits one short prompt took 0.2 us more.)
  auto plus = [](int a, int b) { return static_cast<int>(min(static_cast<uint32_t>(a) + static_cast<uint32_t>(b), 0x7FFFFFFFu)); };
  int mine = 0, some = 0, longest = 0;       // of this thread's items: places, those with queries, tiles
  for (int i = tid * per; i < min((tid + 1) * per, n_items); ++i) {
    const PromptGroup g = prompt_group(p, i);
    mine = plus(mine, key_cost(g) * p.Hv);
    some += g.n > 0;
    longest = max(longest, g.tiles);
  }
  int incl = mine, incl_some = some;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int a = __shfl_up_sync(0xFFFFFFFFu, incl, d), b = __shfl_up_sync(0xFFFFFFFFu, incl_some, d);
    if (lane >= d) {
      incl = plus(incl, a);
      incl_some += b;
    }
  }
  longest = __reduce_max_sync(0xFFFFFFFFu, longest);
  int* sums = reinterpret_cast<int*>(sh.s_stat);
  if (lane == 31) {
    sums[warp] = incl;
    sums[16 + warp] = incl_some;
    sums[32 + warp] = longest;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int before = 0, total = 0, before_some = 0, total_some = 0;
#pragma unroll 4
  for (int w = 0; w < kPaThreads / 32; ++w) {
    const int x = sums[w], y = sums[16 + w];
    if (w < warp) {
      before = plus(before, x);
      before_some += y;
    }
    total = plus(total, x);
    total_some += y;
    longest = max(longest, sums[32 + w]);
  }
  if (total >= kPaMost) total = total_some = 0;
  sh.s_first[tid] = before_some + incl_some - some;
  const int blocks = static_cast<int>(gridDim.x);
  Share share;
  share.keys = total_some * p.Hv;
  const int chunk = share.chunk = max((total + blocks - 1) / blocks, p.min_chunk);
  share.uncut = kPaPlaces * longest > 2 * chunk ? kPaWholeFew : kPaWhole;
  const int top = kPaPlaces * longest + kPaKeyCost;          // the longest key's places
  share.whole = longest <= share.uncut || chunk >= kPaEven * kPaPlaces * longest ||
                (chunk >= top && 4 * static_cast<int64_t>(total) <= 3 * static_cast<int64_t>(share.keys) * top);
  const int f0 = share.f0 = static_cast<int>(min(static_cast<int64_t>(blockIdx.x) * chunk, static_cast<int64_t>(total)));
  const int f1 = share.f1 = static_cast<int>(min(static_cast<int64_t>(f0) + chunk, static_cast<int64_t>(total)));
  const int excl = plus(before, incl - mine);
  if (!share.whole && f0 < f1 && excl <= f0 && f0 < excl + mine) {
    int at = excl, i = tid * per;
    for (;; ++i) {
      const int n = key_cost(prompt_group(p, i)) * p.Hv;
      if (f0 < at + n) break;
      at += n;
    }
    sh.s_start[0] = i;
    sh.s_start[1] = f0 - at;
  }
  __syncthreads();
  const uint32_t tmem = *sh.tmem_holder;
  if (p.cu_q && warp >= 8 && warp < 12) clear_rows<D>(p, blockIdx.x * 4 + warp - 8, gridDim.x * 4);
  if (share.whole ? static_cast<int>(blockIdx.x) < share.keys : f0 < f1) {
    bool ok = true;
    if (warp < 8) {
      ok = softmax<D, kF16>(tmem, p.Gt, p.qt, p.causal, p.window, p.scale_log2);
    } else if (warp < 12) {
      ok = rows_out<D, kF16, kPrefix>(p, tmem);
    } else if (warp < 14) {
      ok = products<D, kF16>(tmem, warp - 12);
      // nothing of this block's is under way when the tensor memory goes back
      if (elect_one()) tc_commit(sh.drained);
      __syncwarp();
      __all_sync(0xFFFFFFFFu, wait_bounded(sh.drained, 0, sh.abort_flag));
    } else {
      ok = warp == 14 ? walk<D>(p, share) : look_over<D, kF16>();
    }
    if (!ok && lane == 0) {
      report_timeout(p.status);
      *sh.abort_flag = 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(tmem, 512);
}

bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool off4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

constexpr size_t a256(size_t n) { return (n + 255) & ~size_t(255); }
constexpr size_t kWsArrived = 256;
constexpr size_t kWsHanded = a256(kWsArrived + kPaMaxCtas * 8 * sizeof(uint32_t));
constexpr size_t kWsPartials = kWsHanded + 256;
constexpr size_t ws_total(int D) { return a256(kWsPartials + size_t(2) * kPaMaxCtas * kPaRows * (D + 2) * 4); }

// [rows][heads][D] of 16-bit values, boxes of 64 channels, box_heads and box_rows.
bool encode_heads(CUtensorMap* map, const void* base, bool f16, int64_t rows, int64_t heads, int D, int64_t row_stride,
                  int64_t head_stride, uint32_t box_heads, uint32_t box_rows) {
  auto encode = tensor_map_encoder();
  if (!encode) return false;
  // (the distance of the only one of a kind is never used; it has to be valid)
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(heads > 1 ? head_stride : D) * 2,
                                 static_cast<cuuint64_t>(rows > 1 ? row_stride : D) * 2};
  const cuuint32_t box[3] = {64, box_heads, box_rows}, step[3] = {1, 1, 1};
  return encode(map, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
                const_cast<void*>(base), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The tiles of a key at most: of all keys, or of a window over the group's queries.
int64_t most_tiles(const PromptParams& p) {
  const int64_t tiles = (static_cast<int64_t>(p.max_k) + kPaTile - 1) / kPaTile;
  if (p.window <= 0) return tiles;
  return std::min(tiles, (static_cast<int64_t>(p.window) + 2 * p.qt + kPaTile - 2) / kPaTile + 1);
}
// Items, and keys that have queries, of a call at most where a key has up to `span` of them: T
// queries in B sequences are T / span + B groups, however many max_q leaves room for.
int64_t most_items(const PromptParams& p, int span) { return p.B * ((static_cast<int64_t>(p.max_q) + span - 1) / span); }
int64_t most_keys(const PromptParams& p, int span) { return std::min(most_items(p, span), p.T / span + p.B) * p.Hv; }
// Whether the device can count its places, and whether a block's stretch of one key (all of its tiles,
// or those of the block's places: a GB300 has more than 128 blocks) ends while the rows' way out still waits for it.
bool countable(const PromptParams& p, int span) {
  const int64_t tiles = most_tiles(p), cost = kPaPlaces * tiles + kPaKeyCost;
  return most_items(p, span) < (int64_t(1) << 30) && most_keys(p, span) <= (kPaMost - 1) / cost &&
         std::min(tiles, most_keys(p, span) * cost / (128 * kPaPlaces)) <= kPaMostTiles;
}

template <int D, bool kF16, bool kPrefix>
nvr_status launch(PromptParams& p, cudaStream_t s) {
  using Sm = PaSmem<D>;
  static_assert(Sm::kTotal <= 227 * 1024, "shared memory");
  static bool attr_set[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return NVR_ERR_CUDA;
  const int sms = device_sm_count();
  if (sms <= 0) return NVR_ERR_CUDA;
  if (!attr_set[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(prompt_attention_kernel<D, kF16, kPrefix>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sm::kTotal);
    if (e != cudaSuccess) return cuda_status(e);
    attr_set[dev] = true;
  }
  // Two row tiles a key; one where no more than three blocks of four would have one (the rows of a
  // block's two tiles go out, and are joined, one after the other): a prompt of 37 tokens, 32 heads,
  // 10.8 us, and 8.8 so; 700 of 16 heads with a prefix 24.4 and 17.6; 128 tokens of 8 heads over 8320 keys
  // 64 and 38.5; 600 of 16 heads (38 keys of two row tiles) 18.5 and 14.9, over 4000 more 57 and 44.  At 70
  // keys two are faster where they are long: 1100 tokens over 4000 more 59 and 64.5; with more keys
  // than blocks, 2000 and 1500 tokens over 5000 and 4000 keys, 103 and 132.
  p.span = 2 * p.qt;
  if (most_keys(p, p.span) * 4 <= sms * int64_t(3) && countable(p, p.qt)) p.span = p.qt;
  p.groups = (p.max_q + p.span - 1) / p.span;
  const int64_t tiles = most_tiles(p), most = most_keys(p, p.span) * (kPaPlaces * tiles + kPaKeyCost);
  int64_t grid = sms < kPaMaxCtas ? sms : kPaMaxCtas;
  p.min_chunk = kPaMinChunk;
  while (static_cast<int64_t>(p.min_chunk) * p.min_chunk < kPaPlaces * kPaPlaces * tiles) ++p.min_chunk;
  // (rows that no sequence covers are many where the batch is padded: they are cleared by all blocks)
  const int64_t blocks = (most + p.min_chunk - 1) / p.min_chunk, clearing = p.cu_q ? (p.T + kPaRows - 1) / kPaRows : 0;
  if (grid > blocks) grid = blocks > clearing ? blocks : clearing < grid ? clearing : grid;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kPaThreads);
  cfg.dynamicSmemBytes = Sm::kTotal;
  cfg.stream = s;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, prompt_attention_kernel<D, kF16, kPrefix>, p));
}

}  // namespace

}  // namespace nvr

using namespace nvr;

extern "C" size_t prompt_attention_workspace_size(int Hq, int Hkv, int D) {
  if (Hkv < 1 || Hq < 1 || Hq % Hkv || (D != 64 && D != 128)) return 0;
  return ws_total(D);
}

extern "C" nvr_status prompt_attention(const void* q, int64_t q_stride, int64_t q_head_stride, const void* k,
                                       int64_t k_stride, int64_t k_head_stride, const void* v, int64_t v_stride,
                                       int64_t v_head_stride, nvr_dtype dt, int64_t T, int64_t Tk, int Hq, int Hkv,
                                       int D, const int32_t* cu_q, const int32_t* cu_k, int64_t B, int max_q,
                                       int max_k, float scale, int causal, int window, const void* prefix_out,
                                       const float* prefix_lse, void* out, float* lse, void* workspace,
                                       size_t ws_bytes, nvr_stream_t stream) {
  if (T < 0 || Tk < 0 || B < 0 || Hq < 1 || Hkv < 1 || Hq % Hkv || Hq > 65536) return NVR_ERR_INVALID_ARG;
  if (dt != NVR_BF16 && dt != NVR_F16) return NVR_ERR_INVALID_ARG;
  if (max_q < 0 || max_k < 0 || window < 0 || (window > 0 && !causal)) return NVR_ERR_INVALID_ARG;
  const float scale_log2 = scale * 1.44269504088896341f;     // (finite as well: times a score of 0 it would be a NaN)
  if (!(scale_log2 > -INFINITY && scale_log2 < INFINITY)) return NVR_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return NVR_ERR_UNSUPPORTED;
  if (!workspace || (prefix_out != nullptr) != (prefix_lse != nullptr)) return NVR_ERR_INVALID_ARG;
  if (T > 0 && (!q || !out || B < 1 || max_q < 1 || out == q || out == k || out == v)) return NVR_ERR_INVALID_ARG;
  if (Tk > 0 && (!k || !v)) return NVR_ERR_INVALID_ARG;
  if (T > INT32_MAX - 1024 || Tk > INT32_MAX - 1024 || B > kPaMaxB) return NVR_ERR_UNSUPPORTED;
  if (cu_q && max_q > T) max_q = static_cast<int>(T);        // (no sequence has more)
  if (!cu_q && T != B * max_q) return NVR_ERR_INVALID_ARG;
  if (!cu_k && Tk != T) return NVR_ERR_INVALID_ARG;
  // heads may lie in any order, 16 bytes apart at least, but not in front of the first
  auto bad = [&](int64_t rows, int64_t heads, int64_t stride, int64_t head_stride) {
    return (rows > 1 && (stride < D || stride % 8)) || (heads > 1 && (head_stride < D || head_stride % 8)) ||
           stride >= (int64_t(1) << 38) || head_stride >= (int64_t(1) << 38);
  };
  if (bad(T, Hq, q_stride, q_head_stride) || bad(Tk, Hkv, k_stride, k_head_stride) ||
      bad(Tk, Hkv, v_stride, v_head_stride))
    return NVR_ERR_INVALID_ARG;
  PromptParams p;
  p.T = T; p.Tk = Tk;
  p.Hq = Hq; p.G = Hq / Hkv;
  // Heads of a KV head that share a row tile: the most that divide them and fill 7/8 of its
  // 128 rows with whole queries (one always does).
  p.Gt = 1;
  for (int g = 2; g <= p.G && g <= kPaTile; ++g)
    if (p.G % g == 0 && kPaTile / g * g >= kPaTile * 7 / 8) p.Gt = g;
  p.qt = kPaTile / p.Gt;
  p.chunks = p.G / p.Gt;
  p.Hv = Hq / p.Gt;
  p.cu_q = cu_q; p.cu_k = cu_k;
  p.B = static_cast<int>(B); p.max_q = max_q;
  p.max_k = cu_k ? max_k : max_q;
  if (p.max_k > Tk) p.max_k = static_cast<int>(Tk);
  p.window = window >= Tk ? 0 : window;                      // (then it hides nothing)
  if (!countable(p, 2 * p.qt)) return NVR_ERR_UNSUPPORTED;
  if (off16(q) || off16(k) || off16(v) || off16(out) || off16(prefix_out) || off4(cu_q) || off4(cu_k) || off4(lse) ||
      off4(prefix_lse) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return NVR_ERR_ALIGNMENT;
  if (ws_bytes < ws_total(D)) return NVR_ERR_WORKSPACE;
  if (T == 0) return NVR_OK;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.scale_log2 = scale_log2;
  p.causal = causal != 0;
  p.v = static_cast<const uint16_t*>(v); p.v_stride = v_stride; p.v_head = v_head_stride;
  p.prefix_out = static_cast<const uint16_t*>(prefix_out); p.prefix_lse = prefix_lse;
  p.out = static_cast<uint16_t*>(out); p.lse = lse;
  p.status = reinterpret_cast<uint32_t*>(ws + kWsStatus);
  p.arrived = reinterpret_cast<uint32_t*>(ws + kWsArrived);
  p.handed = reinterpret_cast<uint32_t*>(ws + kWsHanded);
  p.partials = reinterpret_cast<float*>(ws + kWsPartials);
  const bool f16 = dt == NVR_F16;
  // (without keys nothing is loaded: the maps are of the queries, to be valid)
  const bool keys = Tk > 0;
  if (!encode_heads(&p.tm_q, q, f16, T, Hq, D, q_stride, q_head_stride, p.Gt, p.qt) ||
      !encode_heads(&p.tm_k, keys ? k : q, f16, keys ? Tk : 1, keys ? Hkv : 1, D, k_stride, k_head_stride, 1, kPaTile) ||
      !encode_heads(&p.tm_v, keys ? v : q, f16, keys ? Tk : 1, keys ? Hkv : 1, D, v_stride, v_head_stride, 1, kPaTile))
    return NVR_ERR_UNSUPPORTED;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  auto go = [&](auto prefix) {
    constexpr bool kPrefix = decltype(prefix)::value;
    if (D == 128) return f16 ? launch<128, true, kPrefix>(p, s) : launch<128, false, kPrefix>(p, s);
    return f16 ? launch<64, true, kPrefix>(p, s) : launch<64, false, kPrefix>(p, s);
  };
  return prefix_lse ? go(std::true_type{}) : go(std::false_type{});
}
