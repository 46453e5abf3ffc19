// kv_prefill.cu -- softmax attention over the paged NVFP4 key/value cache for
// many (query, head) columns (sm_103a): prompt chunks, drafts of many tokens.
// Bound by the tensor cores: 4 D flops for every column and token against 9/8 D
// bytes of cache read once for 256 columns.
//
// Mathematics: as csrc/kv_attention.cu (running maximum moved in steps, fp32
// sums, fp16 weights).  Here S = Q K^T and O += P V run on tcgen05 with the
// columns as the 128 rows of an accumulator in tensor memory: a thread owns a
// row, so that its maximum and sum need no exchange.
//
// A block (one per SM) takes 256 columns of a sequence that share a KV head as
// two row tiles and walks the tokens in tiles of 128:
//   warps 0-3, 4-7  softmax of row tile 0 and 1: scale the queries into fp16, read S
//                   from tensor memory, write P (fp16) over it, rescale O when the
//                   maximum moves, store the rows at the end of a key;
//   warps 8-11      expand the cache: codes and scales from the pages to
//                   registers one tile ahead, code * scale (exact in fp16) into
//                   swizzled shared memory, two stages of K and of V;
//   warp 12         issues the products, alternating the row tiles, so that one
//                   tile's softmax runs under the other's products;
//   warp 13         walks the work and hands every role its runs;
//   warp 14         fetches the pages of the coming tiles into L2;
//   warp 15         copies the query rows of the coming run into shared memory, the
//                   heads of a query in one bulk copy (a copy a row: each run 4 us longer).
// A group of at most 128 columns uses both halves as well: the same rows in
// both, each taking every other token tile, joined at the end.
//
// Tensor memory, 512 columns: S0 | S1 (128 each, P over the first half of its
// S), O0 | O1 (D each).  S of the next tile follows P V of this one in issue
// order, so S is never overwritten early and a complete S implies the earlier
// P V complete.  P comes in two halves of 64 tokens: P V of the first runs under
// the softmax of the second.
//
// The work is cut as in csrc/kv_attention.cu: all keys' tiles end to end in
// equal chunks, one per block, the rows of cut keys joined by csrc/kv_join.cu.
//
// Measured (D = 128, 8 KV heads): 2048 queries of 64 heads over 8192 tokens 385 us,
// 1249 TFLOP/s, 0.66 of the cuBLAS bf16 rate; nine ragged prompts of up to 1500
// queries of 32 heads over 2500 tokens 113 us.  A tile of 128 tokens and 256 columns takes
// 1.8 us (3400 clocks; its products 2050): each row tile's softmax 2200 clocks and
// then 1000 of waiting for its next S, which the full tensor memory leaves no room to
// make earlier.  A run of a key costs 4.6 us on top (queries in, rows out).  Tried and
// slower: loops around the issue of the products (510 us for the chunk), unrolled
// halves of the softmax (450: fetching the instructions), eight warps that expand
// (450: 96 registers a thread), other splits of the registers (equal), scores in
// halves of 64 tokens that are made while the other half is weighed (536), S loaded a
// half ahead (388), each where this took 383.
#include <type_traits>

#include "kv_attention.cuh"

namespace nvr {

namespace {

constexpr int kPTile = 128;                // tokens of a tile, rows of a row tile
constexpr int kPThreads = 512;
// Starting and ending a key (queries in, rows out, an empty pipeline) counts as this many
// tiles: 4.6 us beside 1.8 us for a tile of two row tiles and 1.4 for one.  2, 3, 4, 5
// tiles, us: the ragged prompts above 121, 113.5, 113, 116; 32 sequences of up to 4096
// tokens with eight queries of 64 heads 85, 71.7, 68.9, 68.5; six prompts of up to 700
// queries of 48 heads over 5000 tokens 135, 134.5, 135.5, 135; the chunk 387, 386, 386, 388.
constexpr int kPKeyCost = 4;
constexpr int kRuns = 3;                   // runs handed out ahead
constexpr int kLive = 4;                   // tiles whose live tokens are kept: expanded at most three ahead
constexpr int kAhead = 6;                  // tiles fetched into L2 before they are expanded
constexpr float kMostSum = 32768.0f;       // 2^kMostWeight

// A key's stretch of tiles in this block's chunk.
struct alignas(16) Run {
  int tiles;                               // -1: the end
  int tile0, b, head;
  int kv, n_q, q0, n_cols;
  int iq0, rem0, lo, hi;
  int dual;                                // both halves on different rows (else on alternate tiles)
  int whole, slot;                         // all of its key, or a part: in this slot
  float k_gsa, v_gsa;
  int col0;                                // the column of half 1's row 0 (half 0's: column 0)
  int nan;                                 // values of the run have NaNs among their scales (written while it is expanded)
  int pad;
};

template <int D>
struct PrefillSmem {
  static constexpr int kTileBytes = kPTile * D * 2;          // fp16 rows in 128-byte swizzled atoms of 64 channels
  static constexpr int kQ = 0;
  static constexpr int kK = kQ + 2 * kTileBytes;
  static constexpr int kV = kK + 2 * kTileBytes;
  static constexpr int kOut = kV + 2 * kTileBytes;           // 128 bytes of each row on their way out
  static constexpr int kRunsAt = kOut + 2 * kPTile * 128;
  static constexpr int kRowAt = kRunsAt + kRuns * static_cast<int>(sizeof(Run));   // per row: m, l of half 1
  static constexpr int kBarAt = kRowAt + 2 * kPTile * 4;
  static constexpr int kTotal = kBarAt + 48 * 8 + 64 + 1024;
};

__device__ __forceinline__ uint32_t idesc_f16(int M, int N, bool b_mn_major) {
  // D fp32 (1 in bits 4-5), A and B fp16 (0), B transposed in bit 16, N >> 3 in
  // bits 17-22, M >> 4 in bits 24-28
  return (1u << 4) | (b_mn_major ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}

// The two words of a matrix descriptor: 128-byte swizzle, 8-row groups 1024 bytes
// apart; the low one holds the address and the distance of 64-channel atoms (used
// by the transposed operand alone).  The next step of a product is an addition to
// the low word: the issuing warp's instructions are on the critical path.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(const void* tile, uint32_t atom_distance) {
  return ((smem_u32(tile) & 0x3FFFFu) >> 4) | ((atom_distance >> 4) << 16);
}

// D[tmem] (+)= A[smem] . B[smem], fp16 operands; descriptors by their low words.
__device__ __forceinline__ void tc_mma_f16(uint32_t d_tmem, uint32_t a_low, uint32_t b_low, uint32_t idesc,
                                           bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}"
      :: "r"(d_tmem), "r"(a_low), "r"(b_low), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)), "r"(kDescHigh)
      : "memory");
}
// The same with A in tensor memory (two fp16 of a row to a column).
__device__ __forceinline__ void tc_mma_f16_ta(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_low, uint32_t idesc,
                                              bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %4, 0;\n\tmov.b64 b, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}"
      :: "r"(d_tmem), "r"(a_tmem), "r"(b_low), "r"(idesc), "r"(static_cast<uint32_t>(accumulate)), "r"(kDescHigh)
      : "memory");
}

__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// 32 columns of this warp's lanes without the wait, and the wait: the registers
// pass through it so that nothing reads them early.
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
__device__ __forceinline__ int key_cost(const Group& g) { return g.tiles ? g.tiles + kPKeyCost : 0; }

template <int D>
__global__ void __launch_bounds__(kPThreads, 1)
kv_prefill_kernel(const AttnParams p) {
  using Sm = PrefillSmem<D>;
  constexpr int NC = kPrefillCols;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Run* s_runs = reinterpret_cast<Run*>(smem + Sm::kRunsAt);
  float* s_row = reinterpret_cast<float*>(smem + Sm::kRowAt);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Sm::kBarAt);
  uint64_t *run_full = bars, *run_empty = run_full + kRuns, *k_full = run_empty + kRuns, *k_empty = k_full + 2,
           *v_full = k_empty + 2, *v_empty = v_full + 2, *q_full = v_empty + 2, *s_full = q_full + 2,
           *p_full = s_full + 2, *o_full = p_full + 2, *meet = o_full + 2, *x_ready = meet + 2, *x_full = x_ready + 1,
           *x_free = x_full + 1, *drained = x_free + 1, *q_raw = drained + 1, *h_full = q_raw + 2,
           *p_half = h_full + 2, *q_empty = p_half + 2;
  int* s_words = reinterpret_cast<int*>(q_empty + 2);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(s_words);
  volatile int* abort_flag = s_words + 1;
  int* s_start = s_words + 2;                                // item, offset inside it
  volatile int* s_done = s_words + 10;                       // tiles expanded
  volatile uint32_t* s_live = reinterpret_cast<volatile uint32_t*>(s_words + 6);   // [kLive] tokens in groups of 16
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int i = 0; i < kRuns; ++i) { mbar_init(run_full + i, 1); mbar_init(run_empty + i, 15); }
    for (int i = 0; i < 2; ++i) {
      mbar_init(k_full + i, 4); mbar_init(k_empty + i, 1);
      mbar_init(v_full + i, 4); mbar_init(v_empty + i, 1);
      mbar_init(q_full + i, 4); mbar_init(s_full + i, 1);
      mbar_init(p_full + i, 4); mbar_init(o_full + i, 1);
      mbar_init(meet + i, 4); mbar_init(q_raw + i, 1); mbar_init(h_full + i, 1); mbar_init(p_half + i, 4);
      mbar_init(q_empty + i, 5);
    }
    mbar_init(x_ready, 4); mbar_init(x_full, 4); mbar_init(x_free, 4); mbar_init(drained, 1);
    *abort_flag = 0;
    *s_done = 0;
    for (int i = 0; i < kLive; ++i) s_live[i] = 0;
    fence_mbar_init();
  }
  if (warp == 12) tmem_alloc(tmem_holder, 512);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");

  // ---- this block's chunk of the flat order
  const int n_items = p.B * p.groups;
  const int per = (n_items + kPThreads - 1) / kPThreads;
  int mine = 0;
  for (int i = tid * per; i < min((tid + 1) * per, n_items); ++i) mine += key_cost(group_of<NC, kPTile>(p, i)) * p.Hkv;
  int incl = mine;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int a = __shfl_up_sync(0xFFFFFFFFu, incl, d);
    if (lane >= d) incl += a;
  }
  if (lane == 31) reinterpret_cast<int*>(s_row)[warp] = incl;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int before = 0, total = 0;
  for (int w = 0; w < kPThreads / 32; ++w) {
    const int x = reinterpret_cast<int*>(s_row)[w];
    if (w < warp) before += x;
    total += x;
  }
  const int chunk = max((total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x), kMinChunk);
  const int f0 = min(static_cast<int64_t>(blockIdx.x) * chunk, static_cast<int64_t>(total));
  const int f1 = min(f0 + chunk, total);
  const int excl = before + incl - mine;
  if (f0 < f1 && excl <= f0 && f0 < excl + mine) {
    int at = excl, i = tid * per;
    for (;; ++i) {
      const int n = key_cost(group_of<NC, kPTile>(p, i)) * p.Hkv;
      if (f0 < at + n) break;
      at += n;
    }
    s_start[0] = i;
    s_start[1] = f0 - at;
  }
  __syncthreads();
  const uint32_t tmem = *tmem_holder;

  auto give_up = [&]() {
    if (lane == 0) {
      report_timeout(p.status);
      *abort_flag = 1;
    }
  };
  auto wait_all = [&](uint64_t* bar, uint32_t parity) {
    return __all_sync(0xFFFFFFFFu, wait_bounded(bar, parity, abort_flag)) != 0;
  };

  if (tid == 13 * 32) p.joins[blockIdx.x].n_parts = 0;       // (until this block turns out to start a cut key)
  if (p.cu_q && warp < 8) clear_uncovered<D>(p, blockIdx.x * 8 + warp, gridDim.x * 8);
  if (f0 < f1) {
    int n_taken = 0;
    Run run;
    // the next run, or false (with run.tiles == -1 at the end)
    auto take = [&]() {
      const int s = n_taken % kRuns;
      if (!wait_all(run_full + s, (n_taken / kRuns) & 1)) return false;
      run = s_runs[s];
      __syncwarp();
      if (lane == 0) mbar_arrive(run_empty + s);
      ++n_taken;
      return true;
    };
    if (warp == 13) {
      // ------------------------------------------------------------ the walk
      int item = s_start[0], off = s_start[1], f = f0, n_run = 0;
      bool ok = true;
      auto hand_out = [&](const Run& r) {
        const int s = n_run % kRuns;
        if (!wait_all(run_empty + s, ((n_run / kRuns) & 1) ^ 1)) return false;
        if (lane == 0) {
          s_runs[s] = r;
          mbar_arrive(run_full + s);
        }
        __syncwarp();
        ++n_run;
        return true;
      };
      Group next = {};
      for (bool primed = false; f < f1 && ok;) {
        const Group g = next;
        next = group_of<NC, kPTile>(p, min(primed ? item + 1 : item, n_items - 1));
        if (!primed) {
          primed = true;
          continue;
        }
        const int cost = key_cost(g);
        while (off < cost * p.Hkv && f < f1 && ok) {
          const int head = off / cost, at = off - head * cost;
          const int key_f0 = f - at, end = min(f1, key_f0 + cost);
          const int ta = min(at, g.tiles), tb = min(end - key_f0, g.tiles);
          if (ta < tb) {
            Run r = {};
            r.tiles = tb - ta;
            r.tile0 = g.tile0 + ta; r.b = g.b; r.head = head;
            r.kv = g.kv; r.n_q = g.n_q; r.q0 = g.q0; r.n_cols = g.n_cols;
            r.iq0 = g.c0 / p.G; r.rem0 = g.c0 - r.iq0 * p.G; r.lo = g.lo; r.hi = g.hi;
            r.dual = g.n_cols > kPTile;
            // (up to half a tile's columns: half 1 has them in its upper rows, whose
            // warps run on the other two of the SM's four schedulers)
            r.col0 = r.dual ? kPTile : g.n_cols <= kPTile / 2 ? -kPTile / 2 : 0;
            const int first_chunk = key_f0 / chunk, n_parts = (key_f0 + g.tiles - 1) / chunk - first_chunk + 1;
            const int inside = key_f0 > f0;
            r.whole = n_parts == 1;
            r.slot = 2 * blockIdx.x + inside;
            r.k_gsa = __ldg(p.k_gsa + head);
            r.v_gsa = __ldg(p.v_gsa + head);
            // this block holds a cut key's first part
            if (lane == 0 && n_parts > 1 && ta == 0)
              p.joins[blockIdx.x] = {n_parts, inside, g.q0 + r.iq0, r.rem0, g.n_cols, head, r.v_gsa, 0};
            ok = hand_out(r);
          }
          off += end - f;
          f = end;
        }
        off = 0;
        ++item;
      }
      if (ok) {
        Run r = {};
        r.tiles = -1;
        ok = hand_out(r);
      }
      if (!ok) give_up();
    } else if (warp == 12) {
      // -------------------------------------------------------- the products
      const uint32_t id_s = idesc_f16(128, kPTile, false), id_o = idesc_f16(128, D, true);
      int tk = 0, tv = 0;                                  // tiles of K and V taken
      uint32_t ph_q[2] = {0, 0}, ph_p[2] = {0, 0};
      auto products = [&]() -> bool {
        const uint32_t q_low = desc_low(smem + Sm::kQ, 16), k_low = desc_low(smem + Sm::kK, 16);
        const uint32_t v_low = desc_low(smem + Sm::kV, kPTile * 128);
        constexpr uint32_t kTileLow = Sm::kTileBytes >> 4;
        auto score = [&](int w, int stage) {
          const uint32_t q = q_low + w * kTileLow, k = k_low + stage * kTileLow, d = tmem + w * kPTile;
          if (elect_one()) {
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
              const uint32_t o = ((i / 4) * (kPTile * 128) + (i % 4) * 32) >> 4;
              tc_mma_f16(d, q + o, k + o, id_s, i != 0);
            }
          }
          __syncwarp();
        };
        auto weigh = [&](int w, int stage, bool add, int half) {
          const uint32_t v = v_low + stage * kTileLow, d = tmem + 2 * kPTile + w * D, a = tmem + w * kPTile;
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kPTile / 32; ++k) {
              // 16 tokens: two groups of eight 128-byte rows; 64-channel atoms a tile of rows apart
              const int i = half * (kPTile / 32) + k;
              tc_mma_f16_ta(d, a + 8 * i, v + (i * 2048 >> 4), id_o, add || i != 0);
            }
          }
          __syncwarp();
        };
        auto commit = [&](uint64_t* bar) {
          if (elect_one()) tc_commit(bar);
          __syncwarp();
        };
        auto have = [&](uint64_t* bar, uint32_t parity) {
          const bool ok = wait_all(bar, parity);
          tc_fence_after();
          return ok;
        };
        for (;;) {
          if (!take()) return false;
          const int n = run.tiles;
          if (n < 0) return true;
          const int k0 = tk, v0 = tv;
          tk += n;
          tv += n;
          auto k_ready = [&](int j) { return have(k_full + (k0 + j) % 2, ((k0 + j) / 2) & 1); };
          auto v_ready = [&](int j) { return have(v_full + (v0 + j) % 2, ((v0 + j) / 2) & 1); };
          auto q_ready = [&](int w) { const bool ok = have(q_full + w, ph_q[w]); ph_q[w] ^= 1u; return ok; };
          auto p_ready = [&](int w, int half) { return have((half ? p_full : p_half) + w, ph_p[w]); };
          // Row tile w: O += P V of its tile `cur`, then S of its tile `nxt`; both row
          // tiles walk all tiles (dual) or every other.  K and V of a tile wait for
          // its first reader and are free after its last.
          auto step = [&](bool dual, int w, int cur, int nxt) -> bool {
            const bool first = !dual || w == 0, last = !dual || w == 1;
            if (cur >= 0) {
              if ((first && !v_ready(cur)) || !p_ready(w, 0)) return false;
              weigh(w, (v0 + cur) % 2, cur > (dual ? 0 : 1), 0);
              commit(h_full + w);
              if (!p_ready(w, 1)) return false;
              ph_p[w] ^= 1u;
              weigh(w, (v0 + cur) % 2, true, 1);
              if (last) commit(v_empty + (v0 + cur) % 2);
            }
            if (nxt < n) {
              if (nxt < (dual ? 1 : 2) && !q_ready(w)) return false;
              if (first && !k_ready(nxt)) return false;
              score(w, (k0 + nxt) % 2);
              commit(s_full + w);
              if (nxt + (dual ? 1 : 2) >= n) commit(q_empty + w);
              if (last) commit(k_empty + (k0 + nxt) % 2);
            } else if (cur >= 0) {
              commit(o_full + w);
            }
            return true;
          };
          if (run.dual) {
#pragma unroll 1
            for (int j = -1; j < n; ++j)
              if (!step(true, 0, j, j + 1) || !step(true, 1, j, j + 1)) return false;
          } else {
#pragma unroll 1
            for (int j = -2; j < n; ++j)
              if (!step(false, j & 1, j, j + 2)) return false;
          }
        }
      };
      if (!products()) give_up();
      // nothing of this block's is under way when the tensor memory goes back
      if (elect_one()) tc_commit(drained);
      __syncwarp();
      wait_all(drained, 0);
    } else if (warp == 14) {
      // ------------------------------- the pages of the coming tiles into L2
      // (the expanding warps read one tile ahead, less than a trip to memory)
      const int S = 1 << p.page_shift, pieces = kPTile / S;
      int n_tile = 0;
      bool ok = true;
      while (ok) {
        ok = take() && run.tiles >= 0;
        const int32_t* table = p.page_table + static_cast<int64_t>(run.b) * p.max_pages;
        for (int j = 0; ok && j < run.tiles; ++j, ++n_tile) {
          const uint64_t limit = globaltimer_ns() + 1000000000ull;
          while (n_tile > *s_done + kAhead && !*abort_flag && globaltimer_ns() < limit) __nanosleep(100);
          const int t = (run.tile0 + j) * kPTile + lane * S;
          if (lane < pieces && t < run.hi && t + S > run.lo) {
            const int page = __ldg(table + (t >> p.page_shift));
            if (page >= 0 && page < p.n_pages)
              asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;"
                           :: "l"(p.cache + (static_cast<int64_t>(page) * p.Hkv + run.head) * KvPage<D>::bytes(S)),
                              "r"(KvPage<D>::bytes(S)) : "memory");
          }
          __syncwarp();
        }
      }
    } else if (warp == 15) {
      // -------------- the query rows of the coming run, raw into the halves' tiles
      const float inv_G = 1.0f / static_cast<float>(p.G);
      uint32_t sent[2] = {0, 0};
      auto queries = [&]() -> bool {
        for (;;) {
          if (!take()) return false;
          if (run.tiles < 0) return true;
          for (int w = 0; w < 2; ++w) {
            if (!run.dual && run.tiles <= w) continue;
            if (!wait_all(q_empty + w, (sent[w] & 1) ^ 1)) return false;
            ++sent[w];
            uint8_t* tile = smem + Sm::kQ + w * Sm::kTileBytes;
            // the columns [from, to) are in the tile; a query's lie next to each other
            const int c0 = w ? run.col0 : 0, from = max(c0, 0), to = min(c0 + kPTile, run.n_cols);
            if (lane == 0) mbar_arrive_expect_tx(q_raw + w, (to - from) * D * 2);
            __syncwarp();
            for (int dq = div_small(run.rem0 + from, inv_G) + lane; dq * p.G - run.rem0 < to; dq += 32) {
              const int a = max(from, dq * p.G - run.rem0), b = min(to, (dq + 1) * p.G - run.rem0);
              bulk_load(tile + (a - c0) * D * 2,
                        p.q + (run.q0 + run.iq0 + dq) * p.q_stride +
                            static_cast<int64_t>(run.head * p.G + run.rem0 + a - dq * p.G) * D,
                        (b - a) * D * 2, q_raw + w);
            }
            __syncwarp();
          }
        }
      };
      if (!queries()) give_up();
      if (*abort_flag) {
        // copies in flight land before the block's memory goes away
        const uint64_t drain = globaltimer_ns() + 1000000000ull;
        for (int w = 0; w < 2; ++w)
          while (sent[w] && !mbar_try_wait(q_raw + w, (sent[w] - 1) & 1))
            if (globaltimer_ns() > drain) break;
      }
    } else if (warp >= 8) {
      // ---------------------------------------------------- expanding the cache
      const int w = warp - 8, tok = lane & 7, qd = lane >> 3;
      const int S = 1 << p.page_shift;
      int n_tile = 0;                                      // tiles expanded
      constexpr int BL = D / 64;                           // blocks of 16 channels a lane takes of a token
      // Where this lane's codes and scales lie in the page of its warp's first 16
      // tokens, and how much further the other 16 are when they share the page
      // (pages of 32 tokens or more): the same in every tile, a tile holds whole
      // pages or lies in one
      const int o0 = ((32 * w) & (S - 1)) + tok;
      const uint32_t k_code = o0 * (D / 2) + qd * 8 * BL, k_scale = KvPage<D>::key_scales(S) + o0 * (D / 16) + qd * BL;
      const uint32_t v_code = KvPage<D>::value_codes(S) + KvPage<D>::value_code(o0, qd * BL);
      const uint32_t v_scale = KvPage<D>::value_scales(S) + KvPage<D>::value_scale(o0, qd * BL);
      const bool one_page = S >= 32;
      const uint32_t page_stride = static_cast<uint32_t>(p.Hkv) * KvPage<D>::bytes(S);
      auto expand = [&]() -> bool {
        for (;;) {
          if (!take()) return false;
          if (run.tiles < 0) return true;
          const int32_t* table = p.page_table + static_cast<int64_t>(run.b) * p.max_pages;
          uint2 kc[4][BL], vc[4][BL];
          uint32_t ks[4], vs[4][BL], k_mask[4], v_mask[4];
          // A half without its page reads the first page of the cache, under scales
          // of zero; so do the values of tokens outside [lo, hi), which no column sees
          // (whatever their bytes: a NaN scale would pass through a weight of zero).
          const uint8_t* head_at = p.cache + static_cast<int64_t>(run.head) * KvPage<D>::bytes(S);
          const uint8_t* base[2];                          // this head in the pages of the warp's two halves
          int limit[2];                                    // the tokens of a half from run.lo to this have scales
          int at = -1, entries = -1;
          // the pages of a tile; which are in the cache
          auto find = [&](int tile) {
            const int x = (tile * kPTile) >> p.page_shift; // the tile's first page
            if ((x & ~31) != at) {
              at = x & ~31;
              entries = at + lane < p.max_pages ? __ldg(table + at + lane) : -1;
            }
            const int t = tile * kPTile + 32 * w, e = (t >> p.page_shift) - at;
            int page = __shfl_sync(0xFFFFFFFFu, entries, e);
            bool ok = page >= 0 && page < p.n_pages;
            uint32_t live = ok ? 3u : 0u;
            ok = ok && t < run.hi && t + (one_page ? 32 : 16) > run.lo;
            base[0] = base[1] = head_at + static_cast<uint64_t>(static_cast<uint32_t>(ok ? page : 0)) * page_stride;
            limit[0] = limit[1] = ok ? run.hi : 0;
            if (!one_page) {                               // pages of 16: the second half's is the next
              page = __shfl_sync(0xFFFFFFFFu, entries, e + 1);
              ok = page >= 0 && page < p.n_pages;
              live = (live & 1u) | (ok ? 2u : 0u);
              ok = ok && t + 16 < run.hi && t + 32 > run.lo;
              base[1] = head_at + static_cast<uint64_t>(static_cast<uint32_t>(ok ? page : 0)) * page_stride;
              limit[1] = ok ? run.hi : 0;
            }
            return live;
          };
          const int step_c = one_page ? 16 * (D / 2) : 0, step_s = one_page ? 16 * (D / 16) : 0;
          auto load_k = [&](int tile) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint8_t* c = base[h] + (k_code + h * step_c);
              const uint8_t* s = base[h] + (k_scale + h * step_s);
              const int t = tile * kPTile + 32 * w + 16 * h + tok;
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                if (BL == 2) {
                  const uint4 u = __ldg(reinterpret_cast<const uint4*>(c + i * 8 * (D / 2)));
                  kc[2 * h + i][0] = make_uint2(u.x, u.y);
                  kc[2 * h + i][BL - 1] = make_uint2(u.z, u.w);
                  ks[2 * h + i] = __ldg(reinterpret_cast<const uint16_t*>(s + i * 8 * (D / 16)));
                } else {
                  kc[2 * h + i][0] = __ldg(reinterpret_cast<const uint2*>(c + i * 8 * (D / 2)));
                  ks[2 * h + i] = __ldg(s + i * 8 * (D / 16));
                }
                k_mask[2 * h + i] = t + 8 * i < limit[h] ? 0xFFFFu : 0u;
              }
            }
          };
          auto load_v = [&](int tile) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint8_t* c = base[h] + (v_code + h * step_c);
              const uint8_t* s = base[h] + (v_scale + h * step_s);
              const int t = tile * kPTile + 32 * w + 16 * h + tok;
#pragma unroll
              for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int x = 0; x < BL; ++x) {
                  vc[2 * h + i][x] = __ldg(reinterpret_cast<const uint2*>(c + i * 8 * (D / 2) + 64 * x));
                  vs[2 * h + i][x] = __ldg(s + i * 8 * (D / 16) + 8 * x);
                }
                v_mask[2 * h + i] = t + 8 * i < limit[h] && t + 8 * i >= run.lo ? 0xFFFFu : 0u;
              }
            }
          };
          // one group of eight tokens: codes times scales into the swizzled tile
          uint32_t odd = 0;
          // (A value's NaN would reach the columns that do not see it, through a weight of
          // zero: its scale becomes finite, the run's rows get their NaNs at its end.  386
          // and 113 us for the chunk and the ragged prompts, 384 and 111 without.)
          auto put = [&](uint8_t* tile, int i, const uint2 (&c)[BL], uint32_t two, bool value) {
            uint32_t s2 = e4m3x2_to_f16(two);
            if (value) {
              const uint32_t is = s2;
              s2 = h2_min(is, 0x5F005F00u);                // 448 in place of a NaN
              odd |= s2 ^ is;
            }
            uint8_t* row = tile + (32 * w + 8 * i + tok) * 128;
#pragma unroll
            for (int x = 0; x < BL; ++x) {
              const uint32_t sb = __byte_perm(s2, 0, x == 0 ? 0x1010 : 0x3232);
              uint32_t a[8];
              e2m1x8_to_f16(c[x].x, a[0], a[1], a[2], a[3]);
              e2m1x8_to_f16(c[x].y, a[4], a[5], a[6], a[7]);
#pragma unroll
              for (int y = 0; y < 8; ++y) a[y] = h2_mul(a[y], sb);
              const int blk = qd * BL + x;                 // channels 16 blk ..
              uint8_t* atom = row + (blk / 4) * (kPTile * 128);
              const int ch = 2 * (blk % 4);
              *reinterpret_cast<uint4*>(atom + ((ch ^ tok) << 4)) = make_uint4(a[0], a[1], a[2], a[3]);
              *reinterpret_cast<uint4*>(atom + (((ch + 1) ^ tok) << 4)) = make_uint4(a[4], a[5], a[6], a[7]);
            }
          };
          uint32_t live = find(run.tile0);
          load_k(run.tile0);
          load_v(run.tile0);
          for (int j = 0; j < run.tiles; ++j, ++n_tile) {
            const int st = n_tile % 2;
            const uint32_t ph = ((n_tile / 2) & 1) ^ 1;
            if (!wait_all(k_empty + st, ph)) return false;
#pragma unroll
            for (int i = 0; i < 4; ++i) put(smem + Sm::kK + st * Sm::kTileBytes, i, kc[i], ks[i] & k_mask[i], false);
            fence_proxy_async_smem();
            __syncwarp();
            // this warp's byte of the word: its two groups of 16 tokens
            if (lane == 0) {
              reinterpret_cast<volatile uint8_t*>(s_live + n_tile % kLive)[w] = static_cast<uint8_t>(live);
              mbar_arrive(k_full + st);
            }
            const int more = run.tile0 + j + 1;
            uint32_t live_next = 0;
            if (j + 1 < run.tiles) {
              live_next = find(more);
              load_k(more);
            }
            if (!wait_all(v_empty + st, ph)) return false;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              put(smem + Sm::kV + st * Sm::kTileBytes, i, vc[i], (vs[i][0] | (vs[i][BL - 1] << 8)) & v_mask[i], true);
            if (odd) reinterpret_cast<volatile Run*>(s_runs + (n_taken - 1) % kRuns)->nan = 1;
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(v_full + st);
            if (w == 0 && lane == 0) *s_done = n_tile + 1;
            if (j + 1 < run.tiles) load_v(more);
            live = live_next;
          }
        }
      };
      if (!expand()) give_up();
    } else {
      // ------------------------------------------------------------- softmax
      const int w = warp >> 2, wl = warp & 3, row = tid & 127;
      const uint32_t lanes = static_cast<uint32_t>(wl * 32) << 16;
      const uint32_t t_s = tmem + lanes + w * kPTile, t_o = tmem + lanes + 2 * kPTile + w * D;
      const float inv_G = 1.0f / static_cast<float>(p.G);
      uint32_t ph_h = 0, ph_q = 0, ph_s = 0, ph_o = 0, ph_meet = 0, ph_x = 0;
      int n_tile = 0;                                      // tiles before the run
      auto sync_half = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(meet + w);
        const bool ok = wait_all(meet + w, ph_meet);
        ph_meet ^= 1u;
        return ok;
      };
      // A run stays in shared memory meanwhile: its fields are read where they are needed.
      auto my_tiles = [&](const volatile Run& run) { return run.dual ? run.tiles : (run.tiles + 1 - w) / 2; };
      auto col_of = [&](const volatile Run& run) { return w == 0 ? row : row + run.col0; };
      auto is_on = [&](const volatile Run& run) {
        return static_cast<uint32_t>(col_of(run)) < static_cast<uint32_t>(run.n_cols);
      };
      // the query of the row, and its row of the result
      auto quotient = [&](const volatile Run& run) {
        return div_small(run.rem0 + (is_on(run) ? col_of(run) : 0), inv_G);
      };
      auto out_row = [&](const volatile Run& run) {
        const int dq = quotient(run);
        return static_cast<int64_t>(run.q0 + run.iq0 + dq) * p.Hq + run.head * p.G + run.rem0 +
               (is_on(run) ? col_of(run) : 0) - dq * p.G;
      };
      float to_log2 = 0.0f, m_neg = INFINITY, l = 0.0f;
      // ---- a run's queries: the raw row of each thread, scaled into fp16's range,
      // into the swizzled tile.  Vector f(i) of a row is its thread's i-th: with f(i)
      // = i xor (x times the row) in GF(8), both f and f xor the row (the swizzle)
      // take all values over eight rows: neither side has bank conflicts.
      auto start = [&](const volatile Run& run) -> bool {
        if (my_tiles(run) == 0) return true;
        uint8_t* tile = smem + Sm::kQ + w * Sm::kTileBytes;
        if (!wait_all(q_raw + w, ph_q)) return false;
        ph_q ^= 1u;
        const bool on = is_on(run);
        const int turn = ((row << 1) ^ (row & 4 ? 3 : 0)) & 7;
        uint4 u[D / 8];
        uint32_t big2 = 0;                                 // the largest magnitudes of the even and odd channels
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          u[i] = on ? *reinterpret_cast<const uint4*>(tile + row * D * 2 + ((i & 8) | ((i ^ turn) & 7)) * 16)
                    : make_uint4(0u, 0u, 0u, 0u);
          const uint32_t v[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            asm("max.u16x2 %0, %0, %1;" : "+r"(big2) : "r"(v[k] & 0x7FFF7FFFu));
        }
        if (!sync_half()) return false;
        float up, down;
        query_scale(max(big2 & 0xFFFFu, big2 >> 16), up, down);
        to_log2 = down * (p.scale_log2 * run.k_gsa);
#pragma unroll
        for (int i = 0; i < D / 8; ++i) {
          const uint32_t v[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
          uint32_t h[4];
#pragma unroll
          for (int k = 0; k < 4; ++k)
            h[k] = pack_f16(__uint_as_float(v[k] << 16) * up, __uint_as_float(v[k] & 0xFFFF0000u) * up);
          *reinterpret_cast<uint4*>(tile + (i / 8) * (kPTile * 128) + row * 128 + (((i ^ turn ^ row) & 7) << 4)) =
              make_uint4(h[0], h[1], h[2], h[3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(q_full + w);
          if (run.dual) mbar_arrive(q_empty + w);          // (this half has nothing more to do with the tile)
        }
        return true;
      };
      // ---- its tiles
      auto weigh = [&](const volatile Run& run) -> bool {
        const int n_my = my_tiles(run);
        const bool on = is_on(run), any_on = __any_sync(0xFFFFFFFFu, on);
        const int pos = run.kv - run.n_q + run.iq0 + quotient(run);
        const int hi = !on ? 0 : p.causal ? pos + 1 : run.kv;
        const int lo = p.window > 0 ? pos + 1 - p.window : 0;
        m_neg = INFINITY;
        l = 0.0f;
        for (int i = 0; i < n_my; ++i) {
          const int j = run.dual ? i : 2 * i + w;
          const int t0 = (run.tile0 + j) * kPTile;
          if (!wait_all(s_full + w, ph_s)) return false;
          ph_s ^= 1u;
          tc_fence_after();
          if (!any_on) {
            // (rows that nobody asked for: their P may be anything)
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(p_half + w);
              mbar_arrive(p_full + w);
            }
            ph_h ^= 1u;
            continue;
          }
          const uint32_t bytes = s_live[(n_tile + j) % kLive];
          // bit i: tokens 16 i .. of the tile are in the cache
          const uint32_t live = (bytes & 3u) | ((bytes >> 6) & 0xCu) | ((bytes >> 12) & 0x30u) | ((bytes >> 18) & 0xC0u);
          const bool masked = __any_sync(0xFFFFFFFFu, t0 + kPTile > hi || t0 < lo || live != 0xFFu);
          // bit x: the row sees token t0 + c + x (c a multiple of 32)
          const int from = lo - t0, to = hi - t0;
          auto seen32 = [&](int c) {
            const int a = min(max(from - c, 0), 32), b = min(max(to - c, 0), 32);
            const uint32_t m = (a < 32 ? 0xFFFFFFFFu << a : 0u) & (b > 0 ? 0xFFFFFFFFu >> (32 - b) : 0u);
            const uint32_t two = live >> (c / 16);
            return m & ((two & 1u ? 0xFFFFu : 0u) | (two & 2u ? 0xFFFF0000u : 0u));
          };
          // In two halves of 64 tokens: P V of the first starts under the second.
#pragma unroll 1
          for (int c0 = 0; c0 < kPTile; c0 += kPTile / 2) {
            uint32_t pr[kPTile / 4];
            float sum;
            auto weights = [&](auto hidden) {              // hidden: some tokens are not seen
              uint64_t sum2 = f2_pack(0.0f, 0.0f);
              const uint64_t k2 = f2_pack(to_log2, to_log2), m2 = f2_pack(m_neg, m_neg);
              uint32_t s[2][32];
              tmem_load32_start(t_s + c0, s[0]);
#pragma unroll
              for (int c = 0; c < kPTile / 2; c += 32) {
                uint32_t (&now)[32] = s[(c / 32) % 2];
                tmem_load32_finish(now);
                if (c + 32 < kPTile / 2) tmem_load32_start(t_s + c0 + c + 32, s[(c / 32 + 1) % 2]);
                const uint32_t see = hidden ? seen32(c0 + c) : 0xFFFFFFFFu;
#pragma unroll
                for (int x = 0; x < 32; x += 2) {
                  const uint64_t v =
                      f2_fma(f2_pack(__uint_as_float(now[x]), __uint_as_float(now[x + 1])), k2, m2);
                  float v0 = f2_lo(v), v1 = f2_hi(v);
                  if (hidden) {
                    v0 = see & (1u << x) ? v0 : -INFINITY;
                    v1 = see & (2u << x) ? v1 : -INFINITY;
                  }
                  const float a = ex2(v0), b = ex2(v1);
                  sum2 = f2_add(sum2, f2_pack(a, b));
                  pr[(c + x) / 2] = pack_f16(a, b);
                }
              }
              sum = f2_lo(sum2) + f2_hi(sum2);
            };
            // Weights that add up to more than 2^kMostWeight hold a score far above the
            // largest that m was set by (a weight above 4 times its 2^kLift, at least): no
            // maximum is taken of the others.  (No score above it: at most 64 weights of
            // 2^kLift.)
            for (bool move = i == 0 && c0 == 0;; move = true) {
              if (move) {
                // m is set by the largest score so far, this half's included
                float top = -INFINITY;
#pragma unroll 1
                for (int c = c0; c < c0 + kPTile / 2; c += 32) {
                  uint32_t s[32];
                  tmem_load32_start(t_s + c, s);
                  tmem_load32_finish(s);
                  const uint32_t see = masked ? seen32(c) : 0xFFFFFFFFu;
#pragma unroll
                  for (int x = 0; x < 32; ++x)
                    top = fmaxf(top, see & (1u << x) ? __uint_as_float(s[x]) * to_log2 : -INFINITY);
                }
                const float now = fminf(m_neg, kLift - top);
                const float shrink = now < m_neg ? ex2(now - m_neg) : 1.0f;
                m_neg = now;
                l *= shrink;
                if (i > 0 || c0 > 0) {
                  // (earlier tiles are in O, S came after them; the first half may be on its way)
                  if (c0 > 0) {
                    if (!wait_all(h_full + w, ph_h)) return false;
                    tc_fence_after();
                  }
#pragma unroll 1
                  for (int c = 0; c < D; c += 16) {
                    float o[16];
                    uint32_t y[16];
                    tmem_load16(t_o + c, o);
#pragma unroll
                    for (int x = 0; x < 16; ++x) y[x] = __float_as_uint(o[x] * shrink);
                    tmem_store16(t_o + c, y);
                  }
                }
              }
              if (masked) weights(std::true_type{});
              else weights(std::false_type{});
              if (move || !__any_sync(0xFFFFFFFFu, sum > kMostSum)) break;
            }
            l += sum;
            // P over the columns of S that have been read
#pragma unroll
            for (int c = 0; c < kPTile / 4; c += 16) {
              uint32_t x[16];
#pragma unroll
              for (int k = 0; k < 16; ++k) x[k] = pr[c + k];
              tmem_store16(t_s + c0 / 2 + c, x);
            }
            tmem_store_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive((c0 ? p_full : p_half) + w);
          }
          ph_h ^= 1u;
        }
        n_tile += run.tiles;
        if (n_my > 0) {
          if (!wait_all(o_full + w, ph_o)) return false;
          ph_o ^= 1u;
          tc_fence_after();
        }
        return true;
      };
      // NaNs for the rows that see a value with NaNs among its scales, in its 16 channels:
      // the run's scales once more, 32 tokens at a time (of no consequence for the time of a
      // cache that append has written, which holds none).
      auto give_nans = [&](const volatile Run& run) {
        const bool on = is_on(run);
        const int pos = run.kv - run.n_q + run.iq0 + quotient(run);
        const int hi = !on ? 0 : p.causal ? pos + 1 : run.kv, lo = p.window > 0 ? pos + 1 - p.window : 0;
        const int from = max(run.lo, run.tile0 * kPTile), to = min(run.hi, (run.tile0 + run.tiles) * kPTile);
        const int S = 1 << p.page_shift;
        uint32_t blocks = 0;
#pragma unroll 1
        for (int t0 = from & ~31; t0 < to; t0 += 32) {
          const int t = t0 + lane;
          const int page = t >= from && t < to ? __ldg(p.page_table + static_cast<int64_t>(run.b) * p.max_pages + (t >> p.page_shift)) : -1;
          const bool have = page >= 0 && page < p.n_pages;
          const uint8_t* at = p.cache + (static_cast<int64_t>(have ? page : 0) * p.Hkv + run.head) * KvPage<D>::bytes(S) +
                              KvPage<D>::value_scales(S) + KvPage<D>::value_scale(t & (S - 1), 0);
#pragma unroll 1
          for (int b = 0; b < D / 16; ++b) {
            const bool nan = have && (__ldg(at + KvPage<D>::value_scale(0, b)) & 0x7Fu) == 0x7Fu;
            if (__ballot_sync(0xFFFFFFFFu, nan) & tokens32(t0, lo, hi)) blocks |= 1u << b;
          }
        }
#pragma unroll 1
        for (int b = 0; b < D / 16; ++b) {
          float o[16];
          uint32_t y[16];
          tmem_load16(t_o + 16 * b, o);
#pragma unroll
          for (int x = 0; x < 16; ++x) y[x] = (blocks >> b) & 1u ? 0x7FFFFFFFu : __float_as_uint(o[x]);
          tmem_store16(t_o + 16 * b, y);
        }
        tmem_store_wait();
      };
      // ---- its rows
      auto finish = [&](const volatile Run& run) -> bool {
        const int col = col_of(run);
        const bool on = is_on(run);
        float m = -m_neg;
        // both halves on one set of rows: half 1 hands its rows over, through the
        // query tiles (their scores are complete)
        const bool cross = !run.dual && run.tiles > 1;
        float keep = 1.0f, other = 0.0f;
        const int x_row = col & (kPTile - 1);
        float* x_rows = reinterpret_cast<float*>(smem + Sm::kQ) + x_row * D;
        if (cross) {
          if (w == 0) {
            __syncwarp();
            if (lane == 0) mbar_arrive(x_ready);           // (its scores are done with the queries)
            if (!wait_all(x_full, ph_x)) return false;
            const float m1 = s_row[x_row], l1 = s_row[kPTile + x_row];
            const float top = fmaxf(m, m1), base = top == -INFINITY ? 0.0f : top;
            keep = ex2(m - base);
            other = ex2(m1 - base);
            l = l * keep + l1 * other;
            m = top;
          } else {
            if (!wait_all(x_ready, ph_x)) return false;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              float o[32];
              tmem_load32(t_o + c, o);
#pragma unroll
              for (int x = 0; x < 32; x += 4)
                *reinterpret_cast<float4*>(x_rows + c + (((x / 4) ^ (row & 7)) * 4)) =
                    make_float4(o[x], o[x + 1], o[x + 2], o[x + 3]);
            }
            s_row[x_row] = m;
            s_row[kPTile + x_row] = l;
            __syncwarp();
            if (lane == 0) mbar_arrive(x_full);
            if (!wait_all(x_free, ph_x)) return false;
          }
          ph_x ^= 1u;
        }
        if (run.dual || w == 0) {
          if (run.nan) give_nans(run);
          const bool whole = run.whole;
          float* part = p.partials + static_cast<size_t>(run.slot) * NC * (D + 2);
          const float inv = out_factor(run.v_gsa, l);
          // 128 bytes of each row at a time through shared memory, so that the warp
          // stores whole lines; 16-byte vectors are swizzled by the row
          uint8_t* rows_at = smem + Sm::kOut + warp * 32 * 128;
          // (a lane stores vector lane % 8 of every fourth row)
          const int64_t row_at = whole ? out_row(run) * (D * 2) : static_cast<int64_t>(col) * (D * 4);
          const uint32_t rows_on = __ballot_sync(0xFFFFFFFFu, on) >> (lane / 8);
          uint8_t* base = whole ? reinterpret_cast<uint8_t*>(p.out) : reinterpret_cast<uint8_t*>(part + 2 * NC);
          uint8_t* to[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            to[i] = base + __shfl_sync(0xFFFFFFFFu, row_at, 4 * i + lane / 8) + (lane % 8) * 16;
          auto put_vector = [&](int i, uint4 v) {
            *reinterpret_cast<uint4*>(rows_at + lane * 128 + (((i ^ lane) & 7) << 4)) = v;
          };
          // every row's eight vectors, to byte `at` of each row's place
          auto store_rows = [&](int at) {
            __syncwarp();
            const int r = lane / 8;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const uint4 v = *reinterpret_cast<const uint4*>(rows_at + (4 * i + r) * 128 +
                                                              (((lane ^ (4 * i + r)) & 7) << 4));
              if ((rows_on >> (4 * i)) & 1u) *reinterpret_cast<uint4*>(to[i] + at) = v;
            }
            __syncwarp();
          };
#pragma unroll 1
          for (int c = 0; c < D; c += 32) {
            float o[32];
            tmem_load32(t_o + c, o);
            if (cross) {
#pragma unroll
              for (int x = 0; x < 32; x += 4) {
                const float4 y = *reinterpret_cast<const float4*>(x_rows + c + (((x / 4) ^ (row & 7)) * 4));
                o[x] = o[x] * keep + y.x * other;
                o[x + 1] = o[x + 1] * keep + y.y * other;
                o[x + 2] = o[x + 2] * keep + y.z * other;
                o[x + 3] = o[x + 3] * keep + y.w * other;
              }
            }
            if (whole) {
              // (a row that saw nothing has l = 0; what lies in its accumulator is finite)
#pragma unroll
              for (int x = 0; x < 32; x += 8) {
                uint32_t h[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const __nv_bfloat162 y = __floats2bfloat162_rn(o[x + 2 * k] * inv, o[x + 2 * k + 1] * inv);
                  h[k] = *reinterpret_cast<const uint32_t*>(&y);
                }
                put_vector((c % 64 + x) / 8, make_uint4(h[0], h[1], h[2], h[3]));
              }
              if (c % 64) store_rows((c - 32) * 2);
            } else {
#pragma unroll
              for (int x = 0; x < 32; x += 4)
                put_vector(x / 4, make_uint4(__float_as_uint(o[x]), __float_as_uint(o[x + 1]),
                                             __float_as_uint(o[x + 2]), __float_as_uint(o[x + 3])));
              store_rows(c * 4);
            }
          }
          if (cross) {
            __syncwarp();
            if (lane == 0) mbar_arrive(x_free);
          }
          if (whole) {
            if (on && p.lse) p.lse[out_row(run)] = lse_of(m, l);
          } else if (on) {
            part[col] = m;
            part[NC + col] = l;
          }
        }
        tc_fence_before();
        if (!run.dual && my_tiles(run) > 0) {
          fence_proxy_async_smem();                        // (rows went through the query tiles)
          __syncwarp();
          if (lane == 0) mbar_arrive(q_empty + w);
        }
        return true;
      };
      auto softmax = [&]() -> bool {
        for (int n = 0;; ++n) {
          const int s = n % kRuns;
          if (!wait_all(run_full + s, (n / kRuns) & 1)) return false;
          const volatile Run& run = s_runs[s];
          if (run.tiles < 0) return true;
          if (!start(run) || !weigh(run) || !finish(run)) return false;
          __syncwarp();
          if (lane == 0) mbar_arrive(run_empty + s);
        }
      };
      if (!softmax()) give_up();
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 12) tmem_dealloc(tmem, 512);
}

template <int D>
nvr_status launch(AttnParams& p, int max_kv, cudaStream_t s) {
  using Sm = PrefillSmem<D>;
  static_assert(Sm::kTotal <= 227 * 1024, "shared memory");
  static bool attr_set[kMaxDevices] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return NVR_ERR_CUDA;
  const int sms = device_sm_count();
  if (sms <= 0) return NVR_ERR_CUDA;
  if (!attr_set[dev]) {
    const cudaError_t e =
        cudaFuncSetAttribute(kv_prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Sm::kTotal);
    if (e != cudaSuccess) return cuda_status(e);
    attr_set[dev] = true;
  }
  p.groups = static_cast<int>((static_cast<int64_t>(p.max_q) * p.G + kPrefillCols - 1) / kPrefillCols);
  const int64_t items = static_cast<int64_t>(p.B) * p.groups;
  const int64_t most = items * p.Hkv * ((max_kv + kPTile - 1) / kPTile + 1 + kPKeyCost);
  if (items >= (int64_t(1) << 30) || most >= (int64_t(1) << 31) - (1 << 24)) return NVR_ERR_UNSUPPORTED;
  int64_t grid = sms < kPrefillMaxCtas ? sms : kPrefillMaxCtas;
  if (grid > most) grid = most;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kPThreads);
  cfg.dynamicSmemBytes = Sm::kTotal;
  cfg.stream = s;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kv_prefill_kernel<D>, p);
  if (e != cudaSuccess) return cuda_status(e);
  return launch_kv_join(p, D, static_cast<int>(grid), kPrefillCols, items * p.Hkv, s);
}

}  // namespace

nvr_status launch_kv_prefill(AttnParams& p, int D, int max_kv, cudaStream_t s) {
  return D == 128 ? launch<128>(p, max_kv, s) : launch<64>(p, max_kv, s);
}

}  // namespace nvr
