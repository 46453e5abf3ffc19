// kv_attention.cuh -- what the two attention kernels over the NVFP4 key/value
// cache share: parameters, the rows and tokens of a column group, and small
// device functions (sm_103a).
#pragma once

#include "kv_layout.cuh"
#include "nvr_internal.h"
#include "nvr_tcgen05.cuh"

namespace nvr {

// A row's weights are 2^(s - m) with m set to its largest score less kLift (base 2), and
// set again when one passes 2^kMostWeight: between those of the largest score at the
// upper end of fp16 (2^16) and the smallest that its subnormals hold lie 2^32, so that
// the many small weights beside a dominant token still count.
constexpr float kLift = 7.0f;
constexpr float kMostWeight = 15.0f;

// Fewest places of a block in the flat order of the tiles.
constexpr int kMinChunk = 2;

// A key that a chunk border cuts, written by the share (a block's or a team's) that has
// its first chunk: its parts, whether the first lies in the share's second slot, its rows.
struct KeyJoin {
  int n_parts, tail;
  int q0, rem0, n_cols;       // the first column is head rem0 of the KV head's at query row q0
  int head;
  float v_gsa;
  int pad;
};

struct AttnParams {
  const __nv_bfloat16* q;
  int64_t q_stride;
  int64_t T;
  int Hq, Hkv, G;
  const uint8_t* cache;
  int64_t n_pages;
  int page_shift;
  const int32_t* page_table;
  int B, max_pages;
  const int32_t* kv_lens;
  const int32_t* cu_q;
  int max_q;
  const float *k_gsa, *v_gsa;
  float scale_log2;           // scale * log2(e)
  int causal, window;
  int groups;                 // column groups per sequence
  __nv_bfloat16* out;
  float* lse;
  uint32_t* status;
  KeyJoin* joins;             // [shares]
  // [2 * shares][NC m, NC l, NC x D O]: a share's first run is in its slot 0 when it
  // is part of a cut key, its last one in slot 1 unless the key starts the chunk
  float* partials;
};

// What the queries and the tokens of a column group are.
struct Group {
  int b, q0, n_q, kv;         // sequence, its first query row, its queries (max_q of them have columns), its tokens
  int c0, n_cols;             // first column, columns of the group (0: none)
  int lo, hi;                 // tokens any of the columns sees: [lo, hi)
  int tile0, tiles;
};

template <int NC, int TILE>
__device__ __forceinline__ Group group_of(const AttnParams& p, int item) {
  Group g;
  g.b = item / p.groups;
  const int cg = item - g.b * p.groups;
  g.kv = min(max(__ldg(p.kv_lens + g.b), 0), p.max_pages << p.page_shift);
  if (p.cu_q) {
    const int64_t a = min(max(static_cast<int64_t>(__ldg(p.cu_q + g.b)), int64_t(0)), p.T);
    const int64_t e = min(max(static_cast<int64_t>(__ldg(p.cu_q + g.b + 1)), a), p.T);
    g.q0 = static_cast<int>(a);
    g.n_q = static_cast<int>(e - a);
  } else {
    g.q0 = g.b * p.max_q;
    g.n_q = p.max_q;
  }
  g.c0 = cg * NC;
  g.n_cols = min(min(g.n_q, p.max_q) * p.G - g.c0, NC);
  if (g.n_cols <= 0) {
    g.n_cols = 0;
    g.lo = g.hi = g.tile0 = g.tiles = 0;
    return g;
  }
  g.lo = 0;
  g.hi = g.kv;
  if (p.causal) {
    const int first = g.kv - g.n_q + g.c0 / p.G;                       // position of the first column's query
    const int last = g.kv - g.n_q + (g.c0 + g.n_cols - 1) / p.G;
    g.hi = max(last + 1, 0);
    if (p.window > 0) g.lo = min(max(first + 1 - p.window, 0), g.hi);
  }
  g.tile0 = g.lo / TILE;
  g.tiles = max((g.hi + TILE - 1) / TILE - g.tile0, 1);                // a group that sees nothing still writes its rows
  return g;
}

// Zeros, and an lse of -inf, for the rows that no sequence covers: in front of the first
// one, behind the last one (a batch padded for a captured graph), past max_q in one.  By
// the warps `unit` of `units`, while the first loads of the work are under way.
template <int D>
__device__ __forceinline__ void clear_uncovered(const AttnParams& p, int unit, int units) {
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

// Waits for a phase of the barrier, about a second at most: a try that fails
// takes 4 us on this GPU (measured), and 2^18 of them are made.  A count keeps the
// wait to a few instructions; there are many waits, and the kernels' rarely run
// parts are bound by fetching their instructions.
__device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
#pragma unroll 1
  for (int n = 0; n < (1 << 18); ++n) {
    if (mbar_try_wait(bar, parity)) return true;
    if (*abort_flag) return false;
  }
  return false;
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

// What a row's result is multiplied by, and its lse: a row that sees no token has a sum
// of 0 (zeros and -inf), one with a NaN among its scores a NaN, which both keep.
__device__ __forceinline__ float out_factor(float v_gsa, float sum) {
  return sum == 0.0f ? 0.0f : __fdividef(v_gsa, sum);
}
__device__ __forceinline__ float lse_of(float top, float sum) {
  return sum == 0.0f ? -INFINITY : (top + log2f(sum)) * 0.693147180559945309f;
}

// Bit i: token t + i is in [lo, hi).
__device__ __forceinline__ uint32_t tokens32(int t, int lo, int hi) {
  const int a = min(max(lo - t, 0), 32), b = min(max(hi - t, 0), 32);
  return (a < 32 ? 0xFFFFFFFFu << a : 0u) & (b > 0 ? 0xFFFFFFFFu >> (32 - b) : 0u);
}

// x / G for the small numerators of a group (below 2^17, G at most 2^16):
// exact in fp32, the quotient's distance from an integer is at least 1 / (2 G).
__device__ __forceinline__ int div_small(int x, float inv_G) {
  return static_cast<int>((static_cast<float>(x) + 0.5f) * inv_G);
}

// 2^(14 - exponent of the largest magnitude) brings a row of bf16 queries into
// the upper range of fp16 (fewer significant bits: exact, but for channels 2^28
// below the largest, which lose their last bits).  `big`: the largest magnitude's
// bf16 bits; up and its inverse are normal fp32 numbers.
__device__ __forceinline__ void query_scale(uint32_t big, float& up, float& down) {
  const int e = min(max(static_cast<int>(big >> 7), 16), 254);
  up = __uint_as_float(static_cast<uint32_t>(268 - e) << 23);
  down = __uint_as_float(static_cast<uint32_t>(e - 14) << 23);
}

// Workspace of an attention call (csrc/kv_attention.cu): control words, the cut
// keys, the partial results.
constexpr int kAttnMaxShares = 2048;    // teams of the streaming kernel at most
constexpr int kPrefillMaxCtas = 160;       // blocks of the tensor-memory kernel
constexpr int kPrefillCols = 256;          // its columns
constexpr int kAttnMaxCols = 16384;        // columns * teams of the streaming kernel at most
static_assert(kPrefillMaxCtas * kPrefillCols >= kAttnMaxCols, "the partials hold either kernel's");

// Joins the cut keys of `blocks` blocks, of `keys` keys at most (csrc/kv_join.cu);
// the last launch of a call.
nvr_status launch_kv_join(const AttnParams& p, int D, int blocks, int NC, int64_t keys, cudaStream_t s);

// The tensor-memory kernel (csrc/kv_prefill.cu).
nvr_status launch_kv_prefill(AttnParams& p, int D, int max_kv, cudaStream_t s);

}  // namespace nvr
