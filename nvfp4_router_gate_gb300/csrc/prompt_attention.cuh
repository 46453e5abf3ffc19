// prompt_attention.cuh -- what the kernels of prompt_attention share: parameters,
// the rows and tokens of a group of queries, the workspace (sm_103a).
#pragma once

#include <cuda_fp16.h>

#include "kv_attention.cuh"

namespace nvr {

constexpr int kPaTile = 128;               // tokens of a tile, rows of a row tile
constexpr int kPaRows = 2 * kPaTile;       // rows of a key: two row tiles
constexpr int kPaMaxCtas = 160;

struct PromptParams {
  CUtensorMap tm_q, tm_k, tm_v;
  int64_t T, Tk;
  int Hq, G;
  int Gt, chunks, Hv;                      // heads of a row tile; row tiles' head groups of a KV head, of all
  int qt;                                  // queries of a row tile: Gt * qt <= 128 rows
  const int32_t *cu_q, *cu_k;
  int B, max_q, max_k;
  float scale_log2;                        // scale * log2(e)
  int causal, window;
  int span, groups;                        // queries of a group (one or two row tiles), groups of a sequence
  const uint16_t* v;
  int64_t v_stride, v_head;
  const uint16_t* prefix_out;
  const float* prefix_lse;
  uint16_t* out;
  float* lse;
  uint32_t* status;
  int min_chunk;                           // places of a block at least
  // [blocks][8 warps of rows]: written parts of the key whose first one is the block's; zero
  // between calls
  uint32_t* arrived;
  uint32_t* handed;                        // keys handed out behind the blocks' first ones; zero between calls
  // [2 * blocks][256 m, 256 l, D / 4 x 256 x 4 O]: a block's first stretch is in its slot 0 when it
  // is part of a cut key, its last one in slot 1 unless the key starts the chunk
  float* partials;
};

// A key: the queries of a sequence that one block takes, for one group of heads.
struct PromptGroup {
  int b, q0, k0;                           // sequence, its first rows of q and of k
  int i0, n;                               // first query of the group, its queries (0: none)
  int shift, kmax;                         // position of query i: shift + i; keys that exist
  int tile0, tiles;                        // key tiles that some row sees
  int first[2], last[2];                   // of each row tile, from tile0: [first, last)
};

// The keys that a query of a position sees: [begin, end)
__device__ __forceinline__ int seen_end(int causal, int pos, int kmax) {
  return causal ? min(max(pos + 1, 0), kmax) : kmax;
}
__device__ __forceinline__ int seen_begin(int window, int pos) {
  return window > 0 ? max(max(pos + 1, 0) - window, 0) : 0;
}

__device__ __forceinline__ PromptGroup prompt_group(const PromptParams& p, int item) {
  PromptGroup g;
  // (a sequence's last queries, which see most, come first)
  const int turn = item / p.B;
  g.b = item - turn * p.B;
  g.i0 = (p.groups - 1 - turn) * p.span;
  int n_q, n_k;
  if (p.cu_q) {
    const int64_t a = min(max(static_cast<int64_t>(__ldg(p.cu_q + g.b)), int64_t(0)), p.T);
    n_q = static_cast<int>(min(max(static_cast<int64_t>(__ldg(p.cu_q + g.b + 1)), a), p.T) - a);
    g.q0 = static_cast<int>(a);
  } else {
    g.q0 = g.b * p.max_q;
    n_q = p.max_q;
  }
  if (p.cu_k) {
    const int64_t a = min(max(static_cast<int64_t>(__ldg(p.cu_k + g.b)), int64_t(0)), p.Tk);
    n_k = static_cast<int>(min(max(static_cast<int64_t>(__ldg(p.cu_k + g.b + 1)), a), p.Tk) - a);
    g.k0 = static_cast<int>(a);
  } else {
    g.k0 = g.q0;
    n_k = n_q;
  }
  g.shift = n_k - n_q;
  g.kmax = min(n_k, p.max_k);
  g.n = max(min(min(n_q, p.max_q) - g.i0, p.span), 0);
  int begin = INT32_MAX, end = 0;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int a = g.shift + g.i0 + w * p.qt, m = min(g.n - w * p.qt, p.qt);
    const int hi = m > 0 ? seen_end(p.causal, a + m - 1, g.kmax) : 0, lo = min(seen_begin(p.window, a), hi);
    g.first[w] = lo / kPaTile;
    g.last[w] = hi > lo ? (hi + kPaTile - 1) / kPaTile : g.first[w];
    if (hi > lo) {
      begin = min(begin, g.first[w]);
      end = max(end, g.last[w]);
    }
  }
  g.tile0 = end > 0 ? begin : 0;
  g.tiles = max(end - g.tile0, 0);
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    if (g.first[w] >= g.last[w]) g.first[w] = g.last[w] = g.tile0;
    g.first[w] -= g.tile0;
    g.last[w] -= g.tile0;
  }
  return g;
}

// lse of the own keys and of the prefix's: the factors of both results, the lse of all.
// (A prefix of which nothing was seen does not count, whatever its rows hold.)
__device__ __forceinline__ float join_prefix(float own, float before, float& f_own, float& f_before) {
  const float top = fmaxf(own, before);
  if (top == -INFINITY) {
    f_own = own != own ? own : 0.0f;
    f_before = before != before ? before : 0.0f;
    return own + before;
  }
  const float a = ex2((own - top) * 1.44269504088896341f), b = ex2((before - top) * 1.44269504088896341f);
  const float s = a + b;
  f_own = a / s;
  f_before = b / s;
  return top + logf(s);
}

template <bool kF16>
__device__ __forceinline__ uint32_t pack_16(float lo, float hi) {
  uint32_t d;
  if (kF16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
template <bool kF16>
__device__ __forceinline__ float2 unpack_16(uint32_t u) {
  if (kF16) return __half22float2(*reinterpret_cast<const __half2*>(&u));
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
}

}  // namespace nvr
