// kv_join.cu -- joins the partial results of attention keys that were cut over
// several blocks (sm_103a).
//
//   m = max m_i,  w_i = 2^(m_i - m),  out = sum w_i O_i / sum w_i l_i,
//   lse = (m + log2 sum w_i l_i) / log2 e
// for every row, over the parts i of its key in chunk order; D / 32 channels a lane.
// Bound by the latency of a few dependent reads from L2, so a warp has as many on
// their way as it can: of keys with few parts it takes four rows at a time, the (m, l)
// of eight parts of each in its lanes; of a key with many (one long sequence: 57
// parts) four warps share one row, each taking every fourth part, the (m, l) of 32
// of them in the lanes.  Blocks without a cut key leave at once.
#include "kv_attention.cuh"

namespace nvr {

namespace {

constexpr int kJoinWarps = 4;
constexpr int kJoinRows = 4;               // rows a warp takes at a time

// The place of a row: its query's row and its head.
__device__ __forceinline__ int64_t out_row(const KeyJoin& k, int n, int Hq, int G) {
  const int dq = div_small(k.rem0 + n, 1.0f / static_cast<float>(G));
  return static_cast<int64_t>(k.q0 + dq) * Hq + k.head * G + (k.rem0 + n - dq * G);
}

template <int CH>
__device__ __forceinline__ void load_channels(const float* src, float (&y)[CH]) {
  if (CH == 4) {
    const float4 v = *reinterpret_cast<const float4*>(src);
    y[0] = v.x; y[1] = v.y; y[CH - 2] = v.z; y[CH - 1] = v.w;
  } else {
    const float2 v = *reinterpret_cast<const float2*>(src);
    y[0] = v.x; y[1] = v.y;
  }
}

template <int CH>
__device__ __forceinline__ void store_channels(__nv_bfloat16* dst, const float (&acc)[CH], float inv) {
#pragma unroll
  for (int x = 0; x < CH; x += 2)
    *reinterpret_cast<__nv_bfloat162*>(dst + x) = __floats2bfloat162_rn(acc[x] * inv, acc[x + 1] * inv);
}

// Part i of a key is in the first slot of its block, but the key's first one if the
// key starts inside the chunk.
__device__ __forceinline__ const float* part_of(const float* partials, const KeyJoin& k, int i, size_t slot) {
  return partials + (2 * (blockIdx.x + static_cast<size_t>(i)) + (i == 0 ? k.tail : 0)) * slot;
}

template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps)
kv_join_few_kernel(const KeyJoin* __restrict__ joins, const float* __restrict__ partials, int NC, int Hq, int G,
                   __nv_bfloat16* __restrict__ out, float* __restrict__ lse) {
  constexpr int CH = D / 32, R = kJoinRows, P = 32 / R;      // rows of a warp, parts at a time
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const KeyJoin k = joins[blockIdx.x];
  if (k.n_parts < 2) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t slot = static_cast<size_t>(NC) * (D + 2);
  const int n0 = (blockIdx.y * (blockDim.x / 32) + warp) * R;
  if (n0 >= k.n_cols) return;
  const int mine = n0 + lane / P;                            // this lane's row among the (m, l)
  float top = -INFINITY, sum = 0.0f, acc[R][CH];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int x = 0; x < CH; ++x) acc[r][x] = 0.0f;
  // (rows past the last: the last row again, not stored)
  auto load = [&](int i, float (&y)[R][CH]) {
#pragma unroll
    for (int r = 0; r < R; ++r)
      load_channels<CH>(part_of(partials, k, i, slot) + 2 * NC + min(n0 + r, k.n_cols - 1) * D + lane * CH, y[r]);
  };
  constexpr int N = 4;                                       // parts whose channels are on their way
  float y[N][R][CH];
#pragma unroll
  for (int i = 0; i < N; ++i) load(min(i, k.n_parts - 1), y[i]);
  for (int b = 0; b < k.n_parts; b += P) {
    const int m = min(P, k.n_parts - b);
    float w = -INFINITY, l = 0.0f;
    if (lane % P < m && mine < k.n_cols) {
      const float* src = part_of(partials, k, b + lane % P, slot) + mine;
      w = src[0];
      l = src[NC];
    }
    float high = fmaxf(top, w);
#pragma unroll
    for (int d = P / 2; d > 0; d >>= 1) high = fmaxf(high, __shfl_xor_sync(0xFFFFFFFFu, high, d));
    const float base = high == -INFINITY ? 0.0f : high, shrink = ex2(top - base);
    top = high;
    w = ex2(w - base);
    sum = sum * shrink + w * l;
    if (b > 0) {
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float f = __shfl_sync(0xFFFFFFFFu, shrink, r * P);
#pragma unroll
        for (int x = 0; x < CH; ++x) acc[r][x] *= f;
      }
    }
    for (int i0 = 0; i0 < m; i0 += N) {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        // (past the end of the batch: a weight of zero)
        const float wi = i0 + i < m ? w : 0.0f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float f = __shfl_sync(0xFFFFFFFFu, wi, r * P + ((i0 + i) % P));
#pragma unroll
          for (int x = 0; x < CH; ++x) acc[r][x] += f * y[i][r][x];
        }
      }
      if (b + i0 + N < k.n_parts) {
#pragma unroll
        for (int i = 0; i < N; ++i) load(min(b + i0 + N + i, k.n_parts - 1), y[i]);
      }
    }
  }
#pragma unroll
  for (int d = P / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const float s = __shfl_sync(0xFFFFFFFFu, sum, r * P);
    if (n0 + r < k.n_cols)
      store_channels<CH>(out + out_row(k, n0 + r, Hq, G) * D + lane * CH, acc[r], out_factor(k.v_gsa, s));
  }
  if (lse && lane % P == 0 && mine < k.n_cols) lse[out_row(k, mine, Hq, G)] = lse_of(top, sum);
}

template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps)
kv_join_many_kernel(const KeyJoin* __restrict__ joins, const float* __restrict__ partials, int NC, int Hq, int G,
                    __nv_bfloat16* __restrict__ out, float* __restrict__ lse) {
  constexpr int CH = D / 32, W = kJoinWarps;
  __shared__ float s_top[W], s_sum[W], s_acc[W][32][CH];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const KeyJoin k = joins[blockIdx.x];
  if (k.n_parts < 2) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const size_t slot = static_cast<size_t>(NC) * (D + 2);
  const int parts = (k.n_parts - warp + W - 1) / W;          // this warp's: warp, warp + W, ...
  for (int n = blockIdx.y; n < k.n_cols; n += gridDim.y) {
    float top = -INFINITY, sum = 0.0f, acc[CH];
#pragma unroll
    for (int x = 0; x < CH; ++x) acc[x] = 0.0f;
    for (int b = 0; b < parts; b += 32) {
      const int m = min(32, parts - b);
      float w = -INFINITY, l = 0.0f;
      if (lane < m) {
        const float* src = part_of(partials, k, (b + lane) * W + warp, slot) + n;
        w = src[0];
        l = src[NC];
      }
      float high = fmaxf(top, w);
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) high = fmaxf(high, __shfl_xor_sync(0xFFFFFFFFu, high, d));
      const float base = high == -INFINITY ? 0.0f : high, shrink = ex2(top - base);
      top = high;
      w = ex2(w - base);
      sum = sum * shrink + w * l;
#pragma unroll
      for (int x = 0; x < CH; ++x) acc[x] *= shrink;
      for (int i0 = 0; i0 < m; i0 += 8) {
        float y[8][CH];
#pragma unroll
        for (int i = 0; i < 8; ++i)
          // (past the end: the last part, under a weight of zero)
          load_channels<CH>(part_of(partials, k, (b + min(i0 + i, m - 1)) * W + warp, slot) + 2 * NC + n * D + lane * CH, y[i]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float wi = __shfl_sync(0xFFFFFFFFu, w, i0 + i);
#pragma unroll
          for (int x = 0; x < CH; ++x) acc[x] += wi * y[i][x];
        }
      }
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    // the warps of the row, in order
    __syncthreads();                                         // (the last row's are read)
    if (lane == 0) {
      s_top[warp] = top;
      s_sum[warp] = sum;
    }
#pragma unroll
    for (int x = 0; x < CH; ++x) s_acc[warp][lane][x] = acc[x];
    __syncthreads();
    if (warp) continue;
#pragma unroll
    for (int i = 1; i < W; ++i) top = fmaxf(top, s_top[i]);
    const float base = top == -INFINITY ? 0.0f : top;
    sum = 0.0f;
#pragma unroll
    for (int x = 0; x < CH; ++x) acc[x] = 0.0f;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float w = ex2(s_top[i] - base);
      sum += w * s_sum[i];
#pragma unroll
      for (int x = 0; x < CH; ++x) acc[x] += w * s_acc[i][lane][x];
    }
    const int64_t row = out_row(k, n, Hq, G);
    store_channels<CH>(out + row * D + lane * CH, acc, out_factor(k.v_gsa, sum));
    if (lse && lane == 0) lse[row] = lse_of(top, sum);
  }
}

}  // namespace

nvr_status launch_kv_join(const AttnParams& p, int D, int blocks, int NC, int64_t keys, cudaStream_t s) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  // A key has about blocks / keys parts and at most `cols` rows.  From eight parts on (32,
  // where a key has many rows to share out) a row gets a block: one sequence of 131072
  // tokens, 57 parts: 49.6 -> 41.1 us for the call.  At most 64 rows of a key at once: of
  // the blocks most have no key, and 152 x 256 of them took 35 us (two sequences of 695
  // tokens, 16 queries of 24 and 6 heads: 45.6 -> 13.2 us).
  const int64_t all = static_cast<int64_t>(p.max_q) * p.G;
  const int cols = static_cast<int>(all < NC ? all : NC);
  const bool many = keys * (cols > 32 ? 32 : 8) <= blocks;
  const int warps = many || cols > kJoinRows * (kJoinWarps - 1) ? kJoinWarps : (cols + kJoinRows - 1) / kJoinRows;
  const int rows = warps * kJoinRows;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks),
                     static_cast<unsigned>(many ? (cols < 64 ? cols : 64) : (cols + rows - 1) / rows));
  cfg.blockDim = dim3(32 * warps);
  cfg.stream = s;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  auto go = [&](auto kernel) {
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, static_cast<const KeyJoin*>(p.joins),
                                          static_cast<const float*>(p.partials), NC, p.Hq, p.G, p.out, p.lse));
  };
  if (many) return D == 128 ? go(kv_join_many_kernel<128>) : go(kv_join_many_kernel<64>);
  return D == 128 ? go(kv_join_few_kernel<128>) : go(kv_join_few_kernel<64>);
}

}  // namespace nvr
