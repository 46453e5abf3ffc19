// kv_join.cu -- joins the partial results of attention keys that were cut over
// several blocks (sm_103a).
//
//   m = max m_i,  w_i = 2^(m_i - m),  out = sum w_i O_i / sum w_i l_i,
//   lse = (m + log2 sum w_i l_i) / log2 e
// for every row, over the parts i of its key in chunk order.  A row has one warp,
// or four that take every fourth part where keys have many (one long sequence: 57
// parts); D / 32 channels a lane, the (m, l) of 32 parts in the lanes, eight parts'
// vectors under way.  Bound by the latency of three or four dependent reads from
// L2; blocks without a cut key leave at once.
#include "kv_attention.cuh"

namespace nvr {

namespace {

constexpr int kJoinWarps = 4;

template <int D, int WPR>                        // warps of a row
__global__ void __launch_bounds__(32 * kJoinWarps)
kv_join_kernel(const KeyJoin* __restrict__ joins, const float* __restrict__ partials, int NC, int Hq, int G,
               __nv_bfloat16* __restrict__ out, float* __restrict__ lse) {
  constexpr int CH = D / 32;
  __shared__ float s_top[kJoinWarps], s_sum[kJoinWarps], s_acc[WPR > 1 ? kJoinWarps : 1][32][CH];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const KeyJoin k = joins[blockIdx.x];
  if (k.n_parts < 2) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, mine = warp % WPR;
  const float inv_G = 1.0f / static_cast<float>(G);
  const size_t slot = static_cast<size_t>(NC) * (D + 2);
  // part i is in the first slot of its block, but the key's first one if the key
  // starts inside the chunk
  auto part_at = [&](int i) { return partials + (2 * (blockIdx.x + i) + (i == 0 ? k.tail : 0)) * slot; };
  const int parts = (k.n_parts - mine + WPR - 1) / WPR;      // this warp's: mine, mine + WPR, ...
  constexpr int RB = kJoinWarps / WPR;                       // rows of the block at a time
  for (int n = blockIdx.y * RB + warp / WPR; n < k.n_cols; n += gridDim.y * RB) {
    float top = -INFINITY, sum = 0.0f, acc[CH];
#pragma unroll
    for (int x = 0; x < CH; ++x) acc[x] = 0.0f;
    for (int b = 0; b < parts; b += 32) {
      const int m = min(32, parts - b);
      float w = -INFINITY, l = 0.0f;
      if (lane < m) {
        const float* src = part_at((b + lane) * WPR + mine) + n;
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
        for (int i = 0; i < 8; ++i) {
          // (past the end: the last part, under a weight of zero)
          const float* src = part_at((b + min(i0 + i, m - 1)) * WPR + mine) + 2 * NC + n * D + lane * CH;
          if (CH == 4) {
            const float4 v = *reinterpret_cast<const float4*>(src);
            y[i][0] = v.x; y[i][1] = v.y; y[i][CH - 2] = v.z; y[i][CH - 1] = v.w;
          } else {
            const float2 v = *reinterpret_cast<const float2*>(src);
            y[i][0] = v.x; y[i][1] = v.y;
          }
        }
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
    if (WPR > 1) {
      // the warps of the row, in order
      __syncthreads();                                       // (the last row's are read)
      if (lane == 0) {
        s_top[warp] = top;
        s_sum[warp] = sum;
      }
#pragma unroll
      for (int x = 0; x < CH; ++x) s_acc[WPR > 1 ? warp : 0][lane][x] = acc[x];
      __syncthreads();
      if (mine) continue;
#pragma unroll
      for (int i = 1; i < WPR; ++i) top = fmaxf(top, s_top[warp + i]);
      const float base = top == -INFINITY ? 0.0f : top;
      sum = 0.0f;
#pragma unroll
      for (int x = 0; x < CH; ++x) acc[x] = 0.0f;
#pragma unroll
      for (int i = 0; i < WPR; ++i) {
        const float w = ex2(s_top[warp + i] - base);
        sum += w * s_sum[warp + i];
#pragma unroll
        for (int x = 0; x < CH; ++x) acc[x] += w * s_acc[WPR > 1 ? warp + i : 0][lane][x];
      }
    }
    const int dq = div_small(k.rem0 + n, inv_G);
    const int64_t row = static_cast<int64_t>(k.q0 + dq) * Hq + k.head * G + (k.rem0 + n - dq * G);
    const float inv = sum > 0.0f ? __fdividef(k.v_gsa, sum) : 0.0f;
    __nv_bfloat16* dst = out + row * D + lane * CH;
#pragma unroll
    for (int x = 0; x < CH; x += 2)
      *reinterpret_cast<__nv_bfloat162*>(dst + x) = __floats2bfloat162_rn(acc[x] * inv, acc[x + 1] * inv);
    if (lse && lane == 0) lse[row] = sum > 0.0f ? (top + log2f(sum)) * 0.693147180559945309f : -INFINITY;
  }
}

}  // namespace

nvr_status launch_kv_join(const AttnParams& p, int D, int blocks, int NC, int64_t keys, cudaStream_t s) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  // A key has about blocks / keys parts.  From eight on a row gets a block (one
  // sequence of 131072 tokens, 57 parts: 49.6 -> 41.1 us for the call); below it a
  // warp, two rows (of 256 columns four) to a warp, so that there are few blocks
  // with nothing to do.
  const bool many = keys * 8 <= blocks;
  const int rows = many ? 1 : (NC > 32 ? 4 : 2) * kJoinWarps;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), static_cast<unsigned>((NC + rows - 1) / rows));
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = s;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  auto go = [&](auto kernel) {
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, static_cast<const KeyJoin*>(p.joins),
                                          static_cast<const float*>(p.partials), NC, p.Hq, p.G, p.out, p.lse));
  };
  if (many) return D == 128 ? go(kv_join_kernel<128, 4>) : go(kv_join_kernel<64, 4>);
  return D == 128 ? go(kv_join_kernel<128, 1>) : go(kv_join_kernel<64, 1>);
}

}  // namespace nvr
