// prompt_join.cu -- joins the partial results of prompt_attention's keys that were
// cut over several blocks (sm_103a).
//
//   m = max m_i,  w_i = 2^(m_i - m),  out = sum w_i O_i / sum w_i l_i,
//   lse = (m + log2 sum w_i l_i) / log2 e
// for every row, over the parts i of its key in chunk order, then with the prefix.
// Bound by the latency of dependent reads from L2.  A block takes four rows of a key
// at a time, each of its warps every fourth part of them, D / 32 channels a lane; the
// warps' sums are added in order.
#include "prompt_attention.cuh"

namespace nvr {

namespace {

constexpr int kWarps = 4;
constexpr int kRows = 4;

template <int D, bool kF16>
__global__ void __launch_bounds__(32 * kWarps)
prompt_join_kernel(const PromptJoin* __restrict__ joins, int blocks, const float* __restrict__ partials, int Hq,
                   int Gt, int qt, const uint16_t* prefix_out, const float* prefix_lse, uint16_t* out, float* lse) {
  constexpr int CH = D / 32;
  __shared__ int s_end[kPaMaxCtas];          // rows' quadruples of the keys up to this one
  __shared__ float s_ml[2][kWarps][kRows], s_acc[kWarps][kRows][D];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (warp == 0) {
    int total = 0;
    for (int i0 = 0; i0 < blocks; i0 += 32) {
      const int i = i0 + lane;
      int n = 0;
      if (i < blocks && joins[i].n_parts > 1) {
        // (row tile 0 ends at row Gt * qt, row tile 1 starts at row 128)
        const int nq = joins[i].n_q;
        const int rows = nq <= qt ? nq * Gt : kPaTile + (nq - qt) * Gt;
        n = (rows + kRows - 1) / kRows;
      }
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int a = __shfl_up_sync(0xFFFFFFFFu, n, d);
        if (lane >= d) n += a;
      }
      if (i < blocks) s_end[i] = total + n;
      total += __shfl_sync(0xFFFFFFFFu, n, 31);
    }
  }
  __syncthreads();
  const int total = s_end[blocks - 1];
  constexpr size_t kSlot = static_cast<size_t>(kPaRows) * (D + 2);
  int key = 0;
  for (int u = blockIdx.x; u < total; u += gridDim.x) {
    while (s_end[key] <= u) ++key;
    const PromptJoin k = joins[key];
    const int n0 = (u - (key ? s_end[key - 1] : 0)) * kRows;
    auto part_of = [&](int i) { return partials + (2 * (static_cast<size_t>(key) + i) + (i == 0 ? k.tail : 0)) * kSlot; };
    float m[kRows], l[kRows], acc[kRows][CH];
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      m[r] = -INFINITY;
      l[r] = 0.0f;
#pragma unroll
      for (int x = 0; x < CH; ++x) acc[r][x] = 0.0f;
    }
    for (int i = warp; i < k.n_parts; i += kWarps) {
      const float* part = part_of(i);
      float pm[kRows], pl[kRows], y[kRows][CH];
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        pm[r] = part[n0 + r];
        pl[r] = part[kPaRows + n0 + r];
        const float* src = part + 2 * kPaRows + (n0 + r) * D + lane * CH;
        if (CH == 4) {
          const float4 v = *reinterpret_cast<const float4*>(src);
          y[r][0] = v.x; y[r][1] = v.y; y[r][CH - 2] = v.z; y[r][CH - 1] = v.w;
        } else {
          const float2 v = *reinterpret_cast<const float2*>(src);
          y[r][0] = v.x; y[r][1] = v.y;
        }
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        // (a part that the row sees nothing of has a sum of 0, its row of O may be anything)
        const bool none = pl[r] == 0.0f;
        const float top = none ? m[r] : fmaxf(m[r], pm[r]), base = top == -INFINITY ? 0.0f : top;
        const float keep = ex2(m[r] - base), w = none ? 0.0f : ex2(pm[r] - base);
        m[r] = top;
        l[r] = l[r] * keep + w * pl[r];
#pragma unroll
        for (int x = 0; x < CH; ++x) acc[r][x] = acc[r][x] * keep + (none ? 0.0f : w * y[r][x]);
      }
    }
    __syncthreads();                                        // (the last rows' sums have been read)
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
      if (lane == 0) {
        s_ml[0][warp][r] = m[r];
        s_ml[1][warp][r] = l[r];
      }
#pragma unroll
      for (int x = 0; x < CH; ++x) s_acc[warp][r][lane * CH + x] = acc[r][x];
    }
    __syncthreads();
    // row `warp` of the four
    const int n = n0 + warp, w_tile = n / kPaTile, x = n - w_tile * kPaTile, iq = x / Gt, dq = w_tile * qt + iq;
    if (iq >= qt || dq >= k.n_q) continue;
    float top = -INFINITY, sum = 0.0f, o[CH];
#pragma unroll
    for (int i = 0; i < kWarps; ++i) top = fmaxf(top, s_ml[0][i][warp]);
    const float base = top == -INFINITY ? 0.0f : top;
#pragma unroll
    for (int c = 0; c < CH; ++c) o[c] = 0.0f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      const float w = ex2(s_ml[0][i][warp] - base);
      sum += w * s_ml[1][i][warp];
#pragma unroll
      for (int c = 0; c < CH; ++c) o[c] += w * s_acc[i][warp][lane * CH + c];
    }
    const int64_t row = static_cast<int64_t>(k.q0 + dq) * Hq + k.head + (x - iq * Gt);
    float z = lse_of(top, sum), f = out_factor(1.0f, sum), f_before = 0.0f;
    if (prefix_lse) {
      const float before = prefix_lse[row];
      float f_own;
      z = join_prefix(z, before, f_own, f_before);
      f *= f_own;
    }
    uint32_t* dst = reinterpret_cast<uint32_t*>(out + row * D + lane * CH);
    const uint32_t* prev = reinterpret_cast<const uint32_t*>(prefix_out + row * D + lane * CH);
#pragma unroll
    for (int c = 0; c < CH; c += 2) {
      float a = o[c] * f, b = o[c + 1] * f;
      if (f_before != 0.0f) {
        const float2 v = unpack_16<kF16>(prev[c / 2]);
        a = fmaf(v.x, f_before, a);
        b = fmaf(v.y, f_before, b);
      }
      dst[c / 2] = pack_16<kF16>(a, b);
    }
    __syncwarp();
    if (lse && lane == 0) lse[row] = z;
  }
}

}  // namespace

nvr_status launch_prompt_join(const PromptParams& p, int D, bool f16, int blocks, int sms, cudaStream_t s) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(sms * 8));
  cfg.blockDim = dim3(32 * kWarps);
  cfg.stream = s;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  auto go = [&](auto kernel) {
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, static_cast<const PromptJoin*>(p.joins), blocks,
                                          static_cast<const float*>(p.partials), p.Hq, p.Gt, p.qt, p.prefix_out,
                                          p.prefix_lse, p.out, p.lse));
  };
  if (D == 128) return f16 ? go(prompt_join_kernel<128, true>) : go(prompt_join_kernel<128, false>);
  return f16 ? go(prompt_join_kernel<64, true>) : go(prompt_join_kernel<64, false>);
}

}  // namespace nvr
