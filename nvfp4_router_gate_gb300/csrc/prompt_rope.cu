// prompt_rope.cu -- RMS norm of query and key heads and rotary positions with
// several axes (sm_103a): prompt_rope.
//
//   x <- x w / sqrt(sum x^2 / D + eps),  (a, b) -> (a c - b s, b c + a s),
// with c and s of pair i from row positions[axes[i]] of the tables.
//
// Bound by memory: every byte of the heads is read and written once, the tables'
// rows are read once a token.  A warp takes a run of the head groups of one token,
// so that a lane's eight pairs of angles stay in its registers; the loads of the
// next two groups are under way meanwhile.
#include <cuda_fp16.h>

#include "nvr_internal.h"
#include "../../include/nvfp4_prompt.h"

namespace nvr {

namespace {

constexpr int kRopeThreads = 128;

struct RopeParams {
  const void *q, *k;
  void *q_out, *k_out;
  int64_t q_stride, k_stride, qo_stride, ko_stride;
  int64_t T;
  int Hq, Hkv, D;
  const int32_t* positions;
  int64_t axis_stride;
  const float *cos, *sin;
  int64_t n_pos;
  int rot;
  const float *q_weight, *k_weight;
  float eps;
  int steps_q, steps;     // groups of heads of the queries, of both
  int parts;              // warps of a token
  int shift;              // lanes of a head: 1 << shift
  uint32_t used;          // bit a: some pair goes by axis a
  uint8_t axes[PROMPT_ROPE_MAX_PAIRS];
};

// Eight channels as they lie in memory, and as fp32.
template <typename E>
struct Eight {
  uint4 u;
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    u = __ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at));
  }
  __device__ __forceinline__ void widen(float (&x)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (sizeof(E) == sizeof(__half) && std::is_same<E, __half>::value) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        x[2 * i] = f.x; x[2 * i + 1] = f.y;
      } else {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    }
  }
};
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    const float4* src = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    a = __ldg(src);
    b = __ldg(src + 1);
  }
  __device__ __forceinline__ void widen(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
};

template <typename E>
__device__ __forceinline__ void store8(void* base, int64_t at, const float (&x)[8]) {
  if constexpr (std::is_same<E, float>::value) {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
    dst[0] = make_float4(x[0], x[1], x[2], x[3]);
    dst[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same<E, __half>::value) {
        const __half2 h = __floats2half2_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// The row of the tables of a pair, and whether every position of the token lies in them.
__device__ __forceinline__ bool positions_ok(const RopeParams& p, int64_t t) {
  bool ok = true;
  for (uint32_t left = p.used; left; left &= left - 1) {
    const int64_t pos = __ldg(p.positions + (__ffs(left) - 1) * p.axis_stride + t);
    ok = ok && pos >= 0 && pos < p.n_pos;
  }
  return ok;
}
__device__ __forceinline__ int64_t table_at(const RopeParams& p, int64_t t, int pair) {
  return static_cast<int64_t>(__ldg(p.positions + p.axes[pair] * p.axis_stride + t)) * (p.rot / 2) + pair;
}

// Heads of 64, 128 or 256 channels: 1 << shift lanes a head, two vectors of eight
// channels each.  By halves a lane's vectors hold the two sides of eight pairs (and
// the channels behind the rotated ones are shared out in the same way); with
// neighbouring pairs each vector holds four.
template <typename In, typename Out, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, 6)
prompt_rope_kernel(const __grid_constant__ RopeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int lane = threadIdx.x & 31, L = 1 << p.shift, l = lane & (L - 1), sub_head = lane >> p.shift;
  const int per_step = 32 >> p.shift;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = unit / p.parts;
  if (t >= p.T) return;
  const int part = static_cast<int>(unit - t * p.parts);
  const int s0 = p.steps * part / p.parts, s1 = p.steps * (part + 1) / p.parts;

  int o0, o1;                                  // the channels of this lane's vectors
  bool on0, on1;                               // they turn
  if (kInterleaved) {
    o0 = 8 * l; o1 = 8 * (L + l);
    on0 = o0 < p.rot; on1 = o1 < p.rot;
  } else {
    const int turning = p.rot / 16;
    on0 = on1 = l < turning;
    o0 = on0 ? 8 * l : p.rot + 16 * (l - turning);
    o1 = on0 ? p.rot / 2 + 8 * l : o0 + 8;
  }
  // The vectors of step s; heads past the last one read the first.
  const int64_t row_q = t * p.q_stride, row_k = t * p.k_stride;
  Eight<In> next[2][2];
  auto load = [&](int s, Eight<In> (&v)[2]) {
    const bool key = s >= p.steps_q;
    const int h = (key ? s - p.steps_q : s) * per_step + sub_head, n = key ? p.Hkv : p.Hq;
    const int64_t at = (key ? row_k : row_q) + static_cast<int64_t>(h < n ? h : 0) * p.D;
    v[0].load(key ? p.k : p.q, at + o0);
    v[1].load(key ? p.k : p.q, at + o1);
  };
  load(s0, next[0]);
  if (s0 + 1 < s1) load(s0 + 1, next[1]);

  const bool ok = p.rot == 0 || positions_ok(p, t);
  float c[8], s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    c[i] = 1.0f;
    s[i] = 0.0f;
    const bool on = i < 4 ? on0 : on1;
    const int pair = !kInterleaved ? o0 + i : (i < 4 ? o0 / 2 + i : o1 / 2 + i - 4);
    if (ok && on) {
      const int64_t at = table_at(p, t, pair);
      c[i] = __ldg(p.cos + at);
      s[i] = __ldg(p.sin + at);
    }
  }
  float w[2][8];
  bool norm = false;
  auto weights = [&](const float* src) {
    norm = src != nullptr;
    if (!norm) return;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[0][i] = __ldg(src + o0 + i);
      w[1][i] = __ldg(src + o1 + i);
    }
  };
  weights(s0 < p.steps_q ? p.q_weight : p.k_weight);
  const float inv_D = 1.0f / static_cast<float>(p.D);

  auto step = [&](int st, Eight<In> (&v)[2]) {
    const bool key = st >= p.steps_q;
    if (st == p.steps_q && st > s0) weights(p.k_weight);
    float a[8], b[8];
    v[0].widen(a);
    v[1].widen(b);
    if (st + 2 < s1) load(st + 2, v);
    if (norm) {
      float ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(a[i], a[i], fmaf(b[i], b[i], ss));
      for (int d = L / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
      const float r = 1.0f / sqrtf(fmaf(ss, inv_D, p.eps));
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        a[i] = a[i] * r * w[0][i];
        b[i] = b[i] * r * w[1][i];
      }
    }
    if (kInterleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a0 = a[2 * i], a1 = a[2 * i + 1], b0 = b[2 * i], b1 = b[2 * i + 1];
        if (on0) {
          a[2 * i] = a0 * c[i] - a1 * s[i];
          a[2 * i + 1] = a1 * c[i] + a0 * s[i];
        }
        if (on1) {
          b[2 * i] = b0 * c[i + 4] - b1 * s[i + 4];
          b[2 * i + 1] = b1 * c[i + 4] + b0 * s[i + 4];
        }
      }
    } else if (on0) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float a0 = a[i], b0 = b[i];
        a[i] = a0 * c[i] - b0 * s[i];
        b[i] = b0 * c[i] + a0 * s[i];
      }
    }
    if (!ok) {
#pragma unroll
      for (int i = 0; i < 8; ++i) a[i] = b[i] = 0.0f;
    }
    const int h = (key ? st - p.steps_q : st) * per_step + sub_head;
    if (h < (key ? p.Hkv : p.Hq)) {
      const int64_t at = t * (key ? p.ko_stride : p.qo_stride) + static_cast<int64_t>(h) * p.D;
      store8<Out>(key ? p.k_out : p.q_out, at + o0, a);
      store8<Out>(key ? p.k_out : p.q_out, at + o1, b);
    }
  };
  for (int st = s0; st < s1; st += 2) {
    step(st, next[0]);
    if (st + 1 < s1) step(st + 1, next[1]);
  }
}

template <typename E>
__device__ __forceinline__ float load1(const void* base, int64_t at) {
  return static_cast<float>(static_cast<const E*>(base)[at]);
}
template <typename E>
__device__ __forceinline__ void store1(void* base, int64_t at, float x) {
  if constexpr (std::is_same<E, __half>::value) static_cast<E*>(base)[at] = __float2half_rn(x);
  else if constexpr (std::is_same<E, float>::value) static_cast<E*>(base)[at] = x;
  else static_cast<E*>(base)[at] = __float2bfloat16_rn(x);
}

// Any other even head size, number of rotated channels or alignment: a warp a head, a channel
// a lane at a time (a channel's partner is read again, before anything is stored).
template <typename In, typename Out>
__global__ void __launch_bounds__(kRopeThreads)
prompt_rope_any_kernel(const __grid_constant__ RopeParams p, bool interleaved) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int lane = threadIdx.x & 31;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kRopeThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = unit / (p.Hq + p.Hkv);
  if (t >= p.T) return;
  const int head = static_cast<int>(unit - t * (p.Hq + p.Hkv));
  const bool key = head >= p.Hq;
  const int h = key ? head - p.Hq : head;
  const void* src = key ? p.k : p.q;
  const int64_t from = t * (key ? p.k_stride : p.q_stride) + static_cast<int64_t>(h) * p.D;
  const float* weight = key ? p.k_weight : p.q_weight;
  const bool ok = p.rot == 0 || positions_ok(p, t);
  constexpr int N = PROMPT_ROPE_MAX_D / 32;
  float x[N], z[N], r = 1.0f, ss = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = lane + 32 * i;
    x[i] = z[i] = 0.0f;
    if (e >= p.D) continue;
    x[i] = load1<In>(src, from + e);
    const int f = interleaved ? e ^ 1 : e < p.rot / 2 ? e + p.rot / 2 : e - p.rot / 2;
    if (e < p.rot) z[i] = load1<In>(src, from + f) * (weight ? __ldg(weight + f) : 1.0f);
    ss = fmaf(x[i], x[i], ss);
    if (weight) x[i] *= __ldg(weight + e);
  }
  if (weight) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
    r = 1.0f / sqrtf(fmaf(ss, 1.0f / static_cast<float>(p.D), p.eps));
  }
  __syncwarp();
  void* dst = key ? p.k_out : p.q_out;
  const int64_t to = t * (key ? p.ko_stride : p.qo_stride) + static_cast<int64_t>(h) * p.D;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int e = lane + 32 * i;
    if (e >= p.D) continue;
    float y = x[i] * r;
    if (ok && e < p.rot) {
      const bool second = interleaved ? e & 1 : e >= p.rot / 2;
      const int64_t at = table_at(p, t, interleaved ? e / 2 : second ? e - p.rot / 2 : e);
      const float c = __ldg(p.cos + at), s = __ldg(p.sin + at), b = z[i] * r;
      y = second ? y * c + b * s : y * c - b * s;
    }
    store1<Out>(dst, to + e, ok ? y : 0.0f);
  }
}

bool off4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

}  // namespace

}  // namespace nvr

using namespace nvr;

extern "C" nvr_status prompt_rope(const void* q, int64_t q_stride, const void* k, int64_t k_stride, nvr_dtype dt,
                                  int64_t T, int Hq, int Hkv, int D, const int32_t* positions, int64_t axis_stride,
                                  int n_axes, const uint8_t* axes, const float* cos, const float* sin, int64_t n_pos,
                                  int rot, int interleaved, const float* q_weight, const float* k_weight, float eps,
                                  void* q_out, int64_t q_out_stride, void* k_out, int64_t k_out_stride,
                                  nvr_dtype out_dt, nvr_stream_t stream) {
  if (T < 0 || Hq < 0 || Hq > 65536 || Hkv < 0 || Hkv > 65536 || Hq + Hkv < 1) return NVR_ERR_INVALID_ARG;
  if ((dt != NVR_BF16 && dt != NVR_F32 && dt != NVR_F16) || (out_dt != dt && (dt != NVR_F32 || (out_dt != NVR_BF16 && out_dt != NVR_F16))))
    return NVR_ERR_INVALID_ARG;
  if (D < 2 || D % 2) return NVR_ERR_INVALID_ARG;
  if (D > PROMPT_ROPE_MAX_D) return NVR_ERR_UNSUPPORTED;
  if (rot < 0 || rot > D || rot % 2 || !(eps >= 0.0f)) return NVR_ERR_INVALID_ARG;
  if (rot > 0 && (n_pos < 1 || n_axes < 1 || n_axes > PROMPT_ROPE_MAX_AXES || !axes)) return NVR_ERR_INVALID_ARG;
  if (T > 0 && ((Hq > 0 && (!q || !q_out)) || (Hkv > 0 && (!k || !k_out)))) return NVR_ERR_INVALID_ARG;
  if (T > 0 && rot > 0 && (!positions || !cos || !sin || (n_axes > 1 && axis_stride < 0))) return NVR_ERR_INVALID_ARG;
  RopeParams p;
  p.used = 0;
  for (int i = 0; i < rot / 2; ++i) {
    if (axes[i] >= n_axes) return NVR_ERR_INVALID_ARG;
    p.axes[i] = axes[i];
    p.used |= 1u << axes[i];
  }
  const int64_t row_q = static_cast<int64_t>(Hq) * D, row_k = static_cast<int64_t>(Hkv) * D;
  if ((Hq > 0 && (q_stride < row_q || q_out_stride < row_q)) || (Hkv > 0 && (k_stride < row_k || k_out_stride < row_k)))
    return NVR_ERR_INVALID_ARG;
  const uintptr_t in_bits = reinterpret_cast<uintptr_t>(q) | reinterpret_cast<uintptr_t>(k);
  const uintptr_t out_bits = reinterpret_cast<uintptr_t>(q_out) | reinterpret_cast<uintptr_t>(k_out);
  if (in_bits % (dt == NVR_F32 ? 4 : 2) || out_bits % (out_dt == NVR_F32 ? 4 : 2) || off4(positions) || off4(cos) ||
      off4(sin) || off4(q_weight) || off4(k_weight))
    return NVR_ERR_ALIGNMENT;
  if (T == 0) return NVR_OK;
  const int sms = device_sm_count();
  if (sms <= 0) return NVR_ERR_CUDA;
  p.q = q; p.k = k; p.q_out = q_out; p.k_out = k_out;
  p.q_stride = q_stride; p.k_stride = k_stride; p.qo_stride = q_out_stride; p.ko_stride = k_out_stride;
  p.T = T; p.Hq = Hq; p.Hkv = Hkv; p.D = D;
  p.positions = positions; p.axis_stride = axis_stride; p.cos = cos; p.sin = sin; p.n_pos = n_pos; p.rot = rot;
  p.q_weight = q_weight; p.k_weight = k_weight; p.eps = eps;
  // Whole vectors on both sides of the pairs and of the channels behind them, 16 bytes apart
  const int vec = dt == NVR_F32 ? 4 : 8, out_vec = out_dt == NVR_F32 ? 4 : 8;
  const bool aligned = (in_bits | out_bits) % 16 == 0 && (Hq == 0 || (q_stride % vec == 0 && q_out_stride % out_vec == 0)) &&
                       (Hkv == 0 || (k_stride % vec == 0 && k_out_stride % out_vec == 0));
  const bool vectors = aligned && (D == 64 || D == 128 || D == 256) && rot % (interleaved ? 8 : 16) == 0;
  int64_t units;
  if (vectors) {
    p.shift = D == 64 ? 2 : D == 128 ? 3 : 4;
    const int heads = 32 >> p.shift;
    p.steps_q = (Hq + heads - 1) / heads;
    p.steps = p.steps_q + (Hkv + heads - 1) / heads;
    const int64_t each = (T * p.steps + sms * 24 - 1) / (sms * 24);
    p.parts = each >= p.steps ? 1 : static_cast<int>((p.steps + each - 1) / each);
    units = T * p.parts;
  } else {
    p.shift = 0;
    p.steps_q = p.steps = p.parts = 0;
    units = T * (Hq + Hkv);
  }
  const int64_t blocks = (units + kRopeThreads / 32 - 1) / (kRopeThreads / 32);
  if (blocks > INT32_MAX) return NVR_ERR_UNSUPPORTED;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kRopeThreads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  auto go = [&](auto in, auto out) {
    using In = decltype(in);
    using Out = decltype(out);
    if (!vectors) return cuda_status(cudaLaunchKernelEx(&cfg, prompt_rope_any_kernel<In, Out>, p, interleaved != 0));
    return interleaved ? cuda_status(cudaLaunchKernelEx(&cfg, prompt_rope_kernel<In, Out, true>, p))
                       : cuda_status(cudaLaunchKernelEx(&cfg, prompt_rope_kernel<In, Out, false>, p));
  };
  if (dt == NVR_BF16) return go(__nv_bfloat16(), __nv_bfloat16());
  if (dt == NVR_F16) return go(__half(), __half());
  if (out_dt == NVR_BF16) return go(float(), __nv_bfloat16());
  if (out_dt == NVR_F16) return go(float(), __half());
  return go(float(), float());
}
