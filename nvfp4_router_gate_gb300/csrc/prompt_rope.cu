// prompt_rope.cu -- RMS norm of query and key heads and rotary positions with
// several axes (sm_103a): prompt_rope.
//
//   x <- x w / sqrt(sum x^2 / D + eps),  (a, b) -> (a c - b s, b c + a s),
// with c and s of pair i from row positions[axes[i]] of the tables.
//
// Bound by memory: every byte of the heads is read and written once, the tables' rows are
// read once a token.  Measured (inputs not in L2): 8192 tokens of 72 heads of 128 channels
// with norm, 306 MB, 51 us (6.0 TB/s); one such token 2.6 us, the launch and three loads
// one after the other (position, angle, store).
//
// A warp takes a stretch of all tokens' head groups, equally many for each: with a token a
// warp the last of 2.25 waves was mostly empty (73 us).  A lane's eight pairs of angles stay
// in its registers over a token.  The next two groups' loads are under way through a ring
// in shared memory, a thread's own slots: kept in registers they cost spills, and the moves
// from one group to the next waited for them (59 us).  Then the instructions bind as much
// as the memory: pairs of channels go through the packed fp32 instructions, and addresses
// are worked out where a token or its keys begin.
#include <cuda_fp16.h>

#include "nvr_internal.h"
#include "../../include/nvfp4_prompt.h"

namespace nvr {

namespace {

constexpr int kRopeThreads = 128;
// Of a multiprocessor.  The prompt above: 4 blocks 52 us, 5 52, 6 53; a chunk of 2537 tokens
// of 54 heads 15.5, 15.2, 16.1.
constexpr int kRopeBlocks = 5;
constexpr int kRopeAhead = 2;            // steps whose loads are under way (1: 56 us, 3: 55)

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
  int64_t share, extra;   // steps of a warp, warps that have one more
  int shift;              // lanes of a head: 1 << shift
  uint32_t used;          // bit a: some pair goes by axis a
  alignas(4) uint8_t axes[PROMPT_ROPE_MAX_PAIRS];
};

// Eight channels as they lie in memory (16-bit types one vector of 16 bytes, fp32 two), to
// four pairs of fp32.
template <typename E>
__device__ __forceinline__ void widen(const uint4* u, uint64_t (&x)[4]) {
  const uint4 a = u[0];
  if constexpr (std::is_same<E, float>::value) {
    const uint4 b = u[kRopeThreads];
    x[0] = f2_pack(__uint_as_float(a.x), __uint_as_float(a.y)); x[1] = f2_pack(__uint_as_float(a.z), __uint_as_float(a.w));
    x[2] = f2_pack(__uint_as_float(b.x), __uint_as_float(b.y)); x[3] = f2_pack(__uint_as_float(b.z), __uint_as_float(b.w));
  } else {
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same<E, __half>::value) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        x[i] = f2_pack(f.x, f.y);
      } else {
        x[i] = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
      }
    }
  }
}

__device__ __forceinline__ void copy16(uint4* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(smem_u32(dst)), "l"(src) : "memory");
}

template <typename E>
__device__ __forceinline__ void store8(E* to, const uint64_t (&x)[4]) {
  if constexpr (std::is_same<E, float>::value) {
    float4* dst = reinterpret_cast<float4*>(to);
    dst[0] = make_float4(f2_lo(x[0]), f2_hi(x[0]), f2_lo(x[1]), f2_hi(x[1]));
    dst[1] = make_float4(f2_lo(x[2]), f2_hi(x[2]), f2_lo(x[3]), f2_hi(x[3]));
  } else {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same<E, __half>::value) {
        const __half2 h = __floats2half2_rn(f2_lo(x[i]), f2_hi(x[i]));
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(f2_lo(x[i]), f2_hi(x[i]));
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    *reinterpret_cast<uint4*>(to) = make_uint4(w[0], w[1], w[2], w[3]);
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
__global__ void __launch_bounds__(kRopeThreads, kRopeBlocks)
prompt_rope_kernel(const __grid_constant__ RopeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  constexpr int kVec = sizeof(In) == 4 ? 2 : 1;                  // vectors of eight channels
  __shared__ alignas(16) float weights[2][PROMPT_ROPE_MAX_D];
  __shared__ uint4 ring[kRopeAhead + 1][2 * kVec][kRopeThreads];  // a thread's own vectors alone
  const int lane = threadIdx.x & 31, L = 1 << p.shift, l = lane & (L - 1), sub_head = lane >> p.shift;
  const int per_step = 32 >> p.shift;
  const int64_t warp = static_cast<int64_t>(blockIdx.x) * (kRopeThreads / 32) + (threadIdx.x >> 5);
  int64_t left = p.share + (warp < p.extra ? 1 : 0);
  const int64_t first = p.share * warp + (warp < p.extra ? warp : p.extra);
  int64_t t = first >> 31 ? first / p.steps : static_cast<int>(first) / p.steps;   // (a short division will mostly do)
  int st = static_cast<int>(first - t * p.steps);

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
  const int pair0 = kInterleaved ? o0 / 2 : o0, pair1 = kInterleaved ? o1 / 2 : o0 + 4;   // four pairs from each
  uint32_t ax0 = 0, ax1 = 0;                   // their axes, a byte each
  if (on0) ax0 = *reinterpret_cast<const uint32_t*>(p.axes + pair0);
  if (on1) ax1 = *reinterpret_cast<const uint32_t*>(p.axes + pair1);

  // Lane a holds the position of axis a.
  const bool holds = lane < PROMPT_ROPE_MAX_AXES && (p.used >> lane & 1);
  auto position = [&](int64_t token) { return holds ? __ldg(p.positions + lane * p.axis_stride + token) : 0; };
  int pos = left > 0 ? position(t) : 0, pos_next = left > p.steps - st ? position(t + 1) : 0;

  // The vectors of a step; heads past the last one read the first.
  int64_t t_load = t;
  int s_load = st, slot_load = 0, h_load = 0, n_load = 0;
  const In* from = nullptr;                    // the queries' or keys' row
  auto enter_load = [&]() {
    const bool key = s_load >= p.steps_q;
    h_load = (key ? s_load - p.steps_q : s_load) * per_step + sub_head;
    n_load = key ? p.Hkv : p.Hq;
    from = static_cast<const In*>(key ? p.k : p.q) + t_load * (key ? p.k_stride : p.q_stride);
  };
  auto load = [&]() {
    const In* src = from + (h_load < n_load ? h_load * p.D : 0);
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      copy16(&ring[slot_load][i][threadIdx.x], src + o0 + 4 * i);
      copy16(&ring[slot_load][kVec + i][threadIdx.x], src + o1 + 4 * i);
    }
    slot_load = slot_load == kRopeAhead ? 0 : slot_load + 1;
    h_load += per_step;
    if (++s_load == p.steps) { s_load = 0; ++t_load; }
    if (s_load == 0 || s_load == p.steps_q) enter_load();
  };
  enter_load();
#pragma unroll 1
  for (int i = 0; i < kRopeAhead; ++i) {
    if (i < left) load();
    asm volatile("cp.async.commit_group;");
  }
  for (int e = threadIdx.x; e < p.D; e += kRopeThreads) {
    if (p.q_weight) weights[0][e] = __ldg(p.q_weight + e);
    if (p.k_weight) weights[1][e] = __ldg(p.k_weight + e);
  }
  __syncthreads();

  bool ok;
  float c[8], s[8];
  auto angles = [&]() {
    ok = !__any_sync(0xFFFFFFFFu, holds && (pos < 0 || pos >= p.n_pos));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int row = __shfl_sync(0xFFFFFFFFu, pos, (i < 4 ? ax0 : ax1) >> (8 * (i & 3)) & 31);
      c[i] = 1.0f;
      s[i] = 0.0f;
      if (ok && (i < 4 ? on0 : on1)) {
        const int64_t at = static_cast<int64_t>(row) * (p.rot / 2) + (i < 4 ? pair0 + i : pair1 + i - 4);
        c[i] = __ldg(p.cos + at);
        s[i] = __ldg(p.sin + at);
      }
    }
  };
  const float inv_D = 1.0f / static_cast<float>(p.D);
  const float* w = weights[0];
  Out* to = nullptr;
  int h = 0, n = 0, slot = 0;
  bool norm = false;
  auto enter = [&]() {
    const bool key = st >= p.steps_q;
    h = (key ? st - p.steps_q : st) * per_step + sub_head;
    n = key ? p.Hkv : p.Hq;
    to = static_cast<Out*>(key ? p.k_out : p.q_out) + t * (key ? p.ko_stride : p.qo_stride);
    w = weights[key];
    norm = (key ? p.k_weight : p.q_weight) != nullptr;
  };
  bool turn = true, side = true;               // a token's first step here, the queries' or keys'
#pragma unroll 1
  for (; left > 0; --left) {
    if (turn) {
      angles();
      pos = pos_next;
      if (left > 2 * p.steps - st) pos_next = position(t + 2);
    }
    if (side) enter();
    uint64_t a[4], b[4];
    asm volatile("cp.async.wait_group %0;" :: "n"(kRopeAhead - 1) : "memory");
    widen<In>(&ring[slot][0][threadIdx.x], a);
    widen<In>(&ring[slot][kVec][threadIdx.x], b);
    slot = slot == kRopeAhead ? 0 : slot + 1;
    if (left > kRopeAhead) load();
    asm volatile("cp.async.commit_group;");
    if (norm) {
      uint64_t two = f2_mul(a[0], a[0]);
#pragma unroll
      for (int i = 1; i < 4; ++i) two = f2_fma(a[i], a[i], two);
#pragma unroll
      for (int i = 0; i < 4; ++i) two = f2_fma(b[i], b[i], two);
      float ss = f2_lo(two) + f2_hi(two);
      for (int d = L / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, d);
      const float r = rsqrtf(fmaf(ss, inv_D, p.eps));
      const uint64_t r2 = f2_pack(r, r);
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const float4 wa = *reinterpret_cast<const float4*>(w + o0 + 2 * i), wb = *reinterpret_cast<const float4*>(w + o1 + 2 * i);
        a[i] = f2_mul(f2_mul(a[i], r2), f2_pack(wa.x, wa.y));
        a[i + 1] = f2_mul(f2_mul(a[i + 1], r2), f2_pack(wa.z, wa.w));
        b[i] = f2_mul(f2_mul(b[i], r2), f2_pack(wb.x, wb.y));
        b[i + 1] = f2_mul(f2_mul(b[i + 1], r2), f2_pack(wb.z, wb.w));
      }
    }
    if (kInterleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a0 = f2_lo(a[i]), a1 = f2_hi(a[i]), b0 = f2_lo(b[i]), b1 = f2_hi(b[i]);
        if (on0) a[i] = f2_pack(a0 * c[i] - a1 * s[i], a1 * c[i] + a0 * s[i]);
        if (on1) b[i] = f2_pack(b0 * c[i + 4] - b1 * s[i + 4], b1 * c[i + 4] + b0 * s[i + 4]);
      }
    } else if (on0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint64_t a0 = a[i], c2 = f2_pack(c[2 * i], c[2 * i + 1]), s2 = f2_pack(s[2 * i], s[2 * i + 1]);
        a[i] = f2_fma(b[i], s2 ^ 0x8000000080000000ull, f2_mul(a0, c2));
        b[i] = f2_fma(a0, s2, f2_mul(b[i], c2));
      }
    }
    if (!ok) {
      asm volatile("");                        // (a branch: it is hardly ever taken)
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = b[i] = 0;
    }
    if (h < n) {
      Out* dst = to + h * p.D;
      store8<Out>(dst + o0, a);
      store8<Out>(dst + o1, b);
    }
    h += per_step;
    turn = ++st == p.steps;
    if (turn) { st = 0; ++t; }
    side = st == 0 || st == p.steps_q;
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
// a lane at a time (a channel's partner is read again, before anything is stored).  Accesses of an
// element, and the angles loaded anew for every head, bind it: 4096 tokens of 32 heads of 80 channels
// 115 us (0.4 TB/s), 8192 tokens of 72 heads of 128 channels at odd addresses 720, 51 aligned.
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
  // results over their inputs element by element, or elsewhere
  auto over = [&](const void* in, int64_t stride, const void* out, int64_t out_stride) {
    return in == out && (dt != out_dt || (T > 1 && stride != out_stride));
  };
  if ((Hq > 0 && over(q, q_stride, q_out, q_out_stride)) || (Hkv > 0 && over(k, k_stride, k_out, k_out_stride)) ||
      (Hq > 0 && Hkv > 0 && (q_out == k || k_out == q || q_out == k_out)))
    return NVR_ERR_INVALID_ARG;
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
    const int64_t all = T * p.steps, most = static_cast<int64_t>(sms) * kRopeBlocks * (kRopeThreads / 32);
    units = all < most ? all : most;
    units = (units + kRopeThreads / 32 - 1) / (kRopeThreads / 32) * (kRopeThreads / 32);
    p.share = all / units;
    p.extra = all % units;
  } else {
    p.shift = 0;
    p.steps_q = p.steps = 0;
    p.share = p.extra = 0;
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
