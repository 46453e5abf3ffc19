// kv_cache.cu -- writing the NVFP4 key/value cache and reading it back
// (sm_103a): nvfp4_kv_append (RMS norm of query and key heads, rotary
// positions, NVFP4 quantization, store into the pages) and nvfp4_kv_gather.
//
// Both move each byte once: append reads the fused projection's row, writes the
// query row in bf16 and the token's entry in 4.5 bits a value.  8192 tokens of 64
// query and 8 KV heads of 128 channels, bf16: append 69 us, 0.68 of the copy
// bandwidth (issue slots 63 % busy: every operation rounded by itself; 7 or 8 blocks
// an SM, and fetching a warp's later groups into L2 at its start, were not faster: 69,
// 75 and 74 us), gather 9.7 us, 0.66.  One token: 3.1 and 1.7 us, two launches.
#include "kv_layout.cuh"
#include "nvr_internal.h"
#include "../../include/nvfp4_kv_cache.h"

namespace nvr {

namespace {

constexpr int kAppendThreads = 128;

// How a head's channels are paired by the rotation.
enum : int {
  kRotAny = 0,          // half pairs at any distance (or no rotation)
  kRotInterleaved = 1,
  kRotHalf32 = 2,       // half pairs 32 apart: both in one lane's registers
  kRotHalf64 = 3        // half pairs 64 apart: the same
};

struct AppendParams {
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;
  int64_t T;
  int Hq, Hkv;
  const int32_t *positions, *slots;
  const float *cos, *sin;
  int64_t n_pos;
  int rot;
  const float *q_weight, *k_weight;
  float eps;
  const float *k_gsa, *v_gsa;
  uint8_t* cache;
  int64_t n_slots;
  int page_shift;       // page_size == 1 << page_shift
  __nv_bfloat16* q_out;
  int quads_q, quads_kv;           // groups of four heads
  int parts_q, parts_kv;           // warps for a token's queries, its keys (values)
};

// Four channels as they lie in memory, and as two fp32 pairs.
template <bool kBF16>
struct Raw {
  uint2 u;
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    u = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + at));
  }
  __device__ __forceinline__ void widen(uint64_t (&x)[2]) const {
    x[0] = f2_pack(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u));
    x[1] = f2_pack(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xFFFF0000u));
  }
};
template <>
struct Raw<false> {
  float4 u;
  __device__ __forceinline__ void load(const void* base, int64_t at) {
    u = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(base) + at));
  }
  __device__ __forceinline__ void widen(uint64_t (&x)[2]) const {
    x[0] = f2_pack(u.x, u.y);
    x[1] = f2_pack(u.z, u.w);
  }
};

template <bool kBF16>
__device__ __forceinline__ float load1(const void* base, int64_t at) {
  if (kBF16) return __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(base) + at)) << 16);
  return __ldg(static_cast<const float*>(base) + at);
}

__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
// a b + c d and a b - c d with every product rounded: scalar operations, which
// are never contracted (a packed product feeding a packed sum was, nvcc 13.0).
__device__ __forceinline__ uint64_t f2_mul_add_mul(uint64_t a, uint64_t b, uint64_t c, uint64_t d) {
  return f2_pack(__fadd_rn(__fmul_rn(f2_lo(a), f2_lo(b)), __fmul_rn(f2_lo(c), f2_lo(d))),
                 __fadd_rn(__fmul_rn(f2_hi(a), f2_hi(b)), __fmul_rn(f2_hi(c), f2_hi(d))));
}
__device__ __forceinline__ uint64_t f2_mul_sub_mul(uint64_t a, uint64_t b, uint64_t c, uint64_t d) {
  return f2_pack(__fsub_rn(__fmul_rn(f2_lo(a), f2_lo(b)), __fmul_rn(f2_lo(c), f2_lo(d))),
                 __fsub_rn(__fmul_rn(f2_hi(a), f2_hi(b)), __fmul_rn(f2_hi(c), f2_hi(d))));
}

__device__ __forceinline__ uint64_t shfl_xor2(uint64_t v, int d) {
  return f2_pack(__shfl_xor_sync(0xFFFFFFFFu, f2_lo(v), d), __shfl_xor_sync(0xFFFFFFFFu, f2_hi(v), d));
}

// E2M1 codes of four values under the block scale s of global scale qs, the
// quantizer's exact arithmetic; magnitudes are cut where the quotient is still
// far from overflow (they saturate from 2688 gsa on).
__device__ __noinline__ uint32_t codes4_exact(float4 v, float gsa, float s) {
  const QuantScale qs = quant_scale_of(gsa);
  const float cut = __fmul_rn(gsa, 4096.0f), rs = __frcp_rn(s);
  const float x[4] = {v.x, v.y, v.z, v.w};
  float c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = div_rn_short(quant_divide(fmaxf(fminf(x[i], cut), -cut), qs), s, rs);
  return e2m1_pack8(c[0], c[1], c[2], c[3], 0.0f, 0.0f, 0.0f, 0.0f);
}

// A warp takes one token and a run of groups of four heads of its queries, keys
// or values, eight lanes to a head.  Lane l of the eight holds channels
// 4 l + 32 j + i (j < D / 32, i < 4): the first levels of the norm's halving sum
// (D/2 .. 32 apart) and the usual half pairs of the rotation are then inside one
// lane, 16, 8 and 4 apart are lanes 4, 2 and 1 away, and a 16-channel scale block
// is four lanes.  Every operation is rounded by itself; the next group's loads are
// under way meanwhile, the rows of the tables and the weights stay in registers.
template <int D, bool kBF16, int kRot>
__global__ void __launch_bounds__(kAppendThreads, 6)
kv_append_kernel(const AppendParams p) {
  constexpr int J = D / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int lane = threadIdx.x & 31, l8 = lane & 7, hq4 = lane >> 3;
  int64_t unit = static_cast<int64_t>(blockIdx.x) * (kAppendThreads / 32) + (threadIdx.x >> 5);
  // section 0: queries, 1: keys, 2: values, one after the other over all tokens
  // (the warps of a block then do equal work); this warp's groups [g0, g1)
  const int64_t n_q = p.T * p.parts_q, n_kv = p.T * p.parts_kv;
  const int sec = unit < n_q ? 0 : unit < n_q + n_kv ? 1 : 2;
  if (unit >= n_q + 2 * n_kv) return;
  unit -= sec == 0 ? 0 : n_q + (sec - 1) * n_kv;
  const int64_t t = unit / (sec == 0 ? p.parts_q : p.parts_kv);
  const int sub = static_cast<int>(unit - t * (sec == 0 ? p.parts_q : p.parts_kv));
  const int groups = sec == 0 ? p.quads_q : p.quads_kv, parts = sec == 0 ? p.parts_q : p.parts_kv;
  const int g0 = groups * sub / parts, g1 = groups * (sub + 1) / parts;
  const int n_heads = sec == 0 ? p.Hq : p.Hkv;
  const void* base = sec == 0 ? p.q : sec == 1 ? p.k : p.v;
  const int64_t row = t * (sec == 0 ? p.q_stride : sec == 1 ? p.k_stride : p.v_stride) + 4 * l8;
  int head = 4 * g0 + hq4;                       // of this lane; heads past the last read the first
  Raw<kBF16> nxt[J];
  auto load = [&](int h) {
    const int64_t at = row + static_cast<int64_t>(h < n_heads ? h : 0) * D;
#pragma unroll
    for (int j = 0; j < J; ++j) nxt[j].load(base, at + 32 * j);
  };
  load(head);

  const int64_t pos = p.rot ? __ldg(p.positions + t) : 0;
  const int64_t slot = __ldg(p.slots + t);
  const bool pos_ok = p.rot == 0 || (pos >= 0 && pos < p.n_pos);
  if (sec > 0 && (!pos_ok || slot < 0 || slot >= p.n_slots)) return;      // nothing is stored
  const int half = p.rot / 2;
  const float* weight = sec == 0 ? p.q_weight : sec == 1 ? p.k_weight : nullptr;
  constexpr int kCs = kRot == kRotHalf64 ? 2 : kRot == kRotHalf32 ? 1 : J;
  uint64_t cs[kCs][2], sn[kCs][2]; // this lane's channels, pairs of neighbours
  if (sec < 2) {
    const float* cosr = p.cos + (pos_ok ? pos : 0) * half;
    const float* sinr = p.sin + (pos_ok ? pos : 0) * half;
#pragma unroll
    for (int j = 0; j < kCs; ++j) {
      float c[4], s[4];
      if (kRot == kRotHalf32 || kRot == kRotHalf64) {
        const float4 cv = __ldg(reinterpret_cast<const float4*>(cosr + 4 * l8 + 32 * j));
        const float4 sv = __ldg(reinterpret_cast<const float4*>(sinr + 4 * l8 + 32 * j));
        c[0] = cv.x; c[1] = cv.y; c[2] = cv.z; c[3] = cv.w;
        s[0] = sv.x; s[1] = sv.y; s[2] = sv.z; s[3] = sv.w;
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = 4 * l8 + 32 * j + i;
          const int f = kRot == kRotInterleaved ? e / 2 : (e < half ? e : e - half);
          const bool on = e < p.rot;
          c[i] = on ? __ldg(cosr + f) : 1.0f;
          s[i] = on ? __ldg(sinr + f) : 0.0f;
          // interleaved: the even channel of a pair takes -sin of the odd one
          if (kRot == kRotInterleaved && i % 2 == 0) s[i] = -s[i];
        }
      }
      cs[j][0] = f2_pack(c[0], c[1]); cs[j][1] = f2_pack(c[2], c[3]);
      sn[j][0] = f2_pack(s[0], s[1]); sn[j][1] = f2_pack(s[2], s[3]);
    }
  }

  // x of head h: norm and rotation
  auto turn = [&](uint64_t (&x)[J][2], int h) {
    float r = 1.0f;
    if (weight) {
      uint64_t u[J][2];                          // squares of chunks j and j + J / 2, added
#pragma unroll
      for (int j = 0; j < J / 2; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          u[j][i] = f2_mul_add_mul(x[j][i], x[j][i], x[j + J / 2][i], x[j + J / 2][i]);
#pragma unroll
      for (int k = J / 4; k > 0; k >>= 1)
#pragma unroll
        for (int j = 0; j < k; ++j) {
          u[j][0] = f2_add(u[j][0], u[j + k][0]);
          u[j][1] = f2_add(u[j][1], u[j + k][1]);
        }
#pragma unroll
      for (int d = 4; d > 0; d >>= 1) {
        u[0][0] = f2_add(u[0][0], shfl_xor2(u[0][0], d));
        u[0][1] = f2_add(u[0][1], shfl_xor2(u[0][1], d));
      }
      const uint64_t two = f2_add(u[0][0], u[0][1]);
      const float ss = __fadd_rn(f2_lo(two), f2_hi(two));
      r = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(ss, 1.0f / D), p.eps)));
      const uint64_t r2 = f2_pack(r, r);
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const float4 w = __ldg(reinterpret_cast<const float4*>(weight + 4 * l8 + 32 * j));
        x[j][0] = f2_mul(f2_mul(x[j][0], r2), f2_pack(w.x, w.y));
        x[j][1] = f2_mul(f2_mul(x[j][1], r2), f2_pack(w.z, w.w));
      }
    }
    if (kRot == kRotHalf32 || kRot == kRotHalf64) {
      constexpr int o = kRot == kRotHalf64 ? 2 : 1;
#pragma unroll
      for (int j = 0; j < (J >= 2 * o ? o : 0); ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint64_t a = x[j][i], b = x[j + o][i];
          x[j][i] = f2_mul_sub_mul(a, cs[j][i], b, sn[j][i]);
          x[j + o][i] = f2_mul_add_mul(b, cs[j][i], a, sn[j][i]);
        }
    } else if (kRot == kRotInterleaved) {
      // (a, b) -> (a c + b (-s), b c + a s)
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint64_t turned =
              f2_mul_add_mul(x[j][i], cs[j][i], f2_pack(f2_hi(x[j][i]), f2_lo(x[j][i])), sn[j][i]);
          if (4 * l8 + 32 * j + 2 * i < p.rot) x[j][i] = turned;
        }
    } else if (p.rot) {
      // the partner channel is another lane's: read it again and put it through
      // the same norm
      const int64_t at = row - 4 * l8 + static_cast<int64_t>(h < n_heads ? h : 0) * D;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int e = 4 * l8 + 32 * j + i;
          const uint64_t xv = x[j][i / 2], cv = cs[j][i / 2], sv = sn[j][i / 2];
          y[i] = i % 2 ? f2_hi(xv) : f2_lo(xv);
          if (e < p.rot) {
            const int f = e < half ? e + half : e - half;
            float z = load1<kBF16>(base, at + f);
            if (weight) z = __fmul_rn(__fmul_rn(z, r), __ldg(weight + f));
            const float xc = __fmul_rn(y[i], i % 2 ? f2_hi(cv) : f2_lo(cv));
            const float zs = __fmul_rn(z, i % 2 ? f2_hi(sv) : f2_lo(sv));
            y[i] = e < half ? __fsub_rn(xc, zs) : __fadd_rn(xc, zs);
          }
        }
        x[j][0] = f2_pack(y[0], y[1]);
        x[j][1] = f2_pack(y[2], y[3]);
      }
    }
  };

  if (sec == 0) {
    __nv_bfloat16* out = p.q_out + t * p.Hq * D + static_cast<int64_t>(head) * D + 4 * l8;
#pragma unroll 1
    for (int g = g0; g < g1; ++g) {
      uint64_t x[J][2];
#pragma unroll
      for (int j = 0; j < J; ++j) nxt[j].widen(x[j]);
      const int now = head;
      head += 4;
      if (g + 1 < g1) load(head);
      turn(x, now);
      if (now < n_heads) {
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const __nv_bfloat162 lo = __floats2bfloat162_rn(f2_lo(x[j][0]), f2_hi(x[j][0])),
                               hi = __floats2bfloat162_rn(f2_lo(x[j][1]), f2_hi(x[j][1]));
          uint2 u = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
          if (!pos_ok) u = make_uint2(0u, 0u);
          *reinterpret_cast<uint2*>(out + 32 * j) = u;
        }
      }
      out += 4 * D;
    }
    return;
  }

  const int S = 1 << p.page_shift, tok = static_cast<int>(slot) & (S - 1);
  // codes and scales of this token's first block; 16 channels on they are
  // code_step and scale_step bytes further
  const bool key = sec == 1;
  const int code_at = key ? tok * KvPage<D>::kCodeRow : KvPage<D>::value_codes(S) + KvPage<D>::value_code(tok, 0);
  const int scale_at = key ? KvPage<D>::key_scales(S) + tok * KvPage<D>::kScaleRow
                           : KvPage<D>::value_scales(S) + KvPage<D>::value_scale(tok, 0);
  const int code_step = key ? 8 : 64, scale_step = key ? 1 : 8;
#pragma unroll 1
  for (int g = g0; g < g1; ++g) {
    uint64_t x[J][2];
#pragma unroll
    for (int j = 0; j < J; ++j) nxt[j].widen(x[j]);
    const int now = head;
    head += 4;
    if (g + 1 < g1) load(head);
    if (key) turn(x, now);
    const bool live = now < n_heads;
    const float gsa = __ldg((key ? p.k_gsa : p.v_gsa) + (live ? now : 0));
    const QuantScale qs = quant_scale_of(gsa);
    uint8_t* page = p.cache + ((slot >> p.page_shift) * p.Hkv + now) * KvPage<D>::bytes(S);
    // The four lanes of a block have the largest magnitude of each of their J
    // blocks; lane j of them finds the scale of block j.  RN(|x| / gsa) is
    // monotone: a block's largest quotient is that of its largest magnitude.
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      float m = fmaxf(fmaxf(fabsf(f2_lo(x[j][0])), fabsf(f2_hi(x[j][0]))),
                      fmaxf(fabsf(f2_lo(x[j][1])), fabsf(f2_hi(x[j][1]))));
      m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      if ((l8 & 3) == j) amax = m;
    }
    const uint32_t my_byte = quant_scale_byte(fminf(amax, __fmul_rn(gsa, 4096.0f)), qs);
    const float my_c = my_byte ? __fmul_rn(qs.rgsa, __frcp_rn(e4m3_value(my_byte))) : 0.0f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const uint32_t byte = __shfl_sync(0xFFFFFFFFu, my_byte, (lane & ~3) + j);
      const float c = __shfl_sync(0xFFFFFFFFu, my_c, (lane & ~3) + j);
      uint32_t code = 0;
      if (byte) {
        // x c brackets the exact quotient when c is off by a little more than all
        // roundings: equal codes on both sides are the exact ones (as in
        // quant_block16_bracket)
        const float c_lo = __fmul_rn(c, 0.99999904632568359375f), c_hi = __fmul_rn(c, 1.00000095367431640625f);
        const uint64_t lo2 = f2_pack(c_lo, c_lo), hi2 = f2_pack(c_hi, c_hi);
        const uint64_t a0 = f2_mul(x[j][0], lo2), a1 = f2_mul(x[j][1], lo2);
        const uint64_t b0 = f2_mul(x[j][0], hi2), b1 = f2_mul(x[j][1], hi2);
        code = e2m1_pack8(f2_lo(a0), f2_hi(a0), f2_lo(a1), f2_hi(a1), f2_lo(b0), f2_hi(b0), f2_lo(b1), f2_hi(b1));
        const bool same = (code >> 16) == (code & 0xFFFFu) && qs.mode == 1;
        code &= 0xFFFFu;
        if (!same)
          code = codes4_exact(make_float4(f2_lo(x[j][0]), f2_hi(x[j][0]), f2_lo(x[j][1]), f2_hi(x[j][1])), gsa,
                              e4m3_value(byte));
        // the conversion gives +0 for a negative value that rounds to zero
        code |= (__float_as_uint(f2_lo(x[j][0])) >> 31 << 3) | (__float_as_uint(f2_hi(x[j][0])) >> 31 << 7) |
                (__float_as_uint(f2_lo(x[j][1])) >> 31 << 11) | (__float_as_uint(f2_hi(x[j][1])) >> 31 << 15);
      }
      __syncwarp();
      // the block's eight code bytes to its first lane
      code |= __shfl_down_sync(0xFFFFFFFFu, code, 1) << 16;
      const uint32_t hi = __shfl_down_sync(0xFFFFFFFFu, code, 2);
      if (live && (l8 & 3) == 0) {
        const int b = 2 * j + (l8 >> 2);
        *reinterpret_cast<uint2*>(page + code_at + b * code_step) = make_uint2(code, hi);
        page[scale_at + b * scale_step] = static_cast<uint8_t>(byte);
      }
    }
  }
}

template <int D, bool kBF16>
cudaError_t launch_append(int rot_kind, cudaLaunchConfig_t* cfg, const AppendParams& p) {
  switch (rot_kind) {
    case kRotInterleaved: return cudaLaunchKernelEx(cfg, kv_append_kernel<D, kBF16, kRotInterleaved>, p);
    case kRotHalf32: return cudaLaunchKernelEx(cfg, kv_append_kernel<D, kBF16, kRotHalf32>, p);
    case kRotHalf64:
      if (D == 128) return cudaLaunchKernelEx(cfg, kv_append_kernel<D, kBF16, D == 128 ? kRotHalf64 : kRotAny>, p);
      break;
    default: break;
  }
  return cudaLaunchKernelEx(cfg, kv_append_kernel<D, kBF16, kRotAny>, p);
}

// ------------------------------------------------------------------ gather
// One thread per (slot, head, 16-channel block): its key and its value block.
template <int D, bool kOutBF16>
__global__ void __launch_bounds__(256)
kv_gather_kernel(const uint8_t* __restrict__ cache, int64_t n_slots, int page_shift, int Hkv,
                 const int32_t* __restrict__ slots, int64_t n, const float* __restrict__ k_gsa,
                 const float* __restrict__ v_gsa, void* __restrict__ k_out, void* __restrict__ v_out) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  constexpr int NB = D / 16;
  const int S = 1 << page_shift;
  const int64_t total = n * Hkv * NB;
  for (int64_t g = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x; g < total;
       g += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t row = g / NB;                   // (slot, head)
    const int b = static_cast<int>(g - row * NB);
    const int64_t i = row / Hkv;
    const int h = static_cast<int>(row - i * Hkv);
    const int64_t slot = __ldg(slots + i);
    const bool ok = slot >= 0 && slot < n_slots;
    const int tok = static_cast<int>(slot) & (S - 1);
    const uint8_t* page = cache + ((ok ? slot >> page_shift : 0) * Hkv + h) * KvPage<D>::bytes(S);
#pragma unroll
    for (int kv = 0; kv < 2; ++kv) {
      float y[16];
      if (ok) {
        const uint2 c = *reinterpret_cast<const uint2*>(
            kv == 0 ? page + tok * KvPage<D>::kCodeRow + 8 * b
                    : page + KvPage<D>::value_codes(S) + KvPage<D>::value_code(tok, b));
        const uint32_t byte = kv == 0 ? page[KvPage<D>::key_scales(S) + tok * KvPage<D>::kScaleRow + b]
                                      : page[KvPage<D>::value_scales(S) + KvPage<D>::value_scale(tok, b)];
        const uint32_t s2 = e4m3x2_to_f16(byte);
        const float s = __low2float(*reinterpret_cast<const __half2*>(&s2));
        const float gsa = __ldg((kv == 0 ? k_gsa : v_gsa) + h);
        uint32_t f[8];
        e2m1x8_to_f16(c.x, f[0], f[1], f[2], f[3]);
        e2m1x8_to_f16(c.y, f[4], f[5], f[6], f[7]);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&f[e]));
          y[2 * e] = __fmul_rn(__fmul_rn(v.x, s), gsa);       // code * scale is exact
          y[2 * e + 1] = __fmul_rn(__fmul_rn(v.y, s), gsa);
        }
      } else {
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] = 0.0f;
      }
      void* out = kv == 0 ? k_out : v_out;
      if (kOutBF16) {
        uint32_t w[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const __nv_bfloat162 v = __floats2bfloat162_rn(y[2 * e], y[2 * e + 1]);
          w[e] = *reinterpret_cast<const uint32_t*>(&v);
        }
        uint4* o = reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + row * D + 16 * b);
        o[0] = make_uint4(w[0], w[1], w[2], w[3]);
        o[1] = make_uint4(w[4], w[5], w[6], w[7]);
      } else {
        float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + row * D + 16 * b);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = make_float4(y[4 * e], y[4 * e + 1], y[4 * e + 2], y[4 * e + 3]);
      }
    }
  }
}

int page_shift_of(int S) { return S == 16 ? 4 : S == 32 ? 5 : S == 64 ? 6 : 7; }

bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool off4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

}  // namespace

}  // namespace nvr

using namespace nvr;

extern "C" size_t nvfp4_kv_page_bytes(int page_size, int D) {
  if (!kv_page_size_ok(page_size) || !kv_head_dim_ok(D)) return 0;
  return static_cast<size_t>(page_size) * D * 9 / 8;
}

extern "C" nvr_status nvfp4_kv_append(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                      int64_t v_stride, nvr_dtype dt, int64_t T, int Hq, int Hkv, int D,
                                      const int32_t* positions, const int32_t* slots, const float* cos,
                                      const float* sin, int64_t n_pos, int rot, int interleaved,
                                      const float* q_weight, const float* k_weight, float eps, const float* k_gsa,
                                      const float* v_gsa, uint8_t* cache, int64_t n_pages, int page_size, void* q_out,
                                      nvr_stream_t stream) {
  if (T < 0 || Hq < 0 || Hq > 65536 || Hkv < 1 || Hkv > 65536 || n_pages < 1) return NVR_ERR_INVALID_ARG;
  if (dt != NVR_BF16 && dt != NVR_F32) return NVR_ERR_INVALID_ARG;
  if (!kv_head_dim_ok(D) || !kv_page_size_ok(page_size)) return NVR_ERR_UNSUPPORTED;
  if (rot < 0 || rot > D || rot % 2 != 0 || (rot > 0 && n_pos < 1)) return NVR_ERR_INVALID_ARG;
  if (!(eps >= 0.0f)) return NVR_ERR_INVALID_ARG;
  if (!k_gsa || !v_gsa || !cache) return NVR_ERR_INVALID_ARG;
  if (T > 0 && (!k || !v || !slots || (Hq > 0 && (!q || !q_out)))) return NVR_ERR_INVALID_ARG;
  if (T > 0 && rot > 0 && (!positions || !cos || !sin)) return NVR_ERR_INVALID_ARG;
  if (n_pages > INT32_MAX / page_size) return NVR_ERR_UNSUPPORTED;     // slots are int32
  const int vec = dt == NVR_BF16 ? 8 : 4;                              // elements of 16 bytes
  if ((Hq > 0 && (q_stride < static_cast<int64_t>(Hq) * D || q_stride % vec)) ||
      k_stride < static_cast<int64_t>(Hkv) * D || k_stride % vec || v_stride < static_cast<int64_t>(Hkv) * D ||
      v_stride % vec)
    return NVR_ERR_INVALID_ARG;
  if (off16(q) || off16(k) || off16(v) || off16(cache) || off16(q_out) || off16(cos) || off16(sin) ||
      off16(q_weight) || off16(k_weight) || off4(positions) || off4(slots) || off4(k_gsa) || off4(v_gsa))
    return NVR_ERR_ALIGNMENT;
  if (T == 0) return NVR_OK;
  const int sms = device_sm_count();
  if (sms <= 0) return NVR_ERR_CUDA;
  AppendParams p;
  p.q = q; p.k = k; p.v = v;
  p.q_stride = q_stride; p.k_stride = k_stride; p.v_stride = v_stride;
  p.T = T; p.Hq = Hq; p.Hkv = Hkv;
  p.positions = positions; p.slots = slots; p.cos = cos; p.sin = sin; p.n_pos = n_pos; p.rot = rot;
  p.q_weight = q_weight; p.k_weight = k_weight; p.eps = eps; p.k_gsa = k_gsa; p.v_gsa = v_gsa;
  p.cache = cache; p.n_slots = n_pages * page_size; p.page_shift = page_shift_of(page_size);
  p.q_out = static_cast<__nv_bfloat16*>(q_out);
  p.quads_q = (Hq + 3) / 4;
  p.quads_kv = (Hkv + 3) / 4;
  // A warp takes as many groups of four heads as let all warps run at once (24 an SM),
  // up to sixteen of queries and four of keys or of values: they share the rows of the
  // tables and the weights.  64 and 8 heads of 128 channels, one group a warp / this /
  // sixteen: 128 tokens 4.4 / 4.4 / 7.1 us, 600: 9.2 / 7.7 / 8.9, 1000: 14.0 / 11.0 /
  // 16.6, 2000: 25.6 / 17.9 / 17.3, 8192: 111 / 69 / 69.
  const int64_t each = (T * (p.quads_q + 2 * p.quads_kv) + sms * 24 - 1) / (sms * 24);
  const int per_q = each < 16 ? static_cast<int>(each) : 16, per_kv = each < 4 ? static_cast<int>(each) : 4;
  p.parts_q = (p.quads_q + per_q - 1) / per_q;
  p.parts_kv = (p.quads_kv + per_kv - 1) / per_kv;
  const int64_t units = T * (p.parts_q + 2 * p.parts_kv);
  const int64_t blocks = (units + kAppendThreads / 32 - 1) / (kAppendThreads / 32);
  if (blocks > INT32_MAX) return NVR_ERR_UNSUPPORTED;
  int kind = kRotAny;
  if (rot > 0 && interleaved) kind = kRotInterleaved;
  else if (rot == 128) kind = kRotHalf64;
  else if (rot == 64) kind = kRotHalf32;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(kAppendThreads);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  const bool bf16 = dt == NVR_BF16;
  return cuda_status(D == 128 ? (bf16 ? launch_append<128, true>(kind, &cfg, p) : launch_append<128, false>(kind, &cfg, p))
                              : (bf16 ? launch_append<64, true>(kind, &cfg, p) : launch_append<64, false>(kind, &cfg, p)));
}

extern "C" nvr_status nvfp4_kv_gather(const uint8_t* cache, int64_t n_pages, int page_size, int Hkv, int D,
                                      const int32_t* slots, int64_t n, const float* k_gsa, const float* v_gsa,
                                      void* k_out, void* v_out, nvr_dtype out_dt, nvr_stream_t stream) {
  if (n < 0 || Hkv < 1 || Hkv > 65536 || n_pages < 1) return NVR_ERR_INVALID_ARG;
  if (out_dt != NVR_BF16 && out_dt != NVR_F32) return NVR_ERR_INVALID_ARG;
  if (!kv_head_dim_ok(D) || !kv_page_size_ok(page_size)) return NVR_ERR_UNSUPPORTED;
  if (!cache || !k_gsa || !v_gsa) return NVR_ERR_INVALID_ARG;
  if (n > 0 && (!slots || !k_out || !v_out)) return NVR_ERR_INVALID_ARG;
  if (n_pages > INT32_MAX / page_size) return NVR_ERR_UNSUPPORTED;
  if (off16(cache) || off16(k_out) || off16(v_out) || off4(slots) || off4(k_gsa) || off4(v_gsa))
    return NVR_ERR_ALIGNMENT;
  if (n == 0) return NVR_OK;
  const int sms = device_sm_count();
  if (sms <= 0) return NVR_ERR_CUDA;
  int64_t grid = (n * Hkv * (D / 16) + 255) / 256;
  if (grid > static_cast<int64_t>(sms) * 32) grid = static_cast<int64_t>(sms) * 32;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(256);
  cfg.stream = reinterpret_cast<cudaStream_t>(stream);
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  const int64_t n_slots = n_pages * page_size;
  const int shift = page_shift_of(page_size);
  auto go = [&](auto kernel) {
    return cuda_status(cudaLaunchKernelEx(&cfg, kernel, cache, n_slots, shift, Hkv, slots, n, k_gsa, v_gsa, k_out, v_out));
  };
  if (D == 128) return out_dt == NVR_BF16 ? go(kv_gather_kernel<128, true>) : go(kv_gather_kernel<128, false>);
  return out_dt == NVR_BF16 ? go(kv_gather_kernel<64, true>) : go(kv_gather_kernel<64, false>);
}
