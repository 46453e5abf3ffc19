// kv_cache.cu -- writing the NVFP4 key/value cache and reading it back
// (sm_103a): nvfp4_kv_append (RMS norm of query and key heads, rotary
// positions, NVFP4 quantization, store into the pages) and nvfp4_kv_gather.
//
// Both move each byte once and are bound by memory: append reads the fused
// projection's row, writes the query row in bf16 and the token's entry in 4.5
// bits a value.
#include "kv_layout.cuh"
#include "nvr_internal.h"
#include "../../include/nvfp4_kv_cache.h"

namespace nvr {

namespace {

constexpr int kAppendThreads = 256;

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
  int quads_q, quads_kv, parts;
};

template <bool kBF16>
__device__ __forceinline__ float4 load4(const void* base, int64_t at) {
  if (kBF16) {
    const uint2 u = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(base) + at));
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xFFFF0000u));
  }
  return __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(base) + at));
}

template <bool kBF16>
__device__ __forceinline__ float load1(const void* base, int64_t at) {
  if (kBF16) return __uint_as_float(static_cast<uint32_t>(__ldg(static_cast<const uint16_t*>(base) + at)) << 16);
  return __ldg(static_cast<const float*>(base) + at);
}

// One warp: `quads_per_part` groups of four heads of one token, eight lanes to
// a head.  Lane l of the eight holds channels 4 l + 32 j + i (j < D / 32, i < 4):
// the first levels of the norm's halving sum (D/2 .. 32 apart) and the usual
// half pairs of the rotation are then inside one lane, 16, 8 and 4 apart are
// lanes 4, 2 and 1 away, and a 16-channel scale block is four lanes.
template <int D, bool kBF16, int kRot>
__global__ void __launch_bounds__(kAppendThreads)
kv_append_kernel(const AppendParams p) {
  constexpr int J = D / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;");
  const int lane = threadIdx.x & 31, l8 = lane & 7, hq4 = lane >> 3;
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kAppendThreads / 32) + (threadIdx.x >> 5);
  const int64_t t = unit / p.parts;
  if (t >= p.T) return;
  const int part = static_cast<int>(unit - t * p.parts);
  const int n_quads = p.quads_q + 2 * p.quads_kv;
  const int q0 = static_cast<int>(static_cast<int64_t>(n_quads) * part / p.parts);
  const int q1 = static_cast<int>(static_cast<int64_t>(n_quads) * (part + 1) / p.parts);
  const int64_t pos = p.rot ? __ldg(p.positions + t) : 0;
  const bool pos_ok = p.rot == 0 || (pos >= 0 && pos < p.n_pos);
  const int64_t slot = pos_ok ? __ldg(p.slots + t) : -1;
  const bool stored = slot >= 0 && slot < p.n_slots;
  const int half = p.rot / 2;
  const float* cosr = p.cos + (pos_ok ? pos : 0) * half;
  const float* sinr = p.sin + (pos_ok ? pos : 0) * half;

  // this lane's rows of the tables, kept over the heads of the token
  constexpr int kCs = kRot == kRotHalf64 ? 2 : kRot == kRotHalf32 ? 1 : J;
  float cs[kCs][4], sn[kCs][4];
#pragma unroll
  for (int j = 0; j < kCs; ++j) {
    if (kRot == kRotHalf32 || kRot == kRotHalf64) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(cosr + 4 * l8 + 32 * j));
      const float4 s = __ldg(reinterpret_cast<const float4*>(sinr + 4 * l8 + 32 * j));
      cs[j][0] = c.x; cs[j][1] = c.y; cs[j][2] = c.z; cs[j][3] = c.w;
      sn[j][0] = s.x; sn[j][1] = s.y; sn[j][2] = s.z; sn[j][3] = s.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = 4 * l8 + 32 * j + i;
        const int f = kRot == kRotInterleaved ? e / 2 : (e < half ? e : e - half);
        const bool on = e < p.rot;
        cs[j][i] = on ? __ldg(cosr + f) : 1.0f;
        sn[j][i] = on ? __ldg(sinr + f) : 0.0f;
      }
    }
  }

  for (int qd = q0; qd < q1; ++qd) {
    // section 0: queries, 1: keys, 2: values
    const int sec = qd < p.quads_q ? 0 : (qd < p.quads_q + p.quads_kv ? 1 : 2);
    const int head = 4 * (qd - (sec == 0 ? 0 : sec == 1 ? p.quads_q : p.quads_q + p.quads_kv)) + hq4;
    const int n_heads = sec == 0 ? p.Hq : p.Hkv;
    const bool live = head < n_heads;
    const void* base = sec == 0 ? p.q : sec == 1 ? p.k : p.v;
    const int64_t row = t * (sec == 0 ? p.q_stride : sec == 1 ? p.k_stride : p.v_stride) +
                        static_cast<int64_t>(live ? head : 0) * D;
    float x[J][4];
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const float4 a = load4<kBF16>(base, row + 4 * l8 + 32 * j);
      x[j][0] = a.x; x[j][1] = a.y; x[j][2] = a.z; x[j][3] = a.w;
    }
    if (sec < 2) {
      const float* weight = sec == 0 ? p.q_weight : p.k_weight;
      float r = 1.0f;
      if (weight) {
        float s[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float u[J];
#pragma unroll
          for (int j = 0; j < J; ++j) u[j] = __fmul_rn(x[j][i], x[j][i]);
#pragma unroll
          for (int h = J / 2; h > 0; h >>= 1)
#pragma unroll
            for (int j = 0; j < h; ++j) u[j] = __fadd_rn(u[j], u[j + h]);
          s[i] = u[0];
        }
#pragma unroll
        for (int d = 4; d > 0; d >>= 1)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[i] = __fadd_rn(s[i], __shfl_xor_sync(0xFFFFFFFFu, s[i], d));
        const float ss = __fadd_rn(__fadd_rn(s[0], s[2]), __fadd_rn(s[1], s[3]));
        r = __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(ss, 1.0f / D), p.eps)));
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const float4 w = __ldg(reinterpret_cast<const float4*>(weight + 4 * l8 + 32 * j));
          x[j][0] = __fmul_rn(__fmul_rn(x[j][0], r), w.x);
          x[j][1] = __fmul_rn(__fmul_rn(x[j][1], r), w.y);
          x[j][2] = __fmul_rn(__fmul_rn(x[j][2], r), w.z);
          x[j][3] = __fmul_rn(__fmul_rn(x[j][3], r), w.w);
        }
      }
      if (kRot == kRotHalf32 || kRot == kRotHalf64) {
        constexpr int o = kRot == kRotHalf64 ? 2 : 1;
#pragma unroll
        for (int j = 0; j < (J >= 2 * o ? o : 0); ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float a = x[j][i], b = x[j + o][i];
            x[j][i] = __fsub_rn(__fmul_rn(a, cs[j][i]), __fmul_rn(b, sn[j][i]));
            x[j + o][i] = __fadd_rn(__fmul_rn(b, cs[j][i]), __fmul_rn(a, sn[j][i]));
          }
      } else if (kRot == kRotInterleaved) {
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            if (4 * l8 + 32 * j + i < p.rot) {
              const float a = x[j][i], b = x[j][i + 1];
              x[j][i] = __fsub_rn(__fmul_rn(a, cs[j][i]), __fmul_rn(b, sn[j][i]));
              x[j][i + 1] = __fadd_rn(__fmul_rn(b, cs[j][i]), __fmul_rn(a, sn[j][i]));
            }
          }
      } else {
        // the partner channel is another lane's: read it again and put it
        // through the same norm
#pragma unroll
        for (int j = 0; j < J; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e = 4 * l8 + 32 * j + i;
            if (e < p.rot) {
              const int f = e < half ? e + half : e - half;
              float y = load1<kBF16>(base, row + f);
              if (weight) y = __fmul_rn(__fmul_rn(y, r), __ldg(weight + f));
              const float xc = __fmul_rn(x[j][i], cs[j][i]), ys = __fmul_rn(y, sn[j][i]);
              x[j][i] = e < half ? __fsub_rn(xc, ys) : __fadd_rn(xc, ys);
            }
          }
      }
    }
    if (sec == 0) {
      if (live) {
        __nv_bfloat16* o = p.q_out + (t * p.Hq + head) * D + 4 * l8;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const __nv_bfloat162 lo = __floats2bfloat162_rn(x[j][0], x[j][1]), hi = __floats2bfloat162_rn(x[j][2], x[j][3]);
          uint2 u = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
          if (!pos_ok) u = make_uint2(0u, 0u);
          *reinterpret_cast<uint2*>(o + 32 * j) = u;
        }
      }
      continue;
    }
    if (!stored) continue;                       // warp-uniform: one token per warp
    const float gsa = __ldg((sec == 1 ? p.k_gsa : p.v_gsa) + (live ? head : 0));
    const QuantScale qs = quant_scale_of(gsa);
    // beyond 2688 gsa every magnitude gets the largest scale and code: cut where
    // the quotient is still far from overflow
    const float cut = __fmul_rn(gsa, 4096.0f);
#pragma unroll
    for (int j = 0; j < J; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[j][i] = fmaxf(fminf(x[j][i], cut), -cut);
    const int S = 1 << p.page_shift, tok = static_cast<int>(slot) & (S - 1);
    uint8_t* page = p.cache + ((slot >> p.page_shift) * p.Hkv + head) * KvPage<D>::bytes(S);
#pragma unroll
    for (int j = 0; j < J; ++j) {
      // RN(|x| / gsa) is monotone: the block's largest quotient is the quotient
      // of its largest magnitude
      float m = fmaxf(fmaxf(fabsf(x[j][0]), fabsf(x[j][1])), fmaxf(fabsf(x[j][2]), fabsf(x[j][3])));
      m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      const uint32_t byte = quant_scale_byte(m, qs);
      uint32_t code = 0;
      if (byte) {
        const float s = e4m3_value(byte), rs = __frcp_rn(s);
        float c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) c[i] = div_rn_short(quant_divide(x[j][i], qs), s, rs);
        code = e2m1_pack8(c[0], c[1], c[2], c[3], 0.0f, 0.0f, 0.0f, 0.0f);
        // the conversion gives +0 for a negative value that rounds to zero
#pragma unroll
        for (int i = 0; i < 4; ++i) code |= (__float_as_uint(x[j][i]) >> 31) << (4 * i + 3);
      }
      // the block's eight code bytes to its first lane
      code |= __shfl_down_sync(0xFFFFFFFFu, code, 1) << 16;
      const uint32_t hi = __shfl_down_sync(0xFFFFFFFFu, code, 2);
      if (live && (l8 & 3) == 0) {
        const int b = 2 * j + (l8 >> 2);
        if (sec == 1) {
          *reinterpret_cast<uint2*>(page + tok * KvPage<D>::kCodeRow + 8 * b) = make_uint2(code, hi);
          page[KvPage<D>::key_scales(S) + tok * KvPage<D>::kScaleRow + b] = static_cast<uint8_t>(byte);
        } else {
          *reinterpret_cast<uint2*>(page + KvPage<D>::value_codes(S) + KvPage<D>::value_code(tok, b)) =
              make_uint2(code, hi);
          page[KvPage<D>::value_scales(S) + KvPage<D>::value_scale(tok, b)] = static_cast<uint8_t>(byte);
        }
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
  if (n_pages * page_size > INT32_MAX) return NVR_ERR_UNSUPPORTED;     // slots are int32
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
  // A warp takes a part of one token's groups of four heads.  While a group per
  // warp does not fill the GPU (eight warps of work per scheduler), every
  // group gets its own warp; beyond that a warp takes about five, so that the
  // rows of the tables are loaded once for them.
  const int n_quads = p.quads_q + 2 * p.quads_kv;
  p.parts = T * n_quads <= static_cast<int64_t>(sms) * 32 ? n_quads : (n_quads + 4) / 5;
  const int64_t units = T * p.parts;
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
  if (n_pages * page_size > INT32_MAX) return NVR_ERR_UNSUPPORTED;
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
