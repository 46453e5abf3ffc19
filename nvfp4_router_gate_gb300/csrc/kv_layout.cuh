// kv_layout.cuh -- the NVFP4 key/value cache's page layout and the conversions
// its kernels share (sm_103a).  include/nvfp4_kv_cache.h describes the layout.
#pragma once

#include <cuda_fp16.h>

#include "nvr_device.cuh"

namespace nvr {

// Byte offsets of the four regions of one page of one KV head (S tokens).
template <int D>
struct KvPage {
  static constexpr int kCodeRow = D / 2;       // code bytes of one token
  static constexpr int kScaleRow = D / 16;     // scale bytes of one token
  __host__ __device__ static constexpr int key_scales(int S) { return S * kCodeRow; }
  __host__ __device__ static constexpr int value_codes(int S) { return S * (kCodeRow + kScaleRow); }
  __host__ __device__ static constexpr int value_scales(int S) { return S * (2 * kCodeRow + kScaleRow); }
  __host__ __device__ static constexpr int bytes(int S) { return 2 * S * (kCodeRow + kScaleRow); }
  // value code bytes / scale byte of (token t, channel block b)
  __host__ __device__ static constexpr int value_code(int t, int b) {
    return (t >> 3) * (8 * kCodeRow) + b * 64 + (t & 7) * 8;
  }
  __host__ __device__ static constexpr int value_scale(int t, int b) {
    return (t >> 3) * (8 * kScaleRow) + b * 8 + (t & 7);
  }
};

inline bool kv_page_size_ok(int S) { return S == 16 || S == 32 || S == 64 || S == 128; }
inline bool kv_head_dim_ok(int D) { return D == 64 || D == 128; }

// The four code bytes of a word as four half2 (element 2j in the low half).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t& a, uint32_t& b, uint32_t& c, uint32_t& d) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(a), "=r"(b), "=r"(c), "=r"(d) : "r"(w));
}

// Two scale bytes as half2 (the low byte in the low half); exact, NaN kept.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t two) {
  uint32_t r;
  asm("{\n\t.reg .b16 h, hi;\n\tmov.b32 {h, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(two));
  return r;
}

__device__ __forceinline__ uint32_t h2_mul(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

// Per half the smaller one; the other one for a NaN.
__device__ __forceinline__ uint32_t h2_min(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("min.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

}  // namespace nvr
