// sa_kv8_device.cuh -- device helpers of the 8-bit paged cache: tokens and
// pages, scales, and the conversions between codes and 16-bit floats.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <stdint.h>

#include "sa_device.cuh"
#include "sa_kv8.h"

namespace sa {

__device__ __forceinline__ int k8_quot(const K8Div& v, int n) { return (int)(__umulhi(2u * (uint32_t)n, v.m) >> v.s); }
__device__ __forceinline__ int k8_rem(const K8Div& v, int n) { return n - k8_quot(v, n) * v.d; }

// Every read of the caller's memory is an ordinary load (or a copy): the kernels start while the call before them
// still writes, and the non-coherent loads are only for what nothing writes as long as a kernel lives.
template <typename T>
__device__ __forceinline__ T k8_read(const T* p) {
  return *p;
}

// Scales as the kernels use them: [2^-60, 2^60], NaN as 2^-60 (fmaxf drops it).
__device__ __forceinline__ float k8_scale(float s) { return fminf(fmaxf(s, 0x1p-60f), 0x1p60f); }

// The tokens of sequence b: [t0, t0 + n), its rows L, and the row of its first token.
struct K8Seq {
  int t0, n, L, first;
};
__device__ __forceinline__ int k8_cu(const K8Cache& c, int b) {
  return c.cu ? min(max(k8_read(c.cu + b), 0), c.T) : b * c.s_q;
}
__device__ __forceinline__ int k8_len(const K8Cache& c, int b) {
  return min(max(k8_read(c.lens + b), 0), c.max_pages * c.ps);
}
__device__ __forceinline__ K8Seq k8_seq(const K8Cache& c, int b) {
  K8Seq s;
  s.t0 = k8_cu(c, b);
  s.n = max(k8_cu(c, b + 1) - s.t0, 0);
  s.L = k8_len(c, b);
  s.first = s.L - s.n;
  return s;
}
// Two e4m3 codes (low byte first) -> two halves; exact.
__device__ __forceinline__ uint32_t k8_e4m3x2(uint32_t two) {
  uint32_t r;
  asm("{\n .reg .b16 t;\n cvt.u16.u32 t, %1;\n cvt.rn.f16x2.e4m3x2 %0, t;\n}\n" : "=r"(r) : "r"(two));
  return r;
}
__device__ __forceinline__ float k8_code(uint8_t c, int fmt) {
  if (fmt == kFmtInt8) return (float)(int8_t)c;
  const uint32_t h = k8_e4m3x2(c);
  return __half2float(__ushort_as_half((unsigned short)h));
}
// Two floats -> two codes, rounded to nearest even and saturated.  NaN: the e4m3 NaN, 0 in integers.
__device__ __forceinline__ uint32_t k8_round2(float lo, float hi, int fmt) {
  if (fmt == kFmtInt8) {
    const int a = __float2int_rn(fminf(fmaxf(lo, -127.f), 127.f)), b = __float2int_rn(fminf(fmaxf(hi, -127.f), 127.f));
    return (uint32_t)((lo == lo ? a : 0) & 255) | ((uint32_t)((hi == hi ? b : 0) & 255) << 8);
  }
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;\n" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

}  // namespace sa
