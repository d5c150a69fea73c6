// Device helpers shared by the operators around a projection (norm.hip,
// adapters.hip): fp32 / bf16 element access and rounding.
#pragma once

#include "ql_device.h"

namespace ql {

// fp32 -> bf16, round to nearest even (v_cvt_pk_bf16_f32; NaN stays NaN).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const bf16x2 v = {(__bf16)lo, (__bf16)hi};
  return __builtin_bit_cast(uint32_t, v);
}
__device__ __forceinline__ uint16_t bf16_bits(float v) { return __builtin_bit_cast(uint16_t, (__bf16)v); }

// Element types of a stream of values: fp32 or bf16 bit patterns.
struct F32 {
  typedef float type;
  static __device__ __forceinline__ float load(const void *p, int64_t i) { return static_cast<const float *>(p)[i]; }
  static __device__ __forceinline__ void store(void *p, int64_t i, float v) { static_cast<float *>(p)[i] = v; }
  static __device__ __forceinline__ void load4(const void *p, int64_t i, float (&f)[4]) {
    const f32x4 v = *reinterpret_cast<const f32x4 *>(static_cast<const float *>(p) + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = v[e];
  }
  static __device__ __forceinline__ void store4(void *p, int64_t i, const float (&f)[4]) {
    *reinterpret_cast<f32x4 *>(static_cast<float *>(p) + i) = f32x4{f[0], f[1], f[2], f[3]};
  }
  static __device__ __forceinline__ void load8(const void *p, int64_t i, float (&f)[8]) {
    const f32x4 *s = reinterpret_cast<const f32x4 *>(static_cast<const float *>(p) + i);
    const f32x4 a = s[0], b = s[1];
#pragma unroll
    for (int e = 0; e < 4; ++e) f[e] = a[e], f[4 + e] = b[e];
  }
  static __device__ __forceinline__ void store8(void *p, int64_t i, const float (&f)[8]) {
    f32x4 *d = reinterpret_cast<f32x4 *>(static_cast<float *>(p) + i);
    d[0] = f32x4{f[0], f[1], f[2], f[3]};
    d[1] = f32x4{f[4], f[5], f[6], f[7]};
  }
};

struct BF16 {
  typedef uint16_t type;
  static __device__ __forceinline__ float load(const void *p, int64_t i) {
    return __uint_as_float((uint32_t)static_cast<const uint16_t *>(p)[i] << 16);
  }
  static __device__ __forceinline__ void store(void *p, int64_t i, float v) {
    static_cast<uint16_t *>(p)[i] = bf16_bits(v);
  }
  static __device__ __forceinline__ void load4(const void *p, int64_t i, float (&f)[4]) {
    const u32x2 v = *reinterpret_cast<const u32x2 *>(static_cast<const uint16_t *>(p) + i);
#pragma unroll
    for (int e = 0; e < 2; ++e) f[2 * e] = bf16_lo(v[e]), f[2 * e + 1] = bf16_hi(v[e]);
  }
  static __device__ __forceinline__ void store4(void *p, int64_t i, const float (&f)[4]) {
    *reinterpret_cast<u32x2 *>(static_cast<uint16_t *>(p) + i) = u32x2{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])};
  }
  static __device__ __forceinline__ void load8(const void *p, int64_t i, float (&f)[8]) {
    const u32x4 v = *reinterpret_cast<const u32x4 *>(static_cast<const uint16_t *>(p) + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[2 * e] = bf16_lo(v[e]), f[2 * e + 1] = bf16_hi(v[e]);
  }
  static __device__ __forceinline__ void store8(void *p, int64_t i, const float (&f)[8]) {
    *reinterpret_cast<u32x4 *>(static_cast<uint16_t *>(p) + i) =
        u32x4{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])};
  }
};

}  // namespace ql
