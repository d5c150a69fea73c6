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
};

struct BF16 {
  typedef uint16_t type;
  static __device__ __forceinline__ float load(const void *p, int64_t i) {
    return __uint_as_float((uint32_t)static_cast<const uint16_t *>(p)[i] << 16);
  }
  static __device__ __forceinline__ void store(void *p, int64_t i, float v) {
    static_cast<uint16_t *>(p)[i] = bf16_bits(v);
  }
};

}  // namespace ql
