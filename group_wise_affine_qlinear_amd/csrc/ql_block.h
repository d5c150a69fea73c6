// Device helpers shared by the operators around a projection (norm.hip,
// adapters.hip) and between two (heads.hip, attention.hip): fp32 / bf16 element
// access and rounding, reductions over lanes.
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

// op over a lane and the one that a DPP move gives it. A lane that the move
// leaves out takes `op(v, 0)`: the sum, and the maximum of magnitudes.
template <int CTRL, int ROWS = 0xF, typename Op>
__device__ __forceinline__ float dpp(float v, Op op) {
  const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xF, false);
  return op(v, __builtin_bit_cast(float, o));
}
struct Sum {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct Max {  // of magnitudes
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};

}  // namespace ql
