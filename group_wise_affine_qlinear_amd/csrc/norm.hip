// The norm on either side of a projection, fused with its AdaLN modulation,
// its gate and the scaled residual update (qlinear_block_norm).
//
//   z = N_post(y) * w_post + b_post
//   r = residual_scale * residual + gate[s] * z            -> residual_out
//   h = (N_pre(r) * w_pre + b_pre) * (1 + scale[s]) + shift[s]  -> h (bf16), x16 + rowscale (FAST activations)
//
// s is the row's sample; N is the identity, v / sqrt(mean v^2 + eps) or
// (v - mean) / sqrt(mean (v - mean)^2 + eps).
//
// A row is held in registers by W waves, C chunks of 8 values per lane, so
// every input is read once and every output written once: the kernel is bound
// by those bytes. Everything is fp32; each output is rounded once, and h is
// made from the unrounded r.
#include "ql_block.h"
#include "ql_kernels.h"

namespace ql {

namespace {

struct None {};

// a (op) a's partner lane, over the 64 lanes; every lane gets the result.
// Butterfly order: the same tree for every row, independent of its position.
template <typename Op>
__device__ __forceinline__ float wave_all(float v, Op op) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = op(v, __shfl_xor(v, o));
  return v;
}

struct Sum {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct Max {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};

// Reduction over the W waves of a row. Each call uses the next of four LDS
// lines in turn: two calls that share a line have three barriers between
// them, so no wave still reads what another overwrites. W == 1 needs neither
// LDS nor a barrier (a block then holds several rows).
template <typename Op>
__device__ __forceinline__ float row_all(float v, int W, float (*lds)[16], int &turn, Op op) {
  v = wave_all(v, op);
  if (W == 1) return v;
  float *line = lds[turn & 3];
  ++turn;
  if ((threadIdx.x & 63) == 0) line[threadIdx.x >> 6] = v;
  __syncthreads();
  float t = line[0];
  for (int w = 1; w < W; ++w) t = op(t, line[w]);
  return t;
}

// Row exponent of the FAST activations, as qlinear_fast_activations defines it.
__device__ __forceinline__ int fast_exponent(float mx) {
  if (!(mx > 0.f)) return 0;
  const int ex = ilogbf(mx);
  return ex > 134 ? 120 : min(max(ex - 14, -126), 120);
}

// Element index of value e of a lane's chunk j: 8 consecutive values per lane
// (VEC), or every row-width-th value (rows of any length and alignment).
template <bool VEC>
__device__ __forceinline__ int at(int j, int e, int lane, int lanes) {
  return VEC ? (j * lanes + lane) * 8 + e : (j * 8 + e) * lanes + lane;
}

template <typename T, int C, bool VEC>
__device__ __forceinline__ void load_row(const void *p, int64_t base, int D, int lane, int lanes, float (&v)[C][8]) {
#pragma unroll
  for (int j = 0; j < C; ++j) {
    if constexpr (VEC) {
      const int i = at<true>(j, 0, lane, lanes);
      if (i < D) {
        T::load8(p, base + i, v[j]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[j][e] = 0.f;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = at<false>(j, e, lane, lanes);
        v[j][e] = i < D ? T::load(p, base + i) : 0.f;
      }
    }
  }
}

template <typename T, int C, bool VEC>
__device__ __forceinline__ void store_row(void *p, int64_t base, int D, int lane, int lanes, const float (&v)[C][8]) {
#pragma unroll
  for (int j = 0; j < C; ++j) {
    if constexpr (VEC) {
      const int i = at<true>(j, 0, lane, lanes);
      if (i < D) T::store8(p, base + i, v[j]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = at<false>(j, e, lane, lanes);
        if (i < D) T::store(p, base + i, v[j][e]);
      }
    }
  }
}

// f(value, parameter) over the row for an fp32 parameter vector p (skipped when null).
template <int C, bool VEC, typename F>
__device__ __forceinline__ void with_vector(const float *p, int D, int lane, int lanes, float (&v)[C][8], F f) {
  if (!p) return;
#pragma unroll
  for (int j = 0; j < C; ++j) {
    float w[8];
    if constexpr (VEC) {
      const int i = at<true>(j, 0, lane, lanes);
      if (i >= D) continue;
      F32::load8(p, i, w);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int i = at<false>(j, e, lane, lanes);
        w[e] = i < D ? p[i] : 0.f;
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[j][e] = f(v[j][e], w[e]);
  }
}

// v <- N(v) over the D values of a row. Values past D are zero on entry and
// are not counted; they hold no meaning afterwards. The mean is taken first
// and the squares of the centred values second (both from registers), so a
// large mean cancels nothing. Where the sums leave fp32 although every value
// is finite, they are taken again of the values times the power of two that
// brings the largest into [1, 4).
template <int C, bool VEC>
__device__ __forceinline__ void normalise(int kind, float eps, int D, int lane, int lanes, int W, float (*lds)[16],
                                          int &turn, float (&v)[C][8]) {
  if (kind == 0) return;
  const float inv_d = 1.0f / (float)D;
  float unit = 1.0f, mean, rstd;
  for (int pass = 0;; ++pass) {
    mean = 0.f;
    if (kind == 2) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < C; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) s += v[j][e] * unit;
      mean = row_all(s, W, lds, turn, Sum{}) * inv_d;
    }
    float q = 0.f;
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float c = at<VEC>(j, e, lane, lanes) < D ? v[j][e] * unit - mean : 0.f;
        q = __builtin_fmaf(c, c, q);
      }
    const float var = row_all(q, W, lds, turn, Sum{}) * inv_d;
    // the scaled eps may underflow; in the scaled pass a variance that is not
    // zero is far above 2^-126, so a row of equal values still gives zeros
    rstd = rsqrtf(var + fmaxf(eps * unit * unit, 0x1p-126f));
    if (pass == 1 || __builtin_isfinite(var)) break;
    float mx = 0.f;
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(v[j][e]));
    mx = row_all(mx, W, lds, turn, Max{});
    if (!(mx < __builtin_inff())) break;  // an infinity or a NaN among the values: the formula's own result
    unit = __uint_as_float((uint32_t)max(254 - (int)(__float_as_uint(mx) >> 23), 1) << 23);
  }
#pragma unroll
  for (int j = 0; j < C; ++j)
#pragma unroll
    for (int e = 0; e < 8; ++e) v[j][e] = (v[j][e] * unit - mean) * rstd;
}

template <typename YT, typename RT, int C, bool VEC>
__global__ __launch_bounds__(1024) void block_norm_kernel(BlockNormArgs a, int W) {
  constexpr bool AFTER = !__is_same(YT, None);
  __shared__ float lds[4][16];
  int turn = 0;
  const int D = a.D;
  const int lanes = 64 * W;
  const int in_block = W == 1 ? (int)(threadIdx.x >> 6) : 0;  // row of this wave in the block
  const int lane = W == 1 ? (int)(threadIdx.x & 63) : (int)threadIdx.x;
  const int64_t m = W == 1 ? (int64_t)blockIdx.x * (blockDim.x >> 6) + in_block : (int64_t)blockIdx.x;
  if (m >= a.M) return;  // whole rows only: W == 1 has no barrier, W > 1 one row per block
  int64_t s = 0;
  if (a.row_sample) {
    s = a.row_sample[m];
    if (s < 0 || s >= a.samples) return;  // behind the last sample: left as it is
  } else if (a.mod_rows) {
    s = (int64_t)((uint64_t)m / (uint64_t)a.mod_rows);
  }
  const int64_t base = m * D;
  float v[C][8], r[C][8];
  if constexpr (AFTER) load_row<YT, C, VEC>(a.y, base, D, lane, lanes, v);
  // both rows in flight at once; at the widest rows y is finished first, for
  // two rows and their loads do not fit the 128 registers of a 16-wave block
  if constexpr (!AFTER || C < 8) load_row<RT, C, VEC>(a.residual, base, D, lane, lanes, r);
  if constexpr (AFTER) {
    normalise<C, VEC>(a.post_norm, a.post_eps, D, lane, lanes, W, lds, turn, v);
    with_vector<C, VEC>(a.post_weight, D, lane, lanes, v, [](float x, float w) { return x * w; });
    with_vector<C, VEC>(a.post_bias, D, lane, lanes, v, [](float x, float w) { return x + w; });
    if (a.gate) {
      with_vector<C, VEC>(a.gate + s * a.gate_ld, D, lane, lanes, v, [](float x, float w) { return x * w; });
    }
    if constexpr (C >= 8) load_row<RT, C, VEC>(a.residual, base, D, lane, lanes, r);
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) r[j][e] = __builtin_fmaf(a.residual_scale, r[j][e], v[j][e]);
    if (a.residual_out) store_row<RT, C, VEC>(a.residual_out, base, D, lane, lanes, r);
    if (!a.h && !a.x16) return;
    // what lies past the row must not count in the next sums
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (at<VEC>(j, e, lane, lanes) >= D) r[j][e] = 0.f;
  } else if (a.residual_scale != 1.0f) {
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) r[j][e] *= a.residual_scale;
  }
  normalise<C, VEC>(a.pre_norm, a.pre_eps, D, lane, lanes, W, lds, turn, r);
  with_vector<C, VEC>(a.pre_weight, D, lane, lanes, r, [](float x, float w) { return x * w; });
  with_vector<C, VEC>(a.pre_bias, D, lane, lanes, r, [](float x, float w) { return x + w; });
  if (a.scale)
    with_vector<C, VEC>(a.scale + s * a.scale_ld, D, lane, lanes, r, [](float x, float w) { return x * (1.0f + w); });
  if (a.shift)
    with_vector<C, VEC>(a.shift + s * a.shift_ld, D, lane, lanes, r, [](float x, float w) { return x + w; });
  if (a.h) store_row<BF16, C, VEC>(a.h, base, D, lane, lanes, r);
  if (a.x16) {
    float mx = 0.f;
#pragma unroll
    for (int j = 0; j < C; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (at<VEC>(j, e, lane, lanes) < D) mx = fmaxf(mx, fabsf(r[j][e]));
    const int ex = fast_exponent(row_all(mx, W, lds, turn, Max{}));
    const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
    if (lane == 0) a.rowscale[m] = __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
    for (int j = 0; j < C; ++j) {
      if constexpr (VEC) {
        const int i = at<true>(j, 0, lane, lanes);
        if (i >= D) continue;
        u32x4 o;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const _Float16 lo = (_Float16)(r[j][2 * e] * down), hi = (_Float16)(r[j][2 * e + 1] * down);
          o[e] = (uint32_t)__builtin_bit_cast(uint16_t, lo) | ((uint32_t)__builtin_bit_cast(uint16_t, hi) << 16);
        }
        *reinterpret_cast<u32x4 *>(a.x16 + base + i) = o;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int i = at<false>(j, e, lane, lanes);
          if (i < D) a.x16[base + i] = __builtin_bit_cast(uint16_t, (_Float16)(r[j][e] * down));
        }
      }
    }
  }
}

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <typename YT, typename RT, int C>
void launch_c(const BlockNormArgs &a, int W, bool vec, hipStream_t stream) {
  const int rows = W == 1 ? 4 : 1;
  const dim3 grid((unsigned)((a.M + rows - 1) / rows)), block(64 * W * rows);
  if (vec) hipLaunchKernelGGL((block_norm_kernel<YT, RT, C, true>), grid, block, 0, stream, a, W);
  else hipLaunchKernelGGL((block_norm_kernel<YT, RT, C, false>), grid, block, 0, stream, a, W);
}

template <typename YT, typename RT>
void launch_types(const BlockNormArgs &a, hipStream_t stream) {
  // 16-byte accesses where every row of every array starts on 16 bytes
  bool vec = a.D % 8 == 0;
  for (const void *p : {(const void *)a.residual, a.y, (const void *)a.residual_out, (const void *)a.h, (const void *)a.x16,
                        (const void *)a.post_weight, (const void *)a.post_bias, (const void *)a.pre_weight,
                        (const void *)a.pre_bias, (const void *)a.gate, (const void *)a.scale, (const void *)a.shift})
    vec = vec && aligned(p, 16);
  vec = vec && a.gate_ld % 4 == 0 && a.scale_ld % 4 == 0 && a.shift_ld % 4 == 0;
  const int chunks = (a.D + 7) / 8;
  // fewest chunks per lane that leave at most 16 waves to a row
  int c = 1;
  while ((chunks + 64 * c - 1) / (64 * c) > 16) c *= 2;
  const int W = (chunks + 64 * c - 1) / (64 * c);
  if (c == 1) launch_c<YT, RT, 1>(a, W, vec, stream);
  else if (c == 2) launch_c<YT, RT, 2>(a, W, vec, stream);
  else if (c == 4) launch_c<YT, RT, 4>(a, W, vec, stream);
  else launch_c<YT, RT, 8>(a, W, vec, stream);
}

}  // namespace

hipError_t launch_block_norm(const BlockNormArgs &a, hipStream_t stream) {
  if (!a.y) {
    if (a.residual_bf16) launch_types<None, BF16>(a, stream);
    else launch_types<None, F32>(a, stream);
  } else if (a.y_bf16) {
    if (a.residual_bf16) launch_types<BF16, BF16>(a, stream);
    else launch_types<BF16, F32>(a, stream);
  } else {
    if (a.residual_bf16) launch_types<F32, BF16>(a, stream);
    else launch_types<F32, F32>(a, stream);
  }
  return hipGetLastError();
}

}  // namespace ql
