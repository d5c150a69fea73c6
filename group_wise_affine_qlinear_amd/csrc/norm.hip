// The norm on either side of a projection, fused with its AdaLN modulation,
// its gate and the scaled residual update (qlinear_block_norm).
//
//   z = N_post(y) * w_post + b_post
//   r = residual_scale * residual + gate[s] * z                 -> residual_out
//   h = (N_pre(r) * w_pre + b_pre) * (1 + scale[s]) + shift[s]  -> h (bf16), x16 + rowscale (FAST activations)
//
// s is the row's sample; N is the identity, v / sqrt(mean v^2 + eps) or
// (v - mean) / sqrt(mean (v - mean)^2 + eps).
//
// A row is held in registers by W waves, C chunks of 8 values per lane, so
// every input is read once and every output written once: the kernel is bound
// by those bytes. Not so for rows by elements (of a length or alignment that
// 16-byte accesses cannot serve) above 16384 values: four and eight chunks of a
// lane do not fit its 128 registers there, since a bf16 value takes one of its
// own, and up to 200 of them go through scratch memory (512 bf16 rows of 53247
// before a block 62 us, of 53248 23; between two 235 and 68; 1000 rows of 20001
// between two 122, of 20000 51). Everything is fp32; each output is rounded
// once, and h is made from the unrounded r.
#include <algorithm>

#include "ql_block.h"
#include "ql_kernels.h"

namespace ql {

namespace {

struct None {};

// op over the 64 lanes by DPP moves in a fixed order (pairs, quads, half rows
// and rows of 16, then rows 0-1 and 2-3, then both halves), in every lane. A
// lane that a move leaves out takes `op(v, 0)`: the sum, and the maximum of
// magnitudes.
template <int CTRL, int ROWS, typename Op>
__device__ __forceinline__ float dpp(float v, Op op) {
  const int o = __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, ROWS, 0xF, false);
  return op(v, __builtin_bit_cast(float, o));
}
template <typename Op>
__device__ __forceinline__ float row16_all(float v, Op op) {
  v = dpp<0xB1, 0xF>(v, op);   // quad_perm [1, 0, 3, 2]
  v = dpp<0x4E, 0xF>(v, op);   // quad_perm [2, 3, 0, 1]
  v = dpp<0x141, 0xF>(v, op);  // row_half_mirror
  return dpp<0x140, 0xF>(v, op);  // row_mirror
}
template <typename Op>
__device__ __forceinline__ float wave_all(float v, Op op) {
  v = row16_all(v, op);
  v = dpp<0x142, 0xA>(v, op);  // row_bcast:15 into rows 1 and 3
  v = dpp<0x143, 0xC>(v, op);  // row_bcast:31 into rows 2 and 3
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(v), 63));
}

struct Sum {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
struct Max {  // of magnitudes
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
};

// The place of a lane in its row, and the LDS lines of the row's reductions.
struct Place {
  int lane, lanes, W;
  float (*lds)[16];
  int turn;
};

// Reduction over the W waves of a row, the same tree for every row. Each call
// uses the next of four LDS lines in turn: two calls that share a line have
// three barriers between them, so no wave still reads what another overwrites.
// W == 1 needs neither LDS nor a barrier (a block then holds several rows).
template <typename Op>
__device__ __forceinline__ float row_all(float v, Place &p, Op op) {
  v = wave_all(v, op);
  if (p.W == 1) return v;
  float *line = p.lds[p.turn & 3];
  ++p.turn;
  if ((threadIdx.x & 63) == 0) line[threadIdx.x >> 6] = v;
  __syncthreads();
  const int w = threadIdx.x & 15;
  return row16_all(w < p.W ? line[w] : 0.f, op);
}

// Row exponent of the FAST activations, as qlinear_fast_activations defines it.
__device__ __forceinline__ int fast_exponent(float mx) {
  if (!(mx > 0.f)) return 0;
  const int ex = ilogbf(mx);
  return ex > 134 ? 120 : min(max(ex - 14, -126), 120);
}

// Element index of value e of a lane's chunk j: 8 consecutive values per lane
// (VEC: rows whose 16-byte pieces start on words), or every row-width-th value
// (rows of any length and alignment).
template <bool VEC>
__device__ __forceinline__ int at(const Place &p, int j, int e) {
  return VEC ? (j * p.lanes + p.lane) * 8 + e : (j * 8 + e) * p.lanes + p.lane;
}

// One row of a stream or one fp32 vector as a buffer of its D values: reads
// past it give zero and writes past it are dropped, so no access needs a
// compare or a 64-bit address of its own.
typedef __amdgpu_buffer_rsrc_t Row;
template <typename T>
__device__ __forceinline__ Row row_of(const void *p, int64_t first, int D) {
  constexpr int size = __is_same(T, F32) ? 4 : 2;
  return make_rsrc(p, first * size, (int64_t)D * size);
}

__device__ __forceinline__ u32x4 load16(Row r, int byte) {
  return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, byte, 0, 0));
}

// A chunk as it is loaded: bf16 values stay packed until they are used.
template <typename T, bool VEC> struct Raw { u32x4 v[VEC && __is_same(T, BF16) ? 1 : 2]; };
template <bool VEC> struct Raw<None, VEC> {};

template <typename T, bool VEC>
__device__ __forceinline__ void fetch(Row row, const Place &pl, int j, Raw<T, VEC> &raw) {
  if constexpr (VEC) {
    const int i = at<true>(pl, j, 0);
    if constexpr (__is_same(T, BF16)) {
      raw.v[0] = load16(row, i * 2);
    } else {
      raw.v[0] = load16(row, i * 4);
      raw.v[1] = load16(row, i * 4 + 16);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = at<false>(pl, j, e);
      if constexpr (__is_same(T, BF16))
        raw.v[e / 4][e % 4] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(row, i * 2, 0, 0) << 16;
      else
        raw.v[e / 4][e % 4] = __builtin_amdgcn_raw_buffer_load_b32(row, i * 4, 0, 0);
    }
  }
}

template <typename T, bool VEC>
__device__ __forceinline__ void unpack(const Raw<T, VEC> &raw, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (VEC && __is_same(T, BF16)) v[e] = e % 2 ? bf16_hi(raw.v[0][e / 2]) : bf16_lo(raw.v[0][e / 2]);
    else v[e] = __uint_as_float(raw.v[e / 4][e % 4]);
  }
}

struct F16 {};  // fp16 bit patterns

__device__ __forceinline__ uint32_t f16_bits(float v) { return __builtin_bit_cast(uint16_t, (_Float16)v); }

template <typename T, bool VEC>
__device__ __forceinline__ void store(Row row, const Place &pl, int j, const float (&v)[8]) {
  if constexpr (VEC) {
    const int i = at<true>(pl, j, 0);
    if constexpr (__is_same(T, F32)) {
      const f32x4 a = {v[0], v[1], v[2], v[3]}, b = {v[4], v[5], v[6], v[7]};
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, a), row, i * 4, 0, 0);
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, b), row, i * 4 + 16, 0, 0);
    } else {
      u32x4 o;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        o[e] = __is_same(T, F16) ? f16_bits(v[2 * e]) | f16_bits(v[2 * e + 1]) << 16 : pack_bf16(v[2 * e], v[2 * e + 1]);
      __builtin_amdgcn_raw_buffer_store_b128(o, row, i * 2, 0, 0);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = at<false>(pl, j, e);
      if constexpr (__is_same(T, F32))
        __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v[e]), row, i * 4, 0, 0);
      else
        __builtin_amdgcn_raw_buffer_store_b16(__is_same(T, F16) ? (uint16_t)f16_bits(v[e]) : bf16_bits(v[e]), row,
                                              i * 2, 0, 0);
    }
  }
}

// Chunk j of an fp32 vector, `other` in every place where there is no vector.
template <bool VEC>
__device__ __forceinline__ void vector8(const float *p, int64_t first, int D, const Place &pl, int j, float other,
                                        float (&w)[8]) {
  if (p) {
    Raw<F32, VEC> raw;
    fetch<F32, VEC>(row_of<F32>(p, first, D), pl, j, raw);
    unpack<F32, VEC>(raw, w);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = other;
  }
}

// A norm's affine step and what follows it, v * mul + add, for chunk j:
// after a block mul = weight * gate, add = bias * gate; before one
// mul = weight * (1 + scale), add = bias * (1 + scale) + shift.
template <bool AFTER, bool VEC, bool ADD>
__device__ __forceinline__ void factors(const BlockNormArgs &a, int64_t s, const Place &pl, int j, float (&mul)[8],
                                        float (&add)[8]) {
  float w[8], t[8];
  vector8<VEC>(AFTER ? a.post_weight : a.pre_weight, 0, a.D, pl, j, 1.f, w);
  vector8<VEC>(AFTER ? a.gate : a.scale, s * (AFTER ? a.gate_ld : a.scale_ld), a.D, pl, j, AFTER ? 1.f : 0.f, t);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if constexpr (!AFTER) t[e] = 1.f + t[e];
    mul[e] = w[e] * t[e];
  }
  if constexpr (ADD) {
    float b[8], sh[8];
    vector8<VEC>(AFTER ? a.post_bias : a.pre_bias, 0, a.D, pl, j, 0.f, b);
    if constexpr (!AFTER) vector8<VEC>(a.shift, s * a.shift_ld, a.D, pl, j, 0.f, sh);
#pragma unroll
    for (int e = 0; e < 8; ++e) add[e] = AFTER ? b[e] * t[e] : __builtin_fmaf(b[e], t[e], sh[e]);
  }
}

// What N does to a row: v -> (v * unit - mean) * rstd.
struct Stats {
  float unit, mean, rstd;
};

// The statistics of N over the D values of a row; get(j, v) gives chunk j,
// zeros past D. The mean is taken first and the squares of the centred values
// second (both from registers), so a large mean cancels nothing. Where the
// sums leave fp32 although every value is finite, they are taken again of the
// values times the power of two that brings the largest into [1, 4).
template <int C, bool VEC, typename Get>
__device__ __forceinline__ Stats statistics(int kind, float eps, int D, Place &pl, Get get) {
  Stats t = {1.f, 0.f, 1.f};
  if (kind == 0) return t;
  const float inv_d = 1.0f / (float)D;
  for (int pass = 0;; ++pass) {
    if (kind == 2) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < C; ++j) {
        float v[8];
        get(j, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) s = __builtin_fmaf(v[e], t.unit, s);
      }
      t.mean = row_all(s, pl, Sum{}) * inv_d;
    }
    float q = 0.f;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      float v[8];
      get(j, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float c = __builtin_fmaf(v[e], t.unit, -t.mean);
        // without a mean the zeros past the row stay zeros
        if (kind == 2 && at<VEC>(pl, j, VEC ? 0 : e) >= D) c = 0.f;
        q = __builtin_fmaf(c, c, q);
      }
    }
    const float var = row_all(q, pl, Sum{}) * inv_d;
    // the scaled eps may underflow; in the scaled pass a variance that is not
    // zero is far above 2^-126, so a row of equal values still gives zeros
    t.rstd = rsqrtf(var + fmaxf(eps * t.unit * t.unit, 0x1p-126f));
    if (pass == 1 || __builtin_isfinite(var)) break;
    float mx = 0.f;
#pragma unroll
    for (int j = 0; j < C; ++j) {
      float v[8];
      get(j, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(v[e]));
    }
    mx = row_all(mx, pl, Max{});
    if (!(mx < __builtin_inff())) break;  // an infinity or a NaN among the values: the formula's own result
    t.unit = __uint_as_float((uint32_t)max(254 - (int)(__float_as_uint(mx) >> 23), 1) << 23);
  }
  return t;
}

__device__ __forceinline__ float apply(const Stats &t, float v) { return __builtin_fmaf(v, t.unit, -t.mean) * t.rstd; }

constexpr int kMostWaves = 16;
constexpr int kCus = 256;  // MI355X

// What a call writes: the updated stream alone, or (with or without it) h, or
// x16 with or without h.
enum class Out { kStream, kH, kX16 };

template <bool B> struct Bool { static constexpr bool value = B; };

// The stream whose norm comes first: y, or the residual where there is no y.
template <typename YT, typename RT> struct First { typedef YT type; };
template <typename RT> struct First<None, RT> { typedef RT type; };

// rows: consecutive rows per block (per wave when W == 1). With one chunk per
// lane (HOLD) the factors of a sample stay in registers from row to row, and
// the next row is in flight while this one is worked on: read again for every
// row, the fp32 factors are up to four times the bytes of a bf16 row itself
// (through L2). Wider rows have no registers for that: there a block has one
// row, its values stay as they were loaded (bf16 packed) until they change,
// and the factors, and the residual after the norm of y, are read by chunks.
template <typename YT, typename RT, Out OUT, int C, bool VEC, bool ADD>
__global__ __launch_bounds__(64 * kMostWaves) void block_norm_kernel(BlockNormArgs a, int W, int rows) {
  constexpr bool AFTER = !__is_same(YT, None);
  constexpr bool HOLD = C == 1;
  constexpr bool PRE = OUT != Out::kStream, X16 = OUT == Out::kX16;
  // x16 needs the row's largest value before its first: its rows are kept unpacked
  constexpr bool KEEP = HOLD || AFTER || X16;
  using T = typename First<YT, RT>::type;
  __shared__ float lds[4][16];
  Place pl;
  pl.W = W;
  pl.lanes = 64 * W;
  pl.lds = lds;
  pl.turn = 0;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  pl.lane = W == 1 ? (int)(threadIdx.x & 63) : (int)threadIdx.x;
  const int D = a.D;
  // W == 1: no barriers, every wave on rows of its own
  int64_t m = ((int64_t)blockIdx.x * (W == 1 ? blockDim.x >> 6 : 1) + (W == 1 ? wave : 0)) * rows;
  const int64_t end = min(a.M, m + rows);
  // the sample of row i, or -1 for a row that is left as it is
  auto sample = [&](int64_t i) -> int64_t {
    if (i >= end) return -1;
    if (a.row_sample) {
      const int64_t s = a.row_sample[i];
      return s < a.samples ? s : -1;
    }
    return a.mod_rows ? (int64_t)((uint64_t)i / (uint64_t)a.mod_rows) : 0;
  };
  const void *const first = AFTER ? a.y : a.residual;
  Raw<T, VEC> x[C];   // the row whose norm comes first
  Raw<RT, VEC> res;   // the residual of an update
  float pm[8], pa[8], qm[8], qa[8];
  auto fetch_row = [&](int64_t i) {
#pragma unroll
    for (int j = 0; j < C; ++j) fetch<T, VEC>(row_of<T>(first, i * D, D), pl, j, x[j]);
    if constexpr (AFTER && HOLD) fetch<RT, VEC>(row_of<RT>(a.residual, i * D, D), pl, 0, res);
  };
  int64_t s = sample(m), held = -1;
  if (!HOLD && s < 0) return;
  if (!HOLD || s >= 0) fetch_row(m);
  do {
    const int64_t next = HOLD ? sample(m + 1) : -1;
    if (HOLD && s < 0) {
      s = next;
      if (s >= 0) fetch_row(m + 1);
      continue;
    }
    const int64_t base = m * D;
    if (HOLD && s != held) {  // the row's own loads are in flight before these
      held = s;
      if constexpr (AFTER) factors<true, VEC, ADD>(a, s, pl, 0, pm, pa);
      if constexpr (PRE) factors<false, VEC, ADD>(a, s, pl, 0, qm, qa);
    }
    float v[C][8], r[8];
    auto values = [&](int j, float (&f)[8]) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = v[j][e];
    };
    auto loaded = [&](int j, float (&f)[8]) {
      if constexpr (!HOLD && VEC && __is_same(T, BF16)) {
        // unpacked anew at each use, or 8 registers would stay taken by every 4
#pragma unroll
        for (auto &w : x[j].v) asm("" : "+v"(w));
      }
      unpack<T, VEC>(x[j], f);
      if constexpr (!AFTER) {
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] *= a.residual_scale;
      }
    };
    if constexpr (HOLD) {
      loaded(0, v[0]);
      if constexpr (AFTER) unpack<RT, VEC>(res, r);
      if (next >= 0) fetch_row(m + 1);
    }
    if constexpr (!HOLD && !AFTER && X16) {
#pragma unroll
      for (int j = 0; j < C; ++j) loaded(j, v[j]);
    }
    // One norm's statistics: of the values as loaded, or as kept in v.
    auto stats = [&](int kind, float eps, auto kept) {
      if constexpr (decltype(kept)::value) return statistics<C, VEC>(kind, eps, D, pl, values);
      else return statistics<C, VEC>(kind, eps, D, pl, loaded);
    };
    if constexpr (AFTER) {
      // v: the updated stream
      const Stats t = stats(a.post_norm, a.post_eps, Bool<HOLD>{});
#pragma unroll
      for (int j = 0; j < C; ++j) {
        if constexpr (!HOLD) {
          fetch<RT, VEC>(row_of<RT>(a.residual, base, D), pl, j, res);
          factors<true, VEC, ADD>(a, s, pl, j, pm, pa);
          unpack<RT, VEC>(res, r);
          loaded(j, v[j]);
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float z = apply(t, v[j][e]) * pm[e];
          const float u = __builtin_fmaf(a.residual_scale, r[e], ADD ? z + pa[e] : z);
          // what lies past the row must not count in the next sums
          v[j][e] = at<VEC>(pl, j, VEC ? 0 : e) < D ? u : 0.f;
        }
        if (a.residual_out) store<RT, VEC>(row_of<RT>(a.residual_out, base, D), pl, j, v[j]);
        // left alone, the loads of all chunks come first and the row spills
        if constexpr (!HOLD) __builtin_amdgcn_sched_barrier(0);
      }
    }
    if constexpr (PRE) {
      const Stats t = stats(a.pre_norm, a.pre_eps, Bool<KEEP>{});
      float mx = 0.f;
#pragma unroll
      for (int j = 0; j < C; ++j) {
        if constexpr (!HOLD) factors<false, VEC, ADD>(a, s, pl, j, qm, qa);
        float o[8];
        if constexpr (KEEP) values(j, o);
        else loaded(j, o);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float n = apply(t, o[e]);
          o[e] = ADD ? __builtin_fmaf(n, qm[e], qa[e]) : n * qm[e];
          if constexpr (X16) {
            v[j][e] = o[e];
            if (at<VEC>(pl, j, VEC ? 0 : e) < D) mx = fmaxf(mx, fabsf(o[e]));
          }
        }
        if (!X16 || a.h) store<BF16, VEC>(row_of<BF16>(a.h, base, D), pl, j, o);
        if constexpr (!HOLD) __builtin_amdgcn_sched_barrier(0);
      }
      if constexpr (X16) {
        const int ex = fast_exponent(row_all(mx, pl, Max{}));
        const float down = __uint_as_float((uint32_t)(127 - ex) << 23);
        if (pl.lane == 0) a.rowscale[m] = __uint_as_float((uint32_t)(127 + ex) << 23);
#pragma unroll
        for (int j = 0; j < C; ++j) {
#pragma unroll
          for (int e = 0; e < 8; ++e) v[j][e] *= down;
          store<F16, VEC>(row_of<F16>(a.x16, base, D), pl, j, v[j]);
        }
      }
    }
    s = next;
  } while (HOLD && ++m < end);
}

bool aligned(const void *p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

template <typename YT, typename RT, Out OUT, int C>
void launch_c(const BlockNormArgs &a, bool vec, bool add, hipStream_t stream) {
  const int chunks = (a.D + 7) / 8;
  const int W = (chunks + 64 * C - 1) / (64 * C);
  const int per_block = W == 1 ? 4 : 1;
  // Rows of a block that holds its factors: as many as leave every CU about
  // `waves` waves, since each block loads the factors once. Measured for RMS
  // over bf16 rows of 4608 (9 waves): before a block 16.2 us at 20 waves per
  // CU, 15.5 at 32, 20.5 at 16 and 21 at a block per row (4096 rows); between
  // two blocks 128 us at 16 waves, 132 at 36, 229 at a block per row (16896).
  constexpr int waves = __is_same(YT, None) ? 32 : OUT == Out::kStream ? 20 : 16;
  const int64_t slots = (int64_t)kCus * std::max(1, waves / (W * per_block));
  const int rows = C == 1 ? (int)std::max<int64_t>(1, (a.M + slots * per_block - 1) / (slots * per_block)) : 1;
  const int64_t units = (a.M + rows - 1) / rows;
  const dim3 grid((unsigned)((units + per_block - 1) / per_block)), block(64 * W * per_block);
  if (vec && !add) hipLaunchKernelGGL((block_norm_kernel<YT, RT, OUT, C, true, false>), grid, block, 0, stream, a, W, rows);
  else if (vec) hipLaunchKernelGGL((block_norm_kernel<YT, RT, OUT, C, true, true>), grid, block, 0, stream, a, W, rows);
  if constexpr (C > 1) {
    if (!vec) hipLaunchKernelGGL((block_norm_kernel<YT, RT, OUT, C, false, true>), grid, block, 0, stream, a, W, rows);
  }
}

template <typename YT, typename RT, Out OUT>
void launch_types(const BlockNormArgs &a, hipStream_t stream) {
  // 16-byte accesses where every row of every array starts on 16 bytes
  bool vec = a.D % 8 == 0;
  for (const void *p : {(const void *)a.residual, a.y, (const void *)a.residual_out, (const void *)a.h, (const void *)a.x16,
                        (const void *)a.post_weight, (const void *)a.post_bias, (const void *)a.pre_weight,
                        (const void *)a.pre_bias, (const void *)a.gate, (const void *)a.scale, (const void *)a.shift})
    vec = vec && aligned(p, 16);
  vec = vec && a.gate_ld % 4 == 0 && a.scale_ld % 4 == 0 && a.shift_ld % 4 == 0;
  const bool add = a.post_bias || a.pre_bias || a.shift;
  const int chunks = (a.D + 7) / 8;
  // Element-wise rows start at two chunks per lane: with one, the factors of
  // every held row cost eight loads each (4096 bf16 rows of 4607 before a
  // block: 19 us at two, 26 at one; 1001 rows of 1003 between: 5.8 and 8.7).
  int c = vec ? 1 : 2;
  while ((chunks + 64 * c - 1) / (64 * c) > kMostWaves) c *= 2;
  if (c == 1) launch_c<YT, RT, OUT, 1>(a, vec, add, stream);
  else if (c == 2) launch_c<YT, RT, OUT, 2>(a, vec, add, stream);
  else if (c == 4) launch_c<YT, RT, OUT, 4>(a, vec, add, stream);
  else launch_c<YT, RT, OUT, 8>(a, vec, add, stream);
}

template <typename YT, typename RT>
void launch_parts(const BlockNormArgs &a, hipStream_t stream) {
  if (a.x16) launch_types<YT, RT, Out::kX16>(a, stream);
  else if (a.h) launch_types<YT, RT, Out::kH>(a, stream);
  else if constexpr (!__is_same(YT, None)) launch_types<YT, RT, Out::kStream>(a, stream);
}

}  // namespace

hipError_t launch_block_norm(const BlockNormArgs &a, hipStream_t stream) {
  if (!a.y) {
    if (a.residual_bf16) launch_parts<None, BF16>(a, stream);
    else launch_parts<None, F32>(a, stream);
  } else if (a.y_bf16) {
    if (a.residual_bf16) launch_parts<BF16, BF16>(a, stream);
    else launch_parts<BF16, F32>(a, stream);
  } else {
    if (a.residual_bf16) launch_parts<F32, BF16>(a, stream);
    else launch_parts<F32, F32>(a, stream);
  }
  return hipGetLastError();
}

}  // namespace ql
