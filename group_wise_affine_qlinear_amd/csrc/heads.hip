// From the output of a fused QKV projection to the heads that attention reads
// (qlinear_qk_norm_rope): per query and key head
//
//   u = N(x) * w                               over the D values of the head
//   t_i = positions[axis_i, m] * freqs[i]      one angle per pair and row
//   (a, b) -> (a cos t_i - b sin t_i, b cos t_i + a sin t_i)
//
// with the pairs (u_i, u_{i + P}) or (u_2i, u_{2i+1}), i < P; values are
// rounded only. N is the identity, v / sqrt(mean v^2 + eps) or
// (v - mean) / sqrt(mean (v - mean)^2 + eps).
//
// A head lies on the power of two of lanes that holds 8 values each, so a
// wave works on 64 / lanes heads at once, every value is read once and written
// once and the sums of a norm are DPP moves. The angles depend on the row
// alone: the threads of a block make each cosine and sine of its row once and
// all heads are turned by them from LDS (made per head and lane, 2047 rows of
// 48 heads of 128 took 19 us instead of 12.4).
//
// Bound by its bytes: 16896 rows of 54 heads of 256 (fp32 in, bf16 out, 1.4 GB)
// 261 us, 5.4 TB/s, as a large copy; 4608 rows 75 us, 5.1 TB/s; 2047 text rows
// (50 MB) 12.4 us in a graph, of which 3 are the launch and a row's first loads
// and angles most of the rest. One row takes 3.4 us, the launch.
#include "ql_block.h"
#include "ql_kernels.h"

namespace ql {

namespace {

// Sum (or maximum of magnitudes) over the aligned groups of 2^lg lanes, in a
// fixed order, in every lane of the group.
template <typename Op>
__device__ __forceinline__ float group_all(float v, int lg, Op op) {
  v = dpp<0xB1>(v, op);                // quad_perm [1, 0, 3, 2]
  v = dpp<0x4E>(v, op);                // quad_perm [2, 3, 0, 1]
  if (lg > 2) v = dpp<0x141>(v, op);   // row_half_mirror
  if (lg > 3) v = dpp<0x140>(v, op);   // row_mirror
  if (lg > 4) {
    // lane ^ 16: rows 0 <-> 1 and 2 <-> 3
    const int o = __builtin_amdgcn_ds_swizzle(__builtin_bit_cast(int, v), 0x401F);
    v = op(v, __builtin_bit_cast(float, o));
  }
  return v;
}

// The 8 values of a lane: four at `lo` and four at `hi` of its head.
template <typename T, bool VEC>
struct Piece {
  u32x4 raw[2];  // bf16: two words of each are used

  __device__ __forceinline__ void load(const void *base, int64_t at, int lo, int hi) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t e = at + (i ? hi : lo);
      if constexpr (__is_same(T, F32)) {
        const float *p = static_cast<const float *>(base) + e;
        if constexpr (VEC) raw[i] = *reinterpret_cast<const u32x4 *>(p);
        else raw[i] = u32x4{__float_as_uint(p[0]), __float_as_uint(p[1]), __float_as_uint(p[2]), __float_as_uint(p[3])};
      } else {
        const uint16_t *p = static_cast<const uint16_t *>(base) + e;
        if constexpr (VEC) {
          const u32x2 w = *reinterpret_cast<const u32x2 *>(p);
          raw[i][0] = w[0];
          raw[i][1] = w[1];
        } else {
          raw[i][0] = p[0] | (uint32_t)p[1] << 16;
          raw[i][1] = p[2] | (uint32_t)p[3] << 16;
        }
      }
    }
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if constexpr (__is_same(T, F32)) v[e] = __uint_as_float(raw[e / 4][e % 4]);
      else v[e] = e % 2 ? bf16_hi(raw[e / 4][e % 4 / 2]) : bf16_lo(raw[e / 4][e % 4 / 2]);
    }
  }
};

template <bool VEC>
__device__ __forceinline__ void store(uint16_t *base, int64_t at, int lo, int hi, const float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint16_t *p = base + at + (i ? hi : lo);
    if constexpr (VEC) {
      *reinterpret_cast<u32x2 *>(p) = u32x2{pack_bf16(v[4 * i], v[4 * i + 1]), pack_bf16(v[4 * i + 2], v[4 * i + 3])};
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) p[e] = bf16_bits(v[4 * i + e]);
    }
  }
}

// N over a head. Lanes past the head hold zeros and `live` false. The mean is
// taken first and the squares of the centred values second, so a large mean
// cancels nothing. Where the sums leave fp32 although every value is finite,
// they are taken again of the values times the power of two that brings the
// largest into [1, 4); the other heads of the wave go along with a factor of 1.
__device__ __forceinline__ void normalise(float (&v)[8], int kind, float eps, float inv_d, int lg, bool live) {
  float unit = 1.f;
  for (int pass = 0;; ++pass) {
    float mean = 0.f;
    if (kind == 2) {
      float s = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) s = __builtin_fmaf(v[e], unit, s);
      mean = group_all(s, lg, Sum{}) * inv_d;
    }
    float q = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float c = __builtin_fmaf(v[e], unit, -mean);
      if (!live) c = 0.f;
      q = __builtin_fmaf(c, c, q);
    }
    const float var = group_all(q, lg, Sum{}) * inv_d;
    // the scaled eps may underflow; a variance that is not zero is then far above 2^-126
    const float rstd = rsqrtf(var + fmaxf(eps * unit * unit, 0x1p-126f));
    float mx = 0.f;
    const bool again = pass == 0 && !__builtin_isfinite(var);
    if (__any(again)) {
#pragma unroll
      for (int e = 0; e < 8; ++e) mx = fmaxf(mx, fabsf(v[e]));
      mx = group_all(mx, lg, Max{});
      if (again && mx < __builtin_inff()) unit = __uint_as_float((uint32_t)max(254 - (int)(__float_as_uint(mx) >> 23), 1) << 23);
      continue;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __builtin_fmaf(v[e], unit, -mean) * rstd;
    return;
  }
}

constexpr int kPairs = 128;  // of a head of 256

// Grid: x rows, y ranges of a row's steps; a step is the 64 >> lg heads that a
// wave holds at once, the steps of q first, then k's, then v's.
template <typename T, bool PAIRS, bool VEC>
__global__ __launch_bounds__(256) void qk_norm_rope_kernel(HeadsArgs a) {
  __shared__ __attribute__((aligned(16))) float turn[kPairs][2];  // cosine and sine
  const int64_t m = blockIdx.x;
  if (a.rows_end && m >= *a.rows_end) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lg = a.lane_bits, slot = lane & ((1 << lg) - 1), sub = lane >> lg, per = 64 >> lg;
  const bool live = slot * 8 < a.D;
  const bool turns = slot < a.pairs / 4;  // the slot holds turned pairs
  const int lo = !PAIRS && turns ? slot * 4 : slot * 8;
  const int hi = !PAIRS && turns ? a.pairs + slot * 4 : slot * 8 + 4;

  const int steps_q = (a.part[0].heads + per - 1) / per, steps_k = (a.part[1].heads + per - 1) / per;
  const int steps = steps_q + steps_k + (a.part[2].heads + per - 1) / per;
  const int stride = 4 * gridDim.y;
  // the part and head of step i; whether the lane has a value of it
  auto where = [&](int i, int &p, int64_t &head) {
    p = i < steps_q ? 0 : i < steps_q + steps_k ? 1 : 2;
    head = (int64_t)(i - (p == 0 ? 0 : p == 1 ? steps_q : steps_q + steps_k)) * per + sub;
    return live && i < steps && head < a.part[p].heads;
  };
  int i = blockIdx.y * 4 + wave;
  // two steps are on their way at any time, the first two while the angles are made
  Piece<T, VEC> next[2] = {};
  auto load = [&](int i, Piece<T, VEC> &to) {
    int p;
    int64_t head;
    if (where(i, p, head)) to.load(a.part[p].in, m * a.part[p].in_ld + head * a.D, lo, hi);
  };
  load(i, next[0]);
  load(i + stride, next[1]);
  // weights of q and k
  float w[2][8];
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    if (a.part[p].weight && live) {
      Piece<F32, VEC> weight;
      weight.load(a.part[p].weight, 0, lo, hi);
      weight.values(w[p]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[p][e] = 1.f;
    }
  }

  if (a.pairs > 0) {
    if ((int)threadIdx.x < a.pairs) {
      const int pair = threadIdx.x, axis = a.pair_axis ? a.pair_axis[pair] : 0;
      float cs = 1.f, sn = 0.f;
      if ((unsigned)axis < (unsigned)a.axes) {
        // in turns, in 64 bits: what is left of a far position's angle after
        // whole turns is then as exact as a near one's
        double x = (double)a.positions[axis * a.M + m] * ((double)a.freqs[pair] * 0.15915494309189533577);
        x -= rint(x);
        sincospif(2.f * (float)x, &sn, &cs);
      }
      turn[pair][0] = cs;
      turn[pair][1] = sn;
    }
    __syncthreads();
  }

  const float inv_d = 1.f / (float)a.D;
  auto step = [&](Piece<T, VEC> &piece) __attribute__((always_inline)) {
    int p;
    int64_t head;
    const bool here = where(i, p, head);
    float v[8];
    piece.values(v);
    load(i + 2 * stride, piece);
    if (p != 2) {
      if (!here) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = 0.f;
      }
      if (a.norm) normalise(v, a.norm, a.eps, inv_d, lg, live);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= p == 0 ? w[0][e] : w[1][e];
      if (turns) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float cs = turn[slot * 4 + e][0], sn = turn[slot * 4 + e][1];
          float &x = v[PAIRS ? 2 * e : e], &y = v[PAIRS ? 2 * e + 1 : e + 4];
          const float x0 = x, y0 = y;
          x = __builtin_fmaf(x0, cs, -(y0 * sn));
          y = __builtin_fmaf(y0, cs, x0 * sn);
        }
      }
    }
    if (here) store<VEC>(a.part[p].out, m * a.part[p].out_ld + head * a.D, lo, hi, v);
  };
  for (; i < steps; i += stride) {
    step(next[0]);
    i += stride;
    if (i >= steps) break;
    step(next[1]);
  }
}

}  // namespace

hipError_t launch_qk_norm_rope(const HeadsArgs &a, hipStream_t stream) {
  // One row to a block: 5.4 TB/s at 16896 rows of 54 heads of 256, where two
  // rows, half a row or a quarter give 5.1, 5.1 and 4.7. Few rows would leave
  // CUs idle: their steps are divided over up to as many blocks as keep 512 in
  // all, each of which makes the row's angles again.
  const int per = 64 >> a.lane_bits;
  int steps = 0;
  for (const auto &p : a.part) steps += (p.heads + per - 1) / per;
  const int most = (steps + 3) / 4;
  const int64_t want = a.M >= 512 ? 1 : 512 / a.M;
  const dim3 grid((unsigned)a.M, (unsigned)(want < most ? want : most));
#define QL_HEADS(T, PAIRS, VEC) qk_norm_rope_kernel<T, PAIRS, VEC><<<grid, 256, 0, stream>>>(a)
#define QL_HEADS_VEC(T, PAIRS) \
  if (a.vec) QL_HEADS(T, PAIRS, true); \
  else QL_HEADS(T, PAIRS, false)
  if (a.in_bf16) {
    if (a.pair_layout) { QL_HEADS_VEC(BF16, true); } else { QL_HEADS_VEC(BF16, false); }
  } else {
    if (a.pair_layout) { QL_HEADS_VEC(F32, true); } else { QL_HEADS_VEC(F32, false); }
  }
#undef QL_HEADS_VEC
#undef QL_HEADS
  return hipGetLastError();
}

}  // namespace ql
