// Softmax attention of packed samples (qlinear_attention):
//
//   out[m, h] = sum_j p_j v[j, h / G] / sum_j p_j,   p_j = exp(scale * q[m, h] . k[j, h / G])
//
// over the kept keys j of row m's sample; G = q_heads / kv_heads.
//
// One pass over the keys with the running maximum and sum of the softmax. A
// wave computes S^T = K Q^T (32 keys x 32 queries per MFMA), so a lane holds
// the scores of one query: the maximum and the sum are taken in registers and
// exchanged once between the two halves of the wave. The weights P^T leave the
// softmax in the very order in which the second product O^T = V^T P^T takes
// its right operand, if V's rows are taken in the order of S^T's rows; V^T
// comes from LDS by transposing reads, so no operand crosses lanes.
//
// Scores, maxima, sums and outputs are fp32; P enters the second product as
// bf16 (its operand type, error 2^-9 of a weight), and the sum is taken of the
// rounded weights, so that what the output is divided by is exactly what it
// was multiplied by. The output is rounded once.
#include <algorithm>

#include "ql_block.h"
#include "ql_kernels.h"

namespace ql {

namespace {

typedef __attribute__((__vector_size__(4 * sizeof(short)))) short s16x4;

constexpr float kLowest = -3.4028234663852886e38f;
// A maximum is followed only when it has grown by more than 2^kSlack: weights
// then stay below 2^kSlack and the sums far below fp32's limit, and the
// outputs are rescaled a few times instead of at every tile.
constexpr float kSlack = 8.f;
constexpr int kOut = 0x7FFFFFFF;  // an offset past every buffer: the load gives zeros

// 16-byte unit that holds unit c of a row in LDS. K is read 16 bytes per lane
// by 32 rows at once (units of eight rows in a row of 128 bytes each), V eight
// bytes per lane from four rows (two units of each).
__device__ __forceinline__ int k_unit(int row, int c) { return c ^ (row & 7); }
__device__ __forceinline__ int v_unit(int row, int c) { return c ^ ((row & 3) * 2); }

__device__ __forceinline__ bf16x8 lds_read8(const unsigned char *p) { return *reinterpret_cast<const bf16x8 *>(p); }

__device__ __forceinline__ s16x4 lds_read_tr(const unsigned char *p) {
  typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
}

__device__ __forceinline__ float other_half(float v) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float((threadIdx.x & 32) ? r[0] : r[1]);
}

// ------------------------------------------------------------------ which block does what

// Rows, keys and tiles of one sample.
struct Sample {
  int64_t q0, k0;
  int rows, keys;  // rows: queries times the heads that share a key head
};

__device__ __forceinline__ Sample sample_of(const AttentionArgs &a, int s) {
  Sample r = {0, 0, (int)(a.Mq * a.group), (int)a.Mk};
  if (a.q_offsets) {
    // whatever the offsets hold, no row outside the arrays is touched
    const int64_t b = min(max((int64_t)a.q_offsets[s], (int64_t)0), a.Mq), e = min((int64_t)a.q_offsets[s + 1], a.Mq);
    r.q0 = b;
    r.rows = (int)(max(e - b, (int64_t)0) * a.group);
  }
  if (a.k_offsets) {
    const int64_t b = min(max((int64_t)a.k_offsets[s], (int64_t)0), a.Mk), e = min((int64_t)a.k_offsets[s + 1], a.Mk);
    r.k0 = b;
    r.keys = (int)max(e - b, (int64_t)0);
  }
  return r;
}

// Inclusive sum over the 64 lanes.
__device__ __forceinline__ int64_t scan(int64_t v) {
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int64_t o = __shfl_up(v, d);
    if ((int)(threadIdx.x & 63) >= d) v += o;
  }
  return v;
}

// The division of a call's tiles over blocks. The first `whole` tiles belong
// to a block each; the keys of the others are cut into pieces of `per` units.
// All of it follows from the offsets, so every block finds the same.
struct Plan {
  int64_t tiles, whole;
  int per;
};

struct Work {
  Sample s;
  int head, tile;       // key head; tile of BQ rows
  int unit0, unit1;     // units of keys
  int64_t slot;         // where its partial sums go, -1: it writes the output
};

template <int BQ, int UNIT>
struct Division {
  static __device__ __forceinline__ int64_t tiles_of(const AttentionArgs &a, const Sample &s) {
    return (int64_t)((s.rows + BQ - 1) / BQ) * a.kv_heads;
  }
  static __device__ __forceinline__ int units_of(const Sample &s) { return max((s.keys + UNIT - 1) / UNIT, 1); }

  // Calls f(sample index or -1, Sample) with 64 samples at a time, a lane each, until f returns true.
  template <typename F>
  static __device__ __forceinline__ void each(const AttentionArgs &a, F f) {
    for (int s0 = 0; s0 < a.samples; s0 += 64) {
      const int s = s0 + (int)(threadIdx.x & 63);
      Sample x = {0, 0, 0, 0};
      if (s < a.samples) x = sample_of(a, s);
      if (f(s < a.samples ? s : -1, x)) return;
    }
  }

  static __device__ __forceinline__ Plan plan(const AttentionArgs &a) {
    Plan p = {0, 0, 1 << 30};
    each(a, [&](int, const Sample &x) {
      p.tiles += __shfl(scan(tiles_of(a, x)), 63);
      return false;
    });
    if (a.slots == 0) {
      p.whole = p.tiles;
      return p;
    }
    p.whole = a.cut_all ? 0 : p.tiles / a.slots * a.slots;
    int64_t first = 0, units = 0;
    each(a, [&](int, const Sample &x) {
      const int64_t n = tiles_of(a, x), incl = scan(n);
      const int64_t begin = first + incl - n, cut = min(max(begin + n - p.whole, (int64_t)0), n);
      units += __shfl(scan(cut * units_of(x)), 63);
      first += __shfl(incl, 63);
      return false;
    });
    p.per = (int)max((units + a.slots - 1) / a.slots, (int64_t)a.least_units);
    return p;
  }

  // The tile `t` (of all, `t` >= 0), or the tile that the piece `b` of the cut ones belongs to (t < 0).
  static __device__ __forceinline__ bool find(const AttentionArgs &a, const Plan &p, int64_t t, int64_t b, Work &w) {
    int64_t first = 0, pieces = 0;
    bool found = false;
    // offsets that decrease may ask for more pieces than there is room for
    if (t < 0 && b >= a.pieces) return false;
    each(a, [&](int s, const Sample &x) {
      const int64_t n = tiles_of(a, x), incl = scan(n);
      const int64_t begin = first + incl - n;
      const int64_t cut = min(max(begin + n - p.whole, (int64_t)0), n);  // the last `cut` tiles of the sample are cut
      const int parts = (units_of(x) + p.per - 1) / p.per;
      const int64_t pincl = scan(cut * parts), pbegin = pieces + pincl - cut * parts;
      const bool mine = s >= 0 && (t >= 0 ? t >= begin && t < begin + n : b >= pbegin && b < pbegin + cut * parts);
      const uint64_t who = __ballot(mine);
      if (who) {
        const int l = __builtin_ctzll(who);
        const int sl = __shfl(s, l), np = __shfl(parts, l);
        const int64_t nl = __shfl(n, l), cl = __shfl(cut, l), bl = __shfl(begin, l), pl = __shfl(pbegin, l);
        w.s = sample_of(a, sl);
        const int64_t in = t >= 0 ? t - bl : nl - cl + (b - pl) / np;
        const int heads_tiles = (w.s.rows + BQ - 1) / BQ;
        w.head = (int)(in / heads_tiles);
        w.tile = (int)(in % heads_tiles);
        const int all = units_of(w.s);
        const bool is_cut = in >= nl - cl && np > 1;
        const int piece = t >= 0 ? 0 : (int)((b - pl) % np);
        w.unit0 = t >= 0 ? 0 : piece * p.per;
        w.unit1 = t >= 0 ? all : min(all, w.unit0 + p.per);
        // of a tile: the slot of its first piece
        w.slot = is_cut ? (t >= 0 ? pl + (in - (nl - cl)) * np : b) : -1;
        found = w.slot + (t >= 0 ? np : 1) <= a.pieces || !is_cut;
        return true;
      }
      first += __shfl(incl, 63);
      pieces += __shfl(pincl, 63);
      return false;
    });
    return found;
  }
};

// Consecutive logical blocks on one XCD, for any number of blocks.
__device__ __forceinline__ int64_t xcd_order(int64_t b, int64_t n) {
  const int64_t x = b & 7, each = n >> 3, more = n & 7;
  return x * each + min(x, more) + (b >> 3);
}

// ------------------------------------------------------------------ the products

// fp32 accumulators of 32 x 32 MFMAs: column lane & 31, register r row
// 8 (r / 4) + 4 (lane / 32) + r % 4.
__device__ __forceinline__ constexpr int acc_row(int r) { return (r >> 2) * 8 + (r & 3); }

template <int DP, int NQ>
struct State {
  bf16x8 q[NQ][DP / 16];     // Q^T: lane's query, 8 values at 16 i + 8 (lane / 32)
  f32x16 o[NQ][DP / 32];     // O^T
  float m[NQ], l[NQ];        // maximum followed (in powers of two), sum of this half's weights
};

// Query rows r0 + 32 i + (lane & 31) of a tile into registers; zeros past the rows and past D.
template <int DP, int NQ>
__device__ __forceinline__ void load_q(const AttentionArgs &a, const Work &w, int r0, State<DP, NQ> &st) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    const int r = r0 + 32 * i + (lane & 31);
    const bool in = r < w.s.rows;
    const int m = in ? r / a.group : 0, g = in ? r % a.group : 0;
    const uint16_t *p = a.q + (w.s.q0 + m) * a.q_ld + (int64_t)(w.head * a.group + g) * a.D;
#pragma unroll
    for (int j = 0; j < DP / 16; ++j) {
      const int d = 16 * j + 8 * (lane >> 5);
      u32x4 v = {0, 0, 0, 0};
      if (in && d < a.D) v = *reinterpret_cast<const u32x4 *>(p + d);
      st.q[i][j] = as_bf16x8(v);
    }
#pragma unroll
    for (int j = 0; j < DP / 32; ++j) st.o[i][j] = f32x16{};
    st.m[i] = kLowest;
    st.l[i] = 0.f;
  }
}

// S^T of 32 keys: K rows [row0, row0 + 32) of the stage at kb.
template <int DP, int NQ>
__device__ __forceinline__ void scores(const unsigned char *kb, int row0, const State<DP, NQ> &st, f32x16 (&s)[NQ]) {
  const int lane = threadIdx.x & 63, row = row0 + (lane & 31), h = lane >> 5;
#pragma unroll
  for (int i = 0; i < NQ; ++i) s[i] = f32x16{};
#pragma unroll
  for (int j = 0; j < DP / 16; ++j) {
    const bf16x8 k = lds_read8(kb + row * (DP * 2) + k_unit(row, 2 * j + h) * 16);
#pragma unroll
    for (int i = 0; i < NQ; ++i) s[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k, st.q[i][j], s[i], 0, 0, 0);
  }
}

// One tile's scores become weights: keys whose bit in `valid` is clear get
// none; the maximum, the sum and, where the maximum is followed, the output so
// far are brought up to date.
template <int DP, int NQ>
__device__ __forceinline__ void weights(State<DP, NQ> &st, f32x16 (&s)[NQ], float c, uint32_t valid, bf16x8 (&p)[NQ][2]) {
  const int h = (threadIdx.x >> 5) & 1;
  if (valid != 0xFFFFFFFFu) {
    const uint32_t mine = valid >> (4 * h);
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const bool keep = (mine >> acc_row(r)) & 1;
#pragma unroll
      for (int i = 0; i < NQ; ++i) s[i][r] = keep ? s[i][r] : -__builtin_inff();
    }
  }
  float mx[NQ];
  bool follow = false;
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    float x = s[i][0];
#pragma unroll
    for (int r = 1; r < 16; ++r) x = fmaxf(x, s[i][r]);
    mx[i] = fmaxf(x, other_half(x)) * c;
    follow |= mx[i] > st.m[i] + kSlack;
  }
  if (__any(follow)) {
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      // each query by its own scores alone
      const float m = mx[i] > st.m[i] + kSlack ? mx[i] : st.m[i];
      const float f = __builtin_amdgcn_exp2f(st.m[i] - m);
      st.m[i] = m;
      st.l[i] *= f;
#pragma unroll
      for (int j = 0; j < DP / 32; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) st.o[i][j][r] *= f;
    }
  }
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    uint32_t w[8];
#pragma unroll
    for (int r = 0; r < 16; r += 2) {
      const float a = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][r], c, -st.m[i]));
      const float b = __builtin_amdgcn_exp2f(__builtin_fmaf(s[i][r + 1], c, -st.m[i]));
      w[r / 2] = pack_bf16(a, b);
    }
#pragma unroll
    for (int r = 0; r < 8; ++r) st.l[i] += bf16_lo(w[r]) + bf16_hi(w[r]);
    p[i][0] = as_bf16x8(u32x4{w[0], w[1], w[2], w[3]});
    p[i][1] = as_bf16x8(u32x4{w[4], w[5], w[6], w[7]});
  }
}

// O^T += V^T P^T over the 32 V rows [row0, row0 + 32) of the stage at vb.
template <int DP, int NQ>
__device__ __forceinline__ void outputs(const unsigned char *vb, int row0, State<DP, NQ> &st, const bf16x8 (&p)[NQ][2]) {
  const int lane = threadIdx.x & 63, h = lane >> 5;
  const int row = row0 + 4 * h + ((lane & 15) >> 2);                  // + 16 t + 8 u
  const int unit = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1), byte = (lane & 1) * 8;  // + 4 j
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int j = 0; j < DP / 32; ++j) {
      const unsigned char *r = vb + (row + 16 * t) * (DP * 2) + v_unit(row, unit + 4 * j) * 16 + byte;
      const s16x4 lo = lds_read_tr(r), hi = lds_read_tr(r + 8 * DP * 2);
      const bf16x8 v = __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
      for (int i = 0; i < NQ; ++i) st.o[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, p[i][t], st.o[i][j], 0, 0, 0);
    }
}

// Rows of K or V of one key head of a sample, from the sample's key `first` on.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const AttentionArgs &a, const uint16_t *x, int64_t ld,
                                                          const Work &w, int first) {
  const int64_t rows = w.s.keys - first;
  return make_rsrc(x + (w.s.k0 + first) * ld + (int64_t)w.head * a.D, 0, rows <= 0 ? 0 : ((rows - 1) * ld + a.D) * 2);
}

// Bits of the keys [first, first + 64) of the sample that are kept.
template <bool MASKED>
__device__ __forceinline__ uint64_t kept(const AttentionArgs &a, const Work &w, int first, int mask_byte) {
  const int rest = w.s.keys - first;
  const uint64_t in = rest >= 64 ? ~0ull : rest <= 0 ? 0ull : (1ull << rest) - 1;
  if constexpr (MASKED) return in & __ballot(mask_byte != 0);
  else return in;
}
__device__ __forceinline__ int mask_byte(const AttentionArgs &a, const Work &w, int first) {
  const int j = first + (int)(threadIdx.x & 63);
  return j < w.s.keys ? a.key_mask[w.s.k0 + j] : 0;
}

// Partial sums of a tile: [DP / 4][rows][4] outputs, then the maxima, then the sums, fp32.
template <int DP, int BQ> __device__ __forceinline__ float *slot_at(const AttentionArgs &a, int64_t slot) {
  return a.partial + slot * (int64_t)(BQ * (DP + 2));
}

__device__ __forceinline__ uint16_t *out_row(const AttentionArgs &a, const Work &w, int r) {
  return a.out + (w.s.q0 + r / a.group) * a.out_ld + (int64_t)(w.head * a.group + r % a.group) * a.D;
}

// Sum over both halves, 1 / it, or 0 where there is no weight at all.
__device__ __forceinline__ float reciprocal(float l) { return l == 0.f ? 0.f : 1.f / l; }

// ------------------------------------------------------------------ tiles of many rows

// A block of four waves, 32 NQ rows each, over keys in stages of 64 that all
// waves read from LDS, the next stage on its way meanwhile.
template <int DP, int NQ, bool MASKED>
__global__ __launch_bounds__(256, 1) void attention_kernel(AttentionArgs a) {
  constexpr int BQ = 128 * NQ, UNIT = 64, kBytes = UNIT * DP * 2;
  constexpr int kUnits = DP / 8;             // 16-byte units of a row
  constexpr int kCopies = UNIT * kUnits / 256;  // copies of 64 units per wave and stage
  __shared__ __attribute__((aligned(16))) unsigned char k0[kBytes], k1[kBytes], v0[kBytes], v1[kBytes];
  using Div = Division<BQ, UNIT>;
  const Plan plan = Div::plan(a);
  Work w;
  if ((int64_t)blockIdx.x < plan.whole) {
    if (!Div::find(a, plan, xcd_order(blockIdx.x, plan.whole), 0, w)) return;
  } else {
    if (!Div::find(a, plan, -1, blockIdx.x - plan.whole, w)) return;
  }
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int r0 = w.tile * BQ + wave * 32 * NQ;
  const bool busy = r0 < w.s.rows;
  State<DP, NQ> st;
  load_q<DP, NQ>(a, w, r0, st);
  const float c = a.scale * 1.4426950408889634f;

  // copy i of this wave: unit (4 i + wave) * 64 + lane of the stage
  int row[kCopies], kofs[kCopies], vofs[kCopies];
#pragma unroll
  for (int i = 0; i < kCopies; ++i) {
    const int id = (4 * i + wave) * 64 + lane;
    row[i] = id / kUnits;
    const int kc = k_unit(row[i], id % kUnits), vc = v_unit(row[i], id % kUnits);
    kofs[i] = kc * 8 < a.D ? (int)(row[i] * a.k_ld + kc * 8) * 2 : kOut;
    vofs[i] = vc * 8 < a.D ? (int)(row[i] * a.v_ld + vc * 8) * 2 : kOut;
  }
  int next_mask = 0;
  auto copy = [&](unsigned char *kb, unsigned char *vb, int first, uint64_t keep) {
    const auto kr = rows_of(a, a.k, a.k_ld, w, first), vr = rows_of(a, a.v, a.v_ld, w, first);
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const bool in = !MASKED || (keep >> row[i] & 1);
      dma16(kr, in ? kofs[i] : kOut, 0, kb + (4 * i + wave) * 1024);
    }
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const bool in = !MASKED || (keep >> row[i] & 1);
      dma16(vr, in ? vofs[i] : kOut, 0, vb + (4 * i + wave) * 1024);
    }
  };
  const int first = w.unit0 * UNIT, end = min(w.unit1 * UNIT, w.s.keys);
  uint64_t keep = 0, keep_next = 0;
  auto stage = [&](unsigned char *kb, unsigned char *vb, unsigned char *kn, unsigned char *vn, int at) {
    dma_barrier();  // this stage has landed everywhere, the one before is free
    keep = keep_next;
    if (at + UNIT < end) {
      keep_next = kept<MASKED>(a, w, at + UNIT, next_mask);
      if constexpr (MASKED) next_mask = mask_byte(a, w, at + 2 * UNIT);
      copy(kn, vn, at + UNIT, keep_next);
    }
    if (!busy || keep == 0) return;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      f32x16 s[NQ];
      bf16x8 p[NQ][2];
      scores<DP, NQ>(kb, 32 * t, st, s);
      weights<DP, NQ>(st, s, c, (uint32_t)(keep >> (32 * t)), p);
      outputs<DP, NQ>(vb, 32 * t, st, p);
    }
  };
  if (first < end) {
    if constexpr (MASKED) next_mask = mask_byte(a, w, first);
    keep_next = kept<MASKED>(a, w, first, next_mask);
    if constexpr (MASKED) next_mask = mask_byte(a, w, first + UNIT);
    copy(k0, v0, first, keep_next);
    for (int at = first; at < end; at += 2 * UNIT) {
      stage(k0, v0, k1, v1, at);
      if (at + UNIT < end) stage(k1, v1, k0, v0, at + UNIT);
    }
  }
  if (!busy) return;
  const int h = lane >> 5;
  float *part = w.slot >= 0 ? slot_at<DP, BQ>(a, w.slot) : nullptr;
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    const int rt = wave * 32 * NQ + 32 * i + (lane & 31), r = w.tile * BQ + rt;
    const float l = st.l[i] + other_half(st.l[i]);
    if (r >= w.s.rows) continue;
    if (part) {
#pragma unroll
      for (int j = 0; j < DP / 32; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g)
          *reinterpret_cast<f32x4 *>(part + ((int64_t)(8 * j + 2 * g + h) * BQ + rt) * 4) =
              f32x4{st.o[i][j][4 * g], st.o[i][j][4 * g + 1], st.o[i][j][4 * g + 2], st.o[i][j][4 * g + 3]};
      if (h == 0) {
        part[(int64_t)BQ * DP + rt] = st.m[i];
        part[(int64_t)BQ * (DP + 1) + rt] = l;
      }
    } else {
      const float f = reciprocal(l);
      uint16_t *o = out_row(a, w, r);
#pragma unroll
      for (int j = 0; j < DP / 32; ++j)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const int d = 32 * j + 8 * g + 4 * h;
          if (d < a.D)
            *reinterpret_cast<u32x2 *>(o + d) = u32x2{pack_bf16(st.o[i][j][4 * g] * f, st.o[i][j][4 * g + 1] * f),
                                                      pack_bf16(st.o[i][j][4 * g + 2] * f, st.o[i][j][4 * g + 3] * f)};
        }
    }
  }
}

// ------------------------------------------------------------------ tiles of few rows

// 32 rows at most: the four waves of a block share them and take every fourth
// tile of 32 keys each, through LDS of their own, without a barrier until
// their sums are joined at the end.
template <int DP, bool MASKED>
__global__ __launch_bounds__(256, 1) void attention_few_kernel(AttentionArgs a) {
  constexpr int BQ = 32, UNIT = 128, kBytes = 32 * DP * 2, kUnits = DP / 8, kCopies = 32 * kUnits / 64;
  __shared__ __attribute__((aligned(16))) unsigned char ks[4 * kBytes], vs[4 * kBytes];
  __shared__ float ms[4][32], ls[4][32];
  using Div = Division<BQ, UNIT>;
  const Plan plan = Div::plan(a);
  Work w;
  if ((int64_t)blockIdx.x < plan.whole) {
    if (!Div::find(a, plan, blockIdx.x, 0, w)) return;
  } else {
    if (!Div::find(a, plan, -1, blockIdx.x - plan.whole, w)) return;
  }
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  State<DP, 1> st;
  load_q<DP, 1>(a, w, w.tile * BQ, st);
  const float c = a.scale * 1.4426950408889634f;
  unsigned char *const kb = ks + wave * kBytes, *const vb = vs + wave * kBytes;
  // copy i of the wave: unit 64 i + lane of its tile
  auto copy = [&](const uint16_t *x, int64_t ld, bool is_k, unsigned char *to, int at, uint32_t keep) {
    const auto r = rows_of(a, x, ld, w, at);
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const int id = 64 * i + lane, row = id / kUnits;
      const int u = is_k ? k_unit(row, id % kUnits) : v_unit(row, id % kUnits);
      const bool in = u * 8 < a.D && (!MASKED || (keep >> row & 1));
      dma16(r, in ? (int)(row * ld + u * 8) * 2 : kOut, 0, to + i * 1024);
    }
  };
  const int end = min(w.unit1 * UNIT, w.s.keys);
  int at = w.unit0 * UNIT + 32 * wave;
  if (at < end) {
    int byte = 0, byte_next = 0;
    if constexpr (MASKED) {
      byte = mask_byte(a, w, at);
      byte_next = mask_byte(a, w, at + 128);
    }
    uint32_t keep = (uint32_t)kept<MASKED>(a, w, at, byte);
    copy(a.k, a.k_ld, true, kb, at, keep);
    copy(a.v, a.v_ld, false, vb, at, keep);
    for (; at < end; at += 128) {
      const bool more = at + 128 < end;
      uint32_t keep_next = 0;
      if (more) {
        keep_next = (uint32_t)kept<MASKED>(a, w, at + 128, byte_next);
        if constexpr (MASKED) byte_next = mask_byte(a, w, at + 256);
      }
      f32x16 s[1];
      bf16x8 p[1][2];
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      scores<DP, 1>(kb, 0, st, s);
      // the reads of K are back before its place is filled again
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (more) copy(a.k, a.k_ld, true, kb, at + 128, keep_next);
      weights<DP, 1>(st, s, c, keep, p);
      outputs<DP, 1>(vb, 0, st, p);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (more) copy(a.v, a.v_ld, false, vb, at + 128, keep_next);
      keep = keep_next;
    }
  }
  // Joined through the waves' own LDS: the first half of the outputs in K's place, the second in V's.
  const int h = lane >> 5, col = lane & 31;
  const float l = st.l[0] + other_half(st.l[0]);
#pragma unroll
  for (int j = 0; j < DP / 32; ++j) {
    f32x4 *const to = reinterpret_cast<f32x4 *>(j < DP / 64 ? kb : vb);
#pragma unroll
    for (int g = 0; g < 4; ++g)
      to[(8 * (j % (DP / 64)) + 2 * g + h) * 32 + col] =
          f32x4{st.o[0][j][4 * g], st.o[0][j][4 * g + 1], st.o[0][j][4 * g + 2], st.o[0][j][4 * g + 3]};
  }
  if (h == 0) {
    ms[wave][col] = st.m[0];
    ls[wave][col] = l;
  }
  __syncthreads();
  const int rt = threadIdx.x & 31, r = w.tile * BQ + rt;
  if (r >= w.s.rows) return;
  float f[4], m = kLowest, sum = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = fmaxf(m, ms[i][rt]);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = __builtin_amdgcn_exp2f(ms[i][rt] - m);
    sum += ls[i][rt] * f[i];
  }
  float *part = w.slot >= 0 ? slot_at<DP, BQ>(a, w.slot) : nullptr;
  if (part && threadIdx.x < 32) {
    part[BQ * DP + rt] = m;
    part[BQ * (DP + 1) + rt] = sum;
  }
  const float inv = reciprocal(sum);
  uint16_t *o = out_row(a, w, r);
  for (int d4 = threadIdx.x >> 5; d4 < DP / 4; d4 += 8) {
    const f32x4 *from = reinterpret_cast<const f32x4 *>(d4 < DP / 8 ? ks : vs) + (d4 % (DP / 8)) * 32 + rt;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4 x = from[i * (kBytes / 16)];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(x[e], f[i], v[e]);
    }
    if (part) *reinterpret_cast<f32x4 *>(part + ((int64_t)d4 * BQ + rt) * 4) = v;
    else if (d4 * 4 < a.D)
      *reinterpret_cast<u32x2 *>(o + d4 * 4) = u32x2{pack_bf16(v[0] * inv, v[1] * inv), pack_bf16(v[2] * inv, v[3] * inv)};
  }
}

// ------------------------------------------------------------------ joining pieces

// The pieces of the cut tiles become outputs. Grid: x cut tiles, y ranges of
// 16 values; a thread has one row.
template <int DP, int BQ, int UNIT>
__global__ __launch_bounds__(BQ < 64 ? 64 : BQ) void attention_join_kernel(AttentionArgs a) {
  using Div = Division<BQ, UNIT>;
  const Plan plan = Div::plan(a);
  Work w;
  if (plan.whole + (int64_t)blockIdx.x >= plan.tiles || !Div::find(a, plan, plan.whole + blockIdx.x, 0, w) || w.slot < 0) return;
  const int rt = threadIdx.x % BQ, r = w.tile * BQ + rt;
  if (r >= w.s.rows) return;
  const int pieces = (w.unit1 + plan.per - 1) / plan.per;
  const float *part = slot_at<DP, BQ>(a, w.slot);
  constexpr int64_t kSlot = BQ * (DP + 2);
  float m = kLowest, sum = 0.f;
  for (int i = 0; i < pieces; ++i) m = fmaxf(m, part[i * kSlot + BQ * DP + rt]);
  // 32 rows: two threads of a row share its values
  constexpr int kShare = BQ < 64 ? 64 / BQ : 1;
  const int d0 = blockIdx.y * 4 + threadIdx.x / BQ;
  f32x4 v[4 / kShare] = {};
  for (int i = 0; i < pieces; ++i) {
    const float f = __builtin_amdgcn_exp2f(part[i * kSlot + BQ * DP + rt] - m);
    sum = __builtin_fmaf(part[i * kSlot + BQ * (DP + 1) + rt], f, sum);
#pragma unroll
    for (int j = 0; j < 4 / kShare; ++j) {
      const f32x4 x = *reinterpret_cast<const f32x4 *>(part + i * kSlot + ((int64_t)(d0 + j * kShare) * BQ + rt) * 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[j][e] = __builtin_fmaf(x[e], f, v[j][e]);
    }
  }
  const float inv = reciprocal(sum);
  uint16_t *o = out_row(a, w, r);
#pragma unroll
  for (int j = 0; j < 4 / kShare; ++j) {
    const int d = 4 * (d0 + j * kShare);
    if (d < a.D)
      *reinterpret_cast<u32x2 *>(o + d) = u32x2{pack_bf16(v[j][0] * inv, v[j][1] * inv), pack_bf16(v[j][2] * inv, v[j][3] * inv)};
  }
}

int padded(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }

constexpr int kCus = 256;  // MI355X

template <int DP, int NQ>
void launch_rows(const AttentionArgs &a, const AttentionPlan &p, hipStream_t stream) {
  const dim3 grid((unsigned)p.blocks);
  if (a.key_mask) attention_kernel<DP, NQ, true><<<grid, 256, 0, stream>>>(a);
  else attention_kernel<DP, NQ, false><<<grid, 256, 0, stream>>>(a);
  if (a.slots) attention_join_kernel<DP, 128 * NQ, 64><<<dim3((unsigned)p.cut, DP / 16), 128 * NQ, 0, stream>>>(a);
}

template <int DP>
void launch_width(const AttentionArgs &a, const AttentionPlan &p, hipStream_t stream) {
  if (p.rows == 32) {
    const dim3 grid((unsigned)p.blocks);
    if (a.key_mask) attention_few_kernel<DP, true><<<grid, 256, 0, stream>>>(a);
    else attention_few_kernel<DP, false><<<grid, 256, 0, stream>>>(a);
    if (a.slots) attention_join_kernel<DP, 32, 128><<<dim3((unsigned)p.cut, DP / 16), 64, 0, stream>>>(a);
  } else if (p.rows == 128) {
    launch_rows<DP, 1>(a, p, stream);
  } else if constexpr (DP <= 128) {
    launch_rows<DP, 2>(a, p, stream);
  }
}

}  // namespace

AttentionPlan attention_plan(int64_t Mq, int64_t Mk, int64_t samples, int q_heads, int kv_heads, int D, bool workspace) {
  AttentionPlan p{};
  const int dp = padded(D);
  const int64_t rows = Mq * (q_heads / kv_heads), each = rows / std::max<int64_t>(samples, 1);
  p.rows = each <= 32 ? 32 : each <= 128 || dp > 128 ? 128 : 256;
  // tiles of all samples at most: whatever the offsets are, one more per sample than without them
  const int64_t tiles = ((rows + p.rows - 1) / p.rows + samples) * kv_heads;
  p.slots = workspace ? (p.rows == 32 ? 2 * kCus : kCus) : 0;
  p.cut_all = p.rows == 32;
  p.least_units = 4;
  // keys that do not reach two pieces are not cut, nor are tiles that fill the blocks several times over
  if (Mk <= (p.rows == 32 ? 128 : 64) * (int64_t)p.least_units || (p.cut_all && tiles >= 4 * (int64_t)p.slots)) p.slots = 0;
  p.cut = p.slots == 0 ? 0 : p.cut_all ? tiles : std::min<int64_t>(tiles, p.slots - 1);
  p.pieces = p.slots == 0 ? 0 : p.slots + p.cut;
  p.blocks = tiles + p.pieces;
  p.partial_bytes = (size_t)p.pieces * p.rows * (dp + 2) * sizeof(float);
  return p;
}

hipError_t launch_attention(const AttentionArgs &args, const AttentionPlan &p, hipStream_t stream) {
  AttentionArgs a = args;
  a.slots = p.slots;
  a.cut_all = p.cut_all;
  a.least_units = p.least_units;
  a.pieces = p.pieces;
  switch (padded(a.D)) {
    case 64: launch_width<64>(a, p, stream); break;
    case 128: launch_width<128>(a, p, stream); break;
    default: launch_width<256>(a, p, stream); break;
  }
  return hipGetLastError();
}

}  // namespace ql
