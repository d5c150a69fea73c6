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
// bf16, and the sum is taken of the rounded weights, so that what the output is
// divided by is exactly what it was multiplied by. That is a choice: MFMAs take
// P in V's type, and a weight as two bf16 parts would ask for half as many MFMAs
// again. A weight is off by up to 2^-8, relative. Outputs, whose own rounding
// makes 1.65e-3 to 1.67e-3 in the mean square against 64 bits, come to 0.4 %
// more than that over 16896 keys, 1.3 % over 4608, 5 % over 512 and 6 % over the
// 130 kept keys of the masked odd samples. The output is rounded once.
//
// Three kernels: attention_kernel for tiles of 128 or 256 rows, bound by the
// matrix unit; attention_few_kernel for up to 32, bound by the bytes of K and V
// or, on few CUs, by their latency; attention_join_kernel for tiles whose keys
// were cut into pieces to fill the card. attention_plan() chooses.
#include <algorithm>
#include <utility>

#include "ql_block.h"
#include "ql_kernels.h"

namespace ql {

namespace {

typedef __attribute__((__vector_size__(4 * sizeof(short)))) short s16x4;

constexpr float kLowest = -3.4028234663852886e38f;
// A maximum is followed only when it has grown by more than 2^kSlack: weights
// then stay below 2^kSlack and the sums far below fp32's limit, and the
// outputs are rescaled a few times instead of every 32 keys (which would take
// as many instructions of the vector unit as the weights themselves).
constexpr float kSlack = 8.f;
constexpr uint32_t kOut = 0x7FFFFFFF;  // an offset past every buffer: the load gives zeros

// 16-byte unit that holds unit c of a row in LDS. K is read 16 bytes per lane,
// the same unit of 32 rows at once: eight rows in turn have theirs at eight
// different places of 128 bytes. V is read eight bytes per lane, two units of
// four rows at once, which lie side by side in 128 bytes. Over twice as many
// places neither is faster (4608 tokens of 18 heads of 256: V 379 us against
// 380, K 383).
__device__ __forceinline__ int k_unit(int row, int c) { return c ^ (row & 7); }
__device__ __forceinline__ int v_unit(int row, int c) { return c ^ ((row & 3) * 2); }

// Values of a row in LDS, whole groups of eight units, for heads of DP values
// (D rounded up to what the kernels are made for).
constexpr int lds_width(int DP) { return (DP + 63) / 64 * 64; }

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

// Rows and keys of one sample.
struct Sample {
  int q0, k0;
  int rows, keys;  // rows: queries times the heads that share a key head
};

__device__ __forceinline__ Sample sample_of(const AttentionArgs &a, int s) {
  Sample r = {0, 0, (int)a.Mq * a.group, (int)a.Mk};
  if (a.q_offsets) {
    // whatever the offsets hold, no row outside the arrays is touched
    const int Mq = (int)a.Mq, Mk = (int)a.Mk;
    const auto within = [](int v, int most) { return min(max(v, 0), most); };
    r.q0 = within(a.q_offsets[s], Mq);
    r.k0 = within(a.k_offsets[s], Mk);
    r.rows = max(within(a.q_offsets[s + 1], Mq) - r.q0, 0) * a.group;
    r.keys = max(within(a.k_offsets[s + 1], Mk) - r.k0, 0);
  }
  return r;
}

struct Plus {
  template <typename T> __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};
struct Most {
  template <typename T> __device__ __forceinline__ T operator()(T a, T b) const { return max(a, b); }
};
// Sums (or maxima of what is not negative) over the lanes up to and with this one.
template <typename T, typename Op = Plus>
__device__ __forceinline__ T scan(T v, Op op = {}) {
  auto add = [&](auto moved) { v = op(v, __builtin_bit_cast(T, moved)); };
  const auto bits = [&] { return __builtin_bit_cast(int, v); };
  add(__builtin_amdgcn_update_dpp(0, bits(), 0x111, 0xF, 0xF, true));   // row_shr:1
  add(__builtin_amdgcn_update_dpp(0, bits(), 0x112, 0xF, 0xF, true));   // row_shr:2
  add(__builtin_amdgcn_update_dpp(0, bits(), 0x114, 0xF, 0xF, true));   // row_shr:4
  add(__builtin_amdgcn_update_dpp(0, bits(), 0x118, 0xF, 0xF, true));   // row_shr:8
  add(__builtin_amdgcn_update_dpp(0, bits(), 0x142, 0xA, 0xF, false));  // row_bcast:15 into rows 1 and 3
  add(__builtin_amdgcn_update_dpp(0, bits(), 0x143, 0xC, 0xF, false));  // row_bcast:31 into rows 2 and 3
  return v;
}
template <typename T> __device__ __forceinline__ T lane_of(T v, int lane) {
  return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

// A value that is the same in every lane, in a scalar register. The compiler
// knows that of most of these, but has some in vector registers all the same
// (loads that it cannot make scalar), and a buffer resource made of such a one
// turns every copy into a loop over the lanes: so it is not told.
__device__ __forceinline__ int uniform(int v) {
  asm("" : "+v"(v));
  return __builtin_amdgcn_readfirstlane(v);
}
__device__ __forceinline__ const uint16_t *uniform(const uint16_t *p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  return reinterpret_cast<const uint16_t *>((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32 | (uint32_t)uniform((int)v));
}

struct Work {
  Sample s;
  int head, tile;    // key head; tile of BQ rows
  int unit0, unit1;  // units of keys
  int slot;          // where its partial sums go (of a cut tile: the first piece's), -1: it writes the output
  int parts;         // pieces of the tile
};

// A block's work in scalar registers. Where it is found it is one value of several branches, so each kernel asks for
// this behind them.
__device__ __forceinline__ Work uniform(const Work &w) {
  return {{uniform(w.s.q0), uniform(w.s.k0), uniform(w.s.rows), uniform(w.s.keys)}, uniform(w.head), uniform(w.tile),
          uniform(w.unit0), uniform(w.unit1), uniform(w.slot), uniform(w.parts)};
}

// The division of a call's tiles over blocks: which sample, head, rows and
// keys a block has. The first `whole` tiles belong to a block each; the keys
// of the others are cut into pieces of `per` units, so that about as many
// pieces come out as blocks run at once (a.slots), or twice as many. All of it
// follows from the offsets, so every wave of every block finds the same.
constexpr int kMostBlocks = 1 << 24;  // of a call that is served

// Tiles of few rows are all cut, of many rows those behind the last whole round
// of blocks; into pieces of this many units at least.
__host__ __device__ constexpr bool cuts_all(int rows) { return rows == 32; }
__host__ __device__ constexpr int least_units(int rows) { return rows == 32 ? 2 : 3; }

// a / b of whole numbers, rounded down; of more than 2^20 it may be off by some. (Every block of every call with
// offsets divides a dozen times before its first load: 1 to 2 us where all digits are taken.)
__host__ __device__ __forceinline__ int quotient(int a, int b) {
#ifdef __HIP_DEVICE_COMPILE__
  const float inverse = __builtin_amdgcn_rcpf((float)b);
#else
  const float inverse = 1.f / (float)b;
#endif
  return (int)((float)a * inverse + 1e-4f);
}

// Units of a piece where `cut` tiles of `units` units each are cut so that
// pieces come out for `blocks` blocks, as many of every tile.
__host__ __device__ __forceinline__ int equal_pieces(int units, int cut, int blocks, int least_units) {
  const int by_blocks = quotient(blocks, cut), by_units = units / least_units;
  const int most = by_blocks < by_units ? by_blocks : by_units;
  return most > 1 ? quotient(units + most - 1, most) : units;
}
// Tiles of many rows are cut into pieces for one round of blocks or for two
// (144 tiles in 256 blocks leave 112 idle in one round, three pieces of each
// fill two), whichever is over first, or not at all. A round takes the units of
// a piece; whole tiles 2 more (outputs); the partial sums of a round of pieces
// go out and come back in 8 units' time, and the launch that joins them takes 4.
// Heads of 256, 256 rows to a tile, not cut and in two rounds: 162 tiles of 36
// units 113 and 149 us, 144 of 64 195 and 189, 164 of 264 behind 1024 whole ones
// 4.53 and 4.23 ms; 104 of 19 behind 256, not cut and in one round: 154 and 141.
// Heads of 128, 256 tiles of 16 units for 512 blocks: not cut 26, cut 37.
// mean, longest: units of the cut tiles. Returns the units of a piece, `longest` if none is to be cut.
__host__ __device__ __forceinline__ int best_length(int mean, int longest, int cut, int slots, int one, int two) {
  const auto cost = [&](int length) {
    if (length >= longest) return longest + 2;
    const int pieces = quotient(mean + length - 1, length) * cut;
    return quotient(pieces + slots - 1, slots) * length + 4 + quotient(8 * pieces, slots);
  };
  const int best = cost(two) < cost(one) ? two : one;
  return cost(best) < longest + 2 ? best : longest;
}

template <int BQ, int UNIT>
struct Division {
  const AttentionArgs &a;
  Sample mine;  // the lane's of the first 64 samples
  int tiles = 0, whole = 0, per = 1 << 30;
  static constexpr bool kAll = cuts_all(BQ);
  static constexpr int kLeast = least_units(BQ);

  __device__ __forceinline__ int whole_of(int tiles) const {
    return a.slots == 0 ? tiles : kAll ? 0 : (int)((unsigned)tiles / (unsigned)a.slots) * a.slots;
  }
  static __device__ __forceinline__ int tiles_of(const AttentionArgs &a, const Sample &s) {
    return (s.rows + BQ - 1) / BQ * a.kv_heads;
  }
  static __device__ __forceinline__ int units_of(const Sample &s) { return max((s.keys + UNIT - 1) / UNIT, 1); }

  // The lane's of the 64 samples from s0 on, an empty one past the last.
  __device__ __forceinline__ Sample lanes_sample(int s0) const {
    const int s = s0 + (int)(threadIdx.x & 63);
    return s < a.samples ? sample_of(a, s) : Sample{0, 0, 0, 0};
  }
  // Calls f with 64 samples at a time, a lane each, until it returns true.
  template <typename F> __device__ __forceinline__ void each(F f) {
    Sample next = mine;
    for (int s0 = 0; s0 < a.samples; s0 += 64) {
      const Sample x = next;
      next = lanes_sample(s0 + 64);  // on its way meanwhile
      if (f(x)) return;
    }
  }
  // Pieces of a cut tile.
  __device__ __forceinline__ int parts_of(const Sample &s) const {
    const int units = units_of(s);
    return units < a.cut_units ? 1 : (units + per - 1) / per;
  }
  // Of a sample's n tiles, whose first is `begin`, those that are cut.
  __device__ __forceinline__ int cut_of(int begin, int n) const { return min(max(begin + n - whole, 0), n); }

  __device__ __forceinline__ explicit Division(const AttentionArgs &args) : a(args) {
    if (a.samples == 1) {
      mine = sample_of(a, 0);
      tiles = tiles_of(a, mine);
      if (!a.q_offsets) {
        whole = a.whole;
        per = a.per;
        return;
      }
      whole = whole_of(tiles);
      const int cut = tiles - whole, units = units_of(mine);
      if (cut == 0) return;
      per = equal_pieces(units, cut, a.slots, kLeast);
      if (!kAll) per = best_length(units, units, cut, a.slots, per, equal_pieces(units, cut, 2 * a.slots, kLeast));
      return;
    }
    mine = lanes_sample(0);
    if (a.slots == 0 && a.samples > 64) {
      whole = kMostBlocks;  // nothing is cut: not worth a pass over the offsets to count
      return;
    }
    each([&](const Sample &x) {
      tiles = min(tiles + lane_of(scan(tiles_of(a, x)), 63), kMostBlocks);
      return false;
    });
    whole = whole_of(tiles);
    if (whole == tiles) return;
    int first = 0, longest = 1;
    float units = 0.f;  // counted to a few parts in a million
    each([&](const Sample &x) {
      const int n = tiles_of(a, x), incl = scan(n);
      const int cut = cut_of(first + incl - n, n);
      units += lane_of(scan((float)cut * (float)units_of(x)), 63);
      if (!kAll) longest = max(longest, lane_of(scan(cut > 0 ? units_of(x) : 0, Most{}), 63));
      first = min(first + lane_of(incl, 63), kMostBlocks);
      return false;
    });
    // half a piece of every tile is empty on average
    const int cut = tiles - whole;
    const auto length = [&](int blocks) {
      return max((int)min(units * __builtin_amdgcn_rcpf((float)max(blocks - cut / 2, blocks / 2)) + 1.f, 1e9f), kLeast);
    };
    per = length(a.slots);
    if (!kAll) {
      const int mean = (int)min(units * __builtin_amdgcn_rcpf((float)cut) + 1.f, 1e9f);
      per = best_length(mean, longest, cut, a.slots, per, length(2 * a.slots));
    }
  }

  __device__ __forceinline__ void set(Work &w, int in, int piece, int parts) const {
    const int row_tiles = (w.s.rows + BQ - 1) / BQ, units = units_of(w.s);
    w.head = (unsigned)in / (unsigned)row_tiles;
    w.tile = in - w.head * row_tiles;
    w.parts = parts;
    w.unit0 = parts > 1 ? piece * per : 0;
    w.unit1 = parts > 1 ? min(units, w.unit0 + per) : units;
  }

  // What tile t (of all, t >= 0), or piece b of the cut ones (t < 0), is of; false if there is none.
  // Of a tile all its pieces, with the first one's slot.
  __device__ __forceinline__ bool find(int t, int b, Work &w) {
    // offsets that decrease may ask for more tiles and pieces than there is room for
    if (t < 0 && (b < 0 || b >= a.pieces)) return false;
    if (a.samples == 1) {
      w.s = mine;
      const int parts = parts_of(mine);
      if (t >= 0) {
        if (t >= tiles) return false;
        set(w, t, 0, 1);
        w.parts = t >= whole ? parts : 1;
        w.slot = w.parts > 1 ? (t - whole) * parts : -1;
      } else {
        const int in = whole + (unsigned)b / (unsigned)parts;
        if (in >= tiles) return false;
        set(w, in, b - (in - whole) * parts, parts);
        w.slot = parts > 1 ? b : -1;
      }
    } else {
      int first = 0, pieces = 0, found = 0;
      each([&](const Sample &x) {
        const int n = tiles_of(a, x), incl = scan(n), begin = first + incl - n;
        const int cut = cut_of(begin, n), parts = parts_of(x);
        const int all = (int)min((int64_t)cut * parts, (int64_t)kMostBlocks);
        const int pincl = scan(all), pbegin = pieces + pincl - all;
        const uint64_t who = __ballot(t >= 0 ? t >= begin && t < begin + n : b >= pbegin && b < pbegin + all);
        if (who) {
          const int l = __builtin_ctzll(who);
          const int nl = lane_of(n, l), cl = lane_of(cut, l), np = lane_of(parts, l), pl = lane_of(pbegin, l);
          w.s = {lane_of(x.q0, l), lane_of(x.k0, l), lane_of(x.rows, l), lane_of(x.keys, l)};
          if (t >= 0) {
            const int in = t - lane_of(begin, l);
            set(w, in, 0, 1);
            w.parts = in >= nl - cl ? np : 1;
            w.slot = w.parts > 1 ? pl + (in - (nl - cl)) * np : -1;
          } else {
            const int in = (unsigned)(b - pl) / (unsigned)np;
            set(w, nl - cl + in, b - pl - in * np, np);
            w.slot = np > 1 ? b : -1;
          }
          found = 1;
          return true;
        }
        first = min(first + lane_of(incl, 63), kMostBlocks);
        pieces = min(pieces + lane_of(pincl, 63), kMostBlocks);
        return false;
      });
      if (!__builtin_amdgcn_readfirstlane(found)) return false;
    }
    return w.slot < 0 || w.slot + (t >= 0 ? w.parts : 1) <= a.pieces;
  }
};

// Consecutive logical blocks on one XCD, for any number of blocks.
__device__ __forceinline__ int xcd_order(int b, int n) {
  const int x = b & 7, each = n >> 3, more = n & 7;
  return x * each + min(x, more) + (b >> 3);
}

// ------------------------------------------------------------------ the products

// fp32 accumulators of 32 x 32 MFMAs: column lane & 31, register r row
// 8 (r / 4) + 4 (lane / 32) + r % 4.
__device__ __forceinline__ constexpr int acc_row(int r) { return (r >> 2) * 8 + (r & 3); }

template <int DP, int NQ>
struct Queries {
  bf16x8 q[NQ][DP / 16];     // Q^T: lane's query, 8 values at 16 i + 8 (lane / 32)
  float m[NQ], l[NQ];        // maximum followed (in powers of two), sum of this half's weights
};
template <int DP>
struct State : Queries<DP, 1> {
  f32x16 o[DP / 32];         // O^T
};

// Row r of a sample's rows: query r / group, head r % group of the key head's.
__device__ __forceinline__ int query_of(const AttentionArgs &a, int r) { return a.group == 1 ? r : (unsigned)r / (unsigned)a.group; }

// Query rows r0 + 32 i + (lane & 31) of a tile into registers; zeros past the rows and past D.
template <int DP, int NQ>
__device__ __forceinline__ void load_q(const AttentionArgs &a, const Work &w, int r0, Queries<DP, NQ> &st) {
  const int lane = threadIdx.x & 63, m0 = query_of(a, r0);
  const uint16_t *const p = a.q + (int64_t)(w.s.q0 + m0) * a.q_ld + (int64_t)w.head * a.group * a.D;
  // 64 rows of a pitch of at most 2^22 values lie within the buffer
  const auto rows = make_rsrc(uniform(p), 0, 0x7FFFFFFF);
#pragma unroll
  for (int i = 0; i < NQ; ++i) {
    const int r = r0 + 32 * i + (lane & 31), m = query_of(a, r);
    const uint32_t at = r < w.s.rows ? (uint32_t)((m - m0) * a.q_ld + (r - m * a.group) * a.D + 8 * (lane >> 5)) * 2 : kOut;
#pragma unroll
    for (int j = 0; j < DP / 16; ++j) {
      const int d = 16 * j + 8 * (lane >> 5);
      st.q[i][j] = as_bf16x8(__builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rows, (int)(d < a.D ? at + 32 * j : kOut), 0, 0)));
    }
    st.m[i] = kLowest;
    st.l[i] = 0.f;
  }
}

// Up to 64 rows of K or V of one key head of a sample, from the sample's key `first` on; what is past them reads as zeros.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const AttentionArgs &a, const uint16_t *x, int64_t ld,
                                                          const Work &w, int first) {
  const int rows = min(w.s.keys - first, 64);
  const uint16_t *p = x + (int64_t)(w.s.k0 + first) * ld + (int64_t)w.head * a.D;
  return make_rsrc(p, 0, rows <= 0 ? 0 : ((rows - 1) * (int)ld + a.D) * 2);
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
  return j < w.s.keys ? a.key_mask[(int64_t)w.s.k0 + j] : 0;
}

// Partial sums of a tile: [DP / 4][rows][4] outputs, then the maxima, then the sums, fp32.
template <int DP, int BQ> __device__ __forceinline__ float *slot_at(const AttentionArgs &a, int slot) {
  return a.partial + slot * (int64_t)(BQ * (DP + 2));
}

__device__ __forceinline__ uint16_t *out_row(const AttentionArgs &a, const Work &w, int r) {
  const int m = query_of(a, r);
  return a.out + (int64_t)(w.s.q0 + m) * a.out_ld + (int64_t)(w.head * a.group + r - m * a.group) * a.D;
}

// 1 / the sum of a query's weights; 0 for a query without a score (its maximum is still the lowest). Scores from some
// 2^31 on, whose maximum is rounded to multiples of 2^8, can have all weights vanish: that is no zero, but NaN.
__device__ __forceinline__ float reciprocal(float l, float m) {
  return l != 0.f ? 1.f / l : m == kLowest ? 0.f : __builtin_nanf("");
}

// ------------------------------------------------------------------ tiles of many rows

// Bytes of a wave's LDS reads: where a lane finds its part of fragment j of 32
// K rows (16 bytes) and of V^T (twice eight bytes). The unit of a row moves in
// bits that repeat every four (two) fragments, so that few bases and constant
// offsets serve all of them.
template <int DP>
struct Lanes {
  static constexpr int kRow = lds_width(DP) * 2;
  int k[4], v[2];

  __device__ __forceinline__ Lanes() {
    const int lane = threadIdx.x & 63, h = lane >> 5, row = lane & 31;
#pragma unroll
    for (int j = 0; j < 4; ++j) k[j] = row * kRow + k_unit(row, 2 * j + h) * 16;
    const int vrow = 4 * h + ((lane & 15) >> 2), unit = ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1);
#pragma unroll
    for (int j = 0; j < 2; ++j) v[j] = vrow * kRow + v_unit(vrow, unit + 4 * j) * 16 + (lane & 1) * 8;
  }
  // 16 values of K's row at 16 j, of the 32 rows at kb
  __device__ __forceinline__ bf16x8 k_frag(const unsigned char *kb, int j) const {
    return lds_read8(kb + k[j & 3] + (j >> 2) * 128);
  }
  // V^T's rows 32 (f % (DP / 32)), of 16 of the 32 keys at vb
  __device__ __forceinline__ bf16x8 v_frag(const unsigned char *vb, int f) const {
    const int t = f / (DP / 32), j = f % (DP / 32);
    const unsigned char *p = vb + v[j & 1] + (16 * t * kRow + (j >> 1) * 128);
    const s16x4 lo = lds_read_tr(p), hi = lds_read_tr(p + 8 * kRow);
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
  }
};

// Accumulators of attention_kernel: tile n (32 values of 32 queries) is in the
// AGPRs a[16 n .. 16 n + 15], named in the instructions themselves. With 64
// queries of 256 values they are all 256 AGPRs of a wave that has a SIMD's
// registers to itself; held as variables, every branch that they live across
// would need free ones to move them through, and the compiler sends hundreds
// of them through scratch memory instead. Nothing else in the kernel uses
// AGPRs: the scores' products are built into VGPRs, and the clobbers keep the
// compiler's own values out (tests/test_qk_attention_host.py looks through the
// assembly for any other use).
#define QL_D(n) "a" #n "0", "a" #n "1", "a" #n "2", "a" #n "3", "a" #n "4", "a" #n "5", "a" #n "6", "a" #n "7", "a" #n "8", "a" #n "9"
#define QL_ACC64 "a0", "a1", "a2", "a3", "a4", "a5", "a6", "a7", "a8", "a9", QL_D(1), QL_D(2), QL_D(3), QL_D(4), QL_D(5), \
    "a60", "a61", "a62", "a63"
#define QL_ACC128 QL_ACC64, "a64", "a65", "a66", "a67", "a68", "a69", QL_D(7), QL_D(8), QL_D(9), QL_D(10), QL_D(11), "a120", \
    "a121", "a122", "a123", "a124", "a125", "a126", "a127"
#define QL_ACC256 QL_ACC128, "a128", "a129", QL_D(13), QL_D(14), QL_D(15), QL_D(16), QL_D(17), QL_D(18), QL_D(19), QL_D(20), \
    QL_D(21), QL_D(22), QL_D(23), QL_D(24), "a250", "a251", "a252", "a253", "a254", "a255"
// An instruction on the accumulators of a kernel of TILES tiles.
#define QL_ACC_ASM(TILES, ...)                                        \
  if constexpr ((TILES) <= 4) asm volatile(__VA_ARGS__ : QL_ACC64);   \
  else if constexpr ((TILES) <= 8) asm volatile(__VA_ARGS__ : QL_ACC128); \
  else asm volatile(__VA_ARGS__ : QL_ACC256)

template <int TILES>
struct Acc {
  // Waits before an accumulator is read or written by anything but a product: 24 states, more than any product asks for.
  static __device__ __forceinline__ void settle() { QL_ACC_ASM(TILES, "s_nop 15\n\ts_nop 7" : :); }

  // Tile N += a b. The wait covers an operand that a VALU instruction wrote just before.
  template <int N> static __device__ __forceinline__ void mfma(bf16x8 a, bf16x8 b) {
    QL_ACC_ASM(TILES, "s_nop 1\n\tv_mfma_f32_32x32x16_bf16 a[%2:%3], %0, %1, a[%2:%3]"
               : : "v"(a), "v"(b), "n"(16 * N), "n"(16 * N + 15));
  }
  template <int R = 0> static __device__ __forceinline__ void clear() {
    if constexpr (R < 16 * TILES) {
      QL_ACC_ASM(TILES, "v_accvgpr_write_b32 a[%0], 0\n\tv_accvgpr_write_b32 a[%1], 0\n\tv_accvgpr_write_b32 a[%2], 0\n\t"
                 "v_accvgpr_write_b32 a[%3], 0" : : "n"(R), "n"(R + 1), "n"(R + 2), "n"(R + 3));
      clear<R + 4>();
    }
  }
  // Four values of tile N, from register R on. The waits: settle() first.
  template <int N, int R> static __device__ __forceinline__ f32x4 get() {
    float a, b, c, d;
    QL_ACC_ASM(TILES, "v_accvgpr_read_b32 %0, a[%4]\n\tv_accvgpr_read_b32 %1, a[%5]\n\tv_accvgpr_read_b32 %2, a[%6]\n\t"
               "v_accvgpr_read_b32 %3, a[%7]" : "=v"(a), "=v"(b), "=v"(c), "=v"(d)
               : "n"(16 * N + R), "n"(16 * N + R + 1), "n"(16 * N + R + 2), "n"(16 * N + R + 3));
    return f32x4{a, b, c, d};
  }
  // Tiles FIRST .. LAST - 1 times f. settle() first; the wait at the end is for the next product.
  template <int FIRST, int LAST> static __device__ __forceinline__ void scale(float f) {
    if constexpr (FIRST < LAST) {
      scale4<16 * FIRST>(f);
      scale<FIRST + 1, LAST>(f);
    }
  }
  template <int R> static __device__ __forceinline__ void scale4(float f) {
    float a, b, c, d;
    QL_ACC_ASM(TILES, "v_accvgpr_read_b32 %0, a[%5]\n\tv_accvgpr_read_b32 %1, a[%6]\n\tv_accvgpr_read_b32 %2, a[%7]\n\t"
               "v_accvgpr_read_b32 %3, a[%8]\n\tv_mul_f32 %0, %0, %4\n\tv_mul_f32 %1, %1, %4\n\tv_mul_f32 %2, %2, %4\n\t"
               "v_mul_f32 %3, %3, %4\n\tv_accvgpr_write_b32 a[%5], %0\n\tv_accvgpr_write_b32 a[%6], %1\n\t"
               "v_accvgpr_write_b32 a[%7], %2\n\tv_accvgpr_write_b32 a[%8], %3\n\ts_nop 1"
               : "=&v"(a), "=&v"(b), "=&v"(c), "=&v"(d) : "v"(f), "n"(R), "n"(R + 1), "n"(R + 2), "n"(R + 3));
    if constexpr (R % 16 != 12) scale4<R + 4>(f);
  }
};

template <int N> struct Count { static constexpr int value = N; };

// f(Count<0>), ..., f(Count<N - 1>): accumulators are named by constants.
template <int... I, typename F>
__device__ __forceinline__ void constants(std::integer_sequence<int, I...>, F f) { (f(Count<I>{}), ...); }
template <int N, typename F>
__device__ __forceinline__ void constants(F f) { constants(std::make_integer_sequence<int, N>{}, f); }

// A block of four waves, 32 NQ rows each, over keys in chunks of 32 that all
// waves read from LDS.
//
// While the scores of chunk i + 1 are multiplied, those of chunk i become
// weights between the MFMAs; while these meet V, the next maximum is taken.
//
// 2 D multiply-adds per row and key: a wave's 32 rows and 32 keys of 256 values
// are 32 MFMAs of 32 cycles and 32 KB of K and V read from LDS, so the matrix
// unit bounds it, and the card's power with it: 16896
// tokens of 18 heads of 256 take 4.2 to 4.5 ms (1170 to 1240 TFLOP/s) with the
// unit busy in 54 % of the cycles of a clock that falls to 2.0 GHz; without the
// exponentials the loop reaches 1099 TFLOP/s where it was at 1051, without the
// softmax 1243, with the MFMAs alone 1315; a library product of 8192^3 1200 to
// 1340. 4608 tokens: 361 to 376 us, 19 of them the join of the last tiles.
// 64 rows per wave (NQ = 2) read LDS half as often for the same products; with
// 32 and without the order below the large call took 7.6 ms. Copies go from
// memory to LDS without registers, and two chunks ahead: all but the newest
// batch are waited for, never all.
template <int DP, int NQ, bool MASKED>
__global__ __launch_bounds__(256, 1) void attention_kernel(AttentionArgs a) {
  constexpr int kRow = lds_width(DP) * 2, BQ = 128 * NQ, UNIT = 64, kBytes = UNIT * kRow, kHalf = kBytes / 2;
  constexpr int kUnits = kRow / 16;             // 16-byte units of a row
  constexpr int kCopies = UNIT * kUnits / 256;  // copies of 64 units per wave and stage
  constexpr int kSteps = DP / 16, kFrags = DP / 16;
  __shared__ __attribute__((aligned(16))) unsigned char k0[kBytes], k1[kBytes], v0[kBytes], v1[kBytes];
  Division<BQ, UNIT> division(a);
  Work w;
  const int block = blockIdx.x, whole = a.rest_from ? a.rest_from : division.whole;
  if (!division.find(block >= whole ? -1 : whole < kMostBlocks ? xcd_order(block, whole) : block, block - whole, w)) return;
  w = uniform(w);
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63, h = lane >> 5;
  const int r0 = w.tile * BQ + wave * 32 * NQ;
  using O = Acc<NQ * DP / 32>;
  constexpr int kTiles = DP / 32;  // of a query block
  Queries<DP, NQ> st;
  const float c = __uint_as_float(uniform((int)__float_as_uint(a.scale * 1.4426950408889634f)));
  const Lanes<DP> at;

  // Copy i of this wave: unit (4 i + wave) * 64 + lane of the stage. Every kKinds
  // copies (one, or three of rows of 24 units) the units of a lane come again,
  // kRows rows on, a multiple of 8.
  constexpr int kKinds = kUnits == 24 ? 3 : 1, kRows = kKinds * 256 / kUnits;
  int row[kKinds];
  uint32_t kofs[kKinds], vofs[kKinds];
#pragma unroll
  for (int b = 0; b < kKinds; ++b) {
    const int id = (4 * b + wave) * 64 + lane;
    row[b] = id / kUnits;
    const int kc = k_unit(row[b], id % kUnits), vc = v_unit(row[b], id % kUnits);
    kofs[b] = kc * 8 < a.D ? (uint32_t)(row[b] * a.k_ld + kc * 8) * 2 : kOut;
    vofs[b] = vc * 8 < a.D ? (uint32_t)(row[b] * a.v_ld + vc * 8) * 2 : kOut;
  }
  const int first = w.unit0 * UNIT, end = min(w.unit1 * UNIT, w.s.keys);
  // The copies of one stage of K or V, requested one at a time.
  struct Copies {
    __amdgpu_buffer_rsrc_t rows;
    uint32_t ofs[kKinds], step;
    unsigned char *to;
    uint64_t keep;
    int row[kKinds];
    __device__ __forceinline__ void one(int i) {
      const int b = i % kKinds;
      dma16(rows, !MASKED || (keep >> (row[b] + i / kKinds * kRows) & 1) ? ofs[b] : kOut, 0, to + i * 4096);
      ofs[b] += step;
    }
    __device__ __forceinline__ void all() {
#pragma unroll
      for (int i = 0; i < kCopies; ++i) one(i);
    }
  };
  auto copies = [&](const uint16_t *x, int64_t ld, const uint32_t (&ofs)[kKinds], unsigned char *to, int from, uint64_t keep)
      __attribute__((always_inline)) {
    Copies c = {rows_of(a, x, ld, w, from), {}, (uint32_t)(kRows * ld * 2), to + wave * 1024, keep, {}};
#pragma unroll
    for (int b = 0; b < kKinds; ++b) {
      c.ofs[b] = ofs[b];
      c.row[b] = row[b];
      asm volatile("" : "+v"(c.ofs[b]));  // or every copy's offset is kept in a register over the loop
    }
    return c;
  };
  // Kept keys of the stages in hand; a stage's bytes of the mask are requested two stages ahead.
  uint64_t keep = 0, keep1 = 0;
  int byte = 0;
  auto next_keep = [&](int from) __attribute__((always_inline)) {
    const uint64_t k = kept<MASKED>(a, w, from, byte);
    if constexpr (MASKED) byte = mask_byte(a, w, from + UNIT);
    return k;
  };

  f32x16 s[2][NQ];
  // The maximum of a chunk's scores is followed if it has grown by more than the slack, each query's by its own alone.
  auto follow = [&](float (&mx)[NQ]) __attribute__((always_inline)) {
    bool grown = false;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      mx[i] = fmaxf(mx[i], other_half(mx[i])) * c;
      grown |= mx[i] > st.m[i] + kSlack;
    }
    if (!__any(grown)) return;
    O::settle();
    float f[NQ];
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const float m = mx[i] > st.m[i] + kSlack ? mx[i] : st.m[i];
      f[i] = __builtin_amdgcn_exp2f(st.m[i] - m);
      st.m[i] = m;
      st.l[i] *= f[i];
    }
    O::template scale<0, kTiles>(f[0]);
    if constexpr (NQ == 2) O::template scale<kTiles, 2 * kTiles>(f[1]);
  };
  auto hide = [&](f32x16 (&x)[NQ], uint32_t valid) __attribute__((always_inline)) {
    if (valid == 0xFFFFFFFFu) return;
    const uint32_t mine = valid >> (4 * h);
#pragma unroll
    for (int r = 0; r < 16; ++r)
#pragma unroll
      for (int i = 0; i < NQ; ++i) x[i][r] = (mine >> acc_row(r)) & 1 ? x[i][r] : -__builtin_inff();
  };
  auto scores_of = [&](const unsigned char *kb, f32x16 (&x)[NQ]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NQ; ++i) x[i] = f32x16{};
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      const bf16x8 k = at.k_frag(kb, j);
#pragma unroll
      for (int i = 0; i < NQ; ++i) x[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k, st.q[i][j], x[i], 0, 0, 0);
    }
  };
  auto largest = [&](f32x16 (&x)[NQ], float (&mx)[NQ]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      mx[i] = x[i][0];
#pragma unroll
      for (int r = 1; r < 16; ++r) mx[i] = fmaxf(mx[i], x[i][r]);
    }
  };

  // One chunk: its scores `x` meet V's rows at vb; meanwhile the next chunk's
  // become y (K rows at kb, kept keys `valid`) and `c2` is requested. An MFMA
  // keeps the matrix unit for 32 cycles: after each one goes what the vector
  // unit can do meanwhile, in this order and no other.
  auto chunk = [&](const unsigned char *kb, const unsigned char *vb, f32x16 (&x)[NQ], f32x16 (&y)[NQ], uint32_t valid, Copies c2)
      __attribute__((always_inline)) {
    uint32_t p[NQ][8];
    float e0 = 0.f, e1 = 0.f, sum = 0.f;
    // half n of the 16 NQ: the exponents and the first power of two weights, then the second and their sum. A chunk's
    // weights are added up by themselves before they meet the sum so far, which so takes no more additions than the outputs.
    auto half = [&](int n) __attribute__((always_inline)) {
      const int i = n / 16, r = n % 16 / 2 * 2;
      if (n % 2 == 0) {
        e0 = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i][r], c, -st.m[i]));
        e1 = __builtin_fmaf(x[i][r + 1], c, -st.m[i]);
      } else {
        p[i][r / 2] = pack_bf16(e0, __builtin_amdgcn_exp2f(e1));
        const bf16x2 one = {(__bf16)1.f, (__bf16)1.f};
        sum = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, p[i][r / 2]), one, r == 0 ? 0.f : sum, false);
        asm volatile("" : "+v"(p[i][r / 2]), "+v"(sum));
        if (r == 14) st.l[i] += sum;
      }
    };
    bf16x8 kf[3];
    kf[0] = at.k_frag(kb, 0);
    kf[1] = at.k_frag(kb, 1);
#pragma unroll
    for (int i = 0; i < NQ; ++i) y[i] = f32x16{};
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int n = 0; n < kSteps * NQ; ++n) {
      const int j = n / NQ, i = n % NQ;
      if (i == 0 && j + 2 < kSteps) kf[(j + 2) % 3] = at.k_frag(kb, j + 2);
      y[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[j % 3], st.q[i][j], y[i], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < (16 + kSteps - 1) / kSteps; ++u)
        if (n * 16 / kSteps + u < (n + 1) * 16 / kSteps) half(n * 16 / kSteps + u);
      if (i == NQ - 1 && j * kCopies / kSteps < (j + 1) * kCopies / kSteps) c2.one(j * kCopies / kSteps);
      __builtin_amdgcn_sched_barrier(0);
    }
    hide(y, valid);
    bf16x8 vf[3];
    vf[0] = at.v_frag(vb, 0);
    vf[1] = at.v_frag(vb, 1);
    float mx[NQ];
    __builtin_amdgcn_sched_barrier(0);
    constants<kFrags * NQ>([&](auto count) __attribute__((always_inline)) {
      constexpr int n = decltype(count)::value, f = n / NQ, i = n % NQ, t = f / kTiles, j = f % kTiles;
      if constexpr (i == 0 && f + 2 < kFrags) vf[(f + 2) % 3] = at.v_frag(vb, f + 2);
      O::template mfma<i * kTiles + j>(vf[f % 3], as_bf16x8(u32x4{p[i][4 * t], p[i][4 * t + 1], p[i][4 * t + 2], p[i][4 * t + 3]}));
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int r = f * 16 / kFrags; r < (f + 1) * 16 / kFrags; ++r) mx[i] = r ? fmaxf(mx[i], y[i][r]) : y[i][0];
      __builtin_amdgcn_sched_barrier(0);
    });
    follow(mx);
  };
  // All but the `ahead` newest of this wave's copies have landed, and so have the other waves'.
  auto landed = [&](auto ahead) __attribute__((always_inline)) {
    constexpr int n = decltype(ahead)::value;
    __builtin_amdgcn_s_waitcnt((n & 0xF) | ((n >> 4) << 14) | 0xF70);
    __syncthreads();
  };

  if (first < end) {
    if constexpr (MASKED) byte = mask_byte(a, w, first);
    keep = next_keep(first);
    keep1 = next_keep(first + UNIT);
    copies(a.k, a.k_ld, kofs, k0, first, keep).all();
    load_q<DP, NQ>(a, w, r0, st);
    copies(a.v, a.v_ld, vofs, v0, first, keep).all();
    copies(a.k, a.k_ld, kofs, k1, first + UNIT, keep1).all();
    O::clear();
    __builtin_amdgcn_s_waitcnt(((2 * kCopies) & 0xF) | (((2 * kCopies) >> 4) << 14) | 0xF70);
    __syncthreads();
    scores_of(k0, s[0]);
    hide(s[0], (uint32_t)keep);
    float mx[NQ];
    largest(s[0], mx);
    follow(mx);
    // Chunks 2 j and 2 j + 1 are stage j. Copies are requested two chunks before their first use: V of stage j + 1
    // at chunk 2 j, K of stage j + 2 at chunk 2 j + 1. What is past the end is requested too (and nothing is read
    // for it), so that the same number of copies is always on the way.
    auto even = [&](unsigned char *kb, unsigned char *vb, unsigned char *vn, int from) __attribute__((always_inline)) {
      landed(Count<kCopies>{});
      chunk(kb + kHalf, vb, s[0], s[1], (uint32_t)(keep >> 32), copies(a.v, a.v_ld, vofs, vn, from + UNIT, keep1));
    };
    auto odd = [&](unsigned char *kb, unsigned char *vb, unsigned char *kn, int from) __attribute__((always_inline)) {
      landed(Count<kCopies>{});
      keep = keep1;
      keep1 = next_keep(from + 2 * UNIT);
      chunk(kn, vb + kHalf, s[1], s[0], (uint32_t)keep, copies(a.k, a.k_ld, kofs, kb, from + 2 * UNIT, keep1));
    };
    for (int from = first;; from += 2 * UNIT) {
      even(k0, v0, v1, from);
      if (from + 32 >= end) break;
      odd(k0, v0, k1, from);
      if (from + 64 >= end) break;
      even(k1, v1, v0, from + UNIT);
      if (from + 96 >= end) break;
      odd(k1, v1, k0, from + UNIT);
      if (from + 128 >= end) break;
    }
    landed(Count<0>{});  // what was requested past the end, before the stages are used again
  } else {
    O::clear();
#pragma unroll
    for (int i = 0; i < NQ; ++i) st.m[i] = kLowest, st.l[i] = 0.f;
  }
  if (r0 >= w.s.rows) return;
  O::settle();
  if (w.slot >= 0) {
    float *const part = slot_at<DP, BQ>(a, w.slot);
    constants<NQ>([&](auto block) __attribute__((always_inline)) {
      constexpr int i = decltype(block)::value;
      const int rt = wave * 32 * NQ + 32 * i + (lane & 31);
      const float l = st.l[i] + other_half(st.l[i]);
      // four values of 8 g + 4 h on of each 32: of the 32 queries side by side
      constants<4 * kTiles>([&](auto four) __attribute__((always_inline)) {
        constexpr int j = decltype(four)::value / 4, g = decltype(four)::value % 4;
        *reinterpret_cast<f32x4 *>(part + ((8 * j + 2 * g + h) * BQ + rt) * 4) = O::template get<i * kTiles + j, 4 * g>();
      });
      if (h == 0) {
        part[BQ * DP + rt] = st.m[i];
        part[BQ * (DP + 1) + rt] = l;
      }
    });
    return;
  }
  // Whole rows leave through the wave's quarter of LDS (a lane holds every
  // eighth four values of a row: stored as they are, a call of 512 keys spends
  // a fifth of its time on it). Units of 16 bytes are moved by the row.
  unsigned char *const rows = wave == 0 ? k0 : wave == 1 ? k1 : wave == 2 ? v0 : v1;
  constants<NQ>([&](auto block) __attribute__((always_inline)) {
    constexpr int i = decltype(block)::value;
    const float f = reciprocal(st.l[i] + other_half(st.l[i]), st.m[i]);
    const int q = 32 * i + (lane & 31);
    constants<4 * kTiles>([&](auto four) __attribute__((always_inline)) {
      constexpr int j = decltype(four)::value / 4, g = decltype(four)::value % 4;
      const f32x4 v = O::template get<i * kTiles + j, 4 * g>();
      *reinterpret_cast<u32x2 *>(rows + q * kRow + ((4 * j + g) ^ (q & 7)) * 16 + h * 8) =
          u32x2{pack_bf16(v[0] * f, v[1] * f), pack_bf16(v[2] * f, v[3] * f)};
    });
  });
#pragma unroll 4
  for (int n = 0; n < 32 * NQ * kUnits / 64; ++n) {
    const int q = (n * 64 + lane) / kUnits, u = (n * 64 + lane) % kUnits;
    const u32x4 v = *reinterpret_cast<const u32x4 *>(rows + q * kRow + (u ^ (q & 7)) * 16);
    if (r0 + q < w.s.rows && u * 8 < a.D) *reinterpret_cast<u32x4 *>(out_row(a, w, r0 + q) + u * 8) = v;
  }
}

// ------------------------------------------------------------------ tiles of few rows

// What a wave of few rows does with 32 keys: S^T of those whose K rows are at kb,
template <int DP>
__device__ __forceinline__ f32x16 scores(const Lanes<DP> &at, const unsigned char *kb, const State<DP> &st) {
  f32x16 s = {};
#pragma unroll
  for (int j = 0; j < DP / 16; ++j) s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(at.k_frag(kb, j), st.q[0][j], s, 0, 0, 0);
  return s;
}

// weights of these scores, none for keys whose bit in `valid` is clear; the
// maximum, the sum and, where the maximum is followed, the output so far are
// brought up to date,
template <int DP>
__device__ __forceinline__ void weights(State<DP> &st, f32x16 s, float c, uint32_t valid, bf16x8 (&p)[2]) {
  const int h = (threadIdx.x >> 5) & 1;
  if (valid != 0xFFFFFFFFu) {
    const uint32_t mine = valid >> (4 * h);
#pragma unroll
    for (int r = 0; r < 16; ++r) s[r] = (mine >> acc_row(r)) & 1 ? s[r] : -__builtin_inff();
  }
  float mx = s[0];
#pragma unroll
  for (int r = 1; r < 16; ++r) mx = fmaxf(mx, s[r]);
  mx = fmaxf(mx, other_half(mx)) * c;
  const bool grown = mx > st.m[0] + kSlack;
  if (__any(grown)) {
    // each query by its own scores alone
    const float m = grown ? mx : st.m[0], f = __builtin_amdgcn_exp2f(st.m[0] - m);
    st.m[0] = m;
    st.l[0] *= f;
#pragma unroll
    for (int j = 0; j < DP / 32; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) st.o[j][r] *= f;
  }
  uint32_t w[8];
#pragma unroll
  for (int r = 0; r < 16; r += 2) {
    const float a = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r], c, -st.m[0]));
    const float b = __builtin_amdgcn_exp2f(__builtin_fmaf(s[r + 1], c, -st.m[0]));
    w[r / 2] = pack_bf16(a, b);
  }
  float sum = 0.f;  // of these keys alone first: the sum so far takes no more additions than the outputs
#pragma unroll
  for (int r = 0; r < 8; ++r) sum += bf16_lo(w[r]) + bf16_hi(w[r]);
  st.l[0] += sum;
  p[0] = as_bf16x8(u32x4{w[0], w[1], w[2], w[3]});
  p[1] = as_bf16x8(u32x4{w[4], w[5], w[6], w[7]});
}

// and O^T += V^T P^T over the V rows at vb.
template <int DP>
__device__ __forceinline__ void outputs(const Lanes<DP> &at, const unsigned char *vb, State<DP> &st, const bf16x8 (&p)[2]) {
  constexpr int kTiles = DP / 32;
#pragma unroll
  for (int f = 0; f < 2 * kTiles; ++f)
    st.o[f % kTiles] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(at.v_frag(vb, f), p[f / kTiles], st.o[f % kTiles], 0, 0, 0);
}

// 32 rows at most: the four waves of a block share them and take every fourth
// tile of 32 keys each, through LDS of their own, without a barrier until
// their sums are joined at the end. REST: the rows of a few tiles that the
// kernel above left, 32 to a block.
//
// Bound by the bytes of K and V where many blocks run (16 queries over 65536
// keys of 8 heads of 128: 56 us, 4.8 TB/s, and 6 for the join), and by what one
// CU has on its way where few do: 128 KB of LDS, so 18 blocks of one query over
// 512 keys of 256 (512 KB each) take 12 us of which 3.4 are the launch.
template <int DP, bool MASKED, bool REST>
__global__ __launch_bounds__(256, 1) void attention_few_kernel(AttentionArgs a) {
  constexpr int kRow = lds_width(DP) * 2, BQ = 32, UNIT = 128, kBytes = 32 * kRow, kUnits = kRow / 16;
  constexpr int kCopies = 32 * kUnits / 64, kTiles = lds_width(DP) / 64;  // tiles of 32 values that K's place holds
  __shared__ __attribute__((aligned(16))) unsigned char ks[4 * kBytes], vs[4 * kBytes];
  __shared__ float ms[4][32], ls[4][32];
  Work w;
  if constexpr (REST) {
    Division<256, 64> division(a);
    if (!division.find(a.rest_from + (int)blockIdx.x / 8, 0, w)) return;
    w = uniform(w);
    w.tile = w.tile * 8 + (int)blockIdx.x % 8;
    if (w.tile * BQ >= w.s.rows) return;
  } else {
    Division<BQ, UNIT> division(a);
    const int block = blockIdx.x, whole = division.whole;
    if (!division.find(block < whole ? block : -1, block - whole, w)) return;
    w = uniform(w);
  }
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  State<DP> st;
  const Lanes<DP> lanes;
  // units are of 64 keys in the kernel above
  const int end = REST ? w.s.keys : min(w.unit1 * UNIT, w.s.keys);
  const float c = __uint_as_float(uniform((int)__float_as_uint(a.scale * 1.4426950408889634f)));
  unsigned char *const kb = ks + wave * kBytes, *const vb = vs + wave * kBytes;
  // copy i of the wave: unit 64 i + lane of its tile
  auto copy = [&](const uint16_t *x, int64_t ld, bool is_k, unsigned char *to, int at, uint32_t keep) {
    const auto r = rows_of(a, x, ld, w, at);
#pragma unroll
    for (int i = 0; i < kCopies; ++i) {
      const int id = 64 * i + lane, row = id / kUnits;
      const int u = is_k ? k_unit(row, id % kUnits) : v_unit(row, id % kUnits);
      const bool in = u * 8 < a.D && (!MASKED || (keep >> row & 1));
      dma16(r, in ? (uint32_t)(row * ld + u * 8) * 2 : kOut, 0, to + i * 1024);
    }
  };
  int at = REST ? 32 * wave : w.unit0 * UNIT + 32 * wave;
  int byte = 0, byte_next = 0;
  uint32_t keep = 0;
  if (at < end) {
    if constexpr (MASKED) {
      byte = mask_byte(a, w, at);
      byte_next = mask_byte(a, w, at + 128);
    }
    keep = (uint32_t)kept<MASKED>(a, w, at, byte);
    copy(a.k, a.k_ld, true, kb, at, keep);
  }
  load_q<DP, 1>(a, w, w.tile * BQ, st);
#pragma unroll
  for (int j = 0; j < DP / 32; ++j) st.o[j] = f32x16{};
  if (at < end) {
    copy(a.v, a.v_ld, false, vb, at, keep);
    for (; at < end; at += 128) {
      // K of the next tile is requested behind this one's scores and V behind its outputs, always, so that what
      // has landed can be counted
      const uint32_t keep_next = (uint32_t)kept<MASKED>(a, w, at + 128, byte_next);
      bf16x8 p[2];
      __builtin_amdgcn_s_waitcnt((kCopies & 0xF) | ((kCopies >> 4) << 14) | 0xF70);  // all but V
      asm volatile("" ::: "memory");
      const f32x16 s = scores(lanes, kb, st);
      // the reads of K are back before its place is filled again
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if constexpr (MASKED) byte_next = mask_byte(a, w, at + 256);
      copy(a.k, a.k_ld, true, kb, at + 128, keep_next);
      weights(st, s, c, keep, p);
      __builtin_amdgcn_s_waitcnt((kCopies & 0xF) | ((kCopies >> 4) << 14) | 0xF70);  // all but the next K
      asm volatile("" ::: "memory");
      outputs(lanes, vb, st, p);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      copy(a.v, a.v_ld, false, vb, at + 128, keep_next);
      keep = keep_next;
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // what was requested past the end
  }
  // Joined through the waves' own LDS: the first half of the outputs in K's place, the second in V's.
  const int h = lane >> 5, col = lane & 31;
  const float l = st.l[0] + other_half(st.l[0]);
#pragma unroll
  for (int j = 0; j < DP / 32; ++j) {
    f32x4 *const to = reinterpret_cast<f32x4 *>(j < kTiles ? kb : vb);
#pragma unroll
    for (int g = 0; g < 4; ++g)
      to[(8 * (j % kTiles) + 2 * g + h) * 32 + col] =
          f32x4{st.o[j][4 * g], st.o[j][4 * g + 1], st.o[j][4 * g + 2], st.o[j][4 * g + 3]};
  }
  if (h == 0) {
    ms[wave][col] = st.m[0];
    ls[wave][col] = l;
  }
  __syncthreads();
  const int rows = min(w.s.rows - w.tile * BQ, BQ);
  float *const part = w.slot >= 0 ? slot_at<DP, BQ>(a, w.slot) : nullptr;
  for (int n = threadIdx.x; n < rows * (DP / 4); n += 256) {
    const int d4 = (unsigned)n / (unsigned)rows, rt = n - d4 * rows;
    float f[4], m = kLowest, sum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, ms[i][rt]);
    const f32x4 *from = reinterpret_cast<const f32x4 *>(d4 < 8 * kTiles ? ks : vs) + d4 % (8 * kTiles) * 32 + rt;
    f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[i] = __builtin_amdgcn_exp2f(ms[i][rt] - m);
      sum = __builtin_fmaf(ls[i][rt], f[i], sum);
      const f32x4 x = from[i * (kBytes / 16)];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __builtin_fmaf(x[e], f[i], v[e]);
    }
    if (part) {
      *reinterpret_cast<f32x4 *>(part + (d4 * BQ + rt) * 4) = v;
      if (d4 == 0) {
        part[BQ * DP + rt] = m;
        part[BQ * (DP + 1) + rt] = sum;
      }
    } else if (d4 * 4 < a.D) {
      const float inv = reciprocal(sum, m);
      *reinterpret_cast<u32x2 *>(out_row(a, w, w.tile * BQ + rt) + d4 * 4) =
          u32x2{pack_bf16(v[0] * inv, v[1] * inv), pack_bf16(v[2] * inv, v[3] * inv)};
    }
  }
}

// ------------------------------------------------------------------ joining pieces

// The pieces of the cut tiles become outputs. Grid: x cut tiles, y parts of
// their work; a thread has one row at a time and 4 N of its values: 16, and 4
// where there are few rows. Mostly latency, for the pieces come from other
// dies' caches: maxima, sums and values of G pieces are requested together
// (512 pieces of 32 rows of 128 values 5.8 us, one at a time 9.0). Pieces of
// 256 rows are bytes: 492 of them, 130 MB, 35 us, 3.7 TB/s.
template <int BQ> constexpr int kJoin = BQ == 32 ? 1 : 4;

template <int DP, int BQ, int UNIT>
__global__ __launch_bounds__(256) void attention_join_kernel(AttentionArgs a) {
  constexpr int N = kJoin<BQ>, G = N == 1 ? 8 : 4, kSlot = BQ * (DP + 2);
  Division<BQ, UNIT> division(a);
  Work w;
  if (!division.find(division.whole + (int)blockIdx.x, 0, w) || w.slot < 0) return;
  w = uniform(w);
  const int rows = min(w.s.rows - w.tile * BQ, BQ), pieces = w.parts;
  const float *const part = slot_at<DP, BQ>(a, w.slot);
  for (int n = blockIdx.y * 256 + threadIdx.x; n < rows * (DP / (4 * N)); n += 256 * gridDim.y) {
    const int d4 = (unsigned)n / (unsigned)rows * N, rt = n - d4 / N * rows;
    if (d4 * 4 >= a.D) break;
    const float *from = part + (d4 * BQ + rt) * 4, *stats = part + BQ * DP + rt;
    float m = kLowest, sum = 0.f;
    f32x4 v[N] = {};
    for (int i0 = 0; i0 < pieces; i0 += G) {
      float pm[G], pl[G];
      f32x4 x[G][N];
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const int64_t at = (int64_t)(i0 + g) * kSlot;
        const bool in = i0 + g < pieces;
        pm[g] = in ? stats[at] : kLowest;
        pl[g] = in ? stats[at + BQ] : 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j) x[g][j] = in ? *reinterpret_cast<const f32x4 *>(from + at + j * BQ * 4) : f32x4{};
      }
      float top = m;
#pragma unroll
      for (int g = 0; g < G; ++g) top = fmaxf(top, pm[g]);
      const float old = __builtin_amdgcn_exp2f(m - top);
      m = top;
      sum *= old;
#pragma unroll
      for (int j = 0; j < N; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) v[j][e] *= old;
#pragma unroll
      for (int g = 0; g < G; ++g) {
        const float f = __builtin_amdgcn_exp2f(pm[g] - m);
        sum = __builtin_fmaf(pl[g], f, sum);
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) v[j][e] = __builtin_fmaf(x[g][j][e], f, v[j][e]);
      }
    }
    const float inv = reciprocal(sum, m);
    uint16_t *o = out_row(a, w, w.tile * BQ + rt) + d4 * 4;
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (d4 * 4 + j * 4 < a.D)
        *reinterpret_cast<u32x2 *>(o + j * 4) = u32x2{pack_bf16(v[j][0] * inv, v[j][1] * inv), pack_bf16(v[j][2] * inv, v[j][3] * inv)};
  }
}

int padded(int D) { return D <= 64 ? 64 : D <= 96 ? 96 : D <= 128 ? 128 : D <= 192 ? 192 : 256; }

constexpr int kCus = 256;  // MI355X

// Parts of a cut tile's join: at most 256 threads' work each.
template <int DP, int BQ>
constexpr int kJoinParts = BQ * DP / (4 * kJoin<BQ>) > 256 ? BQ * DP / (4 * kJoin<BQ>) / 256 : 1;

template <int DP, int NQ>
void launch_rows(const AttentionArgs &a, const AttentionPlan &p, hipStream_t stream) {
  const dim3 grid((unsigned)p.blocks);
  if (a.key_mask) attention_kernel<DP, NQ, true><<<grid, 256, 0, stream>>>(a);
  else attention_kernel<DP, NQ, false><<<grid, 256, 0, stream>>>(a);
  if (p.cut) attention_join_kernel<DP, 128 * NQ, 64><<<dim3((unsigned)p.cut, kJoinParts<DP, 128 * NQ>), 256, 0, stream>>>(a);
}

template <int DP, bool REST>
void launch_few(const AttentionArgs &a, int64_t blocks, hipStream_t stream) {
  const dim3 grid((unsigned)blocks);
  if (a.key_mask) attention_few_kernel<DP, true, REST><<<grid, 256, 0, stream>>>(a);
  else attention_few_kernel<DP, false, REST><<<grid, 256, 0, stream>>>(a);
}

template <int DP>
void launch_width(const AttentionArgs &a, const AttentionPlan &p, hipStream_t stream) {
  if (p.rows == 32) {
    launch_few<DP, false>(a, p.blocks, stream);
    if (p.cut) attention_join_kernel<DP, 32, 128><<<dim3((unsigned)p.cut, kJoinParts<DP, 32>), 256, 0, stream>>>(a);
  } else if (p.rows == 128) {
    launch_rows<DP, 1>(a, p, stream);
  } else if constexpr (DP != 96 && DP != 128) {
    launch_rows<DP, 2>(a, p, stream);
    if constexpr (DP == 256) {
      if (p.rest) launch_few<DP, true>(a, p.rest * 8, stream);
    }
  }
}

}  // namespace

AttentionPlan attention_plan(int64_t Mq, int64_t Mk, int64_t samples, bool offsets, int q_heads, int kv_heads, int D,
                             bool workspace) {
  AttentionPlan p{};
  const int dp = padded(D);
  const int64_t rows = Mq * (q_heads / kv_heads), several = std::max<int64_t>(samples, 1);
  const int64_t each = rows / several, keys = Mk / several;
  auto tiles_of = [&](int64_t tile) {
    // of all samples at most: whatever the offsets are, one more per sample than without them
    const int64_t run = (rows + tile - 1) / tile;
    return (offsets ? run + samples : run) * kv_heads;
  };
  // Rows of a tile (96 goes by 128, 192 by 256). Up to 32 the waves of a block share the keys instead of
  // the rows. 64 rows per wave read LDS half as often as 32, but leave one
  // block to a CU. Heads of 256: 2048 rows of 16 heads over 300 keys 33 us
  // with 64 rows and 23 with 32, 4000 keys 152 and 143, 16000 keys 479 and
  // 512; 8192 rows 441 and 509 (4000 keys). Heads of 64: 16896 tokens of 18
  // heads 1420 and 1544, 3000 rows of 16 heads over 4000 keys 84 and 85, over
  // 1000 keys 37 and 30, 256 rows over 4000 keys 29 and 22. Heads of 128: two blocks of 32 rows per wave on a CU
  // are as fast as one of 64 on the largest (2581 and 2591) and faster on all
  // others.
  if (each <= 32) p.rows = 32;
  else if (each <= 128 || dp == 96 || dp == 128) p.rows = 128;
  else if (dp == 64) p.rows = 2 * tiles_of(256) >= kCus && keys >= 4000 ? 256 : 128;
  else p.rows = 2 * tiles_of(256) > kCus || keys >= 8000 ? 256 : 128;
  // blocks that a CU holds at once, by LDS and registers
  const int held = p.rows == 32 ? (dp == 64 ? 4 : dp <= 128 ? 2 : 1) : dp <= 128 ? 2 : 1;
  const int at_once = kCus * held;
  const int64_t tiles = tiles_of(p.rows);
  // Cutting pays for its second launch from some keys on (units of 128 with
  // 32 rows, else of 64). One query of 16 heads of 256, whole and cut: 512
  // keys 11 and 13 us, 1024 keys 17 and 15, 4096 keys 50 and 21; of 64: 1024
  // keys 7.9 and 9.2, 4096 keys 21 and 11. 256 rows of 16 heads of 256: 300
  // keys 18 and 22, 1000 keys 41 and 25.
  const bool all = cuts_all(p.rows);
  const int least = least_units(p.rows), unit = all ? 128 : 64;
  p.cut_units = !all ? 10 : dp > 128 ? 8 : 16;
  p.slots = workspace ? (all ? std::max(at_once, 2 * kCus) : at_once) : 0;
  // Nor are tiles cut that fill the blocks several times over, or where a
  // sample's keys are far below that on average (a batch of which one sample
  // has most of the keys loses by that).
  const int64_t cut_keys = (int64_t)unit * p.cut_units;
  if (Mk < cut_keys || keys * 2 < cut_keys || (all && tiles >= 4 * (int64_t)p.slots)) p.slots = 0;
  // The last tiles of one sample over few keys: 32 rows to a block (8 of a
  // tile) need no second launch to join them and fill the card where cutting
  // the keys does not: 4096 rows of 18 heads of 256 over 512 keys (32 tiles
  // behind 256 whole ones) 66 us, keys cut 82.
  const int64_t behind = tiles % at_once;
  if (!offsets && dp == 256 && p.rows == 256 && tiles > at_once && behind > 0 && behind * 8 <= at_once && Mk <= 2048) {
    p.rest = behind;
    p.rest_from = (int)(tiles - behind);
    p.slots = 0;
  }
  if (p.slots > 0) p.cut = all ? tiles : offsets ? std::min<int64_t>(tiles, p.slots - 1) : tiles % p.slots;
  p.per = 1 << 30;
  if (p.cut > 0) {
    // about the slots, or two rounds of them, and one of each tile more; without offsets all of it is known
    p.pieces = all ? p.slots + p.cut : 2 * p.slots + p.cut;
    if (!offsets) {
      const int units = (int)((Mk + unit - 1) / unit), cut = (int)p.cut;
      p.per = equal_pieces(units, cut, p.slots, least);
      if (!all) p.per = best_length(units, units, cut, p.slots, p.per, equal_pieces(units, cut, 2 * p.slots, least));
      if (p.per == units) p.slots = 0, p.cut = 0;
      p.pieces = p.cut * ((units + p.per - 1) / p.per);
    }
  }
  p.whole = (int)(tiles - p.cut);
  p.blocks = (offsets ? tiles : p.whole) - p.rest + p.pieces;
  p.longest = p.cut > 0 && p.whole == 0 && !offsets ? (int64_t)p.per * unit : Mk;
  if (all) p.longest = (p.longest + 3) / 4;  // the waves of a block divide them
  p.partial_bytes = (size_t)p.pieces * p.rows * (dp + 2) * sizeof(float);
  return p;
}

hipError_t launch_attention(const AttentionArgs &args, const AttentionPlan &p, hipStream_t stream) {
  AttentionArgs a = args;
  a.slots = p.slots;
  a.cut_units = p.cut_units;
  a.pieces = p.pieces;
  a.whole = p.whole;
  a.per = p.per;
  a.rest_from = p.rest_from;
  switch (padded(a.D)) {
    case 64: launch_width<64>(a, p, stream); break;
    case 96: launch_width<96>(a, p, stream); break;
    case 192: launch_width<192>(a, p, stream); break;
    case 128: launch_width<128>(a, p, stream); break;
    default: launch_width<256>(a, p, stream); break;
  }
  return hipGetLastError();
}

}  // namespace ql
