// Low-rank adapters of many requests beside a shared projection (qlinear_adapters).
//
//   v[m, :] = A[id_m] x[m, :]                    (rank values)
//   t[m, :] = y[m, :] + scaling[id_m] * B[id_m] v[m, :]
//   out     = t | silu(t_gate) * t_up | residual + gate * t
//
// Two launches, for v needs all of K before its first use: "down" (x and A to
// v, K split over blocks and waves) and "up" (v and B onto y, with the
// epilogue). Both work on tiles of consecutive rows. The rows of a tile may
// belong to any adapters: a block takes the tile's distinct adapters one by
// one, multiplies the whole tile by each and keeps the rows that are that
// adapter's (a row of an MFMA product depends on its own row of the operand
// alone, so what other rows hold never reaches it). A row's sums have the
// same order wherever it stands in a tile and whatever its neighbours are.
//
// Every row has one adapter, so blocks that share a tile's adapters write
// different rows: no atomics and no order between blocks.
//
// Numerics: x and A enter the bf16 MFMA as they are (fp16 tables as an exact
// sum of two bf16 terms), v is fp32 and enters the second product as three
// bf16 terms (24 bits), accumulation is fp32, the output is rounded once. A
// term of a finite value may be zero, and an infinite value has no terms behind
// the first: where an infinity enters, a sum over terms can be NaN although
// the sum over the values is infinite. Sums of terms that are not finite are
// therefore taken again from the values one by one, off the fast path.
#include <algorithm>
#include <type_traits>

#include "ql_block.h"
#include "ql_kernels.h"

namespace ql {

namespace {

constexpr int kWaves = 4;
constexpr int kMostSplits = 8;
constexpr int kCus = 256;  // MI355X

// A fragment of eight table values as bf16 terms whose sum is exact.
template <bool F16> struct Terms { static constexpr int n = F16 ? 2 : 1; };

// fp16 -> two bf16 terms: the upper 8 bits of the significand by truncation,
// the remaining 3 bits as an exact bf16.
template <bool F16>
__device__ __forceinline__ void table_terms(u32x4 raw, bf16x8 (&t)[Terms<F16>::n]) {
  if constexpr (!F16) {
    t[0] = as_bf16x8(raw);
  } else {
    u32x4 hi, lo;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t a = __float_as_uint(f16_to_f32((uint16_t)raw[e]));
      const uint32_t b = __float_as_uint(f16_to_f32((uint16_t)(raw[e] >> 16)));
      hi[e] = perm(b, a, 0x07060302u);
      const uint32_t ra = __float_as_uint(__uint_as_float(a) - __uint_as_float(a & 0xFFFF0000u));
      const uint32_t rb = __float_as_uint(__uint_as_float(b) - __uint_as_float(b & 0xFFFF0000u));
      lo[e] = perm(rb, ra, 0x07060302u);
    }
    t[0] = as_bf16x8(hi);
    t[1] = as_bf16x8(lo);
  }
}

// fp32 -> three bf16 terms, each the upper half of what the ones before left
// (truncation: every difference is exact; 8 bits each, 24 in all).
__device__ __forceinline__ void split3(const float (&f)[8], bf16x8 (&t)[3]) {
  float r[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) r[e] = f[e];
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    u32x4 w;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      w[e] = perm(__float_as_uint(r[2 * e + 1]), __float_as_uint(r[2 * e]), 0x07060302u);
      r[2 * e] -= __uint_as_float(__float_as_uint(r[2 * e]) & 0xFFFF0000u);
      r[2 * e + 1] -= __uint_as_float(__float_as_uint(r[2 * e + 1]) & 0xFFFF0000u);
    }
    t[k] = as_bf16x8(w);
  }
}

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Between a wave's writes to its own part of LDS and its reads of what other
// lanes wrote: LDS serves a wave's accesses in order, so only the compiler has
// to keep them there.
__device__ __forceinline__ void wave_lds_fence() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The lane counted anew, of nothing that is at hand: what rarely runs computes
// its addresses from it, and keeps no register while the fast path runs.
__device__ __forceinline__ int another_lane() {
  uint32_t all = ~0u;
  asm volatile("" : "+v"(all));
  return __builtin_amdgcn_mbcnt_hi(all, __builtin_amdgcn_mbcnt_lo(all, 0u));
}

// The address of the kernel's first argument, for reading it anew for the same reason.
typedef __attribute__((address_space(4))) const AdapterArgs *Kernarg;
__device__ __forceinline__ Kernarg another_args() {
  uint64_t at = (uint64_t)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(at));
  return (Kernarg)at;
}

// The adapter of each of a tile's T rows, one lane per row: an index of the
// table, -1 for a row without one (any index outside the table), -2 past M.
template <int T>
__device__ __forceinline__ int tile_id(const int32_t *row_adapter, int64_t m0, int64_t M, int64_t adapters, int lane) {
  const int64_t m = m0 + lane;
  if (lane >= T || m >= M) return -2;
  const int id = row_adapter[m];
  return id >= 0 && id < adapters ? id : -1;
}

// Calls f(adapter, rows) for every slots-th distinct value >= lowest among the
// tile's ids, `rows` being the bit mask of the rows that have it. Uniform over
// the block: every wave holds the same ids.
template <typename F>
__device__ __forceinline__ void each_adapter(int id, int lowest, int slot, int slots, F f) {
  uint64_t left = __ballot(id >= lowest);
  for (int j = 0; left != 0; ++j) {
    const int cur = __builtin_amdgcn_readlane(id, __builtin_ctzll(left));
    const uint64_t rows = __ballot(id == cur) & left;
    left &= ~rows;
    if (j % slots == slot) f(cur, rows);
  }
}

__device__ __forceinline__ int adapter_rank(const AdapterArgs &a, int id) {
  if (id < 0) return 0;
  if (!a.ranks) return a.rank;
  return min(max(a.ranks[id], 0), a.rank);
}

// The partial sums of a 16 x 16 piece, rows from `row` of the tile and ranks
// from r, that the fp16 terms left not finite, taken again over [k0, k1).
__device__ __forceinline__ void sum_values(const AdapterArgs &a, float *v, int cur, int rank, int64_t m0, uint64_t rows,
                                           int row, int r, int k0, int k1) {
  const int lane = another_lane();
  row += lane & 15;
  r += (lane >> 4) * 4;
  if (!((rows >> row) & 1)) return;
  const uint16_t *const x = a.x + (m0 + row) * a.K;
#pragma clang loop unroll(disable)
  for (int e = r; e < min(r + 4, rank); ++e) {
    float *const sum = v + (m0 + row) * a.rank + e;
    if (__builtin_isfinite(*sum)) continue;
    const uint16_t *const w = a.a + ((int64_t)cur * a.rank + e) * a.K;
    float t = 0.f;
#pragma clang loop unroll(disable)
    for (int k = k0; k < k1; ++k) t = __builtin_fmaf(bf16_lo(x[k]), f16_to_f32(w[k]), t);
    *sum = t;
  }
}

// v = A x over a range of K. Block: WR*MI*16 rows, RJ*16 ranks; its waves are
// WR along the rows, and the others take the range's 64-wide K units in turn
// and add their sums in LDS in wave order.
//
// A unit of rows is loaded eight 128-byte lines to an instruction, eight
// neighbouring lanes to a line, and turned into MFMA operands (16 rows to 16
// neighbouring lanes) in LDS of the wave's own, without a barrier: loads in
// operand order, 16 bytes of 16 rows to neighbouring lanes, run at 15 B/clk
// and CU from L2, loads by lines at 45 to 57 (a 64 x 4608 table read by every
// CU). Line r keeps its 16-byte piece c at c ^ (r & 7): no bank conflicts.
// The next unit is requested before this one is multiplied.
template <int MI, int WR, int RJ, bool F16>
__global__ __launch_bounds__(64 * kWaves) void adapter_down_kernel(AdapterArgs a, int slots, int units_per_split) {
  constexpr int NT = Terms<F16>::n;
  constexpr int T = 16 * MI * WR, KW = kWaves / WR;
  constexpr int LINES = 16 * (MI + RJ);            // of one unit: x, then the table
  constexpr int SUMS = (KW - 1) * WR * MI * RJ * 64;  // 16-byte words of the waves' sums
  __shared__ f32x4 lds[SUMS > kWaves * LINES * 8 ? SUMS : kWaves * LINES * 8];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wr = wave % WR, wk = wave / WR;
  const int r16 = lane & 15, g = lane >> 4;
  u32x4 *const stage = reinterpret_cast<u32x4 *>(lds) + wave * LINES * 8;
  const int64_t m0 = (int64_t)blockIdx.x * T;
  const int slot = blockIdx.z % slots;
  const int r0 = (int)(blockIdx.z / slots) * (16 * RJ);
  const int units = (int)(a.K / 64);
  const int u0 = blockIdx.y * units_per_split, u1 = min(units, u0 + units_per_split);
  const int id = tile_id<T>(a.row_adapter, m0, a.M, a.adapters, lane);
  each_adapter(id, 0, slot, slots, [&](int cur, uint64_t rows) {
    const int rank = adapter_rank(a, cur);
    if (r0 >= rank) return;
    // lines of x and of the table as offsets into the tile's and the adapter's part
    const __amdgpu_buffer_rsrc_t x_buf = make_rsrc(a.x, m0 * a.K * 2, INT32_MAX);
    const __amdgpu_buffer_rsrc_t a_buf = make_rsrc(a.a, ((int64_t)cur * a.rank + r0) * a.K * 2, INT32_MAX);
    const int first = wr * (16 * MI);
    int x_at[2 * MI], a_at[2 * RJ];
#pragma unroll
    for (int i = 0; i < 2 * MI; ++i) {
      const int row = first + i * 8 + (lane >> 3);
      const int pick = (rows >> row) & 1 ? row : (int)__builtin_ctzll(rows);  // rows of others: not loaded
      x_at[i] = pick * (int)a.K * 2 + (lane & 7) * 16;
    }
#pragma unroll
    for (int j = 0; j < 2 * RJ; ++j) a_at[j] = min(j * 8 + (lane >> 3), rank - r0 - 1) * (int)a.K * 2 + (lane & 7) * 16;
    f32x4 acc[MI][RJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < RJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    u32x4 line[2 * (MI + RJ)];
    auto load = [&](int u) {
#pragma unroll
      for (int i = 0; i < 2 * MI; ++i)
        line[i] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(x_buf, x_at[i], u * 128, 0));
#pragma unroll
      for (int j = 0; j < 2 * RJ; ++j)
        line[2 * MI + j] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(a_buf, a_at[j], u * 128, 0));
    };
    const int put = (lane >> 3) * 8 + ((lane & 7) ^ (lane >> 3));
    auto operand = [&](int tile, int s) {  // 16 lines from 16 * tile, the 16-byte piece 2 g + s
      return stage[(tile * 16 + r16) * 8 + ((2 * g + s) ^ (r16 & 7))];
    };
    if (((rows >> first) & (~0ull >> (64 - 16 * MI))) != 0 && u0 + wk < u1) {
      load(u0 + wk);
      for (int u = u0 + wk; u < u1; u += KW) {
#pragma unroll
        for (int i = 0; i < 2 * (MI + RJ); ++i) stage[i * 64 + put] = line[i];
        wave_lds_fence();
        load(min(u + KW, u1 - 1));
        __builtin_amdgcn_sched_barrier(0);  // requested before the products
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          bf16x8 x[MI];
#pragma unroll
          for (int i = 0; i < MI; ++i) x[i] = as_bf16x8(operand(i, s));
#pragma unroll
          for (int j = 0; j < RJ; ++j) {
            bf16x8 w[NT];
            table_terms<F16>(operand(MI + j, s), w);
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
              for (int k = 0; k < NT; ++k) acc[i][j] = mfma(w[k], x[i], acc[i][j]);
          }
        }
        wave_lds_fence();
      }
    }
    __syncthreads();  // every wave's operands, and the previous adapter's sums, have been read
    if (wk > 0) {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < RJ; ++j) lds[(((wk - 1) * WR + wr) * (MI * RJ) + i * RJ + j) * 64 + lane] = acc[i][j];
    }
    __syncthreads();
    if (wk == 0) {
      float *v = a.v + (int64_t)blockIdx.y * a.M * a.rank;
      uint32_t again = 0;  // pieces with a sum of fp16 terms that is not finite
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int row = first + i * 16 + r16;
#pragma unroll
        for (int j = 0; j < RJ; ++j) {
          f32x4 t = acc[i][j];
#pragma unroll
          for (int w = 0; w < KW - 1; ++w) t += lds[((w * WR + wr) * (MI * RJ) + i * RJ + j) * 64 + lane];
          const int r = r0 + j * 16 + g * 4;
          const float zero = (t[0] * 0.f + t[1] * 0.f) + (t[2] * 0.f + t[3] * 0.f);  // NaN where a sum is not finite
          if (((rows >> row) & 1) && r < a.rank) *reinterpret_cast<f32x4 *>(v + (m0 + row) * a.rank + r) = t;
          if (F16 && __ballot(!(zero == 0.f)) != 0) again |= 1u << (i * RJ + j);
        }
      }
      for (; again != 0; again &= again - 1) {
        const int piece = __builtin_ctz(again);
        sum_values(a, v, cur, rank, m0, rows, first + piece / RJ * 16, r0 + piece % RJ * 16, u0 * 64, u1 * 64);
      }
    }
    __syncthreads();  // the sums have been read: the next adapter's operands may take their place
  });
}

// silu(g) * u with the hardware exponential and reciprocal; e^-g overflows to
// +inf for g < -88 and the quotient is then -0.
__device__ __forceinline__ float silu_mul(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

// Clears the ranks from `rank` on of a table's entries k .. k + 7, which may hold anything.
__device__ __forceinline__ void mask_ranks(int k, int rank, u32x4 &raw) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (k + 2 * e >= rank) raw[e] = 0;
    else if (k + 2 * e + 1 >= rank) raw[e] &= 0xFFFFu;
  }
}

// Sixteen rows from row m of an array [., row_length], as a buffer: at most
// 16 * 2^22 values (kMaxAdapterColumns) of 4 bytes; of no bytes for no array.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t tile_buffer(const void *p, int64_t m, int64_t row_length, int size) {
  return make_rsrc(p, p ? m * row_length * size : 0, p ? 16 * row_length * size : 0);
}

// Four values of a stream as loaded: packed where they come as 8 or 16 bytes.
template <typename T, bool VEC> struct Raw4 { uint32_t v[VEC && __is_same(T, BF16) ? 2 : 4]; };

template <typename T, bool VEC>
__device__ __forceinline__ void unpack4(const Raw4<T, VEC> &r, float (&f)[4]) {
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    if constexpr (VEC && __is_same(T, BF16)) f[s] = s % 2 ? bf16_hi(r.v[s / 2]) : bf16_lo(r.v[s / 2]);
    else f[s] = __uint_as_float(r.v[s]);
  }
}

// A lane's four columns of rows of `width` values, `pitch` apart: n .. n + 3,
// or one by one n, n + 16, n + 32, n + 48, so that neighbouring lanes have
// neighbouring columns either way. A column past the width, or a row that is
// not live, has its offset past the buffer's end: its loads give zero and its
// stores are dropped.
template <bool VEC> struct Tile {
  int n, width, pitch;
  static constexpr int kPast = 0x7FFFFFF0;
  __device__ __forceinline__ int at(int row, int first, int s, bool live, int size) const {
    const int c = n + (VEC ? s : 16 * s);
    return live && c < width ? (row * pitch + first + c) * size : kPast;
  }
  template <typename T>
  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t r, int row, int first, bool live, Raw4<T, VEC> &raw) const {
    if constexpr (VEC && __is_same(T, F32)) {
      const u32x4 v = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(r, at(row, first, 0, live, 4), 0, 0));
#pragma unroll
      for (int s = 0; s < 4; ++s) raw.v[s] = v[s];
    } else if constexpr (VEC) {
      const u32x2 v = __builtin_bit_cast(u32x2, __builtin_amdgcn_raw_buffer_load_b64(r, at(row, first, 0, live, 2), 0, 0));
      raw.v[0] = v[0], raw.v[1] = v[1];
    } else {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if constexpr (__is_same(T, F32)) raw.v[s] = __builtin_amdgcn_raw_buffer_load_b32(r, at(row, first, s, live, 4), 0, 0);
        else raw.v[s] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(r, at(row, first, s, live, 2), 0, 0) << 16;
      }
    }
  }
  template <typename T>
  __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t r, int row, bool live, const float (&f)[4]) const {
    if constexpr (VEC && __is_same(T, F32)) {
      const f32x4 v = {f[0], f[1], f[2], f[3]};
      __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, v), r, at(row, 0, 0, live, 4), 0, 0);
    } else if constexpr (VEC) {
      __builtin_amdgcn_raw_buffer_store_b64(u32x2{pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3])}, r,
                                            at(row, 0, 0, live, 2), 0, 0);
    } else {
#pragma unroll
      for (int s = 0; s < 4; ++s) {
        if constexpr (__is_same(T, F32))
          __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(f[s]), r, at(row, 0, s, live, 4), 0, 0);
        else
          __builtin_amdgcn_raw_buffer_store_b16(bf16_bits(f[s]), r, at(row, 0, s, live, 2), 0, 0);
      }
    }
  }
};

// One step of the second launch, 16 rows from `first` of the tile by 64 columns
// of out from n0, with sums of terms that are not finite: the same sums, in the
// place of those that are not finite the sums over the values, and the
// epilogue, a column at a time. Looking for such sums costs a multiply-add for
// each of them, 0 to 2 % of a call (us before and with it: QKV 4608 x 4608 ->
// 13824 rank 32 121 and 120, SwiGLU 4096 x 4608 -> 24576 rank 16 89 and 90,
// gated down 16896 x 12288 -> 4608 rank 64 246 and 249).
template <bool F16, typename YT, typename OT, int EPI, bool VEC>
__device__ __forceinline__ void step_by_values(Kernarg args, const f32x4 *vs, int cur, uint64_t rows, int64_t m0, int first,
                                               int n0) {
  constexpr int NT = Terms<F16>::n;
  constexpr int HALVES = EPI == 1 ? 2 : 1;
  const AdapterArgs a = *(const AdapterArgs *)args;
  const int lane = another_lane(), r16 = lane & 15, g = lane >> 4;
  const int64_t width = a.N / HALVES;
  const int rank = adapter_rank(a, cur), units = (a.rank + 31) / 32 * 8;
  const uint16_t *const b = a.b + (int64_t)cur * a.N * a.rank;
#pragma clang loop unroll(disable)
  for (int s = 0; s < 4; ++s) {
    const int64_t c = n0 + (VEC ? 4 * r16 + s : 16 * s + r16);
    f32x4 acc[HALVES];
#pragma unroll
    for (int h = 0; h < HALVES; ++h) {
      const uint16_t *const table = b + (min(c, width - 1) + h * width) * a.rank;
      acc[h] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma clang loop unroll(disable)
      for (int k0 = 0; k0 < rank; k0 += 32) {
        const int row = first + r16, u = k0 / 4 + 2 * g;
        const f32x4 lo = vs[row * units + (u ^ (row & 7))], hi = vs[row * units + ((u + 1) ^ (row & 7))];
        const float f[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        bf16x8 vt[3], bt[NT];
        split3(f, vt);
        u32x4 w = {0, 0, 0, 0};
        const int k = k0 + 8 * g;
        if (k < rank) w = *reinterpret_cast<const u32x4 *>(table + k);
        mask_ranks(k, rank, w);
        table_terms<F16>(w, bt);
#pragma unroll
        for (int q = 2; q >= 0; --q)
#pragma unroll
          for (int p = 0; p < NT; ++p) acc[h] = mfma(vt[q], bt[p], acc[h]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (__builtin_isfinite(acc[h][e])) continue;
        const int row = first + 4 * g + e;
        float t = 0.f;
#pragma clang loop unroll(disable)
        for (int k = 0; k < rank; ++k)
          t = __builtin_fmaf(reinterpret_cast<const float *>(vs + row * units + ((k / 4) ^ (row & 7)))[k % 4],
                             F16 ? f16_to_f32(table[k]) : bf16_lo(table[k]), t);
        acc[h][e] = t;
      }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int row = first + 4 * g + e;
      if (c >= width || !((rows >> row) & 1)) continue;
      const int64_t m = m0 + row;
      float t[HALVES];
#pragma unroll
      for (int h = 0; h < HALVES; ++h) t[h] = (a.y ? YT::load(a.y, m * a.N + h * width + c) : 0.f) + acc[h][e];
      if constexpr (EPI == 1) t[0] = silu_mul(t[0], t[HALVES - 1]);
      if constexpr (EPI == 2)
        t[0] = __builtin_fmaf(a.gate[m / a.gate_rows * width + c], t[0], OT::load(a.residual, m * width + c));
      OT::store(a.out, m * width + c, t[0]);
    }
  }
}

// The same as a function of its own, for the kernels that read B by steps: put
// into the kernel, it slows their loop (SwiGLU 2048 x 4608 -> 24576 rank 72 143
// us, rank 128 146; called 132 and 139). The others have it inside, where a
// call takes registers that the loop needs (4096 x 4608 -> 4608 bf16 rank 64
// four waves per SIMD and 45.3 us, with a call three and 45.9).
template <bool F16, typename YT, typename OT, int EPI, bool VEC>
__device__ __attribute__((noinline)) void step_by_values_called(Kernarg args, const f32x4 *vs, int cur, uint64_t rows,
                                                              int64_t m0, int first, int n0) {
  step_by_values<F16, YT, OT, EPI, VEC>(args, vs, cur, rows, m0, first, n0);
}

// out = epilogue(y + scaling * B v). Block: MI*16 rows; its four waves take
// `chunks` times 256 output columns, 64 each. For one adapter of the tile the
// block first adds the partial sums of v, scales them and keeps them in LDS
// (fp32, zero past the adapter's rank), so that they are read once per block
// and not once per 64 columns. Subtile s of a wave covers columns 4*c + s: a
// lane ends with four consecutive columns of four rows, and 16 lanes load and
// store a contiguous 256 (fp32) or 128 bytes of a row. Rows that do not start
// on four elements have c + 16*s instead, a column to an access. SwiGLU has the same
// columns twice, from the gate and the up half. KB steps of 32 ranks of B
// stay in registers over the rows (0: any rank, B read again for every 16 rows).
//
// One step is 16 rows by 64 columns. What the next step reads of y, residual,
// gate and B is requested before this step's stores: a wait for loads counts
// every memory access before them, so a load behind stores waits for those
// (16384 x 4608 bf16 with residual: 200 us with the loads behind).
template <int MI, int KB, bool F16, typename YT, typename OT, int EPI, bool VEC>
__global__ __launch_bounds__(64 * kWaves) void adapter_up_kernel(AdapterArgs a, int slots, int splits, int col_blocks,
                                                               int chunks, int skip_rows_without) {
  constexpr int NT = Terms<F16>::n;
  constexpr int HALVES = EPI == 1 ? 2 : 1;
  constexpr int T = 16 * MI;
  extern __shared__ f32x4 vs[];  // [T][rank / 4 rounded up to 8], 16-byte units swizzled by the row
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int64_t m0 = (int64_t)(blockIdx.x / (unsigned)col_blocks) * T;
  const int width = (int)(EPI == 1 ? a.N / 2 : a.N);  // of out
  const int first = (int)(blockIdx.x % (unsigned)col_blocks) * chunks;
  const int units = (a.rank + 31) / 32 * 8;
  const int id = tile_id<T>(a.row_adapter, m0, a.M, a.adapters, lane);
  bool later = false;
  each_adapter(id, skip_rows_without ? 0 : -1, blockIdx.y, slots, [&](int cur, uint64_t rows) {
    const int rank = adapter_rank(a, cur);
    const float scaling = cur >= 0 && a.scaling ? a.scaling[cur] : 1.0f;
    const uint16_t *const b = a.b + (int64_t)cur * a.N * a.rank;

    // B of the wave's 64 columns from n0 of half h, ranks k0 .. k0 + 31: rows
    // (columns of out) 4 r16 + s, or r16 + 16 s, ranks 8 g .. 8 g + 7 of subtile s. With TURN,
    // where it is read for every step, it is loaded four neighbouring lanes to
    // a row's 64 bytes and turned in LDS of the wave's own: in operand order
    // neighbouring lanes are 4 rows apart, and such loads run at a quarter of
    // the rate (SwiGLU 2048 x 4608 -> 24576 at rank 128: 202 -> 147 us). Read
    // once for four steps it is not worth the LDS (rank 16: 90 -> 96 us).
    constexpr bool TURN = KB == 0;
    u32x4 *const stage = reinterpret_cast<u32x4 *>(vs + T * units) + wave * 256;
    auto load_b = [&](int n0, int h, int k0, u32x4 (&raw)[4]) {
      const int k = k0 + (TURN ? lane & 3 : g) * 8;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        raw[q] = u32x4{0, 0, 0, 0};
        const int row = TURN ? q * 16 + (lane >> 2) : VEC ? 4 * r16 + q : 16 * q + r16;
        const int64_t col = min(n0 + row, width - 1) + (int64_t)h * width;
        if (k < rank) raw[q] = *reinterpret_cast<const u32x4 *>(b + col * a.rank + k);
      }
    };
    auto turn = [&](u32x4 (&raw)[4]) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        // of column 16 q + lane / 4: its lane r16 and subtile s
        const int row = VEC ? q * 4 + (lane >> 4) : lane >> 2, s = VEC ? (lane >> 2) & 3 : q;
        stage[(s * 16 + row) * 4 + ((lane & 3) ^ (row & 3))] = raw[q];
      }
      wave_lds_fence();
#pragma unroll
      for (int s = 0; s < 4; ++s) raw[s] = stage[(s * 16 + r16) * 4 + (g ^ (r16 & 3))];
      wave_lds_fence();
    };
    auto mask_b = [&](int k0, u32x4 &raw) {
      if (k0 + 32 > rank) mask_ranks(k0 + g * 8, rank, raw);
    };

    // the streams of rows 16 i .., columns of chunk ch
    Raw4<YT, VEC> y_raw[HALVES][4];
    Raw4<OT, VEC> res_raw[4];
    Raw4<F32, VEC> gate_raw;
    u32x4 b_raw[HALVES][KB ? KB : 1][4];
    auto wave_column = [&](int ch) { return (first + ch) * (64 * kWaves) + wave * 64; };
    auto column = [&](int ch) { return wave_column(ch) + (VEC ? 4 * r16 : r16); };
    auto live = [&](int i, int e) -> bool { return (rows >> (16 * i + 4 * g + e)) & 1; };
    auto load_streams = [&](int ch, int i) {
      const int64_t m = m0 + 16 * i;
      const Tile<VEC> y = {column(ch), width, (int)a.N}, out = {column(ch), width, width};
      const __amdgpu_buffer_rsrc_t y_buf = tile_buffer(a.y, m, a.N, sizeof(typename YT::type));
#pragma unroll
      for (int h = 0; h < HALVES; ++h)
#pragma unroll
        for (int e = 0; e < 4; ++e) y.template load<YT>(y_buf, 4 * g + e, h * width, live(i, e), y_raw[h][e]);
      if constexpr (EPI == 2) {
        const __amdgpu_buffer_rsrc_t res_buf = tile_buffer(a.residual, m, width, sizeof(typename OT::type));
#pragma unroll
        for (int e = 0; e < 4; ++e) out.template load<OT>(res_buf, 4 * g + e, 0, live(i, e), res_raw[e]);
        out.template load<F32>(tile_buffer(a.gate, (uint32_t)m / (uint32_t)a.gate_rows, width, 4), 0, 0, true, gate_raw);
      }
    };
    auto load_table = [&](int ch) {
      if constexpr (KB > 0) {
#pragma unroll
        for (int h = 0; h < HALVES; ++h)
#pragma unroll
          for (int k = 0; k < KB; ++k) load_b(wave_column(ch), h, 32 * k, b_raw[h][k]);
      }
    };

    int i = -1, ch = 0;
    auto next_group = [&](int after) -> int {  // the tile's next 16 rows with rows of this adapter
      for (int j = after + 1; j < MI; ++j)
        if ((rows >> (16 * j)) & 0xFFFF) return j;
      return MI;
    };
    const int group0 = next_group(-1);
    i = group0;
    const bool any = first * (64 * kWaves) + wave * 64 < width;
    if (any) {
      load_table(0);
      load_streams(0, i);
    }
    if (later) __syncthreads();  // the previous adapter's v has been read
    later = true;
    for (int u = threadIdx.x; u < T * units; u += 64 * kWaves) {
      const int row = u / units, c = u % units;
      f32x4 t = {0.f, 0.f, 0.f, 0.f};
      if (((rows >> row) & 1) && 4 * c < rank) {
        const float *p = a.v + (m0 + row) * a.rank + 4 * c;
        const int64_t split = a.M * a.rank;
        f32x4 part[kMostSplits];
#pragma unroll
        for (int q = 0; q < kMostSplits; ++q)
          part[q] = q < splits ? *reinterpret_cast<const f32x4 *>(p + q * split) : f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int q = 0; q < kMostSplits; ++q) t += part[q];
#pragma unroll
        for (int e = 0; e < 4; ++e) t[e] = 4 * c + e < rank ? t[e] * scaling : 0.f;
      }
      vs[row * units + (c ^ (row & 7))] = t;
    }
    __syncthreads();
    if (!any) return;
    uint32_t again = 0;  // steps with a sum that is not finite: not stored here, but by step_by_values
    for (;;) {
      f32x4 acc[HALVES][4];
#pragma unroll
      for (int h = 0; h < HALVES; ++h)
#pragma unroll
        for (int s = 0; s < 4; ++s) acc[h][s] = f32x4{0.f, 0.f, 0.f, 0.f};
      auto step = [&](int k, const u32x4 (&raw)[HALVES][4]) {
        const int row = 16 * i + r16, c = 8 * k + 2 * g;
        const f32x4 lo = vs[row * units + (c ^ (row & 7))], hi = vs[row * units + ((c + 1) ^ (row & 7))];
        const float f[8] = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        bf16x8 vt[3];
        split3(f, vt);
#pragma unroll
        for (int h = 0; h < HALVES; ++h)
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            bf16x8 bt[NT];
            u32x4 w = raw[h][s];
            if constexpr (KB > 0) mask_b(32 * k, w);
            table_terms<F16>(w, bt);
#pragma unroll
            for (int q = 2; q >= 0; --q)
#pragma unroll
              for (int p = 0; p < NT; ++p) acc[h][s] = mfma(vt[q], bt[p], acc[h][s]);
          }
      };
      if constexpr (KB > 0) {
#pragma unroll
        for (int k = 0; k < KB; ++k) {
          u32x4 raw[HALVES][4];
#pragma unroll
          for (int h = 0; h < HALVES; ++h)
#pragma unroll
            for (int s = 0; s < 4; ++s) raw[h][s] = b_raw[h][k][s];
          step(k, raw);
        }
      } else {
        // one step of ranks ahead
        u32x4 now[HALVES][4], ahead[HALVES][4];
#pragma unroll
        for (int h = 0; h < HALVES; ++h) load_b(wave_column(ch), h, 0, now[h]);
        for (int k = 0; 32 * k < rank; ++k) {
#pragma unroll
          for (int h = 0; h < HALVES; ++h) load_b(wave_column(ch), h, min(32 * k + 32, 32 * (units / 8 - 1)), ahead[h]);
#pragma unroll
          for (int h = 0; h < HALVES; ++h) turn(now[h]);
          if (32 * k + 32 > rank) {
#pragma unroll
            for (int h = 0; h < HALVES; ++h)
#pragma unroll
              for (int s = 0; s < 4; ++s) mask_ranks(32 * k + g * 8, rank, now[h][s]);
          }
          step(k, now);
#pragma unroll
          for (int h = 0; h < HALVES; ++h)
#pragma unroll
            for (int s = 0; s < 4; ++s) now[h][s] = ahead[h][s];
        }
      }
      const Tile<VEC> out = {column(ch), width, width};
      const uint32_t m32 = (uint32_t)m0 + 16 * i, gate0 = EPI == 2 ? m32 / (uint32_t)a.gate_rows : 0;
      const bool one_gate = EPI != 2 || (m32 + 15) / (uint32_t)a.gate_rows == gate0;
      float o[4][4], zero = 0.f;  // zero: NaN where a sum is not finite
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float t[HALVES][4], res[4], gt[4];
#pragma unroll
        for (int h = 0; h < HALVES; ++h) unpack4<YT, VEC>(y_raw[h][e], t[h]);
        if constexpr (EPI == 2) {
          unpack4<OT, VEC>(res_raw[e], res);
          if (one_gate) {
            unpack4<F32, VEC>(gate_raw, gt);
          } else {  // a boundary of samples among the 16 rows
            const uint32_t at = m32 + 4 * g + e;
            Raw4<F32, VEC> raw;
            out.template load<F32>(tile_buffer(a.gate, gate0, width, 4), (int)(at / (uint32_t)a.gate_rows - gate0), 0,
                                   live(i, e), raw);
            unpack4<F32, VEC>(raw, gt);
          }
        }
#pragma unroll
        for (int s = 0; s < 4; ++s) {
#pragma unroll
          for (int h = 0; h < HALVES; ++h) zero = __builtin_fmaf(acc[h][s][e], 0.f, zero);
          const float v = t[0][s] + acc[0][s][e];
          if constexpr (EPI == 1) o[e][s] = silu_mul(v, t[HALVES - 1][s] + acc[HALVES - 1][s][e]);
          else if constexpr (EPI == 2) o[e][s] = __builtin_fmaf(gt[s], v, res[s]);
          else o[e][s] = v;
        }
      }
      const uint32_t this_step = 1u << (ch * MI + i);
      const __amdgpu_buffer_rsrc_t out_buf = tile_buffer(a.out, m0 + 16 * i, width, sizeof(typename OT::type));
      bool keep[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) keep[e] = live(i, e);
      i = next_group(i);
      bool more = true;
      if (i == MI) {
        i = group0;
        ++ch;
        more = ch < chunks && (first + ch) * (64 * kWaves) + wave * 64 < width;
        if (more) load_table(ch);
      }
      if (more) load_streams(ch, i);
      __builtin_amdgcn_sched_barrier(0);  // the loads stay ahead of the stores
      const bool odd = __ballot(zero != 0.f) != 0;
      if (odd) again |= this_step;
#pragma unroll
      for (int e = 0; e < 4; ++e) out.template store<OT>(out_buf, 4 * g + e, keep[e] && !odd, o[e]);
      __builtin_amdgcn_sched_barrier(0);
      if (!more) break;
    }
    for (; again != 0; again &= again - 1) {
      const int bit = __builtin_ctz(again);
      const int first_row = bit % MI * 16, n0 = wave_column(bit / MI);
      if constexpr (KB == 0) step_by_values_called<F16, YT, OT, EPI, VEC>(another_args(), vs, cur, rows, m0, first_row, n0);
      else step_by_values<F16, YT, OT, EPI, VEC>(another_args(), vs, cur, rows, m0, first_row, n0);
    }
  });
}

template <int MI, int WR, int RJ>
void launch_down(const AdapterArgs &a, const AdapterPlan &p, hipStream_t stream) {
  const int units = (int)(a.K / 64), per = (units + p.splits - 1) / p.splits;
  const int chunks = (a.rank + 16 * RJ - 1) / (16 * RJ);
  const dim3 grid((unsigned)p.tiles, (unsigned)p.splits, (unsigned)(p.slots * chunks)), block(64 * kWaves);
  if (a.ab_f16) hipLaunchKernelGGL((adapter_down_kernel<MI, WR, RJ, true>), grid, block, 0, stream, a, p.slots, per);
  else hipLaunchKernelGGL((adapter_down_kernel<MI, WR, RJ, false>), grid, block, 0, stream, a, p.slots, per);
}

// 64-row tiles: two waves along the rows, or all four along K where a unit of
// the table is as large as the rows' (every wave along the rows reads it again:
// rank 64, 16896 x 12288 -> 4608 gated 266 us along K, 290 us with two and two;
// rank 32, 4608 x 4608 -> 13824 126 and 123 us).
template <int MI>
void launch_down_rank(const AdapterArgs &a, const AdapterPlan &p, hipStream_t stream) {
  constexpr int HALF = MI == 4 ? 2 : 1;
  if (a.rank <= 16) launch_down<MI / HALF, HALF, 1>(a, p, stream);
  else if (a.rank <= 32) launch_down<MI / HALF, HALF, 2>(a, p, stream);
  else launch_down<MI, 1, 4>(a, p, stream);
}

template <int MI, bool F16, typename YT, typename OT, int EPI>
void launch_up(const AdapterArgs &a, const AdapterPlan &p, hipStream_t stream) {
  const int64_t width = EPI == 1 ? a.N / 2 : a.N;
  const int64_t blocks = (width + 64 * kWaves - 1) / (64 * kWaves);
  const int chunks = (int)std::min<int64_t>(p.chunks, blocks);
  const int col_blocks = (int)((blocks + chunks - 1) / chunks);
  const dim3 grid((unsigned)(p.tiles * col_blocks), (unsigned)p.slots), block(64 * kWaves);
  // without an epilogue a row without an adapter is a copy of y, which is
  // nothing to do in place
  const int skip = EPI == 0 && a.y == a.out;
  const unsigned v_bytes = (unsigned)(16 * MI * ((a.rank + 31) / 32 * 32) * 4);  // v of the tile, 64 KB at most
  const auto run = [&](auto kernel, unsigned turn_bytes) {
    const unsigned lds = v_bytes + turn_bytes;
    if (lds > 65536u && hipFuncSetAttribute(reinterpret_cast<const void *>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize,
                                            (int)lds) != hipSuccess)
      return;  // reported by the check after the launches
    hipLaunchKernelGGL(kernel, grid, block, lds, stream, a, p.slots, p.splits, col_blocks, chunks, skip);
  };
  constexpr unsigned turn = kWaves * 4096;
  const auto by_rank = [&](auto vec) {
    constexpr bool VEC = decltype(vec)::value;
    // B stays in registers over a block's rows (KB steps of 32 ranks) where that
    // was measured faster than reading it by steps. Up to 64 ranks (4096 x 512
    // -> 4608 bf16 rank 64: 35 us held, 43 by steps; 500 rows within 7 % either
    // way), but for SwiGLU of rows by elements, whose two halves leave one or
    // two waves per SIMD then (2048 x 512 -> 8002 bf16 rank 64: 49 us held, 40
    // by steps; 500 rows 26 and 18). From 65 to 128 ranks, in 64-row tiles, fp32
    // in and out but for the gated update of whole fours. In us, held and by
    // steps, rank 96, 4096 x 4608 -> 4608 and (by elements) 4609: fp32 plain 86
    // and 88 (92 102), gated 107 and 100; bf16 plain 75 and 67 (80 72), gated 87
    // and 82 (131 100). Rank 128: bf16 plain 79 and 76 (86 83), gated 91 and 92
    // (139 117); 4096 x 512, fp32 plain 64 and 68 (68 70), gated 90 and 88 (95
    // 114).
    if (a.rank <= 32) return run(adapter_up_kernel<MI, 1, F16, YT, OT, EPI, VEC>, 0);
    if constexpr (VEC || EPI != 1) {
      if (a.rank <= 64) return run(adapter_up_kernel<MI, 2, F16, YT, OT, EPI, VEC>, 0);
    }
    constexpr bool F32S = std::is_same<YT, F32>::value && std::is_same<OT, F32>::value;
    if constexpr (MI == 4 && F32S && (EPI == 0 || (EPI == 2 && !VEC))) {
      if (a.rank <= 128) return run(adapter_up_kernel<MI, 4, F16, YT, OT, EPI, VEC>, 0);
    }
    run(adapter_up_kernel<MI, 0, F16, YT, OT, EPI, VEC>, turn);
  };
  if (a.vec) by_rank(std::true_type{});
  else by_rank(std::false_type{});
}

template <int MI, bool F16, typename YT, typename OT>
void launch_up_epi(const AdapterArgs &a, const AdapterPlan &p, hipStream_t stream) {
  if (a.epilogue == 1) launch_up<MI, F16, YT, OT, 1>(a, p, stream);
  else if (a.epilogue == 2) launch_up<MI, F16, YT, OT, 2>(a, p, stream);
  else launch_up<MI, F16, YT, OT, 0>(a, p, stream);
}

template <int MI, bool F16>
void launch_up_types(const AdapterArgs &a, const AdapterPlan &p, hipStream_t stream) {
  if (a.y_bf16) {
    if (a.out_bf16) launch_up_epi<MI, F16, BF16, BF16>(a, p, stream);
    else launch_up_epi<MI, F16, BF16, F32>(a, p, stream);
  } else {
    if (a.out_bf16) launch_up_epi<MI, F16, F32, BF16>(a, p, stream);
    else launch_up_epi<MI, F16, F32, F32>(a, p, stream);
  }
}

template <int MI>
hipError_t launch_mi(const AdapterArgs &a, const AdapterPlan &p, hipStream_t stream) {
  if (a.adapters > 0) launch_down_rank<MI>(a, p, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.ab_f16) launch_up_types<MI, true>(a, p, stream);
  else launch_up_types<MI, false>(a, p, stream);
  return hipGetLastError();
}

}  // namespace

AdapterPlan adapter_plan(int64_t M, int64_t N, int64_t K, int rank, int64_t adapters) {
  AdapterPlan p{};
  // 64-row tiles from 1024 blocks of the second launch and more than 1024 rows,
  // 16-row tiles below: more blocks, and fewer adapters to a tile of short
  // requests (512 rows of 16 requests, 4608 -> 4608 at rank 16: 16.3 us, with
  // 64-row tiles 20.4; 1186 rows of 28, 320 -> 1173 at rank 8: 16.0 and 28.9)
  const int64_t col_blocks = (N + 64 * kWaves - 1) / (64 * kWaves);
  p.row_tile = M > 1024 && M / 64 * col_blocks >= 1024 ? 64 : 16;
  p.tiles = (M + p.row_tile - 1) / p.row_tile;
  // Few tiles: blocks of their own for the adapters of one tile, 128 over all
  // tiles (203 rows of 14 requests: 11.1 us, at 32 over all 16.5; 256 rows of
  // 64 adapters in turn 59 and 87)
  const int64_t distinct = std::min<int64_t>({M, (int64_t)p.row_tile, adapters + 1});
  p.slots = (int)std::min<int64_t>(distinct, std::max<int64_t>(1, (p.row_tile == 16 ? 128 : 1) / p.tiles));
  // columns of a block of the second launch: 512 where 256 leave plenty of
  // blocks, so that v is summed less often (SwiGLU case 105 -> 96 us). The plan
  // is that of a call without an epilogue, and so is the workspace's size: with
  // SwiGLU, out has half of the pieces that are counted here.
  p.chunks = p.tiles * p.slots * col_blocks >= 2048 ? 2 : 1;
  // K ranges of the first launch, by its time and the second's: about 1 us for
  // each 64-wide unit of a wave and 2 us to start, in as many rounds as the
  // blocks need, and 1 ns for every 16 KB of partial sums, which are
  // written once and read by every block of columns. Measured in all: rank 64,
  // 4096 x 4608 -> 4608: 57.6, 46.6, 44.1, 43.5 us at 1, 2, 3, 4 ranges and
  // 46.8 at 8; rank 16, 1 row: 10.3 us at 1, 8.9 at 2, 8.3 at 8.
  const int rj = rank <= 16 ? 1 : rank <= 32 ? 2 : 4;
  const int along_k = p.row_tile == 16 || rj == 4 ? kWaves : kWaves / 2;  // waves of a block
  const int per_cu = p.row_tile == 16 ? (rj == 1 ? 8 : 4) : rj == 1 ? 5 : rj == 2 ? 4 : 2;  // blocks, by the registers of bf16 tables
  const int64_t blocks = p.tiles * p.slots * ((rank + 16 * rj - 1) / (16 * rj)), held = (int64_t)kCus * per_cu;
  const int64_t units = K / 64;
  const int64_t partial = M * rank * ((col_blocks + p.chunks - 1) / p.chunks + 2) / 4096;
  int64_t best = INT64_MAX;
  p.splits = 1;
  for (int64_t n = 1; n <= kMostSplits && n <= std::max<int64_t>(units, 1); ++n) {
    const int64_t per = (units + n - 1) / n;
    if (n > 1 && (units + per - 1) / per != n) continue;  // an empty range
    const int64_t cost = (blocks * n + held - 1) / held * ((per + along_k - 1) / along_k * 1000 + 2000) + n * partial;
    if (cost < best) best = cost, p.splits = (int)n;
  }
  return p;
}

hipError_t launch_adapters(const AdapterArgs &a, const AdapterPlan &p, hipStream_t stream) {
  return p.row_tile == 16 ? launch_mi<1>(a, p, stream) : launch_mi<4>(a, p, stream);
}

}  // namespace ql
