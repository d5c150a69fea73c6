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
// bf16 terms (24 bits), accumulation is fp32, the output is rounded once.
#include <algorithm>

#include "ql_block.h"
#include "ql_kernels.h"

namespace ql {

namespace {

constexpr int kWaves = 4;

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

// v = A x over a range of K. Block: MI*16 rows, RJ*16 ranks, four waves that
// take the range's 64-wide K units in turn and add their sums in LDS in wave
// order. A lane's 32 bytes of a row (two MFMA steps) lie side by side, so the
// four lanes of a row read its whole 128-byte line.
template <int MI, int RJ, bool F16>
__global__ __launch_bounds__(64 * kWaves) void adapter_down_kernel(AdapterArgs a, int slots, int units_per_split) {
  constexpr int NT = Terms<F16>::n;
  __shared__ f32x4 red[kWaves - 1][MI * RJ][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int64_t m0 = (int64_t)blockIdx.x * (16 * MI);
  const int slot = blockIdx.z % slots;
  const int r0 = (int)(blockIdx.z / slots) * (16 * RJ);
  const int units = (int)(a.K / 64);
  const int u0 = blockIdx.y * units_per_split, u1 = min(units, u0 + units_per_split);
  const int id = tile_id<16 * MI>(a.row_adapter, m0, a.M, a.adapters, lane);
  each_adapter(id, 0, slot, slots, [&](int cur, uint64_t rows) {
    const int rank = adapter_rank(a, cur);
    if (r0 >= rank) return;
    const uint16_t *xp[MI], *ap[RJ];
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int row = i * 16 + r16;
      const int pick = (rows >> row) & 1 ? row : (int)__builtin_ctzll(rows);  // rows of others: not loaded
      xp[i] = a.x + (m0 + pick) * a.K + g * 16;
    }
#pragma unroll
    for (int j = 0; j < RJ; ++j)
      ap[j] = a.a + ((int64_t)cur * a.rank + min(r0 + j * 16 + r16, rank - 1)) * a.K + g * 16;
    f32x4 acc[MI][RJ];
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int j = 0; j < RJ; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
    for (int u = u0 + wave; u < u1; u += kWaves) {
      u32x4 xr[MI][2], ar[RJ][2];
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int s = 0; s < 2; ++s) xr[i][s] = *reinterpret_cast<const u32x4 *>(xp[i] + u * 64 + s * 8);
#pragma unroll
      for (int j = 0; j < RJ; ++j)
#pragma unroll
        for (int s = 0; s < 2; ++s) ar[j][s] = *reinterpret_cast<const u32x4 *>(ap[j] + u * 64 + s * 8);
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int j = 0; j < RJ; ++j) {
          bf16x8 t[NT];
          table_terms<F16>(ar[j][s], t);
#pragma unroll
          for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int k = 0; k < NT; ++k) acc[i][j] = mfma(t[k], as_bf16x8(xr[i][s]), acc[i][j]);
        }
    }
    __syncthreads();  // the previous adapter's sums have been read
    if (wave > 0) {
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int j = 0; j < RJ; ++j) red[wave - 1][i * RJ + j][lane] = acc[i][j];
    }
    __syncthreads();
    if (wave > 0) return;
    float *v = a.v + (int64_t)blockIdx.y * a.M * a.rank;
#pragma unroll
    for (int i = 0; i < MI; ++i) {
      const int row = i * 16 + r16;
#pragma unroll
      for (int j = 0; j < RJ; ++j) {
        f32x4 t = acc[i][j];
#pragma unroll
        for (int w = 0; w < kWaves - 1; ++w) t += red[w][i * RJ + j][lane];
        const int r = r0 + j * 16 + g * 4;
        if (((rows >> row) & 1) && r < a.rank) *reinterpret_cast<f32x4 *>(v + (m0 + row) * a.rank + r) = t;
      }
    }
  });
}

// silu(g) * u with the hardware exponential and reciprocal; e^-g overflows to
// +inf for g < -88 and the quotient is then -0.
__device__ __forceinline__ float silu_mul(float g, float u) {
  return g * __builtin_amdgcn_rcpf(1.0f + __expf(-g)) * u;
}

// out = epilogue(y + scaling * B v). Block: MI*16 rows, 256 output columns, 64
// per wave: subtile s of a wave covers columns 4*c + s, so that a lane ends
// with four consecutive columns of four rows and 16 lanes store a contiguous
// 256 (fp32) or 128 bytes of a row. SwiGLU has the same columns twice, from
// the gate and the up half.
template <int MI, bool F16, typename YT, typename OT, int EPI, bool VEC>
__global__ __launch_bounds__(64 * kWaves) void adapter_up_kernel(AdapterArgs a, int slots, int splits, int col_blocks,
                                                               int skip_rows_without) {
  constexpr int NT = Terms<F16>::n;
  constexpr int HALVES = EPI == 1 ? 2 : 1;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, g = lane >> 4;
  const int64_t tile = blockIdx.x / (unsigned)col_blocks;
  const int64_t m0 = tile * (16 * MI);
  const int64_t width = EPI == 1 ? a.N / 2 : a.N;  // of out
  const int64_t n0 = (int64_t)(blockIdx.x % (unsigned)col_blocks) * (64 * kWaves) + wave * 64;
  if (n0 >= width) return;  // no barriers in this kernel
  const int64_t n = n0 + 4 * r16;
  const int id = tile_id<16 * MI>(a.row_adapter, m0, a.M, a.adapters, lane);
  each_adapter(id, skip_rows_without ? 0 : -1, blockIdx.y, slots, [&](int cur, uint64_t rows) {
    const int rank = adapter_rank(a, cur);
    f32x4 acc[HALVES][MI][4];
#pragma unroll
    for (int h = 0; h < HALVES; ++h)
#pragma unroll
      for (int i = 0; i < MI; ++i)
#pragma unroll
        for (int s = 0; s < 4; ++s) acc[h][i][s] = f32x4{0.f, 0.f, 0.f, 0.f};
    const float scaling = cur >= 0 && a.scaling ? a.scaling[cur] : 1.0f;
    for (int k0 = 0; k0 < rank; k0 += 32) {
      const int k = k0 + g * 8;
      bf16x8 bt[HALVES][4][NT];
#pragma unroll
      for (int h = 0; h < HALVES; ++h)
#pragma unroll
        for (int s = 0; s < 4; ++s) {
          const int64_t col = min(n + s, width - 1) + h * width;
          u32x4 raw = {0, 0, 0, 0};
          if (k < rank) raw = *reinterpret_cast<const u32x4 *>(a.b + ((int64_t)cur * a.N + col) * a.rank + k);
          if (k0 + 32 > rank) {
            // table entries past the adapter's own rank may hold anything
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (k + 2 * e >= rank) raw[e] = 0;
              else if (k + 2 * e + 1 >= rank) raw[e] &= 0xFFFFu;
            }
          }
          table_terms<F16>(raw, bt[h][s]);
        }
#pragma unroll
      for (int i = 0; i < MI; ++i) {
        const int row = i * 16 + r16;
        const int pick = (rows >> row) & 1 ? row : (int)__builtin_ctzll(rows);
        float f[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = 0.f;
        if (k < rank) {
          const float *p = a.v + (m0 + pick) * a.rank + k;
          F32::load8(p, 0, f);
          for (int q = 1; q < splits; ++q) {
            float o[8];
            F32::load8(p + (int64_t)q * a.M * a.rank, 0, o);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] += o[e];
          }
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = k + e < rank ? f[e] * scaling : 0.f;
        bf16x8 vt[3];
        split3(f, vt);
#pragma unroll
        for (int t = 2; t >= 0; --t)
#pragma unroll
          for (int h = 0; h < HALVES; ++h)
#pragma unroll
            for (int s = 0; s < 4; ++s)
#pragma unroll
              for (int q = 0; q < NT; ++q) acc[h][i][s] = mfma(vt[t], bt[h][s][q], acc[h][i][s]);
      }
    }
#pragma unroll
    for (int i = 0; i < MI; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = i * 16 + g * 4 + e;
        if (!((rows >> row) & 1)) continue;
        const int64_t m = m0 + row;
        float t[HALVES][4];
        auto get = [&](auto type, const void *p, int64_t at, float (&f)[4]) {
          using T = decltype(type);
          if constexpr (VEC) {
            if (n < width) T::load4(p, at, f);
          } else {
#pragma unroll
            for (int s = 0; s < 4; ++s)
              if (n + s < width) f[s] = T::load(p, at + s);
          }
        };
#pragma unroll
        for (int h = 0; h < HALVES; ++h) {
          float base[4] = {0.f, 0.f, 0.f, 0.f};
          if (a.y) get(YT{}, a.y, m * a.N + h * width + n, base);
#pragma unroll
          for (int s = 0; s < 4; ++s) t[h][s] = base[s] + acc[h][i][s][e];
        }
        float o[4];
        if constexpr (EPI == 1) {
#pragma unroll
          for (int s = 0; s < 4; ++s) o[s] = silu_mul(t[0][s], t[1][s]);
        } else if constexpr (EPI == 2) {
          float res[4] = {0.f, 0.f, 0.f, 0.f}, gt[4] = {0.f, 0.f, 0.f, 0.f};
          get(OT{}, a.residual, m * width + n, res);
          get(F32{}, a.gate, (int64_t)((uint64_t)m / (uint64_t)a.gate_rows) * width + n, gt);
#pragma unroll
          for (int s = 0; s < 4; ++s) o[s] = __builtin_fmaf(gt[s], t[0][s], res[s]);
        } else {
#pragma unroll
          for (int s = 0; s < 4; ++s) o[s] = t[0][s];
        }
        if constexpr (VEC) {
          if (n < width) OT::store4(a.out, m * width + n, o);
        } else {
#pragma unroll
          for (int s = 0; s < 4; ++s)
            if (n + s < width) OT::store(a.out, m * width + n + s, o[s]);
        }
      }
  });
}

template <int MI, int RJ>
void launch_down(const AdapterArgs &a, const AdapterPlan &p, hipStream_t stream) {
  const int units = (int)(a.K / 64), per = (units + p.splits - 1) / p.splits;
  const int chunks = (a.rank + 16 * RJ - 1) / (16 * RJ);
  const dim3 grid((unsigned)p.tiles, (unsigned)p.splits, (unsigned)(p.slots * chunks)), block(64 * kWaves);
  if (a.ab_f16) hipLaunchKernelGGL((adapter_down_kernel<MI, RJ, true>), grid, block, 0, stream, a, p.slots, per);
  else hipLaunchKernelGGL((adapter_down_kernel<MI, RJ, false>), grid, block, 0, stream, a, p.slots, per);
}

template <int MI>
void launch_down_mi(const AdapterArgs &a, const AdapterPlan &p, hipStream_t stream) {
  if (a.rank <= 16) launch_down<MI, 1>(a, p, stream);
  else if (a.rank <= 32) launch_down<MI, 2>(a, p, stream);
  else launch_down<MI, 4>(a, p, stream);
}

template <int MI, bool F16, typename YT, typename OT, int EPI>
void launch_up(const AdapterArgs &a, const AdapterPlan &p, hipStream_t stream) {
  const int64_t width = EPI == 1 ? a.N / 2 : a.N;
  const int col_blocks = (int)((width + 64 * kWaves - 1) / (64 * kWaves));
  const dim3 grid((unsigned)(p.tiles * col_blocks), (unsigned)p.slots), block(64 * kWaves);
  // without an epilogue a row without an adapter is a copy of y, which is
  // nothing to do in place
  const int skip = EPI == 0 && a.y == a.out;
  if (a.vec) hipLaunchKernelGGL((adapter_up_kernel<MI, F16, YT, OT, EPI, true>), grid, block, 0, stream, a, p.slots, p.splits, col_blocks, skip);
  else hipLaunchKernelGGL((adapter_up_kernel<MI, F16, YT, OT, EPI, false>), grid, block, 0, stream, a, p.slots, p.splits, col_blocks, skip);
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
  if (a.adapters > 0) launch_down_mi<MI>(a, p, stream);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (a.ab_f16) launch_up_types<MI, true>(a, p, stream);
  else launch_up_types<MI, false>(a, p, stream);
  return hipGetLastError();
}

}  // namespace

AdapterPlan adapter_plan(int64_t M, int64_t N, int64_t K, int rank, int64_t adapters) {
  AdapterPlan p{};
  (void)N;
  p.row_tile = M <= 256 ? 16 : 64;
  p.tiles = (M + p.row_tile - 1) / p.row_tile;
  // few tiles: blocks of their own for the adapters of one tile
  const int64_t distinct = std::min<int64_t>({M, (int64_t)p.row_tile, adapters + 1});
  p.slots = (int)std::min<int64_t>(distinct, std::max<int64_t>(1, 32 / p.tiles));
  const int chunk = rank <= 16 ? 16 : rank <= 32 ? 32 : 64;
  const int64_t blocks = p.tiles * p.slots * ((rank + chunk - 1) / chunk);
  const int64_t units = K / 64;
  int64_t splits = std::min<int64_t>({16, (units + kWaves - 1) / kWaves, (512 + blocks - 1) / blocks});
  splits = std::max<int64_t>(splits, 1);
  // no empty range
  const int64_t per = std::max<int64_t>((units + splits - 1) / splits, 1);
  p.splits = (int)std::max<int64_t>((units + per - 1) / per, 1);
  return p;
}

hipError_t launch_adapters(const AdapterArgs &a, const AdapterPlan &p, hipStream_t stream) {
  return p.row_tile == 16 ? launch_mi<1>(a, p, stream) : launch_mi<4>(a, p, stream);
}

}  // namespace ql
