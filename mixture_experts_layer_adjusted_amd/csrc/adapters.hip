// Low-rank adapters of many requests, added to a shared projection's output.
//
// Row t has the adapter e = row_adapter[t] (outside [0, n): none), with A_e [r, in], B_e [out, r], a factor s_e and
// a rank r_e <= r:  out_t = base_t + s_e B_e (A_e x_t), the ranks from r_e on left out.
//
// Two products on the bf16 matrix instruction, fp32 sums.  The first contracts 16 rows at a time over `in` (cut into
// slices where there are few rows), the second adds up the slices, takes the factor and splits the fp32 result into bf16
// parts that keep it (two parts, 16 bits, under a bf16 output; three, 24 bits, under an fp32 one), since
// the instruction multiplies bf16: a part more costs the same bytes, and bytes are what bounds both products.
//
// 16 neighbouring rows form a tile.  The rows of a tile may have different adapters: for each that occurs the whole tile is
// multiplied and the rows that have it keep the result, so every adapter in use is read once for a tile and rows need
// no sorting.  Rows of other adapters are computed and dropped, never added as zeros: an infinity or NaN stays in its row.
#include "moe_internal.h"
#include "rows.h"

namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kRows = 16;        // rows of a tile
constexpr int kCols = 64;        // output columns of a wavefront at a time

struct AdapterArgs {
  const uint16_t* x;
  const int32_t* row_adapter;
  const uint16_t *a, *b;
  const float* scale;
  const int32_t* ranks;
  const void* base;
  void* out;
  float* low;                    // [splits, rows, RT * 16]
  int64_t rows, x_ld, base_ld, out_ld;
  int in, outs, n, r;
  int splits, per_split;         // slices of the first product, values of each
  int per_block;                 // columns of a workgroup of the second product
};

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ bf16x8 vector_at(const uint16_t* p) { return *reinterpret_cast<const bf16x8*>(p); }
__device__ __forceinline__ bf16x8 no_values() { return __builtin_bit_cast(bf16x8, make_uint4(0u, 0u, 0u, 0u)); }

// the adapter of row t, -1 for none
__device__ __forceinline__ int adapter_of(const AdapterArgs& g, int64_t t) {
  const int e = t < g.rows ? g.row_adapter[t] : -1;
  return e >= 0 && e < g.n ? e : -1;
}
__device__ __forceinline__ int rank_of(const AdapterArgs& g, int e) {
  return g.ranks ? max(0, min(g.ranks[e], g.r)) : g.r;
}

// Calls f with every adapter of the wavefront's rows (mine: the lane's row's), the same in all lanes.
template <typename F>
__device__ __forceinline__ void for_adapters(int mine, F f) {
  uint64_t left = __ballot(mine >= 0);
  while (left) {
    const int e = __builtin_amdgcn_readlane(mine, __builtin_ctzll(left));
    left &= ~__ballot(mine == e);
    f(e);
  }
}

// The first product, transposed: ranks are the matrix instruction's rows, tokens its columns, so that a lane holds four
// neighbouring ranks of one token.  RT tiles of 16 ranks.  A workgroup's wavefronts take every fourth run of 32.
template <int RT>
__global__ void __launch_bounds__(kThreads) adapters_low_kernel(AdapterArgs g) {
  __shared__ float place[kWaves][kRows][RT * 16 + 4];
  const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4, wave = threadIdx.x >> 6;
  const int64_t t0 = (int64_t)blockIdx.x * kRows, t = t0 + col;
  const int begin = blockIdx.y * g.per_split, end = min(g.in, begin + g.per_split);
  const int mine = adapter_of(g, t);
  const uint16_t* x = g.x + (mine >= 0 ? t : 0) * g.x_ld;
  f32x4 kept[RT];
#pragma unroll
  for (int j = 0; j < RT; ++j) kept[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for_adapters(mine, [&](int e) {
    const int rank = rank_of(g, e);
    const uint16_t* a = g.a + ((int64_t)e * g.r + col) * g.in;
    f32x4 acc[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
    for (int k0 = begin + 32 * wave; k0 < end; k0 += 32 * kWaves) {
      const int k = k0 + 8 * quad;
      const bool in = k < end;
      const bf16x8 xv = in && mine == e ? vector_at(x + k) : no_values();
#pragma unroll
      for (int j = 0; j < RT; ++j)
        acc[j] = mfma(in && 16 * j + col < rank ? vector_at(a + (int64_t)16 * j * g.in + k) : no_values(), xv, acc[j]);
    }
    if (mine == e) {
#pragma unroll
      for (int j = 0; j < RT; ++j) kept[j] = acc[j];
    }
  });
#pragma unroll
  for (int j = 0; j < RT; ++j) *reinterpret_cast<f32x4*>(&place[wave][col][16 * j + 4 * quad]) = kept[j];
  __syncthreads();
  for (int i = threadIdx.x; i < kRows * RT * 4; i += kThreads) {
    const int row = i / (RT * 4), c = i % (RT * 4) * 4;
    if (t0 + row >= g.rows) continue;
    f32x4 s = *reinterpret_cast<f32x4*>(&place[0][row][c]);
#pragma unroll
    for (int w = 1; w < kWaves; ++w) s += *reinterpret_cast<f32x4*>(&place[w][row][c]);
    *reinterpret_cast<f32x4*>(g.low + ((int64_t)blockIdx.y * g.rows + t0 + row) * (RT * 16) + c) = s;
  }
}

// the next bf16 part of v (and what it leaves); nothing is left of what is not finite
__device__ __forceinline__ bf16x8 part_of(float (&v)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    w[i] = bf16_pair(v[2 * i], v[2 * i + 1]);
    const float lo = __uint_as_float(w[i] << 16), hi = __uint_as_float(w[i] & 0xFFFF0000u);
    v[2 * i] = fabsf(lo) < __builtin_inff() ? v[2 * i] - lo : 0.0f;
    v[2 * i + 1] = fabsf(hi) < __builtin_inff() ? v[2 * i + 1] - hi : 0.0f;
  }
  return __builtin_bit_cast(bf16x8, make_uint4(w[0], w[1], w[2], w[3]));
}

// The second product, transposed as well: output columns are the instruction's rows, in an order that leaves a lane 16
// neighbouring columns of its token (row m of tile j is column 16 (m / 4) + 4 j + m % 4 of the wavefront's 64).
// PARTS bf16 parts of the low-rank values.  RT == 1: one run of 32 holds two parts.
template <int RT, int PARTS, typename T>
__global__ void __launch_bounds__(kThreads) adapters_out_kernel(AdapterArgs g) {
  constexpr int kRuns = RT == 1 ? 1 : RT / 2;                       // runs of 32 ranks (RT == 1: 16 ranks twice)
  constexpr int kSteps = RT == 1 ? (PARTS + 1) / 2 : kRuns * PARTS;
  const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4, wave = threadIdx.x >> 6;
  const int64_t t = (int64_t)blockIdx.x * kRows + col;
  const int mine = adapter_of(g, t);
  bf16x8 low[kSteps];
  {
    const float factor = mine >= 0 ? g.scale[mine] : 0.0f;
#pragma unroll
    for (int run = 0; run < kRuns; ++run) {
      const int rank = RT == 1 ? 8 * (quad & 1) : 32 * run + 8 * quad;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.0f;
      if (mine >= 0) {
        const float* p = g.low + t * (RT * 16) + rank;
        for (int s = 0; s < g.splits; ++s) {
          float u[8];
          load8(p + (int64_t)s * g.rows * (RT * 16), u);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] += u[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= factor;
      }
      if constexpr (RT == 1) {
        bf16x8 part[2 * kSteps];
#pragma unroll
        for (int p = 0; p < 2 * kSteps; ++p) part[p] = p < PARTS ? part_of(v) : no_values();
#pragma unroll
        for (int s = 0; s < kSteps; ++s) low[s] = quad < 2 ? part[2 * s] : part[2 * s + 1];
      } else {
#pragma unroll
        for (int p = 0; p < PARTS; ++p) low[p * kRuns + run] = part_of(v);
      }
    }
  }
  const int first = blockIdx.y * g.per_block, end = min(g.outs, first + g.per_block);
  for (int c0 = first + kCols * wave; c0 < end; c0 += kCols * kWaves) {
    const int c = c0 + 16 * quad;   // the lane's 16 columns
    float was[16];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[8];
      if (g.base && t < g.rows && c + 8 * h < g.outs) {
        load8(static_cast<const T*>(g.base) + t * g.base_ld + c + 8 * h, v);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.0f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) was[8 * h + i] = v[i];
    }
    f32x4 kept[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) kept[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for_adapters(mine, [&](int e) {
      const int rank = rank_of(g, e);
      f32x4 acc[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int bc = c0 + 16 * (col >> 2) + 4 * j + (col & 3);
        const uint16_t* b = g.b + ((int64_t)e * g.outs + bc) * g.r;
        acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        bf16x8 bv[kRuns];
#pragma unroll
        for (int run = 0; run < kRuns; ++run) {
          const int k = RT == 1 ? 8 * (quad & 1) : 32 * run + 8 * quad;
          bv[run] = bc < g.outs && k < rank ? vector_at(b + k) : no_values();
          if (k < rank && k + 8 > rank) {   // the rank ends inside: what is behind it does not count, whatever it holds
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (k + i >= rank) bv[run][i] = (__bf16)0.0f;
          }
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s) acc[j] = mfma(bv[RT == 1 ? 0 : s % kRuns], low[s], acc[j]);
      }
      if (mine == e) {
#pragma unroll
        for (int j = 0; j < 4; ++j) kept[j] = acc[j];
      }
    });
    if (t >= g.rows) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (c + 8 * h >= g.outs) continue;
      float v[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {   // (a row without an adapter keeps its base to the sign of a zero)
        const float d = kept[2 * h + i / 4][i % 4];
        v[i] = mine >= 0 ? was[8 * h + i] + d : was[8 * h + i];
      }
      store8(static_cast<T*>(g.out) + t * g.out_ld + c + 8 * h, v);
    }
  }
}

struct AdapterPlan {
  int tiles16;                   // RT
  int splits, per_split, per_block;
};

// Slices of the first product: some 512 workgroups, each of 256 values at least.
AdapterPlan plan_of(const moe_adapter_shape& s) {
  AdapterPlan p;
  p.tiles16 = s.rank <= 16 ? 1 : s.rank <= 32 ? 2 : s.rank <= 64 ? 4 : 8;
  const int64_t tiles = ceil_div(s.rows, kRows);
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(ceil_div(512, std::max<int64_t>(1, tiles)), ceil_div(s.in_cols, 256)));
  p.per_split = (int)(ceil_div(ceil_div(s.in_cols, want), 128) * 128);
  p.splits = (int)ceil_div(s.in_cols, p.per_split);
  int64_t blocks = ceil_div(1024, std::max<int64_t>(1, tiles));
  p.per_block = (int)(ceil_div(ceil_div(s.out_cols, blocks), kCols * kWaves) * kCols * kWaves);
  return p;
}

template <int RT>
hipError_t run_t(const AdapterArgs& g, int out_dtype, hipStream_t st) {
  const unsigned tiles = (unsigned)ceil_div(g.rows, kRows);
  const hipError_t err = launch_kernel(adapters_low_kernel<RT>, dim3(tiles, (unsigned)g.splits), dim3(kThreads), 0, st, g);
  if (err != hipSuccess) return err;
  const dim3 grid(tiles, (unsigned)ceil_div(g.outs, g.per_block));
  return out_dtype == MOE_DTYPE_F32 ? launch_kernel(adapters_out_kernel<RT, 3, float>, grid, dim3(kThreads), 0, st, g)
                                    : launch_kernel(adapters_out_kernel<RT, 2, uint16_t>, grid, dim3(kThreads), 0, st, g);
}

}  // namespace

size_t adapters_workspace(const moe_adapter_shape& s) {
  const AdapterPlan p = plan_of(s);
  return (size_t)p.splits * s.rows * p.tiles16 * 16 * 4;
}

hipError_t launch_adapters(const moe_adapter_shape& s, const void* x, const int32_t* row_adapter, const void* a, const void* b,
                           const float* scale, const int32_t* ranks, const void* base, void* out, float* low,
                           hipStream_t st) {
  const AdapterPlan p = plan_of(s);
  const AdapterArgs g{static_cast<const uint16_t*>(x),
                      row_adapter,
                      static_cast<const uint16_t*>(a),
                      static_cast<const uint16_t*>(b),
                      scale,
                      ranks,
                      base,
                      out,
                      low,
                      s.rows,
                      s.x_ld ? s.x_ld : s.in_cols,
                      s.base_ld ? s.base_ld : s.out_cols,
                      s.out_ld ? s.out_ld : s.out_cols,
                      s.in_cols,
                      s.out_cols,
                      s.n_adapters,
                      s.rank,
                      p.splits,
                      p.per_split,
                      p.per_block};
  switch (p.tiles16) {
    case 1: return run_t<1>(g, s.out_dtype, st);
    case 2: return run_t<2>(g, s.out_dtype, st);
    case 4: return run_t<4>(g, s.out_dtype, st);
    default: return run_t<8>(g, s.out_dtype, st);
  }
}

}  // namespace moe
