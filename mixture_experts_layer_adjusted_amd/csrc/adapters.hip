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

constexpr int kWaves = 4, kThreads = 64 * kWaves;
constexpr int kRows = 16;        // rows of a tile
constexpr int kStep = 64;        // values of a wavefront's step along the first product's contraction
constexpr int kCols = 64;        // output columns of a wavefront at a time
constexpr int kLeadRows = 128;   // rows at most where workgroups go by adapters

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
  int blocks, per_block;         // workgroups of a tile in the second product, columns of each
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

// The rows of a workgroup that goes by adapters: `first` is its row, and if that is the first one with its adapter e
// (or the first without one) the workgroup takes all rows that have the same; otherwise there are none.  Every wavefront
// finds them by itself: a ballot for each 64 rows, and a permutation that brings the rows of e to the lanes in front.
struct LeadRows {
  int count, low, high;   // rows number 0 to 63 and 64 to 127 of e, one a lane
  __device__ __forceinline__ int at(int i) const { return i < 64 ? __shfl(low, i, 64) : __shfl(high, i - 64, 64); }
};
__device__ __forceinline__ int bits_below(uint64_t m) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
}
__device__ __forceinline__ LeadRows lead_rows(const AdapterArgs& g, int first, int e) {
  const int lane = threadIdx.x & 63;
  const bool is0 = lane < g.rows && adapter_of(g, lane) == e, is1 = lane + 64 < g.rows && adapter_of(g, lane + 64) == e;
  const uint64_t m0 = __ballot(is0), m1 = __ballot(is1);
  const uint64_t before = (uint64_t(1) << (first & 63)) - 1;
  LeadRows l{0, 0, 0};
  if (first < 64 ? (m0 & before) != 0 : (m0 != 0 || (m1 & before) != 0)) return l;
  const int n0 = __popcll(m0), n1 = __popcll(m1), b0 = bits_below(m0), b1 = bits_below(m1);
  const int to0 = is0 ? b0 : n0 + lane - b0, to1 = (n0 + (is1 ? b1 : n1 + lane - b1)) & 63;
  const int p0 = __builtin_amdgcn_ds_permute(4 * to0, lane), p1 = __builtin_amdgcn_ds_permute(4 * to1, lane + 64);
  l.count = n0 + n1;
  l.low = lane < n0 ? p0 : p1;
  l.high = p1;
  return l;
}

// The operands of one step of the first product: 64 values along the contraction, two of the instruction's
template <int RT>
struct LowStep {
  bf16x8 x[2], a[2][RT];
};

// The first product, transposed: ranks are the matrix instruction's rows, tokens its columns, so that a lane holds four
// neighbouring ranks of one token.  RT tiles of 16 ranks.  A workgroup's wavefronts take every fourth run of 64.
template <int RT, bool LEAD>
__global__ void __launch_bounds__(kThreads) adapters_low_kernel(AdapterArgs g) {
  constexpr int kAhead = RT == 1 ? 3 : RT <= 4 ? 2 : 1;   // steps whose operands are in flight
  constexpr int kStride = kStep * kWaves;
  __shared__ float place[kWaves][kRows][RT * 16 + 4];
  const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t tile = blockIdx.x / g.splits;
  const int slice = blockIdx.x - (unsigned)tile * g.splits, begin = slice * g.per_split, end = min(g.in, begin + g.per_split);
  // whole steps of the wavefront, and where a last one may end early
  const int first = begin + kStep * wave, n = first + kStep <= end ? (end - kStep - first) / kStride + 1 : 0;
  const int tail = first + n * kStride;
  LeadRows rows{kRows, 0, 0};
  int leader = -1;
  if constexpr (LEAD) {
    leader = adapter_of(g, tile);
    if (leader < 0) return;
    rows = lead_rows(g, (int)tile, leader);
  }
  for (int group = 0; group < rows.count; group += kRows) {
    int64_t t;
    int mine;
    if constexpr (LEAD) {
      t = rows.at(min(group + col, rows.count - 1));
      mine = group + col < rows.count ? leader : -1;
    } else {
      t = tile * kRows + col;
      mine = adapter_of(g, t);
    }
    // (32-bit offsets from the first row of the tile, or of all)
    const uint16_t* x = g.x + (LEAD ? 0 : tile * kRows * g.x_ld);
    const uint32_t at = mine < 0 ? 0u : (LEAD ? (uint32_t)t : (uint32_t)col) * (uint32_t)g.x_ld;
    f32x4 kept[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) kept[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    for_adapters(mine, [&](int e) {
      const int rank = rank_of(g, e);
      if (rank == 0) return;
      const uint16_t* a = g.a + (int64_t)e * g.r * g.in;
      uint32_t row[RT];   // of A; rows past the rank repeat the last one, their sums are dropped
#pragma unroll
      for (int j = 0; j < RT; ++j) row[j] = (uint32_t)min(16 * j + col, rank - 1) * (uint32_t)g.in;
      f32x4 acc[RT];
#pragma unroll
      for (int j = 0; j < RT; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      LowStep<RT> step[kAhead];
      auto load = [&](LowStep<RT>& s, int i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t k = first + i * kStride + 32 * h + 8 * quad;
          s.x[h] = vector_at(x + (at + k));
#pragma unroll
          for (int j = 0; j < RT; ++j) s.a[h][j] = vector_at(a + (row[j] + k));
        }
      };
      auto multiply = [&](const LowStep<RT>& s) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < RT; ++j) acc[j] = mfma(s.a[h][j], s.x[h], acc[j]);
      };
      if (n >= kAhead) {   // (no load under a condition before the last steps: each is waited for alone)
        int i = 0;
#pragma unroll
        for (int d = 0; d < kAhead; ++d) load(step[d], d);
        for (; i + 2 * kAhead <= n; i += kAhead) {
#pragma unroll
          for (int d = 0; d < kAhead; ++d) {
            multiply(step[d]);
            load(step[d], i + d + kAhead);
          }
        }
#pragma unroll
        for (int d = 0; d < kAhead; ++d) {
          multiply(step[d]);
          if (i + d + kAhead < n) load(step[d], i + d + kAhead);
        }
#pragma unroll
        for (int d = 0; d < kAhead; ++d)
          if (i + d + kAhead < n) multiply(step[d]);
      } else {
#pragma unroll
        for (int d = 0; d < kAhead; ++d)
          if (d < n) load(step[d], d);
#pragma unroll
        for (int d = 0; d < kAhead; ++d)
          if (d < n) multiply(step[d]);
      }
      if (tail < end) {   // the contraction ends inside this step
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t k = tail + 32 * h + 8 * quad;
          const bool in = (int)k < end;
          const bf16x8 xv = in ? vector_at(x + (at + k)) : no_values();
#pragma unroll
          for (int j = 0; j < RT; ++j) acc[j] = mfma(in ? vector_at(a + (row[j] + k)) : no_values(), xv, acc[j]);
        }
      }
      if (mine == e) {
#pragma unroll
        for (int j = 0; j < RT; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) kept[j][i] = 16 * j + 4 * quad + i < rank ? acc[j][i] : 0.0f;
      }
    });
    if (LEAD && group > 0) __syncthreads();
#pragma unroll
    for (int j = 0; j < RT; ++j) *reinterpret_cast<f32x4*>(&place[wave][col][16 * j + 4 * quad]) = kept[j];
    __syncthreads();
    for (int i = threadIdx.x; i < kRows * RT * 4; i += kThreads) {
      const int row = i / (RT * 4), c = i % (RT * 4) * 4;
      int64_t to;
      bool in;
      if constexpr (LEAD) {
        in = group + row < rows.count;
        to = rows.at(min(group + row, rows.count - 1));
      } else {
        to = tile * kRows + row;
        in = to < g.rows;
      }
      f32x4 s = *reinterpret_cast<f32x4*>(&place[0][row][c]);
#pragma unroll
      for (int w = 1; w < kWaves; ++w) s += *reinterpret_cast<f32x4*>(&place[w][row][c]);
      if (in) *reinterpret_cast<f32x4*>(g.low + ((int64_t)slice * g.rows + to) * (RT * 16) + c) = s;
    }
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
template <int RT, int PARTS, typename T, bool LEAD>
__global__ void __launch_bounds__(kThreads) adapters_out_kernel(AdapterArgs g) {
  constexpr int kRuns = RT == 1 ? 1 : RT / 2;                       // runs of 32 ranks (RT == 1: 16 ranks twice)
  constexpr int kSteps = RT == 1 ? (PARTS + 1) / 2 : kRuns * PARTS;
  constexpr int kBatch = 8, kShares = 8;   // slices loaded at once; threads at most that share one value's slices
  constexpr int kStride = kCols * kWaves;
  struct Operands {
    Raw8<T> base[2];
    bf16x8 b[4][kRuns];
  };
  __shared__ f32x4 sums[kRows * RT * 4 > kThreads ? kRows * RT * 4 : kThreads];
  const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t tile = blockIdx.x / g.blocks;
  const int block = blockIdx.x - (unsigned)tile * g.blocks;
  const int first = block * g.per_block + kCols * wave, end = min(g.outs, (block + 1) * g.per_block);
  LeadRows rows{kRows, 0, 0};
  int leader = -1;
  if constexpr (LEAD) {
    leader = adapter_of(g, tile);
    rows = lead_rows(g, (int)tile, leader);
  }
  for (int group = 0; group < rows.count; group += kRows) {
    const int here = LEAD ? min(kRows, rows.count - group) : kRows;   // rows of the tile
    auto row_of = [&](int i) -> int64_t {
      if constexpr (LEAD) return rows.at(min(group + i, rows.count - 1));
      else return tile * kRows + i;
    };
    const int64_t t = row_of(col);
    const bool real = LEAD ? col < here : t < g.rows;
    const int64_t row = t < g.rows ? t : g.rows - 1;   // (lanes without a row load another's values, and drop them)
    const int mine = LEAD ? (real ? leader : -1) : adapter_of(g, t);
    const uint64_t with = __ballot(mine >= 0);
    const int e0 = with ? __builtin_amdgcn_readlane(mine, __builtin_ctzll(with)) : -1;
    // one adapter in the tile (and the registers for a second set of operands)
    const bool alone = RT <= 4 && __ballot(mine >= 0 && mine != e0) == 0 && with != 0;
    auto load_base = [&](Raw8<T> (&v)[2], int c0) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        v[h] = raw_at(static_cast<const T*>(g.base) + row * g.base_ld + min(c0 + 16 * quad + 8 * h, g.outs - 8));
    };
    auto load_b = [&](bf16x8 (&v)[4][kRuns], int e, int c0) {
      const uint16_t* b = g.b + (int64_t)e * g.outs * g.r;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t bc = (uint32_t)min(c0 + 16 * (col >> 2) + 4 * j + (col & 3), g.outs - 1) * (uint32_t)g.r;
#pragma unroll
        for (int run = 0; run < kRuns; ++run)
          v[j][run] = vector_at(b + (bc + (uint32_t)min(RT == 1 ? 8 * (quad & 1) : 32 * run + 8 * quad, g.r - 8)));
      }
    };
    Operands now{};
    if (alone && first < end) load_b(now.b, e0, first);
    if (g.base && first < end) load_base(now.base, first);
    bf16x8 low[kSteps];
    if (with) {   // (the wavefronts of a workgroup have the same rows)
      if (LEAD && group > 0) __syncthreads();
      // the slices' sums, slices shared out among threads and loaded in batches
      const int items = here * RT * 4, shares = max(1, min(kShares, kThreads / items));
      for (int i0 = 0; i0 < items * shares; i0 += kThreads) {   // (all lanes: row_of reads other lanes' values)
        const int i = min(i0 + (int)threadIdx.x, items * shares - 1), share = i / items, item = i - share * items;
        const int64_t from = row_of(item / (RT * 4));
        f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
        const float* p = g.low + (from < g.rows ? from : g.rows - 1) * (RT * 16) + item % (RT * 4) * 4;
        for (int s0 = share; s0 < g.splits; s0 += shares * kBatch) {
          f32x4 v[kBatch];
#pragma unroll
          for (int b = 0; b < kBatch; ++b)
            v[b] = *reinterpret_cast<const f32x4*>(p + (int64_t)min(s0 + b * shares, g.splits - 1) * g.rows * (RT * 16));
#pragma unroll
          for (int b = 0; b < kBatch; ++b) sum += s0 + b * shares < g.splits ? v[b] : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        }
        sums[i] = sum;
      }
      const float factor = mine >= 0 ? g.scale[mine] : 0.0f;
      __syncthreads();
#pragma unroll
      for (int run = 0; run < kRuns; ++run) {
        const int at = min(col, here - 1) * RT * 4 + (RT == 1 ? 2 * (quad & 1) : 8 * run + 2 * quad);
        f32x4 lo = sums[at], hi = sums[at + 1];
        for (int w = 1; w < shares; ++w) {
          lo += sums[w * items + at];
          hi += sums[w * items + at + 1];
        }
        float v[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = mine >= 0 ? lo[i] * factor : 0.0f;
          v[4 + i] = mine >= 0 ? hi[i] * factor : 0.0f;
        }
        if constexpr (RT == 1) {
#pragma unroll
          for (int s = 0; s < kSteps; ++s) {   // the lower half of the lanes has one part, the upper half the next
            const bf16x8 even = part_of(v), odd = 2 * s + 1 < PARTS ? part_of(v) : no_values();
            low[s] = quad < 2 ? even : odd;
          }
        } else {
#pragma unroll
          for (int p = 0; p < PARTS; ++p) low[p * kRuns + run] = part_of(v);
        }
      }
    }
    // kept = the products with adapter e's rows of B, for the tokens that have e
    auto multiply = [&](bf16x8 (&bv)[4][kRuns], int e, int rank, f32x4 (&kept)[4]) {
      if (rank < RT * 16) {   // what is behind the rank does not count, whatever it holds
#pragma unroll
        for (int run = 0; run < kRuns; ++run) {
          const int left = rank - (RT == 1 ? 8 * (quad & 1) : 32 * run + 8 * quad);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint4 q = __builtin_bit_cast(uint4, bv[j][run]);
            q.x &= left > 1 ? ~0u : left > 0 ? 0xFFFFu : 0u;
            q.y &= left > 3 ? ~0u : left > 2 ? 0xFFFFu : 0u;
            q.z &= left > 5 ? ~0u : left > 4 ? 0xFFFFu : 0u;
            q.w &= left > 7 ? ~0u : left > 6 ? 0xFFFFu : 0u;
            bv[j][run] = __builtin_bit_cast(bf16x8, q);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < kSteps; ++s) acc = mfma(bv[j][RT == 1 ? 0 : s % kRuns], low[s], acc);
        if (mine == e) kept[j] = acc;
      }
    };
    auto store = [&](const Raw8<T> (&base)[2], const f32x4 (&kept)[4], int c0) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int c = c0 + 16 * quad + 8 * h;   // the lane's 16 columns
        if (!real || c >= g.outs) continue;
        float v[8];
        unpack8(base[h], v);
#pragma unroll
        for (int i = 0; i < 8; ++i)   // (a row without an adapter keeps its base to the sign of a zero)
          v[i] = mine >= 0 ? v[i] + kept[2 * h + i / 4][i % 4] : v[i];
        store8(static_cast<T*>(g.out) + t * g.out_ld + c, v);
      }
    };
    const f32x4 none = {0.0f, 0.0f, 0.0f, 0.0f};
    if (alone) {   // the next columns' operands on their way while these are worked on
      const int rank = rank_of(g, e0);
      int c0 = first;
      for (; c0 + kStride < end; c0 += kStride) {
        Operands next{};
        load_b(next.b, e0, c0 + kStride);
        if (g.base) load_base(next.base, c0 + kStride);
        f32x4 kept[4] = {none, none, none, none};
        multiply(now.b, e0, rank, kept);
        store(now.base, kept, c0);
        now = next;
      }
      if (c0 < end) {
        f32x4 kept[4] = {none, none, none, none};
        multiply(now.b, e0, rank, kept);
        store(now.base, kept, c0);
      }
    } else {
      for (int c0 = first; c0 < end; c0 += kStride) {
        f32x4 kept[4] = {none, none, none, none};
        if (g.base && c0 > first) load_base(now.base, c0);
        for_adapters(mine, [&](int e) {
          load_b(now.b, e, c0);
          multiply(now.b, e, rank_of(g, e), kept);
        });
        store(now.base, kept, c0);
      }
    }
  }
}

struct AdapterPlan {
  int tiles16;                   // RT
  bool lead;                     // workgroups go by adapters
  int splits, per_split, blocks, per_block;
};

AdapterPlan plan_of(const moe_adapter_shape& s) {
  AdapterPlan p;
  p.tiles16 = s.rank <= 16 ? 1 : s.rank <= 32 ? 2 : s.rank <= 64 ? 4 : 8;
  p.lead = s.rows <= kLeadRows;
  const int64_t tiles = std::max<int64_t>(1, ceil_div(s.rows, kRows)), run = kStep * kWaves;
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(ceil_div(2048, tiles), ceil_div(s.in_cols, run)));
  p.per_split = (int)(ceil_div(ceil_div(s.in_cols, want), run) * run);
  p.splits = (int)ceil_div(s.in_cols, p.per_split);
  p.per_block = (int)(ceil_div(ceil_div(s.out_cols, ceil_div(2048, tiles)), kCols * kWaves) * kCols * kWaves);
  p.blocks = (int)ceil_div(s.out_cols, p.per_block);
  return p;
}

template <int RT, bool LEAD>
hipError_t run_t(const AdapterArgs& g, int out_dtype, hipStream_t st) {
  // (the slices or columns of a tile are neighbours in the grid: workgroups at work together cover whole rows)
  const unsigned tiles = (unsigned)(LEAD ? g.rows : ceil_div(g.rows, kRows));
  const hipError_t err = launch_kernel(adapters_low_kernel<RT, LEAD>, dim3(tiles * g.splits), dim3(kThreads), 0, st, g);
  if (err != hipSuccess) return err;
  const dim3 grid(tiles * g.blocks);
  return out_dtype == MOE_DTYPE_F32
             ? launch_kernel(adapters_out_kernel<RT, 3, float, LEAD>, grid, dim3(kThreads), 0, st, g)
             : launch_kernel(adapters_out_kernel<RT, 2, uint16_t, LEAD>, grid, dim3(kThreads), 0, st, g);
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
                      p.blocks,
                      p.per_block};
  switch (p.tiles16) {
    case 1: return p.lead ? run_t<1, true>(g, s.out_dtype, st) : run_t<1, false>(g, s.out_dtype, st);
    case 2: return p.lead ? run_t<2, true>(g, s.out_dtype, st) : run_t<2, false>(g, s.out_dtype, st);
    case 4: return p.lead ? run_t<4, true>(g, s.out_dtype, st) : run_t<4, false>(g, s.out_dtype, st);
    default: return p.lead ? run_t<8, true>(g, s.out_dtype, st) : run_t<8, false>(g, s.out_dtype, st);
  }
}

}  // namespace moe
