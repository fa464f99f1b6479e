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
// Few rows of many adapters (a decode batch) go by adapters instead: a workgroup finds 16 rows of one.
//
// Bound by memory at many rows (traced): 8192 x 7168 -> 4096, rank 16, bf16: 30.3 us for the first product (121 MB, 4.0 TB/s), 33
// for the second (134 MB and B, 4.1 TB/s); by latency at few (one row 3.7 + 4.3 us).  Operands loaded as the matrix instruction
// wants them took 37 + 37 us: the address unit takes a lane at a time there (57 accesses a load in place of 16).
#include "moe_internal.h"
#include "rows.h"

namespace moe {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int16_t s16x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4, kThreads = 64 * kWaves, kWavesOfTile = kWaves;
constexpr int kRows = 16;        // rows of a tile, or of an adapter at a time
constexpr int kStep = 64;        // values of a wavefront's step along the first product's contraction
constexpr int kCols = 64;        // output columns of a wavefront at a time
// Workgroups go by adapters (16 rows of one each) up to so many rows, which each of them looks through, and rows for each adapter
// there is: they read an adapter once for 16 of its rows, a tile of neighbouring rows reads all of its adapters one after the
// other.  In a graph, us, by adapters against by tiles, rows of all adapters mixed, then side by side, then all rows on one
// adapter: 32 adapters of rank 64, 7168 -> 4096: 64 rows 15.0, 31.2; 14.5, 22.6; 12.4, 9.9.  500 rows 21.7, 60; 22.4, 25.6; 16.8,
// 16.5.  1000 rows 30, 138; 31, 34; 24.1, 22.5.  256 of rank 16, 2048 -> 4096: 256 rows 16.0, 22.6; 16.5, 21.2; 15.3, 6.9 (the
// largest loss found); 1000 rows 19.6, 28.3; 19.7, 19.7; 17.6, 10.9.  8 of rank 16, 7168 -> 4096: 128 rows 10.1, 13.4; 10.2, 9.3;
// 9.8, 7.3; above 16 rows an adapter (32 above rank 32) tiles are at least as good side by side and hold few adapters each.  (A
// workgroup for each adapter and all of its rows: 269 with all of 1000 rows on one of 64 adapters of rank 16, 742 on one of 256.)
constexpr int kUnitRows = 1024, kUnitShare = 16;
// Workgroups of a product, or so.  By adapters about as many as the registers let run at once (in a graph, us, 256, 512, 1024,
// mixed: 64 rows, 32 adapters of rank 64, 7168 -> 4096: 15.7, 15.0, 16.2; 500 rows 22.6, 21.7, 24.6; 256 rows, 256 of rank 16,
// 2048 -> 4096: 20.1, 15.9, 15.1; 1000 rows 23.4, 19.6, 22.6).  By tiles 2048, 1024 above rank 32
// (rows of one adapter side by side, 1024 against 2048: 2000 rows of 8 adapters of rank 64, 4096 -> 4096 29.3, 35.2; 600 rows,
// 2048 -> 7168 21.1, 20.1; 2000 rows of 4 of rank 128 47, 58; of rank 16, 7168 -> 4096: 8192 rows 71.5, 61.4)
constexpr int kTileBlocks = 2048, kUnitBlocks = 512;
// One launch in place of two up to so many rows and values of an adapter's A, which every workgroup then reads whole.
// In a graph, us, one kernel against two: 1 row, 16 x 2048 -> 7168: 5.4, 7.1; 16 rows, 32 x 2048 -> 4096: 7.5, 7.7;
// 1 row, 16 x 7168 -> 4096: 8.2, 7.1; 32 rows, 32 x 2048 -> 4096: 8.5, 8.4.
constexpr int kFewRows = 16, kFewValues = 1 << 16;

struct AdapterArgs {
  const uint16_t* x;
  const int32_t* row_adapter;
  const uint16_t *a, *b;
  const float* scale;
  const int32_t* ranks;
  const void* base;
  void* out;
  float* low;                    // [splits, rows, RT * 16]
  int2* found;                   // by adapters: [units, 16] rows and adapters, row -1: none
  int64_t rows, x_ld, base_ld, out_ld;
  int in, outs, n, r;
  int splits, per_split;         // slices of the first product, values of each
  int blocks, per_block;         // workgroups of a tile in the second product, columns of each
  int units;                     // by adapters: groups of rows at most, or adapters (or rows) for few rows
};

__device__ __forceinline__ f32x4 mfma(bf16x8 a, bf16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
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

// The rows of a workgroup that goes by adapters: up to 16 of one adapter, as every wavefront has them.
struct UnitRows {
  int count;          // 0 to 16
  int row, adapter;   // lane i < count: the i-th
};
__device__ __forceinline__ int bits_below(uint64_t m) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(m >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)m, 0));
}
// Rows by adapters are cut into groups of 16, in their order.  Up to kScanRows rows, a unit is first an adapter (with fewer
// rows than adapters: a row, which stands for its adapter if it is the first to have it) and its first 16 rows, which every
// wavefront finds by itself, a ballot for each 64 rows and a permutation that brings those of the adapter to the lanes in
// front; then a number among the further groups.  Beyond, a unit is a number among all groups.  (In a graph, us, against numbers
// among all groups from the first row on, mixed: 64 rows of 64 adapters of rank 16, 7168 -> 4096: 10.6, 12.0; 140 rows of 32 of
// rank 64 16.5, 17.8; 256 rows of 64 of rank 16 14.1, 14.3.)
constexpr int kScanRows = 256;
__host__ __device__ inline int first_units(int64_t rows, int n) { return rows < n ? (int)rows : n; }
__device__ __forceinline__ UnitRows first_rows(const AdapterArgs& g, int unit) {
  const int lane = threadIdx.x & 63, rows = (int)g.rows;
  const bool leads = rows < g.n;
  const int own = leads ? g.row_adapter[unit] : unit;   // (on its way with the rows)
  int e[kScanRows / 64];
#pragma unroll
  for (int k = 0; k < kScanRows / 64; ++k) e[k] = g.row_adapter[min(64 * k + lane, rows - 1)];
  UnitRows u{0, 0, own};
  if (own < 0 || own >= g.n) return u;
#pragma unroll
  for (int k = 0; k < kScanRows / 64; ++k) {
    const int r = 64 * k + lane;
    if (64 * k >= rows || u.count >= kRows) break;
    const bool has = r < rows && e[k] == own;
    const uint64_t m = __ballot(has);
    if (m == 0) continue;
    if (leads && u.count == 0 && 64 * k + __builtin_ctzll(m) != unit) return u;
    const int at = u.count + bits_below(m), more = __builtin_amdgcn_ds_permute(4 * (has && at < kRows ? at : kRows), r);
    if (lane >= u.count) u.row = more;
    u.count += __popcll(m);
  }
  u.count = min(kRows, u.count);
  return u;
}

// A unit that is a group's number, of up to kUnitRows rows; further: among those behind an adapter's first.  The workgroup
// counts the rows of every adapter in LDS, adds up their groups, and gives the rows of its own their places, which go by the
// rows' order alone.  (Above kBuckets adapters, those that are alike in their last bits together: a group may have rows of
// several.)
constexpr int kBuckets = 4 * kThreads;
// whether first_rows finds the first groups
__device__ __forceinline__ bool scanned(const AdapterArgs& g) { return g.rows <= kScanRows && g.n <= kBuckets; }
struct GroupLds {
  int rows_of[kBuckets];
  int groups[kWaves];                    // of a wavefront's buckets
  int bucket, group;                     // the unit's
  int matches[kUnitRows / 64];           // of each 64 rows
  int row[kRows], adapter[kRows];
};
__device__ __forceinline__ UnitRows group_rows(const AdapterArgs& g, int unit, bool further, GroupLds& lds) {
  constexpr int kEach = kUnitRows / kThreads;
  static_assert(kEach * kThreads == kUnitRows && kWaves == 4, "rows of a thread, totals of the wavefronts");
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, rows = (int)g.rows;
  int e[kEach];
#pragma unroll
  for (int k = 0; k < kEach; ++k) e[k] = g.row_adapter[min(k * kThreads + tid, rows - 1)];
  reinterpret_cast<int4*>(lds.rows_of)[tid] = make_int4(0, 0, 0, 0);
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    if (k * kThreads + tid >= rows || e[k] < 0 || e[k] >= g.n) e[k] = -1;
    if (e[k] >= 0) atomicAdd(&lds.rows_of[e[k] & (kBuckets - 1)], 1);
  }
  __syncthreads();
  const int4 c = reinterpret_cast<const int4*>(lds.rows_of)[tid];
  auto groups = [&](int n) { return (int)((uint32_t)max(0, n + (further ? -1 : kRows - 1)) / kRows); };
  const int q[4] = {groups(c.x), groups(c.y), groups(c.z), groups(c.w)};
  const int own = q[0] + q[1] + q[2] + q[3];
  int upto = own;   // with the lanes before: row_shr 1, 2, 4, 8, then the last lane of the row, of the half before
  upto += __builtin_amdgcn_update_dpp(0, upto, 0x111, 0xF, 0xF, true);
  upto += __builtin_amdgcn_update_dpp(0, upto, 0x112, 0xF, 0xF, true);
  upto += __builtin_amdgcn_update_dpp(0, upto, 0x114, 0xF, 0xF, true);
  upto += __builtin_amdgcn_update_dpp(0, upto, 0x118, 0xF, 0xF, true);
  upto += __builtin_amdgcn_update_dpp(0, upto, 0x142, 0xA, 0xF, false);
  upto += __builtin_amdgcn_update_dpp(0, upto, 0x143, 0xC, 0xF, false);
  if (lane == 63) lds.groups[wave] = upto;
  __syncthreads();
  int before = upto - own, total = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    before += w < wave ? lds.groups[w] : 0;
    total += lds.groups[w];
  }
  if (unit >= total) return {0, 0, -1};   // (all threads)
  if (unit >= before && unit < before + own) {
    int bucket = 0, group = unit - before;
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (bucket == i && group >= q[i]) {
        group -= q[i];
        bucket = i + 1;
      }
    lds.bucket = 4 * tid + bucket;
    lds.group = group;
  }
  __syncthreads();
  const int bucket = lds.bucket, from = (lds.group + further) * kRows;
  uint64_t m[kEach];
#pragma unroll
  for (int k = 0; k < kEach; ++k) {
    m[k] = __ballot(e[k] >= 0 && (e[k] & (kBuckets - 1)) == bucket);
    if (lane == 0) lds.matches[k * kWaves + wave] = __popcll(m[k]);
  }
  __syncthreads();
  int seen = 0;
#pragma unroll
  for (int i = 0; i < kEach * kWaves; ++i) {
    if (i % kWaves == wave) {
      const int k = i / kWaves, at = seen + bits_below(m[k]) - from;
      if ((m[k] >> lane & 1) && at >= 0 && at < kRows) {
        lds.row[at] = k * kThreads + tid;
        lds.adapter[at] = e[k];
      }
    }
    seen += lds.matches[i];
  }
  __syncthreads();
  return {min(kRows, seen - from), lds.row[lane & (kRows - 1)], lds.adapter[lane & (kRows - 1)]};
}

// One step of the first product for a tile of 16 rows (of x, or of A): 64 values of each, as they are loaded.  Eight
// neighbouring lanes load a row's 128 bytes: the matrix instruction wants neighbouring lanes on different rows, which
// the address unit takes one lane at a time (64 cycles a load in place of 16: the bound of both products before), so the
// values go through LDS.  There chunk c of row m lies at c ^ (m mod 8): no two lanes of a read on the same banks.
struct StepTile {
  u32x4 q[2];   // rows lane / 8 and 8 + lane / 8
};
constexpr int kTileBytes = kRows * kStep * 2;
__device__ __forceinline__ void tile_to_lds(char* to, const StepTile& s, int lane) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int m = 8 * h + (lane >> 3);
    *reinterpret_cast<u32x4*>(to + m * 128 + ((lane & 7) ^ (m & 7)) * 16) = s.q[h];
  }
}
// the instruction's operand for half h of the step
__device__ __forceinline__ bf16x8 tile_operand(const char* from, int h, int lane) {
  const int m = lane & 15;
  return *reinterpret_cast<const bf16x8*>(from + m * 128 + ((4 * h + (lane >> 4)) ^ (m & 7)) * 16);
}

// LDS of a wavefront in the first product: a tile of x and up to four of A; the sums then take their place
template <int RT>
struct LowLds {
  static constexpr int kAtOnce = RT < 4 ? RT : 4;
  static constexpr int kPitch = RT * 16 + 4;   // values between the sums of neighbouring tokens
  static constexpr int kTiles = (1 + kAtOnce) * kTileBytes, kSums = kRows * kPitch * 4;
  static constexpr int kBytes = kTiles > kSums ? kTiles : kSums;
};

// The first product, transposed: ranks are the matrix instruction's rows, tokens its columns, so that a lane holds four
// neighbouring ranks of one token.  RT tiles of 16 ranks, kept[j]: ranks 16 j + 4 (lane / 16) of token lane mod 16, whose
// adapter is `mine` and whose row of x begins at x + at.  The values from begin on, of which the wavefront takes
// every waves-th run of 64, the operands of kAhead of them in flight.
template <int RT, int kAhead>
__device__ __forceinline__ void low_sums(const AdapterArgs& g, const uint16_t* x, uint32_t at, int mine, int begin, int end,
                                         int wave, int waves, char* lds, f32x4 (&kept)[RT]) {
  constexpr int kAtOnce = LowLds<RT>::kAtOnce;
  const int lane = threadIdx.x & 63, quad = lane >> 4;
  // whole steps of the wavefront, and where a last one may end early
  const int stride = kStep * waves, first = begin + kStep * wave;
  const int n = first + kStep <= end ? (end - kStep - first) / stride + 1 : 0;
  const int tail = first + n * stride;
  const uint32_t chunk = 8 * (lane & 7);
  uint32_t x_row[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) x_row[h] = (uint32_t)__shfl((int)at, 8 * h + (lane >> 3), 64) + chunk;
#pragma unroll
  for (int j = 0; j < RT; ++j) kept[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for_adapters(mine, [&](int e) {
    const int rank = rank_of(g, e);
    if (rank == 0) return;
    const uint16_t* a = g.a + (int64_t)e * g.r * g.in;
    uint32_t a_row[RT][2];   // rows past the rank repeat the last one, their sums are dropped
#pragma unroll
    for (int j = 0; j < RT; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h) a_row[j][h] = (uint32_t)min(16 * j + 8 * h + (lane >> 3), rank - 1) * (uint32_t)g.in + chunk;
    f32x4 acc[RT];
#pragma unroll
    for (int j = 0; j < RT; ++j) acc[j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    struct Step {
      StepTile x, a[RT];
    };
    Step step[kAhead];
    auto load = [&](Step& s, int i) {
      const uint32_t k = first + i * stride;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        s.x.q[h] = *reinterpret_cast<const u32x4*>(x + (x_row[h] + k));
#pragma unroll
        for (int j = 0; j < RT; ++j) s.a[j].q[h] = *reinterpret_cast<const u32x4*>(a + (a_row[j][h] + k));
      }
    };
    auto multiply = [&](const Step& s) {
      // (the LDS operations of one wavefront take effect in program order)
      bf16x8 xv[2];
#pragma unroll
      for (int j0 = 0; j0 < RT; j0 += kAtOnce) {
        __builtin_amdgcn_wave_barrier();
        if (j0 == 0) tile_to_lds(lds, s.x, lane);
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) tile_to_lds(lds + (1 + j) * kTileBytes, s.a[j0 + j], lane);
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (j0 == 0) xv[h] = tile_operand(lds, h, lane);
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j)
            acc[j0 + j] = mfma(tile_operand(lds + (1 + j) * kTileBytes, h, lane), xv[h], acc[j0 + j]);
        }
      }
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
      Step s;
      const bool in = tail + (int)chunk < end;
      const u32x4 zero = {0u, 0u, 0u, 0u};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        s.x.q[h] = in ? *reinterpret_cast<const u32x4*>(x + (x_row[h] + (uint32_t)tail)) : zero;
#pragma unroll
        for (int j = 0; j < RT; ++j)
          s.a[j].q[h] = in ? *reinterpret_cast<const u32x4*>(a + (a_row[j][h] + (uint32_t)tail)) : zero;
      }
      multiply(s);
    }
    if (mine == e) {
#pragma unroll
      for (int j = 0; j < RT; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) kept[j][i] = 16 * j + 4 * quad + i < rank ? acc[j][i] : 0.0f;
    }
  });
}

// leaves the wavefront's sums in its LDS, a token's side by side
template <int RT>
__device__ __forceinline__ void leave_sums(const f32x4 (&kept)[RT], char* lds) {
  const int lane = threadIdx.x & 63;
  __builtin_amdgcn_wave_barrier();
#pragma unroll
  for (int j = 0; j < RT; ++j)
    *reinterpret_cast<f32x4*>(lds + ((lane & 15) * LowLds<RT>::kPitch + 16 * j + 4 * (lane >> 4)) * 4) = kept[j];
}
// the sum over the wavefronts' sums, four ranks from c on of the tile's row
template <int RT, int WAVES, int BYTES>
__device__ __forceinline__ f32x4 sum_of_waves(const char (&lds)[WAVES][BYTES], int row, int c) {
  f32x4 s = *reinterpret_cast<const f32x4*>(lds[0] + (row * LowLds<RT>::kPitch + c) * 4);
#pragma unroll
  for (int w = 1; w < WAVES; ++w) s += *reinterpret_cast<const f32x4*>(lds[w] + (row * LowLds<RT>::kPitch + c) * 4);
  return s;
}

// A slice of the first product for a tile of rows, or for a group of an adapter's rows, which the second product finds
// in `found`.
template <int RT, bool UNITS>
__global__ void __launch_bounds__(kThreads) adapters_low_kernel(AdapterArgs g) {
  union Lds {
    char of[kWaves][LowLds<RT>::kBytes];
    GroupLds group;
  };
  __shared__ __align__(16) Lds lds;
  const int lane = threadIdx.x & 63, col = lane & 15, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int tile = blockIdx.x / g.splits;
  const int slice = blockIdx.x - (unsigned)tile * g.splits, begin = slice * g.per_split, end = min(g.in, begin + g.per_split);
  UnitRows rows{kRows, 0, -1};
  if constexpr (UNITS) {
    const int firsts = scanned(g) ? first_units(g.rows, g.n) : 0;
    rows = tile < firsts ? first_rows(g, tile) : group_rows(g, tile - firsts, firsts > 0, lds.group);
    if (slice == 0 && wave == 0 && lane < kRows)
      g.found[tile * kRows + lane] = lane < rows.count ? make_int2(rows.row, rows.adapter) : make_int2(-1, -1);
    if (rows.count == 0) return;
    __syncthreads();   // (the products' LDS is the groups')
  }
  int64_t t;
  int mine;
  if constexpr (UNITS) {
    const int e = __shfl(rows.adapter, col, 64);
    t = __shfl(rows.row, min(col, rows.count - 1), 64);
    mine = col < rows.count ? e : -1;
  } else {
    t = (int64_t)tile * kRows + col;
    mine = adapter_of(g, t);
  }
  // (32-bit offsets from the first row of the tile, or of all)
  const uint32_t at = mine < 0 ? 0u : (UNITS ? (uint32_t)t : (uint32_t)col) * (uint32_t)g.x_ld;
  f32x4 kept[RT];
  low_sums<RT, RT == 1 ? 3 : RT == 2 ? 2 : 1>(g, g.x + (UNITS ? 0 : (int64_t)tile * kRows * g.x_ld), at, mine, begin, end, wave,
                                              kWaves, lds.of[wave], kept);
  leave_sums<RT>(kept, lds.of[wave]);
  __syncthreads();
  for (int i = threadIdx.x; i < kRows * RT * 4; i += kThreads) {
    const int row = i / (RT * 4), c = i % (RT * 4) * 4;
    int64_t to;
    bool in;
    if constexpr (UNITS) {
      in = row < rows.count;
      to = __shfl(rows.row, min(row, rows.count - 1), 64);
    } else {
      to = (int64_t)tile * kRows + row;
      in = to < g.rows;
    }
    const f32x4 s = sum_of_waves<RT>(lds.of, row, c);
    if (in) *reinterpret_cast<f32x4*>(g.low + ((int64_t)slice * g.rows + to) * (RT * 16) + c) = s;
  }
}

// the next bf16 part of v (and what it leaves).  A finite value's parts are finite, also above 3.396e38, which rounds to
// infinity: its first part is bf16's largest.  Nothing is left of what is not finite.
__device__ __forceinline__ bf16x8 part_of(float (&v)[8]) {
  constexpr float kMost = 0x1.fep127f;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool some[2] = {fabsf(v[2 * i]) < __builtin_inff(), fabsf(v[2 * i + 1]) < __builtin_inff()};
    float c[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) c[h] = some[h] ? __builtin_amdgcn_fmed3f(v[2 * i + h], -kMost, kMost) : v[2 * i + h];
    w[i] = bf16_pair(c[0], c[1]);
    v[2 * i] = some[0] ? v[2 * i] - __uint_as_float(w[i] << 16) : 0.0f;
    v[2 * i + 1] = some[1] ? v[2 * i + 1] - __uint_as_float(w[i] & 0xFFFF0000u) : 0.0f;
  }
  return __builtin_bit_cast(bf16x8, make_uint4(w[0], w[1], w[2], w[3]));
}

// the finite ones of eight bf16 values, zeros for the others (a magnitude from 0x7F80 on carries into the sign's place)
__device__ __forceinline__ bf16x8 finite_of(bf16x8 v) {
  u32x4 w = __builtin_bit_cast(u32x4, v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const s16x2 past = __builtin_bit_cast(s16x2, (w[i] & 0x7FFF7FFFu) + 0x00800080u) >> 15;
    w[i] &= ~__builtin_bit_cast(uint32_t, past);
  }
  return __builtin_bit_cast(bf16x8, w);
}

// four neighbouring values of base or out, as they lie in memory
template <typename T>
struct RawFour;
template <>
struct RawFour<uint16_t> {
  u32x2 w;
  __device__ __forceinline__ float at(int k) const {
    return __uint_as_float(k & 1 ? w[k / 2] & 0xFFFF0000u : w[k / 2] << 16);
  }
  __device__ __forceinline__ void set(const float (&v)[4]) { w = u32x2{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])}; }
};
template <>
struct RawFour<float> {
  u32x4 w;
  __device__ __forceinline__ float at(int k) const { return __uint_as_float(w[k]); }
  __device__ __forceinline__ void set(const float (&v)[4]) {
    w = u32x4{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
  }
};

// The second product: tokens are the matrix instruction's rows, output columns its columns, in an order that leaves a lane
// four neighbouring columns of four tokens (lane n of tile j: column 4 n + j of the wavefront's 64), so that base and out
// go in whole lines.  B, whose rows for neighbouring columns lie side by side, is loaded as it lies and read from LDS, its
// 16-byte chunks turned so that the lanes of a read meet on no bank.  PARTS bf16 parts of the low-rank values (RT == 1: one run
// of 32 holds two).
// FORM: tiles of neighbouring rows, the rows of an adapter, or those with the first product in the same kernel (each
// workgroup computes it whole, for its columns: for few rows and little of A that is less than a launch more).
enum AdapterForm { kTileForm, kUnitForm, kFewForm };
constexpr int kFewWaves = 8;
// wavefronts a SIMD that the registers have to leave room for: three where the kernel would take a little more than that
// allows
constexpr int out_waves(int rt, int form) {
  return form != kFewForm && (rt == 1 || (rt == 2 && form == kTileForm)) ? 3 : 1;
}
template <int RT, int PARTS, typename T, int FORM>
__global__ void __launch_bounds__(FORM == kFewForm ? 64 * kFewWaves : kThreads, out_waves(RT, FORM))
    adapters_out_kernel(AdapterArgs g) {
  constexpr bool UNITS = FORM != kTileForm, FEW = FORM == kFewForm;
  constexpr int kWaves = FEW ? kFewWaves : kWavesOfTile, kThreads = 64 * kWaves;
  constexpr int kRuns = RT == 1 ? 1 : RT / 2;                       // runs of 32 ranks (RT == 1: 16 ranks twice)
  constexpr int kSteps = RT == 1 ? (PARTS + 1) / 2 : kRuns * PARTS;
  // slices loaded at once (in a graph, us, 4 against 8: 1 row, 16 x 7168 -> 4096: 7.1, 7.3; 64 rows, 128 x 4096 -> 4096, side by
  // side: 16.5, 15.1); threads at most that share one value's slices
  constexpr int kBatch = RT <= 2 ? 4 : 8, kShares = 8;
  constexpr int kStride = kCols * kWaves;
  constexpr int kChunks = kCols * RT * 2;                           // 16-byte chunks of B in LDS, RT * 2 a column
  constexpr int kTurn = RT * 8 > 16 ? RT * 8 : 16;                  // chunks after which the next turn begins
  constexpr int kLoads = kChunks / 64;
  struct Operands {
    RawFour<T> base[4];
    u32x4 b[kLoads];
  };
  constexpr int kSums = kRows * RT * 4 > kThreads ? kRows * RT * 4 : kThreads;
  constexpr bool kShared = RT == 8;        // the sums lie where B will (64 KB in all)
  constexpr int kBytes = FEW && LowLds<RT>::kBytes > kChunks * 16 ? LowLds<RT>::kBytes : kChunks * 16;
  __shared__ __align__(16) char lds[kWaves][kBytes];
  __shared__ f32x4 own_sums[kShared ? 1 : kSums];
  f32x4* sums = kShared ? reinterpret_cast<f32x4*>(lds[0]) : own_sums;
  const int lane = threadIdx.x & 63, col = lane & 15, quad = lane >> 4, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  char* mine_lds = lds[wave];
  auto chunk_at = [&](int i) { return mine_lds + ((i & ~15) | ((i + i / kTurn) & 15)) * 16; };
  const int tile = blockIdx.x / g.blocks;
  const bool copy = UNITS && tile >= g.units;   // the rows without an adapter of tile `copied`
  const int copied = tile - g.units;
  const int block = blockIdx.x - (unsigned)tile * g.blocks;
  const int first = block * g.per_block + kCols * wave, end = min(g.outs, (block + 1) * g.per_block);
  UnitRows rows{kRows, 0, -1};
  if constexpr (UNITS) {
    if (copy) {
      const int r = copied * kRows + lane;
      const bool without = lane < kRows && r < g.rows && adapter_of(g, r) < 0;
      const uint64_t m = __ballot(without);
      rows = {(int)__popcll(m), __builtin_amdgcn_ds_permute(4 * (without ? bits_below(m) : kRows), r), -1};
    } else if constexpr (FEW) {
      rows = first_rows(g, tile);
    } else {
      const int2 f = g.found[tile * kRows + col];
      rows = {(int)__popcll(__ballot(lane < kRows && f.x >= 0)), f.x, f.y};
    }
    if (rows.count == 0) return;
  }
  // rows of the tile
  const int here = UNITS ? rows.count : (int)min((int64_t)kRows, g.rows - (int64_t)tile * kRows);
  auto row_of = [&](int i) -> int64_t {   // (rows the tile does not have: its last one)
    if constexpr (UNITS) return __shfl(rows.row, min(i, here - 1), 64);
    else return (int64_t)tile * kRows + min(i, here - 1);
  };
  const int64_t t = row_of(col);
  const int e = UNITS ? __shfl(rows.adapter, col, 64) : adapter_of(g, t), mine = col < here ? e : -1;
  const uint64_t with = __ballot(mine >= 0);
  const int e0 = with ? __builtin_amdgcn_readlane(mine, __builtin_ctzll(with)) : -1;
  const bool alone = RT <= 4 && with != 0 && __ballot(mine >= 0 && mine != e0) == 0;   // one adapter in the tile
  // the lane's four tokens of the result, and their adapters
  int64_t out_row[4];
  int theirs[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    out_row[i] = row_of(4 * quad + i);
    theirs[i] = __shfl(mine, 4 * quad + i, 64);
  }
  auto load_base = [&](Operands& o, int c0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o.base[i] = *reinterpret_cast<const RawFour<T>*>(static_cast<const T*>(g.base) + out_row[i] * g.base_ld +
                                                       min(c0 + 4 * col, g.outs - 4));
  };
  auto load_b = [&](u32x4 (&to)[kLoads], int e, int c0) {
    const uint16_t* b = g.b + (int64_t)e * g.outs * g.r;
#pragma unroll
    for (int l = 0; l < kLoads; ++l) {
      const int i = 64 * l + lane;
      to[l] = *reinterpret_cast<const u32x4*>(b + ((uint32_t)min(c0 + i / (RT * 2), g.outs - 1) * (uint32_t)g.r +
                                                    (uint32_t)min(i % (RT * 2) * 8, g.r - 8)));
    }
  };
  Operands now{};
  if (alone && first < end) load_b(now.b, e0, first);
  if (g.base && first < end) load_base(now, first);
  bf16x8 low[kSteps];
  if (with) {   // (the wavefronts of a workgroup have the same rows)
    const int items = here * RT * 4, shares = FEW ? 1 : max(1, min(kShares, kThreads / items));
    if constexpr (FEW) {
      f32x4 part[RT];
      low_sums<RT, RT == 1 ? 3 : 2>(g, g.x, mine < 0 ? 0u : (uint32_t)t * (uint32_t)g.x_ld, mine, 0, g.in, wave,
                                           kWaves, mine_lds, part);
      leave_sums<RT>(part, mine_lds);
      __syncthreads();
      for (int i = threadIdx.x; i < items; i += kThreads) sums[i] = sum_of_waves<RT>(lds, i / (RT * 4), i % (RT * 4) * 4);
    }
    // the slices' sums, slices shared out among threads and loaded in batches
    for (int i0 = FEW ? items : 0; i0 < items * shares; i0 += kThreads) {   // (all lanes: row_of reads other lanes' values)
      const int i = min(i0 + (int)threadIdx.x, items * shares - 1), share = i / items, item = i - share * items;
      f32x4 sum = {0.0f, 0.0f, 0.0f, 0.0f};
      const float* p = g.low + row_of(item / (RT * 4)) * (RT * 16) + item % (RT * 4) * 4;
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
    if (kShared) __syncthreads();
  }
  // kept = the products with adapter e's rows of B, for the tokens that have e
  auto multiply = [&](const u32x4 (&from)[kLoads], int e, int rank, f32x4 (&kept)[4]) {
    __builtin_amdgcn_wave_barrier();   // (the LDS operations of one wavefront take effect in program order)
#pragma unroll
    for (int l = 0; l < kLoads; ++l) {
      const int i = 64 * l + lane;
      u32x4 q = from[l];
      if (rank < RT * 16) {   // what is behind the rank does not count, whatever it holds
        const int left = rank - i % (RT * 2) * 8;
        q[0] &= left > 1 ? ~0u : left > 0 ? 0xFFFFu : 0u;
        q[1] &= left > 3 ? ~0u : left > 2 ? 0xFFFFu : 0u;
        q[2] &= left > 5 ? ~0u : left > 4 ? 0xFFFFu : 0u;
        q[3] &= left > 7 ? ~0u : left > 6 ? 0xFFFFu : 0u;
      }
      *reinterpret_cast<u32x4*>(chunk_at(i)) = q;
    }
    __builtin_amdgcn_wave_barrier();
    float none_past = 0.0f;            // NaN where a product is not finite
    auto operands = [&](int j, bf16x8 (&bv)[kRuns]) {
      const int c = 4 * col + j;   // the lane's column of this tile
#pragma unroll
      for (int run = 0; run < kRuns; ++run)
        bv[run] = *reinterpret_cast<const bf16x8*>(chunk_at(c * RT * 2 + (RT == 1 ? quad & 1 : 4 * run + quad)));
    };
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      bf16x8 bv[kRuns];
      operands(j, bv);
      f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int s = 0; s < kSteps; ++s) acc = mfma(low[s], bv[RT == 1 ? 0 : s % kRuns], acc);
      none_past = fmaf(acc[0], 0.0f, none_past);
#pragma unroll
      for (int i = 0; i < 4; ++i) kept[j][i] = theirs[i] == e ? acc[i] : kept[j][i];
    }
    // Where B is not finite, the first part of a low-rank value makes the infinity or NaN of it; the others, which may be
    // zero or of another sign, leave it out.  (Such a value leaves no token's product in its column finite, zeros' neither: one
    // of the lane's four is looked at.  In B as it is loaded, with the operands chosen on the way, that cost 2 to 7% of a call.)
    if (__builtin_expect(__ballot(none_past != none_past) != 0, 0)) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        bf16x8 bv[kRuns];
        operands(j, bv);
        f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          const bf16x8 b = bv[RT == 1 ? 0 : s % kRuns], rest = finite_of(b);
          acc = mfma(low[s], RT == 1 ? (s == 0 && quad < 2 ? b : rest) : s < kRuns ? b : rest, acc);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) kept[j][i] = theirs[i] == e ? acc[i] : kept[j][i];
      }
    }
  };
  auto store = [&](const Operands& o, const f32x4 (&kept)[4], int c0) {
    const int c = c0 + 4 * col;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (4 * quad + i >= here || c >= g.outs) continue;
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = o.base[i].at(k) + kept[k][i];
      RawFour<T> p;
      p.set(v);
      if (theirs[i] < 0) p = o.base[i];   // (a row without an adapter keeps its base's bits)
      *reinterpret_cast<RawFour<T>*>(static_cast<T*>(g.out) + out_row[i] * g.out_ld + c) = p;
    }
  };
  const f32x4 none = {0.0f, 0.0f, 0.0f, 0.0f};
  auto clear = [&](f32x4 (&kept)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) kept[j] = none;
  };
  f32x4 kept[4];
  if (alone) {
    const int rank = rank_of(g, e0);
    int c0 = first;
    for (; c0 + kStride < end; c0 += kStride) {
      if constexpr (RT <= 2) {   // the next columns' operands on their way while these are worked on
        Operands next{};
        load_b(next.b, e0, c0 + kStride);
        if (g.base) load_base(next, c0 + kStride);
        clear(kept);
        multiply(now.b, e0, rank, kept);
        store(now, kept, c0);
        now = next;
      } else {   // (no registers for a second set)
        clear(kept);
        multiply(now.b, e0, rank, kept);
        store(now, kept, c0);
        load_b(now.b, e0, c0 + kStride);
        if (g.base) load_base(now, c0 + kStride);
      }
    }
    if (c0 < end) {
      clear(kept);
      multiply(now.b, e0, rank, kept);
      store(now, kept, c0);
    }
  } else {
    for (int c0 = first; c0 < end; c0 += kStride) {
      clear(kept);
      if (g.base && c0 > first) load_base(now, c0);
      for_adapters(mine, [&](int e) {
        load_b(now.b, e, c0);
        multiply(now.b, e, rank_of(g, e), kept);
      });
      store(now, kept, c0);
    }
  }
}

struct AdapterPlan {
  int tiles16;                   // RT
  AdapterForm form;
  int splits, per_split, blocks, per_block;
  int units;
};

AdapterPlan plan_of(const moe_adapter_shape& s) {
  AdapterPlan p;
  p.tiles16 = s.rank <= 16 ? 1 : s.rank <= 32 ? 2 : s.rank <= 64 ? 4 : 8;
  const int64_t n = s.n_adapters, x_ld = s.x_ld ? s.x_ld : s.in_cols;
  p.form = s.rows <= kFewRows && p.tiles16 <= 2 && (int64_t)s.rank * s.in_cols <= kFewValues ? kFewForm
           : s.rows <= kUnitRows && s.rows <= (p.tiles16 <= 2 ? 1 : 2) * kUnitShare * n &&
                     s.rows * x_ld < (int64_t(1) << 32)   // (32-bit offsets)
               ? kUnitForm
               : kTileForm;
  // an adapter's last group may be a part of one: n groups (or as many as there are rows) and one for every whole 16 rows
  p.units = (int)(first_units(s.rows, s.n_adapters) + (p.form == kUnitForm ? s.rows / kRows : 0));
  // (at least one: the size query may be asked for no rows; up to 64 rows hardly any adapter has further groups)
  const int64_t tiles = std::max<int64_t>(
      1, p.form != kUnitForm ? ceil_div(s.rows, kRows) : s.rows <= 64 ? first_units(s.rows, s.n_adapters) : p.units);
  const int64_t some = p.form == kUnitForm ? kUnitBlocks : p.tiles16 <= 2 ? kTileBlocks : kTileBlocks / 2;
  const int64_t run = kStep * kWaves;
  const int64_t want = std::max<int64_t>(1, std::min<int64_t>(ceil_div(some, tiles), ceil_div(s.in_cols, run)));
  p.per_split = (int)(ceil_div(ceil_div(s.in_cols, want), run) * run);
  p.splits = (int)ceil_div(s.in_cols, p.per_split);
  const int64_t stride = kCols * (p.form == kFewForm ? kFewWaves : kWaves);
  p.per_block = (int)(ceil_div(ceil_div(s.out_cols, ceil_div(some, tiles)), stride) * stride);
  p.blocks = (int)ceil_div(s.out_cols, p.per_block);
  return p;
}

template <int RT, int FORM>
hipError_t out_t(const AdapterArgs& g, int out_dtype, dim3 grid, hipStream_t st) {
  const dim3 threads(FORM == kFewForm ? 64 * kFewWaves : kThreads);
  return out_dtype == MOE_DTYPE_F32 ? launch_kernel(adapters_out_kernel<RT, 3, float, FORM>, grid, threads, 0, st, g)
                                    : launch_kernel(adapters_out_kernel<RT, 2, uint16_t, FORM>, grid, threads, 0, st, g);
}

template <int RT>
hipError_t run_t(const AdapterArgs& g, AdapterForm form, int out_dtype, hipStream_t st) {
  // (the slices or columns of a tile are neighbours in the grid: workgroups at work together cover whole rows)
  const int64_t row_tiles = ceil_div(g.rows, kRows);
  const unsigned tiles = (unsigned)(form == kTileForm ? row_tiles : (int64_t)g.units);
  // by adapters, the rows without one are copied by further workgroups, unless they are where they belong
  const dim3 grid((tiles + (unsigned)(form == kTileForm || g.base == g.out ? 0 : row_tiles)) * g.blocks);
  if constexpr (RT <= 2)
    if (form == kFewForm) return out_t<RT, kFewForm>(g, out_dtype, grid, st);
  const hipError_t err =
      form == kTileForm ? launch_kernel(adapters_low_kernel<RT, false>, dim3(tiles * g.splits), dim3(kThreads), 0, st, g)
                        : launch_kernel(adapters_low_kernel<RT, true>, dim3(tiles * g.splits), dim3(kThreads), 0, st, g);
  if (err != hipSuccess) return err;
  return form == kTileForm ? out_t<RT, kTileForm>(g, out_dtype, grid, st) : out_t<RT, kUnitForm>(g, out_dtype, grid, st);
}

}  // namespace

// What any batch of up to so many rows needs (the slices are fewer the more rows there are, and end unevenly): the groups that
// the first product finds, and its slices, which are fewer than some / tiles + 1 and no more than the runs of 256 values: with
// kRows rows a tile or group at most, slices * rows <= kRows * some + rows.
static int64_t found_bytes(const moe_adapter_shape& s) {
  const int64_t rows = std::min<int64_t>(s.rows, kUnitRows);
  return (first_units(rows, s.n_adapters) + rows / kRows) * kRows * sizeof(int2);
}
size_t adapters_workspace(const moe_adapter_shape& s) {
  const AdapterPlan p = plan_of(s);
  if (p.form == kFewForm) return 0;
  const int64_t most = kRows * (p.tiles16 <= 2 ? kTileBlocks : kTileBlocks / 2) + s.rows;
  return (size_t)(found_bytes(s) + std::min(s.rows * ceil_div(s.in_cols, kStep * kWaves), most) * p.tiles16 * 16 * 4);
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
                      low + (found_bytes(s) / 4),
                      reinterpret_cast<int2*>(low),
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
                      p.per_block,
                      p.units};
  switch (p.tiles16) {
    case 1: return run_t<1>(g, p.form, s.out_dtype, st);
    case 2: return run_t<2>(g, p.form, s.out_dtype, st);
    case 4: return run_t<4>(g, p.form, s.out_dtype, st);
    default: return run_t<8>(g, p.form, s.out_dtype, st);
  }
}

}  // namespace moe
