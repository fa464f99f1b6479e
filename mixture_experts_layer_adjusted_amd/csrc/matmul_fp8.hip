// Products of two E4M3 matrices with one fp32 scale per block of 128 (and the transposing quantiser that makes
// the operands of a weight gradient).
//
//   forward       out[m, n] = sum_kb sa[m, kb] sb[n / 128, kb] sum_{k in kb} a[m, k] b[n, k]
//   input grad    out[m, n] = sum_kb sa[m, kb] sb[kb, n / 128] sum_{k in kb} a[m, k] b[k, n]
//   weight grad   out[m, n] = sum_kb sa[m, kb] sb[n, kb]       sum_{k in kb} a[m, k] b[n, k]
//
// with kb the blocks of 128 of the contraction.  A v_mfma_scale_f32_16x16x128_f8f6f4 with unit scales contracts
// one block of a 16 x 16 piece in fp32; its result is folded into the fp32 sum with the factor sa sb, so that the
// scales never touch the codes.  In that instruction b's rows are the first operand: a lane holds four
// neighbouring columns n of one row m of the output.
//
// That instruction adds products in groups of eight neighbouring elements, and a product keeps no bits more than
// 13 below its group's largest: measured against 64 bits, the sum over a block of normal values is 1.3e-5 off
// (1.8e-5 with columns 8 times larger), far less than a bf16 output's own rounding but 100 times fp32's.  So an
// fp32 output takes the v_mfma_f32_16x16x32_f16 instead, on the codes widened to f16 (every E4M3 value is one):
// 1e-8 off, at half the rate.
#include "fp8_codec.h"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kBK = 128;            // elements (bytes) of one scale block
constexpr int kXcds = 8;
constexpr int kE8M0One = 127;       // E8M0 encoding of 2^0
constexpr int kGroupM = 4;          // M-tiles per block of the tile order

typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) i32x2 lds_i32x2;
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void lds_void_t;

struct MatmulArgs {
  const uint8_t* a;
  const float* a_scale;
  const uint8_t* b;
  const float* b_scale;
  void* out;
  float* part;          // [splits, m, n] fp32 sums of a split contraction; null: out is written
  int64_t lda, ldb, ldo;
  int m, n, k;
  int nblk;             // column blocks of b's scales: ceil(n / 128)
  int kb_per_split;     // K blocks of one slice of the contraction
  bool out_f32, accumulate;
};

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const uint32_t a = __float_as_uint(lo), b = __float_as_uint(hi);
  const uint32_t x = lo != lo ? 0x7FC0u : (a + 0x7FFFu + ((a >> 16) & 1u)) >> 16;
  const uint32_t y = hi != hi ? 0x7FC00000u : (b + 0x7FFFu + ((b >> 16) & 1u)) & 0xFFFF0000u;
  return x | y;
}

// four neighbouring outputs of one row, added to what is there if the caller accumulates
__device__ __forceinline__ void store4(const MatmulArgs& g, int64_t row, int col, f32x4 v) {
  if (g.out_f32) {
    f32x4* p = reinterpret_cast<f32x4*>(static_cast<float*>(g.out) + row * g.ldo + col);
    if (g.accumulate) v += *p;
    *p = v;
  } else {
    uint2* p = reinterpret_cast<uint2*>(static_cast<uint16_t*>(g.out) + row * g.ldo + col);
    if (g.accumulate) {
      const uint2 q = *p;
      v += f32x4{__uint_as_float(q.x << 16), __uint_as_float(q.x & 0xFFFF0000u), __uint_as_float(q.y << 16),
                 __uint_as_float(q.y & 0xFFFF0000u)};
    }
    *p = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  }
}

template <int N>
__device__ __forceinline__ void wait_vmcnt() {
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}

// ---- tiles staged in LDS -------------------------------------------------------------------------------------
//
// A staged row is one 128-byte K block as eight 16-byte chunks, chunk q at slot kslot(q) ^ swz(row): a fragment
// read (16 rows x 64 contiguous bytes) then spreads over all banks.
__device__ __forceinline__ int swz(int r) { return (r >> 1) & 7; }
__device__ __forceinline__ int kslot(int q) { return ((q & 1) << 2) | (q >> 1); }
__device__ __forceinline__ int kchunk(int s) { return ((s & 3) << 1) | (s >> 2); }
__device__ __forceinline__ int src_chunk(int r, int s) { return kchunk(s ^ swz(r)) << 4; }

// b as stored [k][n]: 128 K rows of BN bytes.  One transposing read takes 8 bytes from each of 32 rows
// (32 kq + 8 j + 0..7); the 16-byte chunk c of row r sits at slot c ^ kn_swz(r), so that these rows fall on every
// 16-byte unit of the banks twice.
template <int BN>
__device__ __forceinline__ int kn_swz(int r) {
  return BN == 256 ? (r & 7) | (((r >> 5) & 1) << 3) : ((r >> 1) & 3) | (((r >> 5) & 1) << 2);
}

__device__ __forceinline__ i32x8 frag_at(const uint8_t* p0, const uint8_t* p1) {
  const u32x4 a = *reinterpret_cast<const u32x4*>(p0), b = *reinterpret_cast<const u32x4*>(p1);
  return i32x8{(int)a[0], (int)a[1], (int)a[2], (int)a[3], (int)b[0], (int)b[1], (int)b[2], (int)b[3]};
}

// A 16 x 16 block over one K block.  EXACT: in f16, four instructions of eight elements a lane (any order of the
// elements serves, both operands having the same).
template <bool EXACT>
struct Frag;
template <>
struct Frag<false> {
  i32x8 v;
  __device__ __forceinline__ void set(const i32x8& codes) { v = codes; }
};
template <>
struct Frag<true> {
  f16x8 v[4];
  __device__ __forceinline__ void set(const i32x8& codes) {
#pragma unroll
    for (int s = 0; s < 4; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const f16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes[2 * s + h], 1.0f, false);
        const f16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(codes[2 * s + h], 1.0f, true);
        v[s][4 * h] = lo[0], v[s][4 * h + 1] = lo[1], v[s][4 * h + 2] = hi[0], v[s][4 * h + 3] = hi[1];
      }
  }
};
__device__ __forceinline__ f32x4 contract(const Frag<false>& w, const Frag<false>& x) {
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w.v, x.v, zero, 0, 0, 0, kE8M0One, 0, kE8M0One);
}
__device__ __forceinline__ f32x4 contract(const Frag<true>& w, const Frag<true>& x) {
  f32x4 p = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int s = 0; s < 4; ++s) p = __builtin_amdgcn_mfma_f32_16x16x32_f16(w.v[s], x.v[s], p, 0, 0, 0);
  return p;
}

// 64 lanes x 16 (or 4) bytes at base + off + step into LDS at dst + 16 (or 4) lane
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t base, uint8_t* dst, uint32_t off, uint32_t step) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(base, (lds_void_t*)dst, 16, off, step, 0, 0);
}
__device__ __forceinline__ void load_lds4(__amdgpu_buffer_rsrc_t base, uint8_t* dst, uint32_t off, uint32_t step) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(base, (lds_void_t*)dst, 4, off, step, 0, 0);
}

template <int BM, int BN, int WM, int WN, int STAGES>
struct TileShape {
  static constexpr int kWaves = WM * WN, kThreads = kWaves * 64;
  static constexpr int kMB = BM / WM / 16, kNB = BN / WN / 16;
  static constexpr int kADma = BM / 8 / kWaves, kBDma = BN / 8 / kWaves;   // 1 KB loads of a wavefront per stage
  static constexpr int kDataBytes = (BM + BN) * kBK;
  static constexpr int kScaleBytes = kWaves * 256;                          // 64 scales per wavefront
  static constexpr int kLds = STAGES * (kDataBytes + kScaleBytes);
  static_assert(BM % 64 == 0 && (BM + BN) / 64 <= kWaves, "a wavefront loads 64 scales at most");
  static_assert(kADma * 8 * kWaves == BM && kBDma * 8 * kWaves == BN, "whole loads");
};

// One BM x BN tile of the output over the K blocks of slice blockIdx.y.  STAGES stages of one K block each, filled
// by direct loads STAGES - 1 blocks ahead.  Rows and columns past the matrix read a valid row or column and are
// not stored.
template <int FORM, bool EXACT, int BM, int BN, int WM, int WN, int STAGES>
__global__ void __launch_bounds__(WM * WN * 64) matmul_tile_kernel(MatmulArgs g, int MT, int NT) {
  using S = TileShape<BM, BN, WM, WN, STAGES>;
  constexpr bool KN = FORM == MOE_FP8_INPUT_GRAD, ROWS = FORM == MOE_FP8_WEIGHT_GRAD;
  constexpr int kMB = S::kMB, kNB = S::kNB;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  uint8_t* const scales = lds + STAGES * S::kDataBytes;
  const int L = (int)xcd_logical(blockIdx.x);
  if (L >= MT * NT) return;
  const int grp = L / (kGroupM * NT), gm = min(kGroupM, MT - grp * kGroupM), rem = L - grp * kGroupM * NT;
  const int m0 = (grp * kGroupM + rem % gm) * BM, n0 = rem / gm * BN;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int KB = g.k / kBK;
  const int kb0 = blockIdx.y * g.kb_per_split, nk = min(g.kb_per_split, KB - kb0);

  // ---- where this lane's loads come from: 32-bit byte offsets from the tile's first row
  uint32_t aoff[S::kADma], boff[S::kBDma];
#pragma unroll
  for (int i = 0; i < S::kADma; ++i) {
    const int r = (wave * S::kADma + i) * 8 + (lane >> 3);
    aoff[i] = (uint32_t)min(r, g.m - 1 - m0) * (uint32_t)g.lda + src_chunk(r, lane & 7);
  }
#pragma unroll
  for (int i = 0; i < S::kBDma; ++i) {
    if constexpr (KN) {
      constexpr int kLanes = BN / 16;   // lanes of one K row
      const int kr = (wave * S::kBDma + i) * (64 / kLanes) + lane / kLanes;
      const int c = 16 * ((lane % kLanes) ^ kn_swz<BN>(kr));
      boff[i] = (uint32_t)kr * (uint32_t)g.ldb + min(c, g.n - 16 - n0);
    } else {
      const int r = (wave * S::kBDma + i) * 8 + (lane >> 3);
      boff[i] = (uint32_t)min(r, g.n - 1 - n0) * (uint32_t)g.ldb + src_chunk(r, lane & 7);
    }
  }
  // scales: the first BM / 64 wavefronts a's rows, the next b's (its rows, or lane i its column block i);
  // the others repeat a's, so that every wavefront has the same loads in flight
  const float* sbase = g.a_scale + (int64_t)m0 * KB;
  uint32_t soff = 0, sstep = 4;
  if (wave < BM / 64 || wave >= (BM + BN) / 64 || (!ROWS && wave > BM / 64)) {
    soff = (uint32_t)min((wave % (BM / 64)) * 64 + lane, g.m - 1 - m0) * (uint32_t)KB * 4;
  } else if (ROWS) {
    sbase = g.b_scale + (int64_t)n0 * KB;
    soff = (uint32_t)min((wave - BM / 64) * 64 + lane, g.n - 1 - n0) * (uint32_t)KB * 4;
  } else {
    const int blk = min(n0 / kBK + lane, g.nblk - 1);
    sbase = g.b_scale;
    soff = (uint32_t)(KN ? blk : blk * KB) * 4;
    sstep = KN ? g.nblk * 4 : 4;
  }
  const uint8_t* abase = g.a + (int64_t)m0 * g.lda;
  const uint8_t* bbase = KN ? g.b + n0 : g.b + (int64_t)n0 * g.ldb;
  const __amdgpu_buffer_rsrc_t abuf =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(abase), (short)0, -1, 0x00020000);
  const __amdgpu_buffer_rsrc_t sbuf =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(sbase), (short)0, -1, 0x00020000);
  auto issue = [&](int kt) {
    const int slot = kt % STAGES;
    uint8_t* st = lds + slot * S::kDataBytes;
    const uint32_t k0 = (uint32_t)(kb0 + kt) * kBK;
#pragma unroll
    for (int i = 0; i < S::kADma; ++i) load_lds16(abuf, st + (wave * S::kADma + i) * 1024, aoff[i], k0);
    const __amdgpu_buffer_rsrc_t bbuf = __builtin_amdgcn_make_buffer_rsrc(
        const_cast<uint8_t*>(KN ? bbase + (int64_t)k0 * g.ldb : bbase), (short)0, -1, 0x00020000);
#pragma unroll
    for (int i = 0; i < S::kBDma; ++i)
      load_lds16(bbuf, st + BM * kBK + (wave * S::kBDma + i) * 1024, boff[i], KN ? 0u : k0);
    load_lds4(sbuf, scales + slot * S::kScaleBytes + wave * 256, soff, (uint32_t)(kb0 + kt) * sstep);
  };
  constexpr int kLoads = S::kADma + S::kBDma + 1;

  const int l16 = lane & 15, kq = lane >> 4;
  const int mrow = wm * (BM / WM), ncol = wn * (BN / WN);
  // the lane's fragment halves (K chunks 2 kq, 2 kq + 1); every 16th row on has the same swizzle
  const int c0 = (kslot(2 * kq) ^ swz(l16)) << 4, c1 = (kslot(2 * kq + 1) ^ swz(l16)) << 4;
  const int xr = (mrow + l16) * kBK, wr = (BM + ncol + l16) * kBK;
  // slot of the wavefront's column block among the loaded ones
  const int wblk = ROWS ? 0 : (n0 + ncol) / kBK - n0 / kBK;

  f32x4 acc[kMB][kNB];
#pragma unroll
  for (int i = 0; i < kMB; ++i)
#pragma unroll
    for (int j = 0; j < kNB; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s)
    if (s < nk) issue(s);
  for (int kt = 0; kt < nk; ++kt) {
    // stage kt has landed once at most the STAGES - 2 younger ones are in flight
    if (kt + STAGES - 1 <= nk)
      wait_vmcnt<(STAGES - 2) * kLoads>();
    else
      wait_vmcnt<0>();
    // every wavefront's part of stage kt is there, and stage kt - 1 is no longer read
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (kt + STAGES - 1 < nk) issue(kt + STAGES - 1);
    const uint8_t* st = lds + (kt % STAGES) * S::kDataBytes;
    const float* sc = reinterpret_cast<const float*>(scales + (kt % STAGES) * S::kScaleBytes);
    const float sw = ROWS ? 0.0f : sc[BM + wblk];
    // (widened fragments are twice as large: half the wavefront's columns at a time)
    constexpr int kCols = EXACT ? kNB / 2 : kNB;
#pragma unroll
    for (int j0 = 0; j0 < kNB; j0 += kCols) {
      if constexpr (EXACT) __builtin_amdgcn_sched_barrier(0);   // or the second half's reads move up, and spill
      Frag<EXACT> wf[kCols];
      f32x4 swr[kCols];
#pragma unroll
      for (int jj = 0; jj < kCols; ++jj) {
        const int j = j0 + jj;
        if constexpr (KN) {
          // ds_read_b64_tr_b8: within 16 lanes, lane s names row 8 j + s / 2 at columns 8 (s % 2)..+7 of the 16 and
          // receives its own column's eight rows
          const uint8_t* wt = st + BM * kBK;
          const int col = ncol + 16 * j + 8 * (lane & 1);
          i32x8 f;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int r = 32 * kq + 8 * q + (l16 >> 1);
            const i32x2 v = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
                (lds_i32x2*)(wt + r * BN + (((col >> 4) ^ kn_swz<BN>(r)) << 4) + (col & 15)));
            f[2 * q] = v[0];
            f[2 * q + 1] = v[1];
          }
          wf[jj].set(f);
        } else {
          wf[jj].set(frag_at(st + wr + j * 16 * kBK + c0, st + wr + j * 16 * kBK + c1));
        }
        if constexpr (ROWS) swr[jj] = *reinterpret_cast<const f32x4*>(sc + BM + ncol + 16 * j + 4 * kq);
      }
      i32x8 xf_next = frag_at(st + xr + c0, st + xr + c1);
      float sa_next = sc[mrow + l16];
#pragma unroll
      for (int i = 0; i < kMB; ++i) {
        Frag<EXACT> xf;
        xf.set(xf_next);
        const float sa = sa_next;
        if (i + 1 < kMB) {
          xf_next = frag_at(st + xr + (i + 1) * 16 * kBK + c0, st + xr + (i + 1) * 16 * kBK + c1);
          sa_next = sc[mrow + (i + 1) * 16 + l16];
        }
        const float f = sa * sw;
#pragma unroll
        for (int jj = 0; jj < kCols; ++jj) {
          const f32x4 p = contract(wf[jj], xf);
          f32x4& c = acc[i][j0 + jj];
#pragma unroll
          for (int v = 0; v < 4; ++v) c[v] = fmaf(p[v], ROWS ? sa * swr[jj][v] : f, c[v]);
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kMB; ++i) {
    const int row = m0 + mrow + 16 * i + l16;
    if (row >= g.m) continue;
#pragma unroll
    for (int j = 0; j < kNB; ++j) {
      const int col = n0 + ncol + 16 * j + 4 * kq;
      if (col >= g.n) continue;
      if (g.part)
        *reinterpret_cast<f32x4*>(g.part + ((int64_t)blockIdx.y * g.m + row) * g.n + col) = acc[i][j];
      else
        store4(g, row, col, acc[i][j]);
    }
  }
}

// out = the sum of the slices, in their order
__global__ void __launch_bounds__(256) matmul_join_kernel(MatmulArgs g, int splits) {
  const int64_t per = (int64_t)g.m * g.n, quads = per / 4;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < quads; i += (int64_t)gridDim.x * 256) {
    f32x4 v = *reinterpret_cast<const f32x4*>(g.part + 4 * i);
    for (int s = 1; s < splits; ++s) v += *reinterpret_cast<const f32x4*>(g.part + s * per + 4 * i);
    const int64_t row = 4 * i / g.n;
    store4(g, row, (int)(4 * i - row * g.n), v);
  }
}

// ---- few rows ------------------------------------------------------------------------------------------------
//
// Up to 16 MB rows of a: b is read once, straight into the fragments.  A workgroup has 16 columns; its eight
// wavefronts take the K blocks in turn (U of each in flight) and their sums meet in LDS.
constexpr int kRowWaves = 8;
template <int MB, bool EXACT>
__global__ void __launch_bounds__(kRowWaves * 64) matmul_rows_kernel(MatmulArgs g) {
  constexpr int U = MB == 1 ? 8 : 4;
  __shared__ f32x4 sums[kRowWaves][MB][64];
  const int tid = threadIdx.x, lane = tid & 63, l16 = lane & 15, kq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = blockIdx.x * 16, KB = g.k / kBK;
  // a lane has the 16-byte chunks kq and kq + 4 of its row of both operands: a read covers 64 bytes of each row,
  // and the products pair the same elements
  const uint8_t* bp = g.b + (int64_t)(n0 + l16) * g.ldb + kq * 16;
  const uint8_t* ap[MB];
  const float* sp[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i) {
    const int row = min(16 * i + l16, g.m - 1);
    ap[i] = g.a + (int64_t)row * g.lda + kq * 16;
    sp[i] = g.a_scale + (int64_t)row * KB;
  }
  const float* wp = g.b_scale + (int64_t)(n0 / kBK) * KB;
  f32x4 acc[MB];
#pragma unroll
  for (int i = 0; i < MB; ++i) acc[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (int k0 = wave; k0 < KB; k0 += kRowWaves * U) {
    i32x8 wf[U], xf[U][MB];
    float f[U][MB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int kb = min(k0 + u * kRowWaves, KB - 1);   // past the end: the last block again, with the factor 0
      const bool there = k0 + u * kRowWaves < KB;
      wf[u] = frag_at(bp + (int64_t)kb * kBK, bp + (int64_t)kb * kBK + 64);
      const float sw = wp[kb];
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        xf[u][i] = frag_at(ap[i] + (int64_t)kb * kBK, ap[i] + (int64_t)kb * kBK + 64);
        f[u][i] = there ? sp[i][kb] * sw : 0.0f;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      Frag<EXACT> w, x;
      w.set(wf[u]);
#pragma unroll
      for (int i = 0; i < MB; ++i) {
        x.set(xf[u][i]);
        const f32x4 p = contract(w, x);
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][v] = fmaf(p[v], f[u][i], acc[i][v]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < MB; ++i) sums[wave][i][lane] = acc[i];
  __syncthreads();
  for (int j = tid; j < MB * 64; j += kRowWaves * 64) {
    const int i = j >> 6, l = j & 63, row = 16 * i + (l & 15);
    if (row >= g.m) continue;
    f32x4 v = sums[0][i][l];
#pragma unroll
    for (int w = 1; w < kRowWaves; ++w) v += sums[w][i][l];
    store4(g, row, n0 + 4 * (l >> 4), v);
  }
}

// ---- the transposing quantiser -------------------------------------------------------------------------------
//
// codes[c, r] of x[r, c] (bf16), one scale per column and run of 128 rows: amax times fp32(1 / 448), 1 for a run of zeros; rows
// past the last are zeros.  A 128-row x 64-column block goes through LDS in fp32: a thread loads 32 columns of one
// row, then four neighbouring threads take one column's rows, 32 each.
__global__ void __launch_bounds__(256) quant_act_t_kernel(const uint16_t* __restrict__ x, int rows, int cols,
                                                          uint8_t* __restrict__ codes, float* __restrict__ scales) {
  __shared__ float tile[64][129];
  const int64_t r0 = (int64_t)blockIdx.x * 128;
  const int c0 = blockIdx.y * 64, tid = threadIdx.x;
  const int64_t runs = gridDim.x;
  {
    const int rl = tid >> 1, h = (tid & 1) * 32;
    const int64_t r = r0 + rl;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int c = c0 + h + 8 * q;
      uint4 w = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows && c < cols) w = *reinterpret_cast<const uint4*>(x + r * cols + c);   // (cols: a multiple of 8)
      const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        tile[h + 8 * q + 2 * i][rl] = __uint_as_float(v[i] << 16);
        tile[h + 8 * q + 2 * i + 1][rl] = __uint_as_float(v[i] & 0xFFFF0000u);
      }
    }
  }
  __syncthreads();
  const int c = tid >> 2, q = tid & 3;
  float v[32], amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    v[i] = tile[c][32 * q + i];
    amax = fmaxf(amax, fabsf(v[i]));
  }
  amax = fmaxf(amax, __shfl_xor(amax, 1, 64));
  amax = fmaxf(amax, __shfl_xor(amax, 2, 64));
  if (c0 + c >= cols) return;
  const float scale = amax > 0.0f ? amax * (1.0f / 448.0f) : 1.0f;
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    w[i] = e4m3x4_from_f32(__fdiv_rn(v[4 * i], scale), __fdiv_rn(v[4 * i + 1], scale), __fdiv_rn(v[4 * i + 2], scale),
                           __fdiv_rn(v[4 * i + 3], scale));
  uint8_t* p = codes + (int64_t)(c0 + c) * runs * 128 + r0 + 32 * q;
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  *reinterpret_cast<uint4*>(p + 16) = make_uint4(w[4], w[5], w[6], w[7]);
  if (q == 0) scales[(int64_t)(c0 + c) * runs + blockIdx.x] = scale;
}

// ---- which kernel ----------------------------------------------------------------------------------------------

struct Plan {
  int rows_mb;         // > 0: the few-rows kernel with so many blocks of 16 rows
  int bm, bn;          // else the tile
  int splits, kb_per_split;
};

Plan plan_of(const moe_matmul_shape& s) {
  Plan p{0, 0, 0, 1, s.k / kBK};
  if (s.form == MOE_FP8_FORWARD && s.m <= 32) {
    p.rows_mb = s.m <= 16 ? 1 : 2;
    return p;
  }
  const int64_t big = ceil_div(s.m, 256) * ceil_div(s.n, 256);
  p.bm = p.bn = 256;
  if (big < 200) p.bm = p.bn = 128;
  if (s.m <= 64) p.bm = 64, p.bn = 128;
  const int64_t tiles = ceil_div(s.m, p.bm) * ceil_div(s.n, p.bn);
  const int kb = s.k / kBK;
  if (p.bm < 256) {   // the chip has 256 CUs: slices of at least four K blocks
    const int want = (int)std::min<int64_t>(std::min<int64_t>(256 / std::max<int64_t>(tiles, 1), kb / 4), 16);
    if (want > 1) {
      p.kb_per_split = (int)ceil_div(kb, want);
      p.splits = (int)ceil_div(kb, p.kb_per_split);
    }
  }
  return p;
}

template <int FORM, bool EXACT, int BM, int BN, int WM, int WN, int STAGES>
hipError_t launch_tile(const MatmulArgs& g, int splits, hipStream_t st) {
  using S = TileShape<BM, BN, WM, WN, STAGES>;
  static_assert(S::kLds <= 163840, "LDS");
  auto kern = &matmul_tile_kernel<FORM, EXACT, BM, BN, WM, WN, STAGES>;
  const hipError_t err = ensure_dynamic_lds(reinterpret_cast<const void*>(kern), S::kLds);
  if (err != hipSuccess) return err;
  const int64_t MT = ceil_div(g.m, BM), NT = ceil_div(g.n, BN);
  const int64_t grid = ceil_div(MT * NT, kXcds * 32) * (kXcds * 32);
  if (MT * NT >= (int64_t(1) << 31) - 256) return hipErrorInvalidValue;
  hipLaunchKernelGGL(kern, dim3((unsigned)grid, (unsigned)splits), dim3(S::kThreads), S::kLds, st, g, (int)MT, (int)NT);
  return hipGetLastError();
}

template <int FORM, bool EXACT>
hipError_t launch_form(const MatmulArgs& g, const Plan& p, hipStream_t st) {
  if (p.rows_mb) {
    const dim3 grid((unsigned)(g.n / 16)), block(kRowWaves * 64);
    if (p.rows_mb == 1) hipLaunchKernelGGL((matmul_rows_kernel<1, EXACT>), grid, block, 0, st, g);
    else hipLaunchKernelGGL((matmul_rows_kernel<2, EXACT>), grid, block, 0, st, g);
    return hipGetLastError();
  }
  if (p.bm == 256) return launch_tile<FORM, EXACT, 256, 256, 2, 4, 2>(g, p.splits, st);
  if (p.bm == 128) return launch_tile<FORM, EXACT, 128, 128, 2, 2, 4>(g, p.splits, st);
  return launch_tile<FORM, EXACT, 64, 128, 2, 2, 4>(g, p.splits, st);
}

template <int FORM>
hipError_t launch_product(const MatmulArgs& g, const Plan& p, hipStream_t st) {
  return g.out_f32 ? launch_form<FORM, true>(g, p, st) : launch_form<FORM, false>(g, p, st);
}

}  // namespace

size_t matmul_fp8_workspace(const moe_matmul_shape& s) {
  if (s.m == 0 || s.n == 0 || s.k == 0) return 0;
  const Plan p = plan_of(s);
  return p.splits > 1 ? (size_t)p.splits * s.m * s.n * 4 : 0;
}

hipError_t launch_matmul_fp8(const moe_matmul_shape& s, const uint8_t* a, const float* a_scale, const uint8_t* b,
                             const float* b_scale, void* out, float* ws, hipStream_t st) {
  if (s.m == 0 || s.n == 0) return hipSuccess;
  const Plan p = plan_of(s);
  MatmulArgs g{a, a_scale, b, b_scale, out, p.splits > 1 ? ws : nullptr, s.lda ? s.lda : s.k,
               s.ldb ? s.ldb : (s.form == MOE_FP8_INPUT_GRAD ? s.n : s.k), s.ldo ? s.ldo : s.n, s.m, s.n, s.k,
               (int)ceil_div(s.n, kBK), p.kb_per_split, s.out_dtype == MOE_DTYPE_F32, s.accumulate != 0};
  hipError_t err = s.form == MOE_FP8_FORWARD ? launch_product<MOE_FP8_FORWARD>(g, p, st)
                   : s.form == MOE_FP8_INPUT_GRAD ? launch_product<MOE_FP8_INPUT_GRAD>(g, p, st)
                                                  : launch_product<MOE_FP8_WEIGHT_GRAD>(g, p, st);
  if (err != hipSuccess || p.splits == 1) return err;
  const int64_t quads = (int64_t)s.m * s.n / 4;
  hipLaunchKernelGGL(matmul_join_kernel, dim3((unsigned)std::min<int64_t>(ceil_div(quads, 256), 4096)), dim3(256), 0, st, g,
                     p.splits);
  return hipGetLastError();
}

hipError_t launch_quantize_act_t(int rows, int cols, const void* x, uint8_t* codes, float* scales, hipStream_t st) {
  hipLaunchKernelGGL(quant_act_t_kernel, dim3((unsigned)ceil_div(rows, 128), (unsigned)ceil_div(cols, 64)), dim3(256), 0, st,
                     static_cast<const uint16_t*>(x), rows, cols, codes, scales);
  return hipGetLastError();
}

}  // namespace moe
