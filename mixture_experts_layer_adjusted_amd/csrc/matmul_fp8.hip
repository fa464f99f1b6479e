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

// at most N of this wavefront's loads in flight, and none of its LDS reads
template <int N>
__device__ __forceinline__ void wait_counts() {
  static_assert(N < 64, "vmcnt");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4));
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
  const int quarter = (r >> 5) & 1;   // of the K quarters, neighbours apart
  return BN == 256 ? (r & 7) | quarter << 3 : BN == 128 ? ((r >> 1) & 3) | quarter << 2 : ((r >> 2) & 1) | quarter << 1;
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
__device__ __forceinline__ void contract(const Frag<false>* w, const Frag<false>& x, f32x4 (&p)[1]) {
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  p[0] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w->v, x.v, zero, 0, 0, 0, 0, 0, 0);
}
// (U blocks in turn, so that no instruction waits for the one before)
template <int U>
__device__ __forceinline__ void contract(const Frag<true>* w, const Frag<true>& x, f32x4 (&p)[U]) {
#pragma unroll
  for (int u = 0; u < U; ++u) p[u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int s = 0; s < 4; ++s)
#pragma unroll
    for (int u = 0; u < U; ++u) p[u] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[u].v[s], x.v[s], p[u], 0, 0, 0);
}

// 64 lanes x 16 (or 4) bytes at base + off + step into LDS at dst + 16 (or 4) lane
__device__ __forceinline__ void load_lds16(__amdgpu_buffer_rsrc_t base, uint8_t* dst, uint32_t off, uint32_t step) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(base, (lds_void_t*)dst, 16, off, step, 0, 0);
}
__device__ __forceinline__ void load_lds4(__amdgpu_buffer_rsrc_t base, uint8_t* dst, uint32_t off, uint32_t step) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(base, (lds_void_t*)dst, 4, off, step, 0, 0);
}

template <int FORM, int BM, int BN, int WM, int WN, int STAGES>
struct TileShape {
  static constexpr bool KN = FORM == MOE_FP8_INPUT_GRAD, ROWS = FORM == MOE_FP8_WEIGHT_GRAD;
  static constexpr int kWaves = WM * WN, kThreads = kWaves * 64;
  static constexpr int kMB = BM / WM / 16, kNB = BN / WN / 16;
  static constexpr int kADma = BM / 8 / kWaves, kBDma = BN / 8 / kWaves;   // 1 KB loads of a wavefront per stage
  static constexpr int kDataBytes = (BM + BN) * kBK;
  // K blocks whose scales are loaded together (forward 8192 x 4096 x 7168: 219 us with 4, 215 with 8; the input gradient
  // 192 x 3024 x 2176 the other way round, 10.2 and 10.4; the weight gradient's two vectors leave no room for more)
  static constexpr int kSpan = FORM == MOE_FP8_FORWARD ? 8 : ROWS && STAGES == 3 ? 2 : 4;
  static constexpr int kPart = 64 / kSpan;                                  // rows of one scale load
  static constexpr int kAScale = BM * kSpan * 4;                            // a's scales of kSpan K blocks
  static constexpr int kBScale = ROWS ? BN * kSpan * 4 : 256;               // b's: rows, or up to 16 column blocks
  static constexpr int kScales = STAGES * kDataBytes;                        // where they start
  static constexpr int kUnread = kScales + 3 * (kAScale + kBScale);          // where loads go that nothing reads
  static constexpr bool kPrefetch = STAGES == 2 && BM == 256 && !KN;
  static constexpr int kLds = kUnread + (kPrefetch ? kWaves * 256 : 256);
  static_assert(BM % 64 == 0 && BM / 64 + (ROWS ? BN / 64 : 1) <= kWaves, "one scale load of a wavefront per stage");
  static_assert(STAGES - 1 <= kSpan, "three spans of scales hold all that is in use");
  static_assert(kADma * 8 * kWaves == BM && kBDma * 8 * kWaves == BN, "whole loads");
};

// One BM x BN tile of the output over one slice of the K blocks.  STAGES stages of one K block each, filled by direct
// loads.  Rows and columns past the matrix read a valid row or column and are not stored.
//
// A K block is worked off in row blocks of 16.  Before the last one, every fragment of the stage has been read: there
// the wavefronts meet (the next stage has landed, this one may be filled again), and the next K block's first fragments
// are on their way while the last row block's products run, so that the matrix units do not wait at a K block's start.
//
// Scales: a row's are neighbours along K, rows are far apart, and a load costs by the cache lines it touches (64 rows
// a load kept the address unit busy 183 cycles, 29 a load of codes).  So a load takes several K blocks (a span) of fewer
// rows, one load of a wavefront per stage, a span ahead, into one of three spans in LDS: [kPart rows][K block][row].
// Wavefronts without a share load one word, which costs the address unit next to nothing (repeating another's share
// took 4 to 10% of small tiles' time: 1000 x 2816 x 2048 15.4 us -> 14.7).
//
// L2: with two stages, what misses L2 is late (all hits: 199 us against 237 at 8192 x 4096 x 7168).  Of the tiles an XCD
// works on at a time, eight share a's rows and four b's, so each asks for an eighth and a quarter of the lines of the
// stage after those in flight: one load of a wavefront, into LDS that nothing reads (237 -> 210 us; every tile asking
// for all its lines gained nothing).  More stages do not need it.
//
// SETS = 2: where there is no second workgroup for a CU, a second set of wavefronts takes the second half of the K blocks
// in an LDS of its own, and the first adds its sums at the end (77 x 7168 x 2048 to bf16: 9.2 us -> 8.4, to fp32
// 13.7 -> 11.7; 1000 x 2816 x 2048 to fp32: 26.2 -> 22.2; a bf16 input gradient 77 x 2048 x 7168: 14.6 -> 12.6).
template <int FORM, bool EXACT, int BM, int BN, int WM, int WN, int STAGES, int SETS>
__global__ void __launch_bounds__(WM * WN * 64 * SETS) matmul_tile_kernel(MatmulArgs g, int MT, int NT, int splits, int chunk) {
  constexpr bool KN = FORM == MOE_FP8_INPUT_GRAD, ROWS = FORM == MOE_FP8_WEIGHT_GRAD;
  using S = TileShape<FORM, BM, BN, WM, WN, STAGES>;
  constexpr int kMB = S::kMB, kNB = S::kNB;
  extern __shared__ __attribute__((aligned(16))) uint8_t all_lds[];
  constexpr int kSpan = S::kSpan, kPart = S::kPart;
  const int tid = threadIdx.x, lane = tid & 63;
  const int first_wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int set = SETS == 1 ? 0 : first_wave / S::kWaves, wave = first_wave - set * S::kWaves;
  uint8_t* const lds = all_lds + set * S::kLds;
  uint8_t* const ascales = lds + S::kScales;
  uint8_t* const bscales = ascales + 3 * S::kAScale;
  // tiles of one slice after another, dealt to the XCDs in runs of `chunk`
  const int64_t Ls = xcd_logical(blockIdx.x, chunk);
  if (Ls >= (int64_t)MT * NT * splits) return;
  const int slice = (int)(Ls / (MT * NT)), L = (int)(Ls - (int64_t)slice * MT * NT);
  const int grp = L / (kGroupM * NT), gm = min(kGroupM, MT - grp * kGroupM), rem = L - grp * kGroupM * NT;
  const int m0 = (grp * kGroupM + rem % gm) * BM, n0 = rem / gm * BN;
  const int wm = wave / WN, wn = wave % WN;
  const int KB = g.k / kBK;
  int kb0 = slice * g.kb_per_split, nk = min(g.kb_per_split, KB - kb0);
  const int meetings = nk > 0 ? 1 + (nk + SETS - 1) / SETS : 0;   // of the set with the most K blocks
  if constexpr (SETS == 2) {
    kb0 += set * ((nk + 1) / 2);
    nk = (nk + 1 - set) / 2;
  }

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
  // scales: in the load of stage s, lane (kb, r) takes K block kb and row r of part (s mod kSpan) BM / 64 + w of the span
  // after s's; w: the wavefront among the first BM / 64 (a's rows) or the next (b's rows, or all the span's column blocks
  // in each load).  The others load one word into LDS that nothing reads, so that every wavefront has the same loads in
  // flight.
  constexpr int kAW = BM / 64, kBW = ROWS ? BN / 64 : 1;
  const bool idle = wave >= kAW + kBW, for_a = wave < kAW || idle, for_rows = for_a || ROWS;
  const int s_wave = for_a ? wave % kAW : wave - kAW;
  const int s_step = idle ? 0 : for_a ? kAW : ROWS ? kBW : 0;        // parts of one stage's loads
  const int s_row = (for_rows ? s_wave * kPart : n0 / kBK) + lane % kPart;
  const int s_last = for_a ? g.m - 1 - m0 : ROWS ? g.n - 1 - n0 : g.nblk - 1;
  const uint32_t s_rowstep = idle ? 0 : KN && !for_a ? 1 : (uint32_t)KB;
  const uint32_t s_kstep = idle ? 0 : KN && !for_a ? (uint32_t)g.nblk : 1;
  uint8_t* const s_dst = idle ? lds + S::kUnread : (for_a ? ascales : bscales) + (for_rows ? s_wave * 256 : 0);
  const int s_span = idle ? 0 : for_a ? S::kAScale : S::kBScale;
  const uint8_t* abase = g.a + (int64_t)m0 * g.lda;
  const uint8_t* bbase = KN ? g.b + n0 : g.b + (int64_t)n0 * g.ldb;
  const __amdgpu_buffer_rsrc_t abuf =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(abase), (short)0, -1, 0x00020000);
  const float* sbase = for_a ? g.a_scale + (int64_t)m0 * KB : ROWS ? g.b_scale + (int64_t)n0 * KB : g.b_scale;
  const __amdgpu_buffer_rsrc_t sbuf =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<float*>(sbase), (short)0, -1, 0x00020000);
  auto issue_scales = [&](int span, int j) {
    const uint32_t kb = (uint32_t)min(kb0 + span * kSpan + lane / kPart, KB - 1);
    const uint32_t r = (uint32_t)min(s_row + j * s_step * kPart, s_last);
    load_lds4(sbuf, s_dst + span % 3 * s_span + j * s_step * 256, (r * s_rowstep + kb * s_kstep) * 4, 0);
  };
  // load p of this wavefront's share of stage kt: a's codes, b's, scales.  Past the last K block the last one again:
  // no branch in the loop, where the compiler would carry folds across it
  constexpr int kLoads = S::kADma + S::kBDma + 1;
  // what is issued after a stage's loads until the stage has to be there: its prefetch, then STAGES - 2 stages with theirs
  constexpr int kPf = S::kPrefetch ? 1 : 0, kYounger = (STAGES - 2) * (kLoads + kPf) + kPf;
  auto issue_load = [&](int kt, int p) {
    uint8_t* st = lds + kt % STAGES * S::kDataBytes;
    const uint32_t k0 = (uint32_t)(kb0 + min(kt, nk - 1)) * kBK;
    if (p < S::kADma) {
      load_lds16(abuf, st + (wave * S::kADma + p) * 1024, aoff[p], k0);
    } else if (p < kLoads - 1) {
      const __amdgpu_buffer_rsrc_t bbuf = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<uint8_t*>(KN ? bbase + (int64_t)k0 * g.ldb : bbase), (short)0, -1, 0x00020000);
      const int i = p - S::kADma;
      load_lds16(bbuf, st + BM * kBK + (wave * S::kBDma + i) * 1024, boff[i], KN ? 0u : k0);
    } else {
      issue_scales(kt / kSpan + 1, kt % kSpan);
    }
  };

  // L2 prefetch: a wavefront's lines of a's rows (the first quarter of the wavefronts) or of b's
  constexpr int kPfA = S::kWaves / 4, kPfB = S::kWaves - kPfA;
  constexpr int kEachA = (BM / 8 + kPfA - 1) / kPfA, kEachB = (BN / 4 + kPfB - 1) / kPfB;
  static_assert(kEachA <= 64 && kEachB <= 64, "a lane a line");
  const bool pf_a = wave < kPfA;
  const int pf_line = pf_a ? rem / gm % 8 * (BM / 8) + min(wave * kEachA + lane % kEachA, BM / 8 - 1)
                           : rem % gm % 4 * (BN / 4) + min((wave - kPfA) * kEachB + lane % kEachB, BN / 4 - 1);
  const uint32_t pf_off = pf_a ? (uint32_t)min(pf_line, g.m - 1 - m0) * (uint32_t)g.lda
                               : (uint32_t)min(pf_line, g.n - 1 - n0) * (uint32_t)g.ldb;
  const __amdgpu_buffer_rsrc_t pf_buf =
      __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(pf_a ? abase : bbase), (short)0, -1, 0x00020000);
  auto prefetch = [&](int kt) {
    if constexpr (S::kPrefetch)
      load_lds4(pf_buf, lds + S::kUnread + wave * 256, pf_off, (uint32_t)(kb0 + min(kt, nk - 1)) * kBK);
  };

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

  if (nk > 0) {
#pragma unroll
    for (int j = 0; j < kSpan; ++j) issue_scales(0, j);
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) {
#pragma unroll
      for (int p = 0; p < kLoads; ++p) issue_load(s, p);
      prefetch(STAGES - 1 + s);   // (as in the loop, whose waits count on it)
    }
  }

  // Columns are taken kCols blocks at a time (widened fragments are twice as large: half the wavefront's).
  constexpr int kGroups = EXACT ? 2 : 1, kCols = kNB / kGroups;
  static_assert(kNB % kGroups == 0 && kMB > 1, "whole groups, and a row block before the last");
  struct Start {   // a group's column fragments, read ahead
    i32x8 w[kCols];
  };
  i32x8 next;         // the next row block's fragment
  float sa_next;      // and scale
  // reads group h of K block kt (stage kt mod STAGES)
  auto read_start = [&](int kt, int h, Start& s) {
    const uint8_t* st = lds + kt % STAGES * S::kDataBytes;
#pragma unroll
    for (int jj = 0; jj < kCols; ++jj) {
      const int j = h * kCols + jj;
      if constexpr (KN) {
        // ds_read_b64_tr_b8: within 16 lanes, lane s names row 8 q + s / 2 at columns 8 (s % 2)..+7 of the 16 and
        // receives its own column's eight rows
        const uint8_t* wt = st + BM * kBK;
        const int col = ncol + 16 * j + 8 * (lane & 1);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int r = 32 * kq + 8 * q + (l16 >> 1);
          const i32x2 v = __builtin_amdgcn_ds_read_tr8_b64_v2i32(
              (lds_i32x2*)(wt + r * BN + (((col >> 4) ^ kn_swz<BN>(r)) << 4) + (col & 15)));
          s.w[jj][2 * q] = v[0];
          s.w[jj][2 * q + 1] = v[1];
        }
      } else {
        s.w[jj] = frag_at(st + wr + j * 16 * kBK + c0, st + wr + j * 16 * kBK + c1);
      }
    }
  };
  // the scale of row r (a multiple of 16, + what the caller adds) in the spans at `at`
  auto scale_at = [&](const uint8_t* at, int span_bytes, int kt, int r) {
    return reinterpret_cast<const float*>(at + kt / kSpan % 3 * span_bytes) + r / kPart * 64 + kt % kSpan * kPart + r % kPart;
  };
  auto read_rows = [&](int kt, int i) {   // row block i's fragment and scale
    const uint8_t* st = lds + kt % STAGES * S::kDataBytes;
    next = frag_at(st + xr + i * 16 * kBK + c0, st + xr + i * 16 * kBK + c1);
    sa_next = scale_at(ascales, S::kAScale, kt, mrow + 16 * i)[kPart < 16 ? l16 / kPart * 64 + l16 % kPart : l16];
  };
  // Group h of K block kt from `now`; `then` receives the start of the group after it.  Pieces of kUnit blocks: a
  // piece's instructions, then the fold of the piece kLag before it, whose results are there by then, in this order (left
  // to itself the compiler folds each result at once, waiting for it).
  auto group = [&](int kt, int h, const Start& now, Start& then) {
    constexpr int kUnit = EXACT && kCols > 1 ? 2 : 1, kLag = EXACT ? 1 : 2, kPer = kCols / kUnit, kPieces = kMB * kPer;
    f32x4 part[kLag + 1][kUnit];
    Frag<EXACT> wf[kCols], xf;
    float sa[kMB], sw = 0.0f;
    f32x4 swr[kCols];   // weight gradient: the lane's four columns'
    if constexpr (!ROWS) sw = scale_at(bscales, S::kBScale, kt, 0)[wblk];
#pragma unroll
    for (int jj = 0; jj < kCols; ++jj) {
      wf[jj].set(now.w[jj]);
      if constexpr (ROWS) 
        swr[jj] = *reinterpret_cast<const f32x4*>(scale_at(bscales, S::kBScale, kt, ncol + 16 * (h * kCols + jj)) + 4 * kq);
    }
#pragma unroll
    for (int n = 0; n < kPieces + kLag; ++n) {
      if (n < kPieces) {
        const int i = n / kPer, jj = n % kPer * kUnit;
        if (jj == 0) {
          xf.set(next);
          sa[i] = sa_next;
          if (i + 1 < kMB) {
            read_rows(kt, i + 1);
          } else if (h + 1 < kGroups) {
            read_start(kt, h + 1, then);
            read_rows(kt, 0);
          } else {
            // the next stage has landed, and this wavefront's reads of this stage are done
            prefetch(kt + STAGES);
            wait_counts<kYounger>();
            asm volatile("" ::: "memory");
            __builtin_amdgcn_s_barrier();
            asm volatile("" ::: "memory");
            read_start(kt + 1, 0, then);
            read_rows(kt + 1, 0);
          }
        }
        // loads of the stage that the last meeting set free, one at a time between the pieces: issued together they
        // fill the address unit's queue, and the wavefronts stand before it
        constexpr int kSlots = kGroups * kPieces - kPer, kEach = (kLoads + kSlots - 1) / kSlots;   // all before the meeting
#pragma unroll
        for (int p = (h * kPieces + n) * kEach; p < (h * kPieces + n + 1) * kEach; ++p)
          if (p < kLoads) issue_load(kt + STAGES - 1, p);
        contract(&wf[jj], xf, part[n % (kLag + 1)]);
      }
      if (n >= kLag) {
        const int q = n - kLag, i = q / kPer;
#pragma unroll
        for (int u = 0; u < kUnit; ++u) {
          const int jj = q % kPer * kUnit + u;
          const f32x4& p = part[q % (kLag + 1)][u];
          const float f = ROWS ? sa[i] : sa[i] * sw;
          f32x4& c = acc[i][h * kCols + jj];
#pragma unroll
          for (int v = 0; v < 4; ++v) c[v] = fmaf(p[v], ROWS ? f * swr[jj][v] : f, c[v]);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  if (nk > 0) {
    wait_counts<kYounger>();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    Start even, odd;
    read_start(0, 0, even);
    read_rows(0, 0);
    if constexpr (kGroups == 2) {
      for (int kt = 0; kt < nk; ++kt) {
        group(kt, 0, even, odd);
        group(kt, 1, odd, even);
      }
    } else {
      int kt = 0;
      for (; kt + 1 < nk; kt += 2) {
        group(kt, 0, even, odd);
        group(kt + 1, 0, odd, even);
      }
      if (kt < nk) group(kt, 0, even, odd);
    }
  }
  if constexpr (SETS == 2) {
    for (int i = nk > 0 ? 1 + nk : 0; i < meetings; ++i) __builtin_amdgcn_s_barrier();
    // the second set's sums, through its own part of LDS once nothing is on its way there
    wait_counts<0>();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    f32x4* const sums = reinterpret_cast<f32x4*>(all_lds + S::kLds) + wave * (kMB * kNB * 64) + lane;
    static_assert(BM * BN * 4 <= S::kLds, "a tile's sums");
    if (set == 1) {
#pragma unroll
      for (int i = 0; i < kMB; ++i)
#pragma unroll
        for (int j = 0; j < kNB; ++j) sums[(i * kNB + j) * 64] = acc[i][j];
    }
    wait_counts<0>();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (set == 1) return;
#pragma unroll
    for (int i = 0; i < kMB; ++i)
#pragma unroll
      for (int j = 0; j < kNB; ++j) acc[i][j] += sums[(i * kNB + j) * 64];
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
        *reinterpret_cast<f32x4*>(g.part + ((int64_t)slice * g.m + row) * g.n + col) = acc[i][j];
      else
        store4(g, row, col, acc[i][j]);
    }
  }
  wait_counts<0>();   // the loads past the last K block still write to this workgroup's LDS
}

// out = the sum of the slices, in their order
__global__ void __launch_bounds__(256) matmul_join_kernel(MatmulArgs g, int splits) {
  const int64_t per = (int64_t)g.m * g.n, quads = per / 4;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < quads; i += (int64_t)gridDim.x * 256) {
    f32x4 v = *reinterpret_cast<const f32x4*>(g.part + 4 * i);
#pragma unroll 8
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
template <int MB, int U, bool EXACT>
__global__ void __launch_bounds__(kRowWaves * 64) matmul_rows_kernel(MatmulArgs g) {
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
        f32x4 p[1];
        contract(&w, x, p);
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[i][v] = fmaf(p[0][v], f[u][i], acc[i][v]);
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
// codes[c, r] of x[r, c] (bf16), one scale per column and run of 128 rows: amax times fp32(1 / 448), 1 for a run of
// zeros; rows past the last are zeros.  (8100 x 7168: 35.7 us, 174 MB.)  A 128-row x 64-column block goes through LDS as words of two rows: eight lanes
// load 16 bytes each of a row pair (128 bytes of both rows), and four lanes then take one column's rows, 32 each; the
// pitch of 65 words keeps either side on distinct banks.  The quotients are rounded without a division each: with r
// the rounded 1 / scale and q = v r, the remainder v - q scale is exact in one fma and q + remainder r is the rounded
// quotient (Markstein); scales outside 2^-64..2^64, where it could underflow or overflow, divide.
__global__ void __launch_bounds__(256) quant_act_t_kernel(const uint16_t* __restrict__ x, int rows, int cols,
                                                          uint8_t* __restrict__ codes, float* __restrict__ scales) {
  __shared__ uint32_t tile[64][65];
  const int64_t r0 = (int64_t)blockIdx.x * 128;
  const int c0 = blockIdx.y * 64, tid = threadIdx.x;
  const int64_t runs = gridDim.x;
  {
    const int cl = (tid & 7) * 8, c = c0 + cl;
    uint4 w[2][2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int64_t r = r0 + 2 * ((tid >> 3) + 32 * h) + e;
        w[h][e] = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows && c < cols) w[h][e] = *reinterpret_cast<const uint4*>(x + r * cols + c);   // (cols: a multiple of 8)
      }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t lo[4] = {w[h][0].x, w[h][0].y, w[h][0].z, w[h][0].w};
      const uint32_t hi[4] = {w[h][1].x, w[h][1].y, w[h][1].z, w[h][1].w};
      const int p = (tid >> 3) + 32 * h;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        tile[cl + 2 * i][p] = (lo[i] & 0xFFFFu) | (hi[i] << 16);
        tile[cl + 2 * i + 1][p] = (lo[i] >> 16) | (hi[i] & 0xFFFF0000u);
      }
    }
  }
  __syncthreads();
  const int c = tid >> 2, q = tid & 3;
  float v[32], amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t w = tile[c][16 * q + i];
    v[2 * i] = __uint_as_float(w << 16);
    v[2 * i + 1] = __uint_as_float(w & 0xFFFF0000u);
    amax = fmaxf(amax, fmaxf(fabsf(v[2 * i]), fabsf(v[2 * i + 1])));
  }
  amax = fmaxf(amax, __shfl_xor(amax, 1, 64));
  amax = fmaxf(amax, __shfl_xor(amax, 2, 64));
  if (c0 + c >= cols) return;
  const float scale = amax > 0.0f ? amax * (1.0f / 448.0f) : 1.0f;
  const float inv = __fdiv_rn(1.0f, scale);
  if (scale >= 0x1p-64f && scale < 0x1p64f) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const float s = v[i] * inv;
      v[i] = fmaf(fmaf(-s, scale, v[i]), inv, s);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __fdiv_rn(v[i], scale);
  }
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = e4m3x4_from_f32(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  uint8_t* p = codes + (int64_t)(c0 + c) * runs * 128 + r0 + 32 * q;
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  *reinterpret_cast<uint4*>(p + 16) = make_uint4(w[4], w[5], w[6], w[7]);
  if (q == 0) scales[(int64_t)(c0 + c) * runs + blockIdx.x] = scale;
}

// ---- which kernel ----------------------------------------------------------------------------------------------

// The tiles (Sets: two sets of wavefronts, each on half of the K blocks), and for bf16 and for fp32 outputs what a launch
// of one takes apart from its K blocks and what a K block takes with every CU at work (us; 0: not built), fitted to
// 138 shapes from 16 to 9000 rows with up to 8 slices; on 60 others the choice is 2% slower than the best on average.
enum Tile { kT256, kT128x256, kT128, kT128Pair, kT128Sets, kT64Pair, kT64Sets, kTiles };
struct TileCost {
  int bm, bn, per_cu;   // workgroups of a CU at a time
  float base, step, base_f32, step_f32;
};
constexpr TileCost kCost[kTiles] = {{256, 256, 1, 6.8f, 1.59f, 9.9f, 3.19f}, {128, 256, 1, 5.9f, 1.08f, 0.0f, 0.0f},
                                    {128, 128, 1, 5.1f, 0.62f, 0.0f, 0.0f},  {128, 128, 2, 4.5f, 1.44f, 4.8f, 1.88f},
                                    {128, 128, 1, 0.0f, 0.0f, 5.8f, 1.18f},  {64, 64, 2, 4.4f, 0.49f, 3.2f, 1.08f},
                                    {64, 64, 1, 4.8f, 0.23f, 4.5f, 0.52f}};

struct Plan {
  int rows;            // rows of a that the plan covers (from the first)
  int rows_mb;         // > 0: the few-rows kernel with so many blocks of 16 rows
  Tile tile;           // else the tile
  int splits, kb_per_split;
  float us;
};

// The plan for `rows` rows in one kernel (and the join): rounds of tiles over the CUs (1.5 us for the start of each after
// the first), a chip that is not full being up to 22% faster (38% where a CU has one workgroup in place of two), and for
// slices 2.3 us and their sums' way to memory and back.  kb / slices is 2 at least.
Plan plan_one(const moe_matmul_shape& s, int rows) {
  const int kb = s.k / kBK;
  Plan best{rows, 0, kT64Pair, 1, kb, 0.0f};
  if (s.form == MOE_FP8_FORWARD && (rows <= 16 || (rows <= 32 && s.k <= 2048))) {
    // straight from memory (1 x 4096 x 7168: 7.3 us against 10.6 with the best tile; 17 x 1024 x 1024: 4.4 against 5.9)
    best.rows_mb = rows <= 16 ? 1 : 2;
    best.us = 5.0f + (float)s.n * s.k / 1e7f;
    return best;
  }
  const bool f32 = s.out_dtype == MOE_DTYPE_F32;
  for (int i = 0; i < kTiles; ++i) {
    if (i == kT256 && s.form == MOE_FP8_WEIGHT_GRAD && !f32) continue;   // its two vectors of scales spill there
    const TileCost& c = kCost[i];
    const float step = f32 ? c.step_f32 : c.step;
    if (step == 0.0f) continue;
    const float base = f32 ? c.base_f32 : c.base;
    const float faster = c.per_cu == 2 ? 0.38f : 0.22f;
    const int64_t tiles = ceil_div(rows, c.bm) * ceil_div(s.n, c.bn);
    for (int want = 1; want <= 16 && (want == 1 || want * 2 <= kb); ++want) {
      const int per = (int)ceil_div(kb, want), splits = per > 0 ? (int)ceil_div(kb, per) : 1;
      if (splits != want) continue;
      const int64_t total = tiles * splits, at_once = 256 * c.per_cu;
      const float fill = total < at_once ? (float)total / at_once : 1.0f;
      const float rounds = (float)ceil_div(total, at_once);
      float us = base + 1.5f * (rounds - 1.0f) + rounds * per * step * (1.0f - faster * (1.0f - fill));
      if (splits > 1) us += 2.3f + (float)splits * rows * s.n * 8 / 4.2e6f;
      if (best.us == 0.0f || us < best.us)
        best = Plan{rows, 0, (Tile)i, splits, per, us};
    }
  }
  return best;
}

// One kernel for all rows, or one for whole tiles of them and one for the rest (4097 rows: one more row of tiles).
int plan_of(const moe_matmul_shape& s, Plan (&plans)[2]) {
  plans[0] = plan_one(s, s.m);
  int n = 1;
  for (int bm : {256, 128}) {
    const int rest = s.m % bm;
    if (rest == 0 || s.m < bm) continue;
    const Plan whole = plan_one(s, s.m - rest), last = plan_one(s, rest);
    if (whole.us + last.us < (n == 1 ? plans[0].us : plans[0].us + plans[1].us)) {
      plans[0] = whole;
      plans[1] = last;
      n = 2;
    }
  }
  return n;
}

template <int FORM, bool EXACT, int BM, int BN, int WM, int WN, int STAGES, int SETS = 1>
hipError_t launch_tile(const MatmulArgs& g, int splits, hipStream_t st) {
  using S = TileShape<FORM, BM, BN, WM, WN, STAGES>;
  static_assert(SETS * S::kLds <= 163840, "LDS");
  auto kern = &matmul_tile_kernel<FORM, EXACT, BM, BN, WM, WN, STAGES, SETS>;
  const hipError_t err = ensure_dynamic_lds(reinterpret_cast<const void*>(kern), SETS * S::kLds);
  if (err != hipSuccess) return err;
  const int64_t MT = ceil_div(g.m, BM), NT = ceil_div(g.n, BN);
  const int64_t total = MT * NT * splits;
  if (total >= (int64_t(1) << 31) - 256) return hipErrorInvalidValue;
  // an XCD's 32 CUs take neighbouring tiles; fewer at a time where there are not enough for every XCD
  const int chunk = (int)std::min<int64_t>(32, ceil_div(total, kXcds));
  const int64_t grid = ceil_div(total, kXcds * chunk) * (kXcds * chunk);
  return launch_kernel(kern, dim3((unsigned)grid), dim3(SETS * S::kThreads), SETS * S::kLds, st, g, (int)MT, (int)NT, splits, chunk);
}

template <int MB, bool EXACT>
hipError_t launch_rows(const MatmulArgs& g, hipStream_t st) {
  const dim3 grid((unsigned)(g.n / 16)), block(kRowWaves * 64);
  const int each = (int)ceil_div(g.k / kBK, kRowWaves);   // K blocks of a wavefront: all in flight at once if they fit
  if constexpr (MB == 1) {
    if (each > 4) {
      return launch_kernel(matmul_rows_kernel<1, 8, EXACT>, grid, block, 0, st, g);
    }
    if (each > 2) {
      return launch_kernel(matmul_rows_kernel<1, 4, EXACT>, grid, block, 0, st, g);
    }
  }
  // (two blocks of rows come with k <= 2048 only: no wavefront has more than two K blocks)
  return launch_kernel(matmul_rows_kernel<MB, 2, EXACT>, grid, block, 0, st, g);
}

template <int FORM, bool EXACT>
hipError_t launch_form(const MatmulArgs& g, const Plan& p, hipStream_t st) {
  if constexpr (FORM == MOE_FP8_FORWARD) {
    if (p.rows_mb == 1) return launch_rows<1, EXACT>(g, st);
    if (p.rows_mb == 2) return launch_rows<2, EXACT>(g, st);
  }
  switch (p.tile) {
    case kT256:
      if constexpr (FORM != MOE_FP8_WEIGHT_GRAD || EXACT) return launch_tile<FORM, EXACT, 256, 256, 2, 4, 2>(g, p.splits, st);
      return hipErrorInvalidValue;   // never planned
    case kT128x256: {
      // gradients: eight wavefronts side by side, each column of b read by one of them (input gradient 4096 x 2048 x 7168: 67.0 us
      // against 69.0 in two rows of four; the forward the other way round, 65.1 and 64.0)
      constexpr int kRows = FORM == MOE_FP8_FORWARD ? 2 : 1;
      if constexpr (!EXACT) return launch_tile<FORM, EXACT, 128, 256, kRows, 8 / kRows, 3>(g, p.splits, st);
      return hipErrorInvalidValue;
    }
    case kT128:
      if constexpr (!EXACT) return launch_tile<FORM, EXACT, 128, 128, 2, 4, 4>(g, p.splits, st);
      return hipErrorInvalidValue;
    case kT128Pair: return launch_tile<FORM, EXACT, 128, 128, 2, 2, 2>(g, p.splits, st);
    case kT128Sets:
      if constexpr (EXACT) return launch_tile<FORM, EXACT, 128, 128, 2, 2, 2, 2>(g, p.splits, st);
      return hipErrorInvalidValue;
    case kT64Sets: return launch_tile<FORM, EXACT, 64, 64, 2, 2, 4, 2>(g, p.splits, st);
    default: return launch_tile<FORM, EXACT, 64, 64, 2, 2, 4>(g, p.splits, st);
  }
}

template <int FORM>
hipError_t launch_product(const MatmulArgs& g, const Plan& p, hipStream_t st) {
  return g.out_f32 ? launch_form<FORM, true>(g, p, st) : launch_form<FORM, false>(g, p, st);
}

size_t sums_bytes(const moe_matmul_shape& s, const Plan& p) {
  return p.splits > 1 ? (size_t)p.splits * p.rows * s.n * 4 : 0;
}

}  // namespace

size_t matmul_fp8_workspace(const moe_matmul_shape& s) {
  if (s.m == 0 || s.n == 0 || s.k == 0) return 0;
  Plan plans[2];
  const int n = plan_of(s, plans);
  // (the second kernel's sums may take the first one's place: they run in order)
  return std::max(sums_bytes(s, plans[0]), n > 1 ? sums_bytes(s, plans[1]) : 0);
}

hipError_t launch_matmul_fp8(const moe_matmul_shape& s, const uint8_t* a, const float* a_scale, const uint8_t* b,
                             const float* b_scale, void* out, float* ws, hipStream_t st) {
  if (s.m == 0 || s.n == 0) return hipSuccess;
  Plan plans[2];
  const int n = plan_of(s, plans);
  const int64_t lda = s.lda ? s.lda : s.k, ldo = s.ldo ? s.ldo : s.n;
  const bool f32 = s.out_dtype == MOE_DTYPE_F32;
  int64_t row = 0;
  for (int i = 0; i < n; ++i) {
    const Plan& p = plans[i];
    const MatmulArgs g{a + row * lda, a_scale + row * (s.k / kBK), b, b_scale,
                       static_cast<char*>(out) + row * ldo * (f32 ? 4 : 2), p.splits > 1 ? ws : nullptr, lda,
                       s.ldb ? s.ldb : (s.form == MOE_FP8_INPUT_GRAD ? s.n : s.k), ldo, p.rows, s.n, s.k,
                       (int)ceil_div(s.n, kBK), p.kb_per_split, f32, s.accumulate != 0};
    hipError_t err = s.form == MOE_FP8_FORWARD      ? launch_product<MOE_FP8_FORWARD>(g, p, st)
                     : s.form == MOE_FP8_INPUT_GRAD ? launch_product<MOE_FP8_INPUT_GRAD>(g, p, st)
                                                    : launch_product<MOE_FP8_WEIGHT_GRAD>(g, p, st);
    if (err == hipSuccess && p.splits > 1) {
      const int64_t quads = (int64_t)p.rows * s.n / 4;
      err = launch_kernel(matmul_join_kernel, dim3((unsigned)std::min<int64_t>(ceil_div(quads, 256), 4096)), dim3(256), 0, st,
                          g, p.splits);
    }
    if (err != hipSuccess) return err;
    row += p.rows;
  }
  return hipSuccess;
}

hipError_t launch_quantize_act_t(int rows, int cols, const void* x, uint8_t* codes, float* scales, hipStream_t st) {
  return launch_kernel(quant_act_t_kernel, dim3((unsigned)ceil_div(rows, 128), (unsigned)ceil_div(cols, 64)), dim3(256), 0, st,
                     static_cast<const uint16_t*>(x), rows, cols, codes, scales);
}

}  // namespace moe
