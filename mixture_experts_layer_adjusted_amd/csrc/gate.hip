// Routing from given logits, and its gradient.
//
// For a token's logits l[0..N), a bias b (or none) and K picks:
//   s_i = 1 / (1 + exp(-l_i))   or   s_i = exp(l_i) / sum_j exp(l_j);
//   c_i = s_i + b_i ranks the experts; l_i = -inf or b_i = -inf takes expert i out;
//   with G groups of N / G neighbouring experts, only the TG groups with the largest score (the largest c,
//   or the sum of the two largest) stay; the K largest c left are the picks, equal ones by index;
//   g_k = scale s_k / sum of the picked s, or scale s_k.
// The gradient holds the picks fixed.  With q_k = s_k / sum of the picked s, and D = sum_k dg_k q_k:
//   sigmoid  renormalised   dl_k = scale (dg_k - D) q_k (1 - s_k);  plain  dl_k = scale dg_k s_k (1 - s_k)
//   softmax  renormalised   dl_k = scale (dg_k - D) q_k
//   softmax  plain          dl_i = scale p_i (dg_i [i picked] - sum_j dg_j p_j), every i
// and zero elsewhere.
//
// Lanes hold neighbouring experts: lane i of a token has the experts CPL i .. CPL i + CPL - 1 (one vector load), in
// lists of four sorted by key, so that a round of the selection is the largest head over the lanes and one pop, and
// equal keys leave in index order (lowest lane first, the sort being stable).
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr uint32_t kOut = 0u;       // key of an expert that is out (masked, in a closed group, or taken)
constexpr uint32_t kNanKey = 1u;    // a NaN ranks below every number
constexpr float kNegInf = -__builtin_inff();

// larger score, larger key; -0 and +0 are one score
__device__ __forceinline__ uint32_t key_of(float c) {
  const uint32_t b = __float_as_uint(c + 0.0f);
  const uint32_t k = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  return c != c ? kNanKey : k;
}
__device__ __forceinline__ float score_of(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key ^ 0x80000000u) : ~key);
}

// exp(x) from the 2^y instruction: y = x log2(e) rounded, and what the rounding (and the constant's) left out as a
// factor 1 + r.  Within 2 units in the last place; results below 2^-126 are 0, infinities and NaN as they should be.
__device__ __forceinline__ float exp_of(float x) {
  const float y = x * 1.44269502f;
  float r = fmaf(x, 1.44269502f, -y);
  r = fmaf(x, 1.92596299e-8f, r);
  const float e = __builtin_amdgcn_exp2f(y);
  return fabsf(x) < 150.0f ? fmaf(e, r * 0.693147182f, e) : e;   // (e may be infinite, and r NaN)
}

// CPL neighbouring logits (rows start anywhere: the loads need no more than the element's alignment)
template <int CPL>
__device__ __forceinline__ void load_run(const float* p, int left, float (&v)[CPL]) {
  if (left >= CPL) {
    struct __attribute__((packed, aligned(4))) Run { float v[CPL]; };
    const Run q = *reinterpret_cast<const Run*>(p);
#pragma unroll
    for (int j = 0; j < CPL; ++j) v[j] = q.v[j];
  } else {
#pragma unroll
    for (int j = 0; j < CPL; ++j) v[j] = j < left ? p[j] : kNegInf;
  }
}
template <int CPL>
__device__ __forceinline__ void load_run(const uint16_t* p, int left, float (&v)[CPL]) {
  if (left >= CPL) {
    struct __attribute__((packed, aligned(2))) Run { uint16_t v[CPL]; };
    const Run q = *reinterpret_cast<const Run*>(p);
#pragma unroll
    for (int j = 0; j < CPL; ++j) v[j] = __uint_as_float((uint32_t)q.v[j] << 16);
  } else {
#pragma unroll
    for (int j = 0; j < CPL; ++j) v[j] = j < left ? __uint_as_float((uint32_t)p[j] << 16) : kNegInf;
  }
}
__device__ __forceinline__ uint16_t to_bf16(float v) {
  const uint32_t b = __float_as_uint(v);
  return v != v ? (uint16_t)0x7FC0u : (uint16_t)((b + 0x7FFFu + ((b >> 16) & 1u)) >> 16);
}
__device__ __forceinline__ void store_run4(float* p, int left, const float (&v)[4]) {
  if (left >= 4) {
    struct __attribute__((packed, aligned(4))) Run { float v[4]; };
    *reinterpret_cast<Run*>(p) = Run{{v[0], v[1], v[2], v[3]}};
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < left) p[j] = v[j];
  }
}
__device__ __forceinline__ void store_run4(uint16_t* p, int left, const float (&v)[4]) {
  if (left >= 4) {
    struct __attribute__((packed, aligned(2))) Run { uint16_t v[4]; };
    *reinterpret_cast<Run*>(p) = Run{{to_bf16(v[0]), to_bf16(v[1]), to_bf16(v[2]), to_bf16(v[3])}};
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (j < left) p[j] = to_bf16(v[j]);
  }
}

// v from the lane that the DPP control names; lanes without one, or outside row_mask, get `other`
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ uint32_t moved(uint32_t other, uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)other, (int)v, CTRL, ROW_MASK, 0xF, false);
}

// A reduction over the L lanes of a token, the result in each of them.  L = 16: four rotations of the 16-lane row
// (row_ror:8, 4, 2, 1).  L = 32: then the other row by a shuffle.  L = 64: row shifts by 1, 2, 4, 8, row 0's and 2's
// result into the row after (row_bcast:15), lane 31's into the upper rows (row_bcast:31), and lane 63's to all.
// The order is fixed, so sums repeat to the bit.
template <int L, typename Op>
__device__ __forceinline__ uint32_t reduce(uint32_t v, uint32_t neutral, Op op) {
  if constexpr (L == 64) {
    v = op(v, moved<0x111, 0xF>(neutral, v));
    v = op(v, moved<0x112, 0xF>(neutral, v));
    v = op(v, moved<0x114, 0xF>(neutral, v));
    v = op(v, moved<0x118, 0xF>(neutral, v));
    v = op(v, moved<0x142, 0xA>(neutral, v));
    v = op(v, moved<0x143, 0xC>(neutral, v));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
  } else {
    v = op(v, moved<0x128, 0xF>(v, v));
    v = op(v, moved<0x124, 0xF>(v, v));
    v = op(v, moved<0x122, 0xF>(v, v));
    v = op(v, moved<0x121, 0xF>(v, v));
    if constexpr (L == 32) v = op(v, (uint32_t)__shfl_xor((int)v, 16, 64));
    return v;
  }
}
template <int L>
__device__ __forceinline__ uint32_t max_of(uint32_t v) {
  return reduce<L>(v, 0u, [](uint32_t a, uint32_t b) { return max(a, b); });
}
template <int L>
__device__ __forceinline__ float max_of(float v) {
  return __uint_as_float(reduce<L>(__float_as_uint(v), __float_as_uint(kNegInf), [](uint32_t a, uint32_t b) {
    return __float_as_uint(fmaxf(__uint_as_float(a), __uint_as_float(b)));
  }));
}
template <int L>
__device__ __forceinline__ float sum_of(float v) {
  return __uint_as_float(reduce<L>(__float_as_uint(v), 0u, [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

struct GateArgs {
  const void* logits;
  int64_t ld;
  const float* bias;
  int T, N, K, G, TG;
  bool top2, renorm;
  float scale;
  int32_t* idx;
  float* gate;
  int32_t* counts;   // [gridDim.x, N] picks of each expert in each workgroup; null: not counted
};

// Bits of the groups that stay open.  keys: the token's keys in LDS.  2^p lanes work on a group (as many as
// leave a lane set for every group), each on every 2^p-th expert; their two largest join by shuffles.  A
// group's score counts numbers only: a NaN or an absent second adds nothing.
__device__ __forceinline__ uint64_t open_groups(const uint32_t* keys, const GateArgs& a, int lane, int lanes_log2) {
  const int gs = a.N / a.G, per = 1 << lanes_log2;
  const int g = lane >> lanes_log2;
  uint32_t k1 = kOut, k2 = kOut;
  if (g < a.G) {
    for (int i = lane & (per - 1); i < gs; i += per) {
      const uint32_t k = keys[g * gs + i];
      k2 = max(k2, min(k1, k));
      k1 = max(k1, k);
    }
  }
  for (int m = 1; m < per; m <<= 1) {
    const uint32_t o1 = __shfl_xor(k1, m, 64), o2 = __shfl_xor(k2, m, 64);
    k2 = max(max(k2, o2), min(k1, o1));
    k1 = max(k1, o1);
  }
  uint32_t score = k1;
  if (a.top2 && k2 > kNanKey) score = key_of(score_of(k1) + score_of(k2));
  // the rank of the lane's group: groups above it, or equal to it and before it
  int rank = 0;
  for (int h = 0; h < a.G; ++h) {
    const uint32_t o = (uint32_t)__builtin_amdgcn_readlane((int)score, h << lanes_log2);
    rank += (o > score || (o == score && h < g)) ? 1 : 0;
  }
  const uint64_t first = __ballot(g < a.G && rank < a.TG);
  uint64_t open = 0;
  for (int h = 0; h < a.G; ++h) open |= ((first >> (h << lanes_log2)) & 1ull) << h;
  return open;
}

// L lanes a token: 64, or 16 where a token's experts are few (four tokens a wavefront).
template <int CPL, int L, typename TL, bool SOFTMAX>
__global__ void __launch_bounds__(kThreads) gate_kernel(GateArgs a, int lanes_log2) {
  constexpr int kTokens = 64 / L;                    // tokens of a wavefront
  constexpr int kLists = (CPL + 3) / 4, kLen = CPL < 4 ? CPL : 4;
  __shared__ int32_t hist[kMaxRouted];
  __shared__ uint32_t keys[L == 64 ? kWaves : 1][kMaxRouted];
  __shared__ int2 won[kWaves][kTokens][kMaxTopK];    // the picks: expert, and its score (softmax renormalised: logit)
  const int tid = threadIdx.x, wl = tid & 63, lane = wl & (L - 1), slot = wl / L;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int N = a.N, K = a.K;
  for (int e = tid; e < N; e += kThreads) hist[e] = 0;
  const bool limited = L == 64 && a.TG < a.G;
  const int first = lane * CPL, left = N - first;
  float bias[CPL];
  int group[CPL];
#pragma unroll
  for (int j = 0; j < CPL; ++j) {
    bias[j] = j < left ? (a.bias ? a.bias[first + j] : 0.0f) : kNegInf;
    group[j] = limited && j < left ? (first + j) / (N / a.G) : 0;
  }
  // lanes before this one in its token's 16 (for the first of equals)
  const uint32_t before = L == 64 ? 0u : ((1u << lane) - 1u) << (wl & 16);
  __syncthreads();
  const int64_t per_block = (int64_t)kWaves * kTokens;
  for (int64_t t0 = (int64_t)blockIdx.x * per_block + wave * kTokens; t0 < a.T; t0 += (int64_t)gridDim.x * per_block) {
    const int64_t t = t0 + slot;
    const bool real = t < a.T;   // (16 lanes a token: the last wavefront may have fewer than four)
    float l[CPL], s[CPL];
    load_run<CPL>(static_cast<const TL*>(a.logits) + (real ? t : t0) * a.ld + first, left, l);
    if constexpr (SOFTMAX) {
      float top = l[0];
#pragma unroll
      for (int j = 1; j < CPL; ++j) top = fmaxf(top, l[j]);
      top = max_of<L>(top);
      if (top == kNegInf) top = 0.0f;
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < CPL; ++j) {
        s[j] = exp_of(l[j] - top);
        sum += s[j];
      }
      sum = sum_of<L>(sum);
      const float r = sum == 0.0f ? 0.0f : 1.0f / sum;   // 0: every expert masked
#pragma unroll
      for (int j = 0; j < CPL; ++j) s[j] *= r;
    } else {
#pragma unroll
      for (int j = 0; j < CPL; ++j) s[j] = __builtin_amdgcn_rcpf(1.0f + exp_of(-l[j]));
    }
    uint32_t key[kLists][4];
    uint32_t order[kLists];       // which expert of the lane each entry is, a byte each
#pragma unroll
    for (int q = 0; q < kLists; ++q) {
      order[q] = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = 4 * q + j;
        key[q][j] = j < kLen && !(l[i] == kNegInf || bias[i] == kNegInf) ? key_of(s[i] + bias[i]) : kOut;
      }
    }
    if (limited) {
#pragma unroll
      for (int j = 0; j < CPL; ++j)
        if (j < left) keys[wave][first + j] = key[j / 4][j % 4];
      __builtin_amdgcn_wave_barrier();   // LDS operations of one wavefront take effect in program order
      const uint64_t open = open_groups(keys[wave], a, lane, lanes_log2);
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int j = 0; j < CPL; ++j)
        if (!((open >> group[j]) & 1ull)) key[j / 4][j % 4] = kOut;
    }
    // each list in descending order, equal keys as they stand (neighbours change places only if the later is larger)
#pragma unroll
    for (int q = 0; q < kLists; ++q) {
      uint32_t at[4] = {4u * q, 4u * q + 1u, 4u * q + 2u, 4u * q + 3u};
#pragma unroll
      for (int end = kLen - 1; end > 0; --end)
#pragma unroll
        for (int j = 0; j < end; ++j) {
          const bool swap = key[q][j + 1] > key[q][j];
          const uint32_t hi = max(key[q][j], key[q][j + 1]), lo = min(key[q][j], key[q][j + 1]);
          const uint32_t x = swap ? at[j + 1] : at[j], y = swap ? at[j] : at[j + 1];
          key[q][j] = hi, key[q][j + 1] = lo, at[j] = x, at[j + 1] = y;
        }
      order[q] = at[0] | (at[1] << 8) | (at[2] << 16) | (at[3] << 24);
    }
    for (int k = lane; k < K; k += L) won[wave][slot][k] = make_int2(-1, __float_as_int(kNegInf));
    __builtin_amdgcn_wave_barrier();
    for (int k = 0; k < K; ++k) {
      uint32_t head = key[0][0];
      if constexpr (kLists > 1) head = max(head, key[1][0]);
      const uint32_t best = max_of<L>(head);
      if (L == 64 ? best == kOut : __ballot(best != kOut) == 0) break;
      const uint64_t at = __ballot(head == best && best != kOut);
      bool mine;
      if constexpr (L == 64) {
        mine = wl == __builtin_ctzll(at);
      } else {
        const uint32_t half = wl < 32 ? (uint32_t)at : (uint32_t)(at >> 32);
        mine = head == best && best != kOut && (half & before) == 0;
      }
      if (mine) {
        const int q = kLists == 1 || key[0][0] == best ? 0 : 1;   // the first list's expert comes first
        uint32_t j = order[0] & 0xFFu;
        if (kLists > 1 && q == 1) j = order[kLists - 1] & 0xFFu;
        float v = (SOFTMAX && a.renorm) ? l[0] : s[0];
#pragma unroll
        for (int i = 1; i < CPL; ++i)
          if (j == (uint32_t)i) v = (SOFTMAX && a.renorm) ? l[i] : s[i];
        // (a softmax over a NaN has no number: the score says so where the logit may not)
        if (SOFTMAX && a.renorm && best == kNanKey) v = __builtin_nanf("");
        won[wave][slot][k] = make_int2(first + (int)j, __float_as_int(v));
#pragma unroll
        for (int p = 0; p < kLists; ++p)
          if (p == q) {
#pragma unroll
            for (int i = 0; i + 1 < kLen; ++i) key[p][i] = key[p][i + 1];
            key[p][kLen - 1] = kOut;
            order[p] >>= 8;
          }
      }
    }
    __builtin_amdgcn_wave_barrier();
    constexpr int kHalves = L == 16 ? 2 : 1;   // 16 lanes hold up to 32 picks
    float g[kHalves], v[kHalves];
    int e[kHalves];
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      e[h] = -1, v[h] = kNegInf;
      if (lane + L * h < K) {
        const int2 w = won[wave][slot][lane + L * h];
        e[h] = w.x, v[h] = __int_as_float(w.y);
      }
    }
    float top = 0.0f;
    if (SOFTMAX && a.renorm) {   // from the picked logits, so that no picked score has underflowed
      top = v[0];
#pragma unroll
      for (int h = 1; h < kHalves; ++h) top = fmaxf(top, v[h]);
      top = max_of<L>(top);
    }
    float sum = 0.0f;
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      g[h] = e[h] < 0 ? 0.0f : SOFTMAX && a.renorm ? exp_of(v[h] - top) : v[h];
      sum += g[h];
    }
    if (a.renorm) {
      sum = sum_of<L>(sum);
#pragma unroll
      for (int h = 0; h < kHalves; ++h) g[h] = sum == 0.0f ? 0.0f : g[h] / sum;
    }
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
      if (real && lane + L * h < K) {
        a.idx[t * K + lane + L * h] = e[h];
        a.gate[t * K + lane + L * h] = a.scale * g[h];
        if (e[h] >= 0) atomicAdd(&hist[e[h]], 1);
      }
    __builtin_amdgcn_wave_barrier();
  }
  if (!a.counts) return;
  __syncthreads();
  for (int e = tid; e < N; e += kThreads) a.counts[(int64_t)blockIdx.x * N + e] = hist[e];
}

// load[e] = sum over the workgroups of counts[w, e]: 64 experts per workgroup, its wavefronts every 16th row
__global__ void __launch_bounds__(kThreads) gate_load_kernel(const int32_t* __restrict__ counts, int rows, int N,
                                                             int32_t* __restrict__ load) {
  __shared__ int32_t part[kWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = blockIdx.x * 64 + lane;
  int c = 0;
  if (e < N) {
#pragma unroll 16
    for (int r = wave; r < rows; r += kWaves) c += counts[(int64_t)r * N + e];
  }
  part[wave][lane] = c;
  __syncthreads();
  if (wave == 0 && e < N) {
    int sum = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) sum += part[w][lane];
    load[e] = sum;
  }
}

__global__ void gate_zero_kernel(int32_t* p, int n) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) p[i] = 0;
}

struct GateBwdArgs {
  const void* logits;
  int64_t ld, d_ld;
  const int32_t* idx;
  const float* d_gate;
  void* d_logits;
  int T, N, K;
  bool renorm;
  float scale;
};

// L lanes a token (16, or 32 for more than 16 picks).  The picks' lanes work out the gradients and put them into the
// token's row in LDS, zero otherwise, from where it leaves in runs of four.  DENSE (a softmax whose gates are not
// renormalised): every expert has one; C runs of four a lane.
constexpr int kBwdThreads = 256, kBwdWaves = kBwdThreads / 64;
template <int L, int C, typename TL, bool SOFTMAX, bool DENSE>
__global__ void __launch_bounds__(kBwdThreads) gate_bwd_kernel(GateBwdArgs a) {
  constexpr int kTokens = 64 / L;
  extern __shared__ float4 rows4[];
  const int tid = threadIdx.x, wl = tid & 63, lane = wl & (L - 1), slot = wl / L;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int N = a.N, K = a.K, quads = (N + 3) / 4;
  float4* row4 = rows4 + (wave * kTokens + slot) * quads;
  float* row = reinterpret_cast<float*>(row4);
  for (int q = lane; q < quads; q += L) row4[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const int64_t per_block = kBwdWaves * kTokens;
  for (int64_t t0 = (int64_t)blockIdx.x * per_block + wave * kTokens; t0 < a.T; t0 += (int64_t)gridDim.x * per_block) {
    const bool real = t0 + slot < a.T;
    const int64_t t = real ? t0 + slot : t0;
    const TL* lrow = static_cast<const TL*>(a.logits) + t * a.ld;
    TL* drow = static_cast<TL*>(a.d_logits) + t * a.d_ld;
    const int e = lane < K ? a.idx[t * K + lane] : -1;
    const bool ok = e >= 0 && e < N;
    const float dg = ok ? a.d_gate[t * K + lane] : 0.0f;
    float p[C][4];
    float dot = 0.0f;
    __builtin_amdgcn_wave_barrier();   // LDS operations of one wavefront take effect in program order
    if constexpr (DENSE) {
      float top = kNegInf;
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int first = 4 * (c * L + lane);
        load_run<4>(lrow + first, N - first, p[c]);
#pragma unroll
        for (int j = 0; j < 4; ++j) top = fmaxf(top, p[c][j]);
      }
      top = max_of<L>(top);
      if (top == kNegInf) top = 0.0f;
      float sum = 0.0f;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          p[c][j] = exp_of(p[c][j] - top);
          sum += p[c][j];
        }
      sum = sum_of<L>(sum);
      const float r = sum == 0.0f ? 0.0f : 1.0f / sum;
      if (ok) row[e] = dg;
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int c = 0; c < C; ++c) {
        const int q = c * L + lane;
        const float4 d = q < quads ? row4[q] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        const float dv[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          p[c][j] *= r;
          dot = fmaf(dv[j], p[c][j], dot);
        }
      }
      dot = sum_of<L>(dot);
    } else {
      const uint16_t* l16 = reinterpret_cast<const uint16_t*>(lrow);
      float l = kNegInf;
      if (ok) l = sizeof(TL) == 4 ? reinterpret_cast<const float*>(lrow)[e] : __uint_as_float((uint32_t)l16[e] << 16);
      float q, rest = 1.0f;   // the pick's share (or score), and 1 - s for the sigmoid
      if constexpr (SOFTMAX) {
        float top = max_of<L>(l);
        if (top == kNegInf) top = 0.0f;
        q = ok ? exp_of(l - top) : 0.0f;
      } else {
        const float x = exp_of(-fabsf(l));   // s and 1 - s without a difference of near values
        const float big = 1.0f / (1.0f + x), small = x * big;
        q = ok ? (l >= 0.0f ? big : small) : 0.0f;
        rest = l >= 0.0f ? small : big;
        if (l != l) q = rest = l;
      }
      float dl = dg;
      if (a.renorm) {
        const float sum = sum_of<L>(q);
        q = sum == 0.0f ? 0.0f : q / sum;
        dl -= sum_of<L>(dg * q);
      }
      if (ok) row[e] = a.scale * dl * q * rest;
      __builtin_amdgcn_wave_barrier();
    }
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int q = c * L + lane;
      if (q < quads) {
        const float4 d = row4[q];
        float o[4] = {d.x, d.y, d.z, d.w};
        if constexpr (DENSE) {
#pragma unroll
          for (int j = 0; j < 4; ++j) o[j] = a.scale * p[c][j] * (o[j] - dot);
        }
        if (real) store_run4(drow + 4 * q, N - 4 * q, o);
      }
    }
    __builtin_amdgcn_wave_barrier();
    if (ok) row[e] = 0.0f;
  }
}

// 16 lanes a token where they hold its experts (no group limit: that one wants the wavefront)
bool narrow(const moe_gate_config& c) { return c.n_routed <= 64 && c.topk_groups >= c.n_groups; }

template <typename TL, bool SOFTMAX>
hipError_t gate_forward_t(const GateArgs& a, bool few, int lanes_log2, unsigned grid, hipStream_t st) {
#define MOE_GATE_CASE(C, L) \
  hipLaunchKernelGGL((gate_kernel<C, L, TL, SOFTMAX>), dim3(grid), dim3(kThreads), 0, st, a, lanes_log2)
  if (few) {
    if (a.N <= 16) MOE_GATE_CASE(1, 16);
    else if (a.N <= 32) MOE_GATE_CASE(2, 16);
    else MOE_GATE_CASE(4, 16);
  } else if (a.N <= 64) {
    MOE_GATE_CASE(1, 64);
  } else if (a.N <= 128) {
    MOE_GATE_CASE(2, 64);
  } else if (a.N <= 256) {
    MOE_GATE_CASE(4, 64);
  } else {
    MOE_GATE_CASE(8, 64);
  }
#undef MOE_GATE_CASE
  return hipGetLastError();
}

template <int L, typename TL, bool SOFTMAX, bool DENSE>
hipError_t gate_backward_t(const GateBwdArgs& a, hipStream_t st) {
  const int64_t per_block = kBwdWaves * (64 / L);
  const unsigned grid = (unsigned)std::min<int64_t>(ceil_div(a.T, per_block), 4096);
  const size_t lds = (size_t)per_block * ((a.N + 3) / 4) * 16;   // at most 32 KB
#define MOE_GATE_CASE(C) \
  hipLaunchKernelGGL((gate_bwd_kernel<L, C, TL, SOFTMAX, DENSE>), dim3(grid), dim3(kBwdThreads), lds, st, a)
  if (a.N <= 4 * L) MOE_GATE_CASE(1);
  else if (a.N <= 8 * L) MOE_GATE_CASE(2);
  else if (a.N <= 16 * L) MOE_GATE_CASE(4);
  else MOE_GATE_CASE(8);
#undef MOE_GATE_CASE
  return hipGetLastError();
}

template <typename TL>
hipError_t gate_backward_l(const GateBwdArgs& a, bool softmax, hipStream_t st) {
  const bool dense = softmax && !a.renorm;
  if (a.K <= 16)
    return dense     ? gate_backward_t<16, TL, true, true>(a, st)
           : softmax ? gate_backward_t<16, TL, true, false>(a, st)
                     : gate_backward_t<16, TL, false, false>(a, st);
  return dense     ? gate_backward_t<32, TL, true, true>(a, st)
         : softmax ? gate_backward_t<32, TL, true, false>(a, st)
                   : gate_backward_t<32, TL, false, false>(a, st);
}

}  // namespace

int64_t gate_blocks(const moe_gate_config& c) {
  return std::min<int64_t>(ceil_div(c.tokens, narrow(c) ? 4 * kWaves : kWaves), 512);
}

hipError_t launch_gate(const moe_gate_config& c, const void* logits, const float* bias, int32_t* idx, float* gate,
                       int32_t* load, int32_t* counts, hipStream_t st) {
  if (c.tokens == 0) {
    if (!load) return hipSuccess;
    hipLaunchKernelGGL(gate_zero_kernel, dim3((unsigned)ceil_div(c.n_routed, 256)), dim3(256), 0, st, load, c.n_routed);
    return hipGetLastError();
  }
  const unsigned grid = (unsigned)gate_blocks(c);
  const GateArgs a{logits, c.logits_ld ? c.logits_ld : c.n_routed, bias, c.tokens, c.n_routed, c.top_k, c.n_groups,
                   c.topk_groups, c.group_score == MOE_GROUP_TOP2, c.renormalize != 0, c.scale, idx, gate,
                   load ? (grid == 1 ? load : counts) : nullptr};
  int lanes_log2 = 0;   // as many lanes per group as leave a set for every group
  while ((2 << lanes_log2) * c.n_groups <= 64) ++lanes_log2;
  const bool f32 = c.logits_dtype == MOE_DTYPE_F32, few = narrow(c);
  hipError_t err;
  if (c.score == MOE_SCORE_SOFTMAX)
    err = f32 ? gate_forward_t<float, true>(a, few, lanes_log2, grid, st)
              : gate_forward_t<uint16_t, true>(a, few, lanes_log2, grid, st);
  else
    err = f32 ? gate_forward_t<float, false>(a, few, lanes_log2, grid, st)
              : gate_forward_t<uint16_t, false>(a, few, lanes_log2, grid, st);
  if (err != hipSuccess || !load || grid == 1) return err;
  hipLaunchKernelGGL(gate_load_kernel, dim3((unsigned)ceil_div(c.n_routed, 64)), dim3(kThreads), 0, st, counts, (int)grid,
                     c.n_routed, load);
  return hipGetLastError();
}

hipError_t launch_gate_backward(const moe_gate_config& c, const void* logits, const int32_t* idx, const float* d_gate,
                                void* d_logits, int64_t d_ld, hipStream_t st) {
  if (c.tokens == 0) return hipSuccess;
  const GateBwdArgs a{logits, c.logits_ld ? c.logits_ld : c.n_routed, d_ld ? d_ld : c.n_routed, idx, d_gate, d_logits,
                      c.tokens, c.n_routed, c.top_k, c.renormalize != 0, c.scale};
  const bool softmax = c.score == MOE_SCORE_SOFTMAX;
  return c.logits_dtype == MOE_DTYPE_F32 ? gate_backward_l<float>(a, softmax, st) : gate_backward_l<uint16_t>(a, softmax, st);
}

}  // namespace moe
