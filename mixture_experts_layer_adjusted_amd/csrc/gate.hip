// Routing from given logits, and its gradient.
//
// For a token's logits l[0..N), a bias b (or none) and K picks:
//   s_i = 1 / (1 + exp(-l_i))   or   s_i = exp(l_i) / sum_j exp(l_j);
//   c_i = s_i + b_i ranks the experts; l_i = -inf or b_i = -inf takes expert i out;
//   (a softmax whose b_i are all 0, or -inf, ranks by l_i: the same order, which exp(l_i) below 2^-126 would lose)
//   with G groups of N / G neighbouring experts, only the TG groups with the largest score (the largest c,
//   or the sum of the two largest) stay; the K largest c left are the picks, equal ones by index;
//   g_k = scale s_k / sum of the picked s, or scale s_k.
// The gradient holds the picks fixed.  With q_k = s_k / sum of the picked s, and D = sum_k dg_k q_k:
//   sigmoid  renormalised   dl_k = scale (dg_k - D) q_k (1 - s_k);  plain  dl_k = scale dg_k s_k (1 - s_k)
//   softmax  renormalised   dl_k = scale (dg_k - D) q_k
//   softmax  plain          dl_i = scale p_i (dg_i [i picked] - sum_j dg_j p_j), every i
// and zero elsewhere.
//
// L lanes hold a token, CPL neighbouring experts each (one load of up to 64 bytes), in lists of four sorted by key: a
// round of the selection is the largest head over the lanes and one pop, and equal keys leave in index order (lowest
// lane, lowest list, stable sort).  What bounds it is instructions, not bytes (a 64-lane round costs 30 for one token, a
// 16-lane one 50 for four): T=16384, 256 experts in 8 groups: 15.5 us with 64 lanes, 9.8 with 16; T=32768, 64 experts:
// 16.6 and 6.2; one token of 256 experts 3.9 and 5.0.  Fewer lanes (8, 4) lose what they save in rounds to their longer
// runs.
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kWaves = 16;   // wavefronts of a workgroup at most
constexpr int kMaxBlocks = 512;
constexpr uint32_t kOut = 0u;       // key of an expert that is out (masked, in a closed group, or taken)
constexpr uint32_t kNanKey = 1u;    // a NaN ranks below every number
constexpr float kNegInf = -__builtin_inff();

// larger score, larger key (a score, a sum with a term that is no less than +0, is never -0)
__device__ __forceinline__ uint32_t key_of(float c) {
  const uint32_t b = __float_as_uint(c);
  const uint32_t k = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  return c != c ? kNanKey : k;
}
__device__ __forceinline__ float score_of(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key ^ 0x80000000u) : ~key);
}

// exp(x) from the 2^y instruction: y = x log2(e) rounded, and r = x - y ln(2) (ln(2) in two parts) as a factor 1 + r.
// Within 2 units in the last place; results below 2^-126 are 0, infinities and NaN as they should be.
__device__ __forceinline__ float exp_of(float x) {
  const float y = x * 1.44269502f;
  const float r = fmaf(y, 1.90465421e-9f, fmaf(y, -0.693147182f, x));
  const float e = __builtin_amdgcn_exp2f(y);
  return fabsf(x) < 150.0f ? fmaf(e, r, e) : e;   // (e may be infinite, and r NaN)
}

__device__ __forceinline__ float sigmoid_of(float l) { return __builtin_amdgcn_rcpf(1.0f + exp_of(-l)); }

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

// v from the lane that the DPP control names, where every lane has one (rotations, permutations)
template <int CTRL>
__device__ __forceinline__ uint32_t turned(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
}

// A reduction over the L lanes of a token, the result in each of them: neighbours first, then pairs of them and so on
// (quad_perm 1 0 3 2, quad_perm 2 3 0 1, row_half_mirror, row_mirror, the odd rows, the upper half).  With sum_run the
// order of a sum is that of its terms alone, however many lanes and registers they lie in.
template <int L, typename Op>
__device__ __forceinline__ uint32_t reduce(uint32_t v, Op op) {
  v = op(v, turned<0xB1>(v));
  v = op(v, turned<0x4E>(v));
  v = op(v, turned<0x141>(v));
  v = op(v, turned<0x140>(v));
  if constexpr (L >= 32) {
    const auto p = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = op(p[0], p[1]);
  }
  if constexpr (L >= 64) {
    const auto p = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = op(p[0], p[1]);
  }
  return v;
}
template <int L>
__device__ __forceinline__ uint32_t max_of(uint32_t v) {
  return reduce<L>(v, [](uint32_t a, uint32_t b) { return max(a, b); });
}
// (as integers of the same order: a float maximum would quiet each operand first.  A NaN is the largest or ignored: what
// uses the maximum of a row with one has no number anyway.)
template <int L>
__device__ __forceinline__ float max_of(float v) {
  const int32_t b = __float_as_int(v);
  const uint32_t m = reduce<L>((uint32_t)(b ^ ((b >> 31) & 0x7FFFFFFF)),
                               [](uint32_t a, uint32_t b) { return (uint32_t)max((int32_t)a, (int32_t)b); });
  const int32_t r = (int32_t)m;
  return __int_as_float(r ^ ((r >> 31) & 0x7FFFFFFF));
}
template <int L>
__device__ __forceinline__ float sum_of(float v) {
  return __uint_as_float(reduce<L>(__float_as_uint(v), [](uint32_t a, uint32_t b) {
    return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
  }));
}

// the sum of a lane's run, in the order of `reduce`
template <int N>
__device__ __forceinline__ float sum_run(const float (&v)[N]) {
  float s[N];
#pragma unroll
  for (int j = 0; j < N; ++j) s[j] = v[j];
#pragma unroll
  for (int w = 1; w < N; w *= 2)
#pragma unroll
    for (int j = 0; j < N; j += 2 * w) s[j] += s[j + w];
  return s[0];
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
// leave a lane set for every group), each on every 2^p-th expert; their two largest join by shuffles.
// score_pair: the key of a group's score from those of its two largest, where both count.
template <typename Score>
__device__ __forceinline__ uint64_t open_groups(const uint32_t* keys, const GateArgs& a, int lane, int lanes_log2,
                                                Score score_pair) {
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
  const uint32_t score = a.top2 ? score_pair(k1, k2) : k1;
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

// Whether the lane's group stays open, groups being `per` whole lanes: the lanes' two largest join over the group, and
// the group's rank counts the groups above it, or equal to it and before it.  Scores as in open_groups.
template <int L, typename Score>
__device__ __forceinline__ bool group_open(uint32_t k1, uint32_t k2, const GateArgs& a, int lane, int per,
                                           Score score_pair) {
  auto join = [&](uint32_t o1, uint32_t o2) {
    k2 = max(max(k2, o2), min(k1, o1));
    k1 = max(k1, o1);
  };
  if (per >= 2) join(turned<0xB1>(k1), turned<0xB1>(k2));       // quad_perm: lanes 1 0 3 2
  if (per >= 4) join(turned<0x4E>(k1), turned<0x4E>(k2));       // lanes 2 3 0 1
  if (per >= 8) join(turned<0x141>(k1), turned<0x141>(k2));     // row_half_mirror
  if (per >= 16) join(turned<0x140>(k1), turned<0x140>(k2));    // row_mirror
  if (L >= 32 && per >= 32) join(__shfl_xor(k1, 16, 64), __shfl_xor(k2, 16, 64));
  if (L >= 64 && per >= 64) join(__shfl_xor(k1, 32, 64), __shfl_xor(k2, 32, 64));
  const uint32_t score = a.top2 ? score_pair(k1, k2) : k1;
  const int g = lane / per;
  int rank = 0;
  for (int h = 0; h < a.G; ++h) {
    const uint32_t o = (uint32_t)__shfl((int)score, h * per, L);
    rank += (o > score || (o == score && h < g)) ? 1 : 0;
  }
  return rank < a.TG;
}

// `per`: lanes of a group where groups are whole lanes (0: they are not; 64 lanes only)
template <int CPL, int L, typename TL, bool SOFTMAX>
__global__ void __launch_bounds__(kWaves * 64) gate_kernel(GateArgs a, int per, int lanes_log2) {
  constexpr int kTokens = 64 / L;                    // tokens of a wavefront
  constexpr int kLists = (CPL + 3) / 4, kLen = CPL < 4 ? CPL : 4;
  __shared__ int32_t hist[kMaxRouted];
  __shared__ uint32_t keys[L == 64 ? kWaves : 1][kMaxRouted];
  __shared__ int32_t won[kWaves][kTokens][kMaxTopK];
  const int tid = threadIdx.x, wl = tid & 63, lane = wl & (L - 1), slot = wl / L;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int N = a.N, K = a.K;
  const int threads = blockDim.x;
  for (int e = tid; e < N; e += threads) hist[e] = 0;
  const bool limited = a.TG < a.G;
  const int first = lane * CPL, left = N - first;
  float bias[CPL];   // -inf past the last expert
  if (a.bias) {
    load_run<CPL>(a.bias + first, left, bias);
  } else {
#pragma unroll
    for (int j = 0; j < CPL; ++j) bias[j] = j < left ? 0.0f : kNegInf;
  }
  __syncthreads();
  const int64_t per_block = threads / L;
  for (int64_t t0 = (int64_t)blockIdx.x * per_block + wave * kTokens; t0 < a.T; t0 += (int64_t)gridDim.x * per_block) {
    const bool real = t0 + slot < a.T;   // (several tokens a wavefront: the last one may have fewer)
    const int64_t t = real ? t0 + slot : t0;
    const TL* row = static_cast<const TL*>(a.logits) + t * a.ld;
    uint32_t key[kLists][4];
    uint32_t order[kLists];              // which expert of the lane each entry is, a byte each
    float total = 0.0f, top = 0.0f;      // softmax: the row's sum and maximum
    float l[CPL];
    load_run<CPL>(row + first, left, l);
    bool by_logit = false;
    {
      float s[CPL];
      if constexpr (SOFTMAX) {
        top = l[0];
#pragma unroll
        for (int j = 1; j < CPL; ++j) top = fmaxf(top, l[j]);
        top = max_of<L>(top);
        if (top == kNegInf) top = 0.0f;
#pragma unroll
        for (int j = 0; j < CPL; ++j) s[j] = exp_of(l[j] - top);
        total = sum_of<L>(sum_run<CPL>(s));
        total = total == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(total);   // (1 ulp) 0: every expert masked
      } else {
#pragma unroll
        for (int j = 0; j < CPL; ++j) s[j] = sigmoid_of(l[j]);
      }
      // the biases, from here on unknown to the compiler: it would wait for them before the logits are asked for, and keep
      // a mask for each of their comparisons
#pragma unroll
      for (int j = 0; j < CPL; ++j) asm volatile("" : "+v"(bias[j]));
      float factor = 1.0f;   // of what ranks the experts: the scores before their division by the sum, or the logits
      if constexpr (SOFTMAX) {
        bool none = true;
#pragma unroll
        for (int j = 0; j < CPL; ++j) none = none && __builtin_amdgcn_classf(bias[j], 0x044);   // +0 or -inf: then no key is -0
        by_logit = __builtin_amdgcn_ballot_w64(!none) == 0;   // (a wavefront sees all the biases)
        factor = by_logit ? fmaf(total, 0.0f, 1.0f) : total;   // (a row without a number has none of either)
      }
#pragma unroll
      for (int q = 0; q < kLists; ++q)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j >= kLen) {
            key[q][j] = kOut;
            continue;
          }
          const int i = 4 * q + j;
          const float c = SOFTMAX ? fmaf(by_logit ? l[i] : s[i], factor, bias[i]) : s[i] + bias[i];
          const uint32_t k = key_of(c);
          key[q][j] = l[i] == kNegInf || bias[i] == kNegInf ? kOut : k;   // (not by c: a NaN score's is a NaN)
        }
    }
    // The key of a group's score, the sum of its two largest.  It counts numbers only: a NaN or an absent second adds
    // nothing.  By logits, of exp(l1 - top) + exp(l2 - top) the logarithm.
    auto score_pair = [&](uint32_t k1, uint32_t k2) {
      if (SOFTMAX && by_logit) {
        const float l1 = score_of(k1), x = k2 > kNanKey ? exp_of(score_of(k2) - l1) : 0.0f;
        return k1 > kNanKey ? key_of(fmaf(__builtin_amdgcn_logf(1.0f + x), 0.693147182f, l1 - top)) : k1;
      }
      return k2 > kNanKey ? key_of(score_of(k1) + score_of(k2)) : k1;
    };
    if (limited && per == 0) {
      if constexpr (L == 64) {
#pragma unroll
        for (int j = 0; j < CPL; ++j)
          if (j < left) keys[wave][first + j] = key[j / 4][j % 4];
        __builtin_amdgcn_wave_barrier();   // LDS operations of one wavefront take effect in program order
        const uint64_t open = open_groups(keys[wave], a, lane, lanes_log2, score_pair);
        __builtin_amdgcn_wave_barrier();
        const float inv = (float)a.G / (float)N;   // (small integers: half a step in, the quotient is exact enough)
#pragma unroll
        for (int j = 0; j < CPL; ++j)
          if (!((open >> (int)(((float)(first + j) + 0.5f) * inv)) & 1ull)) key[j / 4][j % 4] = kOut;
      }
    }
    // each list in descending order, equal keys as they stand: an entry's place is the number of larger ones, and of
    // equal ones before it
#pragma unroll
    for (int q = 0; q < kLists; ++q) {
      uint32_t(&k)[4] = key[q];
      if constexpr (kLen == 4) {
        const uint32_t c01 = k[1] > k[0] ? 8 : 0, c02 = k[2] > k[0] ? 8 : 0, c03 = k[3] > k[0] ? 8 : 0;
        const uint32_t c12 = k[2] > k[1] ? 8 : 0, c13 = k[3] > k[1] ? 8 : 0, c23 = k[3] > k[2] ? 8 : 0;
        order[q] = (1u << (8 - c01 + c12 + c13)) + (2u << (16 - c02 - c12 + c23)) + (3u << (24 - c03 - c13 - c23)) +
                   4u * q * 0x01010101u;
        const uint32_t hi0 = max(k[0], k[1]), lo0 = min(k[0], k[1]), hi1 = max(k[2], k[3]), lo1 = min(k[2], k[3]);
        k[0] = max(hi0, hi1), k[3] = min(lo0, lo1);
        const uint32_t x = min(hi0, hi1), y = max(lo0, lo1);
        k[1] = max(x, y), k[2] = min(x, y);
      } else if constexpr (kLen == 2) {
        order[q] = k[1] > k[0] ? 0x0001u : 0x0100u;
        const uint32_t hi = max(k[0], k[1]);
        k[1] = min(k[0], k[1]), k[0] = hi;
      } else {
        order[q] = 0;
      }
    }
    if (limited && per > 0) {
      uint32_t k1 = kOut, k2 = kOut;
#pragma unroll
      for (int q = 0; q < kLists; ++q) {
        k2 = max(max(k2, kLen > 1 ? key[q][1] : kOut), min(k1, key[q][0]));
        k1 = max(k1, key[q][0]);
      }
      if (!group_open<L>(k1, k2, a, lane, per, score_pair)) {
#pragma unroll
        for (int q = 0; q < kLists; ++q)
#pragma unroll
          for (int j = 0; j < kLen; ++j) key[q][j] = kOut;
      }
    }
    for (int k = lane; k < K; k += L) won[wave][slot][k] = -1;
    __builtin_amdgcn_wave_barrier();
    for (int k = 0; k < K; ++k) {
      uint32_t head = key[0][0];
#pragma unroll
      for (int q = 1; q < kLists; ++q) head = max(head, key[q][0]);
      const uint32_t best = max_of<L>(head);
      // of the lanes that have it the token's lowest: the lowest set bit in each L bits (a field with its top bit set
      // less one, without a borrow from the next)
      const uint64_t at = __builtin_amdgcn_ballot_w64(head == best) & __builtin_amdgcn_ballot_w64(best != kOut);
      constexpr uint64_t kLow = L == 16 ? 0x0001000100010001ull : L == 32 ? 0x0000000100000001ull : 1ull;
      const uint64_t lowest = at & ~((at | kLow << (L - 1)) - kLow);
      if (__builtin_amdgcn_inverse_ballot_w64(lowest)) {   // the first list whose head it is
        bool found = false;
        uint32_t j = 0;
#pragma unroll
        for (int q = 0; q < kLists; ++q) {
          const bool here = !found && (q == kLists - 1 || key[q][0] == best);
          found = found || here;
          j = here ? order[q] & 0xFFu : j;
          order[q] = here ? order[q] >> 8 : order[q];
#pragma unroll
          for (int i = 0; i < kLen; ++i) key[q][i] = here ? (i + 1 < kLen ? key[q][i + 1] : kOut) : key[q][i];
        }
        won[wave][slot][k] = first + (int)j;
      }
    }
    __builtin_amdgcn_wave_barrier();
    // the picks' gates, from their logits again
    constexpr int kHalves = L == 16 ? 2 : 1;   // 16 lanes hold up to 32 picks
    const int halves = kHalves == 2 && K > L ? 2 : 1;
    float g[kHalves], v[kHalves];
    int e[kHalves];
    float most = kNegInf;
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      e[h] = -1;
      v[h] = kNegInf;
      g[h] = 0.0f;
      if (h >= halves) continue;
      if (lane + L * h < K) e[h] = won[wave][slot][lane + L * h];
      if constexpr (L == 64 && CPL <= 4) {   // from the lane that has it: sooner, though more instructions
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
          const float o = __shfl(l[j], max(e[h], 0) / CPL, L);
          if (e[h] >= 0 && e[h] % CPL == j) v[h] = o;
        }
      } else {
        if (e[h] >= 0) load_run<1>(row + e[h], 1, reinterpret_cast<float(&)[1]>(v[h]));
      }
      most = fmaxf(most, v[h]);
    }
    if (SOFTMAX && a.renorm) {   // over the picks alone, so that no picked score has underflowed
      most = max_of<L>(most);
      if (most == kNegInf) most = 0.0f;
    }
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      if (h >= halves) continue;
      if constexpr (SOFTMAX) {   // (total is NaN where a NaN or an infinity leaves the row without a number)
        g[h] = exp_of(v[h] - (a.renorm ? most : top));
        g[h] = a.renorm ? (total != total ? total : g[h]) : g[h] * total;
      } else {
        g[h] = sigmoid_of(v[h]);
      }
      if (e[h] < 0) g[h] = 0.0f;
    }
    if (a.renorm) {   // (picks are 32 at most: two runs of 16 lanes, or one of 32)
      float sum = sum_of<kHalves == 2 ? 16 : 32>(g[0]);
      if (halves == 2) sum += sum_of<16>(g[kHalves - 1]);
#pragma unroll
      for (int h = 0; h < kHalves; ++h)
        if (h < halves) g[h] = sum == 0.0f ? 0.0f : g[h] / sum;
    }
#pragma unroll
    for (int h = 0; h < kHalves; ++h)
      if (h < halves && real && lane + L * h < K) {
        a.idx[t * K + lane + L * h] = e[h];
        a.gate[t * K + lane + L * h] = e[h] >= 0 ? a.scale * g[h] : 0.0f;   // (an empty place's share of a NaN sum is one)
        if (e[h] >= 0) atomicAdd(&hist[e[h]], 1);
      }
    __builtin_amdgcn_wave_barrier();
  }
  if (!a.counts) return;
  __syncthreads();
  for (int e = tid; e < N; e += threads) a.counts[(int64_t)blockIdx.x * N + e] = hist[e];
}

// load[e] = sum over the workgroups of counts[w, e]: 64 experts per workgroup, its wavefronts every 16th row
__global__ void __launch_bounds__(kWaves * 64) gate_load_kernel(const int32_t* __restrict__ counts, int rows, int N,
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
// renormalised): every expert has one; C runs of four a lane.  Bound by memory: T=16384, 256 experts, 6.4 to
// 7.9 us for 26 MB, dense 7.8 us for 35 MB.
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

// How a call's tokens lie on lanes: 16 lanes a token (32 above 256 experts), or 64 for groups that do not fall on a power
// of two of whole lanes, and for up to four tokens, where a token's own time counts (one token, 256 experts: 3.9 us
// against 5.0).  Sums do not depend on it, so a token's gates are the same in every batch.  Workgroups are small while
// kMaxBlocks of them hold every token, and so reach more CUs (T=4096, 256 experts: 8.8 us against 12.6).
struct GateLanes {
  int lanes, cpl;
  int per;     // lanes of a group, 0 where groups are not whole lanes
  int waves;   // of a workgroup
};
GateLanes lanes_of(const moe_gate_config& c) {
  auto with = [&](int lanes) {
    GateLanes g{lanes, 1, 0, 4};
    while (g.cpl * lanes < c.n_routed) g.cpl *= 2;
    const int gs = c.n_routed / c.n_groups;
    const int per = gs % g.cpl == 0 ? gs / g.cpl : 0;
    if (per > 0 && (per & (per - 1)) == 0) g.per = per;
    if (c.tokens > kMaxBlocks * 4 * (64 / lanes)) g.waves = kWaves;
    return g;
  };
  if (c.tokens <= 4 && c.n_routed > 64) return with(64);
  const GateLanes few = with(c.n_routed <= 256 ? 16 : 32);
  const bool limited = c.topk_groups < c.n_groups;
  return !limited || few.per > 0 ? few : with(64);
}

template <typename TL, bool SOFTMAX>
hipError_t gate_forward_t(const GateArgs& a, const GateLanes& g, int lanes_log2, unsigned grid, hipStream_t st) {
#define MOE_GATE_CASE(C, L)                                                                                            \
  case L * 100 + C:                                                                                                    \
    return launch_kernel(gate_kernel<C, L, TL, SOFTMAX>, dim3(grid), dim3(g.waves * 64), 0, st, a, g.per, lanes_log2)
  switch (g.lanes * 100 + g.cpl) {
    MOE_GATE_CASE(1, 16);
    MOE_GATE_CASE(2, 16);
    MOE_GATE_CASE(4, 16);
    MOE_GATE_CASE(8, 16);
    MOE_GATE_CASE(16, 16);
    MOE_GATE_CASE(16, 32);
    MOE_GATE_CASE(1, 64);
    MOE_GATE_CASE(2, 64);
    MOE_GATE_CASE(4, 64);
    MOE_GATE_CASE(8, 64);
  }
#undef MOE_GATE_CASE
  return hipErrorInvalidValue;
}

template <int L, typename TL, bool SOFTMAX, bool DENSE>
hipError_t gate_backward_t(const GateBwdArgs& a, hipStream_t st) {
  const int64_t per_block = kBwdWaves * (64 / L);
  const unsigned grid = (unsigned)std::min<int64_t>(ceil_div(a.T, per_block), 4096);
  const size_t lds = (size_t)per_block * ((a.N + 3) / 4) * 16;   // at most 32 KB
#define MOE_GATE_CASE(C) \
  return launch_kernel(gate_bwd_kernel<L, C, TL, SOFTMAX, DENSE>, dim3(grid), dim3(kBwdThreads), lds, st, a)
  if (a.N <= 4 * L) MOE_GATE_CASE(1);
  if (a.N <= 8 * L) MOE_GATE_CASE(2);
  if (L == 32 || a.N <= 16 * L) MOE_GATE_CASE(4);   // (512 experts at most)
  if constexpr (L == 16) MOE_GATE_CASE(8);
#undef MOE_GATE_CASE
  return hipErrorInvalidValue;
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
  const GateLanes g = lanes_of(c);
  return std::min<int64_t>(ceil_div(c.tokens, g.waves * (64 / g.lanes)), kMaxBlocks);
}

hipError_t launch_gate(const moe_gate_config& c, const void* logits, const float* bias, int32_t* idx, float* gate,
                       int32_t* load, int32_t* counts, hipStream_t st) {
  if (c.tokens == 0) {
    if (!load) return hipSuccess;
    return launch_kernel(gate_zero_kernel, dim3((unsigned)ceil_div(c.n_routed, 256)), dim3(256), 0, st, load, c.n_routed);
  }
  const unsigned grid = (unsigned)gate_blocks(c);
  const GateArgs a{logits, c.logits_ld ? c.logits_ld : c.n_routed, bias, c.tokens, c.n_routed, c.top_k, c.n_groups,
                   c.topk_groups, c.group_score == MOE_GROUP_TOP2, c.renormalize != 0, c.scale, idx, gate,
                   load ? (grid == 1 ? load : counts) : nullptr};
  int lanes_log2 = 0;   // as many lanes per group as leave a set for every group
  while ((2 << lanes_log2) * c.n_groups <= 64) ++lanes_log2;
  const bool f32 = c.logits_dtype == MOE_DTYPE_F32;
  const GateLanes g = lanes_of(c);
  hipError_t err;
  if (c.score == MOE_SCORE_SOFTMAX)
    err = f32 ? gate_forward_t<float, true>(a, g, lanes_log2, grid, st)
              : gate_forward_t<uint16_t, true>(a, g, lanes_log2, grid, st);
  else
    err = f32 ? gate_forward_t<float, false>(a, g, lanes_log2, grid, st)
              : gate_forward_t<uint16_t, false>(a, g, lanes_log2, grid, st);
  if (err != hipSuccess || !load || grid == 1) return err;
  return launch_kernel(gate_load_kernel, dim3((unsigned)ceil_div(c.n_routed, 64)), dim3(kWaves * 64), 0, st, counts, (int)grid,
                     c.n_routed, load);
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
