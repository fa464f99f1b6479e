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
// One wavefront holds one token: lane i has the experts i, i + 64, ...
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 1024;
constexpr int kWaves = kThreads / 64;
constexpr uint32_t kOut = 0u;       // key of an expert that is out (masked, in a closed group, or taken)
constexpr uint32_t kNanKey = 1u;    // a NaN ranks below every number
constexpr float kNegInf = -__builtin_inff();

__device__ __forceinline__ float load_logit(const float* p) { return *p; }
__device__ __forceinline__ float load_logit(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(uint16_t* p, float v) {
  const uint32_t b = __float_as_uint(v);
  *p = v != v ? (uint16_t)0x7FC0u : (uint16_t)((b + 0x7FFFu + ((b >> 16) & 1u)) >> 16);
}

// larger score, larger key; -0 and +0 are one score
__device__ __forceinline__ uint32_t key_of(float c) {
  if (c != c) return kNanKey;
  const uint32_t b = __float_as_uint(c + 0.0f);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}
__device__ __forceinline__ float score_of(uint32_t key) {
  return __uint_as_float((key & 0x80000000u) ? (key ^ 0x80000000u) : ~key);
}

// v from the lane that the DPP control names; lanes without one, or outside row_mask, get `other`
template <int CTRL, int ROW_MASK>
__device__ __forceinline__ uint32_t moved(uint32_t other, uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)other, (int)v, CTRL, ROW_MASK, 0xF, false);
}

// Over the 64 lanes, the same value in each lane: row shifts by 1, 2, 4, 8, then row 0's result into row 1
// and row 2's into row 3 (row_bcast:15), and lane 31's into the upper rows (row_bcast:31); lane 63 has all.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, moved<0x111, 0xF>(v, v));
  v = max(v, moved<0x112, 0xF>(v, v));
  v = max(v, moved<0x114, 0xF>(v, v));
  v = max(v, moved<0x118, 0xF>(v, v));
  v = max(v, moved<0x142, 0xA>(v, v));
  v = max(v, moved<0x143, 0xC>(v, v));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}
__device__ __forceinline__ float wave_fmax(float v) {
  auto step = [&](uint32_t m) { v = fmaxf(v, __uint_as_float(m)); };
  step(moved<0x111, 0xF>(__float_as_uint(v), __float_as_uint(v)));
  step(moved<0x112, 0xF>(__float_as_uint(v), __float_as_uint(v)));
  step(moved<0x114, 0xF>(__float_as_uint(v), __float_as_uint(v)));
  step(moved<0x118, 0xF>(__float_as_uint(v), __float_as_uint(v)));
  step(moved<0x142, 0xA>(__float_as_uint(v), __float_as_uint(v)));
  step(moved<0x143, 0xC>(__float_as_uint(v), __float_as_uint(v)));
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ float wave_sum(float v) {
  auto step = [&](uint32_t m) { v += __uint_as_float(m); };
  step(moved<0x111, 0xF>(0u, __float_as_uint(v)));
  step(moved<0x112, 0xF>(0u, __float_as_uint(v)));
  step(moved<0x114, 0xF>(0u, __float_as_uint(v)));
  step(moved<0x118, 0xF>(0u, __float_as_uint(v)));
  step(moved<0x142, 0xA>(0u, __float_as_uint(v)));
  step(moved<0x143, 0xC>(0u, __float_as_uint(v)));
  return __uint_as_float((uint32_t)__builtin_amdgcn_readlane(__float_as_int(v), 63));
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
  uint64_t first = __ballot(g < a.G && rank < a.TG);
  uint64_t open = 0;
  for (int h = 0; h < a.G; ++h) open |= ((first >> (h << lanes_log2)) & 1ull) << h;
  return open;
}

template <int CPL, typename TL, bool SOFTMAX>
__global__ void __launch_bounds__(kThreads) gate_kernel(GateArgs a, int lanes_log2) {
  __shared__ int32_t hist[kMaxRouted];
  __shared__ uint32_t keys[kWaves][kMaxRouted];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int N = a.N, K = a.K;
  for (int e = tid; e < N; e += kThreads) hist[e] = 0;
  const bool limited = a.TG < a.G;
  float bias[CPL];
  int group[CPL];
#pragma unroll
  for (int j = 0; j < CPL; ++j) {
    const int e = lane + 64 * j;
    bias[j] = e < N ? (a.bias ? a.bias[e] : 0.0f) : kNegInf;
    group[j] = e < N ? e / (N / a.G) : 0;
  }
  __syncthreads();
  for (int64_t t = (int64_t)blockIdx.x * kWaves + wave; t < a.T; t += (int64_t)gridDim.x * kWaves) {
    const TL* row = static_cast<const TL*>(a.logits) + t * a.ld;
    float l[CPL], s[CPL];
    uint32_t key[CPL];
#pragma unroll
    for (int j = 0; j < CPL; ++j) l[j] = lane + 64 * j < N ? load_logit(row + lane + 64 * j) : kNegInf;
    if constexpr (SOFTMAX) {
      float top = l[0];
#pragma unroll
      for (int j = 1; j < CPL; ++j) top = fmaxf(top, l[j]);
      top = wave_fmax(top);
      if (top == kNegInf) top = 0.0f;
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < CPL; ++j) {
        s[j] = expf(l[j] - top);
        sum += s[j];
      }
      sum = wave_sum(sum);
      if (sum == 0.0f) sum = 1.0f;   // every expert masked
#pragma unroll
      for (int j = 0; j < CPL; ++j) s[j] = s[j] / sum;
    } else {
#pragma unroll
      for (int j = 0; j < CPL; ++j) s[j] = 1.0f / (1.0f + expf(-l[j]));
    }
#pragma unroll
    for (int j = 0; j < CPL; ++j)
      key[j] = (l[j] == kNegInf || bias[j] == kNegInf) ? kOut : key_of(s[j] + bias[j]);
    if (limited) {
#pragma unroll
      for (int j = 0; j < CPL; ++j)
        if (lane + 64 * j < N) keys[wave][lane + 64 * j] = key[j];
      __builtin_amdgcn_wave_barrier();   // LDS operations of one wavefront take effect in program order
      const uint64_t open = open_groups(keys[wave], a, lane, lanes_log2);
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int j = 0; j < CPL; ++j)
        if (!((open >> group[j]) & 1ull)) key[j] = kOut;
    }
    // K rounds: the largest key of the wavefront, then the first expert that has it
    int my_idx = -1;
    float my_s = 0.0f, my_l = kNegInf;
    for (int k = 0; k < K; ++k) {
      uint32_t best = key[0];
#pragma unroll
      for (int j = 1; j < CPL; ++j) best = max(best, key[j]);
      best = wave_max(best);
      if (best == kOut) break;
      bool found = false;
#pragma unroll
      for (int j = 0; j < CPL; ++j) {
        if (!found) {
          const uint64_t at = __ballot(key[j] == best);
          if (at) {
            found = true;
            const int owner = __builtin_ctzll(at);
            if (lane == owner) key[j] = kOut;
            const float sw = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(s[j]), owner));
            const float lw = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(l[j]), owner));
            if (lane == k) {
              my_idx = owner + 64 * j;
              my_s = sw;
              my_l = lw;
            }
          }
        }
      }
    }
    float g = my_s;
    if (a.renorm) {
      if constexpr (SOFTMAX) {   // from the picked logits, so that no picked score has underflowed
        float top = wave_fmax(my_l);
        if (top == kNegInf) top = 0.0f;
        g = my_idx < 0 ? 0.0f : my_s != my_s ? my_s : expf(my_l - top);
      }
      const float sum = wave_sum(g);
      g = sum == 0.0f ? 0.0f : g / sum;
    }
    if (lane < K) {
      a.idx[t * K + lane] = my_idx;
      a.gate[t * K + lane] = a.scale * g;
      if (my_idx >= 0) atomicAdd(&hist[my_idx], 1);
    }
  }
  if (!a.counts) return;
  __syncthreads();
  for (int e = tid; e < N; e += kThreads) a.counts[(int64_t)blockIdx.x * N + e] = hist[e];
}

// load[e] = sum over the workgroups of counts[w, e]: 64 experts per workgroup, 16 runs of rows
__global__ void __launch_bounds__(kThreads) gate_load_kernel(const int32_t* __restrict__ counts, int rows, int N,
                                                             int32_t* __restrict__ load) {
  __shared__ int32_t part[kWaves][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int e = blockIdx.x * 64 + lane;
  int c = 0;
  if (e < N) {
#pragma unroll 8
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

template <int CPL, typename TL, bool SOFTMAX>
__global__ void __launch_bounds__(kThreads) gate_bwd_kernel(GateBwdArgs a) {
  __shared__ float rows[kWaves][kMaxRouted];   // per wavefront: one row, zero but where the picks write
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int N = a.N, K = a.K;
  float* row = rows[wave];
#pragma unroll
  for (int j = 0; j < CPL; ++j)
    if (lane + 64 * j < N) row[lane + 64 * j] = 0.0f;
  for (int64_t t = (int64_t)blockIdx.x * kWaves + wave; t < a.T; t += (int64_t)gridDim.x * kWaves) {
    const TL* lrow = static_cast<const TL*>(a.logits) + t * a.ld;
    TL* drow = static_cast<TL*>(a.d_logits) + t * a.d_ld;
    const int e = lane < K ? a.idx[t * K + lane] : -1;
    const bool ok = e >= 0 && e < N;
    const float dg = ok ? a.d_gate[t * K + lane] : 0.0f;
    float out[CPL];
    if (SOFTMAX && !a.renorm) {
      float p[CPL];
      float top = kNegInf;
#pragma unroll
      for (int j = 0; j < CPL; ++j) {
        p[j] = lane + 64 * j < N ? load_logit(lrow + lane + 64 * j) : kNegInf;
        top = fmaxf(top, p[j]);
      }
      top = wave_fmax(top);
      if (top == kNegInf) top = 0.0f;
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < CPL; ++j) {
        p[j] = expf(p[j] - top);
        sum += p[j];
      }
      sum = wave_sum(sum);
      if (sum == 0.0f) sum = 1.0f;
      if (ok) row[e] = dg;
      __builtin_amdgcn_wave_barrier();
      float dot = 0.0f;
#pragma unroll
      for (int j = 0; j < CPL; ++j) {
        p[j] = p[j] / sum;
        out[j] = lane + 64 * j < N ? row[lane + 64 * j] : 0.0f;
        dot = fmaf(out[j], p[j], dot);
      }
      dot = wave_sum(dot);
#pragma unroll
      for (int j = 0; j < CPL; ++j) out[j] = a.scale * p[j] * (out[j] - dot);
    } else {
      const float l = ok ? load_logit(lrow + e) : kNegInf;
      float q, rest = 1.0f;   // the pick's share (or score), and 1 - s for the sigmoid
      if constexpr (SOFTMAX) {
        float top = wave_fmax(l);
        if (top == kNegInf) top = 0.0f;
        q = ok ? expf(l - top) : 0.0f;
      } else {
        const float x = expf(-fabsf(l));   // s and 1 - s without a difference of near values
        const float big = 1.0f / (1.0f + x), small = x * big;
        q = ok ? (l >= 0.0f ? big : small) : 0.0f;
        rest = l >= 0.0f ? small : big;
        if (l != l) q = rest = l;
      }
      float dl = dg;
      if (a.renorm) {
        const float sum = wave_sum(q);
        q = sum == 0.0f ? 0.0f : q / sum;
        dl -= wave_sum(dg * q);
      }
      dl = a.scale * dl * q * rest;
      if (ok) row[e] = dl;
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int j = 0; j < CPL; ++j) out[j] = lane + 64 * j < N ? row[lane + 64 * j] : 0.0f;
    }
    __builtin_amdgcn_wave_barrier();
    if (ok) row[e] = 0.0f;
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int j = 0; j < CPL; ++j)
      if (lane + 64 * j < N) store_logit(drow + lane + 64 * j, out[j]);
  }
}

template <typename TL, bool SOFTMAX>
hipError_t gate_forward_t(const GateArgs& a, int lanes_log2, unsigned grid, hipStream_t st) {
#define MOE_GATE_CASE(C) hipLaunchKernelGGL((gate_kernel<C, TL, SOFTMAX>), dim3(grid), dim3(kThreads), 0, st, a, lanes_log2)
  if (a.N <= 64) MOE_GATE_CASE(1);
  else if (a.N <= 128) MOE_GATE_CASE(2);
  else if (a.N <= 256) MOE_GATE_CASE(4);
  else MOE_GATE_CASE(8);
#undef MOE_GATE_CASE
  return hipGetLastError();
}

template <typename TL, bool SOFTMAX>
hipError_t gate_backward_t(const GateBwdArgs& a, unsigned grid, hipStream_t st) {
#define MOE_GATE_CASE(C) hipLaunchKernelGGL((gate_bwd_kernel<C, TL, SOFTMAX>), dim3(grid), dim3(kThreads), 0, st, a)
  if (a.N <= 64) MOE_GATE_CASE(1);
  else if (a.N <= 128) MOE_GATE_CASE(2);
  else if (a.N <= 256) MOE_GATE_CASE(4);
  else MOE_GATE_CASE(8);
#undef MOE_GATE_CASE
  return hipGetLastError();
}

}  // namespace

int64_t gate_blocks(const moe_gate_config& c) {
  return std::min<int64_t>(ceil_div(c.tokens, kWaves), 512);
}

hipError_t launch_gate(const moe_gate_config& c, const void* logits, const float* bias, int32_t* idx, float* gate,
                       int32_t* load, int32_t* counts, hipStream_t st) {
  if (c.tokens == 0) {
    if (load) {
      hipLaunchKernelGGL(gate_zero_kernel, dim3((unsigned)ceil_div(c.n_routed, 256)), dim3(256), 0, st, load, c.n_routed);
      return hipGetLastError();
    }
    return hipSuccess;
  }
  const unsigned grid = (unsigned)gate_blocks(c);
  const GateArgs a{logits, c.logits_ld ? c.logits_ld : c.n_routed, bias, c.tokens, c.n_routed, c.top_k, c.n_groups,
                   c.topk_groups, c.group_score == MOE_GROUP_TOP2, c.renormalize != 0, c.scale, idx, gate,
                   load ? (grid == 1 ? load : counts) : nullptr};
  int lanes_log2 = 0;   // as many lanes per group as leave a set for every group
  while ((2 << lanes_log2) * c.n_groups <= 64) ++lanes_log2;
  const bool f32 = c.logits_dtype == MOE_DTYPE_F32;
  hipError_t err;
  if (c.score == MOE_SCORE_SOFTMAX)
    err = f32 ? gate_forward_t<float, true>(a, lanes_log2, grid, st) : gate_forward_t<uint16_t, true>(a, lanes_log2, grid, st);
  else
    err = f32 ? gate_forward_t<float, false>(a, lanes_log2, grid, st) : gate_forward_t<uint16_t, false>(a, lanes_log2, grid, st);
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
  const unsigned grid = (unsigned)std::min<int64_t>(ceil_div(c.tokens, kWaves), 1024);
  const bool f32 = c.logits_dtype == MOE_DTYPE_F32;
  if (c.score == MOE_SCORE_SOFTMAX)
    return f32 ? gate_backward_t<float, true>(a, grid, st) : gate_backward_t<uint16_t, true>(a, grid, st);
  return f32 ? gate_backward_t<float, false>(a, grid, st) : gate_backward_t<uint16_t, false>(a, grid, st);
}

}  // namespace moe
