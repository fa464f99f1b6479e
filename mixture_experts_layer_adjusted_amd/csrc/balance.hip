// The balance loss of a router, from its logits and picks, and its gradient.
//
// For a sequence of tokens, N experts, K picks a token (entries outside [0, N) are no picks; a token without one is
// padding and counts nowhere):
//   p_t = softmax(l_t), or s_t / sum s_t with s = 1 / (1 + exp(-l));
//   n_i = picks of expert i, L = the sequence's tokens;  f_i = N n_i / (K L),  P_i = sum_t p_{t,i} / L;
//   loss = alpha sum_i f_i P_i.
// The gradient holds the picks, and so f, fixed.  With c_i = d_loss alpha f_i / L and D = sum_i p_i c_i:
//   softmax  dl_i = p_i (c_i - D);   sigmoid  dl_i = p_i (1 - s_i) (c_i - D).
//
// Sequences lie one behind the other and may begin anywhere.  16 lanes hold a token, each runs of four neighbouring
// experts.  A workgroup takes a chunk of tokens and writes its sums of p and its counts once for every sequence that it
// meets: chunk c and sequence s have the place c + s, which no other pair has (from one pair to the next, at least one of
// the two grows).  A second kernel adds up the places of each sequence, in order: no floating-point atomics.
#include "lanes.h"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kLanes = 16, kTokens = 64 / kLanes;             // lanes of a token, tokens of a wavefront at a time
constexpr int kPartWaves = 16, kPartThreads = 64 * kPartWaves;  // of a workgroup of the forward pass
constexpr int kWaves = 4, kThreads = 64 * kWaves;             // of a workgroup of the backward pass
constexpr int kJoinThreads = 1024;

// the places' layout: N sums of p (fp32), N counts, the number of tokens
__host__ __device__ inline int64_t place_words(int n) { return 2 * (int64_t)n + 4; }

struct BalanceArgs {
  const void* logits;
  int64_t ld;
  const int32_t *idx, *start;
  int64_t T;
  int N, K, S;
  float alpha;
};

// The sequence that token t lies in (-1: before the first, S: behind the last), the same in all lanes: the number of
// starts at or before t, less one.  A wavefront looks at 64 of them at once.
__device__ __forceinline__ int sequence_of(const BalanceArgs& a, int64_t t) {
  if (!a.start) return 0;
  const int lane = threadIdx.x & 63;
  int lo = 0, hi = a.S + 1;   // the number is in [lo, hi]
  while (hi > lo) {
    const int step = (hi - lo + 63) / 64, at = lo + lane * step;
    const uint64_t below = __ballot(at < hi && a.start[at] <= t);
    const int c = __popcll(below);
    if (c == 0) break;
    if (step == 1) {
      lo += c;
      break;
    }
    const int from = lo + (c - 1) * step;
    hi = min(hi, from + step);
    lo = from + 1;
  }
  return lo - 1;
}

// the end of the piece of sequence s that begins at t, inside [t + 1, end]
__device__ __forceinline__ int64_t piece_end(const BalanceArgs& a, int s, int64_t t, int64_t end) {
  if (!a.start || s >= a.S) return end;
  const int64_t e = a.start[s + 1];
  return e <= t ? t + 1 : e < end ? e : end;
}

// The token's p, and for the sigmoid 1 - s; C runs of four a lane.  Where no logit of the token is positive the sigmoid's
// shares come from exp(l - largest l) / (1 + exp(l)): they keep their value where every s is below 2^-126.  Reciprocals are the
// instruction's, one unit in the last place.
template <int C, bool SOFTMAX>
__device__ __forceinline__ void shares(float (&l)[C][4], float (&rest)[C][4]) {
  float top = kNegInf;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) top = fmaxf(top, l[c][j]);
  top = max_of<kLanes>(top);
  if (top == kNegInf) top = 0.0f;
  float part[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float v = l[c][j];
      if constexpr (SOFTMAX) {
        l[c][j] = exp_of(v - top);
      } else {
        const float x = exp_of(-fabsf(v)), r = __builtin_amdgcn_rcpf(1.0f + x);
        const bool up = v >= 0.0f;
        rest[c][j] = (up ? x : 1.0f) * r;
        l[c][j] = (up ? 1.0f : top < 0.0f ? exp_of(v - top) : x) * r;
      }
    }
    part[c] = sum_run<4>(l[c]);
  }
  const float sum = sum_of<kLanes>(sum_run<C>(part));
  const float r = sum == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(sum);
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) l[c][j] *= r;
}

template <int C, typename TL>
__device__ __forceinline__ void load_token(const TL* row, int N, int lane, float (&l)[C][4]) {
#pragma unroll
  for (int c = 0; c < C; ++c) {
    const int first = 4 * (c * kLanes + lane);
    if (first < N) load_run<4>(row + first, N - first, l[c]);
    else
#pragma unroll
      for (int j = 0; j < 4; ++j) l[c][j] = kNegInf;
  }
}

// the sum over the four tokens of a wavefront
__device__ __forceinline__ float slots_sum(float v) {
  const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  return __uint_as_float(q[0]) + __uint_as_float(q[1]);
}

// chunk: tokens of a workgroup, in blocks of 64 that lie in registers together
template <int C, typename TL, bool SOFTMAX>
__global__ void __launch_bounds__(kPartThreads) balance_part_kernel(BalanceArgs a, int chunk, float* __restrict__ places,
                                                                    int32_t* __restrict__ tickets) {
  extern __shared__ float lds[];   // [kPartWaves][N] sums, then int [N] counts, int [1] tokens
  constexpr int kBlock = kPartWaves * kTokens;
  const int lane = threadIdx.x & (kLanes - 1), wl = threadIdx.x & 63, slot = wl / kLanes, wave = threadIdx.x >> 6;
  const int64_t begin = (int64_t)blockIdx.x * chunk, end = begin + chunk < a.T ? begin + chunk : a.T;
  int* counts = reinterpret_cast<int*>(lds + kPartWaves * a.N);
  if (tickets)   // (for the second kernel)
    for (int64_t i = (int64_t)blockIdx.x * kPartThreads + threadIdx.x; i < a.S; i += (int64_t)gridDim.x * kPartThreads) tickets[i] = 0;
  for (int i = threadIdx.x; i < a.N + 1; i += kPartThreads) counts[i] = 0;
  float total[C][4];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) total[c][j] = 0.0f;
  int seq = -1;   // the sequence of what has been summed so far
  // writes the sums of sequence `seq` and begins anew
  auto leave = [&]() {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = 4 * (c * kLanes + lane) + j;
        const float v = slots_sum(total[c][j]);
        if (slot == 0 && i < a.N) lds[wave * a.N + i] = v;
        total[c][j] = 0.0f;
      }
    __syncthreads();
    float* place = places + ((int64_t)blockIdx.x + seq) * place_words(a.N);
    for (int i = threadIdx.x; i < a.N + 1; i += kPartThreads) {
      if (i < a.N) {
        float v[kPartWaves];
#pragma unroll
        for (int w = 0; w < kPartWaves; ++w) v[w] = lds[w * a.N + i];
        place[i] = sum_run<kPartWaves>(v);
      }
      reinterpret_cast<int*>(place)[a.N + i] = counts[i];
      counts[i] = 0;
    }
    __syncthreads();
  };
  __syncthreads();
  for (int64_t block = begin; block < end; block += kBlock) {
    const int64_t t = block + wave * kTokens + slot, stop = block + kBlock < end ? block + kBlock : end;
    const bool in = t < stop;
    float l[C][4], rest[C][4];
    load_token<C>(static_cast<const TL*>(a.logits) + (in ? t : block) * a.ld, a.N, lane, l);
    int pick[2];   // (at most 32)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = lane + h * kLanes;
      pick[h] = in && k < a.K ? a.idx[t * a.K + k] : -1;
      if (pick[h] >= a.N) pick[h] = -1;
    }
    const bool real = max_of<kLanes>((uint32_t)(pick[0] >= 0 || pick[1] >= 0)) != 0;
    shares<C, SOFTMAX>(l, rest);
    for (int64_t t0 = block; t0 < stop;) {
      const int s = sequence_of(a, t0);
      const int64_t t1 = s < 0 ? (a.start[0] < stop ? a.start[0] : stop) : piece_end(a, s, t0, stop);
      const bool some = s >= 0 && s < a.S;
      if (seq >= 0 && s != seq) {
        __syncthreads();   // (the counts of the piece before)
        leave();
      }
      seq = some ? s : -1;
      if (some && real && t >= t0 && t < t1) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) total[c][j] += l[c][j];
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (pick[h] >= 0) atomicAdd(&counts[pick[h]], 1);
        if (lane == 0) atomicAdd(&counts[a.N], 1);
      }
      t0 = t1;
    }
  }
  if (seq >= 0) {
    __syncthreads();
    leave();
  }
}

struct BalanceOut {
  float* loss;
  int32_t *counts, *tokens;
  float* prob_sum;   // or null
};

// A workgroup adds up 64 columns of a sequence's places, its wavefronts every so many-th place, then their sums.  The loss is a
// sum over the columns: with several workgroups a sequence, each leaves its share and the last of them (by a ticket that the
// first kernel cleared) adds the shares in their order.
__global__ void __launch_bounds__(kJoinThreads) balance_join_kernel(BalanceArgs a, int chunk, const float* __restrict__ places,
                                                                    BalanceOut o, int32_t* tickets, float* dots) {
  constexpr int kBatch = 8;
  __shared__ float sums[kJoinThreads / 64][64];
  __shared__ int counts[kJoinThreads / 64][64];
  __shared__ int lens[kJoinThreads / 64];
  const int s = blockIdx.x, lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int i = blockIdx.y * 64 + lane, col = min(i, a.N - 1);
  int64_t b = a.start ? a.start[s] : 0, e = a.start ? a.start[s + 1] : a.T;
  b = b < 0 ? 0 : b;
  e = e > a.T ? a.T : e;
  float p = 0.0f;
  int n = 0, len = 0;
  if (b < e) {
    const int64_t last = (e - 1) / chunk;
    for (int64_t c0 = b / chunk + wave; c0 <= last; c0 += (int64_t)waves * kBatch) {
      float v[kBatch];
      int m[kBatch], q[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int64_t c = c0 + (int64_t)k * waves < last ? c0 + (int64_t)k * waves : last;
        const float* place = places + (c + s) * place_words(a.N);
        v[k] = place[col];
        m[k] = reinterpret_cast<const int*>(place)[a.N + col];
        q[k] = reinterpret_cast<const int*>(place)[2 * a.N];
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (c0 + (int64_t)k * waves <= last) {
          p += v[k];
          n += m[k];
          len += q[k];
        }
    }
  }
  sums[wave][lane] = p;
  counts[wave][lane] = n;
  if (lane == 0) lens[wave] = len;
  __syncthreads();
  if (wave != 0) return;
  p = 0.0f;
  n = len = 0;
  for (int w = 0; w < waves; ++w) {
    p += sums[w][lane];
    n += counts[w][lane];
    len += lens[w];
  }
  const bool in = i < a.N;
  if (in) {
    o.counts[(int64_t)s * a.N + i] = n;
    if (o.prob_sum) o.prob_sum[(int64_t)s * a.N + i] = p;
  }
  float dot = sum_of<64>(in ? (float)n * p : 0.0f);
  if (lane != 0) return;
  if (blockIdx.y == 0) o.tokens[s] = len;
  if (gridDim.y > 1) {
    float* mine = dots + (int64_t)s * gridDim.y;
    __hip_atomic_store(&mine[blockIdx.y], dot, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (__hip_atomic_fetch_add(&tickets[s], 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) != (int)gridDim.y - 1) return;
    dot = 0.0f;
    for (unsigned k = 0; k < gridDim.y; ++k) dot += __hip_atomic_load(&mine[k], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  o.loss[s] = len == 0 ? 0.0f : a.alpha * (dot / (float)len) * ((float)a.N / ((float)a.K * (float)len));
}

__global__ void balance_zero_kernel(BalanceOut o, int S, int N) {
  const int64_t at = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (at < S) {
    o.loss[at] = 0.0f;
    o.tokens[at] = 0;
  }
  if (at >= (int64_t)S * N) return;
  o.counts[at] = 0;
  if (o.prob_sum) o.prob_sum[at] = 0.0f;
}

struct BalanceBwdArgs {
  const int32_t *counts, *tokens;
  const float* d_loss;
  void* d_logits;
  int64_t d_ld;
};

// The sequence of the token that the lane's 16 lanes hold, as sequence_of; 16 starts at once.
__device__ __forceinline__ int sequence_of_lanes(const BalanceArgs& a, int64_t t) {
  if (!a.start) return 0;
  const int lane = threadIdx.x & (kLanes - 1), shift = threadIdx.x & 63 & ~(kLanes - 1);
  int lo = 0, hi = a.S + 1;
  while (hi > lo) {
    const int step = (hi - lo + kLanes - 1) / kLanes, at = lo + lane * step;
    const int c = __popc((uint32_t)(__ballot(at < hi && a.start[at] <= t) >> shift) & 0xFFFFu);
    if (c == 0) break;
    if (step == 1) {
      lo += c;
      break;
    }
    const int from = lo + (c - 1) * step;
    hi = min(hi, from + step);
    lo = from + 1;
  }
  return lo - 1;
}

// Four tokens a wavefront, each with its own sequence.
template <int C, typename TL, bool SOFTMAX, bool ADD>
__global__ void __launch_bounds__(kThreads) balance_bwd_kernel(BalanceArgs a, BalanceBwdArgs w) {
  const int lane = threadIdx.x & (kLanes - 1), slot = (threadIdx.x & 63) / kLanes, wave = threadIdx.x >> 6;
  constexpr int kBlock = kWaves * kTokens;
  for (int64_t t = (int64_t)blockIdx.x * kBlock + wave * kTokens + slot; t < a.T; t += (int64_t)gridDim.x * kBlock) {
    float l[C][4], rest[C][4], pull[C][4];
    load_token<C>(static_cast<const TL*>(a.logits) + t * a.ld, a.N, lane, l);
    bool some = false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = lane + h * kLanes, e = k < a.K ? a.idx[t * a.K + k] : -1;
      some |= e >= 0 && e < a.N;
    }
    const int s = sequence_of_lanes(a, t);
    const bool real = s >= 0 && s < a.S && max_of<kLanes>((uint32_t)some) != 0;
    const float len = real ? (float)w.tokens[s] : 0.0f;
    const float each = len > 0.0f ? w.d_loss[s] * a.alpha * ((float)a.N / ((float)a.K * len)) / len : 0.0f;
    const int32_t* n = w.counts + (real ? (int64_t)s * a.N : 0);
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int first = 4 * (c * kLanes + lane);
      if (first + 4 <= a.N) {
        struct __attribute__((packed, aligned(4))) Run { int32_t v[4]; };
        const Run q = *reinterpret_cast<const Run*>(n + first);
#pragma unroll
        for (int j = 0; j < 4; ++j) pull[c][j] = each * (float)q.v[j];
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) pull[c][j] = first + j < a.N ? each * (float)n[first + j] : 0.0f;
      }
    }
    shares<C, SOFTMAX>(l, rest);
    float part[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) q[j] = l[c][j] * pull[c][j];
      part[c] = sum_run<4>(q);
    }
    const float dot = sum_of<kLanes>(sum_run<C>(part));
    TL* row = static_cast<TL*>(w.d_logits) + t * w.d_ld;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int first = 4 * (c * kLanes + lane);
      if (first >= a.N || (ADD && !real)) continue;
      float d[4], was[4];
      if constexpr (ADD) load_run<4>(row + first, a.N - first, was);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        d[j] = l[c][j] * (pull[c][j] - dot);
        if constexpr (!SOFTMAX) d[j] *= rest[c][j];
        if (!real) d[j] = 0.0f;
        if constexpr (ADD) d[j] += was[j];
      }
      store_run4(row + first, a.N - first, d);
    }
  }
}

// Tokens of a workgroup of the forward pass: 64, or more where that would make over 1024 places
int chunk_of(const moe_balance_config& c) {
  int64_t chunk = 64;
  while (ceil_div(c.tokens, chunk) > 1024) chunk *= 2;
  return (int)chunk;
}

BalanceArgs args_of(const moe_balance_config& c, const void* logits, const int32_t* idx, const int32_t* start) {
  return {logits, c.logits_ld ? c.logits_ld : c.n_routed, idx, start, c.tokens, c.n_routed, c.top_k, c.n_seqs, c.alpha};
}

// f(integral_constant) with the runs of four a lane that hold N experts
template <typename F>
hipError_t with_runs(int n, F f) {
  if (n <= 64) return f(std::integral_constant<int, 1>{});
  if (n <= 128) return f(std::integral_constant<int, 2>{});
  if (n <= 256) return f(std::integral_constant<int, 4>{});
  return f(std::integral_constant<int, 8>{});
}

template <typename TL, bool SOFTMAX>
hipError_t part_t(const BalanceArgs& a, int chunk, float* places, int32_t* tickets, hipStream_t st) {
  const size_t lds = (size_t)(kPartWaves * a.N + a.N + 4) * 4;
  return with_runs(a.N, [&](auto c) {
    return launch_kernel(balance_part_kernel<decltype(c)::value, TL, SOFTMAX>, dim3((unsigned)ceil_div(a.T, chunk)),
                         dim3(kPartThreads), lds, st, a, chunk, places, tickets);
  });
}

template <typename TL, bool SOFTMAX>
hipError_t bwd_t(const BalanceArgs& a, const BalanceBwdArgs& w, bool add, hipStream_t st) {
  const unsigned grid = (unsigned)std::min<int64_t>(ceil_div(a.T, kWaves * kTokens), 1 << 16);
  return with_runs(a.N, [&](auto c) {
    return add ? launch_kernel(balance_bwd_kernel<decltype(c)::value, TL, SOFTMAX, true>, dim3(grid), dim3(kThreads), 0, st, a, w)
               : launch_kernel(balance_bwd_kernel<decltype(c)::value, TL, SOFTMAX, false>, dim3(grid), dim3(kThreads), 0, st, a, w);
  });
}

}  // namespace

// the workspace: places, then (more than 64 experts) a ticket and a share of the loss per 64 columns for each sequence
size_t balance_workspace(const moe_balance_config& c) {
  if (c.tokens == 0) return 0;
  const size_t places = (size_t)(ceil_div(c.tokens, chunk_of(c)) + c.n_seqs) * place_words(c.n_routed) * 4;
  return places + (c.n_routed > 64 ? (size_t)c.n_seqs * (1 + ceil_div(c.n_routed, 64)) * 4 : 0);
}

hipError_t launch_balance_loss(const moe_balance_config& c, const void* logits, const int32_t* idx, const int32_t* start,
                               float* loss, int32_t* counts, int32_t* tokens, float* prob_sum, float* places,
                               hipStream_t st) {
  const BalanceArgs a = args_of(c, logits, idx, start);
  const BalanceOut o{loss, counts, tokens, prob_sum};
  if (c.tokens == 0)
    return launch_kernel(balance_zero_kernel, dim3((unsigned)ceil_div((int64_t)c.n_seqs * c.n_routed, 256)), dim3(256), 0, st,
                         o, c.n_seqs, c.n_routed);
  const int chunk = chunk_of(c);
  float* dots = places + (ceil_div(c.tokens, chunk) + c.n_seqs) * place_words(c.n_routed);
  int32_t* tickets = c.n_routed > 64 ? reinterpret_cast<int32_t*>(dots + c.n_seqs * ceil_div(c.n_routed, 64)) : nullptr;
  const bool f32 = c.logits_dtype == MOE_DTYPE_F32;
  hipError_t err;
  if (c.score == MOE_SCORE_SOFTMAX)
    err = f32 ? part_t<float, true>(a, chunk, places, tickets, st) : part_t<uint16_t, true>(a, chunk, places, tickets, st);
  else
    err = f32 ? part_t<float, false>(a, chunk, places, tickets, st) : part_t<uint16_t, false>(a, chunk, places, tickets, st);
  if (err != hipSuccess) return err;
  // wavefronts: 16, or 4 where a sequence has few places
  const unsigned threads = c.tokens / c.n_seqs >= 8 * chunk ? kJoinThreads : 256;
  return launch_kernel(balance_join_kernel, dim3((unsigned)c.n_seqs, (unsigned)ceil_div(c.n_routed, 64)), dim3(threads), 0, st, a,
                       chunk, places, o, tickets, dots);
}

hipError_t launch_balance_backward(const moe_balance_config& c, const void* logits, const int32_t* idx, const int32_t* start,
                                   const int32_t* counts, const int32_t* tokens, const float* d_loss, void* d_logits,
                                   int64_t d_ld, bool add, hipStream_t st) {
  if (c.tokens == 0) return hipSuccess;
  const BalanceArgs a = args_of(c, logits, idx, start);
  const BalanceBwdArgs w{counts, tokens, d_loss, d_logits, d_ld ? d_ld : c.n_routed};
  const bool f32 = c.logits_dtype == MOE_DTYPE_F32;
  if (c.score == MOE_SCORE_SOFTMAX)
    return f32 ? bwd_t<float, true>(a, w, add, st) : bwd_t<uint16_t, true>(a, w, add, st);
  return f32 ? bwd_t<float, false>(a, w, add, st) : bwd_t<uint16_t, false>(a, w, add, st);
}

}  // namespace moe
