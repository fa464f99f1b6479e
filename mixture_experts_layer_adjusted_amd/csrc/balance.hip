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

constexpr int kThreads = 256, kWaves = 4, kLanes = 16;
constexpr int kTokens = 64 / kLanes;          // tokens of a wavefront at a time
constexpr int kBwdChunk = 16;                 // tokens of a workgroup of the backward pass
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

// The token's p, and for the sigmoid 1 - s; C runs of four a lane.  The sigmoid's shares are those of
// exp(min(l, 0) - m) / (1 + exp(-|l|)) with m = min(largest l, 0): they keep their value where every s is below 2^-126.
template <int C, bool SOFTMAX>
__device__ __forceinline__ void shares(float (&l)[C][4], float (&rest)[C][4]) {
  float top = kNegInf;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) top = fmaxf(top, l[c][j]);
  top = max_of<kLanes>(top);
  if (top == kNegInf) top = 0.0f;
  const float m = fminf(top, 0.0f);
  float part[C];
#pragma unroll
  for (int c = 0; c < C; ++c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float v = l[c][j];
      if constexpr (SOFTMAX) {
        l[c][j] = exp_of(v - top);
      } else {
        const float x = exp_of(-fabsf(v)), r = 1.0f / (1.0f + x);
        rest[c][j] = v >= 0.0f ? x * r : r;
        l[c][j] = v >= 0.0f ? r : (m == 0.0f ? x : exp_of(v - m)) * r;
        if (v != v) l[c][j] = rest[c][j] = v;
      }
    }
    part[c] = sum_run<4>(l[c]);
  }
  const float sum = sum_of<kLanes>(sum_run<C>(part));
  const float r = sum == 0.0f ? 0.0f : 1.0f / sum;
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

// chunk: tokens of a workgroup
template <int C, typename TL, bool SOFTMAX>
__global__ void __launch_bounds__(kThreads) balance_part_kernel(BalanceArgs a, int chunk, float* __restrict__ places) {
  extern __shared__ float lds[];   // [kWaves * kTokens][N] sums, then int [N] counts, int [1] tokens
  const int lane = threadIdx.x & (kLanes - 1), wl = threadIdx.x & 63, slot = wl / kLanes, wave = threadIdx.x >> 6;
  const int64_t begin = (int64_t)blockIdx.x * chunk, end = begin + chunk < a.T ? begin + chunk : a.T;
  int* counts = reinterpret_cast<int*>(lds + kWaves * kTokens * a.N);
  for (int64_t t0 = begin; t0 < end;) {
    const int s = sequence_of(a, t0);
    const int64_t t1 = s < 0 ? (a.start[0] < end ? a.start[0] : end) : piece_end(a, s, t0, end);
    if (s >= 0 && s < a.S) {
      for (int i = threadIdx.x; i < a.N + 1; i += kThreads) counts[i] = 0;
      __syncthreads();
      float total[C][4];
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) total[c][j] = 0.0f;
      for (int64_t t = t0 + wave * kTokens + slot; t < t1; t += kWaves * kTokens) {   // (lanes of 16 stay together)
        float l[C][4], rest[C][4];
        load_token<C>(static_cast<const TL*>(a.logits) + t * a.ld, a.N, lane, l);
        uint32_t mine = 0;
        for (int k = lane; k < a.K; k += kLanes) {
          const int e = a.idx[t * a.K + k];
          if (e >= 0 && e < a.N) {
            atomicAdd(&counts[e], 1);
            mine = 1;
          }
        }
        const bool real = max_of<kLanes>(mine) != 0;
        shares<C, SOFTMAX>(l, rest);
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) total[c][j] += real ? l[c][j] : 0.0f;
        if (real && lane == 0) atomicAdd(&counts[a.N], 1);
      }
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = 4 * (c * kLanes + lane) + j;
          if (i < a.N) lds[(wave * kTokens + slot) * a.N + i] = total[c][j];
        }
      __syncthreads();
      float* place = places + ((int64_t)blockIdx.x + s) * place_words(a.N);
      for (int i = threadIdx.x; i < a.N; i += kThreads) {
        float v[kWaves * kTokens];
#pragma unroll
        for (int w = 0; w < kWaves * kTokens; ++w) v[w] = lds[w * a.N + i];
        place[i] = sum_run<kWaves * kTokens>(v);
        reinterpret_cast<int*>(place)[a.N + i] = counts[i];
      }
      if (threadIdx.x == 0) reinterpret_cast<int*>(place)[2 * a.N] = counts[a.N];
      __syncthreads();
    }
    t0 = t1;
  }
}

struct BalanceOut {
  float* loss;
  int32_t *counts, *tokens;
  float* prob_sum;   // or null
};

// One workgroup a sequence: its places added up in order, then the loss.  Columns are padded to a power of two, the
// threads beyond them take every further place.
__global__ void __launch_bounds__(kJoinThreads) balance_join_kernel(BalanceArgs a, int chunk, const float* __restrict__ places,
                                                                    BalanceOut o, int cols) {
  __shared__ float sums[kJoinThreads];
  __shared__ int counts[kJoinThreads];
  __shared__ int tokens;
  const int s = blockIdx.x, tid = threadIdx.x, i = tid & (cols - 1), group = tid / cols, groups = kJoinThreads / cols;
  if (tid == 0) tokens = 0;
  int64_t b = a.start ? a.start[s] : 0, e = a.start ? a.start[s + 1] : a.T;
  b = b < 0 ? 0 : b;
  e = e > a.T ? a.T : e;
  __syncthreads();
  float p = 0.0f;
  int n = 0, L = 0;
  if (b < e) {
    const int64_t last = (e - 1) / chunk;
    for (int64_t c = b / chunk + group; c <= last; c += groups) {
      const float* place = places + (c + s) * place_words(a.N);
      if (i < a.N) {
        p += place[i];
        n += reinterpret_cast<const int*>(place)[a.N + i];
      }
      if (i == 0) L += reinterpret_cast<const int*>(place)[2 * a.N];
    }
  }
  if (L) atomicAdd(&tokens, L);
  sums[tid] = p;
  counts[tid] = n;
  __syncthreads();
  float f = 0.0f;
  if (group == 0) {
    for (int g = 1; g < groups; ++g) {
      p += sums[g * cols + i];
      n += counts[g * cols + i];
    }
    if (i < a.N) {
      o.counts[(int64_t)s * a.N + i] = n;
      if (o.prob_sum) o.prob_sum[(int64_t)s * a.N + i] = p;
      f = (float)n * p;
    }
  }
  __syncthreads();
  // the sum over the experts: 64 lanes at a time, then their sums
  f = sum_of<64>(f);
  if ((tid & 63) == 0) sums[tid >> 6] = f;
  __syncthreads();
  if (tid != 0) return;
  float dot = 0.0f;
  for (int w = 0; w < max(1, cols / 64); ++w) dot += sums[w];
  const float len = (float)tokens;
  o.tokens[s] = tokens;
  o.loss[s] = tokens == 0 ? 0.0f : a.alpha * (dot / len) * ((float)a.N / ((float)a.K * len));
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

template <int C, typename TL, bool SOFTMAX, bool ADD>
__global__ void __launch_bounds__(kThreads) balance_bwd_kernel(BalanceArgs a, BalanceBwdArgs w) {
  const int lane = threadIdx.x & (kLanes - 1), slot = (threadIdx.x & 63) / kLanes, wave = threadIdx.x >> 6;
  const int64_t chunks = (a.T + kBwdChunk - 1) / kBwdChunk;
  for (int64_t chunk = blockIdx.x; chunk < chunks; chunk += gridDim.x) {
    const int64_t begin = chunk * kBwdChunk, end = begin + kBwdChunk < a.T ? begin + kBwdChunk : a.T;
    for (int64_t t0 = begin; t0 < end;) {
      const int s = sequence_of(a, t0);
      const int64_t t1 = s < 0 ? (a.start[0] < end ? a.start[0] : end) : piece_end(a, s, t0, end);
      const bool in = s >= 0 && s < a.S;
      const float len = in ? (float)w.tokens[s] : 0.0f;
      const float each = len > 0.0f ? w.d_loss[s] * a.alpha * ((float)a.N / ((float)a.K * len)) / len : 0.0f;
      float pull[C][4];
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int i = 4 * (c * kLanes + lane) + j;
          pull[c][j] = in && i < a.N ? each * (float)w.counts[(int64_t)s * a.N + i] : 0.0f;
        }
      for (int64_t t = t0 + wave * kTokens + slot; t < t1; t += kWaves * kTokens) {
        float l[C][4], rest[C][4];
        load_token<C>(static_cast<const TL*>(a.logits) + t * a.ld, a.N, lane, l);
        uint32_t mine = 0;
        for (int k = lane; k < a.K; k += kLanes) {
          const int e = a.idx[t * a.K + k];
          if (e >= 0 && e < a.N) mine = 1;
        }
        const bool real = in && max_of<kLanes>(mine) != 0;
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
      t0 = t1;
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
hipError_t part_t(const BalanceArgs& a, int chunk, float* places, hipStream_t st) {
  const size_t lds = (size_t)(kWaves * kTokens * a.N + a.N + 4) * 4;
  return with_runs(a.N, [&](auto c) {
    return launch_kernel(balance_part_kernel<decltype(c)::value, TL, SOFTMAX>, dim3((unsigned)ceil_div(a.T, chunk)),
                         dim3(kThreads), lds, st, a, chunk, places);
  });
}

template <typename TL, bool SOFTMAX>
hipError_t bwd_t(const BalanceArgs& a, const BalanceBwdArgs& w, bool add, hipStream_t st) {
  const unsigned grid = (unsigned)std::min<int64_t>(ceil_div(a.T, kBwdChunk), 1 << 16);
  return with_runs(a.N, [&](auto c) {
    return add ? launch_kernel(balance_bwd_kernel<decltype(c)::value, TL, SOFTMAX, true>, dim3(grid), dim3(kThreads), 0, st, a, w)
               : launch_kernel(balance_bwd_kernel<decltype(c)::value, TL, SOFTMAX, false>, dim3(grid), dim3(kThreads), 0, st, a, w);
  });
}

}  // namespace

size_t balance_workspace(const moe_balance_config& c) {
  return c.tokens == 0 ? 0 : (size_t)(ceil_div(c.tokens, chunk_of(c)) + c.n_seqs) * place_words(c.n_routed) * 4;
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
  const bool f32 = c.logits_dtype == MOE_DTYPE_F32;
  hipError_t err;
  if (c.score == MOE_SCORE_SOFTMAX)
    err = f32 ? part_t<float, true>(a, chunk, places, st) : part_t<uint16_t, true>(a, chunk, places, st);
  else
    err = f32 ? part_t<float, false>(a, chunk, places, st) : part_t<uint16_t, false>(a, chunk, places, st);
  if (err != hipSuccess) return err;
  int cols = 1;
  while (cols < c.n_routed) cols *= 2;
  return launch_kernel(balance_join_kernel, dim3((unsigned)c.n_seqs), dim3(kJoinThreads), 0, st, a, chunk, places, o, cols);
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
