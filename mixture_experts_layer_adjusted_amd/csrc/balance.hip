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
// Sequences lie one behind the other and may begin anywhere.  16 lanes hold a token (32 above 128 experts, 64 above 256),
// each one or two runs of four neighbouring experts.  A workgroup takes a chunk of tokens and writes its sums of p and its
// counts once for every sequence that it meets: chunk c and sequence s have the place c + s, which no other pair has (from
// one pair to the next, at least one of the two grows).  A second kernel adds up the places of each sequence, in order: no
// floating-point atomics.  (A sum over several workgroups a sequence, the last by a ticket, cost 2 us of device-wide
// atomics and gained less.)  Few tokens take one kernel, a workgroup a sequence.
//
// Bound by latency and instructions (traced): 32768 tokens of 64 experts, softmax: 6.1 us (8.4 MB), the second kernel 5.1, the
// gradient 6.4 (16.8 MB); 16384 tokens of 256 experts, sigmoid: 10.2 (16.8 MB; 330 vector instructions for two tokens), 6.5, 9.4
// (33.6 MB).  Loads of one value each where four lie side by side cost the gradient 14.0 in place of 9.4.  7 sequences of 1021
// tokens of 60 experts, softmax: 7.2 in one kernel (5.6 + 3.9 in two), the gradient 3.2.
#include "lanes.h"
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kPartWaves = 16, kPartThreads = 64 * kPartWaves;  // of a workgroup of the forward pass
constexpr int kWaves = 4, kThreads = 64 * kWaves;             // of a workgroup of the backward pass
constexpr int kJoinThreads = 1024;                            // of the second kernel
// Places for the whole batch, or so: T=32768, 64 experts, 512 of them 8.8 + 5.7 us, 256 6.2 + 5.8; T=16384, 256 experts 12.7 +
// 5.8, 10.0 + 5.9.
constexpr int kPlaces = 256;

// the places' layout: sums of p (fp32), counts, the number of tokens, columns rounded up to fours
__host__ __device__ inline int place_cols(int n) { return (n + 3) & ~3; }
__host__ __device__ inline int place_words(int n) { return 2 * place_cols(n) + 4; }

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
  if (a.S < 64) return __popcll(__ballot(a.start[min(lane, a.S)] <= t && lane <= a.S)) - 1;
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

// where sequence s (as sequence_of has it) ends
__device__ __forceinline__ int64_t sequence_end(const BalanceArgs& a, int s) {
  return !a.start || s >= a.S ? a.T : a.start[s + 1];
}

// The token's p, and for the sigmoid 1 - s; C runs of four a lane.  Where no logit of the token is positive the sigmoid's
// shares come from exp(l - largest l) / (1 + exp(l)): they keep their value where every s is below 2^-126.  Reciprocals are the
// instruction's, one unit in the last place.
template <int L, int C, bool SOFTMAX>
__device__ __forceinline__ void shares(float (&l)[C][4], float (&rest)[C][4]) {
  float top = kNegInf;
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) top = fmaxf(top, l[c][j]);
  top = max_of<L>(top);
  if (top == kNegInf) top = 0.0f;
  float part[C];
  const bool low = top < 0.0f;
  // some_low: a token of the wavefront has no positive logit
  auto each = [&](auto some_low) {
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
          float part_of_s = x;
          if constexpr (decltype(some_low)::value) {
            const float alike = exp_of(v - top);
            part_of_s = low ? alike : x;
          }
          rest[c][j] = (up ? x : 1.0f) * r;
          l[c][j] = (up ? 1.0f : part_of_s) * r;
        }
      }
      part[c] = sum_run<4>(l[c]);
    }
  };
  if (!SOFTMAX && __ballot(low) != 0) each(std::true_type{});
  else each(std::false_type{});
  const float sum = sum_of<L>(sum_run<C>(part));
  const float r = sum == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(sum);
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) l[c][j] *= r;
}

// Four neighbouring values of a row of n, from `first` on (any alignment), as they lie in memory: loads ahead of their use.
// No lane goes round a load, lanes behind the row's end load other values of it.  WHOLE: n is a multiple of four (known to
// the compiler: it would make four loads of one and a choice of addresses out of a branch).
template <bool WHOLE, typename T>
struct Four {
  uint32_t w[WHOLE ? sizeof(T) : 4];
};
template <bool WHOLE, typename T>
__device__ __forceinline__ Four<WHOLE, T> four_at(const T* row, int first, int n) {
  Four<WHOLE, T> q;
  if constexpr (WHOLE) {
    struct __attribute__((packed, aligned(sizeof(T)))) Run { uint32_t w[sizeof(T)]; };
    const Run r = *reinterpret_cast<const Run*>(row + (first < n ? first : 0));
#pragma unroll
    for (int j = 0; j < (int)sizeof(T); ++j) q.w[j] = r.w[j];
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const T* at = row + min(first + j, n - 1);
      if constexpr (sizeof(T) == 2) q.w[j] = (uint32_t)*at << 16;
      else q.w[j] = *reinterpret_cast<const uint32_t*>(at);
    }
  }
  return q;
}
// the values, `fill` behind the row's end
template <bool WHOLE, typename T>
__device__ __forceinline__ void values(const Four<WHOLE, T>& q, int first, int n, float fill, float (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if constexpr (WHOLE && sizeof(T) == 2)
      v[j] = __uint_as_float(j & 1 ? q.w[j / 2] & 0xFFFF0000u : q.w[j / 2] << 16);
    else v[j] = __uint_as_float(q.w[j]);
    v[j] = (WHOLE ? first : first + j) < n ? v[j] : fill;
  }
}

// a token's logits
template <int L, int C, bool WHOLE, typename TL>
__device__ __forceinline__ void load_token(const TL* row, int N, int lane, Four<WHOLE, TL> (&q)[C]) {
#pragma unroll
  for (int c = 0; c < C; ++c) q[c] = four_at<WHOLE>(row, 4 * (c * L + lane), N);
}
template <int L, int C, bool WHOLE, typename TL>
__device__ __forceinline__ void unpack_token(const Four<WHOLE, TL> (&q)[C], int N, int lane, float (&l)[C][4]) {
#pragma unroll
  for (int c = 0; c < C; ++c) values(q[c], 4 * (c * L + lane), N, kNegInf, l[c]);
}

// the sum over the tokens of a wavefront
template <int L>
__device__ __forceinline__ float slots_sum(float v) {
  if constexpr (L == 16) {
    const auto p = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(p[0]) + __uint_as_float(p[1]);
  }
  if constexpr (L <= 32) {
    const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(q[0]) + __uint_as_float(q[1]);
  }
  return v;
}

// the token's entries of topk_idx that the lane holds, -1 behind the last (at most 32 picks: two of 16 lanes)
template <int L>
constexpr int kPicks = L == 16 ? 2 : 1;
template <int L>
__device__ __forceinline__ void load_picks(const BalanceArgs& a, int64_t t, int lane, int (&pick)[kPicks<L>]) {
#pragma unroll
  for (int h = 0; h < kPicks<L>; ++h) pick[h] = lane + h * L < a.K ? a.idx[t * a.K + lane + h * L] : -1;
}

struct BalanceOut {
  float* loss;
  int32_t *counts, *tokens;
  float* prob_sum;   // or null
};

// the loss from sum_i n_i sum_t p_{t,i} and L
__device__ __forceinline__ float balance_of(const BalanceArgs& a, float dot, int len) {
  return len == 0 ? 0.0f : a.alpha * (dot / (float)len) * ((float)a.N / ((float)a.K * (float)len));
}

// Few tokens (few_tokens, below): a workgroup a sequence does all of it.
template <int L, int C, bool WHOLE, typename TL, bool SOFTMAX>
__global__ void __launch_bounds__(kPartThreads) balance_few_kernel(BalanceArgs a, BalanceOut o) {
  extern __shared__ float lds[];   // [kPartWaves][N] sums, then int [N] counts, int [1] tokens
  __shared__ float dots[kPartWaves];
  constexpr int kTokens = 64 / L, kBlock = kPartWaves * kTokens;
  const int lane = threadIdx.x & (L - 1), slot = (threadIdx.x & 63) / L, wave = threadIdx.x >> 6, s = blockIdx.x;
  int* counts = reinterpret_cast<int*>(lds + kPartWaves * a.N);
  const int T = (int)a.T, begin = a.start ? max(0, a.start[s]) : 0, end = a.start ? min(T, a.start[s + 1]) : T;
  float total[C][4];
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) total[c][j] = 0.0f;
  // a block's logits and picks, on their way while the block before is worked on
  Four<WHOLE, TL> next[C];
  int next_pick[kPicks<L>];
  auto load = [&](int block) {
    const int t = min(block + wave * kTokens + slot, end - 1);
    load_token<L, C, WHOLE>(static_cast<const TL*>(a.logits) + t * a.ld, a.N, lane, next);
    load_picks<L>(a, t, lane, next_pick);
  };
  if (begin < end) load(begin);
  for (int i = threadIdx.x; i < a.N + 1; i += kPartThreads) counts[i] = 0;
  __syncthreads();
  for (int block = begin; block < end; block += kBlock) {
    float l[C][4], rest[C][4];
    int pick[kPicks<L>];
    bool some = false;
    unpack_token<L, C, WHOLE>(next, a.N, lane, l);
#pragma unroll
    for (int h = 0; h < kPicks<L>; ++h) {
      pick[h] = next_pick[h] < a.N ? next_pick[h] : -1;
      some |= pick[h] >= 0;
    }
    if (block + kBlock < end) load(block + kBlock);
    const bool real = max_of<L>((uint32_t)some) != 0 && block + wave * kTokens + slot < end;
    shares<L, C, SOFTMAX>(l, rest);
    if (real) {
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) total[c][j] += l[c][j];
#pragma unroll
      for (int h = 0; h < kPicks<L>; ++h)
        if (pick[h] >= 0) atomicAdd(&counts[pick[h]], 1);
      if (lane == 0) atomicAdd(&counts[a.N], 1);
    }
  }
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = 4 * (c * L + lane) + j;
      const float v = slots_sum<L>(total[c][j]);
      if (slot == 0 && i < a.N) lds[wave * a.N + i] = v;
    }
  __syncthreads();
  const int i = threadIdx.x;
  float term = 0.0f;
  if (i < a.N) {   // (N is at most 512)
    float v[kPartWaves];
#pragma unroll
    for (int w = 0; w < kPartWaves; ++w) v[w] = lds[w * a.N + i];
    const float p = sum_run<kPartWaves>(v);
    const int n = counts[i];
    term = (float)n * p;
    o.counts[(int64_t)s * a.N + i] = n;
    if (o.prob_sum) o.prob_sum[(int64_t)s * a.N + i] = p;
  }
  term = sum_of<64>(term);
  if ((i & 63) == 0) dots[wave] = term;
  __syncthreads();
  if (i != 0) return;
  float dot = 0.0f;
  for (int w = 0; 64 * w < a.N; ++w) dot += dots[w];
  const int len = counts[a.N];
  o.tokens[s] = len;
  o.loss[s] = balance_of(a, dot, len);
}

// L lanes a token.  chunk: tokens of a workgroup, in blocks that lie in registers together.  After kHeld blocks a lane's sums go
// into second ones: thousands of fp32 additions one after another may all round the same way (2^26 tokens of 64 experts, all
// alike, 4096 additions: 2^-14 of the sum; 2^-19 with these).  Chunks of up to kHeld blocks (2^20 tokens at 64 experts) do not.
template <int L, int C, bool WHOLE, typename TL, bool SOFTMAX>
__global__ void __launch_bounds__(kPartThreads) balance_part_kernel(BalanceArgs a, int chunk, float* __restrict__ places) {
  extern __shared__ float lds[];   // [kPartWaves][N] sums, then int [N] counts, int [1] tokens
  constexpr int kTokens = 64 / L, kBlock = kPartWaves * kTokens, kHeld = 64;
  const int lane = threadIdx.x & (L - 1), slot = (threadIdx.x & 63) / L, wave = threadIdx.x >> 6;
  const int64_t begin = (int64_t)blockIdx.x * chunk, end = begin + chunk < a.T ? begin + chunk : a.T;
  int* counts = reinterpret_cast<int*>(lds + kPartWaves * a.N);
  float total[C][4], before[C][4];
  int held = 0;   // blocks whose sums are in total
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) total[c][j] = before[c][j] = 0.0f;
  int seq = -1;   // the sequence of what has been summed so far
  // writes the sums of sequence `seq` and begins anew
  auto leave = [&]() {
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = 4 * (c * L + lane) + j;
        const float v = slots_sum<L>(before[c][j] + total[c][j]);
        if (slot == 0 && i < a.N) lds[wave * a.N + i] = v;
        total[c][j] = before[c][j] = 0.0f;
      }
    __syncthreads();
    float* place = places + ((int64_t)blockIdx.x + seq) * place_words(a.N);
    const int cols = place_cols(a.N);
    for (int i = threadIdx.x; i < a.N + 1; i += kPartThreads) {
      if (i < a.N) {
        float v[kPartWaves];
#pragma unroll
        for (int w = 0; w < kPartWaves; ++w) v[w] = lds[w * a.N + i];
        place[i] = sum_run<kPartWaves>(v);
      }
      reinterpret_cast<int*>(place)[i < a.N ? cols + i : 2 * cols] = counts[i];
      counts[i] = 0;
    }
    __syncthreads();
  };
  // a block's logits and picks, on their way while the block before is worked on
  Four<WHOLE, TL> next[C];
  int next_pick[kPicks<L>];
  auto load = [&](int64_t block) {
    const int64_t t = block + wave * kTokens + slot;
    load_token<L, C, WHOLE>(static_cast<const TL*>(a.logits) + (t < end ? t : end - 1) * a.ld, a.N, lane, next);
    load_picks<L>(a, t < end ? t : end - 1, lane, next_pick);
  };
  load(begin);
  for (int i = threadIdx.x; i < a.N + 1; i += kPartThreads) counts[i] = 0;
  int s = sequence_of(a, begin);
  int64_t s_end = sequence_end(a, s);
  __syncthreads();
  for (int64_t block = begin; block < end; block += kBlock) {
    const int64_t t = block + wave * kTokens + slot, stop = block + kBlock < end ? block + kBlock : end;
    float l[C][4], rest[C][4];
    int pick[kPicks<L>];
    bool some = false;
    unpack_token<L, C, WHOLE>(next, a.N, lane, l);
#pragma unroll
    for (int h = 0; h < kPicks<L>; ++h) {
      pick[h] = next_pick[h] < a.N ? next_pick[h] : -1;
      some |= pick[h] >= 0;
    }
    if (block + kBlock < end) load(block + kBlock);
    const bool real = max_of<L>((uint32_t)some) != 0;
    shares<L, C, SOFTMAX>(l, rest);
    for (int64_t t0 = block; t0 < stop;) {
      if (t0 >= s_end && t0 > begin) {
        s = sequence_of(a, t0);
        s_end = sequence_end(a, s);
      }
      const int64_t t1 = s_end <= t0 ? t0 + 1 : s_end < stop ? s_end : stop;
      const bool inside = s >= 0 && s < a.S;
      if (seq >= 0 && s != seq) {
        __syncthreads();   // (the counts of the piece before)
        leave();
      }
      seq = inside ? s : -1;
      if (inside && real && t >= t0 && t < t1) {
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
          for (int j = 0; j < 4; ++j) total[c][j] += l[c][j];
#pragma unroll
        for (int h = 0; h < kPicks<L>; ++h)
          if (pick[h] >= 0) atomicAdd(&counts[pick[h]], 1);
        if (lane == 0) atomicAdd(&counts[a.N], 1);
      }
      t0 = t1;
    }
    if (++held == kHeld) {
      held = 0;
#pragma unroll
      for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          before[c][j] += total[c][j];
          total[c][j] = 0.0f;
        }
    }
  }
  if (seq >= 0) {
    __syncthreads();
    leave();
  }
}

// One workgroup a sequence: its places added up in order, then the loss, which is a sum over all columns.  `quads` threads (a
// power of two, 16 at least) take four columns each, groups of them every further place, four loads at once.
__global__ void __launch_bounds__(kJoinThreads) balance_join_kernel(BalanceArgs a, int chunk, const float* __restrict__ places,
                                                                    BalanceOut o, int quads) {
  typedef float f32x4 __attribute__((ext_vector_type(4)));
  typedef int i32x4 __attribute__((ext_vector_type(4)));
  constexpr int kBatch = 4, kMost = kJoinThreads / 64;
  __shared__ f32x4 sums[kMost][64];
  __shared__ i32x4 counts[kMost][64];
  __shared__ int lens[kMost];
  __shared__ float dots[2];
  const int s = blockIdx.x, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, waves = blockDim.x >> 6;
  const int cols = place_cols(a.N), words = place_words(a.N), col = min(4 * (tid & (quads - 1)), cols - 4);
  const int group = tid / quads, groups = blockDim.x / quads;
  int64_t b = a.start ? a.start[s] : 0, e = a.start ? a.start[s + 1] : a.T;
  b = b < 0 ? 0 : b;
  e = e > a.T ? a.T : e;
  f32x4 p = {0.0f, 0.0f, 0.0f, 0.0f};
  i32x4 n = {0, 0, 0, 0};
  int len = 0;
  if (b < e) {
    const int first = (int)(b / chunk), last = (int)((e - 1) / chunk);
    const float* at = places + (int64_t)s * words;
    for (int c0 = first + group; c0 <= last; c0 += groups * kBatch) {
      f32x4 v[kBatch];
      i32x4 m[kBatch];
      int q[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const float* place = at + (int64_t)min(c0 + k * groups, last) * words;
        v[k] = *reinterpret_cast<const f32x4*>(place + col);
        m[k] = *reinterpret_cast<const i32x4*>(place + cols + col);
        q[k] = reinterpret_cast<const int*>(place)[2 * cols];
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k)
        if (c0 + k * groups <= last) {
          p += v[k];
          n += m[k];
          len += q[k];
        }
    }
  }
  // the groups of a wavefront, then the wavefronts
  auto over = [&](auto add) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      p[j] = __uint_as_float(add(__float_as_uint(p[j]), [](uint32_t x, uint32_t y) {
        return __float_as_uint(__uint_as_float(x) + __uint_as_float(y));
      }));
      n[j] = (int)add((uint32_t)n[j], [](uint32_t x, uint32_t y) { return x + y; });
    }
    len = (int)add((uint32_t)len, [](uint32_t x, uint32_t y) { return x + y; });
  };
  if (quads < 32)
    over([](uint32_t v, auto op) {
      const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
      return op(r[0], r[1]);
    });
  if (quads < 64)
    over([](uint32_t v, auto op) {
      const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
      return op(r[0], r[1]);
    });
  sums[wave][lane] = p;
  counts[wave][lane] = n;
  if (lane == 0) lens[wave] = len;
  __syncthreads();
  const int wide = quads > 64 ? 2 : 1;   // wavefronts of a row of columns
  if (wide == 1 && wave > 0) return;
  const int half = wave & (wide - 1);
  p = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  n = i32x4{0, 0, 0, 0};
  len = 0;
  for (int w0 = half; w0 < waves; w0 += 4 * wide) {   // (four loads at once; waves is a multiple of wide)
    f32x4 v[4];
    i32x4 m[4];
    int q[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int w = min(w0 + k * wide, waves - wide + half);
      v[k] = sums[w][lane];
      m[k] = counts[w][lane];
      q[k] = lens[w];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (w0 + k * wide < waves) {
        p += v[k];
        n += m[k];
        len += q[k];
      }
  }
  float term[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int i = 4 * tid + j;
    const bool in = i < a.N && tid < quads;
    term[j] = in ? (float)n[j] * p[j] : 0.0f;
    if (in) {
      o.counts[(int64_t)s * a.N + i] = n[j];
      if (o.prob_sum) o.prob_sum[(int64_t)s * a.N + i] = p[j];
    }
  }
  float dot = sum_of<64>(sum_run<4>(term));
  if (wide == 2) {
    if (lane == 0 && wave < 2) dots[wave] = dot;
    __syncthreads();
    dot = dots[0] + dots[1];
  }
  if (tid != 0) return;
  o.tokens[s] = len;
  o.loss[s] = balance_of(a, dot, len);
}

__global__ void balance_zero_kernel(BalanceOut o, int S, int N) {
  const int64_t step = (int64_t)gridDim.x * blockDim.x;
  for (int64_t at = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; at < (int64_t)S * N; at += step) {
    if (at < S) {
      o.loss[at] = 0.0f;
      o.tokens[at] = 0;
    }
    o.counts[at] = 0;
    if (o.prob_sum) o.prob_sum[at] = 0.0f;
  }
}

struct BalanceBwdArgs {
  const int32_t *counts, *tokens;
  const float* d_loss;
  void* d_logits;
  int64_t d_ld;
};

// The sequence of the token that the lane's L lanes hold, as sequence_of; L starts at once.
template <int L>
__device__ __forceinline__ int sequence_of_lanes(const BalanceArgs& a, int64_t t) {
  if (!a.start) return 0;
  const int lane = threadIdx.x & (L - 1), shift = threadIdx.x & 63 & ~(L - 1);
  auto bits = [&](uint64_t m) { return __popcll(L == 64 ? m : (m >> shift) & ((uint64_t(1) << (L & 63)) - 1)); };
  if (a.S < L) return bits(__ballot(a.start[min(lane, a.S)] <= t && lane <= a.S)) - 1;
  int lo = 0, hi = a.S + 1;
  while (hi > lo) {
    const int step = (hi - lo + L - 1) / L, at = lo + lane * step;
    const int c = bits(__ballot(at < hi && a.start[at] <= t));
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

// Every token with its own sequence.
template <int L, int C, bool WHOLE, typename TL, bool SOFTMAX, bool ADD>
__global__ void __launch_bounds__(kThreads) balance_bwd_kernel(BalanceArgs a, BalanceBwdArgs w) {
  constexpr int kTokens = 64 / L, kBlock = kWaves * kTokens;
  const int lane = threadIdx.x & (L - 1), slot = (threadIdx.x & 63) / L, wave = threadIdx.x >> 6;
  for (int64_t t = (int64_t)blockIdx.x * kBlock + wave * kTokens + slot; t < a.T; t += (int64_t)gridDim.x * kBlock) {
    float l[C][4], rest[C][4], pull[C][4];
    Four<WHOLE, TL> raw[C];
    Four<WHOLE, int32_t> raw_counts[C];
    int pick[kPicks<L>];
    load_token<L, C, WHOLE>(static_cast<const TL*>(a.logits) + t * a.ld, a.N, lane, raw);
    load_picks<L>(a, t, lane, pick);
    const int s = sequence_of_lanes<L>(a, t), at = s < 0 ? 0 : s < a.S ? s : a.S - 1;
    const float len = (float)w.tokens[at], d_loss = w.d_loss[at];
#pragma unroll
    for (int c = 0; c < C; ++c) raw_counts[c] = four_at<WHOLE>(w.counts + (int64_t)at * a.N, 4 * (c * L + lane), a.N);
    bool some = false;
#pragma unroll
    for (int h = 0; h < kPicks<L>; ++h) some |= pick[h] >= 0 && pick[h] < a.N;
    const bool real = max_of<L>((uint32_t)some) != 0 && s == at;
    unpack_token<L, C, WHOLE>(raw, a.N, lane, l);
    shares<L, C, SOFTMAX>(l, rest);
#pragma unroll
    for (int c = 0; c < C; ++c)   // (behind the row's end p is 0)
#pragma unroll
      for (int j = 0; j < 4; ++j) pull[c][j] = (float)(int32_t)raw_counts[c].w[j];
    float part[C];
#pragma unroll
    for (int c = 0; c < C; ++c) {
      float q[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) q[j] = l[c][j] * pull[c][j];
      part[c] = sum_run<4>(q);
    }
    const float dot = sum_of<L>(sum_run<C>(part));
    const float each = real && len > 0.0f ? d_loss * a.alpha * ((float)a.N / ((float)a.K * len)) / len : 0.0f;
    TL* row = static_cast<TL*>(w.d_logits) + t * w.d_ld;
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const int first = 4 * (c * L + lane);
      float d[4], was[4];
      if constexpr (ADD) values(four_at<WHOLE>(row, first, a.N), first, a.N, 0.0f, was);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        d[j] = l[c][j] * (each * (pull[c][j] - dot));
        if constexpr (!SOFTMAX) d[j] *= rest[c][j];
        if (!real) d[j] = 0.0f;   // (whatever its logits are)
        if constexpr (ADD) d[j] += was[j];
      }
      if (first < a.N && (!ADD || real)) store_run4(row + first, WHOLE ? 4 : a.N - first, d);
    }
  }
}

// (any other number of experts than a multiple of four: 64 lanes whatever their number, one kernel in place of four)
int lanes_of(int n) { return n % 4 != 0 ? 64 : n <= 128 ? 16 : n <= 256 ? 32 : 64; }

// Tokens of a workgroup of the forward pass: whole blocks of what its wavefronts hold at once
int chunk_of(const moe_balance_config& c) {
  const int64_t block = kPartWaves * (64 / lanes_of(c.n_routed));
  return (int)(block * std::max<int64_t>(1, ceil_div(ceil_div(c.tokens, block), kPlaces)));
}

BalanceArgs args_of(const moe_balance_config& c, const void* logits, const int32_t* idx, const int32_t* start) {
  return {logits, c.logits_ld ? c.logits_ld : c.n_routed, idx, start, c.tokens, c.n_routed, c.top_k, c.n_seqs, c.alpha};
}

// f(lanes of a token, runs of four a lane, whether runs are whole) as integral constants
template <typename F>
hipError_t with_lanes(int n, F f) {
  using std::bool_constant;
  using std::integral_constant;
  if (n % 4 != 0) return f(integral_constant<int, 64>{}, integral_constant<int, 2>{}, bool_constant<false>{});
  if (n <= 64) return f(integral_constant<int, 16>{}, integral_constant<int, 1>{}, bool_constant<true>{});
  if (n <= 128) return f(integral_constant<int, 16>{}, integral_constant<int, 2>{}, bool_constant<true>{});
  if (n <= 256) return f(integral_constant<int, 32>{}, integral_constant<int, 2>{}, bool_constant<true>{});
  return f(integral_constant<int, 64>{}, integral_constant<int, 2>{}, bool_constant<true>{});
}

// One kernel, a workgroup a sequence, for few tokens: a block of them costs such a workgroup 0.75 us (1.5 us where a lane has
// two runs), and two kernels cost more the more sequences there are.  How the tokens are shared out is not known here.  In a
// graph, us with the gradient, one kernel against two, cut at random, evenly, and all tokens in one sequence; blocks of 64 tokens
// of 64 experts: 1 sequence: 4 blocks 8.0, 9.3; 6 9.4, 9.4; 8 10.9, 9.4.  3 sequences: 8 blocks 8.2, 10.5; 7.3, 10.6; 10.9, 9.4; 12
// blocks 10.5, 10.6; 8.3, 9.6; 13.9, 9.7.  7: 16 blocks 10.1, 11.4; 7.4, 10.7; 17.0, 9.8; 24 blocks 10.5, 10.7; 8.2, 10.6; 23.0,
// 9.9.  15: 32 blocks 11.5, 11.8; 7.5, 10.8; 28.8, 9.9.  64: 32 blocks 7.2, 18.0; 6.7, 12.1; 29.0, 10.6.  256 experts, sigmoid, half
// the blocks (of 32 tokens): 7 sequences, 8 blocks 10.9, 13.7; 8.5, 12.1; 18.7, 11.0; 64, 16 blocks 8.8, 22.6; 7.6, 16.4; 29.6, 12.5.
// So random cuts of 1, 3, 7 and 15 sequences are even at 6, 12, 24 and 32 blocks; the rule stays at two thirds of that up to 7
// sequences, which bounds what a batch loses whose tokens are all in one of them: 1.7 times up to 7 sequences, 2.9 beyond.
bool few_tokens(const moe_balance_config& c) {
  const int runs = c.n_routed <= 64 && c.n_routed % 4 == 0 ? 1 : 2;
  const int64_t blocks = ceil_div(c.tokens, kPartWaves * (64 / lanes_of(c.n_routed)));
  return blocks * runs <= std::min<int64_t>(2 * (int64_t)c.n_seqs + 2, 32) && c.n_seqs <= 4096;
}

template <typename TL, bool SOFTMAX>
hipError_t few_t(const BalanceArgs& a, const BalanceOut& o, hipStream_t st) {
  const size_t lds = (size_t)(kPartWaves * a.N + a.N + 4) * 4;
  return with_lanes(a.N, [&](auto l, auto c, auto whole) {
    return launch_kernel(balance_few_kernel<decltype(l)::value, decltype(c)::value, decltype(whole)::value, TL, SOFTMAX>,
                         dim3((unsigned)a.S), dim3(kPartThreads), lds, st, a, o);
  });
}

template <typename TL, bool SOFTMAX>
hipError_t part_t(const BalanceArgs& a, int chunk, float* places, hipStream_t st) {
  const size_t lds = (size_t)(kPartWaves * a.N + a.N + 4) * 4;
  return with_lanes(a.N, [&](auto l, auto c, auto whole) {
    return launch_kernel(balance_part_kernel<decltype(l)::value, decltype(c)::value, decltype(whole)::value, TL, SOFTMAX>,
                         dim3((unsigned)ceil_div(a.T, chunk)), dim3(kPartThreads), lds, st, a, chunk, places);
  });
}

template <typename TL, bool SOFTMAX, bool ADD>
hipError_t bwd_t(const BalanceArgs& a, const BalanceBwdArgs& w, hipStream_t st) {
  const unsigned grid = (unsigned)std::min<int64_t>(ceil_div(a.T, kWaves * (64 / lanes_of(a.N))), 1 << 16);
  return with_lanes(a.N, [&](auto l, auto c, auto whole) {
    return launch_kernel(balance_bwd_kernel<decltype(l)::value, decltype(c)::value, decltype(whole)::value, TL, SOFTMAX, ADD>,
                         dim3(grid), dim3(kThreads), 0, st, a, w);
  });
}

template <typename TL>
hipError_t bwd_l(const BalanceArgs& a, const BalanceBwdArgs& w, bool softmax, bool add, hipStream_t st) {
  if (softmax) return add ? bwd_t<TL, true, true>(a, w, st) : bwd_t<TL, true, false>(a, w, st);
  return add ? bwd_t<TL, false, true>(a, w, st) : bwd_t<TL, false, false>(a, w, st);
}

}  // namespace

// What any batch of up to so many tokens and sequences needs: chunks of whole blocks, kPlaces of them at most, and a place more
// for each sequence.  (None where one kernel does all, for these sequences and for a single one.)
size_t balance_workspace(const moe_balance_config& c) {
  moe_balance_config one = c;
  one.n_seqs = 1;
  if (c.tokens == 0 || (few_tokens(c) && few_tokens(one))) return 0;
  const int64_t blocks = ceil_div(c.tokens, kPartWaves * (64 / lanes_of(c.n_routed)));
  return (size_t)(std::min<int64_t>(blocks, kPlaces) + c.n_seqs) * place_words(c.n_routed) * 4;
}

bool balance_in_one_kernel(const moe_balance_config& c) { return c.tokens == 0 || few_tokens(c); }

hipError_t launch_balance_loss(const moe_balance_config& c, const void* logits, const int32_t* idx, const int32_t* start,
                               float* loss, int32_t* counts, int32_t* tokens, float* prob_sum, float* places,
                               hipStream_t st) {
  const BalanceArgs a = args_of(c, logits, idx, start);
  const BalanceOut o{loss, counts, tokens, prob_sum};
  if (c.tokens == 0) {
    const int64_t blocks = std::min<int64_t>(ceil_div((int64_t)c.n_seqs * c.n_routed, 256), 1 << 16);
    return launch_kernel(balance_zero_kernel, dim3((unsigned)blocks), dim3(256), 0, st, o, c.n_seqs, c.n_routed);
  }
  const bool f32 = c.logits_dtype == MOE_DTYPE_F32;
  hipError_t err;
  if (few_tokens(c)) {
    if (c.score == MOE_SCORE_SOFTMAX) return f32 ? few_t<float, true>(a, o, st) : few_t<uint16_t, true>(a, o, st);
    return f32 ? few_t<float, false>(a, o, st) : few_t<uint16_t, false>(a, o, st);
  }
  const int chunk = chunk_of(c);
  if (c.score == MOE_SCORE_SOFTMAX)
    err = f32 ? part_t<float, true>(a, chunk, places, st) : part_t<uint16_t, true>(a, chunk, places, st);
  else
    err = f32 ? part_t<float, false>(a, chunk, places, st) : part_t<uint16_t, false>(a, chunk, places, st);
  if (err != hipSuccess) return err;
  int quads = 16;
  while (4 * quads < c.n_routed) quads *= 2;
  // groups of columns: about as many as an average sequence has places
  unsigned threads = kJoinThreads;
  while (threads > 128 && (int64_t)(threads / quads) * chunk * c.n_seqs > 2 * (int64_t)c.tokens) threads /= 2;
  return launch_kernel(balance_join_kernel, dim3((unsigned)c.n_seqs), dim3(threads), 0, st, a, chunk, places, o, quads);
}

hipError_t launch_balance_backward(const moe_balance_config& c, const void* logits, const int32_t* idx, const int32_t* start,
                                   const int32_t* counts, const int32_t* tokens, const float* d_loss, void* d_logits,
                                   int64_t d_ld, bool add, hipStream_t st) {
  if (c.tokens == 0) return hipSuccess;
  const BalanceArgs a = args_of(c, logits, idx, start);
  const BalanceBwdArgs w{counts, tokens, d_loss, d_logits, d_ld ? d_ld : c.n_routed};
  const bool softmax = c.score == MOE_SCORE_SOFTMAX;
  return c.logits_dtype == MOE_DTYPE_F32 ? bwd_l<float>(a, w, softmax, add, st) : bwd_l<uint16_t>(a, w, softmax, add, st);
}

}  // namespace moe
