// The residual's addition and the root-mean-square norm behind it, with an 8-bit output, and its gradient.
//
// Forward, for a row of n values:
//   h = x + r, rounded to the stream's type (it is kept, and the backward pass reads it);
//   rstd = 1 / sqrt(sum h^2 / n + eps);  y = h rstd w;
//   a run of 128 of y: scale = amax / 448 (1 where that is 0), code = E4M3 of the fp32 quotient y / scale, as quant_act_kernel
//   (bias_quant.hip) has them, from y in fp32 and not from its bf16 rounding.
// Backward, with g = dy w and u = h rstd:
//   dh = rstd (g - u sum(g u) / n) + what arrives at h from behind;  dw = sum over the rows of dy u.
// Squares, sums, y and the gradients are fp32.
//
// A row lies in the registers of one wavefront (up to 2048 values) or of one workgroup, eight neighbouring values a lane
// and load, so that it is read once.  The order of its sums goes by its length alone: a row's results are the same bits in
// every batch.  16 lanes hold a run of 128.  The weight's gradient: every thread sums its own columns over the
// workgroup's rows, the workgroups' sums are joined in a fixed order by a second kernel; for few rows, further workgroups
// sum up columns in the same kernel.
// Bound by memory (traced): 16384 x 7168 in bf16, forward with y and codes 178 us for 1.06 GB (6.0 TB/s), backward 182 us for
// 0.94 GB (5.2 TB/s) and 5 us for the join; 8192 x 7168 forward with codes alone 77 us for 0.41 GB (5.4 TB/s).  Few rows by
// latency: one row of 7168 3.2 us, 77 of 2048 3.5 us.
#include "fp8_codec.h"
#include "lanes.h"
#include "moe_internal.h"
#include "rows.h"

namespace moe {
namespace {

constexpr int kParts = 256;   // workgroups at most that sum up the weight's gradient by rows: one a CU
constexpr int kMostBlocks = 1 << 21;   // of a forward pass along x, the others along y: fewer than 2^32 threads in each

struct NormArgs {
  const void *x, *residual;
  const float* weight;
  void *sum, *y;
  uint8_t* codes;
  float *scales, *rstd;
  int64_t rows, x_ld, y_ld;
  int cols;
  float eps;
};

// The sum of the lanes' V parts over the row.  WAVE: the row's own wavefront.  Otherwise the workgroup: the wavefronts'
// sums meet in LDS (`at` alternates between two places, so that one barrier a row is enough).  A wavefront with four parts a
// lane adds them up as two wavefronts with two parts each would: the same bits.
template <bool WAVE, int V>
__device__ __forceinline__ float row_sum(const float (&part)[V], float (&place)[2][16], int at) {
  if constexpr (WAVE && V == 4) return sum_of<64>(part[0] + part[2]) + sum_of<64>(part[1] + part[3]);
  const float v = sum_of<64>(sum_run<V>(part));
  if constexpr (WAVE) return v;
  const int waves = blockDim.x >> 6;
  if ((threadIdx.x & 63) == 0) place[at][threadIdx.x >> 6] = v;
  __syncthreads();
  float s = place[at][0];
  for (int w = 1; w < waves; ++w) s += place[at][w];
  return s;
}

// the quotients of eight values and the scale of their run, correctly rounded without a division each (with r the rounded
// 1 / scale and q = v r, the remainder v - q scale is exact in one fma: Markstein); scales below 2^-64, where it could
// underflow, divide
__device__ __forceinline__ uint2 e4m3_codes8(const float (&v)[8], float scale) {
  float q[8];
  if (scale >= 0x1p-64f && scale <= 0x1p64f) {
    const float r = __fdiv_rn(1.0f, scale);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      q[i] = v[i] * r;
      q[i] = fmaf(-fmaf(q[i], scale, -v[i]), r, q[i]);   // (signs so that -0 stays -0)
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(v[i], scale);
  }
  return make_uint2(e4m3x4_from_f32(q[0], q[1], q[2], q[3]), e4m3x4_from_f32(q[4], q[5], q[6], q[7]));
}

__device__ __forceinline__ float run_amax(const float (&v)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
  m = fmaxf(m, __uint_as_float(turned<0x128>(__float_as_uint(m))));   // row_ror:8, 4, 2, 1
  m = fmaxf(m, __uint_as_float(turned<0x124>(__float_as_uint(m))));
  m = fmaxf(m, __uint_as_float(turned<0x122>(__float_as_uint(m))));
  return fmaxf(m, __uint_as_float(turned<0x121>(__float_as_uint(m))));
}

// V vectors of eight a lane; MOST: threads of a workgroup at most, 64: a row to a wavefront.  One row each:
// rows that a workgroup goes through with the next one's values on their way measured 5.1 TB/s against 5.6 (16384 x 7168).
template <typename T, int V, int MOST>
__global__ void __launch_bounds__(MOST == 64 ? 256 : MOST) norm_fwd_kernel(NormArgs a) {
  constexpr bool WAVE = MOST == 64;
  __shared__ float place[2][16];
  const int lanes = WAVE ? 64 : blockDim.x, lane = WAVE ? threadIdx.x & 63 : threadIdx.x;
  const int64_t block = (int64_t)blockIdx.y * gridDim.x + blockIdx.x;
  const int64_t r = WAVE ? block * 4 + (threadIdx.x >> 6) : block;
  if (r >= a.rows) return;
  Raw8<T> x[V], res[V];
  Raw8<float> w[V];
  float h[V][8], part[V];
  // (lanes past the row's end load its first values, and drop them)
  auto column = [&](int j) {
    const int c = (j * lanes + lane) * 8;
    return c < a.cols ? c : 0;
  };
#pragma unroll
  for (int j = 0; j < V; ++j) x[j] = raw_at(static_cast<const T*>(a.x) + r * a.x_ld + column(j));
  if (a.residual) {
#pragma unroll
    for (int j = 0; j < V; ++j) res[j] = raw_at(static_cast<const T*>(a.residual) + r * a.x_ld + column(j));
  }
#pragma unroll
  for (int j = 0; j < V; ++j) w[j] = raw_at(a.weight + column(j));
#pragma unroll
  for (int j = 0; j < V; ++j) {
    unpack8(x[j], h[j]);
    if (a.residual) {
      float v[8];
      unpack8(res[j], v);
#pragma unroll
      for (int i = 0; i < 8; ++i) h[j][i] += v[i];
      round8<T>(h[j]);
    }
    float sq[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) sq[i] = h[j][i] * h[j][i];
    part[j] = (j * lanes + lane) * 8 < a.cols ? sum_run<8>(sq) : 0.0f;
  }
  const float rstd = 1.0f / sqrtf(row_sum<WAVE>(part, place, 0) / (float)a.cols + a.eps);
  if (a.rstd && lane == 0) a.rstd[r] = rstd;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (j * lanes + lane) * 8;
    const bool in = c < a.cols;   // (with codes: of the 16 lanes of a run all or none)
    if (!in) continue;
    if (a.sum) store8(static_cast<T*>(a.sum) + r * a.x_ld + c, h[j]);
    float y[8];
    unpack8(w[j], y);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] *= h[j][i] * rstd;
    if (a.y) store8(static_cast<T*>(a.y) + r * a.y_ld + c, y);
    if (a.codes) {
      const float amax = run_amax(y);
      const float share = __fdiv_rn(amax, 448.0f), scale = share > 0.0f ? share : 1.0f;   // (amax below 3.2e-43: 0)
      *reinterpret_cast<uint2*>(a.codes + r * a.cols + c) = e4m3_codes8(y, scale);
      if ((lane & 15) == 0) a.scales[r * (a.cols / 128) + c / 128] = scale;
    }
  }
}

struct NormBwdArgs {
  const void *d_y, *d_sum, *h;
  const float *weight, *rstd;
  void* d_x;
  float* parts;   // [workgroups, cols], or null
  int64_t rows, x_ld, y_ld;
  int cols;
  float* d_weight;   // where workgroups 0 to column_blocks - 1 sum up columns in place of parts
  int column_blocks;
};

// The weight's gradient of 64 bytes of neighbouring columns, for a batch of few rows: what the workgroups of the rows do
// not wait for.  Four lanes a row; every thread sums its rows, then the threads of a wavefront, then the wavefronts.
template <typename T>
__device__ __forceinline__ void sum_columns(const NormBwdArgs& a, float (&place)[16][32]) {
  constexpr int kVals = 16 / sizeof(T), kBatch = 8;   // rows loaded at once
  struct __attribute__((aligned(16))) Raw { uint4 q; };
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6, step = waves * 16;
  const int column = blockIdx.x * (4 * kVals) + (lane & 3) * kVals, at = min(column, a.cols - kVals);
  const int rows = (int)a.rows;
  const T *d_y = static_cast<const T*>(a.d_y) + at, *h = static_cast<const T*>(a.h) + at;
  float dw[kVals];
#pragma unroll
  for (int i = 0; i < kVals; ++i) dw[i] = 0.0f;
  for (int r0 = wave * 16 + (lane >> 2); r0 < rows; r0 += step * kBatch) {
    Raw g[kBatch], u[kBatch];
    float rstd[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int64_t r = min(r0 + k * step, rows - 1);
      g[k] = *reinterpret_cast<const Raw*>(d_y + r * a.y_ld);
      u[k] = *reinterpret_cast<const Raw*>(h + r * a.x_ld);
      rstd[k] = a.rstd[r];
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (r0 + k * step >= rows) break;
      const uint32_t gw[4] = {g[k].q.x, g[k].q.y, g[k].q.z, g[k].q.w}, uw[4] = {u[k].q.x, u[k].q.y, u[k].q.z, u[k].q.w};
#pragma unroll
      for (int i = 0; i < kVals; ++i) {
        auto value = [&](const uint32_t (&w)[4]) {
          if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
          else return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
        };
        dw[i] = fmaf(value(gw), value(uw) * rstd[k], dw[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kVals; ++i) {
#pragma unroll
    for (int off = 4; off < 64; off *= 2) dw[i] += __shfl_xor(dw[i], off, 64);
    if (lane < 4) place[wave][lane * kVals + i] = dw[i];
  }
  __syncthreads();
  const int c = blockIdx.x * (4 * kVals) + threadIdx.x;
  if (threadIdx.x >= 4 * kVals || c >= a.cols) return;
  float sum = place[0][threadIdx.x];
  for (int w = 1; w < waves; ++w) sum += place[w][threadIdx.x];
  a.d_weight[c] = sum;
}

// kAhead: a workgroup goes through its rows with the next one's values on their way, which lets one workgroup a CU reach what
// the memory gives (16384 x 7168, bf16, in a graph with the join: 169 us with 256 workgroups, 183 with 512, 230 with one row
// each).  Where
// the registers do not hold both rows, they are loaded one after the other.
template <typename T, int V, int MOST>
__global__ void __launch_bounds__(MOST == 64 ? 256 : MOST) norm_bwd_kernel(NormBwdArgs a) {
  constexpr bool WAVE = MOST == 64, kAhead = MOST == 512 || (WAVE && V * sizeof(T) <= 8);
  __shared__ float place[2][16];
  const int lanes = WAVE ? 64 : blockDim.x, lane = WAVE ? threadIdx.x & 63 : threadIdx.x;
  const int per = WAVE ? blockDim.x >> 6 : 1;
  const int first = WAVE ? threadIdx.x >> 6 : 0;
  const int64_t step = (int64_t)(gridDim.x - a.column_blocks) * per;
  const float n = (float)a.cols;
  if ((int)blockIdx.x < a.column_blocks) {
    __shared__ float columns[16][32];
    sum_columns<T>(a, columns);
    return;
  }
  const int64_t block = blockIdx.x - a.column_blocks;
  float dw[V][8];
  Raw8<float> w[V];
  Raw8<T> h[V], d_y[V], d_sum[V];
  float next_rstd = 0.0f;
  // (lanes past the row's end load its first values, and drop them)
  auto column = [&](int j) {
    const int c = (j * lanes + lane) * 8;
    return c < a.cols ? c : 0;
  };
  auto load = [&](int64_t r) {
    next_rstd = a.rstd[r];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      h[j] = raw_at(static_cast<const T*>(a.h) + r * a.x_ld + column(j));
      d_y[j] = raw_at(static_cast<const T*>(a.d_y) + r * a.y_ld + column(j));
    }
    if (a.d_sum) {
#pragma unroll
      for (int j = 0; j < V; ++j) d_sum[j] = raw_at(static_cast<const T*>(a.d_sum) + r * a.x_ld + column(j));
    }
  };
  int64_t r = block * per + first;
  if (kAhead && r < a.rows) load(r);
#pragma unroll
  for (int j = 0; j < V; ++j) {
    d_sum[j] = a.d_sum && kAhead ? d_sum[j] : Raw8<T>{};
    if constexpr (kAhead) w[j] = raw_at(a.weight + column(j));
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = 0.0f;
  }
  if constexpr (kAhead) {   // the weights are waited for here: in the loop that would wait for the next row as well
#pragma unroll
    for (int j = 0; j < V; ++j)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        asm volatile("" : "+v"(w[j].q[i].x), "+v"(w[j].q[i].y), "+v"(w[j].q[i].z), "+v"(w[j].q[i].w));
  }
  for (int at = 0; r < a.rows; r += step, at ^= 1) {
    if constexpr (!kAhead) {
      load(r);
#pragma unroll
      for (int j = 0; j < V; ++j) w[j] = raw_at(a.weight + column(j));
    }
    const float rstd = next_rstd;
    float u[V][8], g[V][8], part[V];
    Raw8<T> behind[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float p[8], wv[8];
      unpack8(w[j], wv);
      unpack8(h[j], u[j]);
      unpack8(d_y[j], g[j]);
      behind[j] = d_sum[j];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        u[j][i] *= rstd;
        dw[j][i] = fmaf(g[j][i], u[j][i], dw[j][i]);
        g[j][i] *= wv[i];
        p[i] = g[j][i] * u[j][i];
      }
      part[j] = (j * lanes + lane) * 8 < a.cols ? sum_run<8>(p) : 0.0f;
    }
    if (kAhead && r + step < a.rows) load(r + step);
    const float mean = row_sum<WAVE>(part, place, at) / n;
    T* d_x = static_cast<T*>(a.d_x) + r * a.x_ld;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * lanes + lane) * 8;
      if (c >= a.cols) continue;
      float d[8];
      unpack8(behind[j], d);
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] += rstd * (g[j][i] - u[j][i] * mean);
      store8(d_x + c, d);
    }
  }
  if (!a.parts) return;
  float* mine = a.parts + block * a.cols;
  if constexpr (WAVE) {   // the four wavefronts' sums, in their order
    __shared__ float sums[4][V * 512];
#pragma unroll
    for (int j = 0; j < V; ++j) store8(&sums[first][(j * 64 + lane) * 8], dw[j]);
    __syncthreads();
    for (int c = threadIdx.x * 4; c < a.cols; c += 1024) {
      f32x4 v = *reinterpret_cast<f32x4*>(&sums[0][c]);
#pragma unroll
      for (int w = 1; w < 4; ++w) v += *reinterpret_cast<f32x4*>(&sums[w][c]);
      *reinterpret_cast<f32x4*>(mine + c) = v;
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * lanes + lane) * 8;
      if (c < a.cols) store8(mine + c, dw[j]);
    }
  }
}

// d_weight from `count` rows of partial sums: 16 columns a workgroup, 64 threads a column, every 64th row a thread
__global__ void __launch_bounds__(1024) norm_join_kernel(const float* __restrict__ parts, int count, int cols,
                                                         float* __restrict__ d_weight) {
  __shared__ float place[16][16];
  constexpr int kBatch = 8;   // rows loaded at once
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = blockIdx.x * 16 + (lane & 15);
  const int at = wave * 4 + (lane >> 4);
  float s = 0.0f;
  for (int p0 = at; p0 < count; p0 += 64 * kBatch) {
    float v[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) v[b] = parts[(int64_t)min(p0 + 64 * b, count - 1) * cols + min(c, cols - 1)];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) s += p0 + 64 * b < count ? v[b] : 0.0f;
  }
  s += __shfl_xor(s, 16, 64);
  s += __shfl_xor(s, 32, 64);
  if (lane < 16) place[wave][lane] = s;
  __syncthreads();
  if (threadIdx.x >= 16 || c >= cols) return;
  float v[16];
#pragma unroll
  for (int w = 0; w < 16; ++w) v[w] = place[w][lane];
  d_weight[c] = sum_run<16>(v);
}

__global__ void norm_zero_kernel(float* __restrict__ p, int n) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) p[i] = 0.0f;
}

// How a row lies on lanes: a wavefront up to 2048 values, a workgroup of up to 512 threads up to 8192, of up to 1024
// beyond; vectors of eight a lane.  By the row's length alone.
struct NormLanes {
  int vectors, most;
  unsigned threads;   // of a workgroup
  int per;            // rows of a workgroup at a time
};
NormLanes lanes_of(int cols) {
  const int vecs = cols / 8;
  if (vecs <= 256) return {vecs <= 64 ? 1 : vecs <= 128 ? 2 : 4, 64, 256, 4};
  const int v = vecs <= 2048 ? 2 : 4;
  return {v, vecs <= 1024 ? 512 : 1024, (unsigned)(64 * ceil_div(vecs, 64 * v)), 1};
}

// f(vectors, most) as integral constants
template <typename F>
hipError_t with_lanes(const NormLanes& l, F f) {
  using std::integral_constant;
  if (l.most == 64) {
    if (l.vectors == 1) return f(integral_constant<int, 1>{}, integral_constant<int, 64>{});
    if (l.vectors == 2) return f(integral_constant<int, 2>{}, integral_constant<int, 64>{});
    return f(integral_constant<int, 4>{}, integral_constant<int, 64>{});
  }
  if (l.most == 512) return f(integral_constant<int, 2>{}, integral_constant<int, 512>{});
  if (l.vectors == 2) return f(integral_constant<int, 2>{}, integral_constant<int, 1024>{});
  return f(integral_constant<int, 4>{}, integral_constant<int, 1024>{});
}

// Workgroups of a backward pass that sums up the weight's gradient by rows, each with its own sums: half as many for few rows
// of a workgroup each, whose sums cost as much as the rows (7168 values in bf16, us with the second kernel, 128 workgroups
// against 256: 512 rows 13.1, 14.9; 700 rows 14.7, 14.8; 1024 rows 17.5, 17.0; but rows of a wavefront, 1408 values in
// fp32: 600 rows 8.7, 7.3; 1021 rows 9.7, 9.0)
int64_t norm_blocks(const NormLanes& l, int64_t rows) {
  const int64_t each = ceil_div(rows, l.per);
  return std::min<int64_t>(each, l.per == 1 && each <= 5 * (kParts / 2) ? kParts / 2 : kParts);
}

// Up to so many rows and bytes of them, the weight's gradient is summed by columns in the kernel of the rows: one launch in
// place of two, against reading dy and h twice.  In a graph, us, one against two: 1408 in fp32: 1 row 2.5, 4.7; 300 rows 4.5,
// 6.1; 512 rows 6.9, 6.8; 1021 rows 11.8, 8.9.  7168 in bf16: 64 rows 4.8, 7.4; 384 rows 11.0, 10.7; in fp32 300 rows 13.7,
// 13.8; 384 rows 17.8, 14.5.
bool by_columns(const moe_norm_shape& s) {
  return s.rows <= 384 && (int64_t)s.rows * s.cols * (s.dtype == MOE_DTYPE_F32 ? 4 : 2) <= (8 << 20);
}

// Rows of 1025 to 2048 values, up to 4096 of them: two wavefronts a row, more loads at once (in a graph, us, two
// wavefronts against one: 1 x 2048 2.8, 3.5; 77 x 2048 3.1, 4.0; 4096 x 2048 11.0, 11.7; 65536 x 2048 166, 163)
NormLanes forward_lanes_of(int cols, int64_t rows) {
  const NormLanes l = lanes_of(cols);
  return l.most == 64 && l.vectors == 4 && rows <= 4096 ? NormLanes{2, 512, 128, 1} : l;
}

template <typename T>
hipError_t norm_forward_t(const NormLanes& l, const NormArgs& a, hipStream_t st) {
  const int64_t blocks = ceil_div(a.rows, l.per);
  const dim3 grid((unsigned)std::min<int64_t>(blocks, kMostBlocks), (unsigned)ceil_div(blocks, kMostBlocks));
  return with_lanes(l, [&](auto v, auto most) {
    return launch_kernel(norm_fwd_kernel<T, decltype(v)::value, decltype(most)::value>, grid, dim3(l.threads), 0, st, a);
  });
}

template <typename T>
hipError_t norm_backward_t(const NormLanes& l, const NormBwdArgs& a, unsigned grid, hipStream_t st) {
  return with_lanes(l, [&](auto v, auto most) {
    return launch_kernel(norm_bwd_kernel<T, decltype(v)::value, decltype(most)::value>, dim3(grid), dim3(l.threads), 0, st, a);
  });
}

}  // namespace

size_t norm_workspace(const moe_norm_shape& s) {
  const NormLanes l = lanes_of(s.cols);
  return by_columns(s) ? 0 : (size_t)norm_blocks(l, s.rows) * s.cols * 4;
}

hipError_t launch_norm_forward(const moe_norm_shape& s, const void* x, const void* residual, const float* weight, void* sum,
                               void* y, uint8_t* codes, float* scales, float* rstd, hipStream_t st) {
  const NormArgs a{x,    residual, weight, sum, y, codes, scales, rstd, s.rows, s.x_ld ? s.x_ld : s.cols,
                   s.y_ld ? s.y_ld : s.cols, s.cols, s.eps};
  const NormLanes l = forward_lanes_of(s.cols, s.rows);
  return s.dtype == MOE_DTYPE_F32 ? norm_forward_t<float>(l, a, st) : norm_forward_t<uint16_t>(l, a, st);
}

hipError_t launch_norm_backward(const moe_norm_shape& s, const void* d_y, const void* d_sum, const void* h,
                                const float* weight, const float* rstd, void* d_x, float* d_weight, float* parts,
                                hipStream_t st) {
  if (s.rows == 0)
    return launch_kernel(norm_zero_kernel, dim3((unsigned)ceil_div(s.cols, 256)), dim3(256), 0, st, d_weight, s.cols);
  const NormLanes l = lanes_of(s.cols);
  const bool columns = by_columns(s);
  const int elem = s.dtype == MOE_DTYPE_F32 ? 4 : 2;
  const int column_blocks = columns && d_weight ? (int)ceil_div(s.cols * elem, 64) : 0;
  const unsigned blocks = (unsigned)(columns ? ceil_div(s.rows, l.per) : norm_blocks(l, s.rows));
  const NormBwdArgs a{d_y, d_sum, h, weight, rstd, d_x, d_weight && !columns ? parts : nullptr, s.rows,
                      s.x_ld ? s.x_ld : s.cols, s.y_ld ? s.y_ld : s.cols, s.cols, d_weight, column_blocks};
  const unsigned grid = blocks + column_blocks;
  const hipError_t err =
      s.dtype == MOE_DTYPE_F32 ? norm_backward_t<float>(l, a, grid, st) : norm_backward_t<uint16_t>(l, a, grid, st);
  if (err != hipSuccess || !d_weight || columns) return err;
  return launch_kernel(norm_join_kernel, dim3((unsigned)ceil_div(s.cols, 16)), dim3(1024), 0, st, parts,
                       (int)blocks, s.cols, d_weight);
}

}  // namespace moe
