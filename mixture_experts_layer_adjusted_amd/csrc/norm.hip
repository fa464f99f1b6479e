// The residual's addition and the root-mean-square norm behind it, with an 8-bit output, and its gradient.
//
// Forward, for a row of n values:
//   h = x + r, rounded to the stream's type (it is kept, and the backward pass reads it);
//   rstd = 1 / sqrt(sum h^2 / n + eps);  y = h rstd w;
//   a run of 128 of y: scale = amax / 448 (1 for zeros), code = E4M3 of the fp32 quotient y / scale, as quant_act_kernel
//   (bias_quant.hip) has them, from y in fp32 and not from its bf16 rounding.
// Backward, with g = dy w and u = h rstd:
//   dh = rstd (g - u sum(g u) / n) + what arrives at h from behind;  dw = sum over the rows of dy u.
// Squares, sums, y and the gradients are fp32.
//
// A row lies in the registers of one wavefront (up to 2048 values) or of one workgroup, eight neighbouring values a lane
// and load, so that it is read once; which of the two goes by the row's length alone, so a row's results are the same bits
// in every batch.  16 lanes hold a run of 128.  The weight's gradient: every thread sums its own columns over the
// workgroup's rows, the workgroups' sums are joined in a fixed order by a second kernel.
// Bound by memory.
#include "fp8_codec.h"
#include "lanes.h"
#include "moe_internal.h"
#include "rows.h"

namespace moe {
namespace {

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

// The sum of v over the row's lanes.  WAVE: the row's own wavefront.  Otherwise the workgroup: the wavefronts' sums
// meet in LDS (`at` alternates between two places, so that one barrier a row is enough).
template <bool WAVE>
__device__ __forceinline__ float row_sum(float v, float (&place)[2][16], int at) {
  v = sum_of<64>(v);
  if constexpr (WAVE) return v;
  const int waves = blockDim.x >> 6;
  if ((threadIdx.x & 63) == 0) place[at][threadIdx.x >> 6] = v;
  __syncthreads();
  float s = 0.0f;
  for (int w = 0; w < waves; ++w) s += place[at][w];
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

// V vectors of eight a lane; WAVE: a row to a wavefront
template <typename T, int V, bool WAVE>
__global__ void __launch_bounds__(WAVE ? 256 : 1024) norm_fwd_kernel(NormArgs a) {
  __shared__ float place[2][16];
  const int lanes = WAVE ? 64 : blockDim.x, lane = WAVE ? threadIdx.x & 63 : threadIdx.x;
  const int per = WAVE ? blockDim.x >> 6 : 1;   // rows of the workgroup at a time
  const int first = WAVE ? threadIdx.x >> 6 : 0;
  const float n = (float)a.cols;
  int at = 0;
  for (int64_t r = (int64_t)blockIdx.x * per + first; r < a.rows; r += (int64_t)gridDim.x * per, at ^= 1) {
    const T* x = static_cast<const T*>(a.x) + r * a.x_ld;
    float h[V][8];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * lanes + lane) * 8;
      if (c < a.cols) load8(x + c, h[j]);
      else
#pragma unroll
        for (int i = 0; i < 8; ++i) h[j][i] = 0.0f;
    }
    if (a.residual) {
      const T* res = static_cast<const T*>(a.residual) + r * a.x_ld;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = (j * lanes + lane) * 8;
        float v[8];
        if (c < a.cols) {
          load8(res + c, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) h[j][i] += v[i];
          round8<T>(h[j]);
        }
      }
    }
    float part[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      float sq[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) sq[i] = h[j][i] * h[j][i];
      part[j] = sum_run<8>(sq);
    }
    const float rstd = 1.0f / sqrtf(row_sum<WAVE>(sum_run<V>(part), place, at) / n + a.eps);
    if (a.rstd && lane == 0) a.rstd[r] = rstd;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * lanes + lane) * 8;
      const bool in = c < a.cols;   // (with codes: of the 16 lanes of a run all or none)
      if (!in) continue;
      if (a.sum) store8(static_cast<T*>(a.sum) + r * a.x_ld + c, h[j]);
      float w[8], y[8];
      load8(a.weight + c, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = h[j][i] * rstd * w[i];
      if (a.y) store8(static_cast<T*>(a.y) + r * a.y_ld + c, y);
      if (a.codes) {
        const float amax = run_amax(y);
        const float scale = amax > 0.0f ? __fdiv_rn(amax, 448.0f) : 1.0f;
        *reinterpret_cast<uint2*>(a.codes + r * a.cols + c) = e4m3_codes8(y, scale);
        if ((lane & 15) == 0) a.scales[r * (a.cols / 128) + c / 128] = scale;
      }
    }
  }
}

struct NormBwdArgs {
  const void *d_y, *d_sum, *h;
  const float *weight, *rstd;
  void* d_x;
  float* parts;   // [gridDim.x * rows at a time, cols], or null
  int64_t rows, x_ld, y_ld;
  int cols;
};

template <typename T, int V, bool WAVE>
__global__ void __launch_bounds__(WAVE ? 256 : 1024) norm_bwd_kernel(NormBwdArgs a) {
  __shared__ float place[2][16];
  const int lanes = WAVE ? 64 : blockDim.x, lane = WAVE ? threadIdx.x & 63 : threadIdx.x;
  const int per = WAVE ? blockDim.x >> 6 : 1;
  const int first = WAVE ? threadIdx.x >> 6 : 0;
  const float n = (float)a.cols;
  float dw[V][8];
#pragma unroll
  for (int j = 0; j < V; ++j)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[j][i] = 0.0f;
  int at = 0;
  for (int64_t r = (int64_t)blockIdx.x * per + first; r < a.rows; r += (int64_t)gridDim.x * per, at ^= 1) {
    const T* h = static_cast<const T*>(a.h) + r * a.x_ld;
    const T* d_y = static_cast<const T*>(a.d_y) + r * a.y_ld;
    const float rstd = a.rstd[r];
    float u[V][8], g[V][8], part[V];
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * lanes + lane) * 8;
      part[j] = 0.0f;
      if (c < a.cols) {
        float w[8], p[8];
        load8(h + c, u[j]);
        load8(d_y + c, g[j]);
        load8(a.weight + c, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          u[j][i] *= rstd;
          dw[j][i] = fmaf(g[j][i], u[j][i], dw[j][i]);
          g[j][i] *= w[i];
          p[i] = g[j][i] * u[j][i];
        }
        part[j] = sum_run<8>(p);
      }
    }
    const float mean = row_sum<WAVE>(sum_run<V>(part), place, at) / n;
    T* d_x = static_cast<T*>(a.d_x) + r * a.x_ld;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = (j * lanes + lane) * 8;
      if (c >= a.cols) continue;
      float d[8];
      if (a.d_sum) load8(static_cast<const T*>(a.d_sum) + r * a.x_ld + c, d);
      else
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) d[i] += rstd * (g[j][i] - u[j][i] * mean);
      store8(d_x + c, d);
    }
  }
  if (!a.parts) return;
  float* mine = a.parts + ((int64_t)blockIdx.x * per + first) * a.cols;
#pragma unroll
  for (int j = 0; j < V; ++j) {
    const int c = (j * lanes + lane) * 8;
    if (c < a.cols) store8(mine + c, dw[j]);
  }
}

// d_weight from `count` rows of partial sums: 64 columns a workgroup, its 16 wavefronts every 16th row
__global__ void __launch_bounds__(1024) norm_join_kernel(const float* __restrict__ parts, int count, int cols,
                                                         float* __restrict__ d_weight) {
  __shared__ float place[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, c = blockIdx.x * 64 + lane;
  float s = 0.0f;
  if (c < cols)
    for (int p = wave; p < count; p += 16) s += parts[(int64_t)p * cols + c];
  place[wave][lane] = s;
  __syncthreads();
  if (wave != 0 || c >= cols) return;
  float v[16];
#pragma unroll
  for (int w = 0; w < 16; ++w) v[w] = place[w][lane];
  d_weight[c] = sum_run<16>(v);
}

__global__ void norm_zero_kernel(float* __restrict__ p, int n) {
  const int i = blockIdx.x * blockDim.x + threadIdx.x;
  if (i < n) p[i] = 0.0f;
}

// How a row lies on lanes: wavefronts of a row, vectors of eight a lane.  By the row's length alone.
struct NormLanes {
  int vectors;
  bool wave;
  unsigned threads;   // of a workgroup
  int per;            // rows of a workgroup at a time
};
NormLanes lanes_of(int cols) {
  const int vecs = cols / 8;
  if (vecs <= 64) return {1, true, 256, 4};
  if (vecs <= 128) return {2, true, 256, 4};
  if (vecs <= 256) return {4, true, 256, 4};
  const int v = vecs <= 2048 ? 2 : 4;
  return {v, false, (unsigned)(64 * ceil_div(vecs, 64 * v)), 1};
}

// Workgroups of a backward pass, each with its own sums of the weight's gradient: as many as keep those sums near 16 MB
int64_t norm_blocks(const NormLanes& l, int64_t rows, int cols) {
  const int64_t most = std::max<int64_t>(256, std::min<int64_t>(4096, (int64_t(1) << 22) / cols));
  return std::min<int64_t>(ceil_div(rows, l.per), most / l.per);
}

template <typename T>
hipError_t norm_forward_t(const NormLanes& l, const NormArgs& a, hipStream_t st) {
  const unsigned grid = (unsigned)std::min<int64_t>(ceil_div(a.rows, l.per), 1 << 20);
  if (l.wave) {
    if (l.vectors == 1) return launch_kernel(norm_fwd_kernel<T, 1, true>, dim3(grid), dim3(l.threads), 0, st, a);
    if (l.vectors == 2) return launch_kernel(norm_fwd_kernel<T, 2, true>, dim3(grid), dim3(l.threads), 0, st, a);
    return launch_kernel(norm_fwd_kernel<T, 4, true>, dim3(grid), dim3(l.threads), 0, st, a);
  }
  if (l.vectors == 2) return launch_kernel(norm_fwd_kernel<T, 2, false>, dim3(grid), dim3(l.threads), 0, st, a);
  return launch_kernel(norm_fwd_kernel<T, 4, false>, dim3(grid), dim3(l.threads), 0, st, a);
}

template <typename T>
hipError_t norm_backward_t(const NormLanes& l, const NormBwdArgs& a, unsigned grid, hipStream_t st) {
  if (l.wave) {
    if (l.vectors == 1) return launch_kernel(norm_bwd_kernel<T, 1, true>, dim3(grid), dim3(l.threads), 0, st, a);
    if (l.vectors == 2) return launch_kernel(norm_bwd_kernel<T, 2, true>, dim3(grid), dim3(l.threads), 0, st, a);
    return launch_kernel(norm_bwd_kernel<T, 4, true>, dim3(grid), dim3(l.threads), 0, st, a);
  }
  if (l.vectors == 2) return launch_kernel(norm_bwd_kernel<T, 2, false>, dim3(grid), dim3(l.threads), 0, st, a);
  return launch_kernel(norm_bwd_kernel<T, 4, false>, dim3(grid), dim3(l.threads), 0, st, a);
}

}  // namespace

size_t norm_workspace(const moe_norm_shape& s) {
  const NormLanes l = lanes_of(s.cols);
  return (size_t)(norm_blocks(l, s.rows, s.cols) * l.per) * s.cols * 4;
}

hipError_t launch_norm_forward(const moe_norm_shape& s, const void* x, const void* residual, const float* weight, void* sum,
                               void* y, uint8_t* codes, float* scales, float* rstd, hipStream_t st) {
  const NormArgs a{x,    residual, weight, sum, y, codes, scales, rstd, s.rows, s.x_ld ? s.x_ld : s.cols,
                   s.y_ld ? s.y_ld : s.cols, s.cols, s.eps};
  const NormLanes l = lanes_of(s.cols);
  return s.dtype == MOE_DTYPE_F32 ? norm_forward_t<float>(l, a, st) : norm_forward_t<uint16_t>(l, a, st);
}

hipError_t launch_norm_backward(const moe_norm_shape& s, const void* d_y, const void* d_sum, const void* h,
                                const float* weight, const float* rstd, void* d_x, float* d_weight, float* parts,
                                hipStream_t st) {
  if (s.rows == 0)
    return launch_kernel(norm_zero_kernel, dim3((unsigned)ceil_div(s.cols, 256)), dim3(256), 0, st, d_weight, s.cols);
  const NormLanes l = lanes_of(s.cols);
  const unsigned grid = (unsigned)norm_blocks(l, s.rows, s.cols);
  const NormBwdArgs a{d_y, d_sum, h, weight, rstd, d_x, d_weight ? parts : nullptr, s.rows, s.x_ld ? s.x_ld : s.cols,
                      s.y_ld ? s.y_ld : s.cols, s.cols};
  const hipError_t err =
      s.dtype == MOE_DTYPE_F32 ? norm_backward_t<float>(l, a, grid, st) : norm_backward_t<uint16_t>(l, a, grid, st);
  if (err != hipSuccess || !d_weight) return err;
  return launch_kernel(norm_join_kernel, dim3((unsigned)ceil_div(s.cols, 64)), dim3(1024), 0, st, parts,
                       (int)grid * l.per, s.cols, d_weight);
}

}  // namespace moe
