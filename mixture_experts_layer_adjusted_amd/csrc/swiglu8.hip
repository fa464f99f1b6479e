// SwiGLU whose inputs are kept for the backward pass in 8 bits.
//
// Forward, for a row's inputs a[I] and b[I]:  h = a sg(a) b, sg(a) = 1 / (1 + exp(-a)).  Kept: for every run of
// 128 values of a and of b, scale = amax times fp32(1 / 127) (1 for a run of zeros) and code = the integer nearest to
// x / scale (even at a half), -127..127.  Backward, with a~ = code scale and b~ likewise:
//   dA = dh b~ sg(a~) (1 + a~ (1 - sg(a~))),   dB = dh a~ sg(a~),   H = a~ sg(a~) b~.
// Integers and not E4M3: what reaches the gradients is the absolute error of a and b, which the integers keep at
// amax / 254 over the run, against x / 16 for E4M3's values (for normal values 0.6% of their size against 2.3%).
// A run with an infinity or NaN gets the scale NaN, so that its gradients are NaN and not plausible numbers.
//
// The layer's rows (moe_forward_train8, moe_backward_gates) are those of the permuted layout: as many as *row_end says;
// the backward pass weighs dh by the row's gate, writes padding rows (row_token < 0) as zeros and hands back, for every
// row and run, the sum of dh H before the gate (its share of the gate's gradient).
//
// 16 lanes share one run of 128 features of a row, 8 features a lane: 16-byte loads and stores, the run's amax by
// four row rotations.  Bound by memory: 32768 x 2048, forward 100 to 114 us for 541 MB, backward 116 to 121 us for 675 MB.
#include "moe_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const uint32_t a = __float_as_uint(lo), b = __float_as_uint(hi);
  const uint32_t x = lo != lo ? 0x7FC0u : (a + 0x7FFFu + ((a >> 16) & 1u)) >> 16;
  const uint32_t y = hi != hi ? 0x7FC00000u : (b + 0x7FFFu + ((b >> 16) & 1u)) & 0xFFFF0000u;
  return x | y;
}

__device__ __forceinline__ void unpack8(const uint4& q, float (&v)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
}

template <int CTRL>
__device__ __forceinline__ uint32_t rotated(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, false);
}

// the run's scale: the largest magnitude as bits (a NaN's are above infinity's, those above every number's)
__device__ __forceinline__ float run_scale(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  m = max(m, rotated<0x128>(m));   // row_ror:8, 4, 2, 1: all 16 lanes get the row's largest
  m = max(m, rotated<0x124>(m));
  m = max(m, rotated<0x122>(m));
  m = max(m, rotated<0x121>(m));
  if (m >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
  return m == 0u ? 1.0f : __uint_as_float(m) * (1.0f / 127.0f);
}

// The codes of a lane's eight values.  The quotients are correctly rounded without a division each: with r the
// rounded 1 / scale and q = x r, the remainder e = x - q scale is exact in one fma and q + e r is the rounded quotient
// (Markstein).  Scales below 2^-64, where the remainder could underflow, divide (and a subnormal scale is so coarse
// that its quotients can pass 127).
__device__ __forceinline__ uint2 code8(const float (&v)[8], float scale) {
  float q[8];
  if (scale >= 0x1p-64f) {
    const float r = __fdiv_rn(1.0f, scale);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      q[i] = v[i] * r;
      q[i] = fmaf(fmaf(-q[i], scale, v[i]), r, q[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] = fminf(fmaxf(__fdiv_rn(v[i], scale), -127.0f), 127.0f);
  }
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i / 4] |= ((uint32_t)(int)rintf(q[i]) & 0xFFu) << (8 * (i % 4));
  return scale != scale ? make_uint2(0u, 0u) : make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void decode8(const uint2& q, float scale, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[i] = (float)(int8_t)(q.x >> (8 * i)) * scale;
    v[4 + i] = (float)(int8_t)(q.y >> (8 * i)) * scale;
  }
}

// h may be null (the codes alone); row_end may be null (rows)
__global__ void __launch_bounds__(kThreads) swiglu8_fwd_kernel(const uint16_t* __restrict__ ab, int64_t rows,
                                                               const int32_t* __restrict__ row_end, int I,
                                                               uint16_t* __restrict__ h, int8_t* __restrict__ codes,
                                                               float* __restrict__ scales) {
  const int sub = threadIdx.x & 15, per_row = I / 128;
  const int64_t units = (row_end ? (int64_t)*row_end : rows) * per_row, step = (int64_t)gridDim.x * (kThreads / 16);
  for (int64_t u = (int64_t)blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4); u < units; u += step) {
    const int64_t r = u / per_row;
    const int run = (int)(u - r * per_row), f = run * 128 + sub * 8;
    float a[8], b[8];
    unpack8(*reinterpret_cast<const uint4*>(ab + r * 2 * I + f), a);
    unpack8(*reinterpret_cast<const uint4*>(ab + r * 2 * I + I + f), b);
    // (the 16 lanes of a run are all here or none: units are whole runs)
    const float sa = run_scale(a), sb = run_scale(b);
    *reinterpret_cast<uint2*>(codes + r * 2 * I + f) = code8(a, sa);
    *reinterpret_cast<uint2*>(codes + r * 2 * I + I + f) = code8(b, sb);
    if (sub == 0) {
      scales[r * 2 * per_row + run] = sa;
      scales[r * 2 * per_row + per_row + run] = sb;
    }
    if (h) {
      float o[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) o[i] = a[i] / (1.0f + __expf(-a[i])) * b[i];
      *reinterpret_cast<uint4*>(h + r * I + f) = pack8(o);
    }
  }
}

struct Swiglu8Rows {
  const int32_t* row_end;
  const float* row_gate;
  const int32_t* row_token;
  float* dg_part;   // [rows, I / 128]
};

// h may be null (LAYER: it is not)
template <bool LAYER>
__global__ void __launch_bounds__(kThreads) swiglu8_bwd_kernel(const uint16_t* __restrict__ dh,
                                                               const int8_t* __restrict__ codes,
                                                               const float* __restrict__ scales, int64_t rows, int I,
                                                               uint16_t* __restrict__ dab, uint16_t* __restrict__ h,
                                                               Swiglu8Rows w) {
  const int sub = threadIdx.x & 15, per_row = I / 128;
  const int64_t units = (LAYER ? (int64_t)*w.row_end : rows) * per_row, step = (int64_t)gridDim.x * (kThreads / 16);
  for (int64_t u = (int64_t)blockIdx.x * (kThreads / 16) + (threadIdx.x >> 4); u < units; u += step) {
    const int64_t r = u / per_row;
    const int run = (int)(u - r * per_row), f = run * 128 + sub * 8;
    float a[8], b[8], d[8], da[8], db[8], o[8];
    decode8(*reinterpret_cast<const uint2*>(codes + r * 2 * I + f), scales[r * 2 * per_row + run], a);
    decode8(*reinterpret_cast<const uint2*>(codes + r * 2 * I + I + f), scales[r * 2 * per_row + per_row + run], b);
    unpack8(*reinterpret_cast<const uint4*>(dh + r * I + f), d);
    const bool pad = LAYER && w.row_token[r] < 0;
    const float gate = LAYER ? w.row_gate[r] : 1.0f;
    float part = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float sg = 1.0f / (1.0f + __expf(-a[i])), dg = LAYER ? gate * d[i] : d[i];
      da[i] = pad ? 0.0f : dg * b[i] * sg * (1.0f + a[i] * (1.0f - sg));
      db[i] = pad ? 0.0f : dg * a[i] * sg;
      o[i] = pad ? 0.0f : a[i] * sg * b[i];
      if (LAYER) part = pad ? 0.0f : fmaf(d[i], o[i], part);
    }
    *reinterpret_cast<uint4*>(dab + r * 2 * I + f) = pack8(da);
    *reinterpret_cast<uint4*>(dab + r * 2 * I + I + f) = pack8(db);
    if (h) *reinterpret_cast<uint4*>(h + r * I + f) = pack8(o);
    if constexpr (LAYER) {
      part += __uint_as_float(rotated<0x128>(__float_as_uint(part)));
      part += __uint_as_float(rotated<0x124>(__float_as_uint(part)));
      part += __uint_as_float(rotated<0x122>(__float_as_uint(part)));
      part += __uint_as_float(rotated<0x121>(__float_as_uint(part)));
      if (sub == 0) w.dg_part[r * per_row + run] = part;
    }
  }
}

unsigned blocks_for(int64_t units) {
  return (unsigned)std::min<int64_t>(ceil_div(units, kThreads / 16), 8192);
}

}  // namespace

hipError_t launch_swiglu8_forward(int64_t rows, const int32_t* row_end, int I, const void* ab, void* h, int8_t* codes,
                                  float* scales, hipStream_t st) {
  const int64_t units = rows * (I / 128);
  if (units == 0) return hipSuccess;
  return launch_kernel(swiglu8_fwd_kernel, dim3(blocks_for(units)), dim3(kThreads), 0, st,
                     static_cast<const uint16_t*>(ab), rows, row_end, I, static_cast<uint16_t*>(h), codes, scales);
}

hipError_t launch_swiglu8_backward(int64_t rows, int I, const void* dh, const int8_t* codes, const float* scales,
                                   void* dab, void* h, hipStream_t st) {
  const int64_t units = rows * (I / 128);
  if (units == 0) return hipSuccess;
  return launch_kernel(swiglu8_bwd_kernel<false>, dim3(blocks_for(units)), dim3(kThreads), 0, st,
                     static_cast<const uint16_t*>(dh), codes, scales, rows, I, static_cast<uint16_t*>(dab),
                     static_cast<uint16_t*>(h), Swiglu8Rows{});
}

hipError_t launch_swiglu_bwd_saved8(const int8_t* codes, const float* scales, const void* dhu, const float* row_gate,
                                    const int32_t* row_token, const int32_t* row_end, int64_t max_rows, int I, void* dab,
                                    void* h, float* dg_part, hipStream_t st) {
  const int64_t units = max_rows * (I / 128);
  if (units == 0) return hipSuccess;
  return launch_kernel(swiglu8_bwd_kernel<true>, dim3(blocks_for(units)), dim3(kThreads), 0, st,
                     static_cast<const uint16_t*>(dhu), codes, scales, max_rows, I, static_cast<uint16_t*>(dab),
                     static_cast<uint16_t*>(h), Swiglu8Rows{row_end, row_gate, row_token, dg_part});
}

}  // namespace moe
