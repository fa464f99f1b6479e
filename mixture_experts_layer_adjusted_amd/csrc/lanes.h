// Runs of a row's neighbouring values in registers, and reductions over the lanes that hold a row: what the kernels
// on logits share.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {
namespace {

constexpr float kNegInf = -__builtin_inff();

// exp(x) from the 2^y instruction: y = x log2(e) rounded, and r = x - y ln(2) (ln(2) in two parts) as a factor 1 + r.
// Within 2 units in the last place; results below 2^-126 are 0, infinities and NaN as they should be.
__device__ __forceinline__ float exp_of(float x) {
  const float y = x * 1.44269502f;
  const float r = fmaf(y, 1.90465421e-9f, fmaf(y, -0.693147182f, x));
  const float e = __builtin_amdgcn_exp2f(y);
  return fabsf(x) < 150.0f ? fmaf(e, r, e) : e;   // (e may be infinite, and r NaN)
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

}  // namespace
}  // namespace moe
