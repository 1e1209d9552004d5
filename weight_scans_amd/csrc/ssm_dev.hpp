// ssm_dev.hpp -- device helpers of the selective scan, the short convolution and
// the norms around a block.
#pragma once

#include "dev_common.hpp"
#include "ssm.hpp"

namespace gls {

// One rounding to bf16 (to nearest, ties to even), by the hardware.
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  typedef __bf16 two __attribute__((ext_vector_type(2)));
  typedef float ftwo __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((ftwo){a, b}, two));
}
template <typename IO, typename S>
__device__ __forceinline__ void put(IO* p, S v) {
  if constexpr (sizeof(IO) == 2) reinterpret_cast<uint16_t*>(p)[0] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
  else p[0] = static_cast<IO>(v);
}

// Sixteen bytes as the registers hold them.
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr double kLog2e = 1.4426950408889634;

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ double exp2_(double x) { return exp2(x); }
__device__ __forceinline__ float rcp_(float x) { return __builtin_amdgcn_rcpf(x); }
__device__ __forceinline__ double rcp_(double x) { return 1.0 / x; }
__device__ __forceinline__ float sqrt_(float x) { return sqrtf(x); }
__device__ __forceinline__ double sqrt_(double x) { return sqrt(x); }

// 1 / (1 + e^-x): e^-x overflows to infinity and the quotient to 0 below -88.
template <typename S>
__device__ __forceinline__ S sigmoid_(S x) {
  return rcp_(S(1) + exp2_(static_cast<S>(-kLog2e) * x));
}

// log(1 + e^x) = max(x, 0) + log(1 + y) with y = e^-|x| <= 1 and
// log(1 + y) = 2 artanh(s), s = y / (2 + y) <= 1/3: the series in s^2 <= 1/9 to its
// seventh term leaves 2e-8 of the sum (Abramowitz and Stegun 4.1.27), where
// log(1 + y) loses y's last places for small y.
__device__ __forceinline__ float softplus_(float x) {
  const float y = exp2_(static_cast<float>(-kLog2e) * fabsf(x));
  const float s = y * rcp_(2.0f + y), q = s * s;
  float p = 2.0f / 13.0f;
  p = fmaf(p, q, 2.0f / 11.0f);
  p = fmaf(p, q, 2.0f / 9.0f);
  p = fmaf(p, q, 2.0f / 7.0f);
  p = fmaf(p, q, 2.0f / 5.0f);
  p = fmaf(p, q, 2.0f / 3.0f);
  p = fmaf(p, q, 2.0f);
  return fmaf(p, s, x != x ? x : fmaxf(x, 0.0f));
}
__device__ __forceinline__ double softplus_(double x) { return log1p(exp(-fabs(x))) + (x != x ? x : fmax(x, 0.0)); }

__device__ __forceinline__ float fma_(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ double fma_(double a, double b, double c) { return fma(a, b, c); }

// Sixteen bytes of consecutive elements, 16-byte aligned, in the compute type.
template <typename IO>
struct Vec;
template <>
struct Vec<bf16> {
  static constexpr int n = 8;
  template <typename S>
  __device__ static __forceinline__ void ld(const bf16* p, S* v) {
    const uint4 t = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  template <typename S>
  __device__ static __forceinline__ void st(bf16* p, const S* v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec<float> {
  static constexpr int n = 4;
  template <typename S>
  __device__ static __forceinline__ void ld(const float* p, S* v) {
    const float4 t = *reinterpret_cast<const float4*>(p);
    v[0] = t.x; v[1] = t.y; v[2] = t.z; v[3] = t.w;
  }
  template <typename S>
  __device__ static __forceinline__ void st(float* p, const S* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <>
struct Vec<double> {
  static constexpr int n = 2;
  template <typename S>
  __device__ static __forceinline__ void ld(const double* p, S* v) {
    const double2 t = *reinterpret_cast<const double2*>(p);
    v[0] = t.x; v[1] = t.y;
  }
  template <typename S>
  __device__ static __forceinline__ void st(double* p, const S* v) {
    *reinterpret_cast<double2*>(p) = make_double2(v[0], v[1]);
  }
};

// W elements from p: one vector, or one element.
template <typename IO, typename S, int W>
__device__ __forceinline__ void load_w(const IO* p, S* v) {
  if constexpr (W == 1) {
    v[0] = load_as<S>(p, 0);
  } else {
    static_assert(W == Vec<IO>::n, "16 bytes");
    Vec<IO>::ld(p, v);
  }
}
template <typename IO, typename S, int W>
__device__ __forceinline__ void store_w(IO* p, const S* v) {
  if constexpr (W == 1) {
    put(p, v[0]);
  } else {
    static_assert(W == Vec<IO>::n, "16 bytes");
    Vec<IO>::st(p, v);
  }
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
inline bool aligned16(int io, const Rows& s) {
  const int m = io == IO_BF16 ? 8 : io == IO_F32 ? 4 : 2;
  return s.b % m == 0 && s.t % m == 0 && s.g % m == 0;
}
inline int vec_of(int io) { return io == IO_BF16 ? 8 : io == IO_F32 ? 4 : 2; }

// Work-groups that follow one another in the grid go to the eight XCDs in turn;
// this gives each XCD a run of neighbouring tiles instead, so that tiles that
// share cache lines meet in one L2.
__device__ __forceinline__ int64_t xcd_order(int64_t i, int64_t n) {
  const int64_t q = n / 8, r = n % 8, x = i % 8, k = i / 8;
  return x * q + (x < r ? x : r) + k;
}

}  // namespace gls
