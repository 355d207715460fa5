// Device helpers of the kernels at a block's ends (ssm_add_norm.hip, ssm_quantize.hip, ssm_matmul_fp8.hip): eight consecutive
// elements of a row at any alignment; magnitudes, scales and codes of 8-bit values with a scale for each block of 128.
#pragma once

#include "packed.hpp"

namespace ssm57 {

constexpr int kBlock = SSM57_BLOCK;
constexpr float kTop = 448.0f;                  // the largest e4m3 value
constexpr uint32_t kLeastBits = 0x0d800000u;    // 2^-100

// 4-byte (2-byte) alignment is all that a 16-byte access of fp32 (bf16) elements needs.
typedef uint32_t pu4e __attribute__((ext_vector_type(4), aligned(2)));
typedef uint32_t pu2e __attribute__((ext_vector_type(2), aligned(8)));

// Eight consecutive elements: raw registers, their load, conversion and store.  `cnt` < 8 elements belong to the row:
// the others are read as zero and not written.
template <typename T>
struct Eight;
template <>
struct Eight<float> {
  pf4 raw[2];
  __device__ __forceinline__ void load(const float* p) {
    raw[0] = *reinterpret_cast<const pf4u*>(p);
    raw[1] = *reinterpret_cast<const pf4u*>(p + 4);
  }
  __device__ __forceinline__ void load(const float* p, int cnt) {
#pragma unroll
    for (int i = 0; i < 8; ++i) raw[i >> 2][i & 3] = i < cnt ? p[i] : 0.0f;
  }
  __device__ __forceinline__ void zero() { raw[0] = raw[1] = pf4{0.0f, 0.0f, 0.0f, 0.0f}; }
  __device__ __forceinline__ void get(float* o) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = raw[i >> 2][i & 3];
  }
  static __device__ __forceinline__ void store(float* p, const float* v) { store_floats<8>(p, v); }
  static __device__ __forceinline__ void store(float* p, const float* v, int cnt) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < cnt) p[i] = v[i];
  }
};
template <>
struct Eight<uint16_t> {
  pu4 raw;
  __device__ __forceinline__ void load(const uint16_t* p) { raw = *reinterpret_cast<const pu4e*>(p); }
  __device__ __forceinline__ void load(const uint16_t* p, int cnt) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = 2 * i < cnt ? p[2 * i] : 0, b = 2 * i + 1 < cnt ? p[2 * i + 1] : 0;
      raw[i] = a | (b << 16);
    }
  }
  __device__ __forceinline__ void zero() { raw = pu4{0, 0, 0, 0}; }
  __device__ __forceinline__ void get(float* o) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = lo_f32(raw[i]);
      o[2 * i + 1] = hi_f32(raw[i]);
    }
  }
  static __device__ __forceinline__ void store(uint16_t* p, const float* v) {
    *reinterpret_cast<pu4e*>(p) =
        pu4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
  }
  static __device__ __forceinline__ void store(uint16_t* p, const float* v, int cnt) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < cnt) Elem<uint16_t>::st(p, i, v[i]);
  }
};

// Magnitudes are compared as bit patterns: the order is the same, and infinities and NaN come out on top.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ uint32_t largest(const float* v) {
  uint32_t m = magnitude(v[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max(m, magnitude(v[i]));
  return m;
}
template <int K>
__device__ __forceinline__ uint32_t row_ror_bits(uint32_t v) { return __float_as_uint(row_ror<K>(__uint_as_float(v))); }
// the largest over the 16 lanes of a row (eight elements each: a block), in all of them
__device__ __forceinline__ uint32_t row_largest(uint32_t m) {
  m = max(m, row_ror_bits<8>(m));
  m = max(m, row_ror_bits<4>(m));
  m = max(m, row_ror_bits<2>(m));
  return max(m, row_ror_bits<1>(m));
}

__device__ __forceinline__ float scale_of(uint32_t most) { return __uint_as_float(max(most, kLeastBits)) / kTop; }

// Codes of four values that are at most 448 (1 + 2^-22) in magnitude, or NaN.
__device__ __forceinline__ uint32_t codes(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true));
}
// Codes of eight values of a block: their fp32 quotients by the scale, rounded to nearest, then to the nearest code.  bf16
// values often lie halfway between two codes, where a product with the rounded reciprocal went to the wrong side (6 codes in
// 10,000), so the quotient's remainder, which a fma has exactly, corrects it: two more operations for a code, with the same
// codes as a division for each (tried on the host at every border between codes for every divisor's mantissa).  Measured
// beside the product alone: 8191 x 5120 bf16, rows and columns, 42.9 us and 39.6; 16384 rows of 2560 of the norm 86.6 and 84.9.
__device__ __forceinline__ pu2 codes8(const float* v, float scale) {
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = v[i];
  if (scale < 0x1p-90f) {   // (remainders would be subnormal)
    scale *= 0x1p64f;
#pragma unroll
    for (int i = 0; i < 8; ++i) q[i] *= 0x1p64f;
  }
  const float inv = 1.0f / scale;
  const float s = scale < __builtin_inff() ? scale : 0.0f;   // (of a block with an infinity: finite values have code 0)
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float near = q[i] * inv;
    q[i] = fmaf(-fmaf(near, s, -q[i]), inv, near);
  }
  return pu2{codes(q[0], q[1], q[2], q[3]), codes(q[4], q[5], q[6], q[7])};
}

inline int64_t up16(int64_t n) { return (n + 15) / 16 * 16; }
inline int64_t blocks_of(int64_t n) { return (n + kBlock - 1) / kBlock; }

}  // namespace ssm57
