// Device helpers shared by the kernels over packed sequences (ssm_packed_conv.hip, ssm_packed_ssd.hip,
// ssm_packed_ssd_bwd.hip) and by the norm (ssm_gated_norm.hip): vector element access with a scalar form for rows that
// are not 16-byte aligned, and the places of sequences and states.
#pragma once

#include "common.hpp"

namespace ssm57 {

typedef float pf4 __attribute__((ext_vector_type(4)));
typedef float pf2 __attribute__((ext_vector_type(2)));
typedef __bf16 pbf2 __attribute__((ext_vector_type(2)));
typedef uint32_t pu4 __attribute__((ext_vector_type(4)));
typedef uint32_t pu2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ float lo_f32(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f32(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }
// two fp32 -> packed bf16 pair (first value in the low half), round to nearest even
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(pf2{a, b}, pbf2));
}

// V consecutive elements of type T (float or bf16 bits): raw registers, their load, conversion and store.  V > 1 is
// one 16-byte access (4 floats or 8 bf16), V = 1 a single element.  Outputs stream out once: non-temporal stores.
template <typename T, int V>
struct Pack {
  static_assert(V == 1);
  T raw;
  __device__ __forceinline__ void load(const T* p) { raw = *p; }
  __device__ __forceinline__ void get(float* o) const { o[0] = Elem<T>::cvt(raw); }
  static __device__ __forceinline__ void store(T* p, const float* v) { Elem<T>::st(p, 0, v[0]); }
};
template <>
struct Pack<float, 4> {
  pf4 raw;
  __device__ __forceinline__ void load(const float* p) { raw = *reinterpret_cast<const pf4*>(p); }
  __device__ __forceinline__ void get(float* o) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = raw[i];
  }
  static __device__ __forceinline__ void store(float* p, const float* v) {
    __builtin_nontemporal_store(pf4{v[0], v[1], v[2], v[3]}, reinterpret_cast<pf4*>(p));
  }
};
template <>
struct Pack<uint16_t, 8> {
  pu4 raw;
  __device__ __forceinline__ void load(const uint16_t* p) { raw = *reinterpret_cast<const pu4*>(p); }
  __device__ __forceinline__ void get(float* o) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = lo_f32(raw[i]);
      o[2 * i + 1] = hi_f32(raw[i]);
    }
  }
  static __device__ __forceinline__ void store(uint16_t* p, const float* v) {
    __builtin_nontemporal_store(pu4{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]),
                                    pack_bf16(v[6], v[7])},
                                reinterpret_cast<pu4*>(p));
  }
};

// M consecutive floats in as few loads (stores) as they make up; 4-byte alignment is all a 16-byte access needs here.
typedef float pf4u __attribute__((ext_vector_type(4), aligned(4)));
template <int M>
__device__ __forceinline__ void load_floats(const float* p, float* o) {
#pragma unroll
  for (int i = 0; i + 4 <= M; i += 4) {
    const pf4u v = *reinterpret_cast<const pf4u*>(p + i);
#pragma unroll
    for (int k = 0; k < 4; ++k) o[i + k] = v[k];
  }
#pragma unroll
  for (int i = M / 4 * 4; i < M; ++i) o[i] = p[i];
}
template <int M>
__device__ __forceinline__ void store_floats(float* p, const float* o) {
#pragma unroll
  for (int i = 0; i + 4 <= M; i += 4) *reinterpret_cast<pf4u*>(p + i) = pf4u{o[i], o[i + 1], o[i + 2], o[i + 3]};
#pragma unroll
  for (int i = M / 4 * 4; i < M; ++i) p[i] = o[i];
}

__device__ __forceinline__ float sigmoid(float v) { return hw_rcp(1.0f + hw_exp2(-v * kLog2e)); }

// The last s in [0, nseqs] with cu[s] <= t (empty sequences at t are passed over), or -1: token t belongs to sequence
// s when 0 <= s < nseqs; s == nseqs means it lies behind the last one.
__device__ __forceinline__ int find_seq(const int32_t* cu, int nseqs, int t) {
  int lo = -1, hi = nseqs + 1;   // cu[lo] <= t < cu[hi], with cu[-1] = -inf and cu[nseqs + 1] = inf
  while (hi - lo > 1) {
    const int mid = lo + (hi - lo) / 2;
    if (cu[mid] <= t) lo = mid; else hi = mid;
  }
  return lo;
}

// First token and end of sequence s, held inside [0, ntokens] whatever cu holds.
__device__ __forceinline__ void seq_range(const int32_t* cu, int s, int ntokens, int& begin, int& end) {
  begin = min(max(cu[s], 0), ntokens);
  end = min(max(cu[s + 1], begin), ntokens);
}

// Slot of sequence (or row) s: idx[s], or s itself without idx; -1 where that is no slot.
__device__ __forceinline__ int64_t slot_of(const int32_t* idx, int s, int64_t nslots) {
  const int64_t k = idx ? idx[s] : s;
  return k >= 0 && k < nslots ? k : -1;
}

// A launch takes fewer than 2^32 threads along a dimension of its grid.
inline bool fits_launch(int64_t blocks, int threads) { return blocks * threads < (int64_t(1) << 32); }

}  // namespace ssm57
