// quantize_common.hpp -- loads and maxima of the quantizers: eight values of a
// row from any element's address, and |x| by its bit pattern, whose integer order
// is |x|'s own, with a NaN above every number.
#pragma once

#include "grouped_common.hpp"

namespace tla {
namespace {

template <int kCode>
struct RowVec;  // eight values of a row
template <int kCode>
  requires(kCode != kF32)
struct RowVec<kCode> {
  i32x4 v;
  __device__ __forceinline__ void load(const uint8_t* x, int64_t i) { v = load16_even(x + i * 2); }
  __device__ __forceinline__ uint32_t amax() const {
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    u16x2 m = {0, 0};
#pragma unroll
    for (int w = 0; w < 4; ++w)
      m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[w] & 0x7FFF7FFF));
    return m[0] > m[1] ? m[0] : m[1];
  }
  __device__ __forceinline__ float get(int e) const {
    return e & 1 ? widen_hi<kCode == kBF16>((uint32_t)v[e >> 1])
                 : widen_lo<kCode == kBF16>((uint32_t)v[e >> 1]);
  }
};
template <>
struct RowVec<kF32> {
  i32x4 lo, hi;
  __device__ __forceinline__ void load(const uint8_t* x, int64_t i) {
    typedef int i32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
    lo = *(const i32x4_a4*)(x + i * 4);
    hi = *(const i32x4_a4*)(x + i * 4 + 16);
  }
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      m = max(m, (uint32_t)lo[w] & 0x7FFFFFFFu);
      m = max(m, (uint32_t)hi[w] & 0x7FFFFFFFu);
    }
    return m;
  }
  __device__ __forceinline__ float get(int e) const {
    return __builtin_bit_cast(float, e < 4 ? lo[e] : hi[e - 4]);
  }
};

// |x|'s bits of one element, and the float of such bits
template <int kCode>
__device__ __forceinline__ uint32_t abs_bits(const uint8_t* x, int64_t i) {
  if constexpr (kCode == kF32) return ((const uint32_t*)x)[i] & 0x7FFFFFFFu;
  else return ((const uint16_t*)x)[i] & 0x7FFFu;
}
template <int kCode>
__device__ __forceinline__ float from_bits(uint32_t b) {
  if constexpr (kCode == kF32) return __builtin_bit_cast(float, b);
  else return widen_lo<kCode == kBF16>(b);
}

}  // namespace
}  // namespace tla
