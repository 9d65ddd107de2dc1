// quantize.hip -- int8 codes and one fp32 scale for each row.
//
//   a = max |x|,  s = a * fl(1/127),  q = x / s rounded to nearest, ties to even
//
// Memory-bound: each value is read once, kept in registers over the row's
// reduction and written as one byte.  kTpr threads share a row; the row's
// columns are cut where the codes' address is a multiple of 8, so stores are
// whole 8-byte vectors whatever the pitch, and the few columns before and
// after go one by one.  |x| compares like its bit pattern, so the maximum is
// an integer maximum and a NaN, larger than every number, wins it.
//
// Exact rounding without a division: q0 = x (1/s) rounded through the
// addition of 1.5 * 2^23 is within 1.6e-5 of x / s before rounding, so it can
// only be wrong where |x (1/s) - q0| is within that of 1/2.  There the
// remainder d = x - q0 s decides: q0 s has at most 31 bits, d is a multiple of
// half a unit of s's last place and at most s/2 in size up to that error, so
// the fused multiply-add gives it exactly, and comparing it with s/2 rounds as
// the true quotient does.
//
// Measured: 16384 x 8191 bf16 76 us (403 MB: 5.3 TB/s), 12608 x 811 fp32 11 us,
// 64 x 4096 bf16 4.4 us (a launch).
#include "grouped_common.hpp"

namespace tla {
namespace {

constexpr float kRcp127 = 1.0f / 127.0f;
constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: its low byte is 0

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

// The row's divisor.  mul: 2^64 for scales below 2^-100, whose reciprocal and
// remainders would leave the normal range (x and s times 2^64 have the same
// quotient; there s itself was rounded to few bits, so codes need the clamp).
struct Divisor {
  float s, inv, mul;
  bool zero, tiny;  // zero: every code is 0 (s is 0, infinite or NaN)
};

// The exact rounding of x / s near a tie, from q0 = t - kMagic
__device__ __forceinline__ float settle(float x, float t, const Divisor& d) {
  const float q = t - kMagic, r = fmaf(-q, d.s, x), h = 0.5f * d.s;
  const bool odd = __builtin_bit_cast(uint32_t, t) & 1u;
  if (r > h || (r == h && odd)) return t + 1.f;
  if (r < -h || (r == -h && odd)) return t - 1.f;
  return t;
}

__device__ __forceinline__ uint32_t code1(float x, const Divisor& d) {
  x *= d.mul;
  float t = settle(x, fmaf(x, d.inv, kMagic), d);
  t = fminf(fmaxf(t, kMagic - 127.f), kMagic + 127.f);
  return d.zero ? 0u : __builtin_bit_cast(uint32_t, t) & 0xFFu;
}

template <int kCode>
__device__ __forceinline__ uint2 codes8(const RowVec<kCode>& v, const Divisor& d) {
  if (d.zero) return uint2{0u, 0u};
  uint32_t w[8];
  if (d.tiny) {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = code1(v.get(e), d);
  } else {
    float t[8], far = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float x = v.get(e);
      t[e] = fmaf(x, d.inv, kMagic);
      far = fmaxf(far, fabsf(fmaf(x, d.inv, kMagic - t[e])));
    }
    if (far > 0.49997f) {
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = settle(v.get(e), t[e], d);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = __builtin_bit_cast(uint32_t, t[e]);
  }
  auto pack4 = [](uint32_t a, uint32_t b, uint32_t c, uint32_t e) {
    const uint32_t lo = __builtin_amdgcn_perm(b, a, 0x0C0C0400u);
    const uint32_t hi = __builtin_amdgcn_perm(e, c, 0x0C0C0400u);
    return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
  };
  return uint2{pack4(w[0], w[1], w[2], w[3]), pack4(w[4], w[5], w[6], w[7])};
}

template <int kCode, int kTpr, int kV>
__global__ __launch_bounds__(256) void quantize_rows_kernel(const uint8_t* X, int64_t ldx,
                                                            int8_t* Q, int64_t ldq, float* scale,
                                                            int64_t M, int64_t K) {
  constexpr int kEB = type_bytes(kCode), kRows = 256 / kTpr;
  const int tid = threadIdx.x, t = tid % kTpr;
  const int64_t row = (int64_t)blockIdx.x * kRows + tid / kTpr;
  const bool live = row < M;
  const int64_t r = live ? row : M - 1;
  const uint8_t* x = X + r * ldx * kEB;
  uint8_t* q = (uint8_t*)Q + r * ldq;
  // columns [0, head) and [K - tail, K) one by one, the rest in vectors of 8
  const int64_t to8 = (-(uintptr_t)q) & 7;
  const int64_t head = to8 < K ? to8 : K, nv = (K - head) / 8, tail = K - head - 8 * nv;
  const int64_t one = t < head ? t : (t >= 8 && t - 8 < tail ? K - tail + t - 8 : -1);
  x += head * kEB;
  RowVec<kCode> v[kV];
  uint32_t m = one >= 0 ? abs_bits<kCode>(x - head * kEB, one) : 0u;
#pragma unroll
  for (int i = 0; i < kV; ++i)
    if (t + i * kTpr < nv) v[i].load(x, 8 * (int64_t)(t + i * kTpr));
#pragma unroll
  for (int i = 0; i < kV; ++i)
    if (t + i * kTpr < nv) m = max(m, v[i].amax());
  for (int64_t i = t + kV * kTpr; i < nv; i += kTpr) {  // rows past the registers: read again below
    RowVec<kCode> u;
    u.load(x, 8 * i);
    m = max(m, u.amax());
  }
#pragma unroll
  for (int d = 32; d; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
  if constexpr (kTpr > 64) {
    __shared__ uint32_t part[4];
    if ((tid & 63) == 0) part[tid >> 6] = m;
    __syncthreads();
    m = max(max(part[0], part[1]), max(part[2], part[3]));
  }
  if (!live) return;
  const float a = from_bits<kCode>(m);
  Divisor d;
  const float s = a * kRcp127;
  d.zero = !(s > 0.f && s <= 3.40282347e38f);
  d.tiny = s < 0x1p-100f;
  d.mul = d.tiny ? 0x1p64f : 1.f;
  d.s = s * d.mul;
  d.inv = 1.0f / d.s;
  if (t == 0) scale[row] = s;
#pragma unroll
  for (int i = 0; i < kV; ++i)
    if (t + i * kTpr < nv)
      *(uint2*)(q + head + 8 * (int64_t)(t + i * kTpr)) = codes8<kCode>(v[i], d);
  for (int64_t i = t + kV * kTpr; i < nv; i += kTpr) {
    RowVec<kCode> u;
    u.load(x, 8 * i);
    *(uint2*)(q + head + 8 * i) = codes8<kCode>(u, d);
  }
  if (one >= 0) {
    const uint8_t* o = x - head * kEB;
    float val;
    if constexpr (kCode == kF32) val = ((const float*)o)[one];
    else val = widen_lo<kCode == kBF16>(((const uint16_t*)o)[one]);
    q[one] = (uint8_t)code1(val, d);
  }
}

// The rows in launches of fewer than 2^32 threads.
template <int kCode, int kTpr, int kV>
int launch(int64_t M, int64_t K, const void* X, int64_t ldx, int8_t* Q, int64_t ldq, float* scale,
           hipStream_t s) {
  constexpr int64_t kRows = 256 / kTpr, kMost = kRows * (kMaxThreads / 256);
  if (M > kRows * 0x7FFFFFFF) return TLA_ERR_UNSUPPORTED;
  for (int64_t r = 0; r < M; r += kMost) {
    const int64_t rows = M - r < kMost ? M - r : kMost;
    const unsigned grid = (unsigned)((rows + kRows - 1) / kRows);
    hipLaunchKernelGGL((quantize_rows_kernel<kCode, kTpr, kV>), dim3(grid), dim3(256), 0, s,
                       (const uint8_t*)X + r * ldx * type_bytes(kCode), ldx, Q + r * ldq, ldq,
                       scale + r, rows, K);
    if (hipGetLastError() != hipSuccess) return TLA_ERR_HIP;
  }
  return TLA_OK;
}

// The narrowest form whose registers hold the row: a wavefront for each row
// up to 2048 columns, the workgroup for longer ones.
template <int kCode>
int dispatch(int64_t M, int64_t K, const void* X, int64_t ldx, int8_t* Q, int64_t ldq,
             float* scale, hipStream_t s) {
  if (K <= 512) return launch<kCode, 64, 1>(M, K, X, ldx, Q, ldq, scale, s);
  if (K <= 1024) return launch<kCode, 64, 2>(M, K, X, ldx, Q, ldq, scale, s);
  if (K <= 2048) return launch<kCode, 64, 4>(M, K, X, ldx, Q, ldq, scale, s);
  if (K <= 4096) return launch<kCode, 256, 2>(M, K, X, ldx, Q, ldq, scale, s);
  if (K <= 8192) return launch<kCode, 256, 4>(M, K, X, ldx, Q, ldq, scale, s);
  return launch<kCode, 256, 8>(M, K, X, ldx, Q, ldq, scale, s);
}

}  // namespace

int launch_quantize_rows(int64_t M, int64_t K, const void* X, int type, int64_t ldx, int8_t* Q,
                         int64_t ldq, float* scale, hipStream_t s) {
  switch (type) {
    case TLA_F16: return dispatch<kF16>(M, K, X, ldx, Q, ldq, scale, s);
    case TLA_BF16: return dispatch<kBF16>(M, K, X, ldx, Q, ldq, scale, s);
    case TLA_F32: return dispatch<kF32>(M, K, X, ldx, Q, ldq, scale, s);
    default: return TLA_ERR_UNSUPPORTED;
  }
}

}  // namespace tla
