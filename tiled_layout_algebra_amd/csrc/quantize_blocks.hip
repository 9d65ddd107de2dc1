// quantize_blocks.hip -- e4m3 codes and an fp32 scale for each block of 1 x 128
// or 128 x 128 values.
//
//   a = max |x|,  s = a / 448,  q = x / s rounded to e4m3, ties to even
//
// Memory-bound: each value is read once, kept in registers over its block's
// reduction and written as one byte.  1 x 128: sixteen lanes share a block, eight
// values each.  128 x 128: a workgroup has a block, 16 lanes a row, 8 rows a lane.
//
// Exact rounding without a division: with i the rounded 1 / s, x i (1 - 2^-22) and
// x i (1 + 2^-22), rounding errors included, lie on either side of x / s.  Rounding
// is monotone, so where both convert to one code that is the quotient's; where
// they do not, the sign of x - m s, m the midpoint of the two codes, decides: the
// fused multiply-add has it exactly.
#include "quantize_common.hpp"

namespace tla {
namespace {

// A block's divisor.  mul: 2^64 for scales below 2^-100, whose reciprocal and
// remainders would leave the normal range (there s itself was rounded to few
// bits, so quotients need the clamp).
struct BlockScale {
  float s, lo, hi, mul;
  bool zero, tiny;  // zero: every code is 0 (s is 0, infinite or NaN)
};
__device__ __forceinline__ BlockScale block_scale(float amax, float& s) {
  BlockScale d;
  s = amax / 448.f;
  d.zero = !(s > 0.f && s <= 3.40282347e38f);
  d.tiny = s < 0x1p-100f;
  d.mul = d.tiny ? 0x1p64f : 1.f;
  d.s = s * d.mul;
  const float inv = 1.f / d.s;
  d.lo = fmaf(inv, -0x1p-22f, inv);
  d.hi = fmaf(inv, 0x1p-22f, inv);
  return d;
}

__device__ __forceinline__ uint32_t codes2(float a, float b) {
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false) & 0xFFFFu;
}
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false), true);
}
// The exactly rounded code of one value
__device__ __forceinline__ uint32_t settle(float x, const BlockScale& d) {
  const float ax = fabsf(x) * d.mul;
  // (no clamp changes a code below the largest, and none above it is one)
  const uint32_t w = codes2(fminf(ax * d.lo, 448.f), fminf(ax * d.hi, 448.f));
  uint32_t lo = w & 0xFFu;
  const uint32_t hi = w >> 8;
  if (lo != hi) {
    const float m = 0.5f * (__builtin_amdgcn_cvt_f32_fp8((int)lo, 0) + __builtin_amdgcn_cvt_f32_fp8((int)hi, 0));
    const float r = fmaf(-m, d.s, ax);
    if (r > 0.f || (r == 0.f && (lo & 1u))) lo = hi;
  }
  return d.zero ? 0u : lo | (__builtin_bit_cast(uint32_t, x) >> 24 & 0x80u);
}

template <int kCode>
__device__ __forceinline__ uint2 block_codes8(const RowVec<kCode>& v, const BlockScale& d) {
  if (d.zero) return uint2{0u, 0u};
  uint32_t w[2] = {0, 0};
  bool sure = !d.tiny;
  if (sure) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float x[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = v.get(4 * h + e);
      w[h] = codes4(x[0] * d.lo, x[1] * d.lo, x[2] * d.lo, x[3] * d.lo);
      sure &= w[h] == codes4(x[0] * d.hi, x[1] * d.hi, x[2] * d.hi, x[3] * d.hi);
    }
  }
  if (!sure) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      w[h] = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) w[h] |= settle(v.get(4 * h + e), d) << (8 * e);
    }
  }
  return uint2{w[0], w[1]};
}

// eight values of a row from column c, zeros from column K on
template <int kCode>
__device__ __forceinline__ void load8(RowVec<kCode>& v, const uint8_t* row, int64_t c, int64_t K) {
  constexpr int kEB = type_bytes(kCode);
  if (c + 8 <= K) {
    v.load(row, c);
    return;
  }
  uint32_t w[kEB * 2] = {};
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (c + e < K) {
      if constexpr (kCode == kF32) w[e] = ((const uint32_t*)row)[c + e];
      else w[e / 2] |= (uint32_t)((const uint16_t*)row)[c + e] << (16 * (e & 1));
    }
  }
  v.load((const uint8_t*)w, 0);
}
__device__ __forceinline__ void store8(uint8_t* q, int64_t c, int64_t K, uint2 w) {
  typedef uint32_t u32x2_a1 __attribute__((ext_vector_type(2), aligned(1)));
  if (c + 8 <= K) {
    *(u32x2_a1*)(q + c) = u32x2_a1{w.x, w.y};
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (c + e < K) q[c + e] = (uint8_t)((e < 4 ? w.x : w.y) >> (8 * (e & 3)));
}

struct QuantArgs {
  const uint8_t* X;
  uint8_t* Q;
  float* scale;
  int64_t ldx, ldq, s_row, s_kb, M, K;
  int kbs, groups, shift;  // blocks in a row; workgroups along a row; log2 of a workgroup's blocks along it
};

// Workgroup b runs on XCD b % 8: each XCD gets a run of neighbours, so that lines
// which two blocks share are read into one L2 (16384 x 8191 bf16, whose rows begin
// anywhere in a line: TIME).
__device__ __forceinline__ unsigned in_runs(unsigned b, unsigned n) {
  const unsigned per = n / 8, rest = n % 8, xcd = b & 7;
  return xcd * per + min(xcd, rest) + (b >> 3);
}

// 1 x 128: a workgroup's sixteen blocks are 2^shift neighbours of 16 / 2^shift rows.
template <int kCode>
__global__ __launch_bounds__(256) void quantize_row_blocks_kernel(const QuantArgs a) {
  const int tid = threadIdx.x, unit = tid >> 4;
  const unsigned id = in_runs(blockIdx.x, gridDim.x);
  const int band = id / (unsigned)a.groups, group = id % (unsigned)a.groups;
  const int64_t row = ((int64_t)band << (4 - a.shift)) + (unit >> a.shift);
  const int kb = (group << a.shift) + (unit & ((1 << a.shift) - 1));
  if (row >= a.M || kb >= a.kbs) return;
  const int64_t c = (int64_t)kb * 128 + 8 * (tid & 15);
  RowVec<kCode> v;
  load8<kCode>(v, a.X + row * a.ldx * type_bytes(kCode), c, a.K);
  uint32_t m = v.amax();
#pragma unroll
  for (int d = 8; d; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
  float s;
  const BlockScale d = block_scale(from_bits<kCode>(m), s);
  if ((tid & 15) == 0) a.scale[row * a.s_row + kb * a.s_kb] = s;
  store8(a.Q + row * a.ldq, c, a.K, block_codes8<kCode>(v, d));
}

// 128 x 128: a workgroup a block.
template <int kCode>
__global__ __launch_bounds__(256) void quantize_square_blocks_kernel(const QuantArgs a) {
  const int tid = threadIdx.x;
  const unsigned id = in_runs(blockIdx.x, gridDim.x);
  const int64_t band = id / (unsigned)a.kbs;
  const int kb = id % (unsigned)a.kbs;
  const int64_t row0 = band * 128 + (tid >> 4), c = (int64_t)kb * 128 + 8 * (tid & 15);
  RowVec<kCode> v[8];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    load8<kCode>(v[i], a.X + min(row0 + 16 * i, a.M - 1) * a.ldx * type_bytes(kCode), c, a.K);
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, v[i].amax());  // (rows past the last are that row again)
#pragma unroll
  for (int d = 32; d; d >>= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d));
  __shared__ uint32_t part[4];
  if ((tid & 63) == 0) part[tid >> 6] = m;
  __syncthreads();
  m = max(max(part[0], part[1]), max(part[2], part[3]));
  float s;
  const BlockScale d = block_scale(from_bits<kCode>(m), s);
  if (tid == 0) a.scale[band * a.s_row + kb * a.s_kb] = s;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (row0 + 16 * i < a.M) store8(a.Q + (row0 + 16 * i) * a.ldq, c, a.K, block_codes8<kCode>(v[i], d));
}

// In launches of fewer than 2^32 threads, bands of rows at a time.
template <int kCode>
int launch(QuantArgs a, int block_rows, hipStream_t s) {
  const int64_t most = kMaxThreads / 256;  // workgroups
  a.kbs = (int)((a.K + 127) / 128);
  a.shift = 0;
  while (a.shift < 4 && (1 << a.shift) < a.kbs) ++a.shift;
  a.groups = block_rows == 1 ? (a.kbs + (1 << a.shift) - 1) >> a.shift : a.kbs;
  const int64_t rows = block_rows == 1 ? 16 >> a.shift : 128;  // of a workgroup
  const int64_t bands = (a.M + rows - 1) / rows, step = most / a.groups;
  if (step < 1) return TLA_ERR_UNSUPPORTED;
  const int64_t M = a.M;
  for (int64_t b = 0; b < bands; b += step) {
    const int64_t n = bands - b < step ? bands - b : step;
    QuantArgs x = a;
    x.X += b * rows * a.ldx * type_bytes(kCode);
    x.Q += b * rows * a.ldq;
    x.scale += b * (block_rows == 1 ? rows : 1) * a.s_row;
    x.M = M - b * rows;
    const dim3 grid((unsigned)(n * a.groups));
    if (block_rows == 1)
      hipLaunchKernelGGL((quantize_row_blocks_kernel<kCode>), grid, dim3(256), 0, s, x);
    else
      hipLaunchKernelGGL((quantize_square_blocks_kernel<kCode>), grid, dim3(256), 0, s, x);
    if (hipGetLastError() != hipSuccess) return TLA_ERR_HIP;
  }
  return TLA_OK;
}

}  // namespace

int launch_quantize_blocks(int64_t M, int64_t K, const void* X, int type, int64_t ldx,
                           int block_rows, uint8_t* Q, int64_t ldq, float* scale, int64_t s_row,
                           int64_t s_kb, hipStream_t s) {
  QuantArgs a{};
  a.X = (const uint8_t*)X;
  a.Q = Q;
  a.scale = scale;
  a.ldx = ldx;
  a.ldq = ldq;
  a.s_row = s_row;
  a.s_kb = s_kb;
  a.M = M;
  a.K = K;
  switch (type) {
    case TLA_F16: return launch<kF16>(a, block_rows, s);
    case TLA_BF16: return launch<kBF16>(a, block_rows, s);
    case TLA_F32: return launch<kF32>(a, block_rows, s);
    default: return TLA_ERR_UNSUPPORTED;
  }
}

}  // namespace tla
