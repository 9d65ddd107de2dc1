// quantize_blocks.hip -- e4m3 codes and an fp32 scale for each block of 1 x 128
// or 128 x 128 values.
//
//   a = max |x|,  s = a / 448,  q = x / s rounded to e4m3, ties to even
//
// Memory-bound: each value is read once, kept in registers over its block's
// reduction and written as one byte.  1 x 128: sixteen lanes share a block, eight
// values each.  128 x 128: a workgroup has a block, 16 lanes a row, 8 rows a lane.
// Measured: 16384 x 8192 bf16 (403 MB) 84 us in 1 x 128 and 81 in 128 x 128, 4.8 and
// 5.0 TB/s of a large copy's 6.6; 8191 columns, whose rows begin anywhere in a line, 92
// and 93; 8192 x 8192 fp32 62 us; 64 x 4096 3.5 us on the card, a launch.
//
// Exact rounding without a division: with i the hardware's reciprocal of s (one
// unit off at most), x i (1 - 2^-21) and x i (1 + 2^-21), rounding errors included,
// lie on either side of x / s.  Rounding is monotone, so where both convert to one
// code that is the quotient's; where they do not, the sign of x - m s, m the
// midpoint of the two codes, decides: the fused multiply-add has it exactly.
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
// a / 448 correctly rounded: from the product q with the rounded reciprocal, whose
// remainder a - 448 q is exact, one correction (checked over every significand on
// the host); below 2^-91 the remainder could underflow.
__device__ __forceinline__ float over448(float a) {
  constexpr float r = 1.f / 448.f;
  const float q = a * r, y = fmaf(fmaf(-448.f, q, a), r, q);
  return a >= 0x1p-91f && a <= 3.40282347e38f ? y : a / 448.f;
}
__device__ __forceinline__ BlockScale block_scale(float amax, float& s) {
  BlockScale d;
  s = over448(amax);
  d.zero = !(s > 0.f && s <= 3.40282347e38f);
  d.tiny = s < 0x1p-100f;
  d.mul = d.tiny ? 0x1p64f : 1.f;
  d.s = s * d.mul;
  const float inv = __builtin_amdgcn_rcpf(d.s);
  d.lo = fmaf(inv, -0x1p-21f, inv);
  d.hi = fmaf(inv, 0x1p-21f, inv);
  return d;
}

// The largest of 16 neighbouring lanes' values, in each of them
__device__ __forceinline__ uint32_t max16(uint32_t m) {
  auto turn = [&](auto n) {  // rotated by n lanes within the sixteen
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x120 + n, 0xF, 0xF, false));
  };
  turn(std::integral_constant<int, 8>{});
  turn(std::integral_constant<int, 4>{});
  turn(std::integral_constant<int, 2>{});
  turn(std::integral_constant<int, 1>{});
  return m;
}

__device__ __forceinline__ int any_int() {  // a register as it is
  int x;
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("" : "=v"(x));
#else
  x = 0;
#endif
  return x;
}
__device__ __forceinline__ uint32_t codes2(float a, float b) {
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(a, b, any_int(), false) & 0xFFFFu;
}
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(
      c, d, __builtin_amdgcn_cvt_pk_fp8_f32(a, b, any_int(), false), true);
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


// Eight values of each of kN rows from a column on, zeros from column K on: without a
// branch where the whole wavefront is inside (its loads then go out together).
template <int kCode, int kN, class C, class F>
__device__ __forceinline__ void load_rows(RowVec<kCode> (&v)[kN], int64_t K, C&& col, F&& row) {
  constexpr int kEB = type_bytes(kCode);
  bool inside = true;
#pragma unroll
  for (int i = 0; i < kN; ++i) inside &= col(i) + 8 <= K;
  if (__all(inside)) {
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i].load(row(i), col(i));
    return;
  }
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    uint32_t w[kEB * 2] = {};
    const uint8_t* x = row(i);
    const int64_t c = col(i);
    if (c + 8 <= K) {
      v[i].load(x, c);
      continue;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (c + e < K) {
        if constexpr (kCode == kF32) w[e] = ((const uint32_t*)x)[c + e];
        else w[e / 2] |= (uint32_t)((const uint16_t*)x)[c + e] << (16 * (e & 1));
      }
    }
    v[i].load((const uint8_t*)w, 0);
  }
}
__device__ __forceinline__ void store8(uint8_t* q, int64_t c, int64_t K, uint2 w) {
  typedef uint32_t u32x2_a1 __attribute__((ext_vector_type(2), aligned(1)));
  if (c + 8 <= K) {
    __builtin_nontemporal_store(u32x2_a1{w.x, w.y}, (u32x2_a1*)(q + c));
    return;
  }
#pragma unroll 1
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
// anywhere in a line, in blocks of 128 x 128: 131 us without, 93 with).
__device__ __forceinline__ unsigned in_runs(unsigned b, unsigned n) {
  const unsigned per = n / 8, rest = n % 8, xcd = b & 7;
  return xcd * per + min(xcd, rest) + (b >> 3);
}

// 1 x 128: a workgroup has 16 kUnits blocks, 2^shift neighbours of each of its rows
// (whole rows of up to 64 blocks: the workgroup's loads, all in front of its stores,
// run through memory in order); a lane has eight values of kUnits of them.
template <int kCode, int kUnits>
__global__ __launch_bounds__(256) void quantize_row_blocks_kernel(const QuantArgs a) {
  const int tid = threadIdx.x, unit = tid >> 4;
  const unsigned id = in_runs(blockIdx.x, gridDim.x);
  const int band = id / (unsigned)a.groups, group = id % (unsigned)a.groups;
  const int mask = (1 << a.shift) - 1;
  const int64_t row0 = (int64_t)band * (16 * kUnits >> a.shift);
  auto row_of = [&](int i) { return row0 + ((unit + 16 * i) >> a.shift); };
  auto block_of = [&](int i) { return (group << a.shift) + ((unit + 16 * i) & mask); };
  auto col_of = [&](int i) { return (int64_t)block_of(i) * 128 + 8 * (tid & 15); };
  RowVec<kCode> v[kUnits];
  load_rows<kCode>(v, a.K, col_of, [&](int i) {
    return a.X + min(row_of(i), a.M - 1) * a.ldx * type_bytes(kCode);
  });
#pragma unroll
  for (int i = 0; i < kUnits; ++i) {
    const uint32_t m = max16(v[i].amax());
    float s;
    const BlockScale d = block_scale(from_bits<kCode>(m), s);
    const int64_t row = row_of(i);
    const int kb = block_of(i);
    if (row < a.M && kb < a.kbs) {
      if ((tid & 15) == 0) a.scale[row * a.s_row + kb * a.s_kb] = s;
      store8(a.Q + row * a.ldq, col_of(i), a.K, block_codes8<kCode>(v[i], d));
    }
  }
}

// 128 x 128: a workgroup a block.  (Four neighbouring blocks and 1024 threads, whose
// loads are 1 KiB of a row: 134 us instead of 93 for 16384 x 8191 bf16.)
template <int kCode>
__global__ __launch_bounds__(512) void quantize_square_blocks_kernel(const QuantArgs a) {
  const int tid = threadIdx.x;
  const unsigned id = in_runs(blockIdx.x, gridDim.x);
  const int64_t band = id / (unsigned)a.kbs;
  const int kb = id % (unsigned)a.kbs;
  const int64_t row0 = band * 128 + (tid >> 4), c = (int64_t)kb * 128 + 8 * (tid & 15);
  RowVec<kCode> v[4];
  uint32_t m = 0;
  load_rows<kCode>(v, a.K, [&](int) { return c; }, [&](int i) {
    return a.X + min(row0 + 32 * i, a.M - 1) * a.ldx * type_bytes(kCode);
  });
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, v[i].amax());  // (rows past the last are that row again)
  m = max16(m);
  m = max(m, (uint32_t)__shfl_xor((int)m, 16));
  m = max(m, (uint32_t)__shfl_xor((int)m, 32));
  __shared__ uint32_t part[8];
  if ((tid & 63) == 0) part[tid >> 6] = m;
  __syncthreads();
  for (int w = 0; w < 8; ++w) m = max(m, part[w]);
  float s;
  const BlockScale d = block_scale(from_bits<kCode>(m), s);
  if (tid == 0) a.scale[band * a.s_row + kb * a.s_kb] = s;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (row0 + 32 * i < a.M) store8(a.Q + (row0 + 32 * i) * a.ldq, c, a.K, block_codes8<kCode>(v[i], d));
}

// In launches of fewer than 2^32 threads, bands of rows at a time.
template <int kCode>
int launch(QuantArgs a, int block_rows, hipStream_t s) {
  const int64_t most = kMaxThreads / 512;  // workgroups
  a.kbs = (int)((a.K + 127) / 128);
  // 1 x 128: four blocks a lane where that still gives each compute unit eight
  // workgroups, else one
  const bool deep = a.M * (int64_t)a.kbs >= 2048 * 64;
  const int units = deep ? 64 : 16;
  a.shift = 0;
  while ((1 << a.shift) < units && (1 << a.shift) < a.kbs) ++a.shift;
  a.groups = block_rows == 1 ? (a.kbs + (1 << a.shift) - 1) >> a.shift : a.kbs;
  const int64_t rows = block_rows == 1 ? units >> a.shift : 128;  // of a workgroup
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
    if (block_rows != 1)
      hipLaunchKernelGGL((quantize_square_blocks_kernel<kCode>), grid, dim3(512), 0, s, x);
    else if (deep)
      hipLaunchKernelGGL((quantize_row_blocks_kernel<kCode, 4>), grid, dim3(256), 0, s, x);
    else
      hipLaunchKernelGGL((quantize_row_blocks_kernel<kCode, 1>), grid, dim3(256), 0, s, x);
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
