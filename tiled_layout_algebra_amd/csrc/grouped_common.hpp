// grouped_common.hpp -- what the expert-grouped kernels share: the lookup of
// a workgroup's tile from the experts' row offsets, the int8 matrix-core
// atom and the epilogue of the grouped products.
#pragma once

#include "gemm_common.hpp"
#include "operators.hpp"

namespace tla {

typedef int i32x16 __attribute__((ext_vector_type(16)));

// A matrix-core step of each operand type: MfmaAtom's 32x32 instruction with
// the accumulator type beside it.  int8 takes 16 bytes of K per lane like the
// 16-bit types (32x32x32, exact 32-bit sums), so it shares their slabs,
// fragment reads and instruction schedule.
template <int kCode>
struct OpAtom : MfmaAtom<kCode> {
  typedef f32x16 Acc;
};
template <>
struct OpAtom<kI8> {
  static constexpr int kK = 32;
  static constexpr int kLaneBytes = 16;
  typedef i32x4 Frag;
  typedef i32x16 Acc;
  static __device__ __forceinline__ void mma(i32x16& acc, const Frag& a, const Frag& b) {
    acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(a, b, acc, 0, 0, 0);
  }
};
// e4m3 through the 16-bit instruction, as f16, which holds every e4m3 value:
// the same fragments as the 8-bit instruction's (32 consecutive K per lane,
// taken 8 at a time).  The 8-bit instructions align a step's products to the
// largest and drop what falls below about its 2^-15 (measured: 2^-14.3 of two
// terms' magnitudes, 2^-15.8 of 64 terms'), which only sums of many steps
// bury under their own fp32 rounding; here every product and sum is fp32.
struct E4m3AsF16 {
  static constexpr int kK = 64;
  static constexpr int kLaneBytes = 32;
  typedef i32x8 Frag;
  typedef f32x16 Acc;
  static __device__ __forceinline__ i32x4 widen(const Frag& f, int q) {
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    i32x4 r;
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const f16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(f[2 * q + w], 1.0f, false);
      const f16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(f[2 * q + w], 1.0f, true);
      r[2 * w] = __builtin_bit_cast(int, lo);
      r[2 * w + 1] = __builtin_bit_cast(int, hi);
    }
    return r;
  }
  static __device__ __forceinline__ void mma(f32x16& acc, const Frag& a, const Frag& b) {
#pragma unroll
    for (int q = 0; q < 4; ++q) MfmaAtom<kF16>::mma(acc, widen(a, q), widen(b, q));
  }
};
// e4m3 sixteen bytes a lane at a time, like the other types: two of the
// unscaled 8-bit instructions.
struct E4m3Bytes {
  static constexpr int kK = 32;
  static constexpr int kLaneBytes = 16;
  typedef i32x4 Frag;
  typedef f32x16 Acc;
  static __device__ __forceinline__ void mma(f32x16& acc, const Frag& a, const Frag& b) {
    typedef long i64x2 __attribute__((ext_vector_type(2)));
    const i64x2 x = __builtin_bit_cast(i64x2, a), y = __builtin_bit_cast(i64x2, b);
    acc = __builtin_amdgcn_mfma_f32_32x32x16_fp8_fp8(x[0], y[0], acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_32x32x16_fp8_fp8(x[1], y[1], acc, 0, 0, 0);
  }
};
// load_frag's geometry depends only on the bytes of a K step and of a lane's
// share of it, which int8 shares with the 16-bit types.
template <int kCode>
constexpr int kFragCode = kCode == kI8 ? (int)kBF16 : kCode;

namespace {

// ------------------------------------------------------------- tile lookup
// The rows of expert e, clamped into [0, rows] and in order, so no offsets
// array, however wrong, leads an access outside A, D or Z.
__device__ __forceinline__ void expert_rows(const GroupedParams& p, int e, int& lo, int& hi) {
  if (!p.offsets) {
    lo = 0;
    hi = p.rows;
    return;
  }
  lo = min(max(p.offsets[e], 0), p.rows);
  hi = min(max(p.offsets[e + 1], lo), p.rows);
}

__device__ __forceinline__ int wave_scan(int x, int lane) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  return x;
}

// Workgroup `bid`'s tile of the ragged tiling: experts one after another,
// each cut into blocks of BM rows.  The grid holds the largest number of
// tiles that any offsets could need (row_tiles_bound); workgroups past the
// actual number get false.  Every wave finds the tile by itself with a scan
// over the experts' block counts, 64 experts at a time.  Tiles are handed to
// the XCDs (bid % 8) in contiguous runs, kGroupM blocks of rows at a time,
// rows fastest, so the workgroups sharing an L2 share an expert's columns.
struct RowTile {
  int e, r0, r1, tn;  // expert, first row, end of the expert's rows, column tile
};
template <int BM, int kGroupM = 4>
__device__ __forceinline__ bool row_tile(const GroupedParams& p, int bid, RowTile& t) {
  const int lane = threadIdx.x & 63;
  auto blocks = [&](int e) {
    int lo, hi;
    if (e >= p.groups) return 0;
    expert_rows(p, e, lo, hi);
    return (int)(((int64_t)hi - lo + BM - 1) / BM);
  };
  int total = 0, incl = 0;
  for (int g0 = 0; g0 < p.groups; g0 += 64) {
    incl = wave_scan(blocks(g0 + lane), lane);
    total += __builtin_amdgcn_readlane(incl, 63);
  }
  const int64_t tiles = (int64_t)total * p.tiles_n;
  if (bid >= tiles) return false;
  const int per = (int)(tiles / 8), rest = (int)(tiles % 8), xcd = bid & 7;
  const int id = xcd * per + min(xcd, rest) + (bid >> 3);
  const int per_group = kGroupM * p.tiles_n;
  const int first = (id / per_group) * kGroupM;
  const int gm = min(total - first, kGroupM);
  const int in = id % per_group;
  const int tm = first + in % gm;
  t.tn = in / gm;
  int before = 0;
  for (int g0 = 0; g0 < p.groups; g0 += 64) {
    if (p.groups > 64) incl = wave_scan(blocks(g0 + lane), lane);
    const uint64_t mask = __ballot(tm < before + incl);
    if (mask) {
      const int l = __builtin_ctzll(mask);
      const int excl = l ? __builtin_amdgcn_readlane(incl, l - 1) : 0;
      t.e = g0 + l;
      int lo, hi;
      expert_rows(p, t.e, lo, hi);
      t.r0 = __builtin_amdgcn_readfirstlane(lo + (tm - before - excl) * BM);
      t.r1 = __builtin_amdgcn_readfirstlane(hi);
      lo = __builtin_amdgcn_readfirstlane(lo);
      // (wrong offsets could have overflowed the sums)
      return t.r0 >= lo && t.r0 < t.r1 && (unsigned)t.tn < (unsigned)p.tiles_n;
    }
    before += __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
}

// ---------------------------------------------------------------- epilogue
// Activations that hand a NaN on (a comparison with NaN is false, so it takes
// the branch that keeps it).
__device__ __forceinline__ float relu_nan(float y) { return y < 0.f ? 0.f : y; }

// |y|, cut at 16, from where on both functions below have met their limits
__device__ __forceinline__ float abs16(float y) {
  const float a = fabsf(y);
  return a > 16.f ? 16.f : a;
}

// GELU(y) = y Phi(y) = max(y, 0) - |y| h, h = erfc(|y| / sqrt 2) / 2 = 2^P(|y|): P,
// of degree 6, is the fit of log2 h on [0, 6.5] that has the least largest error
// in h (fitted here by reweighted least squares); beyond, P keeps falling faster
// than log2 h, so h is cut off early where it no longer counts.  |Phi - exact| <=
// 1.5e-7, so GELU is off by 1.5e-7 |y| and a rounding; for y << 0, where it gets
// small itself, that is 3e-5 of the value down to y = -3, 0.25 % at -4, 2.1 % at -5 (-1.4e-6)
// and 8.9 % at -6 (-5.9e-9).  14 operations' time (56 cycles a wave), the hardware exp2
// among them; a rational erfc with its reciprocal took 21 (84) at 3e-7.  The
// epilogue applies it to 128 values a lane: int8 3001 x 4096 x 4096 with bias and
// GELU 61.8 -> 60.4 us, 8192^3 487 -> 482, and one row, which shares the code's
// size and not its work, 6.85 -> 6.24.
__device__ __forceinline__ float gelu_nan(float y) {
  const float a = abs16(y);
  float p = fmaf(a, 1.91763193e-05f, -0.000658615434f);
  p = fmaf(a, p, 0.00775443483f);
  p = fmaf(a, p, -0.0529654212f);
  p = fmaf(a, p, -0.459060252f);
  p = fmaf(a, p, -1.15112209f);
  p = fmaf(a, p, -0.999999702f);
  return fmaf(-a, __builtin_amdgcn_exp2f(p), fmaxf(y, 0.f));
}
// d/dz z Phi(z) = Phi(z) + z phi(z) = g for z < 0 and 1 - g otherwise, g = h - |z|
// phi(z) = e^(-z^2/2) R(|z|): R, of degree 9, is the fit of erfcx(|z| / sqrt 2) / 2
// - |z| / sqrt(2 pi) on [0, 6] with the least largest error in g.  In fp32 g is off
// by at most 3.2e-7, and 1 - g, rounded once more, by 3.6e-7.
__device__ __forceinline__ float gelu_slope(float z) {
  const float a = abs16(z), b = a * 0.8493218003f;  // |z| sqrt(log2(e) / 2)
  float r = fmaf(a, -8.06307162e-06f, 0.000151941887f);
  r = fmaf(a, r, -0.00127116218f);
  r = fmaf(a, r, 0.00638280576f);
  r = fmaf(a, r, -0.0222308766f);
  r = fmaf(a, r, 0.0594967976f);
  r = fmaf(a, r, -0.131772891f);
  r = fmaf(a, r, 0.249752298f);
  r = fmaf(a, r, -0.797864914f);
  r = fmaf(a, r, 0.499999732f);
  const float g = r * __builtin_amdgcn_exp2f(b * -b);
  return z < 0.f ? g : 1.f - g;
}

// 16 bytes from an even address (one load: vector loads need no alignment
// beyond the element's here)
__device__ __forceinline__ i32x4 load16_even(const uint8_t* p) {
  typedef int i32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
  return *(const i32x4_a2*)p;
}

// A wave's 32 FM x 32 FN piece of D in 16-bit form in its LDS region: rows
// of 64 FN bytes, the 16-byte chunks XOR-swizzled by row so that the
// lane-per-row accesses of the MFMA layout fall into distinct banks.  Lane l
// holds row 32 i + l % 32, columns 32 j + 8 g + 4 (l / 32) .. + 3.
template <int FM, int FN>
struct WaveRegion {
  static constexpr int kRowB = 64 * FN, kCh = kRowB / 16, kRowsPerKiB = 1024 / kRowB;
  static constexpr int kIters = 32 * FM * kRowB / 1024;
  static_assert(kCh == 4 || kCh == 8 || kCh == 16, "row width");
  static __device__ __forceinline__ int swz(int r, int c) {
    return c ^ ((r / (16 / kCh)) & (kCh - 1));
  }
  static __device__ __forceinline__ uint8_t* slot(uint8_t* region, int lane, int i, int j, int g) {
    const int r = 32 * i + (lane & 31);
    return region + r * kRowB + swz(r, 4 * j + g) * 16 + 8 * (lane >> 5);
  }
  // region -> rows x cols of a row-major 16-bit matrix at `base`, whole rows
  // per instruction; v16: rows are 16-byte aligned
  static __device__ __forceinline__ void store(uint8_t* base, int64_t ld, const uint8_t* region,
                                               int lane, int rows, int cols, bool v16) {
    const int rr = lane / kCh, cs = lane % kCh;
#pragma unroll
    for (int t = 0; t < kIters; ++t) {
      const int r = kRowsPerKiB * t + rr;
      const int c0 = 8 * swz(r, cs);
      const i32x4 v = *(const i32x4*)(region + t * 1024 + lane * 16);
      uint8_t* dst = base + ((int64_t)r * ld + c0) * 2;
      if (r < rows) {
        if (c0 + 8 <= cols) {
          if (v16) *(i32x4*)dst = v;
          else store16_even(dst, v);
        } else if (c0 < cols) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (c0 + e < cols)
              ((uint16_t*)dst)[e] = (uint16_t)((uint32_t)v[e >> 1] >> (16 * (e & 1)));
        }
      }
    }
  }
  // the other way round; elements outside rows x cols are left as they are
  static __device__ __forceinline__ void load(const uint8_t* base, int64_t ld, uint8_t* region,
                                              int lane, int rows, int cols) {
    const int rr = lane / kCh, cs = lane % kCh;
#pragma unroll
    for (int t = 0; t < kIters; ++t) {
      const int r = kRowsPerKiB * t + rr;
      const int c0 = 8 * swz(r, cs);
      const uint8_t* src = base + ((int64_t)min(r, rows - 1) * ld + c0) * 2;
      i32x4 x = {0, 0, 0, 0};
      if (c0 + 8 <= cols) x = load16_even(src);
      else if (c0 < cols) x = gather16<2>(src - c0 * 2, 2, c0, cols, cols - 1);
      *(i32x4*)(region + t * 1024 + lane * 16) = x;
    }
  }
};

template <int FM, int FN, class F>
__device__ __forceinline__ void each_group(F&& f) {
  static_for<FM>([&](auto i) {
    static_for<FN>([&](auto j) { static_for<4>([&](auto g) { f(i, j, g); }); });
  });
}

// Scale and bias of a lane's four column groups of fragment j: columns
// n + 8 g .. + 3 of a row of N, clamped to the last column.
struct ColumnTerms {
  f32x4 s[4], b[4];
};
template <bool kScaled>
__device__ __forceinline__ void load_columns(const GroupedParams& p, int e, int n, ColumnTerms& t) {
  const bool vec = (p.flags & kOpVec4) && n + 27 < p.N;
  static_for<4>([&](auto g) {
    t.s[g] = f32x4{1.f, 1.f, 1.f, 1.f};
    t.b[g] = f32x4{0.f, 0.f, 0.f, 0.f};
  });
  auto fetch = [&](const uint8_t* base, int type, f32x4 (&x)[4]) {
    if (vec && type == TLA_F32) {
      static_for<4>([&](auto g) { x[g] = *(const f32x4*)((const float*)base + n + 8 * g); });
    } else if (vec) {
      uint2 u[4];
      static_for<4>([&](auto g) { u[g] = *(const uint2*)((const uint16_t*)base + n + 8 * g); });
      static_for<4>([&](auto g) {
        x[g] = type == TLA_BF16
                   ? f32x4{widen_lo<true>(u[g].x), widen_hi<true>(u[g].x), widen_lo<true>(u[g].y),
                           widen_hi<true>(u[g].y)}
                   : f32x4{widen_lo<false>(u[g].x), widen_hi<false>(u[g].x),
                           widen_lo<false>(u[g].y), widen_hi<false>(u[g].y)};
      });
    } else {
      static_for<4>([&](auto g) {
        static_for<4>([&](auto q) { x[g][(int)q] = load_elem(base, type, min(n + 8 * g + q, p.N - 1)); });
      });
    }
  };
  if (p.bias) fetch(p.bias + (int64_t)e * p.N * type_bytes(p.bias_type), p.bias_type, t.b);
  if constexpr (kScaled) {
    if (p.sb) fetch((const uint8_t*)(p.sb + (int64_t)e * p.N), TLA_F32, t.s);
  }
}

// What the epilogue makes of y: itself, its activation, or y times the
// activation's derivative at a stored z.
enum EpiOp : int { kSame, kRelu, kGelu, kReluGrad, kGeluGrad };
template <int kOp>
__device__ __forceinline__ float epi_op(float y, float z) {
  if constexpr (kOp == kRelu) return relu_nan(y);
  if constexpr (kOp == kGelu) return gelu_nan(y);
  if constexpr (kOp == kReluGrad) return y * (z > 0.f ? 1.f : 0.f);
  if constexpr (kOp == kGeluGrad) return y * gelu_slope(z);
  return y;
}

// One pass over a wave's accumulators into its region: op(sa s acc + b), four
// columns at a time, in the MFMA layout; the derivatives read their z from
// the slot they write.  A fragment's column terms are loaded while the one
// before it is worked on.
template <int kCode, int kOp, bool kBf, int FM, int FN>
__device__ __forceinline__ void epilogue_pass(const GroupedParams& p, int e, int col, int lane,
                                              const typename OpAtom<kCode>::Acc (&acc)[FM][FN],
                                              const float (&sa)[FM], uint8_t* region) {
  using R = WaveRegion<FM, FN>;
  constexpr bool kScaled = kCode == kI8 || kCode == kE4M3;
  constexpr bool kSlope = kOp == kReluGrad || kOp == kGeluGrad;
  const int n0 = col + 4 * (lane >> 5);
  ColumnTerms t[2];
  load_columns<kScaled>(p, e, n0, t[0]);
  static_for<FN>([&](auto j) {
    if constexpr (j + 1 < FN) load_columns<kScaled>(p, e, n0 + 32 * (j + 1), t[(j + 1) & 1]);
    const ColumnTerms& c = t[j & 1];
    static_for<4>([&](auto g) {
      static_for<FM>([&](auto i) {
        uint8_t* slot = R::slot(region, lane, i, j, g);
        float z[4] = {0.f, 0.f, 0.f, 0.f}, y[4];
        if constexpr (kSlope) {
          const uint2 u = *(const uint2*)slot;
          z[0] = widen_lo<kBf>(u.x);
          z[1] = widen_hi<kBf>(u.x);
          z[2] = widen_lo<kBf>(u.y);
          z[3] = widen_hi<kBf>(u.y);
        }
        static_for<4>([&](auto q) {
          const float a = (float)acc[i][j][4 * g + q];
          const float v = kScaled ? fmaf(a * sa[i], c.s[g][(int)q], c.b[g][(int)q]) : a + c.b[g][(int)q];
          y[q] = epi_op<kOp>(v, z[q]);
        });
        *(uint2*)slot = uint2{pack2<kBf>(y[0], y[1]), pack2<kBf>(y[2], y[3])};
      });
    });
  });
}

// The grouped product's epilogue for one wave's accumulators: rows row ..,
// columns col .. of D, the expert's rows end at r1.
//   y = sa sb acc + bias;  D = act(y), or y act'(Z);  Z = y when it is kept.
// fp32 throughout; one rounding to D's type at the store (Z holds y rounded
// to the same type).  region: 64 FN x 32 FM bytes of LDS of the wave's own.
template <int kCode, int FM, int FN>
__device__ __forceinline__ void grouped_epilogue(const GroupedParams& p, int e, int r1, int row,
                                                 int col, int lane,
                                                 const typename OpAtom<kCode>::Acc (&acc)[FM][FN],
                                                 uint8_t* region) {
  using R = WaveRegion<FM, FN>;
  const int rows = min(32 * FM, r1 - row), cols = min(32 * FN, p.N - col);
  if (rows <= 0 || cols <= 0) return;
  const bool bf = p.d_type == TLA_BF16, v16 = p.flags & kOpD16;
  float sa[FM];
  static_for<FM>([&](auto i) {
    sa[i] = p.sa ? p.sa[row + min(32 * (int)i + (lane & 31), rows - 1)] : 1.f;
  });
  auto fence = [&]() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); };
  auto pass = [&](auto op, uint8_t* out, int64_t ld) {
    if (bf) epilogue_pass<kCode, op, true, FM, FN>(p, e, col, lane, acc, sa, region);
    else epilogue_pass<kCode, op, false, FM, FN>(p, e, col, lane, acc, sa, region);
    fence();
    R::store(out + ((int64_t)row * ld + col) * 2, ld, region, lane, rows, cols, v16);
  };
  if (p.z_mode == TLA_Z_GRAD) {
    R::load(p.Z + ((int64_t)row * p.ldz + col) * 2, p.ldz, region, lane, rows, cols);
    fence();
    if (p.act == TLA_ACT_RELU) pass(std::integral_constant<int, kReluGrad>{}, p.D, p.ldd);
    else pass(std::integral_constant<int, kGeluGrad>{}, p.D, p.ldd);
    return;
  }
  if (p.z_mode == TLA_Z_STORE) {
    pass(std::integral_constant<int, kSame>{}, p.Z, p.ldz);
    fence();
  }
  if (p.act == TLA_ACT_RELU) pass(std::integral_constant<int, kRelu>{}, p.D, p.ldd);
  else if (p.act == TLA_ACT_GELU) pass(std::integral_constant<int, kGelu>{}, p.D, p.ldd);
  else pass(std::integral_constant<int, kSame>{}, p.D, p.ldd);
}

// The weight gradient's epilogue: D_e rows m .., columns n .. of M x N, row
// major, in fp32 or rounded once to 16 bits.
template <int FM, int FN>
__device__ __forceinline__ void wgrad_epilogue(const GroupedParams& p, int e, int m, int n,
                                               int lane, const f32x16 (&acc)[FM][FN],
                                               uint8_t* region) {
  using R = WaveRegion<FM, FN>;
  const int rows = min(32 * FM, p.M - m), cols = min(32 * FN, p.N - n);
  if (rows <= 0 || cols <= 0) return;
  const int64_t at = (int64_t)e * p.stride_d + (int64_t)m * p.ldd + n;
  const bool v16 = p.flags & kOpD16;
  if (p.d_type == TLA_F32) {
    float* D = (float*)p.D + at;
    each_group<FM, FN>([&](auto i, auto j, auto g) {
      const int r = 32 * i + (lane & 31), c = 32 * j + 8 * g + 4 * (lane >> 5);
      if (r < rows) {
        float* d = D + (int64_t)r * p.ldd + c;
        if (c + 3 < cols) {
          // vector stores need the element's alignment only
          typedef float f32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
          *(f32x4_a4*)d = f32x4_a4{acc[i][j][4 * g], acc[i][j][4 * g + 1], acc[i][j][4 * g + 2],
                             acc[i][j][4 * g + 3]};
        } else {
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (c + q < cols) d[q] = acc[i][j][4 * g + q];
        }
      }
    });
    return;
  }
  auto run = [&](auto kb) {
    each_group<FM, FN>([&](auto i, auto j, auto g) {
      *(uint2*)R::slot(region, lane, i, j, g) =
          uint2{pack2<kb>(acc[i][j][4 * g], acc[i][j][4 * g + 1]),
                pack2<kb>(acc[i][j][4 * g + 2], acc[i][j][4 * g + 3])};
    });
  };
  if (p.d_type == TLA_BF16) run(std::true_type{});
  else run(std::false_type{});
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  R::store(p.D + at * 2, p.ldd, region, lane, rows, cols, v16);
}

// The bias gradient beside the weight gradient: sums over k of each line (a
// column of dY) of an operand's fragments.  A 32x32 fragment's lane l holds eight
// values of line l % 32, K half l / 32.  The matrix instruction of sixteen 4x4
// blocks takes each lane as a column of its own block, so with ones as the other
// operand every result of lane l is the sum of that lane's four values: two of
// them a fragment, and a line never meets another one, whose infinity or NaN (a
// neighbour's, or the padding's behind the last column) stays in its own sum.
// Four registers a fragment.  One block of tiles along the other extent does it:
// 516 us instead of 505 for 16384 rows on 8 experts of 4096 x 4096, where a pass
// over dY of its own took 26; it reads nothing more.
template <int kCode, int kN>
struct LineSums {
  f32x4 s[kN];
  __device__ __forceinline__ void init() {
    static_for<kN>([&](auto i) { s[i] = f32x4{0.f, 0.f, 0.f, 0.f}; });
  }
  template <int kI>
  __device__ __forceinline__ void add(const i32x4& f) {
    typedef int i32x2 __attribute__((ext_vector_type(2)));
    static_for<2>([&](auto h) {
      const i32x2 x = {f[2 * h], f[2 * h + 1]};
      if constexpr (kCode == kBF16) {
        const i32x2 ones = {0x3F803F80, 0x3F803F80};
        s[kI] = __builtin_amdgcn_mfma_f32_4x4x4bf16_1k(__builtin_bit_cast(s16x4, ones),
                                                       __builtin_bit_cast(s16x4, x), s[kI], 0, 0, 0);
      } else {
        typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
        const i32x2 ones = {0x3C003C00, 0x3C003C00};
        s[kI] = __builtin_amdgcn_mfma_f32_4x4x4f16(__builtin_bit_cast(f16x4, ones),
                                                   __builtin_bit_cast(f16x4, x), s[kI], 0, 0, 0);
      }
    });
  }
  // the sums of fragment i's lines first + 32 i .. that lie below `lines`
  template <int kCount>
  __device__ __forceinline__ void write(float* out, int first, int lines, int lane) const {
    static_for<kCount>([&](auto i) {
      const float sum = s[i][0] + __shfl_xor(s[i][0], 32);  // the two K halves
      const int n = first + 32 * i + lane;
      if (lane < 32 && n < lines) out[n] = sum;
    });
  }
};

// Workgroup `bid`'s tile of the weight gradient: expert e, tile (tm, tn) of
// its D_e; an XCD's run of tiles stays within one expert, whose rows its L2
// then serves to all of them.
__device__ __forceinline__ void wgrad_tile(const GroupedParams& p, int bid, int total, int& e,
                                           int& tm, int& tn) {
  const int per = total / 8, rest = total % 8, xcd = bid & 7;
  const int id = xcd * per + min(xcd, rest) + (bid >> 3);
  const int tiles = p.tiles_m * p.tiles_n;
  e = id / tiles;
  const int in_e = id - e * tiles;
  const int per_group = 4 * p.tiles_n;
  const int first = (in_e / per_group) * 4;
  const int gm = min(p.tiles_m - first, 4);
  const int in = in_e % per_group;
  tm = first + in % gm;
  tn = in / gm;
}

}  // namespace
}  // namespace tla
