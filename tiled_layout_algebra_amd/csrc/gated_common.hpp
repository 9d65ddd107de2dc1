// gated_common.hpp -- what the kernels of the gated feed-forward products and
// of the block-scaled e4m3 product share: the block-scaled matrix-core atom and
// the epilogues.
//
//   forward   g = sum + bias, u = sum + bias, H = act(g) u
//   backward  dh = sum;  dgate = dh u act'(g),  dup = dh act(g),  H = act(g) u
//   SiLU      z s(z), derivative s(z) (1 + z (1 - s(z))), s(z) = 1 / (1 + e^-z)
//   GELU      the polynomials of grouped_common.hpp
// All in fp32 from the fp32 sums; each result is rounded once, when it is written.
#pragma once

#include "grouped_common.hpp"

namespace tla {

// e4m3 with a scale for each block of 128 along K: the 16x16x128 instruction
// takes a whole block, from a zero accumulator, and the caller adds its result
// times the two operands' scales to an fp32 sum.  (A 32x32 result would hold 16
// registers of a block's partial sums at a time instead of 4.)  Lane l holds 32
// consecutive K of row l % 16; results: row l % 16 of the second operand,
// columns 4 (l / 16) .. + 3 of the first.
template <>
struct OpAtom<kE4M3Blocks> {
  static constexpr int kK = 128;
  static constexpr int kLaneBytes = 32;
  typedef i32x8 Frag;
  typedef f32x4 Acc;
  static __device__ __forceinline__ f32x4 block(const Frag& a, const Frag& b) {
    const f32x4 zero = {0.f, 0.f, 0.f, 0.f};
    // (scales of 0: the form of the instruction without any, which issues a cycle or two sooner)
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, zero, 0, 0, 0, 0, 0, 0);
  }
};

namespace {

// The sums of a wave's MFMA tiles over blocks of 128 of K: acc += scale part, a
// tile's sum kAhead instructions behind its matrix instruction, so that these
// follow each other without waiting for a result.  s[0]: the scales of the plain
// sums or of the first half of the columns (the gate's), s[1]: of the other half.
// mma: a k-tile's matrix instructions and all but the last kAhead sums; b holds FB
// of the FN column fragments, and after(j) is called behind the last use of fragment
// j where j + FB < FN, to read fragment j + FB in its place.  finish: those last
// sums, which may wait (with their scales) until the matrix cores are another
// wave's.
template <int FM, int FN, bool kTwo>
struct BlockSums {
  static constexpr int kN = FM * FN, kAhead = 3;
  f32x4 acc[FM][FN], part[kAhead];
  __device__ __forceinline__ void init() {
    static_for<FM>([&](auto i) { static_for<FN>([&](auto j) { acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f}; }); });
  }
  template <int y>
  __device__ __forceinline__ void add(const float (&s)[2][FM]) {
    constexpr int i = y % FM, j = y / FM;
    const float c = s[kTwo && j >= FN / 2][i];
    static_for<4>([&](auto q) {
      acc[i][j][(int)q] = fmaf(part[y % kAhead][(int)q], c, acc[i][j][(int)q]);
    });
  }
  template <int FB, class F>
  __device__ __forceinline__ void mma(const i32x8 (&a)[FM], i32x8 (&b)[FB], const float (&s)[2][FM],
                                      F&& after) {
    static_for<kN>([&](auto x) {
      if constexpr (x >= kAhead) add<x - kAhead>(s);
      part[x % kAhead] = OpAtom<kE4M3Blocks>::block(b[x / FM % FB], a[x % FM]);
      if constexpr (x % FM == FM - 1 && x / FM + FB < FN) after(std::integral_constant<int, x / FM>{});
      __builtin_amdgcn_sched_barrier(0);  // in this order
    });
  }
  // The whole k-tile with e4m3 widened to f16, which holds every e4m3 value: here each
  // product and sum is fp32, where the 8-bit instruction drops what lies far below a
  // block's largest term.
  __device__ __forceinline__ void mma_wide(const i32x8 (&a)[FM], const i32x8 (&b)[FN],
                                           const float (&s)[2][FM]) {
    i32x4 wa[FM][4];
    static_for<FM>([&](auto i) { static_for<4>([&](auto q) { wa[i][q] = E4m3AsF16::widen(a[i], q); }); });
    static_for<FN>([&](auto j) {
      i32x4 wb[4];
      static_for<4>([&](auto q) { wb[q] = E4m3AsF16::widen(b[j], q); });
      static_for<FM>([&](auto i) {
        f32x4 x = {0.f, 0.f, 0.f, 0.f};
        static_for<4>([&](auto q) {
          x = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, wb[q]),
                                                     __builtin_bit_cast(f16x8, wa[i][q]), x, 0, 0, 0);
        });
        const float c = s[kTwo && j >= FN / 2][i];
        static_for<4>([&](auto q) { acc[i][j][(int)q] = fmaf(x[(int)q], c, acc[i][j][(int)q]); });
      });
    });
  }
  __device__ __forceinline__ void finish(const float (&s)[2][FM]) {
    static_for<kAhead>([&](auto x) { add<kN - kAhead + x>(s); });
  }
  // keeps the matrix instructions in front of what follows
  __device__ __forceinline__ void pin() {
#if defined(__HIP_DEVICE_COMPILE__)
    static_for<kAhead>([&](auto x) { asm volatile("" : "+v"(part[x])); });
#endif
  }
};

// sigmoid(z) = 1 / (1 + 2^(-z log2 e)) by the hardware's exp2 and reciprocal
// (one unit each, 2 2^-24).  The constant is off by 0.22 2^-24 and the product rounds
// by 2^-24, of |z| in the exponent: with the sum's rounding at most (1.25 |z| + 5) 2^-24
// of its value (largest seen: 0.92 of that, over 2^24 values of each range to -87).
__device__ __forceinline__ float sigmoid(float z) {
  return __builtin_amdgcn_rcpf(1.f + __builtin_amdgcn_exp2f(z * -1.44269504f));
}

// The activation of a kernel: kLinear is ReLU, or with p.act TLA_ACT_NONE nothing
// (one code for both), the others themselves.
enum Act : int { kLinear = TLA_ACT_RELU, kGeluAct = TLA_ACT_GELU, kSiluAct = TLA_ACT_SILU };
template <int kAct>
__device__ __forceinline__ float act_value(float z, bool none) {
  if constexpr (kAct == kGeluAct) return gelu_nan(z);
  if constexpr (kAct == kSiluAct) return z * sigmoid(z);
  return z < 0.f && !none ? 0.f : z;
}
// act(z) and act'(z); SiLU: p + z p (1 - p), p = sigmoid(z)
template <int kAct>
__device__ __forceinline__ void act_both(float z, bool none, float& value, float& slope) {
  if constexpr (kAct == kSiluAct) {
    const float s = sigmoid(z);
    value = z * s;
    slope = fmaf(value, 1.f - s, s);
  } else {
    value = act_value<kAct>(z, none);
    slope = kAct == kGeluAct ? gelu_slope(z) : z > 0.f || none ? 1.f : 0.f;
  }
}
// f(integral_constant<Act>) for p.act
template <class F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  if (act == TLA_ACT_SILU) f(std::integral_constant<int, kSiluAct>{});
  else if (act == TLA_ACT_GELU) f(std::integral_constant<int, kGeluAct>{});
  else f(std::integral_constant<int, kLinear>{});
}
__device__ __forceinline__ float act_any(float z, int act) {
  float y = z;
  with_act(act, [&](auto a) { y = act_value<a>(z, act == TLA_ACT_NONE); });
  return y;
}

// v, which the compiler has to take for different in each lane: a load at this offset
// is a vector load, in order with the others in vmcnt, where one that is the same for
// all lanes may become a scalar load, which vmcnt does not count.
__device__ __forceinline__ int64_t per_lane(int64_t v) {
#if defined(__HIP_DEVICE_COMPILE__)
  asm volatile("" : "+v"(v));
#endif
  return v;
}

// Orders a wave's LDS accesses of different types
__device__ __forceinline__ void wave_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

// A wave's WM x WN piece of a row-major 16-bit matrix in LDS (WaveRegion) seen from
// MFMA tiles of FR rows: FR 32: lane l holds row 32 i + l % 32, columns 32 j + 8 g +
// 4 (l / 32) .. + 3; FR 16: row 16 i + l % 16, columns 16 j + 4 (l / 16) .. + 3.
// WM <= 64.
template <int FR, int WM, int WN>
struct Piece {
  using R = WaveRegion<WM / 32, WN / 32>;
  static constexpr int kG = FR == 32 ? 4 : 1, kBytes = WM * WN * 2, kIters = R::kIters;
  static __device__ __forceinline__ int column(int lane, int j, int g) {
    return FR * j + 8 * g + 4 * (lane / FR);
  }
  static __device__ __forceinline__ uint2* slot(uint8_t* region, int lane, int i, int j, int g) {
    const int r = FR * i + lane % FR, c = column(lane, j, g);
    return (uint2*)(region + r * R::kRowB + R::swz(r, c / 8) * 16 + (c & 4) * 2);
  }
  // row and first column of the 16-byte chunk at region + 1024 t + 16 lane
  static __device__ __forceinline__ int row(int lane, int t) { return R::kRowsPerKiB * t + lane / R::kCh; }
  static __device__ __forceinline__ int chunk(int lane, int t) { return 8 * R::swz(row(lane, t), lane % R::kCh); }
  // where element c of row r lies in the region
  static __device__ __forceinline__ uint16_t* elem(uint8_t* region, int r, int c) {
    return (uint16_t*)(region + r * R::kRowB + R::swz(r, c / 8) * 16 + (c & 7) * 2);
  }
  // rows x cols of a piece into registers (whole chunks of them) ...  These loads and
  // the stores below pass the caches by: operands stay there instead (8192 x 8192 x
  // 4096, the gradient 579 us -> 539, the gated product with gate and up kept 860 -> 845).
  typedef int i32x4_a2 __attribute__((ext_vector_type(4), aligned(2)));
  static __device__ __forceinline__ void fetch(const uint8_t* base, int64_t ld, i32x4 (&v)[kIters],
                                               int lane, int rows, int cols) {
    const uint8_t* from = base + (int64_t)(lane / R::kCh) * ld * 2;
#pragma unroll
    for (int t = 0; t < kIters; ++t) {
      v[t] = i32x4{0, 0, 0, 0};
      if (row(lane, t) < rows && chunk(lane, t) + 8 <= cols)
        v[t] = __builtin_nontemporal_load(
            (const i32x4_a2*)(from + (int64_t)(R::kRowsPerKiB * t) * ld * 2 + chunk(lane, t) * 2));
    }
  }
  // ... and from there into the region, with the elements of the chunk that the
  // last column cuts, a lane a row
  static __device__ __forceinline__ void put(const uint8_t* base, int64_t ld, const i32x4 (&v)[kIters],
                                             uint8_t* region, int lane, int rows, int cols) {
#pragma unroll
    for (int t = 0; t < kIters; ++t) *(i32x4*)(region + t * 1024 + lane * 16) = v[t];
    if (cols < WN && cols % 8 != 0 && lane < rows) {
      wave_fence();
#pragma unroll 1
      for (int c = cols & ~7; c < cols; ++c)
        *elem(region, lane, c) = ((const uint16_t*)base)[(int64_t)lane * ld + c];
    }
  }
  // region -> rows x cols of the matrix; v16: its rows are 16-byte aligned
  static __device__ __forceinline__ void store(uint8_t* base, int64_t ld, uint8_t* region, int lane,
                                               int rows, int cols, bool v16) {
    uint8_t* to = base + (int64_t)(lane / R::kCh) * ld * 2;
#pragma unroll
    for (int t = 0; t < kIters; ++t) {
      const i32x4 v = *(const i32x4*)(region + t * 1024 + lane * 16);
      uint8_t* dst = to + (int64_t)(R::kRowsPerKiB * t) * ld * 2 + chunk(lane, t) * 2;
      if (row(lane, t) < rows && chunk(lane, t) + 8 <= cols) {
        if (v16) __builtin_nontemporal_store(v, (i32x4*)dst);
        else store16_even(dst, v);
      }
    }
    if (cols < WN && cols % 8 != 0 && lane < rows) {
#pragma unroll 1
      for (int c = cols & ~7; c < cols; ++c)
        ((uint16_t*)base)[(int64_t)lane * ld + c] = *elem(region, lane, c);
    }
  }
};

// Four bias values from column n (clamped to the last) of expert e
__device__ __forceinline__ f32x4 bias4(const GroupedParams& p, const uint8_t* bias, int e, int n) {
  f32x4 x;
  const int64_t at = (int64_t)e * p.N;
  static_for<4>([&](auto q) { x[(int)q] = load_elem(bias, p.bias_type, at + min(n + q, p.N - 1)); });
  return x;
}

// One pass over pairs of sums: f(gate, up) packed into a region.
template <int FR, int WM, int WN, bool kBf, class Acc, int FM, int FN, class F>
__device__ __forceinline__ void pair_pass(int lane, const Acc (&acc)[FM][FN], uint8_t* region, F&& f) {
  using P = Piece<FR, WM, WN>;
  static_for<FN / 2>([&](auto j) {
    static_for<P::kG>([&](auto g) {
      static_for<FM>([&](auto i) {
        float y[4];
        static_for<4>([&](auto q) { y[q] = f(acc[i][j][4 * g + q], acc[i][j + FN / 2][4 * g + q]); });
        *P::slot(region, lane, i, j, g) = uint2{pack2<kBf>(y[0], y[1]), pack2<kBf>(y[2], y[3])};
      });
    });
  });
}

// The gated product's epilogue for a wave's sums: rows row .., columns col ..
// (WN of them) of the hidden layer, the expert's rows end at r1; tiles j < FN / 2
// are the gate's, the others the up projection's.  fp32 throughout, one rounding
// for each output.  region: 2 WM WN 16-bit values.
template <int FR, int WM, int WN, int kAct, bool kBf, class Acc, int FM, int FN>
__device__ __forceinline__ void gated_epilogue(const GroupedParams& p, int e, int r1, int row,
                                               int col, int lane, Acc (&acc)[FM][FN],
                                               uint8_t* region) {
  using P = Piece<FR, WM, WN>;
  const int rows = min(WM, r1 - row), cols = min(WN, p.N - col);
  if (rows <= 0 || cols <= 0) return;
  const bool v16 = p.flags & kOpD16, none = p.act == TLA_ACT_NONE;
  if (p.bias || p.bias2) {
    static_for<FN>([&](auto j) {
      const uint8_t* bias = j < FN / 2 ? p.bias : p.bias2;
      if (bias) {
        static_for<P::kG>([&](auto g) {
          const f32x4 b = bias4(p, bias, e, col + P::column(lane, j % (FN / 2), g));
          static_for<FM>([&](auto i) {
            static_for<4>([&](auto q) { acc[i][j][4 * g + q] += b[(int)q]; });
          });
        });
      }
    });
  }
  if (p.Z) {
    pair_pass<FR, WM, WN, kBf>(lane, acc, region, [](float g, float) { return g; });
    pair_pass<FR, WM, WN, kBf>(lane, acc, region + P::kBytes, [](float, float u) { return u; });
    wave_fence();
    const int64_t at = ((int64_t)row * p.ldz + col) * 2;
    P::store(p.Z + at, p.ldz, region, lane, rows, cols, v16);
    P::store(p.Z2 + at, p.ldz, region + P::kBytes, lane, rows, cols, v16);
    wave_fence();
  }
  pair_pass<FR, WM, WN, kBf>(lane, acc, region,
                             [&](float g, float u) { return act_value<kAct>(g, none) * u; });
  wave_fence();
  P::store(p.D + ((int64_t)row * p.ldd + col) * 2, p.ldd, region, lane, rows, cols, v16);
}

// What the gradient's epilogue reads: a part's gate and up as whole rows, in
// registers.  Parts are half a wave's columns, or all 32.
template <int WM, int WN>
struct GateParts {
  static constexpr int kPart = WN >= 64 ? WN / 2 : WN, kParts = WN / kPart;
  using P = Piece<32, WM, kPart>;
  i32x4 g[P::kIters], u[P::kIters];
  __device__ __forceinline__ void ask(const GroupedParams& p, int r1, int row, int col, int lane, int part) {
    const int c = col + part * kPart, rows = min(WM, r1 - row), cols = min(kPart, p.N - c);
    const int64_t at = ((int64_t)row * p.ldz + c) * 2;
    P::fetch(p.Z + at, p.ldz, g, lane, rows, cols);
    P::fetch(p.Z2 + at, p.ldz, u, lane, rows, cols);
  }
};

// The gradient's epilogue: acc is dh; D = dh up act'(gate), D2 = dh act(gate),
// H = act(gate) up with gate and up read from Z and Z2.  z holds the first part;
// the next one comes while a part is worked on.  A part goes through LDS into the
// MFMA layout, the gradients go back the same way, the hidden layer waits in the
// sums' registers.  region: WM WN 16-bit values, 2 WM WN for WN = 32.
template <int WM, int WN, int kAct, bool kBf, int FM, int FN>
__device__ __forceinline__ void gate_grad_epilogue(const GroupedParams& p, int r1, int row, int col,
                                                   int lane, f32x16 (&acc)[FM][FN],
                                                   GateParts<WM, WN>& z, uint8_t* region) {
  using G = GateParts<WM, WN>;
  using P = typename G::P;
  constexpr int kPart = G::kPart, FP = kPart / 32, kParts = G::kParts;
  const int rows = min(WM, r1 - row);
  if (rows <= 0 || col >= p.N) return;
  const bool v16 = p.flags & kOpD16, none = p.act == TLA_ACT_NONE;
  uint8_t* region2 = region + P::kBytes;
  static_for<kParts>([&](auto part) {
    const int c = col + part * kPart, cols = min(kPart, p.N - c);
    if (cols <= 0) return;
    const int64_t dat = ((int64_t)row * p.ldd + c) * 2, zat = ((int64_t)row * p.ldz + c) * 2;
    P::put(p.Z + zat, p.ldz, z.g, region, lane, rows, cols);
    P::put(p.Z2 + zat, p.ldz, z.u, region2, lane, rows, cols);
    if constexpr (part + 1 < kParts) z.ask(p, r1, row, col, lane, part + 1);
    wave_fence();
    static_for<FP>([&](auto jj) {
      constexpr int j = part * FP + jj;
      static_for<4>([&](auto g) {
        static_for<FM>([&](auto i) {
          uint2 *gate = P::slot(region, lane, i, jj, g), *up = P::slot(region2, lane, i, jj, g);
          const uint2 wg = *gate, wu = *up;
          const float g4[4] = {widen_lo<kBf>(wg.x), widen_hi<kBf>(wg.x), widen_lo<kBf>(wg.y),
                               widen_hi<kBf>(wg.y)};
          const float u4[4] = {widen_lo<kBf>(wu.x), widen_hi<kBf>(wu.x), widen_lo<kBf>(wu.y),
                               widen_hi<kBf>(wu.y)};
          float dg[4], du[4];
          static_for<4>([&](auto q) {
            float value, slope;
            act_both<kAct>(g4[q], none, value, slope);
            const float dh = acc[i][j][4 * g + q];
            dg[q] = dh * (u4[q] * slope);
            du[q] = dh * value;
            acc[i][j][4 * g + q] = value * u4[q];
          });
          *gate = uint2{pack2<kBf>(dg[0], dg[1]), pack2<kBf>(dg[2], dg[3])};
          *up = uint2{pack2<kBf>(du[0], du[1]), pack2<kBf>(du[2], du[3])};
        });
      });
    });
    wave_fence();
    P::store(p.D + dat, p.ldd, region, lane, rows, cols, v16);
    P::store(p.D2 + dat, p.ldd, region2, lane, rows, cols, v16);
    wave_fence();
    if (p.H) {
      static_for<FP>([&](auto jj) {
        constexpr int j = part * FP + jj;
        static_for<4>([&](auto g) {
          static_for<FM>([&](auto i) {
            *P::slot(region, lane, i, jj, g) =
                uint2{pack2<kBf>(acc[i][j][4 * g], acc[i][j][4 * g + 1]),
                      pack2<kBf>(acc[i][j][4 * g + 2], acc[i][j][4 * g + 3])};
          });
        });
      });
      wave_fence();
      P::store(p.H + ((int64_t)row * p.ldh + c) * 2, p.ldh, region, lane, rows, cols, v16);
      wave_fence();
    }
  });
}

// The block-scaled product's epilogue: D = act(sum + bias).
template <int WM, int WN, int kAct, bool kBf, int FM, int FN>
__device__ __forceinline__ void blocks_epilogue(const GroupedParams& p, int e, int r1, int row,
                                                int col, int lane, f32x4 (&acc)[FM][FN],
                                                uint8_t* region) {
  using P = Piece<16, WM, WN>;
  const int rows = min(WM, r1 - row), cols = min(WN, p.N - col);
  if (rows <= 0 || cols <= 0) return;
  const bool none = p.act == TLA_ACT_NONE;
  if (p.bias) {
    static_for<FN>([&](auto j) {
      const f32x4 b = bias4(p, p.bias, e, col + P::column(lane, j, 0));
      static_for<FM>([&](auto i) { acc[i][j] += b; });
    });
  }
  static_for<FN>([&](auto j) {
    static_for<FM>([&](auto i) {
      float y[4];
      static_for<4>([&](auto q) { y[q] = act_value<kAct>(acc[i][j][(int)q], none); });
      *P::slot(region, lane, i, j, 0) = uint2{pack2<kBf>(y[0], y[1]), pack2<kBf>(y[2], y[3])};
    });
  });
  wave_fence();
  P::store(p.D + ((int64_t)row * p.ldd + col) * 2, p.ldd, region, lane, rows, cols, p.flags & kOpD16);
}

template <int kCode, int kAct, class F>
__device__ __forceinline__ void with_act_and_type(const GroupedParams& p, F&& run) {
  auto typed = [&](auto act) {
    if constexpr (kCode == kBF16 || kCode == kF16) run(act, std::bool_constant<kCode == kBF16>{});
    else if (p.d_type == TLA_BF16) run(act, std::true_type{});
    else run(act, std::false_type{});
  };
  if constexpr (kAct > 0) typed(std::integral_constant<int, kAct>{});
  else with_act(p.act, typed);
}

// A wave's epilogue in the role and operand code of its kernel.  16-bit roles: the
// outputs have the operands' type.  The two-group kernel is compiled for each
// activation (kAct > 0), the others branch.
template <int kCode, int kRole, int kAct, int FR, int WM, int WN, class Acc, int FM, int FN>
__device__ __forceinline__ void role_epilogue(const GroupedParams& p, int e, int r1, int row, int col,
                                              int lane, Acc (&acc)[FM][FN], uint8_t* region) {
  with_act_and_type<kCode, kAct>(p, [&](auto act, auto bf) {
    if constexpr (kRole == kGated)
      gated_epilogue<FR, WM, WN, act, bf>(p, e, r1, row, col, lane, acc, region);
    else
      blocks_epilogue<WM, WN, act, bf>(p, e, r1, row, col, lane, acc, region);
  });
}
template <int kCode, int kAct, int WM, int WN, int FM, int FN>
__device__ __forceinline__ void grad_epilogue(const GroupedParams& p, int r1, int row, int col, int lane,
                                              f32x16 (&acc)[FM][FN], GateParts<WM, WN>& z,
                                              uint8_t* region) {
  with_act_and_type<kCode, kAct>(p, [&](auto act, auto bf) {
    gate_grad_epilogue<WM, WN, act, bf>(p, r1, row, col, lane, acc, z, region);
  });
}

}  // namespace
}  // namespace tla
