// grouped_few_rows.hpp -- the product for experts with few rows (decoding
// steps), where reading the weights is all that costs.
//
// A workgroup takes up to 16 MT rows of one expert and 16 NT columns; its
// waves split K between them and each keeps the whole 16 MT x 16 NT piece in
// registers.  A weight is used by one wave only, so nothing is staged: lane l
// of a step loads 16 bytes of K of column l % 16 (and of row l % 16 of A, from
// the caches) straight into the operands of the 16x16 matrix instruction --
// any assignment of K to lanes is right while both operands share it.  kU steps are loaded before the first is used.
// The waves' partial sums meet in LDS in a fixed order, and the epilogue runs
// element by element, consecutive lanes along a row of D.
//
// Weights of 8 bits are read as they are: int8 goes to the integer
// instruction, e4m3 is widened to f16, which holds it exactly.
//
// Bound by memory.  Measured: bf16, 128 rows on 32 experts of 2048 x 4096 106 us
// (537 MB of weights: 5.1 TB/s; a large copy reaches 6.7, reads and writes together),
// two rows on two experts of 4096 x 4096 12-13 us (67 MB: 5 TB/s and more); one
// row x 4096 x 4096 6.3 us in int8 and in e4m3, of which about 4 are a launch's; 128
// e4m3 rows on the 32 experts 43 us.  Gated (the NT fragments are as many of the gate's
// columns and the same of up's), one bf16 row x 8192 x 4096, SiLU: 26.9 us a call, 22.8
// on the card (134 MB: 5.9 TB/s).  Block scales (kBlocks: two steps of 64 are a block, whose
// partial sums are scaled into the sums): one row x 4096 x 4096 7.2 us, 128 rows on the
// 32 experts 52-55 (253 MB: 4.9 TB/s).
#pragma once

#include "gated_common.hpp"

namespace tla {
namespace {

// 16x16 step over the 16 bytes of K a lane holds of each operand
template <int kCode>
struct Step16 {
  typedef f32x4 Acc;
  static __device__ __forceinline__ void mma(f32x4& c, const i32x4& a, const i32x4& b) {
    if constexpr (kCode == kBF16)
      c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                  __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    else
      c = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                 __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
  }
};
template <>
struct Step16<kI8> {
  typedef i32x4 Acc;
  static __device__ __forceinline__ void mma(i32x4& c, const i32x4& a, const i32x4& b) {
    c = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
  }
};
template <>
struct Step16<kE4M3> {
  typedef f32x4 Acc;
  static __device__ __forceinline__ void mma(f32x4& c, const i32x4& a, const i32x4& b) {
    const i32x8 a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, b8 = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
#pragma unroll
    for (int q = 0; q < 2; ++q) Step16<kF16>::mma(c, E4m3AsF16::widen(a8, q), E4m3AsF16::widen(b8, q));
  }
};

// Sixteen bytes of a row.  kDword: rows start on dwords, one load.  Otherwise
// the dword-aligned sixteen bytes and the dword after them, shifted into place
// when they are used (128 bf16 rows on 32 experts of 2048 x 4095: 163 us so, 243
// with loads at the rows' own addresses).
template <bool kDword>
struct Chunk {
  i32x4 v;
  uint32_t hi;
  __device__ __forceinline__ void load(const uint8_t* p) {
    typedef int i32x4_a4 __attribute__((ext_vector_type(4), aligned(4)));
    if constexpr (kDword) v = *(const i32x4_a4*)p;
    else load16_split(p, v, hi);
  }
  __device__ __forceinline__ i32x4 get(uint32_t sh) const {
    if constexpr (kDword) return v;
    else return realign16(v, hi, sh);
  }
};

// kBlocks: e4m3 with block scales.  A wave takes whole blocks of 128 of K, two
// steps each, and adds a block's sum to its own with the block's scales.
template <>
struct Step16<kE4M3Blocks> : Step16<kE4M3> {};

template <int kCode, int MT, int NT, int kWaves, bool kDword, int kRole = kPlain>
__global__ __launch_bounds__(64 * kWaves) void grouped_few_rows_kernel(const GroupedParams p, int first) {
  using S = Step16<kCode>;
  typedef typename S::Acc Acc;
  constexpr bool kBlocks = kCode == kE4M3Blocks;
  // kGated: the first half of the column pieces are the gate's, the others the
  // same columns of the up projection
  constexpr bool kTwo = kRole == kGated;
  constexpr int NH = kTwo ? NT / 2 : NT;
  constexpr int EB = type_bytes(kCode), BM = 16 * MT, BN = 16 * NH;
  constexpr int kU = MT + NT <= 2 ? 8 : 4;  // steps in flight
  __shared__ Acc part[kWaves][MT * NT][64];

  RowTile t;
  if (!row_tile<BM>(p, first + (int)blockIdx.x, t)) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = t.tn * BN;
  const int rows = min(BM, t.r1 - t.r0), cols = min(BN, p.N - n0);
  // K in steps of 64 bytes, each wave a run of them
  const int64_t kbytes = (int64_t)p.K * EB;
  const int steps = (int)((kbytes + 63) / 64);
  constexpr int kUnit = kBlocks ? 2 : 1;  // steps a wave takes together
  const int units = (steps + kUnit - 1) / kUnit;
  const int s0 = kUnit * (int)((int64_t)units * wave / kWaves);
  const int s1 = min(steps, kUnit * (int)((int64_t)units * (wave + 1) / kWaves));
  const uint8_t *pa[MT], *pb[NT];
  static_for<MT>([&](auto i) {
    const int r = t.r0 + min(16 * (int)i + (lane & 15), rows - 1);
    pa[i] = p.A + (int64_t)r * p.lda * EB + 16 * (lane >> 4);
  });
  static_for<NT>([&](auto j) {
    const int n = n0 + min(16 * ((int)j % NH) + (lane & 15), cols - 1);
    const uint8_t* B = kTwo && j >= NH ? p.B2 : p.B;
    pb[j] = B + ((int64_t)t.e * p.stride_b + (int64_t)n * p.ldb) * EB + 16 * (lane >> 4);
  });
  // rows 16 apart share a byte shift, the two operands of kTwo need not
  const uint32_t sa = (uint32_t)(uintptr_t)pa[0] & 3u;
  const uint32_t sb[2] = {(uint32_t)(uintptr_t)pb[0] & 3u, (uint32_t)(uintptr_t)pb[NT - 1] & 3u};
  Acc acc[MT][NT];
  static_for<MT>([&](auto i) { static_for<NT>([&](auto j) { acc[i][j] = Acc{}; }); });

  // kBlocks: the scales of block kb: of each piece's rows, and of its columns
  // (16 of them never cross a block: n0 is a multiple of 16)
  struct Scales {
    float a[MT], b[kTwo ? 2 : 1];
  };
  const float *ra[MT], *rb[2];
  if constexpr (kBlocks) {
    static_for<MT>([&](auto i) {
      ra[i] = p.sa + (int64_t)(t.r0 + min(16 * (int)i + (lane & 15), rows - 1)) * p.sa_row;
    });
    const int64_t at = (int64_t)t.e * p.stride_sb + (int64_t)(n0 >> 7) * p.sb_col;
    rb[0] = p.sb + at;
    rb[1] = kTwo ? p.sb2 + at : nullptr;
  }
  auto scales = [&](int kb) {
    Scales x;
    static_for<MT>([&](auto i) { x.a[i] = ra[i][(int64_t)kb * p.sa_kb]; });
    static_for<kTwo ? 2 : 1>([&](auto h) { x.b[h] = rb[h][(int64_t)kb * p.sb_kb]; });
    return x;
  };
  auto add_block = [&](const Acc (&part)[MT][NT], const Scales& x) {
    static_for<MT>([&](auto i) {
      static_for<NT>([&](auto j) {
        const float c = x.a[i] * x.b[kTwo && j >= NH];
        static_for<4>([&](auto q) { acc[i][j][(int)q] = fmaf(part[i][j][(int)q], c, acc[i][j][(int)q]); });
      });
    });
  };

  // Loads run kU steps ahead of the matrix instructions: unit v's are asked for
  // again as soon as its step (kBlocks: its two) has been taken.  (All kU loaded,
  // then all used, twice as many: bf16, 128 rows on 32 experts of 2048 x 4096 112 us
  // instead of 106; and the steps left over one at a time: one row, 8192 x 1050 e4m3
  // 14.4 instead of 9.7.)
  const int whole = min(s1, (int)(kbytes / 64));  // steps inside K
  constexpr int kSlots = kU / kUnit;
  Chunk<kDword> a[kU][MT], b[kU][NT];
  Scales x[kBlocks ? kSlots : 1];
  auto load = [&](int s, auto v) {
    static_for<kUnit>([&](auto h) {
      constexpr int u = kUnit * v + h;
      static_for<NT>([&](auto j) { b[u][j].load(pb[j] + (int64_t)(s + h) * 64); });
      static_for<MT>([&](auto i) { a[u][i].load(pa[i] + (int64_t)(s + h) * 64); });
    });
    if constexpr (kBlocks) x[v] = scales(s / 2);
  };
  auto use = [&](auto v) {
    Acc part[MT][NT];
    if constexpr (kBlocks)
      static_for<MT>([&](auto i) { static_for<NT>([&](auto j) { part[i][j] = Acc{}; }); });
    static_for<kUnit>([&](auto h) {
      constexpr int u = kUnit * v + h;
      i32x4 bb[NT];
      static_for<NT>([&](auto j) { bb[j] = b[u][j].get(sb[kTwo && j >= NH]); });
      static_for<MT>([&](auto i) {
        const i32x4 aa = a[u][i].get(sa);
        static_for<NT>([&](auto j) {
          if constexpr (kBlocks) S::mma(part[i][j], bb[j], aa);
          else S::mma(acc[i][j], bb[j], aa);
        });
      });
    });
    if constexpr (kBlocks) add_block(part, x[v]);
  };
  int s = s0;
  if (s + kU <= whole) {
    static_for<kSlots>([&](auto v) { load(s + kUnit * v, v); });
    for (; s + 2 * kU <= whole; s += kU) {
      static_for<kSlots>([&](auto v) {
        use(v);
        load(s + kU + kUnit * v, v);
        __builtin_amdgcn_sched_barrier(0);  // (or the registers of v double)
      });
    }
    static_for<kSlots>([&](auto v) { use(v); });
    s += kU;
  }
  // what is left of the whole steps, in halves of kU
  static_for<3>([&](auto h) {
    constexpr int n = kU >> (h + 1);
    if constexpr (n >= kUnit) {
      if (s + n <= whole) {
        static_for<n / kUnit>([&](auto v) { load(s + kUnit * v, v); });
        static_for<n / kUnit>([&](auto v) { use(v); });
        s += n;
      }
    }
  });
  for (; s < s1; ++s) {
    // the last step; a lane's bytes past K are zeros, gathered
    // where they begin inside its sixteen
    const int left = (int)min(kbytes - (int64_t)s * 64, (int64_t)64) - 16 * (lane >> 4);
    auto get = [&](const uint8_t* base) {
      const uint8_t* q = base + (int64_t)s * 64;
      i32x4 x = {0, 0, 0, 0};
      if (left >= 16) {
        Chunk<false> c;
        c.load(q);
        return c.get((uint32_t)(uintptr_t)q & 3u);
      }
      if (left > 0) x = gather16<EB>(q, EB, 0, left / EB, left / EB - 1);
      return x;
    };
    i32x4 a[MT], b[NT];
    static_for<NT>([&](auto j) { b[j] = get(pb[j]); });
    static_for<MT>([&](auto i) { a[i] = get(pa[i]); });
    if constexpr (kBlocks) {
      // (each of a block's two steps by itself: the scales distribute)
      Acc part[MT][NT];
      static_for<MT>([&](auto i) {
        static_for<NT>([&](auto j) {
          part[i][j] = Acc{};
          S::mma(part[i][j], b[j], a[i]);
        });
      });
      add_block(part, scales(s / 2));
    } else {
      static_for<MT>([&](auto i) { static_for<NT>([&](auto j) { S::mma(acc[i][j], b[j], a[i]); }); });
    }
  }
  // lane l, value r of piece (i, j): row 16 i + l % 16, column 16 j + 4 (l / 16) + r
  static_for<MT>([&](auto i) {
    static_for<NT>([&](auto j) { part[wave][i * NT + j][lane] = acc[i][j]; });
  });
  __syncthreads();
  for (int x = tid; x < BM * BN; x += 64 * kWaves) {
    const int m = x / BN, n = x % BN;
    if (m >= rows || n >= cols) continue;
    const int piece = (m / 16) * NT + n / 16, l = (m & 15) + 16 * ((n & 15) >> 2), v = n & 3;
    auto total = [&](int at) {
      auto sum = part[0][at][l][v];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) sum += part[w][at][l][v];
      return sum;
    };
    const int64_t row = t.r0 + m, col = n0 + n;
    float y = (float)total(piece);
    if constexpr (kCode == kI8 || kCode == kE4M3) {
      const float sa = p.sa ? p.sa[row] : 1.f;
      y = y * sa * (p.sb ? p.sb[(int64_t)t.e * p.N + col] : 1.f);
    }
    auto bias = [&](const uint8_t* b) {
      return load_elem(b + (int64_t)t.e * p.N * type_bytes(p.bias_type), p.bias_type, col);
    };
    if (p.bias) y += bias(p.bias);
    uint16_t* Z = (uint16_t*)p.Z + row * p.ldz + col;
    if constexpr (kTwo) {
      float u = (float)total(piece + NH);
      if (p.bias2) u += bias(p.bias2);
      if (p.Z) {
        *Z = to_bits(y, p.d_type);
        ((uint16_t*)p.Z2)[row * p.ldz + col] = to_bits(u, p.d_type);
      }
      y = act_any(y, p.act) * u;
    } else if constexpr (kBlocks) {
      y = act_any(y, p.act);
    } else if (p.z_mode == TLA_Z_GRAD) {
      const float z = load_elem((const uint8_t*)Z, p.d_type, 0);
      y = p.act == TLA_ACT_RELU ? epi_op<kReluGrad>(y, z) : epi_op<kGeluGrad>(y, z);
    } else {
      if (p.z_mode == TLA_Z_STORE) *Z = to_bits(y, p.d_type);
      if (p.act == TLA_ACT_RELU) y = relu_nan(y);
      else if (p.act == TLA_ACT_GELU) y = gelu_nan(y);
    }
    ((uint16_t*)p.D)[row * p.ldd + col] = to_bits(y, p.d_type);
  }
}

constexpr int64_t kMaxTiles = (int64_t(1) << 31) - 4096;  // counted in 32 bits

template <int kCode, int MT, int NT, int kWaves, int kRole = kPlain>
int launch(const GroupedParams& p0, hipStream_t stream) {
  constexpr int EB = type_bytes(kCode);
  GroupedParams p = p0;
  constexpr int kCols = 16 * (kRole == kGated ? NT / 2 : NT);
  p.tiles_n = (p.N + kCols - 1) / kCols;
  const int64_t grid = row_tiles_bound(p.rows, p.groups, 16 * MT) * p.tiles_n;
  if (grid <= 0) return TLA_OK;
  if (grid > kMaxTiles) return TLA_ERR_UNSUPPORTED;
  const bool dword = aligned(p.A, 4) && aligned(p.B, 4) && (kRole != kGated || aligned(p.B2, 4)) && p.lda * EB % 4 == 0 &&
                     p.ldb * EB % 4 == 0 && (p.groups == 1 || p.stride_b * EB % 4 == 0);
  // launches of fewer than 2^32 threads, each a multiple of the eight XCDs (the last: what is left)
  constexpr int64_t kStep = kMaxThreads / (64 * kWaves) / 8 * 8;
  for (int64_t first = 0; first < grid; first += kStep) {
    const dim3 blocks((unsigned)(grid - first < kStep ? grid - first : kStep)), threads(64 * kWaves);
    if (dword)
      hipLaunchKernelGGL((grouped_few_rows_kernel<kCode, MT, NT, kWaves, true, kRole>), blocks, threads, 0,
                         stream, p, (int)first);
    else
      hipLaunchKernelGGL((grouped_few_rows_kernel<kCode, MT, NT, kWaves, false, kRole>), blocks, threads, 0,
                         stream, p, (int)first);
    if (hipGetLastError() != hipSuccess) return TLA_ERR_HIP;
  }
  return TLA_OK;
}

}  // namespace
}  // namespace tla
