// grouped_few_rows.hip -- the product for experts with few rows (decoding
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
// Bound by memory.  Measured: bf16, 128 rows on 32 experts of 2048 x 4096 110 us
// (537 MB of weights: 4.9 TB/s; a large copy reaches 6.7, reads and writes together),
// two rows on two experts of 4096 x 4096 12-13.6 us (67 MB: 5 TB/s and more); one
// row x 4096 x 4096 6.3 us in int8 and in e4m3, of which about 4 are a launch's; 128
// e4m3 rows on the 32 experts 43 us.
#include "grouped_common.hpp"

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

template <int kCode, int MT, int NT, int kWaves, bool kDword>
__global__ __launch_bounds__(64 * kWaves) void grouped_few_rows_kernel(const GroupedParams p) {
  using S = Step16<kCode>;
  typedef typename S::Acc Acc;
  constexpr int EB = type_bytes(kCode), BM = 16 * MT, BN = 16 * NT;
  constexpr int kU = MT + NT <= 3 ? 8 : 4;  // steps in flight
  __shared__ Acc part[kWaves][MT * NT][64];

  RowTile t;
  if (!row_tile<BM>(p, blockIdx.x, t)) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int n0 = t.tn * BN;
  const int rows = min(BM, t.r1 - t.r0), cols = min(BN, p.N - n0);
  // K in steps of 64 bytes, each wave a run of them
  const int64_t kbytes = (int64_t)p.K * EB;
  const int steps = (int)((kbytes + 63) / 64);
  const int s0 = (int)((int64_t)steps * wave / kWaves), s1 = (int)((int64_t)steps * (wave + 1) / kWaves);
  const uint8_t *pa[MT], *pb[NT];
  static_for<MT>([&](auto i) {
    const int r = t.r0 + min(16 * (int)i + (lane & 15), rows - 1);
    pa[i] = p.A + (int64_t)r * p.lda * EB + 16 * (lane >> 4);
  });
  static_for<NT>([&](auto j) {
    const int n = n0 + min(16 * (int)j + (lane & 15), cols - 1);
    pb[j] = p.B + ((int64_t)t.e * p.stride_b + (int64_t)n * p.ldb) * EB + 16 * (lane >> 4);
  });
  // rows 16 apart share a byte shift
  const uint32_t sa = (uint32_t)(uintptr_t)pa[0] & 3u, sb = (uint32_t)(uintptr_t)pb[0] & 3u;
  Acc acc[MT][NT];
  static_for<MT>([&](auto i) { static_for<NT>([&](auto j) { acc[i][j] = Acc{}; }); });

  const int whole = min(s1, (int)(kbytes / 64));  // steps inside K
  int s = s0;
  for (; s + kU <= whole; s += kU) {
    Chunk<kDword> a[kU][MT], b[kU][NT];
    static_for<kU>([&](auto u) {
      static_for<NT>([&](auto j) { b[u][j].load(pb[j] + (int64_t)(s + u) * 64); });
      static_for<MT>([&](auto i) { a[u][i].load(pa[i] + (int64_t)(s + u) * 64); });
    });
    static_for<kU>([&](auto u) {
      i32x4 bb[NT];
      static_for<NT>([&](auto j) { bb[j] = b[u][j].get(sb); });
      static_for<MT>([&](auto i) {
        const i32x4 aa = a[u][i].get(sa);
        static_for<NT>([&](auto j) { S::mma(acc[i][j], bb[j], aa); });
      });
    });
  }
  for (; s < s1; ++s) {
    // the rest one step at a time; a lane's bytes past K are zeros, gathered
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
    static_for<MT>([&](auto i) { static_for<NT>([&](auto j) { S::mma(acc[i][j], b[j], a[i]); }); });
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
    auto sum = part[0][piece][l][v];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) sum += part[w][piece][l][v];
    const int64_t row = t.r0 + m, col = n0 + n;
    float y = (float)sum;
    if constexpr (kCode == kI8 || kCode == kE4M3) {
      const float sa = p.sa ? p.sa[row] : 1.f;
      y = y * sa * (p.sb ? p.sb[(int64_t)t.e * p.N + col] : 1.f);
    }
    if (p.bias)
      y += load_elem(p.bias + (int64_t)t.e * p.N * type_bytes(p.bias_type), p.bias_type, col);
    uint16_t* Z = (uint16_t*)p.Z + row * p.ldz + col;
    if (p.z_mode == TLA_Z_GRAD) {
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

template <int kCode, int MT, int NT, int kWaves>
int launch(const GroupedParams& p0, hipStream_t stream) {
  constexpr int EB = type_bytes(kCode);
  GroupedParams p = p0;
  p.tiles_n = (p.N + 16 * NT - 1) / (16 * NT);
  const int64_t grid = row_tiles_bound(p.rows, p.groups, 16 * MT) * p.tiles_n;
  if (grid <= 0) return TLA_OK;
  if (!grid_fits(grid, 64 * kWaves)) return TLA_ERR_UNSUPPORTED;
  const bool dword = aligned(p.A, 4) && aligned(p.B, 4) && p.lda * EB % 4 == 0 &&
                     p.ldb * EB % 4 == 0 && (p.groups == 1 || p.stride_b * EB % 4 == 0);
  if (dword)
    hipLaunchKernelGGL((grouped_few_rows_kernel<kCode, MT, NT, kWaves, true>), dim3((unsigned)grid),
                       dim3(64 * kWaves), 0, stream, p);
  else
    hipLaunchKernelGGL((grouped_few_rows_kernel<kCode, MT, NT, kWaves, false>),
                       dim3((unsigned)grid), dim3(64 * kWaves), 0, stream, p);
  return hipGetLastError() == hipSuccess ? TLA_OK : TLA_ERR_HIP;
}

template <int kCode>
int pick(const GroupedParams& p, int mt, hipStream_t s) {
  const bool narrow = few_rows_narrow(p.rows, p.groups, p.N);
  if (mt == 1) return narrow ? launch<kCode, 1, 1, 8>(p, s) : launch<kCode, 1, 2, 4>(p, s);
  if (mt == 2) return narrow ? launch<kCode, 2, 1, 8>(p, s) : launch<kCode, 2, 2, 4>(p, s);
  return narrow ? launch<kCode, 4, 1, 8>(p, s) : launch<kCode, 4, 2, 4>(p, s);
}

}  // namespace

int launch_grouped_few_rows(const GroupedParams& p, int type, int mt, hipStream_t s) {
  switch (type) {
    case TLA_BF16: return pick<kBF16>(p, mt, s);
    case TLA_F16: return pick<kF16>(p, mt, s);
    case TLA_E4M3: return pick<kE4M3>(p, mt, s);
    case TLA_I8: return pick<kI8>(p, mt, s);
    default: return TLA_ERR_UNSUPPORTED;
  }
}

}  // namespace tla
