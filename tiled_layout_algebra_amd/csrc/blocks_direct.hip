// blocks_direct.hip -- the block-scaled e4m3 product, plain and gated, on tiles
// of 64 or 128 rows and 128 columns.
//
// A k-tile is a block of 128 of K, 128 bytes a row.  LDS holds kStages slabs of
// A and of B, filled by direct global -> LDS copies; the loop has one barrier a
// k-tile: wait for the tile's copies, read its fragments, start the copies of the
// tile kStages - 1 ahead, multiply.  The scales come a k-tile ahead by plain
// loads in front of the copies: a lane's rows' (col-major scales: 16 neighbours
// together) and the one or two of the workgroup's columns.
//
// kWide (K < 512): the fragments are widened to f16 and every product and sum is fp32,
// as in the other e4m3 products of that length: what the 8-bit instruction drops of
// terms of like sizes lies under fp32's own rounding bound in long sums only.  8192 rows x 4096 x 384 43 us (without 35), gated 82 (52 in
// the two-group kernel, which has no such form); 300 rows 7.0 (6.1), 9 (8.7).  The
// few-row kernel, which sums the same way, takes 361 and 326 for the 8192 rows.
//
// Bound by its copies: a workgroup's k-tile takes 0.45 us alone on a compute unit with 64
// rows, 0.72 with 128.  Measured, 4096 x 4096 weights, 32 k-tiles: 96 rows 18.6 us (64
// x 128), 800 rows 26.7 and 28 (128 x 128); gated, 48 rows 19 and 27.
#include "gated_common.hpp"

namespace tla {
namespace {

template <int BM, int kStages, int kWM, int kWN, bool kTwo, bool kWide>
__global__ __launch_bounds__(64 * kWM * kWN) void blocks_direct_kernel(const GroupedParams p) {
  constexpr int BN = 128, kRowBytes = 128, NT = 64 * kWM * kWN;
  using Swz = typename Slab<kRowBytes>::Swz;
  constexpr int kChunks = Slab<kRowBytes>::kChunks;
  constexpr int WM = BM / kWM, WN = BN / kWN, FM = WM / 16, FN = WN / 16, FH = FN / 2;
  constexpr int SLAB_A = BM * kRowBytes, SLAB_B = BN * kRowBytes, STAGE = SLAB_A + SLAB_B;
  constexpr int IA = BM * kChunks / NT, IB = BN * kChunks / NT, kLoads = IA + IB;
  constexpr int BNO = kTwo ? BN / 2 : BN;  // columns of D
  static_assert(IA * NT == BM * kChunks && IB * NT == BN * kChunks && IB % 2 == 0, "whole copies");
  static_assert(kWM * kWN * WM * WN * 2 <= kStages * STAGE && kStages * STAGE <= 160 * 1024, "LDS");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kStages * STAGE];

  RowTile t;
  if (!row_tile<BM>(p, blockIdx.x, t)) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int e = __builtin_amdgcn_readfirstlane(t.e), m0 = t.r0, m_end = t.r1;
  const int n0 = __builtin_amdgcn_readfirstlane(t.tn) * BNO, K = p.K;
  const int wm0 = (wave % kWM) * WM, wn0 = (wave / kWM) * WN, wb0 = kTwo ? wn0 / 2 : wn0;
  const int KT = (K + 127) / 128, KTf = K / 128;  // tile KTf, if K ends inside it, is ragged
  const uint8_t* A = p.A + (int64_t)m0 * p.lda;
  const uint8_t* B = p.B + (int64_t)e * p.stride_b + (int64_t)n0 * p.ldb;
  const int64_t up_by = kTwo ? p.B2 - p.B : 0;
  // each operand's bytes up to the last dword that it needs
  const int a_last = m_end - 1 - m0, b_last = p.N - 1 - n0;
  const int a_bytes = (int)((min(a_last, BM - 1) * (uint32_t)p.lda + K + 3) & ~3u);
  const int b_bytes = (int)((min(b_last, BNO - 1) * (uint32_t)p.ldb + K + 3) & ~3u);
  // copy q: slab row tid / 8 + (NT / 8) q' (of its half slab), the chunk that the
  // swizzle assigns to slot tid + NT q', from the row clamped to the matrix
  uint32_t off[kLoads], tail_past = 0;
  static_for<kLoads>([&](auto q) {
    constexpr bool kA = q < IA;
    constexpr int qq = kA ? (int)q : kTwo ? (q - IA) % (IB / 2) : q - IA;
    const int r = tid / kChunks + (NT / kChunks) * qq, c = Swz::chunk(r, tid % kChunks) * 16;
    off[q] = (uint32_t)(min(r, kA ? a_last : b_last) * (uint32_t)(kA ? p.lda : p.ldb) + c);
    if (c >= K - KTf * 128) tail_past |= 1u << q;
  });
  // tiles past K reload the last one; chunks past K read zeros from past the records
  auto copy_tile = [&](int kt, auto slot) {
    const int tt = min(kt, KT - 1);
    static_for<kLoads>([&](auto q) {
      const uint32_t o = tt == KTf && ((tail_past >> q) & 1) ? 0x80000000u : off[q];
      uint8_t* to = smem + slot * STAGE + (q < IA ? 0 : SLAB_A) +
                    (wave * 64 + NT * (q < IA ? (int)q : q - IA)) * 16;
      const uint8_t* from = q < IA ? A : B;
      if constexpr (kTwo && q >= IA + IB / 2) from += up_by;
      dma16_buf(from, o, (uint32_t)tt * kRowBytes, to, q < IA ? a_bytes : b_bytes);
    });
  };
  // what the last k-tile's crossing chunk holds past K (the next row's bytes)
  auto clear_tail = [&](int kt, auto slot) {
    if (kt != KTf || K % 16 == 0) return;
    for (int r = tid; r < BM + BN; r += NT) {
      const int rr = r < BM ? r : r - BM;
      uint8_t* row = smem + slot * STAGE + (r < BM ? 0 : SLAB_A) + rr * kRowBytes;
      const int first = K - KTf * 128, end = (first + 15) / 16 * 4;
      for (int d = first >> 2; d < end; ++d) {
        uint32_t* w = (uint32_t*)(row + Swz::chunk(rr, d >> 2) * 16 + (d & 3) * 4);
        *w = d == first >> 2 ? *w & ((1u << (8 * (first & 3))) - 1u) : 0u;
      }
    }
    __syncthreads();
  };
  // the scales of block kt: of this lane's rows, of the columns
  const float* sa_at[FM];
  static_for<FM>([&](auto i) {
    sa_at[i] = p.sa + (int64_t)(m0 + min(wm0 + 16 * (int)i + (lane & 15), a_last)) * p.sa_row;
  });
  const int64_t sb_at = (int64_t)e * p.stride_sb + (int64_t)(n0 >> 7) * p.sb_col;
  float raw_a[FM], raw_b[2];
  auto ask_scales = [&](int kt) {
    const int k = min(kt, KT - 1);
    static_for<FM>([&](auto i) { raw_a[i] = sa_at[i][(int64_t)k * p.sa_kb]; });
    raw_b[0] = p.sb[sb_at + (int64_t)k * p.sb_kb];
    raw_b[1] = kTwo ? p.sb2[sb_at + (int64_t)k * p.sb_kb] : 0.f;
  };

  const uint32_t fa = (uint32_t)((wm0 + (lane & 15)) * kRowBytes), fb = (uint32_t)((wb0 + (lane & 15)) * kRowBytes);
  // logical chunks lane / 16 and the fourth after it, as the two-group kernel's
  // (whose comment says why); the swizzle repeats in 16 rows
  const uint32_t c0 = Swz::chunk(lane & 15, lane >> 4) * 16;
  auto frag = [&](uint32_t at) {
    const i32x4 lo = *(const i32x4*)(smem + at + c0), hi = *(const i32x4*)(smem + at + (c0 ^ 64u));
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };
  BlockSums<FM, FN, kTwo> sums;
  sums.init();

  auto tile = [&](int kt, auto S) {
    using Fill = std::integral_constant<int, (S + kStages - 1) % kStages>;
    __builtin_amdgcn_s_waitcnt(0xC07F);    // this wave's reads of tile kt - 1 (lgkmcnt 0)
    wait_vmcnt<(kStages - 2) * kLoads>();  // tile kt's copies and scales (this thread's)
    stage_barrier();                       // everyone's; tile kt - 1's slot is free
    clear_tail(kt, S);
    float s[2][FM];
    static_for<FM>([&](auto i) {
      s[0][i] = raw_a[i] * raw_b[0];
      s[1][i] = raw_a[i] * raw_b[1];
    });
    ask_scales(kt + 1);
    copy_tile(kt + kStages - 1, Fill{});
    i32x8 a[FM], b[FN];
    static_for<FM>([&](auto i) { a[i] = frag(fa + S * STAGE + 16 * i * kRowBytes); });
    static_for<FN>([&](auto j) {
      constexpr int at = kTwo ? j % FH * 16 * kRowBytes + j / FH * (SLAB_B / 2) : j * 16 * kRowBytes;
      b[j] = frag(fb + S * STAGE + SLAB_A + at);
    });
    if constexpr (kWide) {
      sums.mma_wide(a, b, s);
    } else {
      sums.mma(a, b, s, [](auto) {});
      sums.finish(s);
    }
  };
  if (KT > 0) {
    // the first tile's scales before its copies, so that the loop's first wait covers them
    ask_scales(0);
    static_for<kStages - 1>([&](auto q) { copy_tile(q, q); });
    for (int kt = 0; kt < KT; kt += kStages) {
      static_for<kStages>([&](auto s) {
        if (kt + s < KT) tile(kt + s, s);
      });
    }
    wait_vmcnt<0>();  // no copy may land in LDS after this point
  }
  __syncthreads();  // the stages become the waves' epilogue regions
  uint8_t* region = smem + wave * WM * WN * 2;
  role_epilogue<kE4M3Blocks, kTwo ? kGated : kPlain, 0, 16, WM, kTwo ? WN / 2 : WN>(
      p, e, m_end, m0 + wm0, n0 + wb0, lane, sums.acc, region);
}

template <int BM, int kStages, int kWM, int kWN, bool kTwo, bool kWide>
int launch_form(const GroupedParams& p0, hipStream_t stream) {
  GroupedParams p = p0;
  p.tiles_n = kTwo ? (p.N + 63) / 64 : (p.N + 127) / 128;
  const int64_t grid = row_tiles_bound(p.rows, p.groups, BM) * p.tiles_n;
  if (grid <= 0) return TLA_OK;
  if (!grid_fits(grid, 64 * kWM * kWN)) return TLA_ERR_UNSUPPORTED;
  hipLaunchKernelGGL((blocks_direct_kernel<BM, kStages, kWM, kWN, kTwo, kWide>), dim3((unsigned)grid),
                     dim3(64 * kWM * kWN), 0, stream, p);
  return hipGetLastError() == hipSuccess ? TLA_OK : TLA_ERR_HIP;
}

template <int BM, int kStages, int kWM, int kWN, bool kTwo>
int launch(const GroupedParams& p, hipStream_t s) {
  return p.K < kMinKE4m3 ? launch_form<BM, kStages, kWM, kWN, kTwo, true>(p, s)
                         : launch_form<BM, kStages, kWM, kWN, kTwo, false>(p, s);
}

}  // namespace

int launch_blocks_direct(const GroupedParams& p, int bm, bool gated, hipStream_t s) {
  if (bm == 64) return gated ? launch<64, 3, 2, 2, true>(p, s) : launch<64, 3, 2, 2, false>(p, s);
  return gated ? launch<128, 2, 2, 2, true>(p, s) : launch<128, 2, 2, 2, false>(p, s);
}

}  // namespace tla
