// grouped_general.hip -- the register-staged kernel of the expert-grouped
// products: any pitch, alignment, order and length.
//
// A workgroup of four wavefronts owns 128 x 128 of D, each wave 64 x 64 of
// it, two LDS stages of 128 bytes of K.  Product: tiles come from the ragged
// lookup (row_tile), A and B are read through gemm_common.hpp's
// register-staged loaders (16-byte chunks at any byte address, shifted into
// place on the way to LDS), B K-contiguous, 16-bit N-contiguous (its slab as
// k rows of n, read back transposed) or 8-bit N-contiguous (element by
// element).  Weight gradient: the sum runs over an expert's rows, so both
// operands are k-row slabs.  Tile kt + 1 is loaded into registers before the
// MFMAs of tile kt and written to the other stage after them; whole and
// ragged k-tiles have loops of their own.
#include "grouped_common.hpp"

namespace tla {
namespace {

enum : int { kBKc = 0, kBElem = 1, kBRows = 2 };

template <int kCode, int kBView, bool kWgrad>
__global__ __launch_bounds__(kThreads, kBView == kBElem ? 1 : 2) void grouped_general_kernel(
    const GroupedParams p) {
  using Atom = std::conditional_t<kCode == kE4M3, E4m3AsF16, OpAtom<kCode>>;
  using Frag = typename Atom::Frag;
  constexpr int kF = kFragCode<kCode>;
  constexpr int EB = type_bytes(kCode), BM = 128, BN = 128, kRowBytes = 128, BK = kRowBytes / EB;
  constexpr int WM = 64, WN = 64, FM = 2, FN = 2, KSTEPS = BK / Atom::kK;
  constexpr bool kAT = kWgrad, kNT = kBView == kBRows;
  constexpr int SLAB_A = BM * kRowBytes, STAGE = (BM + BN) * kRowBytes;
  static_assert(!kWgrad || kNT, "the weight gradient sums over rows of both operands");
  static_assert(4 * WM * 64 * FN <= 2 * STAGE, "epilogue regions");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * STAGE];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int e, m0, m_end, n0, K;
  const uint8_t *A = p.A, *B = p.B;
  if constexpr (kWgrad) {
    int tm, tn, lo, hi;
    wgrad_tile(p, blockIdx.x, gridDim.x, e, tm, tn);
    expert_rows(p, e, lo, hi);
    m0 = tm * BM;
    n0 = tn * BN;
    m_end = p.M;
    K = hi - lo;
    A += (int64_t)lo * p.lda * EB;
    B += (int64_t)lo * p.ldb * EB;
  } else {
    RowTile t;
    if (!row_tile<BM>(p, blockIdx.x, t)) return;
    e = t.e;
    m0 = t.r0;
    m_end = t.r1;
    n0 = t.tn * BN;
    K = p.K;
    B += (int64_t)e * p.stride_b * EB;
  }
  const int wm0 = (wave & 1) * WM, wn0 = (wave >> 1) * WN;
  const int N = p.N;

  typename Atom::Acc acc[FM][FN];
  static_for<FM>([&](auto i) { static_for<FN>([&](auto j) { acc[i][j] = typename Atom::Acc{}; }); });
  Frag a[2][FM], b[2][FN];
  auto read_frags = [&](auto buf, const uint8_t* stage, auto ks) {
    static_for<FM>([&](auto i) {
      if constexpr (kAT) a[buf][i] = load_frag_nt<2 * BM>(stage, wm0 + 32 * i, ks, lane);
      else a[buf][i] = load_frag<kF, kRowBytes>(stage, wm0 + 32 * i + (lane & 31), ks, lane);
    });
    static_for<FN>([&](auto j) {
      if constexpr (kNT) b[buf][j] = load_frag_nt<2 * BN>(stage + SLAB_A, wn0 + 32 * j, ks, lane);
      else
        b[buf][j] = load_frag<kF, kRowBytes>(stage + SLAB_A, wn0 + 32 * j + (lane & 31), ks, lane);
    });
  };
  auto compute = [&](const uint8_t* stage) {
    read_frags(std::integral_constant<int, 0>{}, stage, std::integral_constant<int, 0>{});
    static_for<KSTEPS>([&](auto ks) {
      constexpr int cur = ks & 1;
      if constexpr (ks + 1 < KSTEPS)
        read_frags(std::integral_constant<int, cur ^ 1>{}, stage,
                   std::integral_constant<int, ks + 1>{});
      static_for<FM * FN>([&](auto q) {
        Atom::mma(acc[q / FN][q % FN], b[cur][q % FN], a[cur][q / FN]);
      });
    });
  };

  using RA = std::conditional_t<kAT, RegSlabNT<BM, BK>, RegSlab<BM, EB, kRowBytes, true>>;
  using RB = std::conditional_t<kNT, RegSlabNT<BN, BK>, RegSlab<BN, EB, kRowBytes, kBView == kBKc>>;
  RA ra;
  RB rb;
  const int KT = (K + BK - 1) / BK;
  // Whole tiles: inside K; where a k-rows slab's tile crosses its matrix's
  // edge also before the tile that holds row K - 1 (whole chunks there read
  // on into the next row).
  const bool m_edge = kAT && m0 + BM > m_end, n_edge = kNT && n0 + BN > N;
  const int KTw = kBView == kBElem ? 0
                  : (m_edge || n_edge)
                      ? ((m_edge && m_end < 8) || (n_edge && N < 8) ? 0 : (K - 1) / BK)
                      : K / BK;
  auto load = [&](int k0, auto whole) {
    if constexpr (whole) {
      ra.load_whole(A, p.lda, m0, m_end, k0, tid);
      if constexpr (kBView != kBElem) rb.load_whole(B, p.ldb, n0, N, k0, tid);
    } else {
      ra.load_edge(A, p.lda, m0, m_end, k0, K, tid);
      rb.load_edge(B, p.ldb, n0, N, k0, K, tid);
    }
  };
  auto store = [&](uint8_t* st) {
    ra.store(st, tid);
    rb.store(st + SLAB_A, tid);
  };
  auto step = [&](int kt, auto whole) {  // load tile kt + 1, multiply tile kt
    load((kt + 1) * BK, whole);
    __builtin_amdgcn_sched_barrier(0);
    compute(smem + (kt & 1) * STAGE);
    __builtin_amdgcn_sched_barrier(0);
    store(smem + ((kt + 1) & 1) * STAGE);
    __syncthreads();
  };
  if (KT > 0) {
    if (KTw > 0) load(0, std::true_type{});
    else load(0, std::false_type{});
    store(smem);
    __syncthreads();
    int kt = 0;
    for (; kt + 1 < KTw; ++kt) step(kt, std::true_type{});
    for (; kt + 1 < KT; ++kt) step(kt, std::false_type{});
    compute(smem + (kt & 1) * STAGE);
  }
  __syncthreads();  // the stages become the waves' epilogue regions
  uint8_t* region = smem + wave * WM * 64 * FN;
  if constexpr (kWgrad)
    wgrad_epilogue<FM, FN>(p, e, m0 + wm0, n0 + wn0, lane, acc, region);
  else
    grouped_epilogue<kCode, FM, FN>(p, e, m_end, m0 + wm0, n0 + wn0, lane, acc, region);
}

template <int kCode, int kBView, bool kWgrad>
int launch(const GroupedParams& p0, hipStream_t stream) {
  GroupedParams p = p0;
  p.tiles_n = (p.N + 127) / 128;
  p.tiles_m = (p.M + 127) / 128;
  const int64_t grid = kWgrad ? (int64_t)p.groups * p.tiles_m * p.tiles_n
                              : row_tiles_bound(p.rows, p.groups, 128) * p.tiles_n;
  if (grid <= 0) return TLA_OK;
  if (grid > 0x7FFFFFFF) return TLA_ERR_UNSUPPORTED;
  hipLaunchKernelGGL((grouped_general_kernel<kCode, kBView, kWgrad>), dim3((unsigned)grid),
                     dim3(kThreads), 0, stream, p);
  return hipGetLastError() == hipSuccess ? TLA_OK : TLA_ERR_HIP;
}

// Column sums of each expert's rows of Y, 64 columns a workgroup: 8 lanes
// cover a row's 128 bytes, 32 rows at a time; the 32 partial sums of a column
// are joined in LDS in a fixed order.
template <int kCode>
__global__ __launch_bounds__(256) void group_colsum_kernel(const GroupedParams p, const uint8_t* Y,
                                                           int64_t ldy, int N) {
  __shared__ float part[32][65];
  const int e = blockIdx.y, c0 = blockIdx.x * 64, tid = threadIdx.x;
  const int c = c0 + 8 * (tid & 7), r0 = tid >> 3;
  int lo, hi;
  expert_rows(p, e, lo, hi);
  float s[8] = {};
  auto add = [&](const i32x4& v) {
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      s[2 * w] += widen_lo<kCode == kBF16>((uint32_t)v[w]);
      s[2 * w + 1] += widen_hi<kCode == kBF16>((uint32_t)v[w]);
    }
  };
  if (c + 8 <= N) {
    int r = lo + r0;
    for (; r + 7 * 32 < hi; r += 8 * 32) {
      i32x4 v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = load16_even(Y + ((int64_t)(r + 32 * u) * ldy + c) * 2);
#pragma unroll
      for (int u = 0; u < 8; ++u) add(v[u]);
    }
    for (; r < hi; r += 32) add(load16_even(Y + ((int64_t)r * ldy + c) * 2));
  } else if (c < N) {
    for (int r = lo + r0; r < hi; r += 32)
      add(gather16<2>(Y + (int64_t)r * ldy * 2, 2, c, N, N - 1));
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) part[r0][8 * (tid & 7) + q] = s[q];
  __syncthreads();
  if (tid < 64 && c0 + tid < N) {
    float t = 0.f;
#pragma unroll
    for (int r = 0; r < 32; ++r) t += part[r][tid];
    p.dbias[(int64_t)e * N + c0 + tid] = t;
  }
}

}  // namespace

int launch_grouped_general(const GroupedParams& p, int type, bool b_kc, hipStream_t s) {
  switch (type) {
    case TLA_BF16:
      return b_kc ? launch<kBF16, kBKc, false>(p, s) : launch<kBF16, kBRows, false>(p, s);
    case TLA_F16:
      return b_kc ? launch<kF16, kBKc, false>(p, s) : launch<kF16, kBRows, false>(p, s);
    case TLA_E4M3:
      return b_kc ? launch<kE4M3, kBKc, false>(p, s) : launch<kE4M3, kBElem, false>(p, s);
    case TLA_I8:
      return b_kc ? launch<kI8, kBKc, false>(p, s) : launch<kI8, kBElem, false>(p, s);
    default: return TLA_ERR_UNSUPPORTED;
  }
}

int launch_wgrad_general(const GroupedParams& p, int type, hipStream_t s) {
  switch (type) {
    case TLA_BF16: return launch<kBF16, kBRows, true>(p, s);
    case TLA_F16: return launch<kF16, kBRows, true>(p, s);
    default: return TLA_ERR_UNSUPPORTED;
  }
}

int launch_group_colsum(const GroupedParams& p, const uint8_t* Y, int64_t ldy, int type, int N,
                        hipStream_t s) {
  const dim3 grid((unsigned)((N + 63) / 64), (unsigned)p.groups);
  if (type == TLA_BF16)
    hipLaunchKernelGGL(group_colsum_kernel<kBF16>, grid, dim3(256), 0, s, p, Y, ldy, N);
  else
    hipLaunchKernelGGL(group_colsum_kernel<kF16>, grid, dim3(256), 0, s, p, Y, ldy, N);
  return hipGetLastError() == hipSuccess ? TLA_OK : TLA_ERR_HIP;
}

}  // namespace tla
