// grouped_general.hip -- the register-staged kernel of the expert-grouped
// products: any pitch, alignment, order and length.
//
// A workgroup of four wavefronts owns 128 x 128 of D, each wave 64 x 64 of
// it, two LDS stages of 128 bytes of K.  Product: tiles come from the ragged
// lookup (row_tile), B K-contiguous, 16-bit N-contiguous (its slab as k rows
// of n, read back transposed) or 8-bit N-contiguous.  Weight gradient: the sum
// runs over an expert's rows, so both operands are k-row slabs.
//
// Chunks of sixteen bytes are loaded through dword-aligned addresses and
// shifted into place on the way to LDS.  A chunk that would pass the end of
// its line starts early enough to end with it and is shifted down by the
// difference, which puts zeros past the end: no load is predicated, none
// leaves the matrix, and every k-tile runs the same code, two tiles ahead of
// the MFMAs in two register sets.  (One loop for whole and another, chunk by
// chunk, for ragged k-tiles: 555 rows' gradient 277 x 1688 took 29 us, 11.6
// now.)  Lines shorter than a chunk and 8-bit N-contiguous weights go element by
// element.
//
// Bound by LDS (fragment reads and the staged writes) at one workgroup's share
// of two a compute unit.  Measured: bf16, 16384 rows on 8 experts, [K, N] weights
// of 4095 x 4095 1075 us, the weight gradient 4095 x 4095 1085 us; 4096 rows x 4096 x
// 4096 with 8-bit [K, N] weights, a byte a load, 311 us in int8 and 342 in e4m3; 4096
// e4m3 rows on 8 experts of 4096 x 256 28 us.
#include "grouped_common.hpp"

namespace tla {
namespace {

enum : int { kBKc = 0, kBElem = 1, kBRows = 2 };

// Sixteen bytes shifted down by n bytes, zeros coming in; 16 and more: zeros.
__device__ __forceinline__ i32x4 shift_down(const i32x4& v, int n) {
  const bool one = n & 4, two = n & 8, out = n >= 16;
  const uint32_t v0 = v[0], v1 = v[1], v2 = v[2], v3 = v[3], sh = (uint32_t)n & 3u;
  const uint32_t a0 = one ? v1 : v0, a1 = one ? v2 : v1, a2 = one ? v3 : v2, a3 = one ? 0u : v3;
  const uint32_t b0 = two ? a2 : a0, b1 = two ? a3 : a1, b2 = two ? 0u : a2, b3 = two ? 0u : a3;
  return i32x4{out ? 0 : (int)__builtin_amdgcn_alignbyte(b1, b0, sh),
               out ? 0 : (int)__builtin_amdgcn_alignbyte(b2, b1, sh),
               out ? 0 : (int)__builtin_amdgcn_alignbyte(b3, b2, sh),
               out ? 0 : (int)__builtin_amdgcn_alignbyte(0u, b3, sh)};
}

// One operand's slab of a k-tile in registers: 1024 chunks, four a thread.
// kRows: 64 rows of k, each 128 columns (16-bit; chunk c of row r stored at
// c ^ 4 (r % 4), as load_frag_nt reads it); otherwise 128 rows of 128 bytes of
// K (load_frag's swizzle).  Lines hold at least one chunk.
template <int EB, bool kRows>
struct LooseSlab {
  static constexpr int kCE = 16 / EB, kI = 4;
  i32x4 v[kI];
  uint32_t hi[kI];
  uint32_t shifts;

  static __device__ __forceinline__ int row(int tid, int it) {
    return (tid + 256 * it) / (kRows ? 16 : 8);
  }
  static __device__ __forceinline__ int col(int tid, int it) {
    return (tid + 256 * it) % (kRows ? 16 : 8) * kCE;
  }
  // lines first + row (clamped to the last one), elements at + col
  __device__ __forceinline__ void load(const uint8_t* __restrict__ base, int64_t ld, int first,
                                       int lines, int at, int len, int tid) {
    shifts = 0;
#pragma unroll
    for (int it = 0; it < kI; ++it) {
      const int r = min(first + row(tid, it), lines - 1), c = min(at + col(tid, it), len - kCE);
      shifts |= load16_split(base + ((int64_t)r * ld + c) * EB, v[it], hi[it]) << (4 * it);
    }
  }
  // cut: the tile passes the lines' end; gone: (kRows) passes the last line
  __device__ __forceinline__ void store(uint8_t* slab, int first, int lines, int at, int len,
                                        int tid) const {
    const bool cut = at + (kRows ? 128 : 128 / EB) > len;
    const bool gone = kRows && first + 64 > lines;
#pragma unroll
    for (int it = 0; it < kI; ++it) {
      i32x4 x = realign16(v[it], hi[it], shifts >> (4 * it));
      const int r = row(tid, it), c = col(tid, it);
      if (cut) x = shift_down(x, max(at + c - (len - kCE), 0) * EB);
      if (gone && first + r >= lines) x = i32x4{0, 0, 0, 0};
      if constexpr (kRows)
        *(i32x4*)(slab + r * 256 + ((c / 8) ^ (4 * (r & 3))) * 16) = x;
      else
        *(i32x4*)(slab + r * 128 + Slab<128>::Swz::chunk(r, c / kCE) * 16) = x;
    }
  }
};

template <int kCode, int kBView, bool kWgrad, bool kLoose>
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
  bool sum_a = false, sum_b = false;  // gradient: this wave sums dY's lines
  const uint8_t *A = p.A, *B = p.B;
  if constexpr (kWgrad) {
    int tm, tn, lo, hi;
    wgrad_tile(p, blockIdx.x, gridDim.x, e, tm, tn);
    expert_rows(p, e, lo, hi);
    sum_a = p.dbias && (p.flags & kOpSumA) && tn == 0 && !(wave >> 1);
    sum_b = p.dbias && !(p.flags & kOpSumA) && tm == 0 && !(wave & 1);
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
  LineSums<kCode, FM> sums;
  if constexpr (kWgrad) sums.init();
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
      if constexpr (kWgrad) {
        if (sum_b) static_for<FN>([&](auto j) { sums.template add<j>(b[cur][j]); });
        if (sum_a) static_for<FM>([&](auto i) { sums.template add<i>(a[cur][i]); });
      }
    });
  };

  const int KT = (K + BK - 1) / BK;
  if constexpr (kLoose) {
    LooseSlab<EB, kAT> ra[2];
    LooseSlab<EB, kNT> rb[2];
    auto load = [&](int kt, auto set) {
      const int k0 = min(kt, KT - 1) * BK;
      if constexpr (kAT) ra[set].load(A, p.lda, k0, K, m0, m_end, tid);
      else ra[set].load(A, p.lda, m0, m_end, k0, K, tid);
      if constexpr (kNT) rb[set].load(B, p.ldb, k0, K, n0, N, tid);
      else rb[set].load(B, p.ldb, n0, N, k0, K, tid);
    };
    auto store = [&](int kt, auto set) {
      uint8_t* st = smem + (kt & 1) * STAGE;
      const int k0 = kt * BK;
      if constexpr (kAT) ra[set].store(st, k0, K, m0, m_end, tid);
      else ra[set].store(st, m0, m_end, k0, K, tid);
      if constexpr (kNT) rb[set].store(st + SLAB_A, k0, K, n0, N, tid);
      else rb[set].store(st + SLAB_A, n0, N, k0, K, tid);
    };
    using S0 = std::integral_constant<int, 0>;
    using S1 = std::integral_constant<int, 1>;
    auto fenced_compute = [&](int kt) {
      __builtin_amdgcn_sched_barrier(0);
      compute(smem + (kt & 1) * STAGE);
      __builtin_amdgcn_sched_barrier(0);
    };
    // tile kt in LDS, tile kt + 1 in set S ^ 1: load tile kt + 2 into set S,
    // multiply, hand tile kt + 1 on.  No branch in the loop, so the waits for
    // loads count exactly.
    auto step = [&](int kt, auto S) {
      load(kt + 2, S);
      fenced_compute(kt);
      store(kt + 1, std::integral_constant<int, S ^ 1>{});
      __syncthreads();
    };
    if (KT > 0) {
      load(0, S0{});
      load(1, S1{});  // (past the end: the last tile again)
      store(0, S0{});
      __syncthreads();
      int kt = 0;
      for (; kt + 2 < KT; kt += 2) {
        step(kt, S0{});
        step(kt + 1, S1{});
      }
      if (kt + 1 < KT) {
        fenced_compute(kt);
        store(kt + 1, S1{});
        __syncthreads();
        ++kt;
      }
      compute(smem + (kt & 1) * STAGE);
    }
  } else {
    using RA = std::conditional_t<kAT, RegSlabNT<BM, BK>, RegSlab<BM, EB, kRowBytes, true>>;
    using RB =
        std::conditional_t<kNT, RegSlabNT<BN, BK>, RegSlab<BN, EB, kRowBytes, kBView == kBKc>>;
    RA ra;
    RB rb;
    auto load = [&](int k0) {
      ra.load_edge(A, p.lda, m0, m_end, k0, K, tid);
      rb.load_edge(B, p.ldb, n0, N, k0, K, tid);
    };
    if (KT > 0) load(0);
    for (int kt = 0; kt < KT; ++kt) {
      ra.store(smem, tid);
      rb.store(smem + SLAB_A, tid);
      __syncthreads();
      if (kt + 1 < KT) load((kt + 1) * BK);
      compute(smem);
      __syncthreads();
    }
  }
  __syncthreads();  // the stages become the waves' epilogue regions
  uint8_t* region = smem + wave * WM * 64 * FN;
  if constexpr (kWgrad) {
    if (sum_b) sums.template write<FN>(p.dbias + (int64_t)e * p.N, n0 + wn0, p.N, lane);
    if (sum_a) sums.template write<FM>(p.dbias + (int64_t)e * p.M, m0 + wm0, p.M, lane);
  }
  if constexpr (kWgrad)
    wgrad_epilogue<FM, FN>(p, e, m0 + wm0, n0 + wn0, lane, acc, region);
  else
    grouped_epilogue<kCode, FM, FN>(p, e, m_end, m0 + wm0, n0 + wn0, lane, acc, region);
}

template <int kCode, int kBView, bool kWgrad, bool kLoose>
int launch_form(const GroupedParams& p0, hipStream_t stream) {
  GroupedParams p = p0;
  p.tiles_n = (p.N + 127) / 128;
  p.tiles_m = (p.M + 127) / 128;
  const int64_t grid = kWgrad ? (int64_t)p.groups * p.tiles_m * p.tiles_n
                              : row_tiles_bound(p.rows, p.groups, 128) * p.tiles_n;
  if (grid <= 0) return TLA_OK;
  if (!grid_fits(grid, kThreads)) return TLA_ERR_UNSUPPORTED;
  hipLaunchKernelGGL((grouped_general_kernel<kCode, kBView, kWgrad, kLoose>), dim3((unsigned)grid),
                     dim3(kThreads), 0, stream, p);
  return hipGetLastError() == hipSuccess ? TLA_OK : TLA_ERR_HIP;
}

template <int kCode, int kBView, bool kWgrad>
int launch(const GroupedParams& p, hipStream_t stream) {
  if constexpr (kBView != kBElem) {
    constexpr int kCE = 16 / type_bytes(kCode);
    // the lines: of K (A, or both), of N, of both extents of the gradient
    const bool a_long = kWgrad ? p.M >= kCE : p.K >= kCE;
    const bool b_long = kBView == kBKc ? p.K >= kCE : p.N >= kCE;
    if (a_long && b_long) return launch_form<kCode, kBView, kWgrad, true>(p, stream);
  }
  return launch_form<kCode, kBView, kWgrad, false>(p, stream);
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

}  // namespace tla
