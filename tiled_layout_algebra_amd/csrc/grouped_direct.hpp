// grouped_direct.hpp -- the grouped products' kernel for tiles of 128 rows
// and columns, filled by direct global -> LDS copies.
//
// The loop is gemm.hip's single-group one: a software pipeline over every
// MFMA step, the copies of a later k-tile between the MFMAs of the current
// one, one barrier a k-tile, the next step's fragments read a step ahead.
// LDS holds kStages A slabs and kStages B slabs of 128 bytes of K.  With two
// stages two workgroups share a compute unit, so one's prologue and epilogue
// run under the other's loop.  Forms and tile lookup as in
// grouped_two_group.hpp, but the rows of kNKShift bring the dword after their
// window with them, so a k-tile is the whole window.
//
// Bound by LDS reads (a 64 x 32 wave tile reads three 16-byte fragments for two
// MFMAs: about 1020 of a k-tile's 1190 cycles) or, with few rows an expert, by
// the weights' way from memory.  Measured: bf16, 4096 rows on 32 experts of
// 2048 x 4096 151 us (128 x 128; 537 MB of weights: 3.6 TB/s), 2048 rows 117 us
// (64 x 128; 4.6 TB/s), int8 512 rows x 4096 x 4096 17 us; kNKShift, 4096 rows 2048 x
// 4095 241 us (its dword loads and copies across two lines cost the difference);
// 777 rows' fp32 gradients on 16 experts of 512 x 1024 12 us (33.5 MB written).  The
// gated forms (Role, as in grouped_two_group.hpp; half as many columns of the result):
// bf16, 4096 x 4096, 96 rows or fewer 23 us (64 x 128), 400 rows 35-38 (128 x 128).
#pragma once

#include "gated_common.hpp"

namespace tla {
namespace {

enum Form : int { kNK = 0, kKN = 1, kGrad = 2, kNKShift = 3 };

// dma16_buf for a dword a lane
__device__ __forceinline__ void dma4_buf(const uint8_t* base, uint32_t voffset, uint32_t soffset,
                                         uint8_t* lds, int records) {
#if defined(__HIP_DEVICE_COMPILE__)
  __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc((void*)base, 0, records, 0x00020000);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 4, voffset,
                                           soffset, 0, 0);
#endif
}

template <int kCode, int kForm, int BM, int BN, int kStages, int kFront, int kWM, int kWN,
          int kRole = kPlain>
__global__ __launch_bounds__(64 * kWM * kWN) void grouped_direct_kernel(const GroupedParams p) {
  constexpr bool kShift = kForm == kNKShift;
  using Atom = std::conditional_t<kShift && kCode == kE4M3, E4m3Bytes, OpAtom<kCode>>;
  constexpr int kRowBytes = 128;
  constexpr bool kBT = kForm == kKN || kForm == kGrad, kAT = kForm == kGrad;
  using Frag = typename Atom::Frag;
  using Swz = typename Slab<kRowBytes>::Swz;
  constexpr int NT = 64 * kWM * kWN;  // kWM x kWN wavefronts
  constexpr int EB = type_bytes(kCode);
  constexpr int BK = kRowBytes / EB;
  constexpr int WM = BM / kWM, WN = BN / kWN;
  constexpr int FM = WM / 32, FN = WN / 32;
  constexpr int KSTEPS = BK / Atom::kK;
  static_assert(BK % Atom::kK == 0 && KSTEPS >= 2 && KSTEPS % 2 == 0,
                "fragment buffers alternate per step");
  static_assert(kStages >= 2, "copies need a free slot");
  constexpr int SLAB_A = BM * kRowBytes, SLAB_B = BN * kRowBytes;
  constexpr int B_BASE = kStages * SLAB_A;
  static_assert(kStages * (SLAB_A + SLAB_B) <= 160 * 1024, "LDS budget");
  static_assert(!kBT || (EB == 2 && BN >= 128), "N-contiguous B: 16-bit");
  static_assert(!kAT || (EB == 2 && BM >= 128), "M-contiguous A: 16-bit");
  // kGated: the first half of B's slab is the gate's columns, the other half the
  // same columns of the up projection (an N-contiguous slab: 64 rows of each); a
  // wave's first FN / 2 MFMA tiles are the gate's
  constexpr bool kTwo = kRole == kGated;
  constexpr int BNO = kTwo ? BN / 2 : BN, FH = FN / 2;  // columns of D; of a wave's tiles, one operand's
  static_assert(!kTwo || FN % 2 == 0, "a wave holds both sums of an element");
  constexpr int kRowBT = BNO * 2;                  // bytes per k row of an N-contiguous slab
  constexpr int kChBT = kRowBT / 16;
  constexpr int kRowAT = BM * 2;                   // bytes per k row of an M-contiguous slab
  constexpr int kChAT = kRowAT / 16;
  static_assert(kStages * SLAB_A <= 65536 && kStages * SLAB_B <= 65536, "fragment immediates");
  constexpr int kChunks = Slab<kRowBytes>::kChunks;
  static_assert((1 << Slab<kRowBytes>::kRowShift) * kChunks <= 32, "swizzle period divides 32 rows");
  constexpr int IA = BM * kChunks / NT, IB = BN * kChunks / NT;
  static_assert(IA * NT == BM * kChunks && IB * NT == BN * kChunks, "whole copy instructions");
  // copies per thread per tile; kShift: the last one a dword a row
  constexpr int kLoads = IA + IB + (kShift ? 1 : 0);
  constexpr int TAIL_BASE = kStages * (SLAB_A + SLAB_B), kTail = kShift ? 4 * NT : 0;
  static_assert(!kShift || (kWM * kWN * 64 >= BM + BN && BM % 64 == 0), "a wave's rows are A's or B's");
  constexpr int kSub = Atom::kLaneBytes / 16;      // 16-byte reads per fragment
  constexpr int kReads =
      kShift ? 2 * (FM + FN) : (kAT ? 2 * FM : FM * kSub) + (kBT ? 2 * FN : FN * kSub);
  constexpr int kMfmas = FM * FN;
  constexpr int kStepBytes = Atom::kK * EB;
  // Copies per full step, the rest go into the first half of the last step.
  // kFront > 0 puts all copies into the first kFront steps instead.
  constexpr int kSpread = kFront > 0 && kFront < KSTEPS ? kFront : KSTEPS;
  constexpr int kPerStep = (kLoads + kSpread - 1) / kSpread;
  constexpr int kFull = kPerStep * (KSTEPS - 1) < kLoads ? kPerStep * (KSTEPS - 1) : kLoads;
  constexpr int kLast = kLoads - kFull;
  constexpr int kWait = (kStages - 2) * kLoads;  // copies allowed in flight past the next tile
  __shared__ __attribute__((aligned(1024))) uint8_t smem[TAIL_BASE + kStages * kTail];

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  int e, m0, m_end, n0, K;
  bool sum_a = false, sum_b = false;  // gradient: this wave sums dY's lines
  const uint8_t *A = p.A, *B = p.B;
  if constexpr (kForm == kGrad) {
    int tm, tn, lo, hi;
    wgrad_tile(p, blockIdx.x, gridDim.x, e, tm, tn);
    expert_rows(p, e, lo, hi);
    sum_a = p.dbias && (p.flags & kOpSumA) && tn == 0 && wave / kWM == 0;
    sum_b = p.dbias && !(p.flags & kOpSumA) && tm == 0 && wave % kWM == 0;
    m0 = tm * BM;
    m_end = p.M;
    n0 = tn * BN;
    K = hi - lo;
    A += (int64_t)lo * p.lda * EB;
    B += (int64_t)lo * p.ldb * EB;
  } else {
    RowTile rt;
    if (!row_tile<BM>(p, blockIdx.x, rt)) return;
    e = rt.e;
    m0 = rt.r0;
    m_end = rt.r1;
    n0 = rt.tn * BNO;
    K = p.K;
    // 32-bit offsets count from the tile's first row
    A += (int64_t)m0 * p.lda * EB;
    B += ((int64_t)e * p.stride_b + (kBT ? 0 : (int64_t)n0 * p.ldb)) * EB;
  }
  const int wm0 = (wave % kWM) * WM, wn0 = (wave / kWM) * WN;
  const int wb0 = kTwo ? wn0 / 2 : wn0;  // the wave's first column
  const int64_t up_by = kTwo ? p.B2 - p.B : 0;
  const int KT = (K + BK - 1) / BK;
  const int KTf = K / BK;  // whole k-tiles; tile KTf, if K ends inside it, is ragged

  // kShift: rows begin at any byte.  Copies start at each row's dword, so its
  // bytes land `row_shift` late and the window's last ones in a dword of its
  // own (tail), a row a lane.
  const uint32_t a_rb = (uint32_t)(p.lda * EB), b_rb = (uint32_t)(p.ldb * EB);
  const uint32_t a_off = kShift ? (uint32_t)(uintptr_t)A & 3u : 0u;
  const uint32_t b_off = kShift ? (uint32_t)(uintptr_t)B & 3u : 0u;
  auto row_shift = [&](bool is_a, int r) {
    return ((is_a ? a_off : b_off) + (uint32_t)r * (is_a ? a_rb : b_rb)) & 3u;
  };
  const int a_last = m_end - 1 - m0, b_last = p.N - 1 - n0;
  if constexpr (kShift) {
    A -= a_off;
    B -= b_off;
  }
  // each operand's bytes from its base up to the last dword that it needs
  auto k_rows_bytes = [&](int64_t ld, int lines) {
    return K > 0 ? (int)min((((K - 1) * ld + lines) * EB + 3) & ~(int64_t)3, (int64_t)0x7FFFFFFC) : 0;
  };
  const int a_bytes = kAT ? k_rows_bytes(p.lda, p.M)
                          : (int)((min(a_last, BM - 1) * a_rb + K * EB + a_off + 3) & ~3u);
  const int b_bytes = kBT ? k_rows_bytes(p.ldb, p.N)
                          : (int)((min(b_last, BNO - 1) * b_rb + K * EB + b_off + 3) & ~3u);
  // Copy q (A for q < IA, else B): slab row r = tid/kChunks + (NT/kChunks)*q',
  // landing at slab slot wave*64 + NT*q' (lane-linear); the lane fetches the
  // global chunk the swizzle assigns to that slot, from row r clamped to the
  // matrix (rows past M or N are never stored).
  uint32_t off[kLoads];
  static_for<kLoads>([&](auto q) {
    constexpr bool kA = q < IA;
    constexpr int qq = kA ? q : q - IA;
    if constexpr (q == IA + IB) {
      const int r = tid < BM ? tid : tid - BM;
      const bool is_a = tid < BM;
      const int row = min(r, is_a ? a_last : b_last);
      off[q] = tid < BM + BN ? ((uint32_t)row * (is_a ? a_rb : b_rb) + (is_a ? a_off : b_off)) / 4 * 4 +
                                   kRowBytes
                             : 0x80000000u;
    } else if constexpr (kA && kAT) {
      // as for an N-contiguous B: k row r, stored chunk pc holding columns
      // m0 + 8 (pc ^ 4 (r % 4)) .. + 7, clamped to M's last chunk (whose
      // columns past M feed nothing that is stored)
      const int sc = tid + NT * qq, r = sc / kChAT, pc = sc % kChAT;
      const int m = min(m0 + 8 * (pc ^ (4 * (r & 3))), (p.M - 1) & ~7);
      off[q] = (uint32_t)(((int64_t)r * p.lda + m) * EB);
    } else if constexpr (!kA && kBT) {
      // slab chunk tid + NT q': k row r, stored chunk pc, which holds logical
      // chunk pc ^ 4 (r % 4): columns n0 + 8 lc .. + 7, clamped to the
      // matrix' last chunk (columns past N are never stored)
      // (kTwo: of the half slab, whose 128-byte rows swap halves by r / 2)
      constexpr int qh = kTwo ? qq % (IB / 2) : qq;
      const int sc = tid + NT * qh, r = sc / kChBT, pc = sc % kChBT;
      const int n = min(n0 + 8 * (pc ^ (4 * (kTwo ? (r >> 1) & 1 : r & 3))), (p.N - 1) & ~7);
      off[q] = (uint32_t)(((int64_t)r * p.ldb + n) * EB);
    } else {
      constexpr int qh = kTwo && !kA ? qq % (IB / 2) : qq;
      const int r = tid / kChunks + (NT / kChunks) * qh;
      const int64_t row = kA ? min(r, m_end - 1 - m0) : min(r, p.N - 1 - n0);
      const int64_t rb = (kA ? p.lda : p.ldb) * EB;
      off[q] = (uint32_t)(row * rb + Swz::chunk(r, tid % kChunks) * 16);
      if constexpr (kShift)
        off[q] = (uint32_t)(row * rb + (kA ? a_off : b_off)) / 4 * 4 +
                 Swz::chunk(r, tid % kChunks) * 16;
    }
  });
  // The ragged last k-tile: bit q is set when copy q's K-contiguous chunk lies
  // past K -- that copy then reads from past every record and the range check
  // returns zeros (the chunk that crosses K: clear_tail).  An N-contiguous B
  // slab's rows past K lie past its record count (K rows).
  uint32_t tail_past = 0;
  static_for<kShift ? 0 : kLoads>([&](auto q) {
    constexpr bool kA = q < IA;
    constexpr int qq = kA ? q : q - IA;
    if constexpr (kA ? !kAT : !kBT) {
      const int r = tid / kChunks + (NT / kChunks) * qq;
      if (Swz::chunk(r, tid % kChunks) * 16 >= (K - KTf * BK) * EB) tail_past |= 1u << q;
    }
  });
  // Fragment bases for each k-step (and each 16-byte half of a 32-byte
  // fragment): row wm0 + lane%32 of the A slot, wn0 + lane%32 of the B slot.
  uint32_t fa[KSTEPS][kSub], fb[KSTEPS][kSub];
  static_for<KSTEPS>([&](auto ks) {
    static_for<kSub>([&](auto u) {
      const int c = (ks * kStepBytes + (lane >> 5) * Atom::kLaneBytes) / 16 + u;
      const int ra = wm0 + (lane & 31), rb = wb0 + (lane & 31);
      fa[ks][u] = (uint32_t)(ra * kRowBytes + Swz::chunk(ra, c) * 16);
      fb[ks][u] = (uint32_t)(B_BASE + rb * kRowBytes + Swz::chunk(rb, c) * 16);
    });
  });
  // N-contiguous B: the two transpose reads of k-step ks (k0 = 16 ks +
  // 8 (quarter-wave / 2) + 4 h) for lane a = lane % 16 of its quarter-wave
  uint32_t fbt[kBT ? KSTEPS : 1][kBT ? FN : 1][2];
  if constexpr (kBT) {
    const int qw = lane >> 4, a4 = lane & 15;
    static_for<KSTEPS>([&](auto ks) {
      static_for<FN>([&](auto j) {
        static_for<2>([&](auto h) {
          const int k = 16 * ks + 8 * (qw >> 1) + 4 * h + (a4 >> 2);
          const int jj = kTwo ? (int)j % FH : (int)j;
          const int n = wb0 + 32 * jj + 16 * (qw & 1) + 4 * (a4 & 3);
          const int swap = 4 * (kTwo ? (k >> 1) & 1 : k & 3);
          fbt[ks][j][h] = (uint32_t)(B_BASE + (kTwo && j >= FH ? SLAB_B / 2 : 0) + k * kRowBT +
                                     (((n >> 3) ^ swap) * 16) + (n & 7) * 2);
        });
      });
    });
  }

  // M-contiguous A: the same two reads for each 32-row fragment i (the
  // swizzle does not commute with the 32-row step, so each has its bases)
  uint32_t fat[kAT ? KSTEPS : 1][kAT ? FM : 1][2];
  if constexpr (kAT) {
    const int qw = lane >> 4, a4 = lane & 15;
    static_for<KSTEPS>([&](auto ks) {
      static_for<FM>([&](auto i) {
        static_for<2>([&](auto h) {
          const int k = 16 * ks + 8 * (qw >> 1) + 4 * h + (a4 >> 2);
          const int m = wm0 + 32 * i + 16 * (qw & 1) + 4 * (a4 & 3);
          fat[ks][i][h] = (uint32_t)(k * kRowAT + (((m >> 3) ^ (4 * (k & 3))) * 16) + (m & 7) * 2);
        });
      });
    });
  }

  // kShift: the dword after the fragment of step ks is dword 0 of the next
  // chunk, or the row's tail dword after chunk 7 (the last step's upper lanes):
  // its address, the distance between slots and between 32-row fragments
  uint32_t na[kShift ? KSTEPS : 1], nb[kShift ? KSTEPS : 1], sh_a = 0, sh_b = 0;
  uint32_t step_a = SLAB_A, step_b = SLAB_B, frag32 = 32 * kRowBytes;
  if constexpr (kShift) {
    const int ra = wm0 + (lane & 31), rb = wn0 + (lane & 31), half = lane >> 5;
    sh_a = row_shift(true, ra);
    sh_b = row_shift(false, rb);
    static_for<KSTEPS>([&](auto ks) {
      const int c = 2 * ks + half + 1;
      na[ks] = c < 8 ? ra * kRowBytes + Swz::chunk(ra, c & 7) * 16 : TAIL_BASE + 4 * ra;
      nb[ks] = c < 8 ? B_BASE + rb * kRowBytes + Swz::chunk(rb, c & 7) * 16
                     : TAIL_BASE + 4 * (BM + rb);
    });
    if (half) {  // of the last step
      step_a = step_b = kTail;
      frag32 = 32 * 4;
    }
  }
  uint32_t xa[kShift ? 2 : 1][FM], xb[kShift ? 2 : 1][FN];
  typename Atom::Acc acc[FM][FN];
  static_for<FM>([&](auto i) { static_for<FN>([&](auto j) { acc[i][j] = typename Atom::Acc{}; }); });
  LineSums<kCode, (FM > FN ? FM : FN)> sums;
  if constexpr (kForm == kGrad) sums.init();
  Frag a[2][FM], b[2][FN];
  auto lds_frag = [&](const uint32_t (&base)[kSub], int imm) -> Frag {
    if constexpr (kSub == 1) {
      return *(const i32x4*)(smem + base[0] + imm);
    } else {
      const i32x4 lo = *(const i32x4*)(smem + base[0] + imm);
      const i32x4 hi = *(const i32x4*)(smem + base[1] + imm);
      return Frag{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    }
  };
  auto lds_frag_t = [&](const uint32_t (&base)[2], int imm) -> Frag {
    typedef int s32x2 __attribute__((ext_vector_type(2)));
    const s16x4 lo = ds_read_tr16(smem + base[0] + imm);
    const s16x4 hi = ds_read_tr16(smem + base[1] + imm);
    const s32x2 l2 = __builtin_bit_cast(s32x2, lo), h2 = __builtin_bit_cast(s32x2, hi);
    return Frag{l2[0], l2[1], h2[0], h2[1]};
  };
  auto read_frags = [&](auto buf, auto slot, auto ks) {
    if constexpr (kAT)
      static_for<FM>([&](auto i) { a[buf][i] = lds_frag_t(fat[ks][i], slot * SLAB_A); });
    else
      static_for<FM>([&](auto i) { a[buf][i] = lds_frag(fa[ks], slot * SLAB_A + i * 32 * kRowBytes); });
    if constexpr (kBT)
      static_for<FN>([&](auto j) { b[buf][j] = lds_frag_t(fbt[ks][j], slot * SLAB_B); });
    else
      static_for<FN>([&](auto j) {
        constexpr int at = kTwo ? j % FH * 32 * kRowBytes + j / FH * (SLAB_B / 2) : j * 32 * kRowBytes;
        b[buf][j] = lds_frag(fb[ks], slot * SLAB_B + at);
      });
    if constexpr (kShift) {
      static_for<FM>([&](auto i) {
        const uint32_t at = ks + 1 < KSTEPS ? na[ks] + slot * SLAB_A + i * 32 * kRowBytes
                                            : na[ks] + slot * step_a + i * frag32;
        xa[buf][i] = *(const uint32_t*)(smem + at);
      });
      static_for<FN>([&](auto j) {
        const uint32_t at = ks + 1 < KSTEPS ? nb[ks] + slot * SLAB_B + j * 32 * kRowBytes
                                            : nb[ks] + slot * step_b + j * frag32;
        xb[buf][j] = *(const uint32_t*)(smem + at);
      });
    }
  };
  // kShift: a step's fragments moved into place before its MFMAs
  auto place = [&](auto buf) {
    if constexpr (kShift) {
      auto shift = [](Frag& w, uint32_t x, uint32_t sh) {
        const uint32_t w0 = w[0], w1 = w[1], w2 = w[2], w3 = w[3];
        w[0] = (int)__builtin_amdgcn_alignbyte(w1, w0, sh);
        w[1] = (int)__builtin_amdgcn_alignbyte(w2, w1, sh);
        w[2] = (int)__builtin_amdgcn_alignbyte(w3, w2, sh);
        w[3] = (int)__builtin_amdgcn_alignbyte(x, w3, sh);
      };
      static_for<FM>([&](auto i) { shift(a[buf][i], xa[buf][i], sh_a); });
      static_for<FN>([&](auto j) { shift(b[buf][j], xb[buf][j], sh_b); });
    }
  };
  // Clears what a last k-tile that ends inside a chunk holds past K (the next
  // row's bytes) in slot S, a thread a row, between its landing and its first
  // reader
  auto clear_tail = [&](int kt, auto S) {
    if constexpr (kForm != kGrad) {
      if (kt != KTf || !(kShift || K * EB % 16 != 0)) return;
      if (tid < (kBT ? BM : BM + BN)) {
        const bool is_a = tid < BM;
        const int r = is_a ? tid : tid - BM;  // (the swizzle repeats within half a slab)
        uint8_t* row = smem + (is_a ? S * SLAB_A : B_BASE + S * SLAB_B) + r * kRowBytes;
        const int first = (kShift ? (int)row_shift(is_a, min(r, is_a ? a_last : b_last)) : 0) +
                          (K - KTf * BK) * EB;
        const int end = kShift ? 33 : (first + 15) / 16 * 4;
        for (int d = first >> 2; d < end; ++d) {
          uint32_t* w = d < 32 ? (uint32_t*)(row + Swz::chunk(r, d >> 2) * 16 + (d & 3) * 4)
                               : (uint32_t*)(smem + TAIL_BASE + S * kTail + 4 * tid);
          *w = d == first >> 2 ? *w & ((1u << (8 * (first & 3))) - 1u) : 0u;
        }
      }
      __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
      stage_barrier();
    }
  };
  auto mma = [&](auto buf, auto idx) {
    Atom::mma(acc[idx / FN][idx % FN], b[buf][idx % FN], a[buf][idx / FN]);
  };
  // copy q of tile t into slot `slot`; tiles past K reload the last one
  auto copy = [&](int t, auto slot, auto q) {
    const int tt = min(t, KT - 1);
    const uint32_t kb = (uint32_t)tt * kRowBytes;
    const uint32_t o = (tt == KTf && ((tail_past >> q) & 1)) ? 0x80000000u : off[q];
    if constexpr (q == IA + IB) {
      const bool is_a = wave * 64 < BM;
      dma4_buf(is_a ? A : B, off[q], kb, smem + TAIL_BASE + slot * kTail + wave * 256,
               is_a ? a_bytes : b_bytes);
    } else if constexpr (q < IA && kAT)
      dma16_buf(A, off[q], (uint32_t)(tt * BK) * (uint32_t)(p.lda * EB),
                smem + slot * SLAB_A + (wave * 64 + NT * q) * 16, a_bytes);
    else if constexpr (q < IA)
      dma16_buf(A, o, kb, smem + slot * SLAB_A + (wave * 64 + NT * q) * 16, a_bytes);
    else {
      const uint8_t* from = B;
      if constexpr (kTwo && q - IA >= IB / 2) from += up_by;
      if constexpr (kBT)
        dma16_buf(from, off[q], (uint32_t)(tt * BK) * (uint32_t)(p.ldb * EB),
                  smem + B_BASE + slot * SLAB_B + (wave * 64 + NT * (q - IA)) * 16, b_bytes);
      else
        dma16_buf(from, o, kb, smem + B_BASE + slot * SLAB_B + (wave * 64 + NT * (q - IA)) * 16,
                  b_bytes);
    }
  };
  // MFMAs [lo, hi) of a step with copies [q0, q0 + nq) of tile t spread
  // evenly between them: after MFMA k come copies [k*nq/n, (k+1)*nq/n).
  auto mfmas_with_copies = [&](auto buf, auto lo, auto hi, int t, auto slot, auto q0, auto nq) {
    constexpr int n = hi - lo;
    static_for<n>([&](auto k) {
      mma(buf, std::integral_constant<int, lo + k>{});
      constexpr int c0 = k * nq / n, c1 = (k + 1) * nq / n;
      static_for<c1 - c0>([&](auto c) { copy(t, slot, std::integral_constant<int, q0 + c0 + c>{}); });
    });
    static_for<n>([&](auto k) {
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      constexpr int c0 = k * nq / n, c1 = (k + 1) * nq / n;
      if constexpr (c1 > c0) __builtin_amdgcn_sched_group_barrier(0x020, c1 - c0, 0);
    });
  };
  // k-tile kt, which lives in slot S (= kt % kStages)
  auto tile = [&](int kt, auto S) {
    using Next = std::integral_constant<int, (S + 1) % kStages>;
    using Fill = std::integral_constant<int, (S + kStages - 1) % kStages>;
    const int ct = kt + kStages - 1;  // tile whose copies are issued now
    static_for<KSTEPS>([&](auto ks) {
      constexpr int cur = ks & 1;
      place(std::integral_constant<int, cur>{});
      if constexpr (kForm == kGrad) {
        if (sum_b) static_for<FN>([&](auto j) { sums.template add<j>(b[cur][j]); });
        if (sum_a) static_for<FM>([&](auto i) { sums.template add<i>(a[cur][i]); });
      }
      if constexpr (ks + 1 < KSTEPS) {
        read_frags(std::integral_constant<int, cur ^ 1>{}, S, std::integral_constant<int, ks + 1>{});
        __builtin_amdgcn_sched_group_barrier(0x100, kReads, 0);
        constexpr int q0 = ks * kPerStep < kFull ? ks * kPerStep : kFull;
        constexpr int q1 = (ks + 1) * kPerStep < kFull ? (ks + 1) * kPerStep : kFull;
        mfmas_with_copies(std::integral_constant<int, cur>{}, std::integral_constant<int, 0>{},
                          std::integral_constant<int, kMfmas>{}, ct, Fill{},
                          std::integral_constant<int, q0>{}, std::integral_constant<int, q1 - q0>{});
      } else {
        mfmas_with_copies(std::integral_constant<int, cur>{}, std::integral_constant<int, 0>{},
                          std::integral_constant<int, kMfmas / 2>{}, ct, Fill{},
                          std::integral_constant<int, kFull>{}, std::integral_constant<int, kLast>{});
        if (kt + 1 < KT) {
          wait_vmcnt<kWait>();  // tile kt+1 landed (this thread's copies)
          stage_barrier();      // ... everyone's; tile kt-1's slot is free
          clear_tail(kt + 1, Next{});
          read_frags(std::integral_constant<int, cur ^ 1>{}, Next{}, std::integral_constant<int, 0>{});
        }
        static_for<kMfmas - kMfmas / 2>([&](auto k) {
          mma(std::integral_constant<int, cur>{}, std::integral_constant<int, kMfmas / 2 + k>{});
        });
      }
    });
  };

  // the gradient's first gate and up values, under the loop
  GateParts<kRole == kGateGrad ? WM : 32, kRole == kGateGrad ? WN : 32> z;
  if constexpr (kRole == kGateGrad) z.ask(p, m_end, m0 + wm0, n0 + wn0, lane, 0);
  if (KT > 0) {
    static_for<kStages - 1>([&](auto t) {
      static_for<kLoads>([&](auto q) { copy(t, t, q); });
    });
    wait_vmcnt<kWait>();
    stage_barrier();
    clear_tail(0, std::integral_constant<int, 0>{});
    read_frags(std::integral_constant<int, 0>{}, std::integral_constant<int, 0>{},
               std::integral_constant<int, 0>{});
    for (int kt = 0; kt < KT; kt += kStages) {
      static_for<kStages>([&](auto s) {
        if (kt + s < KT) tile(kt + s, s);
      });
    }
    wait_vmcnt<0>();  // no copy may land in LDS after this point
  }

  // Every wave is past its last LDS read: the slots become the waves'
  // epilogue regions.
  static_assert((NT / 64) * WM * 64 * FN <= kStages * (SLAB_A + SLAB_B), "epilogue regions");
  __syncthreads();
  uint8_t* region = smem + wave * WM * 64 * FN;
  if constexpr (kForm == kGrad) {
    if (sum_b) sums.template write<FN>(p.dbias + (int64_t)e * p.N, n0 + wn0, p.N, lane);
    if (sum_a) sums.template write<FM>(p.dbias + (int64_t)e * p.M, m0 + wm0, p.M, lane);
  }
  if constexpr (kForm == kGrad)
    wgrad_epilogue<FM, FN>(p, e, m0 + wm0, n0 + wn0, lane, acc, region);
  else if constexpr (kRole == kGateGrad)
    grad_epilogue<kCode, 0>(p, m_end, m0 + wm0, n0 + wn0, lane, acc, z, region);
  else if constexpr (kRole != kPlain)
    role_epilogue<kCode, kRole, 0, 32, WM, kTwo ? WN / 2 : WN>(p, e, m_end, m0 + wm0, n0 + wb0, lane,
                                                               acc, region);
  else
    grouped_epilogue<kCode, FM, FN>(p, e, m_end, m0 + wm0, n0 + wn0, lane, acc, region);
}

template <int kCode, int kForm, int BM, int BN, int kStages, int kFront, int kWM, int kWN,
          int kRole = kPlain>
int launch(const GroupedParams& p0, hipStream_t stream) {
  GroupedParams p = p0;
  constexpr int kCols = kRole == kGated ? BN / 2 : BN;
  p.tiles_n = (p.N + kCols - 1) / kCols;
  p.tiles_m = (p.M + BM - 1) / BM;
  const int64_t grid = kForm == kGrad ? (int64_t)p.groups * p.tiles_m * p.tiles_n
                                      : row_tiles_bound(p.rows, p.groups, BM) * p.tiles_n;
  if (grid <= 0) return TLA_OK;
  if (!grid_fits(grid, 64 * kWM * kWN)) return TLA_ERR_UNSUPPORTED;
  hipLaunchKernelGGL((grouped_direct_kernel<kCode, kForm, BM, BN, kStages, kFront, kWM, kWN, kRole>),
                     dim3((unsigned)grid), dim3(64 * kWM * kWN), 0, stream, p);
  return hipGetLastError() == hipSuccess ? TLA_OK : TLA_ERR_HIP;
}

}  // namespace
}  // namespace tla
