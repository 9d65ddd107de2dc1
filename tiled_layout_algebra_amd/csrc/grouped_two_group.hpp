// grouped_two_group.hpp -- the 256 x 256 kernel of the expert-grouped
// products, for tiles enough to fill the card.
//
// The tile program is the two-group one of gemm_pingpong.hip: eight
// wavefronts in two groups of four, one wave of each group on a SIMD; a group
// alternates between a memory phase (a k-tile's fragments from LDS, the
// direct global -> LDS copies of a later one in between) and a compute phase
// (the k-tile's 32 MFMAs, nothing else), half a period apart from the other
// group, so that one multiplies while the other moves data.  LDS holds two A
// slabs and three B slabs of 128 bytes of K: all 160 KiB.  What differs:
//   tiles     come from the ragged lookup, so the last block of an expert's
//             rows ends inside the tile; copies past it read zeros through
//             the buffer range check, and waves without a row skip their
//             MFMAs
//   kNK, kKN  the product with B K-contiguous ([N, K] weights) or
//             N-contiguous (16-bit [K, N] weights: a slab of k rows, read
//             back by transposing LDS reads)
//   kGrad     the weight gradient: the sum runs over the expert's rows, both
//             operands are slabs of k rows, and the rows past the expert's
//             last lie past the copies' record counts, so any number of rows
//             works
//   int8      the 16-bit geometry with 32 K a step and integer sums
//   kNKShift  the product for rows at any byte address.  Copies take 16-byte
//             chunks from each row's dword-aligned address, so a row's bytes
//             land 0 to 3 bytes late; a fragment is its sixteen bytes and the
//             dword after them, moved into place by v_alignbyte (4 vector
//             operations a fragment, under the other group's MFMAs).  A k-tile
//             uses 96 of the window's 128 bytes, so that dword is always in it:
//             three MFMA steps a period instead of four.
//   Role      kGated: half of B's slab is columns of the gate's projection, half the
//             same columns of up's, so that a lane holds both sums of an element and
//             the epilogue has act(gate) up without meeting another lane; a tile is
//             256 x 128 of the result.  kGateGrad: a plain product whose epilogue
//             reads gate and up and writes both gradients (and the hidden values):
//             the product itself is never stored.
//   e4m3 with block scales  a k-tile is a block of 128 of K.  The matrix instruction
//             starts from zero and its result is scaled into the sums by vector
//             multiply-adds, which run under the other group's MFMAs.  Scales travel
//             with the fragments' lanes and are spread by register swaps (by LDS
//             permutes: 456 us for 8192^3 instead of 442).
//
// Bound by the matrix cores (busy 0.72 of the time in the int8 case below, at
// the clock that leaves).  Measured, calls in a row on the same buffers; boxes
// differ by up to 8 %: bf16, 16384 rows, one expert of 4096 x 4096 423 us = 1300
// TFLOP/s, [K, N] weights 421 us; the same rows over 8 experts with GELU, bias and
// the pre-activation kept 546 us, the input gradient of 16001 rows with GELU's
// derivative 557 us, the weight gradient 516 us in bf16 (618 where every call finds
// other buffers) and 587 in fp32 (a tile's epilogue writes 128 KiB, 256 KiB with the
// pre-activation or in fp32, and every compute unit does so at once); 8192^3 with
// bias and GELU 472 us = 2330 TOP/s in int8, 411 us = 2670 TFLOP/s in e4m3; kNKShift
// on 8 experts of 4096 x 4095 720 us.  A round of tiles that fills part of the card
// costs most of a whole one: see two_group_lookup.  kGated, bf16, 8192 rows x 8192
// columns x 4096, SiLU, gate and up kept: 820-845 us = 1320 TFLOP/s, of which the 400
// MB written are 60 (MFMA busy 0.78).  kGateGrad at the same sizes, SiLU, hidden
// written: 538 us; a tile's epilogue moves 640 KiB, and every compute unit does so at
// once (busy 0.56); beside the sums and a part's gate and up 52 to 66 registers spill
// there, none in the loop.  Every other unit begun half a tile ahead, so that epilogues meet
// products: 616 instead of 579 then, its half tiles cost more.  Block scales: 8192^3
// 440 us = 2500 TFLOP/s, e4m3 without scales 390 on that box, at 1.66 GHz both by the
// card's power (busy 0.65; 16 to 66 registers spill); gated, 2048 x 8192 x 4096, 120 us,
// two rounds of tiles.
#pragma once

#include "gated_common.hpp"
#include "two_group_lds.hpp"

namespace tla {
namespace {

enum Form : int { kNK = 0, kKN = 1, kGrad = 2, kNKShift = 3 };

// Where a workgroup's tile lies: rows m0 .. of the expert, which end at m_end;
// columns n0 ..; the operands' bases, and the length of the sum.  Product: rows
// of A and of D.  Gradient: the expert's rows are the K of both operands, m0
// and n0 columns of them; sum_a / sum_b: this wave sums dY's lines.
struct TileSpan {
  int e, m0, m_end, n0, K;
  const uint8_t *A, *B, *B2;  // (B2: role kGated)
  bool sum_a, sum_b;
};

// The tile program.  kHalf: 128 x 256 instead of 256 x 256, for blocks of at
// most 128 rows: both groups share the rows and take half the columns each, so
// every wave multiplies 64 x 64 (16 MFMAs a k-tile, not 32) and none idles.
template <int kCode, int kForm, bool kHalf, int kRole, int kAct>
__device__ __forceinline__ void two_group_tile(const GroupedParams& p, const TileSpan& ts,
                                               uint8_t* smem) {
  constexpr bool kShift = kForm == kNKShift;
  using Atom = std::conditional_t<kShift && kCode == kE4M3, E4m3Bytes, OpAtom<kCode>>;
  using Frag = typename Atom::Frag;
  constexpr int kRowBytes = 128;
  using Swz = typename Slab<kRowBytes>::Swz;
  constexpr int kChunks = Slab<kRowBytes>::kChunks;
  constexpr int EB = type_bytes(kCode);
  constexpr bool kBT = kForm == kKN || kForm == kGrad, kAT = kForm == kGrad;
  constexpr int kUsed = kShift ? 96 : kRowBytes;  // bytes of K in a k-tile
  constexpr int BK = kUsed / EB;                // K elements per k-tile
  constexpr int BM = kHalf ? 128 : 256, BN = 256;
  constexpr int WM = 64, WN = kHalf ? 64 : 128;  // wave tile
  constexpr bool kBlocks = kCode == kE4M3Blocks;
  constexpr int FR = kBlocks ? 16 : 32;         // rows of an MFMA tile
  constexpr int FM = WM / FR, FN = WN / FR;     // MFMA tiles per wave
  constexpr int KSTEPS = BK / Atom::kK;         // MFMA k-steps per k-tile
  constexpr int kSub = Atom::kLaneBytes / 16;   // 16-byte reads per fragment
  constexpr int kStepBytes = Atom::kK * EB;
  constexpr int SLAB = BN * kRowBytes;          // 32 KiB: one operand, one k-tile
  constexpr int B_BASE = kTwoGroupB;            // LDS: [A0 A1 | B0 B1 B2]
  constexpr int kCopies = SLAB / (256 * 16);    // 16-byte copies per thread per slab
  constexpr int kCopiesA = BM * kRowBytes / (256 * 16);
  constexpr int kRowBT = kRole == kGated ? 256 : 512;  // bytes of a k row in B's slab
  static_assert(BK % Atom::kK == 0 && kCopies == 8, "k-tile geometry");
  static_assert(!kShift || (kSub == 1 && kStepBytes == 32), "a dword follows every fragment");
  static_assert((1 << Slab<kRowBytes>::kRowShift) * kChunks <= 32,
                "the swizzle repeats within 32 rows");
  static_assert(SLAB == kTwoGroupSlab && kTwoGroupLds <= 160 * 1024, "LDS budget");
  static_assert(!kHalf || kForm != kGrad, "blocks of rows");
  static_assert(!kBT || EB == 2, "slabs of k rows: 16-bit operands");

  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int grp = wave >> 2;                    // 0: waves 0-3, 1: waves 4-7
  const int t = tid & 255;                      // thread index inside the group
  const int e = ts.e, m0 = ts.m0, m_end = ts.m_end, n0 = ts.n0, K = ts.K;
  const uint8_t *A = ts.A, *B = ts.B;
  const bool sum_a = ts.sum_a, sum_b = ts.sum_b;
  const int wm0 = kHalf ? WM * (wave & 1) : 128 * grp + WM * (wave & 1);
  const int wn0 = WN * (kHalf ? 2 * grp + ((wave >> 1) & 1) : ((wave >> 1) & 1));
  // kGated: the first half of B's slab is the gate's columns n0 .., the other
  // half the same columns of the up projection; a wave's first FN / 2 MFMA tiles
  // are the gate's, so a lane holds both sums of an element
  constexpr bool kTwo = kRole == kGated;
  constexpr int FH = FN / 2;
  const int wb0 = kTwo ? wn0 / 2 : wn0;         // the wave's first column
  const bool busy = kForm == kGrad || m0 + wm0 < m_end;  // a wave without a row multiplies nothing
  const int KT = (K + BK - 1) / BK;
  const int KTf = K / BK;  // whole k-tiles; tile KTf, if K ends inside it, is ragged

  // ---- copies: group 0 moves A (two LDS slots), group 1 moves B (three
  // slots), 8 instructions per slab.  Thread t fills slot byte 16 (t + 256q)
  // (lane-linear), i.e. row r0 + 32q, physical chunk t % 8, and fetches the
  // logical chunk the swizzle puts there; rows 32q.. of the tile start the
  // buffer resource of copy q, whose record count ends at the last real row.
  const int r0 = t / kChunks;
  const int64_t rb = (grp == 0 ? p.lda : p.ldb) * EB;   // row pitch in bytes
  const uint8_t* op = (grp == 0 ? A + m0 * rb : B + n0 * rb);  // the tile's first row
  const int rows_left = (grp == 0 ? m_end - m0 : p.N - n0); // real rows from there on
  uint32_t voff = (uint32_t)(r0 * rb + Swz::chunk(r0, t % kChunks) * 16);
  const int lds_op = grp == 0 ? 0 : B_BASE;
  int recs[kCopies];
  const uint32_t off = kShift ? (uint32_t)(uintptr_t)op & 3u : 0u;
  static_for<kCopies>([&](auto q) {
    // up to the dword that holds the last row's last byte
    const int n = min(rows_left - 32 * (kTwo && grp ? (int)q % 4 : (int)q), 32);
    recs[q] = n > 0 ? (int)((uint32_t)((n - 1) * rb + (int64_t)K * EB + off + 3) & ~3u) : 0;
  });
  // per group: the byte step of a k-tile, and (N-contiguous B) of a copy
  uint32_t kt_bytes = kUsed, q_bytes = 0;
  const uint8_t* qbase = op;
  if constexpr (kShift) {
    // every row from the dword that holds its first byte; the window's last
    // chunk is never read
    qbase = op - off;
    const int c = Swz::chunk(r0, t % kChunks);
    voff = c == 7 ? 0x80000000u : (uint32_t)((off + (uint32_t)(r0 * rb)) & ~3u) + c * 16;
  }
  // a k-rows operand of `lines` columns: up to its last element's dword
  auto k_rows_bytes = [&](int64_t ld, int lines) {
    return K > 0 ? (int)min((((K - 1) * ld + lines) * EB + 3) & ~(int64_t)3, (int64_t)0x7FFFFFFC) : 0;
  };
  int64_t q_stride = 32 * rb;
  if constexpr (kBT && kTwo) {
    if (grp == 1) {
      // each half slab 64 rows of k x 128 columns: chunk t + 256 (q % 4) of the
      // half is row t / 16 (+ 16 (q % 4)), stored chunk t % 16
      const int rt = t >> 4;
      const int n = min(n0 + 8 * ((t & 15) ^ (4 * (rt & 3))), (p.N - 1) & ~7);
      voff = (uint32_t)((rt * p.ldb + n) * EB);
      kt_bytes = (uint32_t)(BK * p.ldb * EB);
      q_bytes = (uint32_t)(16 * p.ldb * EB);
      qbase = B;
      q_stride = 0;
      const int whole = k_rows_bytes(p.ldb, p.N);
      static_for<kCopies>([&](auto q) { recs[q] = whole; });
    }
  } else if constexpr (kBT) {
    if (grp == 1) {
      // slab chunk t + 256 q: row r0 = t / 32 (+ 8 q), stored chunk t % 32
      // holding columns n0 + 8 ((t % 32) ^ 4 (r0 % 4)) .. + 7
      const int64_t ldb = p.ldb;
      const int rt = t >> 5;
      const int n = min(n0 + 8 * ((t & 31) ^ (4 * (rt & 3))), (p.N - 1) & ~7);
      voff = (uint32_t)((rt * ldb + n) * EB);
      kt_bytes = (uint32_t)(BK * ldb * EB);
      q_bytes = (uint32_t)(8 * ldb * EB);
      qbase = B;
      q_stride = 0;
      const int whole = k_rows_bytes(ldb, p.N);
      static_for<kCopies>([&](auto q) { recs[q] = whole; });
    }
  }
  if constexpr (kAT) {
    if (grp == 0) {
      // the same for an M-contiguous A (column-major M x K, pitch lda):
      // row rt (+ 8 q) of k, stored chunk t % 32 holding columns
      // m0 + 8 ((t % 32) ^ 4 (rt % 4)) .. + 7, clamped to M's last chunk
      // (whose columns past M feed nothing that is stored)
      const int64_t lda = p.lda;
      const int rt = t >> 5;
      const int m = min(m0 + 8 * ((t & 31) ^ (4 * (rt & 3))), (p.M - 1) & ~7);
      voff = (uint32_t)((rt * lda + m) * EB);
      kt_bytes = (uint32_t)(BK * lda * EB);
      q_bytes = (uint32_t)(8 * lda * EB);
      qbase = A;
      q_stride = 0;
      const int whole = k_rows_bytes(lda, p.M);
      static_for<kCopies>([&](auto q) { recs[q] = whole; });
    }
  }
  // The ragged last k-tile: a lane whose K-contiguous chunk lies past K reads
  // from past every record, so the range check returns zeros (the chunk that
  // crosses K: clear_tail); the rows past K of a k-rows slab (an M- or
  // N-contiguous operand) are past its records already.
  uint32_t voff_tail = voff;
  if (!kShift && ((grp == 0 && !kAT) || (grp == 1 && !kBT))) {
    if (Swz::chunk(r0, t % kChunks) * 16 >= (K - KTf * BK) * EB) voff_tail = 0x80000000u;
  }
  // Copy q of k-tile kt into `slot`.  A copy past the last k-tile still runs
  // (so the instruction stream and the wait counts never change) but with no
  // records: it writes zeros into a slot nobody reads any more.
  // kTwo: copies 4 .. 7 of B are the up projection's, `up_by` bytes from the gate's
  const int64_t up_by = kTwo && grp ? ts.B2 - ts.B : 0;
  auto copy_one = [&](int kt, int slot, bool live, auto q) {
    const int qq = kTwo && grp ? (int)q % 4 : (int)q;
    const uint8_t* base = qbase + (int64_t)qq * q_stride;
    if constexpr (kTwo && q >= 4) base += up_by;
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
        (void*)base, 0, __builtin_amdgcn_readfirstlane(recs[q] & -(int)live), 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        r, (__attribute__((address_space(3))) void*)(smem + lds_op + slot * SLAB + q * 4096 +
                                                     (wave & 3) * 1024),
        16, kt == KTf ? voff_tail : voff, (uint32_t)kt * kt_bytes + (uint32_t)qq * q_bytes, 0, 0);
  };
  auto copy_slab = [&](int kt, int slot, bool live, auto n) {
    static_for<n>([&](auto q) { copy_one(kt, slot, live, q); });
  };
  using CopiesA = std::integral_constant<int, kCopiesA>;
  using CopiesB = std::integral_constant<int, kCopies>;

  // ---- fragments: one base register per k-step; the A slot and the 32-row
  // fragment are immediates, the B slot (three of them: immediates would
  // pass 64 KiB) is added into the B bases as they move from slot to slot.
  // A 32-byte (e4m3) fragment is logical chunks 2u, 2u+1 of the row: the
  // swizzle XORs the chunk index, so the second chunk sits at the first
  // one's address XOR 16 (every other term of the address is a multiple of
  // 128), formed in the loop rather than held.
  // kBlocks: lane l holds chunks l / 16 and l / 16 + 4 (XOR 64).  A 16-byte LDS read
  // takes lanes 0 .. 3, 12 .. 15 and 20 .. 27 at a time, rows 4 .. 11 of them
  // sixteen lanes on: with chunks 2 (l / 16) and the next one these hit the banks
  // of the others' (bank conflicts 46 % of the LDS's cycles), with neighbours they
  // do not.  Both operands share the order, so the sums are the same.
  static_assert(kSub == 1 || (Atom::kLaneBytes == 32 && kStepBytes % 32 == 0), "chunk pairs");
  uint32_t fa[kAT ? 1 : KSTEPS], fb[kBT ? 1 : KSTEPS];
  static_for<KSTEPS>([&](auto ks) {
    const int c = kBlocks ? lane / FR : (ks * kStepBytes + lane / FR * Atom::kLaneBytes) / 16;
    const int ra = wm0 + lane % FR, rbw = wb0 + lane % FR;
    if constexpr (!kAT) fa[ks] = (uint32_t)(ra * kRowBytes + Swz::chunk(ra, c) * 16);
    if constexpr (!kBT)
      fb[ks] = (uint32_t)(B_BASE + rbw * kRowBytes + Swz::chunk(rbw, c) * 16);  // B slot 0
  });
  // kShift: the dword after a fragment's sixteen bytes begins the next logical
  // chunk, c + 1 for c = 2 ks + lane / 32, which sits at the fragment's address
  // XOR 16 (c ^ (c + 1)); each lane's byte shift (rows 32 apart share it)
  uint32_t next02 = 0, next1 = 0, sh_a = 0, sh_b = 0;
  if constexpr (kShift) {
    next02 = lane < 32 ? 16 : 48;
    next1 = lane < 32 ? 16 : 112;
    sh_a = ((uint32_t)(uintptr_t)A +
            (uint32_t)(m0 + wm0 + (lane & 31)) * (uint32_t)(p.lda * EB)) & 3u;
    sh_b = ((uint32_t)(uintptr_t)B +
            (uint32_t)(n0 + wn0 + (lane & 31)) * (uint32_t)(p.ldb * EB)) & 3u;
  }
  if constexpr (kAT) {
    // as for an N-contiguous B below, with rows m = wm0 + ... of A slot 0
    // (wm0 is a multiple of 64, so fragment i is again XOR 64 i)
    const int qw = lane >> 4, a4 = lane & 15;
    const int k = 8 * (qw >> 1) + (a4 >> 2);
    const int m = wm0 + 16 * (qw & 1) + 4 * (a4 & 3);
    fa[0] = (uint32_t)(k * 512 + (((m >> 3) ^ (4 * (k & 3))) * 16) + (m & 7) * 2);
  }
  if constexpr (kBT) {
    // transpose read h of k-step ks for lane a of quarter-wave qw: row
    // k = 16 ks + 8 (qw / 2) + 4 h + a / 4, columns n = wn0 + 16 (qw % 2) +
    // 4 (a % 4) of the first 32-column fragment, stored chunk
    // (n / 8) ^ 4 (k % 4).  k % 4 = a / 4 whatever ks and h, so one base
    // (ks = h = 0) serves all: + 8192 ks + 2048 h, and XOR 64 j for
    // fragment j
    const int qw = lane >> 4, a4 = lane & 15;
    // (kTwo: rows of 128 columns, so + 4096 ks + 1024 h)
    const int k = 8 * (qw >> 1) + (a4 >> 2);
    const int n = wb0 + 16 * (qw & 1) + 4 * (a4 & 3);
    fb[0] = (uint32_t)(B_BASE + k * kRowBT + (((n >> 3) ^ (4 * (k & 3))) * 16) + (n & 7) * 2);
  }
  // kBlocks: six of B's fragments at a time, the others read between the MFMAs: 256
  // registers do not hold the sums, both operands and the partial sums (four at a
  // time: 477 us for 8192^3 instead of 456)
  constexpr int FB = kBlocks && FN > 6 ? 6 : FN;
  Frag a[KSTEPS][FM], b[KSTEPS][FB];
  uint32_t xa[kShift ? KSTEPS : 1][FM], xb[kShift ? KSTEPS : 1][FN];
  auto lds_frag = [&](uint32_t base, int imm) -> Frag {
    if constexpr (kSub == 1) {
      return *(const i32x4*)(smem + base + imm);
    } else {
      uint32_t base_hi = base ^ (kBlocks ? 64u : 16u);
      asm volatile("" : "+v"(base_hi));  // keep the XOR in the loop
      const i32x4 lo = *(const i32x4*)(smem + base + imm);
      const i32x4 hi = *(const i32x4*)(smem + base_hi + imm);
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  };
  // k-tile kt: A slot kt % 2 (immediate), B slot kt % 3 (in fb); afterwards
  // fb moves on to B slot (kt + 1) % 3
  auto lds_frag_t = [&](uint32_t addr, auto row_bytes) -> Frag {
    typedef int s32x2 __attribute__((ext_vector_type(2)));
    const s16x4 lo = ds_read_tr16(smem + addr);
    const s16x4 hi = ds_read_tr16(smem + addr + 4 * row_bytes);
    const s32x2 l2 = __builtin_bit_cast(s32x2, lo), h2 = __builtin_bit_cast(s32x2, hi);
    return Frag{l2[0], l2[1], h2[0], h2[1]};
  };
  auto read_frag = [&](int kt, auto r) {
    constexpr int ks = r / (FM + FN), f = r % (FM + FN);
    // B's MFMA tile: its place among the wave's columns, and the half slab
    constexpr int j = kTwo ? (f - FM) % FH : f - FM, up = kTwo && f - FM >= FH ? SLAB / 2 : 0;
    if constexpr (f < FM && kAT)
      a[ks][f] = lds_frag_t((fa[0] ^ (64u * f)) + 8192 * ks + (kt & 1) * SLAB,
                            std::integral_constant<int, 512>{});
    else if constexpr (f < FM)
      a[ks][f] = lds_frag(fa[ks], (kt & 1) * SLAB + f * FR * kRowBytes);
    else if constexpr (kBT)
      b[ks][f - FM] = lds_frag_t((fb[0] ^ (64u * j)) + 16 * kRowBT * ks + up,
                                 std::integral_constant<int, kRowBT>{});
    else
      b[ks][(f - FM) % FB] = lds_frag(fb[ks], j * FR * kRowBytes + up);
    if constexpr (kShift) {
      uint32_t base = (f < FM ? fa[ks] : fb[ks]) ^ (ks == 1 ? next1 : next02);
#if defined(__HIP_DEVICE_COMPILE__)
      asm volatile("" : "+v"(base));  // keep the XOR in the loop
#endif
      if constexpr (f < FM)
        xa[ks][f] = *(const uint32_t*)(smem + base + (kt & 1) * SLAB + f * 32 * kRowBytes);
      else
        xb[ks][f - FM] = *(const uint32_t*)(smem + base + (f - FM) * 32 * kRowBytes);
    }
  };
  // kShift: the fragments' bytes moved into place
  auto place = [&]() {
    if constexpr (kShift) {
      auto shift = [](Frag& w, uint32_t x, uint32_t sh) {
        const uint32_t w0 = w[0], w1 = w[1], w2 = w[2], w3 = w[3];
        w[0] = (int)__builtin_amdgcn_alignbyte(w1, w0, sh);
        w[1] = (int)__builtin_amdgcn_alignbyte(w2, w1, sh);
        w[2] = (int)__builtin_amdgcn_alignbyte(w3, w2, sh);
        w[3] = (int)__builtin_amdgcn_alignbyte(x, w3, sh);
      };
      static_for<KSTEPS>([&](auto ks) {
        static_for<FM>([&](auto i) { shift(a[ks][i], xa[ks][i], sh_a); });
        static_for<FN>([&](auto j) { shift(b[ks][j], xb[ks][j], sh_b); });
      });
    }
  };
  // Clears what a last k-tile that ends inside a chunk holds past K (the next
  // row's bytes), a thread a row of its group's slab, before anyone reads it.
  const bool ragged = kForm != kGrad && KTf < KT && (kShift || K * EB % 16 != 0);
  auto clear_tail = [&]() {
    const int kt = KT - 1, slot = grp == 0 ? (kt & 1) : kt % 3;
    if ((kHalf && grp == 0 && t >= BM) || (kBT && grp == 1)) return;
    uint8_t* row = smem + lds_op + slot * SLAB + t * kRowBytes;
    const uint32_t sh =
        kShift ? ((uint32_t)(uintptr_t)op + (uint32_t)t * (uint32_t)rb) & 3u : 0u;
    const int first = (int)sh + K * EB - KTf * kUsed;  // of the window's bytes, the first past K
    const int end = kShift ? 28 : (first + 15) / 16 * 4;
    for (int d = first >> 2; d < end; ++d) {
      uint32_t* w = (uint32_t*)(row + Swz::chunk(t, d >> 2) * 16 + (d & 3) * 4);
      *w = d == first >> 2 ? *w & ((1u << (8 * (first & 3))) - 1u) : 0u;
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup");
  };
  auto advance_b = [&](int kt) {
    const int step = (kt % 3 == 2) ? -2 * SLAB : SLAB;
    static_for<kBT ? 1 : KSTEPS>([&](auto ks) { fb[ks] += step; });
  };
  // A memory phase: read k-tile kt's fragments and copy k-tile ct into
  // `slot`.  Under load the copy path accepts a direct-to-LDS copy only every
  // few dozen cycles, and a wave issues in order, so the copies go out
  // between the LDS reads (kReads / kCopies fragments after each copy, the
  // remainder spread over the first copies): the TA and the LDS then work
  // side by side instead of one after the other.  Measured in the ungrouped
  // kernel per k-tile of 256 x 256 x 128 bytes: 2508 cycles interleaved against 2590 with the
  // copies after the reads (16-bit), 3728 against 3952 (reads first) and
  // 4276 (copies first) for e4m3.
  constexpr int kReads = KSTEPS * (FM + FB);  // fragments per k-tile
  // LDS read instructions of fragments [first, first + n)
  auto read_insts = [](int first, int n) constexpr {
    int c = 0;
    for (int r = first; r < first + n; ++r)
      c += kShift ? 2 : (r % (FM + FN) < FM) ? (kAT ? 2 : kSub) : (kBT ? 2 : kSub);
    return c;
  };
  BlockSums<kBlocks ? FM : 1, kBlocks ? FN : 1, kTwo> block_sums;
  typename Atom::Acc plain_sums[kBlocks ? 1 : FM][kBlocks ? 1 : FN];
  auto& acc = [&]() -> auto& {
    if constexpr (kBlocks) return block_sums.acc;
    else return plain_sums;
  }();
  static_for<FM>([&](auto i) { static_for<FN>([&](auto j) { acc[i][j] = typename Atom::Acc{}; }); });
  // kBlocks: the scales of a block of k.  Lane l asks for row wm0 + l's and, by
  // its parity, for the gate's (or only) and the up projection's of the wave's
  // columns, a period before they are used: two loads in front of the period's
  // copies, so a wait for earlier copies leaves them in flight.
  constexpr int kScaleLoads = kBlocks ? 2 : 0;
  const float *sa_at = nullptr, *sb_at = nullptr;
  float raw_a = 0.f, raw_b = 0.f, scale[2][FM];
  if constexpr (kBlocks) {
    sa_at = p.sa + (int64_t)min(m0 + wm0 + lane, m_end - 1) * p.sa_row;
    // (per_lane: the waits for copies count both loads)
    sb_at = (kTwo && (lane & 1) ? p.sb2 : p.sb) +
            per_lane((int64_t)e * p.stride_sb + (int64_t)(min(n0 + wb0, p.N - 1) >> 7) * p.sb_col);
  }
  if constexpr (kBlocks) {
    // the first k-tile finds nothing to finish
    static_for<block_sums.kAhead>([&](auto x) { block_sums.part[x] = f32x4{0.f, 0.f, 0.f, 0.f}; });
    static_for<FM>([&](auto i) { scale[0][i] = scale[1][i] = 0.f; });
  }
  auto ask_scales = [&](int kt) {
    if constexpr (kBlocks) {
      const int k = min(kt, KT - 1);
      raw_a = sa_at[(int64_t)k * p.sa_kb];
      raw_b = sb_at[(int64_t)k * p.sb_kb];
    }
  };
  // the scales of this lane's rows, 16 i + l % 16, from those that lanes 16 i + l %
  // 16 asked for: sixteen lanes' values spread over the others by swaps of halves
  auto place_scales = [&]() {
    static_assert(!kBlocks || FM == 4, "sixteen lanes a tile");
    if constexpr (kBlocks) {
      static_for<kTwo ? 2 : 1>([&](auto h) {
        const uint32_t s = __builtin_bit_cast(
            uint32_t, raw_a * __builtin_bit_cast(float, __builtin_amdgcn_readlane(
                                                            __builtin_bit_cast(int, raw_b), h)));
        typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
        const u32x2 half = __builtin_amdgcn_permlane32_swap(s, s, false, false);
        static_for<2>([&](auto x) {
          const uint32_t two = half[(int)x];
          const u32x2 row = __builtin_amdgcn_permlane16_swap(two, two, false, false);
          const uint32_t first = row[0], second = row[1];
          scale[h][2 * x] = __builtin_bit_cast(float, first);
          scale[h][2 * x + 1] = __builtin_bit_cast(float, second);
        });
      });
    }
  };
  auto memory_phase = [&](int kt, int ct, int slot, bool live, auto copies) {
    constexpr int kPer = kReads / copies, kRem = kReads % copies;
    if constexpr (kBlocks) {
      // (the k-tile before's last sums, under the other group's MFMAs)
      __builtin_amdgcn_sched_barrier(0);
      block_sums.finish(scale);
      place_scales();
      ask_scales(kt + 1);
    }
    __builtin_amdgcn_sched_barrier(0);
    static_for<copies>([&](auto q) {
      copy_one(ct, slot, live, q);
      constexpr int first = kPer * q + (q < kRem ? q : kRem);
      constexpr int n = kPer + (q < kRem ? 1 : 0);
      static_for<n>([&](auto u) { read_frag(kt, std::integral_constant<int, first + u>{}); });
    });
    static_for<copies>([&](auto q) {
      constexpr int first = kPer * q + (q < kRem ? q : kRem);
      constexpr int n = kPer + (q < kRem ? 1 : 0);
      __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
      __builtin_amdgcn_sched_group_barrier(0x100, read_insts(first, n), 0);
    });
    place();
    if constexpr (!kBlocks) advance_b(kt);
    __builtin_amdgcn_sched_barrier(0);
  };
  LineSums<kCode, FN> sums;
  if constexpr (kForm == kGrad) sums.init();
  // one k-tile of MFMAs, fenced off from the scheduler on both sides so that
  // no wait or memory instruction of a neighbouring phase moves into it
  auto compute = [&](int kt) {
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (kBlocks) {
      // (also without a row: a branch would join the partial sums by moves, which
      // wait for them)
      block_sums.mma(a[0], b[0], scale, [&](auto j) {
        read_frag(kt, std::integral_constant<int, FM + j + FB>{});
      });
      advance_b(kt);
    } else if (busy) {
      static_for<KSTEPS * FM * FN>([&](auto idx) {
        constexpr int ks = idx / (FM * FN), i = (idx / FN) % FM, j = idx % FN;
        Atom::mma(acc[i][j], b[ks][j], a[ks][i]);
      });
    }
    if constexpr (kForm == kGrad) {
      static_for<KSTEPS>([&](auto ks) {
        if (sum_b) static_for<FN>([&](auto j) { sums.template add<j>(b[ks][j]); });
        if (sum_a) static_for<FM>([&](auto i) { sums.template add<i>(a[ks][i]); });
      });
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // keeps the MFMAs in front of a conditional barrier
  auto pin = [&]() {
#if defined(__HIP_DEVICE_COMPILE__)  // a type of the template: the host pass has no such register
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) asm volatile("" ::"v"(acc[i][j]));
    if constexpr (kBlocks) block_sums.pin();
#endif
  };
  auto wait_lgkmcnt0 = [&]() { __builtin_amdgcn_s_waitcnt(0xC07F); };
  auto barrier = [&]() {
    __builtin_amdgcn_sched_barrier(0);
    stage_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };

  // Each group runs its own program with exactly one MFMA sequence; copies
  // are issued only between LDS reads.  Period kt ends at barrier 2kt+1:
  //   group 0: read k-tile kt's fragments and copy A of kt+1 into A slot
  //     (kt+1)%2 (it held kt-1, read by both groups in period kt-1), then
  //     multiply kt and wait for its copies;
  //   group 1: multiply kt-1 (fragments read in period kt-1), then read
  //     kt's fragments and copy B of kt+2 into B slot (kt+2)%3 (it held
  //     kt-1), then wait for B of kt+1 (copied in period kt-1); in period
  //     0 it only reads.
  // Every slab is thus complete one barrier before its first reader.  A
  // second barrier splits each period between its halves: group 0 reads
  // while group 1 multiplies, then the other way round.  An MFMA holds its
  // wave's issue for its whole run, so without the split group 0 starts
  // multiplying before group 1 is done, both share the matrix core and the
  // period grows (the ungrouped kernel, 16-bit: 3084 cycles per k-tile against 2508; the e4m3
  // 8192^3 GEMM with GELU: 440 us with one barrier per period, 396 us with
  // two).
  //
  // Group 1's second barrier is skipped after the last k-tile, and the
  // compiler is free to sink the MFMAs, plain register arithmetic, past
  // such a conditional barrier into the next period (it does so for e4m3,
  // which then measured 3664 cycles per k-tile): an empty asm reading every
  // accumulator keeps them in front of it.
  // The columns' bias and scales come into the cache under the loop: a byte of
  // each is asked for here and waited for with the first slabs, so that no
  // epilogue pass begins with a trip to memory.
  [[maybe_unused]] uint32_t warm = 0;
  if constexpr (kForm != kGrad) {
    const int64_t at = (int64_t)e * p.N + min(n0 + wb0 + 2 * lane, p.N - 1);
    if (p.bias) warm = p.bias[at * type_bytes(p.bias_type)];
    if constexpr (kTwo) {
      if (p.bias2) warm += p.bias2[at * type_bytes(p.bias_type)];
    }
    if constexpr (EB == 1 && !kBlocks) {
      if (p.sb) warm += *(const uint8_t*)(p.sb + at);
    }
  }
  auto warmed = [&]() {
#if defined(__HIP_DEVICE_COMPILE__)
    if constexpr (kForm != kGrad) asm volatile("" ::"v"(warm));
#endif
  };
  if (KT > 0) {
    if (grp == 0) {
      ask_scales(0);
      copy_slab(0, 0, true, CopiesA{});
      wait_vmcnt<0>();
      warmed();
      barrier();
      for (int kt = 0; kt < KT; ++kt) {
        if constexpr (kForm != kGrad) {
          if (ragged && kt + 1 == KT) {
            clear_tail();
            barrier();
          }
        }
        memory_phase(kt, kt + 1, (kt + 1) & 1, kt + 1 < KT, CopiesA{});
        wait_lgkmcnt0();
        barrier();
        compute(kt);
        if constexpr (kForm != kGrad) pin();
        wait_vmcnt<0>();                             // A of kt+1 landed
        barrier();
      }
    } else {
      ask_scales(0);
      copy_slab(0, 0, true, CopiesB{});
      copy_slab(1, 1, KT > 1, CopiesB{});
      wait_vmcnt<kCopies>();
      warmed();
      barrier();
      if constexpr (kForm != kGrad) {
        if (ragged && KT == 1) {
          clear_tail();
          barrier();
        }
      }
      barrier();
      // one iteration reads k-tile kt (end of period kt) and multiplies it
      // (start of period kt+1): the fragments never live across iterations
      for (int kt = 0; kt < KT; ++kt) {
        memory_phase(kt, kt + 2, (kt + 2) % 3, kt + 2 < KT, CopiesB{});
        wait_lgkmcnt0();
        if (kt + 1 < KT) wait_vmcnt<kCopies + kScaleLoads>();  // B of kt+1 landed
        else wait_vmcnt<0>();  // behind this barrier no copy, record-less or not, lands in a region
        barrier();
        if constexpr (kForm != kGrad) {
          // while group 0 clears the last k-tile's A, before it reads it
          if (ragged && kt + 2 == KT) {
            clear_tail();
            barrier();
          }
        }
        compute(kt);
        pin();
        if (kt + 1 < KT) barrier();
      }
    }
    if constexpr (kBlocks) block_sums.finish(scale);
  }
  // The epilogue's regions lie where nothing is read or copied any more: group 0
  // starts while group 1 still multiplies the last k-tile, a wave of group 1 while
  // the group's others do.
  constexpr bool kLate = FB < FN;  // fragments of B are read between the MFMAs
  static_assert(!kLate || 2 * WM * WN * 2 <= SLAB, "two regions in a B slot");
  uint8_t* region = smem + two_group_region(wave, WM * WN * 2, kLate, KT);
  if constexpr (kForm == kGrad) {
    if (sum_b) sums.template write<FN>(p.dbias + (int64_t)e * p.N, n0 + wn0, p.N, lane);
    if (sum_a) sums.template write<FM>(p.dbias + (int64_t)e * p.M, m0 + wm0, p.M, lane);
  }
  if constexpr (kForm == kGrad)
    wgrad_epilogue<FM, FN>(p, e, m0 + wm0, n0 + wn0, lane, acc, region);
  else if constexpr (kRole == kGateGrad) {
    GateParts<WM, WN> z;
    z.ask(p, m_end, m0 + wm0, n0 + wn0, lane, 0);
    grad_epilogue<kCode, kAct>(p, m_end, m0 + wm0, n0 + wn0, lane, acc, z, region);
  } else if constexpr (kRole != kPlain || kBlocks)
    role_epilogue<kCode, kRole, kAct, FR, WM, kTwo ? WN / 2 : WN>(p, e, m_end, m0 + wm0, n0 + wb0, lane,
                                                                 acc, region);
  else
    grouped_epilogue<kCode, FM, FN>(p, e, m_end, m0 + wm0, n0 + wn0, lane, acc, region);
}

// Which blocks of rows a workgroup may get.  Experts are cut into blocks of
// 256 rows and, where at most 128 are left, a half block.  The whole tiles come
// first; when the last round of them would not fill the card's compute units,
// they are split into halves if the halves then end sooner (a half tile takes
// about 0.55 of a whole one's time).  p.flags & kOpHalves: half blocks only.
// As in row_tile, a segment's tiles go to the XCDs in contiguous runs, four
// blocks of rows at a time.
struct HalfTile {
  int e, r0, r1, tn;
  bool half;
};
__device__ __forceinline__ bool two_group_lookup(const GroupedParams& p, int bid, HalfTile& t) {
  constexpr int kUnits = 256;  // compute units of the card, one workgroup on each
  const int lane = threadIdx.x & 63;
  const bool halves = p.flags & kOpHalves;
  auto count = [&](int e, int& full, int& half) {
    full = half = 0;
    if (e >= p.groups) return;
    int lo, hi;
    expert_rows(p, e, lo, hi);
    const int rows = hi - lo, rest = rows & 255;
    full = halves ? 0 : (rows >> 8) + (rest > 128);
    half = halves ? (rows >> 7) + ((rows & 127) > 0) : rest > 0 && rest <= 128;
  };
  int tf = 0, th = 0, fi = 0, hi_ = 0, f, h;
  for (int g0 = 0; g0 < p.groups; g0 += 64) {
    count(g0 + lane, f, h);
    fi = wave_scan(f, lane);
    hi_ = wave_scan(h, lane);
    tf += __builtin_amdgcn_readlane(fi, 63);
    th += __builtin_amdgcn_readlane(hi_, 63);
  }
  const int64_t n_full = (int64_t)tf * p.tiles_n, n_half = (int64_t)th * p.tiles_n;
  const int over = (int)(n_full % kUnits);
  int split = 0;
  if (over) {
    auto half_rounds = [](int64_t n) { return 0.55f * (float)((n + kUnits - 1) / kUnits); };
    const int64_t room = kUnits - over;
    const float whole = 1.f + half_rounds(n_half > room ? n_half - room : 0);
    if (half_rounds(2 * over + n_half) < whole) split = over;
  }
  const int64_t whole_tiles = n_full - split, half_tiles = 2 * (int64_t)split + n_half;
  const bool in_full = bid < whole_tiles;
  if (!in_full && bid - whole_tiles >= half_tiles) return false;
  const int n = (int)(in_full ? whole_tiles : half_tiles);
  const int at = (int)(in_full ? bid : bid - whole_tiles);
  const int per = n / 8, rest = n % 8, xcd = at & 7;
  int id = xcd * per + min(xcd, rest) + (at >> 3);
  int part = 0;
  bool of_full = in_full;
  if (!in_full) {
    if (id < 2 * split) {
      of_full = true;
      part = id & 1;
      id = (int)whole_tiles + (id >> 1);
    } else {
      id -= 2 * split;
    }
  }
  const int total = of_full ? tf : th;
  const int per_group = 4 * p.tiles_n, first = (id / per_group) * 4;
  const int gm = min(total - first, 4), in = id % per_group;
  const int block = first + in % gm;
  t.tn = in / gm;
  t.half = !in_full;
  int before = 0;
  for (int g0 = 0; g0 < p.groups; g0 += 64) {
    if (p.groups > 64) {
      count(g0 + lane, f, h);
      fi = wave_scan(f, lane);
      hi_ = wave_scan(h, lane);
    }
    const int incl = of_full ? fi : hi_;
    const uint64_t mask = __ballot(block < before + incl);
    if (mask) {
      const int l = __builtin_ctzll(mask);
      const int excl = l ? __builtin_amdgcn_readlane(incl, l - 1) : 0;
      t.e = g0 + l;
      int lo, hi, ef, eh;
      expert_rows(p, t.e, lo, hi);
      count(t.e, ef, eh);
      const int local = block - before - excl;
      const int r0 = of_full ? lo + local * 256 + part * 128 : lo + ef * 256 + local * 128;
      t.r0 = __builtin_amdgcn_readfirstlane(r0);
      t.r1 = __builtin_amdgcn_readfirstlane(hi);
      lo = __builtin_amdgcn_readfirstlane(lo);
      // (wrong offsets could have overflowed the sums)
      return t.r0 >= lo && t.r0 < t.r1 && (unsigned)t.tn < (unsigned)p.tiles_n;
    }
    before += __builtin_amdgcn_readlane(incl, 63);
  }
  return false;
}

template <int kCode, int kForm, int kRole = kPlain, int kAct = 0>
__global__ __launch_bounds__(512) void grouped_two_group_kernel(const GroupedParams p) {
  constexpr int EB = type_bytes(kCode);
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kTwoGroupLds];
  TileSpan ts{};
  if constexpr (kForm == kGrad) {
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), grp = wave >> 2;
    int tm, tn, lo, hi;
    wgrad_tile(p, blockIdx.x, gridDim.x, ts.e, tm, tn);
    expert_rows(p, ts.e, lo, hi);
    ts.sum_a = p.dbias && (p.flags & kOpSumA) && tn == 0 && !((wave >> 1) & 1);
    ts.sum_b = p.dbias && !(p.flags & kOpSumA) && tm == 0 && grp == 0 && !(wave & 1);
    ts.m0 = tm * 256;
    ts.m_end = p.M;
    ts.n0 = tn * 256;
    ts.K = hi - lo;
    ts.A = p.A + (int64_t)lo * p.lda * EB;
    ts.B = p.B + (int64_t)lo * p.ldb * EB;
    two_group_tile<kCode, kForm, false, kRole, kAct>(p, ts, smem);
  } else {
    HalfTile t;
    if (!two_group_lookup(p, blockIdx.x, t)) return;
    // scalars for certain: copies whose buffer lies in vector registers loop
    ts.e = __builtin_amdgcn_readfirstlane(t.e);
    ts.m0 = __builtin_amdgcn_readfirstlane(t.r0);
    ts.m_end = __builtin_amdgcn_readfirstlane(t.r1);
    ts.n0 = __builtin_amdgcn_readfirstlane(t.tn) * (kRole == kGated ? 128 : 256);
    ts.K = p.K;
    ts.A = p.A;
    ts.B = p.B + (int64_t)ts.e * p.stride_b * EB;
    if constexpr (kRole == kGated) ts.B2 = p.B2 + (int64_t)ts.e * p.stride_b * EB;
    if (t.half) two_group_tile<kCode, kForm, true, kRole, kAct>(p, ts, smem);
    else two_group_tile<kCode, kForm, false, kRole, kAct>(p, ts, smem);
  }
}

template <int kCode, int kForm, int kRole = kPlain, int kAct = 0>
int launch(const GroupedParams& p0, hipStream_t stream) {
  GroupedParams p = p0;
  p.tiles_n = kRole == kGated ? (p.N + 127) / 128 : (p.N + 255) / 256;
  p.tiles_m = (p.M + 255) / 256;
  // a split round adds fewer than 256 tiles
  const int64_t grid =
      kForm == kGrad ? (int64_t)p.groups * p.tiles_m * p.tiles_n
      : p.flags & kOpHalves ? row_tiles_bound(p.rows, p.groups, 128) * p.tiles_n
                            : row_tiles_bound(p.rows, p.groups, 256) * p.tiles_n + 256;
  if (grid <= 0) return TLA_OK;
  if (!grid_fits(grid, 512)) return TLA_ERR_UNSUPPORTED;
  hipLaunchKernelGGL((grouped_two_group_kernel<kCode, kForm, kRole, kAct>), dim3((unsigned)grid), dim3(512), 0,
                     stream, p);
  return hipGetLastError() == hipSuccess ? TLA_OK : TLA_ERR_HIP;
}

// The kernel of the problem's activation
template <int kCode, int kForm, int kRole>
int launch_act(const GroupedParams& p, hipStream_t s) {
  if (p.act == TLA_ACT_SILU) return launch<kCode, kForm, kRole, kSiluAct>(p, s);
  if (p.act == TLA_ACT_GELU) return launch<kCode, kForm, kRole, kGeluAct>(p, s);
  return launch<kCode, kForm, kRole, kLinear>(p, s);
}

}  // namespace
}  // namespace tla
