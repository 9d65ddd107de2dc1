// operators.hpp -- internal launch interface of the expert-grouped and 8-bit
// integer products and of the token quantizer (declarations and contracts:
// include/tla.h).  Every function assumes arguments validated by
// operators_api.cpp and returns a TLA_* status.
#pragma once

#include "kernels.hpp"

namespace tla {

constexpr int kI8 = TLA_I8;

// Bytes of an element of any type code of the public header.
constexpr int type_bytes(int code) {
  return code == TLA_F32 ? 4 : (code == TLA_E4M3 || code == TLA_I8 ? 1 : 2);
}

// One problem: rows r of A, grouped by expert (rows offsets[e] .. offsets[e +
// 1] - 1 belong to expert e; offsets == nullptr: one expert with every row).
//   product            D[r, n] = epilogue(sum_k A[r, k] B_e(k, n))
//   weight gradient    D_e(m, n) = sum over e's rows r of A[r, m] B[r, n]
// For the weight gradient M x N is D_e's extent, B holds `rows` rows of N,
// and the sum runs over the expert's rows.  Leading dimensions and strides
// are in elements.
struct GroupedParams {
  const int32_t* offsets;
  const uint8_t* A;
  const uint8_t* B;
  uint8_t* D;
  uint8_t* Z;
  const float* sa;       // per row, or null
  const float* sb;       // groups x N, or null
  const uint8_t* bias;   // groups x N, or null
  float* dbias;          // groups x (extent of the gradient's dY side), or null
  int64_t lda, ldb, stride_b, ldd, stride_d, ldz;
  int groups, rows, M, N, K;
  int d_type, bias_type, act, z_mode;
  int tiles_m, tiles_n;  // weight gradient: tiles of one D_e; product: tiles_n only
  int flags;
};
enum : int {
  kOpD16 = 1,    // D (and Z) rows are 16-byte aligned
  kOpVec4 = 2,   // sb and bias rows allow aligned 4-element vectors
  kOpSumA = 4,   // gradient: dY is operand A (column-major D), else B
  kOpHalves = 8, // two-group product: blocks of 128 rows throughout
};

// Blocks of BM rows that `rows` rows in `groups` groups can need: every
// non-empty group's last block may hold a single row.
inline int64_t row_tiles_bound(int64_t rows, int64_t groups, int64_t BM) {
  const int64_t live = rows < groups ? rows : groups;
  return (rows + live * (BM - 1)) / BM;
}

// The register-staged kernel: any order, pitch, alignment (b_kc: B is
// K-contiguous).
int launch_grouped_general(const GroupedParams& p, int type, bool b_kc, hipStream_t stream);
int launch_wgrad_general(const GroupedParams& p, int type, hipStream_t stream);

// The direct-copy kernels: every row starts on a dword.  Product: A's rows and,
// for nk, B's are less than 8 MiB apart; kn: B is 16-bit, a matrix (of 64 rows
// if it has fewer) below 2 GiB.  Gradient: each operand (likewise) below 2 GiB.
// 256 x 256 tiles (grouped_two_group.hpp)
int launch_two_group_nk16(const GroupedParams& p, int type, hipStream_t stream);
int launch_two_group_nk8(const GroupedParams& p, int type, hipStream_t stream);
int launch_two_group_kn(const GroupedParams& p, int type, hipStream_t stream);
// any alignment, B K-contiguous, rows less than 8 MiB apart
int launch_two_group_shift(const GroupedParams& p, int type, hipStream_t stream);
int launch_wgrad_two_group(const GroupedParams& p, int type, hipStream_t stream);
// 64 or 128 x 128 tiles, two or three LDS stages (grouped_direct.hpp)
enum DirectShape : int { kDirect64x3, kDirect128x2, kDirect128x3 };
int launch_grouped_direct(const GroupedParams& p, int type, int shape, hipStream_t stream);
int launch_grouped_direct_kn(const GroupedParams& p, int type, int shape, hipStream_t stream);
int launch_grouped_direct_shift(const GroupedParams& p, int type, int shape, hipStream_t stream);
int launch_wgrad_direct(const GroupedParams& p, int type, int shape, hipStream_t stream);

// The kernel for few rows an expert (grouped_few_rows.hip): B K-contiguous,
// any pitch and alignment; blocks of 16 mt rows, mt 1, 2 or 4, of 32 columns and
// four waves, or, where that would leave compute units without one, 16 columns
// and eight waves.
inline bool few_rows_narrow(int64_t rows, int64_t groups, int64_t N) {
  return (rows < groups ? rows : groups) * ((N + 31) / 32) <= 512;
}
int launch_grouped_few_rows(const GroupedParams& p, int type, int mt, hipStream_t stream);

int launch_quantize_rows(int64_t M, int64_t K, const void* X, int type, int64_t ldx, int8_t* Q,
                         int64_t ldq, float* scale, hipStream_t stream);

}  // namespace tla
