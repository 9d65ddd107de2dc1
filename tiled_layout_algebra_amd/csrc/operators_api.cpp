// operators_api.cpp -- the C entry points of the expert-grouped and 8-bit
// integer products and of the token quantizer: argument validation, status
// codes and the choice of kernel.  Contracts: include/tla.h.
#include <string.h>

#include "operators.hpp"

using namespace tla;

namespace {

constexpr int64_t kLimit = int64_t(1) << 31;
// Extents: the kernels count tiles (up to 256 past an extent) and experts (64 at
// a time) in 32 bits.
constexpr int64_t kMaxExtent = kLimit - 4096;
bool too_large(int64_t groups, int64_t rows, int64_t N, int64_t K) {
  return groups > kMaxExtent || rows > kMaxExtent || N > kMaxExtent || K > kMaxExtent;
}
// products of int8 values sum exactly in 32 bits while K * 128 * 128 < 2^31
constexpr int64_t kMaxKI8 = 131071;

bool out16(int t) { return t == TLA_F16 || t == TLA_BF16; }
bool aux_type(int t) { return out16(t) || t == TLA_F32; }

bool aligned_to(const void* p, int64_t bytes) { return (uintptr_t)p % (uintptr_t)bytes == 0; }

const char* const kNames[TLA_GROUPED_VARIANTS] = {
    "grouped_general_128x128", "grouped_two_group_256x256", "grouped_direct_128x128",
    "grouped_direct_64x128", "grouped_few_rows_64", "grouped_few_rows_32", "grouped_few_rows_16",
    "grouped_two_group_shift_256x256", "grouped_direct_shift_128x128", "grouped_direct_shift_64x128"};

struct Plan {
  GroupedParams p;
  int type;
  bool b_kc;
  Kernel kernel;
};

// Rows of `ld` elements of eb bytes at p start on dwords.
bool dword_rows(const void* p, int64_t ld, int eb) { return aligned_to(p, 4) && ld * eb % 4 == 0; }

// Whether the direct copies' 32-bit offsets reach a slab of k rows `ld` elements
// apart.  A slab has 64 rows however few the sum has, and the range check that
// zeroes the ones past its end needs their offsets unwrapped: below 2^31 bytes
// for max(k, 64) rows, so below 2^32 for the last slab's.
bool k_rows_fit(int64_t k, int64_t ld, int eb) {
  return ld <= (kLimit - 1) / ((k > 64 ? k : 64) * eb);
}

// Whether a launch holds the kernel's workgroups.  bands: the few-row kernel's may go
// out in several launches, while 32 bits count them (16 columns each at the least), for
// products that may have no other kernel (gated_api.cpp); where the grouped products'
// do not fit, the general kernel takes the call.
bool launches(Kernel k, const tla_grouped_gemm_args* a, bool bands) {
  auto blocks = [&](int64_t bm, int64_t bn) {
    return row_tiles_bound(a->rows, a->groups, bm) * ((a->N + bn - 1) / bn);
  };
  auto fits = [&](int64_t bm, int64_t bn, int threads, int64_t more) {
    return grid_fits(blocks(bm, bn) + more, threads);
  };
  const bool narrow = few_rows_narrow(a->rows, a->groups, a->N);
  auto few = [&](int64_t bm) {
    return bands ? blocks(bm, 16) <= kMaxExtent : fits(bm, narrow ? 16 : 32, narrow ? 512 : 256, 0);
  };
  switch (k) {
    case kFewRows1: return few(16);
    case kFewRows2: return few(32);
    case kFewRows4: return few(64);
    case kDirect64: case kDirect64Shift: return fits(64, 128, 256, 0);
    case kDirect128: case kDirect128Shift: return fits(128, 128, 512, 0);
    // half tiles throughout, or whole ones and fewer than 256 halves
    case kTwoGroup: case kTwoGroupShift: return fits(128, 256, 512, 256);
    default: return fits(128, 128, 256, 0);
  }
}

// Whether a kernel takes the problem.
bool takes(Kernel k, const tla_grouped_gemm_args* a, int eb, bool b_kc, bool bands = false) {
  if (k == kGeneral) return true;
  if (a->K == 0 || !launches(k, a, bands)) return false;
  if (k == kFewRows1 || k == kFewRows2 || k == kFewRows4) return b_kc;
  if (a->type == TLA_E4M3 && a->K < kMinKE4m3) return false;
  // 32-bit offsets within a tile's rows
  if (a->lda >= (kLimit >> 8) / eb || (b_kc && a->ldb >= (kLimit >> 8) / eb)) return false;
  if (k >= kTwoGroupShift) return b_kc;
  if (k == kDirect64 && !b_kc) return false;
  if (!dword_rows(a->A, a->lda, eb) || !dword_rows(a->B, a->ldb, eb) ||
      (a->groups > 1 && a->stride_b * eb % 4 != 0))
    return false;
  return b_kc || (eb == 2 && k_rows_fit(a->K, a->ldb, eb));
}

// Blocks of bm rows the experts need, about: a block at least for each that
// has any, otherwise its rows' share and three quarters of a block for its
// ragged end (a half when the experts are even, more when they are not).
double row_blocks(const tla_grouped_gemm_args* a, double bm) {
  const double live = (double)(a->rows < a->groups ? a->rows : a->groups);
  const double blocks = (double)a->rows / live / bm + (a->groups > 1 ? 0.75 : 0.0);
  return live * (blocks > 1.0 ? blocks : 1.0);
}

// Rounds of 256 x 256 tiles (1.6 us a k-tile) the two-group kernel takes, its
// last one in half tiles (0.9) where that is shorter, or half tiles throughout.
double two_group_rounds(const tla_grouped_gemm_args* a, bool halves) {
  const double tiles_n = (double)((a->N + 255) / 256);
  auto up = [](double x) { return (double)(int64_t)((x + 255.0) / 256.0); };
  if (halves) return 0.56 * up(row_blocks(a, 128) * tiles_n);
  const double tiles = row_blocks(a, 256) * tiles_n, whole = (double)(int64_t)(tiles / 256.0);
  const double last = 0.56 * up(2.0 * (tiles - 256.0 * whole));
  return whole + (last < 1.0 ? last : 1.0);
}

// The kernel with the smallest estimated time (us).  These kernels read the
// weights at 5.0 TB/s at most.  Measured with [N, K] weights of 4096 x 4096
// int8 (32 k-tiles of 128 bytes), one expert, M rows:
//      M     few 16   few 32   few 64   64x128   128x128   256x256
//      1       6.3      6.7      7.4     12.8      15.5      23.6
//     32      10.5      9.0     10.1     13.0      15.6      24.3
//     64      19.0     14.5     12.8     13.3      16.0      24.6
//    512       118       88       75     16.7      19.0      27.3
//   2048       453      340      286     51.3      45.8      40.5
//   3001       662      497      416     78.8      67.2      55.4
// and in bf16 for 32 experts of 2048 x 4096: 128 rows 110 (few 16), 123
// (64x128), 4096 rows 174 (64x128), 144 (128x128), 147 (256x256); for 8
// experts of 4096 x 4096 with 2000 rows 129, 123, 89.
// What differs for the operators on these kernels (gated_api.cpp): `own`, MB/us of
// the weights at which a few-row kernel takes an expert's first block of rows and
// each further one, and us a k-tile of the block-scaled kernels of 64 and 128 rows.
struct Rates {
  bool own = false, blocks = false;
  double few[3][2] = {{5.0, 5.0}, {3.3, 3.3}, {2.2, 2.2}};
};
Kernel choose(const tla_grouped_gemm_args* a, int eb, bool b_kc, unsigned allowed, const Rates& r) {
  const double live = (double)(a->rows < a->groups ? a->rows : a->groups);
  const double matrix = (double)a->N * (double)a->K * eb * 1e-6;  // MB
  const double weights = live * matrix / 5.0;
  const double kt = (double)((a->K * eb + 127) / 128);
  Kernel best = kNoop;
  double best_us = 1e30;
  auto consider = [&](Kernel k, double us) {
    if (!(allowed >> k & 1) || !takes(k, a, eb, b_kc, r.own)) return;
    us = us > weights + 4.0 ? us : weights + 4.0;
    if (us < best_us) {
      best = k;
      best_us = us;
    }
  };
  auto tiles = [&](double bm, double bn) {
    return row_blocks(a, bm) * (double)((a->N + (int64_t)bn - 1) / (int64_t)bn);
  };
  // rounds of workgroups, one a compute unit
  auto rounds = [](double t) { return (double)(int64_t)((t + 255.0) / 256.0); };
  // each block of rows reads the weights again, at the rate the matrix
  // instructions and A's rows leave
  auto few = [&](double least, int64_t bm, const double (&rate)[2]) {
    if (!r.own) return least + row_blocks(a, (double)bm) * matrix / rate[0];
    // one expert's blocks are a whole number
    const double n = a->groups == 1 ? (double)((a->rows + bm - 1) / bm) : row_blocks(a, (double)bm);
    const double once = n < live ? n : live;
    return least + matrix * (once / rate[0] + (n - once) / rate[1]);
  };
  consider(kFewRows1, few(4.0, 16, r.few[0]));
  consider(kFewRows2, few(4.3, 32, r.few[1]));
  consider(kFewRows4, few(5.0, 64, r.few[2]));
  const double t64 = tiles(64, 128), t128 = tiles(128, 128);
  auto at_least = [](double least, double us) { return us > least ? us : least; };
  if (r.blocks) {
    consider(kDirect64, 4.2 + kt * at_least(0.45, 0.0018 * t64));
    consider(kDirect128, 4.5 + kt * (t128 <= 256.0 ? 0.72 : at_least(1.15, 1.15 / 512.0 * t128)));
  } else {
    consider(kDirect64, 4.2 + kt * at_least(0.3, (eb == 1 ? 0.0015 : 0.0019) * t64));
    consider(kDirect128, 4.5 + kt * (t128 <= 128.0 ? 0.4 : t128 <= 256.0 ? 0.54 : 0.62 * rounds(t128)));
  }
  const double mixed = two_group_rounds(a, false), halved = two_group_rounds(a, true);
  const double two = mixed < halved ? mixed : halved;
  consider(kTwoGroup, at_least(4.0 + 1.2 * weights, 5.0 + kt * 1.6 * two));
  // any alignment: with B 4096 x 4095 int8, 3001 rows: 122 us (64 rows), 99
  // (128), 69 (256), 99 (general); with 988 x 2371, 400 rows 16, 18, 29, 28;
  // bf16, 4096 rows on 32 experts of 2048 x 4095: 324, 241, 254, 234
  const double kt96 = (double)(a->K * eb / 96 + 1);
  consider(kDirect64Shift, 4.5 + kt * at_least(0.6, (eb == 1 ? 0.0024 : 0.0032) * t64));
  consider(kDirect128Shift, 4.8 + kt * 0.96 * rounds(t128));
  consider(kTwoGroupShift, 6.0 + kt96 * 1.6 * two);
  consider(kGeneral, 4.5 + kt * at_least(1.5, 2.05 * rounds(t128 / 2.0)));
  return best;
}

int plan_product(const tla_grouped_gemm_args* a, Plan* out) {
  if (!a) return TLA_ERR_INVALID_ARG;
  if (a->groups < 0 || a->rows < 0 || a->N < 0 || a->K < 0) return TLA_ERR_INVALID_ARG;
  if (a->b_order != TLA_ROW_MAJOR && a->b_order != TLA_COL_MAJOR) return TLA_ERR_INVALID_ARG;
  if (a->act < TLA_ACT_NONE || a->act > TLA_ACT_GELU) return TLA_ERR_INVALID_ARG;
  if (a->z_mode < TLA_Z_NONE || a->z_mode > TLA_Z_GRAD) return TLA_ERR_INVALID_ARG;
  const bool eight = a->type == TLA_E4M3 || a->type == TLA_I8;
  if (!eight && !out16(a->type)) return TLA_ERR_UNSUPPORTED;
  if (!out16(a->d_type)) return TLA_ERR_UNSUPPORTED;
  if (a->bias && !aux_type(a->bias_type)) return TLA_ERR_UNSUPPORTED;
  if (!eight && (a->scale_a || a->scale_b)) return TLA_ERR_UNSUPPORTED;
  if (too_large(a->groups, a->rows, a->N, a->K)) return TLA_ERR_UNSUPPORTED;
  if (a->type == TLA_I8 && a->K > kMaxKI8) return TLA_ERR_UNSUPPORTED;
  *out = Plan{};
  out->kernel = kNoop;
  if (a->groups == 0 || a->rows == 0 || a->N == 0) return TLA_OK;
  if (!a->offsets && a->groups != 1) return TLA_ERR_INVALID_ARG;
  if (!a->D || a->ldd < a->N) return TLA_ERR_INVALID_ARG;
  const bool b_kc = a->b_order == TLA_COL_MAJOR;
  if (a->K > 0) {
    if (!a->A || !a->B || a->lda < a->K || a->ldb < (b_kc ? a->K : a->N) || a->stride_b < 0)
      return TLA_ERR_INVALID_ARG;
  }
  // without an activation its derivative is 1 and Z is not needed
  const int z_mode = a->z_mode == TLA_Z_GRAD && a->act == TLA_ACT_NONE ? TLA_Z_NONE : a->z_mode;
  if (z_mode != TLA_Z_NONE && (!a->Z || a->ldz < a->N || a->Z == a->D))
    return TLA_ERR_INVALID_ARG;
  const int eb = type_bytes(a->type), bb = type_bytes(a->bias_type);
  if (!aligned_to(a->offsets, 4) || !aligned_to(a->A, eb) || !aligned_to(a->B, eb) ||
      !aligned_to(a->D, 2) || (z_mode != TLA_Z_NONE && !aligned_to(a->Z, 2)) ||
      !aligned_to(a->scale_a, 4) || !aligned_to(a->scale_b, 4) ||
      (a->bias && !aligned_to(a->bias, bb)))
    return TLA_ERR_INVALID_ARG;
  GroupedParams& p = out->p;
  p.offsets = a->offsets;
  p.A = (const uint8_t*)a->A;
  p.B = (const uint8_t*)a->B;
  p.D = (uint8_t*)a->D;
  p.Z = z_mode == TLA_Z_NONE ? nullptr : (uint8_t*)a->Z;
  p.sa = a->scale_a;
  p.sb = a->scale_b;
  p.bias = (const uint8_t*)a->bias;
  p.lda = a->lda;
  p.ldb = a->ldb;
  p.stride_b = a->stride_b;
  p.ldd = a->ldd;
  p.ldz = a->ldz;
  p.groups = (int)a->groups;
  p.rows = (int)a->rows;
  p.N = (int)a->N;
  p.K = (int)a->K;
  p.d_type = a->d_type;
  p.bias_type = a->bias_type;
  p.act = a->act;
  p.z_mode = z_mode;
  if (a->ldd % 8 == 0 && aligned_to(a->D, 16) && (!p.Z || (a->ldz % 8 == 0 && aligned_to(p.Z, 16))))
    p.flags |= kOpD16;
  if ((a->N % 4 == 0 || a->groups == 1) && aligned_to(a->scale_b, 16) &&
      (!a->bias || aligned_to(a->bias, 4 * bb)))
    p.flags |= kOpVec4;
  // no other kernel needs fewer threads than the one that takes everything
  if (!launches(kGeneral, a, false)) return TLA_ERR_UNSUPPORTED;
  out->type = a->type;
  out->b_kc = b_kc;
  out->kernel = choose(a, eb, b_kc, kAnyKernel, Rates{});
  return TLA_OK;
}

// forced: a variant id, or -1 for the estimate's choice
int run_product(const tla_grouped_gemm_args* a, hipStream_t stream, int forced = -1) {
  Plan plan;
  const int rc = plan_product(a, &plan);
  if (rc) return rc;
  if (forced >= 0 && plan.kernel != kNoop) {
    if (!takes((Kernel)forced, a, type_bytes(a->type), plan.b_kc)) return TLA_ERR_UNSUPPORTED;
    plan.kernel = (Kernel)forced;
  }
  GroupedParams& p = plan.p;
  if (product_halves(a)) p.flags |= kOpHalves;
  const int t = plan.type;
  switch (plan.kernel) {
    case kNoop: return TLA_OK;
    case kTwoGroup:
      if (!plan.b_kc) return launch_two_group_kn(p, t, stream);
      return type_bytes(t) == 1 ? launch_two_group_nk8(p, t, stream)
                                : launch_two_group_nk16(p, t, stream);
    case kDirect128Shift: return launch_grouped_direct_shift(p, t, kDirect128x3, stream);
    case kDirect64Shift: return launch_grouped_direct_shift(p, t, kDirect64x3, stream);
    case kTwoGroupShift: return launch_two_group_shift(p, t, stream);
    case kDirect64: return launch_grouped_direct(p, t, kDirect64x3, stream);
    case kDirect128: {
      if (plan.b_kc) return launch_grouped_direct(p, t, kDirect128x3, stream);
      // three stages while every workgroup has a compute unit of its own (500
      // rows on 4 experts of 1024 x 1024: 10.2 us against 12.2 with two), two
      // stages and two workgroups a unit beyond (16000 rows on 8: 57 against 63)
      const int64_t blocks = row_tiles_bound(p.rows, p.groups, 128) * ((p.N + 127) / 128);
      return launch_grouped_direct_kn(p, t, blocks <= 256 ? kDirect128x3 : kDirect128x2, stream);
    }
    case kFewRows1: return launch_grouped_few_rows(p, t, 1, stream);
    case kFewRows2: return launch_grouped_few_rows(p, t, 2, stream);
    case kFewRows4: return launch_grouped_few_rows(p, t, 4, stream);
    case kGeneral: return launch_grouped_general(p, t, plan.b_kc, stream);
  }
  return TLA_ERR_UNSUPPORTED;
}

}  // namespace

namespace tla {

// Measured, 4096 x 4096 (us; few 16, 32, 64, then 64 x 128, 128 x 128, 256 x 256):
//   block-scaled         24 rows  10.4   8.2  10.3   18.7  27  32
//                        48       14    14.3  11.5   18.7  27  32
//                        96       24    19    24     18.6  27  32
//                       800                          26.7  28  33
//                      1600                                41  34
//   gated, block-scaled  24       14    10.7  12     19     27  33
//                        48       19    20    14.5   19     27  33
//                        96       35    30    27     19     27  34
//   gated, bf16          24       24    16.5  18     23     25  40
//                        48       35    31    22.7   23     26  41
//                       400                          35-38      58
Kernel choose_product(const tla_grouped_gemm_args* a, int eb, bool b_kc, unsigned allowed) {
  Rates rates;
  rates.own = true;
  rates.blocks = eb == 1;
  const double few[3][2] = {{5.0, 5.0}, {4.5, 2.8}, {3.0, 1.8}};
  for (int i = 0; i < 3; ++i)
    for (int j = 0; j < 2; ++j) rates.few[i][j] = few[i][j];
  return choose(a, eb, b_kc, allowed, rates);
}
bool product_halves(const tla_grouped_gemm_args* a) {
  return two_group_rounds(a, true) < two_group_rounds(a, false);
}

}  // namespace tla

extern "C" {

int tla_grouped_gemm(const tla_grouped_gemm_args* args, void* stream) {
  return run_product(args, (hipStream_t)stream);
}

int tla_grouped_gemm_variant(const tla_grouped_gemm_args* args, char* buf, int32_t cap) {
  if (!buf || cap < 1) return TLA_ERR_INVALID_ARG;
  Plan plan;
  const int rc = plan_product(args, &plan);
  if (rc) return rc;
  strncpy(buf, plan.kernel == kNoop ? "noop" : kNames[plan.kernel], (size_t)cap - 1);
  buf[cap - 1] = '\0';
  return TLA_OK;
}

int tla_grouped_gemm_run_variant(const tla_grouped_gemm_args* args, int32_t variant,
                                 void* stream) {
  if (variant < 0 || variant >= TLA_GROUPED_VARIANTS) return TLA_ERR_INVALID_ARG;
  return run_product(args, (hipStream_t)stream, variant);
}

int tla_gemm_i8(const tla_gemm_i8_args* a, void* stream) {
  if (!a) return TLA_ERR_INVALID_ARG;
  tla_grouped_gemm_args g{};
  g.groups = 1;
  g.rows = a->M;
  g.N = a->N;
  g.K = a->K;
  g.A = a->A;
  g.type = TLA_I8;
  g.lda = a->lda;
  g.B = a->B;
  g.b_order = a->b_order;
  g.ldb = a->ldb;
  g.D = a->D;
  g.d_type = a->d_type;
  g.ldd = a->ldd;
  g.scale_a = a->scale_a;
  g.scale_b = a->scale_b;
  g.bias = a->bias;
  g.bias_type = a->bias_type;
  g.act = a->act;
  return run_product(&g, (hipStream_t)stream);
}

int tla_grouped_gemm_wgrad(const tla_grouped_wgrad_args* a, void* stream) {
  if (!a) return TLA_ERR_INVALID_ARG;
  if (a->groups < 0 || a->rows < 0 || a->N < 0 || a->K < 0) return TLA_ERR_INVALID_ARG;
  if (a->d_order != TLA_ROW_MAJOR && a->d_order != TLA_COL_MAJOR) return TLA_ERR_INVALID_ARG;
  if (!out16(a->type) || !aux_type(a->d_type)) return TLA_ERR_UNSUPPORTED;
  if (too_large(a->groups, a->rows, a->N, a->K)) return TLA_ERR_UNSUPPORTED;
  if (a->groups == 0 || a->K == 0 || a->N == 0) return TLA_OK;
  if (!a->offsets && a->groups != 1) return TLA_ERR_INVALID_ARG;
  if (a->rows > 0 && (!a->Y || a->ldy < a->N)) return TLA_ERR_INVALID_ARG;
  const bool row = a->d_order == TLA_ROW_MAJOR;
  const int64_t outer = row ? a->K : a->N, inner = row ? a->N : a->K;
  if (!a->D || a->ldd < inner) return TLA_ERR_INVALID_ARG;
  if (a->rows > 0 && (!a->A || a->lda < a->K)) return TLA_ERR_INVALID_ARG;
  // the experts' matrices must not overlap
  if (a->groups > 1 && a->stride_d < (outer - 1) * a->ldd + inner) return TLA_ERR_INVALID_ARG;
  const int db = type_bytes(a->d_type);
  if (!aligned_to(a->offsets, 4) || !aligned_to(a->A, 2) || !aligned_to(a->Y, 2) ||
      !aligned_to(a->D, db) || !aligned_to(a->dbias, 4))
    return TLA_ERR_INVALID_ARG;
  GroupedParams p{};
  p.offsets = a->offsets;
  p.groups = (int)a->groups;
  p.rows = (int)a->rows;
  p.dbias = a->dbias;
  p.D = (uint8_t*)a->D;
  p.d_type = a->d_type;
  p.ldd = a->ldd;
  p.stride_d = a->stride_d;
  // a column-major D_e is the row-major product of the operands swapped
  p.A = (const uint8_t*)(row ? a->A : a->Y);
  p.B = (const uint8_t*)(row ? a->Y : a->A);
  p.lda = row ? a->lda : a->ldy;
  p.ldb = row ? a->ldy : a->lda;
  p.M = (int)(row ? a->K : a->N);
  p.N = (int)(row ? a->N : a->K);
  const int per16 = 16 / db;
  if (a->ldd % per16 == 0 && a->stride_d % per16 == 0 && aligned_to(a->D, 16)) p.flags |= kOpD16;
  if (!row) p.flags |= kOpSumA;
  // the direct copies' layout (operators.hpp, launch_wgrad_two_group)
  const bool direct = dword_rows(a->A, a->lda, 2) && dword_rows(a->Y, a->ldy, 2) &&
                      k_rows_fit(a->rows, a->lda, 2) && k_rows_fit(a->rows, a->ldy, 2);
  // 256 x 256 tiles when they give every compute unit one (8000 rows on 16
  // experts of 2048 x 2048: 105 us against 124 for 128 x 128); below, 128 x 128
  // with two stages (777 rows, 16 experts of 512 x 1024: 11.7 us against 17.0
  // and 13.5 with three), three stages when they all fit at once (1000 rows, 2
  // experts of 1024 x 1024: 9.0 against 10.7)
  const int64_t tiles = a->groups * ((a->K + 255) / 256) * ((a->N + 255) / 256);
  const int64_t tiles128 = a->groups * ((a->K + 127) / 128) * ((a->N + 127) / 128);
  if (direct && tiles >= 256) return launch_wgrad_two_group(p, a->type, (hipStream_t)stream);
  if (direct)
    return launch_wgrad_direct(p, a->type, tiles128 <= 256 ? kDirect128x3 : kDirect128x2,
                               (hipStream_t)stream);
  return launch_wgrad_general(p, a->type, (hipStream_t)stream);
}

int tla_quantize_rows(int64_t M, int64_t K, const void* X, int32_t x_type, int64_t ldx, void* Q,
                      int64_t ldq, float* scale, void* stream) {
  if (M < 0 || K < 0) return TLA_ERR_INVALID_ARG;
  if (!aux_type(x_type)) return TLA_ERR_UNSUPPORTED;
  if (M == 0) return TLA_OK;
  if (!scale || !aligned_to(scale, 4)) return TLA_ERR_INVALID_ARG;
  if (K > 0 && (!X || !Q || ldx < K || ldq < K || !aligned_to(X, type_bytes(x_type))))
    return TLA_ERR_INVALID_ARG;
  return launch_quantize_rows(M, K, X, x_type, ldx, (int8_t*)Q, ldq, scale, (hipStream_t)stream);
}

}  // extern "C"
