// gated_api.cpp -- the C entry points of the gated feed-forward products, the
// block-scaled e4m3 product and its quantizer: argument validation, status codes
// and the choice of kernel.  Contracts: include/tla.h.
#include "operators.hpp"

using namespace tla;

namespace {

constexpr int64_t kMaxExtent = (int64_t(1) << 31) - 4096;

bool out16(int t) { return t == TLA_F16 || t == TLA_BF16; }
bool aux_type(int t) { return out16(t) || t == TLA_F32; }
bool order_ok(int o) { return o == TLA_ROW_MAJOR || o == TLA_COL_MAJOR; }
bool aligned_to(const void* p, int64_t bytes) { return (uintptr_t)p % (uintptr_t)bytes == 0; }
int64_t blocks_of(int64_t n) { return (n + 127) / 128; }
// of a matrix of scales, outer x inner in `order`
bool scales_ok(const float* s, int order, int64_t ld, int64_t rows, int64_t cols) {
  return s && aligned_to(s, 4) && ld >= (order == TLA_ROW_MAJOR ? cols : rows);
}
bool rows16(const void* p, int64_t ld) { return !p || (ld % 8 == 0 && aligned_to(p, 16)); }

// kernels that a role has
constexpr unsigned kFewRows = 1u << kFewRows1 | 1u << kFewRows2 | 1u << kFewRows4;
constexpr unsigned kTiles = 1u << kTwoGroup | 1u << kDirect128 | 1u << kDirect64;

// The problem as the estimates of the grouped products see it: the gated
// product's tiles hold columns of both matrices, so it counts twice the columns.
struct Plan {
  GroupedParams p;
  tla_grouped_gemm_args shape;
  int type, role;
  bool b_kc;
  unsigned allowed;
  Kernel kernel;
};

// Fills in what the three products share and picks the kernel (forced: that one).
int finish(Plan* out, int forced) {
  GroupedParams& p = out->p;
  const tla_grouped_gemm_args& a = out->shape;
  p.offsets = a.offsets;
  p.A = (const uint8_t*)a.A;
  p.B = (const uint8_t*)a.B;
  p.lda = a.lda;
  p.ldb = a.ldb;
  p.stride_b = a.stride_b;
  p.groups = (int)a.groups;
  p.rows = (int)a.rows;
  p.K = (int)a.K;
  const bool blocks = out->type == TLA_E4M3;
  // copies of whole dwords from the second matrix too
  if (p.B2 && !aligned_to(p.B2, 4)) out->allowed &= ~kTiles;
  const int eb = type_bytes(out->type);
  if (forced >= 0) out->allowed &= 1u << forced;
  // short sums are fp32 throughout: of the tile kernels only the direct ones have that form
  else if (blocks && a.K < kMinKE4m3) out->allowed &= ~(1u << kTwoGroup);
  // (the few-row kernel takes any block-scaled problem; with K = 0 every kernel
  // but the general one stands back)
  if (a.K == 0 && blocks && out->allowed & 1u << kFewRows1) out->kernel = kFewRows1;
  else out->kernel = choose_product(&a, eb, out->b_kc, out->allowed);
  if (out->kernel == kNoop) return TLA_ERR_UNSUPPORTED;
  if (product_halves(&a)) p.flags |= kOpHalves;
  return TLA_OK;
}

int run(const Plan& plan, hipStream_t s) {
  const GroupedParams& p = plan.p;
  const int t = plan.type, role = plan.role;
  if (t == TLA_E4M3) {
    const bool gated = role == kGated;
    switch (plan.kernel) {
      case kTwoGroup: return launch_blocks_two_group(p, gated, s);
      case kDirect128: return launch_blocks_direct(p, 128, gated, s);
      case kDirect64: return launch_blocks_direct(p, 64, gated, s);
      case kFewRows4: return launch_blocks_few_rows(p, 4, gated, s);
      case kFewRows2: return launch_blocks_few_rows(p, 2, gated, s);
      case kFewRows1: return launch_blocks_few_rows(p, 1, gated, s);
      default: return TLA_ERR_UNSUPPORTED;
    }
  }
  switch (plan.kernel) {
    case kTwoGroup:
      if (role == kGated)
        return plan.b_kc ? launch_two_group_gated_nk(p, t, s) : launch_two_group_gated_kn(p, t, s);
      return plan.b_kc ? launch_two_group_grad_nk(p, t, s) : launch_two_group_grad_kn(p, t, s);
    case kDirect128:
      return plan.b_kc ? launch_gated_direct_nk(p, t, kDirect128x3, role, s)
                       : launch_gated_direct_kn(p, t, role, s);
    case kDirect64: return launch_gated_direct_nk(p, t, kDirect64x3, role, s);
    case kFewRows4: return launch_gated_few_rows(p, t, 4, s);
    case kFewRows2: return launch_gated_few_rows(p, t, 2, s);
    case kFewRows1: return launch_gated_few_rows(p, t, 1, s);
    case kGeneral: return launch_gated_general(p, t, plan.b_kc, role, s);
    default: return TLA_ERR_UNSUPPORTED;
  }
}

// The checks that the three products share.
int check_shape(int64_t groups, int64_t rows, int64_t N, int64_t K, int act, int w_order) {
  if (groups < 0 || rows < 0 || N < 0 || K < 0) return TLA_ERR_INVALID_ARG;
  if (!order_ok(w_order)) return TLA_ERR_INVALID_ARG;
  if (act < TLA_ACT_NONE || act > TLA_ACT_SILU) return TLA_ERR_INVALID_ARG;
  if (groups > kMaxExtent || rows > kMaxExtent || N > kMaxExtent / 2 || K > kMaxExtent)
    return TLA_ERR_UNSUPPORTED;
  return TLA_OK;
}

int plan_gated(const tla_gated_gemm_args* a, Plan* out, int forced) {
  *out = Plan{};
  out->kernel = kNoop;
  if (!a) return TLA_ERR_INVALID_ARG;
  if (const int rc = check_shape(a->groups, a->rows, a->N, a->K, a->act, a->w_order)) return rc;
  const bool blocks = a->type == TLA_E4M3;
  if (!blocks && !out16(a->type)) return TLA_ERR_UNSUPPORTED;
  if (blocks ? !out16(a->h_type) : a->h_type != a->type) return TLA_ERR_UNSUPPORTED;
  if ((a->b_gate || a->b_up) && !aux_type(a->bias_type)) return TLA_ERR_UNSUPPORTED;
  const bool b_kc = a->w_order == TLA_COL_MAJOR;
  if (blocks ? !b_kc : a->scale_x || a->scale_gate || a->scale_up) return TLA_ERR_UNSUPPORTED;
  if (blocks && (!order_ok(a->sx_order) || !order_ok(a->sw_order))) return TLA_ERR_INVALID_ARG;
  if (a->groups == 0 || a->rows == 0 || a->N == 0) return TLA_OK;
  if (!a->offsets && a->groups != 1) return TLA_ERR_INVALID_ARG;
  const int eb = type_bytes(a->type), bb = type_bytes(a->bias_type);
  if (!a->H || a->ldh < a->N || !aligned_to(a->H, 2)) return TLA_ERR_INVALID_ARG;
  if (a->K > 0) {
    if (!a->X || !a->W_gate || !a->W_up || a->ldx < a->K || a->ldw < (b_kc ? a->K : a->N) ||
        a->stride_w < 0)
      return TLA_ERR_INVALID_ARG;
    const int64_t kb = blocks_of(a->K), nb = blocks_of(a->N);
    if (blocks && (!scales_ok(a->scale_x, a->sx_order, a->ldsx, a->rows, kb) ||
                   !scales_ok(a->scale_gate, a->sw_order, a->ldsw, nb, kb) ||
                   !scales_ok(a->scale_up, a->sw_order, a->ldsw, nb, kb) || a->stride_sw < 0))
      return TLA_ERR_INVALID_ARG;
  }
  if (!a->Z_gate != !a->Z_up) return TLA_ERR_INVALID_ARG;
  if (a->Z_gate && (a->ldz < a->N || a->Z_gate == a->Z_up || a->Z_gate == a->H ||
                    a->Z_up == a->H || !aligned_to(a->Z_gate, 2) || !aligned_to(a->Z_up, 2)))
    return TLA_ERR_INVALID_ARG;
  if (!aligned_to(a->offsets, 4) || !aligned_to(a->X, eb) || !aligned_to(a->W_gate, eb) ||
      !aligned_to(a->W_up, eb) || !aligned_to(a->b_gate, a->b_gate ? bb : 1) ||
      !aligned_to(a->b_up, a->b_up ? bb : 1))
    return TLA_ERR_INVALID_ARG;
  GroupedParams& p = out->p;
  tla_grouped_gemm_args& s = out->shape;
  s.groups = a->groups;
  s.rows = a->rows;
  s.N = 2 * a->N;
  s.K = a->K;
  s.offsets = a->offsets;
  s.A = a->X;
  s.type = blocks ? TLA_I8 : a->type;  // (for the estimates; short sums: finish)
  s.lda = a->ldx;
  s.B = a->W_gate;
  s.b_order = a->w_order;
  s.ldb = a->ldw;
  s.stride_b = a->stride_w;
  p.N = (int)a->N;
  p.B2 = (const uint8_t*)a->W_up;
  p.bias = (const uint8_t*)a->b_gate;
  p.bias2 = (const uint8_t*)a->b_up;
  p.bias_type = a->bias_type;
  p.act = a->act;
  p.D = (uint8_t*)a->H;
  p.d_type = a->h_type;
  p.ldd = a->ldh;
  p.Z = (uint8_t*)a->Z_gate;
  p.Z2 = (uint8_t*)a->Z_up;
  p.ldz = a->ldz;
  if (blocks) {
    const bool xr = a->sx_order == TLA_ROW_MAJOR, wr = a->sw_order == TLA_ROW_MAJOR;
    p.sa = a->scale_x;
    p.sa_row = xr ? a->ldsx : 1;
    p.sa_kb = xr ? 1 : a->ldsx;
    p.sb = a->scale_gate;
    p.sb2 = a->scale_up;
    p.sb_col = wr ? a->ldsw : 1;
    p.sb_kb = wr ? 1 : a->ldsw;
    p.stride_sb = a->stride_sw;
  }
  if (rows16(p.D, p.ldd) && rows16(p.Z, p.ldz) && rows16(p.Z2, p.ldz)) p.flags |= kOpD16;
  out->type = a->type;
  out->role = kGated;
  out->b_kc = b_kc;
  out->allowed = kTiles | kFewRows | (blocks ? 0u : 1u << kGeneral);
  return finish(out, forced);
}

int plan_grad(const tla_gated_grad_args* a, Plan* out, int forced) {
  *out = Plan{};
  out->kernel = kNoop;
  if (!a) return TLA_ERR_INVALID_ARG;
  if (const int rc = check_shape(a->groups, a->rows, a->N, a->K, a->act, a->w_order)) return rc;
  if (!out16(a->type) || a->d_type != a->type) return TLA_ERR_UNSUPPORTED;
  if (a->groups == 0 || a->rows == 0 || a->N == 0) return TLA_OK;
  if (!a->offsets && a->groups != 1) return TLA_ERR_INVALID_ARG;
  const bool b_kc = a->w_order == TLA_COL_MAJOR;
  if (a->K > 0 && (!a->dY || !a->W || a->ldy < a->K || a->ldw < (b_kc ? a->K : a->N) ||
                   a->stride_w < 0))
    return TLA_ERR_INVALID_ARG;
  const void* in[2] = {a->Z_gate, a->Z_up};
  const void* outs[3] = {a->dZ_gate, a->dZ_up, a->H};
  for (const void* x : in)
    if (!x || !aligned_to(x, 2)) return TLA_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i) {
    if ((i < 2 && !outs[i]) || !aligned_to(outs[i], 2)) return TLA_ERR_INVALID_ARG;
    for (int j = 0; outs[i] && j < 3; ++j)
      if ((j < i && outs[j] == outs[i]) || (j < 2 && in[j] == outs[i])) return TLA_ERR_INVALID_ARG;
  }
  if (a->ldz < a->N || a->ldd < a->N || (a->H && a->ldh < a->N)) return TLA_ERR_INVALID_ARG;
  if (!aligned_to(a->offsets, 4) || !aligned_to(a->dY, 2) || !aligned_to(a->W, 2))
    return TLA_ERR_INVALID_ARG;
  GroupedParams& p = out->p;
  tla_grouped_gemm_args& s = out->shape;
  s.groups = a->groups;
  s.rows = a->rows;
  s.N = a->N;
  s.K = a->K;
  s.offsets = a->offsets;
  s.A = a->dY;
  s.type = a->type;
  s.lda = a->ldy;
  s.B = a->W;
  s.b_order = a->w_order;
  s.ldb = a->ldw;
  s.stride_b = a->stride_w;
  p.N = (int)a->N;
  p.act = a->act;
  p.Z = (uint8_t*)a->Z_gate;
  p.Z2 = (uint8_t*)a->Z_up;
  p.ldz = a->ldz;
  p.D = (uint8_t*)a->dZ_gate;
  p.D2 = (uint8_t*)a->dZ_up;
  p.ldd = a->ldd;
  p.d_type = a->d_type;
  p.H = (uint8_t*)a->H;
  p.ldh = a->ldh;
  if (rows16(p.D, p.ldd) && rows16(p.D2, p.ldd) && rows16(p.H, p.ldh)) p.flags |= kOpD16;
  out->type = a->type;
  out->role = kGateGrad;
  out->b_kc = b_kc;
  out->allowed = kTiles | 1u << kGeneral;
  return finish(out, forced);
}

int plan_blocks(const tla_gemm_blocks_args* a, Plan* out, int forced) {
  *out = Plan{};
  out->kernel = kNoop;
  if (!a) return TLA_ERR_INVALID_ARG;
  if (const int rc = check_shape(a->groups, a->rows, a->N, a->K, a->act, TLA_COL_MAJOR)) return rc;
  if (!order_ok(a->sa_order) || !order_ok(a->sb_order)) return TLA_ERR_INVALID_ARG;
  if (!out16(a->d_type) || (a->bias && !aux_type(a->bias_type))) return TLA_ERR_UNSUPPORTED;
  if (a->groups == 0 || a->rows == 0 || a->N == 0) return TLA_OK;
  if (!a->offsets && a->groups != 1) return TLA_ERR_INVALID_ARG;
  if (!a->D || a->ldd < a->N || !aligned_to(a->D, 2)) return TLA_ERR_INVALID_ARG;
  if (a->K > 0) {
    const int64_t kb = blocks_of(a->K), nb = blocks_of(a->N);
    if (!a->A || !a->B || a->lda < a->K || a->ldb < a->K || a->stride_b < 0 ||
        !scales_ok(a->scale_a, a->sa_order, a->ldsa, a->rows, kb) ||
        !scales_ok(a->scale_b, a->sb_order, a->ldsb, nb, kb) || a->stride_sb < 0)
      return TLA_ERR_INVALID_ARG;
  }
  if (!aligned_to(a->offsets, 4) || (a->bias && !aligned_to(a->bias, type_bytes(a->bias_type))))
    return TLA_ERR_INVALID_ARG;
  GroupedParams& p = out->p;
  tla_grouped_gemm_args& s = out->shape;
  s.groups = a->groups;
  s.rows = a->rows;
  s.N = a->N;
  s.K = a->K;
  s.offsets = a->offsets;
  s.A = a->A;
  s.type = TLA_I8;  // (for the estimates; short sums: finish)
  s.lda = a->lda;
  s.B = a->B;
  s.b_order = TLA_COL_MAJOR;
  s.ldb = a->ldb;
  s.stride_b = a->stride_b;
  p.N = (int)a->N;
  p.bias = (const uint8_t*)a->bias;
  p.bias_type = a->bias_type;
  p.act = a->act;
  p.D = (uint8_t*)a->D;
  p.d_type = a->d_type;
  p.ldd = a->ldd;
  const bool ar = a->sa_order == TLA_ROW_MAJOR, br = a->sb_order == TLA_ROW_MAJOR;
  p.sa = a->scale_a;
  p.sa_row = ar ? a->ldsa : 1;
  p.sa_kb = ar ? 1 : a->ldsa;
  p.sb = a->scale_b;
  p.sb_col = br ? a->ldsb : 1;
  p.sb_kb = br ? 1 : a->ldsb;
  p.stride_sb = a->stride_sb;
  if (rows16(p.D, p.ldd)) p.flags |= kOpD16;
  out->type = TLA_E4M3;
  out->role = kPlain;
  out->b_kc = true;
  out->allowed = kTiles | kFewRows;
  return finish(out, forced);
}

template <class Args>
int call(int (*plan)(const Args*, Plan*, int), const Args* args, int forced, void* stream) {
  Plan p;
  const int rc = plan(args, &p, forced);
  return rc || p.kernel == kNoop ? rc : run(p, (hipStream_t)stream);
}
bool variant_ok(int32_t v) { return v >= 0 && v < TLA_GROUPED_VARIANTS; }

}  // namespace

extern "C" {

int tla_gated_gemm(const tla_gated_gemm_args* a, void* stream) { return call(plan_gated, a, -1, stream); }
int tla_gated_gemm_run_variant(const tla_gated_gemm_args* a, int32_t variant, void* stream) {
  return variant_ok(variant) ? call(plan_gated, a, variant, stream) : TLA_ERR_INVALID_ARG;
}

int tla_gated_gemm_grad(const tla_gated_grad_args* a, void* stream) { return call(plan_grad, a, -1, stream); }
int tla_gated_gemm_grad_run_variant(const tla_gated_grad_args* a, int32_t variant, void* stream) {
  return variant_ok(variant) ? call(plan_grad, a, variant, stream) : TLA_ERR_INVALID_ARG;
}

int tla_gemm_blocks(const tla_gemm_blocks_args* a, void* stream) { return call(plan_blocks, a, -1, stream); }
int tla_gemm_blocks_run_variant(const tla_gemm_blocks_args* a, int32_t variant, void* stream) {
  return variant_ok(variant) ? call(plan_blocks, a, variant, stream) : TLA_ERR_INVALID_ARG;
}

int tla_quantize_blocks(const tla_quantize_blocks_args* a, void* stream) {
  if (!a || a->M < 0 || a->K < 0 || (a->block_rows != 1 && a->block_rows != 128) ||
      !order_ok(a->s_order))
    return TLA_ERR_INVALID_ARG;
  if (!aux_type(a->x_type) || a->M > kMaxExtent || a->K > kMaxExtent) return TLA_ERR_UNSUPPORTED;
  if (a->M == 0 || a->K == 0) return TLA_OK;
  const int64_t rows = a->block_rows == 1 ? a->M : blocks_of(a->M);
  if (!a->X || !a->Q || a->ldx < a->K || a->ldq < a->K || !aligned_to(a->X, type_bytes(a->x_type)) ||
      !scales_ok(a->scale, a->s_order, a->lds, rows, blocks_of(a->K)))
    return TLA_ERR_INVALID_ARG;
  const bool row = a->s_order == TLA_ROW_MAJOR;
  return launch_quantize_blocks(a->M, a->K, a->X, a->x_type, a->ldx, a->block_rows, (uint8_t*)a->Q,
                                a->ldq, a->scale, row ? a->lds : 1, row ? 1 : a->lds,
                                (hipStream_t)stream);
}

}  // extern "C"
