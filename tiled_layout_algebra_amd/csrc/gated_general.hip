// gated_general.hip -- the gated product and its gradient for operands of any
// pitch and alignment: launches of the register-staged kernel
// (grouped_general.hpp), and a plain kernel for lines shorter than a 16-byte
// chunk, which that one does not take.
#include "grouped_general.hpp"

namespace tla {
namespace {

// The element at row, n of the hidden layer, the sums in order.
template <int kRole>
__device__ __forceinline__ void gated_small(const GroupedParams& p, int type, bool b_kc, int row, int n) {
  // the last expert that starts at or before the row
  int e = 0, lo, hi;
  for (int above = p.groups; above - e > 1;) {
    const int mid = e + (above - e) / 2;
    expert_rows(p, mid, lo, hi);
    if (lo <= row) e = mid;
    else above = mid;
  }
  expert_rows(p, e, lo, hi);
  if (row < lo || row >= hi) return;  // a row of no expert
  const uint8_t* a = p.A + (int64_t)row * p.lda * 2;
  const int64_t first = (int64_t)e * p.stride_b + (b_kc ? n * p.ldb : n), step = b_kc ? 1 : p.ldb;
  float g = 0.f, u = 0.f;
  for (int k = 0; k < p.K; ++k) {
    const float v = load_elem(a, type, k);
    g = fmaf(v, load_elem(p.B, type, first + k * step), g);
    if constexpr (kRole == kGated) u = fmaf(v, load_elem(p.B2, type, first + k * step), u);
  }
  const int64_t z = (int64_t)row * p.ldz + n, d = (int64_t)row * p.ldd + n;
  if constexpr (kRole == kGated) {
    if (p.bias) g += load_elem(p.bias, p.bias_type, (int64_t)e * p.N + n);
    if (p.bias2) u += load_elem(p.bias2, p.bias_type, (int64_t)e * p.N + n);
    if (p.Z) {
      ((uint16_t*)p.Z)[z] = to_bits(g, p.d_type);
      ((uint16_t*)p.Z2)[z] = to_bits(u, p.d_type);
    }
    ((uint16_t*)p.D)[d] = to_bits(act_any(g, p.act) * u, p.d_type);
  } else {
    const float dh = g, gate = load_elem(p.Z, p.d_type, z), up = load_elem(p.Z2, p.d_type, z);
    with_act(p.act, [&](auto act) {
      float value, slope;
      act_both<act>(gate, p.act == TLA_ACT_NONE, value, slope);
      ((uint16_t*)p.D)[d] = to_bits(dh * (up * slope), p.d_type);
      ((uint16_t*)p.D2)[d] = to_bits(dh * value, p.d_type);
      if (p.H) ((uint16_t*)p.H)[(int64_t)row * p.ldh + n] = to_bits(value * up, p.d_type);
    });
  }
}

// A thread an element, or, past the largest grid, several.  Extents below eight
// elements only, where no kernel's tiles would be a tenth full, and K = 0.
template <int kRole>
__global__ __launch_bounds__(256) void gated_small_kernel(const GroupedParams p, int type, bool b_kc) {
  const int64_t all = (int64_t)p.rows * p.N, step = (int64_t)gridDim.x * 256;
  for (int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x; x < all; x += step)
    gated_small<kRole>(p, type, b_kc, (int)(x / p.N), (int)(x % p.N));
}

template <int kRole>
int launch_small(const GroupedParams& p, int type, bool b_kc, hipStream_t s) {
  const int64_t need = ((int64_t)p.rows * p.N + 255) / 256, most = kMaxThreads / 256;
  const int64_t grid = need < most ? need : most;
  hipLaunchKernelGGL((gated_small_kernel<kRole>), dim3((unsigned)grid), dim3(256), 0, s, p, type, b_kc);
  return hipGetLastError() == hipSuccess ? TLA_OK : TLA_ERR_HIP;
}

template <int kCode, int kRole>
int launch(const GroupedParams& p, bool b_kc, hipStream_t s) {
  if (p.K < 8 || (!b_kc && p.N < 8)) return launch_small<kRole>(p, kCode, b_kc, s);
  return b_kc ? launch_form<kCode, kBKc, false, true, kRole>(p, s)
              : launch_form<kCode, kBRows, false, true, kRole>(p, s);
}

}  // namespace

int launch_gated_general(const GroupedParams& p, int type, bool b_kc, int role, hipStream_t s) {
  if (role == kGated)
    return type == TLA_BF16 ? launch<kBF16, kGated>(p, b_kc, s) : launch<kF16, kGated>(p, b_kc, s);
  return type == TLA_BF16 ? launch<kBF16, kGateGrad>(p, b_kc, s) : launch<kF16, kGateGrad>(p, b_kc, s);
}

}  // namespace tla
