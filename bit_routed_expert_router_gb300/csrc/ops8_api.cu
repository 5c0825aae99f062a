// C entry points of the norm, of the 8-bit operators and of the layer for a few
// tokens: argument checks, then the launches (norm.cu, grouped_mm8.cu,
// token_layer.cu).  No context, no allocation.
#include <cmath>

#include "op_checks.h"
#include "ops8.h"

namespace {

using namespace moe;

bool is16(int dtype) { return dtype == MOE_BF16 || dtype == MOE_F16; }

bool norm_ok(int dtype, int m, int d, const void* weight, float eps) {
  return is16(dtype) && m >= 0 && m <= kMaxRows && d >= 8 && d <= kNormMaxD && d % 8 == 0 && aligned(weight, 16) &&
         eps >= 0.f && std::isfinite(eps);
}

// x, w and their scales; n: rows of an expert's weights
bool product8_ok(const void* x, int64_t ldx, const float* sx, int m, const int32_t* offsets, int n_experts, const void* w,
                 const float* sw, int k) {
  return m >= 0 && m <= kMaxRows && n_experts >= 1 && n_experts <= kMaxExperts && offsets && aligned(offsets, 4) && k >= 16 &&
         k <= kMaxSide && k % 16 == 0 && rows_ok(x, m, ldx, k, 16) && (sx || m == 0) && aligned(sx, 4) && w &&
         aligned(w, 16) && sw && aligned(sw, 4);
}

}  // namespace

extern "C" moe_status moe_rmsnorm(int dtype, const void* h, int64_t ldh, const void* delta, int64_t ldd, int delta_dtype,
                                  const void* weight, float eps, int m, int d, void* h_out, int64_t ldo, void* y,
                                  int64_t ldy, void* y8, int64_t ldy8, float* scale, void* stream) {
  if (!norm_ok(dtype, m, d, weight, eps) || !rows_ok(h, m, ldh, d)) return MOE_EINVAL;
  if (delta) {
    if (delta_dtype != dtype && delta_dtype != MOE_F32) return MOE_EINVAL;
    if (!rows_ok(delta, m, ldd, d, delta_dtype == MOE_F32 ? 4 : 8) || !rows_ok(h_out, m, ldo, d)) return MOE_EINVAL;
  } else if (h_out) {
    return MOE_EINVAL;
  }
  if (m > 0 && !y && !y8) return MOE_EINVAL;
  if (y && !rows_ok(y, m, ldy, d)) return MOE_EINVAL;
  if (y8 && (!aligned(y8, 8) || ldy8 < d || ldy8 % 8 || ldy8 >= (int64_t{1} << 36) || !scale || !aligned(scale, 4)))
    return MOE_EINVAL;
  if (!y8 && scale) return MOE_EINVAL;
  if (m == 0) return MOE_OK;
  NormParams p;
  p.h = h, p.ldh = ldh, p.delta = delta, p.ldd = ldd, p.weight = weight, p.h_out = h_out, p.ldo = ldo;
  p.y = y, p.ldy = ldy, p.y8 = static_cast<uint8_t*>(y8), p.ldy8 = ldy8, p.scale = scale;
  p.m = m, p.d = d, p.eps = eps;
  return status(launch_norm(dtype == MOE_BF16, delta_dtype == MOE_F32, p, static_cast<cudaStream_t>(stream)));
}

extern "C" moe_status moe_rmsnorm_grad(int dtype, const void* h, int64_t ldh, const void* dy, int64_t lddy,
                                       const void* dres, int64_t lddres, const void* weight, float eps, int m, int d,
                                       void* dh, int64_t lddh, float* dweight, void* workspace, uint64_t workspace_bytes,
                                       void* stream) {
  if (!norm_ok(dtype, m, d, weight, eps) || !rows_ok(h, m, ldh, d) || !rows_ok(dy, m, lddy, d) || !rows_ok(dh, m, lddh, d))
    return MOE_EINVAL;
  if (dres && !rows_ok(dres, m, lddres, d)) return MOE_EINVAL;
  const uint64_t need = 4ull * d * (m < kNormParts ? m : kNormParts);
  if (dweight && (!weight || !aligned(dweight, 16) || !aligned(workspace, 16) || (m > 0 && !workspace) || workspace_bytes < need))
    return MOE_EINVAL;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (m == 0) return status(!dweight || cudaMemsetAsync(dweight, 0, sizeof(float) * d, s) == cudaSuccess);
  NormGradParams p;
  p.h = h, p.ldh = ldh, p.dy = dy, p.lddy = lddy, p.dres = dres, p.lddres = lddres, p.weight = weight;
  p.dh = dh, p.lddh = lddh, p.dweight = dweight, p.part = dweight ? static_cast<float*>(workspace) : nullptr;
  p.m = m, p.d = d, p.eps = eps;
  return status(launch_norm_grad(dtype == MOE_BF16, p, s));
}

extern "C" moe_status moe_grouped_mm8(const void* x, int64_t ldx, const float* sx, int m, const int32_t* offsets,
                                      int n_experts, const void* w, const float* sw, int n, int k, void* y, int64_t ldy,
                                      int out_dtype, void* stream) {
  if (!product8_ok(x, ldx, sx, m, offsets, n_experts, w, sw, k) || n < 8 || n > kMaxSide || n % 8) return MOE_EINVAL;
  if ((!is16(out_dtype) && out_dtype != MOE_F32) || !rows_ok(y, m, ldy, n)) return MOE_EINVAL;
  if (m == 0) return MOE_OK;
  Mm8Params p;
  p.x = static_cast<const uint8_t*>(x), p.ldx = ldx, p.sx = sx, p.offsets = offsets, p.E = n_experts, p.m = m;
  p.w = static_cast<const uint8_t*>(w), p.sw = sw, p.n = n, p.k = k, p.y = y, p.ldy = ldy, p.out = out_dtype;
  return status(launch_grouped8(false, p, static_cast<cudaStream_t>(stream)));
}

extern "C" moe_status moe_grouped_geglu8(int gelu_variant, const void* x, int64_t ldx, const float* sx, int m,
                                         const int32_t* offsets, int n_experts, const void* w, const float* sw, int f, int k,
                                         void* a, int64_t lda, float* sa, void* stream) {
  if (!gelu_ok(gelu_variant) || !product8_ok(x, ldx, sx, m, offsets, n_experts, w, sw, k)) return MOE_EINVAL;
  if (f < 16 || f > kMaxSide / 2 || f % 16 || !rows_ok(a, m, lda, f, 16) || (m > 0 && !sa) || !aligned(sa, 4)) return MOE_EINVAL;
  if (m == 0) return MOE_OK;
  Mm8Params p;
  p.x = static_cast<const uint8_t*>(x), p.ldx = ldx, p.sx = sx, p.offsets = offsets, p.E = n_experts, p.m = m;
  p.w = static_cast<const uint8_t*>(w), p.sw = sw, p.n = 2 * f, p.k = k, p.y = a, p.ldy = lda, p.sa = sa;
  p.gelu = gelu_variant;
  return status(launch_grouped8(true, p, static_cast<cudaStream_t>(stream)));
}

extern "C" moe_status moe_token_layer(int dtype, int gelu_variant, const void* x, int64_t ldx, int t, const int32_t* ids,
                                      const float* gates, int top_k, int n_experts, const moe_ffn_weights* routed,
                                      const moe_ffn_weights* shared, int d, int f, int f_shared, void* y, int64_t ldy,
                                      int out_dtype, void* workspace, uint64_t workspace_bytes, void* stream) {
  if (!is16(dtype) || !gelu_ok(gelu_variant) || (out_dtype != dtype && out_dtype != MOE_F32)) return MOE_EINVAL;
  if (t < 0 || t > kLayerTokens || top_k < 1 || top_k > kLayerTopK || n_experts < 1 || n_experts > kMaxExperts || !routed)
    return MOE_EINVAL;
  const auto side_ok = [](int v, int most) { return v >= 16 && v <= most && v % 16 == 0; };
  if (!side_ok(d, kMaxSide) || !side_ok(f, kMaxSide / 2) || (shared ? !side_ok(f_shared, kMaxSide / 2) : f_shared != 0))
    return MOE_EINVAL;
  const bool eight = routed->gate_up_scale != nullptr;
  for (const moe_ffn_weights* w : {routed, shared}) {
    if (!w) continue;
    if (!w->gate_up || !w->down || !aligned(w->gate_up, 16) || !aligned(w->down, 16)) return MOE_EINVAL;
    if ((w->gate_up_scale != nullptr) != eight || (w->down_scale != nullptr) != eight || !aligned(w->gate_up_scale, 4) ||
        !aligned(w->down_scale, 4))
      return MOE_EINVAL;
  }
  if (!rows_ok(x, t, ldx, d) || !rows_ok(y, t, ldy, d) || !aligned(ids, 4) || !aligned(gates, 4)) return MOE_EINVAL;
  if (t == 0) return MOE_OK;
  if (!ids || !gates || !workspace || !aligned(workspace, 16)) return MOE_EINVAL;
  if (workspace_bytes < 2ull * t * (static_cast<uint64_t>(top_k) * f + f_shared)) return MOE_EINVAL;
  LayerParams p;
  p.x = static_cast<const uint16_t*>(x), p.ldx = ldx, p.ids = ids, p.gates = gates;
  p.t = t, p.k = top_k, p.E = n_experts, p.d = d, p.f = f, p.fs = f_shared;
  p.routed = {routed->gate_up, routed->down, routed->gate_up_scale, routed->down_scale};
  if (shared) p.shared = {shared->gate_up, shared->down, shared->gate_up_scale, shared->down_scale};
  p.a = static_cast<uint16_t*>(workspace), p.y = y, p.ldy = ldy;
  p.bf16 = dtype == MOE_BF16, p.out_f32 = out_dtype == MOE_F32, p.gelu = gelu_variant;
  return status(launch_layer(eight, p, static_cast<cudaStream_t>(stream)));
}
