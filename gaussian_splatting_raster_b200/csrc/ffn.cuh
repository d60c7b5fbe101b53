// Feed-forward block over rows: the arguments its kernels share and the activation.
//
//   a = x Wg^T,  u = x Wu^T,  h = act(a) * u,  y = h Wd^T          x [M, D], Wg, Wu [F, D]
//   without Wg:  a = x Wu^T,  h = act(a)                            Wd [O, F], y [M, O]
//   gradients:   dh = dy Wd,  da = dh u act'(a),  du = dh act(a)    (u = 1 without Wg)
//                dx = da Wg + du Wu,  dWg = da^T x,  dWu = du^T x,  dWd = dy^T h
//
// "Research Proposal: Renderer Score Tokens for Recurrent Gaussian Splatting", Final Token and
// Updater: a shared linear - GELU - linear projection of the token rows z_g. The rows are as many
// as there are Gaussians (up to millions), their widths small (tokens have 12 to 57 values, the
// attribute render takes at most 64 channels), so all three products of a row tile stay on chip:
// h and its gradients are never written to memory.
#pragma once

#include "rows.cuh"

namespace splat {
namespace rows {

constexpr int kMaxWidth = 128;   // D and O
constexpr int kMaxHidden = 1024; // F
constexpr int kChunk = 64;       // hidden units taken at a time

struct FfnArgs {
  const void *x, *wg, *wu, *wd, *dy;
  void *y, *dx, *dwg, *dwu, *dwd;
  long long ldx, ldy, lddy, lddx;
  int M, D, F, O;
  float* part;   // [splits] partial weight gradients, fp32: dWg, dWu [F, D] each, dWd^T [F, O]
  int splits;
  unsigned* dy_max;  // fp16 gradients: [kMaxParts] largest finite |dy|, by CTAs
};
constexpr int kMaxParts = 592;

// 2^v and 1 / v of the special function unit: relative errors below 2^-22 and 2^-23.
__device__ __forceinline__ float ex2_fast(float v) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float rcp_fast(float v) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
  return r;
}

// Phi(a), and e = e^{-a^2/2}, which the density shares. Phi(-|a|) = r P(r) e with
// r = 1 / (1 + 0.375 z), z = |a| / sqrt 2: erfc(z) e^{z^2} / 2 is smooth in r, and P of degree 8 (a
// minimax fit of the relative error over z in [0, 9.45], weights from a linear program on Chebyshev
// nodes) is off by 1.2e-8 of it. So Phi keeps its digits on the left, where 1 + erf cancels (57 %
// off at a = -5.5, zero from -5.7 on): rounding adds at most (12 + 2 a^2) 2^-24 of Phi(-|a|), most
// of it the exponent's. e is zero below 2^-126.
__device__ __forceinline__ float normal_cdf(float a, float& e) {
  const float r = rcp_fast(fmaf(0.375f * 0.70710678118654752f, fabsf(a), 1.0f));
  float q = fmaf(r, 0.030848359689116478f, -0.14403793215751648f);
  q = fmaf(q, r, 0.21694736182689667f);
  q = fmaf(q, r, -0.11553873866796494f);
  q = fmaf(q, r, 0.13742241263389587f);
  q = fmaf(q, r, 0.06051934137940407f);
  q = fmaf(q, r, 0.10271524637937546f);
  q = fmaf(q, r, 0.10531674325466156f);
  q = fmaf(q, r, 0.10580720752477646f);
  e = ex2_fast(a * a * -0.72134752044448170f);
  q = q * r * e;
  return a >= 0.0f ? 1.0f - q : q;
}

// act(a) and act'(a) in fp32.
//   silu: a s, s (1 + a (1 - s)) with s = 1 / (1 + e^-a)
//   gelu: a Phi(a), Phi(a) + a phi(a), Phi the normal distribution function, phi its density
template <int ACT>
__device__ __forceinline__ float act_of(float a) {
  if (ACT == SPLAT_ACT_SILU) return a / (1.0f + expf(-a));
  float e;
  return a * normal_cdf(a, e);
}

template <int ACT>
__device__ __forceinline__ float act_and_slope(float a, float& slope) {
  if (ACT == SPLAT_ACT_SILU) {
    const float s = 1.0f / (1.0f + expf(-a));
    slope = s * fmaf(a, 1.0f - s, 1.0f);
    return a * s;
  }
  float e;
  const float cdf = normal_cdf(a, e);
  slope = fmaf(a * 0.3989422804014327f, e, cdf);
  return a * cdf;
}

// tensor-core kernels (ffn_tc.cu; bf16 and fp16): bytes of the packed weights, row splits of the
// weight gradients, and the kernels but for the splits' sum
size_t ffn_tc_image_bytes(int D, int F, int O, bool gated);
int ffn_tc_splits(long long M, int D, int F, int O);
int ffn_tc_parts(int D, int F, int O);  // partial sums a split leaves
int ffn_tc_run(const FfnArgs& f, int dtype, int act, bool backward, void* img, cudaStream_t st);

}  // namespace rows
}  // namespace splat
