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
};

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

// act(a) and act'(a) in fp32.
//   silu: a s, s (1 + a (1 - s)) with s = 1 / (1 + e^-a)
//   gelu: a Phi(a), Phi(a) + a phi(a), Phi the normal distribution function, phi its density
template <int ACT>
__device__ __forceinline__ float act_of(float a) {
  if (ACT == SPLAT_ACT_SILU) return a / (1.0f + expf(-a));
  return 0.5f * a * (1.0f + erff(a * 0.70710678118654752f));
}

template <int ACT>
__device__ __forceinline__ float act_and_slope(float a, float& slope) {
  if (ACT == SPLAT_ACT_SILU) {
    const float s = 1.0f / (1.0f + expf(-a));
    slope = s * fmaf(a, 1.0f - s, 1.0f);
    return a * s;
  }
  const float cdf = 0.5f * (1.0f + erff(a * 0.70710678118654752f));
  slope = fmaf(a * 0.3989422804014327f, expf(-0.5f * a * a), cdf);
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
