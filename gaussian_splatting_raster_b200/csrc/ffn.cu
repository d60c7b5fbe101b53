// Feed-forward block over rows: entry points, and the kernels on the fp32 lanes.
//
// One CTA takes a tile of rows through all products: its rows stay in shared memory while the
// hidden units pass in chunks of 64 (their weights staged per chunk, transposed so that every
// inner product reads along rows). Bound by the fp32 lanes: 2 M F (2 D + O) operations against
// 4 M (D + O) bytes, which at D = 57, F = 256, O = 64 is 188 operations a byte.
#include "ffn.cuh"

namespace splat {
namespace rows {
namespace {

constexpr int kT = 256;  // 16 x 16 threads: thread (tx, ty) has rows ty * RT .., units tx * 4 ..

// rows [r0, r0 + R) of src (cols columns) transposed into dst[k * ld + r]; rows >= M are zero
template <typename T, int R>
__device__ __forceinline__ void stage_rows(const T* src, long long lds, long long r0, int M,
                                           int cols, float* dst, int ld) {
  for (int i = threadIdx.x; i < R * cols; i += kT) {
    const int r = i / cols, k = i - r * cols;
    dst[k * ld + r] = r0 + r < M ? to_f<T>(src[(r0 + r) * lds + k]) : 0.0f;
  }
}

// units [f0, f0 + 64) of w [F, D] transposed into dst[k * ld + j]; units >= F are zero
template <typename T>
__device__ __forceinline__ void stage_units(const T* w, int F, int D, int f0, float* dst, int ld) {
  for (int i = threadIdx.x; i < kChunk * D; i += kT) {
    const int j = i / D, k = i - j * D;
    dst[k * ld + j] = f0 + j < F ? to_f<T>(w[(size_t)(f0 + j) * D + k]) : 0.0f;
  }
}

// units [f0, f0 + 64) of wd [O, F]: dst[o * ldo + j * ldj]
template <typename T>
__device__ __forceinline__ void stage_down(const T* wd, int F, int O, int f0, float* dst, int ldo,
                                           int ldj) {
  for (int i = threadIdx.x; i < kChunk * O; i += kT) {
    const int o = i / kChunk, j = i % kChunk;
    dst[o * ldo + j * ldj] = f0 + j < F ? to_f<T>(wd[(size_t)o * F + f0 + j]) : 0.0f;
  }
}

// acc[i][j] += sum_k rowsT[k][ty RT + i] w[k][tx 4 + j]
template <int RT>
__device__ __forceinline__ void product(const float* rowsT, int ldr, const float* w, int ldw,
                                        int K, float (&acc)[RT][4]) {
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
#pragma unroll 4
  for (int k = 0; k < K; ++k) {
    float xr[RT], wv[4];
#pragma unroll
    for (int i = 0; i < RT; i += 4)
      *reinterpret_cast<float4*>(xr + i) =
          *reinterpret_cast<const float4*>(rowsT + k * ldr + ty * RT + i);
    *reinterpret_cast<float4*>(wv) = *reinterpret_cast<const float4*>(w + k * ldw + tx * 4);
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(xr[i], wv[j], acc[i][j]);
  }
}

template <int N, int M>
__device__ __forceinline__ void clear(float (&a)[N][M]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < M; ++j) a[i][j] = 0.0f;
}

constexpr int kFwdRows = 128;
constexpr int kFwdLd = kFwdRows + 4;
constexpr int kGuLd = 2 * kChunk + 4;
constexpr int kLd = 64 + 4;

int fwd_smem(int D, int O) {
  const int Op = O <= 64 ? 64 : 128;
  return 4 * (D * kFwdLd + D * kGuLd + kChunk * (Op + 4) + kChunk * kFwdLd);
}

template <typename T, int ACT, bool GATED, int NO>  // NO: 64-wide pieces of O
__global__ void __launch_bounds__(kT, 1) k_ffn(FfnArgs p) {
  extern __shared__ __align__(16) float sm[];
  constexpr int RT = kFwdRows / 16, ldo = NO * 64 + 4;
  float* Xs = sm;                          // [D][132]
  float* Ws = Xs + p.D * kFwdLd;           // [D][132]: 64 gate units, 64 up units
  float* Ds = Ws + p.D * kGuLd;            // [64][ldo]
  float* Hs = Ds + kChunk * ldo;           // [64][132]
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const long long r0 = (long long)blockIdx.x * kFwdRows;
  const T *x = (const T*)p.x, *wg = (const T*)p.wg, *wu = (const T*)p.wu, *wd = (const T*)p.wd;
  stage_rows<T, kFwdRows>(x, p.ldx, r0, p.M, p.D, Xs, kFwdLd);
  for (int i = threadIdx.x; i < kChunk * ldo; i += kT) Ds[i] = 0.0f;  // columns >= O stay zero
  float yv[NO][RT][4];
#pragma unroll
  for (int n = 0; n < NO; ++n) clear(yv[n]);
  for (int f0 = 0; f0 < p.F; f0 += kChunk) {
    __syncthreads();
    if (GATED) stage_units(wg, p.F, p.D, f0, Ws, kGuLd);
    stage_units(wu, p.F, p.D, f0, Ws + (GATED ? kChunk : 0), kGuLd);
    stage_down(wd, p.F, p.O, f0, Ds, 1, ldo);
    __syncthreads();
    float a[RT][4], u[RT][4];
    clear(a);
    product<RT>(Xs, kFwdLd, Ws, kGuLd, p.D, a);
    if (GATED) {
      clear(u);
      product<RT>(Xs, kFwdLd, Ws + kChunk, kGuLd, p.D, u);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < RT; i += 4) {
        float h[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          h[q] = act_of<ACT>(a[i + q][j]);
          if (GATED) h[q] *= u[i + q][j];
        }
        *reinterpret_cast<float4*>(Hs + (tx * 4 + j) * kFwdLd + ty * RT + i) =
            *reinterpret_cast<float4*>(h);
      }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NO; ++n) product<RT>(Hs, kFwdLd, Ds + n * 64, ldo, kChunk, yv[n]);
  }
  T* y = (T*)p.y;
#pragma unroll
  for (int n = 0; n < NO; ++n)
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int o = n * 64 + tx * 4 + j;
        const long long r = r0 + ty * RT + i;
        if (o < p.O && r < p.M) y[r * p.ldy + o] = from_f<T>(yv[n][i][j]);
      }
}

// ---------------------------------------------------------------------------------------------
// a few rows
// ---------------------------------------------------------------------------------------------
// Bound by latency: the weights have to come from L2 once. A cluster of eight CTAs shares kFew
// rows; each CTA takes every eighth group of hidden units, a warp four units at a time (its lanes
// along D, then one sum over the warp for each), and forms its part of y from them; the first CTA
// adds the eight parts in order through distributed shared memory. x and the weights are read in
// whole rows by neighbouring lanes whatever their alignment.
constexpr int kCluster = 8;
constexpr int kFew = 4;        // rows of a cluster
constexpr int kFewThreads = 256;
constexpr int kFewSingle = 18;   // up to one cluster a row fills the machine
constexpr int kFewRows = 128;    // most rows taken this way

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <typename T, int ACT, bool GATED, int R>
__global__ void __cluster_dims__(kCluster, 1, 1) __launch_bounds__(kFewThreads)
k_ffn_few(FfnArgs p) {
  constexpr int kUnits = kMaxHidden / kCluster;  // most units of a CTA
  __shared__ float s_h[R][kUnits];
  __shared__ float s_y[kCluster][R][kMaxWidth];  // (the first CTA's is used)
  // (the wait below: every CTA of the cluster has started before its shared memory is written)
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const int rank = blockIdx.x % kCluster, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long r0 = (long long)(blockIdx.x / kCluster) * R;
  const T *x = (const T*)p.x, *wg = (const T*)p.wg, *wu = (const T*)p.wu, *wd = (const T*)p.wd;
  const int per = (p.F + kCluster - 1) / kCluster;
  const int f0 = min(p.F, rank * per), n = min(p.F, f0 + per) - f0;
  float xr[R][4];  // columns lane + 32 k
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int d = lane + 32 * k;
      xr[i][k] = d < p.D && r0 + i < p.M ? to_f<T>(x[(r0 + i) * p.ldx + d]) : 0.0f;
    }
  constexpr int U = 4;
  for (int j0 = warp * U; j0 < n; j0 += kFewThreads / 32 * U) {
    float wa[U][4], wb[U][4];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int d = lane + 32 * k;
        const bool ok = d < p.D && j0 + u < n;
        const size_t at = (size_t)(f0 + j0 + u) * p.D + d;
        wa[u][k] = ok ? to_f<T>((GATED ? wg : wu)[at]) : 0.0f;
        if (GATED) wb[u][k] = ok ? to_f<T>(wu[at]) : 0.0f;
      }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < R; ++i) {
        float a = 0.0f, b = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          a = fmaf(xr[i][k], wa[u][k], a);
          if (GATED) b = fmaf(xr[i][k], wb[u][k], b);
        }
        a = warp_sum(a);
        float h = act_of<ACT>(a);
        if (GATED) h *= warp_sum(b);
        if (lane == 0 && j0 + u < n) s_h[i][j0 + u] = to_f<T>(from_f<T>(h));
      }
  }
  __syncthreads();
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  // this CTA's part of y, written into the first CTA's shared memory
  float* dst = &s_y[rank][0][0];
  uint64_t remote;
  asm("mapa.u64 %0, %1, 0;" : "=l"(remote) : "l"(dst));
  for (int o = warp; o < p.O; o += kFewThreads / 32) {
    float acc[R];
#pragma unroll
    for (int i = 0; i < R; ++i) acc[i] = 0.0f;
    for (int j = lane; j < n; j += 32) {
      const float w = to_f<T>(wd[(size_t)o * p.F + f0 + j]);
#pragma unroll
      for (int i = 0; i < R; ++i) acc[i] = fmaf(s_h[i][j], w, acc[i]);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) {
      acc[i] = warp_sum(acc[i]);
      if (lane == 0) reinterpret_cast<float*>(remote)[i * kMaxWidth + o] = acc[i];
    }
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
  if (rank != 0) return;
  T* y = (T*)p.y;
  for (int q = threadIdx.x; q < R * p.O; q += kFewThreads) {
    const int i = q / p.O, o = q - i * p.O;
    float v = 0.0f;
#pragma unroll
    for (int c = 0; c < kCluster; ++c) v += s_y[c][i][o];
    if (r0 + i < p.M) y[(r0 + i) * p.ldy + o] = from_f<T>(v);
  }
}

// a, u, dh of one 64-row tile and chunk, turned into da, du (and h) in place
template <int ACT, bool GATED>
__device__ __forceinline__ void hidden_grads(const float* Xs, const float* Ys, const float* Ws,
                                             const float* Ds, int D, int O, float (&da)[4][4],
                                             float (&du)[4][4], float (&h)[4][4]) {
  float a[4][4], u[4][4], dh[4][4];
  clear(a);
  clear(dh);
  product<4>(Xs, kLd, Ws, kGuLd, D, a);
  if (GATED) {
    clear(u);
    product<4>(Xs, kLd, Ws + kChunk, kGuLd, D, u);
  }
  product<4>(Ys, kLd, Ds, kLd, O, dh);
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float s;
      const float f = act_and_slope<ACT>(a[i][j], s);
      h[i][j] = GATED ? f * u[i][j] : f;
      da[i][j] = GATED ? dh[i][j] * u[i][j] * s : dh[i][j] * s;
      du[i][j] = GATED ? dh[i][j] * f : 0.0f;
    }
}

int dx_smem(int D, int O) { return 4 * (D * kLd + O * kLd + D * kGuLd + O * kLd + 2 * 64 * kLd); }
int dw_smem(int D, int O) { return 4 * (D * kLd + O * kLd + D * kGuLd + O * kLd + 3 * 64 * kLd); }

// dx of one 64-row tile: all chunks in turn
template <typename T, int ACT, bool GATED>
__global__ void __launch_bounds__(kT, 1) k_ffn_dx(FfnArgs p) {
  extern __shared__ __align__(16) float sm[];
  float* Xs = sm;                    // [D][68]
  float* Ys = Xs + p.D * kLd;        // [O][68]
  float* Ws = Ys + p.O * kLd;        // [D][132]
  float* Ds = Ws + p.D * kGuLd;      // [O][68]
  float* As = Ds + p.O * kLd;        // [64 units][68 rows] da, then du
  float* Us = As + kChunk * kLd;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const long long r0 = (long long)blockIdx.x * 64;
  const T *wg = (const T*)p.wg, *wu = (const T*)p.wu, *wd = (const T*)p.wd;
  stage_rows<T, 64>((const T*)p.x, p.ldx, r0, p.M, p.D, Xs, kLd);
  stage_rows<T, 64>((const T*)p.dy, p.lddy, r0, p.M, p.O, Ys, kLd);
  float acc[8][4];  // columns tx + 16 c, rows ty * 4 + i
  clear(acc);
  for (int f0 = 0; f0 < p.F; f0 += kChunk) {
    __syncthreads();
    if (GATED) stage_units(wg, p.F, p.D, f0, Ws, kGuLd);
    stage_units(wu, p.F, p.D, f0, Ws + (GATED ? kChunk : 0), kGuLd);
    stage_down(wd, p.F, p.O, f0, Ds, kLd, 1);
    __syncthreads();
    float da[4][4], du[4][4], h[4][4];
    hidden_grads<ACT, GATED>(Xs, Ys, Ws, Ds, p.D, p.O, da, du, h);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      *reinterpret_cast<float4*>(As + (tx * 4 + j) * kLd + ty * 4) =
          make_float4(da[0][j], da[1][j], da[2][j], da[3][j]);
      if (GATED)
        *reinterpret_cast<float4*>(Us + (tx * 4 + j) * kLd + ty * 4) =
            make_float4(du[0][j], du[1][j], du[2][j], du[3][j]);
    }
    __syncthreads();
    for (int f = 0; f < kChunk; ++f) {
      float av[4], uv[4];
      *reinterpret_cast<float4*>(av) = *reinterpret_cast<const float4*>(As + f * kLd + ty * 4);
      if (GATED)
        *reinterpret_cast<float4*>(uv) = *reinterpret_cast<const float4*>(Us + f * kLd + ty * 4);
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const int d = tx + 16 * c;
        if (d >= p.D) break;
        const float g = Ws[d * kGuLd + f], v = GATED ? Ws[d * kGuLd + kChunk + f] : 0.0f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          acc[c][i] = fmaf(av[i], g, acc[c][i]);
          if (GATED) acc[c][i] = fmaf(uv[i], v, acc[c][i]);
        }
      }
    }
  }
  T* dx = (T*)p.dx;
#pragma unroll
  for (int c = 0; c < 8; ++c)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = tx + 16 * c;
      const long long r = r0 + ty * 4 + i;
      if (d < p.D && r < p.M) dx[r * p.lddx + d] = from_f<T>(acc[c][i]);
    }
}

// partial weight gradients of chunk blockIdx.x over the row tiles blockIdx.y, + splits, ...
template <typename T, int ACT, bool GATED>
__global__ void __launch_bounds__(kT, 1) k_ffn_dw(FfnArgs p) {
  extern __shared__ __align__(16) float sm[];
  float* Xs = sm;
  float* Ys = Xs + p.D * kLd;
  float* Ws = Ys + p.O * kLd;
  float* Ds = Ws + p.D * kGuLd;
  float* As = Ds + p.O * kLd;        // [64 rows][68 units] da, du, h
  float* Us = As + 64 * kLd;
  float* Hs = Us + 64 * kLd;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int f0 = blockIdx.x * kChunk;
  const T *wg = (const T*)p.wg, *wu = (const T*)p.wu, *wd = (const T*)p.wd;
  if (GATED) stage_units(wg, p.F, p.D, f0, Ws, kGuLd);
  stage_units(wu, p.F, p.D, f0, Ws + (GATED ? kChunk : 0), kGuLd);
  stage_down(wd, p.F, p.O, f0, Ds, kLd, 1);
  float ga[8][4], gu[8][4], gd[8][4];  // rows (of D or O) ty + 16 c, units tx * 4 + j
  clear(ga);
  clear(gu);
  clear(gd);
  const int tiles = (int)(((long long)p.M + 63) / 64);
  for (int t = blockIdx.y; t < tiles; t += p.splits) {
    __syncthreads();
    stage_rows<T, 64>((const T*)p.x, p.ldx, (long long)t * 64, p.M, p.D, Xs, kLd);
    stage_rows<T, 64>((const T*)p.dy, p.lddy, (long long)t * 64, p.M, p.O, Ys, kLd);
    __syncthreads();
    float da[4][4], du[4][4], h[4][4];
    hidden_grads<ACT, GATED>(Xs, Ys, Ws, Ds, p.D, p.O, da, du, h);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int at = (ty * 4 + i) * kLd + tx * 4;
      *reinterpret_cast<float4*>(As + at) = *reinterpret_cast<float4*>(da[i]);
      if (GATED) *reinterpret_cast<float4*>(Us + at) = *reinterpret_cast<float4*>(du[i]);
      *reinterpret_cast<float4*>(Hs + at) = *reinterpret_cast<float4*>(h[i]);
    }
    __syncthreads();
    for (int r = 0; r < 64; r += 4) {
      float av[4][4], uv[4][4], hv[4][4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int at = (r + q) * kLd + tx * 4;
        *reinterpret_cast<float4*>(av[q]) = *reinterpret_cast<const float4*>(As + at);
        if (GATED) *reinterpret_cast<float4*>(uv[q]) = *reinterpret_cast<const float4*>(Us + at);
        *reinterpret_cast<float4*>(hv[q]) = *reinterpret_cast<const float4*>(Hs + at);
      }
#pragma unroll
      for (int c = 0; c < 8; ++c) {
        const int k = ty + 16 * c;
        if (k < p.D) {
          float xv[4];
          *reinterpret_cast<float4*>(xv) = *reinterpret_cast<const float4*>(Xs + k * kLd + r);
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              ga[c][j] = fmaf(xv[q], av[q][j], ga[c][j]);
              if (GATED) gu[c][j] = fmaf(xv[q], uv[q][j], gu[c][j]);
            }
        }
        if (k < p.O) {
          float yv[4];
          *reinterpret_cast<float4*>(yv) = *reinterpret_cast<const float4*>(Ys + k * kLd + r);
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int j = 0; j < 4; ++j) gd[c][j] = fmaf(yv[q], hv[q][j], gd[c][j]);
        }
      }
    }
  }
  const size_t FD = (size_t)p.F * p.D;
  float* part = p.part + blockIdx.y * ((GATED ? 2 : 1) * FD + (size_t)p.O * p.F);
#pragma unroll
  for (int c = 0; c < 8; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = ty + 16 * c, f = f0 + tx * 4 + j;
      if (f >= p.F) continue;
      if (k < p.D) {
        part[(size_t)f * p.D + k] = ga[c][j];
        if (GATED) part[FD + (size_t)f * p.D + k] = gu[c][j];
      }
      if (k < p.O) part[(GATED ? 2 : 1) * FD + (size_t)f * p.O + k] = gd[c][j];
    }
}

// The splits' partial gradients: a CTA has 32 sums, each of its warps every eighth split of all of
// them, the warps' sums added in order.
template <typename T, bool GATED>
__global__ void __launch_bounds__(kT) k_ffn_join(FfnArgs p) {
  __shared__ float s_sum[kT / 32][32];
  const size_t FD = (size_t)p.F * p.D, n = (GATED ? 2 : 1) * FD + (size_t)p.O * p.F;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t i = (size_t)blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (i < n) {
#pragma unroll 4
    for (int k = warp; k < p.splits; k += kT / 32) s += p.part[k * n + i];
  }
  s_sum[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || i >= n) return;
  s = 0.0f;
#pragma unroll
  for (int w = 0; w < kT / 32; ++w) s += s_sum[w][lane];
  const size_t down = i - (GATED ? 2 : 1) * FD;  // of dWd^T, when i is past the others
  if (GATED && i < FD) {
    if (p.dwg) ((T*)p.dwg)[i] = from_f<T>(s);
  } else if (i < (GATED ? 2 : 1) * FD) {
    if (p.dwu) ((T*)p.dwu)[GATED ? i - FD : i] = from_f<T>(s);
  } else if (p.dwd) {
    ((T*)p.dwd)[down % p.O * p.F + down / p.O] = from_f<T>(s);
  }
}

int last_error() {
  return cudaGetLastError() == cudaSuccess ? SPLAT_OK : SPLAT_ERR_CUDA;
}

template <typename K>
bool allow_smem(K kernel, int bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) ==
         cudaSuccess;
}

// row splits of the weight gradients: enough CTAs for the machine, and at most 8,192 rows a split
// (an fp32 sum of n products is off by about sqrt(n) 2^-25 of its size)
int dw_splits(long long M, int F) {
  const int chunks = (F + kChunk - 1) / kChunk;
  const long long tiles = (M + 63) / 64;
  long long s = (148 + chunks - 1) / chunks;
  if (s < (tiles + 127) / 128) s = (tiles + 127) / 128;
  if (s > tiles) s = tiles;
  if (s > 65535) s = 65535;  // the grid's limit
  return (int)(s < 1 ? 1 : s);
}

template <typename T, int ACT, bool GATED>
int run_few(const FfnArgs& p, cudaStream_t st) {
  if (p.M <= kFewSingle) {
    k_ffn_few<T, ACT, GATED, 1><<<p.M * kCluster, kFewThreads, 0, st>>>(p);
  } else {
    k_ffn_few<T, ACT, GATED, kFew>
        <<<(p.M + kFew - 1) / kFew * kCluster, kFewThreads, 0, st>>>(p);
  }
  return last_error();
}

template <typename T, int ACT, bool GATED>
int run_forward(const FfnArgs& p, cudaStream_t st) {
  const int smem = fwd_smem(p.D, p.O);
  const unsigned grid = (unsigned)(((long long)p.M + kFwdRows - 1) / kFwdRows);
  if (p.O <= 64) {
    if (!allow_smem(k_ffn<T, ACT, GATED, 1>, smem)) return SPLAT_ERR_CUDA;
    k_ffn<T, ACT, GATED, 1><<<grid, kT, smem, st>>>(p);
  } else {
    if (!allow_smem(k_ffn<T, ACT, GATED, 2>, smem)) return SPLAT_ERR_CUDA;
    k_ffn<T, ACT, GATED, 2><<<grid, kT, smem, st>>>(p);
  }
  return last_error();
}

template <typename T, bool GATED> int run_join(const FfnArgs& p, cudaStream_t st) {
  const size_t n = ((GATED ? 2 : 1) * (size_t)p.D + p.O) * p.F;
  k_ffn_join<T, GATED><<<(unsigned)((n + 31) / 32), kT, 0, st>>>(p);
  return last_error();
}

template <typename T, int ACT, bool GATED>
int run_backward(const FfnArgs& p, cudaStream_t st) {
  if (p.dx && p.M > 0) {
    const int smem = dx_smem(p.D, p.O);
    if (!allow_smem(k_ffn_dx<T, ACT, GATED>, smem)) return SPLAT_ERR_CUDA;
    k_ffn_dx<T, ACT, GATED><<<(unsigned)(((long long)p.M + 63) / 64), kT, smem, st>>>(p);
  }
  if (p.dwg || p.dwu || p.dwd) {
    const int smem = dw_smem(p.D, p.O);
    if (!allow_smem(k_ffn_dw<T, ACT, GATED>, smem)) return SPLAT_ERR_CUDA;
    const dim3 grid((p.F + kChunk - 1) / kChunk, p.splits);
    k_ffn_dw<T, ACT, GATED><<<grid, kT, smem, st>>>(p);
    return run_join<T, GATED>(p, st);
  }
  return last_error();
}

// A few rows by the clusters; otherwise fp32 on the fp32 lanes, bf16 and fp16 on the tensor cores.
template <typename T, int ACT, bool GATED>
int run(FfnArgs& p, int dtype, bool backward, void* scratch, cudaStream_t st) {
  if (!backward && p.M <= kFewRows) return run_few<T, ACT, GATED>(p, st);
  if constexpr (sizeof(T) == 4) {
    p.part = (float*)scratch;
    p.splits = dw_splits(p.M, p.F);
    return backward ? run_backward<T, ACT, GATED>(p, st) : run_forward<T, ACT, GATED>(p, st);
  } else {
    p.part = (float*)((char*)scratch + ffn_tc_image_bytes(p.D, p.F, p.O, GATED));
    p.splits = ffn_tc_splits(p.M, p.F);
    const int rc = ffn_tc_run(p, dtype, ACT, backward, scratch, st);
    if (rc != SPLAT_OK || !(p.dwg || p.dwu || p.dwd)) return rc;
    return run_join<T, GATED>(p, st);
  }
}

template <typename T>
int run_type(FfnArgs& p, int dtype, int act, bool backward, void* scratch, cudaStream_t st) {
  if (act == SPLAT_ACT_SILU)
    return p.wg ? run<T, SPLAT_ACT_SILU, true>(p, dtype, backward, scratch, st)
                : run<T, SPLAT_ACT_SILU, false>(p, dtype, backward, scratch, st);
  return p.wg ? run<T, SPLAT_ACT_GELU, true>(p, dtype, backward, scratch, st)
              : run<T, SPLAT_ACT_GELU, false>(p, dtype, backward, scratch, st);
}

int dispatch(FfnArgs& p, int dtype, int act, bool backward, void* scratch, cudaStream_t st) {
  if (dtype == SPLAT_F32) return run_type<float>(p, dtype, act, backward, scratch, st);
  if (dtype == SPLAT_BF16) return run_type<__nv_bfloat16>(p, dtype, act, backward, scratch, st);
  return run_type<__half>(p, dtype, act, backward, scratch, st);
}

int check_sizes(int M, int D, int F, int O, int dtype, int act) {
  if (!elem_size(dtype) || (act != SPLAT_ACT_SILU && act != SPLAT_ACT_GELU) || M < 0 || D < 1 ||
      F < 1 || O < 1)
    return SPLAT_ERR_INVALID_ARG;
  if (D > kMaxWidth || O > kMaxWidth || F > kMaxHidden) return SPLAT_ERR_CAPACITY;
  return SPLAT_OK;
}

}  // namespace
}  // namespace rows
}  // namespace splat

using namespace splat::rows;

extern "C" {

long long splat_ffn_scratch(int M, int D, int F, int O, int dtype, int gated, int backward) {
  if (check_sizes(M, D, F, O, dtype, SPLAT_ACT_SILU) != SPLAT_OK) return 0;
  if (!backward && M <= kFewRows) return 0;
  const bool tc = dtype != SPLAT_F32;
  long long n = tc ? (long long)ffn_tc_image_bytes(D, F, O, gated != 0) : 0;
  if (backward)
    n += (long long)F * ((gated ? 2 : 1) * D + O) * 4 *
         (tc ? ffn_tc_splits(M, F) : dw_splits(M, F));
  return (n + 255) & ~255LL;
}

int splat_ffn(const void* x, long long ld_x, const void* w_gate, const void* w_up,
              const void* w_down, void* y, long long ld_y, int M, int D, int F, int O, int dtype,
              int act, void* scratch, long long scratch_bytes, void* stream) {
  int rc = check_sizes(M, D, F, O, dtype, act);
  if (rc != SPLAT_OK) return rc;
  if (M == 0) return SPLAT_OK;
  const int es = elem_size(dtype);
  const long long need = splat_ffn_scratch(M, D, F, O, dtype, w_gate != nullptr, 0);
  if (scratch_bytes < need) return SPLAT_ERR_INVALID_ARG;
  const Span s[] = {{x, M, D, ld_x, es, false},
                    {w_gate, w_gate ? F : 0, D, D, es, false},
                    {w_up, F, D, D, es, false},
                    {w_down, O, F, F, es, false},
                    {y, M, O, ld_y, es, true},
                    {scratch, need ? 1 : 0, need / 16, 0, 16, true}};
  if ((rc = check_spans(s, 6)) != SPLAT_OK) return rc;
  FfnArgs p = {};
  p.x = x;
  p.wg = w_gate;
  p.wu = w_up;
  p.wd = w_down;
  p.y = y;
  p.ldx = ld_x;
  p.ldy = ld_y;
  p.M = M;
  p.D = D;
  p.F = F;
  p.O = O;
  cudaStream_t st = (cudaStream_t)stream;
  return dispatch(p, dtype, act, false, scratch, st);
}

int splat_ffn_backward(const void* dy, long long ld_dy, const void* x, long long ld_x,
                       const void* w_gate, const void* w_up, const void* w_down, void* dx,
                       long long ld_dx, void* dw_gate, void* dw_up, void* dw_down, int M, int D,
                       int F, int O, int dtype, int act, void* scratch, long long scratch_bytes,
                       void* stream) {
  int rc = check_sizes(M, D, F, O, dtype, act);
  if (rc != SPLAT_OK) return rc;
  if (dw_gate && !w_gate) return SPLAT_ERR_INVALID_ARG;
  if (!dx && !dw_gate && !dw_up && !dw_down) return SPLAT_ERR_INVALID_ARG;
  const int es = elem_size(dtype);
  const long long need = splat_ffn_scratch(M, D, F, O, dtype, w_gate != nullptr, 1);
  if (scratch_bytes < need) return SPLAT_ERR_INVALID_ARG;
  const Span s[] = {{dy, M, O, ld_dy, es, false},
                    {x, M, D, ld_x, es, false},
                    {w_gate, w_gate ? F : 0, D, D, es, false},
                    {w_up, F, D, D, es, false},
                    {w_down, O, F, F, es, false},
                    {dx, dx ? M : 0, D, ld_dx, es, true},
                    {dw_gate, dw_gate ? F : 0, D, D, es, true},
                    {dw_up, dw_up ? F : 0, D, D, es, true},
                    {dw_down, dw_down ? O : 0, F, F, es, true},
                    {scratch, need ? 1 : 0, need / 16, 0, 16, true}};
  if ((rc = check_spans(s, 10)) != SPLAT_OK) return rc;
  FfnArgs p = {};
  p.dy = dy;
  p.x = x;
  p.wg = w_gate;
  p.wu = w_up;
  p.wd = w_down;
  p.dx = dx;
  p.dwg = dw_gate;
  p.dwu = dw_up;
  p.dwd = dw_down;
  p.ldx = ld_x;
  p.lddy = ld_dy;
  p.lddx = ld_dx;
  p.M = M;
  p.D = D;
  p.F = F;
  p.O = O;
  cudaStream_t st = (cudaStream_t)stream;
  return dispatch(p, dtype, act, true, scratch, st);
}

}  // extern "C"
