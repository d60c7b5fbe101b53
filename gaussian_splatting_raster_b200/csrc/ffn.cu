// Feed-forward block over rows: entry points, and the kernels on the fp32 lanes.
//
// One CTA takes a tile of rows through all products: its rows stay in shared memory while the
// hidden units pass in chunks of 64, 16 or 4 (their weights staged per chunk, transposed so that
// every inner product reads along rows). Bound by the fp32 lanes and by the shared-memory loads
// that feed them: 2 M F (2 D + O) operations against 4 M (D + O) bytes, which at D = 57, F = 256, O
// = 64 is 188 operations a byte. There, gated, 200,000 rows take 438 us with gelu (42 TFLOP/s, 56 %
// of the lanes' 74) and 492 with silu (37); the gradients of 100,000 rows 491 and 514 us for dx (30
// and 29 TFLOP/s), 664 and 692 us for the weights (27 and 26). 50,000 rows of 128 / 512 / 128 silu
// take 473 us (42), dx 938 us (35), weights 1,085 us (36).
#include <algorithm>

#include "ffn.cuh"

namespace splat {
namespace rows {
namespace {

constexpr int kT = 256;
// UC units are taken at a time: 64 (16 x 16 threads), or 16 (4 x 64) or 4 (1 x 256) for a few
// hidden units. Thread (tx, ty) has rows ty * RT .. and units (or output columns) tx * 4 .. of
// every UC.

// ---------------------------------------------------------------------------------------------
// packed weights and staging
// ---------------------------------------------------------------------------------------------
// Per chunk of UC units: [Wg | Wu]^T as D rows of gu_ld (UC gate, UC up units); then, forward, Wd^T
// as UC rows of down_ld(O), or, for the gradients, Wd as O rows of h_ld (UC units) and [Wg; Wu] as
// 2 UC rows of down_ld(D): zeros beyond F, D and O. A chunk is then copied to shared memory in
// 16-byte pieces, asynchronously, while the one before is worked on (where two fit).
__host__ __device__ constexpr int gu_ld(int UC) { return 2 * UC + 4; }
__host__ __device__ constexpr int h_ld(int UC) { return UC + 4; }
__host__ __device__ constexpr int down_ld(int O) { return (O <= 64 ? 64 : 128) + 4; }
__host__ __device__ constexpr int fwd_floats(int UC, int D, int O) {
  return D * gu_ld(UC) + UC * down_ld(O);
}
__host__ __device__ constexpr int dw_floats(int UC, int D, int O) {
  return D * gu_ld(UC) + O * h_ld(UC);
}
__host__ __device__ constexpr int bwd_floats(int UC, int D, int O) {
  return dw_floats(UC, D, O) + 2 * UC * down_ld(D);
}

__global__ void __launch_bounds__(kT)
k_pack32(FfnArgs p, int UC, bool backward, float* __restrict__ img) {
  const int per = backward ? bwd_floats(UC, p.D, p.O) : fwd_floats(UC, p.D, p.O);
  const int c = blockIdx.y, f0 = c * UC;
  const float *wg = (const float*)p.wg, *wu = (const float*)p.wu, *wd = (const float*)p.wd;
  // unit j of a chunk's gate and up units: its weights (NULL beyond F)
  auto unit = [&](int j) -> const float* {
    const int u = wg && j >= UC ? j - UC : j;
    if (u >= UC || f0 + u >= p.F) return nullptr;
    return (wg && j < UC ? wg : wu) + (size_t)(f0 + u) * p.D;
  };
  for (int i = blockIdx.x * kT + threadIdx.x; i < per; i += gridDim.x * kT) {
    float v = 0.0f;
    const int q = i - p.D * gu_ld(UC);
    if (q < 0) {
      const int k = i / gu_ld(UC);
      const float* w = unit(i - k * gu_ld(UC));
      if (w) v = w[k];
    } else if (backward && i >= dw_floats(UC, p.D, p.O)) {
      const int ld = down_ld(p.D), r = i - dw_floats(UC, p.D, p.O), k = r % ld;
      const float* w = unit(r / ld);
      if (w && k < p.D) v = w[k];
    } else if (backward) {
      const int o = q / h_ld(UC), u = q - o * h_ld(UC);
      if (u < UC && f0 + u < p.F) v = wd[(size_t)o * p.F + f0 + u];
    } else {
      const int ld = down_ld(p.O), u = q / ld, o = q - u * ld;
      if (o < p.O && f0 + u < p.F) v = wd[(size_t)o * p.F + f0 + u];
    }
    img[(size_t)c * per + i] = v;
  }
}

__device__ __forceinline__ void copy_chunk(float* dst, const float* src, int floats) {
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
  for (int i = threadIdx.x; i < floats / 4; i += kT)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(d + i * 16), "l"(src + i * 4)
                 : "memory");
  asm volatile("cp.async.commit_group;" ::: "memory");
}
// all copies but the newest `left` (0 or 1) are there
__device__ __forceinline__ void chunks_left(int left) {
  if (left)
    asm volatile("cp.async.wait_group 1;" ::: "memory");
  else
    asm volatile("cp.async.wait_group 0;" ::: "memory");
}

// rows [r0, r0 + R) of src transposed into dst[k * (R + 4) + r] by asynchronous copies; rows >= M
// are zero
template <int R>
__device__ __forceinline__ void copy_rows(const float* src, long long lds, long long r0, int M,
                                          int cols, float* dst) {
  const int lane = threadIdx.x & 31;
  const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
  for (int r = threadIdx.x >> 5; r < R; r += kT / 32) {
    const bool in = r0 + r < M;
    const float* row = src + (in ? r0 + r : 0) * lds;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int k = lane + 32 * q;
      if (k < cols)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(
                         d + 4 * (k * (R + 4) + r)),
                     "l"(row + k), "r"(in ? 4 : 0)
                     : "memory");
    }
  }
}

// acc[i][j] += sum_k rowsT[k][ty RT + i] w[k][tx 4 + j], two units an instruction
template <int RT, int UC>
__device__ __forceinline__ void product(const float* rowsT, int ldr, const float* w, int ldw,
                                        int K, float2 (&acc)[RT][2]) {
  const int tx = threadIdx.x % (UC / 4), ty = threadIdx.x / (UC / 4);
  const float* xp = rowsT + ty * RT;
  const float* wp = w + tx * 4;
#pragma unroll(RT <= 2 ? 8 : 4)
  for (int k = 0; k < K; ++k, xp += ldr, wp += ldw) {
    float xr[RT];
    if constexpr (RT == 1) {
      xr[0] = *xp;
    } else if constexpr (RT == 2) {
      *reinterpret_cast<float2*>(xr) = *reinterpret_cast<const float2*>(xp);
    } else {
#pragma unroll
      for (int i = 0; i < RT; i += 4)
        *reinterpret_cast<float4*>(xr + i) = *reinterpret_cast<const float4*>(xp + i);
    }
    const float4 wv = *reinterpret_cast<const float4*>(wp);
    const float2 w0 = make_float2(wv.x, wv.y), w1 = make_float2(wv.z, wv.w);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const float2 x2 = make_float2(xr[i], xr[i]);
      acc[i][0] = __ffma2_rn(x2, w0, acc[i][0]);
      acc[i][1] = __ffma2_rn(x2, w1, acc[i][1]);
    }
  }
}

// the same with two sets of units, UC apart
template <int RT, int UC>
__device__ __forceinline__ void product_pair(const float* rowsT, int ldr, const float* w, int ldw,
                                             int K, float2 (&a)[RT][2], float2 (&b)[RT][2]) {
  const int tx = threadIdx.x % (UC / 4), ty = threadIdx.x / (UC / 4);
  const float* xp = rowsT + ty * RT;
  const float* wp = w + tx * 4;
#pragma unroll(RT <= 2 ? 8 : 4)
  for (int k = 0; k < K; ++k, xp += ldr, wp += ldw) {
    float xr[RT];
    if constexpr (RT == 1) {
      xr[0] = *xp;
    } else if constexpr (RT == 2) {
      *reinterpret_cast<float2*>(xr) = *reinterpret_cast<const float2*>(xp);
    } else {
#pragma unroll
      for (int i = 0; i < RT; i += 4)
        *reinterpret_cast<float4*>(xr + i) = *reinterpret_cast<const float4*>(xp + i);
    }
    const float4 wv = *reinterpret_cast<const float4*>(wp);
    const float4 vv = *reinterpret_cast<const float4*>(wp + UC);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const float2 x2 = make_float2(xr[i], xr[i]);
      a[i][0] = __ffma2_rn(x2, make_float2(wv.x, wv.y), a[i][0]);
      a[i][1] = __ffma2_rn(x2, make_float2(wv.z, wv.w), a[i][1]);
      b[i][0] = __ffma2_rn(x2, make_float2(vv.x, vv.y), b[i][0]);
      b[i][1] = __ffma2_rn(x2, make_float2(vv.z, vv.w), b[i][1]);
    }
  }
}

// acc[n] += the product with columns n UC .. of w, up to `cols` of them, two sets at a time
template <int N, int RT, int UC>
__device__ __forceinline__ void products(const float* rowsT, int ldr, const float* w, int ldw,
                                         int K, int cols, float2 (&acc)[N][RT][2]) {
#pragma unroll
  for (int n = 0; n < N; n += 2) {
    if constexpr (N > 1) {
      if ((n + 1) * UC < cols) {
        product_pair<RT, UC>(rowsT, ldr, w + n * UC, ldw, K, acc[n], acc[n + 1]);
        continue;
      }
    }
    if (n * UC < cols) product<RT, UC>(rowsT, ldr, w + n * UC, ldw, K, acc[n]);
  }
}

template <int N>
__device__ __forceinline__ void clear(float2 (&a)[N][2]) {
#pragma unroll
  for (int i = 0; i < N; ++i) a[i][0] = a[i][1] = make_float2(0.0f, 0.0f);
}
template <int N, int M>
__device__ __forceinline__ void clear(float (&a)[N][M]) {
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < M; ++j) a[i][j] = 0.0f;
}
__device__ __forceinline__ float pick(const float2 (&a)[2], int j) {
  return j == 0 ? a[0].x : j == 1 ? a[0].y : j == 2 ? a[1].x : a[1].y;
}
// the thread's RT rows of one unit
template <int RT>
__device__ __forceinline__ void put_rows(float* dst, const float* v) {
  if constexpr (RT == 1) {
    *dst = v[0];
  } else if constexpr (RT == 2) {
    *reinterpret_cast<float2*>(dst) = make_float2(v[0], v[1]);
  } else {
#pragma unroll
    for (int i = 0; i < RT; i += 4)
      *reinterpret_cast<float4*>(dst + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  }
}

// Results (a thread's RT rows of 4 columns in each of N pieces of UC) to a row array. Where one
// thread has whole rows of 32 columns or more (UC = 4) they go through shared memory (all of it is
// free; `floats` of it) and out by whole warps: 560,000 rows of 61 took 202 us instead of 263 (of 3
// columns, 153 instead of 89).
template <int N, int RT, int UC, int R>
__device__ __forceinline__ void write_rows(const float2 (&v)[N][RT][2], float* sm, int floats,
                                           float* dst, long long ld, int cols, long long r0,
                                           int M) {
  constexpr int ldr = R + 1;
  const int tx = threadIdx.x % (UC / 4), ty = threadIdx.x / (UC / 4);
  const bool through = UC == 4 && cols >= 32 && cols * ldr <= floats;
  if (through) __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = n * UC + tx * 4 + j, r = ty * RT + i;
        if (c >= cols) continue;
        if (through)
          sm[c * ldr + r] = pick(v[n][i], j);
        else if (r0 + r < M)
          dst[(r0 + r) * ld + c] = pick(v[n][i], j);
      }
  if (!through) return;
  __syncthreads();
  for (int r = threadIdx.x >> 5; r < R && r0 + r < M; r += kT / 32)
    for (int c = threadIdx.x & 31; c < cols; c += 32) dst[(r0 + r) * ld + c] = sm[c * ldr + r];
}

// The CTAs of a cluster (S of them, along y) have the same rows and every S-th chunk of units each:
// their results are added in order, each CTA adding and writing R / S of the rows.
__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
constexpr int join_floats(int R, int width) { return R * (width + 4); }

template <int N, int RT, int UC, int R>
__device__ __forceinline__ void join_rows(const float2 (&v)[N][RT][2], float* sm, float* dst,
                                          long long ld, int cols, long long r0, int M) {
  constexpr int ldc = N * UC + 4;
  const int tx = threadIdx.x % (UC / 4), ty = threadIdx.x / (UC / 4);
#pragma unroll
  for (int n = 0; n < N; ++n)
#pragma unroll
    for (int i = 0; i < RT; ++i)
      *reinterpret_cast<float4*>(sm + (ty * RT + i) * ldc + n * UC + tx * 4) =
          make_float4(v[n][i][0].x, v[n][i][0].y, v[n][i][1].x, v[n][i][1].y);
  cluster_barrier();
  const int S = gridDim.y, per = R / S, f = blockIdx.y * per;
  const uint32_t base = (uint32_t)__cvta_generic_to_shared(sm);
  for (int r = f + (threadIdx.x >> 5); r < f + per && r0 + r < M; r += kT / 32)
    for (int c = threadIdx.x & 31; c < cols; c += 32) {
      float sum = 0.0f;
      for (int q = 0; q < S; ++q) {
        uint32_t at;
        float w;
        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                     : "=r"(at)
                     : "r"(base + 4 * (r * ldc + c)), "r"(q));
        asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(w) : "r"(at) : "memory");
        sum += w;
      }
      dst[(r0 + r) * ld + c] = sum;
    }
  cluster_barrier();  // until all have read this CTA's sums
}

// ---------------------------------------------------------------------------------------------
// forward, R rows a CTA
// ---------------------------------------------------------------------------------------------
int fwd_smem(int UC, int R, int D, int O, int bufs) {
  return 4 * (D * (R + 4) + bufs * fwd_floats(UC, D, O) + UC * (R + 4));
}

template <int ACT, bool GATED, int NO, int UC, int R>  // NO: 64-wide pieces of O
__global__ void __launch_bounds__(kT, 1) k_ffn(FfnArgs p, const float* __restrict__ img,
                                               int bufs) {
  extern __shared__ __align__(16) float sm[];
  constexpr int RT = R * UC / 1024, ldr = R + 4, ldo = NO * 64 + 4, P = 64 / UC;
  float* Xs = sm;                     // [D][ldr]
  float* Hs = Xs + p.D * ldr;         // [UC][ldr]
  float* Ws = Hs + UC * ldr;          // [bufs] of a chunk
  const int per = fwd_floats(UC, p.D, p.O);
  const int tx = threadIdx.x % (UC / 4), ty = threadIdx.x / (UC / 4);
  const long long r0 = (long long)blockIdx.x * R;
  const int nch = (p.F + UC - 1) / UC;
  const int S = gridDim.y, c0 = blockIdx.y;  // the cluster's CTAs; the first chunk of this one
  copy_rows<R>((const float*)p.x, p.ldx, r0, p.M, p.D, Xs);
  copy_chunk(Ws, img + (size_t)c0 * per, per);
  float2 yv[NO * P][RT][2];
#pragma unroll
  for (int n = 0; n < NO * P; ++n) clear(yv[n]);
  for (int c = c0, b = 0; c < nch; c += S, b ^= bufs - 1) {
    float* W = Ws + b * per;
    const bool more = c + S < nch, ahead = bufs > 1 && more;
    if (ahead) copy_chunk(Ws + (b ^ 1) * per, img + (size_t)(c + S) * per, per);
    chunks_left(ahead);
    __syncthreads();
    float2 a[RT][2], u[RT][2];
    clear(a);
    if (GATED) {
      clear(u);
      product_pair<RT, UC>(Xs, ldr, W, gu_ld(UC), p.D, a, u);
    } else {
      product<RT, UC>(Xs, ldr, W, gu_ld(UC), p.D, a);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float h[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) {
        h[i] = act_of<ACT>(pick(a[i], j));
        if (GATED) h[i] *= pick(u[i], j);
      }
      put_rows<RT>(Hs + (tx * 4 + j) * ldr + ty * RT, h);
    }
    __syncthreads();
    products<NO * P, RT, UC>(Hs, ldr, W + p.D * gu_ld(UC), ldo, UC, p.O, yv);
    __syncthreads();
    if (bufs == 1 && more) copy_chunk(Ws, img + (size_t)(c + S) * per, per);
  }
  if constexpr (UC >= 16)
    if (S > 1) {
      join_rows<NO * P, RT, UC, R>(yv, sm, (float*)p.y, p.ldy, p.O, r0, p.M);
      return;
    }
  write_rows<NO * P, RT, UC, R>(yv, sm, p.D * ldr + UC * ldr + bufs * per, (float*)p.y, p.ldy, p.O,
                                r0, p.M);
}

// ---------------------------------------------------------------------------------------------
// a few rows
// ---------------------------------------------------------------------------------------------
// Bound by latency: the weights have to come from L2 once. A cluster of eight CTAs shares kFew
// rows; each CTA takes every eighth group of hidden units, a warp four units at a time (its lanes
// along D, then one sum over the warp for each), and forms its part of y from them; the first CTA
// adds the eight parts in order through distributed shared memory. x and the weights are read in
// whole rows by neighbouring lanes whatever their alignment. (57 / 256 / 64, nothing in L2, fp32:
// one row 8.8 us, 64 rows 9.5, 128 rows 9.8, in one launch; by tiles 129 to 300 rows take 8.0 after
// 2.5 for the packing. bf16: 128 rows 11.1 us; on the tensor cores 129 take 11.6 after 2.3.) Hidden
// values stay in fp32.
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
        if (lane == 0 && j0 + u < n) s_h[i][j0 + u] = h;
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

// ---------------------------------------------------------------------------------------------
// gradients, R rows a tile
// ---------------------------------------------------------------------------------------------

// a, u, dh of one tile and chunk, turned into da, du (and h)
template <int ACT, bool GATED, int RT, int UC>
__device__ __forceinline__ void hidden_grads(const float* Xs, const float* Ys, int ldr,
                                             const float* W, int D, int O, float (&da)[RT][4],
                                             float (&du)[RT][4], float (&h)[RT][4]) {
  float2 a[RT][2], u[RT][2], dh[RT][2];
  clear(a);
  clear(dh);
  if (GATED) {
    clear(u);
    product_pair<RT, UC>(Xs, ldr, W, gu_ld(UC), D, a, u);
  } else {
    product<RT, UC>(Xs, ldr, W, gu_ld(UC), D, a);
  }
  product<RT, UC>(Ys, ldr, W + D * gu_ld(UC), h_ld(UC), O, dh);
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float s;
      const float f = act_and_slope<ACT>(pick(a[i], j), s), g = pick(dh[i], j);
      const float v = GATED ? pick(u[i], j) : 1.0f;
      h[i][j] = GATED ? f * v : f;
      da[i][j] = GATED ? g * v * s : g * s;
      du[i][j] = GATED ? g * f : 0.0f;
    }
}

// bufs 0: the chunk's two halves (for the hidden values, for dx) take turns in one place
int dx_smem(int UC, int R, int D, int O, int bufs) {
  const int half = std::max(dw_floats(UC, D, O), 2 * UC * down_ld(D));
  return 4 * ((D + O) * (R + 4) + 2 * UC * (R + 4) +
              (bufs ? bufs * bwd_floats(UC, D, O) : half));
}
int dw_smem(int UC, int R, int D, int O, int bufs) {
  return 4 * (bufs * (D + O) * (R + 4) + 3 * R * h_ld(UC) + dw_floats(UC, D, O));
}

// dx of one tile: all chunks in turn
template <int ACT, bool GATED, int ND, int UC, int R>  // ND: 64-wide pieces of D
__global__ void __launch_bounds__(kT, 1) k_ffn_dx(FfnArgs p, const float* __restrict__ img,
                                                  int bufs) {
  extern __shared__ __align__(16) float sm[];
  constexpr int RT = R * UC / 1024, ldr = R + 4, P = 64 / UC;
  float* Xs = sm;                    // [D][ldr]
  float* Ys = Xs + p.D * ldr;        // [O][ldr]
  float* As = Ys + p.O * ldr;        // [UC units][ldr] da, then du
  float* Us = As + UC * ldr;
  float* Ws = Us + UC * ldr;         // [bufs] of a chunk
  const int per = bwd_floats(UC, p.D, p.O), nch = (p.F + UC - 1) / UC;
  const int tx = threadIdx.x % (UC / 4), ty = threadIdx.x / (UC / 4);
  const long long r0 = (long long)blockIdx.x * R;
  copy_rows<R>((const float*)p.x, p.ldx, r0, p.M, p.D, Xs);
  copy_rows<R>((const float*)p.dy, p.lddy, r0, p.M, p.O, Ys);
  const int first = dw_floats(UC, p.D, p.O);  // a chunk's part for the hidden values
  const int S = gridDim.y, c0 = blockIdx.y;  // the cluster's CTAs; the first chunk of this one
  copy_chunk(Ws, img + (size_t)c0 * per, bufs ? per : first);
  float2 acc[ND * P][RT][2];
#pragma unroll
  for (int n = 0; n < ND * P; ++n) clear(acc[n]);
  for (int ch = c0, b = 0; ch < nch; ch += S, b ^= bufs > 1) {
    float* W = Ws + b * per;
    const bool more = ch + S < nch, ahead = bufs > 1 && more;
    if (ahead) copy_chunk(Ws + (b ^ 1) * per, img + (size_t)(ch + S) * per, per);
    chunks_left(ahead);
    __syncthreads();
    float da[RT][4], du[RT][4], h[RT][4];
    hidden_grads<ACT, GATED, RT, UC>(Xs, Ys, ldr, W, p.D, p.O, da, du, h);
    if (bufs == 0) {
      __syncthreads();
      copy_chunk(Ws, img + (size_t)ch * per + first, per - first);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v[RT];
#pragma unroll
      for (int i = 0; i < RT; ++i) v[i] = da[i][j];
      put_rows<RT>(As + (tx * 4 + j) * ldr + ty * RT, v);
      if (GATED) {
#pragma unroll
        for (int i = 0; i < RT; ++i) v[i] = du[i][j];
        put_rows<RT>(Us + (tx * 4 + j) * ldr + ty * RT, v);
      }
    }
    if (bufs == 0) chunks_left(0);
    __syncthreads();
    const float* N = bufs ? W + first : Ws;
    constexpr int ldd = ND * 64 + 4;
    products<ND * P, RT, UC>(As, ldr, N, ldd, UC, p.D, acc);
    if (GATED) products<ND * P, RT, UC>(Us, ldr, N + UC * ldd, ldd, UC, p.D, acc);
    __syncthreads();
    if (bufs < 2 && more) copy_chunk(Ws, img + (size_t)(ch + S) * per, bufs ? per : first);
  }
  if constexpr (UC >= 16)
    if (S > 1) {
      join_rows<ND * P, RT, UC, R>(acc, sm, (float*)p.dx, p.lddx, p.D, r0, p.M);
      return;
    }
  write_rows<ND * P, RT, UC, R>(acc, sm, (p.D + p.O) * ldr + 2 * UC * ldr + bufs * per,
                                (float*)p.dx, p.lddx, p.D, r0, p.M);
}

// partial weight gradients of chunk blockIdx.x over the row tiles blockIdx.y, + splits, ...
template <int ACT, bool GATED, int UC, int R>
__global__ void __launch_bounds__(kT, 1) k_ffn_dw(FfnArgs p, const float* __restrict__ img,
                                                  int bufs) {
  extern __shared__ __align__(16) float sm[];
  constexpr int RT = R * UC / 1024, ldr = R + 4, kLd = h_ld(UC);
  // rows of D or O a thread has: ty + TY c
  constexpr int TY = 1024 / UC, C = TY < kMaxWidth ? kMaxWidth / TY : 1;
  float* rows = sm;                  // [bufs] of X [D][ldr] and dY [O][ldr]
  const int both = (p.D + p.O) * ldr;
  float* As = rows + bufs * both;       // [R rows][kLd units] da, du, h
  float* Us = As + R * kLd;
  float* Hs = Us + R * kLd;
  float* W = Hs + R * kLd;
  const int tx = threadIdx.x % (UC / 4), ty = threadIdx.x / (UC / 4);
  const int f0 = blockIdx.x * UC, per = bwd_floats(UC, p.D, p.O);
  copy_chunk(W, img + (size_t)blockIdx.x * per, dw_floats(UC, p.D, p.O));
  float2 ga[C][2], gu[C][2], gd[C][2];
  clear(ga);
  clear(gu);
  clear(gd);
  const int tiles = (int)(((long long)p.M + R - 1) / R);
  auto fetch = [&](int t, int b) {
    float* X = rows + b * both;
    copy_rows<R>((const float*)p.x, p.ldx, (long long)t * R, p.M, p.D, X);
    copy_rows<R>((const float*)p.dy, p.lddy, (long long)t * R, p.M, p.O, X + p.D * ldr);
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if ((int)blockIdx.y < tiles) fetch(blockIdx.y, 0);
  int b = 0;
  for (int t = blockIdx.y; t < tiles; t += p.splits, b ^= bufs - 1) {
    const bool more = t + p.splits < tiles, ahead = more && bufs > 1;
    if (ahead) fetch(t + p.splits, b ^ 1);
    chunks_left(ahead);
    __syncthreads();
    const float* Xs = rows + b * both;
    const float* Ys = Xs + p.D * ldr;
    float da[RT][4], du[RT][4], h[RT][4];
    hidden_grads<ACT, GATED, RT, UC>(Xs, Ys, ldr, W, p.D, p.O, da, du, h);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const int at = (ty * RT + i) * kLd + tx * 4;
      *reinterpret_cast<float4*>(As + at) = make_float4(da[i][0], da[i][1], da[i][2], da[i][3]);
      if (GATED)
        *reinterpret_cast<float4*>(Us + at) = make_float4(du[i][0], du[i][1], du[i][2], du[i][3]);
      *reinterpret_cast<float4*>(Hs + at) = make_float4(h[i][0], h[i][1], h[i][2], h[i][3]);
    }
    __syncthreads();
    for (int r = 0; r < R; r += 2) {
      float4 av[2], uv[2], hv[2];
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        const int at = (r + q) * kLd + tx * 4;
        av[q] = *reinterpret_cast<const float4*>(As + at);
        if (GATED) uv[q] = *reinterpret_cast<const float4*>(Us + at);
        hv[q] = *reinterpret_cast<const float4*>(Hs + at);
      }
      auto add = [](float2 (&g)[2], float x, const float4& v) {
        const float2 x2 = make_float2(x, x);
        g[0] = __ffma2_rn(x2, make_float2(v.x, v.y), g[0]);
        g[1] = __ffma2_rn(x2, make_float2(v.z, v.w), g[1]);
      };
      float2 x[C], y[C];  // all loads first, then the products without a wait
#pragma unroll
      for (int c = 0; c < C; ++c) {
        x[c] = *reinterpret_cast<const float2*>(Xs + min(ty + TY * c, p.D - 1) * ldr + r);
        y[c] = *reinterpret_cast<const float2*>(Ys + min(ty + TY * c, p.O - 1) * ldr + r);
      }
#pragma unroll
      for (int c = 0; c < C; ++c) {
        if (TY * c < p.D) {
          add(ga[c], x[c].x, av[0]);
          add(ga[c], x[c].y, av[1]);
          if (GATED) {
            add(gu[c], x[c].x, uv[0]);
            add(gu[c], x[c].y, uv[1]);
          }
        }
        if (TY * c < p.O) {
          add(gd[c], y[c].x, hv[0]);
          add(gd[c], y[c].y, hv[1]);
        }
      }
    }
    __syncthreads();  // the tile's place is free
    if (more && bufs == 1) fetch(t + p.splits, 0);
  }
  const size_t FD = (size_t)p.F * p.D;
  float* part = p.part + blockIdx.y * ((GATED ? 2 : 1) * FD + (size_t)p.O * p.F);
#pragma unroll
  for (int c = 0; c < C; ++c)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int k = ty + TY * c, f = f0 + tx * 4 + j;
      if (f >= p.F) continue;
      if (k < p.D) {
        part[(size_t)f * p.D + k] = pick(ga[c], j);
        if (GATED) part[FD + (size_t)f * p.D + k] = pick(gu[c], j);
      }
      if (k < p.O) part[(GATED ? 2 : 1) * FD + (size_t)f * p.O + k] = pick(gd[c], j);
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

constexpr int kSmemMax = 232448 - 1024;

// A kernel's limit is always the same: it belongs to the kernel, not to a launch, and another host
// thread may set it between this thread's setting it and its launch.
template <typename K>
bool allow_smem(K kernel) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax) ==
         cudaSuccess;
}

// Units taken at a time: 16 or 4 for a few hidden units, whose chunk of 64 would be mostly zeros (4
// where its 256-row tiles fit); 16 also where the other side (O forward, D for dx) is so narrow
// that pieces of 64 columns would cost more than the better use of a load by 64 units saves, about
// a third (566,585 rows of 13, 156 units to one column, no gate: 730 us with 64, 359 with 16).
int chunk_of(int D, int F, int O, bool backward) {
  if (F <= 4 && D + O <= 180) return 4;
  if (F <= 32) return 16;
  auto cost = [&](int UC) {
    auto up = [&](int c) { return (c + UC - 1) / UC * UC; };
    return backward ? 2 * D + O + 2 * up(D) : 2 * D + up(O);
  };
  return 3 * cost(16) < 2 * cost(64) ? 16 : 64;
}

// Rows of a tile and CTAs of its cluster. A thread's products of RT rows by 4 (or, of both inputs,
// 8) units read RT + 4 (RT + 8) words from shared memory for each input column, which is what
// bounds them, so tall tiles read least a row; short ones and clusters, which share a tile's
// chunks, fill the machine (of which 15 clusters of eight or 33 of four have place at once). The
// time of a choice is about its waves of CTAs times the words a warp reads, 600 more a chunk for
// its barriers and 1,000 a CTA, or 2,500 with a cluster's join. (Forward, 128 / 1024 / 128 gated:
// 300 rows 30 us, without clusters 148; 20,000 rows 432 us, 667; gradients of 1,000 rows of 57 /
// 256 / 64: dx 13 us, 34.)
struct Tile { int R, S; };
Tile tile_of(int UC, int most, bool backward, long long M, int D, int F, int O, bool gated) {
  const int nch = (F + UC - 1) / UC, wide = gated ? 8 : 4;
  const int least = UC == 4 ? 256 : UC == 16 ? 64 : 16;
  if (UC == 4) return {256, 1};
  Tile best = {most, 1};
  double t = 1e300;
  for (int R = most; R >= least; R >>= 1)
    for (int S = 1; S <= 8 && S <= nch; S <<= 1) {
      const int RT = R * UC / 1024, out = ((backward ? D : O) + UC - 1) / UC * UC;
      const double second = out > UC ? out * 0.5 * (RT + 8) : (double)out * (RT + 4);
      double words = (double)D * (RT + wide) + second;
      if (backward) words += (double)O * (RT + 4) + (gated ? second : 0.0);
      const long long ctas = (M + R - 1) / R * S, fit = S == 8 ? 120 : S == 4 ? 132 : 148;
      const double cost = (double)((ctas + fit - 1) / fit) *
                          ((nch + S - 1) / S * (words + 600) + (S > 1 ? 2500 : 1000));
      if (cost < t) t = cost, best = {R, S};
    }
  return best;
}
bool many(long long M) { return M > 64 * 148; }
int dw_rows(int UC, long long M, int D, int O) {
  if (UC == 4) return 256;
  const int most = UC == 64 ? 64 : 128;
  return many(M) && dw_smem(UC, most, D, O, 1) <= kSmemMax ? most : most / 2;
}

// row splits of the weight gradients: enough CTAs for the machine, and at most 8,192 rows a split
// (an fp32 sum of n products is off by about sqrt(n) 2^-25 of its size)
int dw_splits(long long M, int D, int F, int O) {
  const int UC = chunk_of(D, F, O, true), chunks = (F + UC - 1) / UC, R = dw_rows(UC, M, D, O);
  const long long tiles = (M + R - 1) / R;
  const long long least = std::max((M + 8191) / 8192, 1LL), waves = (least * chunks + 147) / 148;
  // where an SM holds one CTA, no wave of CTAs is left with a few
  long long s = dw_smem(UC, R, D, O, 1) > kSmemMax / 2 ? waves * 148 / chunks
                                                        : (waves * 148 + chunks - 1) / chunks;
  if (s < least) s = least;
  if (s > tiles) s = tiles;
  if (s > 65535) s = 65535;  // the grid's limit
  return (int)(s < 1 ? 1 : s);
}

size_t pack32_bytes(int D, int F, int O, bool backward) {
  const int UC = chunk_of(D, F, O, backward);
  const size_t n = (size_t)((F + UC - 1) / UC) *
                   (backward ? bwd_floats(UC, D, O) : fwd_floats(UC, D, O)) * 4;
  return (n + 255) & ~(size_t)255;
}

void pack32(const FfnArgs& p, bool backward, float* img, cudaStream_t st) {
  const int UC = chunk_of(p.D, p.F, p.O, backward);
  const int per = backward ? bwd_floats(UC, p.D, p.O) : fwd_floats(UC, p.D, p.O);
  k_pack32<<<dim3((per + kT - 1) / kT, (p.F + UC - 1) / UC), kT, 0, st>>>(p, UC, backward, img);
}

// `kernel` on tiles of R rows, each taken by a cluster of S CTAs
template <typename K>
int launch_tiles(K kernel, const FfnArgs& p, const float* img, int bufs, int smem, int R, int S,
                 cudaStream_t st) {
  if (!allow_smem(kernel)) return SPLAT_ERR_CUDA;
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)(((long long)p.M + R - 1) / R), S);
  c.blockDim = dim3(kT);
  c.dynamicSmemBytes = smem;
  c.stream = st;
  cudaLaunchAttribute at = {};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = 1;
  at.val.clusterDim.y = S;
  at.val.clusterDim.z = 1;
  c.attrs = &at;
  c.numAttrs = S > 1 ? 1 : 0;
  if (cudaLaunchKernelEx(&c, kernel, p, img, bufs) != cudaSuccess) {
    cudaGetLastError();
    return SPLAT_ERR_CUDA;
  }
  return SPLAT_OK;
}

template <int ACT, bool GATED, int NO, int UC, int R>
int launch_fwd(const FfnArgs& p, const float* img, int S, cudaStream_t st) {
  const int bufs = p.F > UC * S && fwd_smem(UC, R, p.D, p.O, 2) <= kSmemMax ? 2 : 1;
  const int smem =
      std::max(fwd_smem(UC, R, p.D, p.O, bufs), S > 1 ? 4 * join_floats(R, NO * 64) : 0);
  return launch_tiles(k_ffn<ACT, GATED, NO, UC, R>, p, img, bufs, smem, R, S, st);
}

template <int ACT, bool GATED, int NO>
int run_forward(const FfnArgs& p, float* img, cudaStream_t st) {
  pack32(p, false, img, st);
  const int UC = chunk_of(p.D, p.F, p.O, false);
  const Tile t = tile_of(UC, 128, false, p.M, p.D, p.F, p.O, GATED);
  if (UC == 4) return launch_fwd<ACT, GATED, NO, 4, 256>(p, img, 1, st);
  if (UC == 16)
    return t.R == 128 ? launch_fwd<ACT, GATED, NO, 16, 128>(p, img, t.S, st)
                      : launch_fwd<ACT, GATED, NO, 16, 64>(p, img, t.S, st);
  switch (t.R) {
    case 128: return launch_fwd<ACT, GATED, NO, 64, 128>(p, img, t.S, st);
    case 64: return launch_fwd<ACT, GATED, NO, 64, 64>(p, img, t.S, st);
    case 32: return launch_fwd<ACT, GATED, NO, 64, 32>(p, img, t.S, st);
  }
  return launch_fwd<ACT, GATED, NO, 64, 16>(p, img, t.S, st);
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

template <typename T, bool GATED> int run_join(const FfnArgs& p, cudaStream_t st) {
  const size_t n = ((GATED ? 2 : 1) * (size_t)p.D + p.O) * p.F;
  k_ffn_join<T, GATED><<<(unsigned)((n + 31) / 32), kT, 0, st>>>(p);
  return last_error();
}

template <int ACT, bool GATED, int ND, int UC, int R>
int launch_dx(const FfnArgs& p, const float* img, int S, cudaStream_t st) {
  const int bufs = p.F > UC * S && dx_smem(UC, R, p.D, p.O, 2) <= kSmemMax ? 2
                   : dx_smem(UC, R, p.D, p.O, 1) <= kSmemMax               ? 1
                                                                           : 0;
  const int smem =
      std::max(dx_smem(UC, R, p.D, p.O, bufs), S > 1 ? 4 * join_floats(R, ND * 64) : 0);
  return launch_tiles(k_ffn_dx<ACT, GATED, ND, UC, R>, p, img, bufs, smem, R, S, st);
}

template <int ACT, bool GATED, int UC, int R>
int launch_dw(const FfnArgs& p, const float* img, cudaStream_t st) {
  const int bufs = dw_smem(UC, R, p.D, p.O, 2) <= kSmemMax ? 2 : 1;
  const int smem = dw_smem(UC, R, p.D, p.O, bufs);
  if (!allow_smem(k_ffn_dw<ACT, GATED, UC, R>)) return SPLAT_ERR_CUDA;
  const dim3 grid((p.F + UC - 1) / UC, p.splits);
  k_ffn_dw<ACT, GATED, UC, R><<<grid, kT, smem, st>>>(p, img, bufs);
  return run_join<float, GATED>(p, st);
}

template <int ACT, bool GATED, int ND>
int run_dx(const FfnArgs& p, const float* img, cudaStream_t st) {
  const int UC = chunk_of(p.D, p.F, p.O, true);
  const int most = UC == 16 && dx_smem(16, 128, p.D, p.O, 1) > kSmemMax ? 64 : UC == 16 ? 128 : 64;
  const Tile t = tile_of(UC, most, true, p.M, p.D, p.F, p.O, GATED);
  if (UC == 4) return launch_dx<ACT, GATED, ND, 4, 256>(p, img, 1, st);
  if (UC == 16)
    return t.R == 128 ? launch_dx<ACT, GATED, ND, 16, 128>(p, img, t.S, st)
                      : launch_dx<ACT, GATED, ND, 16, 64>(p, img, t.S, st);
  return t.R == 64   ? launch_dx<ACT, GATED, ND, 64, 64>(p, img, t.S, st)
         : t.R == 32 ? launch_dx<ACT, GATED, ND, 64, 32>(p, img, t.S, st)
                     : launch_dx<ACT, GATED, ND, 64, 16>(p, img, t.S, st);
}

template <int ACT, bool GATED>
int run_backward(const FfnArgs& p, float* img, cudaStream_t st) {
  pack32(p, true, img, st);
  int rc = SPLAT_OK;
  if (p.dx && p.M > 0)
    rc = p.D <= 64 ? run_dx<ACT, GATED, 1>(p, img, st) : run_dx<ACT, GATED, 2>(p, img, st);
  if (rc != SPLAT_OK || !(p.dwg || p.dwu || p.dwd)) return rc;
  const int UC = chunk_of(p.D, p.F, p.O, true), R = dw_rows(UC, p.M, p.D, p.O);
  if (UC == 4) return launch_dw<ACT, GATED, 4, 256>(p, img, st);
  if (UC == 16)
    return R == 128 ? launch_dw<ACT, GATED, 16, 128>(p, img, st)
                    : launch_dw<ACT, GATED, 16, 64>(p, img, st);
  return R == 64 ? launch_dw<ACT, GATED, 64, 64>(p, img, st)
                 : launch_dw<ACT, GATED, 64, 32>(p, img, st);
}

// A few rows by the clusters; otherwise fp32 on the fp32 lanes, bf16 and fp16 on the tensor cores.
template <typename T, int ACT, bool GATED>
int run(FfnArgs& p, int dtype, bool backward, void* scratch, cudaStream_t st) {
  if (!backward && p.M <= kFewRows) return run_few<T, ACT, GATED>(p, st);
  if constexpr (sizeof(T) == 4) {
    p.part = (float*)((char*)scratch + pack32_bytes(p.D, p.F, p.O, backward));
    p.splits = dw_splits(p.M, p.D, p.F, p.O);
    if (backward) return run_backward<ACT, GATED>(p, (float*)scratch, st);
    return p.O <= 64 ? run_forward<ACT, GATED, 1>(p, (float*)scratch, st)
                     : run_forward<ACT, GATED, 2>(p, (float*)scratch, st);
  } else {
    p.part = (float*)((char*)scratch + ffn_tc_image_bytes(p.D, p.F, p.O, GATED));
    p.splits = ffn_tc_splits(p.M, p.D, p.F, p.O);
    if (backward && dtype == SPLAT_F16)
      p.dy_max = (unsigned*)(p.part + (size_t)p.F * ((GATED ? 2 : 1) * p.D + p.O) * p.splits *
                                          ffn_tc_parts(p.D, p.F, p.O));
    const int rc = ffn_tc_run(p, dtype, ACT, backward, scratch, st);
    if (rc != SPLAT_OK || !(p.dwg || p.dwu || p.dwd)) return rc;
    p.splits *= ffn_tc_parts(p.D, p.F, p.O);
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
  long long n = tc ? (long long)ffn_tc_image_bytes(D, F, O, gated != 0)
                   : (long long)pack32_bytes(D, F, O, backward != 0);
  if (backward)
    n += (long long)F * ((gated ? 2 : 1) * D + O) * 4 *
         (tc ? ffn_tc_splits(M, D, F, O) * ffn_tc_parts(D, F, O) : dw_splits(M, D, F, O));
  if (backward && dtype == SPLAT_F16) n += kMaxParts * 4;
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
