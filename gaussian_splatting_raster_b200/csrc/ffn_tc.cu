// Feed-forward block over rows on the tensor cores (bf16 and fp16).
//
// Three persistent kernels of one skeleton, one CTA per SM:
//   forward   per 128-row tile and chunk of 64 hidden units:
//               [A|U] = X [Wg;Wu]^T -> TMEM -> h -> shared memory -> Y += H Wd^T (TMEM)
//   dx        [A|U] again, dH = dY Wd -> da, du -> shared memory -> dX += [da|du] [Wg;Wu]
//   weights   a CTA keeps one chunk and walks row tiles: da, du, h as above, then
//               dWg, dWu += [da|du]^T X,  dWd += h^T dY, accumulated in TMEM over all its tiles
// so hidden values and their gradients never leave the SM. dx and the weight gradients are two
// kernels because the sums run along different axes: with both in one, either dX or dW would have
// to leave TMEM per tile and chunk (M F D / 64 fp32 sums), which costs more than computing the
// hidden values twice.
//
// A CTA has up to two groups of eight warps, each with its own tile, shared memory and TMEM, which
// take turns: while one turns accumulators into hidden values, the tensor cores work for the
// other. One thread issues all MMAs, one all weight loads. Weights are packed once per call into
// the layout the MMAs read (zeros beyond F, D and O), so a chunk is one contiguous bulk copy; all
// chunks stay in shared memory where they fit. Row tiles are read with plain loads, which take any
// row distance and alignment (token rows have odd widths), straight into the swizzled layout.
#include "ffn.cuh"
#include "tc.cuh"

namespace splat {
namespace rows {
namespace {

using namespace tc;

enum Mode { kFwd, kDx, kDw };

constexpr int kGroupThreads = 256;
constexpr int kMaxGroups = 2;
constexpr int kTcThreads = kMaxGroups * kGroupThreads + 64;  // + MMA warp + weight warp
constexpr int kMaxStages = 16;
constexpr int kTile = 128;
constexpr int kSmemLimit = 232448 - 2048;  // 227 KB less the alignment slack and the barriers

__device__ unsigned int g_rows_status;

struct TcArgs {
  FfnArgs f;
  const uint8_t* img;   // packed weights, chunk after chunk
  int nch, stage_bytes; // chunks; bytes of one
  int nst, ng;          // weight stages in shared memory; groups
  int dp, op;           // D and O rounded up to 16
  int x_vec, dy_vec, out_vec;  // bytes per access of x, dy, and y or dx
  uint32_t x_magic, dy_magic;  // dividers by the 16-byte pieces per row
  long long tiles;
};

template <typename T> struct Two;
template <> struct Two<__nv_bfloat16> {
  static constexpr bool kBf16 = true;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};
template <> struct Two<__half> {
  static constexpr bool kBf16 = false;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    const __half2 v = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
};

// 1 / v and e^v from the special function unit (relative error below 2^-22 each; the results are
// rounded to 8 or 11 bits)
__device__ __forceinline__ float rcp_fast(float v) { return __fdividef(1.0f, v); }
__device__ __forceinline__ float exp_fast(float v) { return __expf(v); }

// Phi(a) and e^{-a^2/2}: Abramowitz and Stegun 7.1.26 for erfc at |a| / sqrt 2, absolute error
// 0.75e-7 in Phi; one exponential serves Phi and the density.
__device__ __forceinline__ float normal_cdf(float a, float& e) {
  const float z = fabsf(a) * 0.70710678118654752f;
  const float t = rcp_fast(fmaf(0.3275911f, z, 1.0f));
  e = exp_fast(-z * z);
  float q = fmaf(1.061405429f, t, -1.453152027f);
  q = fmaf(q, t, 1.421413741f);
  q = fmaf(q, t, -0.284496736f);
  q = fmaf(q, t, 0.254829592f);
  q = 0.5f * (q * t) * e;
  return a >= 0.0f ? 1.0f - q : q;
}

template <int ACT> __device__ __forceinline__ float act_fast(float a) {
  if (ACT == SPLAT_ACT_SILU) return a * rcp_fast(1.0f + exp_fast(-a));
  float e;
  return a * normal_cdf(a, e);
}

template <int ACT> __device__ __forceinline__ float act_slope_fast(float a, float& slope) {
  if (ACT == SPLAT_ACT_SILU) {
    const float s = rcp_fast(1.0f + exp_fast(-a)), f = a * s;
    slope = fmaf(f, 1.0f - s, s);
    return f;
  }
  float e;
  const float c = normal_cdf(a, e);
  slope = fmaf(a * 0.3989422804014327f, e, c);
  return a * c;
}

// ---------------------------------------------------------------------------------------------
// packed weights
// ---------------------------------------------------------------------------------------------
// Chunk c: [Wg units | Wu units] (128 rows, 64 without a gate) in blocks of 64 columns of D, then
// Wd's columns of the chunk (op rows of 64). One thread per 16-byte piece.
template <typename T, bool GATED>
__global__ void __launch_bounds__(256)
k_pack(TcArgs p, uint8_t* __restrict__ img) {
  constexpr int WR = GATED ? 128 : 64;
  const int nb = (p.f.D + 63) >> 6, pieces = p.stage_bytes >> 4, gu = nb * WR * 8;
  const int i = blockIdx.x * 256 + threadIdx.x;
  if (i >= p.nch * pieces) return;
  const int c = i / pieces, q = i - c * pieces;
  const T* src = nullptr;
  int n = 0, row;
  if (q < gu) {
    row = (q >> 3) % WR;
    const int b = (q >> 3) / WR, col = b * 64 + (((q & 7) ^ (row & 7)) << 3);
    const int f = c * kChunk + (row & 63);
    if (f < p.f.F) {
      src = (const T*)(GATED && row < 64 ? p.f.wg : p.f.wu) + (size_t)f * p.f.D + col;
      n = p.f.D - col;
    }
  } else {
    row = (q - gu) >> 3;
    const int col = c * kChunk + ((((q - gu) & 7) ^ (row & 7)) << 3);
    if (row < p.f.O) {
      src = (const T*)p.f.wd + (size_t)row * p.f.F + col;
      n = p.f.F - col;
    }
  }
  union {
    uint4 v;
    T e[8];
  } o;
  o.v = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
  for (int k = 0; k < 8; ++k)
    if (k < n) o.e[k] = src[k];
  *reinterpret_cast<uint4*>(img + (size_t)i * 16) = o.v;
}

// ---------------------------------------------------------------------------------------------
// row tiles
// ---------------------------------------------------------------------------------------------

// elements [8 c, 8 c + 8) of a row of `cols`, zeros behind its end
__device__ __forceinline__ uint4 fetch8(const uint16_t* row, int c, int cols, int vec) {
  const int e0 = c * 8;
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (vec == 16) {
    if (e0 < cols) v = __ldg(reinterpret_cast<const uint4*>(row + e0));
  } else if (vec == 8) {
    const uint2* s = reinterpret_cast<const uint2*>(row + e0);
    uint2 a = make_uint2(0u, 0u), b = a;
    if (e0 < cols) a = __ldg(s);
    if (e0 + 4 < cols) b = __ldg(s + 1);
    v = make_uint4(a.x, a.y, b.x, b.y);
  } else if (vec == 4) {
    const uint32_t* s = reinterpret_cast<const uint32_t*>(row + e0);
    if (e0 < cols) v.x = __ldg(s);
    if (e0 + 2 < cols) v.y = __ldg(s + 1);
    if (e0 + 4 < cols) v.z = __ldg(s + 2);
    if (e0 + 6 < cols) v.w = __ldg(s + 3);
  } else {
    uint32_t h[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) h[k] = e0 + k < cols ? (uint32_t)__ldg(row + e0 + k) : 0u;
    v = make_uint4(h[0] | (h[1] << 16), h[2] | (h[3] << 16), h[4] | (h[5] << 16),
                   h[6] | (h[7] << 16));
  }
  return v;
}

// One group's tile of rows [r0, r0 + 128) in registers (each thread np pieces), then in shared
// memory. np = pieces per row / 2 <= 8; rows >= M are zeros.
struct RowRegs {
  uint4 v[8];
};

__device__ __forceinline__ void fetch_rows(RowRegs& g, const void* src, long long ld, long long r0,
                                           long long M, int cols, int pieces, uint32_t magic,
                                           int vec, int tid) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (2 * k >= pieces) break;
    const int q = tid + k * kGroupThreads;
    const int r = (int)__umulhi((uint32_t)q, magic), c = q - r * pieces;
    g.v[k] = make_uint4(0u, 0u, 0u, 0u);
    if (r0 + r < M) g.v[k] = fetch8((const uint16_t*)src + (r0 + r) * ld, c, cols, vec);
  }
}

__device__ __forceinline__ void store_rows(const RowRegs& g, uint8_t* dst, int pieces,
                                           uint32_t magic, int tid) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (2 * k >= pieces) break;
    const int q = tid + k * kGroupThreads;
    const int r = (int)__umulhi((uint32_t)q, magic), c = q - r * pieces;
    *reinterpret_cast<uint4*>(dst + (c >> 3) * 16384 + r * 128 + (((c & 7) ^ (r & 7)) << 4)) =
        g.v[k];
  }
}

// 8 values of a row from column e0, those before `cols`
__device__ __forceinline__ void put8(uint16_t* row, int e0, int cols, uint4 v, int vec) {
  if (e0 >= cols) return;
  if (vec == 16) {
    *reinterpret_cast<uint4*>(row + e0) = v;
  } else if (vec == 8) {
    *reinterpret_cast<uint2*>(row + e0) = make_uint2(v.x, v.y);
    if (e0 + 4 < cols) *reinterpret_cast<uint2*>(row + e0 + 4) = make_uint2(v.z, v.w);
  } else {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (vec == 4) {
        if (e0 + 2 * k < cols) *reinterpret_cast<uint32_t*>(row + e0 + 2 * k) = w[k];
      } else {
        if (e0 + 2 * k < cols) row[e0 + 2 * k] = (uint16_t)w[k];
        if (e0 + 2 * k + 1 < cols) row[e0 + 2 * k + 1] = (uint16_t)(w[k] >> 16);
      }
    }
  }
}

// ---------------------------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------------------------

// TMEM columns of one group: forward A|U 128, Y; dx A|U 128, dH 64, dX; weights A|U 128, dH 64
// (dW accumulators behind both groups').
__host__ __device__ constexpr int tmem_group(int mode, int dp, int op) {
  return mode == kFwd ? 128 + ((op + 31) & ~31)
                      : mode == kDx ? 192 + ((dp + 31) & ~31) : 192;
}

// shared memory of one group: its row tiles, and its hidden operand (h; da, du; da, du, h)
__host__ __device__ constexpr int smem_group(int mode, int dp, int op, bool gated) {
  return ((dp + 63) / 64 + (mode == kFwd ? 0 : (op + 63) / 64) +
          (mode == kFwd ? 1 : (gated ? 2 : 1) + (mode == kDw ? 1 : 0))) * 16384;
}

template <int MODE, typename T, int ACT, bool GATED>
__global__ void __launch_bounds__(kTcThreads, 1) k_ffn_tc(TcArgs p) {
  extern __shared__ uint8_t raw[];
  __shared__ __align__(8) uint64_t s_bar[2 * kMaxStages + 4 * kMaxGroups + 1];
  __shared__ uint32_t s_tmem;
  __shared__ int s_failed;
  constexpr int WR = GATED ? 128 : 64;
  constexpr bool BF = Two<T>::kBf16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint8_t* smem = raw + ((1024 - (smem_addr(raw) & 1023)) & 1023);
  const uint32_t sbase = smem_addr(smem);
  const int nbx = (p.dp + 63) >> 6, nby = (p.op + 63) >> 6;
  const uint32_t groups0 = p.nst * p.stage_bytes;
  const int gbytes = smem_group(MODE, p.dp, p.op, GATED);
  const uint32_t bars = smem_addr(s_bar);
  // weights of a stage: full, empty; per group: accumulators ready, hidden operand ready, second
  // product done, row tile ready (weights only)
  auto full = [&](int s) { return bars + 8 * s; };
  auto empty = [&](int s) { return bars + 8 * (kMaxStages + s); };
  auto gu_full = [&](int g) { return bars + 8 * (2 * kMaxStages + 4 * g); };
  auto h_ready = [&](int g) { return bars + 8 * (2 * kMaxStages + 4 * g + 1); };
  auto out_done = [&](int g) { return bars + 8 * (2 * kMaxStages + 4 * g + 2); };
  auto x_ready = [&](int g) { return bars + 8 * (2 * kMaxStages + 4 * g + 3); };
  const uint32_t all_done = bars + 8 * (2 * kMaxStages + 4 * kMaxGroups);
  volatile int* failed = &s_failed;
  unsigned int* status = &g_rows_status;

  if (threadIdx.x == 0) {
    s_failed = 0;
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), 1);
    }
    for (int g = 0; g < kMaxGroups; ++g) {
      mbar_init(gu_full(g), 1);
      mbar_init(h_ready(g), kGroupThreads / 32);
      mbar_init(out_done(g), 1);
      mbar_init(x_ready(g), kGroupThreads / 32);
    }
    mbar_init(all_done, 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    fence_async_shared();
  }
  constexpr uint32_t kCols = 512;
  if (warp == kMaxGroups * 8) tmem_alloc(smem_addr(&s_tmem), kCols);
  fence_before();
  __syncthreads();
  fence_after();
  const uint32_t tmem = s_tmem;

  const int chunk0 = MODE == kDw ? blockIdx.x % p.nch : 0;
  const int nch = MODE == kDw ? 1 : p.nch;
  const int ctas = MODE == kDw ? p.f.splits : gridDim.x;
  const int me = MODE == kDw ? blockIdx.x / p.nch : blockIdx.x;
  const long long step = (long long)ctas * p.ng;
  // steps of this CTA (both groups take the same number; a group without a tile has zero rows)
  const long long first = (long long)me * p.ng;
  const int nt = first < p.tiles ? (int)((p.tiles - first + step - 1) / step) : 0;
  const uint32_t tg = tmem_group(MODE, p.dp, p.op);
  const uint32_t acc_gu = tmem + p.ng * tg;  // weights: [da|du]^T X, then [du|h]^T dY
  const uint32_t acc_d = acc_gu + ((p.dp + 31) & ~31);

  if (warp == kMaxGroups * 8) {
    // ------------------------------------------------------------------------- MMA issue
    if (lane == 0 && nt > 0) {
      const int kx = p.dp >> 4, ko = p.op >> 4;
      const uint32_t id_gu = idesc(BF, WR, false, false), id_dh = idesc(BF, 64, false, true);
      const uint32_t id_y = idesc(BF, p.op, false, false), id_dx = idesc(BF, p.dp, false, true);
      const uint32_t id_wx = idesc(BF, p.dp, true, true), id_wy = idesc(BF, p.op, true, true);
      auto xs = [&](int g) { return sbase + groups0 + g * gbytes; };
      auto ys = [&](int g) { return xs(g) + nbx * 16384; };
      auto hs = [&](int g) { return xs(g) + (nbx + (MODE == kFwd ? 0 : nby)) * 16384; };
      auto ws = [&](int s) { return sbase + s * p.stage_bytes; };
      auto down = [&](int s) { return ws(s) + nbx * WR * 128; };
      // A|U (and dH) of group g from stage s
      auto first_product = [&](int g, int s) {
        const uint32_t d = tmem + g * tg;
        for (int k = 0; k < kx; ++k)
          mma(d, desc(xs(g) + (k >> 2) * 16384 + (k & 3) * 32, 16),
              desc(ws(s) + (k >> 2) * (WR * 128) + (k & 3) * 32, 16), id_gu, k > 0);
        if (MODE != kFwd)
          for (int k = 0; k < ko; ++k)
            mma(d + 128, desc(ys(g) + (k >> 2) * 16384 + (k & 3) * 32, 16),
                desc(down(s) + k * 2048, 16), id_dh, k > 0);
        commit(gu_full(g));
      };
      uint32_t ph_h[kMaxGroups] = {0, 0}, ph_x[kMaxGroups] = {0, 0};
      auto wait_h = [&](int g) {
        mbar_wait(h_ready(g), ph_h[g], failed, status);
        ph_h[g] ^= 1;
        fence_after();
      };
      auto wait_x = [&](int g) {
        mbar_wait(x_ready(g), ph_x[g], failed, status);
        ph_x[g] ^= 1;
        fence_after();
      };
      const bool ring = nch > p.nst;
      auto wait_full = [&](long long j) {  // j-th chunk use
        if (ring || j < nch)
          mbar_wait(full((int)(j % p.nst)), (uint32_t)((j / p.nst) & 1), failed, status);
      };
      const long long total = (long long)nt * nch;
      wait_full(0);
      for (int g = 0; g < p.ng; ++g) {
        wait_x(g);
        first_product(g, 0);
      }
      for (long long j = 0; j < total; ++j) {
        const int c = (int)(j % nch);
        const int s = ring ? (int)(j % p.nst) : c;
        const int sn = ring ? (int)((j + 1) % p.nst) : (c + 1) % nch;
        if (j + 1 < total) wait_full(j + 1);
        for (int g = 0; g < p.ng; ++g) {
          const uint32_t d = tmem + g * tg;
          wait_h(g);
          if (MODE == kFwd) {
            for (int k = 0; k < 4; ++k)
              mma(d + 128, desc(hs(g) + k * 32, 16), desc(down(s) + k * 32, 16), id_y,
                  c > 0 || k > 0);
          } else if (MODE == kDx) {
            for (int k = 0; k < WR / 16; ++k)
              mma(d + 192, desc(hs(g) + (k >> 2) * 16384 + (k & 3) * 32, 16),
                  desc(ws(s) + k * 2048, WR * 128), id_dx, c > 0 || k > 0);
          } else {
            for (int k = 0; k < 8; ++k)
              mma(acc_gu, desc(hs(g) + k * 2048, 16384), desc(xs(g) + k * 2048, 16384), id_wx,
                  j > 0 || g > 0 || k > 0);
            for (int k = 0; k < 8; ++k)
              mma(acc_d, desc(hs(g) + (GATED ? 16384 : 0) + k * 2048, 16384),
                  desc(ys(g) + k * 2048, 16384), id_wy, j > 0 || g > 0 || k > 0);
          }
          if (MODE == kDw || c == nch - 1) commit(out_done(g));
          if (ring && g == p.ng - 1) commit(empty(s));
          if (j + 1 < total) {
            if (MODE == kDw) wait_x(g);
            first_product(g, sn);
          }
        }
      }
      commit(all_done);
    }
  } else if (warp == kMaxGroups * 8 + 1) {
    // ------------------------------------------------------------------------- weight loads
    if (lane == 0 && nt > 0) {
      const bool ring = nch > p.nst;
      const long long total = ring ? (long long)nt * nch : nch;
      for (long long j = 0; j < total; ++j) {
        const int s = (int)(j % p.nst);
        if (j >= p.nst)
          mbar_wait(empty(s), (uint32_t)((j / p.nst - 1) & 1), failed, status);
        mbar_expect(full(s), p.stage_bytes);
        bulk_load(sbase + s * p.stage_bytes,
                  p.img + (size_t)(chunk0 + (int)(j % nch)) * p.stage_bytes, p.stage_bytes,
                  full(s));
      }
      // no copy may be in flight when the CTA ends, after a failed wait either
      for (long long j = total > p.nst ? total - p.nst : 0; j < total; ++j) {
        const long long t0 = clock64();
        while (!mbar_try(full((int)(j % p.nst)), (uint32_t)((j / p.nst) & 1)) &&
               clock64() - t0 < kWaitClocks) {
        }
      }
    }
  } else {
    // ------------------------------------------------------------------------- row groups
    const int g = warp >> 3, tid = threadIdx.x & (kGroupThreads - 1);
    if (g < p.ng && nt > 0) {
      uint8_t* Xs = smem + groups0 + (size_t)g * gbytes;
      uint8_t* Ys = Xs + nbx * 16384;
      uint8_t* Hs = Xs + (nbx + (MODE == kFwd ? 0 : nby)) * 16384;
      const uint32_t row_lanes = (uint32_t)(warp & 3) << 21;  // 32 * quadrant in the lane field
      const uint32_t d = tmem + g * tg + row_lanes;
      const int row = (warp & 3) * 32 + lane, half = (warp >> 2) & 1;
      const int xp = p.dp >> 3, yp = p.op >> 3;  // 16-byte pieces per row
      RowRegs xr, yr;
      auto fetch = [&](int n) {
        const long long r0 = (first + g + n * step) * kTile;
        fetch_rows(xr, p.f.x, p.f.ldx, r0, p.f.M, p.f.D, xp, p.x_magic, p.x_vec, tid);
        if (MODE != kFwd)
          fetch_rows(yr, p.f.dy, p.f.lddy, r0, p.f.M, p.f.O, yp, p.dy_magic, p.dy_vec, tid);
      };
      auto store = [&]() {
        store_rows(xr, Xs, xp, p.x_magic, tid);
        if (MODE != kFwd) store_rows(yr, Ys, yp, p.dy_magic, tid);
      };
      auto arrive = [&](uint32_t bar) {
        fence_async_shared();
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
      };
      fetch(0);
      store();
      arrive(x_ready(g));
      uint32_t ph_gu = 0, ph_out = 0;
      for (int n = 0; n < nt; ++n) {
        for (int c = 0; c < nch; ++c) {
          const bool more = c == nch - 1 && n + 1 < nt;
          if (more) fetch(n + 1);
          mbar_wait(gu_full(g), ph_gu, failed, status);
          ph_gu ^= 1;
          fence_after();
          // this thread: row `row`, units half * 32 .. + 32
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int u0 = half * 32 + q * 8;
            uint32_t ra[8], ru[8], rd[8];
            tmem_ld8(d + u0, ra);
            if (GATED) tmem_ld8(d + 64 + u0, ru);
            if (MODE != kFwd) tmem_ld8(d + 128 + u0, rd);
            tmem_wait(ra);
            if (GATED) tmem_wait(ru);
            if (MODE != kFwd) tmem_wait(rd);
            float h[8], da[8], du[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const float a = __uint_as_float(ra[e]);
              const float u = GATED ? __uint_as_float(ru[e]) : 1.0f;
              if (MODE == kFwd) {
                h[e] = act_fast<ACT>(a);
                if (GATED) h[e] *= u;
              } else {
                const float dh = __uint_as_float(rd[e]);
                float sl;
                const float f = act_slope_fast<ACT>(a, sl);
                h[e] = GATED ? f * u : f;
                da[e] = GATED ? dh * u * sl : dh * sl;
                du[e] = dh * f;
              }
            }
            const int at = row * 128 + (((u0 >> 3) ^ (row & 7)) << 4);
            auto put = [&](int block, const float* v) {
              *reinterpret_cast<uint4*>(Hs + block * 16384 + at) =
                  make_uint4(Two<T>::pack(v[0], v[1]), Two<T>::pack(v[2], v[3]),
                             Two<T>::pack(v[4], v[5]), Two<T>::pack(v[6], v[7]));
            };
            if (MODE == kFwd) {
              put(0, h);
            } else {
              put(0, da);
              if (GATED) put(1, du);
              if (MODE == kDw) put(GATED ? 2 : 1, h);
            }
          }
          // the tile's last first product is done: its rows may make room for the next tile's
          if (MODE != kDw && more) store();
          arrive(h_ready(g));
        }
        // the second product is done
        mbar_wait(out_done(g), ph_out, failed, status);
        ph_out ^= 1;
        fence_after();
        if (MODE == kDw) {
          if (n + 1 < nt) {
            store();
            arrive(x_ready(g));
          }
        } else {
          const long long r = (first + g + n * step) * kTile + row;
          const int cols = MODE == kFwd ? p.f.O : p.f.D;
          const long long ld = MODE == kFwd ? p.f.ldy : p.f.lddx;
          uint16_t* out = (uint16_t*)(MODE == kFwd ? p.f.y : p.f.dx) + r * ld;
          const uint32_t src = d + (MODE == kFwd ? 128 : 192);
          for (int e0 = half * 8; e0 < cols; e0 += 16) {
            uint32_t v[8];
            tmem_ld8(src + e0, v);
            tmem_wait(v);
            float o[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = __uint_as_float(v[e]);
            if (r < p.f.M)
              put8(out, e0, cols,
                   make_uint4(Two<T>::pack(o[0], o[1]), Two<T>::pack(o[2], o[3]),
                              Two<T>::pack(o[4], o[5]), Two<T>::pack(o[6], o[7])),
                   p.out_vec);
          }
        }
      }
    }
  }

  if (MODE == kDw && warp < 8) {
    // the CTA's sums: lanes are units (gate, up | up or gate, h), columns D or O
    const int row = (warp & 3) * 32 + lane, half = warp >> 2;
    const uint32_t row_lanes = (uint32_t)(warp & 3) << 21;
    const size_t FD = (size_t)p.f.F * p.f.D;
    float* part = p.f.part + (size_t)me * ((GATED ? 2 : 1) * FD + (size_t)p.f.F * p.f.O);
    const int f = chunk0 * kChunk + (row & 63);
    if (nt > 0) {
      mbar_wait(all_done, 0, failed, status);
      fence_after();
    }
    for (int which = 0; which < 2; ++which) {
      const int cols = which ? p.f.O : p.f.D;
      const bool mine = f < p.f.F && (which ? row >= 64 : GATED || row < 64);
      float* dst = part + (which ? (GATED ? 2 : 1) * FD + (size_t)f * p.f.O
                                 : (row >= 64 ? FD : 0) + (size_t)f * p.f.D);
      for (int e0 = half * 8; e0 < cols; e0 += 16) {
        uint32_t v[8];
        tmem_ld8((which ? acc_d : acc_gu) + row_lanes + e0, v);
        tmem_wait(v);
        if (mine)
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (e0 + e < cols) dst[e0 + e] = nt > 0 ? __uint_as_float(v[e]) : 0.0f;
      }
    }
  }
  fence_before();
  __syncthreads();
  if (warp == kMaxGroups * 8) {
    // every MMA is done before TMEM is given back
    if (nt > 0) mbar_wait(all_done, 0, failed, status);
    fence_after();
    __syncwarp();
    tmem_free(tmem, kCols);
  }
}

// ---------------------------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------------------------

int vec_of(const void* p, long long ld, int cols) {
  const uintptr_t all = (uintptr_t)p | (uintptr_t)(ld * 2) | (uintptr_t)(cols * 2);
  int v = 16;
  while (v > 2 && (all & (uintptr_t)(v - 1))) v >>= 1;
  return v;
}

uint32_t magic_of(int d) { return (uint32_t)(((1ULL << 32) + d - 1) / d); }

int pad16(int v) { return (v + 15) & ~15; }

int stage_bytes(int D, int O, bool gated) {
  return (D + 63) / 64 * (gated ? 128 : 64) * 128 + pad16(O) * 128;
}

template <int MODE, typename T, int ACT, bool GATED>
int launch(TcArgs p, cudaStream_t st) {
  p.x_vec = vec_of(p.f.x, p.f.M > 1 ? p.f.ldx : 0, p.f.D);
  if (MODE != kFwd) p.dy_vec = vec_of(p.f.dy, p.f.M > 1 ? p.f.lddy : 0, p.f.O);
  if (MODE == kFwd) p.out_vec = vec_of(p.f.y, p.f.M > 1 ? p.f.ldy : 0, p.f.O);
  if (MODE == kDx) p.out_vec = vec_of(p.f.dx, p.f.M > 1 ? p.f.lddx : 0, p.f.D);
  p.x_magic = magic_of(p.dp >> 3);
  p.dy_magic = magic_of(p.op >> 3);
  const int nch = MODE == kDw ? 1 : p.nch, gb = smem_group(MODE, p.dp, p.op, GATED);
  const int extra = MODE == kDw ? ((p.dp + 31) & ~31) + ((p.op + 31) & ~31) : 0;
  // two groups where tensor memory and shared memory hold them with two weight stages
  const int min_st = nch < 2 ? nch : 2;
  p.ng = 2 * tmem_group(MODE, p.dp, p.op) + extra <= 512 &&
                 2 * gb + min_st * p.stage_bytes <= kSmemLimit && p.tiles > 1
             ? 2
             : 1;
  int nst = (kSmemLimit - p.ng * gb) / p.stage_bytes;
  if (nst > kMaxStages) nst = kMaxStages;
  if (nst > nch) nst = nch;
  // (a ring needs two stages: the MMA thread asks for the next chunk before it frees this one)
  if (nst < min_st || p.ng * tmem_group(MODE, p.dp, p.op) + extra > 512) return SPLAT_ERR_CAPACITY;
  p.nst = nst;
  const int smem = p.nst * p.stage_bytes + p.ng * gb + 1024;
  long long grid = MODE == kDw ? (long long)p.nch * p.f.splits : (p.tiles + p.ng - 1) / p.ng;
  if (MODE != kDw && grid > 148) grid = 148;
  auto kernel = k_ffn_tc<MODE, T, ACT, GATED>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) !=
      cudaSuccess)
    return SPLAT_ERR_CUDA;
  kernel<<<(unsigned)grid, kTcThreads, smem, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? SPLAT_OK : SPLAT_ERR_CUDA;
}

template <typename T, int ACT, bool GATED>
int run(const FfnArgs& f, bool backward, uint8_t* img, cudaStream_t st) {
  TcArgs p = {};
  p.f = f;
  p.img = img;
  p.nch = (f.F + kChunk - 1) / kChunk;
  p.stage_bytes = stage_bytes(f.D, f.O, GATED);
  p.dp = pad16(f.D);
  p.op = pad16(f.O);
  p.tiles = ((long long)f.M + kTile - 1) / kTile;
  const int pieces = p.nch * (p.stage_bytes >> 4);
  k_pack<T, GATED><<<(pieces + 255) / 256, 256, 0, st>>>(p, img);
  int rc = SPLAT_OK;
  if (!backward) return launch<kFwd, T, ACT, GATED>(p, st);
  if (f.dx) rc = launch<kDx, T, ACT, GATED>(p, st);
  if (rc == SPLAT_OK && (f.dwg || f.dwu || f.dwd)) rc = launch<kDw, T, ACT, GATED>(p, st);
  return rc;
}

template <typename T>
int run_type(const FfnArgs& f, int act, bool backward, uint8_t* img, cudaStream_t st) {
  if (act == SPLAT_ACT_SILU)
    return f.wg ? run<T, SPLAT_ACT_SILU, true>(f, backward, img, st)
                : run<T, SPLAT_ACT_SILU, false>(f, backward, img, st);
  return f.wg ? run<T, SPLAT_ACT_GELU, true>(f, backward, img, st)
              : run<T, SPLAT_ACT_GELU, false>(f, backward, img, st);
}

}  // namespace

size_t ffn_tc_image_bytes(int D, int F, int O, bool gated) {
  return (size_t)((F + kChunk - 1) / kChunk) * stage_bytes(D, O, gated);
}

int ffn_tc_splits(long long M, int F) {
  const int chunks = (F + kChunk - 1) / kChunk;
  const long long tiles = (M + kTile - 1) / kTile, s = 148 / chunks;
  return (int)(s < tiles ? (s < 1 ? 1 : s) : tiles);
}

int ffn_tc_run(const FfnArgs& f, int dtype, int act, bool backward, void* img, cudaStream_t st) {
  return dtype == SPLAT_BF16 ? run_type<__nv_bfloat16>(f, act, backward, (uint8_t*)img, st)
                             : run_type<__half>(f, act, backward, (uint8_t*)img, st);
}

cudaError_t rows_status_take(unsigned int* out, cudaStream_t st) {
  const unsigned int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbolAsync(out, g_rows_status, sizeof *out, 0,
                                            cudaMemcpyDeviceToHost, st);
  if (e == cudaSuccess)
    e = cudaMemcpyToSymbolAsync(g_rows_status, &zero, sizeof zero, 0, cudaMemcpyHostToDevice, st);
  return e == cudaSuccess ? cudaStreamSynchronize(st) : e;
}

}  // namespace rows
}  // namespace splat
